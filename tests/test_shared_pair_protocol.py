"""The meetings of a pair of softmax warps in the tensor-core kernel over a
shared prefix (kvarn_shared_tc.cu, meet and leave), as a model that is
searched exhaustively: the pair's named barrier has no time limit, so no order
of the two warps' steps, of their own time-outs and of another role's raising
of the abort flag may leave one of them waiting for a partner that is gone."""
import pytest

STAGES = 4


def stuck(leaves_when_told):
    """A state in which a warp waits and nobody can move, or None. A warp is
    (stage, step): "wait" (its bounded waits: they succeed, or run out at any
    time), "meet" (arrives and waits), "held" (at the barrier), "look" (reads
    the flag behind it), "gone"."""
    first = ((0, "wait"), (0, "wait"), False, 0)  # two warps, abort flag, arrivals at the barrier
    seen, todo = {first}, [first]
    while todo:
        state = todo.pop()
        a, b, flag, count = state
        nexts = [] if flag else [(a, b, True, count)]  # another role gives up

        def arrive(warps, i, becomes):
            """Warp i arrives and goes to `becomes`; the second arrival lets the barrier's waiters go."""
            warps = list(warps)
            warps[i] = becomes
            if count + 1 < 2:
                return warps, count + 1
            return [(w[0], "look") if w[1] == "held" else w for w in warps], 0

        for i, (stage, step) in enumerate((a, b)):
            if step == "wait":
                warps = [a, b]
                warps[i] = (stage, "meet")
                nexts.append((*warps, flag, count))
                warps, n = arrive((a, b), i, (stage, "gone"))  # ran out: sets the flag, then leaves
                nexts.append((*warps, True, n))
            elif step == "meet":
                warps, n = arrive((a, b), i, (stage, "held"))
                nexts.append((*warps, flag, n))
            elif step == "look":
                if not flag:
                    warps, n = [a, b], count
                    warps[i] = (stage + 1, "wait") if stage + 1 < STAGES else (stage, "gone")
                elif leaves_when_told:
                    warps, n = arrive((a, b), i, (stage, "gone"))
                else:
                    warps, n = [a, b], count
                    warps[i] = (stage, "gone")
                nexts.append((*warps, flag, n))
        moves = [n for n in nexts if n[:2] != (a, b)]
        if not moves and "held" in (a[1], b[1]):
            return state
        for n in nexts:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return None


def test_no_order_of_events_leaves_a_warp_waiting():
    assert stuck(leaves_when_told=True) is None


def test_the_model_finds_the_warp_that_goes_without_its_arrival():
    state = stuck(leaves_when_told=False)
    assert state is not None and {w[1] for w in state[:2]} == {"held", "gone"} and state[2]


@pytest.mark.parametrize("call", ["if (!meet(s, mine, other))", "if (s >= 2 && !wait(B_OF", "if (!wait(B_SF", "if (!wait(B_OF"])
def test_the_kernel_leaves_wherever_the_model_does(call):
    """Each early exit of the kernel's stage loop arrives at the barrier first."""
    from quantized_kv_cache_kvarn_gb300 import build
    with open(f"{build.CSRC}/kvarn_shared_tc.cu") as f:
        text = f.read()
    at = text.index(call)
    assert text.find(call, at + 1) < 0
    block = text[at:text.index("break;", at)]
    assert "ok = false;" in block and "leave();" in block
