"""The meetings of a pair of softmax warps in the tensor-core kernel over a
shared prefix (kvarn_shared_tc.cu, meet and leave), as a model that is
searched exhaustively: the pair's named barrier has no time limit, so no order
of the two warps' steps, of their own time-outs and of another role's raising
of the abort flag may leave one of them waiting for a partner that is gone,
nor an arrival at the barrier that nobody meets."""
import pytest

STAGES = 4


def search(one_view):
    """(a state in which a warp waits and nobody can move, a final state with
    an arrival left over), None where there is none. A warp is (stage, step):
    "wait" (its bounded waits: they succeed, or run out at any time), "write"
    (its view of the flag, where the warps exchange it), "meet" (arrives and
    waits), "held" (at the barrier), "look" (decides behind it), "gone".
    one_view: the decision is on the two views exchanged before the barrier,
    else on the flag itself, read behind it."""
    # two warps, abort flag, arrivals at the barrier, views [stage parity][warp]
    first = ((0, "wait"), (0, "wait"), False, 0, ((0, 0), (0, 0)))
    seen, todo, bad, left = {first}, [first], None, None
    while todo:
        state = todo.pop()
        a, b, flag, count, views = state
        moved = []

        def put(i, warp, warps=None, n=count, f=flag, v=views):
            warps = list(warps or (a, b))
            warps[i] = warp
            moved.append((*warps, f, n, v))

        def view(stage, i, value):
            rows = [list(r) for r in views]
            rows[stage & 1][i] = value
            return tuple(tuple(r) for r in rows)

        def arrive(i, becomes, f=flag, v=views):
            """Warp i arrives and goes to `becomes`; the second arrival lets the barrier's waiters go."""
            warps = [a, b]
            warps[i] = becomes
            if count + 1 < 2:
                moved.append((*warps, f, count + 1, v))
            else:
                moved.append((*[(w[0], "look") if w[1] == "held" else w for w in warps], f, 0, v))

        for i, (stage, step) in enumerate((a, b)):
            if step == "wait":
                put(i, (stage, "write"))
                arrive(i, (stage, "gone"), f=True, v=view(stage, i, 1))  # ran out: sets the flag, says so, leaves
            elif step == "write":
                put(i, (stage, "meet"), v=view(stage, i, int(flag)))
            elif step == "meet":
                arrive(i, (stage, "held"))
            elif step == "look":
                go = any(views[stage & 1]) if one_view else flag
                put(i, (stage, "gone") if go or stage + 1 == STAGES else (stage + 1, "wait"))
        if not moved:
            if "held" in (a[1], b[1]):
                bad = state
            elif count:
                left = state
        if not flag:
            moved.append((a, b, True, count, views))  # another role gives up
        for n in moved:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return bad, left


def test_no_order_of_events_leaves_a_warp_waiting():
    assert search(one_view=True) == (None, None)


def test_the_model_finds_the_warp_that_waits_for_one_that_is_gone():
    state, _ = search(one_view=False)
    assert state is not None and {w[1] for w in state[:2]} == {"held", "gone"} and state[2]


@pytest.fixture(scope="module")
def text():
    from quantized_kv_cache_kvarn_gb300 import build
    with open(f"{build.CSRC}/kvarn_shared_tc.cu") as f:
        return f.read()


def test_the_kernel_meets_as_the_model_does(text):
    body = text[text.index("auto meet = "):text.index("auto leave = ")]
    at = [body.index(s) for s in ("half) * kM + r] = gone ? kGone", "bar.sync", "!gone && word != kGone")]
    assert at == sorted(at) and "abort_flag" not in body  # the flag is read by the caller, before
    body = text[text.index("auto leave = "):text.index("const float kq")]
    at = [body.index(s) for s in ("half) * kM + r] = kGone;", "__syncwarp();", "bar.arrive")]
    assert at == sorted(at)


@pytest.mark.parametrize("wait,stage", [("if (s >= 2 && !wait(B_OF", "s"), ("if (!wait(B_SF", "s"), ("if (!wait(B_OF", "s + 1")])
def test_the_kernel_leaves_wherever_the_model_does(text, wait, stage):
    """A wait that runs out arrives at the pair's next meeting."""
    at = text.index(wait)
    assert text.find(wait, at + 1) < 0
    block = text[at:text.index("break;", at)]
    assert "ok = false;" in block and f"leave({stage});" in block
