"""kvarn_fork_sequences over counts that do not agree with the tables' rows: the list of freed pages is that of the
counts before and after, whatever the order in which rows give their references back."""
import pytest
import torch

import quantized_kv_cache_kvarn_gb300 as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_kvarn_gb300 import build
    build.build()
    kv.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("start", [-1, 0, 1, 2])
def test_a_count_that_passes_through_zero(start, in_place):
    """Page 0 is held by a row that goes on twice and by one that ends, page 1 by the same in the other order, page 2 by
    two that end: the counts of pages 0 and 1 end where they began."""
    lay = kv.q8_layout(128, 1, 3)
    for _ in range(10):
        refs = i32([start, start, 2])
        refs_out, out, table = refs if in_place else i32([9, 9, 9]), i32([0] * 4), i32([[7]] * 4)
        gone, count, err = i32([5] * 3), i32([5]), kv.new_error_word()
        kv.fork_sequences(i32([0, 0, 3, 3]), i32([16] * 6), i32([[0], [0], [1], [1], [2], [2]]), refs, lay, 16, out, table, refs_out, gone,
                          count, err)
        assert refs_out.tolist() == [start, start, 0] and table.flatten().tolist() == [0, 0, 1, 1]
        assert int(count) == 1 and gone.tolist() == [2, -1, -1]
        assert kv.read_error_flags(err) == 0


def test_counts_that_fall_below_zero_or_rise_from_it():
    """A count that falls from above 0 past it is listed; one that was not above 0 is not, wherever it ends."""
    lay = kv.q8_layout(128, 1, 4)
    refs, out, table = i32([1, 0, 1, -3]), i32([0] * 3), i32([[7]] * 3)
    gone, count, err = i32([5] * 4), i32([5]), kv.new_error_word()
    # page 0: two rows end; page 1: one ends; page 2: one goes on three times; page 3: one ends
    kv.fork_sequences(i32([3, 3, 3]), i32([16] * 5), i32([[0], [0], [1], [2], [3]]), refs, lay, 16, out, table, refs, gone, count, err)
    assert refs.tolist() == [-1, -1, 3, -4] and int(count) == 1 and gone.tolist() == [0, -1, -1, -1]
