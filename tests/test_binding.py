"""The binding's marshalling (no GPU: nothing is launched)."""
import ctypes

import pytest

from mixture_experts_layer_histogram_amd import moe

PTRS = [0x7F0000000000, 0x7F0000000100, 0x7F0000000200]


class Tensor:
    def __init__(self, ptr):
        self.ptr = ptr

    def data_ptr(self):
        return self.ptr


@pytest.mark.parametrize("make", [list, tuple, iter, lambda p: (q for q in p), lambda p: map(int, p), dict.fromkeys,
                                  lambda p: (ctypes.c_void_p * 3)(*p), lambda p: [Tensor(q) for q in p],
                                  lambda p: (Tensor(q) for q in p), lambda p: {q: Tensor(q) for q in p}.values()])
def test_rank_tables_of_any_iterable(make):
    assert list(moe._table(make(PTRS))) == PTRS


def test_rank_tables_with_no_pointer():
    assert moe._table(None) is None
    assert list(moe._table([PTRS[0], None])) == [PTRS[0], None]
    assert len(moe._table([])) == 0 and len(moe._table(iter([]))) == 0


def test_a_generator_of_ranks_reaches_the_library():
    """The second rank's rows are misaligned: the table arrived whole."""
    s, p = moe.Shape(2, 64, 1024, 16, 4, 512, moe.MOE_BF16), moe.Placement(PTRS[0], 8)
    call = lambda y: moe.moe_combine_merge(s, p, PTRS[0], PTRS[0], PTRS[0], y, stream=0, check=False)  # noqa: E731
    assert call(q for q in (PTRS[1], PTRS[1] + 8)) == -2
    assert call(q for q in (PTRS[1], None)) == -1
