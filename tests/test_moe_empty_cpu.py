"""Empty operands of the routed-experts C ABI, without a GPU: an empty tensor
has no address, so that a NULL for it is not a missing operand."""
import pytest

from activation_epilogue_amd import moe

OK, INVALID, BF16 = 0, 1, 2
P = [0x100000000 * (i + 1) for i in range(8)]


@pytest.mark.parametrize("T,k,S", [(0, 2, 0), (0, 0, 0), (5, 0, 0), (0, 2, 7)])
def test_gradients_of_a_combination_without_slots(T, k, S):
    lib = moe._lib()
    assert lib.fl_moe_combine_bwd(P[0] if T else None, P[1] if S else None, None, None, P[2] if S else None, None, T, k,
                                  S, 32, BF16, None) == OK


def test_gradients_of_a_combination_of_rows_without_columns():
    """(its dweights are zeros, which a launch writes: none is asked for here)"""
    lib = moe._lib()
    assert lib.fl_moe_combine_bwd(None, None, P[0], None, None, None, 4, 2, 8, 0, BF16, None) == OK
    assert lib.fl_moe_combine_bwd(P[0], P[1], P[2], None, None, None, 4, 2, 8, 16, BF16, None) == INVALID
    assert "both NULL" in lib.fl_moe_last_error().decode()
