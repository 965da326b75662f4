"""The integer entry points refuse sizes that one launch does not hold (fewer than 2^32
threads), and take the largest that it does."""
import pytest

from test_int8_cpu import SHAPE, quant



@pytest.mark.parametrize("rows", [1, 512, 513])
def test_columns_of_one_launch(rows):
    """A workgroup of 1024 threads for each 64 columns: 2^22 - 1 of them."""
    most = (1 << 28) - 64
    for cols in (most + 8, most + 56, 1 << 28):
        assert quant(axis=1, rows=rows, cols=cols, ld=cols, ldq=528) == SHAPE
    # the bound itself passes the size check and meets the next one: a missing tensor
    assert quant(axis=1, rows=rows, cols=most, ld=most, ldq=528, x=None) == 1
