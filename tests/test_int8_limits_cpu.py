"""The integer entry points refuse sizes that one launch does not hold (fewer than 2^32
threads), and take the largest that it does."""
import pytest

from test_int8_cpu import NULL, SHAPE, grouped, quant



@pytest.mark.parametrize("rows", [1, 512, 513])
def test_columns_of_one_launch(rows):
    """A workgroup of 1024 threads for each 64 columns: 2^22 - 1 of them."""
    most = (1 << 28) - 64
    for cols in (most + 8, most + 56, 1 << 28):
        assert quant(axis=1, rows=rows, cols=cols, ld=cols, ldq=528) == SHAPE
    # the bound itself passes the size check and meets the next one: a missing tensor
    assert quant(axis=1, rows=rows, cols=most, ld=most, ldq=528, x=None) == NULL


@pytest.mark.parametrize("rows_per_group,tile_m,tile_n", [(5, 64, 128), (32, 64, 128), (33, 128, 128), (127, 128, 128),
                                                          (128, 256, 256)])
def test_tiles_of_one_launch(rows_per_group, tile_m, tile_n):
    """Fewer than 2^24 workgroups of 256 threads: a tile per started tile_m rows of each
    group at most, for each tile_n columns."""
    G = 65535
    rows = G * rows_per_group
    per_column = rows // tile_m + G
    most = ((1 << 24) - 8) // per_column                    # column tiles
    size = lambda N, **o: grouped(M=rows, N=N, K=16, G=G, lda=16, ldb=16, bsg=0, ssg=0, ldc=N, **o)
    assert size((most + 1) * tile_n) == SHAPE and size(most * tile_n + 8) == SHAPE
    assert size(most * tile_n, a=None) == NULL              # past the size check: a missing tensor
