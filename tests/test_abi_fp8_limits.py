"""The largest sizes that the FP8 quantisers name: a size is refused as such, not left to fail at the launch.

16 rows make a workgroup of 256 threads and a launch holds fewer than 2^32 threads along x, so
2^28 - 16 rows are the most.  No pointer is dereferenced (a null one is refused after the sizes)."""
import pytest

OK, ERR_NULL, ERR_SHAPE = range(3)
MOST = (1 << 28) - 16


@pytest.mark.parametrize("rows", [MOST + 1, (1 << 28) - 1, 1 << 28, 1 << 40])
def test_too_many_rows(lib, rows):
    assert lib.fp8_quantize_rows(None, 0, rows, 256, None, 0, None, None, None) == ERR_SHAPE
    assert lib.fp8_swiglu_quantize(None, 0, rows, 256, None, 4, None, None, None, None, None, None) == ERR_SHAPE


def test_the_most_rows(lib):
    assert -(-MOST // 16) * 256 < 1 << 32 <= -(-(MOST + 1) // 16) * 256
    assert lib.fp8_quantize_rows(None, 0, MOST, 256, None, 0, None, None, None) == ERR_NULL
    assert lib.fp8_swiglu_quantize(None, 0, MOST, 256, None, 4, None, None, None, None, None, None) == ERR_NULL
