"""4-bit cache rows: strides whose rows would lie beyond any memory are refused (no kernel runs)."""
import pytest

from sparse_compressed_attention_gb300 import _lib as L
from tests.test_cache_host import append, lib, read, refused           # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows,stride", [(1 << 24, 1 << 40), (1 << 20, 1 << 40), (1 << 24, 1 << 26)])
def test_rows_beyond_any_memory(lib, rows, stride, dtype):                # noqa: F811
    refused(lib, append(lib, rows=rows, xr=stride, dtype=dtype), L.V4_ERR_INVALID_ARG, "10^15")
    refused(lib, read(lib, rows=rows, yr=stride, dtype=dtype), L.V4_ERR_INVALID_ARG, "10^15")
