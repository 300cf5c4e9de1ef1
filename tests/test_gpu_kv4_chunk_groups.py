"""Chunk attention where one kv head serves many query heads, so that a token's
heads fill a tile of 128 rows or more, on the GPU; tolerances as in test_gpu_kv4_chunk."""

import pytest

from test_gpu_kv4_chunk import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv,rows,heads,kv_heads,dim,page,window", [
    ([100, 5], [3, 70], 48, 1, 64, 16, 0),      # tokens end inside a tile
    ([300], [5], 130, 1, 128, 32, 0),           # and tiles inside a token
    ([900, 64], [2, 9], 260, 2, 64, 16, 0),     # a token is a tile and some rows; shared runs
    ([200, 0], [70, 40], 128, 1, 64, 64, 50),
    ([150], [1], 400, 1, 256, 16, 100),
])
def test_against_the_definition(kv, rows, heads, kv_heads, dim, page, window, dtype):
    c = Case(35, kv, rows, heads, kv_heads, dim, page, dtype)
    c.check(*c.run(window), window)
