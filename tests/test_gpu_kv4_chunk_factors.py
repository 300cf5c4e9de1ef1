"""Chunk attention where the factor of its scores leaves fp32's normal range, on
the GPU: queries of zeros (padding) and scales at the ends of what is taken.
Every score is 0, so each row is the mean of the values it sees; tolerances as
in test_gpu_kv4_chunk."""

import pytest
import torch

from quantized_weight_skinny_amd import decode_api as qd
from test_gpu_kv4_chunk import V_SCALE, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("k_scale,scale", [
    (1e-9, None),          # a cache of small keys; bf16 takes 2^-126 out of a row of zeros
    (1e-20, 1e-30),        # their product is below fp32's range
    (1e-45, 1e-45),
    (3e38, 3e38),          # above it
    (1e-45, 3e38),
])
def test_zero_queries_give_the_mean(k_scale, scale, dtype):
    c = Case(33, [100, 37, 0], [5, 70, 130], 4, 2, 128, 16, dtype)
    c.q.zero_()
    c.cache = qd.KV4Cache.wrap(c.pool, c.page, c.kv_heads, c.dim, k_scale, V_SCALE)
    c.table[0, 2] = -1
    out, lse = c.run(scale=scale)
    assert not torch.isnan(out).any()
    c.check(out, lse)
    out, lse = c.run(window=30, scale=scale)
    c.check(out, lse, 30)
