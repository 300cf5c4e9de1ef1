"""Attention over the 4-bit cache where the factor of its scores leaves fp32's
normal range, on the GPU: queries of zeros (padding) and scales at the ends of what is
taken. Every score is 0, so each row is the mean of the n values it sees: sums of n
equal weights and exact values in fp32 (2^-24 of the magnitudes an add), rounded once."""

import math

import pytest
import torch

from gpu_helpers import DEV
from quantized_weight_skinny_amd import decode_api as qd
from test_gpu_kv4_chunk import V_SCALE, Case, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("k_scale,scale", [
    (1e-9, None),          # a cache of small keys; bf16 takes 2^-126 out of a row of zeros
    (1e-20, 1e-30),        # their product is below fp32's range
    (3e38, 3e38),          # above it
])
def test_zero_queries_give_the_mean(k_scale, scale, dim, dtype):
    c = Case(34, [100, 37, 700], [5, 3, 16], 4, 2, dim, 16, dtype)
    c.q.zero_()
    cache = qd.KV4Cache.wrap(c.pool, c.page, c.kv_heads, dim, k_scale, V_SCALE)
    out, lse = qd.kv4_attention(c.q, cache, c.table, c.kv_len, q_start=c.q_start, max_q_len=16, scale=scale)
    for b, (n, rows) in enumerate(zip(c.kv, c.rows)):
        t = torch.arange(n, device=DEV)
        v = _values(c.pool[0], c.page, c.kv_heads, dim, c.table[b].long()[t // c.page] * c.page + t % c.page, True)
        for i in range(rows):
            seen = n - rows + i + 1
            for h in range(c.heads):
                ref, size = v[:seen, h // 2].mean(0), v[:seen, h // 2].abs().mean(0)
                tol = (seen + 8) * 2.0 ** -24 * size
                tol = tol + torch.finfo(c.q.dtype).eps / 2 * (ref.abs() + tol) + 2.0 ** -25
                row = c.start[b] + i
                assert ((out[row, h].double() - ref).abs() <= tol).all(), (b, i, h)
                # log2 of the weights' sum, n 2^8 in [2^8, 2^18), is good to a step of fp32 at 16: 2^-19; less 8, times ln 2
                assert abs(float(lse[row, h]) - math.log(seen)) <= 2.0 ** -19
