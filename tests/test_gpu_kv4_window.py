"""Attention over the 4-bit cache with a window, on the GPU: what cached tokens in
front of the windows of all rows hold, NaN scales among it, has no effect. No tolerance:
nothing of such tokens enters the rows, so they keep their bits."""

import pytest
import torch

import oracle.kv4 as ok
from gpu_helpers import DEV
from quantized_weight_skinny_amd import decode_api as qd
from test_gpu_kv4_chunk import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,rows,page,window", [
    ([300, 90], [1, 1], 16, 37),
    ([3000], [1], 64, 2000),        # shared by many
    ([300, 700, 40], [5, 16, 3], 32, 100),
    ([5000, 64], [16, 16], 128, 1),
])
def test_tokens_in_front_of_every_window_may_hold_anything(kv, rows, page, window, dim, dtype):
    c = Case(36, kv, rows, 4, 2, dim, page, dtype)
    call = lambda: qd.kv4_attention(c.q, c.cache, c.table, c.kv_len, q_start=c.q_start, max_q_len=max(rows),  # noqa: E731
                                    max_kv_len=max(kv), window=window)
    clean, clean_lse = call()
    assert clean.isfinite().all() and clean_lse.isfinite().all()
    seg = c.pool[0].view(c.pool.shape[1], c.kv_heads, -1)
    for b, (n, r) in enumerate(zip(kv, rows)):
        first = n - r + 1 - window   # what the first row sees first
        for t in range(max(0, first - 80), max(0, first)):
            for of_v in (False, True):
                byte, _, scale = ok.kv4_places(dim, page, t % page, of_v)
                for at in (byte, scale):
                    seg[int(c.table[b, t // page]), :, torch.from_numpy(at).to(DEV)] = 0x7F
    out, lse = call()
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
