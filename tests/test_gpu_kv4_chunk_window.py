"""Chunk attention with a window, on the GPU: what cached tokens in front of a
row's window hold, NaN scales of their values and keys among it, has no effect on the row.

No tolerance: a value's scale enters neither scores nor references, so the rows that
do not see it keep their bits, and those that do are NaN in that block of 16 elements alone."""

import pytest
import torch

import oracle.kv4 as ok
from gpu_helpers import DEV
from test_gpu_kv4_chunk import Case

pytestmark = pytest.mark.gpu

RUNS = [
    # kv, rows, heads, kv_heads, page, window
    ([300, 90], [70, 140], 4, 2, 16, 100),     # short runs, a workgroup each
    ([3000], [90], 4, 2, 16, 2000),            # long ones, shared by many
    ([700, 64], [33, 5], 3, 1, 64, 64),
    ([5000, 10, 2100], [200, 20, 1], 8, 2, 128, 1500),
]


def _scale(c, b, t, head, block, of_v, byte):
    """The scale byte of 16 elements of token t of sequence b."""
    at = ok.kv4_places(c.dim, c.page, t % c.page, of_v)[2][16 * block]
    c.pool[c.layer].view(c.pool.shape[1], c.kv_heads, -1)[int(c.table[b, t // c.page]), head, at] = byte


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,rows,heads,kv_heads,page,window", RUNS)
def test_nan_scales_of_values_reach_only_the_rows_that_see_them(kv, rows, heads, kv_heads, page, window, dim, dtype):
    c = Case(31, kv, rows, heads, kv_heads, dim, page, dtype)
    clean, clean_lse = c.run(window)
    c.check(clean, clean_lse, window, only=slice(None, None, 7))
    group, head, blocks = heads // kv_heads, kv_heads - 1, dim // 16
    bad = torch.zeros_like(clean, dtype=torch.bool)
    for b, (old, n) in enumerate(zip(kv, rows)):
        first, last = old - window + 1, old + n - window   # what the first and the last row see first
        # in front of all rows; seen by the first rows only; by all
        for j, t in enumerate((first - 1, first - 2, first // 64 * 64, first, first + 1, first + 10, first + 33, last - 1,
                               last, last + 3)):
            if not 0 <= t < old:
                continue
            block = j % blocks
            _scale(c, b, t, head, block, True, 0xFF if j % 2 else 0x7F)
            for i in range(n):
                if t > old + i - window:
                    bad[c.start[b] + i, head * group:(head + 1) * group, 16 * block:16 * block + 16] = True
    out, lse = c.run(window)
    assert torch.equal(lse, clean_lse)
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,rows,heads,kv_heads,page,window", RUNS)
def test_tokens_in_front_of_every_window_may_hold_anything(kv, rows, heads, kv_heads, page, window, dim):
    c = Case(32, kv, rows, heads, kv_heads, dim, page, "bf16")
    clean, clean_lse = c.run(window)
    seg = c.pool[c.layer].view(c.pool.shape[1], kv_heads, -1)
    for b, old in enumerate(kv):
        for t in range(max(0, old - window - 140), max(0, old - window + 1)):   # (two steps of 64 and more)
            for of_v in (False, True):
                byte, _, scale = ok.kv4_places(dim, page, t % page, of_v)
                for at in (byte, scale):
                    seg[int(c.table[b, t // page]), :, torch.from_numpy(at).to(DEV)] = 0x7F
    out, lse = c.run(window)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
