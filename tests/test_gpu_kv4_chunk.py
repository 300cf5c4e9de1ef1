"""Attention of chunks of new tokens over the 4-bit cache and themselves, on the
GPU, against the definition in 64 bits.

Tolerance of an output (a_old, a_new = sum p |v| over the cached and the new
tokens a row sees, s = max sum |q k| scale): p is rounded to fp16 for cached
tokens (half a step, 2^-11) and to q's type for new ones (2^-11 or 2^-8); its
exponent is an fp32 sum of D products (2^-24 each against s) times a factor,
less a reference (4 more), and an exponential good to 2^-22; sums over tokens
add 2^-24 an add; p below fp16's normal range is off by 2^-25 where the largest
is at least 2^8. The result is rounded to its type once (half a step)."""

import math

import numpy as np
import pytest
import torch

import oracle.kv4 as ok
from gpu_helpers import DEV, say
from quantized_weight_skinny_amd import QpnError
from quantized_weight_skinny_amd import decode_api as qd
from quantized_weight_skinny_amd import prompt_api as qp

pytestmark = pytest.mark.gpu
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
K_SCALE, V_SCALE = 0.01, 0.02


def _values(pool, page, kv_heads, dim, slots, of_v):
    """float64 [tokens, kv_heads, dim] of what slots stand for, by the oracle's places."""
    places = [ok.kv4_places(dim, page, off, of_v) for off in range(page)]
    byte, shift, scale = (torch.from_numpy(np.stack([p[j] for p in places])).to(DEV) for j in range(3))
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    seg = pool.view(pool.shape[0], kv_heads, -1)[slots // page]
    off = slots % page
    pick = lambda at: seg.gather(2, at[off][:, None].expand(-1, kv_heads, -1))  # noqa: E731
    code = (pick(byte).long() >> shift[off][:, None]) & 15
    v = e2m1[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    return v * pick(scale).view(torch.float8_e4m3fn).double() * (V_SCALE if of_v else K_SCALE)


class Case:
    def __init__(self, seed, kv, rows, heads, kv_heads, dim, page, dtype, q_scale=1.0, spare=2, layers=1, layer=0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.kv, self.rows, self.heads, self.kv_heads, self.dim, self.page = kv, rows, heads, kv_heads, dim, page
        held = [-(-n // page) for n in kv]
        pages = sum(held) + spare
        seg = ok.kv4_segment_bytes(dim, page)
        pool = rng.integers(0, 256, (layers, pages, kv_heads, seg), dtype=np.uint8)
        pool[..., page * dim:] = rng.integers(0x28, 0x58, pool[..., page * dim:].shape, dtype=np.uint8)
        self.pool = torch.from_numpy(pool.reshape(layers, pages, -1)).to(DEV)
        order = rng.permutation(pages).astype(np.int32)
        table = np.full((len(kv), max(held)), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).to(DEV)
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device=DEV)
        self.start = [0] + np.cumsum(rows).tolist()
        self.q_start = torch.tensor(self.start, dtype=torch.int32, device=DEV)
        total = self.start[-1]
        qkv = torch.randn((total, (heads + 2 * kv_heads) * dim), device=DEV, generator=gen)
        qkv[:, :heads * dim] *= q_scale
        qkv = qkv.to(TYPES[dtype])
        self.q = qkv[:, :heads * dim].view(total, heads, dim)
        self.k = qkv[:, heads * dim:(heads + kv_heads) * dim].view(total, kv_heads, dim)
        self.v = qkv[:, (heads + kv_heads) * dim:].view(total, kv_heads, dim)
        self.layer = layer
        self.cache = qd.KV4Cache.wrap(self.pool, page, kv_heads, dim, K_SCALE, V_SCALE)

    def run(self, window=0, **kw):
        say("kv4_chunk_attention", self.kv, self.rows, self.heads, self.kv_heads, self.dim, self.page, self.q.dtype, window)
        kw = {"q_start": self.q_start, "max_q_len": max(self.rows), "max_kv_len": max(self.kv), **kw}
        return qp.kv4_chunk_attention(self.q, self.k, self.v, self.cache, self.table, self.kv_len, window=window,
                                      layer=self.layer, **kw)

    def check(self, out, lse, window=0, cut=None, only=None):
        """Compares sequences' rows (only: a slice of each's) with the definition."""
        group, dim = self.heads // self.kv_heads, self.dim
        for b, (old, n) in enumerate(zip(self.kv, self.rows)):
            if n == 0:
                continue
            old = old if cut is None else min(old, cut)
            t = torch.arange(old, device=DEV)
            page = self.table[b].long()[t // self.page] if old else t
            here = (page >= 0) & (page < self.pool.shape[1])
            slots = torch.where(here, page, 0) * self.page + t % self.page
            mine = slice(self.start[b], self.start[b + 1])
            pick = torch.arange(n, device=DEV)[only or slice(None)]
            pos = old + pick[:, None]
            place = torch.arange(old + n, device=DEV)[None]
            seen = place <= pos
            if window:
                seen &= place > pos - window
            seen[:, :old] &= here
            ck, cv = (_values(self.pool[self.layer], self.page, self.kv_heads, dim, slots, x) for x in (False, True))
            for h in range(self.kv_heads):
                k = torch.cat((ck[:, h], self.k[mine, h].double()))
                v = torch.cat((cv[:, h], self.v[mine, h].double()))
                for g in range(h * group, (h + 1) * group):
                    q = self.q[mine, g][pick].double()
                    x = torch.where(seen, q @ k.T * dim ** -0.5, -math.inf)
                    size = torch.where(seen, q.abs() @ k.abs().T * dim ** -0.5, 0.0).amax(1)
                    z = torch.logsumexp(x, 1)
                    p = torch.exp(x - z[:, None])
                    ref = p @ v
                    a_old, a_new = p[:, :old] @ v[:old].abs(), p[:, old:] @ v[old:].abs()
                    a = a_old + a_new
                    half = torch.finfo(self.q.dtype).eps / 2
                    common = (dim + 4) * 2.0 ** -24 * size[:, None] + 2.0 ** -22 + (old + n + 64) * 2.0 ** -24
                    tol = a_old * 2.0 ** -11 + a_new * half + a * common
                    tol = tol + (old + n) * v.abs().max() * 2.0 ** -33 + half * (ref.abs() + tol) + 2.0 ** -25
                    off = (out[mine, g][pick].double() - ref).abs()
                    assert (off <= tol).all(), (b, g, float((off / tol).max()))
                    ltol = (dim + 4) * 2.0 ** -24 * size + (old + n + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + z.abs())
                    loff = (lse[mine, g][pick].double() - z).abs()
                    assert (loff <= ltol).all(), (b, g, float((loff / ltol).max()))


CASES = [
    # kv, rows, heads, kv_heads, dim, page, window
    ([0], [1], 1, 1, 64, 16, 0),
    ([1], [1], 2, 1, 128, 16, 0),
    ([0], [200], 4, 2, 128, 64, 0),
    ([300], [5], 40, 8, 128, 64, 0),
    ([63, 64, 65], [63, 64, 65], 5, 1, 128, 32, 0),
    ([0, 17, 1000], [130, 1, 0], 6, 3, 64, 16, 0),
    ([129, 5], [33, 300], 8, 1, 256, 128, 0),
    ([700], [257], 3, 3, 256, 256, 0),
    ([100, 0, 40], [70, 140, 1], 8, 2, 128, 16, 1),
    ([100, 300, 40], [70, 140, 1], 8, 2, 64, 32, 7),
    ([190, 64], [70, 140], 10, 2, 128, 64, 64),
    ([500, 64], [70, 340], 4, 1, 256, 64, 100),
    ([90, 64], [70, 40], 4, 1, 128, 64, 2 ** 31 - 1),
    ([5000], [9], 10, 2, 128, 16, 0),        # few rows, many splits
    ([9000, 20], [40, 3], 5, 1, 64, 64, 0),
    ([4000], [20], 8, 1, 256, 32, 3000),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv,rows,heads,kv_heads,dim,page,window", CASES)
def test_against_the_definition(kv, rows, heads, kv_heads, dim, page, window, dtype):
    c = Case(len(kv) + heads, kv, rows, heads, kv_heads, dim, page, dtype)
    c.check(*c.run(window), window)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_more_than_64_sequences(dtype):
    rng = np.random.default_rng(7)
    kv = rng.integers(0, 200, 150).tolist()
    rows = rng.integers(0, 70, 150).tolist()
    c = Case(3, kv, rows, 4, 2, 64, 16, dtype)
    c.check(*c.run(), only=slice(None, None, 9))


def test_long_chunk_and_prefix():
    c = Case(5, [20000], [1500], 10, 2, 128, 64, "fp16")
    c.check(*c.run(), only=slice(None, None, 97))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_strong_scores(dtype):
    """Scores of tens to hundreds: nearly one-hot rows, references that move."""
    c = Case(11, [300, 10], [100, 90], 4, 2, 128, 64, dtype, q_scale=30.0)
    c.check(*c.run())


def test_equal_lengths_without_starts_and_defaults():
    c = Case(12, [64, 100, 30], [40, 40, 40], 4, 2, 64, 16, "bf16")
    out, lse = qp.kv4_chunk_attention(c.q, c.k, c.v, c.cache, c.table, c.kv_len)
    c.check(out, lse)
    full, full_lse = c.run()
    assert torch.equal(out, full) and torch.equal(lse, full_lse)


def test_no_cache_at_all():
    """Prompts from their beginning: a table of no columns, a pool of no pages."""
    c = Case(13, [0, 0], [100, 30], 4, 2, 128, 16, "fp16")
    c.table = torch.zeros((2, 0), dtype=torch.int32, device=DEV)
    c.check(*c.run(max_kv_len=0))
    empty = qd.KV4Cache(0, 16, 2, 128)
    out, lse = qp.kv4_chunk_attention(c.q, c.k, c.v, empty, torch.zeros((2, 3), dtype=torch.int32, device=DEV),
                                      torch.tensor([9, 40], dtype=torch.int32, device=DEV), q_start=c.q_start,
                                      max_q_len=100)
    c.check(out, lse)


def test_lengths_beyond_the_bound_are_cut():
    c = Case(14, [200, 90], [30, 20], 2, 1, 64, 16, "fp16")
    c.check(*c.run(max_kv_len=100), cut=100)
    c.kv_len[1] = -5
    c.kv[1] = 0
    c.check(*c.run(max_kv_len=100), cut=100)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 90])
def test_absent_pages_and_foreign_bytes(dim, window):
    """Pages outside the pool are not seen; bytes of tokens past the end, NaN scales among them, change nothing."""
    c = Case(15, [150, 70], [40, 130], 4, 2, dim, 16, "bf16")
    c.table[0, 3], c.table[0, 7], c.table[1, 0] = -1, c.pool.shape[1], 2 ** 31 - 1
    out, lse = c.run(window)
    c.check(out, lse, window)
    seg = c.pool[0].view(c.pool.shape[1], 2, -1)
    used = torch.zeros((c.pool.shape[1] * 16,), dtype=torch.bool, device=DEV)
    for b, n in enumerate(c.kv):
        t = torch.arange(n, device=DEV)
        p = c.table[b].long()[t // 16]
        ok_ = (p >= 0) & (p < c.pool.shape[1])
        used[(p * 16 + t % 16)[ok_]] = True
    for off in range(16):
        for of_v in (False, True):
            byte, _, scale = ok.kv4_places(dim, 16, off, of_v)
            free = ~used.view(-1, 16)[:, off]
            for at in (byte, scale):
                at = torch.from_numpy(at).to(DEV)
                seg[:, :, at] = torch.where(free[:, None, None], torch.full_like(seg[:, :, at], 0x7F), seg[:, :, at])
    again, lse2 = c.run(window)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_odd_values_reach_only_the_rows_that_see_them(dim, dtype):
    """inf and NaN in the values and keys of a token: rows before it, and rows whose window has left it, are as without."""
    for window in (0, 50):
        c = Case(16, [70, 10], [200, 90], 4, 2, dim, 16, dtype)
        clean, clean_lse = c.run(window)
        bad = {30: float("inf"), 64: float("nan"), 130: float("-inf")}
        for t, x in bad.items():
            c.v[t, 1, 5 + t % 7] = x
        out, lse = c.run(window)
        assert torch.equal(lse, clean_lse)
        for row in range(200):
            for d in range(dim):
                hit = [x for t, x in bad.items() if d == 5 + t % 7 and t <= row and (window == 0 or t > row - window)]
                if hit:
                    break
        seen = torch.zeros_like(out, dtype=torch.bool)
        for t in bad:
            last = 200 if window == 0 else min(200, t + window)
            seen[t:last, 2:4, 5 + t % 7] = True
        assert torch.equal(out[~seen], clean[~seen])
        assert not out[seen].isfinite().any()
        for t, x in bad.items():
            col = out[t:200 if window == 0 else min(200, t + window), 2:4, 5 + t % 7]
            others = [y for u, y in bad.items() if u != t and 5 + u % 7 == 5 + t % 7]
            if not others:
                assert torch.isnan(col).all() if math.isnan(x) else (col == x).all()
        # a NaN key: its own row and those after it; the other head and sequence nothing
        c.v[:] = torch.where(c.v.isfinite(), c.v, torch.zeros_like(c.v))
        base, _ = c.run(window)
        c.k[77, 0, 3] = float("nan")
        out, lse = c.run(window)
        last = 200 if window == 0 else 127
        assert torch.isnan(out[77:last, 0:2]).all()
        keep = torch.ones_like(out, dtype=torch.bool)
        keep[77:last, 0:2] = False
        assert torch.equal(out[keep], base[keep])


def test_rows_of_no_sequence_are_left_and_their_contents_do_not_matter():
    c = Case(17, [30, 40], [50, 60], 4, 2, 128, 16, "bf16")
    full, full_lse = c.run()
    start = torch.tensor([0, 50, 80], dtype=torch.int32, device=DEV)
    c.q[80:], c.k[80:], c.v[80:] = float("nan"), float("nan"), float("inf")
    out, lse = torch.full_like(full, 7.0), torch.full_like(full_lse, 7.0)
    c.run(q_start=start, out=out, lse=lse)
    assert torch.equal(out[:80], full[:80]) and torch.equal(lse[:80], full_lse[:80])
    assert (out[80:] == 7).all() and (lse[80:] == 7).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_strides_and_alignment(dim):
    c = Case(18, [100, 20], [70, 33], 4, 2, dim, 16, "fp16")
    full, full_lse = c.run()
    def apart(x):
        wide = torch.full((x.shape[0], 3, x.shape[1], dim + 3), float("nan"), dtype=x.dtype, device=DEV)
        wide[:, 1, :, 1:1 + dim] = x
        return wide[:, 1, :, 1:1 + dim]
    c.q, c.k, c.v = apart(c.q), apart(c.k), apart(c.v)
    out, lse = c.run()
    assert torch.equal(out, full) and torch.equal(lse, full_lse)
    # heads before tokens, a table whose rows lie apart
    swap = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    c.q, c.k, c.v = swap(c.q), swap(c.k), swap(c.v)
    wide = torch.full((2, c.table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    out, lse = c.run()
    assert torch.equal(out, full) and torch.equal(lse, full_lse)


def test_one_chunk_or_several_with_appends_between():
    """A prompt in chunks: later chunks see the earlier ones' tokens as the cache holds them."""
    heads, kvh, dim, page = 4, 2, 128, 16
    gen = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn((150, n, dim), device=DEV, generator=gen).half() for n in (heads, kvh, kvh))
    cache = qd.KV4Cache(12, page, kvh, dim)
    table = torch.arange(11, -1, -1, dtype=torch.int32, device=DEV)[None]
    slots = table[0].long()[torch.arange(150, device=DEV) // page] * page + torch.arange(150, device=DEV) % page
    outs = []
    for at, n in ((0, 60), (60, 50), (110, 40)):
        part = slice(at, at + n)
        out, _ = qp.kv4_chunk_attention(q[part], k[part], v[part], cache, table,
                                        torch.tensor([at], dtype=torch.int32, device=DEV))
        outs.append(out)
        qd.kv4_append(cache, k[part], v[part], slots[part])
    rk, rv = qd.kv4_read(cache, slots, dtype=torch.float32)
    for at, n, out in ((0, 60, outs[0]), (60, 50, outs[1]), (110, 40, outs[2])):
        kk = torch.cat((rk[:at].double(), k[at:at + n].double()))
        vv = torch.cat((rv[:at].double(), v[at:at + n].double()))
        for h in range(heads):
            s = q[at:at + n, h].double() @ kk[:, h // 2].T * dim ** -0.5
            s = s.masked_fill(torch.arange(at + n, device=DEV)[None] > at + torch.arange(n, device=DEV)[:, None], -math.inf)
            ref = torch.softmax(s, 1) @ vv[:, h // 2]
            assert (out[:, h].double() - ref).abs().max() <= 2.0 ** -10 * vv.abs().max()


def test_captured_call_follows_lengths_and_tables():
    c = Case(19, [400, 90], [60, 20], 8, 2, 128, 16, "fp16", spare=8)
    ws = qp.kv4_chunk_workspace(c.cache, 80, 8, 2, 80, 432)
    out, lse = torch.empty((80, 8, 128), dtype=torch.float16, device=DEV), torch.empty((80, 8), device=DEV)
    wide = torch.full((2, 27), -1, dtype=torch.int32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    kw = dict(max_q_len=80, max_kv_len=432, out=out, lse=lse, workspace=ws)
    c.run(**kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(**kw)
    for kv, rows in (([400, 90], [60, 20]), ([0, 33], [1, 79]), ([399, 0], [80, 0]), ([17, 90], [0, 80])):
        c.kv, c.rows, c.start = kv, rows, [0, rows[0], 80]
        c.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        c.q_start.copy_(torch.tensor(c.start, dtype=torch.int32))
        c.q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_streams_layers_and_repeats():
    c = Case(20, [3000], [30], 8, 2, 64, 16, "bf16", layers=3, layer=2)
    out, lse = c.run()
    c.check(out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, other_lse = c.run()
    again, again_lse = c.run()
    torch.cuda.synchronize()
    assert torch.equal(out, other) and torch.equal(out, again)
    assert torch.equal(lse, other_lse) and torch.equal(lse, again_lse)


def test_offsets_beyond_32_bits():
    """A pool of 5 GB whose last pages are read, and strides that take rows beyond 2^32 bytes."""
    page, kvh, dim = 256, 1, 256
    nbytes = 256 * 256 * 9 // 8
    pages = 5 * 2 ** 30 // nbytes
    c = Case(21, [500], [40], 1, 1, dim, page, "fp16")
    big = torch.zeros((1, pages, nbytes), dtype=torch.uint8, device=DEV)
    big[0, -c.pool.shape[1]:] = c.pool[0]
    full, full_lse = c.run()
    c.cache = qd.KV4Cache.wrap(big, page, kvh, dim, K_SCALE, V_SCALE)
    c.table = torch.where(c.table >= 0, c.table + pages - c.pool.shape[1], c.table).to(torch.int32)
    step = 60_000_000
    room = torch.empty((40 * step + 1024,), dtype=torch.float16, device=DEV)
    def far(x, at):
        y = room[at:].as_strided((40, 1, dim), (step, dim, 1))
        y.copy_(x)
        return y
    c.q, c.k, c.v = far(c.q, 0), far(c.k, 256), far(c.v, 512)
    out, lse = c.run()
    assert torch.equal(out, full) and torch.equal(lse, full_lse)


def test_refusals():
    c = Case(22, [40], [8], 4, 2, 64, 16, "fp16")
    with pytest.raises(ValueError, match="k must"):
        qp.kv4_chunk_attention(c.q, c.k[:4], c.v, c.cache, c.table, c.kv_len)
    with pytest.raises(ValueError, match="v must"):
        qp.kv4_chunk_attention(c.q, c.k, c.v.bfloat16(), c.cache, c.table, c.kv_len)
    with pytest.raises(ValueError, match="q must"):
        qp.kv4_chunk_attention(c.q.float(), c.k, c.v, c.cache, c.table, c.kv_len)
    with pytest.raises(ValueError, match="multiple"):
        qp.kv4_chunk_attention(c.q[:, :3], c.k, c.v, c.cache, c.table, c.kv_len)
    with pytest.raises(ValueError, match="table"):
        qp.kv4_chunk_attention(c.q, c.k, c.v, c.cache, c.table.long(), c.kv_len)
    with pytest.raises(ValueError, match="max_kv_len"):
        qp.kv4_chunk_attention(c.q, c.k, c.v, c.cache, c.table, c.kv_len, max_kv_len=1000)
    with pytest.raises(ValueError, match="max_q_len"):
        qp.kv4_chunk_attention(c.q, c.k, c.v, c.cache, c.table, c.kv_len, q_start=c.q_start)
    with pytest.raises(ValueError, match="contiguous"):
        t = torch.empty((8, 64, 4), dtype=torch.float16, device=DEV).transpose(1, 2)
        qp.kv4_chunk_attention(t, c.k, c.v, c.cache, c.table, c.kv_len)
    with pytest.raises(QpnError):
        qp.kv4_chunk_attention(c.q, c.k, c.v, c.cache, c.table, c.kv_len, scale=float("nan"))
    with pytest.raises(ValueError, match="layer"):
        qp.kv4_chunk_attention(c.q, c.k, c.v, c.cache, c.table, c.kv_len, layer=1)
