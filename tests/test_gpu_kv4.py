"""GPU parity of the 4-bit paged cache and the attention over it against the
float64 oracle: bytes exactly, attention within its roundings.

Tolerance of an attention output (derived, in the oracle's units a = sum p |v|
and s = max sum |q k| scale): p is rounded to fp16 (half a step, 2^-11), its
exponent is an fp32 sum of D products (relative 2^-24 each against s) times a
factor, less a reference (2 more), and an exponential good to 2^-22; sums of
tokens add 2^-24 for each add of a lane; p below fp16's normal range is off by
2^-25 where the largest is at least 2^8. The result is rounded to its type once
(half a step of it)."""

import math

import numpy as np
import pytest
import torch

import oracle.kv4 as ok
from gpu_helpers import DEV, say, to_host
from quantized_weight_skinny_amd import decode_api as qd

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def attention_tolerance(out, a, s, tokens, vmax, dim, dtype):
    rel = 2.0 ** -11 + (dim + 4) * 2.0 ** -24 * s[:, None] + 2.0 ** -22 + (tokens + 64) * 2.0 ** -24
    return a * rel + tokens * vmax * 2.0 ** -33 + torch.finfo(dtype).eps / 2 * (np.abs(out) + a * rel) + 2.0 ** -25


def lse_tolerance(lse, s, tokens, dim):
    return (dim + 4) * 2.0 ** -24 * s + (tokens + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(lse))


def random_pool(rng, layers, pages, page, kv_heads, dim):
    """Random codes and block scales between 2^-2 and 30 (any code, NaN scales left out)."""
    seg = ok.kv4_segment_bytes(dim, page)
    pool = rng.integers(0, 256, (layers, pages, kv_heads, seg), dtype=np.uint8)
    pool[..., page * dim:] = rng.integers(0x28, 0x60, pool[..., page * dim:].shape, dtype=np.uint8)
    return pool.reshape(layers, pages, kv_heads * seg)


class Case:
    """A pool with sequences of the given tokens and rows, on the device and for the oracle."""

    def __init__(self, seed, kv, rows, heads, kv_heads, dim, page, dtype, layers=1, layer=0, q_scale=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.kv, self.rows, self.heads, self.kv_heads, self.dim, self.page = kv, rows, heads, kv_heads, dim, page
        self.layer, self.dtype = layer, dtype
        held = [-(-n // page) for n in kv]
        self.pages = sum(held) + spare
        self.pool = random_pool(rng, layers, self.pages, page, kv_heads, dim)
        order = rng.permutation(self.pages).astype(np.int32)
        width = max(held) if held else 0
        self.table = np.full((len(kv), max(width, 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        q = rng.standard_normal((int(self.start[-1]), heads, dim)).astype(np.float32) * q_scale
        self.q = torch.from_numpy(q).to(TYPES[dtype])
        self.k_scale, self.v_scale = 0.01, 0.02
        self.scale = dim ** -0.5

    def device(self):
        data = torch.from_numpy(self.pool.copy()).to(DEV)
        cache = qd.KV4Cache.wrap(data, self.page, self.kv_heads, self.dim, self.k_scale, self.v_scale)
        return cache, torch.from_numpy(self.table).to(DEV), torch.tensor(self.kv, dtype=torch.int32, device=DEV), \
            torch.from_numpy(self.start).to(DEV)

    def run(self, window=0, **kw):
        cache, table, kv_len, start = self.device()
        say("kv4_attention", self.kv, self.rows, self.heads, self.kv_heads, self.dim, self.page, self.dtype, window, kw)
        return qd.kv4_attention(self.q.to(DEV), cache, table, kv_len, q_start=start, max_q_len=max(self.rows),
                                layer=self.layer, window=window, scale=self.scale, **kw)

    def expected(self, window=0, absent=()):
        """Per sequence and kv head: (rows slice, heads slice, out, lse, tolerances)."""
        group = self.heads // self.kv_heads
        for b, n in enumerate(self.kv):
            r = self.rows[b]
            if r == 0:
                continue
            seen = ok.visible(r, n, window)
            k, v = np.zeros((n, self.kv_heads, self.dim)), np.zeros((n, self.kv_heads, self.dim))
            for t in range(n):
                p = self.table[b, t // self.page]
                if p < 0 or p >= self.pages:
                    seen[:, t] = False
                    continue
                (kc, ks), (vc, vs) = ok.kv4_load(self.pool[self.layer], self.page, self.kv_heads, self.dim,
                                                 int(p) * self.page + t % self.page)
                k[t], v[t] = ok.kv4_values(kc, ks, self.k_scale), ok.kv4_values(vc, vs, self.v_scale)
            rows = slice(int(self.start[b]), int(self.start[b + 1]))
            for h in range(self.kv_heads):
                heads = slice(h * group, (h + 1) * group)
                q = self.q[rows, heads].double().numpy().reshape(r * group, self.dim)
                o, lse, a, s = ok.attention(q, k[:, h], v[:, h], np.repeat(seen, group, axis=0), self.scale)
                vmax = np.abs(v[:, h]).max() if n else 0.0
                ot = attention_tolerance(o, a, s, n, vmax, self.dim, TYPES[self.dtype])
                lt = lse_tolerance(np.where(np.isfinite(lse), lse, 0.0), s, n, self.dim)
                shape = (r, group, self.dim)
                yield rows, heads, o.reshape(shape), lse.reshape(r, group), ot.reshape(shape), lt.reshape(r, group)

    def check(self, got, window=0):
        out, lse = to_host(got[0].double()), to_host(got[1].double())
        for rows, heads, o, l, ot, lt in self.expected(window):
            assert np.all(np.abs(out[rows, heads] - o) <= ot), (rows, heads, np.max(np.abs(out[rows, heads] - o) / ot))
            none = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[rows, heads]), none)
            assert np.all(np.abs(lse[rows, heads][~none] - l[~none]) <= lt[~none]), (
                rows, heads, np.max(np.abs(lse[rows, heads][~none] - l[~none]) / lt[~none]))
            assert np.all(out[rows, heads][none] == 0)


# ---------------------------------------------------------------- append, read, copy

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_writes_the_oracles_bytes(dim, page, dtype):
    say("append", dim, page, dtype)
    rng = np.random.default_rng(dim * page)
    kvh, pages, tokens = 3, 4, 37
    pool = random_pool(rng, 2, pages, page, kvh, dim)
    cache = qd.KV4Cache.wrap(torch.from_numpy(pool.copy()).to(DEV), page, kvh, dim, [0.5, 0.01], [0.25, 0.003])
    # a fused projection's output: k and v are strided views; odd-sized magnitudes, zeros and extremes among them
    x = rng.standard_normal((tokens, 2 * kvh + 1, dim)).astype(np.float32)
    x *= np.exp(rng.uniform(-12, 6, (tokens, 2 * kvh + 1, 1))).astype(np.float32)
    x[3] = 0
    x[4, :, 5], x[5, :, 7], x[6, :, 9] = np.inf, -np.inf, np.nan
    x[7, :, :16] = -0.0
    x[8] = 60000.0
    xd = torch.from_numpy(x).to(TYPES[dtype])
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[10], slots[11], slots[12] = -1, pages * page, 1 << 40
    dev = xd.to(DEV)
    qd.kv4_append(cache, dev[:, 1:1 + kvh], dev[:, 1 + kvh:], torch.from_numpy(slots).to(DEV), layer=1)
    f = xd.float().numpy()
    ref = pool.copy()
    for t in range(tokens):
        ok.kv4_store(ref[1], page, kvh, dim, int(slots[t]), ok.kv4_quantize(f[t, 1:1 + kvh], 0.01),
                     ok.kv4_quantize(f[t, 1 + kvh:], 0.003))
    assert np.array_equal(to_host(cache.data), ref)
    # and back, in each type
    for kind, t in (("fp16", torch.float16), ("bf16", torch.bfloat16), ("fp32", torch.float32)):
        k, v = qd.kv4_read(cache, torch.from_numpy(slots).to(DEV), layer=1, dtype=t)
        want = np.zeros((2, tokens, kvh, dim))
        for i, slot in enumerate(slots):
            if 0 <= slot < pages * page:
                (kc, ks), (vc, vs) = ok.kv4_load(ref[1], page, kvh, dim, int(slot))
                want[0, i], want[1, i] = ok.kv4_values(kc, ks, 0.01), ok.kv4_values(vc, vs, 0.003)
        for got, w in ((k, want[0]), (v, want[1])):
            # one fp32 product, one rounding to the type (and fp16's smallest step)
            tol = np.abs(w) * (2.0 ** -24 + torch.finfo(t).eps / 2 * (1 + 2.0 ** -24)) + (2.0 ** -25 if kind == "fp16" else 0)
            assert np.all(np.abs(to_host(got.double()) - w) <= tol), kind


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_append_rounds_division_like_ieee(dim):
    """Many random blocks: every quotient lands on the code that IEEE division
    and the nearest-even rule give, ties and near ties among them."""
    say("append division", dim)
    rng = np.random.default_rng(7)
    tokens, page, kvh = 4096, 64, 2
    cache = qd.KV4Cache(tokens // page, page, kvh, dim, k_scale=1 / 600, v_scale=1.0)
    x = rng.standard_normal((tokens, 2 * kvh, dim)).astype(np.float32)
    x[:, kvh:] = rng.integers(-24, 25, (tokens, kvh, dim)) / 4  # on and between the grid's midpoints
    xd = torch.from_numpy(x).to(torch.float16)
    slots = torch.arange(tokens, dtype=torch.int64, device=DEV)
    qd.kv4_append(cache, xd[:, :kvh].to(DEV), xd[:, kvh:].to(DEV), slots)
    k, v = qd.kv4_read(cache, slots, dtype=torch.float32)
    f = xd.float().numpy()
    for got, src, s in ((k, f[:, :kvh], 1 / 600), (v, f[:, kvh:], 1.0)):
        codes, sc = ok.kv4_quantize(src, s)
        want = ok.kv4_values(codes, sc, s)
        assert np.all(np.abs(to_host(got.double()) - want) <= np.abs(want) * 2.0 ** -23)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scales", [(0.001, 2.0 ** -50), (2.0 ** -70, 2.0 ** 70), (2.0 ** 59, 1.0)])
def test_append_values_at_the_end_of_bf16(dim, scales):
    """Magnitudes up to 2^127 and down to bf16's smallest, beside each other:
    quotients that leave fp32 count as infinite, those that vanish as zeros."""
    say("append extremes", dim, scales)
    rng = np.random.default_rng(dim)
    tokens, page, kvh = 48, 16, 2
    x = rng.standard_normal((tokens, 2 * kvh, dim)) * 2.0 ** rng.uniform(-133, 126, (tokens, 2 * kvh, dim))
    x[0::3] = rng.standard_normal((tokens // 3, 2 * kvh, dim)) * 2.0 ** 125
    x[1::3] = rng.standard_normal((tokens // 3, 2 * kvh, dim)) * 2.0 ** rng.uniform(-130, 120, (tokens // 3, 2 * kvh, 1))
    xd = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    cache = qd.KV4Cache(tokens // page, page, kvh, dim, k_scale=scales[0], v_scale=scales[1])
    ref = to_host(cache.data).copy()
    qd.kv4_append(cache, xd[:, :kvh].to(DEV), xd[:, kvh:].to(DEV), torch.arange(tokens, dtype=torch.int64, device=DEV))
    f = xd.float().numpy()
    with np.errstate(all="ignore"):
        for t in range(tokens):
            ok.kv4_store(ref[0], page, kvh, dim, t, ok.kv4_quantize(f[t, :kvh], scales[0]),
                         ok.kv4_quantize(f[t, kvh:], scales[1]))
    assert np.array_equal(to_host(cache.data), ref)


def test_append_unaligned_rows():
    say("append unaligned")
    rng = np.random.default_rng(3)
    kvh, dim, page, tokens = 2, 128, 16, 9
    x = torch.from_numpy(rng.standard_normal((tokens * 3 * kvh * (dim + 3) + 8)).astype(np.float32)).half()
    slots = torch.arange(tokens, dtype=torch.int64, device=DEV)
    dev = x.to(DEV)
    def views(t):
        a = t[1:1 + tokens * kvh * (dim + 3)].view(tokens, kvh, dim + 3)[..., :dim]
        b = t[4:4 + tokens * kvh * (dim + 3)].view(tokens, kvh, dim + 3)[..., 3:]
        return a, b
    one, two = (qd.KV4Cache(1, page, kvh, dim) for _ in range(2))
    qd.kv4_append(one, *views(dev), slots)
    qd.kv4_append(two, *(v.contiguous() for v in views(dev)), slots)
    assert torch.equal(one.data, two.data)


@pytest.mark.parametrize("page,kvh,dim,layers,count", [(16, 1, 64, 1, 1), (64, 8, 128, 5, 33), (256, 3, 256, 2, 7)])
def test_copy_pages(page, kvh, dim, layers, count):
    say("copy", page, kvh, dim, layers, count)
    rng = np.random.default_rng(count)
    pages = 2 * count + 3
    data = torch.from_numpy(random_pool(rng, layers, pages, page, kvh, dim)).to(DEV)
    before = data.clone()
    cache = qd.KV4Cache.wrap(data, page, kvh, dim)
    order = torch.from_numpy(rng.permutation(pages).astype(np.int32)).to(DEV)
    src, dst = order[:count].clone(), order[count:2 * count].clone()
    if count > 4:
        src[1], dst[2], dst[3] = -1, pages, 1 << 30   # skipped
    qd.kv4_copy_pages(cache, src, dst)
    want = before.clone()
    for s, d in zip(src.tolist(), dst.tolist()):
        if 0 <= s < pages and 0 <= d < pages:
            want[:, d] = before[:, s]
    assert torch.equal(cache.data, want)


def test_empty_calls():
    say("empty calls")
    cache = qd.KV4Cache(0, 16, 2, 64)
    none = torch.zeros((0, 2, 64), dtype=torch.float16, device=DEV)
    slots = torch.zeros(0, dtype=torch.int64, device=DEV)
    qd.kv4_append(cache, none, none, slots)
    k, v = qd.kv4_read(cache, slots)
    assert k.shape == (0, 2, 64)
    some = torch.ones((3, 2, 64), dtype=torch.float16, device=DEV)
    three = torch.arange(3, dtype=torch.int64, device=DEV)
    qd.kv4_append(cache, some, some, three)          # no slot exists
    k, v = qd.kv4_read(cache, three)
    assert not to_host(k).any() and not to_host(v).any()
    ints = torch.zeros(0, dtype=torch.int32, device=DEV)
    qd.kv4_copy_pages(cache, ints, ints)
    # sequences without tokens in a pool without pages
    out, lse = qd.kv4_attention(some, cache, torch.full((3, 2), -1, dtype=torch.int32, device=DEV),
                                torch.tensor([0, 5, 32], dtype=torch.int32, device=DEV))
    assert not to_host(out).any() and np.isneginf(to_host(lse)).all()
    out, lse = qd.kv4_attention(none, cache, torch.zeros((0, 2), dtype=torch.int32, device=DEV), ints)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("group", [1, 3, 5, 8])
def test_attention_head_layouts(dim, dtype, group):
    # rows x group from a third of a tile to several row tiles
    for rows in ([1, 1, 1], [7, 2, 16], [16, 16, 3]):
        c = Case(dim + group, [1, 77, 300], rows, 2 * group, 2, dim, 32, dtype)
        c.check(c.run())


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kv", [[1], [15, 16, 17], [31, 32, 33], [63, 64, 65, 127, 128, 129], [511, 513, 1000]])
def test_attention_lengths_and_pages(page, kv):
    c = Case(page, kv, [1] * len(kv), 10, 2, 128, page, "fp16")
    c.check(c.run())
    c = Case(page + 1, kv, [8] * len(kv), 10, 2, 128, page, "bf16")
    c.check(c.run())


@pytest.mark.parametrize("window", [1, 2, 31, 33, 200, 5000])
def test_attention_window(window):
    c = Case(window, [3, 40, 700, 1501], [1, 9, 5, 16], 8, 2, 128, 16, "fp16")
    c.check(c.run(window=window), window)


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1])
def test_attention_window_as_wide_as_its_type_hides_nothing(window):
    """Also where rows lie before the sequence's start, so that a position less the window is lowest."""
    c = Case(21, [4, 0, 40, 600], [16, 5, 9, 16], 6, 2, 64, 16, "fp16")
    got, want = c.run(window=window), c.run(window=0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(got)


def test_attention_refuses_numbers_beyond_32_bits():
    c = Case(22, [40], [2], 2, 1, 64, 16, "fp16")
    for kw in (dict(window=(1 << 32) + 7), dict(window=-1), dict(max_kv_len=(1 << 32) + 40), dict(max_kv_len=-1)):
        with pytest.raises(ValueError, match="must be 0"):
            c.run(**kw)


def test_attention_empty_rows():
    """Lengths of zero, blocks longer than their sequence (rows before its
    start) and sequences without rows."""
    c = Case(5, [0, 3, 0, 40, 1], [4, 7, 0, 0, 2], 6, 2, 64, 16, "fp16")
    got = c.run()
    c.check(got)
    assert np.isneginf(to_host(got[1])[:4]).all()      # no tokens
    assert np.isneginf(to_host(got[1])[4:8]).all()     # positions below 0


def test_attention_long_splits_and_joins():
    """One sequence spread over all compute units, and very uneven lengths."""
    c = Case(9, [9000], [8], 5, 1, 128, 64, "fp16")
    c.check(c.run())
    c = Case(10, [6000, 1, 33, 2500, 0, 700], [2, 1, 16, 4, 3, 1], 4, 2, 64, 16, "bf16")
    c.check(c.run())


def test_attention_many_sequences():
    """More sequences than a wavefront has lanes."""
    rng = np.random.default_rng(1)
    kv = [int(x) for x in rng.integers(0, 60, 150)]
    rows = [int(x) for x in rng.integers(0, 4, 150)]
    c = Case(11, kv, rows, 2, 1, 64, 16, "fp16")
    c.check(c.run())


def test_attention_many_sequences_cut_into_shares():
    """The same where the tiles are laid end to end: more sequences than lanes,
    some empty, some without rows, one much longer than the others."""
    rng = np.random.default_rng(2)
    kv = [int(x) for x in rng.integers(0, 90, 140)]
    rows = [int(x) for x in rng.integers(0, 4, 140)]
    kv[77], rows[77], kv[139], rows[139] = 5000, 3, 2300, 2
    c = Case(24, kv, rows, 3, 1, 64, 32, "bf16")
    c.check(c.run())


def test_attention_long_block():
    """A block of many rows: several row tiles a sequence, causal across tiles."""
    c = Case(12, [150, 70], [130, 70], 3, 1, 128, 32, "fp16")
    c.check(c.run())


def test_attention_peaked_rows():
    """Scores hundreds apart, rising along the sequence: the running reference
    moves many times, and all but a few probabilities vanish."""
    c = Case(13, [900, 400], [3, 8], 4, 2, 128, 64, "fp16", q_scale=60.0)
    c.check(c.run())
    c = Case(14, [900], [5], 4, 2, 256, 64, "bf16", q_scale=60.0)
    c.check(c.run())


def test_attention_absent_and_bad_pages():
    """Page indices outside the pool hold no tokens."""
    c = Case(15, [200, 130], [4, 2], 4, 2, 128, 32, "fp16")
    c.table[0, 1], c.table[0, 6], c.table[1, 0] = -1, c.pages, np.iinfo(np.int32).max
    c.check(c.run())
    c.table[1, :] = np.iinfo(np.int32).min
    c.check(c.run())


def test_attention_garbage_outside_the_sequences():
    """NaN scales in every byte that belongs to no seen token change nothing."""
    for page in (16, 64):
        c = Case(16, [37, 100, 5], [2, 1, 7], 4, 2, 128, page, "fp16")
        clean = c.run()
        keep = np.zeros((c.pages * page,), bool)
        for b, n in enumerate(c.kv):
            for t in range(n):
                keep[c.table[b, t // page] * page + t % page] = True
        seg = ok.kv4_segment_bytes(c.dim, page)
        for slot in np.flatnonzero(~keep):
            for of_v in (False, True):
                byte, _, scale = ok.kv4_places(c.dim, page, slot % page, of_v)
                view = c.pool[0, slot // page].reshape(c.kv_heads, seg)
                view[:, byte], view[:, scale] = 0xFF, 0x7F
        dirty = c.run()
        c.check(dirty)
        assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_attention_nan_and_inf_queries_stay_in_their_rows():
    c = Case(17, [90], [6], 4, 2, 128, 32, "fp16")
    good = [to_host(x.double()) for x in c.run()]
    c.q[2, 1, 5], c.q[4, 3, 0] = float("nan"), float("inf")
    out, lse = (to_host(x.double()) for x in c.run())
    bad = np.zeros((6, 4), bool)
    bad[2, 1] = bad[4, 3] = True
    assert np.isnan(out[bad]).all()
    assert np.array_equal(out[~bad], good[0][~bad]) and np.array_equal(lse[~bad], good[1][~bad])


def test_attention_strided_and_unaligned_queries():
    for dim, dtype in ((64, "fp16"), (128, "bf16")):
        c = Case(18, [50, 200], [3, 5], 6, 2, dim, 16, dtype)
        want = c.run()
        cache, table, kv_len, start = c.device()
        n = c.q.shape[0]
        for lead, pad in ((0, 8), (1, 3)):     # whole vectors, and rows that start anywhere
            buf = torch.zeros(n * 9 * (dim + pad) + 8, dtype=c.q.dtype, device=DEV)
            view = buf[lead:lead + n * 9 * (dim + pad)].view(n, 9, dim + pad)[:, 2:8, :dim]
            view.copy_(c.q)
            say("strided", dim, lead, pad)
            got = qd.kv4_attention(view, cache, table, kv_len, q_start=start, max_q_len=5)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # a transposed layout: heads outermost
        view = c.q.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
        got = qd.kv4_attention(view, cache, table, kv_len, q_start=start, max_q_len=5)
        assert torch.equal(got[0], want[0])


def test_attention_layers_uniform_blocks_and_bounds():
    """A later layer with its own scales, no q_start, a close max_kv_len, a
    caller's outputs and workspace, and a table that is a slice."""
    c = Case(19, [120, 33, 64], [4, 4, 4], 8, 4, 128, 32, "fp16", layers=3, layer=2)
    cache, table, kv_len, _ = c.device()
    cache = qd.KV4Cache.wrap(cache.data, 32, 4, 128, [9.0, 9.0, c.k_scale], [9.0, 9.0, c.v_scale])
    wide = torch.full((3, table.shape[1] + 5), 7, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    q = c.q.to(DEV)
    ws = qd.kv4_attention_workspace(cache, 12, 8, 3, 4, 120)
    out, lse = torch.full_like(q, 7.0), torch.full((12, 8), 7.0, device=DEV)
    say("layers")
    got = qd.kv4_attention(q, cache, wide[:, :table.shape[1]], kv_len, layer=2, max_kv_len=120, out=out, lse=lse,
                           workspace=ws, scale=c.scale)
    assert got[0] is out and got[1] is lse
    c.check(got)


def test_attention_same_bits_every_time():
    """No atomics in the sums: repeated calls, and other calls in between, give the same bits."""
    c = Case(20, [3000, 17, 900], [8, 3, 1], 10, 2, 128, 64, "fp16")
    first = c.run()
    Case(21, [500], [2], 10, 2, 128, 64, "fp16").run()
    again = c.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_pool_beyond_32_bit_offsets():
    """Pages whose bytes lie past 4 GiB."""
    say("large pool")
    page, kvh, dim, tokens = 256, 8, 128, 300
    nbytes = qd.qpn_kv4_page_bytes(page, kvh, dim)
    pages = (5 << 30) // nbytes
    cache = qd.KV4Cache(pages, page, kvh, dim, k_scale=0.002, v_scale=0.002)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    k, v, q = (torch.randn((tokens, kvh, dim), device=DEV, generator=g).half() for _ in range(3))
    slots = torch.cat([torch.arange(256) + (pages - 1) * page, torch.arange(44) + (pages - 3) * page]).to(DEV)
    qd.kv4_append(cache, k, v, slots)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=DEV)
    far = qd.kv4_attention(q[:4], cache, table, torch.tensor([tokens], dtype=torch.int32, device=DEV))
    qd.kv4_copy_pages(cache, torch.tensor([pages - 1, pages - 3], dtype=torch.int32, device=DEV),
                      torch.tensor([0, 1], dtype=torch.int32, device=DEV))
    near = qd.kv4_attention(q[:4], cache, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV),
                            torch.tensor([tokens], dtype=torch.int32, device=DEV))
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    kr, vr = qd.kv4_read(cache, slots, dtype=torch.float32)
    s = torch.einsum("qhd,thd->qht", q[:4].float().cpu(), kr.cpu()) * dim ** -0.5
    pos = tokens - 4 + torch.arange(4)
    s = s.masked_fill(torch.arange(tokens)[None, None] > pos[:, None, None], -math.inf)
    want = torch.einsum("qht,thd->qhd", torch.softmax(s, -1), vr.cpu())
    assert (far[0].float().cpu() - want).abs().max() < 4e-3   # fp16 roundings of p and of the result, |v| < 6


def test_attention_graph_replays_follow_lengths_and_tables():
    """Captured once, replayed with other lengths, tables, queries and slots."""
    c = Case(22, [200, 90], [2, 2], 4, 2, 128, 32, "fp16")
    cache, table, kv_len, start = c.device()
    q = c.q.to(DEV)
    k, v = (torch.randn((4, 2, 128), device=DEV).half() for _ in range(2))
    slots = torch.full((4,), -1, dtype=torch.int64, device=DEV)
    ws = qd.kv4_attention_workspace(cache, 4, 4, 2, 2, 224)
    out, lse = torch.empty_like(q), torch.empty((4, 4), device=DEV)

    def step():
        qd.kv4_append(cache, k, v, slots)
        qd.kv4_attention(q, cache, table, kv_len, q_start=start, max_q_len=2, max_kv_len=224, out=out, lse=lse,
                         workspace=ws)

    say("graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, (lens, at) in enumerate((([200, 90], -1), ([3, 91], 5), ([0, 64], 40), ([224, 1], 70))):
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        slots.copy_(torch.tensor([at, -1, at + 3, -1]))
        q.copy_(torch.randn(q.shape, device=DEV).half())
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i


def test_operators_on_a_side_stream():
    c = Case(23, [500, 40], [3, 1], 4, 2, 128, 32, "bf16")
    want = c.run()
    cache, table, kv_len, start = c.device()
    q = c.q.to(DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = qd.kv4_attention(q, cache, table, kv_len, q_start=start, max_q_len=3)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
