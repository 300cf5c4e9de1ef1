"""GPU parity of attention where runs of tiles are cut into shares and joined
(bounds above 512 tokens and few runs), and where a wavefront walks more than the
64 tiles whose pages it looks up at once. Tolerances are those of
test_gpu_kv4.py."""

import functools

import numpy as np
import pytest
import torch

import oracle.kv4 as ok
from gpu_helpers import DEV, say, to_host
from quantized_weight_skinny_amd import decode_api as qd
from test_gpu_kv4 import Case

pytestmark = pytest.mark.gpu

PLACES = functools.lru_cache(maxsize=None)(ok.kv4_places)


@pytest.fixture(autouse=True)
def places_once(monkeypatch):
    """The oracle's byte places are worked out element by element: once an offset is enough."""
    monkeypatch.setattr(ok, "kv4_places", PLACES)


# (dim, rows of the longest sequence, query heads a kv head, type): one to four 16-row tiles of 64, one to three
# of 128, one and two of 256
SHAPES = [(64, 1, 4, "fp16"), (64, 8, 3, "bf16"), (64, 9, 4, "fp16"), (64, 16, 4, "bf16"), (128, 2, 5, "bf16"),
          (128, 4, 8, "fp16"), (128, 8, 5, "fp16"), (128, 16, 3, "bf16"), (256, 3, 5, "fp16"), (256, 4, 8, "bf16")]
LENGTHS = [1500, 40, 700]


def case(seed, shape, kv=LENGTHS, page=32, **kw):
    dim, rows, group, dtype = shape
    c = Case(seed, kv, [rows, max(1, rows // 2), rows], 2 * group, 2, dim, page, dtype, **kw)
    cache = qd.KV4Cache(0, page, 2, dim)
    ws = qd.kv4_attention_workspace(cache, c.q.shape[0], 2 * group, 3, rows, c.table.shape[1] * page)
    assert ws is not None                # the call cuts its runs
    return c, ws


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window", [0, 600])
def test_shapes(shape, window):
    c, _ = case(1, shape)
    c.check(c.run(window=window), window)


@pytest.mark.parametrize("shape", SHAPES)
def test_a_callers_workspace_needs_no_preparation(shape):
    c, ws = case(2, shape)
    want = c.run()
    for byte in (0xFF, 0x00, 0x7F):      # NaN, zeros, large numbers
        ws.fill_(byte)
        got = c.run(workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(got)


@pytest.mark.parametrize("shape", SHAPES)
def test_absent_and_bad_pages(shape):
    c, _ = case(3, shape)
    c.table[0, 1], c.table[0, 17], c.table[0, 46] = -1, c.pages, np.iinfo(np.int32).max
    c.table[2, 5:12] = np.iinfo(np.int32).min
    c.check(c.run())
    c.table[0, :30] = -1                 # whole shares without a token
    c.table[2, :] = -1
    c.check(c.run())


@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[6], SHAPES[9], SHAPES[0]])
def test_garbage_outside_the_sequences(shape):
    """NaN scales in every byte that belongs to no seen token change nothing."""
    c, _ = case(4, shape)
    clean = c.run()
    keep = np.zeros(c.pages * c.page, bool)
    for b, n in enumerate(c.kv):
        for t in range(n):
            keep[c.table[b, t // c.page] * c.page + t % c.page] = True
    seg = ok.kv4_segment_bytes(c.dim, c.page)
    for slot in np.flatnonzero(~keep):
        for of_v in (False, True):
            byte, _, scale = ok.kv4_places(c.dim, c.page, slot % c.page, of_v)
            view = c.pool[0, slot // c.page].reshape(c.kv_heads, seg)
            view[:, byte], view[:, scale] = 0xFF, 0x7F
    dirty = c.run()
    c.check(dirty)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("shape", SHAPES)
def test_nan_and_inf_queries_stay_in_their_rows(shape):
    c, _ = case(5, shape)
    good = [to_host(x.double()) for x in c.run()]
    last = c.q.shape[0] - 1
    c.q[0, 1, 5], c.q[last, 3, 0] = float("nan"), float("inf")
    out, lse = (to_host(x.double()) for x in c.run())
    bad = np.zeros(out.shape[:2], bool)
    bad[0, 1] = bad[last, 3] = True
    assert np.isnan(out[bad]).all()
    assert np.array_equal(out[~bad], good[0][~bad]) and np.array_equal(lse[~bad], good[1][~bad])


@pytest.mark.parametrize("shape", SHAPES)
def test_strided_and_unaligned_queries(shape):
    c, _ = case(6, shape)
    want = c.run()
    cache, table, kv_len, start = c.device()
    n, heads, dim = c.q.shape
    for lead, pad in ((0, 8), (1, 3)):   # whole vectors, and rows that start anywhere
        buf = torch.zeros(n * (heads + 3) * (dim + pad) + 8, dtype=c.q.dtype, device=DEV)
        view = buf[lead:lead + n * (heads + 3) * (dim + pad)].view(n, heads + 3, dim + pad)[:, 2:2 + heads, :dim]
        view.copy_(c.q)
        say("strided", shape, lead, pad)
        got = qd.kv4_attention(view, cache, table, kv_len, q_start=start, max_q_len=max(c.rows))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[6], SHAPES[9]])
def test_on_a_side_stream(shape):
    c, _ = case(7, shape)
    want = c.run()
    cache, table, kv_len, start = c.device()
    q = c.q.to(DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = qd.kv4_attention(q, cache, table, kv_len, q_start=start, max_q_len=max(c.rows))
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[6], SHAPES[9]])
def test_graph_replays_follow_lengths_and_tables(shape):
    """Captured once with a caller's workspace, replayed with other lengths, tables, blocks and queries; runs are cut
    elsewhere, or not at all, each time."""
    c, ws = case(8, shape, kv=[1500, 1400, 700])
    cache, table, kv_len, start = c.device()
    q, most = c.q.to(DEV), max(c.rows)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    bound = table.shape[1] * c.page

    def step():
        qd.kv4_attention(q, cache, table, kv_len, q_start=start, max_q_len=most, max_kv_len=bound, out=out, lse=lse,
                         workspace=ws, scale=c.scale)

    say("graph", shape)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(0)
    # (no longer than what the tables hold)
    for i, lens in enumerate(([1500, 1400, 700], [3, 0, 700], [1500, 1, 33], [0, 0, 0], [900, 1400, 5], [1499, 1399, 699])):
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        c.table[0, :c.table.shape[1] // 2] = rng.permutation(c.table[0, :c.table.shape[1] // 2])
        table.copy_(torch.from_numpy(c.table))
        c.q = torch.from_numpy(rng.standard_normal(tuple(c.q.shape)).astype(np.float32)).to(c.q.dtype)
        q.copy_(c.q)
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        c.kv = lens
        c.check(got)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i


# ---------------------------------------------------------------- more than 64 tiles a wavefront

@pytest.mark.parametrize("shape", [(128, 8, 5, "fp16"), (128, 1, 4, "bf16"), (64, 8, 8, "fp16"), (256, 4, 8, "bf16")])
@pytest.mark.parametrize("batch", [320, 160])
def test_wavefronts_of_more_than_64_tiles(shape, batch):
    """Many sequences over the same pages, one oracle for all: 320 of 8 kv heads go whole (71 tiles a wavefront), 160
    are cut into shares of 377 tiles and more. Page 128 of 64 tokens is where the 65th tile begins."""
    dim, rows, group, dtype = shape
    kvh, page, tokens = 8, 64, 9000
    c = Case(dim + batch, [tokens], [rows], kvh * group, kvh, dim, page, dtype)
    c.table[0, [0, 63, 64, 127, 129, 140]] = -1
    cache = qd.KV4Cache.wrap(torch.from_numpy(c.pool).to(DEV), page, kvh, dim, c.k_scale, c.v_scale)
    table = torch.from_numpy(c.table).to(DEV).repeat(batch, 1)
    whole = qd.kv4_attention_workspace(cache, batch * rows, kvh * group, batch, rows, tokens) is None
    assert whole == (batch == 320)
    say("long walks", shape, batch, "whole" if whole else "cut")
    out, lse = qd.kv4_attention(c.q.to(DEV).repeat(batch, 1, 1), cache, table,
                                torch.full((batch,), tokens, dtype=torch.int32, device=DEV), max_kv_len=tokens,
                                scale=c.scale)
    out, lse = to_host(out.float()).reshape(batch, rows, kvh * group, dim), to_host(lse).reshape(batch, rows, -1)
    for _, heads, o, l, ot, lt in c.expected():
        assert (np.abs(out[:, :, heads] - o) <= ot).all(), np.max(np.abs(out[:, :, heads] - o) / ot)
        assert (np.abs(lse[:, :, heads] - l) <= lt).all()
    if whole:
        assert (out == out[0]).all() and (lse == lse[0]).all()
