"""The oracle of the 4-bit cache and of draft verification against something
other than itself: hand cases, torch's attention by definition, a round trip
through the byte layout, and the theorem of speculative sampling."""

import numpy as np
import pytest
import torch

import oracle
import oracle.kv4 as ok


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_places_cover_a_segment_once(dim, page):
    seen = np.zeros((ok.kv4_segment_bytes(dim, page), 2), int)
    for of_v in (False, True):
        for off in range(page):
            byte, shift, scale = ok.kv4_places(dim, page, off, of_v)
            for d in range(dim):
                seen[byte[d], shift[d] // 4] += 1
            for s in scale[::16]:
                seen[s] += 1
            assert all(np.unique(scale[i:i + 16]).size == 1 for i in range(0, dim, 16))
    assert (seen == 1).all()


def test_places_by_hand():
    # D 128, page 16: token 5's element 9 of K: byte 5 * 64 + 4, high nibble
    byte, shift, scale = ok.kv4_places(128, 16, 5, False)
    assert (byte[9], shift[9], scale[9]) == (5 * 64 + 4, 4, 16 * 128 + 5 * 8)
    # of V: quad 1, group 1 (elements 8..15), token 1 of the quad, byte 0 of its four, high nibble
    byte, shift, scale = ok.kv4_places(128, 16, 5, True)
    assert (byte[9], shift[9]) == (16 * 64 + 1 * 256 + 1 * 16 + 1 * 4, 4)
    assert scale[9] == 16 * 128 + 16 * 8 + 1 * 32 + 0 * 4 + 1


def test_store_and_load_round_trip():
    rng = np.random.default_rng(1)
    pool = rng.integers(0, 256, (3, 2 * ok.kv4_segment_bytes(64, 16)), dtype=np.uint8)
    want = {}
    for slot in (0, 17, 18, 47, 33):
        k = ok.kv4_quantize(rng.standard_normal((2, 64)), 0.01)
        v = ok.kv4_quantize(rng.standard_normal((2, 64)), 0.02)
        ok.kv4_store(pool, 16, 2, 64, slot, k, v)
        want[slot] = (k, v)
    ok.kv4_store(pool, 16, 2, 64, -1, *want[0])
    ok.kv4_store(pool, 16, 2, 64, 48, *want[0])
    for slot, pair in want.items():
        for (c, s), (wc, ws) in zip(ok.kv4_load(pool, 16, 2, 64, slot), pair):
            assert np.array_equal(c, wc) and np.array_equal(s, ws)


def test_quantize_agrees_with_the_weights_recipe():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((40, 128)) * np.exp(rng.uniform(-4, 2, (40, 1)))).astype(np.float32)
    codes, scales = ok.kv4_quantize(x, 0.01)
    wc, ws, _ = oracle.quantize_nvfp4(x, tensor_scale=0.01)
    assert np.array_equal(codes, wc) and np.array_equal(scales, ws)


def test_quantize_extremes():
    x = np.zeros((1, 48), np.float32)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = np.inf, -np.inf, np.nan, 1.0
    x[0, 16:32] = -0.0
    x[0, 32] = 1e9
    codes, scales = ok.kv4_quantize(x, 1.0)
    assert scales[0].tolist() == [0x7E, 0, 0x7E]              # 448, 0, saturated
    assert codes[0, :4].tolist() == [7, 15, 0, 0]             # 6, -6, 0, and 1 / 448 rounds to 0
    assert (codes[0, 16:32] == 8).all() and codes[0, 32] == 7


def test_attention_against_torch():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 16), (30, 16), (30, 16)))
    for window in (0, 4):
        seen = ok.visible(5, 30, window)
        out, lse, a, s = ok.attention(q.numpy(), k.numpy(), v.numpy(), seen, 0.25)
        x = (q @ k.T * 0.25).masked_fill(~torch.from_numpy(seen), -torch.inf)
        assert np.allclose(out, (torch.softmax(x, 1) @ v).numpy(), atol=1e-13)
        assert np.allclose(lse, torch.logsumexp(x, 1).numpy(), atol=1e-13)
        assert (np.abs(out) <= a + 1e-15).all()


def test_visible_by_hand():
    assert ok.visible(2, 4, 0).tolist() == [[True, True, True, False], [True] * 4]
    assert ok.visible(2, 4, 2).tolist() == [[False, True, True, False], [False, False, True, True]]
    assert ok.visible(3, 1, 0).tolist() == [[False], [False], [True]]     # rows before the start see nothing
    out, lse, _, _ = ok.attention(np.ones((3, 2)), np.ones((1, 2)), np.ones((1, 2)), ok.visible(3, 1, 0), 1.0)
    assert out.tolist() == [[0, 0], [0, 0], [1, 1]] and np.isneginf(lse[:2]).all() and lse[2] == 2


def test_verify_by_hand():
    p = np.log(np.array([[[0.5, 0.25, 0.25], [0.1, 0.1, 0.8]]]))
    q = np.log(np.array([[[0.25, 0.5, 0.25]]]))
    def go(d, u, v, draft=q, temperature=None):
        return [x.tolist() for x in ok.verify(p, draft, np.array([[d]]), None, temperature, np.array([[u]]),
                                              np.array([v]), False)[:3]]
    # draft 1: p/q = 1/2
    t, a, lp = go(1, 0.49, 0.15)
    assert t == [[1, 1]] and a == [1] and np.allclose(lp, [[np.log(0.25), np.log(0.1)]])
    # rejected: max(p - q, 0) is all on token 0
    t, a, _ = go(1, 0.51, 0.99)
    assert t == [[0, -1]] and a == [0]
    # draft 0 is always accepted, then the next row's 0.1, 0.2, 1.0
    assert go(0, 0.999, 0.05)[0] == [[0, 0]] and go(0, 0.999, 0.5)[0] == [[0, 2]]
    # without a draft row: accepted with p = 1/4; else from p without the draft (2/3, -, 1/3)
    assert go(1, 0.24, 0.15, None)[0] == [[1, 1]]
    assert go(1, 0.26, 0.6, None)[0] == [[0, -1]] and go(1, 0.26, 0.7, None)[0] == [[2, -1]]
    # greedy
    assert go(0, 0.9, 0.9, q, np.array([0.0]))[0] == [[0, 2]] and go(1, 0.0, 0.0, q, np.array([0.0]))[0] == [[0, -1]]


def test_verify_keeps_the_targets_distribution():
    rng = np.random.default_rng(4)
    n, vocab = 20000, 5
    p, q = rng.dirichlet(np.ones(vocab)), rng.dirichlet(np.ones(vocab))
    drafts = rng.choice(vocab, (n, 1), p=q)
    tokens, _, _, _ = ok.verify(np.broadcast_to(p, (n, 2, vocab)), np.broadcast_to(q, (n, 1, vocab)), drafts, None, None,
                                rng.random((n, 1)), rng.random(n), True)
    freq = np.bincount(tokens[:, 0], minlength=vocab) / n
    assert (np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / n)).all()
