"""The 4-bit paged key/value cache and attention over it, element by element
(test-only oracle, float64 where numbers are computed).

A page of P tokens keeps, for each kv head of D elements, one segment
  K codes [P][D/2], V codes [P/4][16][4][D/32], K scales [P][D/16],
  V scales [P/4][D/16][4]
of bytes; an element is E2M1(code) * E4M3(block scale) * tensor scale, 16
elements a block. Quantization is the recipe of ``quantize_nvfp4`` with a given
tensor scale, except that the cache takes any input: the block scale saturates
at 448, an infinity is held as its block's largest value and NaN as 0.
"""

import numpy as np

from .formats import decode_e2m1, decode_e4m3, encode_e2m1, encode_e4m3


def kv4_segment_bytes(dim, page):
    return page * dim + page * dim // 8


def kv4_places(dim, page, off, of_v):
    """(code byte, code shift, scale byte) of each of the D elements of the
    token at offset `off`, within its segment."""
    byte = np.zeros(dim, np.int64)
    shift = np.zeros(dim, np.int64)
    scale = np.zeros(dim, np.int64)
    for d in range(dim):
        shift[d] = 4 * (d % 2)
        if of_v:
            each = dim // 16                  # elements of a token that lie together
            group, inner = d // each, d % each
            byte[d] = page * dim // 2 + ((off // 4) * 16 + group) * (4 * each // 2) + (off % 4) * (each // 2) + inner // 2
            scale[d] = page * dim + page * dim // 16 + ((off // 4) * (dim // 16) + d // 16) * 4 + off % 4
        else:
            byte[d] = off * (dim // 2) + d // 2
            scale[d] = page * dim + off * (dim // 16) + d // 16
    return byte, shift, scale


def kv4_quantize(x, tensor_scale):
    """(codes uint8 [..., D], block scale codes uint8 [..., D/16]) of float32 x."""
    x = np.asarray(x, np.float32)
    s_t = np.float32(tensor_scale)
    b = x.reshape(x.shape[:-1] + (-1, 16))
    with np.errstate(all="ignore"):
        mag = np.where(np.isnan(b), np.float32(0), np.abs(b))
        ratio = np.minimum((mag.max(axis=-1) / np.float32(6)) / s_t, np.float32(448))
        sc = encode_e4m3(ratio).astype(np.uint8)
        d = (decode_e4m3(sc).astype(np.float32) * s_t)[..., None]
        q = b / np.where(d == 0, np.float32(1), d)
    sign = (np.signbit(b).astype(np.uint8) << 3)
    q = np.clip(np.where(np.isnan(q), np.float32(0), q), np.float32(-6), np.float32(6))
    codes = np.where((d == 0) | np.isnan(b), sign, encode_e2m1(q)).astype(np.uint8)
    return codes.reshape(x.shape), sc


def kv4_values(codes, scales, tensor_scale):
    """float64 values of codes [..., D] and block scale codes [..., D/16]."""
    v = decode_e2m1(codes).astype(np.float64)
    s = np.repeat(decode_e4m3(scales).astype(np.float64), 16, axis=-1)
    return v * s * np.float64(np.float32(tensor_scale))


def kv4_store(pool, page, kv_heads, dim, slot, k, v):
    """Writes one token's (codes [kv_heads, D], scales [kv_heads, D/16]) pairs
    into a layer `pool` uint8 [pages, page_bytes]; a slot outside is skipped."""
    if slot < 0 or slot >= pool.shape[0] * page:
        return
    seg = pool[slot // page].reshape(kv_heads, kv4_segment_bytes(dim, page))
    for of_v, (codes, scales) in ((False, k), (True, v)):
        byte, shift, scale = kv4_places(dim, page, slot % page, of_v)
        for h in range(kv_heads):
            for d in range(dim):
                seg[h, byte[d]] = (seg[h, byte[d]] & (0xF0 >> shift[d])) | (int(codes[h, d]) << shift[d])
            seg[h, scale[::16]] = scales[h]


def kv4_load(pool, page, kv_heads, dim, slot):
    """((k codes, k scales), (v codes, v scales)) of one slot."""
    seg = pool[slot // page].reshape(kv_heads, kv4_segment_bytes(dim, page))
    out = []
    for of_v in (False, True):
        byte, shift, scale = kv4_places(dim, page, slot % page, of_v)
        out.append(((seg[:, byte] >> shift) & 15, seg[:, scale[::16]]))
    return out


def attention(q, k, v, seen, scale):
    """(out, lse, a, s) of one head: q [n, D], k and v [t, D] float64, seen
    [n, t] truth values. a = sum_t p |v| and s = max_t sum_d |q k| * scale are
    what rounding errors are measured in. A row that sees nothing: 0, -inf."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, dim = q.shape
    out, mag = np.zeros((n, dim)), np.zeros((n, dim))
    lse, size = np.full(n, -np.inf), np.zeros(n)
    for i in range(n):
        t = np.flatnonzero(seen[i])
        if t.size == 0:
            continue
        x = k[t] @ q[i] * scale
        m = x.max()
        p = np.exp(x - m)
        lse[i] = m + np.log(p.sum())
        p /= p.sum()
        out[i], mag[i] = p @ v[t], p @ np.abs(v[t])
        size[i] = (np.abs(k[t]) @ np.abs(q[i])).max() * scale
    return out, lse, mag, size


def visible(rows, kv_len, window):
    """[rows, kv_len]: which tokens the last `rows` positions see."""
    pos = kv_len - rows + np.arange(rows)[:, None]
    t = np.arange(kv_len)[None]
    seen = t <= pos
    if window:
        seen &= t > pos - window
    return seen


def verify(target, draft, draft_tokens, num_draft, temperature, u_accept, u_sample, probabilities):
    """(tokens, accepted, logprobs, margin) of a batch of verify blocks, by the
    definition, token by token. margin[b] is the smallest relative distance of
    any decision of sequence b from its border (an accept test, the place of
    u_sample among the running sums): where it is not well above the rounding
    of the arithmetic compared with, the decision may go either way."""
    target = np.asarray(target, np.float64)
    batch, places, vocab = target.shape
    tokens = np.full((batch, places), -1, np.int32)
    accepted = np.zeros(batch, np.int32)
    logprobs = np.zeros((batch, places))
    margin = np.full(batch, np.inf)

    def probs(x, t):
        x = np.asarray(x, np.float64)
        if probabilities:
            return np.where(x > 0, x, 0.0)
        x = np.where(np.isnan(x), -np.inf, x)
        m = x.max()
        if m == -np.inf:
            return np.zeros(vocab)
        with np.errstate(invalid="ignore"):
            w = np.where(x == m, 1.0, np.exp((x - m) / t))
        return w / w.sum()

    for b in range(batch):
        n = places - 1 if num_draft is None else int(min(max(num_draft[b], 0), places - 1))
        t = 1.0 if temperature is None else float(temperature[b])
        greedy = not probabilities and not t > 0
        t = t if t > 0 else 1.0
        rest = None
        for i in range(n + 1):
            p = probs(target[b, i], t)
            best = int(np.argmax(np.where(np.isnan(target[b, i]), -np.inf, target[b, i])))
            if i == n:
                rest = p
                break
            d = int(draft_tokens[b, i])
            known = 0 <= d < vocab
            if greedy:
                if not (known and p[d] > 0 and best == d):
                    rest = p
                    break
            else:
                q = probs(draft[b, i], t) if draft is not None else None
                pd = p[d] if known else 0.0
                qd = (q[d] if q is not None else 1.0) if known else 1.0
                lhs = float(u_accept[b, i]) * qd
                if known and max(lhs, pd) > 0:
                    margin[b] = min(margin[b], abs(lhs - pd) / max(lhs, pd))
                if not (known and lhs < pd):
                    if q is not None:
                        rest = np.maximum(p - q, 0)
                    else:
                        rest = p.copy()
                        if known:
                            rest[d] = 0
                    if not rest.sum() > 0:
                        rest = p
                    break
            tokens[b, i] = d
            with np.errstate(divide="ignore"):
                logprobs[b, i] = np.log(p[d])
            accepted[b] += 1
        a = accepted[b]
        token = -1
        if p.sum() > 0:
            if greedy:
                token = best
            else:
                cum = np.cumsum(rest)
                aim = float(u_sample[b]) * cum[-1]
                over = np.flatnonzero(cum > aim)
                token = int(over[0]) if over.size else int(np.flatnonzero(rest > 0)[-1])
                live = np.flatnonzero(rest > 0)
                margin[b] = min(margin[b], np.abs(cum[live[live < vocab - 1]] - aim).min(initial=np.inf) / cum[-1]
                                if live.size > 1 else np.inf)
        tokens[b, a] = token
        if token >= 0:
            logprobs[b, a] = np.log(p[token])
    return tokens, accepted, logprobs, margin
