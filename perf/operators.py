"""The work that decides how fast a verify step's memory and its answer are:
cases over the 4-bit paged key/value cache (append, attention, page copies)
and over the verification of drafted tokens, each in a plain form written with
elementary torch operations, and as calls of this package.

The cache (one byte buffer ``data[layers, pages, page_bytes]``): a page holds
``page`` tokens, and in it every kv head has one segment of four arrays,

  K codes   [page][D / 2]             byte j: elements 2j (low nibble), 2j + 1
  V codes   [page / 4][16][4][D / 32] 4 tokens interleaved per D / 16 elements
  K scales  [page][D / 16]            one E4M3 byte per 16 elements
  V scales  [page / 4][D / 16][4]

A value is E2M1(code) * E4M3(block scale) * tensor scale. Token t of sequence
b lives in page ``table[b, t / page]`` at offset ``t % page``; a slot is
``page_index * page + offset``.
"""

import math

import torch

own = False

DEV = "cuda"

# Sizes: a ~27B dense decoder with 5120 query and 2 x 1024 key/value features
# (40 query and 8 kv heads of 128), its share under 4-way tensor parallelism
# (10 and 2), 64 layers, an output head of 151936 rows, and verify blocks of
# up to 16 rows.
HEADS, KV_HEADS, VOCAB, LAYERS = 40, 8, 151936, 64


def listed():
    return [
        # the first tokens of a chat: one sequence, one row, a few hundred tokens; latency is all there is
        attention("attn 1x1 len 300", 1, 1, 300, 300, "fp16"),
        # one user's long document: the 8 rows of a verify block over 128k tokens
        attention("attn 1x8 len 131072", 1, 8, 131072, 131072, "fp16"),
        # a server's batch: 48 sequences of very different lengths, each with its verify block
        attention("attn 48x8 len 200-16384", 48, 8, 200, 16384, "bf16"),
        # one rank of four, plain decoding of 24 sequences, small pages
        attention("attn 24x1 len 20000-33000", 24, 1, 20000, 33000, "fp16", heads=10, kv_heads=2, page=16),
        # wide heads, ragged short blocks, a sliding window over most of the context
        attention("attn 9x1-4 window 4096", 9, 4, 3000, 40000, "bf16", heads=24, kv_heads=4, dim=256, page=32,
                  window=4096, ragged=True),
        # the verify block's own keys and values enter the cache, cut out of the qkv projection's output
        append("append 8", 8, "fp16"),
        # a prompt's keys and values
        append("append 16389", 16389, "bf16"),
        # a sequence forks: its last, half-full page is copied in every layer
        copy("copy 1 page", 1, LAYERS, 64),
        # a pool is compacted
        copy("copy 2500 pages", 2500, 8, 7000),
        # the rows of one verify block straight from the output head; the drafts were taken greedily
        verify("verify 1x7", 1, 7, VOCAB, "fp16", "none"),
        # a server's batch with the drafter's own logits, some sequences greedy
        verify("verify 32x7 draft logits", 32, 7, VOCAB, "fp16", "logits", ragged=True),
        # probabilities after a filter, fewer drafts, an odd vocabulary
        verify("verify 40x3 probabilities", 40, 3, 50021, "fp32", "probs"),
    ]


def attention(name, batch, rows, shortest, longest, dtype, heads=HEADS, kv_heads=KV_HEADS, dim=128, page=64, window=0,
              ragged=False):
    return {"name": name, "op": "attention", "batch": batch, "rows": rows, "shortest": shortest, "longest": longest,
            "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window,
            "ragged": ragged}


def append(name, tokens, dtype, heads=HEADS, kv_heads=KV_HEADS, dim=128, page=64):
    return {"name": name, "op": "append", "tokens": tokens, "dtype": dtype, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page}


def copy(name, count, layers, pages, kv_heads=KV_HEADS, dim=128, page=64):
    return {"name": name, "op": "copy", "count": count, "layers": layers, "pages": pages, "kv_heads": kv_heads,
            "dim": dim, "page": page}


def verify(name, batch, drafts, vocab, dtype, draft, ragged=False):
    return {"name": name, "op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab, "dtype": dtype,
            "draft": draft, "ragged": ragged}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "copy", "verify", "verify"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = _log(rng, 1, 8)
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "attention":
        batch, rows, group = _log(rng, 1, 64), rng.randint(1, 16), rng.randint(1, 8)
        # at most the long document's cache and products: 131072 tokens in 8 heads of 128, 40 rows each
        most = 131072 * 8 * 128 * 40 // (batch * kv_heads * dim * max(40, rows * group))
        longest = _log(rng, 1, max(64, min(131072, most)))
        case = attention("", batch, rows, _log(rng, 1, longest), longest, dtype, kv_heads * group, kv_heads, dim, page,
                         rng.choice([0, 0, 0, _log(rng, 1, 8192)]), rng.random() < 0.3)
    elif op == "append":
        case = append("", _log(rng, 1, 16000), dtype, kv_heads * rng.randint(1, 8), kv_heads, dim, page)
    elif op == "copy":
        layers, count = _log(rng, 1, 64), _log(rng, 1, 3000)
        count = max(1, min(count, 10 ** 9 // (layers * page * kv_heads * dim * 9 // 8)))
        case = copy("", count, layers, 2 * count + rng.randint(1, 9), kv_heads, dim, page)
    else:
        drafts = rng.randint(1, 15)
        case = verify("", max(1, min(_log(rng, 1, 64), 250 // drafts)), drafts, _log(rng, 1000, 151936),
                      rng.choice(["fp16", "bf16", "fp32"]), rng.choice(["none", "logits", "probs"]),
                      rng.random() < 0.5)
        if case["draft"] == "probs":
            case["dtype"] = "fp32"
    case.pop("name")
    return case


TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ inputs

def segment_bytes(dim, page):
    return page * dim + page * dim // 8


def _cache(gen, layers, pages, page, kv_heads, dim):
    """A pool whose bytes are those of quantized normal values of deviation 1
    (with the tensor scale below): block maxima near twice the deviation, codes
    as such blocks hold them."""
    table = torch.arange(65536, device=DEV)
    nibble = torch.arange(256, device=DEV, dtype=torch.float64)
    # 256 equally likely normal values scaled by 6 / 2.1 and rounded to a code
    x = torch.special.ndtri((nibble + 0.5) / 256) * (6 / 2.1)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV, dtype=torch.float64)
    code = torch.bucketize(x.abs(), mids) + 8 * (x < 0)
    table = (code[table & 255] | (code[table >> 8] << 4)).to(torch.uint8)
    seg = segment_bytes(dim, page)
    data = torch.empty((layers, pages, kv_heads, seg), dtype=torch.uint8, device=DEV)
    for la in range(layers):
        for p in range(0, pages, 4096):
            part = data[la, p:p + 4096]
            r = torch.randint(0, 65536, (part.shape[0], kv_heads, page * dim), device=DEV, generator=gen,
                              dtype=torch.int32)
            part[:, :, :page * dim] = table[r]
            s = torch.randn((part.shape[0], kv_heads, page * dim // 8), device=DEV, generator=gen) * 0.4 + 2.1
            s = (s.clamp(0.9, 4.0) * 100).to(torch.float8_e4m3fn)
            part[:, :, page * dim:] = s.view(torch.uint8)
    return data.reshape(layers, pages, kv_heads * seg)


SCALE = 1 / 600.0  # a block maximum of 2.1 is code 6 times block scale 210


def _lengths(case):
    """Each sequence's rows and tokens: spread over the range by golden-ratio
    steps, so that they are known without asking the GPU."""
    n = case["batch"]
    share = [(0.618033988749895 * i) % 1.0 for i in range(n)]
    share[-1] = 1.0
    lo, hi = case["shortest"], case["longest"]
    kv = [int(round(math.exp(math.log(lo) + s * (math.log(hi) - math.log(lo))))) for s in share]
    rows = [1 + (i * 7 + 3) % case["rows"] if case["ragged"] else case["rows"] for i in range(n)]
    rows[-1] = case["rows"]
    return rows, kv


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"attention": _prepare_attention, "append": _prepare_append, "copy": _prepare_copy,
            "verify": _prepare_verify}[case["op"]](case, gen)


def _prepare_attention(case, gen):
    page, dim, kvh = case["page"], case["dim"], case["kv_heads"]
    rows, kv = _lengths(case)
    held = [-(-n // page) for n in kv]
    pages = sum(held) + 3
    data = _cache(gen, 1, pages, page, kvh, dim)
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((case["batch"], max(held)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    # queries as the projection leaves them, in front of the keys and values of the same tokens
    qkv = torch.randn((start[-1], (case["heads"] + 2 * kvh) * dim), device=DEV, generator=gen) * 1.5
    qkv = qkv.to(TYPES[case["dtype"]])
    q = qkv[:, :case["heads"] * dim].view(start[-1], case["heads"], dim)
    return {"case": case, "data": data, "q": q, "table": table,
            "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV),
            "q_start": torch.tensor(start, dtype=torch.int32, device=DEV),
            "max_rows": max(rows), "max_kv": max(kv)}


def _prepare_append(case, gen):
    page, dim, kvh, tokens = case["page"], case["dim"], case["kv_heads"], case["tokens"]
    pages = -(-tokens // page) + 5
    data = _cache(gen, 1, pages, page, kvh, dim)
    order = torch.randperm(pages, device=DEV, generator=gen)
    t = torch.arange(tokens, device=DEV) + 3  # the block begins inside a page
    slots = order[t // page] * page + t % page
    width = (case["heads"] + 2 * kvh) * dim
    qkv = torch.randn((tokens, width), device=DEV, generator=gen)
    # keys have a few strong channels
    strong = torch.rand((width,), device=DEV, generator=gen) < 0.02
    qkv = torch.where(strong, qkv * 6, qkv).to(TYPES[case["dtype"]])
    k = qkv[:, case["heads"] * dim:(case["heads"] + kvh) * dim].view(tokens, kvh, dim)
    v = qkv[:, (case["heads"] + kvh) * dim:].view(tokens, kvh, dim)
    return {"case": case, "data": data, "k": k, "v": v, "slots": slots}


def _prepare_copy(case, gen):
    data = _cache(gen, case["layers"], case["pages"], case["page"], case["kv_heads"], case["dim"])
    order = torch.randperm(case["pages"], device=DEV, generator=gen).to(torch.int32)
    return {"case": case, "data": data, "src": order[:case["count"]].contiguous(),
            "dst": order[case["count"]:2 * case["count"]].contiguous()}


def _prepare_verify(case, gen):
    batch, n, vocab, kind = case["batch"], case["drafts"], case["vocab"], TYPES[case["dtype"]]
    # logits with the long tail of a language model's: a few tokens carry most of the mass
    draft = torch.randn((batch, n, vocab), device=DEV, generator=gen) * 2.5
    lift = torch.randint(0, vocab, (batch, n, 6), device=DEV, generator=gen)
    draft.scatter_add_(2, lift, torch.rand((batch, n, 6), device=DEV, generator=gen) * 12)
    target = torch.cat([draft + 0.7 * torch.randn((batch, n, vocab), device=DEV, generator=gen),
                        torch.randn((batch, 1, vocab), device=DEV, generator=gen) * 3], dim=1)
    temperature = torch.rand((batch,), device=DEV, generator=gen) + 0.3
    if case["draft"] != "probs":
        temperature[2::5] = 0
    t = torch.where(temperature > 0, temperature, torch.ones_like(temperature))[:, None, None]
    if case["draft"] == "none":
        tokens = draft.argmax(dim=2)
    else:
        noise = -torch.log(-torch.log(torch.rand((batch, n, vocab), device=DEV, generator=gen).clamp(1e-7, 1 - 1e-7)))
        tokens = (draft / t + noise).argmax(dim=2)
    if case["draft"] == "probs":
        # a filter has left each row its tokens above a thousandth of the largest
        target, draft = (torch.softmax(x / t, dim=2) for x in (target, draft))
        target, draft = (torch.where(x >= 1e-3 * x.amax(2, True), x, 0) for x in (target, draft))
        target, draft = (x / x.sum(2, True) for x in (target, draft))
    count = [1 + (3 * b + 2) % n if case["ragged"] else n for b in range(batch)]
    count[0] = 0 if case["ragged"] and batch > 2 else count[0]
    return {"case": case, "target": target.to(kind), "draft": None if case["draft"] == "none" else draft.to(kind),
            "tokens": tokens.to(torch.int32), "num_draft": torch.tensor(count, dtype=torch.int32, device=DEV),
            "temperature": temperature, "u_accept": torch.rand((batch, n), device=DEV, generator=gen),
            "u_sample": torch.rand((batch,), device=DEV, generator=gen)}


# ------------------------------------------------------------------ one pass

def run(state):
    return {"attention": _run_attention, "append": _run_append, "copy": _run_copy,
            "verify": _run_verify}[state["case"]["op"]](state)


def _handle(state):
    """The cache object and the workspace that a program keeps."""
    if "handle" not in state:
        from quantized_weight_skinny_amd import decode_api as qd
        c = state["case"]
        cache = qd.KV4Cache.wrap(state["data"], c["page"], c["kv_heads"], c["dim"], SCALE, SCALE)
        ws = None
        if c["op"] == "attention":
            ws = qd.kv4_attention_workspace(cache, state["q"].shape[0], c["heads"], c["batch"], state["max_rows"],
                                            state["max_kv"])
        state["handle"] = (qd, cache, ws)
    return state["handle"]


def _split(data, case):
    """K codes, V codes, K scales and V scales of pages [..., page_bytes], in token order."""
    page, dim = case["page"], case["dim"]
    lead = data.shape[:-1] + (case["kv_heads"],)
    seg = data.reshape(*lead, segment_bytes(dim, page))
    half, n = page * dim // 2, len(lead)
    kc = seg[..., :half].reshape(*lead, page, dim // 2)
    vc = seg[..., half:2 * half].reshape(*lead, page // 4, 16, 4, dim // 32).transpose(n + 1, n + 2)
    ks = seg[..., 2 * half:2 * half + half // 8].reshape(*lead, page, dim // 16)
    vs = seg[..., 2 * half + half // 8:].reshape(*lead, page // 4, dim // 16, 4).transpose(n + 1, n + 2)
    return kc, vc.reshape(*lead, page, dim // 2), ks, vs.reshape(*lead, page, dim // 16)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(codes, scales, scale):
    """float32 values of code bytes [..., D / 2] and E4M3 scale bytes [..., D / 16]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    both = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), dim=1)  # byte -> its two values
    x = both[codes.to(torch.int32)].flatten(-2)
    s = scales.view(torch.float8_e4m3fn).to(torch.float32)
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * scale


def _run_attention(state):
    c = state["case"]
    if own:
        qd, cache, ws = _handle(state)
        return qd.kv4_attention(state["q"], cache, state["table"], state["kv_len"], q_start=state["q_start"],
                                max_q_len=state["max_rows"], max_kv_len=state["max_kv"], window=c["window"],
                                workspace=ws)
    q, page, group = state["q"], c["page"], c["heads"] // c["kv_heads"]
    batch, total, rows = c["batch"], state["q"].shape[0], state["max_rows"]
    start, kv_len = state["q_start"].long(), state["kv_len"].long()
    # [batch, kv head, tokens, dim] in float32
    kc, vc, ks, vs = _split(state["data"][0][state["table"].clamp(min=0).long()], c)
    k = _values(kc, ks, SCALE).permute(0, 2, 1, 3, 4).flatten(2, 3)
    v = _values(vc, vs, SCALE).permute(0, 2, 1, 3, 4).flatten(2, 3)
    # queries padded to the longest block: [batch, kv head, rows * group, dim]
    i = torch.arange(rows, device=q.device)
    here = i[None] < (start[1:] - start[:-1])[:, None]
    at = (start[:-1, None] + i[None]).clamp(max=total - 1)
    qp = q[at].float().view(batch, rows, c["kv_heads"], group, c["dim"])
    qp = qp.permute(0, 2, 1, 3, 4).reshape(batch * c["kv_heads"], rows * group, c["dim"])
    s = torch.bmm(qp, k.flatten(0, 1).transpose(1, 2).contiguous()) / math.sqrt(c["dim"])
    s = s.view(batch, c["kv_heads"], rows, group, -1)
    # row i of a sequence sits at position kv_len - rows + i and sees the window's tokens up to its own
    pos = (kv_len - (start[1:] - start[:-1]))[:, None] + i[None]
    t = torch.arange(k.shape[2], device=q.device)
    seen = t <= pos[..., None]
    if c["window"]:
        seen &= t > pos[..., None] - c["window"]
    s = s.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = s.amax(-1, True)
    p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
    z = p.sum(-1, True)
    o = torch.bmm(p.view(batch * c["kv_heads"], rows * group, -1), v.flatten(0, 1).contiguous())
    o = o.view(batch, c["kv_heads"], rows, group, c["dim"]) / torch.where(z > 0, z, 1.0)
    lse = (top + torch.log(z)).squeeze(-1)
    # back to [tokens, heads, ...]
    o = o.permute(0, 2, 1, 3, 4)[here].reshape(total, c["heads"], c["dim"]).to(q.dtype)
    return o, lse.permute(0, 2, 1, 3)[here].reshape(total, c["heads"])


def _quantize(x, scale):
    """E2M1 codes packed in bytes [..., D / 2] and E4M3 scale bytes [..., D / 16] of x."""
    b = x.float().unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / 6.0 / scale).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s.float() * scale)[..., None]
    a = (b / torch.where(d > 0, d, 1.0)).abs() * (d > 0)
    # the midpoints of the grid; an equal distance goes to the even code
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * torch.signbit(b)).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), s.view(torch.uint8)


def _places(c, slots):
    """Byte places in a pool of the four arrays of each slot's token: [tokens, kv_heads, bytes]."""
    page, dim, kvh = c["page"], c["dim"], c["kv_heads"]
    seg, half = segment_bytes(dim, page), page * dim // 2
    slots = slots.long()[:, None, None]
    off = slots % page
    base = slots // page * (kvh * seg) + torch.arange(kvh, device=slots.device)[None, :, None] * seg
    j = torch.arange(dim // 2, device=slots.device)
    m = torch.arange(dim // 16, device=slots.device)
    wide = dim // 32
    return (base + off * (dim // 2) + j,
            base + half + off // 4 * (2 * dim) + j // wide * (4 * wide) + off % 4 * wide + j % wide,
            base + 2 * half + off * (dim // 16) + m,
            base + 2 * half + half // 8 + off // 4 * (dim // 4) + m * 4 + off % 4)


def _run_append(state):
    c = state["case"]
    if own:
        qd, cache, _ = _handle(state)
        qd.kv4_append(cache, state["k"], state["v"], state["slots"])
        return qd.kv4_read(cache, state["slots"], dtype=state["k"].dtype)
    flat = state["data"].view(-1)
    kc_at, vc_at, ks_at, vs_at = _places(c, state["slots"])
    kc, ks = _quantize(state["k"], SCALE)
    vc, vs = _quantize(state["v"], SCALE)
    flat[kc_at], flat[ks_at], flat[vc_at], flat[vs_at] = kc, ks, vc, vs
    return (_values(flat[kc_at], flat[ks_at], SCALE).to(state["k"].dtype),
            _values(flat[vc_at], flat[vs_at], SCALE).to(state["v"].dtype))


def _run_copy(state):
    if own:
        qd, cache, _ = _handle(state)
        qd.kv4_copy_pages(cache, state["src"], state["dst"])
        return state["data"]
    state["data"][:, state["dst"].long()] = state["data"][:, state["src"].long()]
    return state["data"]


def _run_verify(state):
    c = state["case"]
    if own:
        from quantized_weight_skinny_amd import decode_api as qd
        if "workspace" not in state:
            state["workspace"] = qd.verify_workspace(c["batch"], c["drafts"], c["vocab"])
        return qd.verify_drafts(state["target"], state["tokens"], state["u_accept"], state["u_sample"],
                                draft=state["draft"], num_draft=state["num_draft"],
                                temperature=None if c["draft"] == "probs" else state["temperature"],
                                probabilities=c["draft"] == "probs", workspace=state["workspace"])
    # sums of exponentials and the place of a random number among them are held in 64 bits: a vocabulary's
    # running sums lie closer together than 32 bits tell apart
    n, vocab, tokens = c["drafts"], c["vocab"], state["tokens"].long()
    target = state["target"].double()
    draft = state["draft"].double() if state["draft"] is not None else None
    greedy = torch.zeros(c["batch"], dtype=torch.bool, device=target.device)
    p, q = target, draft
    if c["draft"] != "probs":
        greedy = state["temperature"] <= 0
        t = torch.where(greedy, 1.0, state["temperature"].double())[:, None, None]
        p = torch.softmax(target / t, dim=2)
        q = torch.softmax(draft / t, dim=2) if draft is not None else None
    best = target.argmax(dim=2)
    pd = p[:, :n].gather(2, tokens[..., None])[..., 0]
    qd_ = q.gather(2, tokens[..., None])[..., 0] if q is not None else 1.0
    ok = state["u_accept"].double() * qd_ < pd
    ok = torch.where(greedy[:, None], best[:, :n] == tokens, ok)
    step = torch.arange(n, device=target.device)
    ok &= step[None] < state["num_draft"][:, None]
    accepted = ok.long().cumprod(dim=1).sum(dim=1)
    # the next token: from what the draft left over at the first rejected place, or from the row after the last draft
    row = torch.arange(c["batch"], device=target.device)
    w = p[row, accepted]
    rejected = accepted < state["num_draft"]
    at = accepted.clamp(max=n - 1)
    if q is not None:
        over = (w - q[row, at]).clamp(min=0)
    else:
        over = w.scatter(1, tokens[row, at][:, None], 0.0)
    over = torch.where(over.sum(1, True) > 0, over, w)
    w = torch.where(rejected[:, None], over, w)
    cum = w.cumsum(dim=1)
    place = (cum <= state["u_sample"].double()[:, None] * cum[:, -1:]).sum(dim=1)
    last = (vocab - 1) - (w.flip(1) > 0).to(torch.uint8).argmax(dim=1)
    token = torch.where(greedy, best[row, accepted], torch.minimum(place, last))
    steps = torch.arange(n + 1, device=target.device)[None]
    out = torch.where(steps < accepted[:, None], torch.nn.functional.pad(tokens, (0, 1)), -1)
    out = torch.where(steps == accepted[:, None], token[:, None], out)
    # the target's log-probability of each token that is given
    logp = torch.log(p.gather(2, out.clamp(min=0)[..., None]))[..., 0]
    logp = torch.where(out >= 0, logp, 0.0)
    return out.to(torch.int32), accepted.to(torch.int32), logp.float()


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "attention":
        rows, kv = _lengths(case)
        dim, kvh, heads, w = case["dim"], case["kv_heads"], case["heads"], case["window"]
        tokens = sum(n if not w else min(n, w + r - 1) for r, n in zip(rows, kv))
        pairs = 0
        for r, n in zip(rows, kv):
            for i in range(r):
                seen = max(0, n - r + i + 1)
                pairs += min(seen, w) if w else seen
        io = sum(rows) * heads * (dim * 2 * 2 + 4) + 4 * sum(-(-n // case["page"]) for n in kv)
        return {"bytes": tokens * kvh * (dim + dim // 8) + io, "flops": 4 * dim * heads * pairs}
    if op == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"]
        # values in, codes and scales out; read again as values
        return {"bytes": 2 * n * 2 + 2 * (n + n // 8) + 2 * n * 2, "flops": 2 * n * 6}
    if op == "copy":
        page = case["kv_heads"] * segment_bytes(case["dim"], case["page"])
        return {"bytes": 2 * case["count"] * case["layers"] * page, "flops": 0}
    size = {"fp16": 2, "bf16": 2, "fp32": 4}[case["dtype"]]
    rows = case["batch"] * (case["drafts"] + 1 + (case["drafts"] if case["draft"] != "none" else 0))
    return {"bytes": rows * case["vocab"] * size, "flops": rows * case["vocab"] * 4}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    if case["op"] == "verify":
        return _exact_verify(prepare(case, seed))
    return None  # bytes


def _e2m1(code):
    """Sign, two exponent bits (bias 1), one fraction bit."""
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.pow(2.0, (e - 1).double()), m / 2)
    return torch.where(code & 8 > 0, -mag, mag)


def _e4m3(byte):
    """Sign, four exponent bits (bias 7), three fraction bits."""
    e, m = (byte >> 3) & 15, (byte & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, (e - 7).double()), m / 8 * 2.0 ** -6)
    return torch.where(byte & 128 > 0, -mag, mag)


def _token_values(seg, off, dim, page, of_v):
    """Values [tokens, dim] of the tokens at offsets `off` of segments [tokens, bytes], element by element."""
    d = torch.arange(dim, device=seg.device)[None]
    off = off[:, None]
    if of_v:
        wide = dim // 16  # elements of a token that lie together
        byte = page * dim // 2 + (off // 4) * 2 * dim + (d // wide) * 2 * wide + (off % 4) * (wide // 2) + d % wide // 2
        scale = page * dim + page * dim // 16 + (off // 4) * (dim // 4) + (d // 16) * 4 + off % 4
    else:
        byte = off * (dim // 2) + d // 2
        scale = page * dim + off * (dim // 16) + d // 16
    codes = seg.gather(1, byte).int()
    return _e2m1((codes >> (4 * (d % 2)).int()) & 15) * _e4m3(seg.gather(1, scale).int()) * SCALE


def _exact_attention(state):
    c = state["case"]
    page, dim, kvh, group = c["page"], c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    start, kv_len = state["q_start"].tolist(), state["kv_len"].tolist()
    pool = state["data"][0].view(-1, kvh, segment_bytes(dim, page))
    out = torch.zeros((start[-1], c["heads"], dim), dtype=torch.float64, device=DEV)
    lse = torch.full((start[-1], c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        t = torch.arange(kv_len[b], device=DEV)
        pages = state["table"][b].long()[t // page]
        for h in range(kvh):
            seg = pool[:, h][pages]
            k = _token_values(seg, t % page, dim, page, False)
            v = _token_values(seg, t % page, dim, page, True)
            q = state["q"][start[b]:start[b + 1], h * group:(h + 1) * group].double()
            n = q.shape[0]
            s = (q.reshape(-1, dim) @ k.T).view(n, group, -1) * dim ** -0.5
            pos = kv_len[b] - n + torch.arange(n, device=DEV)
            unseen = t[None] > pos[:, None]
            if c["window"]:
                unseen |= t[None] <= pos[:, None] - c["window"]
            s[unseen[:, None].expand_as(s)] = -math.inf
            z = torch.logsumexp(s, dim=2)
            p = torch.exp(s - torch.where(z.isinf(), 0.0, z)[..., None])
            out[start[b]:start[b + 1], h * group:(h + 1) * group] = (p.flatten(0, 1) @ v).view(n, group, dim)
            lse[start[b]:start[b + 1], h * group:(h + 1) * group] = z
    return out, lse


def _exact_append(state):
    """What the cache then stands for: each block's scale is its largest magnitude over 6 and the tensor scale,
    the nearest E4M3 value; each element is the nearest E2M1 value times both scales."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def stand(x):
        b = x.double().unflatten(-1, (-1, 16))
        s = torch.clamp(b.abs().amax(-1, True) / 6 / SCALE, max=448.0)
        step = torch.pow(2.0, torch.floor(torch.log2(s.clamp(min=2.0 ** -6)))) / 8
        d = torch.round(s / step) * step * SCALE
        a = b.abs() / torch.where(d > 0, d, 1.0)
        mids = (grid[1:] + grid[:-1]) / 2
        lower = torch.bucketize(a, mids)               # ties below
        upper = torch.bucketize(a, mids, right=True)   # ties above
        code = torch.where(lower % 2 == 0, lower, upper)
        return (grid[code] * torch.sign(b) * d).flatten(-2)

    return stand(state["k"]), stand(state["v"])


def _exact_verify(state):
    """Sequence by sequence, place by place: accept a draft with probability min(1, p / q); the first that is not
    accepted is replaced by a draw from max(p - q, 0), and a block that is accepted whole is followed by a draw from p."""
    c = state["case"]
    n, temperature = c["drafts"], state["temperature"].tolist()
    tokens, counts = state["tokens"].tolist(), state["num_draft"].tolist()
    u_accept, u_sample = state["u_accept"].tolist(), state["u_sample"].tolist()
    out, logps, accepted = [], [], []
    for b in range(c["batch"]):
        t = temperature[b] or 1.0
        greedy = c["draft"] != "probs" and temperature[b] == 0

        def logs(x):
            x = x.double()
            return x.log() if c["draft"] == "probs" else x / t - torch.logsumexp(x / t, 0)

        given, logp, rest = [], [], None
        for i in range(counts[b]):
            d = tokens[b][i]
            lp = logs(state["target"][b, i])
            if greedy:
                good = int(state["target"][b, i].argmax()) == d
            elif state["draft"] is None:
                good = u_accept[b][i] < float(lp[d].exp())
                left = lp.exp()
                left[d] = 0
            else:
                lq = logs(state["draft"][b, i])
                good = u_accept[b][i] * float(lq[d].exp()) < float(lp[d].exp())
                left = torch.relu(lp.exp() - lq.exp())
            if not good:
                rest = lp.exp() if greedy or not float(left.sum()) > 0 else left
                break
            given.append(d)
            logp.append(float(lp[d]))
        accepted.append(len(given))
        lp = logs(state["target"][b, len(given)])
        rest = lp.exp() if rest is None else rest
        sums = torch.cumsum(rest, 0)
        at = int(torch.searchsorted(sums, sums[-1:] * u_sample[b], right=True))
        token = int(state["target"][b, len(given)].argmax()) if greedy else min(at, int(rest.nonzero()[-1]))
        logp.append(float(lp[token]))
        pad = n - len(given)
        out.append(given + [token] + [-1] * pad)
        logps.append(logp + [0.0] * pad)
    return (torch.tensor(out, dtype=torch.int32), torch.tensor(accepted, dtype=torch.int32),
            torch.tensor(logps, dtype=torch.float64))
