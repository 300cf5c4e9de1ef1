"""The work of a prompt's step: cases over the product in 8-bit floating point
with a scale for each block of 128, the attention of a chunk of new tokens over
the 4-bit paged cache, and the log-probabilities of given tokens, each in a
plain form written with elementary torch operations, and as calls of this
package.

Products. x [m, k] is quantized to E4M3 with one scale for each row and 128
columns, the least power of two that takes the largest magnitude to 448 or
below (1 for zeros); w [n, k] is held as E4M3 codes with one fp32 scale for
each 128 rows and 128 columns:
  y[m, n] = sum_k (code_x scale_x)[m, k] (code_w scale_w)[n, k].

Attention. Sequence b has kv_len[b] tokens in the cache and brings a chunk of
rows q_start[b] .. q_start[b + 1] - 1 with queries, keys and values; row i of
the chunk sees the cached tokens and the chunk's own up to i (with a window w
only the last w of them all). The cache (one byte buffer [pages, page_bytes])
holds in every page, for every kv head, one segment of four arrays,
  K codes   [page][D / 2]             byte j: elements 2j (low nibble), 2j + 1
  V codes   [page / 4][16][4][D / 32] 4 tokens interleaved per D / 16 elements
  K scales  [page][D / 16]            one E4M3 byte per 16 elements
  V scales  [page / 4][D / 16][4]
and a value is E2M1(code) * E4M3(block scale) * tensor scale.

Log-probabilities. With l = logits / temperature: l[token] - log sum exp l, the
entropy of softmax(l), how many tokens come before the given one (larger, or
equal with a lower index), and the first few tokens in that order.
"""

import math

import torch

own = False

DEV = "cuda"

# Sizes: a ~27B dense decoder (hidden size 5120, 40 query and 8 kv heads of
# 128, an output head of 151936 rows), its share under 4-way tensor
# parallelism, and prompts cut into chunks of up to 2048 rows.
HEADS, KV_HEADS, VOCAB = 40, 8, 151936


def listed():
    return [
        # one token through the attention's projection: the latency of a small call, the weights' bytes
        product("product 1 x 7168 x 5120", 1, 7168, 5120, "fp16"),
        # a verify block or 16 users through the down projection: the weights' bytes
        product("product 16 x 5120 x 17408", 16, 5120, 17408, "bf16"),
        # the end of a prompt on one rank of four, an output whose partial sums go to an all-reduce; ragged in every size
        product("product 777 x 1795 x 1296", 777, 1795, 1296, "bf16", out="fp32"),
        # a full chunk through gate_up: the matrix cores
        product("product 2048 x 34816 x 5120", 2048, 34816, 5120, "bf16"),
        # a short message after a short chat: latency
        chunk("chunk 1x5 after 300", 1, 5, 5, 300, 300, "fp16"),
        # a question about a long document, on one rank of four: few rows, a long cache
        chunk("chunk 1x60 after 100000", 1, 60, 60, 100000, 100000, "bf16", heads=10, kv_heads=2),
        # a full chunk of a long prompt
        chunk("chunk 1x2048 after 30000", 1, 2048, 2048, 30000, 30000, "fp16"),
        # a server's batch of messages, some the first of their chat, small pages
        chunk("chunk 24x1-700 after 0-9000", 24, 1, 700, 0, 9000, "bf16", page=16),
        # prompts from their beginning, wide heads, a sliding window
        chunk("chunk 3x900-2000 window 1024", 3, 900, 2000, 0, 0, "bf16", heads=24, kv_heads=4, dim=256, page=32,
              window=1024),
        # the token that was just sampled, with its alternatives
        logprob("logprob 1 x 151936 top 20", 1, VOCAB, "fp16", 20),
        # an odd vocabulary in 32 bits, scores alone, each row at its own temperature
        logprob("logprob 37 x 50021", 37, 50021, "fp32", 0, tempered=True),
        # a prompt's chunk, scored token by token
        logprob("logprob 2048 x 151936 top 5", 2048, VOCAB, "bf16", 5),
    ]


def product(name, rows, n, k, dtype, out=None):
    return {"name": name, "op": "product", "rows": rows, "n": n, "k": k, "dtype": dtype, "out": out or dtype}


def chunk(name, batch, fewest, most, shortest, longest, dtype, heads=HEADS, kv_heads=KV_HEADS, dim=128, page=64,
          window=0):
    return {"name": name, "op": "chunk", "batch": batch, "fewest": fewest, "most": most, "shortest": shortest,
            "longest": longest, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "window": window}


def logprob(name, rows, vocab, dtype, top, tempered=False):
    return {"name": name, "op": "logprob", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top,
            "tempered": tempered}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "chunk", "logprob"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "product":
        n, k = _log(rng, 16, 34816), 16 * _log(rng, 4, 1088)
        rows = _log(rng, 1, max(1, min(8192, 2048 * 34816 * 5120 // (n * k))))
        case = product("", rows, n, k, dtype, rng.choice([dtype, dtype, "fp32"]))
    elif op == "chunk":
        batch, kv_heads, group = _log(rng, 1, 32), _log(rng, 1, 8), rng.randint(1, 8)
        dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
        most = _log(rng, 1, max(1, 2048 // batch))
        pairs = 2048 * 30000 * 40 * 128 // (batch * most * kv_heads * group * dim)
        longest = rng.choice([0, _log(rng, 1, 500), *[_log(rng, 500, max(500, min(131072 // batch, pairs)))] * 2])
        longest = min(longest, pairs)
        case = chunk("", batch, rng.randint(1, most), most, min(longest, rng.choice([0, longest, longest // 3])),
                     longest, dtype, kv_heads * group, kv_heads, dim, page,
                     rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    else:
        case = logprob("", _log(rng, 1, 1500), _log(rng, 100, VOCAB), rng.choice(["fp16", "bf16", "fp32"]),
                       rng.choice([0, 1, 5, 20, 33]), rng.random() < 0.5)
    case.pop("name")
    return case


TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"product": _prepare_product, "chunk": _prepare_chunk, "logprob": _prepare_logprob}[case["op"]](case, gen)


def _prepare_product(case, gen):
    m, n, k = case["rows"], case["n"], case["k"]
    x = torch.randn((m, k), device=DEV, generator=gen)
    # activations have a few strong channels
    x = torch.where(torch.rand((k,), device=DEV, generator=gen) < 0.01, x * 12, x)
    w = torch.randn((n, k), device=DEV, generator=gen) * 0.02
    # a checkpoint's form: the largest magnitude of each 128 x 128 is code 448
    pad = torch.nn.functional.pad(w.abs(), (0, -k % 128, 0, -n % 128))
    scales = pad.view(pad.shape[0] // 128, 128, -1, 128).amax((1, 3)) / 448.0
    codes = (w / scales.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]).to(torch.float8_e4m3fn)
    return {"case": case, "x": x.to(TYPES[case["dtype"]]), "codes": codes, "scales": scales}


def _spread(count, lo, hi):
    """`count` numbers from lo to hi by golden-ratio steps (evenly over the logarithm where lo is above 0), the last
    of them hi."""
    share = [(0.618033988749895 * i) % 1.0 for i in range(count)]
    share[-1] = 1.0
    if lo == 0:
        return [int(s * hi) for s in share]
    return [int(round(math.exp(math.log(lo) + s * (math.log(hi) - math.log(lo))))) for s in share]


def _lengths(case):
    """Each sequence's new rows and cached tokens, known without asking the GPU."""
    rows = _spread(case["batch"], case["fewest"], case["most"])
    return rows, _spread(case["batch"], case["shortest"], case["longest"])[::-1]


def segment_bytes(dim, page):
    return page * dim + page * dim // 8


SCALE = 1 / 600.0  # a block maximum of 2.1 is code 6 times block scale 210


def _pool(gen, pages, page, kv_heads, dim):
    """Pages whose bytes are those of quantized normal values of deviation 1 (with the scale above)."""
    # 256 equally likely normal values scaled by 6 / 2.1 and rounded to a code
    level = (torch.arange(256, device=DEV, dtype=torch.float64) + 0.5) / 256
    x = torch.special.ndtri(level) * (6 / 2.1)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV, dtype=torch.float64)
    code = torch.bucketize(x.abs(), mids) + 8 * (x < 0)
    pair = torch.arange(65536, device=DEV)
    pair = (code[pair & 255] | (code[pair >> 8] << 4)).to(torch.uint8)
    data = torch.empty((pages, kv_heads, segment_bytes(dim, page)), dtype=torch.uint8, device=DEV)
    for p in range(0, pages, 4096):
        part = data[p:p + 4096]
        r = torch.randint(0, 65536, (part.shape[0], kv_heads, page * dim), device=DEV, generator=gen,
                          dtype=torch.int32)
        part[:, :, :page * dim] = pair[r]
        s = torch.randn((part.shape[0], kv_heads, page * dim // 8), device=DEV, generator=gen) * 0.4 + 2.1
        part[:, :, page * dim:] = (s.clamp(0.9, 4.0) * 100).to(torch.float8_e4m3fn).view(torch.uint8)
    return data.view(pages, -1)


def _prepare_chunk(case, gen):
    page, dim, kvh, heads = case["page"], case["dim"], case["kv_heads"], case["heads"]
    rows, kv = _lengths(case)
    held = [-(-n // page) for n in kv]
    pages = sum(held) + 3
    data = _pool(gen, pages, page, kvh, dim)
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((case["batch"], max(held)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    # queries, keys and values as the projection leaves them, side by side
    qkv = torch.randn((start[-1], (heads + 2 * kvh) * dim), device=DEV, generator=gen)
    qkv[:, :heads * dim] *= 1.5
    qkv = qkv.to(TYPES[case["dtype"]])
    return {"case": case, "data": data, "table": table,
            "q": qkv[:, :heads * dim].view(start[-1], heads, dim),
            "k": qkv[:, heads * dim:(heads + kvh) * dim].view(start[-1], kvh, dim),
            "v": qkv[:, (heads + kvh) * dim:].view(start[-1], kvh, dim),
            "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV),
            "q_start": torch.tensor(start, dtype=torch.int32, device=DEV), "max_rows": max(rows), "max_kv": max(kv)}


def _prepare_logprob(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    # logits with the long tail of a language model's: a few tokens carry most of the mass, some are ruled out
    x = torch.randn((rows, vocab), device=DEV, generator=gen) * 2.5
    lift = torch.randint(0, vocab, (rows, 6), device=DEV, generator=gen)
    x.scatter_add_(1, lift, torch.rand((rows, 6), device=DEV, generator=gen) * 12)
    x[:, torch.randint(0, vocab, (max(1, vocab // 500),), device=DEV, generator=gen)] = -math.inf
    # a prompt's tokens: mostly likely ones, now and then any; the first of a prompt has none
    tokens = lift[:, 0].clone()
    tokens[::3] = torch.randint(0, vocab, tokens[::3].shape, device=DEV, generator=gen)
    tokens[5::400] = -1
    temperature = torch.rand((rows,), device=DEV, generator=gen) + 0.4 if case["tempered"] else None
    return {"case": case, "logits": x.to(TYPES[case["dtype"]]), "tokens": tokens.to(torch.int32),
            "temperature": temperature}


# ------------------------------------------------------------------ one pass

def run(state):
    return {"product": _run_product, "chunk": _run_chunk, "logprob": _run_logprob}[state["case"]["op"]](state)


def _run_product(state):
    c = state["case"]
    if own:
        from quantized_weight_skinny_amd import prompt_api as qp
        if "weight" not in state:
            state["weight"] = qp.BlockWeight(state["codes"], state["scales"])
            state["workspace"] = qp.fp8_block_workspace(c["rows"], c["n"], c["k"])
        return qp.fp8_block_linear(state["x"], state["weight"], dtype=TYPES[c["out"]], workspace=state["workspace"])
    n, k = c["n"], c["k"]
    x = torch.nn.functional.pad(state["x"].float(), (0, -k % 128)).unflatten(1, (-1, 128))
    # the largest magnitude is f 2^e with f in [0.5, 1), and 448 is 0.875 2^9
    f, e = torch.frexp(x.abs().amax(2, True))
    e = torch.where(f > 0, torch.where(f <= 0.875, e - 9, e - 8).clamp(min=-126), 0)
    scale = ((e + 127) << 23).view(torch.float32)  # 2^e to the bit: many quotients are ties of the rounding
    x = ((x / scale).to(torch.float8_e4m3fn).float() * scale).flatten(1)[:, :k]
    w = state["codes"].float() * state["scales"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return (x @ w.T).to(TYPES[c["out"]])


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _cached(state, b, length):
    """Keys and values [kv heads, tokens, dim] of sequence b's cached tokens, in float32."""
    c = state["case"]
    page, dim, kvh = c["page"], c["dim"], c["kv_heads"]
    held = -(-length // page)
    seg = state["data"][state["table"][b, :held].long()].view(held, kvh, segment_bytes(dim, page))
    half = page * dim // 2
    kc = seg[..., :half].reshape(held, kvh, page, dim // 2)
    vc = seg[..., half:2 * half].reshape(held, kvh, page // 4, 16, 4, dim // 32).transpose(3, 4)
    ks = seg[..., 2 * half:2 * half + half // 8].reshape(held, kvh, page, dim // 16)
    vs = seg[..., 2 * half + half // 8:].reshape(held, kvh, page // 4, dim // 16, 4).transpose(3, 4)
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=seg.device)
    both = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), dim=1)  # byte -> its two values

    def values(codes, scales):
        x = both[codes.reshape(held, kvh, page, dim // 2).to(torch.int32)].flatten(-2)
        s = scales.reshape(held, kvh, page, dim // 16).view(torch.float8_e4m3fn).float()
        x = (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * SCALE
        return x.transpose(0, 1).flatten(1, 2)[:, :length]

    return values(kc, ks), values(vc, vs)


def _run_chunk(state):
    c = state["case"]
    if own:
        from quantized_weight_skinny_amd import decode_api as qd
        from quantized_weight_skinny_amd import prompt_api as qp
        if "cache" not in state:
            state["cache"] = qd.KV4Cache.wrap(state["data"][None], c["page"], c["kv_heads"], c["dim"], SCALE, SCALE)
            state["workspace"] = qp.kv4_chunk_workspace(state["cache"], state["q"].shape[0], c["heads"], c["batch"],
                                                        state["max_rows"], state["max_kv"])
        return qp.kv4_chunk_attention(state["q"], state["k"], state["v"], state["cache"], state["table"],
                                      state["kv_len"], q_start=state["q_start"], max_q_len=state["max_rows"],
                                      max_kv_len=state["max_kv"], window=c["window"], workspace=state["workspace"])
    kvh, dim, group = c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    outs, lses, at = [], [], 0
    for b, (n, cached) in enumerate(zip(*_lengths(c))):
        ck, cv = _cached(state, b, cached)
        k = torch.cat((ck, state["k"][at:at + n].float().transpose(0, 1)), 1)
        v = torch.cat((cv, state["v"][at:at + n].float().transpose(0, 1)), 1)
        # [kv head, rows * group, dim]
        q = state["q"][at:at + n].float().view(n, kvh, group, dim).transpose(0, 1).reshape(kvh, n * group, dim)
        s = torch.bmm(q, k.transpose(1, 2).contiguous()).view(kvh, n, group, cached + n) / math.sqrt(dim)
        t = torch.arange(cached + n, device=s.device)
        pos = cached + torch.arange(n, device=s.device)[:, None]
        unseen = t > pos
        if c["window"]:
            unseen |= t <= pos - c["window"]
        s.masked_fill_(unseen[:, None], -math.inf)
        top = s.amax(-1, True)
        p = torch.exp_(s.sub_(top))
        z = p.sum(-1, True)
        o = torch.bmm(p.view(kvh, n * group, -1), v.contiguous()).view(kvh, n, group, dim) / z
        outs.append(o.transpose(0, 1).reshape(n, c["heads"], dim))
        lses.append((top + torch.log(z))[..., 0].transpose(0, 1).reshape(n, c["heads"]))
        at += n
    return torch.cat(outs).to(state["q"].dtype), torch.cat(lses)


def _run_logprob(state):
    c = state["case"]
    if own:
        from quantized_weight_skinny_amd import prompt_api as qp
        if "workspace" not in state:
            state["workspace"] = qp.token_logprobs_workspace(c["rows"], c["vocab"], c["top"])
        return qp.token_logprobs(state["logits"], state["tokens"], top=c["top"], temperature=state["temperature"],
                                 workspace=state["workspace"])
    x, given = state["logits"].float(), state["tokens"].long()
    t = state["temperature"][:, None] if state["temperature"] is not None else 1.0
    index = torch.arange(c["vocab"], device=x.device)
    top = x.amax(1, True)
    e = torch.exp((x - top) / t)
    z = e.sum(1, True)
    log_z = torch.log(z)
    # log p = (x - top) / t - log z
    at = given.clamp(min=0)[:, None]
    chosen = x.gather(1, at)
    logp = torch.where(given >= 0, ((chosen - top) / t - log_z)[:, 0], 0.0)
    entropy = (log_z - torch.where(e > 0, e * ((x - top) / t), 0.0).sum(1, True) / z)[:, 0]
    rank = ((x > chosen) | ((x == chosen) & (index < at))).sum(1)
    rank = torch.where(given >= 0, rank, -1).to(torch.int32)
    # larger first, then the lower index: one whole number that orders both
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * 2 ** 25 - index
    best = torch.topk(order, c["top"], dim=1).indices
    best_logp = (x.gather(1, best) - top) / t - log_z
    return logp, entropy, rank, best.to(torch.int32), best_logp


# ------------------------------------------------------------------ what a pass cannot do without

SIZES = {"fp16": 2, "bf16": 2, "fp32": 4}


def work(case):
    if case["op"] == "product":
        m, n, k = case["rows"], case["n"], case["k"]
        blocks = -(-n // 128) * -(-k // 128)
        return {"bytes": m * k * SIZES[case["dtype"]] + n * k + 4 * blocks + m * n * SIZES[case["out"]],
                "flops": 2 * m * n * k}
    if case["op"] == "chunk":
        rows, kv = _lengths(case)
        dim, kvh, heads, w = case["dim"], case["kv_heads"], case["heads"], case["window"]
        tokens = pairs = 0
        for r, n in zip(rows, kv):
            tokens += min(n, w - 1) if w else n
            pairs += sum(min(n + i + 1, w) if w else n + i + 1 for i in range(r))
        io = sum(rows) * ((2 * heads + 2 * kvh) * dim * 2 + heads * 4)
        return {"bytes": tokens * kvh * (dim + dim // 8) + io, "flops": 4 * dim * heads * pairs}
    elements = case["rows"] * case["vocab"]
    return {"bytes": elements * SIZES[case["dtype"]] + case["rows"] * (16 + 8 * case["top"]), "flops": 4 * elements}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return {"product": _exact_product, "chunk": _exact_chunk, "logprob": _exact_logprob}[case["op"]](
        prepare(case, seed))


def _e4m3(byte):
    """Sign, four exponent bits (bias 7), three fraction bits."""
    e, m = (byte >> 3) & 15, (byte & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, (e - 7).double()), m / 8 * 2.0 ** -6)
    return torch.where(byte & 128 > 0, -mag, mag)


def _e2m1(code):
    """Sign, two exponent bits (bias 1), one fraction bit."""
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.pow(2.0, (e - 1).double()), m / 2)
    return torch.where(code & 8 > 0, -mag, mag)


def _power(x):
    """The largest power of two not above x > 0: the fraction bits struck out."""
    return (x.view(torch.int64) & ~((1 << 52) - 1)).view(torch.float64)


def _exact_product(state):
    """Block column by block column: the quantized values of x from the grid's spacing, the products' sum."""
    c = state["case"]
    codes = state["codes"].view(torch.uint8)
    y = torch.zeros((c["rows"], c["n"]), dtype=torch.float64, device=DEV)
    row_block = torch.arange(c["n"], device=DEV) // 128
    for j, k0 in enumerate(range(0, c["k"], 128)):
        x = state["x"][:, k0:k0 + 128].double()
        big = x.abs().amax(1, True)
        scale = _power(big.clamp(min=1e-300)) / 256  # 448 is 1.75 * 256
        scale = torch.where(big > 448 * scale, scale * 2, scale)
        scale = torch.where(big > 0, scale.clamp(min=2.0 ** -126), 1.0)
        a = x / scale
        # E4M3 has three fraction bits down to 2^-6 and steps of 2^-9 below; round() takes ties to even
        step = _power(a.abs().clamp(min=2.0 ** -6)) / 8
        x = torch.round(a / step) * step * scale
        w = _e4m3(codes[:, k0:k0 + 128].int()) * state["scales"].double()[row_block, j][:, None]
        y += x @ w.T
    return y


def _exact_chunk(state):
    """Row by row of the group, head by head: weights exp(s - lse), their products with the values."""
    c = state["case"]
    page, dim, kvh, group = c["page"], c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    start, kv_len = state["q_start"].tolist(), state["kv_len"].tolist()
    pool = state["data"].view(-1, kvh, segment_bytes(dim, page))
    out = torch.empty((start[-1], c["heads"], dim), dtype=torch.float64, device=DEV)
    lse = torch.empty((start[-1], c["heads"]), dtype=torch.float64, device=DEV)
    d = torch.arange(dim, device=DEV)[None]
    wide = dim // 16
    for b in range(c["batch"]):
        mine = slice(start[b], start[b + 1])
        n = start[b + 1] - start[b]
        t = torch.arange(kv_len[b], device=DEV)
        pages, off = state["table"][b].long()[t // page], (t % page)[:, None]
        k_byte, k_scale = off * (dim // 2) + d // 2, page * dim + off * wide + d // 16
        v_byte = page * dim // 2 + (off // 4) * 2 * dim + (d // wide) * 2 * wide + (off % 4) * (wide // 2) + d % wide // 2
        v_scale = page * dim + page * wide + (off // 4) * (dim // 4) + (d // 16) * 4 + off % 4
        pos = kv_len[b] + torch.arange(n, device=DEV)[:, None]
        place = torch.arange(kv_len[b] + n, device=DEV)[None]
        seen = place <= pos
        if c["window"]:
            seen &= place > pos - c["window"]
        for h in range(kvh):
            seg = pool[:, h][pages]
            old = []
            for byte, scale in ((k_byte, k_scale), (v_byte, v_scale)):
                code = (seg.gather(1, byte).int() >> (4 * (d % 2)).int()) & 15
                old.append(_e2m1(code) * _e4m3(seg.gather(1, scale).int()) * SCALE)
            k = torch.cat((old[0], state["k"][mine, h].double()))
            v = torch.cat((old[1], state["v"][mine, h].double()))
            for g in range(h * group, (h + 1) * group):
                s = (state["q"][mine, g].double() @ k.T) * dim ** -0.5
                s = torch.where(seen, s, -math.inf)
                z = torch.logsumexp(s, 1)
                out[mine, g] = torch.exp(s - z[:, None]) @ v
                lse[mine, g] = z
    return out, lse


def _exact_logprob(state):
    """Row by row, from a stable sort."""
    c = state["case"]
    logp, entropy, rank, best, best_logp = [], [], [], [], []
    tokens = state["tokens"].tolist()
    for r in range(c["rows"]):
        x = state["logits"][r].double()
        t = float(state["temperature"][r]) if state["temperature"] is not None else 1.0
        lp = x / t - torch.logsumexp(x / t, 0)
        p = lp.exp()
        entropy.append(-(p[p > 0] * lp[p > 0]).sum())
        order = torch.sort(x, descending=True, stable=True).indices
        best.append(order[:c["top"]])
        best_logp.append(lp[best[-1]])
        g = tokens[r]
        logp.append(lp[g] if g >= 0 else lp.new_zeros(()))
        rank.append((order == g).to(torch.uint8).argmax() if g >= 0 else torch.full((), -1, device=x.device))
    return (torch.stack(logp), torch.stack(entropy), torch.stack(rank).to(torch.int32),
            torch.stack(best).to(torch.int32), torch.stack(best_logp))
