"""Torch plumbing over the entry points of ``include/qpn_prompt.h``: a prompt's
step, where ``torch_api`` and ``decode_api`` serve steps of up to 16 rows.
Device memory and the current stream only; every step runs in the library's
HIP kernels.

    w = BlockWeight(codes, scales)                    # E4M3 and a scale for each 128 x 128, as they are
    y = fp8_block_linear(x, w)                        # any number of rows
    out, lse = kv4_chunk_attention(q, k, v, cache, table, kv_len, layer=layer)
    logprobs, entropy, rank, top, top_logprobs = token_logprobs(logits, tokens, top=5)
"""

import functools

import torch

from .decode_api import (DTYPES, HALVES, INT32_MAX, _exactly, _on_device, _out, _rows, _sizes, _stream,  # noqa: F401
                         _workspace)
from .decode import qpn_kv4_cache
from .prompt import (
    QPN_DT_E4M3,
    qpn_fp8_block_gemm,
    qpn_fp8_block_gemm_args,
    qpn_fp8_block_quantize,
    qpn_fp8_block_workspace_bytes,
    qpn_kv4_chunk_args,
    qpn_kv4_chunk_attention,
    qpn_kv4_chunk_workspace_bytes,
    qpn_logprobs_args,
    qpn_token_logprobs,
    qpn_token_logprobs_workspace_bytes,
)

BLOCK = 128  # elements under one scale
CODES = (torch.uint8, torch.float8_e4m3fn)
FLOATS = tuple(DTYPES)


def _blocks(n):
    return -(-n // BLOCK)


def _matrix(t, name, device, dtypes, shape=None):
    """A tensor [rows, columns] with contiguous rows any distance apart; returns
    its address and that distance."""
    _on_device(t, name, device)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, not {t.dtype}")
    sizes = t.shape
    if len(sizes) != 2 or (shape is not None and sizes != shape):
        raise ValueError(f"{name} must have shape {shape or ('rows', 'columns')}, not {tuple(sizes)}")
    rows, columns = sizes
    stride, step = t.stride()
    if step != 1 and columns > 1 and rows:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), stride if rows > 1 and columns > 0 else columns


def _block_scales(t, shape, name, device):
    """fp32 scales of this shape, any strides; returns address and strides."""
    _on_device(t, name, device)
    if t.dtype is not torch.float32 or t.shape != shape:
        raise ValueError(f"{name} must be a torch.float32 tensor of shape {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else 1, t.stride(1) if shape[1] > 1 else 1


def _quantize(x, block_rows, codes, scales):
    dev = x.device if isinstance(x, torch.Tensor) else None
    xp, stride = _matrix(x, "x", dev, FLOATS)
    rows, k = x.shape
    if codes is None:
        codes = torch.empty((rows, -(-k // 16) * 16), dtype=torch.float8_e4m3fn, device=dev)[:, :k]
    cp, code_stride = _matrix(codes, "codes", dev, CODES, (rows, k))
    shape = (-(-rows // block_rows), _blocks(k))
    if scales is None:
        # a block's scales of neighbouring rows lie together, as the product reads them
        scales = torch.empty(shape[::-1], dtype=torch.float32, device=dev).t()
    sp, sr, sb = _block_scales(scales, shape, "scales", dev)
    qpn_fp8_block_quantize(xp, DTYPES[x.dtype], rows, k, stride, block_rows, cp, code_stride, sp, sr, sb, _stream(dev))
    return codes, scales


def quantize_fp8_rows(x, codes=None, scales=None):
    """(codes [rows, k] float8_e4m3fn, scales fp32 [rows, ceil(k / 128)]) of x
    [rows, k] fp16, bf16 or fp32: activations, a scale for each row and 128
    columns. A scale is the least power of two that takes the block's largest
    magnitude to 448 or below (1 for zeros), so every code is the E4M3 value
    nearest to x / scale; inf and NaN get the NaN code. codes may also be uint8;
    the rows of all three any distance apart, scales with any strides."""
    return _quantize(x, 1, codes, scales)


def quantize_fp8_blocks(w, codes=None, scales=None):
    """The same for a weight w [n, k], with a scale for each 128 rows and 128
    columns: scales fp32 [ceil(n / 128), ceil(k / 128)]."""
    return _quantize(w, BLOCK, codes, scales)


class BlockWeight:
    """A weight [n, k] as E4M3 codes (float8_e4m3fn or uint8; rows a multiple of
    16 bytes apart and 16-byte aligned, k a multiple of 16) and fp32 scales
    [ceil(n / 128), ceil(k / 128)], any strides. It keeps both as they are:
    nothing is copied or laid out anew."""

    _FIXED = frozenset(("codes", "scales", "device", "n", "k", "_fields"))

    def __init__(self, codes, scales):
        _on_device(codes, "codes")
        dev = codes.device
        cp, stride = _matrix(codes, "codes", dev, CODES)
        n, k = codes.shape
        if k % 16 or stride % 16 or cp % 16:
            raise ValueError(f"codes need a number of columns ({k}) and of bytes from row to row ({stride}) that 16 "
                             "divides, and 16-byte alignment")
        sp, sr, sb = _block_scales(scales, (_blocks(n), _blocks(k)), "scales", dev)
        self.codes, self.scales, self.device, self.n, self.k = codes, scales, dev, n, k
        self._fields = (cp, sp, stride, sr, sb)

    def __setattr__(self, name, value):
        """Calls take the tensors' addresses and strides from here, so neither tensor
        is replaced: their contents may change, other tensors are another weight."""
        if name in self._FIXED and name in self.__dict__:
            raise AttributeError(f"a weight's {name} does not change: make another weight of the other tensors")
        super().__setattr__(name, value)

    @classmethod
    def quantize(cls, w):
        """From w [n, k] fp16, bf16 or fp32 (see quantize_fp8_blocks)."""
        return cls(*quantize_fp8_blocks(w))


_fp8_workspace_bytes = functools.lru_cache(maxsize=256)(qpn_fp8_block_workspace_bytes)


def fp8_block_workspace(m, n, k, device="cuda"):
    """A workspace for fp8_block_linear and fp8_block_gemm with these sizes
    (None when none is needed). It carries nothing from call to call, but two
    calls that may run at once need one each."""
    _sizes(m=m, n=n, k=k)
    need = _fp8_workspace_bytes(m, n, k)
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def _product(x, scales, w, dtype, out, workspace):
    dev = w.device
    n, k = w.n, w.k
    coded = scales is not None
    xp, x_stride = _matrix(x, "codes" if coded else "x", dev, CODES if coded else FLOATS)
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError(f"{'codes' if coded else 'x'} must have shape (rows, {k}), not {tuple(x.shape)}")
    if coded:
        if x_stride % 16 or xp % 16:
            raise ValueError("codes must be 16-byte aligned, with a number of bytes from row to row that 16 divides")
        sp, sr, sb = _block_scales(scales, (m, _blocks(k)), "scales", dev)
    else:
        sp, sr, sb = None, 0, 0
    if out is None:
        out = torch.empty(m, n, dtype=dtype, device=dev)
        yp, y_stride = out.data_ptr(), n
    else:
        yp, y_stride = _matrix(out, "out", dev, (dtype,), (m, n))
    cp, wp, w_stride, wr, wb = w._fields
    a = qpn_fp8_block_gemm_args(xp, sp, cp, wp, yp, x_stride, sr, sb, w_stride, wr, wb, y_stride, m, n, k,
                                QPN_DT_E4M3 if coded else DTYPES[x.dtype], DTYPES[dtype])
    workspace, ws, nbytes = _workspace(_fp8_workspace_bytes(m, n, k), workspace, dev)
    qpn_fp8_block_gemm(a, ws, nbytes, _stream(dev))
    return out


def _out_dtype(dtype, out, default):
    if dtype is None:
        dtype = out.dtype if isinstance(out, torch.Tensor) else default
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be one of {', '.join(str(d) for d in DTYPES)}, not {dtype}")
    return dtype


def fp8_block_linear(x, w, dtype=None, out=None, workspace=None):
    """y [rows, n] = x @ w.T for x [rows, k] fp16, bf16 or fp32 and a
    BlockWeight: x is quantized as by quantize_fp8_rows, the blocks' scaled sums
    are added in fp32, y is rounded once to dtype (default: x's). For fp32
    results a block's own sum is fp32 too; for 16 bits it keeps its products to
    about 2^-11 of the largest (random blocks: 1.4e-5 of a result). Rows of x
    and out any distance apart."""
    _on_device(x, "x")
    return _product(x, None, w, _out_dtype(dtype, out, x.dtype), out, workspace)


def fp8_block_gemm(codes, scales, w, dtype=None, out=None, workspace=None):
    """The same from codes [rows, k] and scales fp32 [rows, ceil(k / 128)] that
    are there already (any scales; codes as a BlockWeight's). dtype defaults to
    bf16."""
    return _product(codes, scales, w, _out_dtype(dtype, out, torch.bfloat16), out, workspace)


@functools.lru_cache(maxsize=256)
def _chunk_workspace_bytes(page_size, kv_heads, head_dim, rows, heads, batch, max_q_len, max_kv_len):
    c = qpn_kv4_cache(None, 0, 1, page_size, kv_heads, head_dim, 1.0, 1.0)
    a = qpn_kv4_chunk_args()
    a.heads, a.batch, a.rows, a.max_q_len, a.max_kv_len = heads, batch, rows, max_q_len, max_kv_len
    return qpn_kv4_chunk_workspace_bytes(c, a)


def kv4_chunk_workspace(cache, rows, heads, batch, max_q_len, max_kv_len):
    """A workspace for kv4_chunk_attention with these sizes (None when none is
    needed). It carries nothing from call to call, but two calls that may run
    at once need one each."""
    _sizes(rows=rows, heads=heads, batch=batch, max_q_len=max_q_len, max_kv_len=max_kv_len)
    need = _chunk_workspace_bytes(cache.page_size, cache.kv_heads, cache.head_dim, rows, heads, batch, max_q_len,
                                  max_kv_len)
    return torch.empty(need, dtype=torch.uint8, device=cache.device) if need else None


def kv4_chunk_attention(q, k, v, cache, table, kv_len, q_start=None, max_q_len=None, max_kv_len=None, layer=0,
                        scale=None, window=0, out=None, lse=None, workspace=None):
    """(out, lse): attention of each sequence's new tokens over its cached
    tokens and themselves, causal.

    q [rows, heads, head_dim], k and v [rows, kv_heads, head_dim], fp16 or bf16
    (any strides with a contiguous last dimension: slices of a fused
    projection's output will do). The new tokens' keys and values are read from
    k and v as they are, so they may be appended before or after; table int32
    [batch, pages a sequence at most] and kv_len int32 [batch] are of the tokens
    that were cached before (table may have no columns). q_start int32 [batch +
    1] from 0 to rows, with max_q_len the longest (None: rows / batch rows
    each); max_kv_len bounds the lengths (default: what the table can hold).
    window > 0: a row sees the last `window` tokens up to its own. out [rows,
    heads, head_dim] like q, lse fp32 [rows, heads]. What is rounded to fewer bits is in
    qpn_prompt.h; sums are fp32."""
    dev = cache.device
    dim, kv_heads = cache.head_dim, cache.kv_heads
    _on_device(q, "q", dev)
    if q.dim() != 3:
        raise ValueError(f"q must have shape (rows, heads, {dim}), not {tuple(q.shape)}")
    rows, heads, _ = q.shape
    qp, qt, qh = _rows(q, (rows, heads, dim), "q", dev, HALVES)
    kp, kt, kh = _rows(k, (rows, kv_heads, dim), "k", dev, (q.dtype,))
    vp, vt, vh = _rows(v, (rows, kv_heads, dim), "v", dev, (q.dtype,))
    if heads == 0 or heads % kv_heads:
        raise ValueError(f"q's {heads} heads must be a multiple of the cache's {kv_heads}")
    _on_device(table, "table", dev)
    if table.dtype is not torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be an int32 [batch, pages] tensor with contiguous rows")
    batch, pages = table.shape
    lp = _exactly(kv_len, torch.int32, (batch,), "kv_len", dev)
    if q_start is not None:
        sp = _exactly(q_start, torch.int32, (batch + 1,), "q_start", dev)
        if max_q_len is None:
            raise ValueError("q_start needs max_q_len, the longest sequence's rows")
    else:
        sp = None
        each = rows // batch if batch else 0
        if each * batch != rows or (max_q_len is not None and max_q_len != each):
            raise ValueError(f"{rows} rows are not {batch} sequences of as many: give q_start and max_q_len")
        max_q_len = each
    if max_kv_len is None:
        max_kv_len = pages * cache.page_size
    if not (0 <= window <= INT32_MAX and 0 <= max_q_len <= INT32_MAX and 0 <= max_kv_len <= INT32_MAX):
        raise ValueError(f"window {window}, max_q_len {max_q_len} and max_kv_len {max_kv_len} must be 0 .. {INT32_MAX}")
    if max_kv_len > pages * cache.page_size:   # (a slice's rows may lie further apart than they are long)
        raise ValueError(f"max_kv_len {max_kv_len} is more than a table row's {pages} pages of {cache.page_size} hold")
    out = _out(out, q.dtype, (rows, heads, dim), "out", dev)
    lse = _out(lse, torch.float32, (rows, heads), "lse", dev)
    a = qpn_kv4_chunk_args(qp, kp, vp, out.data_ptr(), lse.data_ptr(), table.data_ptr(), lp, sp, qt, qh, kt, kh, vt, vh,
                           table.stride(0) if batch > 1 and pages > 0 else pages, DTYPES[q.dtype], layer, heads, batch,
                           rows, max_q_len, max_kv_len, window, dim ** -0.5 if scale is None else scale, 0)
    workspace, wp, nbytes = _workspace(
        _chunk_workspace_bytes(cache.page_size, kv_heads, dim, rows, heads, batch, max_q_len, max_kv_len), workspace,
        dev)
    qpn_kv4_chunk_attention(cache.desc(layer), a, wp, nbytes, _stream(dev))
    return out, lse


_logprobs_workspace_bytes = functools.lru_cache(maxsize=256)(qpn_token_logprobs_workspace_bytes)


def token_logprobs_workspace(rows, vocab, top=0, device="cuda"):
    """A workspace for token_logprobs with these sizes. It carries nothing from
    call to call, but two calls that may run at once need one each."""
    _sizes(rows=rows, vocab=vocab, top=top)
    need = _logprobs_workspace_bytes(rows, vocab, top)
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def token_logprobs(logits, tokens, top=0, temperature=None, logprobs=None, entropy=None, rank=None, top_tokens=None,
                   top_logprobs=None, workspace=None):
    """(logprobs fp32 [rows], entropy fp32 [rows], rank int32 [rows], top_tokens
    int32 [rows, top], top_logprobs fp32 [rows, top]) of logits [rows, vocab]
    (fp16, bf16 or fp32, rows any distance apart) at tokens int32 [rows].

    With p = softmax(logits / temperature) (fp32 [rows]; None, 0 or below: 1):
    log p of the given token (0 for one outside the vocabulary), the entropy of
    p, how many tokens come before the given one (-1), and the first `top` (0
    to 64) tokens. Larger logits come first, equal ones in the order of their
    index; NaN counts as -inf."""
    xp, stride = _matrix(logits, "logits", None, FLOATS)
    dev = logits.device
    rows, vocab = logits.shape
    if not (0 <= top <= INT32_MAX and rows <= INT32_MAX and vocab <= INT32_MAX):
        raise ValueError(f"{rows} rows, a vocabulary of {vocab} and top {top} must be 0 .. {INT32_MAX}")
    tp = _exactly(tokens, torch.int32, (rows,), "tokens", dev)
    fp = None if temperature is None else _exactly(temperature, torch.float32, (rows,), "temperature", dev)
    logprobs = _out(logprobs, torch.float32, (rows,), "logprobs", dev)
    entropy = _out(entropy, torch.float32, (rows,), "entropy", dev)
    rank = _out(rank, torch.int32, (rows,), "rank", dev)
    top_tokens = _out(top_tokens, torch.int32, (rows, top), "top_tokens", dev)
    top_logprobs = _out(top_logprobs, torch.float32, (rows, top), "top_logprobs", dev)
    a = qpn_logprobs_args(xp, tp, fp, logprobs.data_ptr(), entropy.data_ptr(), rank.data_ptr(), top_tokens.data_ptr(),
                          top_logprobs.data_ptr(), stride, DTYPES[logits.dtype], rows, vocab, top)
    workspace, wp, nbytes = _workspace(_logprobs_workspace_bytes(rows, vocab, top), workspace, dev)
    qpn_token_logprobs(a, wp, nbytes, _stream(dev))
    return logprobs, entropy, rank, top_tokens, top_logprobs
