"""Torch plumbing over the entry points of ``include/qpn_decode.h``: what a
verify step does between and after its weight products. Device memory and the
current stream only; every step runs in the library's HIP kernels.

    cache = KV4Cache(pages, 64, kv_heads=8, head_dim=128, layers=64)
    kv4_append(cache, k, v, slots, layer)          # the step's keys and values, quantized into pages
    out, lse = kv4_attention(q, cache, table, kv_len, layer=layer)
    tokens, accepted, logprobs = verify_drafts(logits, drafts, u_accept, u_sample)

``PagePool`` keeps the books of a cache's pages on the host: allocation, forks
that share pages, copies on write, release and compaction.
"""

import functools
import math

import torch

from .decode import (
    QPN_DT_BF16,
    QPN_DT_F16,
    QPN_DT_F32,
    qpn_kv4_append,
    qpn_kv4_attention,
    qpn_kv4_attention_args,
    qpn_kv4_attention_workspace_bytes,
    qpn_kv4_cache,
    qpn_kv4_copy_pages,
    qpn_kv4_page_bytes,
    qpn_kv4_read,
    qpn_verify,
    qpn_verify_args,
    qpn_verify_workspace_bytes,
)
from .page_pool import NotWritten, OutOfPages, PagePool  # noqa: F401  (part of this module's interface)

DTYPES = {torch.float16: QPN_DT_F16, torch.bfloat16: QPN_DT_BF16, torch.float32: QPN_DT_F32}
HALVES = (torch.float16, torch.bfloat16)
INT32_MAX = 2**31 - 1  # ctypes cuts a larger number to its low 32 bits without a word


def _sizes(**sizes):
    for name, x in sizes.items():
        if not 0 <= x <= INT32_MAX:
            raise ValueError(f"{name} must be 0 .. {INT32_MAX}, not {x}")


# A verify step makes these calls once a layer, so what Python adds to each
# counts: checks compare plain attributes, the descriptors of a cache are built
# once, and the current stream is taken as the raw handle that torch keeps.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _stream(device):
    """The device's current stream. A kernel runs on the current device, so that
    must be the tensors'."""
    if _current_device() != device.index:
        raise ValueError(f"the tensors are on {device}, which is not the current device: call under torch.cuda.device")
    return _raw_stream(device.index)


def _on_device(t, name, device=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _exactly(t, dtype, shape, name, device):
    """A contiguous tensor of this type and shape; returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.device == device):
        _on_device(t, name, device)
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, not {t.dtype} "
                         f"{tuple(t.shape)}")
    return t.data_ptr()


def _rows(t, shape, name, device, dtypes):
    """A tensor of this shape whose last dimension is contiguous, other strides
    free; returns its address and those strides."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.device == device):
        _on_device(t, name, device)
        if t.dtype not in dtypes:
            raise ValueError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, not {t.dtype}")
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    st = t.stride()
    if st[2] != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), st[0], st[1]


def _out(t, dtype, shape, name, device):
    """The caller's output, checked, or a new one."""
    if t is None:
        return torch.empty(*shape, dtype=dtype, device=device)  # 0.7 us less than one tuple
    _exactly(t, dtype, shape, name, device)
    return t


def _workspace(need, workspace, device):
    """(tensor, address, bytes) of the caller's workspace where it is large
    enough, or of a new one."""
    if not need:
        return None, None, 0
    if workspace is not None:
        _on_device(workspace, "workspace", device)
        if not workspace.is_contiguous():   # its elements would not be its bytes
            raise ValueError("workspace must be contiguous")
        have = workspace.numel() * workspace.element_size()
        if have >= need:
            return workspace, workspace.data_ptr(), have
    workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, workspace.data_ptr(), need


class KV4Cache:
    """Pages of keys and values in 4 bits: ``data`` uint8 [layers, pages,
    page_bytes] (the layout is in qpn_decode.h). ``k_scale`` and ``v_scale``
    are tensor scales, one number or one a layer: the largest magnitude a
    block holds exactly is 2688 times the scale, the finest step of a block's
    scale 2^-9 of it, so amax / 2688 of typical keys (values) is the choice."""

    _FIXED = frozenset(("data", "device", "layers", "pages", "page_size", "kv_heads", "head_dim", "k_scale", "v_scale"))

    def __init__(self, pages, page_size, kv_heads, head_dim, layers=1, k_scale=1.0 / 128, v_scale=1.0 / 128,
                 device="cuda"):
        _sizes(page_size=page_size, kv_heads=kv_heads, head_dim=head_dim)
        nbytes = qpn_kv4_page_bytes(page_size, kv_heads, head_dim)
        if nbytes == 0:
            raise ValueError(f"a page of {page_size} tokens, {kv_heads} heads of {head_dim} is not supported: 16, 32, "
                             "64, 128 or 256 tokens, 1 to 1024 heads of 64, 128 or 256")
        data = torch.zeros((layers, pages, nbytes), dtype=torch.uint8, device=device)
        self._init(data, page_size, kv_heads, head_dim, k_scale, v_scale)

    @classmethod
    def wrap(cls, data, page_size, kv_heads, head_dim, k_scale=1.0 / 128, v_scale=1.0 / 128):
        """A cache over an existing buffer, uint8 [layers, pages, page_bytes]."""
        self = cls.__new__(cls)
        _sizes(page_size=page_size, kv_heads=kv_heads, head_dim=head_dim)
        _on_device(data, "data")
        nbytes = qpn_kv4_page_bytes(page_size, kv_heads, head_dim)
        if data.dtype != torch.uint8 or data.dim() != 3 or not data.is_contiguous() or data.shape[2] != nbytes or not nbytes:
            raise ValueError(f"data must be a contiguous uint8 [layers, pages, {nbytes}] tensor")
        self._init(data, page_size, kv_heads, head_dim, k_scale, v_scale)
        return self

    def _init(self, data, page_size, kv_heads, head_dim, k_scale, v_scale):
        k_scale, v_scale = (
            [float(s)] * data.shape[0] if isinstance(s, (int, float)) else [float(x) for x in s]
            for s in (k_scale, v_scale))
        if len(k_scale) != data.shape[0] or len(v_scale) != data.shape[0]:
            raise ValueError("k_scale and v_scale take one number, or one a layer")
        if not all(math.isfinite(s) and s > 0 for s in k_scale + v_scale):
            raise ValueError("tensor scales must be finite and above 0")
        self.data, self.device = data, data.device
        self.layers, self.pages = data.shape[0], data.shape[1]
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        self.k_scale, self.v_scale = tuple(k_scale), tuple(v_scale)
        self._descs = [None] * self.layers

    def __setattr__(self, name, value):
        """The descriptors hold the buffer's address, its sizes and the scales, so
        none of these is replaced: a new buffer is a new cache."""
        if name in self._FIXED and name in self.__dict__:
            raise AttributeError(f"a cache's {name} does not change: wrap the other buffer in a cache of its own")
        super().__setattr__(name, value)

    def desc(self, layer=0):
        """The C descriptor with one layer's scales."""
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer must be 0 .. {self.layers - 1}, not {layer}")
        d = self._descs[layer]
        if d is None:
            _on_device(self.data, "the cache's data")
            d = self._descs[layer] = qpn_kv4_cache(self.data.data_ptr(), self.pages, self.layers, self.page_size,
                                                   self.kv_heads, self.head_dim, self.k_scale[layer],
                                                   self.v_scale[layer])
        return d


def kv4_append(cache, k, v, slots, layer=0):
    """Quantizes k and v ([tokens, kv_heads, head_dim] fp16 or bf16, any
    strides with a contiguous last dimension: slices of a fused projection's
    output will do) into the pages' slots (int64 [tokens], page * page_size +
    offset; one outside the pool is skipped, none may be given twice)."""
    dev = cache.device
    tokens = slots.shape[0]
    shape = (tokens, cache.kv_heads, cache.head_dim)
    kp, kt, kh = _rows(k, shape, "k", dev, HALVES)
    vp, vt, vh = _rows(v, shape, "v", dev, (k.dtype,))
    sp = _exactly(slots, torch.int64, (tokens,), "slots", dev)
    qpn_kv4_append(cache.desc(layer), layer, kp, vp, DTYPES[k.dtype], tokens, kt, kh, vt, vh, sp,
                   _stream(dev))


def kv4_read(cache, slots, layer=0, dtype=torch.float16, k=None, v=None):
    """(k, v) [tokens, kv_heads, head_dim]: the values that the slots (int64
    [tokens]) stand for, zeros for one outside the pool."""
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be one of {', '.join(str(d) for d in DTYPES)}, not {dtype}")
    dev = cache.device
    tokens = slots.shape[0]
    sp = _exactly(slots, torch.int64, (tokens,), "slots", dev)
    shape = (tokens, cache.kv_heads, cache.head_dim)
    k = _out(k, dtype, shape, "k", dev)
    v = _out(v, dtype, shape, "v", dev)
    qpn_kv4_read(cache.desc(layer), layer, sp, tokens, DTYPES[dtype], k.data_ptr(), v.data_ptr(),
                 _stream(dev))
    return k, v


def kv4_copy_pages(cache, src, dst):
    """Copies pages src[i] onto dst[i] (int32 [n]) in every layer, in one
    launch. No page may be both a source and a destination, or a destination
    twice; a pair with a page outside the pool is skipped."""
    dev = cache.device
    n = src.shape[0]
    sp = _exactly(src, torch.int32, (n,), "src", dev)
    dp = _exactly(dst, torch.int32, (n,), "dst", dev)
    qpn_kv4_copy_pages(cache.desc(), sp, dp, n, _stream(dev))


@functools.lru_cache(maxsize=256)
def _attention_workspace_bytes(page_size, kv_heads, head_dim, rows, heads, batch, max_q_len, max_kv_len):
    c = qpn_kv4_cache(None, 0, 1, page_size, kv_heads, head_dim, 1.0, 1.0)
    a = qpn_kv4_attention_args()
    a.heads, a.batch, a.rows, a.max_q_len, a.max_kv_len = heads, batch, rows, max_q_len, max_kv_len
    return qpn_kv4_attention_workspace_bytes(c, a)


def kv4_attention_workspace(cache, rows, heads, batch, max_q_len, max_kv_len):
    """A workspace for kv4_attention with these sizes (None when none is
    needed). It carries nothing from call to call, but two calls that may run
    at once need one each."""
    _sizes(rows=rows, heads=heads, batch=batch, max_q_len=max_q_len, max_kv_len=max_kv_len)
    need = _attention_workspace_bytes(cache.page_size, cache.kv_heads, cache.head_dim, rows, heads, batch, max_q_len,
                                      max_kv_len)
    return torch.empty(need, dtype=torch.uint8, device=cache.device) if need else None


def kv4_attention(q, cache, table, kv_len, q_start=None, max_q_len=None, max_kv_len=None, layer=0, scale=None,
                  window=0, out=None, lse=None, workspace=None):
    """(out, lse): attention of each sequence's last rows over its cached
    tokens, the rows' own among them.

    q [rows, heads, head_dim] fp16 or bf16 (strides as of kv4_append); table
    int32 [batch, pages a sequence at most]; kv_len int32 [batch]; q_start
    int32 [batch + 1] from 0 to rows, with max_q_len the longest (None: rows /
    batch rows each). max_kv_len bounds the lengths (default: what the table
    can hold); a bound of 512 or less spares a small call its second launch.
    window > 0: a row sees the last `window` tokens up to its own. out [rows,
    heads, head_dim] like q, lse fp32 [rows, heads]; a row that sees no token
    gets zeros and -inf. The softmax weights are rounded to fp16 before the
    product with the values, and so are bf16 queries, scaled first (bounds in
    qpn_decode.h); sums are fp32."""
    dev = cache.device
    dim, kv_heads = cache.head_dim, cache.kv_heads
    _on_device(q, "q", dev)
    if q.dim() != 3:
        raise ValueError(f"q must have shape (rows, heads, {dim}), not {tuple(q.shape)}")
    rows, heads, _ = q.shape
    qp, qt, qh = _rows(q, (rows, heads, dim), "q", dev, HALVES)
    if heads == 0 or heads % kv_heads:
        raise ValueError(f"q's {heads} heads must be a multiple of the cache's {kv_heads}")
    _on_device(table, "table", dev)
    if table.dtype is not torch.int32 or table.dim() != 2 or (table.stride(1) != 1 and table.shape[1] > 1):
        raise ValueError("table must be an int32 [batch, pages] tensor with contiguous rows")
    batch, held = table.shape
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
        max_kv_len = held * cache.page_size
    if not (0 <= window <= INT32_MAX and 0 <= max_q_len <= INT32_MAX and 0 <= max_kv_len <= INT32_MAX):
        raise ValueError(f"window {window}, max_q_len {max_q_len} and max_kv_len {max_kv_len} must be 0 .. {INT32_MAX}")
    if max_kv_len > held * cache.page_size:   # (a slice's rows may lie further apart than they are long)
        raise ValueError(f"max_kv_len {max_kv_len} is more than a table row's {held} pages of {cache.page_size} hold")
    out = _out(out, q.dtype, (rows, heads, dim), "out", dev)
    lse = _out(lse, torch.float32, (rows, heads), "lse", dev)
    a = qpn_kv4_attention_args(qp, out.data_ptr(), lse.data_ptr(), table.data_ptr(), lp, sp, qt, qh,
                               table.stride(0) if batch > 1 else held, DTYPES[q.dtype], layer, heads, batch, rows,
                               max_q_len, max_kv_len, window, dim ** -0.5 if scale is None else scale, 0)
    workspace, wp, nbytes = _workspace(
        _attention_workspace_bytes(cache.page_size, kv_heads, dim, rows, heads, batch, max_q_len, max_kv_len), workspace,
        dev)
    qpn_kv4_attention(cache.desc(layer), a, wp, nbytes, _stream(dev))
    return out, lse


_verify_workspace_bytes = functools.lru_cache(maxsize=256)(qpn_verify_workspace_bytes)


def verify_workspace(batch, drafts, vocab, device="cuda"):
    """A workspace for verify_drafts with these sizes. It carries nothing from
    call to call, but two calls that may run at once need one each."""
    _sizes(batch=batch, drafts=drafts, vocab=vocab)
    need = _verify_workspace_bytes(batch, drafts, vocab)
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def verify_drafts(target, draft_tokens, u_accept, u_sample, draft=None, num_draft=None, temperature=None,
                  probabilities=False, tokens=None, accepted=None, logprobs=None, workspace=None):
    """(tokens int32 [batch, drafts + 1], accepted int32 [batch], logprobs fp32
    [batch, drafts + 1]): speculative sampling of a batch of verify blocks.

    target [batch, drafts + 1, vocab]: the target's logits at the drafts'
    places and the one after (fp16, bf16 or fp32, rows contiguous); draft
    [batch, drafts, vocab]: the drafter's, None where it chose without chance;
    draft_tokens int32 [batch, drafts]; num_draft int32 [batch]: how many of
    them each sequence has (None: all); temperature fp32 [batch] (0: greedy;
    None: 1); u_accept fp32 [batch, drafts] and u_sample fp32 [batch]: random
    numbers in [0, 1). probabilities=True: target and draft are fp32
    probabilities instead, taken as they are. The accepted drafts come first,
    then the token that replaces or follows them, then -1 (log-probability 0).
    Accept tests and log-probabilities of logits use p and q to about 2^-21 of
    themselves, the pick of the token 64 bits."""
    _on_device(target, "target")
    dev = target.device
    if target.dim() != 3:
        raise ValueError(f"target must have shape (batch, drafts + 1, vocab), not {tuple(target.shape)}")
    batch, places, vocab = target.shape
    drafts = places - 1
    if drafts < 0:
        raise ValueError("target needs a row for the token after the drafts")
    tp, tb, tr = _rows(target, (batch, places, vocab), "target", dev, (torch.float32,) if probabilities else DTYPES)
    dp, db, dr = (None, 0, 0) if draft is None else _rows(draft, (batch, drafts, vocab), "draft", dev, (target.dtype,))
    np_ = None if num_draft is None else _exactly(num_draft, torch.int32, (batch,), "num_draft", dev)
    if temperature is None:
        tmp = None
    else:
        if probabilities:
            raise ValueError("probabilities are taken as they are: no temperature")
        tmp = _exactly(temperature, torch.float32, (batch,), "temperature", dev)
    if vocab > INT32_MAX:
        raise ValueError(f"a vocabulary of {vocab} is more than {INT32_MAX}")
    tokens = _out(tokens, torch.int32, (batch, places), "tokens", dev)
    accepted = _out(accepted, torch.int32, (batch,), "accepted", dev)
    logprobs = _out(logprobs, torch.float32, (batch, places), "logprobs", dev)
    a = qpn_verify_args(tp, dp, _exactly(draft_tokens, torch.int32, (batch, drafts), "draft_tokens", dev), np_, tmp,
                        _exactly(u_accept, torch.float32, (batch, drafts), "u_accept", dev),
                        _exactly(u_sample, torch.float32, (batch,), "u_sample", dev), tokens.data_ptr(),
                        accepted.data_ptr(), logprobs.data_ptr(), tb, tr, db, dr, DTYPES[target.dtype],
                        1 if probabilities else 0, batch, drafts, vocab, 0)
    workspace, wp, nbytes = _workspace(_verify_workspace_bytes(batch, drafts, vocab), workspace, dev)
    qpn_verify(a, wp, nbytes, _stream(dev))
    return tokens, accepted, logprobs
