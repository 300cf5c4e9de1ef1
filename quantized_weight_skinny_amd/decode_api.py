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
from .torch_api import _output, _stream

DTYPES = {torch.float16: QPN_DT_F16, torch.bfloat16: QPN_DT_BF16, torch.float32: QPN_DT_F32}


def _on_device(t, name, device=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t


def _ints(t, dtype, shape, name, device):
    """A contiguous tensor of whole numbers of exactly this shape."""
    _on_device(t, name, device)
    if t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, not {t.dtype} "
                         f"{tuple(t.shape)}")
    return t


def _floats(t, shape, name, device):
    _on_device(t, name, device)
    if t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)}, not {t.dtype} "
                         f"{tuple(t.shape)}")
    return t


def _rows(t, shape, name, device, dtypes):
    """A tensor of this shape whose last dimension is contiguous, other strides free."""
    _on_device(t, name, device)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t


def _workspace(need, workspace, device):
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if not need:
        return None, 0
    _on_device(workspace, "workspace", device)
    return workspace, workspace.numel() * workspace.element_size()


class KV4Cache:
    """Pages of keys and values in 4 bits: ``data`` uint8 [layers, pages,
    page_bytes] (the layout is in qpn_decode.h). ``k_scale`` and ``v_scale``
    are tensor scales, one number or one a layer: the largest magnitude a
    block holds exactly is 2688 times the scale, the finest step of a block's
    scale 2^-9 of it, so amax / 2688 of typical keys (values) is the choice."""

    def __init__(self, pages, page_size, kv_heads, head_dim, layers=1, k_scale=1.0 / 128, v_scale=1.0 / 128,
                 device="cuda"):
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
        _on_device(data, "data")
        nbytes = qpn_kv4_page_bytes(page_size, kv_heads, head_dim)
        if data.dtype != torch.uint8 or data.dim() != 3 or not data.is_contiguous() or data.shape[2] != nbytes or not nbytes:
            raise ValueError(f"data must be a contiguous uint8 [layers, pages, {nbytes}] tensor")
        self._init(data, page_size, kv_heads, head_dim, k_scale, v_scale)
        return self

    def _init(self, data, page_size, kv_heads, head_dim, k_scale, v_scale):
        self.data = data
        self.layers, self.pages = data.shape[0], data.shape[1]
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        self.k_scale, self.v_scale = (
            [float(s)] * self.layers if isinstance(s, (int, float)) else [float(x) for x in s]
            for s in (k_scale, v_scale))
        if len(self.k_scale) != self.layers or len(self.v_scale) != self.layers:
            raise ValueError("k_scale and v_scale take one number, or one a layer")
        if not all(math.isfinite(s) and s > 0 for s in self.k_scale + self.v_scale):
            raise ValueError("tensor scales must be finite and above 0")

    @property
    def device(self):
        return self.data.device

    def layer(self, layer):
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer must be 0 .. {self.layers - 1}, not {layer}")
        return layer

    def desc(self, layer=0):
        return qpn_kv4_cache(self.data.data_ptr(), self.pages, self.layers, self.page_size, self.kv_heads,
                             self.head_dim, self.k_scale[layer], self.v_scale[layer])


def kv4_append(cache, k, v, slots, layer=0):
    """Quantizes k and v ([tokens, kv_heads, head_dim] fp16 or bf16, any
    strides with a contiguous last dimension: slices of a fused projection's
    output will do) into the pages' slots (int64 [tokens], page * page_size +
    offset; one outside the pool is skipped)."""
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    _rows(k, shape, "k", cache.device, (torch.float16, torch.bfloat16))
    _rows(v, shape, "v", cache.device, (k.dtype,))
    _ints(slots, torch.int64, (shape[0],), "slots", cache.device)
    qpn_kv4_append(cache.desc(cache.layer(layer)), layer, k.data_ptr(), v.data_ptr(), DTYPES[k.dtype], shape[0],
                   k.stride(0), k.stride(1), v.stride(0), v.stride(1), slots.data_ptr(), _stream())


def kv4_read(cache, slots, layer=0, dtype=torch.float16, k=None, v=None):
    """(k, v) [tokens, kv_heads, head_dim]: the values that the slots (int64
    [tokens]) stand for, zeros for one outside the pool."""
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be one of {', '.join(str(d) for d in DTYPES)}, not {dtype}")
    _on_device(slots, "slots", cache.device)
    _ints(slots, torch.int64, (slots.numel(),), "slots", cache.device)
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    k = _output(k, shape, dtype, cache.data, "k")
    v = _output(v, shape, dtype, cache.data, "v")
    qpn_kv4_read(cache.desc(cache.layer(layer)), layer, slots.data_ptr(), shape[0], DTYPES[dtype], k.data_ptr(),
                 v.data_ptr(), _stream())
    return k, v


def kv4_copy_pages(cache, src, dst):
    """Copies pages src[i] onto dst[i] (int32 [n]) in every layer, in one
    launch. No page may be both a source and a destination, or a destination
    twice; a pair with a page outside the pool is skipped."""
    _on_device(src, "src", cache.device)
    _ints(src, torch.int32, (src.numel(),), "src", cache.device)
    _ints(dst, torch.int32, tuple(src.shape), "dst", cache.device)
    qpn_kv4_copy_pages(cache.desc(), src.data_ptr(), dst.data_ptr(), src.shape[0], _stream())


def _attention_sizes(rows, heads, batch, max_q_len, max_kv_len):
    a = qpn_kv4_attention_args()
    a.heads, a.batch, a.rows, a.max_q_len, a.max_kv_len = heads, batch, rows, max_q_len, max_kv_len
    return a


def kv4_attention_workspace(cache, rows, heads, batch, max_q_len, max_kv_len):
    """A workspace for kv4_attention with these sizes (None when none is
    needed). It carries nothing from call to call, but two calls that may run
    at once need one each."""
    need = qpn_kv4_attention_workspace_bytes(cache.desc(),
                                             _attention_sizes(rows, heads, batch, max_q_len, max_kv_len))
    return torch.empty(need, dtype=torch.uint8, device=cache.device) if need else None


def kv4_attention(q, cache, table, kv_len, q_start=None, max_q_len=None, max_kv_len=None, layer=0, scale=None,
                  window=0, out=None, lse=None, workspace=None):
    """(out, lse): attention of each sequence's last rows over its cached
    tokens, the rows' own among them.

    q [rows, heads, head_dim] fp16 or bf16 (strides as of kv4_append); table
    int32 [batch, pages a sequence at most]; kv_len int32 [batch]; q_start
    int32 [batch + 1] from 0 to rows, with max_q_len the longest (None: rows /
    batch rows each). max_kv_len bounds the lengths (default: what the table
    can hold); a close bound spares a small call its second launch. window > 0:
    a row sees the last `window` tokens up to its own. out [rows, heads,
    head_dim] like q, lse fp32 [rows, heads]; a row that sees no token gets
    zeros and -inf."""
    _on_device(q, "q", cache.device)
    if q.dim() != 3:
        raise ValueError(f"q must have shape (rows, heads, {cache.head_dim}), not {tuple(q.shape)}")
    rows, heads = q.shape[0], q.shape[1]
    _rows(q, (rows, heads, cache.head_dim), "q", cache.device, (torch.float16, torch.bfloat16))
    if heads == 0 or heads % cache.kv_heads:
        raise ValueError(f"q's {heads} heads must be a multiple of the cache's {cache.kv_heads}")
    _on_device(table, "table", cache.device)
    if table.dim() != 2 or table.dtype != torch.int32 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be an int32 [batch, pages] tensor with contiguous rows")
    batch = table.shape[0]
    _ints(kv_len, torch.int32, (batch,), "kv_len", cache.device)
    if q_start is not None:
        _ints(q_start, torch.int32, (batch + 1,), "q_start", cache.device)
        if max_q_len is None:
            raise ValueError("q_start needs max_q_len, the longest sequence's rows")
    else:
        each = rows // batch if batch else 0
        if each * batch != rows or (max_q_len is not None and max_q_len != each):
            raise ValueError(f"{rows} rows are not {batch} sequences of as many: give q_start and max_q_len")
        max_q_len = each
    if max_kv_len is None:
        max_kv_len = table.shape[1] * cache.page_size
    out = _output(out, (rows, heads, cache.head_dim), q.dtype, q)
    lse = _output(lse, (rows, heads), torch.float32, q, "lse")
    a = _attention_sizes(rows, heads, batch, max_q_len, max_kv_len)
    a.q, a.out, a.lse = q.data_ptr(), out.data_ptr(), lse.data_ptr()
    a.table, a.kv_len = table.data_ptr(), kv_len.data_ptr()
    a.q_start = q_start.data_ptr() if q_start is not None else None
    a.q_token_stride, a.q_head_stride = q.stride(0), q.stride(1)
    a.table_stride = table.stride(0) if batch > 1 else table.shape[1]
    a.dtype, a.layer, a.window = DTYPES[q.dtype], cache.layer(layer), window
    a.scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else scale
    d = cache.desc(layer)
    workspace, nbytes = _workspace(qpn_kv4_attention_workspace_bytes(d, a), workspace, q.device)
    qpn_kv4_attention(d, a, workspace.data_ptr() if nbytes else None, nbytes, _stream())
    return out, lse


def verify_workspace(batch, drafts, vocab, device="cuda"):
    """A workspace for verify_drafts with these sizes."""
    need = qpn_verify_workspace_bytes(batch, drafts, vocab)
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
    then the token that replaces or follows them, then -1 (log-probability 0)."""
    _on_device(target, "target")
    dev = target.device
    if target.dim() != 3:
        raise ValueError(f"target must have shape (batch, drafts + 1, vocab), not {tuple(target.shape)}")
    batch, drafts, vocab = target.shape[0], target.shape[1] - 1, target.shape[2]
    if drafts < 0:
        raise ValueError("target needs a row for the token after the drafts")
    kinds = (torch.float32,) if probabilities else tuple(DTYPES)
    _rows(target, (batch, drafts + 1, vocab), "target", dev, kinds)
    if draft is not None:
        _rows(draft, (batch, drafts, vocab), "draft", dev, (target.dtype,))
    _ints(draft_tokens, torch.int32, (batch, drafts), "draft_tokens", dev)
    _floats(u_accept, (batch, drafts), "u_accept", dev)
    _floats(u_sample, (batch,), "u_sample", dev)
    if num_draft is not None:
        _ints(num_draft, torch.int32, (batch,), "num_draft", dev)
    if temperature is not None:
        if probabilities:
            raise ValueError("probabilities are taken as they are: no temperature")
        _floats(temperature, (batch,), "temperature", dev)
    tokens = _output(tokens, (batch, drafts + 1), torch.int32, target, "tokens")
    accepted = _output(accepted, (batch,), torch.int32, target, "accepted")
    logprobs = _output(logprobs, (batch, drafts + 1), torch.float32, target, "logprobs")
    a = qpn_verify_args()
    a.target, a.draft = target.data_ptr(), draft.data_ptr() if draft is not None else None
    a.draft_tokens = draft_tokens.data_ptr()
    a.num_draft = num_draft.data_ptr() if num_draft is not None else None
    a.temperature = temperature.data_ptr() if temperature is not None else None
    a.u_accept, a.u_sample = u_accept.data_ptr(), u_sample.data_ptr()
    a.tokens, a.accepted, a.logprobs = tokens.data_ptr(), accepted.data_ptr(), logprobs.data_ptr()
    a.target_batch_stride, a.target_row_stride = target.stride(0), target.stride(1)
    if draft is not None:
        a.draft_batch_stride, a.draft_row_stride = draft.stride(0), draft.stride(1)
    a.dtype, a.probabilities = DTYPES[target.dtype], int(probabilities)
    a.batch, a.drafts, a.vocab = batch, drafts, vocab
    workspace, nbytes = _workspace(qpn_verify_workspace_bytes(batch, drafts, vocab), workspace, dev)
    qpn_verify(a, workspace.data_ptr() if nbytes else None, nbytes, _stream())
    return tokens, accepted, logprobs
