"""Binding of the entry points of ``include/qpn_decode.h`` (the 4-bit paged
cache, attention over it, page copies, verification of drafted tokens), one
for one: integer device pointers and sizes in, the qpn_status code checked (a
negative one raises ``QpnError``). ``decode_api`` has the torch helpers."""

import ctypes

from . import _check
from . import lib as _base_lib

QPN_DT_F16 = 1
QPN_DT_BF16 = 2
QPN_DT_F32 = 3

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float


class qpn_kv4_cache(ctypes.Structure):
    _fields_ = [
        ("data", _P),
        ("pages", _I64),
        ("layers", _I32),
        ("page_size", _I32),
        ("kv_heads", _I32),
        ("head_dim", _I32),
        ("k_scale", _F),
        ("v_scale", _F),
    ]


class qpn_kv4_attention_args(ctypes.Structure):
    _fields_ = [
        ("q", _P),
        ("out", _P),
        ("lse", _P),
        ("table", _P),
        ("kv_len", _P),
        ("q_start", _P),
        ("q_token_stride", _I64),
        ("q_head_stride", _I64),
        ("table_stride", _I64),
        ("dtype", _I32),
        ("layer", _I32),
        ("heads", _I32),
        ("batch", _I32),
        ("rows", _I32),
        ("max_q_len", _I32),
        ("max_kv_len", _I32),
        ("window", _I32),
        ("scale", _F),
        ("reserved", _I32),
    ]


class qpn_verify_args(ctypes.Structure):
    _fields_ = [
        ("target", _P),
        ("draft", _P),
        ("draft_tokens", _P),
        ("num_draft", _P),
        ("temperature", _P),
        ("u_accept", _P),
        ("u_sample", _P),
        ("tokens", _P),
        ("accepted", _P),
        ("logprobs", _P),
        ("target_batch_stride", _I64),
        ("target_row_stride", _I64),
        ("draft_batch_stride", _I64),
        ("draft_row_stride", _I64),
        ("dtype", _I32),
        ("probabilities", _I32),
        ("batch", _I32),
        ("drafts", _I32),
        ("vocab", _I32),
        ("reserved", _I32),
    ]


_C = ctypes.POINTER(qpn_kv4_cache)
_A = ctypes.POINTER(qpn_kv4_attention_args)
_V = ctypes.POINTER(qpn_verify_args)

# name -> (restype, argtypes); the declarations of include/qpn_decode.h
SIGNATURES = {
    "qpn_kv4_page_bytes": (_SZ, [_I32, _I32, _I32]),
    "qpn_kv4_append": (_I32, [_C, _I32, _P, _P, _I32, _I64, _I64, _I64, _I64, _I64, _P, _P]),
    "qpn_kv4_read": (_I32, [_C, _I32, _P, _I64, _I32, _P, _P, _P]),
    "qpn_kv4_copy_pages": (_I32, [_C, _P, _P, _I64, _P]),
    "qpn_kv4_attention_workspace_bytes": (_SZ, [_C, _A]),
    "qpn_kv4_attention": (_I32, [_C, _A, _P, _SZ, _P]),
    "qpn_verify_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "qpn_verify": (_I32, [_V, _P, _SZ, _P]),
}

_lib = None


def lib():
    """The loaded libqpn.so with these entry points declared."""
    global _lib
    if _lib is None:
        handle = _base_lib()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def qpn_kv4_page_bytes(page_size, kv_heads, head_dim):
    return lib().qpn_kv4_page_bytes(page_size, kv_heads, head_dim)


def qpn_kv4_append(cache, layer, k, v, dtype, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                   slots, stream):
    return _check(lib().qpn_kv4_append(ctypes.byref(cache), layer, k, v, dtype, tokens, k_token_stride, k_head_stride,
                                       v_token_stride, v_head_stride, slots, stream), "qpn_kv4_append")


def qpn_kv4_read(cache, layer, slots, tokens, dtype, k, v, stream):
    return _check(lib().qpn_kv4_read(ctypes.byref(cache), layer, slots, tokens, dtype, k, v, stream), "qpn_kv4_read")


def qpn_kv4_copy_pages(cache, src, dst, count, stream):
    return _check(lib().qpn_kv4_copy_pages(ctypes.byref(cache), src, dst, count, stream), "qpn_kv4_copy_pages")


def qpn_kv4_attention_workspace_bytes(cache, args):
    return lib().qpn_kv4_attention_workspace_bytes(ctypes.byref(cache), ctypes.byref(args))


def qpn_kv4_attention(cache, args, workspace, workspace_bytes, stream):
    return _check(lib().qpn_kv4_attention(ctypes.byref(cache), ctypes.byref(args), workspace, workspace_bytes, stream),
                  "qpn_kv4_attention")


def qpn_verify_workspace_bytes(batch, drafts, vocab):
    return lib().qpn_verify_workspace_bytes(batch, drafts, vocab)


def qpn_verify(args, workspace, workspace_bytes, stream):
    return _check(lib().qpn_verify(ctypes.byref(args), workspace, workspace_bytes, stream), "qpn_verify")
