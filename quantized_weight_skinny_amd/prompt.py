"""Binding of the entry points of ``include/qpn_prompt.h`` (8-bit products with
a scale for each block of 128, attention of a chunk of new tokens over the
4-bit cache, log-probabilities of given tokens), one for one: integer device
pointers and sizes in, the qpn_status code checked (a negative one raises
``QpnError``). ``prompt_api`` has the torch helpers."""

import ctypes

from . import _check
from . import lib as _base_lib
from .decode import qpn_kv4_cache

QPN_DT_E4M3 = 4

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


class qpn_fp8_block_gemm_args(ctypes.Structure):
    _fields_ = [
        ("x", _P),
        ("x_scales", _P),
        ("w", _P),
        ("w_scales", _P),
        ("y", _P),
        ("x_stride", _I64),
        ("x_scale_row_stride", _I64),
        ("x_scale_block_stride", _I64),
        ("w_stride", _I64),
        ("w_scale_row_stride", _I64),
        ("w_scale_block_stride", _I64),
        ("y_stride", _I64),
        ("m", _I64),
        ("n", _I64),
        ("k", _I64),
        ("x_dtype", _I32),
        ("y_dtype", _I32),
    ]


class qpn_kv4_chunk_args(ctypes.Structure):
    _fields_ = [
        ("q", _P),
        ("k", _P),
        ("v", _P),
        ("out", _P),
        ("lse", _P),
        ("table", _P),
        ("kv_len", _P),
        ("q_start", _P),
        ("q_token_stride", _I64),
        ("q_head_stride", _I64),
        ("k_token_stride", _I64),
        ("k_head_stride", _I64),
        ("v_token_stride", _I64),
        ("v_head_stride", _I64),
        ("table_stride", _I64),
        ("dtype", _I32),
        ("layer", _I32),
        ("heads", _I32),
        ("batch", _I32),
        ("rows", _I32),
        ("max_q_len", _I32),
        ("max_kv_len", _I32),
        ("window", _I32),
        ("scale", ctypes.c_float),
        ("reserved", _I32),
    ]


class qpn_logprobs_args(ctypes.Structure):
    _fields_ = [
        ("logits", _P),
        ("tokens", _P),
        ("temperature", _P),
        ("logprobs", _P),
        ("entropy", _P),
        ("rank", _P),
        ("top_tokens", _P),
        ("top_logprobs", _P),
        ("row_stride", _I64),
        ("dtype", _I32),
        ("rows", _I32),
        ("vocab", _I32),
        ("top", _I32),
    ]


_C = ctypes.POINTER(qpn_kv4_cache)
_G = ctypes.POINTER(qpn_fp8_block_gemm_args)
_A = ctypes.POINTER(qpn_kv4_chunk_args)
_L = ctypes.POINTER(qpn_logprobs_args)

# name -> (restype, argtypes); the declarations of include/qpn_prompt.h
SIGNATURES = {
    "qpn_fp8_block_quantize": (_I32, [_P, _I32, _I64, _I64, _I64, _I32, _P, _I64, _P, _I64, _I64, _P]),
    "qpn_fp8_block_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "qpn_fp8_block_gemm": (_I32, [_G, _P, _SZ, _P]),
    "qpn_kv4_chunk_workspace_bytes": (_SZ, [_C, _A]),
    "qpn_kv4_chunk_attention": (_I32, [_C, _A, _P, _SZ, _P]),
    "qpn_token_logprobs_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "qpn_token_logprobs": (_I32, [_L, _P, _SZ, _P]),
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


def qpn_fp8_block_quantize(x, dtype, rows, k, stride, block_rows, codes, code_stride, scales, scale_row_stride,
                           scale_block_stride, stream):
    return _check(lib().qpn_fp8_block_quantize(x, dtype, rows, k, stride, block_rows, codes, code_stride, scales,
                                               scale_row_stride, scale_block_stride, stream), "qpn_fp8_block_quantize")


def qpn_fp8_block_workspace_bytes(m, n, k):
    return lib().qpn_fp8_block_workspace_bytes(m, n, k)


def qpn_fp8_block_gemm(args, workspace, workspace_bytes, stream):
    return _check(lib().qpn_fp8_block_gemm(ctypes.byref(args), workspace, workspace_bytes, stream),
                  "qpn_fp8_block_gemm")


def qpn_kv4_chunk_workspace_bytes(cache, args):
    return lib().qpn_kv4_chunk_workspace_bytes(ctypes.byref(cache), ctypes.byref(args))


def qpn_kv4_chunk_attention(cache, args, workspace, workspace_bytes, stream):
    return _check(lib().qpn_kv4_chunk_attention(ctypes.byref(cache), ctypes.byref(args), workspace, workspace_bytes,
                                                stream), "qpn_kv4_chunk_attention")


def qpn_token_logprobs_workspace_bytes(rows, vocab, top):
    return lib().qpn_token_logprobs_workspace_bytes(rows, vocab, top)


def qpn_token_logprobs(args, workspace, workspace_bytes, stream):
    return _check(lib().qpn_token_logprobs(ctypes.byref(args), workspace, workspace_bytes, stream),
                  "qpn_token_logprobs")
