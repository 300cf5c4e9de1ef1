"""CPU checks of include/qpn_prompt.h: every entry point is exported and bound,
the header is C99 with the binding's struct layouts, and bad arguments are
refused on the host before any HIP call (these run without a GPU; no compute
entry point is exercised)."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import quantized_weight_skinny_amd as q
from quantized_weight_skinny_amd import decode as qdec
from quantized_weight_skinny_amd import decode_api as qd
from quantized_weight_skinny_amd import prompt as qpr
from quantized_weight_skinny_amd import prompt_api as qp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qpn_prompt.h")
FAKE = 0x7F0000000000  # an aligned non-null "device" address; never dereferenced
BAD, SMALL, UNSUPPORTED, OK = q.QPN_ERR_INVALID_ARG, q.QPN_ERR_BUFFER_TOO_SMALL, q.QPN_ERR_UNSUPPORTED, q.QPN_OK
F16, BF16, F32, E4M3 = qdec.QPN_DT_F16, qdec.QPN_DT_BF16, qdec.QPN_DT_F32, qpr.QPN_DT_E4M3


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(qpn_[a-z0-9_]+)\s*\(", text)))


def test_library_exports_every_declared_function():
    lib = qpr.lib()
    assert set(_declared()) == set(qpr.SIGNATURES)
    for name in _declared():
        assert hasattr(lib, name), name


def test_header_is_c99_with_the_bindings_layouts(tmp_path):
    structs = {"qpn_fp8_block_gemm_args": qpr.qpn_fp8_block_gemm_args, "qpn_kv4_chunk_args": qpr.qpn_kv4_chunk_args,
               "qpn_logprobs_args": qpr.qpn_logprobs_args}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "qpn_prompt.h"', "typedef void (*entry_fn)(void);",
             "int main(void) {", "  const entry_fn entries[] = {" + ", ".join(f"(entry_fn){n}" for n in _declared()) + "};",
             "  unsigned i;", "  for (i = 0; i < sizeof entries / sizeof entries[0]; ++i) if (!entries[i]) return 1;",
             '  printf("e4m3 %d\\n", QPN_DT_E4M3);']
    for name, cls in structs.items():
        lines.append(f'  printf("{name} %zu\\n", sizeof({name}));')
        for field, _ in cls._fields_:
            lines.append(f'  printf("{name}.{field} %zu\\n", offsetof({name}, {field}));')
    lines += ["  return 0;", "}"]
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text("\n".join(lines))
    libdir = os.path.dirname(q.LIB_PATH)
    cmd = ["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src),
           "-o", str(exe), "-L", libdir, "-lqpn", f"-Wl,-rpath,{libdir}"]
    if os.path.isdir("/opt/rocm/lib"):
        cmd.append("-Wl,-rpath-link,/opt/rocm/lib")
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0
    got = dict(line.split() for line in run.stdout.splitlines())
    assert int(got["e4m3"]) == E4M3
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for field, _ in cls._fields_:
            assert int(got[f"{name}.{field}"]) == getattr(cls, field).offset, (name, field)


def _quantize(**kw):
    a = dict(x=FAKE, dtype=F16, rows=3, k=100, stride=100, block_rows=1, codes=FAKE, code_stride=100, scales=FAKE,
             scale_row_stride=1, scale_block_stride=3)
    a.update(kw)
    return qpr.lib().qpn_fp8_block_quantize(*a.values(), None)


def test_quantizer_refuses_bad_arguments():
    for kw in (dict(x=None), dict(x=FAKE + 1), dict(x=FAKE + 2, dtype=F32), dict(dtype=0), dict(dtype=E4M3), dict(rows=-1),
               dict(rows=(1 << 24) + 1), dict(k=-1), dict(k=(1 << 20) + 1), dict(stride=-1), dict(stride=1 << 41),
               dict(block_rows=0), dict(block_rows=2), dict(codes=None), dict(code_stride=99), dict(scales=None),
               dict(scales=FAKE + 2), dict(scale_row_stride=-1), dict(scale_block_stride=-1)):
        assert _quantize(**kw) == BAD, kw
    assert _quantize(rows=0, x=None, codes=None, scales=None) == OK
    assert _quantize(k=0, x=None, codes=None, scales=None) == OK
    assert _quantize(rows=1 << 24, k=1 << 20, stride=1 << 20, code_stride=1 << 20) == UNSUPPORTED


def _gemm(ws=FAKE, ws_bytes=1 << 44, **kw):
    a = qpr.qpn_fp8_block_gemm_args(x=FAKE, x_scales=FAKE, w=FAKE, w_scales=FAKE, y=FAKE, x_stride=256,
                                    x_scale_row_stride=1, x_scale_block_stride=20, w_stride=256, w_scale_row_stride=2,
                                    w_scale_block_stride=1, y_stride=40, m=20, n=40, k=256, x_dtype=E4M3, y_dtype=BF16)
    for k, v in kw.items():
        setattr(a, k, v)
    return qpr.lib().qpn_fp8_block_gemm(ctypes.byref(a), ws, ws_bytes, None)


def test_product_refuses_bad_arguments():
    assert qpr.lib().qpn_fp8_block_gemm(None, FAKE, 1 << 40, None) == BAD
    for kw in (dict(x=None), dict(x=FAKE + 8), dict(x_scales=None), dict(x_scales=FAKE + 1), dict(w=None), dict(w=FAKE + 8),
               dict(w_scales=None), dict(w_scales=FAKE + 2), dict(y=None), dict(y=FAKE + 1), dict(y=FAKE + 2, y_dtype=F32),
               dict(x_stride=264), dict(x_stride=240), dict(x_stride=1 << 23), dict(x_stride=-16), dict(w_stride=240),
               dict(w_stride=264), dict(w_stride=1 << 23), dict(y_stride=39), dict(x_scale_row_stride=-1),
               dict(x_scale_row_stride=1 << 23), dict(x_scale_block_stride=-1), dict(w_scale_row_stride=-1),
               dict(w_scale_block_stride=1 << 41), dict(m=-1), dict(m=(1 << 22) + 1), dict(n=-1), dict(k=-16), dict(k=250),
               dict(k=(1 << 20) + 16), dict(x_dtype=0), dict(x_dtype=5), dict(y_dtype=E4M3), dict(y_dtype=0), dict(ws=None),
               dict(ws=FAKE + 8), dict(x_dtype=F16), dict(x_dtype=F32, x_scales=None, x=FAKE + 2)):
        assert _gemm(**kw) == BAD, kw
    need = qpr.qpn_fp8_block_workspace_bytes(20, 40, 256)
    assert need > 0 and _gemm(ws_bytes=need - 1) == SMALL
    assert _gemm(m=0, x=None, y=None) == OK and _gemm(n=0, w=None, y=None) == OK
    assert qpr.qpn_fp8_block_workspace_bytes(20, 40, 250) == 0 and qpr.qpn_fp8_block_workspace_bytes(-1, 40, 256) == 0


def _cache(**kw):
    c = qdec.qpn_kv4_cache(FAKE, 10, 2, 64, 8, 128, 0.5, 0.25)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _chunk_args(**kw):
    a = qpr.qpn_kv4_chunk_args(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, table=FAKE, kv_len=FAKE, q_start=FAKE,
                               q_token_stride=5120, q_head_stride=128, k_token_stride=1024, k_head_stride=128,
                               v_token_stride=1024, v_head_stride=128, table_stride=16, dtype=F16, layer=1, heads=40,
                               batch=3, rows=24, max_q_len=8, max_kv_len=1000, window=0, scale=0.1, reserved=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _chunk(ws=FAKE, ws_bytes=1 << 40, cache=None, **kw):
    c = _cache() if cache is None else cache
    return qpr.lib().qpn_kv4_chunk_attention(ctypes.byref(c), ctypes.byref(_chunk_args(**kw)), ws, ws_bytes, None)


def test_chunk_attention_refuses_bad_arguments():
    lib = qpr.lib()
    assert lib.qpn_kv4_chunk_attention(None, ctypes.byref(_chunk_args()), FAKE, 1 << 40, None) == BAD
    assert lib.qpn_kv4_chunk_attention(ctypes.byref(_cache()), None, FAKE, 1 << 40, None) == BAD
    for kw in (dict(data=None), dict(pages=-1), dict(layers=0), dict(page_size=24), dict(head_dim=80), dict(k_scale=0.0),
               dict(v_scale=float("nan"))):
        assert _chunk(cache=_cache(**kw)) == BAD, kw
    for kw in (dict(q=None), dict(q=FAKE + 1), dict(k=None), dict(k=FAKE + 1), dict(v=None), dict(v=FAKE + 1), dict(out=None),
               dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(table=None), dict(table=FAKE + 2), dict(kv_len=None),
               dict(kv_len=FAKE + 1), dict(q_start=FAKE + 2), dict(q_token_stride=-1), dict(q_head_stride=1 << 41),
               dict(k_token_stride=-1), dict(k_head_stride=1 << 41), dict(v_token_stride=-1), dict(v_head_stride=-1),
               dict(table_stride=-1), dict(table_stride=15), dict(dtype=F32), dict(dtype=0), dict(layer=-1), dict(layer=2),
               dict(heads=0), dict(heads=12), dict(heads=-8), dict(heads=65544), dict(batch=-1), dict(batch=65537),
               dict(batch=0), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(max_q_len=-1), dict(max_q_len=0),
               dict(max_q_len=(1 << 20) + 1), dict(max_kv_len=-1), dict(max_kv_len=(1 << 30) + 1), dict(window=-1),
               dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(reserved=1),
               dict(q_start=None, rows=23), dict(ws=None), dict(ws=FAKE + 8)):
        assert _chunk(**kw) == BAD, kw
    need = qpr.qpn_kv4_chunk_workspace_bytes(_cache(), _chunk_args())
    assert need == qpr.qpn_kv4_chunk_workspace_bytes(_cache(), _chunk_args(q=None, k=None, out=None, table=None))
    assert need > 0 and _chunk(ws_bytes=need - 1) == SMALL
    assert _chunk(rows=0, q=None, out=None) == OK and _chunk(batch=0, rows=0, q=None, kv_len=None) == OK
    assert _chunk(rows=1 << 24, max_q_len=1 << 20, heads=65536) == UNSUPPORTED


def _logprobs(ws=FAKE, ws_bytes=1 << 40, **kw):
    a = qpr.qpn_logprobs_args(logits=FAKE, tokens=FAKE, temperature=FAKE, logprobs=FAKE, entropy=FAKE, rank=FAKE,
                              top_tokens=FAKE, top_logprobs=FAKE, row_stride=100, dtype=F16, rows=3, vocab=100, top=5)
    for k, v in kw.items():
        setattr(a, k, v)
    return qpr.lib().qpn_token_logprobs(ctypes.byref(a), ws, ws_bytes, None)


def test_token_logprobs_refuses_bad_arguments():
    assert qpr.lib().qpn_token_logprobs(None, FAKE, 1 << 40, None) == BAD
    for kw in (dict(logits=None), dict(logits=FAKE + 1), dict(logits=FAKE + 2, dtype=F32), dict(tokens=None),
               dict(tokens=FAKE + 2), dict(temperature=FAKE + 1), dict(logprobs=FAKE + 2), dict(entropy=FAKE + 2),
               dict(rank=FAKE + 2), dict(top_tokens=None), dict(top_logprobs=None), dict(top_tokens=FAKE + 2),
               dict(top_logprobs=FAKE + 1), dict(row_stride=-1), dict(row_stride=1 << 41), dict(dtype=0), dict(dtype=E4M3),
               dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(top=-1), dict(top=65),
               dict(vocab=4), dict(ws=None), dict(ws=FAKE + 8)):
        assert _logprobs(**kw) == BAD, kw
    need = qpr.qpn_token_logprobs_workspace_bytes(3, 100, 5)
    assert need > 0 and _logprobs(ws_bytes=need - 1) == SMALL
    assert _logprobs(rows=0, logits=None, ws=None) == OK


# ------------------------------------------------------------------ the torch layer (tensors stay on the host)

@pytest.fixture
def on_host(monkeypatch):
    monkeypatch.setattr(qd, "_on_device", lambda *a: None)
    monkeypatch.setattr(qp, "_on_device", lambda *a: None)


def test_sizes_beyond_32_bits_are_refused():
    for call in (lambda: qp.fp8_block_workspace(1 << 32, 16, 16), lambda: qp.token_logprobs_workspace(1, 1 << 32),
                 lambda: qp.token_logprobs_workspace(1, 100, -1)):
        with pytest.raises(ValueError, match="must be 0 .."):
            call()
    cache = qd.KV4Cache(4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="must be 0 .."):
        qp.kv4_chunk_workspace(cache, 1, 4, 1, 1, 1 << 33)


def test_chunk_attention_takes_no_longer_bound_than_the_table_holds(on_host):
    cache = qd.KV4Cache(4, 16, 2, 64, device="cpu")
    x, kv = torch.zeros((2, 4, 64), dtype=torch.float16), torch.zeros((2, 2, 64), dtype=torch.float16)
    lengths = torch.zeros(2, dtype=torch.int32)
    wide = torch.zeros((2, 50), dtype=torch.int32)
    for table in (wide[:, :3], wide[:, 47:], wide[:, 3:6].contiguous()):
        for bound in (49, 800):
            with pytest.raises(ValueError, match="max_kv_len"):
                qp.kv4_chunk_attention(x, kv, kv, cache, table, lengths, max_kv_len=bound)
    for bad in (dict(window=-1), dict(window=1 << 32), dict(max_kv_len=-1)):
        with pytest.raises(ValueError, match="must be 0 .."):
            qp.kv4_chunk_attention(x, kv, kv, cache, wide, lengths, **bad)


def test_weights_keep_to_whole_pieces(on_host):
    ones = torch.ones((1, 1))
    for codes in (torch.zeros((4, 24), dtype=torch.uint8), torch.zeros((4, 40), dtype=torch.uint8)[:, :32]):
        with pytest.raises(ValueError, match="16"):
            qp.BlockWeight(codes, ones)
    with pytest.raises(ValueError, match="scales"):
        qp.BlockWeight(torch.zeros((129, 32), dtype=torch.uint8), ones)
    with pytest.raises(ValueError, match="one of"):
        qp.BlockWeight(torch.zeros((4, 32), dtype=torch.int8), ones)
