"""CPU checks of include/qpn_decode.h: every entry point is exported and
bound, the header is C99 with the binding's struct layouts, sizes are what the
layout says, and bad arguments are refused on the host before any HIP call
(these run without a GPU; no compute entry point is exercised)."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import quantized_weight_skinny_amd as q
from quantized_weight_skinny_amd import decode as qdec
from quantized_weight_skinny_amd import decode_api as qd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qpn_decode.h")
FAKE = 0x7F0000000000  # an aligned non-null "device" address; never dereferenced
BAD, SMALL, UNSUPPORTED = q.QPN_ERR_INVALID_ARG, q.QPN_ERR_BUFFER_TOO_SMALL, q.QPN_ERR_UNSUPPORTED


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(qpn_[a-z0-9_]+)\s*\(", text)))


def test_library_exports_every_declared_function():
    lib = qdec.lib()
    assert set(_declared()) == set(qdec.SIGNATURES)
    for name in _declared():
        assert hasattr(lib, name), name


def test_header_is_c99_with_the_bindings_layouts(tmp_path):
    structs = {"qpn_kv4_cache": qdec.qpn_kv4_cache, "qpn_kv4_attention_args": qdec.qpn_kv4_attention_args,
               "qpn_verify_args": qdec.qpn_verify_args}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "qpn_decode.h"', "typedef void (*entry_fn)(void);",
             "int main(void) {", "  const entry_fn entries[] = {" + ", ".join(f"(entry_fn){n}" for n in _declared()) + "};",
             "  unsigned i;", "  for (i = 0; i < sizeof entries / sizeof entries[0]; ++i) if (!entries[i]) return 1;"]
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
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for field, _ in cls._fields_:
            assert int(got[f"{name}.{field}"]) == getattr(cls, field).offset, (name, field)


def test_page_bytes():
    assert qdec.qpn_kv4_page_bytes(64, 8, 128) == 64 * 8 * 2 * (64 + 8)
    assert qdec.qpn_kv4_page_bytes(16, 1, 64) == 16 * 2 * (32 + 4)
    for bad in ((8, 1, 64), (48, 1, 64), (512, 1, 64), (64, 0, 64), (64, 1025, 64), (64, 1, 96), (64, 1, 0), (-64, 1, 64)):
        assert qdec.qpn_kv4_page_bytes(*bad) == 0


def _cache(**kw):
    c = qdec.qpn_kv4_cache(FAKE, 10, 2, 64, 8, 128, 0.5, 0.25)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [dict(data=None), dict(data=FAKE + 8), dict(pages=-1), dict(pages=1 << 31), dict(layers=0),
              dict(page_size=24), dict(kv_heads=0), dict(head_dim=80), dict(k_scale=0.0), dict(v_scale=-1.0),
              dict(k_scale=float("inf")), dict(v_scale=float("nan"))]


def _append(cache=None, layer=0, k=FAKE, v=FAKE, dtype=qdec.QPN_DT_F16, tokens=3, strides=(1024, 128, 1024, 128),
            slots=FAKE):
    c = _cache() if cache is None else cache
    return qdec.lib().qpn_kv4_append(ctypes.byref(c), layer, k, v, dtype, tokens, *strides, slots, None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(kw):
    c, lib = _cache(**kw), qdec.lib()
    assert _append(c) == BAD
    assert lib.qpn_kv4_read(ctypes.byref(c), 0, FAKE, 3, qdec.QPN_DT_F16, FAKE, FAKE, None) == BAD
    assert lib.qpn_kv4_copy_pages(ctypes.byref(c), FAKE, FAKE, 3, None) == BAD
    assert lib.qpn_kv4_attention(ctypes.byref(c), ctypes.byref(_args()), FAKE, 1 << 40, None) == BAD


def test_append_read_and_copy_refuse_bad_arguments():
    assert qdec.lib().qpn_kv4_append(None, 0, FAKE, FAKE, 1, 1, 0, 0, 0, 0, FAKE, None) == BAD
    for kw in (dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(k=FAKE + 1), dict(v=FAKE + 1),
               dict(dtype=qdec.QPN_DT_F32), dict(dtype=0), dict(tokens=-1), dict(tokens=1 << 31),
               dict(strides=(-1, 128, 1024, 128)), dict(strides=(1024, 128, 1024, 1 << 41)), dict(slots=None),
               dict(slots=FAKE + 4)):
        assert _append(**kw) == BAD, kw
    assert _append(tokens=0, k=None, v=None, slots=None) == q.QPN_OK
    assert _append(_cache(pages=0, data=None)) == q.QPN_OK     # no slot exists
    lib, c = qdec.lib(), ctypes.byref(_cache())
    for a in ((c, -1, FAKE, 3, 1, FAKE, FAKE), (c, 2, FAKE, 3, 1, FAKE, FAKE), (c, 0, None, 3, 1, FAKE, FAKE),
              (c, 0, FAKE + 4, 3, 1, FAKE, FAKE), (c, 0, FAKE, -1, 1, FAKE, FAKE), (c, 0, FAKE, 3, 4, FAKE, FAKE),
              (c, 0, FAKE, 3, 1, None, FAKE), (c, 0, FAKE, 3, 1, FAKE, FAKE + 8)):
        assert lib.qpn_kv4_read(*a, None) == BAD
    assert lib.qpn_kv4_read(c, 0, None, 0, 1, None, None, None) == q.QPN_OK
    for a in ((c, None, FAKE, 3), (c, FAKE, None, 3), (c, FAKE + 2, FAKE, 3), (c, FAKE, FAKE, -1), (c, FAKE, FAKE, 1 << 31)):
        assert lib.qpn_kv4_copy_pages(*a, None) == BAD
    assert lib.qpn_kv4_copy_pages(c, None, None, 0, None) == q.QPN_OK


def _args(**kw):
    a = qdec.qpn_kv4_attention_args(q=FAKE, out=FAKE, lse=FAKE, table=FAKE, kv_len=FAKE, q_start=FAKE,
                                    q_token_stride=40 * 128, q_head_stride=128, table_stride=16,
                                    dtype=qdec.QPN_DT_F16, layer=1, heads=40, batch=3, rows=24, max_q_len=8,
                                    max_kv_len=1000, window=0, scale=0.1, reserved=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _attention(ws=FAKE, ws_bytes=1 << 40, cache=None, **kw):
    c = _cache() if cache is None else cache
    return qdec.lib().qpn_kv4_attention(ctypes.byref(c), ctypes.byref(_args(**kw)), ws, ws_bytes, None)


def test_attention_refuses_bad_arguments():
    lib = qdec.lib()
    assert lib.qpn_kv4_attention(None, ctypes.byref(_args()), FAKE, 1 << 40, None) == BAD
    assert lib.qpn_kv4_attention(ctypes.byref(_cache()), None, FAKE, 1 << 40, None) == BAD
    for kw in (dict(q=None), dict(q=FAKE + 1), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(table=None),
               dict(table=FAKE + 2), dict(kv_len=None), dict(kv_len=FAKE + 1), dict(q_start=FAKE + 2),
               dict(q_token_stride=-1), dict(q_head_stride=1 << 41), dict(table_stride=-1),
               dict(table_stride=15), dict(dtype=qdec.QPN_DT_F32), dict(dtype=0), dict(layer=-1), dict(layer=2),
               dict(heads=0), dict(heads=12), dict(heads=-8), dict(batch=-1), dict(batch=65537), dict(rows=-1),
               dict(batch=0), dict(max_q_len=-1), dict(max_q_len=0), dict(max_q_len=65537), dict(max_kv_len=-1),
               dict(max_kv_len=(1 << 30) + 1), dict(window=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(reserved=1), dict(q_start=None, rows=23),
               dict(ws=None), dict(ws=FAKE + 8)):
        assert _attention(**kw) == BAD, kw
    assert _attention(ws_bytes=10) == SMALL
    assert _attention(rows=1 << 20, q_start=FAKE) == UNSUPPORTED
    assert _attention(batch=0, rows=0, q=None, out=None, kv_len=None) == q.QPN_OK
    assert _attention(rows=0, q=None, out=None) == q.QPN_OK


def test_attention_workspace():
    c = _cache()
    need = qdec.qpn_kv4_attention_workspace_bytes(c, _args())
    # pointers do not matter, and one byte less is too little
    assert need == qdec.qpn_kv4_attention_workspace_bytes(c, _args(q=None, out=None, table=None, kv_len=None))
    assert need > 0 and _attention(ws_bytes=need - 1) == SMALL
    assert qdec.qpn_kv4_attention_workspace_bytes(c, _args(rows=0)) == 0
    assert qdec.qpn_kv4_attention_workspace_bytes(c, _args(heads=7)) == 0


def _vargs(**kw):
    a = qdec.qpn_verify_args(target=FAKE, draft=FAKE, draft_tokens=FAKE, num_draft=FAKE, temperature=FAKE, u_accept=FAKE,
                             u_sample=FAKE, tokens=FAKE, accepted=FAKE, logprobs=FAKE, target_batch_stride=800,
                             target_row_stride=100, draft_batch_stride=700, draft_row_stride=100, dtype=qdec.QPN_DT_F16,
                             probabilities=0, batch=2, drafts=7, vocab=100, reserved=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _verify(ws=FAKE, ws_bytes=1 << 40, **kw):
    return qdec.lib().qpn_verify(ctypes.byref(_vargs(**kw)), ws, ws_bytes, None)


def test_verify_refuses_bad_arguments():
    assert qdec.lib().qpn_verify(None, FAKE, 1 << 40, None) == BAD
    for kw in (dict(target=None), dict(target=FAKE + 1), dict(draft=FAKE + 1), dict(draft_tokens=None),
               dict(draft_tokens=FAKE + 2), dict(num_draft=FAKE + 2), dict(temperature=FAKE + 2), dict(u_accept=None),
               dict(u_sample=None), dict(u_sample=FAKE + 1), dict(tokens=None), dict(accepted=None),
               dict(accepted=FAKE + 2), dict(logprobs=FAKE + 2), dict(target_batch_stride=-1),
               dict(target_row_stride=1 << 41), dict(draft_row_stride=-1), dict(dtype=0), dict(dtype=4),
               dict(probabilities=2), dict(probabilities=1), dict(probabilities=1, dtype=qdec.QPN_DT_F32),
               dict(dtype=qdec.QPN_DT_F32, target=FAKE + 2), dict(batch=-1), dict(batch=65537), dict(drafts=-1),
               dict(drafts=65), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(reserved=3), dict(ws=None),
               dict(ws=FAKE + 4)):
        assert _verify(**kw) == BAD, kw
    need = qdec.qpn_verify_workspace_bytes(2, 7, 100)
    assert need > 0 and _verify(ws_bytes=need - 1) == SMALL
    assert _verify(batch=0, target=None, tokens=None) == q.QPN_OK
    assert qdec.qpn_verify_workspace_bytes(65536, 64, 1 << 24) == 0   # more workgroups than a launch takes
    assert qdec.qpn_verify_workspace_bytes(2, 65, 100) == 0


# ---------------------------------------------------------------- the torch layer's own checks

def test_torch_layer_refuses_cpu_tensors_and_bad_caches():
    with pytest.raises(ValueError):
        qd.KV4Cache(4, 24, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        qd.KV4Cache(4, 16, 2, 64, k_scale=0.0, device="cpu")
    with pytest.raises(ValueError):
        qd.KV4Cache(4, 16, 2, 64, layers=3, v_scale=[1.0, 1.0], device="cpu")
    with pytest.raises(ValueError):
        qd.KV4Cache.wrap(torch.zeros((1, 2, 100), dtype=torch.uint8), 16, 2, 64)
    cache = qd.KV4Cache(4, 16, 2, 64, layers=2, k_scale=[0.5, 0.25], device="cpu")
    assert cache.k_scale == (0.5, 0.25) and cache.layers == 2
    with pytest.raises(ValueError, match="layer"):
        cache.desc(2)
    with pytest.raises(ValueError, match="CUDA"):
        cache.desc(1)
    x = torch.zeros((3, 2, 64), dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        qd.kv4_append(cache, x, x, slots)
    with pytest.raises(ValueError, match="CUDA"):
        qd.kv4_read(cache, slots)
    with pytest.raises(ValueError):
        qd.kv4_read(cache, slots, dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        qd.kv4_copy_pages(cache, slots.int(), slots.int())
    with pytest.raises(ValueError, match="CUDA"):
        qd.kv4_attention(x, cache, slots.int().view(3, 1), slots.int())
    with pytest.raises(ValueError, match="CUDA"):
        qd.verify_drafts(torch.zeros((1, 2, 5)), slots.int()[:1].view(1, 1), torch.zeros(1, 1), torch.zeros(1))
