"""Build-level checks of the decode operators on the CPU: their sources compile
warning-free on both passes, the device code holds no packed fp32 arithmetic,
no store through the scalar data cache, no M0 write, no scratch memory and no
register spills, and their plans and argument checks run clean under
AddressSanitizer and UndefinedBehaviorSanitizer."""

import os
import re
import shutil
import subprocess

import pytest

from quantized_weight_skinny_amd import build as qbuild
from test_build_checks import COMMON, CSRC, HIPCC, INCLUDE, ROOT, _instructions, needs_hipcc

SOURCES = ["qpn_kv4_attention.hip", "qpn_kv4_cache.hip", "qpn_verify.hip", "qpn_decode_api.hip"]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm")
    procs = {s: subprocess.Popen([HIPCC, *COMMON, "--cuda-device-only", "-S", os.path.join(CSRC, s), "-o",
                                  str(out / (s + ".s"))], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for s in SOURCES}
    text = {}
    for s, proc in procs.items():
        log, _ = proc.communicate(timeout=600)
        assert proc.returncode == 0 and "warning" not in log, f"{s}:\n{log[-4000:]}"
        text[s] = (out / (s + ".s")).read_text()
    return text


def test_sources_are_part_of_the_build():
    assert set(SOURCES) | {"qpn_decode_checks.cpp"} <= set(qbuild.SOURCES)


@needs_hipcc
@pytest.mark.parametrize("what,pattern", [
    ("packed fp32", r"\bv_pk_(add|mul|fma)_f32\b"),
    ("scalar stores", r"^s_(store|buffer_store|scratch_store|atomic|buffer_atomic|dcache_wb|dcache_discard)"),
    ("M0 writes", r"^\S+ m0,"),
])
def test_device_code_has_none_of(asm, what, pattern):
    for src, text in asm.items():
        hits = [s for s in _instructions(text) if re.search(pattern, s)]
        assert not hits, f"{src}: {what}: {hits[:5]}"


@needs_hipcc
def test_device_code_no_scratch_or_spills(asm):
    kernels = 0
    for src, text in asm.items():
        for key in (".private_segment_fixed_size", ".sgpr_spill_count", ".vgpr_spill_count"):
            vals = re.findall(re.escape(key) + r":\s+(\d+)", text)
            assert all(v == "0" for v in vals), (src, key, sorted(set(vals)))
        kernels += len(re.findall(r"\.private_segment_fixed_size:", text))
    assert kernels > 40


@needs_hipcc
def test_attention_keeps_its_occupancy(asm):
    """Registers and LDS leave room for the workgroups that the launch counts on."""
    text = asm["qpn_kv4_attention.hip"]
    found = 0
    for m in re.finditer(r"\.group_segment_fixed_size: (\d+).*?\.name:\s+\S*kv4_attention_kernelILi(\d+)ELi(\d+)E.*?"
                         r"\.vgpr_count:\s+(\d+)", text, re.S):
        lds, dim, nq, vgprs = (int(x) for x in m.groups())
        waves = 2 if dim == 256 or nq >= (4 if dim == 64 else 3) else 4 if nq * dim <= 128 else 3
        assert vgprs <= 512 // waves // 8 * 8, (dim, nq, vgprs)
        assert lds * waves <= 160 * 1024, (dim, nq, lds)
        found += 1
    assert found == 18


@needs_hipcc
def test_host_pass_warning_clean():
    for src in SOURCES + ["qpn_decode_checks.cpp"]:
        res = subprocess.run([HIPCC, *COMMON, "--cuda-host-only", "-fsyntax-only", os.path.join(CSRC, src)],
                             capture_output=True, text=True, timeout=300)
        log = res.stdout + res.stderr
        assert res.returncode == 0 and "warning" not in log, f"{src}:\n{log[-4000:]}"


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_plans_and_checks_under_sanitizers(tmp_path):
    exe = tmp_path / "check_decode"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-I", INCLUDE,
           *[os.path.join(CSRC, s) for s in ("qpn_decode_checks.cpp", "qpn_checks.cpp", "qpn_plan.cpp")],
           os.path.join(ROOT, "tests", "host", "check_decode.cpp"), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    out = run.stdout + run.stderr
    assert run.returncode == 0 and out.startswith("ok "), out[-4000:]
    assert int(out.split()[1]) > 1000, out
