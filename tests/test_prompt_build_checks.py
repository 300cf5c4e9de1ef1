"""Build-level checks of the prompt operators on the CPU: their sources compile
warning-free on both passes, the device code holds no packed fp32 arithmetic, no
store through the scalar data cache and no scratch memory, M0 is written only
where a load to LDS takes it, and their plans and argument checks run clean
under AddressSanitizer and UndefinedBehaviorSanitizer."""

import os
import re
import shutil
import subprocess

import pytest

from quantized_weight_skinny_amd import build as qbuild
from test_build_checks import COMMON, CSRC, HIPCC, INCLUDE, ROOT, _instructions, needs_hipcc

SOURCES = ["qpn_fp8_block.hip", "qpn_kv4_chunk.hip", "qpn_logprobs.hip", "qpn_prompt_api.hip"]


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
    assert set(SOURCES) | {"qpn_prompt_checks.cpp"} <= set(qbuild.SOURCES)


@needs_hipcc
@pytest.mark.parametrize("what,pattern", [
    ("packed fp32", r"\bv_pk_(add|mul|fma)_f32\b"),
    ("scalar stores", r"^s_(store|buffer_store|scratch_store|atomic|buffer_atomic|dcache_wb|dcache_discard)"),
])
def test_device_code_has_none_of(asm, what, pattern):
    for src, text in asm.items():
        hits = [s for s in _instructions(text) if re.search(pattern, s)]
        assert not hits, f"{src}: {what}: {hits[:5]}"


@needs_hipcc
def test_m0_belongs_to_the_loads_to_lds(asm):
    """The compiler does not track M0: each write of it stands right in front of its load."""
    for src, text in asm.items():
        ins = list(_instructions(text))
        writes = [i for i, s in enumerate(ins) if re.match(r"^\S+ m0,", s)]
        loads = [i for i, s in enumerate(ins) if "_lds_dword" in s]
        assert [i + 2 for i in writes] == loads, src
        for i in writes:
            assert ins[i].startswith("s_mov_b32 m0, s") and ins[i + 1] == "s_nop 0", (src, ins[i:i + 3])
        assert bool(writes) == (src == "qpn_fp8_block.hip")


@needs_hipcc
def test_device_code_uses_no_scratch(asm):
    kernels = 0
    for src, text in asm.items():
        vals = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)
        assert all(v == "0" for v in vals), (src, sorted(set(vals)))
        kernels += len(vals)
    assert kernels > 30


@needs_hipcc
def test_attention_keeps_two_workgroups_a_compute_unit(asm):
    """Registers and LDS leave room for the workgroups that the launch counts on."""
    found = 0
    for m in re.finditer(r"\.group_segment_fixed_size: (\d+).*?\.name:\s+\S*kv4_chunk_kernelILi(\d+)ELb.*?"
                         r"\.vgpr_count:\s+(\d+)", asm["qpn_kv4_chunk.hip"], re.S):
        lds, dim, vgprs = (int(x) for x in m.groups())
        groups = 1 if dim == 256 else 2
        assert vgprs <= 512 // groups and lds * groups <= 160 * 1024, (dim, vgprs, lds)
        found += 1
    assert found == 6


@needs_hipcc
def test_host_pass_warning_clean():
    for src in SOURCES + ["qpn_prompt_checks.cpp"]:
        res = subprocess.run([HIPCC, *COMMON, "--cuda-host-only", "-fsyntax-only", os.path.join(CSRC, src)],
                             capture_output=True, text=True, timeout=300)
        log = res.stdout + res.stderr
        assert res.returncode == 0 and "warning" not in log, f"{src}:\n{log[-4000:]}"


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_plans_and_checks_under_sanitizers(tmp_path):
    exe = tmp_path / "check_prompt"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-I", INCLUDE,
           *[os.path.join(CSRC, s) for s in ("qpn_prompt_checks.cpp", "qpn_decode_checks.cpp", "qpn_checks.cpp",
                                             "qpn_plan.cpp")],
           os.path.join(ROOT, "tests", "host", "check_prompt.cpp"), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    out = run.stdout + run.stderr
    assert run.returncode == 0 and out.startswith("ok "), out[-4000:]
    assert int(out.split()[1]) > 1000, out
