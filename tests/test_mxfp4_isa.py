"""CPU checks on the MXFP4 kernels' gfx950 code: no packed fp32, no scratch;
the tile kernels that issue their matrix instructions as inline assembly keep
the wait states the compiler does not see to; M0 is set only where a DMA
follows; the debug build poisons every kernel that reuses an LDS stage."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "register_lds_tiled_amd", "csrc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature",
         "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
         "--cuda-device-only", "-S"]
SOURCES = ["mxfp4_cast.hip", "mxfp4_gemm.hip", "mxfp4_rows.hip", "mxfp4_wgemm.hip"]
STAGED = {"mxfp4_gemm.hip": ["mx_tile_kernel", "mx_dma_kernel"], "mxfp4_rows.hip": ["mx_rows_kernel"],
          "mxfp4_wgemm.hip": ["mx_wtile_kernel", "mx_wdma_kernel"]}
POISON = "-DSGEMM_LDS_POISON"


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    d = tmp_path_factory.mktemp("isa")
    jobs = {}
    for name in SOURCES:
        for extra in ((), (POISON,)):
            out = d / (name + "".join(extra) + ".s")
            jobs[name + "".join(extra)] = (out, subprocess.Popen(
                ["/opt/rocm/bin/hipcc", *FLAGS, *extra, os.path.join(CSRC, name), "-o", str(out)],
                stdout=subprocess.DEVNULL, stderr=subprocess.PIPE))
    texts = {}
    for key, (out, proc) in jobs.items():
        log = proc.communicate()[1]
        assert proc.returncode == 0, log.decode(errors="replace")[-2000:]
        texts[key] = out.read_text()
    return texts


def functions(text, pattern):
    for name in re.findall(r"^(_Z\w*\d" + pattern + r"\w*):", text, re.M):
        start = text.index(name + ":")
        lines = [l.split(";")[0].strip() for l in text[start:text.index(".Lfunc_end", start)].splitlines()]
        yield name, [l for l in lines if l and not l.startswith(".") and not l.endswith(":")]


@pytest.mark.parametrize("name", SOURCES)
def test_no_packed_fp32_and_no_scratch(asm, name):
    assert not re.search(r"\bv_pk_(fma|mul|add)_f32\b", asm[name])
    scratch = [int(x) for x in re.findall(r"; ScratchSize: (\d+)", asm[name])]
    assert scratch and max(scratch) == 0, scratch


@pytest.mark.parametrize("name", ["mxfp4_gemm.hip", "mxfp4_wgemm.hip"])
def test_m0_only_before_a_dma(asm, name):
    lines = asm[name].splitlines()
    uses = [i for i, l in enumerate(lines) if re.search(r"\bm0\b", l) and not l.lstrip().startswith(";")]
    assert uses
    for i in uses:
        assert re.match(r"\s*s_mov_b32 m0, s\d+\s*$", lines[i]), lines[i]
        assert "ASMSTART" in lines[i - 1] and re.match(r"\s*global_load_lds_dwordx4\s", lines[i + 1])


def registers(text):
    out = set()
    for one, lo, hi in re.findall(r"\bv(\d+)\b|\bv\[(\d+):(\d+)\]", text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def wait_states(lines):
    return sum(int(l.split()[1]) + 1 for l in lines if l.startswith("s_nop"))


def test_matrix_instruction_pauses(asm):
    """Nothing but matrix instructions touches an accumulator between the first
    and the last of them; at least two wait states lie between a vector
    instruction that writes an operand, or the accumulators' clearing, and the
    matrix instruction; at least 19 between the last one and the first read of
    its result."""
    agpr = re.compile(r"\ba(\d+|\[\d+:\d+\])")
    found = 0
    for name, lines in functions(asm["mxfp4_gemm.hip"], "mx_dma_kernel"):
        found += 1
        mfma = [i for i, l in enumerate(lines) if l.startswith("v_mfma")]
        first, last = mfma[0], mfma[-1]
        for l in lines[first:last]:
            assert l.startswith("v_mfma") or not agpr.search(l), (name, l)
        zero = [i for i, l in enumerate(lines[:first]) if l.startswith("v_accvgpr")]
        assert zero and wait_states(lines[zero[-1] + 1:first]) >= 2, name
        for i in mfma:
            operands, states = registers(lines[i].split(",", 1)[1]), 0
            for l in reversed(lines[max(0, i - 3):i]):
                if states >= 2:
                    break
                if l.startswith("s_nop"):
                    states += int(l.split()[1]) + 1
                    continue
                if l.startswith("v_") and not l.startswith("v_mfma"):
                    assert not registers(l.split(None, 1)[1].split(",")[0]) & operands, (name, l, lines[i])
                states += 1
        uses = [i for i, l in enumerate(lines) if i > last and agpr.search(l)]
        assert uses and wait_states(lines[last + 1:uses[0]]) >= 19, name
    assert found >= 4


@pytest.mark.parametrize("name", list(STAGED))
def test_debug_build_poisons_staged_kernels(asm, name):
    nan = "0x7fc00000"
    assert nan not in asm[name]
    for family in STAGED[name]:
        found = list(functions(asm[name + POISON], family))
        assert found, family
        for fn, lines in found:
            assert any(nan in l for l in lines), fn
