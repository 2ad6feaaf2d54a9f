"""CPU tests of what the 8-bit integer and gated entry points launch: the kernels
chosen and the sizes of their grids, up to the largest dimensions an int holds,
against the stand-in runtime of test_mxfp4_launch.py; and their argument checks
under AddressSanitizer and UndefinedBehaviorSanitizer.  No GPU is used; device
addresses are fake."""
import ctypes
import os
import subprocess

import pytest

from register_lds_tiled_amd import binding as b
from tests.test_mxfp4_launch import RUNTIME

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "register_lds_tiled_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang"
SOURCES = ["layer_api", "i8_cast", "i8_gemm", "i8_gated", "gated_gemm", "gated_backward", "layer_rows"]
TOP = 2 ** 31 - 1

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="ROCm toolchain missing")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    flags = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC", "-w",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    jobs = [subprocess.Popen([HIPCC, *flags, "-c", os.path.join(CSRC, n + ".hip"), "-o", str(d / (n + ".o"))],
                             stdout=subprocess.DEVNULL, stderr=subprocess.PIPE) for n in SOURCES]
    for j in jobs:
        log = j.communicate()[1]
        assert j.returncode == 0, log.decode(errors="replace")[-2000:]
    objs = [str(d / (n + ".o")) for n in SOURCES]
    undefined = subprocess.run(["nm", "-u", *objs], capture_output=True, text=True, check=True).stdout.split()
    images = sorted({s for s in undefined if s.startswith("__hip_fatbin")})
    (d / "runtime.cpp").write_text(
        RUNTIME + 'extern "C" void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}\n'
        + "".join(f'extern "C" {{ char {s}[16]; }}\n' for s in images))
    so = d / "launches.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-w", "-I/opt/rocm/include", "-Wl,-Bsymbolic",
                    str(d / "runtime.cpp"), *objs, "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    i, p = ctypes.c_int, ctypes.c_void_p
    for t in ("f32", "bf16", "f16"):
        getattr(lib, f"gemm_i8_quantize_{t}").argtypes = [i, i, p, i, p, i, p, p]
        getattr(lib, f"gemm_i8_dequantize_{t}").argtypes = [i, i, p, i, p, p, i, p]
        getattr(lib, f"gemm_i8_{t}").argtypes = [i, i, i, p, i, p, p, i, p, p, i, p]
    for t in ("bf16", "f16"):
        getattr(lib, f"gemm_i8_gated_{t}").argtypes = [i, i, i] + [p, i, p] * 3 + [p, i, i, p]
        getattr(lib, f"gemm_gated_{t}").argtypes = [i, i, i] + [p, i] * 6 + [i, p]
        getattr(lib, f"gemm_gated_backward_{t}").argtypes = [i, i, i] + [p, i] * 11 + [i, p]
    lib.record_kernel.restype = lib.record_name.restype = ctypes.c_char_p
    lib.record_groups.restype = lib.record_threads.restype = ctypes.c_ulonglong
    return lib


AT = [0x100_0000_0000_0000 * n for n in range(1, 13)]     # far apart


def ld_of(n, size, pad):
    return -(-n // (16 // size)) * (16 // size) + pad


def i8(lib, t, M, N, K, pad=0):
    lib.record_count()
    ld = ld_of(K, 1, pad)
    return getattr(lib, f"gemm_i8_{t}")(M, N, K, AT[0], ld, AT[1], AT[2], ld, AT[3], AT[4], N, None)


def i8_gated(lib, t, M, N, K, pad=0):
    lib.record_count()
    ld = ld_of(K, 1, pad)
    return getattr(lib, f"gemm_i8_gated_{t}")(M, N, K, AT[0], ld, AT[1], AT[2], ld, AT[3], AT[4], ld, AT[5], AT[6], N, 2, None)


def gated(lib, t, M, N, K, pad=0):
    lib.record_count()
    ld = ld_of(K, 2, pad)
    return getattr(lib, f"gemm_gated_{t}")(M, N, K, AT[0], ld, AT[1], ld, AT[2], ld, None, 0, None, 0, AT[3], N, 2, None)


def backward(lib, t, M, N, K, pad=0, dx=True, dw=True):
    lib.record_count()
    n, k = min(TOP, ld_of(N, 2, pad)), min(TOP, ld_of(K, 2, pad))
    none = (None, 0)
    return getattr(lib, f"gemm_gated_backward_{t}")(
        M, N, K, AT[0], k, AT[1], k, AT[2], k, AT[3], n, AT[4], n, AT[5], n, AT[6], n, AT[7], n,
        *((AT[8], k) if dx else none), *((AT[9], k) if dw else none), *((AT[10], k) if dw else none), 2, None)


WIDE = 64 * (2 ** 24 - 1)     # the widest C that one workgroup of 256 threads per 64 x 64 tile covers


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("call,t", [(i8, "f32"), (i8, "f16"), (i8_gated, "bf16"), (gated, "bf16"), (gated, "f16")])
def test_products_launch_or_are_refused(lib, call, t, pad):
    """The largest C of any form, and beyond it SGEMM_EINVAL_DIM without a launch."""
    for M, N in ((1, 1), (16, 2 ** 26), (16, 2 ** 26 + 1), (32, 2 ** 26 + 64), (64, 2 ** 26), (1, WIDE), (WIDE, 1), (WIDE, 64),
                 (64, WIDE), (33, WIDE), (64 * 4095, 64 * 4096)):
        for K in (7, 16, 64, 128):
            assert call(lib, t, M, N, K, pad) == b.SGEMM_OK, (M, N, K, lib.record_kernel(), lib.record_groups(), lib.record_threads())
            assert lib.record_count() == 1
    for M, N in ((1, WIDE + 1), (1, TOP), (16, TOP), (WIDE + 1, 1), (TOP, 1), (65, WIDE), (TOP, TOP)):
        assert call(lib, t, M, N, 64, pad) == b.SGEMM_EINVAL_DIM, (M, N)
        assert lib.record_count() == 0


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_gradients_launch_or_are_refused(lib, t, pad):
    half = 64 * (2 ** 23 - 1)     # two such results in one launch
    for M, N, K in ((1, 1, 1), (1, half, 1), (WIDE, 1, 1), (1, 1, half), (64 * 4095, 64 * 4096, 64),
                    (64, 64 * 2047, 64 * 4096), (64 * 4095, 64, 64 * 4096), (300, 500, 700)):
        for dx, dw in ((True, True), (True, False), (False, True), (False, False)):
            assert backward(lib, t, M, N, K, pad, dx, dw) == b.SGEMM_OK, (M, N, K, lib.record_kernel(), lib.record_groups())
            assert lib.record_count() == 1 + dx + dw
    for M, N, K in ((1, WIDE + 1, 1), (TOP, 1, 1), (65, WIDE, 1), (1, half + 1, 1), (1, 1, half + 1), (1, WIDE, 1)):
        assert backward(lib, t, M, N, K, pad) == b.SGEMM_EINVAL_DIM
        assert lib.record_count() == 0
    # only what is asked has to fit
    assert backward(lib, t, 1, 65, WIDE, pad, True, False) == b.SGEMM_OK and lib.record_count() == 2
    assert backward(lib, t, 1, 65, WIDE, pad, True, True) == b.SGEMM_EINVAL_DIM and lib.record_count() == 0
    assert backward(lib, t, 1, WIDE, 1, pad, True, False) == b.SGEMM_OK and lib.record_count() == 2
    # empty sums: one launch each
    n, k = 64, 64
    fn = getattr(lib, f"gemm_gated_backward_{t}")
    none = (None, 64)
    assert fn(0, n, k, *none * 3, *none * 5, None, 0, AT[9], k, AT[10], k, 2, None) == b.SGEMM_OK
    assert lib.record_count() == 1
    assert fn(30, 0, k, *none * 3, *none * 5, AT[8], k, None, 0, None, 0, 2, None) == b.SGEMM_OK
    assert lib.record_count() == 1


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_casts_launch(lib, t):
    for R, C in ((1, 1), (1, TOP), (TOP, 1), (TOP, 100), (TOP, 8192), (100, 100000), (2 ** 21 + 1, 5000), (1000, 2 ** 25)):
        lib.record_count()
        assert getattr(lib, f"gemm_i8_quantize_{t}")(R, C, AT[0], C, AT[3], C, AT[6], None) == b.SGEMM_OK, (R, C, lib.record_groups())
        assert getattr(lib, f"gemm_i8_dequantize_{t}")(R, C, AT[3], C, AT[6], AT[0], C, None) == b.SGEMM_OK, (R, C, lib.record_groups())
        assert lib.record_count() == 2


def test_every_kernel_is_launched_by_some_call(lib):
    """The library holds no kernel of these families that no call reaches."""
    known = {lib.record_name(i) for i in range(lib.record_known())}
    assert len(known) > 40
    reached = set()

    def call(status):
        assert status == b.SGEMM_OK
        reached.add(lib.record_kernel())

    for M in (1, 17, 33, 64, 100, 300, 600, 1500, 4200):
        for N in (5, 64, 1000, 2048, 4096, 8192, 20000):
            for K in (3, 200, 1024):
                for pad in (0, 1):
                    for t in ("f32", "bf16", "f16"):
                        call(i8(lib, t, M, N, K, pad))
                    for t in ("bf16", "f16"):
                        call(i8_gated(lib, t, M, N, K, pad))
                        call(gated(lib, t, M, N, K, pad))
                        for dx, dw in ((True, False), (False, True), (False, False)):
                            call(backward(lib, t, M, N, K, pad, dx, dw))
    for t in ("bf16", "f16"):
        call(backward(lib, t, 4200, 64, 4096, 0, True, False))
        call(backward(lib, t, 4200, 1024, 8192, 0, True, False))
        call(i8_gated(lib, t, 4200, 4096, 2048, 0))
    for t in ("f32", "bf16", "f16"):
        call(i8(lib, t, 4200, 8192, 2048, 0))
    for t in ("f32", "bf16", "f16"):
        for R, C in ((1, 100), (1, 8192), (1000, 8192), (1000, 4000), (1000, 100)):
            call(getattr(lib, f"gemm_i8_quantize_{t}")(R, C, AT[0], C, AT[3], C, AT[6], None))
            call(getattr(lib, f"gemm_i8_dequantize_{t}")(R, C, AT[3], C, AT[6], AT[0], C, None))
    assert known == reached, sorted(k.decode() for k in known - reached)


DRIVER = r"""
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include "sgemm.h"
static int bad;
#define IS(call, want) do { int got = (call); if (got != (want)) { printf("%d: %s gave %d\n", __LINE__, #call, got); bad = 1; } } while (0)
int main(void) {
    const int T = INT_MAX;
    char *p = (char *)(uintptr_t)0x1000, *q = (char *)(uintptr_t)(UINTPTR_MAX - 64), *n = 0;
    float *s = (float *)(uintptr_t)0x7000000000000000;
    IS(gemm_i8_quantize_f32(INT_MIN, T, p, T, p, T, s, n), SGEMM_EINVAL_DIM);
    IS(gemm_i8_quantize_f32(T, T, p, INT_MIN, p, T, s, n), SGEMM_EINVAL_LD);
    IS(gemm_i8_quantize_f32(T, T, q, T, p, T, s, n), SGEMM_EINVAL_DIM);
    IS(gemm_i8_quantize_bf16(T, T, p, T, p, T, s, n), SGEMM_EALIAS);
    IS(gemm_i8_dequantize_f16(T, T, p, T, s, q, T, n), SGEMM_EINVAL_DIM);
    IS(gemm_i8_dequantize_f16(T, T, p, T, s, p, INT_MIN, n), SGEMM_EINVAL_LD);
    IS(gemm_i8_f32(T, T, T, p, T, s, p, T, s, (float *)p, T, n), SGEMM_EINVAL_DIM);
    IS(gemm_i8_bf16(T, T, 131071, p, T, s, p, T, s, p, T, n), SGEMM_EINVAL_DIM);
    IS(gemm_i8_f16(4, 4, 131071, q, T, s, p, T, s, p, T, n), SGEMM_EINVAL_DIM);
    IS(gemm_i8_f16(4, 4, 131071, p, T, s, p, T, s, p, T, n), SGEMM_EALIAS);
    IS(gemm_i8_gated_bf16(4, 4, 4, p, T, s, p, T, s, q, T, s, (char *)s - 4096, T, 4, n), SGEMM_EINVAL_DIM);
    IS(gemm_i8_gated_bf16(4, 4, 4, p, T, s, p, T, s, p, T, s, p, T, INT_MAX, n), SGEMM_EINVAL_ACT);
    IS(gemm_gated_f16(T, T, T, p, T, p, T, p, T, n, 0, n, 0, p, T, INT_MIN, n), SGEMM_EINVAL_ACT);
    IS(gemm_gated_f16(T, T, T, p, T, p, T, p, T, n, 0, n, 0, p, T, 0, n), SGEMM_EINVAL_DIM);
    IS(gemm_gated_f16(T, 1, T, p, T, p, T, p, T, n, 0, n, 0, p, T, 0, n), SGEMM_EINVAL_DIM);
    IS(gemm_gated_bf16(64, 1, T, p, T, p, T, p, T, n, 0, n, 0, p, T, 0, n), SGEMM_EALIAS);
    IS(gemm_gated_backward_bf16(T, T, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, 0, n), SGEMM_EINVAL_DIM);
    IS(gemm_gated_backward_bf16(9, 9, T / 8, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, p, T, 0, n), SGEMM_EALIAS);
    IS(gemm_gated_backward_f16(9, 9, 9, p, T, p, T, p, T, q, T, p, T, p, T, s, T, s, T, n, 0, n, 0, n, 0, 0, n), SGEMM_EINVAL_DIM);
    IS(gemm_gated_backward_f16(0, 0, T, n, T, n, T, n, T, n, 1, n, 1, n, 1, n, 1, n, 1, n, T, n, T, n, T, 0, n), SGEMM_OK);
    return bad;
}
"""
STUBS = r"""
#include "layer.h"
namespace sgemm {
hipError_t launch_i8_quantize(const I8CastArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_i8_dequantize(const I8CastArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_i8_nt(const LayerArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_i8_gated(const LayerArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_gated(const LayerArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_gated_slopes(const GateArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_gated_dx(const LayerArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_gated_dw(const LayerArgs&, Elem, hipStream_t) { return hipErrorInvalidDevice; }
}
"""


@pytest.mark.skipif(not os.path.exists(CLANG), reason="clang missing")
def test_argument_checks_under_sanitizers(tmp_path):
    """The argument checks at extreme dimensions and addresses, built for the host
    with the sanitizers; no launch."""
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    host = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g", "-fPIC", "-w",
            "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
            "-Xarch_host", "-fno-sanitize-recover=all"]
    (tmp_path / "drv.c").write_text(DRIVER)
    (tmp_path / "stubs.hip").write_text(STUBS)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-3000:]}\n{r.stderr[-3000:]}"

    run([HIPCC, *host, *inc, "-c", os.path.join(CSRC, "layer_api.hip"), "-o", str(tmp_path / "api.o")])
    run([HIPCC, *host, *inc, "-c", str(tmp_path / "stubs.hip"), "-o", str(tmp_path / "stubs.o")])
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    run([CLANG, "-O1", "-g", *san, *inc, "-c", str(tmp_path / "drv.c"), "-o", str(tmp_path / "drv.o")])
    run([CLANG + "++", *san, *(str(tmp_path / n) for n in ("drv.o", "api.o", "stubs.o")),
         "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", str(tmp_path / "drv")])
    r = subprocess.run([str(tmp_path / "drv")], capture_output=True, text=True,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
