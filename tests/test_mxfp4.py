"""CPU tests of the MXFP4 operators: the definition in oracle/mxfp4.py against
the formats' tables and exact rational arithmetic, and the argument checks of
the C entry points (no GPU is used; device addresses are fake and never
dereferenced)."""
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from oracle import mxfp4 as mx
from register_lds_tiled_amd import binding as b

F = 0x10000000
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- the definition --------------------------------------------------------

def test_element_table():
    """sign, exponent of bias 1, mantissa: every code's value from its fields."""
    for code in range(16):
        s, e, m = code >> 3, (code >> 1) & 3, code & 1
        v = Fraction(m, 2) if e == 0 else (1 + Fraction(m, 2)) * Fraction(2) ** (e - 1)
        assert Fraction(float(mx.element(code))) == (-v if s else v)
    assert np.isnan(mx.scale(255)) and mx.scale(127) == 1.0 and mx.scale(0) == 2.0 ** -127


def test_nearest_code_exhaustive():
    """Every multiple of 1/64 up to 8, both signs, against the nearest of the
    eight magnitudes by exact comparison, ties to the even code."""
    for n in range(0, 8 * 64 + 1):
        v = Fraction(n, 64)
        dist = [abs(v - Fraction(float(x))) for x in mx.MAGNITUDES]
        best = [c for c in range(8) if dist[c] == min(dist)]
        want = best[0] if len(best) == 1 else [c for c in best if c % 2 == 0][0]
        assert mx.nearest_code(float(v)) == want, v
        assert mx.nearest_code(-float(v)) == want + 8, v
    assert mx.nearest_code(-0.0) == 8 and mx.nearest_code(1e30) == 7


def test_quantize_rule():
    """The scale's exponent by exact integer logarithm; the error of an element
    that is not cut off at most half a step; zeros, NaN and infinities."""
    rng = np.random.default_rng(1)
    X = rng.standard_normal((40, 75)) * np.exp2(rng.integers(-130, 120, (40, 1)))
    X[3] = 0.0
    X[4, 40] = np.nan
    X[5, 70] = -np.inf
    codes, byte = mx.quantize(X)
    assert byte.shape == (40, 3) and codes.shape == X.shape
    Y = mx.dequantize(codes, byte)
    for r in range(40):
        for blk in range(3):
            x = X[r, 32 * blk:32 * blk + 32]
            if not np.isfinite(x).all():
                assert byte[r, blk] == 255
                continue
            top = Fraction(float(np.abs(x).max()))
            e = -127
            if top:
                k = top.numerator.bit_length() - top.denominator.bit_length()
                k -= Fraction(2) ** k > top
                e = max(k - 2, -127)
            assert byte[r, blk] == e + 127
            s = Fraction(2) ** e
            for v, y in zip(x, Y[r, 32 * blk:32 * blk + 32]):
                a = abs(Fraction(float(v))) / s
                step = Fraction(1, 2) if a < 2 else 1 if a < 4 else 2
                err = abs(Fraction(float(v)) - Fraction(float(y))) / s
                assert err <= step / 2 or (a > 6 and abs(Fraction(float(y))) / s == 6)
    assert (byte[3] == 0).all() and byte[4, 1] == 255 and byte[5, 2] == 255
    assert byte[4, 0] != 255 and byte[5, 0] != 255


def test_pack_round_trip():
    rng = np.random.default_rng(2)
    for C in (1, 2, 31, 33):
        codes = rng.integers(0, 16, (5, C)).astype(np.uint8)
        assert np.array_equal(mx.unpack(mx.pack(codes, ld=40, fill=0xFF), C), codes)


# ---- refusals --------------------------------------------------------------

X, Q, S, QT, ST, Y = (F + (i << 24) for i in range(6))


@pytest.mark.parametrize("t,size", [("f32", 4), ("bf16", 2), ("f16", 2)])
def test_quantize_refusals(t, size):
    fn = getattr(b, f"gemm_mxfp4_quantize_{t}")
    f = lambda *a: fn(*a, 0, check=False)  # noqa: E731
    assert f(-1, 64, X, 64, Q, 32, S, 2, 0, 0, 0, 0) == b.SGEMM_EINVAL_DIM
    assert f(64, -1, X, 64, Q, 32, S, 2, 0, 0, 0, 0) == b.SGEMM_EINVAL_DIM
    assert f(4, 65, X, 64, Q, 33, S, 3, 0, 0, 0, 0) == b.SGEMM_EINVAL_LD
    assert f(4, 65, X, 65, Q, 32, S, 3, 0, 0, 0, 0) == b.SGEMM_EINVAL_LD    # 33 bytes of codes
    assert f(4, 65, X, 65, Q, 33, S, 2, 0, 0, 0, 0) == b.SGEMM_EINVAL_LD    # 3 scales
    assert f(65, 4, X, 4, 0, 0, 0, 0, QT, 32, ST, 3) == b.SGEMM_EINVAL_LD
    assert f(65, 4, X, 4, 0, 0, 0, 0, QT, 33, ST, 2) == b.SGEMM_EINVAL_LD
    assert f(4, 64, X, 64, 0, 0, 0, 0, 0, 0, 0, 0) == b.SGEMM_EINVAL_PTR    # nothing asked for
    assert f(4, 64, 0, 64, Q, 32, S, 2, 0, 0, 0, 0) == b.SGEMM_EINVAL_PTR
    assert f(4, 64, X, 64, Q, 32, 0, 2, 0, 0, 0, 0) == b.SGEMM_EINVAL_PTR   # half a pair
    assert f(4, 64, X, 64, 0, 32, S, 2, 0, 0, 0, 0) == b.SGEMM_EINVAL_PTR
    assert f(4, 64, X, 64, Q, 32, S, 2, QT, 2, 0, 1) == b.SGEMM_EINVAL_PTR
    assert f(4, 64, X, 64, Q, 32, S, 2, 0, 2, ST, 1) == b.SGEMM_EINVAL_PTR
    # an output on the input's last byte, or on another output
    last = X + 4 * 64 * size - 1
    assert f(4, 64, X, 64, last, 32, S, 2, 0, 0, 0, 0) == b.SGEMM_EALIAS
    assert f(4, 64, X, 64, Q, 32, last, 2, 0, 0, 0, 0) == b.SGEMM_EALIAS
    assert f(4, 64, X, 64, Q, 32, Q + 127, 2, 0, 0, 0, 0) == b.SGEMM_EALIAS
    assert f(4, 64, X, 64, Q, 48, Q + 32, 48, 0, 0, 0, 0) == b.SGEMM_EALIAS  # scales between rows
    assert f(4, 64, X, 64, Q, 32, S, 2, S + 7, 2, ST, 1) == b.SGEMM_EALIAS
    assert f(4, 64, X, 64, Q, 32, S, 2, QT, 2, QT + 127, 1) == b.SGEMM_EALIAS
    # an extent past the end of the address space
    assert f(4, 64, (1 << 64) - 64, 64, Q, 32, S, 2, 0, 0, 0, 0) == b.SGEMM_EINVAL_DIM
    # nothing to do
    assert f(0, 64, 0, 64, 0, 0, 0, 0, 0, 0, 0, 0) == b.SGEMM_OK
    assert f(4, 0, 0, 1, Q, 1, S, 1, QT, 2, ST, 1) == b.SGEMM_OK


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_dequantize_refusals(t):
    fn = getattr(b, f"gemm_mxfp4_dequantize_{t}")
    f = lambda *a: fn(*a, 0, check=False)  # noqa: E731
    assert f(-1, 64, Q, 32, S, 2, Y, 64) == b.SGEMM_EINVAL_DIM
    assert f(4, 65, Q, 32, S, 3, Y, 65) == b.SGEMM_EINVAL_LD
    assert f(4, 65, Q, 33, S, 2, Y, 65) == b.SGEMM_EINVAL_LD
    assert f(4, 65, Q, 33, S, 3, Y, 64) == b.SGEMM_EINVAL_LD
    for a in ((0, S, Y), (Q, 0, Y), (Q, S, 0)):
        assert f(4, 64, a[0], 32, a[1], 2, a[2], 64) == b.SGEMM_EINVAL_PTR
    assert f(4, 64, Q, 32, S, 2, Q + 127, 64) == b.SGEMM_EALIAS
    assert f(4, 64, Q, 32, S, 2, S + 7, 64) == b.SGEMM_EALIAS
    assert f(0, 64, 0, 32, 0, 2, 0, 64) == b.SGEMM_OK


@pytest.mark.parametrize("out,size", [("f32", 4), ("bf16", 2)])
def test_product_refusals(out, size):
    fn = getattr(b, f"gemm_mxfp4_{out}")
    f = lambda *a: fn(*a, 0, check=False)  # noqa: E731
    A, SA, B, SB, C = Q, S, QT, ST, Y
    assert f(-1, 4, 64, A, 32, SA, 2, B, 32, SB, 2, C, 4) == b.SGEMM_EINVAL_DIM
    assert f(4, -1, 64, A, 32, SA, 2, B, 32, SB, 2, C, 4) == b.SGEMM_EINVAL_DIM
    assert f(4, 4, -1, A, 32, SA, 2, B, 32, SB, 2, C, 4) == b.SGEMM_EINVAL_DIM
    assert f(2**31 - 1, 2**31 - 1, 1, A, 1, SA, 1, B, 1, SB, 1, C, 2**31 - 1) == b.SGEMM_EINVAL_DIM
    assert f(4, 4, 65, A, 32, SA, 3, B, 33, SB, 3, C, 4) == b.SGEMM_EINVAL_LD
    assert f(4, 4, 65, A, 33, SA, 2, B, 33, SB, 3, C, 4) == b.SGEMM_EINVAL_LD
    assert f(4, 4, 65, A, 33, SA, 3, B, 32, SB, 3, C, 4) == b.SGEMM_EINVAL_LD
    assert f(4, 4, 65, A, 33, SA, 3, B, 33, SB, 2, C, 4) == b.SGEMM_EINVAL_LD
    assert f(4, 5, 64, A, 32, SA, 2, B, 32, SB, 2, C, 4) == b.SGEMM_EINVAL_LD
    for i in range(5):
        a = [A, SA, B, SB, C]
        a[i] = 0
        assert f(4, 4, 64, a[0], 32, a[1], 2, a[2], 32, a[3], 2, a[4], 4) == b.SGEMM_EINVAL_PTR
    for p, n in ((A, 128), (SA, 8), (B, 128), (SB, 8)):
        assert f(4, 4, 64, A, 32, SA, 2, B, 32, SB, 2, p + n - 1, 4) == b.SGEMM_EALIAS
        assert f(4, 4, 64, A, 32, SA, 2, B, 32, SB, 2, p - 16 * size + 1, 4) == b.SGEMM_EALIAS
    assert f(0, 4, 64, 0, 32, 0, 2, 0, 32, 0, 2, 0, 4) == b.SGEMM_OK
    assert f(4, 0, 64, 0, 32, 0, 2, 0, 32, 0, 2, 0, 1) == b.SGEMM_OK


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_weight_product_refusals(t):
    fn = getattr(b, f"gemm_{t}_mxfp4_f32")
    f = lambda *a: fn(*a, 0, check=False)  # noqa: E731
    A, B, SB, C = X, Q, S, Y
    assert f(-1, 4, 64, A, 64, B, 32, SB, 2, C, 4) == b.SGEMM_EINVAL_DIM
    assert f(4, 4, 65, A, 64, B, 33, SB, 3, C, 4) == b.SGEMM_EINVAL_LD
    assert f(4, 4, 65, A, 65, B, 32, SB, 3, C, 4) == b.SGEMM_EINVAL_LD
    assert f(4, 4, 65, A, 65, B, 33, SB, 2, C, 4) == b.SGEMM_EINVAL_LD
    assert f(4, 5, 64, A, 64, B, 32, SB, 2, C, 4) == b.SGEMM_EINVAL_LD
    for i in range(4):
        a = [A, B, SB, C]
        a[i] = 0
        assert f(4, 4, 64, a[0], 64, a[1], 32, a[2], 2, a[3], 4) == b.SGEMM_EINVAL_PTR
    for p, n in ((A, 512), (B, 128), (SB, 8)):
        assert f(4, 4, 64, A, 64, B, 32, SB, 2, p + n - 1, 4) == b.SGEMM_EALIAS
    assert f(0, 4, 64, 0, 64, 0, 32, 0, 2, 0, 4) == b.SGEMM_OK


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="GPU"):
        b.gemm_mxfp4_quantize_f32(4, 64, torch.zeros(4, 64), 64, Q, 32, S, 2, stream=0)
    with pytest.raises(TypeError):
        b.gemm_mxfp4_quantize_f32(4, 64, "no address", 64, Q, 32, S, 2, stream=0)


HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/llvm/bin/clang"

DRIVER = r"""
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include "sgemm.h"
static int bad;
#define EXPECT(call, want) do { int r_ = (call); if (r_ != (want)) { \
    printf("line %d: %d, expected %d\n", __LINE__, r_, (want)); bad = 1; } } while (0)
int main(void) {
    char *x = (char *)0x10000000, *q = x + (1 << 24), *s = q + (1 << 24), *y = s + (1 << 24);
    char *top = (char *)(UINTPTR_MAX - 63);
    const int m = INT_MAX;
    /* extents past the address space, at the largest dimensions */
    EXPECT(gemm_mxfp4_quantize_f32(m, m, top, m, q, m, s, m, 0, 0, 0, 0, 0), SGEMM_EINVAL_DIM);
    EXPECT(gemm_mxfp4_quantize_bf16(m, m, x, m, top, m, s, m, 0, 0, 0, 0, 0), SGEMM_EINVAL_DIM);
    EXPECT(gemm_mxfp4_quantize_f16(m, m, x, m, 0, 0, 0, 0, q, m, top, m, 0), SGEMM_EINVAL_DIM);
    EXPECT(gemm_mxfp4_dequantize_f32(m, m, q, m, s, m, top, m, 0), SGEMM_EINVAL_DIM);
    EXPECT(gemm_mxfp4_dequantize_bf16(m, m, q, m, s, m, q, m, 0), SGEMM_EALIAS);
    EXPECT(gemm_mxfp4_dequantize_f16(INT_MIN, m, q, m, s, m, y, m, 0), SGEMM_EINVAL_DIM);
    EXPECT(gemm_mxfp4_f32(m, m, m, q, m, s, m, q, m, s, m, (float *)y, m, 0), SGEMM_EINVAL_DIM);
    EXPECT(gemm_mxfp4_bf16(1, 1, m, q, m, s, m, q, m, s, m, q, m, 0), SGEMM_EALIAS);
    EXPECT(gemm_bf16_mxfp4_f32(1, m, m, top, m, q, m, s, m, (float *)y, m, 0), SGEMM_EINVAL_DIM);
    EXPECT(gemm_f16_mxfp4_f32(1, m, m, x, m, top, m, s, m, (float *)y, m, 0), SGEMM_EINVAL_DIM);
    return bad;
}
"""

STUBS = r"""
#include "mxfp4.h"
namespace sgemm {
hipError_t launch_mx_quantize(const MxQuantArgs&, MxType, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_mx_dequantize(const MxDequantArgs&, MxType, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_mx_gemm(const MxGemmArgs&, MxType, hipStream_t) { return hipErrorInvalidDevice; }
hipError_t launch_mx_wgemm(const MxGemmArgs&, MxType, hipStream_t) { return hipErrorInvalidDevice; }
}
"""


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG) and shutil.which("gcc")),
                    reason="ROCm toolchain missing")
def test_argument_checks_under_sanitizers(tmp_path):
    """The argument checks at extreme dimensions and addresses, built for the
    host with AddressSanitizer and UndefinedBehaviorSanitizer; no launch."""
    csrc = os.path.join(ROOT, "register_lds_tiled_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc]
    host = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g", "-fPIC",
            "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
            "-Xarch_host", "-fno-sanitize-recover=all"]
    (tmp_path / "drv.c").write_text(DRIVER)
    (tmp_path / "stubs.hip").write_text(STUBS)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-3000:]}\n{r.stderr[-3000:]}"

    run([HIPCC, *host, *inc, "-c", os.path.join(csrc, "mxfp4_api.hip"), "-o", str(tmp_path / "api.o")])
    run([HIPCC, *host, *inc, "-c", str(tmp_path / "stubs.hip"), "-o", str(tmp_path / "stubs.o")])
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    run([CLANG, "-O1", "-g", *san, *inc, "-c", str(tmp_path / "drv.c"), "-o", str(tmp_path / "drv.o")])
    run([CLANG + "++", *san, *(str(tmp_path / n) for n in ("drv.o", "api.o", "stubs.o")),
         "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", str(tmp_path / "drv")])
    r = subprocess.run([str(tmp_path / "drv")], capture_output=True, text=True,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
