"""GPU tests of the MXFP4 entry points against oracle/mxfp4.py (float64).

Quantising and reading back must match bit for bit: the scale is an exponent,
and rounding to a code is exact.  Products: every product of two elements with
their scales that fp32's normal range holds is exact there (at most 4 significant
bits, or 2 + 11), so C differs from the exact sum only by the additions.  The
matrix cores add 64
(16-bit A: 16 at least, and binary16 A takes two passes) products at a time into
an fp32 accumulator, and the sum over k may be split among up to 16 waves whose
parts are then added: for each output at most
    T = passes * ceil(K / step) + 2 * 16
roundings of partial sums no larger than S = sum |a b|, each off by at most
2^-23 S (truncation included), so |C - R| <= T 2^-23 S.  bfloat16 C adds half
a step, 2^-8 |R|.  Where all partial sums are multiples of 1/4 below 2^22 the
fp32 result is exact.

Bytes past the rows (padding of values and of scales, an odd row's last half
byte) hold garbage that would show: scale bytes 255, codes of 6; buffers
around outputs hold a guard pattern that must survive.
"""
import threading

import numpy as np
import pytest

from oracle import mxfp4 as mx
from register_lds_tiled_amd import binding as b

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GUARD = 0x5A
QUANT = {"f32": b.gemm_mxfp4_quantize_f32, "bf16": b.gemm_mxfp4_quantize_bf16,
         "f16": b.gemm_mxfp4_quantize_f16}
DEQUANT = {"f32": b.gemm_mxfp4_dequantize_f32, "bf16": b.gemm_mxfp4_dequantize_bf16,
           "f16": b.gemm_mxfp4_dequantize_f16}
PRODUCT = {"f32": b.gemm_mxfp4_f32, "bf16": b.gemm_mxfp4_bf16}
WPRODUCT = {"bf16": b.gemm_bf16_mxfp4_f32, "f16": b.gemm_f16_mxfp4_f32}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class Bytes:
    """rows x n bytes, ld apart, off bytes into a device buffer of `fill`,
    with 64 bytes behind."""

    def __init__(self, rows, n, ld=None, off=0, fill=GUARD, data=None):
        self.rows, self.n, self.ld, self.off = rows, n, max(1, n) if ld is None else ld, off
        self.host = np.full(off + rows * self.ld + 64, fill, dtype=np.uint8)
        if data is not None:
            self.view(self.host)[:, :n] = data
        self.dev = torch.from_numpy(self.host).to(DEV)
        self.ptr = self.dev.data_ptr() + off

    def view(self, a):
        return a[self.off:self.off + self.rows * self.ld].reshape(self.rows, self.ld)

    def get(self):
        """The rows' bytes; everything else must be as it was."""
        now = self.dev.cpu().numpy()
        out = self.view(now)[:, :self.n].copy()
        was = self.host.copy()
        self.view(was)[:, :self.n] = 0
        self.view(now)[:, :self.n] = 0
        assert np.array_equal(now, was), "bytes outside the rows were written"
        return out


def as_type(X, t):
    """X rounded to type t: (little-endian bytes R x C*size, float64 values)."""
    y = torch.from_numpy(np.ascontiguousarray(X, dtype=np.float64)).to(TORCH[t])
    raw = y.view(torch.int32 if t == "f32" else torch.int16).numpy()
    return raw.view(np.uint8).reshape(X.shape[0], -1), y.double().numpy()


def same(got, want, what):
    if not np.array_equal(got, want):
        bad = np.argwhere(got != want)
        raise AssertionError(f"{what}: {len(bad)} of {got.size} differ, first at {bad[0]}: "
                             f"{got[tuple(bad[0])]} for {want[tuple(bad[0])]}")


def values(rng, R, C, t, special=True):
    """Rows of very different size, with zeros, ties and (special) blocks that
    hold a NaN or an infinity, extremes of the type and its subnormals."""
    lo, hi = {"f32": (-140, 120), "bf16": (-130, 120), "f16": (-22, 12)}[t]
    X = rng.standard_normal((R, C)) * np.exp2(rng.integers(lo, hi, (R, 1)))
    half = rng.random((R, C)) < 0.3                       # ties between codes
    X = np.where(half, np.round(X / np.exp2(lo)) * np.exp2(lo), X)
    X[rng.random((R, C)) < 0.05] = -0.0
    n = R * C
    if special and n >= 64:
        flat = X.reshape(-1)
        top = {"f32": 3.4028234e38, "bf16": 3.38e38, "f16": 65504.0}[t]
        low = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[t]
        flat[rng.integers(0, n)] = np.nan
        flat[rng.integers(0, n)] = np.inf
        flat[rng.integers(0, n)] = -np.inf
        flat[rng.integers(0, n)] = -top
        r = rng.integers(0, R)
        X[r] = low * rng.integers(-3, 4, C)
    if R > 2:
        X[R // 2] = 0.0
    return X


# ---- quantising ------------------------------------------------------------

SHAPES = [(1, 1), (1, 32), (3, 31), (1, 8192), (5, 33), (33, 5), (64, 64), (127, 129), (128, 128),
          (130, 700), (257, 255), (1000, 777), (31, 2048), (2048, 31)]


def quantize_case(t, R, C, rows, cols, pad=(0, 0, 0, 0, 0), off=(0, 0, 0, 0, 0), seed=0):
    rng = np.random.default_rng(seed + 7 * R + C)
    raw, X = as_type(values(rng, R, C, t), t)
    size = 4 if t == "f32" else 2
    x = Bytes(R, C * size, (C + pad[0]) * size, off[0] * size, 0xFF, raw)   # NaN around X
    q = Bytes(R, (C + 1) // 2, (C + 1) // 2 + pad[1], off[1])
    s = Bytes(R, (C + 31) // 32, (C + 31) // 32 + pad[2], off[2])
    qt = Bytes(C, (R + 1) // 2, (R + 1) // 2 + pad[3], off[3])
    st = Bytes(C, (R + 31) // 32, (R + 31) // 32 + pad[4], off[4])
    ptr = lambda o, on: (o.ptr, o.ld) if on else (0, 0)  # noqa: E731
    QUANT[t](R, C, x.ptr, C + pad[0], *ptr(q, rows), *ptr(s, rows), *ptr(qt, cols), *ptr(st, cols))
    torch.cuda.synchronize()
    for on, Z, oq, os_, what in ((rows, X, q, s, "rows"), (cols, X.T, qt, st, "columns")):
        got_q, got_s = oq.get(), os_.get()
        if not on:
            assert (got_q == GUARD).all() and (got_s == GUARD).all()
            continue
        codes, byte = mx.quantize(Z)
        same(got_s, byte, f"{t} {R}x{C} scales along {what}")
        ok = np.repeat(byte != 255, 32, axis=1)[:, :Z.shape[1]]
        got = mx.unpack(got_q, Z.shape[1])
        same(np.where(ok, got, 0), np.where(ok, codes, 0), f"{t} {R}x{C} codes along {what}")
        if Z.shape[1] % 2 and Z.shape[1] % 32 != 0:
            same((got_q[:, -1] >> 4)[byte[:, -1] != 255], np.zeros((byte[:, -1] != 255).sum(), np.uint8),
                 "an odd row's last half byte")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_quantize(t, shape):
    for rows, cols in ((True, False), (False, True), (True, True)):
        quantize_case(t, *shape, rows, cols)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,off", [((8, 8, 3, 16, 1), (8, 4, 1, 16, 3)), ((1, 1, 0, 1, 0), (1, 1, 1, 1, 1)),
                                     ((0, 2, 5, 3, 2), (0, 2, 0, 0, 0)), ((3, 0, 0, 0, 0), (0, 0, 0, 0, 0))])
def test_quantize_strides_and_alignment(t, pad, off):
    for R, C in ((96, 200), (130, 264), (65, 77)):
        for rows, cols in ((True, False), (True, True)):
            quantize_case(t, R, C, rows, cols, pad, off)


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_quantize_every_16_bit_value(t):
    """Each of the 65536 patterns beside a value that fixes the block's scale."""
    u = np.arange(65536, dtype=np.uint16).reshape(-1, 1)
    f = u.view(np.float16).astype(np.float64) if t == "f16" else \
        (u.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    for top in (2.0 ** -10, 1.0, 1.75, 448.0):
        keep = np.abs(f[:, 0]) <= top
        raw, X = as_type(np.concatenate([f[keep], np.full((keep.sum(), 1), top)], axis=1), t)
        R = X.shape[0]
        x, q, s = Bytes(R, 4, data=raw), Bytes(R, 1), Bytes(R, 1)
        QUANT[t](R, 2, x.ptr, 2, q.ptr, 1, s.ptr, 1)
        torch.cuda.synchronize()
        codes, byte = mx.quantize(X)
        same(s.get(), byte, "scales")
        same(mx.unpack(q.get(), 2), codes, f"{t} codes under {top}")


# ---- reading back ----------------------------------------------------------

def round_to(v, t):
    """float64 values rounded to type t (exact where t holds them), as bytes."""
    with np.errstate(over="ignore"):
        if t == "f16":
            return v.astype(np.float16)
        f = v.astype(np.float32)
        return f if t == "f32" else f


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_dequantize_every_code_and_scale(t):
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8).reshape(256, 1)
    q, s = Bytes(256, 16, data=mx.pack(codes)), Bytes(256, 1, data=byte)
    y = torch.empty((256, 32), dtype=TORCH[t], device=DEV)
    DEQUANT[t](256, 32, q.ptr, 16, s.ptr, 1, y, 32)
    torch.cuda.synchronize()
    want = mx.dequantize(codes, byte)
    got = y.double().cpu().numpy()
    want = round_to(want, t).astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)
    fin = ~np.isnan(want)
    assert np.array_equal(np.signbit(got[fin]), np.signbit(want[fin]))


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_dequantize(t, shape):
    R, C = shape
    rng = np.random.default_rng(R + 3 * C)
    size = 4 if t == "f32" else 2
    for pq, ps, py, off in ((0, 0, 0, 0), (16, 3, 8, 16), (1, 1, 1, 1)):
        codes = rng.integers(0, 16, (R, C)).astype(np.uint8)
        byte = rng.integers(108, 135, (R, (C + 31) // 32)).astype(np.uint8)
        q = Bytes(R, (C + 1) // 2, (C + 1) // 2 + pq, off, 0xFF, mx.pack(codes, fill=0x70))
        s = Bytes(R, byte.shape[1], byte.shape[1] + ps, off, 0xFF, byte)
        y = Bytes(R, C * size, (C + py) * size, off * size)
        DEQUANT[t](R, C, q.ptr, q.ld, s.ptr, s.ld, y.ptr, C + py)
        torch.cuda.synchronize()
        raw, _ = as_type(mx.dequantize(codes, byte), t)
        same(y.get(), raw, f"{t} {R}x{C}")


# ---- products --------------------------------------------------------------

def operand(rng, rows, K, lo=118, hi=134, pad=0, spad=0, off=0):
    codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    byte = rng.integers(lo, hi, (rows, (K + 31) // 32)).astype(np.uint8)
    n = (K + 1) // 2
    q = Bytes(rows, n, n + pad if n + pad else 1, off, 0x77, mx.pack(codes, fill=0x70)[:, :n])
    s = Bytes(rows, byte.shape[1], max(1, byte.shape[1] + spad), off, 0xFF, byte)
    return q, s, mx.dequantize(codes, byte)


def check_product(C, A, B, out, step, passes=1, what=""):
    R, S = mx.product(A, B)
    K = A.shape[1]
    tol = (passes * -(-K // step) + 32) * 2.0 ** -23 * S
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(R)
    err = np.abs(C - R)
    if not (err <= tol).all():
        i = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err - tol)), err.shape)
        raise AssertionError(f"{what}: {(~(err <= tol)).sum()} of {err.size} off, worst at {i}: "
                             f"{C[i]} for {R[i]}, tolerance {tol[i]}")


def run_product(out, M, N, K, a, sa, bq, sb, ldc_pad=0, off=0, stream=None):
    size = 4 if out == "f32" else 2
    c = Bytes(M, N * size, (N + ldc_pad) * size, off * size, 0xFF)     # NaN until written
    PRODUCT[out](M, N, K, a.ptr, a.ld, sa.ptr, sa.ld, bq.ptr, bq.ld, sb.ptr, sb.ld, c.ptr, N + ldc_pad,
                 stream)
    torch.cuda.synchronize()
    return floats(c.get(), out)


def floats(raw, out):
    if out == "f32":
        return np.ascontiguousarray(raw).view(np.float32).astype(np.float64)
    return (np.ascontiguousarray(raw).view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# rows of A from one to those of several tiles, K of one element, of a block
# and its neighbours, of several stages and past them, N beside every tile
PSHAPES = [(1, 1, 1), (1, 17, 31), (2, 16, 32), (3, 33, 33), (16, 64, 128), (17, 65, 129), (1, 300, 1024),
           (5, 100, 777), (16, 130, 2080), (33, 257, 512), (64, 64, 4096), (65, 96, 256), (100, 100, 255),
           (128, 128, 256), (129, 127, 257), (200, 300, 1000), (256, 256, 512), (300, 520, 513),
           (512, 256, 1024), (1, 4096, 8192), (40, 2000, 3001)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", PSHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product(out, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 5 * N + 7 * K)
    n = (K + 1) // 2
    for pad, spad, off in (((-n) % 16, 0, 0), (0, 0, 0), (16 + (-n) % 16, 5, 16), (1, 2, 1)):
        a, sa, A = operand(rng, M, K, pad=pad, spad=spad, off=off)
        bq, sb, B = operand(rng, N, K, pad=pad, spad=spad, off=off)
        C = run_product(out, M, N, K, a, sa, bq, sb, ldc_pad=3 if off else 0, off=1 if off else 0)
        check_product(C, A, B, out, 64, what=f"{out} {shape} pad {pad} offset {off}")


# 256 x 256 tiles (taken where they fill the CUs no worse than two 128 x 128
# do): K within a stage, ending in a pair's first and second stage, in and past
# the 2048 whose scales lie in LDS together, at a whole 16 scales and beside;
# and the same K in 128 x 128 tiles.
BIG = [(4100, 2300, 96), (3900, 2400, 300), (4096, 2304, 2336), (4000, 2400, 2560), (3900, 2310, 4401)]
LONG = [(130, 250, 2049), (200, 300, 2300), (129, 140, 4400), (128, 256, 8192), (100, 130, 520)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", BIG + LONG, ids=lambda s: "x".join(map(str, s)))
def test_product_wide_tiles_and_long_rows(out, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 5 * N + 7 * K)
    a, sa, A = operand(rng, M, K, pad=(-((K + 1) // 2)) % 16)
    bq, sb, B = operand(rng, N, K, pad=(-((K + 1) // 2)) % 16)
    check_product(run_product(out, M, N, K, a, sa, bq, sb), A, B, out, 64, what=f"{out} {shape}")


# few rows against many columns: each form of the few-row kernel, with whole
# spans of 512, with an end and with the end alone
WIDE = [(1, 32770, 1030), (16, 33000, 2100), (5, 40001, 300), (3, 8200, 2600), (16, 8192, 4608), (30, 8200, 700),
        (60, 9000, 1300)]


@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "x".join(map(str, s)))
def test_few_rows_many_columns(shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 5 * N + 7 * K)
    n = (K + 1) // 2
    for off in (0, 1):
        bq, sb, B = operand(rng, N, K, pad=(-n) % 16 + off, spad=off, off=off)
        a, sa, A = operand(rng, M, K, pad=(-n) % 16 + off, spad=off, off=off)
        check_product(run_product("f32", M, N, K, a, sa, bq, sb), A, B, "f32", 64, what=f"{shape} offset {off}")
        for t in ("bf16", "f16"):
            x, X = a16(rng, M, K, t, pad=(-K) % 8 + off, off=off)
            C = run_wproduct(t, M, N, K, x, K + (-K) % 8 + off, bq, sb)
            check_product(C, X, B, "f32", 16, 2, what=f"{t} {shape} offset {off}")
            assert np.array_equal(C, run_wproduct(t, M, N, K, x, K + (-K) % 8 + off, bq, sb)), "a repeat differs"


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("shape", LONG + [(300, 260, 1664)], ids=lambda s: "x".join(map(str, s)))
def test_weight_product_long_rows(t, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 5 * N + 7 * K)
    a, A = a16(rng, M, K, t, pad=(-K) % 8)
    bq, sb, B = operand(rng, N, K, pad=(-((K + 1) // 2)) % 16)
    check_product(run_wproduct(t, M, N, K, a, K + (-K) % 8, bq, sb), A, B, "f32", 16, 2, what=f"{t} {shape}")


@pytest.mark.parametrize("shape", [(1, 200, 4096), (16, 96, 1000), (48, 70, 515), (130, 250, 700),
                                   (512, 512, 2048), (1024, 1100, 320), (4096, 2304, 1280)], ids=lambda s: "x".join(map(str, s)))
def test_product_exact(shape):
    """Equal scales: every partial sum is a multiple of 1/4 below 2^22."""
    M, N, K = shape
    rng = np.random.default_rng(M + N + K)
    a, sa, A = operand(rng, M, K, 127, 128, pad=(-((K + 1) // 2)) % 16)
    bq, sb, B = operand(rng, N, K, 127, 128, pad=(-((K + 1) // 2)) % 16)
    same(run_product("f32", M, N, K, a, sa, bq, sb), A @ B.T, f"exact {shape}")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 20, 140])
def test_product_scale_extremes(out, M):
    """Scales from 2^-127 to 2^127 whose products stay in range; a NaN block
    makes NaN of its row or column and nothing else."""
    N, K = 150, 416
    rng = np.random.default_rng(M)
    a, sa, A = operand(rng, M, K, 0, 20)
    bq, sb, B = operand(rng, N, K, 235, 255)
    C = run_product(out, M, N, K, a, sa, bq, sb)
    check_product(C, A, B, out, 64, what="extreme scales")
    for dst, row, blk in ((sa, M // 2, 3), (sb, 77, 12)):
        dst.view(dst.host)[row, blk] = 255
        dst.dev.copy_(torch.from_numpy(dst.host))
    C = run_product(out, M, N, K, a, sa, bq, sb)
    nan = np.isnan(C)
    want = np.zeros((M, N), bool)
    want[M // 2] = True
    want[:, 77] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product_empty(out):
    size = 4 if out == "f32" else 2
    for M in (3, 70):
        c = Bytes(M, 90 * size, fill=0xFF)
        assert PRODUCT[out](M, 90, 0, 0, 1, 0, 1, 0, 1, 0, 1, c.ptr, 90) == b.SGEMM_OK
        torch.cuda.synchronize()
        assert (c.get() == 0).all()
    assert PRODUCT[out](0, 90, 64, 0, 32, 0, 2, 0, 32, 0, 2, 0, 90) == b.SGEMM_OK
    assert PRODUCT[out](5, 0, 64, 0, 32, 0, 2, 0, 32, 0, 2, 0, 1) == b.SGEMM_OK


def a16(rng, M, K, t, pad=0, off=0, scale_=1.0):
    raw, A = as_type(rng.standard_normal((M, K)) * scale_ * np.exp2(rng.integers(-6, 6, (1, K))), t)
    return Bytes(M, 2 * K, max(2, 2 * (K + pad)), 2 * off, 0xFF, raw), A


def run_wproduct(t, M, N, K, a, lda, bq, sb, ldc_pad=0, off=0):
    c = Bytes(M, N * 4, (N + ldc_pad) * 4, off * 4, 0xFF)
    WPRODUCT[t](M, N, K, a.ptr, lda, bq.ptr, bq.ld, sb.ptr, sb.ld, c.ptr, N + ldc_pad)
    torch.cuda.synchronize()
    return floats(c.get(), "f32")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("shape", PSHAPES, ids=lambda s: "x".join(map(str, s)))
def test_weight_product(t, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 5 * N + 7 * K)
    n = (K + 1) // 2
    for pa, pb, spad, off in (((-K) % 8, (-n) % 16, 0, 0), (0, 0, 0, 0), (8 + (-K) % 8, 16 + (-n) % 16, 5, 16),
                              (1, 1, 2, 1)):
        a, A = a16(rng, M, K, t, pad=pa, off=off)
        bq, sb, B = operand(rng, N, K, pad=pb, spad=spad, off=off)
        C = run_wproduct(t, M, N, K, a, max(1, K + pa), bq, sb, ldc_pad=3 if off else 0, off=1 if off else 0)
        check_product(C, A, B, "f32", 16, 2, what=f"{t} {shape} pads {pa} {pb} offset {off}")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 20, 140])
def test_weight_product_scale_extremes(t, M):
    """B's scales over their whole range (A small where they are large): the
    smallest are subnormal in bfloat16, most are outside binary16's range."""
    N, K = 150, 416
    rng = np.random.default_rng(M)
    for lo, hi, size in ((0, 3, 2.0 ** 8), (0, 60, 1.0), (90, 165, 1.0), (200, 240, 2.0 ** -10), (100, 114, 1.0), (136, 145, 1.0)):
        a, A = a16(rng, M, K, t, scale_=size)
        bq, sb, B = operand(rng, N, K, lo, hi)
        check_product(run_wproduct(t, M, N, K, a, K, bq, sb), A, B, "f32", 16, 2, what=f"{t} scales {lo}..{hi}")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 20, 140])
def test_weight_product_subnormal_activations(t, M):
    """A's values below its type's normal range (2^-14, 2^-126) count as they are."""
    N, K = 150, 416
    rng = np.random.default_rng(M)
    lo, hi, size = {"f16": (110, 130, 2.0 ** -17), "bf16": (137, 147, 2.0 ** -129)}[t]
    a, A = a16(rng, M, K, t, scale_=size)
    assert (np.abs(A[A != 0]) < {"f16": 2.0 ** -14, "bf16": 2.0 ** -126}[t]).mean() > 0.3
    bq, sb, B = operand(rng, N, K, lo, hi)
    check_product(run_wproduct(t, M, N, K, a, K, bq, sb), A, B, "f32", 16, 2, what=f"{t} subnormal A")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [2, 20, 140])
def test_weight_product_nan_and_infinity(t, M):
    N, K = 150, 416
    rng = np.random.default_rng(M)
    raw, A = as_type(rng.standard_normal((M, K)), t)
    bits = {"bf16": (0x7F80, 0x7FC0), "f16": (0x7C00, 0x7E00)}[t]
    raw = raw.copy().view(np.uint16)
    raw[0, 5], raw[1, 400] = bits
    a = Bytes(M, 2 * K, data=raw.view(np.uint8))
    bq, sb, B = operand(rng, N, K)
    sb.view(sb.host)[33, 2] = 255
    sb.dev.copy_(torch.from_numpy(sb.host))
    C = run_wproduct(t, M, N, K, a, K, bq, sb)
    keep = np.ones(N, bool)
    keep[33] = False
    assert np.isnan(C[:, 33]).all() and np.isnan(C[1]).all()
    b5 = B[:, 5]
    assert np.array_equal(C[0, keep & (b5 != 0)], np.inf * np.sign(b5[keep & (b5 != 0)]))
    assert np.isnan(C[0, keep & (b5 == 0)]).all()
    check_product(C[2:, keep], A[2:], B[keep], "f32", 16, 2, what="rows without a NaN")


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_weight_product_exact_and_empty(t):
    """A's whole numbers and equal scales: exact in fp32.  K = 0 stores zeros."""
    for M, N, K in ((1, 300, 4096), (16, 90, 1001), (48, 70, 515), (130, 250, 700), (512, 600, 640)):
        rng = np.random.default_rng(M + K)
        raw, A = as_type(rng.integers(-8, 9, (M, K)).astype(np.float64), t)
        a = Bytes(M, 2 * K, 2 * (K + (-K) % 8), data=raw)
        bq, sb, B = operand(rng, N, K, 127, 128, pad=(-((K + 1) // 2)) % 16)
        same(run_wproduct(t, M, N, K, a, K + (-K) % 8, bq, sb), A @ B.T, f"exact {t} {M}x{N}x{K}")
    for M in (3, 70):
        c = Bytes(M, 360, fill=0xFF)
        WPRODUCT[t](M, 90, 0, 0, 1, 0, 1, 0, 1, c.ptr, 90)
        torch.cuda.synchronize()
        assert (c.get() == 0).all()


# ---- together --------------------------------------------------------------

class Layer:
    """A linear layer's training step in MXFP4 on device tensors."""

    def __init__(self, T, I, O):  # noqa: E741
        self.T, self.I, self.O = T, I, O
        e = lambda r, c: torch.empty((r, c), dtype=torch.uint8, device=DEV)  # noqa: E731
        ld = lambda k: -(-k // 32) * 16  # noqa: E731
        self.q = {}
        for name, (r, c) in {"X": (T, I), "W": (O, I), "G": (T, O)}.items():
            self.q[name] = (e(r, ld(c)), e(r, -(-c // 32)), e(c, ld(r)), e(c, -(-r // 32)))
        self.y = torch.empty((T, O), dtype=torch.bfloat16, device=DEV)
        self.dx = torch.empty((T, I), dtype=torch.float32, device=DEV)
        self.dw = torch.empty((O, I), dtype=torch.float32, device=DEV)

    def step(self, X, W, G, stream=None):
        for name, v in (("X", X), ("W", W), ("G", G)):
            q = self.q[name]
            b.gemm_mxfp4_quantize_bf16(v.shape[0], v.shape[1], v, v.stride(0), q[0], q[0].stride(0), q[1],
                                       q[1].stride(0), q[2], q[2].stride(0), q[3], q[3].stride(0), stream)
        x, w, g = (self.q[n] for n in "XWG")
        mm = lambda f, k, a, sa, bb, sb, c: f(c.shape[0], c.shape[1], k, a, a.stride(0), sa, sa.stride(0),  # noqa: E731
                                              bb, bb.stride(0), sb, sb.stride(0), c, c.stride(0), stream)
        mm(b.gemm_mxfp4_bf16, self.I, x[0], x[1], w[0], w[1], self.y)
        mm(b.gemm_mxfp4_f32, self.O, g[0], g[1], w[2], w[3], self.dx)
        mm(b.gemm_mxfp4_f32, self.T, g[2], g[3], x[2], x[3], self.dw)


def q64(X):
    return mx.dequantize(*mx.quantize(X))


@pytest.mark.parametrize("T,I,O", [(70, 96, 130), (256, 320, 192), (33, 100, 257)])
def test_training_step(T, I, O):  # noqa: E741
    """Forward and both gradients against the formulas on the quantised values."""
    rng = np.random.default_rng(T)
    t = [torch.from_numpy(rng.standard_normal(s) * f).bfloat16().to(DEV)
         for s, f in (((T, I), 1.0), ((O, I), 0.05), ((T, O), 1e-3))]
    layer = Layer(T, I, O)
    layer.step(*t)
    torch.cuda.synchronize()
    X, W, G = (v.double().cpu().numpy() for v in t)
    check_product(layer.y.double().cpu().numpy(), q64(X), q64(W), "bf16", 64, what="y")
    check_product(layer.dx.double().cpu().numpy(), q64(G), q64(W.T), "f32", 64, what="dx")
    check_product(layer.dw.double().cpu().numpy(), q64(G.T), q64(X.T), "f32", 64, what="dw")


def test_gradients_against_differences():
    """On values that both quantisations hold exactly, the step's gradients are
    those of L(X, W) = sum(G * (X W^T)): L is linear in each operand, so the
    difference of two forward runs over a change of one entry is exact."""
    T, I, O = 64, 64, 96  # noqa: E741
    rng = np.random.default_rng(4)
    grid = np.array([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6.0])
    mats = [rng.choice(grid, s) for s in ((T, I), (O, I), (T, O))]
    for m in mats:                          # a 6 in every block of either direction fixes all scales at 1
        for r in range(m.shape[0]):
            for blk in range(0, m.shape[1], 32):
                m[r, blk + r % 32] = 6.0
    layer, fwd = Layer(T, I, O), Layer(T, I, O)
    dev = lambda m: torch.from_numpy(m).bfloat16().to(DEV)  # noqa: E731
    X, W, G = mats
    layer.step(dev(X), dev(W), dev(G))
    torch.cuda.synchronize()
    dx, dw = layer.dx.double().cpu().numpy(), layer.dw.double().cpu().numpy()

    def forward(X, W):
        y = torch.empty((T, O), dtype=torch.float32, device=DEV)
        q = fwd.q
        for n, v in (("X", X), ("W", W)):
            b.gemm_mxfp4_quantize_bf16(v.shape[0], I, dev(v), I, q[n][0], q[n][0].stride(0), q[n][1],
                                       q[n][1].stride(0))
        b.gemm_mxfp4_f32(T, O, I, q["X"][0], q["X"][0].stride(0), q["X"][1], q["X"][1].stride(0),
                         q["W"][0], q["W"][0].stride(0), q["W"][1], q["W"][1].stride(0), y, O)
        torch.cuda.synchronize()
        return float((G * y.double().cpu().numpy()).sum())

    for m, d in ((X, dx), (W, dw)):
        for _ in range(6):
            r, c = rng.integers(0, m.shape[0]), rng.integers(0, m.shape[1])
            if abs(m[r, c]) == 6.0:
                continue
            up, down = m.copy(), m.copy()
            up[r, c], down[r, c] = 4.0, -4.0
            args = (lambda v: (v, W)) if m is X else (lambda v: (X, v))
            assert (forward(*args(up)) - forward(*args(down))) / 8.0 == d[r, c]


def test_serving_step():
    """One token and a batch: activations quantised and multiplied with kept
    weights, and the same weights with 16-bit activations."""
    I, O = 1024, 640  # noqa: E741
    rng = np.random.default_rng(9)
    W = torch.from_numpy(0.02 * rng.standard_normal((O, I))).bfloat16().to(DEV)
    wq = torch.empty((O, I // 2), dtype=torch.uint8, device=DEV)
    ws = torch.empty((O, I // 32), dtype=torch.uint8, device=DEV)
    b.gemm_mxfp4_quantize_bf16(O, I, W, I, wq, I // 2, ws, I // 32)
    W64 = q64(W.double().cpu().numpy())
    for M in (1, 7, 48, 200):
        X = torch.from_numpy(rng.standard_normal((M, I))).bfloat16().to(DEV)
        xq = torch.empty((M, I // 2), dtype=torch.uint8, device=DEV)
        xs = torch.empty((M, I // 32), dtype=torch.uint8, device=DEV)
        y4 = torch.empty((M, O), dtype=torch.bfloat16, device=DEV)
        y16 = torch.empty((M, O), dtype=torch.float32, device=DEV)
        b.gemm_mxfp4_quantize_bf16(M, I, X, I, xq, I // 2, xs, I // 32)
        b.gemm_mxfp4_bf16(M, O, I, xq, I // 2, xs, I // 32, wq, I // 2, ws, I // 32, y4, O)
        b.gemm_bf16_mxfp4_f32(M, O, I, X, I, wq, I // 2, ws, I // 32, y16, O)
        torch.cuda.synchronize()
        X64 = X.double().cpu().numpy()
        check_product(y4.double().cpu().numpy(), q64(X64), W64, "bf16", 64, what=f"M = {M}")
        check_product(y16.double().cpu().numpy(), X64, W64, "f32", 16, what=f"16-bit, M = {M}")


def test_graph_capture_streams_and_repeats():
    """A captured step on a side stream, replayed with eager work between the
    replays that changes the inputs, gives the eager step's bits; so do
    repeated eager steps."""
    T, I, O = 160, 256, 384  # noqa: E741
    rng = np.random.default_rng(5)
    new = lambda: [torch.from_numpy(rng.standard_normal(s)).bfloat16().to(DEV)  # noqa: E731
                   for s in ((T, I), (O, I), (T, O))]
    bufs, layer, eager = new(), Layer(T, I, O), Layer(T, I, O)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        layer.step(*bufs)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            layer.step(*bufs)
    torch.cuda.synchronize()
    for rep in range(4):
        for dst, src in zip(bufs, new()):
            dst.copy_(src)
        for o in (layer.y, layer.dx, layer.dw):
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager.step(*bufs)
        torch.cuda.synchronize()
        for a, e in ((layer.y, eager.y), (layer.dx, eager.dx), (layer.dw, eager.dw)):
            assert torch.equal(a, e), f"replay {rep}"
        first = [o.clone() for o in (eager.y, eager.dx, eager.dw)]
        eager.step(*bufs, stream=s)
        torch.cuda.synchronize()
        for a, e in zip(first, (eager.y, eager.dx, eager.dw)):
            assert torch.equal(a, e), "a repeated step differs"


def test_threads():
    """Four host threads, each with its stream and layer, at once."""
    errors = []

    def worker(i):
        try:
            rng = np.random.default_rng(i)
            T, I, O = 64 + 32 * i, 256, 128 + 64 * i  # noqa: E741
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                t = [torch.from_numpy(rng.standard_normal(x)).bfloat16().to(DEV)
                     for x in ((T, I), (O, I), (T, O))]
                layer = Layer(T, I, O)
                s.synchronize()
                for _ in range(10):
                    layer.step(*t, stream=s)
                s.synchronize()
            X, W, G = (v.double().cpu().numpy() for v in t)
            check_product(layer.y.double().cpu().numpy(), q64(X), q64(W), "bf16", 64)
            check_product(layer.dw.double().cpu().numpy(), q64(G.T), q64(X.T), "f32", 64)
        except Exception as e:  # noqa: BLE001
            errors.append(f"thread {i}: {e!r}")

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not any(t.is_alive() for t in threads) and not errors, errors


def test_large_offsets():
    """Matrices past 2^31 and 2^32 bytes: rows and columns near their ends."""
    # 16-bit X of 70000 x 33000 (4.6 GB), quantised along rows and columns
    R, C = 70000, 33000
    X = torch.zeros((R, C), dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(3)
    tail = torch.from_numpy(rng.standard_normal((200, C))).bfloat16()
    X[R - 200:] = tail.to(DEV)
    ld, ldt = -(-C // 32) * 16, -(-R // 32) * 16
    q = torch.empty((R, ld), dtype=torch.uint8, device=DEV)
    s = torch.empty((R, -(-C // 32)), dtype=torch.uint8, device=DEV)
    qt = torch.empty((C, ldt), dtype=torch.uint8, device=DEV)
    st = torch.empty((C, -(-R // 32)), dtype=torch.uint8, device=DEV)
    b.gemm_mxfp4_quantize_bf16(R, C, X, C, q, ld, s, s.stride(0), qt, ldt, st, st.stride(0))
    torch.cuda.synchronize()
    X64 = tail.double().numpy()
    codes, byte = mx.quantize(X64)
    same(s[R - 200:].cpu().numpy(), byte, "scales of the last rows")
    same(mx.unpack(q[R - 200:].cpu().numpy(), C), codes, "codes of the last rows")
    lo = (R - 200) // 32 * 32 + 32            # whole column blocks inside the tail
    codes, byte = mx.quantize(X64[lo - (R - 200):].T)
    same(st[:, lo // 32:].cpu().numpy(), byte, "scales down the columns")
    same(mx.unpack(qt[:, lo // 2:-(-R // 2)].cpu().numpy(), R - lo), codes, "codes down the columns")
    assert int(q[:R - 200].max()) == 0 and int(s[:R - 200].max()) == 0
    Y = X.fill_(float("nan"))
    b.gemm_mxfp4_dequantize_bf16(R, C, q, ld, s, s.stride(0), Y, C)
    torch.cuda.synchronize()
    same(Y[R - 200:].double().cpu().numpy(), q64(X64), "read back")
    assert int((Y[:R - 200] != 0).sum()) == 0
    del X, Y, qt, st
    # a product whose second operand's last rows lie past 2^32 bytes of row pitch:
    # few rows; the 16-bit tiles' DMA, by offsets past 2^31 (24 MiB), and beyond
    # its reach (40 MiB); the MXFP4 tiles, beyond their DMA's reach in all three
    N, K = 300, 512
    bq, sb, B = operand(np.random.default_rng(1), N, K)
    for M, pitch in ((2, 16 << 20), (100, 16 << 20), (100, 24 << 20), (100, 40 << 20)):
        big = torch.full((N * pitch,), 0x77, dtype=torch.uint8, device=DEV)
        big.view(N, pitch)[:, :K // 2] = torch.from_numpy(bq.view(bq.host)[:, :K // 2].copy()).to(DEV)
        a, sa, A = operand(np.random.default_rng(M), M, K)
        c = torch.empty((M, N), device=DEV)
        b.gemm_mxfp4_f32(M, N, K, a.ptr, a.ld, sa.ptr, sa.ld, big, pitch, sb.ptr, sb.ld, c, N)
        x, A2 = a16(np.random.default_rng(M), M, K, "bf16")
        c2 = torch.empty((M, N), device=DEV)
        b.gemm_bf16_mxfp4_f32(M, N, K, x.ptr, K, big, pitch, sb.ptr, sb.ld, c2, N)
        torch.cuda.synchronize()
        check_product(c.double().cpu().numpy(), A, B, "f32", 64, what=f"far rows, M = {M}")
        check_product(c2.double().cpu().numpy(), A2, B, "f32", 16, what=f"far rows, 16-bit, M = {M}")
        del big


def test_binding_checks_tensors():
    q = torch.empty((4, 32), dtype=torch.uint8, device=DEV)
    s = torch.empty((4, 2), dtype=torch.uint8, device=DEV)
    x = torch.zeros((4, 64), device=DEV)
    with pytest.raises(TypeError):
        b.gemm_mxfp4_quantize_bf16(4, 64, x, 64, q, 32, s, 2)
    with pytest.raises(TypeError):
        b.gemm_mxfp4_quantize_f32(4, 64, x, 64, x, 32, s, 2)
    with pytest.raises(ValueError):
        b.gemm_mxfp4_quantize_f32(4, 64, x, 64, q.cpu(), 32, s, 2)
    with pytest.raises(b.SgemmError) as e:
        b.gemm_mxfp4_dequantize_f32(4, 64, q, 32, s, 2, x, 63)
    assert e.value.status == b.SGEMM_EINVAL_LD
