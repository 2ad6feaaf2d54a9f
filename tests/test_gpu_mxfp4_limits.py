"""GPU tests of the MXFP4 entry points at the ends of their ranges: the widest
matrices, far rows, and products that fp32 does not hold.

Products below fp32's normal range may lose bits down to all of them: each of
the passes * K terms and of the T partial sums (T as derived in
test_gpu_mxfp4.py) is then off by at most 2^-126 more, so
    |C - R| <= T 2^-23 S + (passes * K + T) 2^-126.
Where all terms are positive, a sum R with R (1 - T 2^-23) above the largest
fp32 number is infinite."""
import numpy as np
import pytest

from oracle import mxfp4 as mx
from register_lds_tiled_amd import binding as b
from tests.test_gpu_mxfp4 import Bytes, as_type, check_product, operand, quantize_case, run_product, run_wproduct

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PERIOD = 4099               # rows of B before they repeat: not a multiple of any tile
WIDE = 64 * (2 ** 24 - 1)   # the most columns a product of few rows takes


def repeated(x, n, dim):
    """x repeated along dim to n, on the GPU."""
    reps = [1, 1]
    reps[dim] = -(-n // x.shape[dim])
    return torch.from_numpy(x).to(DEV).repeat(reps).narrow(dim, 0, n)


def same_in_pieces(got, want, period):
    """Columns of got repeat want's: compared on the GPU, a few periods at a time."""
    step = period * 4096
    for at in range(0, got.shape[1], step):
        n = min(step, got.shape[1] - at)
        whole = n // period * period
        assert torch.equal(got[:, at:at + whole].reshape(got.shape[0], -1, period),
                           want[:, None].expand(-1, whole // period, -1)), at
        assert torch.equal(got[:, at + whole:at + n], want[:, :n - whole]), at


@pytest.mark.parametrize("N", [2 ** 29 - 32, 2 ** 29 - 31, 2 ** 29 + 37, WIDE])
@pytest.mark.parametrize("M", [1, 2])
def test_widest_products(M, N):
    """One and two rows against up to 2^30 columns: whole numbers, so exact."""
    rng = np.random.default_rng(M)
    K = 1
    a = rng.integers(0, 16, (M, K)).astype(np.uint8)
    w = rng.integers(0, 16, (PERIOD, K)).astype(np.uint8)
    sw = rng.integers(126, 129, (PERIOD, 1)).astype(np.uint8)
    R = mx.element(a) @ mx.dequantize(w, sw).T
    bq = repeated(mx.pack(w), N, 0).contiguous()
    sb = repeated(sw, N, 0).contiguous()
    aq, sa = torch.from_numpy(mx.pack(a)).to(DEV), torch.full((M, 1), 127, dtype=torch.uint8, device=DEV)
    c = torch.empty((M, N), device=DEV)
    want = torch.from_numpy(R).to(DEV, torch.float32)
    x = torch.from_numpy(mx.element(a)).to(DEV)
    for name in ("mxfp4", "bf16", "f16"):
        c.fill_(float("nan"))
        if name == "mxfp4":
            b.gemm_mxfp4_f32(M, N, K, aq, 1, sa, 1, bq, 1, sb, 1, c, N)
        else:
            fn = b.gemm_bf16_mxfp4_f32 if name == "bf16" else b.gemm_f16_mxfp4_f32
            fn(M, N, K, x.to(TYPES[name]), K, bq, 1, sb, 1, c, N)
        torch.cuda.synchronize()
        same_in_pieces(c, want, PERIOD)


@pytest.mark.parametrize("R,C", [(1, 2 ** 30 - 128), (1, 2 ** 30 + 37), (1, 128 * (2 ** 24 - 1)), (3, 2 ** 30)])
@pytest.mark.parametrize("rows", [False, True])
def test_quantise_widest_along_columns(R, C, rows):
    """Up to 2^31 columns of one to three values each, and the rows with them."""
    rng = np.random.default_rng(R)
    period = 4128            # whole blocks of the rows, no multiple of a tile
    x = torch.from_numpy(rng.standard_normal((R, period)) * np.exp2(rng.integers(-9, 9, (1, period)))).bfloat16()
    X = repeated(x.view(torch.int16).numpy(), C, 1).contiguous().view(torch.bfloat16)
    n, m = -(-R // 2), -(-C // 32) if rows else 1
    qt = torch.full((C, n), 0x5A, dtype=torch.uint8, device=DEV)
    st = torch.full((C, 1), 0x5A, dtype=torch.uint8, device=DEV)
    q = torch.full((R, 16 * m), 0x5A, dtype=torch.uint8, device=DEV)
    s = torch.full((R, m), 0x5A, dtype=torch.uint8, device=DEV)
    if rows:
        b.gemm_mxfp4_quantize_bf16(R, C, X, C, q, 16 * m, s, m, qt, n, st, 1)
    else:
        b.gemm_mxfp4_quantize_bf16(R, C, X, C, None, 0, None, 0, qt, n, st, 1)
    torch.cuda.synchronize()
    x64 = x.double().numpy()
    codes, byte = mx.quantize(x64.T)
    want = torch.from_numpy(np.concatenate([mx.pack(codes), byte], 1).T.copy()).to(DEV)
    same_in_pieces(torch.cat([qt, st], 1).T, want, period)
    if rows:
        codes, byte = mx.quantize(x64)
        full = C // period * period
        for got, per, k in ((q, torch.from_numpy(mx.pack(codes)).to(DEV), 2), (s, torch.from_numpy(byte).to(DEV), 32)):
            same_in_pieces(got[:, :full // k], per, period // k)
        codes, byte = mx.quantize(x64[:, :C - full])
        assert np.array_equal(s[:, full // 32:].cpu().numpy(), byte)
        assert np.array_equal(mx.unpack(q[:, full // 2:full // 2 + -(-(C - full) // 2)].cpu().numpy(), C - full), codes)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("R,C", [(33, 66001), (128, 65664), (129, 66001), (300, 40001), (2100, 7500)])
def test_quantise_in_tiles_of_either_height(t, R, C):
    """Shapes beside the choice between tiles of 128 and 256 rows, odd ends."""
    quantize_case(t, R, C, False, True)
    quantize_case(t, R, C, True, True)


# ---- products that fp32 does not hold ---------------------------------------

FORMS = [(1, 150, 416), (20, 150, 416), (140, 150, 416), (16, 40, 1000), (300, 300, 700)]


def check_range(C, A, B, out, step, passes):
    """C against the exact sums, whose terms may leave fp32's range."""
    K = A.shape[1]
    R, S = mx.product(A, B)
    T = passes * -(-K // step) + 32
    tol = T * 2.0 ** -23 * S + (passes * K + T) * 2.0 ** -126
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(R)
    high = R * (1 - T * 2.0 ** -23) > np.finfo(np.float32).max
    # (bfloat16 rounds to an infinity from half a step below 2^128 on)
    edge = ~high & (S * (1 + T * 2.0 ** -23) >= (2.0 ** 128 - 2.0 ** 119 if out == "bf16" else 2.0 ** 128))
    assert (C[high] == np.inf).all()
    mid = ~high & ~edge
    bad = ~(np.abs(C - R) <= tol)[mid]
    assert not bad.any(), (bad.sum(), C[mid][bad][:4], R[mid][bad][:4], tol[mid][bad][:4])
    return high, mid


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_products_beyond_fp32(out, pad, M, N, K):
    rng = np.random.default_rng(M + pad)
    n = (-((K + 1) // 2)) % 16 + pad
    for (alo, ahi), (blo, bhi) in (((0, 3), (0, 3)), ((40, 80), (50, 90)), ((0, 60), (60, 80)), ((60, 70), (58, 66)),
                                   ((54, 64), (54, 62))):
        a, sa, A = operand(rng, M, K, alo, ahi, pad=n)
        w, sw, W = operand(rng, N, K, blo, bhi, pad=n)
        high, mid = check_range(run_product(out, M, N, K, a, sa, w, sw), A, W, out, 64, 1)
        assert mid.all()
    seen = []
    for (alo, ahi), (blo, bhi) in (((253, 255), (253, 255)), ((185, 193), (180, 192)), ((200, 255), (120, 200)),
                                   ((178, 186), (174, 186))):
        a, sa, A = operand(rng, M, K, alo, ahi, pad=n)
        w, sw, W = operand(rng, N, K, blo, bhi, pad=n)
        for o in (a, w):                              # no minus signs
            o.host &= 0x77
            o.dev.copy_(torch.from_numpy(o.host))
        C = run_product(out, M, N, K, a, sa, w, sw)
        seen.append(check_range(C, np.abs(A), np.abs(W), out, 64, 1)[0].any())
    assert any(seen)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_weight_products_beyond_fp32(t, pad, M, N, K):
    rng = np.random.default_rng(M + pad)
    n = (-((K + 1) // 2)) % 16 + pad
    lda = K + (-K) % 8 + pad

    def a16(x):
        raw, A = as_type(x, t)
        return Bytes(M, 2 * K, 2 * lda, 0, 0xFF, raw), A

    small = {"bf16": (((0, 3), -130), ((20, 60), -60), ((60, 70), -66)), "f16": (((0, 3), -18), ((0, 12), -8))}[t]
    for (lo, hi), e in small:
        a, A = a16(rng.standard_normal((M, K)) * 2.0 ** e)
        w, sw, W = operand(rng, N, K, lo, hi, pad=n)
        high, mid = check_range(run_wproduct(t, M, N, K, a, lda, w, sw), A, W, "f32", 16, 2)
        assert mid.all()
    seen = []
    large = {"bf16": (((200, 252), 60), ((180, 190), 70), ((170, 180), 68)),
             "f16": (((240, 252), 12), ((238, 246), 8), ((232, 240), 8))}[t]
    for (lo, hi), e in large:
        a, A = a16(np.abs(rng.standard_normal((M, K))) * 2.0 ** e)
        w, sw, W = operand(rng, N, K, lo, hi, pad=n)
        w.host &= 0x77
        w.dev.copy_(torch.from_numpy(w.host))
        seen.append(check_range(run_wproduct(t, M, N, K, a, lda, w, sw), A, np.abs(W), "f32", 16, 2)[0].any())
    assert any(seen)


# ---- far rows ---------------------------------------------------------------

@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_wide_tiles_of_far_rows(out):
    """256 x 256 tiles whose rows of B lie past 2^31 bytes from their first, up
    to the last pitch that 32-bit offsets reach."""
    M, N, K, pitch = 32800, 256, 320, (16 << 20) - 16
    rng = np.random.default_rng(1)
    a, sa, A = operand(rng, M, K)
    w, sw, W = operand(rng, N, K)
    big = torch.full((N * pitch,), 0x77, dtype=torch.uint8, device=DEV)
    rows = torch.arange(N, device=DEV)[:, None] * pitch + torch.arange(K // 2, device=DEV)
    big[rows] = torch.from_numpy(w.view(w.host)[:, :K // 2].copy()).to(DEV)
    c = torch.full((M, N), float("nan"), dtype=TYPES[out], device=DEV)
    fn = b.gemm_mxfp4_f32 if out == "f32" else b.gemm_mxfp4_bf16
    fn(M, N, K, a.ptr, a.ld, sa.ptr, sa.ld, big, pitch, sw.ptr, sw.ld, c, N)
    torch.cuda.synchronize()
    check_product(c.double().cpu().numpy(), A, W, out, 64, what=f"far rows, {out}")


# ---- long rows --------------------------------------------------------------

# K at the last row length that the kernels' 32-bit row offsets reach and past
# it: few rows (64 rows of B), MXFP4 tiles (256 rows), 16-bit tiles (128 rows)
LONGEST = [("few", 2, 2 ** 27 - 32), ("few", 2, 2 ** 27 + 33), ("tile", 66, 2 ** 25 - 32), ("tile", 66, 2 ** 25 + 33),
           ("tile16", 66, 2 ** 24 - 8), ("tile16", 66, 2 ** 24 + 9)]


@pytest.mark.parametrize("form,M,K", LONGEST)
def test_longest_rows(form, M, K):
    """A few hundred whole numbers among zeros, the row's ends with them."""
    N = 5
    rng = np.random.default_rng(K % 1000)
    at = np.unique(np.concatenate([rng.integers(0, K, 300), [0, 1, 31, 32, K - 1, K - 2, K - 33]]))
    ld, ls = -(-K // 32) * 16, -(-K // 32)

    def sparse(rows):
        codes = rng.integers(0, 16, (rows, at.size))
        q = torch.zeros((rows, ld), dtype=torch.uint8, device=DEV)
        low, high = at % 2 == 0, at % 2 == 1
        q[:, torch.from_numpy(at[low] // 2).to(DEV)] = torch.from_numpy(codes[:, low].astype(np.uint8)).to(DEV)
        q[:, torch.from_numpy(at[high] // 2).to(DEV)] |= torch.from_numpy((codes[:, high] << 4).astype(np.uint8)).to(DEV)
        s = torch.from_numpy(rng.integers(125, 130, (rows, ls), dtype=np.uint8)).to(DEV)
        byte = s[:, torch.from_numpy(at // 32).to(DEV)].cpu().numpy()
        return q, s, mx.element(codes) * mx.scale(byte)

    w, sw, W = sparse(N)
    c = torch.full((M, N), float("nan"), device=DEV)
    if form != "tile16":
        a, sa, A = sparse(M)
        b.gemm_mxfp4_f32(M, N, K, a, ld, sa, ls, w, ld, sw, ls, c, N)
        torch.cuda.synchronize()
        assert np.array_equal(c.double().cpu().numpy(), A @ W.T)
        del a, sa
    if form != "tile":
        lda = K + (-K) % 8
        for t, fn in (("bf16", b.gemm_bf16_mxfp4_f32), ("f16", b.gemm_f16_mxfp4_f32)):
            A = rng.integers(-8, 9, (M, at.size)).astype(np.float64)
            x = torch.zeros((M, lda), dtype=TYPES[t], device=DEV)
            x[:, torch.from_numpy(at).to(DEV)] = torch.from_numpy(A).to(DEV, TYPES[t])
            c.fill_(float("nan"))
            fn(M, N, K, x, lda, w, ld, sw, ls, c, N)
            torch.cuda.synchronize()
            assert np.array_equal(c.double().cpu().numpy(), A @ W.T), t
