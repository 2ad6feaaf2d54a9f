"""GPU tests of the 8-bit integer operators and the gated feed-forward block
against oracle/layer.py (float64).

Quantising must match bit for bit; a value read back is one fp32 product (2^-24)
and a rounding to the type, half a step of it (eps / 2).

8-bit products: the sum is exact, its conversion and the two scalings round once
each, 3 * 2^-24 relative (and the type's half step).

16-bit products of K terms: the matrix cores add at most 16 products at a time
into an fp32 accumulator and k may be split among up to 16 waves, so each output
has at most T = ceil(K / 16) + 2 * 16 roundings of partial sums no larger than
S = sum |a b|, each off by at most 2^-23 S (truncation included): T 2^-23 S.

H = act(g) u: with g and u off by eg and eu, H is off by at most
    1.2 eg |u| + |act(g)| eu + 1.2 eg eu + E |u|
(no slope exceeds 1.2), where E is the activation's own error.  E: an exponential
of x has the relative error 2^-23 (|x| + 1), the sum, the reciprocal and the
product add 4 * 2^-23 at most; the tanh form's argument is 2 y with y a sum of
three roundings more, |2 y| <= 3 |x| + |x|^3 / 8; erfc's argument x / sqrt 2 has
two roundings, which erfc's tail turns into x^2 2^-23, and its own error is a few
2^-23.  For all of them E <= 2^-23 (8 + 4 |z|) |act| with z = x, 2 y or x^2, and
2^-120 where the hardware's exponential or reciprocal leaves its range.  A slope
is off by less than 2^-13: its terms are bounded by (1 + 0.8 |x| (1 + 0.134 x^2))
s (1 - s), where 1 - s is off by 3 * 2^-23 and s is 1 in fp32 from |x| = 17 on
(tanh form: from |x| = 5.1 on): 40 * 3 * 2^-23 at most, plus the exponential's own.
Rounding to 16 bits adds half a step, and half of the least subnormal.

Around inputs lies NaN (8 bits: -128), around outputs a guard that must survive.
"""
import threading

import numpy as np
import pytest

from oracle import layer as o
from register_lds_tiled_amd import binding as b

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def fn(name, t):
    return getattr(b, f"{name}_{t}")


class Mat:
    """rows x cols of a type in a device buffer: `pad` elements between rows, `off`
    before the first; all else holds NaN (-128), which must survive."""

    def __init__(self, data, t, pad=0, off=0, rows=None, cols=None):
        self.t = t
        if data is not None:
            data = torch.as_tensor(np.ascontiguousarray(data))
            rows, cols = data.shape
        self.rows, self.cols, self.ld, self.off = rows, cols, max(1, cols + pad), off
        guard = -128 if t == "i8" else float("nan")
        self.flat = torch.full((off + rows * self.ld + 64,), guard, dtype=TYPES[t])
        v = self.flat[off:off + rows * self.ld].view(rows, self.ld)
        if data is not None:
            v[:, :cols] = data.to(TYPES[t])
        self.value = v[:, :cols].double().numpy()     # as rounded
        self.dev = self.flat.to(DEV)
        self.ptr = self.dev.data_ptr() + off * self.flat.element_size()

    @property
    def at(self):
        return self.ptr, self.ld

    def get(self):
        now = self.dev.cpu()
        v = now[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)
        out = v[:, :self.cols].clone()
        was = self.flat.clone()
        for x in (now, was):
            x[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = 0
        bits = {1: torch.int8, 2: torch.int16, 4: torch.int32}[now.element_size()]
        assert torch.equal(now.view(bits), was.view(bits)), "something outside the rows was written"
        return out

    def unchanged(self):
        bits = {1: torch.int8, 2: torch.int16, 4: torch.int32}[self.flat.element_size()]
        return torch.equal(self.dev.cpu().view(bits), self.flat.view(bits))


def near(got, want, bound, t, what):
    """|got - want| <= bound + half a step of t."""
    got = got.double().numpy() if hasattr(got, "numpy") else got
    half = torch.finfo(TYPES[t]).eps / 2
    most = bound + half * (np.abs(want) + bound) + TINY[t] / 2
    off = np.abs(got - want)
    bad = ~(off <= most) & ~(np.isnan(got) & np.isnan(want))
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {at}: {got[at]} for {want[at]}, "
                             f"{off[at]:.3g} off where {most[at] if np.ndim(most) else most:.3g} may be")


# ---- quantising ------------------------------------------------------------

def values(rng, R, C, t, special=True):
    lo, hi = {"f32": (-147, 120), "bf16": (-130, 120), "f16": (-22, 12)}[t]
    X = rng.standard_normal((R, C)) * np.exp2(rng.integers(lo, hi, (R, 1)))
    X[rng.random((R, C)) < 0.05] = -0.0
    for r in range(0, R, 3):                            # rows whose scale is a power of two: ties
        e = rng.integers(lo + 20, hi - 8) if hi - 8 > lo + 20 else 0
        X[r] = (rng.integers(-126, 127, C) + 0.5 * rng.integers(0, 2, C)) * np.exp2(float(e))
        X[r, rng.integers(0, C)] = 127.0 * np.exp2(float(e))
    if special:
        top = {"f32": 3.4028234e38, "bf16": 3.38e38, "f16": 65504.0}[t]
        if R > 3:
            X[1] = 0.0
            X[2] = TINY[t] * rng.integers(-3, 4, C)
            X[3, rng.integers(0, C)] = -top
        if R > 6:
            X[4, rng.integers(0, C)] = np.nan
            X[5, rng.integers(0, C)] = np.inf
            X[6, rng.integers(0, C)] = -np.inf
    return X


SHAPES = [(1, 1), (1, 7), (1, 8), (3, 9), (7, 33), (64, 64), (9, 511), (9, 513), (5, 1024), (5, 2047), (5, 2049),
          (3, 8191), (300, 4096), (2, 8200), (300, 8200), (2, 16385), (1, 32768), (3, 40001), (2, 100003), (1000, 777),
          (70000, 3)]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_quantize_and_back(t, R, C):
    rng = np.random.default_rng(R * 7 + C)
    for pad, off in ((0, 0), (5, 3), (16, 16)):
        X = Mat(values(rng, R, C, t), t, pad, off)
        Q, S = Mat(None, "i8", pad, off, R, C), Mat(None, "f32", 0, off % 7, 1, R)
        fn("gemm_i8_quantize", t)(R, C, *X.at, *Q.at, S.ptr)
        q, s = Q.get().numpy(), S.get().numpy()[0]
        want_q, want_s = o.quantize(X.value)
        assert np.array_equal(s, want_s, equal_nan=True), (s[s != want_s][:3], want_s[s != want_s][:3])
        assert np.array_equal(q, want_q), [(i, q[tuple(i)], want_q[tuple(i)]) for i in np.argwhere(q != want_q)[:3]]
        assert X.unchanged()
        Y = Mat(None, t, pad, off, R, C)
        fn("gemm_i8_dequantize", t)(R, C, *Q.at, S.ptr, *Y.at)
        v = o.dequantize(want_q, want_s)
        y = Y.get().double().numpy()
        edge = np.abs(v) > 3.402e38                     # next to the largest number: that or infinite
        assert (np.abs(y[edge]) > 3.4e38).all()
        near(np.where(edge, 0, y), np.where(edge, 0, v), np.where(edge, 0, np.abs(v)) * 2.0 ** -24, t, "read back")


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_quantize_every_pattern(t):
    """Every finite 16-bit pattern beside each of several largest values."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TYPES[t])
    v = bits.double()
    for top in (1.0, 127.0, 100.0, 0.3, 3e-5, 65504.0 if t == "f16" else 3e38):
        keep = v[torch.isfinite(v) & (v.abs() <= top)].numpy()
        X = Mat(np.concatenate([[float(torch.tensor(top).to(TYPES[t]))], keep])[None], t)
        Q, S = Mat(None, "i8", 0, 0, 1, X.cols), Mat(None, "f32", 0, 0, 1, 1)
        fn("gemm_i8_quantize", t)(1, X.cols, *X.at, *Q.at, S.ptr)
        q, s = o.quantize(X.value)
        assert np.array_equal(S.get().numpy()[0], s) and np.array_equal(Q.get().numpy(), q)


# ---- 8-bit products --------------------------------------------------------

PRODUCTS = [(1, 1, 1), (1, 16, 64), (1, 33, 7), (1, 1000, 8192), (2, 100, 300), (3, 5, 7), (16, 100, 33), (16, 128, 512),
            (17, 130, 65), (33, 64, 1000), (64, 64, 64), (64, 300, 2048), (65, 70, 100), (100, 77, 129), (128, 128, 128),
            (129, 257, 191), (256, 256, 256), (255, 512, 320), (300, 200, 1000), (1000, 1500, 777), (520, 776, 1024),
            (1, 8192, 1024), (40, 8200, 256)]
# paddings and offsets of A, B and C, in elements: 16-byte aligned or not
LAYOUTS = {"whole": (0, 0), "padded": (16, 16), "odd": (3, 5)}


def codes(rng, R, C):
    q = rng.integers(-127, 128, (R, C))
    q[rng.random((R, C)) < 0.1] = -128
    return q.astype(np.int8)


def scales(rng, n):
    return (rng.random(n) * np.exp2(rng.integers(-12, 3, n))).astype(np.float32)


def round_up(K, to):
    return -(-K // to) * to - K


def layout(name, K, whole):
    """(padding, offset) of rows of K elements, `whole` of them 16 bytes."""
    pad, off = LAYOUTS[name]
    return (round_up(K, whole) + pad if name == "padded" else pad), off


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("how", list(LAYOUTS))
def test_i8_product(out, M, N, K, how):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    pad, off = layout(how, K, 16)
    A, B = Mat(codes(rng, M, K), "i8", pad, off), Mat(codes(rng, N, K), "i8", pad, off)
    SA, SB = (Mat(scales(rng, n)[None] * (0.01 if out == "f16" else 1), "f32", 0, off % 4) for n in (M, N))
    C = Mat(None, out, pad, off, M, N)
    fn("gemm_i8", out)(M, N, K, *A.at, SA.ptr, *B.at, SB.ptr, *C.at)
    want = o.product(A.value, SA.value[0], B.value, SB.value[0])
    near(C.get(), want, 3.01 * 2.0 ** -24 * np.abs(want), out, f"{out} {M}x{N}x{K} {how}")
    assert A.unchanged() and B.unchanged() and SA.unchanged() and SB.unchanged()


@pytest.mark.parametrize("M,N", [(1, 40), (20, 40), (200, 300)])
def test_i8_longest_sums_are_exact(M, N):
    """K of 131071 codes of -128: the largest sum 32 bits hold."""
    K = 131071
    A = torch.full((M, K + 1), -128, dtype=torch.int8, device=DEV)
    B = torch.full((N, K + 1), -128, dtype=torch.int8, device=DEV)
    B[1::2] = 127
    one_m, one_n = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    C = torch.empty((M, N), device=DEV)
    b.gemm_i8_f32(M, N, K, A, K + 1, one_m, B, K + 1, one_n, C, N)
    want = torch.where(torch.arange(N) % 2 == 0, float(K * 16384), float(-K * 128 * 127)).float()
    assert torch.equal(C.cpu(), want.expand(M, N))


def test_i8_scales_that_are_not_numbers():
    """A NaN scale makes its row or column NaN and nothing else; zero and an infinity
    are multiplied as they are."""
    for M, N, K in ((5, 40, 100), (100, 200, 64), (300, 520, 256)):
        rng = np.random.default_rng(4)
        A, B = codes(rng, M, K), codes(rng, N, K)
        SA, SB = scales(rng, M) + np.float32(0.1), scales(rng, N) + np.float32(0.1)
        SA[1], SB[3], SA[2], SB[5] = np.nan, np.nan, 0.0, np.inf
        C = torch.empty((M, N), device=DEV)
        d = [torch.from_numpy(v).to(DEV) for v in (A, SA, B, SB)]
        b.gemm_i8_f32(M, N, K, d[0], K, d[1], d[2], K, d[3], C, N)
        with np.errstate(invalid="ignore"):
            want = o.product(A, SA, B, SB)
        got = C.cpu().double().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.isnan(got[1]).all() and np.isnan(got[:, 3]).all()
        ok = np.isfinite(want)
        assert np.array_equal(got[~ok], want[~ok], equal_nan=True)
        assert (np.abs(got[ok] - want[ok]) <= 3.01 * 2.0 ** -24 * np.abs(want[ok])).all()


# ---- the gated block -------------------------------------------------------

def act_error(name, g, a):
    z = {"none": 0 * g, "relu": 0 * g, "silu": np.abs(g), "gelu": g * g,
         "gelu_tanh": 3 * np.abs(g) + np.abs(g) ** 3 / 8}[name]
    return 2.0 ** -23 * (8 + 4 * np.minimum(z, 200)) * np.abs(a) + 2.0 ** -120


def product_error(A, B):
    """T 2^-23 S for A.B^T."""
    T = -(-A.shape[1] // 16) + 32
    return T * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T)


def block_error(name, g, u, eg, eu):
    a = o.act(name, g)
    E = act_error(name, np.abs(g) + eg, np.abs(a) + 1.2 * eg)
    return 1.2 * eg * np.abs(u) + np.abs(a) * eu + 1.2 * eg * eu + E * (np.abs(u) + eu) + 2.0 ** -24 * np.abs(a * u)


@pytest.mark.parametrize("act", o.ACTS)
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 100), (5, 70, 256), (33, 100, 65), (100, 130, 192), (300, 200, 512)])
def test_i8_gated(act, t, M, N, K):
    rng = np.random.default_rng(M + 3 * N + K)
    for how in LAYOUTS:
        pad, off = layout(how, K, 16)
        A, G, U = (Mat(codes(rng, r, K), "i8", pad, off) for r in (M, N, N))
        SA, SG, SU = (Mat((rng.random(n) / 64 / np.sqrt(K)).astype(np.float32)[None] * s, "f32")
                      for n, s in ((M, 0.2), (N, 1.0), (N, 1.0)))
        H = Mat(None, t, pad, off, M, N)
        fn("gemm_i8_gated", t)(M, N, K, *A.at, SA.ptr, *G.at, SG.ptr, *U.at, SU.ptr, *H.at, act)
        g, u = o.product(A.value, SA.value[0], G.value, SG.value[0]), o.product(A.value, SA.value[0], U.value, SU.value[0])
        e = 3.01 * 2.0 ** -24
        near(H.get(), o.act(act, g) * u, block_error(act, g, u, e * np.abs(g), e * np.abs(u)), t, f"{how} {act}")


GATED = [(1, 1, 1), (1, 16, 32), (1, 100, 8192), (2, 33, 77), (7, 64, 200), (16, 130, 129), (17, 65, 100), (40, 1000, 64),
         (64, 128, 256), (65, 100, 300), (128, 64, 128), (130, 257, 96), (256, 256, 192), (300, 500, 1000),
         (1000, 1500, 777), (513, 392, 416), (3, 8200, 128)]


def gated_inputs(rng, M, N, K, t, how):
    pad, off = layout(how, K, 8)
    X = Mat(rng.standard_normal((M, K)) * np.exp(0.5 * rng.standard_normal((1, K))), t, pad, off)
    WG, WU = (Mat(1.5 * rng.standard_normal((N, K)) / np.sqrt(K), t, pad, off) for _ in range(2))
    return X, WG, WU


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", GATED)
@pytest.mark.parametrize("how", list(LAYOUTS))
def test_gated(t, M, N, K, how):
    rng = np.random.default_rng(M * 13 + N * 5 + K)
    X, WG, WU = gated_inputs(rng, M, N, K, t, how)
    pad, off = layout(how, N, 8)
    eg, eu = product_error(X.value, WG.value), product_error(X.value, WU.value)
    for act, keep in (("silu", True), ("gelu", False), ("relu", True)):
        H, G, U = (Mat(None, t, pad, off, M, N) for _ in range(3))
        kept = (*G.at, *U.at) if keep else (None, 0, None, 0)
        fn("gemm_gated", t)(M, N, K, *X.at, *WG.at, *WU.at, *kept, *H.at, act)
        h, g, u = o.gated(act, X.value, WG.value, WU.value)
        near(H.get(), h, block_error(act, g, u, eg, eu), t, f"H {M}x{N}x{K} {how} {act}")
        if keep:
            near(G.get(), g, eg, t, "G")
            near(U.get(), u, eu, t, "U")
        else:
            assert G.unchanged() and U.unchanged()
    assert X.unchanged() and WG.unchanged() and WU.unchanged()


@pytest.mark.parametrize("act", o.ACTS)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_activations_over_their_range(act, t):
    """g runs over every size, u is 1: one input channel holds g, another u."""
    for M in (1, 200):
        v = np.concatenate([np.linspace(-40, 40, 3001), [0.0, -0.0, 1e-3, -1e-3, 6e4, -6e4, 90, -90, 300, -300]])
        X = Mat(np.tile([1.0, 0.0], (M, 1)), t)
        WG, WU = Mat(np.stack([v, 0 * v], 1), t), Mat(np.stack([0 * v + 1, 0 * v], 1), t)
        n = len(v)
        H, G, U = (Mat(None, t, 0, 0, M, n) for _ in range(3))
        fn("gemm_gated", t)(M, n, 2, *X.at, *WG.at, *WU.at, *G.at, *U.at, *H.at, act)
        g = WG.value[:, 0][None]
        assert np.array_equal(G.get().double().numpy(), np.tile(g, (M, 1)))
        a = o.act(act, g)
        near(H.get(), np.tile(a, (M, 1)), np.tile(act_error(act, g, a), (M, 1)), t, act)
        DG, DU, DH = Mat(None, t, 0, 0, M, n), Mat(None, t, 0, 0, M, n), Mat(np.ones((M, n)), t)
        fn("gemm_gated_backward", t)(M, n, 2, 0, 2, 0, 2, 0, 2, *G.at, *U.at, *DH.at, *DG.at, *DU.at, None, 0, None, 0,
                                     None, 0, act)
        near(DU.get(), np.tile(a, (M, 1)), np.tile(act_error(act, g, a), (M, 1)), t, act + " dU")
        near(DG.get(), np.tile(o.slope(act, g), (M, 1)), np.full((M, n), 2.0 ** -13), t, act + " dG")


@pytest.mark.parametrize("act", o.ACTS)
def test_what_is_not_a_number_stays_where_it_is(act):
    """A NaN in a row of X reaches that row alone, one in a row of a weight that column
    alone; infinite g of either sign gives no NaN in the gradients of others."""
    for t in ("bf16", "f16"):
        for M, N, K in ((5, 40, 64), (140, 200, 128), (300, 520, 256)):
            rng = np.random.default_rng(3)
            X, WG, WU = (rng.standard_normal(s) for s in ((M, K), (N, K), (N, K)))
            X[1, K - 1], WG[2, 0], WU[3, K // 2] = np.nan, np.nan, np.nan
            d = [torch.from_numpy(v).to(DEV).to(TYPES[t]) for v in (X, WG, WU)]
            H, G, U = (torch.zeros((M, N), dtype=TYPES[t], device=DEV) for _ in range(3))
            fn("gemm_gated", t)(M, N, K, d[0], K, d[1], K, d[2], K, G, N, U, N, H, N, act)
            want = np.zeros((M, N), bool)
            want[1], want[:, 2] = True, True
            assert np.array_equal(torch.isnan(G).cpu().numpy(), want)
            want[:, 2], want[:, 3] = False, True
            want[1] = True
            assert np.array_equal(torch.isnan(U).cpu().numpy(), want)
            want[:, 2] = True
            assert np.array_equal(torch.isnan(H).cpu().numpy(), want)


def backward(t, M, N, K, X, WG, WU, G, U, DH, act, how="whole", dx=True, dw=True):
    pn, on = layout(how, N, 8)
    pk, ok = layout(how, K, 8)
    DG, DU = (Mat(None, t, pn, on, M, N) for _ in range(2))
    DX = Mat(None, t, pk, ok, M, K)
    DWG, DWU = (Mat(None, t, pk, ok, N, K) for _ in range(2))
    none = (None, 0)
    fn("gemm_gated_backward", t)(M, N, K, *(X.at if dw else none), *(WG.at if dx else none), *(WU.at if dx else none),
                                 *G.at, *U.at, *DH.at, *DG.at, *DU.at, *(DX.at if dx else none),
                                 *(DWG.at if dw else none), *(DWU.at if dw else none), act)
    return DG, DU, DX, DWG, DWU


def check_backward(t, act, X, WG, WU, G, U, DH, got, dx=True, dw=True, what=""):
    DG, DU, DX, DWG, DWU = got
    dg, du = o.gated_slopes(act, G.value, U.value, DH.value)
    edg = np.abs(DH.value * U.value) * 2.0 ** -13 + 3 * 2.0 ** -24 * np.abs(dg) + 2.0 ** -120
    a = o.act(act, G.value)
    edu = np.abs(DH.value) * act_error(act, G.value, a) + 2.0 ** -24 * np.abs(du)
    gdg, gdu = DG.get(), DU.get()
    near(gdg, dg, edg, t, what + " dG")
    near(gdu, du, edu, t, what + " dU")
    # the products are those of dG and dU as rounded
    gdg, gdu = gdg.double().numpy(), gdu.double().numpy()
    px, pg, pu = o.gated_products(gdg, gdu, X.value, WG.value, WU.value)
    if dx:
        e = product_error(np.concatenate([gdg, gdu], 1), np.concatenate([WG.value, WU.value], 0).T)
        near(DX.get(), px, e, t, what + " dX")
    else:
        assert DX.unchanged()
    if dw:
        near(DWG.get(), pg, product_error(gdg.T, X.value.T), t, what + " dWg")
        near(DWU.get(), pu, product_error(gdu.T, X.value.T), t, what + " dWu")
    else:
        assert DWG.unchanged() and DWU.unchanged()


BACKWARD = [(1, 1, 1), (1, 64, 32), (2, 33, 77), (7, 64, 200), (16, 130, 129), (32, 128, 128), (33, 65, 100), (64, 32, 256),
            (65, 100, 300), (96, 160, 320), (129, 257, 191), (256, 256, 256), (300, 512, 264), (1000, 1500, 777),
            (1500, 200, 136), (320, 544, 1000)]


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("how", list(LAYOUTS))
def test_gated_backward(t, M, N, K, how):
    rng = np.random.default_rng(M * 11 + N * 3 + K)
    X, WG, WU = gated_inputs(rng, M, N, K, t, how)
    pad, off = layout(how, N, 8)
    G, U, DH = (Mat(rng.standard_normal((M, N)) * s, t, pad, off) for s in (2.0, 1.0, 0.1))
    got = backward(t, M, N, K, X, WG, WU, G, U, DH, "silu", how)
    check_backward(t, "silu", X, WG, WU, G, U, DH, got, what=f"{M}x{N}x{K} {how}")
    assert all(m.unchanged() for m in (X, WG, WU, G, U, DH))


@pytest.mark.parametrize("act", o.ACTS)
def test_gated_backward_in_parts(act):
    M, N, K = 70, 96, 136
    for t in ("bf16", "f16"):
        rng = np.random.default_rng(8)
        X, WG, WU = gated_inputs(rng, M, N, K, t, "whole")
        G, U, DH = (Mat(rng.standard_normal((M, N)), t) for _ in range(3))
        for dx, dw in ((True, True), (True, False), (False, True), (False, False)):
            got = backward(t, M, N, K, X, WG, WU, G, U, DH, act, "whole", dx, dw)
            check_backward(t, act, X, WG, WU, G, U, DH, got, dx, dw, act)


def test_empty_sums_store_zeros():
    for t in ("bf16", "f16"):
        for M, N in ((1, 40), (20, 33), (300, 200)):
            H, G, U = (Mat(None, t, 3, 0, M, N) for _ in range(3))
            fn("gemm_gated", t)(M, N, 0, 0, 1, 0, 1, 0, 1, *G.at, *U.at, *H.at, "silu")
            for m in (H, G, U):
                assert not m.get().any()
            H = Mat(None, t, 3, 0, M, N)
            fn("gemm_i8_gated", t)(M, N, 0, 0, 1, 0, 0, 1, 0, 0, 1, 0, *H.at, "gelu")
            assert not H.get().any()
            C = Mat(None, "f32", 3, 0, M, N)
            b.gemm_i8_f32(M, N, 0, 0, 1, 0, 0, 1, 0, *C.at)
            assert not C.get().any()
        N, K = 40, 72                                  # no tokens: the weights' gradients are zero
        DWG, DWU = Mat(None, t, 0, 0, N, K), Mat(None, t, 0, 0, N, K)
        fn("gemm_gated_backward", t)(0, N, K, 0, K, 0, K, 0, K, 0, N, 0, N, 0, N, 0, N, 0, N, None, 0, *DWG.at, *DWU.at, 2)
        assert not DWG.get().any() and not DWU.get().any()
        DX = Mat(None, t, 0, 0, 30, K)                 # no features: the input's gradient is zero
        fn("gemm_gated_backward", t)(30, 0, K, 0, K, 0, K, 0, K, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1, *DX.at, None, 0, None, 0, 2)
        assert not DX.get().any()


def test_gradients_are_the_differences_of_the_forward_pass():
    """sum(H DH) from the library's forward kernel, differentiated by steps of X: the
    weights' and inputs' values are whole multiples that 16 bits hold, DH one row of
    ones, so that only H's own rounding, half a step of each of N outputs, and the
    curvature stand between the two."""
    M, N, K, t = 4, 64, 32, "f16"
    rng = np.random.default_rng(12)
    X = rng.integers(-8, 9, (M, K)) / 8.0
    WG, WU = (rng.integers(-8, 9, (N, K)) / 32.0 for _ in range(2))
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(DEV).to(torch.float16)  # noqa: E731

    def total(x):
        H = torch.empty((M, N), dtype=torch.float16, device=DEV)
        xd, gd, ud = dev(x), dev(WG), dev(WU)
        b.gemm_gated_f16(M, N, K, xd, K, gd, K, ud, K, None, 0, None, 0, H, N, "silu")
        return H.double().sum(1).cpu().numpy(), H.double().abs().sum(1).cpu().numpy()

    G, U = X @ WG.T, X @ WU.T
    mats = [Mat(v, t) for v in (X, WG, WU, G, U, np.ones((M, N)))]
    got = backward(t, M, N, K, *mats, "silu")
    dx = got[2].get().double().numpy()
    h = 0.125
    for k in range(0, K, 5):
        E = np.zeros((M, K))
        E[:, k] = h
        (up, s1), (down, s2) = total(X + E), total(X - E)
        # third derivative of act(g) u along the step: |w|^3 (|act'''| |u| + 3 |act''|) <= N w^3 (|u| + 1.5)
        curve = h * h / 6 * (np.abs(WG[:, k]) ** 2 * (np.abs(WG[:, k]) * (np.abs(U) + 1) + 3 * 0.5 * np.abs(WU[:, k]))).sum(1)
        rounding = 2.0 ** -11 * (s1 + s2) / (2 * h) + N * 2.0 ** -24 / h
        own = 2.0 ** -11 * np.abs(dx[:, k]) + 2.0 ** -10 * (np.abs(WG[:, k]) * np.abs(U) * 1.1 + np.abs(WU[:, k] * G)).sum(1)
        assert (np.abs((up - down) / (2 * h) - dx[:, k]) <= curve + rounding + own).all()


# ---- together --------------------------------------------------------------

@pytest.mark.parametrize("M,D,F", [(1, 256, 512), (5, 200, 333), (130, 320, 448)])
def test_served_layer(M, D, F):
    """Tokens quantised, the gated block, its result quantised, the down projection:
    each step against the definition on what the step before gave."""
    t = "bf16"
    rng = np.random.default_rng(D)
    X = Mat(rng.standard_normal((M, D)), t)
    W = [o.quantize(np.float32(rng.standard_normal(s) * 0.05)) for s in ((F, D), (F, D), (D, F))]
    (G, SG), (U, SU), (Dn, SD) = [(Mat(q, "i8"), Mat(s[None], "f32")) for q, s in W]
    Q, S, H = Mat(None, "i8", 0, 0, M, D), Mat(None, "f32", 0, 0, 1, M), Mat(None, t, 0, 0, M, F)
    HQ, HS, Y = Mat(None, "i8", 0, 0, M, F), Mat(None, "f32", 0, 0, 1, M), Mat(None, t, 0, 0, M, D)
    b.gemm_i8_quantize_bf16(M, D, *X.at, *Q.at, S.ptr)
    b.gemm_i8_gated_bf16(M, F, D, *Q.at, S.ptr, *G.at, SG.ptr, *U.at, SU.ptr, *H.at, "silu")
    b.gemm_i8_quantize_bf16(M, F, *H.at, *HQ.at, HS.ptr)
    b.gemm_i8_bf16(M, D, F, *HQ.at, HS.ptr, *Dn.at, SD.ptr, *Y.at)
    q, s = o.quantize(X.value)
    assert np.array_equal(Q.get().numpy(), q) and np.array_equal(S.get().numpy()[0], s)
    g, u = o.product(q, s, *W[0]), o.product(q, s, *W[1])
    e = 3.01 * 2.0 ** -24
    h = H.get()
    near(h, o.act("silu", g) * u, block_error("silu", g, u, e * np.abs(g), e * np.abs(u)), t, "H")
    q, s = o.quantize(h.double().numpy())
    assert np.array_equal(HQ.get().numpy(), q) and np.array_equal(HS.get().numpy()[0], s)
    want = o.product(q, s, *W[2])
    near(Y.get(), want, e * np.abs(want), t, "Y")


def test_training_step():
    """Forward keeping G and U, backward on them."""
    for t in ("bf16", "f16"):
        M, N, K = 160, 288, 224
        rng = np.random.default_rng(21)
        X, WG, WU = gated_inputs(rng, M, N, K, t, "whole")
        DH = Mat(0.1 * rng.standard_normal((M, N)), t)
        G, U, H = (Mat(None, t, 0, 0, M, N) for _ in range(3))
        fn("gemm_gated", t)(M, N, K, *X.at, *WG.at, *WU.at, *G.at, *U.at, *H.at, "gelu_tanh")
        G.value, U.value = G.get().double().numpy(), U.get().double().numpy()
        got = backward(t, M, N, K, X, WG, WU, G, U, DH, "gelu_tanh")
        check_backward(t, "gelu_tanh", X, WG, WU, G, U, DH, got)


def some_calls(M, N, K, stream=None):
    """Operands of every kind of call, and a function that makes them all."""
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    x, wg, wu, dh = r(M, K).bfloat16(), (r(N, K) / 8).bfloat16(), (r(N, K) / 8).bfloat16(), r(M, N).bfloat16()
    e = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    q, s, qg, sg, qu, su = e(M, K, dtype=torch.int8), e(M, dtype=torch.float32), e(N, K, dtype=torch.int8), \
        e(N, dtype=torch.float32), e(N, K, dtype=torch.int8), e(N, dtype=torch.float32)
    h, g, u, dg, du, dx, dwg, dwu, hi = e(M, N), e(M, N), e(M, N), e(M, N), e(M, N), e(M, K), e(N, K), e(N, K), e(M, N)
    c, y = e(M, N, dtype=torch.float32), e(M, K)

    def call():
        for a, b_, c_ in ((x, q, s), (wg, qg, sg), (wu, qu, su)):
            b.gemm_i8_quantize_bf16(a.shape[0], K, a, K, b_, K, c_, stream)
        b.gemm_i8_dequantize_bf16(M, K, q, K, s, y, K, stream)
        b.gemm_i8_f32(M, N, K, q, K, s, qg, K, sg, c, N, stream)
        b.gemm_i8_gated_bf16(M, N, K, q, K, s, qg, K, sg, qu, K, su, hi, N, "silu", stream)
        b.gemm_gated_bf16(M, N, K, x, K, wg, K, wu, K, g, N, u, N, h, N, "silu", stream)
        b.gemm_gated_backward_bf16(M, N, K, x, K, wg, K, wu, K, g, N, u, N, dh, N, dg, N, du, N, dx, K, dwg, K, dwu, K,
                                   "silu", stream)

    return call, (x, dh), (q, s, y, c, hi, h, g, u, dg, du, dx, dwg, dwu)


@pytest.mark.parametrize("M,N,K", [(1, 256, 128), (40, 256, 128), (300, 520, 256)])
def test_captured_and_replayed(M, N, K):
    """A graph of all of them, replayed with other inputs and eager work between."""
    call, inputs, outputs = some_calls(M, N, K)
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for i in range(4):
        gen = torch.Generator(device=DEV).manual_seed(i)
        for t in inputs:
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outputs]
        for t in outputs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outputs, want):
            assert torch.equal(t, w), i


def test_four_host_threads():
    jobs = [some_calls(*s) for s in ((1, 200, 100), (33, 256, 128), (130, 300, 264), (300, 512, 256))]
    for call, _, _ in jobs:
        call()
    torch.cuda.synchronize()
    want = [[t.clone() for t in out] for _, _, out in jobs]
    errors = []

    def work(call, out, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    call()
            torch.cuda.synchronize()
            for t, w in zip(out, want):
                assert torch.equal(t, w)
        except Exception as e:  # pragma: no cover - reported below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c, out, w)) for (c, _, out), w in zip(jobs, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors


def test_results_repeat():
    """The same bits from call to call."""
    call, _, outputs = some_calls(300, 776, 1000)
    call()
    first = [t.clone() for t in outputs]
    for _ in range(3):
        for t in outputs:
            t.zero_()
        call()
        for t, w in zip(outputs, first):
            assert torch.equal(t, w)


def test_offsets_past_32_bits():
    """Rows that lie past 4 GiB: the weights of 2^19 outputs of 5000 inputs are read, and
    outputs 2^31 elements apart are written."""
    N, K, ld = 1 << 19, 64, 8704                          # 4.56 GB of codes
    B = torch.zeros((N, ld), dtype=torch.int8, device=DEV)
    B[:, :K] = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    one = torch.ones(N, device=DEV)
    for M in (1, 3, 100):
        A = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV)
        C = torch.empty((M, N), device=DEV)
        b.gemm_i8_f32(M, N, K, A, K, one, B, ld, one, C, N)
        want = A.float() @ B[:, :K].float().t()          # below 2^24: exact
        assert torch.equal(C, want), M
    del B, C, want
    M, N, K, ld = 130, 64, 64, 1 << 25                    # rows of C 64 MB apart: 8.7 GB
    H = torch.zeros((M, ld), dtype=torch.bfloat16, device=DEV)
    X, W = torch.randn((M, K), device=DEV).bfloat16(), torch.randn((N, K), device=DEV).bfloat16()
    b.gemm_gated_bf16(M, N, K, X, K, W, K, W, K, None, 0, None, 0, H, ld, "none")
    small = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    b.gemm_gated_bf16(M, N, K, X, K, W, K, W, K, None, 0, None, 0, small, N, "none")
    assert torch.equal(H[:, :N], small) and not H[:, N:N + 64].any()
    DH = H                                               # the slopes and products read such rows too
    dg, du, dx, dw1, dw2 = (torch.zeros(s, dtype=torch.bfloat16, device=DEV)
                            for s in ((M, N), (M, N), (M, K), (N, K), (N, K)))
    b.gemm_gated_backward_bf16(M, N, K, X, K, W, K, W, K, DH, ld, DH, ld, DH, ld, dg, N, du, N, dx, K, dw1, K, dw2, K, "none")
    assert torch.equal(dg, (small.float() * small.float()).bfloat16())
    s = small.contiguous()
    dx2 = torch.zeros_like(dx)
    b.gemm_gated_backward_bf16(M, N, K, X, K, W, K, W, K, s, N, s, N, s, N, dg, N, du, N, dx2, K, dw1, K, dw2, K, "none")
    assert torch.equal(dx, dx2)


def test_another_stream_is_the_current_one():
    """Tensors are used on the current stream, behind what it holds."""
    M, N, K = 64, 512, 256
    side = torch.cuda.Stream()
    x = torch.randn((M, K), device=DEV).bfloat16()
    w = torch.randn((N, K), device=DEV).bfloat16()
    ref, H = (torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    b.gemm_gated_bf16(M, N, K, x, K, w, K, w, K, None, 0, None, 0, ref, N)
    torch.cuda.synchronize()
    y = torch.zeros_like(x)
    big = torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            big = big @ big * 1e-3
        y.copy_(x)
        b.gemm_gated_bf16(M, N, K, y, K, w, K, w, K, None, 0, None, 0, H, N)
    torch.cuda.synchronize()
    assert torch.equal(H, ref)


def test_checks_hold_after_a_first_call():
    """What the binding refuses it refuses also where the same entry point has run."""
    M, N, K = 8, 24, 32
    i8 = torch.randint(-9, 9, (N, K), dtype=torch.int8, device=DEV)
    A, S = i8[:M], torch.ones(N, device=DEV)
    X, H = torch.randn((N, K), device=DEV).bfloat16(), torch.zeros((M, N), device=DEV).bfloat16()
    C, Q = torch.zeros((M, N), device=DEV), torch.zeros_like(i8)
    mm = lambda A=A, SA=S, C=C, M=M, ldc=N: b.gemm_i8_f32(M, N, K, A, K, SA, i8, K, S, C, ldc)  # noqa: E731
    cast = lambda X=X, Q=Q, S=S, R=N: b.gemm_i8_quantize_bf16(R, K, X, K, Q, K, S)  # noqa: E731
    back = lambda Q=Q, S=S, Y=X, C=K: b.gemm_i8_dequantize_bf16(N, C, Q, K, S, Y, K)  # noqa: E731
    gated = lambda X=X, H=H, act="silu", K=K: b.gemm_gated_bf16(  # noqa: E731
        M, N, K, X, 32, X, 32, X, 32, None, 0, None, 0, H, N, act)
    for call in (mm, cast, back, gated):
        for _ in range(2):
            assert call() == b.SGEMM_OK
    for call, wrong in ((mm, dict(A=X)), (mm, dict(SA=X)), (mm, dict(C=H)), (cast, dict(X=C)), (cast, dict(Q=X)),
                        (back, dict(S=H)), (back, dict(Y=C)), (gated, dict(X=X.half())), (gated, dict(H=C))):
        with pytest.raises(TypeError):
            call(**wrong)
    for call, wrong in ((mm, dict(A=A.cpu())), (mm, dict(SA=S[:M - 1])), (mm, dict(SA=torch.ones(2 * N, device=DEV)[::2])),
                        (cast, dict(S=S[:3])), (cast, dict(X=X.cpu())), (back, dict(S=S[::2])), (back, dict(Q=Q.cpu())),
                        (gated, dict(H=H.cpu())), (mm, dict(M=1 << 32)), (cast, dict(R=1 << 31))):   # too few scales
        with pytest.raises(ValueError):
            call(**wrong)
    for call, wrong in ((mm, dict(ldc=-1 << 40)), (mm, dict(ldc=1 << 31)), (back, dict(C=1 << 35)),
                        (gated, dict(K=1 << 31)), (gated, dict(act=1 << 33))):
        with pytest.raises(OverflowError):
            call(**wrong)
    for call, wrong in ((mm, dict(M=-1)), (mm, dict(ldc=N - 1)), (cast, dict(R=-5)), (gated, dict(act=5)), (gated, dict(K=33))):
        with pytest.raises(b.SgemmError):
            call(**wrong)
    with pytest.raises(KeyError):
        gated(act="tanh")
    torch.cuda.synchronize()
