"""CPU tests of the 8-bit integer operators and the gated block: the float64
definition (oracle/layer.py) against rational arithmetic, differences and torch's
own activations, and every refusal of the entry points (fake addresses, never
dereferenced; no call here reaches a launch)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import layer as o
from register_lds_tiled_amd import binding as b

F = 0x10000000
STEP = 1 << 24


# ---- the definition --------------------------------------------------------

def test_quantize_is_the_nearest_whole_number():
    rng = np.random.default_rng(1)
    X = np.float32(rng.standard_normal((40, 50)) * np.exp2(rng.integers(-140, 120, (40, 1)))).astype(np.float64)
    X[3] = 0.0
    X[4] = np.float32(2.0 ** -149) * rng.integers(-3, 4, 50)
    X[5, 7], X[6, 0] = np.nan, -np.inf
    Q, S = o.quantize(X)
    assert np.isnan(S[5]) and np.isnan(S[6]) and not Q[5].any() and not Q[6].any()
    for r in range(40):
        if r in (5, 6):
            continue
        top = max(Fraction(float(v)) if v >= 0 else -Fraction(float(v)) for v in X[r])
        s = Fraction(float(S[r]))
        exact = top / 127
        if exact < Fraction(2) ** -126:
            assert s == Fraction(2) ** -126
        else:
            assert abs(s - exact) <= exact * Fraction(1, 2 ** 24)
        for c in range(50):
            q, x = Fraction(int(Q[r, c])), Fraction(float(X[r, c]))
            d = abs(x - q * s)
            assert d <= s / 2
            if d == s / 2:
                assert int(Q[r, c]) % 2 == 0


def test_quantize_ties_go_to_even():
    X = np.zeros((1, 300))
    X[0, 0] = 127.0                                  # the scale is exactly 1
    X[0, 1:254] = np.arange(-126, 127) + 0.5
    Q, S = o.quantize(X)
    assert S[0] == 1.0
    assert (Q[0, 1:254] % 2 == 0).all()


def test_product_is_exact():
    rng = np.random.default_rng(2)
    A, B = rng.integers(-128, 128, (5, 33)).astype(np.int8), rng.integers(-128, 128, (7, 33)).astype(np.int8)
    SA, SB = rng.random(5).astype(np.float32), rng.random(7).astype(np.float32)
    C = o.product(A, SA, B, SB)
    for i in range(5):
        for j in range(7):
            want = sum(int(x) * int(y) for x, y in zip(A[i], B[j])) * Fraction(float(SA[i])) * Fraction(float(SB[j]))
            assert abs(Fraction(float(C[i, j])) - want) <= abs(want) * Fraction(1, 2 ** 51)


@pytest.mark.parametrize("name", o.ACTS)
def test_slopes_are_the_activations_differences(name):
    x = np.linspace(-9, 9, 721) + 0.0003
    h = 1e-5
    d = (o.act(name, x + h) - o.act(name, x - h)) / (2 * h)
    # the difference's own error: h^2 / 6 of the third derivative (at most 3 here), and 2^-52 |a| / h
    assert np.abs(d - o.slope(name, x)).max() <= 3 * h * h / 6 + 2 ** -52 * 10 / h


def test_activations_are_the_usual_ones():
    torch = pytest.importorskip("torch")
    x = torch.linspace(-12, 12, 997, dtype=torch.float64)
    want = {"none": x, "relu": torch.relu(x), "silu": torch.nn.functional.silu(x),
            "gelu": torch.nn.functional.gelu(x), "gelu_tanh": torch.nn.functional.gelu(x, approximate="tanh")}
    for name, y in want.items():
        assert np.abs(o.act(name, x.numpy()) - y.numpy()).max() <= 1e-14


@pytest.mark.parametrize("name", o.ACTS)
def test_gradients_are_the_blocks_differences(name):
    """sum(H * DH) differentiated by its inputs, against the formulas."""
    rng = np.random.default_rng(5)
    X, WG, WU = (rng.standard_normal(s) for s in ((4, 6), (5, 6), (5, 6)))
    DH = rng.standard_normal((4, 5))
    H, G, U = o.gated(name, X, WG, WU)
    DG, DU = o.gated_slopes(name, G, U, DH)
    got = dict(zip("XGU", o.gated_products(DG, DU, X, WG, WU)))
    h = 1e-6
    for key, M in (("X", X), ("G", WG), ("U", WU)):
        for at in np.ndindex(M.shape):
            was = M[at]
            M[at] = was + h
            up = (o.gated(name, X, WG, WU)[0] * DH).sum()
            M[at] = was - h
            down = (o.gated(name, X, WG, WU)[0] * DH).sum()
            M[at] = was
            assert abs((up - down) / (2 * h) - got[key][at]) <= 1e-7 * max(1.0, np.abs(got[key]).max())


# ---- refusals --------------------------------------------------------------

def test_quantize_refusals():
    for t, size in (("f32", 4), ("bf16", 2), ("f16", 2)):
        f = lambda *a: getattr(b, f"gemm_i8_quantize_{t}")(*a, 0, check=False)  # noqa: E731,B023
        X, Q, S = F, F + STEP, F + 2 * STEP
        assert f(-1, 8, X, 8, Q, 8, S) == b.SGEMM_EINVAL_DIM
        assert f(8, -1, X, 8, Q, 8, S) == b.SGEMM_EINVAL_DIM
        assert f(8, 8, X, 7, Q, 8, S) == b.SGEMM_EINVAL_LD
        assert f(8, 8, X, 8, Q, 7, S) == b.SGEMM_EINVAL_LD
        assert f(8, 0, X, 0, Q, 1, S) == b.SGEMM_EINVAL_LD
        assert f(0, 8, 0, 8, 0, 8, 0) == b.SGEMM_OK
        assert f(8, 0, 0, 1, 0, 1, 0) == b.SGEMM_OK
        for args in ((0, 8, Q, 8, S), (X, 8, 0, 8, S), (X, 8, Q, 8, 0)):
            assert f(8, 8, *args) == b.SGEMM_EINVAL_PTR
        assert f(8, 8, X, 8, X + 64 * size - 1, 8, S) == b.SGEMM_EALIAS
        assert f(8, 8, X, 8, Q, 8, Q + 60) == b.SGEMM_EALIAS
        assert f(8, 8, X, 8, Q, 8, X + 64 * size - 4) == b.SGEMM_EALIAS
        assert f(2 ** 31 - 1, 2 ** 31 - 1, X, 2 ** 31 - 1, Q, 2 ** 31 - 1, S) == b.SGEMM_EALIAS
        assert f(8, 8, 2 ** 64 - 64, 8, Q, 8, S) == b.SGEMM_EINVAL_DIM


def test_dequantize_refusals():
    for t, size in (("f32", 4), ("bf16", 2), ("f16", 2)):
        f = lambda *a: getattr(b, f"gemm_i8_dequantize_{t}")(*a, 0, check=False)  # noqa: E731,B023
        Q, S, Y = F, F + STEP, F + 2 * STEP
        assert f(-1, 8, Q, 8, S, Y, 8) == b.SGEMM_EINVAL_DIM
        assert f(8, 8, Q, 7, S, Y, 8) == b.SGEMM_EINVAL_LD
        assert f(8, 8, Q, 8, S, Y, 7) == b.SGEMM_EINVAL_LD
        assert f(0, 8, 0, 8, 0, 0, 8) == b.SGEMM_OK
        for args in ((0, 8, S, Y, 8), (Q, 8, 0, Y, 8), (Q, 8, S, 0, 8)):
            assert f(8, 8, *args) == b.SGEMM_EINVAL_PTR
        assert f(8, 8, Q, 8, S, Q + 63, 8) == b.SGEMM_EALIAS
        assert f(8, 8, Q, 8, S, S - 64 * size + 1, 8) == b.SGEMM_EALIAS


@pytest.mark.parametrize("out,size", [("f32", 4), ("bf16", 2), ("f16", 2)])
def test_i8_product_refusals(out, size):
    f = lambda *a: getattr(b, f"gemm_i8_{out}")(*a, 0, check=False)  # noqa: E731
    A, SA, B, SB, C = (F + i * STEP for i in range(5))
    ok = (A, 8, SA, B, 8, SB, C, 8)
    for dims in ((-1, 8, 8), (8, -1, 8), (8, 8, -1)):
        assert f(*dims, *ok) == b.SGEMM_EINVAL_DIM
    assert f(8, 8, 131072, A, 131072, SA, B, 131072, SB, C, 8) == b.SGEMM_EINVAL_DIM
    assert f(8, 8, 8, A, 7, SA, B, 8, SB, C, 8) == b.SGEMM_EINVAL_LD
    assert f(8, 8, 8, A, 8, SA, B, 7, SB, C, 8) == b.SGEMM_EINVAL_LD
    assert f(8, 8, 8, A, 8, SA, B, 8, SB, C, 7) == b.SGEMM_EINVAL_LD
    for i in (0, 2, 3, 5, 6):
        args = list(ok)
        args[i] = 0
        assert f(8, 8, 8, *args) == b.SGEMM_EINVAL_PTR
    assert f(0, 8, 8, 0, 8, 0, 0, 8, 0, 0, 8) == b.SGEMM_OK
    assert f(8, 0, 8, 0, 8, 0, 0, 8, 0, 0, 1) == b.SGEMM_OK
    end = 64 * size
    for at in (A - end + 1, A + 63, SA - end + 4, SA + 28, B - end + 1, B + 63, SB - end + 4, SB + 28):
        assert f(8, 8, 8, A, 8, SA, B, 8, SB, at, 8) == b.SGEMM_EALIAS, hex(at)
    far = 1 << 44
    assert f(2 ** 31 - 1, 2 ** 31 - 1, 8, far, 8, far, far, 8, far, 3 * far, 2 ** 31 - 1) == b.SGEMM_EINVAL_DIM
    assert f(8, 8, 8, 2 ** 64 - 32, 8, SA, B, 8, SB, C, 8) == b.SGEMM_EINVAL_DIM


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_i8_gated_refusals(t):
    f = lambda *a, act=2: getattr(b, f"gemm_i8_gated_{t}")(*a, act, 0, check=False)  # noqa: E731
    A, SA, G, SG, U, SU, H = (F + i * STEP for i in range(7))
    ok = (A, 8, SA, G, 8, SG, U, 8, SU, H, 8)
    for act in (-1, 5):
        assert f(-1, 8, 8, *ok, act=act) == b.SGEMM_EINVAL_ACT
    assert f(8, 8, 131072, A, 131072, SA, G, 131072, SG, U, 131072, SU, H, 8) == b.SGEMM_EINVAL_DIM
    assert f(8, 8, -1, *ok) == b.SGEMM_EINVAL_DIM
    for i in (1, 4, 7, 10):
        args = list(ok)
        args[i] = 7
        assert f(8, 8, 8, *args) == b.SGEMM_EINVAL_LD
    for i in (0, 2, 3, 5, 6, 8, 9):
        args = list(ok)
        args[i] = 0
        assert f(8, 8, 8, *args) == b.SGEMM_EINVAL_PTR
    for at in (A + 62, SA + 28, G + 62, SG + 28, U + 62, SU + 28):
        assert f(8, 8, 8, *ok[:-2], at, 8) == b.SGEMM_EALIAS
    assert f(0, 8, 8, *ok) == b.SGEMM_OK


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_gated_refusals(t):
    f = lambda *a, act=2: getattr(b, f"gemm_gated_{t}")(*a, act, 0, check=False)  # noqa: E731
    X, WG, WU, G, U, H = (F + i * STEP for i in range(6))
    ok = (X, 8, WG, 8, WU, 8, G, 8, U, 8, H, 8)
    for act in (-1, 5):
        assert f(-1, 8, 8, *ok, act=act) == b.SGEMM_EINVAL_ACT
    for dims in ((-1, 8, 8), (8, -1, 8), (8, 8, -1)):
        assert f(*dims, *ok) == b.SGEMM_EINVAL_DIM
    for i in range(1, 12, 2):
        args = list(ok)
        args[i] = 7
        assert f(8, 8, 8, *args) == b.SGEMM_EINVAL_LD
    for i in range(0, 12, 2):                        # one of G and U alone included
        args = list(ok)
        args[i] = 0
        assert f(8, 8, 8, *args) == b.SGEMM_EINVAL_PTR
    for at in (X + 126, WG + 126, WU + 126, G - 126, U + 126):
        assert f(8, 8, 8, *ok[:-2], at, 8) == b.SGEMM_EALIAS
    for i, at in ((6, X + 126), (8, WG + 126), (6, U + 2), (8, WU - 126)):
        args = list(ok)
        args[i] = at
        assert f(8, 8, 8, *args) == b.SGEMM_EALIAS
    assert f(0, 8, 8, 0, 8, 0, 8, 0, 8, 0, 0, 0, 0, 0, 8) == b.SGEMM_OK   # G, U not asked: no ld
    assert f(8, 0, 8, *ok) == b.SGEMM_OK
    far = 1 << 44
    assert f(2 ** 31 - 1, 2 ** 31 - 1, 8, far, 8, far, 8, far, 8, 0, 0, 0, 0, 3 * far, 2 ** 31 - 1) == b.SGEMM_EINVAL_DIM


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_gated_backward_refusals(t):
    f = lambda *a, act=2: getattr(b, f"gemm_gated_backward_{t}")(*a, act, 0, check=False)  # noqa: E731
    names = ("X", "WG", "WU", "G", "U", "DH", "DG", "DU", "DX", "DWG", "DWU")
    at = {n: F + i * STEP for i, n in enumerate(names)}

    def args(**change):
        out = []
        for n in names:
            out += [change.get(n, at[n]), change.get("ld" + n, 8)]
        return out

    for act in (-1, 5):
        assert f(-1, 8, 8, *args(), act=act) == b.SGEMM_EINVAL_ACT
    for dims in ((-1, 8, 8), (8, -1, 8), (8, 8, -1)):
        assert f(*dims, *args()) == b.SGEMM_EINVAL_DIM
    for n in names:
        assert f(8, 8, 8, *args(**{"ld" + n: 7})) == b.SGEMM_EINVAL_LD, n
    for n in names:
        if n == "DX":
            continue
        assert f(8, 8, 8, *args(**{n: 0})) == b.SGEMM_EINVAL_PTR, n
    # what is not asked is not looked at, what is left still is
    assert f(8, 8, 8, *args(DX=0, ldDX=0, WG=0, ldWG=0, WU=0, ldWU=0, DH=0)) == b.SGEMM_EINVAL_PTR
    assert f(8, 8, 8, *args(DX=0, ldDX=0, ldWG=0, ldWU=0, ldDH=7)) == b.SGEMM_EINVAL_LD
    assert f(8, 8, 8, *args(DWG=0, DWU=0, ldDWG=0, ldDWU=0, X=0, ldX=0, DH=0)) == b.SGEMM_EINVAL_PTR
    outputs, inputs = ("DG", "DU", "DX", "DWG", "DWU"), ("X", "WG", "WU", "G", "U", "DH")
    for n in outputs:
        for m in inputs:
            assert f(8, 8, 8, *args(**{n: at[m] + 126})) == b.SGEMM_EALIAS, (n, m)
            assert f(8, 8, 8, *args(**{n: at[m] - 126})) == b.SGEMM_EALIAS, (n, m)
        for m in outputs:
            if n != m:
                assert f(8, 8, 8, *args(**{n: at[m]})) == b.SGEMM_EALIAS, (n, m)
    assert f(0, 0, 8, *args()) == b.SGEMM_OK
    assert f(0, 8, 8, *args(DWG=0, DWU=0)) == b.SGEMM_OK        # no tokens, no weight gradients asked
    assert f(8, 0, 8, *args(DX=0)) == b.SGEMM_OK
    assert f(0, 8, 0, *args()) == b.SGEMM_OK
    top = 2 ** 31 - 1
    far = {n: (i + 1) << 58 for i, n in enumerate(names)}
    assert f(top, top, 8, *args(**far, ldG=top, ldU=top, ldDH=top, ldDG=top, ldDU=top)) == b.SGEMM_EINVAL_DIM


def test_binding_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 4), dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(ValueError):                  # not on the GPU
        b.gemm_i8_f32(4, 4, 4, x, 4, s, x, 4, s, torch.zeros(4, 4), 4)
    with pytest.raises(TypeError):                   # unsigned bytes
        b.gemm_i8_f32(4, 4, 4, x.view(torch.uint8), 4, s, x, 4, s, torch.zeros(4, 4), 4)
    with pytest.raises(ValueError):                  # too few scales
        b.gemm_i8_f32(4, 4, 4, x, 4, s[:3], x, 4, s, torch.zeros(4, 4), 4)
    with pytest.raises(ValueError):                  # scales apart
        b.gemm_i8_f32(4, 4, 4, x, 4, torch.zeros(8)[::2], x, 4, s, torch.zeros(4, 4), 4)
    with pytest.raises(KeyError):
        b.gemm_gated_bf16(4, 4, 4, F, 4, F, 4, F, 4, 0, 0, 0, 0, F, 4, "swish")
    for n in (2 ** 31, -2 ** 31 - 1):
        with pytest.raises(OverflowError):
            b.gemm_gated_bf16(n, 4, 4, F, 4, F, 4, F, 4, 0, 0, 0, 0, F, 4, 0, 0)
        with pytest.raises(OverflowError):
            b.gemm_gated_bf16(4, 4, 4, F, n, F, 4, F, 4, 0, 0, 0, 0, F, 4, 0, 0)
        with pytest.raises(OverflowError):
            b.gemm_gated_bf16(4, 4, 4, F, 4, F, 4, F, 4, 0, 0, 0, 0, F, 4, n, 0)
