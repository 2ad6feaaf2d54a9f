"""GPU tests of the gated block's gradients where G or U holds infinities: gate sums
that 16 bits do not hold.  The forward pass takes act of the fp32 sum, so a finite
sum below its type's range gives a finite H, and the gradients at the -infinity
that G keeps of it are act's and its slope's limits there: 0 of SiLU and both forms
of GELU.  Bounds as in test_gpu_layer.py; which entries are infinite or no number
is compared exactly."""
import numpy as np
import pytest

from oracle import layer as o
from register_lds_tiled_amd import binding as b
from tests.test_gpu_layer import Mat, act_error, backward, fn, near, product_error

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CURVED = ("silu", "gelu", "gelu_tanh")
TOP = {"f16": 65504.0, "bf16": 3.3895313892515355e38}


def limits(act, g):
    """act and its slope, at an infinity their limits."""
    inf = np.isinf(g)
    a, d = o.act(act, np.where(inf, 0, g)), o.slope(act, np.where(inf, 0, g))
    up = g == np.inf
    low = {"none": -np.inf}.get(act, 0.0)
    a = np.where(inf, np.where(up, np.inf, low), a)
    d = np.where(inf, np.where(up, 1.0, 1.0 if act == "none" else 0.0), d)
    return a, d


@pytest.mark.parametrize("act", o.ACTS)
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(5, 40, 64), (140, 200, 128), (33, 65, 100)])
def test_infinite_gates(act, t, M, N, K):
    """G with both infinities and both largest numbers, each in a row and a column of
    its own; no gradient anywhere is NaN, and infinite are those that +infinity (of
    the identity also -infinity) reaches."""
    rng = np.random.default_rng(M + K)
    X, WG, WU = (np.where(rng.random(s) < 0.5, -1.0, 1.0) * (0.5 + rng.random(s)) for s in ((M, K), (N, K), (N, K)))
    G, U, DH = rng.standard_normal((M, N)), rng.standard_normal((M, N)), 0.1 * rng.standard_normal((M, N)) + 0.01
    G[1, 2], G[2, 9], G[3, 17], G[4, 30] = -np.inf, np.inf, -TOP[t], TOP[t] / 64
    X, WG, WU, G, U, DH = (Mat(v, t) for v in (X, WG, WU, G, U, DH))
    got = backward(t, M, N, K, X, WG, WU, G, U, DH, act)
    dg, du, dx, dwg, dwu = (m.get().double().numpy() for m in got)
    a, d = limits(act, G.value)
    want_dg, want_du = DH.value * U.value * d, DH.value * a
    for x in (dg, du, dx, dwg, dwu):
        assert not np.isnan(x).any()
    wild = {(2, 9)} | ({(1, 2)} if act == "none" else set())
    # the identity's -TOP and the others' TOP / 64 stay finite under a DH below 1
    assert {tuple(map(int, i)) for i in np.argwhere(np.isinf(du))} == wild
    assert np.isfinite(dg).all()
    rows = {i for i, _ in wild}
    assert {int(i) for i in np.argwhere(np.isinf(dx))[:, 0]} == rows
    assert np.isfinite(dwg).all()
    assert {int(i) for i in np.argwhere(np.isinf(dwu))[:, 0]} == {j for _, j in wild}
    if act in CURVED or act == "relu":
        assert du[1, 2] == 0 and dg[1, 2] == 0
        if act != "relu":
            assert du[3, 17] == 0 and dg[3, 17] == 0
    ok = np.isfinite(want_du)
    assert np.array_equal(np.isinf(du), ~ok) and (du[~ok] == want_du[~ok]).all()
    want_du = np.where(ok, want_du, 0)
    with np.errstate(over="ignore"):
        edu = np.abs(DH.value) * act_error(act, np.where(np.isinf(G.value), 0, G.value), np.where(ok, a, 0)) + 2.0 ** -24 * np.abs(want_du)
    near(np.where(ok, du, 0), want_du, edu, t, "dU")
    edg = np.abs(DH.value * U.value) * 2.0 ** -13 + 3 * 2.0 ** -24 * np.abs(want_dg) + 2.0 ** -120
    near(dg, want_dg, edg, t, "dG")
    # the products where nothing infinite enters
    px, pg, pu = o.gated_products(dg, np.where(ok, du, 0), X.value, WG.value, WU.value)
    fin = np.where(ok, du, 0)
    e = product_error(np.concatenate([dg, fin], 1), np.concatenate([WG.value, WU.value], 0).T)
    keep = [i for i in range(M) if i not in rows]
    near(dx[keep], px[keep], e[keep], t, "dX")
    near(dwg, pg, product_error(dg.T, X.value.T), t, "dWg")
    cols = [j for j in range(N) if j not in {j for _, j in wild}]
    near(dwu[cols], pu[cols], product_error(fin.T, X.value.T)[cols], t, "dWu")


@pytest.mark.parametrize("act", CURVED)
@pytest.mark.parametrize("t,big,rest", [("f16", -65504.0, -32768.0), ("bf16", -TOP["bf16"], -1.2e36)])
def test_sums_below_the_types_range(act, t, big, rest):
    """Forward and backward together: a gate sum that fp32 holds and the type does not.
    H is finite there, and so are all gradients, with zeros where the gate is shut."""
    M, N, K = 70, 64, 96
    rng = np.random.default_rng(5)
    X, WG, WU = rng.standard_normal((M, K)), rng.standard_normal((N, K)) / 10, rng.standard_normal((N, K)) / 10
    X[:, :2] = 0
    X[6, :2] = 1                                   # token 6 and channel 11 meet
    X[6, 2:] = 0
    WG[:, :2] = 0
    WG[11, :2] = big, rest
    X, WG, WU = (Mat(v, t) for v in (X, WG, WU))
    DH = rng.standard_normal((M, N))
    DH[:, 11] = 0                                  # others' gradients by the large weights are none
    DH[6, 11] = 1.5
    DH = Mat(DH, t)
    H, G, U = (Mat(None, t, 0, 0, M, N) for _ in range(3))
    fn("gemm_gated", t)(M, N, K, *X.at, *WG.at, *WU.at, *G.at, *U.at, *H.at, act)
    g, h = G.get().double().numpy(), H.get().double().numpy()
    assert g[6, 11] == -np.inf and np.isfinite(np.delete(g.ravel(), 6 * N + 11)).all()
    assert np.isfinite(h).all() and h[6, 11] == 0
    G.value, U.value = g, U.get().double().numpy()
    got = backward(t, M, N, K, X, WG, WU, G, U, DH, act)
    dg, du, dx, dwg, dwu = (m.get().double().numpy() for m in got)
    for what, x in (("dG", dg), ("dU", du), ("dX", dx), ("dWg", dwg), ("dWu", dwu)):
        assert np.isfinite(x).all(), what
    assert du[6, 11] == 0 and dg[6, 11] == 0
    px, pg, pu = o.gated_products(dg, du, X.value, WG.value, WU.value)
    e = product_error(np.concatenate([dg, du], 1), np.concatenate([WG.value, WU.value], 0).T)
    near(dx, px, e, t, "dX")
    near(dwg, pg, product_error(dg.T, X.value.T), t, "dWg")
    near(dwu, pu, product_error(du.T, X.value.T), t, "dWu")


@pytest.mark.parametrize("act", CURVED)
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_a_gate_that_is_no_number_stays_so(act, t):
    """NaN in G, U or DH reaches dG and dU where the formulas hold it, and nothing else."""
    M, N, K = 40, 72, 64
    rng = np.random.default_rng(6)
    X, WG, WU = (Mat(rng.standard_normal(s), t) for s in ((M, K), (N, K), (N, K)))
    G, U, DH = (rng.standard_normal((M, N)) for _ in range(3))
    G[1, 3], U[5, 8], DH[9, 20], G[12, 40], DH[13, 41] = np.nan, np.nan, np.nan, -np.inf, np.inf
    G[13, 41] = -np.inf
    G, U, DH = (Mat(v, t) for v in (G, U, DH))
    got = backward(t, M, N, K, X, WG, WU, G, U, DH, act, dx=False, dw=False)
    dg, du = (m.get().double().numpy() for m in got[:2])
    where = lambda x: {tuple(map(int, i)) for i in np.argwhere(np.isnan(x))}  # noqa: E731
    assert where(du) == {(1, 3), (9, 20), (13, 41)}      # infinity times the limit 0 is none
    assert where(dg) == {(1, 3), (5, 8), (9, 20), (13, 41)}
    assert du[12, 40] == 0 and dg[12, 40] == 0


@pytest.mark.parametrize("act", ("relu", *CURVED))
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_infinite_u_behind_a_shut_gate(act, t):
    """U of either infinity: no gradient where the slope is 0, infinite ones where it is
    not; dU does not look at U."""
    M, N, K = 130, 72, 64
    rng = np.random.default_rng(7)
    X, WG, WU = (Mat(rng.standard_normal(s), t) for s in ((M, K), (N, K), (N, K)))
    G, U, DH = (rng.standard_normal((M, N)) for _ in range(3))
    shut = -1.0 if act == "relu" else -1000.0
    for i, (g, u) in enumerate(((shut, np.inf), (shut, -np.inf), (-np.inf, np.inf), (-np.inf, -np.inf))):
        G[20 + i, 3 + 9 * i], U[20 + i, 3 + 9 * i] = g, u
    if act == "relu":
        G[30, 5], U[30, 5] = 0.0, np.inf
    G, U, DH = (Mat(v, t) for v in (G, U, DH))
    got = [m.get().double().numpy() for m in backward(t, M, N, K, X, WG, WU, G, U, DH, act)]
    assert all(np.isfinite(x).all() for x in got)
    assert (got[0][np.isinf(U.value)] == 0).all()
    U.value[50, 60] = np.inf                       # an open gate
    U2, G.value[50, 60] = U.value, 2.0
    got = [m.get().double().numpy() for m in backward(t, M, N, K, X, WG, WU, Mat(G.value, t), Mat(U2, t), DH, act)]
    assert {tuple(map(int, i)) for i in np.argwhere(~np.isfinite(got[0]))} == {(50, 60)} and np.isinf(got[0][50, 60])
    assert np.isfinite(got[1]).all()


def test_infinite_u_of_a_sum_that_fp32_holds():
    """Forward and backward: a channel whose second projection passes binary16's range
    behind a gate that ReLU shuts."""
    M, N, K, t = 33, 40, 64, "f16"
    rng = np.random.default_rng(9)
    X, WG, WU = rng.standard_normal((M, K)), rng.standard_normal((N, K)) / 8, rng.standard_normal((N, K)) / 8
    X[:, :3] = 0
    X[6, :3] = 1
    WG[:, :3], WU[:, :3] = 0, 0
    WG[11, 2], WU[11, :2] = -40.0, (60000.0, 30000.0)
    X, WG, WU = (Mat(v, t) for v in (X, WG, WU))
    DH = rng.standard_normal((M, N))
    DH[:6, 11], DH[7:, 11] = 0, 0
    DH = Mat(DH, t)
    H, G, U = (Mat(None, t, 0, 0, M, N) for _ in range(3))
    b.gemm_gated_f16(M, N, K, *X.at, *WG.at, *WU.at, *G.at, *U.at, *H.at, "relu")
    G.value, U.value = G.get().double().numpy(), U.get().double().numpy()
    assert np.isfinite(H.get().numpy()).all() and U.value[6, 11] == np.inf and G.value[6, 11] < 0
    got = backward(t, M, N, K, X, WG, WU, G, U, DH, "relu")
    assert all(np.isfinite(m.get().numpy()).all() for m in got)
