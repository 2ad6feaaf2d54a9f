"""GPU tests of every kernel that multiplies in the feed-forward layer: each number of
rows and columns a workgroup takes, in every form, operand and result type, against
torch's float64 product with bounds as in test_gpu_layer.py.  Rows and columns are
ragged, k ends inside a span or a stage, row and column scales all differ, what lies
around the matrices is NaN (-128 in 8 bits).  tests/test_layer_reach.py shows that
these sizes reach every kernel on a device of 256 CUs.

A case is the form, the operands' type, the results' type, the product's M, N and K
(of dX: tokens, width, features; of dWg and dWu: features, width, tokens), and
whether rows begin on 16 bytes."""
import pytest

from tests.test_gpu_layer_tiles import TYPES, check, fn, room, untouched

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROWS = [(5, 1000, 200, True), (5, 16400, 200, True), (16, 16500, 2203, True), (20, 1000, 200, True),
        (20, 4100, 200, True), (32, 8200, 1000, True), (27, 4111, 2203, True), (5, 16400, 203, False), (20, 4100, 200, False),
        (40, 1000, 200, False), (40, 4100, 200, False), (64, 8200, 1001, False)]
PLAIN = [*ROWS, (100, 500, 1001, True), (300, 2000, 1001, True), (1500, 2700, 1001, True), (5300, 4300, 1101, True),
         (100, 200, 7, False), (100, 1001, 1003, False), (1000, 1500, 777, False), (1500, 2700, 777, False)]
GATED = [*ROWS, (100, 250, 1001, True), (300, 1000, 1001, True), (1500, 1350, 1001, True), (5300, 2150, 1101, True),
         (100, 100, 7, False), (100, 500, 1003, False), (700, 1000, 777, False), (1500, 1350, 777, False)]
DX = [(100, 500, 128, True), (300, 2000, 256, True), (1500, 2700, 320, True), (4700, 4900, 640, True),
      (100, 99, 5, False), (100, 5, 400, False), (100, 500, 401, False), (1000, 777, 1500, False), (1000, 777, 200, False),
      (1500, 2700, 321, False), (1500, 2700, 321, True)]
DW = [(100, 500, 500, True), (300, 1000, 201, True), (1500, 1350, 1000, True), (2600, 4900, 603, True),
      (5, 100, 100, False), (100, 5, 100, False), (500, 777, 1000, False), (500, 777, 300, False), (1500, 1500, 1000, False)]
CASES = ([("i8", "i8", out, *s) for out in ("f32", "bf16", "f16") for s in PLAIN]
         + [("i8_gated", "i8", out, *s) for out in ("bf16", "f16") for s in GATED]
         + [("gated", t, t, *s) for t in ("bf16", "f16") for s in GATED]
         + [(form, t, t, *s) for t in ("bf16", "f16") for form, sizes in (("dx", DX), ("dw", DW)) for s in sizes])
SIZE = {"i8": 1, "bf16": 2, "f16": 2, "f32": 4}
ACT = {"i8_gated": 4, "gated": 2, "dx": 1, "dw": 1}


def call(case, mat, vec):
    """The entry point's name and its arguments up to the stream; mat(name, rows,
    columns, type) gives an address and a pitch, vec(name, length) an address."""
    form, t, out, M, N, K, _ = case
    none = (None, 0)
    if form == "i8":
        return f"gemm_i8_{out}", (M, N, K, *mat("A", M, K, t), vec("SA", M), *mat("B", N, K, t), vec("SB", N),
                                  *mat("C", M, N, out))
    if form == "i8_gated":
        return f"gemm_i8_gated_{out}", (M, N, K, *mat("A", M, K, t), vec("SA", M), *mat("B", N, K, t), vec("SB", N),
                                        *mat("B2", N, K, t), vec("SB2", N), *mat("C", M, N, out), ACT[form])
    if form == "gated":
        return f"gemm_gated_{t}", (M, N, K, *mat("A", M, K, t), *mat("B", N, K, t), *mat("B2", N, K, t),
                                   *mat("G", M, N, t), *mat("U", M, N, t), *mat("C", M, N, t), ACT[form])
    tokens, features, width = (M, K, N) if form == "dx" else (K, M, N)
    kept = [v for name in ("G", "U", "DH", "DG", "DU") for v in mat(name, tokens, features, t)]
    if form == "dx":
        return f"gemm_gated_backward_{t}", (tokens, features, width, *none, *mat("B", features, width, t),
                                            *mat("B2", features, width, t), *kept, *mat("C", tokens, width, t),
                                            *none, *none, ACT[form])
    return f"gemm_gated_backward_{t}", (tokens, features, width, *mat("A", tokens, width, t), *none, *none, *kept, *none,
                                        *mat("C", features, width, t), *mat("C2", features, width, t), ACT[form])


class Operands:
    """Matrices and scales of a case on the GPU, by name."""

    def __init__(self, case):
        self.m, self.case = {}, case
        self.gen = torch.Generator(device=DEV).manual_seed(case[3] + 3 * case[4] + 7 * case[5])

    def mat(self, name, rows, cols, t):
        x = room(rows, cols, torch.int8 if t == "i8" else torch.float32 if t == "f32" else TYPES[t], self.case[-1])
        if t == "i8":
            x.copy_(torch.randint(-128, 128, (rows, cols), generator=self.gen, device=DEV))
        elif name in ("A", "B", "B2") or (name in ("G", "U", "DH") and self.case[0] in ("dx", "dw")):
            scale = {"B": self.case[5] ** -0.5, "B2": self.case[5] ** -0.5, "DH": 0.1}.get(name, 1.0)
            x.copy_(scale * torch.randn((rows, cols), generator=self.gen, device=DEV))
        self.m[name] = x
        return x.data_ptr(), x.stride(0)

    def vec(self, name, n):
        # sums of size 74^2 sqrt(K) come out near 1
        s = (torch.rand(n, generator=self.gen, device=DEV) + 0.25) / (74 * self.case[5] ** 0.25)
        self.m[name] = s
        return s.data_ptr()

    def __getitem__(self, name):
        return self.m[name].double()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_kernel(case):
    form, t, out, M, N, K, _ = case
    x = Operands(case)
    name, args = call(case, x.mat, x.vec)
    inputs = {n: x.m[n].clone() for n in ("A", "SA", "B", "SB", "B2", "SB2") if n in x.m}
    fn(*name.rsplit("_", 1))(*args)
    for n, was in inputs.items():
        assert torch.equal(x.m[n], was), n
    what = "-".join(map(str, case))
    T = lambda k: (-(-k // 16) + 32) * 2.0 ** -23  # noqa: E731
    if form in ("dx", "dw"):
        g, u, dh, dg, du = (x[n] for n in ("G", "U", "DH", "DG", "DU"))
        check(x.m["DG"], dh * u * (g > 0), (dh * u).abs() * 2.0 ** -23, t, what + " dG")
        check(x.m["DU"], dh * g.clamp(min=0), (dh * g).abs() * 2.0 ** -23, t, what + " dU")
        assert untouched(x.m["C"], N)
        if form == "dx":
            a, b = torch.cat([dg, du], 1), torch.cat([x["B"], x["B2"]], 0)
            check(x.m["C"], a @ b, T(2 * K) * (a.abs() @ b.abs()), t, what)
        else:
            for d, c in ((dg, "C"), (du, "C2")):
                check(x.m[c], d.t() @ x["A"], T(K) * (d.abs().t() @ x["A"].abs()), t, what + c)
            assert untouched(x.m["C2"], N)
        return
    assert untouched(x.m["C"], N)
    if form == "i8":
        want = (x["A"] @ x["B"].t()) * x["SA"][:, None] * x["SB"]
        check(x.m["C"], want, 3.01 * 2.0 ** -24 * want.abs(), out, what)
        return
    if form == "i8_gated":
        e = 3.01 * 2.0 ** -24
        g, u = ((x["A"] @ x[b].t()) * x["SA"][:, None] * x[s] for b, s in (("B", "SB"), ("B2", "SB2")))
        eg, eu = e * g.abs(), e * u.abs()
        act, z = g * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)), 3 * g.abs() + g.abs() ** 3 / 8
    else:
        a = x["A"]
        g, u = a @ x["B"].t(), a @ x["B2"].t()
        eg, eu = (T(K) * (a.abs() @ x[b].abs().t()) for b in ("B", "B2"))
        check(x.m["G"], g, eg, t, what + " G")
        check(x.m["U"], u, eu, t, what + " U")
        assert untouched(x.m["G"], N) and untouched(x.m["U"], N)
        act, z = g * torch.sigmoid(g), g.abs()
    E = 2.0 ** -23 * (8 + 4 * z.clamp(max=200)) * (act.abs() + 1.2 * eg) + 2.0 ** -119
    check(x.m["C"], act * u, 1.2 * eg * u.abs() + act.abs() * eu + 1.2 * eg * eu + E * (u.abs() + eu)
          + 2.0 ** -24 * (act * u).abs(), out, what + " H")
