"""GPU tests of the feed-forward layer's tile kernels on products that fill the
device: every choice of tiles, ragged edges, k of every length around the kernels'
stages.  The reference is torch's float64 product on the GPU; bounds as in
test_gpu_layer.py.  8-bit products with scales of 1 into float32 are exact below
2^24, and are compared bit for bit."""
import pytest

from register_lds_tiled_amd import binding as b

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def fn(name, t):
    return getattr(b, f"{name}_{t}")


def room(rows, cols, dtype, whole=True, fill=float("nan")):
    """rows x cols inside a buffer of `fill`, rows on 16 bytes or packed off them."""
    n = 16 // torch.empty((), dtype=dtype).element_size()
    ld = -(-cols // n) * n + n if whole else cols + 1
    off = n if whole else 1
    flat = torch.full((off + rows * ld + 64,), -128 if dtype == torch.int8 else fill, dtype=dtype, device=DEV)
    return flat[off:off + rows * ld].view(rows, ld)[:, :cols]


def filled(x, dtype, whole=True):
    y = room(x.shape[0], x.shape[1], dtype, whole)
    y.copy_(x)
    return y


def untouched(x, cols):
    """What lies between the rows still holds NaN."""
    rows, ld = x.shape[0], x.stride(0)
    full = torch.as_strided(x, (rows, ld), (ld, 1), x.storage_offset())
    return bool(torch.isnan(full[:-1, cols:].float()).all())


def check(got, want, bound, t, what):
    half = torch.finfo(got.dtype).eps / 2
    most = bound + half * (want.abs() + bound) + 2.0 ** -25
    off = (got.double() - want).abs()
    assert bool((off <= most).all()), f"{what}: {int((~(off <= most)).sum())} off, worst {float((off - most).max()):.3g} past its bound"


# rows, columns: on 256 CUs 32 x 64, 64 x 64, 64 x 128, 128 x 128 and 256 x 256 tiles
# of plain products, each with edges that no tile size divides
SIZES = [(100, 500), (300, 2000), (520, 3500), (1500, 2700), (4200, 4300)]
DEEP = [64, 128, 192, 200, 264, 320, 384, 456, 520, 640, 776, 1000, 1288, 2056]


def depths(M, N):
    return DEEP if M * N < 1 << 22 else DEEP[::3]


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("M,N", SIZES)
def test_i8(M, N, whole):
    gen = torch.Generator(device=DEV).manual_seed(M)
    for K in depths(M, N) + ([48, 80, 144] if whole else [15, 16, 17, 100, 129]):
        if whole:
            K = K // 16 * 16
        A = torch.randint(-128, 128, (M, K), generator=gen, device=DEV)
        B = torch.randint(-128, 128, (N, K), generator=gen, device=DEV)
        want = A.double() @ B.double().t()
        a, w, one = filled(A, torch.int8, whole), filled(B, torch.int8, whole), torch.ones(max(M, N), device=DEV)
        C = room(M, N, torch.float32, whole)
        b.gemm_i8_f32(M, N, K, a, a.stride(0), one, w, w.stride(0), one, C, C.stride(0))
        exact = want.abs() < 2 ** 24
        assert bool((C.double() == want)[exact].all()), (M, N, K)
        check(C, want, want.abs() * 2.0 ** -24, "f32", f"{M}x{N}x{K}")
        assert untouched(C, N)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("M,N", SIZES)
def test_gated(M, N, whole, t):
    gen = torch.Generator(device=DEV).manual_seed(N)
    N //= 2
    for K in depths(M, 2 * N) + ([72, 136] if whole else [9, 65, 101]):
        X, G, U = (filled(s * torch.randn((r, K), generator=gen, device=DEV), TYPES[t], whole)
                   for r, s in ((M, 1.0), (N, K ** -0.5), (N, K ** -0.5)))
        H, g, u = (room(M, N, TYPES[t], whole) for _ in range(3))
        at = [v for m in (X, G, U, g, u, H) for v in (m, m.stride(0))]
        fn("gemm_gated", t)(M, N, K, *at, "silu")
        x, wg, wu = X.double(), G.double(), U.double()
        rg, ru = x @ wg.t(), x @ wu.t()
        T = (-(-K // 16) + 32) * 2.0 ** -23
        eg, eu = T * (x.abs() @ wg.abs().t()), T * (x.abs() @ wu.abs().t())
        what = f"{M}x{N}x{K} {t}"
        check(g, rg, eg, t, what + " G")
        check(u, ru, eu, t, what + " U")
        act = rg * torch.sigmoid(rg)
        E = 2.0 ** -23 * (8 + 4 * rg.abs()) * act.abs()
        check(H, act * ru, 1.2 * eg * ru.abs() + act.abs() * eu + 1.2 * eg * eu + E * (ru.abs() + eu) + 2.0 ** -24 * (act * ru).abs(),
              t, what + " H")
        assert untouched(H, N) and untouched(g, N) and untouched(u, N)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,N", SIZES)
def test_i8_gated(M, N, t):
    gen = torch.Generator(device=DEV).manual_seed(N)
    N //= 2
    for K in (64, 272, 1024):
        A, G, U = (filled(torch.randint(-128, 128, (r, K), generator=gen, device=DEV), torch.int8) for r in (M, N, N))
        sa, sg, su = (torch.rand(n, generator=gen, device=DEV) / 74 / K ** 0.25 for n in (M, N, N))
        H = room(M, N, TYPES[t])
        fn("gemm_i8_gated", t)(M, N, K, A, A.stride(0), sa, G, G.stride(0), sg, U, U.stride(0), su, H, H.stride(0), "gelu_tanh")
        rg = (A.double() @ G.double().t()) * sa.double()[:, None] * sg.double()
        ru = (A.double() @ U.double().t()) * sa.double()[:, None] * su.double()
        act = rg * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (rg + 0.044715 * rg ** 3))
        e = 3.01 * 2.0 ** -24
        E = 2.0 ** -23 * (8 + 4 * (3 * rg.abs() + rg.abs() ** 3 / 8).clamp(max=200)) * act.abs()
        check(H, act * ru, 1.2 * e * (rg * ru).abs() + e * (act * ru).abs() + 1.01 * E * ru.abs() + 2.0 ** -24 * (act * ru).abs(),
              t, f"{M}x{N}x{K}")
        assert untouched(H, N)


# tokens, features, width: the two gradients' products take the sizes (tokens, width)
# over twice the features, and (features, width) over the tokens
BACK = [(100, 128, 500), (300, 256, 2000), (520, 192, 3500), (1500, 320, 2700), (4200, 128, 4300),
        (128, 700, 900), (72, 2000, 1100), (200, 3000, 1500), (500, 3100, 2300), (1000, 1500, 777)]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("M,N,K", BACK)
def test_backward(M, N, K, whole, t):
    gen = torch.Generator(device=DEV).manual_seed(N + K)
    for tokens in (M, M + 1, M // 64 * 64 + 8):
        X, G, U, DH = (filled(s * torch.randn(r, generator=gen, device=DEV), TYPES[t], whole)
                       for r, s in (((tokens, K), 1.0), ((tokens, N), 1.0), ((tokens, N), 1.0), ((tokens, N), 0.1)))
        WG, WU = (filled(torch.randn((N, K), generator=gen, device=DEV) * N ** -0.5, TYPES[t], whole) for _ in range(2))
        DG, DU = (room(tokens, N, TYPES[t], whole) for _ in range(2))
        DX = room(tokens, K, TYPES[t], whole)
        DWG, DWU = (room(N, K, TYPES[t], whole) for _ in range(2))
        at = [v for m in (X, WG, WU, G, U, DH, DG, DU, DX, DWG, DWU) for v in (m, m.stride(0))]
        fn("gemm_gated_backward", t)(tokens, N, K, *at, "relu")
        g, u, dh = G.double(), U.double(), DH.double()
        check(DG, dh * u * (g > 0), (dh * u).abs() * 2.0 ** -23, t, "dG")
        check(DU, dh * g.clamp(min=0), (dh * g).abs() * 2.0 ** -23, t, "dU")
        dg, du, x = DG.double(), DU.double(), X.double()
        a, w = torch.cat([dg, du], 1), torch.cat([WG.double(), WU.double()], 0)
        what = f"{tokens}x{N}x{K} {t}"
        e = lambda k: (-(-k // 16) + 32) * 2.0 ** -23  # noqa: E731
        check(DX, a @ w, e(2 * N) * (a.abs() @ w.abs()), t, what + " dX")
        check(DWG, dg.t() @ x, e(tokens) * (dg.abs().t() @ x.abs()), t, what + " dWg")
        check(DWU, du.t() @ x, e(tokens) * (du.abs().t() @ x.abs()), t, what + " dWu")
        assert untouched(DX, K) and untouched(DWG, K) and untouched(DWU, K) and untouched(DG, N)


def test_backward_with_pitches_of_its_own():
    """dG and dU, Wg and Wu rows apart by different pitches; columns that end inside
    16 bytes."""
    M, N, K, t = 1500, 256, 2700, torch.bfloat16
    gen = torch.Generator(device=DEV).manual_seed(1)
    r = lambda rows, cols, pad: torch.randn((rows, cols + pad), generator=gen, device=DEV).to(t)[:, :cols]  # noqa: E731
    for pads in ((0, 8, 0, 8), (8, 8, 0, 16), (0, 0, 8, 8)):
        X, G, U, DH = r(M, K, 0), r(M, N, 0), r(M, N, 8), r(M, N, 16)
        DG, DU = r(M, N, pads[0]), r(M, N, pads[1])
        WG, WU = r(N, K, pads[2]), r(N, K, pads[3])
        DX, DWG, DWU = r(M, K, 4), r(N, K, 12), r(N, K, 0)
        at = [v for m in (X, WG, WU, G, U, DH, DG, DU, DX, DWG, DWU) for v in (m, m.stride(0))]
        b.gemm_gated_backward_bf16(M, N, K, *at, "none")
        dg, du = DG.double(), DU.double()
        want = dg @ WG.double() + du @ WU.double()
        bound = (2 * N // 16 + 32) * 2.0 ** -23 * (dg.abs() @ WG.double().abs() + du.abs() @ WU.double().abs())
        check(DX, want, bound, "bf16", "dX")
        check(DWU, du.t() @ X.double(), (M // 16 + 33) * 2.0 ** -23 * (du.abs().t() @ X.double().abs()), "bf16", "dWu")


@pytest.mark.parametrize("M,N,K", [(300, 2000, 200), (1500, 2700, 264), (4200, 4300, 136), (4200, 2300, 101)])
def test_what_is_not_a_number_stays_where_it_is(M, N, K):
    """NaN in the last element of a row of X, and infinities around the matrices."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    whole = K % 8 == 0
    X, G, U = (filled(torch.randn((r, K), generator=gen, device=DEV), torch.bfloat16, whole) for r in (M, N, N))
    X[M - 2, K - 1] = float("nan")
    G[N - 3, 0] = float("nan")
    H = room(M, N, torch.bfloat16, whole, 0.0)
    b.gemm_gated_bf16(M, N, K, X, X.stride(0), G, G.stride(0), U, U.stride(0), None, 0, None, 0, H, H.stride(0), "none")
    want = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    want[M - 2], want[:, N - 3] = True, True
    assert torch.equal(torch.isnan(H), want)


def test_large_products_repeat_and_replay():
    """The same bits from call to call and from a graph, on the widest tiles."""
    M, N, K = 4200, 2200, 264
    gen = torch.Generator(device=DEV).manual_seed(6)
    X, G, U, DH = (torch.randn(s, generator=gen, device=DEV).bfloat16() for s in ((M, K), (N, K), (N, K), (M, N)))
    out = [torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((M, N), (M, N), (M, N), (M, N), (M, N), (M, K), (N, K), (N, K))]
    h, g, u, dg, du, dx, dwg, dwu = out

    def call():
        b.gemm_gated_bf16(M, N, K, X, K, G, K, U, K, g, N, u, N, h, N)
        b.gemm_gated_backward_bf16(M, N, K, X, K, G, K, U, K, g, N, u, N, DH, N, dg, N, du, N, dx, K, dwg, K, dwu, K)

    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in out]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(out, first):
            assert torch.equal(t, w)
        call()
        torch.cuda.synchronize()


# k that ends within 16 bytes of rows that begin on them: the rest of the 16 holds
# NaN (-128 in 8 bits), also behind the last row
CUT = [65, 71, 127, 129, 135, 190, 263, 327, 513, 1001, 1990]


@pytest.mark.parametrize("M,N", SIZES)
def test_i8_rows_that_end_within_16_bytes(M, N):
    gen = torch.Generator(device=DEV).manual_seed(M + 1)
    for K in (CUT[2:] if M * N < 1 << 22 else CUT[3::3]):
        A = torch.randint(-128, 128, (M, K), generator=gen, device=DEV)
        B = torch.randint(-128, 128, (N, K), generator=gen, device=DEV)
        want = A.double() @ B.double().t()
        a, w, one = filled(A, torch.int8), filled(B, torch.int8), torch.ones(max(M, N), device=DEV)
        C = room(M, N, torch.float32)
        b.gemm_i8_f32(M, N, K, a, a.stride(0), one, w, w.stride(0), one, C, C.stride(0))
        exact = want.abs() < 2 ** 24
        assert bool((C.double() == want)[exact].all()), (M, N, K)
        check(C, want, want.abs() * 2.0 ** -24, "f32", f"{M}x{N}x{K}")
        assert untouched(C, N)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,N", SIZES)
def test_gated_rows_that_end_within_16_bytes(M, N, t):
    gen = torch.Generator(device=DEV).manual_seed(N + 1)
    N //= 2
    for K in (CUT if M * N < 1 << 21 else CUT[::3]):
        X, G, U = (filled(s * torch.randn((r, K), generator=gen, device=DEV), TYPES[t])
                   for r, s in ((M, 1.0), (N, K ** -0.5), (N, K ** -0.5)))
        H, g, u = (room(M, N, TYPES[t]) for _ in range(3))
        fn("gemm_gated", t)(M, N, K, *[v for m in (X, G, U, g, u, H) for v in (m, m.stride(0))], "none")
        x, wg, wu = X.double(), G.double(), U.double()
        rg, ru = x @ wg.t(), x @ wu.t()
        T = (-(-K // 16) + 32) * 2.0 ** -23
        eg, eu = T * (x.abs() @ wg.abs().t()), T * (x.abs() @ wu.abs().t())
        what = f"{M}x{N}x{K} {t}"
        check(g, rg, eg, t, what + " G")
        check(u, ru, eu, t, what + " U")
        check(H, rg * ru, eg * ru.abs() + rg.abs() * eu + eg * eu + 2.0 ** -24 * (rg * ru).abs(), t, what + " H")
        assert untouched(H, N) and untouched(g, N) and untouched(u, N)


# more than eight stages in more than a round and a quarter of 256 x 256 tiles, of each form
def test_i8_in_the_largest_tiles():
    test_i8(5300, 4300, True)


@pytest.mark.parametrize("t", list(TYPES))
def test_gated_in_the_largest_tiles(t):
    test_gated(5300, 4300, True, t)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,N,K", [(4700, 640, 4900), (600, 2600, 4900)])
def test_backward_in_the_largest_tiles(M, N, K, t):
    test_backward(M, N, K, True, t)


def test_rows_that_end_within_16_bytes_in_the_largest_tiles():
    test_i8_rows_that_end_within_16_bytes(5300, 4300)
    test_gated_rows_that_end_within_16_bytes(5300, 4300, "bf16")
