"""The feed-forward layer's kernels that stage through LDS, with the debug build
that writes NaN over every place of a stage between its last read and its refill:
the same bits in both builds."""
import pytest

from register_lds_tiled_amd import binding as b

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def libs():
    return b.library(), b.ldspoison_library()


def both(libs, name, ints, operands, outputs, tail=()):
    """The call on each build into outputs of its own, which must be equal."""
    got = []
    for lib in libs:
        own = {id(o): torch.full_like(o, 7.0) for o in outputs}
        args = []
        for x in operands:
            x = own.get(id(x), x)
            args += [x.data_ptr()] + ([] if x.dim() == 1 else [x.stride(0)])
        assert getattr(lib, name)(*ints, *args, *tail, torch.cuda.current_stream().cuda_stream) == 0
        got.append([own[id(o)] for o in outputs])
    torch.cuda.synchronize()
    for x, y in zip(*got):
        assert bool(torch.isfinite(x).all()), name
        assert torch.equal(x, y), f"{name} {ints}: the builds differ"


def padded(rows, cols, pad, make):
    return make((rows, cols + pad))[:, :cols]


# on 256 CUs: k divided in 32 x 64 and 64 x 64 tiles (fewer stages than waves, a
# ring gone round several times), 128 x 128 and 256 x 256 (one stage to more than
# five, a first stage partly below k = 0), and with rows off 16 bytes the tiles
# through registers
SHAPES = [(40, 300, 64), (40, 300, 1048), (300, 1500, 128), (300, 1500, 2056), (1500, 2100, 64), (1500, 2100, 200),
          (1500, 2100, 776), (4200, 4300, 64), (4200, 4300, 136), (4200, 4300, 400)]


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(libs, M, N, K, odd):
    gen = torch.Generator(device=DEV).manual_seed(M + K)
    pad = odd if odd else -K % 16 + 16
    K8 = K // 16 * 16 if not odd else K
    codes = lambda s: torch.randint(-127, 128, s, generator=gen, dtype=torch.int8, device=DEV)  # noqa: E731
    A, G, U = (padded(r, K8, pad, codes) for r in (M, N, N // 2))
    s = torch.rand(max(M, N), generator=gen, device=DEV) * 0.01
    C = torch.empty((M, N), device=DEV)
    both(libs, "gemm_i8_f32", (M, N, K8), (A, s, G, s, C), (C,))
    H = torch.empty((M, N // 2), dtype=torch.bfloat16, device=DEV)
    both(libs, "gemm_i8_gated_bf16", (M, N // 2, K8), (A, s, G, s, U, s, H), (H,), (2,))
    for t, dtype in (("bf16", torch.bfloat16), ("f16", torch.float16)):
        if M > 4000 and t == "f16":
            continue
        values = lambda z: (0.1 * torch.randn(z, generator=gen, device=DEV)).to(dtype)  # noqa: E731,B023
        n = N // 2
        X, WG, WU = (padded(r, K, pad, values) for r in (M, n, n))
        g, u, h = (torch.empty((M, n), dtype=dtype, device=DEV) for _ in range(3))
        both(libs, f"gemm_gated_{t}", (M, n, K), (X, WG, WU, g, u, h), (g, u, h), (3,))


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("M,N,K", [(72, 64, 300), (130, 256, 500), (700, 128, 1500), (1500, 320, 2100), (4200, 128, 4300),
                                   (136, 2200, 1000), (400, 3000, 2100), (1000, 4200, 2200)])
def test_gradients(libs, M, N, K, odd):
    gen = torch.Generator(device=DEV).manual_seed(M + N)
    for t, dtype in (("bf16", torch.bfloat16), ("f16", torch.float16)):
        values = lambda z: (0.1 * torch.randn(z, generator=gen, device=DEV)).to(dtype)  # noqa: E731,B023
        X, WG, WU = (padded(r, K, odd if odd else -K % 8, values) for r in (M, N, N))
        G, U, DH, DG, DU = (padded(M, N, odd, values) for _ in range(5))
        DX = torch.empty((M, K), dtype=dtype, device=DEV)
        DWG, DWU = (torch.empty((N, K), dtype=dtype, device=DEV) for _ in range(2))
        # dG and dU are read behind their writing: outputs of each build's own
        DG, DU = (x.contiguous() if not odd else x for x in (DG, DU))
        both(libs, f"gemm_gated_backward_{t}", (M, N, K), (X, WG, WU, G, U, DH, DG, DU, DX, DWG, DWU),
             (DG, DU, DX, DWG, DWU), (2,))


@pytest.mark.parametrize("M,N,K", [(40, 300, 135), (300, 1500, 1001), (1500, 2100, 327), (4200, 4300, 1101)])
def test_rows_that_end_within_16_bytes(libs, M, N, K):
    """What is behind K in the last 16 bytes is cleared between a stage's landing and
    its first read."""
    gen = torch.Generator(device=DEV).manual_seed(M + K)
    codes = lambda s: torch.randint(-127, 128, s, generator=gen, dtype=torch.int8, device=DEV)  # noqa: E731
    A, G, U = (padded(r, K, -K % 16, codes) for r in (M, N, N // 2))
    s = torch.rand(max(M, N), generator=gen, device=DEV) * 0.01
    C = torch.empty((M, N), device=DEV)
    both(libs, "gemm_i8_f32", (M, N, K), (A, s, G, s, C), (C,))
    H = torch.empty((M, N // 2), dtype=torch.bfloat16, device=DEV)
    both(libs, "gemm_i8_gated_bf16", (M, N // 2, K), (A, s, G, s, U, s, H), (H,), (2,))
    real = lambda s: 0.1 * torch.randn(s, generator=gen, device=DEV).half()  # noqa: E731
    X, WG, WU = (padded(r, K, -K % 8, real) for r in (M, N // 2, N // 2))
    g, u, h = (torch.empty((M, N // 2), dtype=torch.float16, device=DEV) for _ in range(3))
    both(libs, "gemm_gated_f16", (M, N // 2, K), (X, WG, WU, g, u, h), (g, u, h), (3,))


def test_the_largest_tiles(libs):
    """More than eight stages in more than a round and a quarter of 256 x 256 tiles."""
    for K in (1101, 2064):
        test_rows_that_end_within_16_bytes(libs, 5300, 4300, K)
    test_gradients(libs, 4700, 640, 4900, 0)
    test_gradients(libs, 600, 2600, 4900, 0)
