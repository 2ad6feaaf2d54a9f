"""The MXFP4 kernels' LDS schedules, with the debug build that writes NaN over
every place of a stage between its last read and its refill: each entry point
that stages through LDS gives the same bits in both builds.  (Codes and scales
of the poison are other values too, so a stale read shows; a few-row case
without the last rows of A leaves their places as they were.)"""
import numpy as np
import pytest

from register_lds_tiled_amd import binding as b

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def libs():
    return b.library(), b.ldspoison_library()


def operand(rng, rows, K, ld):
    q = torch.from_numpy(rng.integers(0, 256, (rows, ld), dtype=np.uint8)).to(DEV)
    s = torch.from_numpy(rng.integers(118, 134, (rows, -(-K // 32)), dtype=np.uint8)).to(DEV)
    return q, s


# few rows (one span, several, an odd end), 128 x 128 tiles by DMA (stages odd
# and even, past 2048) and register-staged (odd pitch), 256 x 256 tiles
SHAPES = [(5, 33000, 1100), (20, 8200, 700), (1, 300, 512), (5, 96, 4096), (17, 64, 3001), (64, 130, 2600), (130, 250, 777), (200, 300, 2304),
          (128, 256, 4401), (4100, 2300, 300), (4096, 2304, 2336)]


# (rows off 16 bytes take the same 128 x 128 kernel at every size)
@pytest.mark.parametrize("shape,odd", [(s, o) for s in SHAPES for o in (0, 1) if not (o and s[0] > 1000)],
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_products(libs, shape, odd):
    M, N, K = shape
    rng = np.random.default_rng(M + K)
    ld = -(-K // 32) * 16 + odd
    a, sa = operand(rng, M, K, ld)
    w, sw = operand(rng, N, K, ld)
    x = torch.randn((M, K + (-K) % 8 + odd), device=DEV)
    for name, act in (("mxfp4_f32", None), ("mxfp4_bf16", None), ("bf16_mxfp4_f32", torch.bfloat16),
                      ("f16_mxfp4_f32", torch.float16)):
        if act is not None and M > 1000:
            continue
        xa = None if act is None else x.to(act)
        outs = []
        for lib in libs:
            c = torch.full((M, N), 7.0, device=DEV, dtype=torch.bfloat16 if name.endswith("bf16") else torch.float32)
            fn = getattr(lib, "gemm_" + name)
            stream = torch.cuda.current_stream().cuda_stream
            if act is None:
                st = fn(M, N, K, a.data_ptr(), ld, sa.data_ptr(), sa.stride(0), w.data_ptr(), ld, sw.data_ptr(),
                        sw.stride(0), c.data_ptr(), N, stream)
            else:
                st = fn(M, N, K, xa.data_ptr(), xa.stride(0), w.data_ptr(), ld, sw.data_ptr(), sw.stride(0),
                        c.data_ptr(), N, stream)
            assert st == 0
            outs.append(c)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(outs[0]).all()), name
        assert torch.equal(outs[0], outs[1]), f"{name}: the builds differ"
