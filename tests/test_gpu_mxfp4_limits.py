"""GPU tests of the MXFP4 entry points at the ends of their ranges: the widest
and longest matrices, far rows, and values past what fp32 holds."""
import numpy as np
import pytest

from oracle import mxfp4 as mx
from register_lds_tiled_amd import binding as b

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
