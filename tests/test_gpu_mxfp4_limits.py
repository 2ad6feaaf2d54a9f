"""GPU tests of the MXFP4 entry points at the ends of their ranges: the widest
matrices."""
import numpy as np
import pytest

from oracle import mxfp4 as mx
from register_lds_tiled_amd import binding as b
from tests.test_gpu_mxfp4 import quantize_case

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
