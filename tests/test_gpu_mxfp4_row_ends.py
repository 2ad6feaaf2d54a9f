"""GPU tests of MXFP4 products whose rows lie off 16 bytes, for every way that K can
end in the last stage of the tiles that go through registers: rows of less than 16
bytes and just more, whole chunks, half a byte, one element past a stage.  Bounds as
in test_gpu_mxfp4.py."""
import numpy as np
import pytest

from tests.test_gpu_mxfp4 import a16, check_product, operand, run_product, run_wproduct

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ENDS = [*range(1, 4), *range(6, 10), *range(28, 36), *range(61, 67), 95, 97, *range(125, 132), 159, 161, *range(222, 228),
        *range(253, 262), 285, 287, 289, 383, 385, 510, 511, 513, 1023, 1025]


@pytest.mark.parametrize("off", [1, 0])
@pytest.mark.parametrize("K", ENDS)
def test_row_ends(K, off):
    M, N = 130, 133
    rng = np.random.default_rng(K)
    pad = 1 if ((K + 1) // 2 + off) % 16 == 0 else off          # off 16 bytes by the pitch at least
    a, sa, A = operand(rng, M, K, pad=pad, spad=off, off=off)
    bq, sb, B = operand(rng, N, K, pad=pad, spad=off, off=off)
    for out in ("f32", "bf16"):
        check_product(run_product(out, M, N, K, a, sa, bq, sb), A, B, out, 64, what=f"{out} {K}")
    for t in ("bf16", "f16"):
        x, X = a16(rng, M, K, t, pad=off, off=off)
        check_product(run_wproduct(t, M, N, K, x, K + off, bq, sb), X, B, "f32", 16, 2, what=f"{t} {K}")
