"""CPU test that the sizes of tests/test_gpu_layer_kernels.py and of the casts' tests
launch every kernel of the feed-forward layer on a device of 256 CUs: they are
replayed, with their alignments, against the stand-in runtime of
test_mxfp4_launch.py.  No GPU is used; device addresses are fake."""
import os

import pytest

from register_lds_tiled_amd import binding as b
from tests.test_gpu_layer import SHAPES
from tests.test_gpu_layer_kernels import CASES, SIZE, call
from tests.test_layer_launch import AT, HIPCC, backward, lib  # noqa: F401

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="ROCm toolchain missing")


def test_the_gpu_tests_reach_every_kernel(lib):  # noqa: F811
    known = {lib.record_name(i) for i in range(lib.record_known())}
    reached = set()

    def launched(status, what):
        assert status == b.SGEMM_OK, what
        reached.add(lib.record_kernel())

    for case in CASES:
        at = iter(AT)

        def mat(name, rows, cols, t):     # as room() of test_gpu_layer_tiles.py lays them out
            n = 16 // SIZE[t]
            ld, off = (-(-cols // n) * n + n, n) if case[-1] else (cols + 1, 1)
            return next(at) + off * SIZE[t], ld

        name, args = call(case, mat, lambda name, n: next(at))
        launched(getattr(lib, name)(*args, None), case)
    for t in ("bf16", "f16"):
        launched(backward(lib, t, 70, 96, 136, 0, False, False), "slopes")
    for t in ("f32", "bf16", "f16"):
        for R, C in SHAPES:
            launched(getattr(lib, f"gemm_i8_quantize_{t}")(R, C, AT[0], C, AT[3], C, AT[6], None), (R, C))
            launched(getattr(lib, f"gemm_i8_dequantize_{t}")(R, C, AT[3], C, AT[6], AT[0], C, None), (R, C))
    assert known == reached, sorted(k.decode() for k in known - reached)
