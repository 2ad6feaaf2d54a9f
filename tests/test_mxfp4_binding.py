"""CPU tests of the binding's own checks of an MXFP4 call's arguments, which the
C library cannot make (no GPU is used; addresses are fake)."""
import pytest

from register_lds_tiled_amd import binding as b

A, SA, B, SB, C, D = (0x1000_0000 + (i << 24) for i in range(6))
# integers that no C int holds, the first of which a cut to 32 bits would make
# another valid size
BEYOND = [2 ** 32 + 64, 2 ** 32, 2 ** 31, -2 ** 31 - 1, 10 ** 30]

# each entry point with valid arguments for nothing to do (no row), and the
# places of its dimensions and leading dimensions
CALLS = {f"gemm_mxfp4_quantize_{t}": ([0, 64, A, 64, SA, 32, B, 2, SB, 1, C, 1], (0, 1, 3, 5, 7, 9, 11))
         for t in ("f32", "bf16", "f16")}
CALLS.update({f"gemm_mxfp4_dequantize_{t}": ([0, 64, A, 32, SA, 2, C, 64], (0, 1, 3, 5, 7))
              for t in ("f32", "bf16", "f16")})
CALLS.update({f"gemm_mxfp4_{t}": ([0, 4, 64, A, 32, SA, 2, B, 32, SB, 2, C, 4], (0, 1, 2, 4, 6, 8, 10, 12))
              for t in ("f32", "bf16")})
CALLS.update({f"gemm_{t}_mxfp4_f32": ([0, 4, 64, A, 64, B, 32, SB, 2, C, 4], (0, 1, 2, 4, 6, 8, 10))
              for t in ("bf16", "f16")})


@pytest.mark.parametrize("name", list(CALLS))
def test_integers_that_no_c_int_holds(name):
    """They are refused, not cut to their lowest 32 bits."""
    args, places = CALLS[name]
    fn = getattr(b, name)
    assert fn(*args, stream=0) == b.SGEMM_OK
    for i in places:
        for v in BEYOND:
            with pytest.raises(OverflowError, match=name):
                fn(*args[:i], v, *args[i + 1:], stream=0)
        # an int's ends reach the library's own checks (with no row, or a negative number of them)
        for v in (-2 ** 31,) if i == 0 else (2 ** 31 - 1, -2 ** 31):
            assert fn(*args[:i], v, *args[i + 1:], stream=0, check=False) in (
                b.SGEMM_OK, b.SGEMM_EINVAL_DIM, b.SGEMM_EINVAL_LD)
