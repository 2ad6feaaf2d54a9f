"""CPU tests of what the MXFP4 entry points launch: the kernels chosen and the
sizes of their grids, up to the largest dimensions an int holds.  The host side
of the library's MXFP4 sources is built against a stand-in for the HIP runtime
that records each launch and, as the runtime does, refuses one of more than
2^32 - 1 threads.  No GPU is used; device addresses are fake."""
import ctypes
import os
import subprocess

import pytest

from register_lds_tiled_amd import binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "register_lds_tiled_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
SOURCES = ["mxfp4_api", "mxfp4_cast", "mxfp4_gemm", "mxfp4_rows", "mxfp4_wgemm"]

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="ROCm toolchain missing")

RUNTIME = r"""
#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>
#include <map>
#include <string>
static std::map<const void*, std::string>& names() { static std::map<const void*, std::string> m; return m; }
static dim3 grid, block;
static size_t shared;
static hipStream_t queue;
static hipError_t last = hipSuccess;
static std::string kernel;
static unsigned long long groups, threads;
static int count;
extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* p; return &p; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
    names()[f] = name;
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, hipStream_t q) {
    grid = g; block = b; shared = s; queue = q;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* s, hipStream_t* q) {
    *g = grid; *b = block; *s = shared; *q = queue;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t, hipStream_t) {
    ++count;
    kernel = names()[f];
    groups = 1ull * g.x * g.y * g.z;
    threads = 1ull * b.x * b.y * b.z;
    if (groups * threads > 0xFFFFFFFFull || groups == 0) last = hipErrorInvalidConfiguration;
    return last;
}
hipError_t hipGetLastError() { hipError_t e = last; last = hipSuccess; return e; }
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipStreamGetDevice(hipStream_t, hipDevice_t* d) { *d = 0; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t a, int) {
    *v = a == hipDeviceAttributeMultiprocessorCount ? 256 : 8;
    return hipSuccess;
}
const char* hipGetErrorName(hipError_t) { return "error"; }
const char* hipGetErrorString(hipError_t) { return "error"; }
int record_known() { return (int)names().size(); }
const char* record_name(int i) { auto it = names().begin(); while (i-- > 0) ++it; return it->second.c_str(); }
const char* record_kernel() { return kernel.c_str(); }
unsigned long long record_groups() { return groups; }
unsigned long long record_threads() { return threads; }
int record_count() { int n = count; count = 0; return n; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    flags = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC", "-w",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    jobs = [subprocess.Popen([HIPCC, *flags, "-c", os.path.join(CSRC, n + ".hip"), "-o", str(d / (n + ".o"))],
                             stdout=subprocess.DEVNULL, stderr=subprocess.PIPE) for n in SOURCES]
    for j in jobs:
        log = j.communicate()[1]
        assert j.returncode == 0, log.decode(errors="replace")[-2000:]
    objs = [str(d / (n + ".o")) for n in SOURCES]
    # what a device image would be called, one per source
    undefined = subprocess.run(["nm", "-u", *objs], capture_output=True, text=True, check=True).stdout.split()
    images = sorted({s for s in undefined if s.startswith("__hip_fatbin")})
    (d / "runtime.cpp").write_text(RUNTIME + "".join(f'extern "C" {{ char {s}[16]; }}\n' for s in images))
    so = d / "launches.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-w", "-I/opt/rocm/include", "-Wl,-Bsymbolic",
                    str(d / "runtime.cpp"), *objs, "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    i, p = ctypes.c_int, ctypes.c_void_p
    for t in ("f32", "bf16", "f16"):
        getattr(lib, f"gemm_mxfp4_quantize_{t}").argtypes = [i, i, p, i, p, i, p, i, p, i, p, i, p]
        getattr(lib, f"gemm_mxfp4_dequantize_{t}").argtypes = [i, i, p, i, p, i, p, i, p]
    for t in ("f32", "bf16"):
        getattr(lib, f"gemm_mxfp4_{t}").argtypes = [i, i, i, p, i, p, i, p, i, p, i, p, i, p]
    for t in ("bf16", "f16"):
        getattr(lib, f"gemm_{t}_mxfp4_f32").argtypes = [i, i, i, p, i, p, i, p, i, p, i, p]
    lib.record_kernel.restype = lib.record_name.restype = ctypes.c_char_p
    lib.record_groups.restype = lib.record_threads.restype = ctypes.c_ulonglong
    return lib


TOP = 2 ** 31 - 1
A, SA, B, SB, C, D = (0x1000_0000_0000 * n for n in range(1, 7))     # 16 TB apart


def product(lib, kind, M, N, K, pad=0):
    """Status of a product whose rows lie 16-byte aligned, or `pad` bytes off."""
    codes, scales = -(-K // 32) * 16 + pad, -(-K // 32)
    lib.record_count()
    if kind in ("f32", "bf16"):
        return getattr(lib, f"gemm_mxfp4_{kind}")(M, N, K, A, codes, SA, scales, B, codes, SB, scales, C, N, None)
    t = kind.split("-")[1]
    return getattr(lib, f"gemm_{t}_mxfp4_f32")(M, N, K, A, -(-K // 8) * 8 + pad, B, codes, SB, scales, C, N, None)


KINDS = ["f32", "bf16", "a-bf16", "a-f16"]
# the widest C that one workgroup of 256 threads per 64 x 64 tile covers
WIDE = 64 * (2 ** 24 - 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 2, 16, 17, 64])
@pytest.mark.parametrize("N", [1, 8192, 32767, 32768, 2 ** 29 - 32, 2 ** 29 - 31, 2 ** 29, 2 ** 29 + 37, WIDE])
def test_products_of_few_rows_launch(lib, kind, M, N):
    """Every number of columns that passes the argument checks is launched."""
    assert product(lib, kind, M, N, 32) == b.SGEMM_OK, (lib.record_kernel(), lib.record_groups(), lib.record_threads())
    assert lib.record_count() == 1
    if M <= 16:
        assert b"mx_rows_kernel" in lib.record_kernel()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [0, 1])
def test_products_launch_or_are_refused(lib, kind, pad):
    """The largest C of any form, and beyond it SGEMM_EINVAL_DIM without a launch."""
    for M, N in ((WIDE, 1), (WIDE, 64), (64, WIDE), (64 * 4095, 64 * 4096), (100, 64 * (2 ** 23 - 1))):
        assert product(lib, kind, M, N, 32, pad) == b.SGEMM_OK, (M, N, lib.record_kernel(), lib.record_groups())
        assert lib.record_count() == 1
    for M, N in ((1, WIDE + 1), (1, TOP), (16, TOP), (WIDE + 1, 1), (TOP, 1), (65, WIDE), (100, 64 * 2 ** 23),
                 (TOP, TOP)):
        assert product(lib, kind, M, N, 1, pad) == b.SGEMM_EINVAL_DIM, (M, N)
        assert lib.record_count() == 0


def quantise(lib, t, R, C, rows, cols):
    codes, scales = (-(-C // 2), -(-C // 32)) if rows else (0, 0)
    codest, scalest = (-(-R // 2), -(-R // 32)) if cols else (0, 0)
    lib.record_count()
    return getattr(lib, f"gemm_mxfp4_quantize_{t}")(R, C, A, C, SA if rows else None, codes, B if rows else None, scales,
                                                    SB if cols else None, codest, D if cols else None, scalest, None)


def test_every_kernel_is_launched_by_some_call(lib):
    """The library holds no MXFP4 kernel that no call reaches."""
    known = {lib.record_name(i) for i in range(lib.record_known())}
    assert len(known) > 20
    reached = set()

    def call(status):
        assert status == b.SGEMM_OK and lib.record_count() == 1
        reached.add(lib.record_kernel())

    for kind in KINDS:
        for M in (1, 2, 16, 17, 32, 33, 64, 65, 1000, 8192):
            for N in (16, 1000, 8191, 8192, 16383, 16384, 32768, 65536):
                for pad in (0, 1):
                    call(product(lib, kind, M, N, 1000, pad))
    for t in ("f32", "bf16", "f16"):
        for R, C_ in ((1, 1), (100, 100), (64, 200000), (300, 200000), (8192, 8192)):
            for rows, cols in ((True, False), (False, True), (True, True)):
                call(quantise(lib, t, R, C_, rows, cols))
            for off in (0, 2):
                fn = getattr(lib, f"gemm_mxfp4_dequantize_{t}")
                call(fn(R, C_, SA, -(-C_ // 2), SB, -(-C_ // 32), C + off, C_ + off, None))
    assert known == reached, sorted(k.decode() for k in known - reached)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_quantising_launches_or_is_refused(lib, t):
    """Along columns, up to the last X that one workgroup of 256 threads per
    128 x 128 tile covers, and beyond it SGEMM_EINVAL_DIM without a launch;
    along rows any X."""
    last = 128 * (2 ** 24 - 1)
    for R, C_ in ((1, 2 ** 30 - 128), (1, 2 ** 30), (1, last), (32, 2 ** 30 + 1), (128, last), (129, 2 ** 30 - 128),
                  (300, 128 * (2 ** 24 // 3)), (last, 1), (2 ** 30, 128), (2 ** 30 - 128, 129)):
        for rows in (False, True):
            assert quantise(lib, t, R, C_, rows, True) == b.SGEMM_OK, (R, C_, lib.record_groups(), lib.record_threads())
            assert lib.record_count() == 1
    for R, C_ in ((1, last + 1), (1, TOP), (TOP, 1), (last + 1, 128), (129, 2 ** 30 + 1), (2 ** 30, 129)):
        for rows in (False, True):
            assert quantise(lib, t, R, C_, rows, True) == b.SGEMM_EINVAL_DIM, (R, C_)
            assert lib.record_count() == 0
        assert quantise(lib, t, R, C_, True, False) == b.SGEMM_OK and lib.record_count() == 1


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_quantising_few_rows_leaves_no_wave_idle(lib, t):
    """A tile of 256 rows for at most 128 would leave half of its waves and more
    without any; from there on it is taken where it fills the CUs."""
    for R, threads in ((1, 256), (32, 256), (128, 256), (129, 512), (256, 512)):
        for rows in (False, True):
            assert quantise(lib, t, R, 65536, rows, True) == b.SGEMM_OK
            assert lib.record_threads() == threads, (R, rows)
            assert quantise(lib, t, R, 65408, rows, True) == b.SGEMM_OK     # 511 tiles for 256 CUs
            assert lib.record_threads() == 256, (R, rows)
