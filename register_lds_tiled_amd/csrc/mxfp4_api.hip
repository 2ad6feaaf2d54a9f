// mxfp4_api.hip -- the C entry points of the MXFP4 operators declared in
// include/sgemm.h: argument validation and launch.  Validation happens before
// any HIP call; nothing is launched when it fails.
#include "api_common.h"
#include "mxfp4.h"

namespace {

using namespace sgemm;

long long value_bytes(int k) { return ((long long)k + 1) / 2; }
long long scale_bytes(int k) { return ((long long)k + 31) / 32; }
long long at_least_1(long long n) { return n > 1 ? n : 1; }

// Up to eight byte ranges, outputs first: every output must keep clear of
// all others.
struct Ranges {
    Range r[8];
    int n = 0, outputs = 0;
    bool ok = true;
    void add(const void* p, long long rows, long long row_elements, long long ld, long long esize,
             bool output = false) {
        r[n] = span(p, rows, row_elements, ld, esize);
        ok = ok && r[n].ok;
        ++n;
        if (output) outputs = n;
    }
    int status() const {
        if (!ok) return SGEMM_EINVAL_DIM;
        for (int i = 0; i < outputs; ++i)
            for (int j = i + 1; j < n; ++j)
                if (overlaps(r[i], r[j])) return SGEMM_EALIAS;
        return SGEMM_OK;
    }
};

int quantize(int R, int C, const void* X, int ldx, void* Q, int ldq, void* S, int lds, void* QT,
             int ldqt, void* ST, int ldst, void* stream, MxType t) {
    if (R < 0 || C < 0) return SGEMM_EINVAL_DIM;
    if (ldx < at_least_1(C)) return SGEMM_EINVAL_LD;
    const bool rows = Q != nullptr || S != nullptr, cols = QT != nullptr || ST != nullptr;
    if (rows && (ldq < at_least_1(value_bytes(C)) || lds < at_least_1(scale_bytes(C))))
        return SGEMM_EINVAL_LD;
    if (cols && (ldqt < at_least_1(value_bytes(R)) || ldst < at_least_1(scale_bytes(R))))
        return SGEMM_EINVAL_LD;
    if (R == 0 || C == 0) return SGEMM_OK;
    if (X == nullptr || !(rows || cols)) return SGEMM_EINVAL_PTR;
    if (rows && (Q == nullptr || S == nullptr)) return SGEMM_EINVAL_PTR;
    if (cols && (QT == nullptr || ST == nullptr)) return SGEMM_EINVAL_PTR;
    // Along columns 256 threads per 128 x 128 tile have to fit a launch; along
    // rows alone the grid is bounded by itself.
    const long long tiles = ((long long)R + 127) / 128 * (((long long)C + 127) / 128);
    if (cols && tiles * 256 > 0xFFFFFFFFll) return SGEMM_EINVAL_DIM;
    Ranges g;
    if (rows) {
        g.add(Q, R, value_bytes(C), ldq, 1, true);
        g.add(S, R, scale_bytes(C), lds, 1, true);
    }
    if (cols) {
        g.add(QT, C, value_bytes(R), ldqt, 1, true);
        g.add(ST, C, scale_bytes(R), ldst, 1, true);
    }
    g.add(X, R, C, ldx, t == MxType::f32 ? 4 : 2);
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    MxQuantArgs a{R, C, X, ldx,
                  static_cast<unsigned char*>(Q), ldq, static_cast<unsigned char*>(S), lds,
                  static_cast<unsigned char*>(QT), ldqt, static_cast<unsigned char*>(ST), ldst};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = device_shape(s, a.cus, a.xcds);
    if (e != hipSuccess) return hip_fail(e);
    e = launch_mx_quantize(a, t, s);
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

int dequantize(int R, int C, const void* Q, int ldq, const void* S, int lds, void* Y, int ldy,
               void* stream, MxType t) {
    if (R < 0 || C < 0) return SGEMM_EINVAL_DIM;
    if (ldq < at_least_1(value_bytes(C)) || lds < at_least_1(scale_bytes(C)) || ldy < at_least_1(C))
        return SGEMM_EINVAL_LD;
    if (R == 0 || C == 0) return SGEMM_OK;
    if (Q == nullptr || S == nullptr || Y == nullptr) return SGEMM_EINVAL_PTR;
    Ranges g;
    g.add(Y, R, C, ldy, t == MxType::f32 ? 4 : 2, true);
    g.add(Q, R, value_bytes(C), ldq, 1);
    g.add(S, R, scale_bytes(C), lds, 1);
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    const MxDequantArgs a{R, C, static_cast<const unsigned char*>(Q), ldq,
                          static_cast<const unsigned char*>(S), lds, Y, ldy};
    const hipError_t e = launch_mx_dequantize(a, t, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

// A product's checks and launch.  mx_a: A is MXFP4 (with SA), else 16-bit of
// type t; t is C's type where mx_a, A's otherwise.
int product(int M, int N, int K, const void* A, int lda, const void* SA, int ldsa, const void* B,
            int ldb, const void* SB, int ldsb, void* C, int ldc, void* stream, bool mx_a, MxType t) {
    if (M < 0 || N < 0 || K < 0) return SGEMM_EINVAL_DIM;
    const long long a_row = mx_a ? value_bytes(K) : K, c_size = mx_a && t != MxType::f32 ? 2 : 4;
    if (lda < at_least_1(a_row) || ldb < at_least_1(value_bytes(K)) ||
        ldsb < at_least_1(scale_bytes(K)) || (mx_a && ldsa < at_least_1(scale_bytes(K))) ||
        ldc < at_least_1(N))
        return SGEMM_EINVAL_LD;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr) return SGEMM_EINVAL_PTR;
    if (K > 0 && (A == nullptr || B == nullptr || SB == nullptr || (mx_a && SA == nullptr)))
        return SGEMM_EINVAL_PTR;
    // 256 threads per 64 x 64 tile fit a launch.  No kernel is launched with
    // more: the few-row forms that take more per column are chosen for narrow
    // C, or where their grid fits (mxfp4_rows.hip).
    const long long tiles = ((long long)M + 63) / 64 * (((long long)N + 63) / 64);
    if (tiles * 256 > 0xFFFFFFFFll) return SGEMM_EINVAL_DIM;
    Ranges g;
    g.add(C, M, N, ldc, c_size, true);
    if (K > 0) {
        g.add(A, M, a_row, lda, mx_a ? 1 : 2);
        if (mx_a) g.add(SA, M, scale_bytes(K), ldsa, 1);
        g.add(B, N, value_bytes(K), ldb, 1);
        g.add(SB, N, scale_bytes(K), ldsb, 1);
    }
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    MxGemmArgs a{M, N, K,
                 static_cast<const unsigned char*>(A), mx_a ? lda : 2ll * lda,
                 static_cast<const unsigned char*>(SA), ldsa,
                 static_cast<const unsigned char*>(B), ldb,
                 static_cast<const unsigned char*>(SB), ldsb, C, ldc};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = device_shape(s, a.cus, a.xcds);
    if (e != hipSuccess) return hip_fail(e);
    e = mx_a ? launch_mx_gemm(a, t, s) : launch_mx_wgemm(a, t, s);
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

}  // namespace

extern "C" {

#define MX_QUANTIZE(NAME)                                                                        \
    int gemm_mxfp4_quantize_##NAME(int R, int C, const void* X, int ldx, void* Q, int ldq,       \
                                   void* S, int lds, void* QT, int ldqt, void* ST, int ldst,     \
                                   void* stream) {                                               \
        return quantize(R, C, X, ldx, Q, ldq, S, lds, QT, ldqt, ST, ldst, stream, MxType::NAME); \
    }
#define MX_DEQUANTIZE(NAME)                                                                      \
    int gemm_mxfp4_dequantize_##NAME(int R, int C, const void* Q, int ldq, const void* S,        \
                                     int lds, void* Y, int ldy, void* stream) {                  \
        return dequantize(R, C, Q, ldq, S, lds, Y, ldy, stream, MxType::NAME);                   \
    }
MX_QUANTIZE(f32)
MX_QUANTIZE(bf16)
MX_QUANTIZE(f16)
MX_DEQUANTIZE(f32)
MX_DEQUANTIZE(bf16)
MX_DEQUANTIZE(f16)
#undef MX_QUANTIZE
#undef MX_DEQUANTIZE

int gemm_mxfp4_f32(int M, int N, int K, const void* A, int lda, const void* SA, int ldsa,
                   const void* B, int ldb, const void* SB, int ldsb, float* C, int ldc,
                   void* stream) {
    return product(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, stream, true, MxType::f32);
}

int gemm_mxfp4_bf16(int M, int N, int K, const void* A, int lda, const void* SA, int ldsa,
                    const void* B, int ldb, const void* SB, int ldsb, void* C, int ldc,
                    void* stream) {
    return product(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, stream, true, MxType::bf16);
}

int gemm_bf16_mxfp4_f32(int M, int N, int K, const void* A, int lda, const void* B, int ldb,
                        const void* SB, int ldsb, float* C, int ldc, void* stream) {
    return product(M, N, K, A, lda, nullptr, 0, B, ldb, SB, ldsb, C, ldc, stream, false,
                   MxType::bf16);
}

int gemm_f16_mxfp4_f32(int M, int N, int K, const void* A, int lda, const void* B, int ldb,
                       const void* SB, int ldsb, float* C, int ldc, void* stream) {
    return product(M, N, K, A, lda, nullptr, 0, B, ldb, SB, ldsb, C, ldc, stream, false,
                   MxType::f16);
}

}  // extern "C"
