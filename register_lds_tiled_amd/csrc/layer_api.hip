// layer_api.hip -- the C entry points of the 8-bit integer operators and of the
// gated feed-forward block declared in include/sgemm.h: argument validation and
// launch.  Validation happens before any HIP call; nothing is launched when it
// fails.
#include "api_common.h"
#include "layer.h"

namespace {

using namespace sgemm;

constexpr int kMostK = 131071;   // of 8-bit products: 131071 * 128 * 128 < 2^31

bool act_known(int act) { return act >= SGEMM_ACT_NONE && act <= SGEMM_ACT_GELU_TANH; }

// 256 threads per 64 x 64 tile of an output, or of all outputs of one launch, fit
// a launch; no kernel here is launched with more.
bool launchable(long long rows, long long cols, int outputs = 1) {
    return (rows + 63) / 64 * ((cols + 63) / 64) * outputs * 256 <= 0xFFFFFFFFll;
}

int quantize(int R, int C, const void* X, int ldx, void* Q, int ldq, float* S, void* stream, Elem t) {
    if (R < 0 || C < 0) return SGEMM_EINVAL_DIM;
    if (ldx < at_least_1(C) || ldq < at_least_1(C)) return SGEMM_EINVAL_LD;
    if (R == 0 || C == 0) return SGEMM_OK;
    if (X == nullptr || Q == nullptr || S == nullptr) return SGEMM_EINVAL_PTR;
    Ranges g;
    g.add(Q, R, C, ldq, 1, true);
    g.add(S, 1, R, R, 4, true);
    g.add(X, R, C, ldx, t == Elem::f32 ? 4 : 2);
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    I8CastArgs a{R, C, X, ldx, Q, ldq, S};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = device_shape(s, a.cus, a.xcds);
    if (e != hipSuccess) return hip_fail(e);
    e = launch_i8_quantize(a, t, s);
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

int dequantize(int R, int C, const void* Q, int ldq, const float* S, void* Y, int ldy, void* stream, Elem t) {
    if (R < 0 || C < 0) return SGEMM_EINVAL_DIM;
    if (ldq < at_least_1(C) || ldy < at_least_1(C)) return SGEMM_EINVAL_LD;
    if (R == 0 || C == 0) return SGEMM_OK;
    if (Q == nullptr || S == nullptr || Y == nullptr) return SGEMM_EINVAL_PTR;
    Ranges g;
    g.add(Y, R, C, ldy, t == Elem::f32 ? 4 : 2, true);
    g.add(Q, R, C, ldq, 1);
    g.add(S, 1, R, R, 4);
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    I8CastArgs a{R, C, Y, ldy, const_cast<void*>(Q), ldq, const_cast<float*>(S)};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = device_shape(s, a.cus, a.xcds);
    if (e != hipSuccess) return hip_fail(e);
    e = launch_i8_dequantize(a, t, s);
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

// gated: B2 and SB2 the second projection.
int i8_product(int M, int N, int K, const void* A, int lda, const float* SA, const void* B, int ldb, const float* SB,
               const void* B2, int ldb2, const float* SB2, void* C, int ldc, int act, void* stream, bool gated,
               Elem out) {
    if (gated && !act_known(act)) return SGEMM_EINVAL_ACT;
    if (M < 0 || N < 0 || K < 0 || K > kMostK) return SGEMM_EINVAL_DIM;
    if (lda < at_least_1(K) || ldb < at_least_1(K) || (gated && ldb2 < at_least_1(K)) || ldc < at_least_1(N))
        return SGEMM_EINVAL_LD;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr) return SGEMM_EINVAL_PTR;
    if (K > 0 && (A == nullptr || B == nullptr || SA == nullptr || SB == nullptr ||
                  (gated && (B2 == nullptr || SB2 == nullptr))))
        return SGEMM_EINVAL_PTR;
    if (!launchable(M, N)) return SGEMM_EINVAL_DIM;
    Ranges g;
    g.add(C, M, N, ldc, out == Elem::f32 ? 4 : 2, true);
    if (K > 0) {
        g.add(A, M, K, lda, 1);
        g.add(SA, 1, M, M, 4);
        g.add(B, N, K, ldb, 1);
        g.add(SB, 1, N, N, 4);
        if (gated) {
            g.add(B2, N, K, ldb2, 1);
            g.add(SB2, 1, N, N, 4);
        }
    }
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    LayerArgs a{M, N, K,
                {static_cast<const unsigned char*>(A), nullptr}, {lda, 0},
                {static_cast<const unsigned char*>(B), static_cast<const unsigned char*>(B2)}, {ldb, ldb2},
                SA, {SB, SB2}, {C, nullptr}, {ldc, 0}};
    a.act = act;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = device_shape(s, a.cus, a.xcds);
    if (e != hipSuccess) return hip_fail(e);
    e = gated ? launch_i8_gated(a, out, s) : launch_i8_nt(a, out, s);
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

int gated(int M, int N, int K, const void* X, int ldx, const void* WG, int ldwg, const void* WU, int ldwu, void* G,
          int ldg, void* U, int ldu, void* H, int ldh, int act, void* stream, Elem t) {
    if (!act_known(act)) return SGEMM_EINVAL_ACT;
    if (M < 0 || N < 0 || K < 0) return SGEMM_EINVAL_DIM;
    const bool keep = G != nullptr || U != nullptr;
    if (ldx < at_least_1(K) || ldwg < at_least_1(K) || ldwu < at_least_1(K) || ldh < at_least_1(N) ||
        (keep && (ldg < at_least_1(N) || ldu < at_least_1(N))))
        return SGEMM_EINVAL_LD;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (H == nullptr || (keep && (G == nullptr || U == nullptr))) return SGEMM_EINVAL_PTR;
    if (K > 0 && (X == nullptr || WG == nullptr || WU == nullptr)) return SGEMM_EINVAL_PTR;
    if (!launchable(M, N)) return SGEMM_EINVAL_DIM;
    Ranges g;
    g.add(H, M, N, ldh, 2, true);
    if (keep) {
        g.add(G, M, N, ldg, 2, true);
        g.add(U, M, N, ldu, 2, true);
    }
    if (K > 0) {
        g.add(X, M, K, ldx, 2);
        g.add(WG, N, K, ldwg, 2);
        g.add(WU, N, K, ldwu, 2);
    }
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    LayerArgs a{M, N, K,
                {static_cast<const unsigned char*>(X), nullptr}, {2ll * ldx, 0},
                {static_cast<const unsigned char*>(WG), static_cast<const unsigned char*>(WU)},
                {2ll * ldwg, 2ll * ldwu},
                nullptr, {nullptr, nullptr}, {H, nullptr}, {ldh, 0}, G, U, ldg, ldu, act};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = device_shape(s, a.cus, a.xcds);
    if (e != hipSuccess) return hip_fail(e);
    e = launch_gated(a, t, s);
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

int gated_backward(int M, int N, int K, const void* X, int ldx, const void* WG, int ldwg, const void* WU, int ldwu,
                   const void* G, int ldg, const void* U, int ldu, const void* DH, int lddh, void* DG, int lddg,
                   void* DU, int lddu, void* DX, int lddx, void* DWG, int lddwg, void* DWU, int lddwu, int act,
                   void* stream, Elem t) {
    if (!act_known(act)) return SGEMM_EINVAL_ACT;
    if (M < 0 || N < 0 || K < 0) return SGEMM_EINVAL_DIM;
    const bool ask_x = DX != nullptr, ask_w = DWG != nullptr || DWU != nullptr;
    const long long n = at_least_1(N), k = at_least_1(K);
    if (ldg < n || ldu < n || lddh < n || lddg < n || lddu < n) return SGEMM_EINVAL_LD;
    if (ask_x && (ldwg < k || ldwu < k || lddx < k)) return SGEMM_EINVAL_LD;
    if (ask_w && (ldx < k || lddwg < k || lddwu < k)) return SGEMM_EINVAL_LD;
    if (ask_w && (DWG == nullptr || DWU == nullptr)) return SGEMM_EINVAL_PTR;
    const bool slopes = M > 0 && N > 0;
    const bool dx = ask_x && M > 0 && K > 0, dw = ask_w && N > 0 && K > 0;
    if (!slopes && !dx && !dw) return SGEMM_OK;
    if (slopes && (G == nullptr || U == nullptr || DH == nullptr || DG == nullptr || DU == nullptr))
        return SGEMM_EINVAL_PTR;
    if (dx && N > 0 && (WG == nullptr || WU == nullptr)) return SGEMM_EINVAL_PTR;
    if (dw && M > 0 && X == nullptr) return SGEMM_EINVAL_PTR;
    if ((slopes && !launchable(M, N)) || (dx && !launchable(M, K)) || (dw && !launchable(N, K, 2)))
        return SGEMM_EINVAL_DIM;
    Ranges g;
    if (slopes) {
        g.add(DG, M, N, lddg, 2, true);
        g.add(DU, M, N, lddu, 2, true);
    }
    if (dx) g.add(DX, M, K, lddx, 2, true);
    if (dw) {
        g.add(DWG, N, K, lddwg, 2, true);
        g.add(DWU, N, K, lddwu, 2, true);
    }
    if (slopes) {
        g.add(G, M, N, ldg, 2);
        g.add(U, M, N, ldu, 2);
        g.add(DH, M, N, lddh, 2);
    }
    if (dx && N > 0) {
        g.add(WG, N, K, ldwg, 2);
        g.add(WU, N, K, ldwu, 2);
    }
    if (dw && M > 0) g.add(X, M, K, ldx, 2);
    const int v = g.status();
    if (v != SGEMM_OK) return v;
    typedef const unsigned char* In;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    int cus = 256, xcds = 8;
    hipError_t e = device_shape(s, cus, xcds);
    if (e == hipSuccess && slopes)
        e = launch_gated_slopes({M, N, (In)G, (In)U, (In)DH, ldg, ldu, lddh, (unsigned char*)DG, (unsigned char*)DU,
                                 lddg, lddu, act, cus}, t, s);
    LayerArgs a{M, K, N,
                {(In)DG, (In)DU}, {2ll * lddg, 2ll * lddu}, {(In)WG, (In)WU}, {2ll * ldwg, 2ll * ldwu},
                nullptr, {nullptr, nullptr}, {DX, nullptr}, {lddx, 0}};
    a.cus = cus;
    a.xcds = xcds;
    if (e == hipSuccess && dx) e = launch_gated_dx(a, t, s);
    a.M = N;
    a.K = M;
    a.B[0] = (In)X;
    a.ldb[0] = 2ll * ldx;
    a.C[0] = DWG;
    a.C[1] = DWU;
    a.ldc[0] = lddwg;
    a.ldc[1] = lddwu;
    if (e == hipSuccess && dw) e = launch_gated_dw(a, t, s);
    return e == hipSuccess ? SGEMM_OK : hip_fail(e);
}

}  // namespace

extern "C" {

#define I8_CASTS(T)                                                                                           \
    int gemm_i8_quantize_##T(int R, int C, const void* X, int ldx, void* Q, int ldq, float* S, void* stream) { \
        return quantize(R, C, X, ldx, Q, ldq, S, stream, Elem::T);                                            \
    }                                                                                                         \
    int gemm_i8_dequantize_##T(int R, int C, const void* Q, int ldq, const float* S, void* Y, int ldy,        \
                               void* stream) {                                                                \
        return dequantize(R, C, Q, ldq, S, Y, ldy, stream, Elem::T);                                          \
    }
I8_CASTS(f32)
I8_CASTS(bf16)
I8_CASTS(f16)
#undef I8_CASTS

int gemm_i8_f32(int M, int N, int K, const void* A, int lda, const float* SA, const void* B, int ldb, const float* SB,
                float* C, int ldc, void* stream) {
    return i8_product(M, N, K, A, lda, SA, B, ldb, SB, nullptr, 0, nullptr, C, ldc, 0, stream, false, Elem::f32);
}
int gemm_i8_bf16(int M, int N, int K, const void* A, int lda, const float* SA, const void* B, int ldb, const float* SB,
                 void* C, int ldc, void* stream) {
    return i8_product(M, N, K, A, lda, SA, B, ldb, SB, nullptr, 0, nullptr, C, ldc, 0, stream, false, Elem::bf16);
}
int gemm_i8_f16(int M, int N, int K, const void* A, int lda, const float* SA, const void* B, int ldb, const float* SB,
                void* C, int ldc, void* stream) {
    return i8_product(M, N, K, A, lda, SA, B, ldb, SB, nullptr, 0, nullptr, C, ldc, 0, stream, false, Elem::f16);
}

#define GATED(T)                                                                                                    \
    int gemm_i8_gated_##T(int M, int N, int K, const void* A, int lda, const float* SA, const void* BG, int ldbg,   \
                          const float* SBG, const void* BU, int ldbu, const float* SBU, void* H, int ldh, int act,  \
                          void* stream) {                                                                           \
        return i8_product(M, N, K, A, lda, SA, BG, ldbg, SBG, BU, ldbu, SBU, H, ldh, act, stream, true, Elem::T);   \
    }                                                                                                               \
    int gemm_gated_##T(int M, int N, int K, const void* X, int ldx, const void* WG, int ldwg, const void* WU,       \
                       int ldwu, void* G, int ldg, void* U, int ldu, void* H, int ldh, int act, void* stream) {     \
        return gated(M, N, K, X, ldx, WG, ldwg, WU, ldwu, G, ldg, U, ldu, H, ldh, act, stream, Elem::T);            \
    }                                                                                                               \
    int gemm_gated_backward_##T(int M, int N, int K, const void* X, int ldx, const void* WG, int ldwg,              \
                                const void* WU, int ldwu, const void* G, int ldg, const void* U, int ldu,           \
                                const void* DH, int lddh, void* DG, int lddg, void* DU, int lddu, void* DX,         \
                                int lddx, void* DWG, int lddwg, void* DWU, int lddwu, int act, void* stream) {      \
        return gated_backward(M, N, K, X, ldx, WG, ldwg, WU, ldwu, G, ldg, U, ldu, DH, lddh, DG, lddg, DU, lddu,    \
                              DX, lddx, DWG, lddwg, DWU, lddwu, act, stream, Elem::T);                              \
    }
GATED(bf16)
GATED(f16)
#undef GATED

}  // extern "C"
