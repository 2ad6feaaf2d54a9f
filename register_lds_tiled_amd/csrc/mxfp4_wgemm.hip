// mxfp4_wgemm.hip -- C = A.B^T with 16-bit A and MXFP4 B (weights kept in
// four bits), on the matrix cores, accumulated in fp32.
//
// An MXFP4 value has at most two significant bits and an exponent between
// -128 and 129, so bfloat16 holds it exactly (2^128 and beyond as infinity):
// B's codes become bfloat16 in registers (v_cvt_scalef32_pk_bf16_fp4, two
// elements with their scale) and multiply in v_mfma_f32_16x16x32_bf16.
// binary16 A: binary16 cannot hold all of B's values, but A splits exactly
// into two bfloat16 terms, hi + lo (11 significant bits in 8 + 8), and both
// multiply the same B.
//
// v_mfma_f32_16x16x32_bf16: lane l holds 8 consecutive k of row l % 16 of each
// operand; D: lane l, register i is row 4 (l / 16) + i of the first operand,
// row l % 16 of the second.  B goes first, so a lane holds four neighbouring
// columns of one row of C.
#include "mxfp4.h"

namespace sgemm {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

// The eight values of four bytes of codes, as bfloat16.
__device__ __forceinline__ uint4 decode8(unsigned q, float s) {
    uint4 v;
    v.x = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
    v.y = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
    v.z = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
    v.w = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
    return v;
}

// Two binary16 values as bfloat16 hi and lo with hi + lo their exact sum: hi
// is the value's upper part (truncated), lo the rest.  An infinity is hi
// alone; a NaN stays NaN in hi (binary16's payload lies in the upper bits).
__device__ __forceinline__ void split2(unsigned h2, unsigned& hi, unsigned& lo) {
    const mx_h2 h = __builtin_bit_cast(mx_h2, h2);
    const float x = (float)h[0], y = (float)h[1];
    const unsigned xb = __float_as_uint(x) & 0xFFFF0000u, yb = __float_as_uint(y) & 0xFFFF0000u;
    const float xh = __uint_as_float(xb), yh = __uint_as_float(yb);
    const float xl = x == xh ? 0.f : x - xh, yl = y == yh ? 0.f : y - yh;
    hi = (xb >> 16) | yb;
    lo = (__float_as_uint(xl) >> 16) | (__float_as_uint(yl) & 0xFFFF0000u);
}

__device__ __forceinline__ mx_f4 mfma_bf16(uint4 b, uint4 a, mx_f4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, b), __builtin_bit_cast(bf8, a),
                                                   acc, 0, 0, 0);
}

__device__ __forceinline__ void store4(const MxGemmArgs& p, long long row, int col, mx_f4 v) {
    if (row >= p.M || col >= p.N) return;
    const int n = min(p.N - col, 4);
    float* c = static_cast<float*>(p.C) + row * p.ldc + col;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) store_c(c + i, v[i]);
}

// 16 bytes of A of which the first n exist (n even).
template <bool VEC>
__device__ __forceinline__ uint4 load_a(const unsigned char* p, long long n) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n >= 16) {
        if constexpr (VEC)
            v = *reinterpret_cast<const uint4*>(p);
        else
            __builtin_memcpy(&v, p, 16);
    } else if (n > 0) {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
        unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (2 * i < n) w[i / 2] |= (unsigned)h[i] << (16 * (i % 2));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

// Tiles: four waves own BM x BN outputs and walk K in stages of 128.  LDS
// holds a stage of A (256 bytes a row, chunk c of row r at c ^ (r & 15)), of
// B's codes (64 bytes a row, chunk c at c ^ ((r >> 1) & 3)) and B's 4 scale
// bytes a row.  Lane group g takes block g of the stage, eight elements of it
// in each of four steps.  k past K reads as 0 in A and in B's codes and scales.
template <int BM_, int BN_, int WM_, int WN_>
struct WTile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 128;
    static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * (BN / WN), NT = NW * 64;
    static constexpr int FM = WM / 16, FN = WN / 16;
};

template <class Cfg, MxType T, bool VEC>
__global__ __launch_bounds__(Cfg::NT) void mx_wtile_kernel(MxGemmArgs p, int tiles_m, int tiles_n) {
    constexpr int BM = Cfg::BM, BN = Cfg::BN, NT = Cfg::NT, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int CA = BM * 16 / NT, CB = BN * 4 / NT;
    static_assert(BM * 16 % NT == 0 && BN * 4 % NT == 0 && BN <= NT, "whole rounds of the loader");
    __shared__ __attribute__((aligned(16))) uint4 as[BM * 16];
    __shared__ __attribute__((aligned(16))) uint4 bs[BN * 4];
    __shared__ unsigned sc[BN];
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, 8, p.xcds, tm, tn);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / Cfg::WAVES_N) * Cfg::WM, wn = (wave % Cfg::WAVES_N) * Cfg::WN;
    const int li = lane & 15, g = lane >> 4;
    const long long m0 = (long long)tm * BM, n0 = (long long)tn * BN;
    const long long ka = 2ll * p.K, ks = ((long long)p.K + 31) / 32;

    uint4 va[CA], vb[CB];
    unsigned s[1];
    auto fetch = [&](long long k0) {
#pragma unroll
        for (int u = 0; u < CA; ++u) {
            const int id = tid + u * NT, r = id >> 4, c = id & 15;
            const long long at = 2 * k0 + 16 * c;
            va[u] = load_a<VEC>(p.A + min(m0 + r, (long long)p.M - 1) * p.lda + at, ka - at);
        }
#pragma unroll
        for (int u = 0; u < CB; ++u) {
            const int id = tid + u * NT, r = id >> 2, c = id & 3;
            vb[u] = mx_codes16<VEC>(p.B + min(n0 + r, (long long)p.N - 1) * p.ldb, k0 / 2 + 16 * c, p.K);
        }
        mx_scales<4>(p.SB + min(n0 + (tid < BN ? tid : 0), (long long)p.N - 1) * p.ldsb, k0 / 32, ks, s);
    };

    mx_f4 acc[FM][FN] = {};
    fetch(0);
    for (long long k0 = 0; k0 < p.K; k0 += Cfg::BK) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < CA; ++u) {
            const int id = tid + u * NT, r = id >> 4, c = id & 15;
            as[r * 16 + (c ^ (r & 15))] = va[u];
        }
#pragma unroll
        for (int u = 0; u < CB; ++u) {
            const int id = tid + u * NT, r = id >> 2, c = id & 3;
            bs[r * 4 + (c ^ ((r >> 1) & 3))] = vb[u];
        }
        if (tid < BN) sc[tid] = s[0];
        __syncthreads();
        if (k0 + Cfg::BK < p.K) fetch(k0 + Cfg::BK);
        uint4 q[FN];
        float sb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int r = wn + 16 * j + li;
            q[j] = bs[r * 4 + (g ^ ((r >> 1) & 3))];
            sb[j] = mx_scale((sc[r] >> (8 * g)) & 255u);
        }
        static_for<4>([&](auto t) {
            uint4 b[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const unsigned w = t == 0 ? q[j].x : t == 1 ? q[j].y : t == 2 ? q[j].z : q[j].w;
                b[j] = decode8(w, sb[j]);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const uint4 a = as[(wm + 16 * i + li) * 16 + ((4 * g + t) ^ li)];
                if constexpr (T == MxType::bf16) {
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[i][j] = mfma_bf16(b[j], a, acc[i][j]);
                } else {
                    uint4 hi, lo;
                    split2(a.x, hi.x, lo.x);
                    split2(a.y, hi.y, lo.y);
                    split2(a.z, hi.z, lo.z);
                    split2(a.w, hi.w, lo.w);
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        acc[i][j] = mfma_bf16(b[j], hi, acc[i][j]);
                        acc[i][j] = mfma_bf16(b[j], lo, acc[i][j]);
                    }
                }
            }
        });
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            store4(p, m0 + wm + 16 * i + li, (int)(n0 + wn + 16 * j + 4 * g), acc[i][j]);
}

template <class Cfg, MxType T>
hipError_t launch_wtile(const MxGemmArgs& a, hipStream_t s) {
    const int tm = (int)(((long long)a.M + Cfg::BM - 1) / Cfg::BM);
    const int tn = (int)(((long long)a.N + Cfg::BN - 1) / Cfg::BN);
    const bool vec = mx_aligned(a.A, a.lda, 16) && mx_aligned(a.B, a.ldb, 16);
    if (vec)
        mx_wtile_kernel<Cfg, T, true><<<(unsigned)tm * tn, Cfg::NT, 0, s>>>(a, tm, tn);
    else
        mx_wtile_kernel<Cfg, T, false><<<(unsigned)tm * tn, Cfg::NT, 0, s>>>(a, tm, tn);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_wgemm(const MxGemmArgs& a, MxType t, hipStream_t s) {
    return t == MxType::bf16 ? launch_wtile<WTile<128, 128, 64, 64>, MxType::bf16>(a, s)
                             : launch_wtile<WTile<128, 128, 64, 64>, MxType::f16>(a, s);
}

}  // namespace sgemm
