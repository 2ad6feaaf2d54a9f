// mxfp4_wgemm.hip -- C = A.B^T with 16-bit A and MXFP4 B (weights kept in
// four bits), on the matrix cores, accumulated in fp32.
//
// An MXFP4 value has at most two significant bits and an exponent between
// -128 and 129, so bfloat16 holds it exactly (2^128 and beyond as infinity):
// B's codes become bfloat16 in registers (v_cvt_scalef32_pk_bf16_fp4, two
// elements with their scale) and multiply in v_mfma_f32_16x16x32_bf16.
// binary16 A: where binary16 holds every value of the blocks at hand (scale
// bytes 104 to 140, any usual weight), they become binary16 and multiply in
// v_mfma_f32_16x16x32_f16.  Where it does not, A splits exactly into two
// bfloat16 terms, hi + lo (11 significant bits in 8 + 8), and both multiply
// the same bfloat16 B.
//
// v_mfma_f32_16x16x32_bf16: lane l holds 8 consecutive k of row l % 16 of each
// operand; D: lane l, register i is row 4 (l / 16) + i of the first operand,
// row l % 16 of the second.  B goes first, so a lane holds four neighbouring
// columns of one row of C.
#include "mxfp4.h"

namespace sgemm {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

// The eight values of four bytes of codes: in A's type, or (SPLIT) in bfloat16.
template <MxType T, bool SPLIT>
__device__ __forceinline__ uint4 decode8(unsigned q, float s) {
    unsigned v[4];
    static_for<4>([&](auto i) {
        if constexpr (T == MxType::bf16 || SPLIT)
            v[i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, i));
        else
            v[i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, i));
    });
    return make_uint4(v[0], v[1], v[2], v[3]);
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

// Whether binary16 holds every value of a block with this scale byte: the
// smallest, 2^(byte - 128), from its least subnormal 2^-24, the largest,
// 6 2^(byte - 127), to 65504.
__device__ __forceinline__ bool f16_holds(unsigned byte) { return byte - 104u <= 36u; }

// acc[j] += a step of 32 k for N tiles of B's rows (decoded by decode8 with
// the same SPLIT) and one tile of A's.
template <MxType T, bool SPLIT, int N>
__device__ __forceinline__ void mfma_row(const uint4 (&b)[N], uint4 a, mx_f4 (&acc)[N]) {
    if constexpr (T == MxType::bf16) {
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = mfma_bf16(b[j], a, acc[j]);
    } else if constexpr (SPLIT) {
        uint4 hi, lo;
        split2(a.x, hi.x, lo.x);
        split2(a.y, hi.y, lo.y);
        split2(a.z, hi.z, lo.z);
        split2(a.w, hi.w, lo.w);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = mfma_bf16(b[j], lo, mfma_bf16(b[j], hi, acc[j]));
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, b[j]),
                                                            __builtin_bit_cast(half8, a), acc[j], 0, 0, 0);
    }
}

__device__ __forceinline__ void store4(const MxGemmArgs& p, long long row, long long col, mx_f4 v) {
    if (row >= p.M || col >= p.N) return;
    const int n = (int)min(p.N - col, 4ll);
    float* c = static_cast<float*>(p.C) + row * p.ldc + col;
    if (n == 4 && ((size_t)c & 15) == 0) {
        store_c4(c, v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) store_c(c + i, v[i]);
    }
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
__global__ __launch_bounds__(Cfg::NT, 2) void mx_wtile_kernel(MxGemmArgs p, int tiles_m, int tiles_n) {
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
        bool in_range = true;
        if constexpr (T == MxType::f16) {
            bool ok = true;
#pragma unroll
            for (int j = 0; j < FN; ++j) ok = ok && f16_holds(__float_as_uint(sb[j]) >> 23);
            in_range = __all(ok);
        }
        auto steps = [&](auto split) {
            static_for<4>([&](auto t) {
                uint4 b[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    b[j] = decode8<T, split>(t == 0 ? q[j].x : t == 1 ? q[j].y : t == 2 ? q[j].z : q[j].w, sb[j]);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const uint4 a = as[(wm + 16 * i + li) * 16 + ((4 * g + t) ^ li)];
                    mfma_row<T, split, FN>(b, a, acc[i]);
                }
            });
        };
        if (in_range)
            steps(std::false_type{});
        else
            steps(std::true_type{});
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            store4(p, m0 + wm + 16 * i + li, n0 + wn + 16 * j + 4 * g, acc[i][j]);
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

// Few rows of A (at most 16 MT): B is streamed once.  A workgroup owns 16 NT
// rows of B; its waves take units of 128 k in turn (four blocks of each row,
// one to each lane group), hold a unit's operands and the next one's in
// registers, and add their parts in LDS at the end, in wave order.
template <MxType T, int MT, int NT, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW) void mx_wrows_kernel(MxGemmArgs p) {
    __shared__ mx_f4 part[NW][MT * NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, g = lane >> 4;
    const long long n0 = (long long)blockIdx.x * (16 * NT);
    const long long ks = ((long long)p.K + 31) / 32;
    const unsigned char *b[NT], *sb[NT], *a[MT];
    bool has[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const long long n = min(n0 + 16 * j + li, (long long)p.N - 1);
        b[j] = p.B + n * p.ldb;
        sb[j] = p.SB + n * p.ldsb;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = 16 * i + li;
        has[i] = m < p.M;
        a[i] = p.A + (has[i] ? m : 0) * p.lda;
    }
    struct Unit {
        uint4 b[NT], a[MT][4];
        unsigned s[NT];
    };
    auto load = [&](Unit& u, long long k0) {
        const long long k = k0 + 32 * g;     // the lane's block
        const bool full = k0 + 128 <= p.K;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (full) {
                u.b[j] = mx_load16<VEC>(b[j] + k / 2, 16);
                u.s[j] = sb[j][k / 32];
            } else {
                u.b[j] = mx_codes16<VEC>(b[j], k / 2, p.K);
                u.s[j] = k / 32 < ks ? sb[j][k / 32] : 127u;
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u.a[i][t] = make_uint4(0u, 0u, 0u, 0u);
                if (has[i])
                    u.a[i][t] = load_a<VEC>(a[i] + 2 * k + 16 * t, full ? 16 : 2 * (p.K - k) - 16 * t);
            }
    };
    mx_f4 acc[MT][NT] = {};
    auto step = [&](const Unit& u, auto split) {
        float s[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) s[j] = mx_scale(u.s[j]);
        static_for<4>([&](auto t) {
            uint4 v[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                v[j] = decode8<T, split>(t == 0 ? u.b[j].x : t == 1 ? u.b[j].y : t == 2 ? u.b[j].z : u.b[j].w, s[j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) mfma_row<T, split, NT>(v, u.a[i][t], acc[i]);
        });
    };
    Unit cur, next;
    long long k0 = 128ll * wave;
    if (k0 < p.K) load(cur, k0);
    while (k0 < p.K) {
        const long long k1 = k0 + 128 * NW;
        if (k1 < p.K) load(next, k1);
        bool in_range = true;
        if constexpr (T == MxType::f16) {
            bool ok = true;
#pragma unroll
            for (int j = 0; j < NT; ++j) ok = ok && f16_holds(cur.s[j]);
            in_range = __all(ok);
        }
        if (in_range)
            step(cur, std::false_type{});
        else
            step(cur, std::true_type{});
        cur = next;
        k0 = k1;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    for (int t = wave; t < MT * NT; t += NW) {
        mx_f4 v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part[w][t][lane];
        store4(p, 16 * (t / NT) + li, n0 + 16 * (t % NT) + 4 * g, v);
    }
}

template <MxType T, int MT, int NT, int NW>
hipError_t launch_wrows_cfg(const MxGemmArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)(((long long)a.N + 16 * NT - 1) / (16 * NT));
    if (mx_aligned(a.A, a.lda, 16) && mx_aligned(a.B, a.ldb, 16))
        mx_wrows_kernel<T, MT, NT, NW, true><<<grid, 64 * NW, 0, s>>>(a);
    else
        mx_wrows_kernel<T, MT, NT, NW, false><<<grid, 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

template <MxType T, int MT>
hipError_t launch_wrows(const MxGemmArgs& a, hipStream_t s) {
    constexpr int NT4 = MT == 1 ? 4 : MT == 2 || T == MxType::bf16 ? 2 : 1, NT2 = NT4 < 2 ? NT4 : 2;
    if ((long long)a.N >= 128ll * a.cus) return launch_wrows_cfg<T, MT, NT4, 8>(a, s);
    if ((long long)a.N >= 32ll * a.cus && a.M > 1) return launch_wrows_cfg<T, MT, NT2, 8>(a, s);
    return launch_wrows_cfg<T, MT, 1, 8>(a, s);
}

template <MxType T>
hipError_t launch_w(const MxGemmArgs& a, hipStream_t s) {
    if (a.M <= 16) return launch_wrows<T, 1>(a, s);
    if (a.M <= 32) return launch_wrows<T, 2>(a, s);
    if (a.M <= 64) return launch_wrows<T, 4>(a, s);
    return launch_wtile<WTile<128, 128, 64, 64>, T>(a, s);
}

}  // namespace

hipError_t launch_mx_wgemm(const MxGemmArgs& a, MxType t, hipStream_t s) {
    return t == MxType::bf16 ? launch_w<MxType::bf16>(a, s) : launch_w<MxType::f16>(a, s);
}

}  // namespace sgemm
