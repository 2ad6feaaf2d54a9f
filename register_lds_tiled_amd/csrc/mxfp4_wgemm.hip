// mxfp4_wgemm.hip -- C = A.B^T with 16-bit A and MXFP4 B (weights kept in
// four bits), on the matrix cores, accumulated in fp32.
//
// An MXFP4 value has at most two significant bits and an exponent between
// -128 and 129, so bfloat16 holds it exactly (2^128 and beyond as infinity):
// B's codes become bfloat16 in registers (v_cvt_scalef32_pk_bf16_fp4, two
// elements with their scale) and multiply in v_mfma_f32_32x32x16_bf16 (16x16x32
// where rows are few or off 16 bytes).  binary16 A: where binary16 holds every
// value of the blocks at hand (scale bytes 104 to 140, any usual weight), they
// become binary16 and multiply in the same instructions' _f16 forms.  Where it
// does not, A splits exactly into two bfloat16 terms, hi + lo (11 significant
// bits in 8 + 8), and both multiply the same bfloat16 B.
//
// Few rows of A (at most 16, or 64 where C is narrow: mx_few_rows):
// mxfp4_rows.hip.  Else 128 x 128 tiles, by DMA where rows are 16-byte aligned:
// 4096 x 8192 x 8192 takes 454 us (1.21 PFLOP/s), 521 with binary16 A, whose
// loop differs by a vote and a branch on the scales' range in every half stage;
// the product of two bfloat16 matrices, whose 1.35 to 1.42 PFLOP/s power bounds,
// has no conversions to do.
#include "mxfp4.h"

namespace sgemm {
namespace {

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

template <class Cfg, MxType T>
__global__ __launch_bounds__(Cfg::NT, 1) void mx_wtile_kernel(MxGemmArgs p, int tiles_m, int tiles_n) {
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
    const long long ka = 2ll * p.K, kb = ((long long)p.K + 1) / 2, ks = ((long long)p.K + 31) / 32;
    const bool rows16 = kb >= 16;

    uint4 va[CA], vb[CB];
    unsigned s[1];
    auto fetch = [&](long long k0) {
        auto load = [&](auto a_chunk, auto b_chunk) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < CA; ++u) {
                const int id = tid + u * NT, r = id >> 4, c = id & 15;
                va[u] = a_chunk(p.A + min(m0 + r, (long long)p.M - 1) * p.lda, 2 * k0 + 16 * c);
            }
#pragma unroll
            for (int u = 0; u < CB; ++u) {
                const int id = tid + u * NT, r = id >> 2, c = id & 3;
                vb[u] = b_chunk(p.B + min(n0 + r, (long long)p.N - 1) * p.ldb, k0 / 2 + 16 * c);
            }
        };
        typedef const unsigned char* Row;
        if (k0 + Cfg::BK > p.K && rows16)
            load([&](Row row, long long at) { return mx_load16(row, at, ka); },
                 [&](Row row, long long at) { return mx_load16(row, at, kb); });
        else
            load([&](Row row, long long at) { return mx_bytes16(row, at, ka); },
                 [&](Row row, long long at) { return mx_codes16(row, at, p.K); });
        mx_scales<4>(p.SB + min(n0 + (tid < BN ? tid : 0), (long long)p.N - 1) * p.ldsb, k0 / 32, ks, s);
    };

    mx_f4 acc[FM][FN] = {};
    fetch(0);
    for (long long k0 = 0; k0 < p.K; k0 += Cfg::BK) {
        if (k0 + Cfg::BK > p.K && rows16) {
#pragma unroll
            for (int u = 0; u < CA; ++u) va[u] = mx_end16(va[u], 2 * k0 + 16 * ((tid + u * NT) & 15), ka);
#pragma unroll
            for (int u = 0; u < CB; ++u) vb[u] = mx_end_codes16(vb[u], k0 / 2 + 16 * ((tid + u * NT) & 3), p.K);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < CA; ++u) {
            const int id = tid + u * NT, r = id >> 4, c = id & 15;
            lds_poison_f4(&as[r * 16 + (c ^ (r & 15))]);
            as[r * 16 + (c ^ (r & 15))] = va[u];
        }
#pragma unroll
        for (int u = 0; u < CB; ++u) {
            const int id = tid + u * NT, r = id >> 2, c = id & 3;
            lds_poison_f4(&bs[r * 4 + (c ^ ((r >> 1) & 3))]);
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
            store4<MxType::f32>(p, m0 + wm + 16 * i + li, n0 + wn + 16 * j + 4 * g, acc[i][j]);
}

// The same tiles where rows lie 16-byte aligned, from v_mfma_f32_32x32x16: A
// and B's codes come by DMA into one of two LDS stages of 128 k, the next
// requested right after the barrier that ends the reads of its place.  Lane
// half g = l / 32 has blocks 2g and 2g + 1 of a stage, eight elements (one
// register of codes, one chunk of A) in each of eight steps.  LDS: A's chunk c
// of row r at c ^ (r & 15), B's at c ^ (r / 4 & 3): the sixteen lanes that LDS
// serves at a time (0-3, 12-15, 20-23, 24-27, and so on) lie in distinct banks.
// Scales: 16 bytes (four stages) of 64 rows by one load, lane 32 t + r row r of
// tile t; one exchange of lane halves per stage brings each tile's four bytes
// to both halves.  Past K: chunks past a row's end are read from the row's last
// one, and what is past K is cleared in LDS in the last stage.
template <int BM_, int BN_, int WM_, int WN_>
struct WDma {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * (BN / WN), NT = NW * 64;
    static constexpr int FM = WM / 32, FN = WN / 32;
};

template <MxType T, bool SPLIT, int N>
__device__ __forceinline__ void mfma_row32(const uint4 (&b)[N], uint4 a, floatx16 (&acc)[N]) {
    auto bf = [](uint4 x) { return __builtin_bit_cast(bf8, x); };
    if constexpr (T == MxType::bf16) {
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf(a), bf(b[j]), acc[j], 0, 0, 0);
    } else if constexpr (SPLIT) {
        uint4 hi, lo;
        split2(a.x, hi.x, lo.x);
        split2(a.y, hi.y, lo.y);
        split2(a.z, hi.z, lo.z);
        split2(a.w, hi.w, lo.w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf(hi), bf(b[j]), acc[j], 0, 0, 0);
            acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf(lo), bf(b[j]), acc[j], 0, 0, 0);
        }
    } else {
        auto h8 = [](uint4 x) { return __builtin_bit_cast(half8, x); };
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(h8(a), h8(b[j]), acc[j], 0, 0, 0);
    }
}

template <class Cfg, MxType T>
__global__ __launch_bounds__(Cfg::NT, 2) void mx_wdma_kernel(MxGemmArgs p, int tiles_m, int tiles_n) {
    constexpr int BM = Cfg::BM, BN = Cfg::BN, NW = Cfg::NW, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int IA = BM * 16 / 64 / NW, IB = BN * 4 / 64 / NW;
    static_assert(IA * NW * 64 == BM * 16 && IB * NW * 64 == BN * 4 && FN % 2 == 0, "whole rounds");
    static_assert(NW % 4 == 0, "a wave's rows of A agree in bits 2 and 3");
    constexpr unsigned STAGE = BM * 256 + BN * 64;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * STAGE];
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, 8, p.xcds, tm, tn);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / Cfg::WAVES_N) * Cfg::WM, wn = (wave % Cfg::WAVES_N) * Cfg::WN;
    const int li = lane & 31, g = lane >> 5;
    const long long m0 = (long long)tm * BM, n0 = (long long)tn * BN;
    const int mlast = (int)min((long long)p.M - 1 - m0, (long long)BM - 1);
    const int nlast = (int)min((long long)p.N - 1 - n0, (long long)BN - 1);
    const unsigned char* const A = p.A + m0 * p.lda;
    const unsigned char* const B = p.B + n0 * p.ldb;
    const int blocks = (int)(((long long)p.K + 31) / 32);           // B's chunks and scales of a row
    const int achunks = (int)(((long long)p.K + 7) / 8);            // A's
    const int stages = (int)(((long long)p.K + 127) / 128);

    // A: instruction u of a wave covers rows 4 (wave + u NW) .. + 3, B: rows 16
    // (wave + u NW) .. + 15; the lane's chunk of its row.
    const int ca = (lane & 15) ^ ((4 * wave + (lane >> 4)) & 15);
    const int cb = (lane & 3) ^ (lane >> 4);
    unsigned va[IA], vb[IB];
#pragma unroll
    for (int u = 0; u < IA; ++u)
        va[u] = (unsigned)min((wave + u * NW) * 4 + (lane >> 4), mlast) * (unsigned)p.lda;
#pragma unroll
    for (int u = 0; u < IB; ++u)
        vb[u] = (unsigned)min((wave + u * NW) * 16 + (lane >> 2), nlast) * (unsigned)p.ldb;
    const unsigned lds0 = lds_addr(lds);
    auto request = [&](int s) {
        const unsigned ata = (unsigned)min(ca, achunks - 1 - 16 * s) * 16u;
        const unsigned atb = (unsigned)min(cb, blocks - 1 - 4 * s) * 16u;
        const unsigned to = lds0 + (s & 1) * STAGE + 1024u * wave;
        const unsigned char* const a = A + 256ll * s;
        const unsigned char* const b = B + 64ll * s;
#pragma unroll
        for (int u = 0; u < IA; ++u)
            lds_dma16s(a, va[u] + ata, __builtin_amdgcn_readfirstlane(to + u * NW * 1024u));
#pragma unroll
        for (int u = 0; u < IB; ++u)
            lds_dma16s(b, vb[u] + atb, __builtin_amdgcn_readfirstlane(to + BM * 256 + u * NW * 1024u));
    };
    const unsigned char* sb[FN / 2];
#pragma unroll
    for (int j = 0; j < FN / 2; ++j) sb[j] = p.SB + (n0 + min(wn + 64 * j + lane, nlast)) * p.ldsb;
    unsigned now[FN / 2][4], next[FN / 2][4];     // scales from this stage on, and of the next four
    floatx16 acc[FM][FN] = {};
    auto multiply = [&](int s) {
        const unsigned char* const st = lds + (s & 1) * STAGE;
        unsigned sc[FN];
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) {
            const auto x = __builtin_amdgcn_permlane32_swap(now[j][0], now[j][0], false, false);
            sc[2 * j] = x[0] >> (16 * g);
            sc[2 * j + 1] = x[1] >> (16 * g);
        }
        static_for<2>([&](auto half) {
            uint4 q[FN];
            bool ok = true, in_range = true;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int r = wn + 32 * j + li;
                q[j] = *reinterpret_cast<const uint4*>(st + BM * 256 + r * 64 + (((2 * g + half) ^ (r >> 2)) & 3) * 16);
                ok = ok && f16_holds(sc[j] >> (8 * half) & 255u);
            }
            if constexpr (T == MxType::f16) in_range = __all(ok);
            auto steps = [&](auto split) __attribute__((always_inline)) {
                static_for<4>([&](auto x) {
                    uint4 b[FN];
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        b[j] = decode8<T, split>(x == 0 ? q[j].x : x == 1 ? q[j].y : x == 2 ? q[j].z : q[j].w,
                                                 mx_scale(sc[j] >> (8 * half) & 255u));
#pragma unroll
                    for (int i = 0; i < FM; ++i) {
                        const int r = wm + 32 * i + li, c = 8 * g + 4 * half + x;
                        mfma_row32<T, split, FN>(b, *reinterpret_cast<const uint4*>(st + r * 256 + ((c ^ r) & 15) * 16),
                                                 acc[i]);
                    }
                });
            };
            if (in_range)
                steps(std::false_type{});
            else
                steps(std::true_type{});
        });
    };
    auto arrived = [&] {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    auto load_scales = [&](int s, unsigned (&to)[FN / 2][4]) {
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) scales16(sb[j], 4 * s, blocks, to[j]);
    };
    auto clear_past = [&](int s) {
        if ((p.K & 127) == 0) return;
        unsigned char* const st = lds + (s & 1) * STAGE;
        for (int id = tid; id < BM * 16; id += Cfg::NT) {
            const int left = (int)(p.K - 128ll * s) - 8 * (((id & 15) ^ (id >> 4)) & 15);
            uint4* const v = reinterpret_cast<uint4*>(st + 16 * id);
            if (left < 8) {
                const uint4 k = *v;
                auto word = [&](unsigned w, int i) {
                    const int n = left - 2 * i;
                    return n >= 2 ? w : n == 1 ? w & 0xFFFFu : 0u;
                };
                *v = make_uint4(word(k.x, 0), word(k.y, 1), word(k.z, 2), word(k.w, 3));
            }
        }
        for (int id = tid; id < BN * 4; id += Cfg::NT) {
            const int left = (int)(p.K - 128ll * s) - 32 * (((id & 3) ^ (id >> 4)) & 3);
            uint4* const v = reinterpret_cast<uint4*>(st + BM * 256 + 16 * id);
            if (left < 32) *v = mx_keep(*v, left);
        }
        __syncthreads();
    };
    if (blocks >= 16) {
        load_scales(0, now);
    } else {
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) scales_few(sb[j], blocks, now[j]);
    }
    request(0);
    for (int s = 0; s < stages; ++s) {
        arrived();
        if ((s & 3) == 0) {
            if (s > 0) {
#pragma unroll
                for (int j = 0; j < FN / 2; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) now[j][i] = next[j][i];
                }
            }
            if (const int past = 4 * s + 16 - blocks; past > 0 && blocks >= 16) {
#pragma unroll
                for (int j = 0; j < FN / 2; ++j) down16(now[j], past);
            }
            if (s + 4 < stages) load_scales(s + 4, next);
        }
        if (s + 1 < stages)
            request(s + 1);
        else
            clear_past(s);
        multiply(s);
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) {
            now[j][0] = now[j][1];
            now[j][1] = now[j][2];
            now[j][2] = now[j][3];
        }
    }
    mx_store_wave<MxType::f32>(p, acc, m0 + wm, n0 + wn, li, g);
}

template <class Cfg, MxType T>
hipError_t launch_wtile(const MxGemmArgs& a, hipStream_t s) {
    const long long tm = ((long long)a.M + Cfg::BM - 1) / Cfg::BM, tn = ((long long)a.N + Cfg::BN - 1) / Cfg::BN;
    if (tm * tn * Cfg::NT > 0xFFFFFFFFll) return hipErrorInvalidValue;
    const bool dma = mx_aligned(a.A, a.lda, 16) && mx_aligned(a.B, a.ldb, 16) && a.K > 0 &&
                     mx_dma_reach(a.lda, Cfg::BM) && mx_dma_reach(a.ldb, Cfg::BN);
    if (dma)
        mx_wdma_kernel<WDma<Cfg::BM, Cfg::BN, Cfg::WM, Cfg::WN>, T>
            <<<(unsigned)(tm * tn), Cfg::NT, 0, s>>>(a, (int)tm, (int)tn);
    else
        mx_wtile_kernel<Cfg, T><<<(unsigned)(tm * tn), Cfg::NT, 0, s>>>(a, (int)tm, (int)tn);
    return hipGetLastError();
}

template <MxType T>
hipError_t launch_w(const MxGemmArgs& a, hipStream_t s) {
    if (mx_few_rows(a)) return launch_mx_rows(a, T, MxType::f32, s);
    return launch_wtile<WTile<128, 128, 64, 64>, T>(a, s);
}

}  // namespace

hipError_t launch_mx_wgemm(const MxGemmArgs& a, MxType t, hipStream_t s) {
    return t == MxType::bf16 ? launch_w<MxType::bf16>(a, s) : launch_w<MxType::f16>(a, s);
}

}  // namespace sgemm
