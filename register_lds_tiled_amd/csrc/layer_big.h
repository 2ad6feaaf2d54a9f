// layer_big.h -- large wave tiles of the feed-forward layer's products, fed by
// direct-to-LDS DMA.
//
// A workgroup of four waves, one per SIMD, owns BM x BN products; each wave holds
// BM/2 x BN/2 of them as accumulator blocks of 32 x 32 in accumulation registers
// (256 x 256 tiles: 4 x 4 blocks, all 256 of them).  Stages of 64 bytes of k go
// round four LDS buffers: stage t + 3 is requested while stage t multiplies,
// into the buffer that stage t - 1 left; one barrier a stage, in its second
// step.  A step's operands are read during the step before, one read or so
// between two matrix instructions.  Every address in the loop is a lane's fixed
// register and an immediate (the DMA's a scalar base and a fixed lane offset), so
// the loop holds no vector ALU instruction, which at one wave per SIMD would
// stall the matrix pipe.
//
// K that is no whole number of stages: the first stage begins below k = 0, where
// its lanes copy zeros.  The rows past M (N) of the last tiles are the last row
// again, the columns past the matrix the tile's first ones: what they give is
// not stored.
#pragma once

#include "layer_tile.h"

namespace sgemm {
// Whether the kernel below takes a product: rows of whole 16 bytes, lane offsets
// of 32 bits, and for the sum of two products whole stages and one pitch for both.
template <class T>
inline bool big_fits(const LayerArgs& a) {
    const int nb = T::GATED || T::PAIRS == 2 ? 2 : 1, na = T::OUTS == 2 || T::PAIRS == 2 ? 2 : 1;
    for (int i = 0; i < na; ++i)
        if (!mx_aligned(a.A[i], a.lda[i], 16) || !mx_dma_reach(a.lda[i], 512)) return false;
    for (int i = 0; i < nb; ++i)
        if (!mx_aligned(a.B[i], a.ldb[i], 16) || !mx_dma_reach(a.ldb[i], 512)) return false;
    if (!T::A_ACROSS && (long long)a.K * T::ES % 16 != 0) return false;
    if (T::PAIRS == 2 && (a.K % T::KST != 0 || a.lda[0] != a.lda[1] || a.ldb[0] != a.ldb[1])) return false;
    return a.K >= T::KST;   // a stage at least: the first one alone may begin below k = 0
}

#ifdef __HIPCC__
namespace layer {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
static __device__ const uint4 kZero16 = {0u, 0u, 0u, 0u};

// The matrix instruction in place on accumulation registers.  The compiler knows
// nothing of its wait states: two after a vector instruction writes an operand,
// 19 before its result is read; the kernel keeps them itself.
template <Elem E>
__device__ __forceinline__ void mfma_in(floatx16& acc, u32x4 a, u32x4 b) {
    if constexpr (E == Elem::bf16)
        asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else if constexpr (E == Elem::f16)
        asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else   // whole numbers in the registers of a float vector
        asm volatile("v_mfma_i32_32x32x32_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

constexpr int kBuffers = 4;

template <class T>
struct Big {
    static constexpr int STAGE = T::SA + T::SB;
    static constexpr int AQ = T::SA / 1024 / T::NW, BQ = T::SB / 1024 / T::NW, NDMA = AQ + BQ;   // DMA per wave and stage
    static constexpr int NMF = T::FM * T::FN;                                                   // per step
    static constexpr int RA = T::A_ACROSS ? 2 : 1, RB = T::B_ACROSS ? 2 : 1;                     // reads per block
    static constexpr int NRD = RA * T::FM + RB * T::FN;
    // A step's reads begin behind this many matrix instructions: in the first
    // step behind the DMA, in the second behind the barrier.
    static constexpr int FIRST = NMF >= 16 ? 4 : 1, PRE = NMF >= 16 ? 2 : 1;
    static constexpr int slot(int j, int n, int first) { return first + j * (NMF - first) / n; }
    static constexpr int MAXW = kBuffers * STAGE > 80 * 1024 ? 1 : 2;   // waves per SIMD that LDS allows
    static_assert(AQ * T::NW * 1024 == T::SA && BQ * T::NW * 1024 == T::SB, "whole DMA instructions");
    static_assert((kBuffers - 2) * NDMA <= 16, "vmcnt range of wait_vmcnt");
    static_assert(kBuffers * STAGE <= 160 * 1024 && T::EPI <= kBuffers * STAGE, "LDS");
    static_assert(T::NW == 4 && PRE + 1 < NMF, "one wave per SIMD, slots for the reads");
};

template <class T>
__global__ __launch_bounds__(256, 1) __attribute__((amdgpu_waves_per_eu(1, Big<T>::MAXW)))
void big_kernel(LayerArgs p, int tiles_m, int tiles_n) {
    using B = Big<T>;
    constexpr int BM = T::BM, BN = T::BN, FM = T::FM, FN = T::FN, KST = T::KST, ES = T::ES, NB = kBuffers;
    constexpr int AQ = B::AQ, BQ = B::BQ, NDMA = B::NDMA, NRD = B::NRD, STAGE = B::STAGE;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[NB * STAGE];
    const int per = tiles_m * tiles_n;
    const int out = T::OUTS == 2 && (int)blockIdx.x >= per ? 1 : 0;
    int tm, tn;
    tile_coords(blockIdx.x - out * per, tiles_m, tiles_n, T::GROUP_M, p.xcds, tm, tn);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave / T::WAVES_N) * T::WM, wn = (wave % T::WAVES_N) * T::WN;
    const int li = lane & 31, g = lane >> 5;
    const long long m0 = (long long)tm * BM, n0 = (long long)tn * T::COLS;
    const int mlast = (int)min((long long)p.M - 1 - m0, (long long)BM - 1);
    const int nlast = (int)min((long long)p.N - 1 - n0, (long long)T::COLS - 1);
    const unsigned lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));

    // Stages: `each` of a pair of matrices, the first `pad` k below zero.
    const int each = (int)(((long long)p.K + KST - 1) / KST), nst = each * T::PAIRS;
    const int pad = (int)((long long)each * KST - p.K);

    // DMA: instruction v of an operand's stage fills its bytes 1024 v + 16 lane.
    // Along k: row 16 v + lane / 4, place lane % 4.  Across: W / 8 places to a k
    // row.  Lane offsets from the stage's first byte in the matrix; kk is the
    // lane's first k in the stage.
    auto along = [&](int v, int row, long long ld, int& kk) __attribute__((always_inline)) {
        const int c = (lane & 3) ^ chunk_at(16 * v + (lane >> 2));
        kk = 16 / ES * c;
        return (unsigned)row * (unsigned)ld + 16u * (unsigned)c;
    };
    auto across = [&](int v, int W, int last, long long ld, int& kk) __attribute__((always_inline)) {
        const int k = v * (512 / W) + lane / (W / 8), c = lane % (W / 8) ^ 4 * (k & 3);
        kk = k;
        return (unsigned)k * (unsigned)ld + (8 * c <= last ? 16u * (unsigned)c : 0u);
    };
    unsigned aoff[AQ], boff[BQ];
    int akk[AQ], bkk[BQ];
    const int pa = T::OUTS == 2 ? out : 0;
    const unsigned char* abase = T::A_ACROSS ? p.A[pa] + 2 * m0 : p.A[pa] + m0 * p.lda[pa];
    const unsigned char* bbase[BQ];
#pragma unroll
    for (int u = 0; u < AQ; ++u) {
        const int v = wave + 4 * u;
        if constexpr (T::A_ACROSS)
            aoff[u] = across(v, BM, mlast, p.lda[pa], akk[u]);
        else
            aoff[u] = along(v, min(16 * v + (lane >> 2), mlast), p.lda[pa], akk[u]);
    }
#pragma unroll
    for (int u = 0; u < BQ; ++u) {
        const int v = wave + 4 * u;
        if constexpr (T::B_ACROSS) {
            bbase[u] = p.B[0] + 2 * n0;
            boff[u] = across(v, BN, nlast, p.ldb[0], bkk[u]);
        } else if constexpr (T::GATED) {
            int m, row;
            gated_row<T>(16 * v, m, row);              // 16 rows of one matrix
            const long long ld = m ? p.ldb[1] : p.ldb[0];
            bbase[u] = (m ? p.B[1] : p.B[0]) + n0 * ld;
            boff[u] = along(v, min(row + (lane >> 2), nlast), ld, bkk[u]);
        } else {
            bbase[u] = p.B[0] + n0 * p.ldb[0];
            boff[u] = along(v, min(16 * v + (lane >> 2), nlast), p.ldb[0], bkk[u]);
        }
    }
    // How far stage s lies from the first of its matrix.
    auto a_step = [&](int s) __attribute__((always_inline)) {
        const long long k = (long long)s * KST - pad;
        return T::A_ACROSS ? k * p.lda[pa] : k * ES;
    };
    auto b_step = [&](int s) __attribute__((always_inline)) {
        const long long k = (long long)s * KST - pad;
        return T::B_ACROSS ? k * p.ldb[0] : k * ES;
    };
    const long long a_pair = T::PAIRS == 2 ? p.A[1] - p.A[0] : 0, b_pair = T::PAIRS == 2 ? p.B[1] - p.B[0] : 0;
    long long sa, sb;                                  // of the stage being requested
    auto at_stage = [&](int s) __attribute__((always_inline)) {
        const bool second = T::PAIRS == 2 && s >= each;
        sa = a_step(second ? s - each : s) + (second ? a_pair : 0);
        sb = b_step(second ? s - each : s) + (second ? b_pair : 0);
    };
    auto to_of = [&](int d, int buf) __attribute__((always_inline)) {
        return lds0 + (unsigned)(buf * STAGE + (d < AQ ? 1024 * (wave + 4 * d) : T::SA + 1024 * (wave + 4 * (d - AQ))));
    };
    auto request = [&](int d, int buf) __attribute__((always_inline)) {
        if (d < AQ)
            lds_dma16s(abase + sa, aoff[d], to_of(d, buf));
        else
            lds_dma16s(bbase[d - AQ] + sb, boff[d - AQ], to_of(d, buf));
    };
    auto barrier = [&](int inflight) __attribute__((always_inline)) {
        asm volatile("" ::: "memory");
        wait_vmcnt(inflight);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    floatx16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
    asm volatile("s_nop 7");

    // Operand addresses: along k one for each buffer and step, blocks 2048 bytes
    // apart; across one for each buffer and block, steps 16 rows of W apart and a
    // read's halves 8.
    constexpr int NA = T::A_ACROSS ? FM : 2, NBB = T::B_ACROSS ? FN : 2;
    unsigned at_a[NB][NA], at_b[NB][NBB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const unsigned buf = lds0 + (unsigned)(b * STAGE);
#pragma unroll
        for (int x = 0; x < NA; ++x)
            at_a[b][x] = buf + (unsigned)(T::A_ACROSS ? across_at<BM>(wm, x, 0, lane) : along_at(wm, 0, x, li, g));
#pragma unroll
        for (int x = 0; x < NBB; ++x)
            at_b[b][x] = buf + T::SA + (unsigned)(T::B_ACROSS ? across_at<BN>(wn, x, 0, lane) : along_at(wn, 0, x, li, g));
    }
    u32x4 Av[2][FM], Bv[2][FN];
    shortx4 Ah[2][FM][2], Bh[2][FN][2];
    auto half = [](unsigned at) __attribute__((always_inline)) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4*)(size_t)at);
    };
    auto whole = [](unsigned at) __attribute__((always_inline)) {
        return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((size_t)at);
    };
    // Read r of step t of buffer b into parity x: A's first block, all of B's,
    // the rest of A's, as the matrix instructions want them.
    auto read_op = [&](auto b_c, auto t_c, int r) __attribute__((always_inline)) {
        constexpr int b = b_c, t = t_c, x = t_c;
        auto rd_a = [&](int i, int h) {
            if constexpr (T::A_ACROSS)
                Ah[x][i][h] = half(at_a[b][i] + (unsigned)((8 * t + 4 * h) * BM * 2));
            else
                Av[x][i] = whole(at_a[b][t] + 2048u * (unsigned)i);
        };
        auto rd_b = [&](int j, int h) {
            if constexpr (T::B_ACROSS)
                Bh[x][j][h] = half(at_b[b][j] + (unsigned)((8 * t + 4 * h) * BN * 2));
            else
                Bv[x][j] = whole(at_b[b][t] + 2048u * (unsigned)j);
        };
        if (r < B::RA)
            rd_a(0, r);
        else if (r < B::RA + B::RB * FN)
            rd_b((r - B::RA) / B::RB, (r - B::RA) % B::RB);
        else
            rd_a((r - B::RB * FN) / B::RA, (r - B::RB * FN) % B::RA);
    };
    auto joined = [](const shortx4 (&h)[2]) __attribute__((always_inline)) {
        const uint2 lo = __builtin_bit_cast(uint2, h[0]), hi = __builtin_bit_cast(uint2, h[1]);
        return u32x4{lo.x, lo.y, hi.x, hi.y};
    };
    auto step = [&](auto x_c, auto&& op) __attribute__((always_inline)) {
        constexpr int x = x_c;
        if constexpr (T::B_ACROSS) static_for<FN>([&](auto j) { Bv[x][j] = joined(Bh[x][j]); });
        static_for<FM>([&](auto i) __attribute__((always_inline)) {
            if constexpr (T::A_ACROSS) Av[x][i] = joined(Ah[x][i]);
            static_for<FN>([&](auto j) __attribute__((always_inline)) {
                op(FN * i + j);
                mfma_in<T::E>(acc[i][j], Av[x][i], Bv[x][j]);
                __builtin_amdgcn_sched_barrier(0);
            });
        });
    };
    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, 1> one{};
    auto stage = [&](auto h_c, int s) __attribute__((always_inline)) {
        constexpr int h = h_c;
        constexpr std::integral_constant<int, (h + 1) % NB> next{};
        at_stage(min(s + NB - 1, nst - 1));   // past the last: it again, where nobody reads
        step(zero, [&](int n) __attribute__((always_inline)) {
#pragma unroll
            for (int d = 0; d < NDMA; ++d)
                if (B::slot(d, NDMA, 0) == n) request(d, (h + NB - 1) % NB);
#pragma unroll
            for (int r = 0; r < NRD; ++r)
                if (B::slot(r, NRD, B::FIRST) == n) read_op(h_c, one, r);
        });
        step(one, [&](int n) __attribute__((always_inline)) {
            if (n == B::PRE) barrier((NB - 2) * NDMA);
#pragma unroll
            for (int r = 0; r < NRD; ++r)
                if (B::slot(r, NRD, B::PRE + 1) == n) read_op(next, zero, r);
        });
    };

    // The first stage, its lanes below k = 0 from zeros.
    at_stage(0);
#pragma unroll
    for (int d = 0; d < NDMA; ++d) {
        const unsigned char* const from = d < AQ ? abase + sa + aoff[d] : bbase[d - AQ] + sb + boff[d - AQ];
        const int kk = d < AQ ? akk[d] : bkk[d - AQ];
        lds_dma16(kk >= pad ? from : reinterpret_cast<const unsigned char*>(&kZero16),
                  __builtin_amdgcn_readfirstlane(to_of(d, 0)));
    }
#pragma unroll
    for (int s = 1; s < NB - 1; ++s) {
        at_stage(min(s, nst - 1));
#pragma unroll
        for (int d = 0; d < NDMA; ++d) request(d, s);
    }
    barrier((NB - 2) * NDMA);
    static_for<NRD>([&](auto r) { read_op(zero, zero, r); });
    int s = 0;
    for (;;) {
        stage(std::integral_constant<int, 0>{}, s);
        if (++s == nst) break;
        stage(std::integral_constant<int, 1>{}, s);
        if (++s == nst) break;
        stage(std::integral_constant<int, 2>{}, s);
        if (++s == nst) break;
        stage(std::integral_constant<int, 3>{}, s);
        if (++s == nst) break;
    }
    // 24 wait states before the results are read; what was requested again past
    // the last stage lands before LDS is used for the results.
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7");
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
    barrier(0);
    epilogue<T>(p, out, acc, reinterpret_cast<float*>(lds) + wave * 32 * T::STR, m0 + wm,
                n0 + (T::GATED ? wn / 2 : wn), lane);
}

// The large tiles where they fit, through registers where not.  WIDE: 256 x 256.
template <Form F, Elem E, Elem OUT>
hipError_t launch_form(const LayerArgs& a, hipStream_t s) {
    using Small = Tile<F, E, OUT, 128, 128, 64, 64>;
    using Wide = Tile<F, E, OUT, 256, 256, 128, 128, 4>;
    if (!big_fits<Small>(a)) return launch_tiles<Small>(tile_kernel<Small>, a, s);
    const long long small = ((long long)a.M + 127) / 128 * (((long long)a.N + Small::COLS - 1) / Small::COLS) * Small::OUTS;
    if (small <= 2ll * a.cus) return launch_tiles<Small>(big_kernel<Small>, a, s);
    return launch_tiles<Wide>(big_kernel<Wide>, a, s);
}

}  // namespace layer
#endif
}  // namespace sgemm
