// layer_big.h -- large wave tiles of the feed-forward layer's products, fed by
// direct-to-LDS DMA.
//
// A workgroup of four waves, one per SIMD, owns BM x BN products; each wave holds
// BM/2 x BN/2 of them as accumulator blocks of 32 x 32 in accumulation registers
// (256 x 256 tiles: 4 x 4 blocks, all 256 of them).
//
// A stage is 128 bytes of k, four steps of matrix instructions, so that a DMA
// reads whole cache lines of rows that run along k: 64-byte pieces come at 22
// TB/s from the L2s of all XCDs, 128-byte pieces at 33, and the multiplication
// wants 18 (8192^3 int8 425 to 433 us, 2.6 POP/s; with stages of 64 bytes it took
// 560, 495 of zeros that cost no power; gated bf16 4096 x 8192 x 8192 780, 1.41
// PFLOP/s).  LDS holds five units, each one operand of a stage: while stage
// t multiplies, B of stage t + 1 and then A of stage t + 2 are requested into the
// units that stage t - 1 left, and the one barrier of a stage, in its last step,
// waits for all but the latter.  A step's operands are read during the step
// before, one read or so between two matrix instructions.  Every address in the
// loop is a lane's fixed register and an immediate (the DMA's a scalar base and a
// fixed lane offset), so the loop holds no vector ALU instruction, which at one
// wave per SIMD would stall the matrix pipe.
//
// Rows along k lie as eight chunks of 16 bytes, chunk c of row r at c ^
// line_at(r); step h gives lane half g the chunk 4g + h.  (In the sets of lanes
// that LDS serves together, see layer_tile.h, the rows of one parity share half
// of the banks, and their line_at differ.)  Rows across k lie as in layer_tile.h,
// 64 of them, lane half g's from 32 g on.
//
// K that is no whole number of stages: what is left of it is the first stage, the
// others follow from k = 0 on.  Lanes of that stage past K copy zeros, and where K
// ends within 16 bytes of rows along k, the elements behind it (of the pitch, or
// of the 16 bytes that the matrix's last row ends in) are cleared in LDS before
// they are read.  (That stage alone is laid and read outside the loop.)  The rows
// past M (N) of the last tiles are the last row again, the columns past the matrix
// the tile's first ones: what they give is not stored.
#pragma once

#include "layer_tile.h"

namespace sgemm {
// Whether the kernel below takes a product: rows that begin on 16 bytes, lane
// offsets of 32 bits, and for the sum of two products whole stages and one pitch
// for both.
template <class T>
inline bool big_fits(const LayerArgs& a) {
    const int nb = T::GATED || T::PAIRS == 2 ? 2 : 1, na = T::OUTS == 2 || T::PAIRS == 2 ? 2 : 1;
    for (int i = 0; i < na; ++i)
        if (!mx_aligned(a.A[i], a.lda[i], 16) || !mx_dma_reach(a.lda[i], 512)) return false;
    for (int i = 0; i < nb; ++i)
        if (!mx_aligned(a.B[i], a.ldb[i], 16) || !mx_dma_reach(a.ldb[i], 512)) return false;
    if (T::PAIRS == 2 && (a.K % (2 * T::KST) != 0 || a.lda[0] != a.lda[1] || a.ldb[0] != a.ldb[1])) return false;
    return a.K >= 2 * T::KST;   // a stage at least: the last one requested has to be whole
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

__device__ __forceinline__ int line_at(int r) { return r >> 1 & 7; }

// Which stage of a matrix is taken as number s: what is left of K first (the sum
// of two products has whole stages only).
template <int PAIRS>
__device__ __forceinline__ int stage_k(int s, int each, bool far) {
    if constexpr (PAIRS == 2) return far ? s - each : s;
    return s == 0 ? each - 1 : s - 1;
}
// Zeros behind the first n bytes of row r of a stage, up to the next 16.
__device__ __forceinline__ void clear_behind(unsigned char* stage, int r, int n) {
    unsigned* const w = reinterpret_cast<unsigned*>(stage + r * 128 + 16 * ((n >> 4) ^ line_at(r)));
    const int last = n >> 2 & 3;   // the word that n ends in
    w[last] = n & 3 ? w[last] & ((1u << 8 * (n & 3)) - 1u) : 0u;
    for (int i = last + 1; i < 4; ++i) w[i] = 0u;
}

constexpr int kUnits = 5;

template <class T>
struct Big {
    static_assert(T::BM == T::BN, "units of one size");
    static constexpr int KST = 2 * T::KST;                                  // k of a stage
    static constexpr int UNIT = 2 * T::SA;                                  // bytes
    static constexpr int NQ = UNIT / 1024 / T::NW;                          // DMA per wave and unit
    static constexpr int NMF = T::FM * T::FN;                               // matrix instructions a step
    static constexpr int RA = T::A_ACROSS ? 2 : 1, RB = T::B_ACROSS ? 2 : 1;   // reads per block
    static constexpr int NRD = RA * T::FM + RB * T::FN;
    // A step's reads begin behind this many matrix instructions, in the last step
    // behind the barrier, which stands before instruction PRE.
    static constexpr int FIRST = NMF >= 16 ? 4 : 1, PRE = NMF >= 16 ? 2 : 1;
    static constexpr int slot(int j, int n, int first) { return first + j * (NMF - first) / n; }
    static constexpr int MAXW = kUnits * UNIT > 80 * 1024 ? 1 : 2;          // waves per SIMD that LDS allows
    static_assert(NQ * T::NW * 1024 == UNIT && NQ <= 16, "whole DMA instructions, vmcnt range of wait_vmcnt");
    static_assert(kUnits * UNIT <= 160 * 1024 && T::EPI <= kUnits * UNIT, "LDS");
    static_assert(T::NW == 4 && PRE + 1 < NMF, "one wave per SIMD, slots for the reads");
};

template <class T>
__global__ __launch_bounds__(256, 1) __attribute__((amdgpu_waves_per_eu(1, Big<T>::MAXW)))
void big_kernel(LayerArgs p, int tiles_m, int tiles_n) {
    using B = Big<T>;
    constexpr int W = T::BM, FM = T::FM, FN = T::FN, KST = B::KST, ES = T::ES;
    constexpr int NQ = B::NQ, NRD = B::NRD, UNIT = B::UNIT;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[kUnits * UNIT];
    const int per = tiles_m * tiles_n;
    const int out = T::OUTS == 2 && (int)blockIdx.x >= per ? 1 : 0;
    int tm, tn;
    tile_coords(blockIdx.x - out * per, tiles_m, tiles_n, T::GROUP_M, p.xcds, tm, tn);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave / T::WAVES_N) * T::WM, wn = (wave % T::WAVES_N) * T::WN;
    const int li = lane & 31, g = lane >> 5;
    const long long m0 = (long long)tm * W, n0 = (long long)tn * T::COLS;
    const int mlast = (int)min((long long)p.M - 1 - m0, (long long)W - 1);
    const int nlast = (int)min((long long)p.N - 1 - n0, (long long)T::COLS - 1);
    const unsigned lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));

    // Stages: `each` of a pair of matrices, the first with `left` of k.
    const int each = (int)(((long long)p.K + KST - 1) / KST), nst = each * T::PAIRS;
    const int left = (int)(p.K - (each - 1ll) * KST);

    // DMA: instruction v of a unit fills its bytes 1024 v + 16 lane.  Along k: row
    // 8 v + lane / 8, place lane % 8.  Across: W / 8 places to a k row.  Lane
    // offsets from the stage's first byte in the matrix; kk is the lane's first k
    // in the stage.
    auto along = [&](int v, int row, long long ld, int& kk) __attribute__((always_inline)) {
        const int c = (lane & 7) ^ line_at(8 * v + (lane >> 3));
        kk = 16 / ES * c;
        return (unsigned)row * (unsigned)ld + 16u * (unsigned)c;
    };
    auto across = [&](int v, int last, long long ld, int& kk) __attribute__((always_inline)) {
        const int k = v * (512 / W) + lane / (W / 8), c = lane % (W / 8) ^ across_swap<W>(k);
        kk = k;
        return (unsigned)k * (unsigned)ld + (8 * c <= last ? 16u * (unsigned)c : 0u);
    };
    // The gated form: the rows of instruction u are the second matrix's.
    auto second = [](int u) { return T::GATED ? 32 * u / (T::WN / 2) & 1 : 0; };
    unsigned aoff[NQ], boff[NQ];
    int akk[NQ], bkk[NQ];
    const int pa = T::OUTS == 2 ? out : 0;
    const unsigned char* const abase = T::A_ACROSS ? p.A[pa] + 2 * m0 : p.A[pa] + m0 * p.lda[pa];
    const unsigned char* const bbase[2] = {T::B_ACROSS ? p.B[0] + 2 * n0 : p.B[0] + n0 * p.ldb[0],
                                           T::GATED ? p.B[1] + n0 * p.ldb[1] : nullptr};
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
        const int v = wave + 4 * u;
        if constexpr (T::A_ACROSS)
            aoff[u] = across(v, mlast, p.lda[pa], akk[u]);
        else
            aoff[u] = along(v, min(8 * v + (lane >> 3), mlast), p.lda[pa], akk[u]);
        if constexpr (T::B_ACROSS) {
            boff[u] = across(v, nlast, p.ldb[0], bkk[u]);
        } else {
            int m = 0, row = 8 * v;
            if constexpr (T::GATED) gated_row<T>(8 * v, m, row);   // 8 rows of one matrix
            boff[u] = along(v, min(row + (lane >> 3), nlast), p.ldb[second(u)], bkk[u]);
        }
    }
    // How far stage s of an operand lies from the first of its (first) matrix.
    const long long a_pair = T::PAIRS == 2 ? p.A[1] - p.A[0] : 0, b_pair = T::PAIRS == 2 ? p.B[1] - p.B[0] : 0;
    auto a_step = [&](int s) __attribute__((always_inline)) {
        const bool far = T::PAIRS == 2 && s >= each;
        const long long k = stage_k<T::PAIRS>(s, each, far) * (long long)KST;
        return (T::A_ACROSS ? k * p.lda[pa] : k * ES) + (far ? a_pair : 0);
    };
    auto b_step = [&](int s) __attribute__((always_inline)) {
        const bool far = T::PAIRS == 2 && s >= each;
        const long long k = stage_k<T::PAIRS>(s, each, far) * (long long)KST;
        return (T::B_ACROSS ? k * p.ldb[0] : k * ES) + (far ? b_pair : 0);
    };
    auto to_of = [&](int unit, int u) __attribute__((always_inline)) {
        return lds0 + (unsigned)(unit * UNIT + 1024 * (wave + 4 * u));
    };
    auto request_a = [&](int u, int unit, long long step) __attribute__((always_inline)) {
        lds_dma16s(abase + step, aoff[u], to_of(unit, u));
    };
    auto request_b = [&](int u, int unit, long long step) __attribute__((always_inline)) {
        lds_dma16s(bbase[second(u)] + step, boff[u], to_of(unit, u));
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

    // Operand addresses in a pair of units (an immediate reaches no further).
    // Along k one for each step, blocks 4096 bytes apart; across one for each
    // block, steps 8 rows apart and a read's halves 4.
    constexpr int NA = T::A_ACROSS ? FM : 4, NB = T::B_ACROSS ? FN : 4, PAIRED = (kUnits + 1) / 2;
    unsigned at_a[PAIRED][NA], at_b[PAIRED][NB];
#pragma unroll
    for (int b = 0; b < PAIRED; ++b) {
        const unsigned unit = lds0 + (unsigned)(2 * b * UNIT);
        auto line = [&](int w, int h) { return (unsigned)((w + li) * 128 + 16 * ((4 * g + h) ^ line_at(li))); };
#pragma unroll
        for (int x = 0; x < NA; ++x) at_a[b][x] = unit + (T::A_ACROSS ? (unsigned)across_at<W, 32>(wm, x, 0, lane) : line(wm, x));
#pragma unroll
        for (int x = 0; x < NB; ++x) at_b[b][x] = unit + (T::B_ACROSS ? (unsigned)across_at<W, 32>(wn, x, 0, lane) : line(wn, x));
    }
    u32x4 Av[2][FM], Bv[2][FN];
    shortx4 Ah[2][FM][2], Bh[2][FN][2];
    auto half = [](unsigned at) __attribute__((always_inline)) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4*)(size_t)at);
    };
    auto whole = [](unsigned at) __attribute__((always_inline)) {
        return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((size_t)at);
    };
    // Read r of step h of the stage whose A lies in unit a: A's first block, all of
    // B's, the rest of A's, as the matrix instructions want them.
    auto read_op = [&](auto a_c, auto h_c, int r) __attribute__((always_inline)) {
        constexpr int a = a_c, b = (a + 1) % kUnits, h = h_c, x = h % 2;
        constexpr unsigned sa = (unsigned)(a % 2 * UNIT), sb = (unsigned)(b % 2 * UNIT);
        constexpr unsigned deep = (unsigned)(8 * h * W * 2);
        auto rd_a = [&](int i, int q) {
            if constexpr (T::A_ACROSS)
                Ah[x][i][q] = half(at_a[a / 2][i] + sa + deep + (unsigned)(4 * q * W * 2));
            else
                Av[x][i] = whole(at_a[a / 2][h] + sa + 4096u * (unsigned)i);
        };
        auto rd_b = [&](int j, int q) {
            if constexpr (T::B_ACROSS)
                Bh[x][j][q] = half(at_b[b / 2][j] + sb + deep + (unsigned)(4 * q * W * 2));
            else
                Bv[x][j] = whole(at_b[b / 2][h] + sb + 4096u * (unsigned)j);
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
    auto step = [&](auto h_c, auto&& op) __attribute__((always_inline)) {
        constexpr int x = h_c % 2;
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
    constexpr std::integral_constant<int, 0> first{};
    // Stage s, whose A lies in unit 2 t % 5 and B in the next one.
    auto stage = [&](auto t_c, int s) __attribute__((always_inline)) {
        constexpr int a = 2 * t_c % kUnits;
        constexpr std::integral_constant<int, a> here{};
        constexpr std::integral_constant<int, (a + 2) % kUnits> next{};
        // past the last stage: that again, where nobody reads it
        const long long sb = b_step(min(s + 1, nst - 1)), sa = a_step(min(s + 2, nst - 1));
        static_for<4>([&](auto h) __attribute__((always_inline)) {
            step(h, [&](int n) __attribute__((always_inline)) {
                if constexpr (h < 2) {
#pragma unroll
                    for (int u = 0; u < NQ; ++u)
                        if (B::slot(u, NQ, 0) == n) {
                            if constexpr (h == 0) request_b(u, (a + 3) % kUnits, sb);
                            if constexpr (h == 1) request_a(u, (a + 4) % kUnits, sa);
                        }
                }
                if constexpr (h == 3)
                    if (n == B::PRE) barrier(NQ);
#pragma unroll
                for (int r = 0; r < NRD; ++r)
                    if (B::slot(r, NRD, h == 3 ? B::PRE + 1 : B::FIRST) == n) {
                        if constexpr (h == 3)
                            read_op(next, first, r);
                        else
                            read_op(here, std::integral_constant<int, (h + 1) % 4>{}, r);
                    }
            });
        });
    };

    // The first stage, its lanes past K from zeros, and A of the second.
    {
        const unsigned char* const zero = reinterpret_cast<const unsigned char*>(&kZero16);
        const long long sa = a_step(0), sb = b_step(0), next = a_step(min(1, nst - 1));
#pragma unroll
        for (int u = 0; u < NQ; ++u)
            lds_dma16(akk[u] < left ? abase + sa + aoff[u] : zero, __builtin_amdgcn_readfirstlane(to_of(0, u)));
#pragma unroll
        for (int u = 0; u < NQ; ++u)
            lds_dma16(bkk[u] < left ? bbase[second(u)] + sb + boff[u] : zero, __builtin_amdgcn_readfirstlane(to_of(1, u)));
#pragma unroll
        for (int u = 0; u < NQ; ++u) request_a(u, 2, next);
    }
    barrier(NQ);
    if constexpr (!T::A_ACROSS && !T::B_ACROSS)
        if (left * ES % 16 != 0) {
            if ((int)threadIdx.x < W) {
                clear_behind(lds, threadIdx.x, left * ES);
                clear_behind(lds + UNIT, threadIdx.x, left * ES);
            }
            barrier(NQ);
        }
    static_for<NRD>([&](auto r) { read_op(first, first, r); });
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
        stage(std::integral_constant<int, 4>{}, s);
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
    epilogue<T>(p, out, acc, reinterpret_cast<float*>(lds), wave, m0 + wm, n0 + (T::GATED ? wn / 2 : wn), lane);
}

}  // namespace layer
#endif
}  // namespace sgemm
