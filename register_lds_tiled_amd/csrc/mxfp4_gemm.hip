// mxfp4_gemm.hip -- C = A.B^T with both operands in MXFP4, on the matrix
// cores, accumulated in fp32.
//
// Few rows of A (at most 16, or 64 where C is narrow: mx_few_rows):
// mxfp4_rows.hip.  Else tiles: 256 x 256 and 128 x 128 by DMA, 128 x 128 through
// registers where rows are not 16-byte aligned.  8192^3 takes 277 us to fp32 C
// and 272 to bfloat16 (4.0 PFLOP/s); the matrix instructions alone would need
// 164 on random codes, where power limits them, and 115 on zeros.
#include "mxfp4.h"

namespace sgemm {
namespace {

// v_mfma_scale_f32_32x32x64_f8f6f4 on 4-bit elements: lane l holds block l / 32
// of row l % 32 of each operand, its scale in byte SEL of one register; D as
// store_tile describes it, its rows the first operand's.  This form runs at the
// matrix cores' full rate from one wave per SIMD (9.6 PFLOP/s on zeros, 6.7
// on random codes, which power limits), where 16 x 16 x 128 reaches 5.3 from
// one wave and 6.9 from two (4.9 and 5.9 on random codes): the tile kernels
// use it.
template <int SEL>
__device__ __forceinline__ floatx16 mfma_mx32(uint4 a, unsigned sa, uint4 b, unsigned sb, floatx16 acc) {
    const mx_i8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const mx_i8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

// Tiles: a workgroup owns BM x BN outputs and walks K in stages of 256 (128
// bytes of a row).  LDS holds a stage of both operands in 16-byte chunks, chunk
// c of row r at c ^ place_of(r).  Step h of a stage gives lane half g the chunk
// 4g + h, so a lane's scales of the stage are four neighbouring bytes, one
// register for all its steps.
//
// place_of: LDS serves a 16-byte read 16 lanes (256 bytes, all banks) at a
// time, lanes 0-3, 12-15, 20-23, 24-27 together and lanes 4-11, 16-19, 28-31
// together.  In the operand reads these are as many rows of one chunk, rows of
// one parity share half of the banks, and r / 2 mod 8 is different for all rows
// of one parity in either set.  (With r mod 8 half of all LDS cycles were bank
// conflicts; this way these reads have none.  A quarter remains, from the
// scales' 4-byte reads.)
__device__ __forceinline__ int place_of(int r) { return r >> 1 & 7; }

template <int BM_, int BN_, int WM_, int WN_, int OCC_ = 1, int GROUP_M_ = 8>
struct MxTile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 256;
    static constexpr int OCC = OCC_, GROUP_M = GROUP_M_;   // waves per SIMD; rows of tiles an XCD walks together
    static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * (BN / WN), NT = NW * 64;
    static constexpr int FM = WM / 32, FN = WN / 32;
};

// mfma_mx32 in place on accumulation registers, as an instruction of its own:
// from the builtin the compiler copies 16-register accumulators about and
// spills in the widest tile (64 per lane and 1000 and more bytes of scratch at
// 128 x 128 outputs a wave).  It knows nothing of the wait states the
// instruction needs: two after a vector instruction writes an operand, and 19
// before its result is read (mfma_settled, mfma_done).
template <int SEL>
__device__ __forceinline__ void mfma_mx32_in(floatx16& acc, uint4 a, unsigned sa, uint4 b, unsigned sb) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 av = {a.x, a.y, a.z, a.w}, bv = {b.x, b.y, b.z, b.w};
    if constexpr (SEL == 0)
        asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
    else if constexpr (SEL == 1)
        asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] "
                     "cbsz:4 blgp:4" : "+a"(acc) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
    else if constexpr (SEL == 2)
        asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[1,1,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
    else
        asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0] "
                     "cbsz:4 blgp:4" : "+a"(acc) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
}
__device__ __forceinline__ void mfma_settled() { asm volatile("s_nop 3" ::: "memory"); }
template <int FM, int FN>
__device__ __forceinline__ void mfma_done(floatx16 (&acc)[FM][FN]) {
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));   // reads stay behind the pause
}

// The register-staged form, for rows of any alignment and pitch.
template <class Cfg, MxType OUT>
__global__ __launch_bounds__(Cfg::NT) void mx_tile_kernel(MxGemmArgs p, int tiles_m, int tiles_n) {
    constexpr int BM = Cfg::BM, BN = Cfg::BN, NT = Cfg::NT, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int ROWS = BM + BN, CH = ROWS * 8 / NT;
    static_assert(ROWS * 8 % NT == 0 && ROWS <= NT, "whole rounds of the loader");
    // A's rows, then B's
    __shared__ __attribute__((aligned(16))) uint4 val[ROWS * 8];
    __shared__ __attribute__((aligned(8))) unsigned char sc[ROWS * 8];
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, Cfg::GROUP_M, p.xcds, tm, tn);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / Cfg::WAVES_N) * Cfg::WM, wn = (wave % Cfg::WAVES_N) * Cfg::WN;
    const int li = lane & 31, g = lane >> 5;
    const long long m0 = (long long)tm * BM, n0 = (long long)tn * BN;
    const long long ks = ((long long)p.K + 31) / 32, len = ((long long)p.K + 1) / 2;

    // The thread's chunks and the row of its scales.  Rows past the matrix
    // read the last one: their products are not stored.
    const unsigned char* src[CH];
    int dst[CH];
#pragma unroll
    for (int u = 0; u < CH; ++u) {
        const int id = tid + u * NT, r = id >> 3, c = id & 7;
        src[u] = r < BM ? p.A + min(m0 + r, (long long)p.M - 1) * p.lda
                        : p.B + min(n0 + r - BM, (long long)p.N - 1) * p.ldb;
        dst[u] = r * 8 + (c ^ place_of(r));
    }
    const int sr = tid < ROWS ? tid : 0;
    const unsigned char* ssrc = sr < BM ? p.SA + min(m0 + sr, (long long)p.M - 1) * p.ldsa
                                        : p.SB + min(n0 + sr - BM, (long long)p.N - 1) * p.ldsb;
    uint4 v[CH];
    unsigned s[2];
    auto fetch = [&](long long k0) {
        if (k0 + Cfg::BK <= p.K) {
#pragma unroll
            for (int u = 0; u < CH; ++u) __builtin_memcpy(&v[u], src[u] + k0 / 2 + 16 * ((tid + u * NT) & 7), 16);
            __builtin_memcpy(s, ssrc + k0 / 32, 8);
        } else {
#pragma unroll
            for (int u = 0; u < CH; ++u) {
                const long long at = k0 / 2 + 16 * ((tid + u * NT) & 7);
                v[u] = len >= 16 ? mx_load16(src[u], at, len) : mx_codes16(src[u], at, p.K);
            }
            mx_scales<8>(ssrc, k0 / 32, ks, s);
        }
    };

    floatx16 acc[FM][FN] = {};
    fetch(0);
    for (long long k0 = 0; k0 < p.K; k0 += Cfg::BK) {
        if (k0 + Cfg::BK > p.K && len >= 16) {
#pragma unroll
            for (int u = 0; u < CH; ++u) v[u] = mx_end_codes16(v[u], k0 / 2 + 16 * ((tid + u * NT) & 7), p.K);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            lds_poison_f4(&val[dst[u]]);
            val[dst[u]] = v[u];
        }
        if (tid < ROWS) *reinterpret_cast<uint2*>(&sc[sr * 8]) = make_uint2(s[0], s[1]);
        __syncthreads();
        if (k0 + Cfg::BK < p.K) fetch(k0 + Cfg::BK);
        unsigned sa[FM], sb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = *reinterpret_cast<const unsigned*>(&sc[(wm + 32 * i + li) * 8 + 4 * g]);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            sb[j] = *reinterpret_cast<const unsigned*>(&sc[(BM + wn + 32 * j + li) * 8 + 4 * g]);
        static_for<4>([&](auto h) {
            const int c = (4 * g + h) ^ place_of(li);
            uint4 a[FM], b[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) a[i] = val[(wm + 32 * i + li) * 8 + c];
#pragma unroll
            for (int j = 0; j < FN; ++j) b[j] = val[(BM + wn + 32 * j + li) * 8 + c];
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma_mx32<h>(a[i], sa[i], b[j], sb[j], acc[i][j]);
        });
    }
    mx_store_wave<OUT>(p, acc, m0 + wm, n0 + wn, li, g);
}

// The same tiles where rows lie 16-byte aligned: both operands come by DMA into
// one of two LDS stages, the next stage requested right after the barrier that
// ends the reads of its place and waited for a stage's multiplication later.
//
// Scales of 2048 k (64 bytes of every row) lie in LDS beside the stages, chunk c
// of row r at c ^ (r / 4 & 3).  They are read along the rows while the last
// stage that needs the ones before multiplies, and written after it.  (Loaded
// straight to the lanes that need them, a row a lane, they took the address
// unit as long as half the codes: 8192^3 to bf16 in 128 x 128 tiles 369 us, 307
// without any scales.)
//
// Past K: a chunk that begins past a row's end is read from the row's last
// one, and what is past K in A's last stage is cleared in LDS; B's codes
// there are finite, and 0 times them is 0.  A scale past the row's end is 0
// (2^-127).
template <class Cfg, MxType OUT>
__global__ __launch_bounds__(Cfg::NT, Cfg::OCC) void mx_dma_kernel(MxGemmArgs p, int tiles_m, int tiles_n) {
    constexpr int BM = Cfg::BM, BN = Cfg::BN, NW = Cfg::NW, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int IA = BM * 8 / 64 / NW, IB = BN * 8 / 64 / NW;   // a wave's DMA instructions per stage
    static_assert(IA * NW * 64 == BM * 8 && IB * NW * 64 == BN * 8, "whole DMA rounds");
    constexpr int IS = (BM + BN) * 4 / Cfg::NT;                   // a thread's 16-byte pieces of scales
    static_assert(IS * Cfg::NT == (BM + BN) * 4, "whole rounds of scales");
    constexpr unsigned STAGE = (BM + BN) * 128;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * STAGE];
    __shared__ __attribute__((aligned(16))) uint4 sc[(BM + BN) * 4];   // A's rows, then B's
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, Cfg::GROUP_M, p.xcds, tm, tn);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / Cfg::WAVES_N) * Cfg::WM, wn = (wave % Cfg::WAVES_N) * Cfg::WN;
    const int li = lane & 31, g = lane >> 5;
    const long long m0 = (long long)tm * BM, n0 = (long long)tn * BN;
    const int mlast = (int)min((long long)p.M - 1 - m0, (long long)BM - 1);
    const int nlast = (int)min((long long)p.N - 1 - n0, (long long)BN - 1);
    const unsigned char* const A = p.A + m0 * p.lda;
    const unsigned char* const B = p.B + n0 * p.ldb;
    const int chunks = (int)(((long long)p.K + 31) / 32);           // 16-byte chunks, and scales, of a row
    const int stages = (int)(((long long)p.K + 255) / 256);

    // Instruction u of this wave, lane l: chunk id 64 (wave + u NW) + l of the
    // operand's stage, row id / 8, place id % 8, which holds chunk place ^ place_of(row).
    static_assert(NW % 2 == 0, "a wave's rows agree in bit 3");
    const int c = (lane & 7) ^ place_of((wave & 1) * 8 + (lane >> 3));
    unsigned va[IA], vb[IB];
#pragma unroll
    for (int u = 0; u < IA; ++u)
        va[u] = (unsigned)min((wave + u * NW) * 8 + (lane >> 3), mlast) * (unsigned)p.lda;
#pragma unroll
    for (int u = 0; u < IB; ++u)
        vb[u] = (unsigned)min((wave + u * NW) * 8 + (lane >> 3), nlast) * (unsigned)p.ldb;
    const unsigned lds0 = lds_addr(lds);
    auto request = [&](int s) __attribute__((always_inline)) {
        const unsigned at = (unsigned)min(c, chunks - 1 - 8 * s) * 16u;
        const unsigned to = lds0 + (s & 1) * STAGE + 1024u * wave;
        const unsigned char* const a = A + 128ll * s;
        const unsigned char* const b = B + 128ll * s;
#pragma unroll
        for (int u = 0; u < IA; ++u)
            lds_dma16s(a, va[u] + at, __builtin_amdgcn_readfirstlane(to + u * NW * 1024u));
#pragma unroll
        for (int u = 0; u < IB; ++u)
            lds_dma16s(b, vb[u] + at, __builtin_amdgcn_readfirstlane(to + BM * 128 + u * NW * 1024u));
    };
    // A row's bytes from 64 panel on; past its end its last 16 instead, moved
    // down when they are placed.
    uint4 piece[IS];
    static_assert(BM * 4 % Cfg::NT == 0, "a round of scales is A's or B's");
    auto scale_row = [&](auto u) __attribute__((always_inline)) {
        constexpr int r0 = u * Cfg::NT / 4;
        const int r = r0 + (tid >> 2);
        if constexpr (r0 < BM)
            return p.SA + (m0 + min(r, mlast)) * p.ldsa;
        else
            return p.SB + (n0 + min(r - BM, nlast)) * p.ldsb;
    };
    const int sat = 16 * (tid & 3);
    auto load_scales = [&](int panel) __attribute__((always_inline)) {
        const int at = min(64 * panel + sat, chunks - 16);
        static_for<IS>([&](auto u) { __builtin_memcpy(&piece[u], scale_row(u) + at, 16); });
    };
    auto place_scales = [&](int panel) __attribute__((always_inline)) {
        const int past = chunks < 16 ? 0 : max(64 * panel + sat - (chunks - 16), 0);
        static_for<IS>([&](auto u) {
            const int r = (tid + u * Cfg::NT) >> 2;
            uint4* const to = &sc[r * 4 + ((tid ^ (r >> 2)) & 3)];
            lds_poison_f4(to);
            *to = past == 0 ? piece[u] : mx_down(piece[u], past);
        });
    };
    unsigned fa[2][FM], fb[2][FN];               // by stage of a pair, a register a tile
    auto read_scales = [&](int s) __attribute__((always_inline)) {
        const int c = s >> 1;                    // the pair's chunk, mod 4
        auto read = [&](int r, unsigned& even, unsigned& odd) {
            const unsigned* const w = reinterpret_cast<const unsigned*>(&sc[r * 4 + ((c ^ (r >> 2)) & 3)]) + g;
            even = w[0];
            odd = w[2];
        };
#pragma unroll
        for (int i = 0; i < FM; ++i) read(wm + 32 * i + li, fa[0][i], fa[1][i]);
#pragma unroll
        for (int j = 0; j < FN; ++j) read(BM + wn + 32 * j + li, fb[0][j], fb[1][j]);
    };

    floatx16 acc[FM][FN] = {};
    // One stage: in step h, lane half g has block 8 s + 4 g + h.
    auto multiply = [&](auto odd) __attribute__((always_inline)) {
        const unsigned char* const st = lds + (odd ? STAGE : 0u);
        // a step's operands are read while the step before multiplies; the
        // barriers keep the compiler from reading the whole stage at once
        uint4 a[2][FM], b[2][FN];
        auto read = [&](auto h) __attribute__((always_inline)) {
            const int at = ((4 * g + h) ^ place_of(li)) * 16;
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[h & 1][j] = *reinterpret_cast<const uint4*>(st + (BM + wn + 32 * j + li) * 128 + at);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                a[h & 1][i] = *reinterpret_cast<const uint4*>(st + (wm + 32 * i + li) * 128 + at);
        };
        read(std::integral_constant<int, 0>{});
        mfma_settled();
        static_for<4>([&](auto h) {
            if constexpr (h < 3) read(std::integral_constant<int, h + 1>{});
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    mfma_mx32_in<h>(acc[i][j], a[h & 1][i], fa[odd][i], b[h & 1][j], fb[odd][j]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // The requested stage is there, for all waves, and the other one's reads
    // are over.
    auto arrived = [&]() __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    // A's elements past K in a stage become 0.
    auto clear_past = [&](int s) __attribute__((always_inline)) {
        if (256ll * (s + 1) <= p.K) return;
        for (int id = tid; id < BM * 8; id += Cfg::NT) {
            const int left = (int)(p.K - 32ll * (8 * s + ((id & 7) ^ place_of(id >> 3))));
            uint4* const v = reinterpret_cast<uint4*>(lds + (s & 1) * STAGE + 16 * id);
            if (left < 32) *v = mx_keep(*v, left);
        }
        __syncthreads();
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    if (chunks >= 16)
        load_scales(0);
    else
        static_for<IS>([&](auto u) __attribute__((always_inline)) {
            piece[u] = mx_bytes16(scale_row(u), sat, chunks);
        });
    request(0);
    place_scales(0);
    // Pairs of stages.  One copy of the multiplication, in the loop: from a
    // second one after it the compiler copies the accumulators, without the
    // wait states that takes.  So where K ends in a pair's first stage, the
    // second multiplies zeros.
    int s = 0;
    do {                                         // K > 0
        arrived();
        read_scales(s);
        clear_past(s);
        if (s + 1 < stages) request(s + 1);
        multiply(even);
        arrived();
        const bool turn = (s & 7) == 6 && s + 2 < stages;   // the panel's last scales have been read
        if (turn) load_scales((s + 2) >> 3);
        clear_past(s + 1);
        if (s + 2 < stages) request(s + 2);
        multiply(odd);
        if (turn) place_scales((s + 2) >> 3);
    } while ((s += 2) < stages);
    mfma_done(acc);
    mx_store_wave<OUT>(p, acc, m0 + wm, n0 + wn, li, g);
}

template <class Cfg>
hipError_t tile_grid(const MxGemmArgs& a, int& tm, int& tn) {
    tm = (int)(((long long)a.M + Cfg::BM - 1) / Cfg::BM);
    tn = (int)(((long long)a.N + Cfg::BN - 1) / Cfg::BN);
    return (long long)tm * tn * Cfg::NT > 0xFFFFFFFFll ? hipErrorInvalidValue : hipSuccess;
}

template <class Cfg, MxType OUT>
hipError_t launch_dma(const MxGemmArgs& a, hipStream_t s) {
    int tm, tn;
    const hipError_t e = tile_grid<Cfg>(a, tm, tn);
    if (e != hipSuccess) return e;
    mx_dma_kernel<Cfg, OUT><<<(unsigned)(tm * tn), Cfg::NT, 0, s>>>(a, tm, tn);
    return hipGetLastError();
}

template <class Cfg, MxType OUT>
hipError_t launch_tile(const MxGemmArgs& a, hipStream_t s) {
    int tm, tn;
    const hipError_t e = tile_grid<Cfg>(a, tm, tn);
    if (e != hipSuccess) return e;
    mx_tile_kernel<Cfg, OUT><<<(unsigned)(tm * tn), Cfg::NT, 0, s>>>(a, tm, tn);
    return hipGetLastError();
}

template <MxType OUT>
hipError_t launch_out(const MxGemmArgs& a, hipStream_t s) {
    if (mx_few_rows(a)) return launch_mx_rows(a, MxType::mxfp4, OUT, s);
    const bool dma = mx_aligned(a.A, a.lda, 16) && mx_aligned(a.B, a.ldb, 16) && a.K > 0 &&
                     mx_dma_reach(a.lda, 256) && mx_dma_reach(a.ldb, 256);
    if (!dma) return launch_tile<MxTile<128, 128, 64, 64>, OUT>(a, s);
    // Rounds of workgroups, one 256 x 256 or two 128 x 128 to a CU, times what a
    // round takes (8192^3: 69 us of four rounds, 39 to 41 of eight).  The wide
    // tiles read half as much through L2, whose rate (25 TB/s and more) bounds
    // the others.  us to fp32 and bfloat16: 8192^3 277 and 272 wide, 310 and 329
    // else; 4096 x 8192 x 4096 91 and 78, 92 and 97; 2048^3, 64 wide tiles, to
    // bfloat16 20 against 11.
    const long long wide = ((long long)a.M + 255) / 256 * (((long long)a.N + 255) / 256);
    const long long small = ((long long)a.M + 127) / 128 * (((long long)a.N + 127) / 128);
    if (5 * ((wide + a.cus - 1) / a.cus) <= 3 * ((small + 2 * a.cus - 1) / (2 * a.cus)))
        return launch_dma<MxTile<256, 256, 128, 64, 2>, OUT>(a, s);
    return launch_dma<MxTile<128, 128, 64, 64, 2>, OUT>(a, s);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& a, MxType out, hipStream_t s) {
    return out == MxType::f32 ? launch_out<MxType::f32>(a, s) : launch_out<MxType::bf16>(a, s);
}

}  // namespace sgemm
