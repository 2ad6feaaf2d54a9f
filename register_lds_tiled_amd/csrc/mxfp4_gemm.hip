// mxfp4_gemm.hip -- C = A.B^T with both operands in MXFP4, on the matrix
// cores, accumulated in fp32.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies a 16 x 128 by a 128 x 16 piece
// of 4-bit elements: lane l holds 32 consecutive elements (16 bytes, one MX
// block) of row l % 16 of each operand, and a scale byte for them in a byte,
// chosen by the instruction, of one register.  The order of the k terms is
// free, so which blocks the four lane groups l / 16 take together is chosen
// for the memory side.  D: lane l, register i is row 4 (l / 16) + i of the
// first operand, row l % 16 of the second.  B's rows are passed first, so a
// lane holds four neighbouring columns of one row of C.  (Layout, scale bytes
// 0 and 255 and the sums' accuracy checked on the GPU: within 2.5e-8 of
// sum |a b| of the exact sum over 128 terms.)
#include "mxfp4.h"

namespace sgemm {
namespace {

// acc += the 16 x 16 x 128 product, with byte SEL of each scale register.
template <int SEL>
__device__ __forceinline__ mx_f4 mfma_mx(uint4 b, unsigned sb, uint4 a, unsigned sa, mx_f4 acc) {
    const mx_i8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    const mx_i8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc, 4, 4, SEL, (int)sb, SEL, (int)sa);
}

// The same for 32 x 32 x 64: lane l holds block l / 32 of row l % 32; D as
// store_tile describes it, its rows the first operand's.  This form runs at
// the matrix cores' full rate from one wave per SIMD (9.6 PFLOP/s on zeros, 6.7
// on random codes, which power limits), where 16 x 16 x 128 reaches 5.3 from
// one wave and 6.9 from two (4.9 and 5.9 on random codes): the tile kernels
// use it.
template <int SEL>
__device__ __forceinline__ floatx16 mfma_mx32(uint4 a, unsigned sa, uint4 b, unsigned sb, floatx16 acc) {
    const mx_i8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const mx_i8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

// One row's four neighbouring outputs from column col on.
template <MxType OUT>
__device__ __forceinline__ void store4(const MxGemmArgs& p, long long row, long long col, mx_f4 v) {
    if (row >= p.M || col >= p.N) return;
    const int n = (int)min(p.N - col, 4ll);
    if constexpr (OUT == MxType::f32) {
        float* c = static_cast<float*>(p.C) + row * p.ldc + col;
        if (n == 4 && ((size_t)c & 15) == 0) {
            store_c4(c, v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) store_c(c + i, v[i]);
        }
    } else {
        __bf16* c = static_cast<__bf16*>(p.C) + row * p.ldc + col;
        typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
        if (n == 4 && ((size_t)c & 7) == 0) {
            *reinterpret_cast<bf4*>(c) = bf4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) c[i] = (__bf16)v[i];
        }
    }
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
// of one parity in either set.  (With r mod 8 half of all LDS cycles are bank
// conflicts; this way the counter reads 0.)
__device__ __forceinline__ int place_of(int r) { return r >> 1 & 7; }

template <int BM_, int BN_, int WM_, int WN_, int OCC_ = 1, int GROUP_M_ = 8>
struct MxTile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 256;
    static constexpr int OCC = OCC_, GROUP_M = GROUP_M_;   // waves per SIMD; rows of tiles an XCD walks together
    static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * (BN / WN), NT = NW * 64;
    static constexpr int FM = WM / 32, FN = WN / 32;
};

// A wave's outputs, whose first is (r0, c0).
template <MxType OUT, int FM, int FN>
__device__ __forceinline__ void store_wave(const MxGemmArgs& p, const floatx16 (&acc)[FM][FN], long long r0,
                                           long long c0, int li, int g) {
    typedef std::conditional_t<OUT == MxType::f32, float, __bf16> T;
    const int rows = (int)min(p.M - r0, 32ll * FM) - 4 * g, cols = (int)min(p.N - c0, 32ll * FN) - li;
    T* c = static_cast<T*>(p.C) + (r0 + 4 * g) * p.ldc + c0 + li;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = 32 * i + 8 * (r / 4) + r % 4;
            T* const at = c + row * p.ldc;
#pragma unroll
            for (int j = 0; j < FN; ++j)
                if (row < rows && 32 * j < cols) {
                    if constexpr (OUT == MxType::f32)
                        store_c(at + 32 * j, acc[i][j][r]);
                    else
                        at[32 * j] = (__bf16)acc[i][j][r];
                }
        }
    }
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
    const long long ks = ((long long)p.K + 31) / 32;

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
            for (int u = 0; u < CH; ++u) v[u] = mx_load16<false>(src[u] + k0 / 2 + 16 * ((tid + u * NT) & 7), 16);
            __builtin_memcpy(s, ssrc + k0 / 32, 8);
        } else {
#pragma unroll
            for (int u = 0; u < CH; ++u)
                v[u] = mx_codes16<false>(src[u], k0 / 2 + 16 * ((tid + u * NT) & 7), p.K);
            mx_scales<8>(ssrc, k0 / 32, ks, s);
        }
    };

    floatx16 acc[FM][FN] = {};
    fetch(0);
    for (long long k0 = 0; k0 < p.K; k0 += Cfg::BK) {
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
    store_wave<OUT>(p, acc, m0 + wm, n0 + wn, li, g);
}

// 16 scale bytes of a row of n, from byte `at` on where they exist; else the
// row's last 16, or its n < 16 and zeros.
__device__ __forceinline__ void scales16(const unsigned char* row, int at, int n, unsigned (&s)[4]) {
    __builtin_memcpy(s, row + min(at, n - 16), 16);
}
__device__ __forceinline__ void scales_few(const unsigned char* row, int n, unsigned (&s)[4]) {
    unsigned char v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = row[min(i, n - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i / 4] |= (i < n ? (unsigned)v[i] : 0u) << (8 * (i % 4));
}
// 16 bytes moved down by n (0 .. 15, wave-uniform), zeros above.
__device__ __forceinline__ void down16(unsigned (&s)[4], int n) {
    for (int k = n >> 2; k > 0; --k) {
        s[0] = s[1];
        s[1] = s[2];
        s[2] = s[3];
        s[3] = 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = __builtin_amdgcn_alignbyte(i < 3 ? s[i + 1] : 0u, s[i], n & 3);
}

// The same tiles where rows lie 16-byte aligned: both operands come by DMA into
// one of two LDS stages, the next stage requested right after the barrier that
// ends the reads of its place and waited for a stage's multiplication later.
//
// Scales come straight to registers, 16 bytes (512 k, two stages) of 64 rows
// by one load: lane 32 t + r holds row r of tile t, in words w0 .. w3.  Lane
// half g needs words g (first stage) and 2 + g (second) of both tiles: one
// exchange of lane halves per stage brings them there.
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
    static_assert(FM % 2 == 0 && FN % 2 == 0, "64 rows of scales at a time");
    constexpr unsigned STAGE = (BM + BN) * 128;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * STAGE];
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
    auto request = [&](int s) {
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
    const unsigned char* sa[FM / 2];
    const unsigned char* sb[FN / 2];
#pragma unroll
    for (int i = 0; i < FM / 2; ++i) sa[i] = p.SA + (m0 + min(wm + 64 * i + lane, mlast)) * p.ldsa;
#pragma unroll
    for (int j = 0; j < FN / 2; ++j) sb[j] = p.SB + (n0 + min(wn + 64 * j + lane, nlast)) * p.ldsb;
    unsigned ra[FM / 2][4], rb[FN / 2][4];       // as loaded for the next pair of stages
    unsigned fa[2][FM], fb[2][FN];               // by stage of the pair, a register a tile
    auto load_scales = [&](int s) {
#pragma unroll
        for (int i = 0; i < FM / 2; ++i) scales16(sa[i], 8 * s, chunks, ra[i]);
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) scales16(sb[j], 8 * s, chunks, rb[j]);
    };
    auto place_scales = [&] {
        static_for<2>([&](auto q) {
#pragma unroll
            for (int i = 0; i < FM / 2; ++i) {
                const auto x = __builtin_amdgcn_permlane32_swap(ra[i][2 * q], ra[i][2 * q + 1], false, false);
                fa[q][2 * i] = x[0];
                fa[q][2 * i + 1] = x[1];
            }
#pragma unroll
            for (int j = 0; j < FN / 2; ++j) {
                const auto x = __builtin_amdgcn_permlane32_swap(rb[j][2 * q], rb[j][2 * q + 1], false, false);
                fb[q][2 * j] = x[0];
                fb[q][2 * j + 1] = x[1];
            }
        });
    };

    floatx16 acc[FM][FN] = {};
    // One stage: in step h, lane half g has block 8 s + 4 g + h.
    auto multiply = [&](auto odd) {
        const unsigned char* const st = lds + (odd ? STAGE : 0u);
        // a step's operands are read while the step before multiplies; the
        // barriers keep the compiler from reading the whole stage at once
        uint4 a[2][FM], b[2][FN];
        auto read = [&](auto h) {
            const int at = ((4 * g + h) ^ place_of(li)) * 16;
#pragma unroll
            for (int j = 0; j < FN; ++j)
                b[h & 1][j] = *reinterpret_cast<const uint4*>(st + (BM + wn + 32 * j + li) * 128 + at);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                a[h & 1][i] = *reinterpret_cast<const uint4*>(st + (wm + 32 * i + li) * 128 + at);
        };
        read(std::integral_constant<int, 0>{});
        static_for<4>([&](auto h) {
            if constexpr (h < 3) read(std::integral_constant<int, h + 1>{});
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = mfma_mx32<h>(a[h & 1][i], fa[odd][i], b[h & 1][j], fb[odd][j], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // The requested stage is there, for all waves, and the other one's reads
    // are over.
    auto arrived = [&] {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };
    // A's elements past K, in the last stage, become 0.
    auto clear_past = [&](int s) {
        if ((p.K & 255) == 0) return;
        for (int id = tid; id < BM * 8; id += Cfg::NT) {
            const int left = p.K - 32 * (8 * s + ((id & 7) ^ place_of(id >> 3)));
            uint4* const v = reinterpret_cast<uint4*>(lds + (s & 1) * STAGE + 16 * id);
            if (left < 32) *v = mx_keep(*v, left);
        }
        __syncthreads();
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    if (chunks >= 16) {
        load_scales(0);
    } else {
#pragma unroll
        for (int i = 0; i < FM / 2; ++i) scales_few(sa[i], chunks, ra[i]);
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) scales_few(sb[j], chunks, rb[j]);
    }
    request(0);
    // Pairs of stages that another follows, then the last pair or single stage.
    int s = 0;
    for (; s + 2 < stages; s += 2) {
        arrived();
        place_scales();
        load_scales(s + 2);
        request(s + 1);
        multiply(even);
        arrived();
        request(s + 2);
        multiply(odd);
    }
    arrived();
    if (const int past = 8 * s + 16 - chunks; past > 0 && chunks >= 16) {
#pragma unroll
        for (int i = 0; i < FM / 2; ++i) down16(ra[i], past);
#pragma unroll
        for (int j = 0; j < FN / 2; ++j) down16(rb[j], past);
    }
    place_scales();
    if (s + 1 < stages) {
        request(s + 1);
        multiply(even);
        arrived();
        clear_past(s + 1);
        multiply(odd);
    } else {
        clear_past(s);
        multiply(even);
    }
    store_wave<OUT>(p, acc, m0 + wm, n0 + wn, li, g);
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

// Few rows of A (at most 16 MT): B is streamed once.  A workgroup owns 16 NT
// rows of B; its waves take the spans of 512 k in turn, hold a span's operands
// and the next one's in registers, and add their parts in LDS at the end, in
// wave order.  Lane group g takes blocks 4g .. 4g + 3 of a span, one in each
// of four steps: a lane's scales of the span are then four neighbouring bytes,
// one register for all steps.
template <int MT, int NT, int NW, MxType OUT, bool VEC>
__global__ __launch_bounds__(64 * NW) void mx_rows_kernel(MxGemmArgs p) {
    __shared__ mx_f4 part[NW > 1 ? NW : 1][MT * NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, g = lane >> 4;
    const long long n0 = (long long)blockIdx.x * (16 * NT);
    const long long ks = ((long long)p.K + 31) / 32;
    const unsigned char *b[NT], *sb[NT], *a[MT], *sa[MT];
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
        sa[i] = p.SA + (has[i] ? m : 0) * p.ldsa;
    }
    struct Span {
        uint4 b[NT][4], a[MT][4];
        unsigned sb[NT], sa[MT];
    };
    auto load_row = [&](const unsigned char* q, const unsigned char* s, long long k0, uint4 (&v)[4], unsigned& sc) {
        const long long at = k0 / 2 + 64 * g;
        unsigned w[1];
        if (k0 + 512 <= p.K) {
#pragma unroll
            for (int h = 0; h < 4; ++h) v[h] = mx_load16<VEC>(q + at + 16 * h, 16);
            __builtin_memcpy(w, s + k0 / 32 + 4 * g, 4);
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) v[h] = mx_codes16<VEC>(q, at + 16 * h, p.K);
            mx_scales<4>(s, k0 / 32 + 4 * g, ks, w);
        }
        sc = w[0];
    };
    auto load = [&](Span& t, long long k0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) load_row(b[j], sb[j], k0, t.b[j], t.sb[j]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int h = 0; h < 4; ++h) t.a[i][h] = make_uint4(0u, 0u, 0u, 0u);
            t.sa[i] = 0u;
            if (has[i]) load_row(a[i], sa[i], k0, t.a[i], t.sa[i]);
        }
    };
    mx_f4 acc[MT][NT] = {};
    Span cur, next;
    long long k0 = 512ll * wave;
    if (k0 < p.K) load(cur, k0);
    while (k0 < p.K) {
        const long long k1 = k0 + 512 * NW;
        if (k1 < p.K) load(next, k1);
        static_for<4>([&](auto h) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = mfma_mx<h>(cur.b[j][h], cur.sb[j], cur.a[i][h], cur.sa[i], acc[i][j]);
        });
        cur = next;
        k0 = k1;
    }
    if constexpr (NW > 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
        __syncthreads();
        for (int t = wave; t < MT * NT; t += NW) {
            mx_f4 v = part[0][t][lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) v += part[w][t][lane];
            store4<OUT>(p, 16 * (t / NT) + li, n0 + 16 * (t % NT) + 4 * g, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) store4<OUT>(p, 16 * i + li, n0 + 16 * j + 4 * g, acc[i][j]);
    }
}

template <int MT, int NT, int NW, MxType OUT>
hipError_t launch_rows_cfg(const MxGemmArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)(((long long)a.N + 16 * NT - 1) / (16 * NT));
    if (mx_aligned(a.A, a.lda, 16) && mx_aligned(a.B, a.ldb, 16))
        mx_rows_kernel<MT, NT, NW, OUT, true><<<grid, 64 * NW, 0, s>>>(a);
    else
        mx_rows_kernel<MT, NT, NW, OUT, false><<<grid, 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

template <int MT, MxType OUT>
hipError_t launch_rows(const MxGemmArgs& a, hipStream_t s) {
    // Two tiles of B's rows to a workgroup where that leaves two workgroups
    // for every CU; waves for the spans there are.
    constexpr int NT = MT < 4 ? 2 : 1;
    const bool two = (long long)a.N >= 64ll * a.cus;
    const int spans = (a.K + 511) / 512;
    if (spans >= 5)
        return two ? launch_rows_cfg<MT, NT, 8, OUT>(a, s) : launch_rows_cfg<MT, 1, 8, OUT>(a, s);
    return two ? launch_rows_cfg<MT, NT, 2, OUT>(a, s) : launch_rows_cfg<MT, 1, 2, OUT>(a, s);
}

template <MxType OUT>
hipError_t launch_out(const MxGemmArgs& a, hipStream_t s) {
    if (a.M <= 16) return launch_rows<1, OUT>(a, s);
    if (a.M <= 32) return launch_rows<2, OUT>(a, s);
    if (a.M <= 64) return launch_rows<4, OUT>(a, s);
    const bool dma = mx_aligned(a.A, a.lda, 16) && mx_aligned(a.B, a.ldb, 16) && a.K > 0 &&
                     mx_dma_reach(a.lda, 256) && mx_dma_reach(a.ldb, 256);
    if (!dma) return launch_tile<MxTile<128, 128, 64, 64>, OUT>(a, s);
#ifdef MXT_
    return launch_dma<MxTile<MXT_>, OUT>(a, s);
#endif
    return launch_dma<MxTile<128, 128, 64, 64, 2>, OUT>(a, s);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& a, MxType out, hipStream_t s) {
    return out == MxType::f32 ? launch_out<MxType::f32>(a, s) : launch_out<MxType::bf16>(a, s);
}

}  // namespace sgemm
