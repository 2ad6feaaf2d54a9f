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

// One row's four neighbouring outputs from column col on.
template <MxType OUT>
__device__ __forceinline__ void store4(const MxGemmArgs& p, long long row, int col, mx_f4 v) {
    if (row >= p.M || col >= p.N) return;
    const int n = min(p.N - col, 4);
    if constexpr (OUT == MxType::f32) {
        float* c = static_cast<float*>(p.C) + row * p.ldc + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) store_c(c + i, v[i]);
    } else {
        __bf16* c = static_cast<__bf16*>(p.C) + row * p.ldc + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) c[i] = (__bf16)v[i];
    }
}

// Tiles: a workgroup of four waves owns BM x BN outputs and walks K in stages
// of 256 (128 bytes of a row).  LDS holds a stage of both operands in 16-byte
// chunks, chunk c of row r at c ^ (r & 7), so that eight rows' equal chunks
// lie in distinct banks, and the stage's 8 scale bytes of every row.  Step h
// of a stage gives lane group g the chunks 2g + h, whose two scales are two
// neighbouring bytes: one 16-bit read serves both steps.
template <int BM_, int BN_, int WM_, int WN_>
struct MxTile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 256;
    static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * (BN / WN), NT = NW * 64;
    static constexpr int FM = WM / 16, FN = WN / 16;
};

template <class Cfg, MxType OUT, bool VEC>
__global__ __launch_bounds__(Cfg::NT) void mx_tile_kernel(MxGemmArgs p, int tiles_m, int tiles_n) {
    constexpr int BM = Cfg::BM, BN = Cfg::BN, NT = Cfg::NT, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int ROWS = BM + BN, CH = ROWS * 8 / NT;
    static_assert(ROWS * 8 % NT == 0 && ROWS <= NT, "whole rounds of the loader");
    // A's rows, then B's
    __shared__ __attribute__((aligned(16))) uint4 val[ROWS * 8];
    __shared__ __attribute__((aligned(8))) unsigned char sc[ROWS * 8];
    int tm, tn;
    tile_coords(blockIdx.x, tiles_m, tiles_n, 8, p.xcds, tm, tn);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / Cfg::WAVES_N) * Cfg::WM, wn = (wave % Cfg::WAVES_N) * Cfg::WN;
    const int li = lane & 15, g = lane >> 4;
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
        dst[u] = r * 8 + (c ^ (r & 7));
    }
    const int sr = tid < ROWS ? tid : 0;
    const unsigned char* ssrc = sr < BM ? p.SA + min(m0 + sr, (long long)p.M - 1) * p.ldsa
                                        : p.SB + min(n0 + sr - BM, (long long)p.N - 1) * p.ldsb;
    uint4 v[CH];
    unsigned s[2];
    auto fetch = [&](long long k0) {
#pragma unroll
        for (int u = 0; u < CH; ++u)
            v[u] = mx_codes16<VEC>(src[u], k0 / 2 + 16 * ((tid + u * NT) & 7), p.K);
        mx_scales<8>(ssrc, k0 / 32, ks, s);
    };

    mx_f4 acc[FM][FN] = {};
    fetch(0);
    for (long long k0 = 0; k0 < p.K; k0 += Cfg::BK) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < CH; ++u) val[dst[u]] = v[u];
        if (tid < ROWS) *reinterpret_cast<uint2*>(&sc[sr * 8]) = make_uint2(s[0], s[1]);
        __syncthreads();
        if (k0 + Cfg::BK < p.K) fetch(k0 + Cfg::BK);
        unsigned sa[FM], sb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] = *reinterpret_cast<const unsigned short*>(&sc[(wm + 16 * i + li) * 8 + 2 * g]);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            sb[j] = *reinterpret_cast<const unsigned short*>(&sc[(BM + wn + 16 * j + li) * 8 + 2 * g]);
        static_for<2>([&](auto h) {
            const int c = (2 * g + h) ^ (li & 7);
            uint4 a[FM], b[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) a[i] = val[(wm + 16 * i + li) * 8 + c];
#pragma unroll
            for (int j = 0; j < FN; ++j) b[j] = val[(BM + wn + 16 * j + li) * 8 + c];
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma_mx<h>(b[j], sb[j], a[i], sa[i], acc[i][j]);
        });
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            store4<OUT>(p, m0 + wm + 16 * i + li, (int)(n0 + wn + 16 * j + 4 * g), acc[i][j]);
}

template <class Cfg, MxType OUT>
hipError_t launch_tile(const MxGemmArgs& a, hipStream_t s) {
    const int tm = (int)(((long long)a.M + Cfg::BM - 1) / Cfg::BM);
    const int tn = (int)(((long long)a.N + Cfg::BN - 1) / Cfg::BN);
    const bool vec = mx_aligned(a.A, a.lda, 16) && mx_aligned(a.B, a.ldb, 16);
    if (vec)
        mx_tile_kernel<Cfg, OUT, true><<<(unsigned)tm * tn, Cfg::NT, 0, s>>>(a, tm, tn);
    else
        mx_tile_kernel<Cfg, OUT, false><<<(unsigned)tm * tn, Cfg::NT, 0, s>>>(a, tm, tn);
    return hipGetLastError();
}

template <MxType OUT>
hipError_t launch_out(const MxGemmArgs& a, hipStream_t s) {
    return launch_tile<MxTile<128, 128, 64, 64>, OUT>(a, s);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& a, MxType out, hipStream_t s) {
    return out == MxType::f32 ? launch_out<MxType::f32>(a, s) : launch_out<MxType::bf16>(a, s);
}

}  // namespace sgemm
