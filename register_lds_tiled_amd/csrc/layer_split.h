// layer_split.h -- small tiles of the feed-forward layer's products whose waves
// divide k, and the choice of a product's tiles.
//
// For products with too few 128 x 128 tiles to fill the CUs (a batch in decoding,
// a short prompt, narrow layers): a workgroup owns 32 or 64 rows and 64 columns of
// products, and each of its four waves the whole tile for every fourth stage of
// 128 bytes of k.  A wave brings its stages by DMA into a ring of its own in LDS,
// and the next into a stage's place as soon as that is in registers, so the loop
// needs no barrier, and nearly all of LDS is on its way from memory all the time:
// such launches are bound by what the caches deliver and by its latency.  Stages
// are whole cache lines because a request for a line that is still on its way
// stalls the ones behind it (with 64 bytes int8 128 x 4096 x 4096 took 11.9 us, 9.6
// so).  The waves' parts are added at the end, in wave order, through LDS.
#pragma once

#include "layer_big.h"

namespace sgemm {
#ifdef __HIPCC__
namespace layer {

constexpr int kSplit = 4;   // waves

template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

// T: the tile with one wave to all of it (WM = BM, WN = BN).
template <class T, int RING>
__global__ __launch_bounds__(64 * kSplit) void split_kernel(LayerArgs p, int tiles_m, int tiles_n) {
    constexpr int BM = T::BM, BN = T::BN, FM = T::FM, FN = T::FN, KST = 2 * T::KST, ES = T::ES;
    constexpr int A_BYTES = 2 * T::SA, B_BYTES = 2 * T::SB, STAGE = A_BYTES + B_BYTES, MINE = RING * STAGE;
    constexpr int AQ = A_BYTES / 1024, BQ = B_BYTES / 1024, NDMA = AQ + BQ;
    constexpr int PART = BM * T::STR * 4;
    static_assert(BM <= 64 && BN <= 64, "a lane to each row");
    static_assert(T::NW == 1 && PART <= MINE, "a wave's part of the result in its ring");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[kSplit * MINE];
    const int per = tiles_m * tiles_n;
    const int out = T::OUTS == 2 && (int)blockIdx.x >= per ? 1 : 0;
    int tm, tn;
    tile_coords(blockIdx.x - out * per, tiles_m, tiles_n, T::GROUP_M, p.xcds, tm, tn);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 31, g = lane >> 5;
    const long long m0 = (long long)tm * BM, n0 = (long long)tn * T::COLS;
    const int mlast = (int)min((long long)p.M - 1 - m0, (long long)BM - 1);
    const int nlast = (int)min((long long)p.N - 1 - n0, (long long)T::COLS - 1);
    const unsigned ring = __builtin_amdgcn_readfirstlane(lds_addr(lds)) + (unsigned)(wave * MINE);

    // Stages as in the large tiles' kernel: the first has what is left of K.
    const int each = (int)(((long long)p.K + KST - 1) / KST), nst = each * T::PAIRS;
    const int left = (int)(p.K - (each - 1ll) * KST);
    const int mine = (nst - wave + kSplit - 1) / kSplit;   // this wave's
    auto along = [&](int v, int row, long long ld, int& kk) __attribute__((always_inline)) {
        const int c = (lane & 7) ^ line_at(8 * v + (lane >> 3));
        kk = 16 / ES * c;
        return (unsigned)row * (unsigned)ld + 16u * (unsigned)c;
    };
    auto across = [&](int v, auto W, int last, long long ld, int& kk) __attribute__((always_inline)) {
        const int k = v * (512 / W) + lane / (W / 8), c = lane % (W / 8) ^ across_swap<W>(k);
        kk = k;
        return (unsigned)k * (unsigned)ld + (8 * c <= last ? 16u * (unsigned)c : 0u);
    };
    const int pa = T::OUTS == 2 ? out : 0;
    const unsigned char* const abase = T::A_ACROSS ? p.A[pa] + 2 * m0 : p.A[pa] + m0 * p.lda[pa];
    const unsigned char* bbase[BQ];
    unsigned aoff[AQ], boff[BQ];
    int akk[AQ], bkk[BQ];
#pragma unroll
    for (int u = 0; u < AQ; ++u) {
        if constexpr (T::A_ACROSS)
            aoff[u] = across(u, std::integral_constant<int, BM>{}, mlast, p.lda[pa], akk[u]);
        else
            aoff[u] = along(u, min(8 * u + (lane >> 3), mlast), p.lda[pa], akk[u]);
    }
#pragma unroll
    for (int u = 0; u < BQ; ++u) {
        if constexpr (T::B_ACROSS) {
            bbase[u] = p.B[0] + 2 * n0;
            boff[u] = across(u, std::integral_constant<int, BN>{}, nlast, p.ldb[0], bkk[u]);
        } else {
            int m = 0, row = 8 * u;
            if constexpr (T::GATED) gated_row<T>(row, m, row);
            bbase[u] = p.B[m] + n0 * p.ldb[m];
            boff[u] = along(u, min(row + (lane >> 3), nlast), p.ldb[m], bkk[u]);
        }
    }
    // Stage i of this wave into its place of the ring.
    auto request = [&](int i) __attribute__((always_inline)) {
        const int s = i * kSplit + wave;
        const int pair = T::PAIRS == 2 && s >= each ? 1 : 0;
        const long long k = stage_k<T::PAIRS>(s, each, pair) * (long long)KST;
        const unsigned char* const a = abase + (T::A_ACROSS ? k * p.lda[pa] : k * ES) + (pair ? p.A[1] - p.A[0] : 0);
        const long long b = (T::B_ACROSS ? k * p.ldb[0] : k * ES) + (pair ? p.B[1] - p.B[0] : 0);
        const unsigned to = ring + (unsigned)(i % RING * STAGE);
        if (s == 0 && left < KST) {   // lanes past K copy zeros
            const unsigned char* const zero = reinterpret_cast<const unsigned char*>(&kZero16);
#pragma unroll
            for (int u = 0; u < AQ; ++u)
                lds_dma16(akk[u] < left ? a + aoff[u] : zero, __builtin_amdgcn_readfirstlane(to + 1024u * u));
#pragma unroll
            for (int u = 0; u < BQ; ++u)
                lds_dma16(bkk[u] < left ? bbase[u] + b + boff[u] : zero,
                          __builtin_amdgcn_readfirstlane(to + A_BYTES + 1024u * u));
        } else {
#pragma unroll
            for (int u = 0; u < AQ; ++u) lds_dma16s(a, aoff[u], __builtin_amdgcn_readfirstlane(to + 1024u * u));
#pragma unroll
            for (int u = 0; u < BQ; ++u)
                lds_dma16s(bbase[u] + b, boff[u], __builtin_amdgcn_readfirstlane(to + A_BYTES + 1024u * u));
        }
    };
    uint4 a[4][FM], b[4][FN];
    auto read = [&](int i) __attribute__((always_inline)) {
        const unsigned char* const st = lds + wave * MINE + i % RING * STAGE;
        auto line = [&](int r, int h) { return (r + li) * 128 + 16 * ((4 * g + h) ^ line_at(li)); };
#pragma unroll
        for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                if constexpr (T::A_ACROSS)
                    a[h][j] = read_across<BM>(st + across_at<BM, 32>(0, j, h, lane));
                else
                    a[h][j] = *reinterpret_cast<const uint4*>(st + line(32 * j, h));
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (T::B_ACROSS)
                    b[h][j] = read_across<BN>(st + A_BYTES + across_at<BN, 32>(0, j, h, lane));
                else
                    b[h][j] = *reinterpret_cast<const uint4*>(st + A_BYTES + line(32 * j, h));
            }
        }
        // the stage is in registers: its place is free
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    acc_of<T::E> acc[FM][FN] = {};
    auto multiply = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma<T::E>(a[h][i], b[h][j], acc[i][j]);
    };
#pragma unroll
    for (int i = 0; i < RING; ++i)
        if (i < mine) request(i);
    if constexpr (!T::A_ACROSS && !T::B_ACROSS)
        if (wave == 0 && left * ES % 16 != 0) {   // K ends within 16 bytes
            wait_loads<0>();
            if (lane < BM) clear_behind(lds, lane, left * ES);
            if (lane < BN) clear_behind(lds + A_BYTES, lane, left * ES);
            lane_order();
        }
    int i = 0;
    for (; i + RING < mine; ++i) {
        wait_loads<(RING - 1) * NDMA>();
        read(i);
        request(i + RING);
        __builtin_amdgcn_sched_barrier(0);
        multiply();
    }
    wait_loads<0>();
    for (; i < mine; ++i) {
        read(i);
        multiply();
    }
    float* const part = reinterpret_cast<float*>(lds + wave * MINE);
    lane_order();
    static_for<FM>([&](auto m) __attribute__((always_inline)) { put_rows<T>(acc[m], part + m * 32 * T::STR, li, g); });
    __syncthreads();
    // a thread has the same eight columns in every row of its
    constexpr int UNITS = T::COLS / 8, STEP = 64 * kSplit / UNITS;
    const int u = threadIdx.x % UNITS;
    const long long at = n0 + 8 * u;
    const int n = (int)min(p.N - at, 8ll);
    if (n <= 0) return;
    Scales8 s;
    load_scales<T>(p, at, n, s);
    for_act<T>(p, [&](auto act) __attribute__((always_inline)) {
        for (int row = threadIdx.x / UNITS; row < min(BM, mlast + 1); row += STEP) {
            const long long R = m0 + row;
            const float sa = T::E == Elem::i8 && p.K > 0 ? p.SA[R] : 0.f;
            float x[8], y[8];
            auto sum = [&](float (&v)[8], int c) __attribute__((always_inline)) {
                const unsigned char* const from = lds + 4 * (row * T::STR + c);
                __builtin_memcpy(v, from, 32);
#pragma unroll
                for (int w = 1; w < kSplit; ++w) {
                    float z[8];
                    __builtin_memcpy(z, from + w * MINE, 32);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if constexpr (T::E == Elem::i8)
                            v[e] = __int_as_float(__float_as_int(v[e]) + __float_as_int(z[e]));
                        else
                            v[e] += z[e];
                    }
                }
            };
            sum(x, 8 * u);
            if constexpr (T::GATED) sum(y, T::COLS + 8 * u);
            finish8<T, act>(p, out, R, at, n, sa, s, x, y);
        }
    });
}

template <class T, int RING>
hipError_t launch_split(const LayerArgs& a, hipStream_t s) {
    const long long tm = ((long long)a.M + T::BM - 1) / T::BM, tn = ((long long)a.N + T::COLS - 1) / T::COLS;
    if (tm * tn * T::OUTS * 64 * kSplit > 0xFFFFFFFFll) return hipErrorInvalidValue;
    split_kernel<T, RING><<<(unsigned)(tm * tn * T::OUTS), 64 * kSplit, 0, s>>>(a, (int)tm, (int)tn);
    return hipGetLastError();
}

// A product's tiles.  32 x 64 or 64 x 64 with divided k where they fit one round of
// workgroups, one to a CU, the latter also two rounds of them (but for a single
// row of tiles, which memory bounds: gated bf16 64 x 16384 x 4096 88 us, 65 in 128 x
// 128); else 128 x 128 up to two to a CU or up to eight stages, where filling and
// draining a tile takes longer than its products (us, 128 x 128 and 256 x 256: int8
// 2096 x 12416 x 1024 40 and 47, x 2048 73 and 69; gated bf16 2096 x 12416 x 128 39
// and 48, x 512 73 and 77, x 1024 125 and 120), and 256 x 256 beyond, but where a
// second round of those would be a quarter full (1.06 rounds: int8 4352 x 4096 x 4096
// 97 and 109, gated bf16 4352 x 2048 x 4096 167 and 178; 1.25: 99 and 113, 173 and
// 184, dW 190 and 186; 1.5: 116 and 118, 203 and 193).  us, K = 4096 (the
// next larger choice in brackets; 8-bit operands from the last-level cache): int8 64
// x 4096 7.5 (9.6), 128 x 4096 9.6 (22), 512 x 4096 19 (22), 1024 x 4096 23 (49);
// gated bf16 64 x 4096 19 (24), 128 x 4096 23 (54), 512 x 2048 35 (51), 1024 x 4096 73
// (92), 1024 x 8192 147 and 111; dX 512 x 4096 69 (100).
// Rows off 16 bytes go through registers, in 64 x 64 (gated: x 128) products where
// 128 x 128 would leave a third of the CUs idle (us, small and large: int8 1000 x
// 1500 x 777 12.2 and 14.7, its dW 20 and 22, dX 26 and 34; the gated form of 192
// tiles 21.5 and 18.9; 2047^3 int8 35 and 25, dX 113 and 75).  The gradients' small
// tiles have two groups of waves for alternate stages where there are 12 and no
// more than two workgroups to a CU (us, one group and two: dX 1000 x 777 x 1500 35
// and 25.5, 70 x 4095 x 4093 91 and 72, of 544 tiles 70.5 and 75; dW 70 x 4095 x
// 4093 46 and 34, of 768 tiles 20 and 22).  Half as large, with two groups (dX:
// four), where those fit one to a CU and there are stages for them: fewer bytes to
// a CU (us, without and with: int8 70 x 4095 x 4093 20 and 15.6, gated bf16 59 and
// 40, 100 x 1001 x 1003 15.7 and 11.8, 300 x 500 x 333 8.5 and 7.2; dX 172 x 2207 x
// 3981 65 and 57, 399 x 82 x 5485 76 and 57; dW of 200 and more gains nothing).
template <Form F, Elem E, Elem OUT>
hipError_t launch_form(const LayerArgs& a, hipStream_t s) {
    using Wide = Tile<F, E, OUT, 256, 256, 128, 128, 4>;
    using Mid = Tile<F, E, OUT, 128, 128, 64, 64>;
    constexpr bool G = F == Form::gated;
    auto tiles = [&](auto t) {
        using T = decltype(t);
        return ((long long)a.M + T::BM - 1) / T::BM * (((long long)a.N + T::COLS - 1) / T::COLS) * T::OUTS;
    };
    if (!big_fits<Mid>(a)) {
        using Small = Tile<F, E, OUT, 64, G ? 128 : 64, 32, G ? 64 : 32>;
        if (!rows_of_16<Mid>(a)) return launch_tiles<Small>(tile_kernel<Small, true>, a, s);
        if constexpr (F != Form::both) {
            using Half = Tile<F, E, OUT, G ? 64 : 32, 64, 32, G ? 64 : 32>;
            constexpr int KS = Half::PAIRS == 2 ? 4 : 2;
            if (tiles(Half{}) <= a.cus && Half::PAIRS * (long long)a.K >= (Half::PAIRS == 2 ? 12 : 4) * 2 * Half::KST)
                return launch_tiles<Half, KS>(tile_kernel<Half, false, KS>, a, s);
        }
        if (3 * tiles(Mid{}) <= 2ll * a.cus) {
            if constexpr (Small::B_ACROSS)
                if (tiles(Small{}) <= 2ll * a.cus && Small::PAIRS * (long long)a.K >= 12 * 2 * Small::KST)
                    return launch_tiles<Small, 2>(tile_kernel<Small, false, 2>, a, s);
            return launch_tiles<Small>(tile_kernel<Small, false>, a, s);
        }
        return launch_tiles<Mid>(tile_kernel<Mid, false>, a, s);
    }
    using S32 = Tile<F, E, OUT, 32, 64, 32, 64>;
    using S64 = Tile<F, E, OUT, 64, 64, 64, 64>;
    if (tiles(S32{}) <= a.cus) return launch_split<S32, 2>(a, s);
    if (tiles(S64{}) <= (a.M > 64 ? 2ll : 1ll) * a.cus) return launch_split<S64, 2>(a, s);
    const long long wide = tiles(Wide{});
    if (tiles(Mid{}) <= 2ll * a.cus || Wide::PAIRS * (long long)a.K <= 8 * 2 * Wide::KST ||
        (wide > a.cus && 4 * wide <= 5ll * a.cus))
        return launch_tiles<Mid>(big_kernel<Mid>, a, s);
    return launch_tiles<Wide>(big_kernel<Wide>, a, s);
}

}  // namespace layer
#endif
}  // namespace sgemm
