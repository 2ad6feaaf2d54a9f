// layer_tile.h -- tile kernels of the feed-forward layer's products on the matrix
// cores, and the epilogue that they share.
//
// One shape serves both element sizes: a matrix instruction of 32 x 32 outputs
// takes 16 bytes of a row of each operand per lane, 16 k in 16 bits
// (v_mfma_f32_32x32x16) and 32 in 8 (v_mfma_i32_32x32x32_i8), in the same number
// of cycles.  A stage is 64 bytes of k (two instructions deep); k terms may come
// in any order, so step t gives lane half h the 16-byte chunk 2h + t.
//
// An operand whose rows run along k lies in LDS as rows of four chunks, chunk c
// of row r at c ^ chunk_at(r).  LDS serves a 16-byte read 16 lanes at a time,
// lanes 0-3, 12-15, 20-23, 24-27 together and lanes 4-11, 16-19, 28-31 together:
// of such rows four share a 64-byte place of the 256-byte window of banks, and
// their chunk_at differ.
//
// An operand of 16-bit elements whose rows run across k lies as 32 k rows of W
// columns, chunk c of row k at c ^ across_swap(k): the four rows that one read
// takes 64 bytes of then lie in the window's four places.  It comes out of LDS
// through the transposing read: within 16 lanes, element e of lane i is element i % 4 of the
// 8 bytes that lane 4e + i / 4 addresses.
//
// The gated form multiplies two matrices by the same rows of A: of a wave's
// columns the first half are rows of the first matrix, the second half the same
// rows of the second, so that both products of an output are in one lane.
#pragma once

#include "layer.h"

namespace sgemm {
#ifdef __HIPCC__
namespace layer {

__device__ __forceinline__ int chunk_at(int r) { return r >> 3 & 3; }
// Four rows of 32 columns fill the window, two of 64, one of 128 and more.
template <int W>
__device__ __forceinline__ int across_swap(int k) { return W == 32 ? 0 : W == 64 ? k << 1 & 4 : (k & 3) << 2; }

template <Elem E>
using acc_of = std::conditional_t<E == Elem::i8, intx16, floatx16>;

template <Elem E>
__device__ __forceinline__ acc_of<E> mfma(uint4 a, uint4 b, acc_of<E> c) {
    if constexpr (E == Elem::i8)
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(intx4, a), __builtin_bit_cast(intx4, b), c, 0,
                                                     0, 0);
    else if constexpr (E == Elem::bf16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0,
                                                       0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0,
                                                      0, 0);
}

template <Form F, Elem E_, Elem OUT_, int BM_, int BN_, int WM_, int WN_, int GROUP_M_ = 8>
struct Tile {
    static constexpr Form FORM = F;
    static constexpr Elem E = E_, OUT = OUT_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, GROUP_M = GROUP_M_;
    static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N, NT = 64 * NW;
    static constexpr int FM = WM / 32, FN = WN / 32;
    static constexpr bool GATED = F == Form::gated;
    static constexpr bool A_ACROSS = F == Form::both, B_ACROSS = F == Form::sum2 || F == Form::both;
    static constexpr int ES = size_of<E>, KST = 64 / ES;          // k of a stage
    static constexpr int SA = BM * 64, SB = BN * 64;              // bytes of 64 of k
    static constexpr int COLS = GATED ? BN / 2 : BN;              // columns of C
    static constexpr int PAIRS = F == Form::sum2 ? 2 : 1;
    static constexpr int OUTS = F == Form::both ? 2 : 1;
    // the epilogue's rows: 32 of WN values, rows four apart in the other half of the banks
    static constexpr int STR = WN + 8;
    static constexpr int EPI = NW * (32 * STR + WM + WN) * 4;     // bytes, with the scales
    static_assert(4 * STR % 64 == 32, "rows four apart");
    static_assert(!GATED || WN % 64 == 0, "two halves of whole blocks");
};

// The scales of eight columns from `at` on, n (1 and up) of them in the matrix.
struct Scales8 {
    float x[8], y[8];
};
template <class T>
__device__ __forceinline__ void load_scales(const LayerArgs& p, long long at, int n, Scales8& s) {
    if constexpr (T::E == Elem::i8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const long long c = at + min(e, n - 1);
            s.x[e] = p.K > 0 ? p.SB[0][c] : 0.f;
            if constexpr (T::GATED) s.y[e] = p.K > 0 ? p.SB[1][c] : 0.f;
        }
    }
}
// Eight neighbouring outputs of row R from column `at` on, n (1 and up) of them
// in the matrix: the sums x (whole numbers in the registers of floats where the
// operands are), in the gated form the second matrix's in y.
template <class T, int ACT>
__device__ __forceinline__ void finish8(const LayerArgs& p, int out, long long R, long long at, int n, float sa,
                                        const Scales8& s, float (&x)[8], float (&y)[8]) {
    typedef type_of<T::OUT> O;
    if constexpr (T::E == Elem::i8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = (float)__float_as_int(x[e]) * sa * s.x[e];
            if constexpr (T::GATED) y[e] = (float)__float_as_int(y[e]) * sa * s.y[e];
        }
    }
    if constexpr (T::GATED) {
        if constexpr (T::E != Elem::i8)
            if (p.G != nullptr) {
                store8<T::OUT>(static_cast<O*>(p.G) + R * p.ldg + at, x, n);
                store8<T::OUT>(static_cast<O*>(p.U) + R * p.ldu + at, y, n);
            }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = act_of<ACT>(x[e]) * y[e];
    }
    store8<T::OUT>(static_cast<O*>(p.C[out]) + R * p.ldc[out] + at, x, n);
}
// f(integral_constant of the activation), none where there is no gate.
template <class T, class F>
__device__ __forceinline__ void for_act(const LayerArgs& p, F&& f) {
    if constexpr (T::GATED)
        with_act(p.act, f);
    else
        f(std::integral_constant<int, 0>{});
}

// A 32-row piece of accumulators to LDS, rows STR words apart.
template <class T, class Acc>
__device__ __forceinline__ void put_rows(const Acc (&acc)[T::FN], float* to, int li, int g) {
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const auto v = acc[j][r];   // (a bit cast of the element itself would take the vector's first)
            to[(8 * (r / 4) + 4 * g + r % 4) * T::STR + 32 * j + li] = __builtin_bit_cast(float, v);
        }
}

// A wave's outputs from its accumulators: 32 rows at a time through LDS (mine:
// 32 STR + WM + WN words of the wave's own), so that a lane has eight neighbouring
// columns and stores them whole.  r0, c0: the first row and column of C.  The
// scales come to LDS before the first row: loaded row by row they cost 8192^3
// int8 40 us.
template <class T, class Acc>
__device__ __forceinline__ void epilogue(const LayerArgs& p, int out, const Acc (&acc)[T::FM][T::FN], float* lds,
                                         int wave, long long r0, long long c0, int lane) {
    constexpr int WCOLS = T::GATED ? T::WN / 2 : T::WN;   // columns of C in a wave
    constexpr int UNITS = WCOLS / 8, STEP = 64 / UNITS;
    float *const mine = lds + wave * (32 * T::STR + T::WM + T::WN), *const row_scales = mine + 32 * T::STR,
                *const col_scales = row_scales + T::WM;
    const int u = lane % UNITS, row0 = lane / UNITS;
    const long long at = c0 + 8 * u;
    const int n = (int)min(p.N - at, 8ll);
    if constexpr (T::E == Elem::i8) {
        if (p.K > 0) {
            for (int r = lane; r < T::WM; r += 64) row_scales[r] = p.SA[min(r0 + r, (long long)p.M - 1)];
            for (int c = lane; c < T::WN; c += 64) {
                const int m = T::GATED ? c / WCOLS : 0;
                col_scales[c] = p.SB[m][min(c0 + c - m * WCOLS, (long long)p.N - 1)];
            }
        } else {
            for (int r = lane; r < T::WM + T::WN; r += 64) row_scales[r] = 0.f;
        }
    }
    static_for<T::FM>([&](auto i) __attribute__((always_inline)) {
        lane_order();
        put_rows<T>(acc[i], mine, lane & 31, lane >> 5);
        lane_order();
        for_act<T>(p, [&](auto act) __attribute__((always_inline)) {
#pragma unroll 1
            for (int row = row0; row < 32; row += STEP) {
                const long long R = r0 + 32 * i + row;
                if (R >= p.M || n <= 0) continue;
                float x[8], y[8], sa = 0.f;
                Scales8 s;
                const float* const from = mine + row * T::STR + 8 * u;
                __builtin_memcpy(x, from, 32);
                if constexpr (T::GATED) __builtin_memcpy(y, from + WCOLS, 32);
                if constexpr (T::E == Elem::i8) {
                    sa = row_scales[32 * i + row];
                    __builtin_memcpy(s.x, col_scales + 8 * u, 32);
                    if constexpr (T::GATED) __builtin_memcpy(s.y, col_scales + WCOLS + 8 * u, 32);
                }
                finish8<T, act>(p, out, R, at, n, sa, s, x, y);
            }
        });
    });
}

// Where a wave's operand lies in a stage: byte offsets of step t's read of block
// j (32 rows or columns from w on).
__device__ __forceinline__ int along_at(int w, int j, int t, int li, int g) {
    return (w + 32 * j + li) * 64 + 16 * ((2 * g + t) ^ chunk_at(li));
}
// The lower read of two (k .. k + 3 of the lane's eight); the upper is 4 rows on.
// HALF: the k rows of one lane half.
template <int W, int HALF = 16>
__device__ __forceinline__ int across_at(int w, int j, int t, int lane) {
    const int q = lane >> 4, e = (lane >> 2) & 3, n = lane & 3;
    const int k = HALF * (q >> 1) + e + 8 * t, col = w + 32 * j + 16 * (q & 1) + 4 * n;
    return 2 * (k * W + (((col >> 3) ^ across_swap<W>(e)) << 3 | (col & 7)));
}
template <int W>
__device__ __forceinline__ uint4 read_across(const unsigned char* at) {
    const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_shortx4*)(__attribute__((address_space(3))) const unsigned char*)at);
    const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_shortx4*)(__attribute__((address_space(3))) const unsigned char*)(at + 8 * W));
    const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
    return make_uint4(l.x, l.y, h.x, h.y);
}

// Row r of B's tile in the gated form: which matrix, and which row from the
// tile's first on.
template <class T>
__device__ __forceinline__ void gated_row(int r, int& m, int& row) {
    constexpr int H = T::WN / 2;
    m = r / H & 1;
    row = r / T::WN * H + r % H;
}

// Tiles through registers: any alignment, pitch and length.  128 bytes of k at a
// time, in two LDS places: while one multiplies the next AHEAD are on their way,
// and one is written to the other place behind it, so there is one barrier to 128
// bytes.  Latency bounds such launches, so the loads are without branches: a chunk
// that would pass its row's end is the row's last 16 bytes, a k row past K the
// last one, and what that brings is moved down or cleared when it is written to
// LDS.  (With the row's end looked after at the load, every load waits for all
// others: dX of 1000 x 1500 x 777 39 us.)  Loads off 4 bytes come at 37 KB/us to a
// CU, on 4 bytes at up to 97: int8 1000 x 1500 x 777 12.2 us, x 780 9.4.  KS groups
// of waves take every KS-th stage each, in places of their own, and the first adds
// the others' sums to its own, in their order.  TINY: rows of less than 16 bytes,
// loaded by bytes.
template <class T, bool TINY, int KS = 1>
__global__ __launch_bounds__(KS * T::NT, 2) void tile_kernel(LayerArgs p, int tiles_m, int tiles_n) {
    constexpr int BM = T::BM, BN = T::BN, NT = T::NT, FM = T::FM, FN = T::FN, KST = 2 * T::KST;
    constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT;             // a thread's chunks
    static_assert(CA * NT == BM * 8 && CB * NT == BN * 8, "whole rounds of the loader");
    constexpr int AHEAD = CA + CB <= 6 ? 3 : 2;
    constexpr int STAGE = 2 * (T::SA + T::SB), ROOM = 2 * STAGE > T::EPI ? 2 * STAGE : T::EPI;
    static_assert(NT * FM * FN * 64 <= ROOM, "a group's sums in its places");
    __shared__ __attribute__((aligned(16))) unsigned char lds[KS * ROOM];
    const int per = tiles_m * tiles_n;
    const int out = T::OUTS == 2 && (int)blockIdx.x >= per ? 1 : 0;
    int tm, tn;
    tile_coords(blockIdx.x - out * per, tiles_m, tiles_n, T::GROUP_M, p.xcds, tm, tn);
    const int tid = threadIdx.x % NT, lane = tid & 63;
    const int group = __builtin_amdgcn_readfirstlane((int)threadIdx.x / NT);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = (wave / T::WAVES_N) * T::WM, wn = (wave % T::WAVES_N) * T::WN;
    const int li = lane & 31, g = lane >> 5;
    unsigned char* const places = lds + group * ROOM;
    const long long m0 = (long long)tm * BM, n0 = (long long)tn * T::COLS;
    const long long row_bytes = (long long)p.K * T::ES;
    const int each = (int)(((long long)p.K + KST - 1) / KST), stages = each * T::PAIRS;

    // The thread's chunk u of an operand.  Along k: a row and 16 bytes of the stage's
    // 128; rows past a matrix are its last one, their products are not stored.
    // Across: a k row of the stage and 16 bytes of a row.
    auto a_row = [&](int u, long long ld) { return min(m0 + ((tid + u * NT) >> 3), (long long)p.M - 1) * ld; };
    auto across_col = [&](int u, int W, long long first) { return 2 * first + 16 * ((tid + u * NT) % (W / 8)); };
    auto across_k = [&](int u, int W) { return (tid + u * NT) / (W / 8); };
    long long arow[CA], brow[CB];           // bytes to the chunk's row, across to its columns
#pragma unroll
    for (int u = 0; u < CA; ++u)
        arow[u] = T::A_ACROSS ? min(across_col(u, BM, m0), 2ll * p.M - (TINY ? 0 : 16)) : a_row(u, p.lda[0]);
#pragma unroll
    for (int u = 0; u < CB; ++u) {
        int m = 0, row = (tid + u * NT) >> 3;
        if constexpr (T::GATED) gated_row<T>(row, m, row);
        if constexpr (T::B_ACROSS)
            brow[u] = min(across_col(u, BN, n0), 2ll * p.N - (TINY ? 0 : 16));
        else
            brow[u] = (m ? p.B[1] - p.B[0] : 0) + min(n0 + row, (long long)p.N - 1) * (m ? p.ldb[1] : p.ldb[0]);
    }
    // Where the last whole 16 bytes of a row begin, from k0 on (before it, maybe).
    auto last_chunk = [&](int k0) { return (int)min(row_bytes - (long long)k0 * T::ES, 1024ll) - 16; };
    // Columns past the matrix: chunks to be moved down.
    const bool a_edge = T::A_ACROSS && m0 + BM > p.M, b_edge = T::B_ACROSS && n0 + BN > p.N;
    uint4 wait_a[AHEAD][CA], wait_b[AHEAD][CB];
    auto fetch = [&](int s, auto slot) __attribute__((always_inline)) {
        uint4(&va)[CA] = wait_a[slot];
        uint4(&vb)[CB] = wait_b[slot];
        const int pair = T::PAIRS == 2 && s >= each ? 1 : 0;
        const int k0 = (s - pair * each) * KST;
        const int ma = T::OUTS == 2 ? out : pair;
        const unsigned char *const A = p.A[ma], *const B = p.B[pair];
        const long long lda = p.lda[ma], ldb = p.ldb[pair];
        const long long start = (long long)k0 * T::ES;
        const int end = last_chunk(k0);
        auto along = [&](const unsigned char* row, int u) __attribute__((always_inline)) {
            const int at = 16 * ((tid + u * NT) & 7);
            if constexpr (TINY) return mx_bytes16(row, start + at, row_bytes);
            uint4 v;
            __builtin_memcpy(&v, row + start + min(at, end), 16);
            return v;
        };
        auto across = [&](const unsigned char* M, long long ld, int k, long long col, int cols) __attribute__((always_inline)) {
            const unsigned char* const row = M + min((unsigned)k0 + k, (unsigned)p.K - 1) * ld;
            if constexpr (TINY) return mx_bytes16(row, col, 2ll * cols);
            uint4 v;
            __builtin_memcpy(&v, row + col, 16);
            return v;
        };
#pragma unroll
        for (int u = 0; u < CA; ++u) {
            if constexpr (T::A_ACROSS)
                va[u] = across(A, lda, across_k(u, BM), arow[u], p.M);
            else
                va[u] = along(A + (T::PAIRS == 2 ? a_row(u, lda) : arow[u]), u);
        }
#pragma unroll
        for (int u = 0; u < CB; ++u) {
            if constexpr (T::B_ACROSS)
                vb[u] = across(B, ldb, across_k(u, BN), brow[u], p.N);
            else
                vb[u] = along(B + brow[u], u);
        }
    };
    auto place = [&](int s, int turn, auto slot) __attribute__((always_inline)) {
        unsigned char* const to = places + (turn & 1) * STAGE;
        const int st = T::PAIRS == 2 && s >= each ? s - each : s;
        const int left = p.K - st * KST;   // k of the stage
        auto put = [](unsigned char* at, uint4 v) {
            lds_poison_f4(at);
            *reinterpret_cast<uint4*>(at) = v;
        };
        // v without its first n bytes, zeros behind them
        auto down = [](uint4 v, unsigned n) {
            const uint4 d = mx_down(v, (int)min(max(n, 1u), 16u));
            return n == 0 ? v : d;
        };
        // 64 bytes of k behind the others
        auto along = [](int id, int S) { return (id >> 2 & 1) * S + (id >> 3) * 64 + 16 * ((id & 3) ^ chunk_at(id >> 3)); };
        auto across = [](int id, auto W) {
            return id / (W / 8) * (2 * W) + 16 * (id % (W / 8) ^ across_swap<W>(id / (W / 8)));
        };
        // The last stage, and tiles at the edge: what the loads brought from elsewhere.
        auto along_end = [&](uint4& v, int u) __attribute__((always_inline)) {
            const int at = 16 * ((tid + u * NT) & 7);
            if constexpr (!TINY) v = down(v, (unsigned)(at - min(at, last_chunk(st * KST))));
        };
        auto across_end = [&](uint4& v, int u, int W, long long first, long long col) __attribute__((always_inline)) {
            if constexpr (!TINY) v = down(v, (unsigned)(across_col(u, W, first) - col));
            if (across_k(u, W) >= left) v = make_uint4(0u, 0u, 0u, 0u);
        };
        uint4(&va)[CA] = wait_a[slot];
        uint4(&vb)[CB] = wait_b[slot];
        if (left < KST || a_edge) {
#pragma unroll
            for (int u = 0; u < CA; ++u) {
                if constexpr (T::A_ACROSS)
                    across_end(va[u], u, BM, m0, arow[u]);
                else
                    along_end(va[u], u);
            }
        }
        if (left < KST || b_edge) {
#pragma unroll
            for (int u = 0; u < CB; ++u) {
                if constexpr (T::B_ACROSS)
                    across_end(vb[u], u, BN, n0, brow[u]);
                else
                    along_end(vb[u], u);
            }
        }
#pragma unroll
        for (int u = 0; u < CA; ++u) {
            const int id = tid + u * NT;
            put(to + (T::A_ACROSS ? across(id, std::integral_constant<int, BM>{}) : along(id, T::SA)), va[u]);
        }
#pragma unroll
        for (int u = 0; u < CB; ++u) {
            const int id = tid + u * NT;
            put(to + 2 * T::SA + (T::B_ACROSS ? across(id, std::integral_constant<int, BN>{}) : along(id, T::SB)), vb[u]);
        }
    };

    acc_of<T::E> acc[FM][FN] = {};
    auto multiply = [&](int buf) __attribute__((always_inline)) {
        const unsigned char* const st = places + buf * STAGE;
        static_for<4>([&](auto h) __attribute__((always_inline)) {
            constexpr int t = h % 2;
            const unsigned char *const sa = st + h / 2 * T::SA, *const sb = st + 2 * T::SA + h / 2 * T::SB;
            uint4 a[FM], b[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (T::A_ACROSS)
                    a[i] = read_across<BM>(sa + across_at<BM>(wm, i, t, lane));
                else
                    a[i] = *reinterpret_cast<const uint4*>(sa + along_at(wm, i, t, li, g));
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                if constexpr (T::B_ACROSS)
                    b[j] = read_across<BN>(sb + across_at<BN>(wn, j, t, lane));
                else
                    b[j] = *reinterpret_cast<const uint4*>(sb + along_at(wn, j, t, li, g));
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma<T::E>(a[i], b[j], acc[i][j]);
        });
    };
    // The group's turn i is stage KS i + group; it waits in registers at i % AHEAD
    // until it is placed.  Past the last stage that one is loaded again: the loads
    // stay without branches.
    constexpr std::integral_constant<int, 0> none{};
    if (stages > 0) {
        const int turns = (stages + KS - 1) / KS;   // of all groups, for the barriers
        auto stage_of = [&](int i) { return KS * i + group; };
        auto bring = [&](int i, auto slot) __attribute__((always_inline)) {
            fetch(min(stage_of(i), stages - 1), slot);
        };
        auto lay = [&](int i, auto slot) __attribute__((always_inline)) {
            if (stage_of(i) < stages) place(stage_of(i), i, slot);
        };
        static_for<AHEAD>([&](auto i) __attribute__((always_inline)) { bring(i, i); });
        lay(0, none);
        bring(AHEAD, none);
        __syncthreads();
        auto turn = [&](int i, auto d) __attribute__((always_inline)) {
            constexpr std::integral_constant<int, (d + 1) % AHEAD> next{};
            lay(i + 1, next);   // where turn i - 1 was read
            bring(i + 1 + AHEAD, next);
            if (KS == 1 || stage_of(i) < stages) multiply(i & 1);
            __syncthreads();
        };
        int i = 0;
        for (;;) {
            turn(i, std::integral_constant<int, 0>{});
            if (++i == turns) break;
            turn(i, std::integral_constant<int, 1 % AHEAD>{});
            if (++i == turns) break;
            if constexpr (AHEAD == 3) {
                turn(i, std::integral_constant<int, 2>{});
                if (++i == turns) break;
            }
        }
    }
    if constexpr (KS > 1) {   // the other groups' sums, in their order
        auto slot = [&](int of, int q) { return reinterpret_cast<uint4*>(lds + of * ROOM) + q * NT + tid; };
        if (group > 0) {
#pragma unroll
            for (int q = 0; q < FM * FN * 4; ++q) {
                uint4 v;
                unsigned w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const auto x = acc[q / 4 / FN][q / 4 % FN][q % 4 * 4 + e];
                    w[e] = __builtin_bit_cast(unsigned, x);
                }
                v = make_uint4(w[0], w[1], w[2], w[3]);
                *slot(group, q) = v;
            }
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int of = 1; of < KS; ++of)
#pragma unroll
            for (int q = 0; q < FM * FN * 4; ++q) {
                const uint4 v = *slot(of, q);
                const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    using V = std::conditional_t<T::E == Elem::i8, int, float>;
                    acc[q / 4 / FN][q / 4 % FN][q % 4 * 4 + e] += __builtin_bit_cast(V, w[e]);
                }
            }
    }
    epilogue<T>(p, out, acc, reinterpret_cast<float*>(lds), wave, m0 + wm, n0 + (T::GATED ? wn / 2 : wn), lane);
}

// Whether every row that the kernel above reads has 16 bytes.
template <class T>
inline bool rows_of_16(const LayerArgs& a) {
    const bool along = (long long)a.K * T::ES >= 16;
    return (T::A_ACROSS ? a.M >= 8 : along) && (T::B_ACROSS ? a.N >= 8 : along);
}

// One workgroup per tile; more threads than a launch holds are refused by the
// argument checks.
template <class T, int KS = 1, class K>
hipError_t launch_tiles(K kernel, const LayerArgs& a, hipStream_t s) {
    const long long tm = ((long long)a.M + T::BM - 1) / T::BM, tn = ((long long)a.N + T::COLS - 1) / T::COLS;
    if (tm * tn * T::OUTS * KS * T::NT > 0xFFFFFFFFll) return hipErrorInvalidValue;
    kernel<<<(unsigned)(tm * tn * T::OUTS), KS * T::NT, 0, s>>>(a, (int)tm, (int)tn);
    return hipGetLastError();
}

}  // namespace layer
#endif
}  // namespace sgemm
