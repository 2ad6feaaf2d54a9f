// layer_rows.h -- products A.B^T of the feed-forward layer for few rows of A (a
// token, or a batch of them in decoding): the weights are streamed once.
//
// Bound by memory: all there is to read are B's rows.  A workgroup owns 16 NT
// columns of C (in the gated form of both matrices); its waves take spans of
// 64 SP bytes of k in turn, each with the next span's operands on their way while
// it multiplies one, and their parts are added in LDS at the end, in wave order.
//
// The matrix instructions take 16 bytes of row l % 16 of each operand from lane
// l, 64 bytes of k together (v_mfma_f32_16x16x32, v_mfma_i32_16x16x64_i8), and
// both operands come from memory that way: an instruction reads 64 neighbouring
// bytes of 16 rows.  B's rows go first, so that a lane holds four neighbouring
// columns of one row of C.
#pragma once

#include "layer.h"

namespace sgemm {
#ifdef __HIPCC__
namespace layer {

template <Elem E>
using part_of = std::conditional_t<E == Elem::i8, intx4, mx_f4>;

template <Elem E>
__device__ __forceinline__ part_of<E> mfma_row(uint4 b, uint4 a, part_of<E> c) {
    if constexpr (E == Elem::i8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, b), __builtin_bit_cast(intx4, a), c, 0,
                                                     0, 0);
    else if constexpr (E == Elem::bf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, b), __builtin_bit_cast(bf8, a), c, 0, 0,
                                                       0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, b), __builtin_bit_cast(half8, a), c, 0,
                                                      0, 0);
}

// MT: 16-row pieces of A.
template <Form F, Elem E, Elem OUT, int MT, int NT, int NW, int SP>
__global__ __launch_bounds__(64 * NW, MT == 1 ? 4 : 2) void rows_kernel(LayerArgs p) {
    constexpr bool GATED = F == Form::gated;
    constexpr int MATS = GATED ? 2 : 1, ES = size_of<E>, SPAN = 64 * SP;
    typedef part_of<E> Part;
    __shared__ __attribute__((aligned(16))) Part parts[NW][MATS * MT * NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, g = lane >> 4;
    const long long n0 = (long long)blockIdx.x * (16 * NT);
    const int nlast = (int)min((long long)p.N - 1 - n0, 16ll * NT - 1);   // rows past B's last read it again
    const long long len = (long long)p.K * ES;
    const unsigned char* bbase[MATS];
    unsigned ob[MATS][NT], oa[MT];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
        bbase[m] = p.B[m] + n0 * p.ldb[m];
#pragma unroll
        for (int j = 0; j < NT; ++j) ob[m][j] = (unsigned)min(16 * j + li, nlast) * (unsigned)p.ldb[m] + 16u * g;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) oa[i] = (unsigned)(16 * i + li) * (unsigned)p.lda[0] + 16u * g;

    struct Span {
        uint4 b[MATS][NT][SP], a[MT][SP];
    };
    // Rows past A's last are not read: what their lanes hold reaches only outputs
    // that do not exist.
    auto load = [&](Span& t, long long k) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < SP; ++h)
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j) __builtin_memcpy(&t.b[m][j][h], bbase[m] + k + 64 * h + ob[m][j], 16);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            if (16 * i + li < p.M) {
#pragma unroll
                for (int h = 0; h < SP; ++h) __builtin_memcpy(&t.a[i][h], p.A[0] + k + 64 * h + oa[i], 16);
            }
    };
    // The span that the rows end in: zeros behind them.
    auto load_end = [&](Span& t, long long k) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < SP; ++h)
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    t.b[m][j][h] = mx_bytes16(bbase[m] + (ob[m][j] - 16u * g), k + 64 * h + 16 * g, len);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            if (16 * i + li < p.M) {
#pragma unroll
                for (int h = 0; h < SP; ++h)
                    t.a[i][h] = mx_bytes16(p.A[0] + (oa[i] - 16u * g), k + 64 * h + 16 * g, len);
            }
    };
    Part acc[MATS][MT][NT] = {};
    auto multiply = [&](const Span& t) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < SP; ++h)
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[m][i][j] = mfma_row<E>(t.b[m][j][h], t.a[i][h], acc[m][i][j]);
    };
    const int spans = (int)(len / SPAN);   // whole ones
    Span cur, next;
    if (wave < spans) load(cur, (long long)wave * SPAN);
    for (int i = wave; i < spans; i += NW) {
        if (i + NW < spans) load(next, (long long)(i + NW) * SPAN);
        multiply(cur);
        cur = next;
    }
    if (spans % NW == wave && (long long)spans * SPAN < len) {
        load_end(cur, (long long)spans * SPAN);
        multiply(cur);
    }
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) parts[wave][(m * MT + i) * NT + j][lane] = acc[m][i][j];
    __syncthreads();
    // A wave to each 16 x 16 piece of C: a lane has row li, columns 4g .. 4g + 3.
    for (int t = wave; t < MT * NT; t += NW) {
        const long long row = 16 * (t / NT) + li, col = n0 + 16 * (t % NT) + 4 * g;
        const int n = (int)min(p.N - col, 4ll);
        if (row >= p.M || n <= 0) continue;
        float x[4], y[4];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            Part v = parts[0][m * MT * NT + t][lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) v += parts[w][m * MT * NT + t][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float f = (float)v[e];
                if constexpr (E == Elem::i8) f = p.K > 0 ? f * p.SA[row] * p.SB[m][col + min(e, n - 1)] : 0.f;
                (m ? y : x)[e] = f;
            }
        }
        typedef type_of<OUT> O;
        auto store = [&](void* C, long long ldc, const float (&v)[4]) __attribute__((always_inline)) {
            O* const c = static_cast<O*>(C) + row * ldc + col;
            const O o[4] = {(O)v[0], (O)v[1], (O)v[2], (O)v[3]};
            if (n == 4) {
                __builtin_memcpy(c, o, sizeof(o));
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (e < n) c[e] = o[e];
            }
        };
        if constexpr (GATED) {
            if constexpr (E != Elem::i8)
                if (p.G != nullptr) {
                    store(p.G, p.ldg, x);
                    store(p.U, p.ldu, y);
                }
            with_act(p.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = act_of<a>(x[e]) * y[e];
            });
        }
        store(p.C[0], p.ldc[0], x);
    }
}

template <Form F, Elem E, Elem OUT, int MT, int NT, int SP>
hipError_t launch_rows(const LayerArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)(((long long)a.N + 16 * NT - 1) / (16 * NT));
    rows_kernel<F, E, OUT, MT, NT, 8, SP><<<grid, 512, 0, s>>>(a);
    return hipGetLastError();
}

// 16 columns to a workgroup give more of them, 32 read A half as often.  us with
// 16 and 32 columns: int8, one row, 8192 x 8192 15.1 and 19.7, 16384 x 2048 9.2 and
// 8.1; 16 rows 18.9 and 20.7, 11.4 and 8.9; 32 rows 4096 x 4096 8.9 and 10.2, 8192 x
// 8192 25 and 21.5.  Gated bf16, 16 rows, 8192 x 8192 56 and 61, 16384 x 2048 32 and
// 28; 32 rows 4096 x 4096 21 and 26, 8192 x 8192 66 and 58.
template <Form F, Elem E, Elem OUT>
hipError_t launch_few(const LayerArgs& a, hipStream_t s) {
    constexpr int SP = F == Form::gated ? 2 : 4;   // of 32 columns of two matrices: registers
    if (a.M <= 16)
        return a.N < 64 * a.cus ? launch_rows<F, E, OUT, 1, 1, 4>(a, s) : launch_rows<F, E, OUT, 1, 2, SP>(a, s);
    if (a.M <= 32)
        return a.N <= 16 * a.cus ? launch_rows<F, E, OUT, 2, 1, 4>(a, s) : launch_rows<F, E, OUT, 2, 2, 2>(a, s);
    return a.N <= 16 * a.cus ? launch_rows<F, E, OUT, 4, 1, 2>(a, s) : launch_rows<F, E, OUT, 4, 2, 2>(a, s);
}

}  // namespace layer
#endif

// Whether a product takes the kernel above: at most 32 rows, or 64 where rows do
// not begin on 16 bytes or are shorter than a stage of the tiles (else tiles whose
// waves divide k: 64 rows, 8192 x 8192 int8 18.7 us against 28, 4096 x 4096 from the
// last-level cache 7.5 against 12); columns that a launch of 512 threads per 16
// holds; and rows in reach of 32-bit offsets.
inline bool few_rows(const LayerArgs& a, int size, bool gated) {
    auto whole = [&](const void* p, long long ld) { return mx_aligned(p, ld, 16); };
    const bool aligned = whole(a.A[0], a.lda[0]) && whole(a.B[0], a.ldb[0]) && (!gated || whole(a.B[1], a.ldb[1])) &&
                         (long long)a.K * size >= 128;
    return a.M <= (aligned ? 32 : 64) && a.N <= 1 << 26 && mx_dma_reach(a.lda[0], 64) && mx_dma_reach(a.ldb[0], 64) &&
           (!gated || mx_dma_reach(a.ldb[1], 64));
}

}  // namespace sgemm
