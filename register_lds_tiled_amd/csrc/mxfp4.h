// mxfp4.h -- internal declarations of the MXFP4 kernels: arguments after
// validation, launchers, and the device helpers that all of them use.
//
// A block is 32 consecutive elements of a row: 16 bytes of codes and one
// scale byte.  gfx950's conversions take the scale as a float of which only
// the exponent counts: the scale byte moved to bits 30:23.  Byte 0 so acts as
// 2^-127 and byte 255 as NaN, exactly as the format says (checked on the GPU
// over every 16-bit input pattern, the ties of every element at scales from
// 2^-127 to 2^125, and all 256 bytes of codes).
#pragma once

#include <hip/hip_runtime.h>

#include <cstring>

#include "lds_dma.h"
#include "tiles.h"

namespace sgemm {

enum class MxType { f32, bf16, f16, mxfp4 };

// X (R x C) -> Q, S along rows and/or QT, ST along columns (null: not asked).
struct MxQuantArgs {
    int R, C;
    const void* X;
    long long ldx;
    unsigned char* Q;
    long long ldq;
    unsigned char* S;
    long long lds;
    unsigned char* QT;
    long long ldqt;
    unsigned char* ST;
    long long ldst;
    int cus = 256, xcds = 8;
};
struct MxDequantArgs {
    int R, C;
    const unsigned char* Q;
    long long ldq;
    const unsigned char* S;
    long long lds;
    void* Y;
    long long ldy;
};
// C = A.B^T.  MXFP4 A: SA and ldsa its scales; 16-bit A: lda in elements.
struct MxGemmArgs {
    int M, N, K;
    const unsigned char* A;
    long long lda;
    const unsigned char* SA;
    long long ldsa;
    const unsigned char* B;
    long long ldb;
    const unsigned char* SB;
    long long ldsb;
    void* C;
    long long ldc;
    int cus = 256, xcds = 8;
};

hipError_t launch_mx_quantize(const MxQuantArgs& a, MxType t, hipStream_t s);
hipError_t launch_mx_dequantize(const MxDequantArgs& a, MxType t, hipStream_t s);
// out: f32 or bf16.
hipError_t launch_mx_gemm(const MxGemmArgs& a, MxType out, hipStream_t s);
// t: the type of A, bf16 or f16; C is fp32.
hipError_t launch_mx_wgemm(const MxGemmArgs& a, MxType t, hipStream_t s);

// Both products where mx_few_rows says so; A's type is a_type (mxfp4, bf16 or
// f16); C's type is out (f32, or bf16 where A is mxfp4).
hipError_t launch_mx_rows(const MxGemmArgs& a, MxType a_type, MxType out, hipStream_t s);

inline bool mx_aligned(const void* p, long long ld_bytes, int n) {
    return ((unsigned long long)(size_t)p | (unsigned long long)ld_bytes) % n == 0;
}

#ifdef __HIPCC__
typedef float mx_f2 __attribute__((ext_vector_type(2)));
typedef float mx_f4 __attribute__((ext_vector_type(4)));
typedef __bf16 mx_bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_h2 __attribute__((ext_vector_type(2)));
typedef int mx_i8 __attribute__((ext_vector_type(8)));

// The scale operand of the conversions for a scale byte.
__device__ __forceinline__ float mx_scale(unsigned byte) { return __uint_as_float(byte << 23); }

// v moved down by n bytes (0 and up), zeros above: whole words by selects, the
// bytes between by v_alignbyte.  A 64-bit vector shift by a register must not
// stand here: one whose amount was the last register that the wave owns
// (184 registers, the amount in v183) read v0 instead as soon as another wave
// shared the SIMD, and moved each row by its thread's number.
__device__ __forceinline__ uint4 mx_down(uint4 v, int n) {
    const int w = n >> 2;
    const bool one = w & 1, two = w & 2, all = w > 3;
    unsigned x = one ? v.y : v.x, y = one ? v.z : v.y, z = one ? v.w : v.z, u = one ? 0u : v.w;
    x = two ? z : x;
    y = two ? u : y;
    z = two ? 0u : z;
    u = two ? 0u : u;
    const unsigned b = (unsigned)n & 3u;
    x = __builtin_amdgcn_alignbyte(y, x, b);
    y = __builtin_amdgcn_alignbyte(z, y, b);
    z = __builtin_amdgcn_alignbyte(u, z, b);
    u = __builtin_amdgcn_alignbyte(0u, u, b);
    return all ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(x, y, z, u);
}

// Bytes at .. at + 15 of a row of len, of any alignment: zeros past its end,
// which is not read.  A piece that crosses the row's end is the row's last 16
// bytes moved down; a row of less than 16 is read by bytes.
__device__ __forceinline__ uint4 mx_bytes16(const unsigned char* row, long long at, long long len) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const long long n = len - at;
    if (n >= 16) {
        __builtin_memcpy(&v, row + at, 16);
    } else if (n > 0) {
        unsigned long long lo = 0, hi = 0;
        if (len >= 16) {
            __builtin_memcpy(&v, row + len - 16, 16);
            return mx_down(v, 16 - (int)n);
        } else {
#pragma unroll 1
            for (int i = (int)n; i-- > 0;) {
                hi = hi << 8 | lo >> 56;
                lo = lo << 8 | row[at + i];
            }
        }
        v = make_uint4((unsigned)lo, (unsigned)(lo >> 32), (unsigned)hi, (unsigned)(hi >> 32));
    }
    return v;
}

// v without the high half of its byte n - 1 (1 <= n <= 16): the half that
// belongs to no element where K is odd and the row ends there.
__device__ __forceinline__ uint4 mx_drop_half(uint4 v, long long n) {
    const unsigned m = ~(0xF0u << (8 * ((n - 1) & 3)));
    const int w = (int)(n - 1) >> 2;
    v.x &= w == 0 ? m : ~0u;
    v.y &= w == 1 ? m : ~0u;
    v.z &= w == 2 ? m : ~0u;
    v.w &= w == 3 ? m : ~0u;
    return v;
}

// 16 bytes of codes at byte `at` of a row of K codes that starts at `row`:
// zeros for elements past K, which are not looked at.
__device__ __forceinline__ uint4 mx_codes16(const unsigned char* row, long long at, int K) {
    const long long len = ((long long)K + 1) / 2, left = len - at;
    uint4 v = mx_bytes16(row, at, len);
    if ((K & 1) && left > 0 && left <= 16) v = mx_drop_half(v, left);
    return v;
}

// The same of rows of at least 16 bytes in two steps, so that many loads are on
// their way together: a piece that passes the row's end is the row's last 16 bytes,
// and is moved down, zeros behind it, when it is put to use.  (Each moved down
// where it was loaded, every load of a row's last stage waited for the one before:
// 1000 x 1500 x 777 12.4 us, 11.4 so; with bfloat16 A 17.8 and 17.2.)
__device__ __forceinline__ uint4 mx_load16(const unsigned char* row, long long at, long long len) {
    uint4 v;
    __builtin_memcpy(&v, row + min(at, len - 16), 16);
    return v;
}
__device__ __forceinline__ uint4 mx_end16(uint4 v, long long at, long long len) {
    return mx_down(v, (int)min(max(at - (len - 16), 0ll), 16ll));
}
__device__ __forceinline__ uint4 mx_end_codes16(uint4 v, long long at, int K) {
    const long long len = ((long long)K + 1) / 2, left = len - at;
    v = mx_end16(v, at, len);
    if ((K & 1) && left > 0 && left <= 16) v = mx_drop_half(v, left);
    return v;
}

// N (4 or 8) scale bytes from byte `at` of a row of n: zeros past n.
template <int N>
__device__ __forceinline__ void mx_scales(const unsigned char* row, long long at, long long n,
                                          unsigned (&s)[N / 4]) {
    if (n - at >= N) {
        __builtin_memcpy(s, row + at, N);
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) s[i] = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n - at) s[i / 4] |= (unsigned)row[at + i] << (8 * (i % 4));
    }
}

// A block's 16 bytes of codes without elements `left` and up (left may be
// negative or past 32).
__device__ __forceinline__ uint4 mx_keep(uint4 v, int left) {
    auto word = [&](unsigned w, int i) {
        const int n = left - 8 * i;
        return n >= 8 ? w : n <= 0 ? 0u : w & ((1u << (4 * n)) - 1u);
    };
    return make_uint4(word(v.x, 0), word(v.y, 1), word(v.z, 2), word(v.w, 3));
}

#endif
// The DMA loaders address a tile's rows by 32-bit offsets from its first row.
inline bool mx_dma_reach(long long ld_bytes, int rows) { return ld_bytes * rows < (1ll << 32); }
// Whether a product takes the few-row kernel: at most 16 rows, or at most 64
// where 128 x 128 tiles would leave half the CUs idle (64 rows, K = 8192: N =
// 8192 takes 19 us in the few-row kernel and 34 in tiles, 16128 37 and 36, 24576
// 54 and 41; with bfloat16 A 35 and 63, 69 and 64, 100 and 66); and 64 rows of
// every operand in reach of 32-bit offsets.
inline bool mx_few_rows(const MxGemmArgs& a) {
    return (a.M <= 16 || (a.M <= 64 && 2 * (((long long)a.N + 127) / 128) < a.cus)) && mx_dma_reach(a.lda, 64) &&
           mx_dma_reach(a.ldsa, 64) && mx_dma_reach(a.ldb, 64) && mx_dma_reach(a.ldsb, 64);
}
#ifdef __HIPCC__
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

// v_mfma_scale_f32_16x16x128_f8f6f4 on 4-bit elements: lane l holds 32
// consecutive elements (16 bytes, one block) of row l % 16 of each operand, and
// their scale in byte SEL of one register.  The order of the k terms is free, so
// which blocks the four lane groups l / 16 take together is chosen for the
// memory side.  D: lane l, register i is row 4 (l / 16) + i of the first operand,
// row l % 16 of the second; B's rows go first, so a lane holds four neighbouring
// columns of one row of C.  (Layout, scale bytes 0 and 255 and the accuracy
// checked on the GPU: within 2.5e-8 sum |a b| of the exact sum of 128 terms.)
template <int SEL>
__device__ __forceinline__ mx_f4 mfma_mx(uint4 b, unsigned sb, uint4 a, unsigned sa, mx_f4 acc) {
    const mx_i8 bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    const mx_i8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, av, acc, 4, 4, SEL, (int)sb, SEL, (int)sa);
}

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

// v_mfma_f32_16x16x32_{bf16,f16}: lane l holds 8 consecutive k of row l % 16 of
// each operand; D as above.
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

// One row's four neighbouring outputs from column col on.
template <MxType OUT>
__device__ __forceinline__ void store4(const MxGemmArgs& p, long long row, long long col, mx_f4 v) {
    if (row >= p.M || col >= p.N) return;
    const int n = (int)min(p.N - col, 4ll);
    if constexpr (OUT == MxType::f32) {
        // (streamed where rows are whole lines: see mx_store_wave)
        float* c = static_cast<float*>(p.C) + row * p.ldc + col;
        if (n == 4) {
            if (((unsigned long long)(size_t)p.C | (unsigned long long)p.ldc * 4) % 128 == 0)
                store_c4(c, v[0], v[1], v[2], v[3]);
            else
                __builtin_memcpy(c, &v, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) c[i] = v[i];
        }
    } else {
        __bf16* c = static_cast<__bf16*>(p.C) + row * p.ldc + col;
        typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
        if (n == 4) {
            const bf4 o = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
            __builtin_memcpy(c, &o, 8);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) c[i] = (__bf16)v[i];
        }
    }
}

// A wave's outputs from 32 x 32 accumulators, the first of them (r0, c0).  fp32
// rows on whole lines stream past the caches (8192^3 277 us against 288); others
// do not, as their pieces of a line meet only there (6336 x 4669 x 90 44 us
// against 64).
template <MxType OUT, int FM, int FN>
__device__ __forceinline__ void mx_store_wave(const MxGemmArgs& p, const floatx16 (&acc)[FM][FN], long long r0,
                                              long long c0, int li, int g) {
    typedef std::conditional_t<OUT == MxType::f32, float, __bf16> T;
    const int rows = (int)min(p.M - r0, 32ll * FM) - 4 * g, cols = (int)min(p.N - c0, 32ll * FN) - li;
    T* c = static_cast<T*>(p.C) + (r0 + 4 * g) * p.ldc + c0 + li;
    auto store = [&](auto stream) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = 32 * i + 8 * (r / 4) + r % 4;
                T* const at = c + row * p.ldc;
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    if (row < rows && 32 * j < cols) {
                        if constexpr (stream)
                            __builtin_nontemporal_store((T)acc[i][j][r], at + 32 * j);
                        else
                            at[32 * j] = (T)acc[i][j][r];
                    }
            }
        }
    };
    if constexpr (OUT == MxType::f32) {
        if (((unsigned long long)(size_t)p.C | (unsigned long long)p.ldc * 4) % 128 == 0)
            store(std::true_type{});
        else
            store(std::false_type{});
    } else {
        store(std::false_type{});
    }
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

#endif
}  // namespace sgemm
