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

enum class MxType { f32, bf16, f16 };

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
    int xcds = 8;
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

// The 16 bytes at p, of which the first n (any sign, at most 16) exist: zeros
// for the rest, which are not read.  ALIGNED: p is 16-byte aligned.
template <bool ALIGNED>
__device__ __forceinline__ uint4 mx_load16(const unsigned char* p, long long n) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n >= 16) {
        if constexpr (ALIGNED)
            v = *reinterpret_cast<const uint4*>(p);
        else
            __builtin_memcpy(&v, p, 16);
    } else if (n > 0) {
        unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (i < n) w[i / 4] |= (unsigned)p[i] << (8 * (i % 4));
        v = make_uint4(w[0], w[1], w[2], w[3]);
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
template <bool ALIGNED>
__device__ __forceinline__ uint4 mx_codes16(const unsigned char* row, long long at, int K) {
    const long long left = ((long long)K + 1) / 2 - at;
    uint4 v = mx_load16<ALIGNED>(row + at, left);
    if ((K & 1) && left > 0 && left <= 16) v = mx_drop_half(v, left);
    return v;
}

// N (4, 8 or 16) scale bytes from byte `at` of a row of n: zeros past n.
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

// The DMA loaders address a tile's rows by 32-bit offsets from its first row.
inline bool mx_dma_reach(long long ld_bytes, int rows) { return ld_bytes * rows < (1ll << 32); }

// Four registers, each holding in lane group t (of 16 lanes) what groups 0 to
// 3 need for tile t; afterwards register t holds in lane group g what group g
// needs for tile t: a transpose across the lane groups.
__device__ __forceinline__ void mx_transpose4(unsigned (&d)[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    const auto x = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = x[0];
    d[1] = x[1];
    d[2] = y[0];
    d[3] = y[1];
}
#endif
}  // namespace sgemm
