// layer.h -- internal declarations of the feed-forward layer's operators:
// products of 8-bit integers with scales, and the gated block in 16 bits and in
// 8 with its backward pass.  Arguments after validation, launchers, and the
// device helpers that the kernels share.
#pragma once

#include <hip/hip_runtime.h>

#include "lds_dma.h"
#include "mxfp4.h"
#include "tiles.h"

namespace sgemm {

enum class Elem { f32, bf16, f16, i8 };

// X (R x C) <-> whole numbers Q with a scale per row.
struct I8CastArgs {
    int R, C;
    const void* X;      // or Y, written
    long long ldx;
    void* Q;            // read where Y is written
    long long ldq;
    float* S;
    int cus = 256, xcds = 8;
};

// The forms of a product.
//   nt     C0 = A0.B0^T                    (A: M x K, B: N x K)
//   gated  C0 = act(A0.B0^T) (A0.B1^T), the two products to G and U if not null
//   sum2   C0 = A0.B0 + A1.B1              (A: M x K, B: K x N)
//   both   C0 = A0^T.B0, C1 = A1^T.B0      (A: K x M, B: K x N)
enum class Form { nt, gated, sum2, both };

struct LayerArgs {
    int M, N, K;
    const unsigned char* A[2];
    long long lda[2];            // bytes
    const unsigned char* B[2];
    long long ldb[2];
    const float* SA = nullptr;   // 8-bit operands: M and N scales
    const float* SB[2] = {nullptr, nullptr};
    void* C[2];
    long long ldc[2];            // elements
    void* G = nullptr;
    void* U = nullptr;
    long long ldg = 0, ldu = 0;
    int act = 0;
    int cus = 256, xcds = 8;
};

// dG = dH U act'(G), dU = dH act(G), all M x N of one 16-bit type.
struct GateArgs {
    int M, N;
    const unsigned char *G, *U, *DH;
    long long ldg, ldu, lddh;    // elements
    unsigned char *DG, *DU;
    long long lddg, lddu;
    int act;
    int cus = 256;
};

hipError_t launch_i8_quantize(const I8CastArgs& a, Elem t, hipStream_t s);
hipError_t launch_i8_dequantize(const I8CastArgs& a, Elem t, hipStream_t s);
// 8-bit operands, out f32, bf16 or f16 (gated: bf16 or f16).
hipError_t launch_i8_nt(const LayerArgs& a, Elem out, hipStream_t s);
hipError_t launch_i8_gated(const LayerArgs& a, Elem out, hipStream_t s);
// 16-bit operands and results.
hipError_t launch_gated(const LayerArgs& a, Elem t, hipStream_t s);
// The same for few rows of A, see few_rows in layer_rows.h.
hipError_t launch_i8_rows(const LayerArgs& a, bool gated, Elem out, hipStream_t s);
hipError_t launch_gated_rows(const LayerArgs& a, Elem t, hipStream_t s);
hipError_t launch_gated_slopes(const GateArgs& a, Elem t, hipStream_t s);
hipError_t launch_gated_dx(const LayerArgs& a, Elem t, hipStream_t s);
hipError_t launch_gated_dw(const LayerArgs& a, Elem t, hipStream_t s);

#ifdef __HIPCC__
typedef int intx16 __attribute__((ext_vector_type(16)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) shortx4 lds_shortx4;

template <Elem T>
using type_of = std::conditional_t<T == Elem::f32, float,
                                   std::conditional_t<T == Elem::bf16, __bf16,
                                                      std::conditional_t<T == Elem::f16, _Float16, signed char>>>;
template <Elem T>
constexpr int size_of = sizeof(type_of<T>);

// ---- activations -----------------------------------------------------------
// The codes of SGEMM_ACT_*: 0 identity, 1 ReLU, 2 SiLU x s(x), 3 GELU x P(x)
// with P the normal distribution's integral, 4 its tanh form x s(2y) with
// y = sqrt(2/pi) (x + 0.044715 x^3); s(x) = 1 / (1 + exp(-x)).
//
// The exponential is 2^(x log2 e) by the hardware's 2^x, the quotient by its
// reciprocal, an ulp each.  What an argument's roundings make of it grows with the
// argument, so an activation is off by at most 2^-23 (8 + 4 z) of its value, z = |x|
// for SiLU, |2y| for the tanh form (its cubic has four roundings more) and x^2 for
// GELU, whose erfc turns its argument's relative error into x^2 of it: 2^-18 up to
// |x| = 2.  (With every rounding emulated the worst is 2^-18.0 for SiLU, 2^-15.8 for
// the tanh form and 2^-16.4 for GELU, all where results are next to 2^-119.)
// Results are rounded to 16 bits, half a step being 2^-8 and 2^-11 of them.  Below
// 2^-119 they may be 0, where the reciprocal has no normal number.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504089f); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp_of(-x)); }
// Within +-lim, NaN as it is.  Past the limit a slope is constant, and the
// products that vanish there would be infinity times zero.
__device__ __forceinline__ float held(float x, float lim) { return x > lim ? lim : x < -lim ? -lim : x; }
constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)

template <int ACT>
__device__ __forceinline__ float act_of(float x) {
    if constexpr (ACT == 1) return x < 0.f ? 0.f : x;
    if constexpr (ACT == 2) return x * sigmoid(x);
    // erfc keeps the left tail's relative accuracy, which 1 + erf would cancel
    if constexpr (ACT == 3) return x * (0.5f * erfcf(x * -0.70710678118654752f));
    if constexpr (ACT == 4) {
        const float h = held(x, 30.f);
        return x * sigmoid(2.f * kGeluC * (h + 0.044715f * h * h * h));
    }
    return x;
}
// Activation and slope of a gate sum as it was kept, in 16 bits: -infinity stands
// for a finite sum as well, so the activation's factor is held at a number whose
// product has long been the limit, 0 (NaN stays: the other factor is NaN then).
template <int ACT>
__device__ __forceinline__ void act_and_slope(float x, float& a, float& d) {
    const float low = fmaxf(x, -1e4f);
    if constexpr (ACT == 0) {
        a = x;
        d = 1.f;
    } else if constexpr (ACT == 1) {
        a = x < 0.f ? 0.f : x;
        d = x <= 0.f ? 0.f : 1.f;
    } else if constexpr (ACT == 2) {
        const float s = sigmoid(x), h = held(x, 100.f);
        a = low * s;
        d = s * (1.f + h * (1.f - s));
    } else if constexpr (ACT == 3) {
        const float p = 0.5f * erfcf(x * -0.70710678118654752f), h = held(x, 30.f);
        a = low * p;
        d = p + h * (0.5f * kGeluC) * exp_of(-0.5f * h * h);
    } else {
        const float h = held(x, 30.f), s = sigmoid(2.f * kGeluC * (h + 0.044715f * h * h * h));
        a = low * s;
        d = s + 2.f * kGeluC * h * s * (1.f - s) * (1.f + 0.134145f * h * h);
    }
}
// f(integral_constant of the activation): one branch for a whole piece of work.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case 1: f(std::integral_constant<int, 1>{}); break;
        case 2: f(std::integral_constant<int, 2>{}); break;
        case 3: f(std::integral_constant<int, 3>{}); break;
        case 4: f(std::integral_constant<int, 4>{}); break;
        default: f(std::integral_constant<int, 0>{}); break;
    }
}

// ---- eight neighbouring values ---------------------------------------------

// Eight values of type T from 16 (32 for f32) bytes.
template <Elem T>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == Elem::bf16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const mx_h2 h = __builtin_bit_cast(mx_h2, w[i]);
            x[2 * i] = (float)h[0];
            x[2 * i + 1] = (float)h[1];
        }
    }
}
template <Elem T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    typedef type_of<T> v2 __attribute__((ext_vector_type(2)));
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const v2 o = {(type_of<T>)x[2 * i], (type_of<T>)x[2 * i + 1]};
        w[i] = __builtin_bit_cast(unsigned, o);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// The first n (1 and up) of eight values to c, rounded to T; any alignment of
// whole elements.
template <Elem T>
__device__ __forceinline__ void store8(type_of<T>* c, const float (&x)[8], int n) {
    if (n >= 8) {
        if constexpr (T == Elem::f32) {
            __builtin_memcpy(c, x, 32);
        } else {
            const uint4 v = pack8<T>(x);
            __builtin_memcpy(c, &v, 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) c[i] = (type_of<T>)x[i];
    }
}
// Values i .. i + 7 of a row of n of a 16-bit type: zeros past n.
template <Elem T>
__device__ __forceinline__ void load8(const unsigned char* row, long long i, long long n, float (&x)[8]) {
    unpack8<T>(mx_bytes16(row, 2 * i, 2 * n), x);
}

// Order between the LDS accesses of one wave's lanes: LDS serves a wave's
// instructions in order, so only the compiler has to keep them.
__device__ __forceinline__ void lane_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
#endif

}  // namespace sgemm
