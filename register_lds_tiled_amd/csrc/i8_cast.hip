// i8_cast.hip -- rows quantised to 8-bit whole numbers with one scale each, and
// read back.
//
// s = max(fl(t / 127), 2^-126) for a row whose largest magnitude is t, and
// q = x / s rounded to nearest, ties to even: |q| <= 127, since t / s is at most
// 127 (1 + 2^-24).  The quotient is not divided out: x times the reciprocal of s,
// added to 3 2^22, leaves in the sum's low byte a whole number q' that is off by
// one at most, and only next to a half.  The rest x - q' s has few enough bits for
// one fused multiply-add to be exact (x and q' s are multiples of s's last bit
// where |x| >= s, their difference no larger than s; below that q' is 0 or +-1,
// and the difference is x or that of two numbers within a factor of two; just
// below s / 2 it may round to s / 2, and the tie goes to 0 as it should).  Where
// no rest of eight values reaches s / 2 all are right; else they are put right
// one by one.
//
// Bound by memory: X is read once (rows of up to kHeld units a thread stay in
// registers between the maximum and the rounding), Q and S are written once; but
// seven vector instructions a value come near (with twenty 8192^2 bf16 took 78
// us).  Threads share a row, or a wave takes a row of its own where rows are
// short.
#include "layer.h"

namespace sgemm {
namespace {

// Eight values: one unit of work.
template <Elem T>
struct Unit {
    unsigned w[T == Elem::f32 ? 8 : 4];
};
template <Elem T>
__device__ __forceinline__ void load_unit(Unit<T>& u, const unsigned char* row, int i, int C) {
    constexpr int B = 8 * size_of<T>;
    const long long at = (long long)i * B, len = (long long)C * size_of<T>;
    if (at + B <= len) {
        __builtin_memcpy(u.w, row + at, B);
    } else {
        const uint4 v = mx_bytes16(row, at, len);
        u.w[0] = v.x, u.w[1] = v.y, u.w[2] = v.z, u.w[3] = v.w;
        if constexpr (T == Elem::f32) {
            const uint4 h = mx_bytes16(row, at + 16, len);
            u.w[4] = h.x, u.w[5] = h.y, u.w[6] = h.z, u.w[7] = h.w;
        }
    }
}
template <Elem T>
__device__ __forceinline__ void values(const Unit<T>& u, float (&x)[8]) {
    if constexpr (T == Elem::f32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u.w[i]);
    } else {
        unpack8<T>(make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]), x);
    }
}
// The largest magnitude's bits in the type's own pattern, where infinities and
// NaN are past every number's: 16-bit types keep two of them, side by side.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
template <Elem T>
__device__ __forceinline__ unsigned top_of(const Unit<T>& u, unsigned top) {
    if constexpr (T == Elem::f32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, u.w[i] & 0x7FFFFFFFu);
        return top;
    } else {
        u16x2 t = __builtin_bit_cast(u16x2, top);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, u.w[i] & 0x7FFF7FFFu));
        return __builtin_bit_cast(unsigned, t);
    }
}
// The larger of two such maxima; the value of one as a float, and whether it is
// a number.
template <Elem T>
__device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    if constexpr (T == Elem::f32) return max(a, b);
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
template <Elem T>
__device__ __forceinline__ float top_value(unsigned top, bool& finite) {
    if constexpr (T == Elem::f32) {
        finite = top < 0x7F800000u;
        return __uint_as_float(top);
    } else {
        const unsigned t = max(top & 0xFFFFu, top >> 16);
        finite = t < (T == Elem::bf16 ? 0x7F80u : 0x7C00u);
        return T == Elem::bf16 ? __uint_as_float(t << 16) : (float)__builtin_bit_cast(_Float16, (unsigned short)t);
    }
}
__device__ __forceinline__ int quotient(float x, float s, float inverse) {
    float q = __builtin_rintf(x * inverse);
    const float r = __builtin_fmaf(-q, s, x), d = 2.f * __builtin_fabsf(r);
    // past a half: the next one; at a half: the even one, which differs where q is odd
    if (d > s || (d == s && ((int)q & 1))) q += r > 0.f ? 1.f : -1.f;
    return (int)q;
}
template <Elem T>
__device__ __forceinline__ void store_unit(const Unit<T>& u, signed char* row, int i, int C, float s, float inverse,
                                           bool finite) {
    constexpr float MAGIC = 12582912.f;   // 3 2^22: the last bit of the sum is 1
    float x[8], rest = 0.f;
    unsigned y[8], b[2];
    values(u, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = __builtin_fmaf(x[e], inverse, MAGIC);
        y[e] = __float_as_uint(f);
        rest = fmaxf(rest, __builtin_fabsf(__builtin_fmaf(MAGIC - f, s, x[e])));
    }
    if (!(rest < 0.5f * s) || !finite) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = finite ? (unsigned)quotient(x[e], s, inverse) : 0u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // the low bytes
        const unsigned lo = __builtin_amdgcn_perm(y[4 * h + 1], y[4 * h], 0x0C0C0400u);
        const unsigned hi = __builtin_amdgcn_perm(y[4 * h + 3], y[4 * h + 2], 0x04000C0Cu);
        b[h] = lo | hi;
    }
    signed char* const to = row + 8ll * i;
    const int n = C - 8 * i;
    if (n >= 8) {
        __builtin_memcpy(to, b, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) to[e] = (signed char)(b[e / 4] >> (8 * (e % 4)));
    }
}

// Units a thread keeps: 64 bytes of X.
template <Elem T>
constexpr int kHeld = T == Elem::f32 ? 2 : 4;

// NT threads to a row, several rows to a workgroup of 256 where NT is 64.
template <Elem T, int NT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void i8_quantize_kernel(I8CastArgs p) {
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, NW = NT / 64;
    __shared__ unsigned tops[2][NW > 1 ? NW : 1];
    const int t = threadIdx.x % NT, units = (int)(((long long)p.C + 7) / 8);
    int turn = 0;
    for (long long r = (long long)blockIdx.x * ROWS + threadIdx.x / NT; r < p.R; r += (long long)gridDim.x * ROWS) {
        const unsigned char* const row = static_cast<const unsigned char*>(p.X) + r * p.ldx * size_of<T>;
        Unit<T> held[kHeld<T>];
        unsigned top = 0;
#pragma unroll
        for (int h = 0; h < kHeld<T>; ++h)
            if (t + h * NT < units) load_unit<T>(held[h], row, t + h * NT, p.C);
#pragma unroll
        for (int h = 0; h < kHeld<T>; ++h)
            if (t + h * NT < units) top = top_of<T>(held[h], top);
        for (int i = t + kHeld<T> * NT; i < units; i += NT) {
            Unit<T> u;
            load_unit<T>(u, row, i, p.C);
            top = top_of<T>(u, top);
        }
#pragma unroll
        for (int d = 32; d > 0; d /= 2) top = larger<T>(top, (unsigned)__shfl_xor((int)top, d));
        if constexpr (NW > 1) {
            // two places in turn, so that a row's are read before they are written again
            if (threadIdx.x % 64 == 0) tops[turn & 1][threadIdx.x / 64] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < NW; ++w) top = larger<T>(top, tops[turn & 1][w]);
            ++turn;
        }
        bool finite;
        const float s = fmaxf(top_value<T>(top, finite) / 127.f, 0x1p-126f), inverse = 1.f / s;
        signed char* const to = static_cast<signed char*>(p.Q) + r * p.ldq;
#pragma unroll
        for (int h = 0; h < kHeld<T>; ++h)
            if (t + h * NT < units) store_unit<T>(held[h], to, t + h * NT, p.C, s, inverse, finite);
        for (int i = t + kHeld<T> * NT; i < units; i += NT) {
            Unit<T> u;
            load_unit<T>(u, row, i, p.C);
            store_unit<T>(u, to, i, p.C, s, inverse, finite);
        }
        if (t == 0) p.S[r] = finite ? s : __builtin_nanf("");
    }
}

// A thread takes units of one column piece down the rows.
template <Elem T>
__global__ __launch_bounds__(256) void i8_dequantize_kernel(I8CastArgs p, int shift) {
    const int units = (int)(((long long)p.C + 7) / 8);
    const long long i = ((long long)blockIdx.x << shift) + (threadIdx.x & ((1 << shift) - 1));
    if (i >= units) return;
    const long long rows = (long long)gridDim.y << (8 - shift);
    for (long long r = ((long long)blockIdx.y << (8 - shift)) + (threadIdx.x >> shift); r < p.R; r += rows) {
        const signed char* const q = static_cast<const signed char*>(p.Q) + r * p.ldq + 8 * i;
        const int n = p.C - 8 * (int)i;
        signed char b[8];
        if (n >= 8) {
            __builtin_memcpy(b, q, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = e < n ? q[e] : (signed char)0;
        }
        const float s = p.S[r];
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)b[e] * s;
        store8<T>(static_cast<type_of<T>*>(const_cast<void*>(p.X)) + r * p.ldx + 8 * i, x, n);
    }
}

template <Elem T, int NT>
hipError_t quantize(const I8CastArgs& a, hipStream_t s) {
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;
    const long long groups = ((long long)a.R + ROWS - 1) / ROWS;
    const long long most = 1ll << 21;   // times 1024 threads: within a launch
    i8_quantize_kernel<T, NT><<<(unsigned)(groups < most ? groups : most), NT < 256 ? 256 : NT, 0, s>>>(a);
    return hipGetLastError();
}

template <Elem T>
hipError_t quantize_t(const I8CastArgs& a, hipStream_t s) {
    const long long units = ((long long)a.C + 7) / 8;
    if (units <= 64 * kHeld<T>) return quantize<T, 64>(a, s);
    if (units <= 256 * kHeld<T> && a.R >= a.cus) return quantize<T, 256>(a, s);
    return quantize<T, 1024>(a, s);
}

template <Elem T>
hipError_t dequantize_t(const I8CastArgs& a, hipStream_t s) {
    const long long units = ((long long)a.C + 7) / 8;
    int shift = 0;
    while (shift < 8 && (1 << shift) < units) ++shift;
    const long long gx = (units + (1 << shift) - 1) >> shift, by = ((long long)a.R + (256 >> shift) - 1) >> (8 - shift);
    long long gy = (64ll * a.cus + gx - 1) / gx;   // rows beyond it go round
    if (gy > by) gy = by;
    if (gy > 65535) gy = 65535;
    i8_dequantize_kernel<T><<<dim3((unsigned)gx, (unsigned)gy), 256, 0, s>>>(a, shift);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_quantize(const I8CastArgs& a, Elem t, hipStream_t s) {
    return t == Elem::f32 ? quantize_t<Elem::f32>(a, s)
                          : t == Elem::bf16 ? quantize_t<Elem::bf16>(a, s) : quantize_t<Elem::f16>(a, s);
}
hipError_t launch_i8_dequantize(const I8CastArgs& a, Elem t, hipStream_t s) {
    return t == Elem::f32 ? dequantize_t<Elem::f32>(a, s)
                          : t == Elem::bf16 ? dequantize_t<Elem::bf16>(a, s) : dequantize_t<Elem::f16>(a, s);
}

}  // namespace sgemm
