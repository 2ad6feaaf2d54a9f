// gated_backward.hip -- the gated block's gradients in 16 bits: dG and dU element
// by element, dX = dG.Wg + dU.Wu as one product over both, dWg = dG^T.X and
// dWu = dU^T.X in one launch.
//
// The products take dG and dU as the call returns them, rounded to 16 bits, because
// the matrix instructions take 16-bit operands; with fp32 dG and dU each would be two
// terms, at twice the instructions.  That rounding and the result's own are of one
// size, so dX, dWg and dWu are off by sqrt 2 of what the latter alone gives (1.5
// times where a few large channels of X carry a gradient).
#include "layer_split.h"

namespace sgemm {
namespace {

// A thread takes eight columns down the rows: three reads, two writes, bound by
// memory.  An infinity in U stands for a finite sum beyond its type's range as
// well (act_and_slope has G's): where the slope is 0, so is dG.  (The branch for
// them: 4096 x 8192 bf16 SiLU 62.8 us, 62.1 without.)
template <Elem E>
__global__ __launch_bounds__(256) void gated_slopes_kernel(GateArgs p, int shift) {
    const int units = (int)(((long long)p.N + 7) / 8);
    const long long i = ((long long)blockIdx.x << shift) + (threadIdx.x & ((1 << shift) - 1));
    if (i >= units) return;
    const int n = p.N - 8 * (int)i;
    const long long rows = (long long)gridDim.y << (8 - shift);
    with_act(p.act, [&](auto act) __attribute__((always_inline)) {
        for (long long r = ((long long)blockIdx.y << (8 - shift)) + (threadIdx.x >> shift); r < p.M; r += rows) {
            float g[8], u[8], dh[8], dg[8], du[8], d[8], top = 0.f;
            load8<E>(p.G + 2 * r * p.ldg, 8 * i, p.N, g);
            load8<E>(p.U + 2 * r * p.ldu, 8 * i, p.N, u);
            load8<E>(p.DH + 2 * r * p.lddh, 8 * i, p.N, dh);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a;
                act_and_slope<act>(g[e], a, d[e]);
                du[e] = dh[e] * a;
                top = fmaxf(top, __builtin_fabsf(u[e]));
            }
            if (top == __builtin_inff()) {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = d[e] == 0.f && __builtin_isinf(u[e]) ? 0.f : u[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) dg[e] = dh[e] * u[e] * d[e];
            typedef type_of<E> O;
            store8<E>(reinterpret_cast<O*>(p.DG) + r * p.lddg + 8 * i, dg, n);
            store8<E>(reinterpret_cast<O*>(p.DU) + r * p.lddu + 8 * i, du, n);
        }
    });
}

template <Elem E>
hipError_t slopes(const GateArgs& a, hipStream_t s) {
    const long long units = ((long long)a.N + 7) / 8;
    int shift = 0;
    while (shift < 8 && (1 << shift) < units) ++shift;
    const long long gx = (units + (1 << shift) - 1) >> shift, by = ((long long)a.M + (256 >> shift) - 1) >> (8 - shift);
    long long gy = (64ll * a.cus + gx - 1) / gx;   // rows beyond it go round
    if (gy > by) gy = by;
    if (gy > 65535) gy = 65535;
    gated_slopes_kernel<E><<<dim3((unsigned)gx, (unsigned)gy), 256, 0, s>>>(a, shift);
    return hipGetLastError();
}

template <Form F, Elem E>
hipError_t launch(const LayerArgs& a, hipStream_t s) {
    return layer::launch_form<F, E, E>(a, s);
}

}  // namespace

hipError_t launch_gated_slopes(const GateArgs& a, Elem t, hipStream_t s) {
    return t == Elem::bf16 ? slopes<Elem::bf16>(a, s) : slopes<Elem::f16>(a, s);
}
hipError_t launch_gated_dx(const LayerArgs& a, Elem t, hipStream_t s) {
    return t == Elem::bf16 ? launch<Form::sum2, Elem::bf16>(a, s) : launch<Form::sum2, Elem::f16>(a, s);
}
hipError_t launch_gated_dw(const LayerArgs& a, Elem t, hipStream_t s) {
    return t == Elem::bf16 ? launch<Form::both, Elem::bf16>(a, s) : launch<Form::both, Elem::f16>(a, s);
}

}  // namespace sgemm
