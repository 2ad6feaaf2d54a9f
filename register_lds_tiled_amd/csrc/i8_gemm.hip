// i8_gemm.hip -- C = A.B^T of 8-bit whole numbers, summed in 32 bits and scaled by
// token and channel, and the gated block on such operands.
#include "layer_big.h"

namespace sgemm {
namespace {

template <Form F, Elem OUT>
hipError_t launch(const LayerArgs& a, hipStream_t s) {
    return layer::launch_form<F, Elem::i8, OUT>(a, s);
}

}  // namespace

hipError_t launch_i8_nt(const LayerArgs& a, Elem out, hipStream_t s) {
    return out == Elem::f32 ? launch<Form::nt, Elem::f32>(a, s)
                            : out == Elem::bf16 ? launch<Form::nt, Elem::bf16>(a, s) : launch<Form::nt, Elem::f16>(a, s);
}
hipError_t launch_i8_gated(const LayerArgs& a, Elem out, hipStream_t s) {
    return out == Elem::bf16 ? launch<Form::gated, Elem::bf16>(a, s) : launch<Form::gated, Elem::f16>(a, s);
}

}  // namespace sgemm
