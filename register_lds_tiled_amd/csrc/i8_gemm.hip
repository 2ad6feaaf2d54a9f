// i8_gemm.hip -- C = A.B^T of 8-bit whole numbers, summed in 32 bits and scaled by
// token and channel.
#include "layer_rows.h"
#include "layer_split.h"

namespace sgemm {

hipError_t launch_i8_nt(const LayerArgs& a, Elem out, hipStream_t s) {
    if (few_rows(a, 1, false)) return launch_i8_rows(a, false, out, s);
    return out == Elem::f32 ? layer::launch_form<Form::nt, Elem::i8, Elem::f32>(a, s)
                            : out == Elem::bf16 ? layer::launch_form<Form::nt, Elem::i8, Elem::bf16>(a, s)
                                                : layer::launch_form<Form::nt, Elem::i8, Elem::f16>(a, s);
}

}  // namespace sgemm
