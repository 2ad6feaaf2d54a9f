// layer_rows.hip -- the few-row kernels of the feed-forward layer: 8-bit products
// and both gated forms.
#include "layer_rows.h"

namespace sgemm {

hipError_t launch_i8_rows(const LayerArgs& a, bool gated, Elem out, hipStream_t s) {
    using namespace layer;
    if (gated)
        return out == Elem::bf16 ? launch_few<Form::gated, Elem::i8, Elem::bf16>(a, s)
                                 : launch_few<Form::gated, Elem::i8, Elem::f16>(a, s);
    return out == Elem::f32 ? launch_few<Form::nt, Elem::i8, Elem::f32>(a, s)
                            : out == Elem::bf16 ? launch_few<Form::nt, Elem::i8, Elem::bf16>(a, s)
                                                : launch_few<Form::nt, Elem::i8, Elem::f16>(a, s);
}

hipError_t launch_gated_rows(const LayerArgs& a, Elem t, hipStream_t s) {
    return t == Elem::bf16 ? layer::launch_few<Form::gated, Elem::bf16, Elem::bf16>(a, s)
                           : layer::launch_few<Form::gated, Elem::f16, Elem::f16>(a, s);
}

}  // namespace sgemm
