// i8_gated.hip -- the gated block on 8-bit operands: two products of one A, scaled
// by token and channel, and H = act(g) u in one kernel.
#include "layer_rows.h"
#include "layer_split.h"

namespace sgemm {

hipError_t launch_i8_gated(const LayerArgs& a, Elem out, hipStream_t s) {
    if (few_rows(a, 1, true)) return launch_i8_rows(a, true, out, s);
    return out == Elem::bf16 ? layer::launch_form<Form::gated, Elem::i8, Elem::bf16>(a, s)
                             : layer::launch_form<Form::gated, Elem::i8, Elem::f16>(a, s);
}

}  // namespace sgemm
