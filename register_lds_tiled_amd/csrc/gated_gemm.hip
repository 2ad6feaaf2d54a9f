// gated_gemm.hip -- the gated block in 16 bits: H = act(X.Wg^T) (X.Wu^T) in one
// kernel.
#include "layer_rows.h"
#include "layer_split.h"

namespace sgemm {

hipError_t launch_gated(const LayerArgs& a, Elem t, hipStream_t s) {
    if (few_rows(a, 2, true)) return launch_gated_rows(a, t, s);
    return t == Elem::bf16 ? layer::launch_form<Form::gated, Elem::bf16, Elem::bf16>(a, s)
                           : layer::launch_form<Form::gated, Elem::f16, Elem::f16>(a, s);
}

}  // namespace sgemm
