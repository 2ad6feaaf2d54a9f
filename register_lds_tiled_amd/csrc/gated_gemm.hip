// gated_gemm.hip -- the gated block in 16 bits: H = act(X.Wg^T) (X.Wu^T) in one
// kernel.
#include "layer_tile.h"

namespace sgemm {
namespace {

template <Elem E>
hipError_t launch(const LayerArgs& a, hipStream_t s) {
    using T = layer::Tile<Form::gated, E, E, 128, 128, 64, 64>;
    return layer::launch_tiles<T>(layer::tile_kernel<T>, a, s);
}

}  // namespace

hipError_t launch_gated(const LayerArgs& a, Elem t, hipStream_t s) {
    return t == Elem::bf16 ? launch<Elem::bf16>(a, s) : launch<Elem::f16>(a, s);
}

}  // namespace sgemm
