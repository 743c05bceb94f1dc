// Kernel specialisations of the normal layout with an epilogue, 192 columns a tile: one for each activation.
#define DG_DEFINE_LAUNCH
#include "dg_launch.cuh"

namespace dg {
template cudaError_t launch<kEpilogue, 192, 1, DG_ACT_NONE>(const Launch&);
template cudaError_t launch<kEpilogue, 192, 1, DG_ACT_RELU>(const Launch&);
template cudaError_t launch<kEpilogue, 192, 1, DG_ACT_GELU>(const Launch&);
template cudaError_t launch<kEpilogue, 192, 1, DG_ACT_GELU_TANH>(const Launch&);
template cudaError_t launch<kEpilogue, 192, 1, DG_ACT_SILU>(const Launch&);
}  // namespace dg
