// Kernel specialisations of the normal layout with an epilogue: the tile widths whose whole tile is staged
// in shared memory, which is where the residual arrives.
#define DG_DEFINE_LAUNCH
#include "dg_launch.cuh"

namespace dg {
template cudaError_t launch<kEpilogue, 64, 1>(const Launch&);
template cudaError_t launch<kEpilogue, 128, 1>(const Launch&);
template cudaError_t launch<kEpilogue, 192, 1>(const Launch&);
template cudaError_t launch<kEpilogue, 256, 2>(const Launch&);
}  // namespace dg
