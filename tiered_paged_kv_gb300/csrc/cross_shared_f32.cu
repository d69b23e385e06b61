// Row tiles over shared prefixes for float32 outputs (cross_tile.cuh).
#include "cross_tile.cuh"

namespace tpk {

cudaError_t launch_shared_tiles_f32(const PagedParams& p, int D, int dtype, int tiles, int groups, int splits, cudaStream_t stream) {
  return launch_tiles_of<kSharedPrefix, 2>(p, D, dtype, tiles, groups, splits, stream);
}

}  // namespace tpk
