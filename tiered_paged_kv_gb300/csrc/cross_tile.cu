// The attention of many query rows over whole histories (cross_tile.cuh).
#include "cross_tile.cuh"

namespace tpk {

cudaError_t launch_cross_tiles(const PagedParams& p, int D, int dtype, int tiles, int groups, int splits,
                               cudaStream_t stream) {
  return launch_tiles_of<kWholeHistory>(p, D, dtype, tiles, groups, splits, stream);
}

}  // namespace tpk
