// The attention of few query rows over whole histories (attn_paged.cuh).
#include "attn_paged.cuh"

namespace tpk {

cudaError_t launch_paged_split(PagedParams& p, int D, int dtype, cudaStream_t stream) {
  return launch_by_rows<kWholeHistory>(p, p.max_pages, D, dtype, stream);
}

}  // namespace tpk
