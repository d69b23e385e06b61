// The attention of few query rows over what requests do not share, for the join with their prefixes (attn_paged.cuh).
#include "attn_paged.cuh"

namespace tpk {

cudaError_t launch_own_split(PagedParams& p, int D, int dtype, cudaStream_t stream) {
  return launch_by_rows<kOwnTokens>(p, p.max_pages, D, dtype, stream);
}

}  // namespace tpk
