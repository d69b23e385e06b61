// The attention of few query rows over prefixes that groups share, and what each request has of its
// own, in one launch (attn_paged.cuh).
#include "attn_paged.cuh"

namespace tpk {

bool shared_split_fits(int n_req, int n_grp) { return n_req + n_grp <= kVirtual; }

cudaError_t launch_shared_split(PagedParams& p, int D, int dtype, cudaStream_t stream) {
  p.whole = 0;
  return dtype == 0 ? launch_dim<Bf16, kSharedPrefix>(p, D, stream) : launch_dim<F16, kSharedPrefix>(p, D, stream);
}

}  // namespace tpk
