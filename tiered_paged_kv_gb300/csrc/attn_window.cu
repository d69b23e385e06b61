// The attention of few query rows through windows (attn_paged.cuh).
#include "attn_paged.cuh"

namespace tpk {

cudaError_t launch_window_split(PagedParams& p, int span_pages, int D, int dtype, cudaStream_t stream) {
  return launch_by_rows<kWindowed>(p, span_pages, D, dtype, stream);
}

}  // namespace tpk
