// Indexer scores with E4M3 queries and keys.
#include "indexer_scores.cuh"

namespace tki {

topk_status launch_scores_e4m3(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream) {
  return launch_scores_of<__nv_fp8_e4m3>(a, dev, sm_count, stream);
}

}  // namespace tki
