// Indexer scores with FP16 queries and keys.
#include "indexer_scores.cuh"

namespace tki {

topk_status launch_scores_fp16(const sparse_scores_args& a, int dev, int sm_count, cudaStream_t stream) {
  return launch_scores_of<__half>(a, dev, sm_count, stream);
}

}  // namespace tki
