// Trees of few rows a sequence: the kernels of kv_step.cuh with a tree's masks.
#include "kv_step.cuh"

namespace splitzip {

int launch_kv_tree_step(const AttentionArgs& a, uint32_t ctas, cudaStream_t s) { return launch_type<true>(a, ctas, s); }

}  // namespace splitzip
