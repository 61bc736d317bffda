// Trees of many rows a sequence: the kernels of kv_chunk.cuh with a tree's masks.
#include "kv_chunk.cuh"

namespace splitzip {

int launch_kv_tree_chunk(const AttentionArgs& a, bool q_half, void* plan, uint32_t ctas, cudaStream_t s) {
    return launch_chunk<true>(a, q_half, plan, ctas, s);
}

}  // namespace splitzip
