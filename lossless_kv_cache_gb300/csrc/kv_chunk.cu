// Chunks of new tokens: the kernels of kv_chunk.cuh without a tree.
#include "kv_chunk.cuh"

namespace splitzip {

uint32_t chunk_ctas(uint64_t rows, uint64_t batch, uint64_t kv_heads, uint64_t keys_max) {
    const uint64_t tiles = std::min<uint64_t>((rows + kRows - 1) / kRows + batch, rows);
    const uint64_t units = tiles * kv_heads * ((keys_max + kUnit - 1) / kUnit + 1);
    return uint32_t(std::min<uint64_t>(kChunkCtas, std::max<uint64_t>(1, units)));
}

uint64_t chunk_plan_bytes(uint32_t ctas) { return plan_bytes(ctas) + uint64_t(ctas) * sizeof(ChunkSplit); }

int launch_kv_chunk(const AttentionArgs& a, bool q_half, void* plan, uint32_t ctas, cudaStream_t s) {
    return launch_chunk<false>(a, q_half, plan, ctas, s);
}

}  // namespace splitzip
