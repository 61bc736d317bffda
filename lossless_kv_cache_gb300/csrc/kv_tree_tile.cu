// Trees of up to 128 rows a sequence: launches of the kernels of kv_tree_tile.cuh.
#include "kv_tree_tile.cuh"

namespace splitzip {

int launch_kv_tree_tile(const AttentionArgs& a, bool q_half, void* plan_at, uint32_t ctas, cudaStream_t s) {
    ChunkPlan* plan = static_cast<ChunkPlan*>(plan_at);
    ChunkMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    // pages too small for the tensor maps, strides that they do not take, or scales that do
    // not lie as the copies want them
    const bool fp8 = a.c.type == SPLITZIP_KV_FP8_E5M2 || a.c.type == SPLITZIP_KV_FP8_E4M3;
    if (a.c.page_shift < 3 || !(fp8 ? make_byte_maps(a, &maps) : make_maps(a, &maps)) ||
        (fp8 && ((reinterpret_cast<uintptr_t>(a.c.k_scale) | reinterpret_cast<uintptr_t>(a.c.v_scale)) & 15u)))
        return launch_kv_tree_chunk(a, q_half, plan_at, ctas, s);
    // the status by all sequences' entries, and where there are many, their plan
    if (a.b.batch > kPlanSequences) {
        kv_chunk_plan_kernel<TileWork><<<1, kPlanThreads, 0, s>>>(a, plan, ctas);
        if (cudaGetLastError() != cudaSuccess) return SPLITZIP_ERR_CUDA;
    } else if (launch_kv_begin(a.b, a.status, nullptr, 0, s) != cudaSuccess) {
        cudaGetLastError();
        return SPLITZIP_ERR_CUDA;
    }
    const bool wide = a.c.head_dim == 128;
    switch (a.c.type) {
        case SPLITZIP_KV_FP8_E5M2:
            return wide ? launch_tile<1, false, 128>(a, plan, maps, ctas, s) : launch_tile<1, false, 64>(a, plan, maps, ctas, s);
        case SPLITZIP_KV_FP8_E4M3:
            return wide ? launch_tile<2, false, 128>(a, plan, maps, ctas, s) : launch_tile<2, false, 64>(a, plan, maps, ctas, s);
        case SPLITZIP_KV_FP16:
            return wide ? launch_tile<0, true, 128>(a, plan, maps, ctas, s) : launch_tile<0, true, 64>(a, plan, maps, ctas, s);
        default:
            return wide ? launch_tile<0, false, 128>(a, plan, maps, ctas, s) : launch_tile<0, false, 64>(a, plan, maps, ctas, s);
    }
}

}  // namespace splitzip
