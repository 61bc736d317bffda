// Decoding steps: the kernels of kv_step.cuh without a tree.
#include "kv_step.cuh"

namespace splitzip {

uint64_t step_part_floats(uint32_t head_dim) { return uint64_t(kStepRows) * (head_dim + 2); }

uint32_t step_ctas(uint64_t items_max, uint64_t keys_max) {
    const uint64_t units = items_max * ((keys_max + kUnit - 1) / kUnit + 1);
    return uint32_t(std::min<uint64_t>(
        kStepCtas, std::max<uint64_t>(std::max<uint64_t>(1, items_max), (units + kMinUnits - 1) / kMinUnits)));
}

int launch_kv_step(const AttentionArgs& a, uint32_t ctas, cudaStream_t s) { return launch_type<false>(a, ctas, s); }

}  // namespace splitzip
