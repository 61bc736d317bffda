// Attention over a paged cache: what its two kernels share (kv_step.cu for
// few rows a sequence, kv_chunk.cu for chunks).
//
// Work is cut the same way in both.  An item is one (sequence, kv head, tile
// of rows), rows being (new token, query head of the group) pairs in token
// order; its keys are cut into units of kUnit positions, aligned to kUnit.
// The units of all items, in item order, are dealt to the CTAs in equal
// contiguous shares, so a batch of any lengths keeps every SM busy to the
// end, and a share ends in the middle of an item where it has to.  The parts
// of such an item (maximum m, sum l and unnormalised sums o of each row) go
// to the workspace, at most two a CTA: the first CTA's part in its slot 1, a
// continuation in slot 0.  They are joined in the order of the parts, so that
// the result does not depend on the timing: by whichever CTA counts the last
// one in a step, where parts are small, and by a kernel of its own in a chunk.
#pragma once

#include "kv_common.cuh"

namespace splitzip {

struct AttentionArgs {
    KvCache c;
    KvBatch b;
    KvRows q, out;
    float* lse;
    uint32_t q_heads, group;
    int q_half;  // the queries and results are FP16, else BF16
    // scale * log2(e).  The chunk kernel takes its magnitude, at least the
    // smallest normal, with its sign (`negate`) given to the queries.
    float scale_log2;
    int negate;
    float lag;  // chunk kernel: how far the reference may lag the maximum, before the scale
    int causal;
    uint32_t window;
    uint32_t* counters;  // workspace, one a CTA (step kernel)
    float* parts;        // workspace, two slots a CTA
    int* status;
};

// The positions that some row of a sequence's rows first .. last (new tokens
// i0 .. i1) sees: [lo, hi).
struct KeyRange {
    int lo, hi;
};

__device__ __forceinline__ KeyRange visible(const AttentionArgs& a, const KvSeq& s, int i) {
    const int p = s.n - s.t + i;
    KeyRange r;
    r.hi = p < 0 ? 0 : (a.causal ? p + 1 : s.n);
    r.lo = a.window && p >= 0 ? max(0, p + 1 - int(a.window)) : 0;
    return r;
}

__device__ __forceinline__ KeyRange visible(const AttentionArgs& a, const KvSeq& s, int i0, int i1) {
    KeyRange r;
    r.hi = visible(a, s, i1).hi;
    r.lo = visible(a, s, max(i0, s.t - s.n)).lo;  // the first row with a place
    return r;
}

// Units that the range covers; one for a range of none, so that its rows are
// written.
__device__ __forceinline__ int unit_count(const KeyRange& r, int unit) {
    return r.hi <= r.lo ? 1 : (r.hi + unit - 1) / unit - r.lo / unit;
}

__device__ __forceinline__ uint64_t share_start(uint64_t units, uint32_t ctas, uint64_t c) { return units * c / ctas; }
// The CTA whose share holds unit u.
__device__ __forceinline__ uint32_t share_of(uint64_t units, uint32_t ctas, uint64_t u) {
    return uint32_t(((u + 1) * ctas - 1) / units);
}

// 2^x; 0 for -infinity.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// kv_step.cu
constexpr int kStepRows = 16;  // rows of a tile at most
uint32_t step_ctas(uint64_t items_max, uint64_t keys_max);
uint64_t step_part_floats(uint32_t head_dim);
int launch_kv_step(const AttentionArgs& a, uint32_t ctas, cudaStream_t s);

// kv_chunk.cu
uint32_t chunk_ctas(uint64_t rows, uint64_t batch, uint64_t kv_heads, uint64_t keys_max);
uint64_t chunk_part_floats(uint32_t head_dim);
uint64_t chunk_plan_bytes(uint32_t ctas);
int launch_kv_chunk(const AttentionArgs& a, bool q_half, void* plan, uint32_t ctas, cudaStream_t s);

}  // namespace splitzip
