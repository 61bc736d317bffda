// Shared by the paged-cache operators (kv_rw.cu, kv_attention.cu, kv_step.cu,
// kv_chunk.cu): their kernel arguments, how a packed row finds its place in
// the pages, and conversions of the FP8 types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "splitzip_internal.cuh"

namespace splitzip {

// splitzip_kv_cache_t with strides in bytes and the page size as a shift.
struct KvCache {
    uint8_t* k;
    uint8_t* v;
    uint8_t* k_scale;
    uint8_t* v_scale;
    uint64_t pool_pages;
    uint64_t page_stride, token_stride, head_stride;
    uint32_t page_shift, kv_heads, head_dim;
    int type;
};

struct KvBatch {
    const int32_t* cu;
    const int32_t* kv_len;
    const int32_t* table;
    uint64_t table_stride;
    uint32_t batch, tokens, max_tokens, max_kv_len;
};

// Packed rows, strides in elements (16-bit).
struct KvRows {
    uint16_t* d;
    uint64_t token_stride, head_stride;
};

// One sequence of a step; ok is false where its entries are out of range, and
// it then counts as having nothing new.
struct KvSeq {
    int row0, t, n;  // first packed row, new tokens, tokens held
    bool ok;
};

__device__ __forceinline__ KvSeq load_seq(const KvBatch& B, uint32_t b) {
    KvSeq s;
    const int c0 = B.cu[b], c1 = B.cu[b + 1];
    s.n = B.kv_len[b];
    s.ok = c0 >= 0 && c0 <= c1 && c1 <= int(B.tokens) && c1 - c0 <= int(B.max_tokens) && s.n >= 0 &&
           s.n <= int(B.max_kv_len);
    s.row0 = s.ok ? c0 : 0;
    s.t = s.ok ? c1 - c0 : 0;
    return s;
}

// 2^(s - 127) of a scale byte.
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s << 23); }

// Two FP8 values (low byte first) as FP16, exactly.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x2_to_half2(uint32_t two) {
    uint32_t r;
    const uint16_t x = uint16_t(two);
    if (E5M2)
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(x));
    else
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    return r;
}

// The low (0) or high (1) two FP8 values of a word as FP16, exactly.  An E5M2
// byte is the upper byte of the FP16 number it stands for.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8_pair_to_half2(uint32_t word, int which) {
    if (E5M2) return __byte_perm(word, 0u, which ? 0x3424u : 0x1404u);
    return fp8x2_to_half2<false>(which ? word >> 16 : word);
}

// Two floats as an FP8 pair (a in the low byte), rounded to nearest even.
// Finite values past the largest would saturate; the callers have none.
template <bool E5M2>
__device__ __forceinline__ uint32_t float2_to_fp8x2(float a, float b) {
    uint16_t r;
    if (E5M2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t h) {
    return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// A kernel chained to its predecessor by programmatic dependent launch starts
// while the predecessor runs; memory that the predecessor writes may be
// touched only after this.
__device__ __forceinline__ void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Host side (kv_rw.cu): argument checks shared by the entry points.
int check_kv(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch, KvCache* c, KvBatch* b, bool need_ptrs);
int check_rows(const splitzip_kv_rows_t* r, const KvBatch& b, uint32_t heads, uint32_t head_dim, KvRows* out);
// Whether rows of `dtype` go with a cache of `type`.
bool kv_dtype_fits(int type, int dtype);

// Sets the status word, by the entries of all sequences (also of those that no
// packed row belongs to, which the kernels after it never look at), and clears
// `count` 32-bit words of a workspace, as the predecessor that the operators'
// kernels are chained to.
cudaError_t launch_kv_begin(const KvBatch& b, int* status, uint32_t* words, uint32_t count, cudaStream_t s);

// Launch configuration of a kernel chained to its predecessor.
struct ChainedLaunch {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    ChainedLaunch(dim3 grid, dim3 block, size_t smem, cudaStream_t s) : cfg{}, attr{} {
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

}  // namespace splitzip
