// Writing new keys and values into the pages of a KV cache, and reading them
// back (splitzip_kv_write, splitzip_kv_read).
//
// Mathematics.  An FP8 cache keeps, for each (token, head), q_i = RN8(x_i /
// 2^k) and the exponent k = min{k : max |x_i| <= M 2^k} of the row's scale, M
// the type's largest value.  M is 1.75 * 2^T (T = 15 for E5M2, 8 for E4M3), so
// with max |x_i| = m 2^e, 1 <= m < 2, k = e - T, plus 1 where m > 1.75: one
// comparison of mantissa bits, no division.  The scale being a power of two,
// x_i / 2^k and q_i 2^k are exact and the only rounding is RN8.
//
// What bounds it: HBM.  Nothing is reused, so a row goes through the registers
// of head_dim / 16 lanes, two 16-byte pieces of the 16-bit side in each (fewer
// lanes a row than one piece each: what is done once a row, its maximum and
// scale, was a third of the instructions, and issue bound the kernel).  A warp
// takes K and V of 4 or 8 heads of one token, so the search for the token's
// sequence and page is done once for all of them while their loads are in
// flight; more rows a warp (two passes) measured the same, with more
// registers.  One GB300: a 32,768-token layer of 8 heads of 128 to E5M2 in
// 34.1 us (5.9 TB/s, 87 % of the measured copy rate), 65,536 E5M2 tokens read
// in 62.9 us (6.4 TB/s, 95 %).
#include "kv_common.cuh"

namespace splitzip {
namespace {

constexpr int kRwWarps = 4;

constexpr int kBeginThreads = 1024;

// Runs beside its successor, which waits for it before its own reports (64 tokens
// are written in 3.08 us, 2.91 if nothing is looked at here; 128 threads: the same).
__global__ void __launch_bounds__(kBeginThreads)
    kv_begin_kernel(const __grid_constant__ KvBatch batch, int* status, uint32_t* words, uint32_t count) {
    release_successor();
    for (uint32_t i = threadIdx.x; i < count; i += kBeginThreads) words[i] = 0;
    bool bad = false;
#pragma unroll 4
    for (uint32_t b = threadIdx.x; b < batch.batch; b += kBeginThreads) bad |= !load_seq(batch, b).ok;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *status = bad ? SPLITZIP_ERR_INVALID_ARG : SPLITZIP_OK;
}

struct RwArgs {
    KvCache c;
    KvBatch b;
    KvRows k, v;
    int* status;
};

// Sixteen elements of a row, quantised; LPR lanes hold the row.  Whole warp.
template <bool E5M2, bool H, int LPR>
__device__ __forceinline__ void quantise16(const uint4 (&x)[2], uint2 (&out)[2], uint32_t* scale) {
    constexpr uint32_t kInf = H ? 0x7C00u : 0x7F80u;
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    // largest magnitude: 16-bit floats order as integers
    uint32_t top = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, d));
    uint32_t most = max(top & 0xFFFFu, top >> 16);
    const bool special = most >= kInf;  // the row has an infinity or a NaN
    if (__any_sync(~0u, special)) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
            top = max(top, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
        }
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
        most = top;
    }
    const uint32_t bits = __float_as_uint(unpack16<H>(most).x);
    int k = int(bits >> 23) - 127 - (E5M2 ? 15 : 8) + ((bits & 0x7FFFFFu) > 0x600000u);
    k = most == 0 ? 0 : max(k, -126);
    *scale = uint32_t(k + 127);
    const float inv = __uint_as_float(uint32_t(127 - k) << 23);
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = mul2(unpack16<H>(w[i]), make_float2(inv, inv));
        q[i] = float2_to_fp8x2<E5M2>(f.x, f.y);
    }
    if (special) {  // the conversion saturates infinities
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if ((w[i] & 0x7FFFu) == kInf) q[i] = (q[i] & 0xFF00u) | (E5M2 ? 0x7Cu : 0x7Fu) | ((w[i] >> 8) & 0x80u);
            if (((w[i] >> 16) & 0x7FFFu) == kInf)
                q[i] = (q[i] & 0x00FFu) | (E5M2 ? 0x7C00u : 0x7F00u) | ((w[i] >> 16) & 0x8000u);
        }
    }
    out[0] = make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
    out[1] = make_uint2(__byte_perm(q[4], q[5], 0x5410), __byte_perm(q[6], q[7], 0x5410));
}

template <bool E5M2, bool H>
__device__ __forceinline__ uint4 dequantise8(const uint2& q, float scale) {
    const uint32_t w[2] = {q.x, q.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = mul2(half2_to_float2(fp8_pair_to_half2<E5M2>(w[i / 2], i & 1)), make_float2(scale, scale));
        o[i] = pack16<H>(f.x, f.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// FMT 0: 16-bit cache, 1: E5M2, 2: E4M3.  LPR lanes hold a row, two 16-byte
// pieces each; a warp takes K and V of 32 / LPR heads of one token.
template <bool WRITE, int FMT, bool H, int LPR>
__global__ void __launch_bounds__(kRwWarps * 32) kv_rw_kernel(const __grid_constant__ RwArgs a) {
    constexpr uint32_t kHeads = 32 / LPR;
    const uint32_t lane = threadIdx.x & 31u, col = lane % LPR;
    const uint32_t parts = (a.c.kv_heads + kHeads - 1) / kHeads;
    const uint64_t warp = uint64_t(blockIdx.x) * kRwWarps + (threadIdx.x >> 5);
    const uint64_t token = warp / parts;
    const uint32_t head = uint32_t(warp - token * parts) * kHeads + lane / LPR;
    const bool there = head < a.c.kv_heads;
    bool bad = false;
    if (token < a.b.tokens) {
        uint4 x[2][2];  // K and V
        uint4* rows[2] = {reinterpret_cast<uint4*>(a.k.d + token * a.k.token_stride + head * a.k.head_stride) + col,
                          reinterpret_cast<uint4*>(a.v.d + token * a.v.token_stride + head * a.v.head_stride) + col};
        if (WRITE) {
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                x[side][0] = x[side][1] = make_uint4(0, 0, 0, 0);
                if (there) {
                    x[side][0] = __ldcs(rows[side]);
                    x[side][1] = __ldcs(rows[side] + LPR);
                }
            }
        }
        const KvPlace at_place = find_place(a.c, a.b, int(token), lane);
        const bool mine = at_place.mine, placed = at_place.placed;
        const uint64_t page = at_place.page;
        const uint32_t slot = at_place.slot;
        bad = at_place.bad;
        // the same in all lanes
        if (mine && !bad && (placed || !WRITE)) {
            const uint64_t at = page * a.c.page_stride + uint64_t(slot) * a.c.token_stride + head * a.c.head_stride +
                                col * (FMT == 0 ? 16u : 8u);
            const uint64_t scale_at = ((page * a.c.kv_heads + head) << a.c.page_shift) + slot;
            if (WRITE) {
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    uint8_t* to = (side ? a.c.v : a.c.k) + at;
                    if (FMT == 0) {
                        uint4* row = reinterpret_cast<uint4*>(to);
                        if (there) row[0] = x[side][0], row[LPR] = x[side][1];
                    } else {
                        uint2 q[2];
                        uint32_t scale;
                        quantise16<FMT == 1, H, LPR>(x[side], q, &scale);
                        uint2* row = reinterpret_cast<uint2*>(to);
                        if (there) row[0] = q[0], row[LPR] = q[1];
                        if (there && col == 0) (side ? a.c.v_scale : a.c.k_scale)[scale_at] = uint8_t(scale);
                    }
                }
            } else if (there) {
                // all loads before the first store; a row without a place reads as zeros
                uint32_t scale[2] = {0, 0};
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    const uint8_t* from = (side ? a.c.v : a.c.k) + at;
                    x[side][0] = x[side][1] = make_uint4(0, 0, 0, 0);
                    if (placed && FMT == 0) {
                        x[side][0] = __ldcs(reinterpret_cast<const uint4*>(from));
                        x[side][1] = __ldcs(reinterpret_cast<const uint4*>(from) + LPR);
                    } else if (placed) {
                        const uint2 q0 = __ldcs(reinterpret_cast<const uint2*>(from));
                        const uint2 q1 = __ldcs(reinterpret_cast<const uint2*>(from) + LPR);
                        x[side][0] = make_uint4(q0.x, q0.y, q1.x, q1.y);
                        scale[side] = (side ? a.c.v_scale : a.c.k_scale)[scale_at];
                    }
                }
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    if (FMT != 0) {
                        const uint4 q = x[side][0];
                        const float f = scale_value(scale[side]);
                        x[side][0] = dequantise8<FMT == 1, H>(make_uint2(q.x, q.y), f);
                        x[side][1] = dequantise8<FMT == 1, H>(make_uint2(q.z, q.w), f);
                    }
                    __stcs(rows[side], x[side][0]);
                    __stcs(rows[side] + LPR, x[side][1]);
                }
            }
        }
    }
    wait_predecessor();  // the status word has been cleared
    if (bad && lane == 0) report(a.status, SPLITZIP_ERR_INVALID_ARG);
}

template <bool WRITE, int FMT, bool H>
cudaError_t launch_rw(const RwArgs& a, cudaStream_t s) {
    const uint32_t lpr = a.c.head_dim / 16, heads = 32 / lpr;
    const uint64_t parts = (a.c.kv_heads + heads - 1) / heads;
    const uint64_t grid = (uint64_t(a.b.tokens) * parts + kRwWarps - 1) / kRwWarps;
    if (grid > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    ChainedLaunch l(dim3(uint32_t(grid)), dim3(kRwWarps * 32), 0, s);
    return lpr == 8 ? cudaLaunchKernelEx(&l.cfg, kv_rw_kernel<WRITE, FMT, H, 8>, a)
                    : cudaLaunchKernelEx(&l.cfg, kv_rw_kernel<WRITE, FMT, H, 4>, a);
}

template <bool WRITE>
int kv_rw_call(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch, const splitzip_kv_rows_t* k,
               const splitzip_kv_rows_t* v, int dtype, int* d_status, cudaStream_t stream) {
    RwArgs a;
    int st = check_kv(cache, batch, &a.c, &a.b, true);
    if (st != SPLITZIP_OK) return st;
    if (!d_status || (reinterpret_cast<uintptr_t>(d_status) & 3u) || !kv_dtype_fits(a.c.type, dtype))
        return SPLITZIP_ERR_INVALID_ARG;
    if ((st = check_rows(k, a.b, a.c.kv_heads, a.c.head_dim, &a.k)) != SPLITZIP_OK) return st;
    if ((st = check_rows(v, a.b, a.c.kv_heads, a.c.head_dim, &a.v)) != SPLITZIP_OK) return st;
    a.status = d_status;
    int sms;
    if ((st = device_sms(&sms)) != SPLITZIP_OK) return st;
    cudaError_t e = launch_kv_begin(a.b, d_status, nullptr, 0, stream);
    if (e == cudaSuccess && a.b.tokens > 0) {
        const bool h = dtype == SPLITZIP_FP16;
        if (a.c.type == SPLITZIP_KV_FP8_E5M2)
            e = h ? launch_rw<WRITE, 1, true>(a, stream) : launch_rw<WRITE, 1, false>(a, stream);
        else if (a.c.type == SPLITZIP_KV_FP8_E4M3)
            e = h ? launch_rw<WRITE, 2, true>(a, stream) : launch_rw<WRITE, 2, false>(a, stream);
        else
            e = launch_rw<WRITE, 0, false>(a, stream);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? SPLITZIP_OK : SPLITZIP_ERR_CUDA;
}

bool multiple_of(uint64_t x, uint64_t m) { return x % m == 0; }

}  // namespace

cudaError_t launch_kv_begin(const KvBatch& b, int* status, uint32_t* words, uint32_t count, cudaStream_t s) {
    kv_begin_kernel<<<1, kBeginThreads, 0, s>>>(b, status, words, count);
    return cudaGetLastError();
}

bool kv_dtype_fits(int type, int dtype) {
    if (dtype != SPLITZIP_BF16 && dtype != SPLITZIP_FP16) return false;
    if (type == SPLITZIP_KV_BF16) return dtype == SPLITZIP_BF16;
    if (type == SPLITZIP_KV_FP16) return dtype == SPLITZIP_FP16;
    return true;
}

int check_batch(const splitzip_kv_batch_t* batch, KvBatch* b, bool need_ptrs) {
    if (!batch) return SPLITZIP_ERR_INVALID_ARG;
    if (need_ptrs && (!batch->d_cu_tokens || !batch->d_kv_len || (reinterpret_cast<uintptr_t>(batch->d_cu_tokens) & 3u) ||
                      (reinterpret_cast<uintptr_t>(batch->d_kv_len) & 3u)))
        return SPLITZIP_ERR_INVALID_ARG;
    if (batch->batch == 0 || batch->max_tokens > batch->tokens) return SPLITZIP_ERR_INVALID_ARG;
    if (batch->batch > 65536u || batch->tokens >= (1u << 30) || batch->max_kv_len >= (1u << 30))
        return SPLITZIP_ERR_UNSUPPORTED;
    b->cu = batch->d_cu_tokens;
    b->kv_len = batch->d_kv_len;
    b->table = batch->d_page_table;
    b->table_stride = batch->table_stride;
    b->batch = batch->batch;
    b->tokens = batch->tokens;
    b->max_tokens = batch->max_tokens;
    b->max_kv_len = batch->max_kv_len;
    return SPLITZIP_OK;
}

int check_kv(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch, KvCache* c, KvBatch* b,
             bool need_ptrs) {
    if (!cache || !batch) return SPLITZIP_ERR_INVALID_ARG;
    const auto addr = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    if (cache->type < SPLITZIP_KV_BF16 || cache->type > SPLITZIP_KV_FP8_E4M3) return SPLITZIP_ERR_INVALID_ARG;
    const bool fp8 = cache->type == SPLITZIP_KV_FP8_E5M2 || cache->type == SPLITZIP_KV_FP8_E4M3;
    const uint64_t size = fp8 ? 1 : 2, quantum = 16 / size;
    const uint32_t pt = cache->page_tokens;
    if (pt == 0 || pt > 65536u || (pt & (pt - 1u)) || cache->kv_heads == 0 || cache->kv_heads > 1024u ||
        cache->pool_pages == 0)
        return SPLITZIP_ERR_INVALID_ARG;
    if (cache->head_dim != 64u && cache->head_dim != 128u) return SPLITZIP_ERR_UNSUPPORTED;
    if (cache->pool_pages > 0x7FFFFFFFull) return SPLITZIP_ERR_UNSUPPORTED;
    if (!multiple_of(cache->page_stride, quantum) || !multiple_of(cache->token_stride, quantum) ||
        !multiple_of(cache->head_stride, quantum))
        return SPLITZIP_ERR_INVALID_ARG;
    // keeps every byte offset below 2^62
    const uint64_t limit = uint64_t(1) << 40;
    if (cache->page_stride > limit || cache->token_stride > limit || cache->head_stride > limit ||
        cache->page_stride > (uint64_t(1) << 48) / cache->pool_pages)
        return SPLITZIP_ERR_UNSUPPORTED;
    if (need_ptrs) {
        if (!cache->d_k || !cache->d_v || (addr(cache->d_k) & 15u) || (addr(cache->d_v) & 15u))
            return SPLITZIP_ERR_INVALID_ARG;
        if (fp8 && (!cache->d_k_scale || !cache->d_v_scale)) return SPLITZIP_ERR_INVALID_ARG;
        if ((!batch->d_page_table && batch->max_kv_len > 0) || (addr(batch->d_page_table) & 3u))
            return SPLITZIP_ERR_INVALID_ARG;
    }
    const int st = check_batch(batch, b, need_ptrs);
    if (st != SPLITZIP_OK) return st;
    uint32_t shift = 0;
    while ((1u << shift) < pt) ++shift;
    if (batch->table_stride < (uint64_t(batch->max_kv_len) + pt - 1u) >> shift ||
        batch->table_stride > (uint64_t(1) << 32))
        return SPLITZIP_ERR_INVALID_ARG;
    c->k = static_cast<uint8_t*>(cache->d_k);
    c->v = static_cast<uint8_t*>(cache->d_v);
    c->k_scale = cache->d_k_scale;
    c->v_scale = cache->d_v_scale;
    c->pool_pages = cache->pool_pages;
    c->page_stride = cache->page_stride * size;
    c->token_stride = cache->token_stride * size;
    c->head_stride = cache->head_stride * size;
    c->page_shift = shift;
    c->kv_heads = cache->kv_heads;
    c->head_dim = cache->head_dim;
    c->type = cache->type;
    return SPLITZIP_OK;
}

int check_rows(const splitzip_kv_rows_t* r, const KvBatch& b, uint32_t heads, uint32_t head_dim, KvRows* out) {
    if (!r || r->token_stride % 8u || r->head_stride % 8u) return SPLITZIP_ERR_INVALID_ARG;
    if (b.tokens > 0 && (!r->d || (reinterpret_cast<uintptr_t>(r->d) & 15u))) return SPLITZIP_ERR_INVALID_ARG;
    // rows must not overlap: heads apart by a row, tokens apart too
    if (heads > 1 && r->head_stride < head_dim) return SPLITZIP_ERR_INVALID_ARG;
    if (b.tokens > 1 && r->token_stride < head_dim) return SPLITZIP_ERR_INVALID_ARG;
    if (r->token_stride > (uint64_t(1) << 32) || r->head_stride > (uint64_t(1) << 32)) return SPLITZIP_ERR_UNSUPPORTED;
    out->d = static_cast<uint16_t*>(r->d);
    out->token_stride = r->token_stride;
    out->head_stride = r->head_stride;
    return SPLITZIP_OK;
}

}  // namespace splitzip

extern "C" int splitzip_kv_write(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch,
                                 const splitzip_kv_rows_t* k, const splitzip_kv_rows_t* v, int dtype, int* d_status,
                                 cudaStream_t stream) {
    return splitzip::kv_rw_call<true>(cache, batch, k, v, dtype, d_status, stream);
}

extern "C" int splitzip_kv_read(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch,
                                const splitzip_kv_rows_t* k, const splitzip_kv_rows_t* v, int dtype, int* d_status,
                                cudaStream_t stream) {
    return splitzip::kv_rw_call<false>(cache, batch, k, v, dtype, d_status, stream);
}
