// Host side of splitzip_kv_attention: argument checks, workspace, and which
// kernel a step takes.
#include <algorithm>
#include <cmath>

#include "kv_attention.cuh"

using namespace splitzip;

namespace {

uint64_t align256(uint64_t x) { return (x + 255u) & ~uint64_t(255); }

// Rows of a sequence (new tokens by query heads of a group) up to which a step
// takes the kernel of 16-row tiles, which is bound by the bytes of the cache,
// rather than the tensor cores' 128-row tiles.  It reads the keys again for
// each tile, so its time grows with the rows where the other's does not.  In us
// for 8 kv heads of 128 and pages of 16, the first kernel by 16 / 32 / 64 rows,
// then the second at any of them:
//   BF16, 1 sequence of 16,384    27 / 30 / 46     34
//   BF16, 8 of 4,096              38 / 48 / 76     51
//   BF16, 32 of 2,048             57 / 97 / 170    91
//   E5M2, 1 of 16,384             33 / 36 / 48     40
//   E5M2, 8 of 4,096              34 / 49 / 80     70
//   E5M2, 32 of 2,048             55 / 88 / 156    130
// At 32 rows the first kernel is the faster but for BF16, 32 of 2,048.  64 dims and
// other numbers of heads follow this table without one of their own.
constexpr uint64_t kStepRowsMax = 32;

struct Plan {
    uint32_t group, ctas;
    bool chunk;
    uint64_t plan_off, parts_off, ws_bytes;
};

// Places the parts of the workspace; returns its size.
uint64_t lay_out(Plan* p, uint64_t plan_bytes, uint64_t counters, uint64_t part_floats) {
    p->plan_off = align256(4ull * counters);
    p->parts_off = align256(p->plan_off + plan_bytes);
    return align256(p->parts_off + 4ull * 2 * p->ctas * part_floats);
}

int plan_for(const KvCache& c, const KvBatch& b, uint32_t q_heads, Plan* p) {
    if (q_heads == 0 || q_heads % c.kv_heads != 0) return SPLITZIP_ERR_INVALID_ARG;
    p->group = q_heads / c.kv_heads;
    // the kernels count a sequence's rows, and up to a tile past them, in an int
    if (p->group > 64 || uint64_t(b.max_tokens) * p->group > 0x7FFFFF00u) return SPLITZIP_ERR_UNSUPPORTED;
    const uint64_t rows = uint64_t(b.tokens) * p->group;
    p->chunk = uint64_t(b.max_tokens) * p->group > kStepRowsMax;
    // tiles of rows over all sequences: each has a partial one at most
    const uint64_t tiles = std::min<uint64_t>((rows + 7) / 8 + b.batch, rows);
    p->ctas = step_ctas(tiles * c.kv_heads, b.max_kv_len);
    p->ws_bytes = lay_out(p, 0, p->ctas, step_part_floats(c.head_dim));
    if (p->chunk) {
        // a step of the same rows, but fewer of a sequence, takes the other kernel:
        // the size is enough for both
        p->ctas = chunk_ctas(rows, b.batch, c.kv_heads, b.max_kv_len);
        p->ws_bytes = std::max(p->ws_bytes, lay_out(p, chunk_plan_bytes(p->ctas), 0, chunk_part_floats(c.head_dim)));
    }
    return SPLITZIP_OK;
}

}  // namespace

extern "C" int splitzip_kv_attention_workspace_size(const splitzip_kv_cache_t* cache,
                                                    const splitzip_kv_batch_t* batch, uint32_t q_heads,
                                                    uint64_t* out_bytes) {
    KvCache c;
    KvBatch b;
    Plan p;
    int st = check_kv(cache, batch, &c, &b, false);
    if (st != SPLITZIP_OK) return st;
    if (!out_bytes) return SPLITZIP_ERR_INVALID_ARG;
    if ((st = plan_for(c, b, q_heads, &p)) != SPLITZIP_OK) return st;
    *out_bytes = p.ws_bytes;
    return SPLITZIP_OK;
}

extern "C" int splitzip_kv_attention(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch,
                                     const splitzip_kv_rows_t* q, const splitzip_kv_rows_t* out, float* d_lse,
                                     int dtype, uint32_t q_heads, float scale, int causal, uint32_t window,
                                     void* d_ws, uint64_t ws_bytes, int* d_status, cudaStream_t stream) {
    AttentionArgs a;
    Plan p;
    int st = check_kv(cache, batch, &a.c, &a.b, true);
    if (st != SPLITZIP_OK) return st;
    if ((st = plan_for(a.c, a.b, q_heads, &p)) != SPLITZIP_OK) return st;
    if (!kv_dtype_fits(a.c.type, dtype) || !std::isfinite(scale)) return SPLITZIP_ERR_INVALID_ARG;
    if ((st = check_rows(q, a.b, q_heads, a.c.head_dim, &a.q)) != SPLITZIP_OK) return st;
    if ((st = check_rows(out, a.b, q_heads, a.c.head_dim, &a.out)) != SPLITZIP_OK) return st;
    if (!d_status || (reinterpret_cast<uintptr_t>(d_status) & 3u) || (reinterpret_cast<uintptr_t>(d_lse) & 3u))
        return SPLITZIP_ERR_INVALID_ARG;
    if (ws_bytes < p.ws_bytes) return SPLITZIP_ERR_CAPACITY;
    if (!d_ws || (reinterpret_cast<uintptr_t>(d_ws) & 15u)) return SPLITZIP_ERR_INVALID_ARG;
    a.lse = d_lse;
    a.q_heads = q_heads;
    a.q_half = dtype == SPLITZIP_FP16;
    a.group = p.group;
    a.scale_log2 = float(double(scale) * 1.4426950408889634);
    a.negate = 0;
    a.lag = 0.f;
    if (p.chunk) {
        a.negate = a.scale_log2 < 0.f;
        a.scale_log2 = std::max(std::fabs(a.scale_log2), 1.17549435e-38f);
        a.lag = 8.f / a.scale_log2;
    }
    a.causal = causal != 0;
    a.window = std::min(window, 1u << 30);  // past every position
    a.counters = static_cast<uint32_t*>(d_ws);
    a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + p.parts_off);
    a.status = d_status;
    int sms;
    if ((st = device_sms(&sms)) != SPLITZIP_OK) return st;
    if (p.chunk && a.b.tokens > 0)
        return launch_kv_chunk(a, a.q_half != 0, static_cast<uint8_t*>(d_ws) + p.plan_off, p.ctas, stream);
    // the step kernel looks at all sequences itself, to share out their units
    if (launch_kv_begin(a.b.tokens > 0 ? KvBatch{} : a.b, d_status, a.counters, p.ctas, stream) != cudaSuccess) {
        cudaGetLastError();
        return SPLITZIP_ERR_CUDA;
    }
    return a.b.tokens > 0 ? launch_kv_step(a, p.ctas, stream) : int(SPLITZIP_OK);
}
