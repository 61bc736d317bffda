// Host side of splitzip_kv_attention and splitzip_kv_tree_attention: argument checks, workspace, and which
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

// The same of trees, whose second kernel (kv_tree_tile.cuh) has one tile of rows
// and is bound by the bytes too: 17 to 32 rows, of which the first reads the keys
// twice, take the second, but for short contexts, where its start counts.  In us
// for 8 kv heads of 128 in pages of 16, the first by 16 / 32 rows, then the second:
//   BF16, 1 sequence of 2,000     13 / 18     21       E5M2    14 / 17     24
//   BF16, 1 of 16,000             30 / 32     30       E5M2    35 / 38     33
//   BF16, 8 of 4,000              39 / 49     39       E5M2    38 / 53     44
//   BF16, 64 of 2,000            101 / 178   111       E5M2    95 / 164   137
//   BF16, 200 of 1,000           149 / 276   183       E5M2   151 / 265   282
// One threshold for all types: FP8, many sequences and just 32 rows is where the
// first would be the faster, by 6 % in the last line.
constexpr uint64_t kTreeStepRowsMax = 16;

struct Plan {
    uint32_t group, ctas;
    bool few;
    bool chunk;
    uint64_t plan_off, parts_off, ws_bytes;
};

// Places the parts of the workspace; returns its size.
uint64_t lay_out(Plan* p, uint64_t plan_bytes, uint64_t counters, uint64_t part_floats) {
    p->plan_off = align256(4ull * counters);
    p->parts_off = align256(p->plan_off + plan_bytes);
    return align256(p->parts_off + 4ull * 2 * p->ctas * part_floats);
}

int plan_for(const KvCache& c, const KvBatch& b, uint32_t q_heads, bool tree, Plan* p) {
    if (q_heads == 0 || q_heads % c.kv_heads != 0) return SPLITZIP_ERR_INVALID_ARG;
    p->group = q_heads / c.kv_heads;
    // the kernels count a sequence's rows, and up to a tile past them, in an int
    if (p->group > 64 || uint64_t(b.max_tokens) * p->group > 0x7FFFFF00u) return SPLITZIP_ERR_UNSUPPORTED;
    const uint64_t rows = uint64_t(b.tokens) * p->group;
    const uint64_t most = uint64_t(b.max_tokens) * p->group;
    p->chunk = most > (tree && !short_tree(b) ? kTreeStepRowsMax : kStepRowsMax);
    // tiles of rows over all sequences: each has a partial one at most
    const uint64_t tiles = std::min<uint64_t>((rows + 7) / 8 + b.batch, rows);
    p->ctas = step_ctas(tiles * c.kv_heads, b.max_kv_len);
    p->ws_bytes = lay_out(p, 0, p->ctas, step_part_floats(c.head_dim));
    p->few = false;
    if (!p->chunk) return SPLITZIP_OK;
    p->ctas = chunk_ctas(rows, b.batch, c.kv_heads, b.max_kv_len);
    const auto chunk_bytes = [&] {
        return lay_out(p, chunk_plan_bytes(p->ctas), 0, uint64_t(p->few ? kFewRows : kChunkRows) * (c.head_dim + 2));
    };
    if (most > kStepRowsMax) {
        // a step of the same rows, but fewer of a sequence, takes the other kernel: the size
        // is enough for both
        p->ws_bytes = std::max(p->ws_bytes, chunk_bytes());
        return SPLITZIP_OK;
    }
    // A tree of rows with which kv_attention takes the step kernel does with that one's size:
    // its parts have few rows, and their number follows what there is room for (all 152 CTAs
    // where the step kernel would have 306, which is so but for short contexts of few heads).
    static_assert(kFewRows == kStepRowsMax, "rows of a part");
    p->few = true;
    while (p->ctas > 1 && chunk_bytes() > p->ws_bytes) --p->ctas;
    return chunk_bytes() <= p->ws_bytes ? SPLITZIP_OK : SPLITZIP_ERR_UNSUPPORTED;
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
    if ((st = plan_for(c, b, q_heads, false, &p)) != SPLITZIP_OK) return st;
    *out_bytes = p.ws_bytes;
    return SPLITZIP_OK;
}

namespace {

// splitzip_kv_attention, and with a tree splitzip_kv_tree_attention.
int attend(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch, const splitzip_kv_tree_t* tree,
           bool is_tree, const splitzip_kv_rows_t* q, const splitzip_kv_rows_t* out, float* d_lse, int dtype,
           uint32_t q_heads, float scale, int causal, uint32_t window, void* d_ws, uint64_t ws_bytes, int* d_status,
           cudaStream_t stream) {
    AttentionArgs a;
    Plan p;
    int st = check_kv(cache, batch, &a.c, &a.b, true);
    if (st != SPLITZIP_OK) return st;
    a.mask = nullptr;
    a.position = nullptr;
    a.words = 0;
    if (is_tree) {
        if (a.b.max_tokens > SPLITZIP_MAX_TREE_TOKENS) return SPLITZIP_ERR_UNSUPPORTED;
        if ((st = check_tree(tree, a.b)) != SPLITZIP_OK) return st;
        a.mask = tree->d_mask;
        a.position = tree->d_position;
        a.words = tree->words;
        window = tree->window;
    }
    if ((st = plan_for(a.c, a.b, q_heads, is_tree, &p)) != SPLITZIP_OK) return st;
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
    a.part_blocks = (p.few ? kFewRows : kChunkRows) / kFewRows;
    a.status = d_status;
    int sms;
    if ((st = device_sms(&sms)) != SPLITZIP_OK) return st;
    if (p.chunk && a.b.tokens > 0) {
        const bool tile = uint64_t(a.b.max_tokens) * p.group <= kTreeTileRows;
        return (!is_tree ? launch_kv_chunk : tile ? launch_kv_tree_tile : launch_kv_tree_chunk)(
            a, a.q_half != 0, static_cast<uint8_t*>(d_ws) + p.plan_off, p.ctas, stream);
    }
    // the step kernel looks at all sequences itself, to share out their units
    if (launch_kv_begin(a.b.tokens > 0 ? KvBatch{} : a.b, d_status, a.counters, p.ctas, stream) != cudaSuccess) {
        cudaGetLastError();
        return SPLITZIP_ERR_CUDA;
    }
    if (a.b.tokens == 0) return SPLITZIP_OK;
    return (is_tree ? launch_kv_tree_step : launch_kv_step)(a, p.ctas, stream);
}

}  // namespace

extern "C" int splitzip_kv_attention(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch,
                                     const splitzip_kv_rows_t* q, const splitzip_kv_rows_t* out, float* d_lse,
                                     int dtype, uint32_t q_heads, float scale, int causal, uint32_t window,
                                     void* d_ws, uint64_t ws_bytes, int* d_status, cudaStream_t stream) {
    return attend(cache, batch, nullptr, false, q, out, d_lse, dtype, q_heads, scale, causal, window, d_ws, ws_bytes,
                  d_status, stream);
}

extern "C" int splitzip_kv_tree_attention(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch,
                                          const splitzip_kv_tree_t* tree, const splitzip_kv_rows_t* q,
                                          const splitzip_kv_rows_t* out, float* d_lse, int dtype, uint32_t q_heads,
                                          float scale, void* d_ws, uint64_t ws_bytes, int* d_status,
                                          cudaStream_t stream) {
    return attend(cache, batch, tree, true, q, out, d_lse, dtype, q_heads, scale, 1, 0, d_ws, ws_bytes, d_status,
                  stream);
}
