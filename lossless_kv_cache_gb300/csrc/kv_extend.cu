// Page tables, lengths, slots and positions of a step, built on the GPU
// (splitzip_kv_extend).
//
// Arithmetic: with n' = n - drop + new tokens and need = ceil(n' / P) pages, a
// sequence gives up max(0, held - need) pages or takes max(0, need - held).
// The free list is a stack, so where each page goes, or comes from, follows
// from sums over the sequences:
//   page j that sequence b gives up  -> free[count + F - less_upto(b) + held_b - 1 - j]
//   page j that sequence b takes     <- free[count + F - 1 - more_before(b) - (j - held_b)]
// (F: all pages given up).  The order does not depend on timing.
//
// What bounds it: latency, of loads that follow one another (lengths, the
// list, the table), for there are 28 bytes a sequence and 12 a row.  One CTA
// checks and sums everything before anything is written, since the arrays may
// be updated in place and a step that does not fit changes nothing.  A page
// that is taken begins with a new token, so the rows' threads enter the pages
// into the tables.  64 sequences of a token take 4.3 us in a graph, 256 with 85,000
// tokens 9.6, of which launches and the plan's chain of loads are 7.
#include "kv_common.cuh"

namespace splitzip {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 128;
constexpr int kWarpRows = 128;  // rows of a warp of the second kernel
// Up to so many rows the planning CTA does them itself: 1,792 rows of 256 sequences
// take 5.3 us so and 7.2 with a second kernel, 4,000 of 8 6.2 and 6.8, 4,096 of 256
// 7.0 and 7.6, 7,936 of them 9.5 and 7.7.
constexpr uint32_t kRowsInPlan = 4096;

struct ExtendArgs {
    int32_t* free;
    const int32_t *count_in, *held_in, *len_in, *more_tokens, *drop;
    int32_t *count, *held, *len, *cu, *table, *position;
    int64_t* slot;
    uint64_t table_stride;
    uint32_t table_pages, pool_pages, page_shift, batch, tokens, max_tokens, max_kv_len;
    int4* plan;  // workspace: of a sequence its length, pages held before, pages taken before it; entry `batch`: top
    int* status;
};

struct Sums {
    uint64_t rows, more, less;
    __device__ Sums& operator+=(const Sums& o) {
        rows += o.rows, more += o.more, less += o.less;
        return *this;
    }
};

// A sequence of the step; not ok: entries out of range.
struct Extent {
    int64_t n;  // tokens after the step
    int t, held, need;
    bool ok;
    __device__ Sums sums() const {
        return Sums{uint64_t(ok ? t : 0), uint64_t(ok && need > held ? need - held : 0),
                    uint64_t(ok && held > need ? held - need : 0)};
    }
};

__device__ __forceinline__ Extent extent_of(const ExtendArgs& a, uint32_t b) {
    const int64_t n = a.len_in[b], d = a.drop ? a.drop[b] : 0, p = (int64_t(1) << a.page_shift) - 1;
    Extent e;
    e.t = a.more_tokens[b];
    e.held = a.held_in[b];
    e.n = n - d + e.t;
    const int64_t need = (e.n + p) >> a.page_shift;
    e.ok = e.t >= 0 && e.t <= int(a.max_tokens) && n >= 0 && d >= 0 && d <= n && e.n <= int64_t(a.max_kv_len) &&
           need <= int64_t(a.table_pages) && e.held >= 0 && int64_t(e.held) >= ((n + p) >> a.page_shift) &&
           e.held <= int64_t(a.table_pages) && e.held <= int64_t(a.pool_pages);
    e.need = e.ok ? int(need) : 0;
    return e;
}

// Positions, slots and new table entries of rows first .. last - 1, by a warp.
// Everything that it reads was written before it came here.
__device__ __forceinline__ void map_rows(const ExtendArgs& a, uint32_t first, uint32_t last) {
    const uint32_t lane = threadIdx.x & 31u;
    // sequences by their starts alone (find_seq reads nothing else)
    KvBatch starts{};
    starts.cu = a.cu;
    starts.batch = a.batch;
    const int seq0 = find_seq(starts, int(first), lane);
    if (seq0 < 0) return;
    uint32_t base = uint32_t(seq0);
    const int top = a.plan[a.batch].x;
    for (uint32_t r0 = first; r0 < last; r0 += 32) {
        const uint32_t row = r0 + lane;
        // the row's sequence: the last whose start is at most `row`, 32 candidates at a time
        uint32_t b = 0;
        bool found = row >= last;
        while (true) {
            const int start = a.cu[min(base + 1 + lane, a.batch)];
            uint32_t upto = 0;  // how many of these starts are at most `row`
#pragma unroll
            for (uint32_t step = 16; step > 0; step >>= 1)
                upto += __shfl_sync(~0u, start, int(upto + step - 1)) <= int(row) ? step : 0;
            upto += __shfl_sync(~0u, start, int(min(upto, 31u))) <= int(row) && upto == 31 ? 1 : 0;
            if (!found && (upto < 32 || base + 32 >= a.batch)) {
                b = base + upto;
                found = true;
            }
            if (__all_sync(~0u, found)) break;
            base += 32;
        }
        const bool there = row < last && b < a.batch;
        if (there) {
            const int4 s = a.plan[b];
            const int pos = s.x - (a.cu[b + 1] - int(row)), j = pos >> a.page_shift;
            const int in_page = pos & ((1 << a.page_shift) - 1);
            int32_t* entry = a.table + uint64_t(b) * a.table_stride + uint32_t(j);
            int32_t page;
            if (j < s.y) {
                page = *entry;
            } else {
                page = a.free[top - 1 - s.z - (j - s.y)];
                if (in_page == 0) *entry = page;
            }
            if (a.position) a.position[row] = pos;
            if (a.slot) a.slot[row] = (int64_t(page) << a.page_shift) + in_page;
        }
        // the next rows begin where the last of these was found
        base = __reduce_max_sync(~0u, there ? b : base);
    }
}

__global__ void __launch_bounds__(kPlanThreads)
    kv_extend_plan_kernel(const __grid_constant__ ExtendArgs a, int map_here) {
    release_successor();
    constexpr uint32_t kWarps = kPlanThreads / 32;
    __shared__ Sums s_warp[kWarps];
    __shared__ uint32_t s_upto[kPlanThreads];
    __shared__ int s_held[kPlanThreads];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    // inclusive sums over the CTA's threads; total: over all of them
    const auto scan = [&](const Sums& mine, Sums* total) -> Sums {
        Sums x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sums y{__shfl_up_sync(~0u, x.rows, d), __shfl_up_sync(~0u, x.more, d), __shfl_up_sync(~0u, x.less, d)};
            if (int(lane) >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        Sums all = s_warp[lane];  // as many warps as lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sums y{__shfl_up_sync(~0u, all.rows, d), __shfl_up_sync(~0u, all.more, d),
                         __shfl_up_sync(~0u, all.less, d)};
            if (int(lane) >= d) all += y;
        }
        const int before = int(warp) - 1 + (warp == 0);
        const Sums b{__shfl_sync(~0u, all.rows, before), __shfl_sync(~0u, all.more, before),
                     __shfl_sync(~0u, all.less, before)};
        if (warp > 0) x += b;
        *total = Sums{__shfl_sync(~0u, all.rows, 31), __shfl_sync(~0u, all.more, 31), __shfl_sync(~0u, all.less, 31)};
        return x;
    };
    static_assert(kWarps == 32, "the scan over warps");

    const int64_t count = *a.count_in;
    Sums all{0, 0, 0}, upto{0, 0, 0};
    Extent e{0, 0, 0, 0, true};
    bool bad = false;
    for (uint32_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        e = Extent{0, 0, 0, 0, true};
        if (b0 + tid < a.batch) e = extent_of(a, b0 + tid);
        bad |= !e.ok;
        Sums round;
        upto = scan(e.sums(), &round);
        all += round;
    }
    bad = __syncthreads_or(bad);
    bad |= count < 0 || uint64_t(count) + all.less > a.pool_pages || all.rows > a.tokens;
    const bool full = !bad && all.more > uint64_t(count) + all.less;
    const bool go = !bad && !full;
    const int64_t top = count + int64_t(go ? all.less : 0);
    Sums before{0, 0, 0};
    for (uint32_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const uint32_t b = b0 + tid;
        const bool there = b < a.batch;
        Sums round = all;  // the only one of up to kPlanThreads sequences
        const uint64_t before_round = before.less;
        if (a.batch > kPlanThreads) {
            e = Extent{0, 0, 0, 0, true};
            if (there) e = extent_of(a, b);
            upto = scan(e.sums(), &round);
            upto += before;
            before += round;
        }
        const Sums own = e.sums();
        if (there && go) {
            a.cu[b] = int(upto.rows - own.rows);
            a.plan[b] = make_int4(int(e.n), e.held, int(upto.more - own.more), 0);
            a.len[b] = int(e.n);
            a.held[b] = e.need;
        } else if (there) {
            const int32_t n = a.len_in[b], h = a.held_in[b];
            a.cu[b] = 0;
            a.len[b] = n;
            a.held[b] = h;
        }
        // Pages given up, a thread each whosever they are: some sequences give many, most none
        // (with a warp a sequence 64 of them, half of which gave up some, took 9.1 us, so 5.0).
        const uint32_t given = go ? uint32_t(round.less) : 0u;
        if (given > 0) {
            __syncthreads();
            s_upto[tid] = uint32_t(upto.less - before_round);
            s_held[tid] = e.held;
            __syncthreads();
            for (uint32_t k = tid; k < given; k += kPlanThreads) {
                uint32_t at = 0, last = kPlanThreads - 1;  // the first sequence that s_upto > k
                while (at < last) {
                    const uint32_t mid = (at + last) / 2;
                    if (s_upto[mid] > k)
                        last = mid;
                    else
                        at = mid + 1;
                }
                const int held = s_held[at], j = held - int(s_upto[at] - k);
                a.free[top - int64_t(before_round) - int64_t(s_upto[at]) + held - 1 - j] =
                    a.table[uint64_t(b0 + at) * a.table_stride + uint32_t(j)];
            }
        }
    }
    if (tid == 0) {
        a.cu[a.batch] = go ? int(all.rows) : 0;
        a.plan[a.batch] = make_int4(int(top), 0, 0, 0);
        *a.count = int(go ? top - int64_t(all.more) : count);
        *a.status = bad ? SPLITZIP_ERR_INVALID_ARG : full ? SPLITZIP_ERR_CAPACITY : SPLITZIP_OK;
    }
    if (!map_here || !go) return;
    __syncthreads();
    const uint32_t rows = uint32_t(all.rows), each = (rows + kWarps - 1) / kWarps;
    if (warp * each < rows) map_rows(a, warp * each, min(rows, (warp + 1) * each));
}

__global__ void __launch_bounds__(kRowThreads) kv_extend_rows_kernel(const __grid_constant__ ExtendArgs a) {
    wait_predecessor();
    const uint32_t rows = uint32_t(a.cu[a.batch]);
    const uint64_t first = (uint64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5)) * kWarpRows;
    if (first < rows) map_rows(a, uint32_t(first), min(rows, uint32_t(first) + kWarpRows));
}

uint64_t workspace(uint32_t batch) { return (uint64_t(batch) + 1) * sizeof(int4); }

bool misaligned(const void* p, uintptr_t by) { return !p || (reinterpret_cast<uintptr_t>(p) & (by - 1u)); }
bool misaligned_or_null(const void* p, uintptr_t by) { return reinterpret_cast<uintptr_t>(p) & (by - 1u); }

}  // namespace
}  // namespace splitzip

using namespace splitzip;

extern "C" int splitzip_kv_extend_workspace_size(uint32_t batch, uint64_t* out_bytes) {
    if (!out_bytes || batch == 0) return SPLITZIP_ERR_INVALID_ARG;
    if (batch > 65536u) return SPLITZIP_ERR_UNSUPPORTED;
    *out_bytes = workspace(batch);
    return SPLITZIP_OK;
}

extern "C" int splitzip_kv_extend(const splitzip_kv_pages_t* pages, const int32_t* d_new, const int32_t* d_drop,
                                  const splitzip_kv_step_t* step, void* d_ws, uint64_t ws_bytes, int* d_status,
                                  cudaStream_t stream) {
    if (!pages || !step) return SPLITZIP_ERR_INVALID_ARG;
    const uint32_t pt = pages->page_tokens;
    if (pt == 0 || pt > 65536u || (pt & (pt - 1u)) || pages->batch == 0 || pages->pool_pages == 0 ||
        step->max_tokens > step->tokens || pages->table_pages > pages->table_stride)
        return SPLITZIP_ERR_INVALID_ARG;
    if (pages->batch > 65536u || pages->pool_pages > 0x7FFFFFFFu || pages->table_pages > 0x7FFFFFFFu ||
        pages->table_stride > (uint64_t(1) << 32) || step->tokens >= (1u << 30) || step->max_kv_len >= (1u << 30))
        return SPLITZIP_ERR_UNSUPPORTED;
    for (const void* p : {static_cast<const void*>(pages->d_free), static_cast<const void*>(pages->d_free_count),
                          static_cast<const void*>(pages->d_held), static_cast<const void*>(pages->d_kv_len),
                          static_cast<const void*>(d_new), static_cast<const void*>(step->d_free_count),
                          static_cast<const void*>(step->d_held), static_cast<const void*>(step->d_kv_len),
                          static_cast<const void*>(step->d_cu_tokens), static_cast<const void*>(d_status)})
        if (misaligned(p, 4)) return SPLITZIP_ERR_INVALID_ARG;
    if (misaligned_or_null(d_drop, 4) || misaligned_or_null(step->d_position, 4) || misaligned_or_null(step->d_slot, 8) ||
        misaligned_or_null(pages->d_page_table, 4) || (!pages->d_page_table && pages->table_pages > 0))
        return SPLITZIP_ERR_INVALID_ARG;
    if (ws_bytes < workspace(pages->batch)) return SPLITZIP_ERR_CAPACITY;
    if (misaligned(d_ws, 16)) return SPLITZIP_ERR_INVALID_ARG;
    ExtendArgs a;
    a.free = pages->d_free;
    a.count_in = pages->d_free_count;
    a.held_in = pages->d_held;
    a.len_in = pages->d_kv_len;
    a.more_tokens = d_new;
    a.drop = d_drop;
    a.count = step->d_free_count;
    a.held = step->d_held;
    a.len = step->d_kv_len;
    a.cu = step->d_cu_tokens;
    a.table = pages->d_page_table;
    a.position = step->d_position;
    a.slot = step->d_slot;
    a.table_stride = pages->table_stride;
    a.table_pages = pages->table_pages;
    a.pool_pages = pages->pool_pages;
    a.page_shift = 0;
    while ((1u << a.page_shift) < pt) ++a.page_shift;
    a.batch = pages->batch;
    a.tokens = step->tokens;
    a.max_tokens = step->max_tokens;
    a.max_kv_len = step->max_kv_len;
    a.plan = static_cast<int4*>(d_ws);
    a.status = d_status;
    int sms, st;
    if ((st = device_sms(&sms)) != SPLITZIP_OK) return st;
    const bool map_here = a.tokens <= kRowsInPlan;
    kv_extend_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, map_here);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && !map_here) {
        const uint32_t per_cta = kRowThreads / 32 * kWarpRows;
        ChainedLaunch l(dim3((a.tokens + per_cta - 1) / per_cta), dim3(kRowThreads), 0, stream);
        e = cudaLaunchKernelEx(&l.cfg, kv_extend_rows_kernel, a);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? SPLITZIP_OK : SPLITZIP_ERR_CUDA;
}
