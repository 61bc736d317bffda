// The accepted branch of a tree of drafted tokens, moved to the front of them
// in every layer's pages (splitzip_kv_keep).
//
// A move in place: new token path[i] goes to the place of new token i.  path
// ascends, so i <= path[i] < path[i + 1], and with the tokens taken in order,
// or a group of them read before the first is written, no source is
// overwritten before it is read.  One warp does all tokens of a sequence for
// its heads, so the order is its own and nobody else's.
//
// What bounds it: latency.  A warp's tokens come eight at a time, a group is a
// chain of path, table, row and store, and a step keeps a few tokens a sequence.
// In a graph, 64 sequences of 16 drafted tokens, 32 layers, 8 heads of 128, bytes
// of the tokens that move (those in their place already are skipped) read and
// written once:
//   125 of 342 kept tokens move    E5M2  8.2 us (2.0 TB/s)    BF16 15.4 (2.1)
//   194 of 258                          10.5 (2.4)                16.2 (3.1)
//   all of 512, every other one         15.8 (4.3)                26.7 (5.0)
// 2 sequences of 7, one layer, take 3.8, which is two launches.
#include <algorithm>
#include <cstring>

#include "kv_common.cuh"

namespace splitzip {
namespace {

constexpr int kWarps = 4;
constexpr int kGroup = 8;       // tokens read before the first of them is written
constexpr uint32_t kLayers = 64;  // of a launch

struct Pools {
    uint8_t *k, *v, *k_scale, *v_scale;
};

struct KeepArgs {
    KvCache c;  // without pointers
    KvBatch b;
    const int32_t *path, *kept;
    uint32_t parts;  // warps for a sequence, side and layer
    int* status;
    Pools layer[kLayers];
};

// LANES 16-byte pieces make a row of a head; a warp takes 32 / LANES heads of
// one side (K or V) of one sequence and layer.
template <bool FP8, int LANES>
__global__ void __launch_bounds__(kWarps * 32) kv_keep_kernel(const __grid_constant__ KeepArgs a) {
    constexpr uint32_t kHeads = 32 / LANES;
    const uint32_t lane = threadIdx.x & 31u, col = lane % LANES;
    const uint64_t warp = uint64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const uint64_t per_seq = 2ull * a.parts;
    const uint64_t seq = warp / per_seq;
    bool bad = false;
    if (seq < a.b.batch) {
        const uint32_t part = uint32_t(warp - seq * per_seq), side = part / a.parts;
        const uint32_t head = (part % a.parts) * kHeads + lane / LANES;
        const bool there = head < a.c.kv_heads;
        const KvSeq s = load_seq(a.b, uint32_t(seq));
        const int kept = a.kept[seq], first = s.n - s.t;
        const int32_t* path = a.path + s.row0;
        bad = !s.ok || kept < 0 || kept > s.t || (s.t > 0 && first < 0);
        if (!bad) {
            for (int i0 = 0; i0 < kept; i0 += 32) {
                const int i = i0 + int(lane);
                const bool in = i < kept;
                const int now = in ? path[i] : 0, last = in && i > 0 ? path[i - 1] : -1;
                bad |= __any_sync(~0u, in && (now <= last || now < 0 || now >= s.t));
            }
        }
        if (!bad) {
            const Pools& pool = a.layer[blockIdx.y];
            uint8_t* base = (side ? pool.v : pool.k) + uint64_t(head) * a.c.head_stride + col * 16u;
            uint8_t* scales = side ? pool.v_scale : pool.k_scale;
            const int32_t* table = a.b.table + seq * a.b.table_stride;
            const uint32_t slots = (1u << a.c.page_shift) - 1u;
            for (int i0 = 0; i0 < kept; i0 += kGroup) {
                // lanes 0 .. 7: where a token of the group comes from, 8 .. 15: where it goes
                const int mine = i0 + int(lane % kGroup);
                int32_t page = -1;
                uint32_t slot = 0;
                if (lane < 2 * kGroup && mine < kept) {
                    const int from = path[mine], pos = first + (lane < kGroup ? from : mine);
                    if (from != mine) {
                        page = table[uint32_t(pos) >> a.c.page_shift];
                        slot = uint32_t(pos) & slots;
                        if (page < 0 || uint64_t(page) >= a.c.pool_pages) {
                            bad = true;
                            page = -1;
                        }
                    }
                }
                uint4 x[kGroup];
                uint32_t scale[kGroup];
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    const int32_t from = __shfl_sync(~0u, page, k), to = __shfl_sync(~0u, page, k + kGroup);
                    const uint32_t at = __shfl_sync(~0u, slot, k);
                    if (from >= 0 && to >= 0 && there) {
                        x[k] = *reinterpret_cast<const uint4*>(base + uint64_t(from) * a.c.page_stride +
                                                               uint64_t(at) * a.c.token_stride);
                        if (FP8 && col == 0)
                            scale[k] = scales[((uint64_t(from) * a.c.kv_heads + head) << a.c.page_shift) + at];
                    }
                }
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    const int32_t from = __shfl_sync(~0u, page, k), to = __shfl_sync(~0u, page, k + kGroup);
                    const uint32_t at = __shfl_sync(~0u, slot, k + kGroup);
                    if (from >= 0 && to >= 0 && there) {
                        *reinterpret_cast<uint4*>(base + uint64_t(to) * a.c.page_stride +
                                                  uint64_t(at) * a.c.token_stride) = x[k];
                        if (FP8 && col == 0)
                            scales[((uint64_t(to) * a.c.kv_heads + head) << a.c.page_shift) + at] = uint8_t(scale[k]);
                    }
                }
            }
        }
    }
    wait_predecessor();  // the status word has been cleared
    if (bad) report(a.status, SPLITZIP_ERR_INVALID_ARG);
}

template <bool FP8, int LANES>
cudaError_t launch_keep(KeepArgs& a, uint32_t layers, cudaStream_t s) {
    constexpr uint32_t kHeads = 32 / LANES;
    a.parts = (a.c.kv_heads + kHeads - 1) / kHeads;
    const uint64_t grid = (uint64_t(a.b.batch) * 2 * a.parts + kWarps - 1) / kWarps;
    ChainedLaunch l(dim3(uint32_t(grid), layers), dim3(kWarps * 32), 0, s);
    return cudaLaunchKernelEx(&l.cfg, kv_keep_kernel<FP8, LANES>, a);
}

}  // namespace
}  // namespace splitzip

using namespace splitzip;

extern "C" int splitzip_kv_keep(const splitzip_kv_cache_t* h_caches, uint32_t count, const splitzip_kv_batch_t* batch,
                                const int32_t* d_path, const int32_t* d_kept, int* d_status, cudaStream_t stream) {
    if (!h_caches || count == 0 || !d_status || (reinterpret_cast<uintptr_t>(d_status) & 3u))
        return SPLITZIP_ERR_INVALID_ARG;
    if (count > SPLITZIP_MAX_LAYERS) return SPLITZIP_ERR_UNSUPPORTED;
    KeepArgs a;
    std::memset(&a, 0, sizeof(a));
    Pools pools[SPLITZIP_MAX_LAYERS];
    for (uint32_t i = 0; i < count; ++i) {
        const splitzip_kv_cache_t &c = h_caches[i], &o = h_caches[0];
        const int st = check_kv(&c, batch, &a.c, &a.b, true);
        if (st != SPLITZIP_OK) return st;
        if (c.pool_pages != o.pool_pages || c.page_stride != o.page_stride || c.token_stride != o.token_stride ||
            c.head_stride != o.head_stride || c.page_tokens != o.page_tokens || c.kv_heads != o.kv_heads ||
            c.head_dim != o.head_dim || c.type != o.type)
            return SPLITZIP_ERR_INVALID_ARG;
        pools[i] = Pools{a.c.k, a.c.v, a.c.k_scale, a.c.v_scale};
    }
    // what is given twice would be moved twice, at once
    const uint8_t* bases[2 * SPLITZIP_MAX_LAYERS];
    const auto twice = [&](uint8_t* Pools::*k, uint8_t* Pools::*v) {
        for (uint32_t i = 0; i < count; ++i) bases[2 * i] = pools[i].*k, bases[2 * i + 1] = pools[i].*v;
        std::sort(bases, bases + 2 * count);
        return std::adjacent_find(bases, bases + 2 * count) != bases + 2 * count;
    };
    if (twice(&Pools::k, &Pools::v)) return SPLITZIP_ERR_INVALID_ARG;
    if (!d_kept || (reinterpret_cast<uintptr_t>(d_kept) & 3u) || (reinterpret_cast<uintptr_t>(d_path) & 3u) ||
        (!d_path && a.b.tokens > 0))
        return SPLITZIP_ERR_INVALID_ARG;
    a.path = d_path;
    a.kept = d_kept;
    a.status = d_status;
    int sms, st;
    if ((st = device_sms(&sms)) != SPLITZIP_OK) return st;
    const bool fp8 = a.c.type == SPLITZIP_KV_FP8_E5M2 || a.c.type == SPLITZIP_KV_FP8_E4M3;
    if (fp8 && twice(&Pools::k_scale, &Pools::v_scale)) return SPLITZIP_ERR_INVALID_ARG;
    // the sequences' entries are looked at by the kernels themselves
    cudaError_t e = launch_kv_begin(KvBatch{}, d_status, nullptr, 0, stream);
    for (uint32_t i = 0; i < count && e == cudaSuccess; i += kLayers) {
        const uint32_t n = std::min(kLayers, count - i);
        std::memcpy(a.layer, pools + i, n * sizeof(Pools));
        if (a.c.head_dim == 128)
            e = fp8 ? launch_keep<true, 8>(a, n, stream) : launch_keep<false, 16>(a, n, stream);
        else
            e = fp8 ? launch_keep<true, 4>(a, n, stream) : launch_keep<false, 8>(a, n, stream);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? SPLITZIP_OK : SPLITZIP_ERR_CUDA;
}
