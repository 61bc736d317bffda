// Masks and positions of trees of drafted tokens (splitzip_kv_tree).
//
// Mathematics: bits(i) = {i} + bits(parent(i)), depth(i) = depth(parent(i)) + 1.
// A warp takes a sequence, 32 tokens at a time, a token a lane.  Doubling its
// reach (bits |= bits of the ancestor reached so far, whose next one it then
// goes on from) finds all ancestors among the 32 in five exchanges of registers;
// what lies before them is the mask of the nearest ancestor there, which has
// been written.
//
// What bounds it: latency.  One CTA takes small steps, so that it can set the
// status word itself and no other launch has to: in a graph 2 trees of 7 tokens
// 1.8 us, 32 of 16 2.2, 64 of 16 3.4 where two launches and many CTAs take 2.8.
// Large trees are slower in one SM's company of others (64 trees of 64 5.0 and
// 3.3 us; 16 of 1,024, whose masks are 32 words, 278 and 105).
#include "kv_common.cuh"

namespace splitzip {
namespace {

constexpr int kThreads = 128;
constexpr uint32_t kSoloSequences = 32, kSoloTokens = 64;  // a step that one CTA takes, a warp a sequence

struct TreeArgs {
    KvBatch b;
    const int32_t* parent;
    uint32_t* mask;
    int32_t* position;
    uint32_t words, window;
    int* status;
};

// One sequence, by a warp; whether it is in order.
__device__ __forceinline__ bool tree_of(const TreeArgs& a, uint32_t seq) {
    const uint32_t lane = threadIdx.x & 31u;
    const KvSeq s = load_seq(a.b, seq);
    if (!s.ok) return false;
    const int32_t* parent = a.parent + s.row0;
    const int first = s.n - s.t;
    bool bad = false;
    for (int i0 = 0; i0 < s.t; i0 += 32) {
        const int i = i0 + int(lane), p = i < s.t ? parent[i] : -1;
        bad |= p < -1 || p >= i;
    }
    bad = __any_sync(~0u, bad);
    for (int i0 = 0; i0 < s.t; i0 += 32) {
        const int i = i0 + int(lane), word = i0 / 32;
        uint32_t bits = 1u << lane;
        int up = i < s.t && !bad ? parent[i] : -1;  // the nearest ancestor that is not among the bits
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const uint32_t theirs = __shfl_sync(~0u, bits, up & 31);
            const int above = __shfl_sync(~0u, up, up & 31);
            if (up >= i0) {
                bits |= theirs;
                up = above;
            }
        }
        // Ancestors descend, so the nearest `window` of them are the highest bits.
        if (i < s.t && word == 0) {
            const int depth = __popc(bits) - 1;
            if (a.window)
                for (int over = depth + 1 - int(min(a.window, 64u)); over > 0; --over) bits &= bits - 1u;
            a.position[s.row0 + i] = first + (bad ? i : depth);
            uint32_t* row = a.mask + uint64_t(uint32_t(s.row0 + i)) * a.words;
            row[0] = bad ? 0u : bits;
            for (uint32_t w = 1; w < a.words; ++w) row[w] = 0;
        } else if (i < s.t) {
            // The mask of the nearest ancestor before these, which has as many of its own,
            // loses its lowest.
            uint32_t* row = a.mask + uint64_t(uint32_t(s.row0 + i)) * a.words;
            const uint32_t* from = up < 0 ? nullptr : a.mask + uint64_t(uint32_t(s.row0 + up)) * a.words;
            const int before = from ? a.position[s.row0 + up] - first + 1 : 0, in = __popc(bits);
            int over = 0;
            if (a.window) over = int(max(int64_t(0), min(int64_t(before), int64_t(a.window)) + in - int64_t(a.window)));
#pragma unroll 4
            for (int w = 0; w < word; ++w) {
                uint32_t x = from ? from[w] : 0u;
                if (over > 0) {
                    const int held = __popc(x);
                    if (over >= held) {
                        over -= held;
                        x = 0;
                    }
                    for (; over > 0 && x; --over) x &= x - 1u;
                }
                row[w] = x;
            }
            for (; over > 0; --over) bits &= bits - 1u;
            row[word] = bad ? 0u : bits;
            for (uint32_t w = uint32_t(word) + 1; w < a.words; ++w) row[w] = 0;
            a.position[s.row0 + i] = first + (bad ? i : before + in - 1);
        }
        __syncwarp();  // the next tokens read these
    }
    return !bad;
}

__global__ void __launch_bounds__(kSoloSequences * 32) kv_tree_solo_kernel(const __grid_constant__ TreeArgs a) {
    const uint32_t seq = threadIdx.x >> 5;
    const bool bad = __syncthreads_or(seq < a.b.batch && !tree_of(a, seq));
    if (threadIdx.x == 0) *a.status = bad ? SPLITZIP_ERR_INVALID_ARG : SPLITZIP_OK;
}

__global__ void __launch_bounds__(kThreads) kv_tree_kernel(const __grid_constant__ TreeArgs a) {
    const uint32_t seq = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const bool bad = seq < a.b.batch && !tree_of(a, seq);
    wait_predecessor();  // the status word has been cleared
    if (bad && (threadIdx.x & 31u) == 0) report(a.status, SPLITZIP_ERR_INVALID_ARG);
}

}  // namespace

int check_tree(const splitzip_kv_tree_t* tree, const KvBatch& b) {
    if (!tree || tree->words > SPLITZIP_MAX_TREE_TOKENS / 32 || tree->words < (b.max_tokens + 31u) / 32 ||
        (reinterpret_cast<uintptr_t>(tree->d_mask) & 3u) || (reinterpret_cast<uintptr_t>(tree->d_position) & 3u) ||
        (b.tokens > 0 && (!tree->d_mask || !tree->d_position)))
        return SPLITZIP_ERR_INVALID_ARG;
    return SPLITZIP_OK;
}

}  // namespace splitzip

using namespace splitzip;

extern "C" int splitzip_kv_tree(const splitzip_kv_batch_t* batch, const int32_t* d_parent, const splitzip_kv_tree_t* tree,
                                int* d_status, cudaStream_t stream) {
    TreeArgs a;
    int st = check_batch(batch, &a.b, true);
    if (st != SPLITZIP_OK) return st;
    if (a.b.max_tokens > SPLITZIP_MAX_TREE_TOKENS) return SPLITZIP_ERR_UNSUPPORTED;
    if ((st = check_tree(tree, a.b)) != SPLITZIP_OK) return st;
    if (!d_status || (reinterpret_cast<uintptr_t>(d_status) & 3u) || (reinterpret_cast<uintptr_t>(d_parent) & 3u) ||
        (a.b.tokens > 0 && !d_parent))
        return SPLITZIP_ERR_INVALID_ARG;
    a.parent = d_parent;
    a.mask = tree->d_mask;
    a.position = tree->d_position;
    a.words = tree->words;
    a.window = tree->window;
    a.status = d_status;
    int sms;
    if ((st = device_sms(&sms)) != SPLITZIP_OK) return st;
    cudaError_t e;
    if (a.b.batch <= kSoloSequences && a.b.max_tokens <= kSoloTokens) {
        kv_tree_solo_kernel<<<1, kSoloSequences * 32, 0, stream>>>(a);
        e = cudaGetLastError();
    } else {
        e = launch_kv_begin(KvBatch{}, d_status, nullptr, 0, stream);
        ChainedLaunch l(dim3((a.b.batch + kThreads / 32 - 1) / (kThreads / 32)), dim3(kThreads), 0, stream);
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&l.cfg, kv_tree_kernel, a);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? SPLITZIP_OK : SPLITZIP_ERR_CUDA;
}
