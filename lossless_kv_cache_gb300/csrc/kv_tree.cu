// Masks and positions of trees of drafted tokens (splitzip_kv_tree).
//
// Mathematics: bits(i) = {i} + bits(parent(i)), depth(i) = depth(parent(i)) + 1.
// A warp takes a sequence.  Of up to 32 tokens a lane holds one, and doubling
// its reach (bits |= bits of the ancestor reached so far, which then becomes
// that one's) finds all ancestors in five exchanges of registers.  A larger
// tree's lanes walk up from their tokens, which leaves masks of a few words.
//
// What bounds it: latency.  For small batches one CTA takes all sequences, so
// that it can set the status word itself and no other launch has to.  (TREE)
#include "kv_common.cuh"

namespace splitzip {
namespace {

constexpr int kSoloThreads = 1024, kThreads = 128;
constexpr uint32_t kSoloSequences = 256;

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
    if (!bad && s.t <= 32) {
        const bool there = int(lane) < s.t;
        const int p = there ? parent[lane] : -1;
        uint32_t bits = 1u << lane;
        int up = p;  // the nearest ancestor that is not among the bits
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const uint32_t theirs = __shfl_sync(~0u, bits, up & 31);
            const int above = __shfl_sync(~0u, up, up & 31);
            if (up >= 0) {
                bits |= theirs;
                up = above;
            }
        }
        const int depth = __popc(bits) - 1;
        // ancestors descend, so the nearest `window` of them are the highest bits
        if (a.window)
            for (int over = depth + 1 - int(min(a.window, 64u)); over > 0; --over) bits &= bits - 1u;
        if (there) {
            a.position[s.row0 + int(lane)] = first + depth;
            uint32_t* row = a.mask + uint64_t(uint32_t(s.row0) + lane) * a.words;
            row[0] = bits;
            for (uint32_t w = 1; w < a.words; ++w) row[w] = 0;
        }
        return true;
    }
    for (int i = int(lane); i < s.t; i += 32) {
        uint32_t* row = a.mask + uint64_t(uint32_t(s.row0 + i)) * a.words;
        uint32_t w = a.words, bits = 0;  // `bits` are of word w - 1, those from w on are written
        int depth = -1;
        for (int j = bad ? -1 : i; j >= 0; j = parent[j]) {
            ++depth;
            if (a.window && uint32_t(depth) >= a.window) continue;
            while (w > uint32_t(j >> 5) + 1u) {
                row[--w] = bits;
                bits = 0;
            }
            bits |= 1u << (j & 31);
        }
        while (w > 0) {
            row[--w] = bits;
            bits = 0;
        }
        a.position[s.row0 + i] = first + (bad ? i : depth);
    }
    return !bad;
}

__global__ void __launch_bounds__(kSoloThreads) kv_tree_solo_kernel(const __grid_constant__ TreeArgs a) {
    bool bad = false;
    for (uint32_t seq = threadIdx.x >> 5; seq < a.b.batch; seq += kSoloThreads / 32) bad |= !tree_of(a, seq);
    bad = __syncthreads_or(bad);
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
    if (a.b.batch <= kSoloSequences) {
        kv_tree_solo_kernel<<<1, kSoloThreads, 0, stream>>>(a);
        e = cudaGetLastError();
    } else {
        e = launch_kv_begin(KvBatch{}, d_status, nullptr, 0, stream);
        ChainedLaunch l(dim3((a.b.batch + kThreads / 32 - 1) / (kThreads / 32)), dim3(kThreads), 0, stream);
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&l.cfg, kv_tree_kernel, a);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? SPLITZIP_OK : SPLITZIP_ERR_CUDA;
}
