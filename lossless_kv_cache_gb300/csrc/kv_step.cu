// Attention of few rows a sequence over a paged cache: decoding steps, one
// new token or a handful of drafted ones.
//
// Mathematics: one pass over the keys with a running maximum and sum (online
// softmax).  For each row m' = max(m, s), l' = l 2^(m-m') + sum 2^(s-m'),
// o' = o 2^(m-m') + sum 2^(s-m') v, in base 2 with the factor log2(e) in the
// score's scale; out = o / l.  Parts over different keys join by the same rule.
//
// What bounds it: HBM.  A tile of 16 rows does 64 operations a byte of a BF16
// cache, far below the ridge, so the layout is chosen for bytes in flight: a
// CTA is four warps, each with its own ring of stages of 16 keys (K and V)
// in shared memory filled by its own 16-byte cp.async copies, and no barrier
// between warps until an item ends.  The query heads that share a kv head are
// rows of one tile, so the cache is read once for all of them.
#include <algorithm>
#include <atomic>

#include "kv_attention.cuh"
#include "tma_pipeline.cuh"

namespace splitzip {
namespace {

constexpr int kUnit = 64;      // keys of a unit: 16 for each of the four warps
constexpr int kWarps = 4;
constexpr int kKeys = 16;      // keys of a stage
constexpr int kMinUnits = 4;   // least share of a CTA
constexpr uint32_t kStepCtas = 304;  // two on each of 152 SMs

__device__ __forceinline__ void mma_16816(bool half, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (half)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// 16 bytes to shared memory, asynchronously; zeros where !there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// FMT 0: cache of the queries' 16-bit type, 1: E5M2, 2: E4M3.
template <int FMT, bool H, int D>
struct Step {
    static constexpr bool kFp8 = FMT != 0;
    static constexpr bool kE5M2 = FMT == 1;
    // P and V are multiplied in FP16 where the cache is FP16, else in BF16: FP8
    // values are exact in it, and weights times V's scales keep their range.
    static constexpr bool kPvHalf = !kFp8 && H;
    // FP16 weights are 2^14 times the exponentials (at most 1), so that those
    // down to 2^-28 keep all bits; the factor cancels in o / l.
    static constexpr float kShift = kPvHalf ? 14.f : 0.f;
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kChunks = kRowBytes / 16;     // 16-byte pieces of a row
    static constexpr int kRowsACopy = 32 / kChunks;    // rows a warp copies with one instruction
    static constexpr int kCopies = kKeys / kRowsACopy;
    static constexpr int kSideBytes = kKeys * kRowBytes;
    static constexpr int kStageBytes = 2 * kSideBytes;
    static constexpr int kStages = 24576 / kStageBytes > 8 ? 8 : 24576 / kStageBytes;
    static constexpr int kRing = kStages * kStageBytes;  // a warp's
    static constexpr int kScaleSlots = kFp8 ? kStages * kKeys * 8 : 0;
    static constexpr int kMergeBytes = kWarps * kStepRows * (D + 2) * 4;
    static constexpr int kRingBytes = kWarps * kRing > kMergeBytes ? kWarps * kRing : kMergeBytes;
    static constexpr int kSmem = kRingBytes + kWarps * kScaleSlots;
    static constexpr int kPartFloats = kStepRows * (D + 2);

    // Where piece c of key row r lies in its side of a stage: permuted within
    // 128-byte lines so that each access below meets every bank once.
    static __device__ __forceinline__ uint32_t place_k(uint32_t r, uint32_t c) {
        if (!kFp8) return r * kRowBytes + ((c ^ (r & 7u)) << 4);
        if (D == 128) return r * kRowBytes + ((c ^ ((r & 1u) << 2)) << 4);
        return r * kRowBytes + (c << 4);
    }
    static __device__ __forceinline__ uint32_t place_v(uint32_t r, uint32_t c) {
        if (!kFp8) return r * kRowBytes + ((c ^ (r & 7u)) << 4);
        if (D == 128) return r * kRowBytes + ((c ^ (r & 6u)) << 4);
        return (r >> 1) * 128u + ((((r & 1u) * 4u + c) ^ (((r >> 1) & 3u) << 1)) << 4);
    }
    // Column of the output that accumulator j, element e of quad lane t holds.
    static __device__ __forceinline__ int out_dim(int j, int t, int e) {
        return kFp8 ? (D / 8) * (2 * t + e) + j : 8 * j + 2 * t + e;
    }
};

// Whether 16 bytes of a cache hold an infinity or a NaN.
template <int FMT, bool H>
__device__ __forceinline__ bool special16(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (FMT == 0) {
            constexpr uint32_t kInf = H ? 0x7C00u : 0x7F80u;
            any |= (w[i] & 0x7FFFu) >= kInf || ((w[i] >> 16) & 0x7FFFu) >= kInf;
        } else {
            constexpr uint32_t kFirst = FMT == 1 ? 0x7Cu : 0x7Fu;
#pragma unroll
            for (int k = 0; k < 4; ++k) any |= ((w[i] >> (8 * k)) & 0x7Fu) >= kFirst;
        }
    }
    return any;
}

template <int FMT, bool H, int D>
__global__ void __launch_bounds__(kWarps * 32) kv_step_kernel(const __grid_constant__ AttentionArgs a) {
    using S = Step<FMT, H, D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_scan[kWarps + 1];
    __shared__ uint32_t s_last;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const int g = int(lane >> 2), t4 = int(lane & 3u);
    uint8_t* ring = smem + warp * S::kRing;
    const uint32_t ring_u32 = smem_u32(ring);
    int64_t* scale_ring = reinterpret_cast<int64_t*>(smem + S::kRingBytes + warp * S::kScaleSlots);
    const uint32_t kv_heads = a.c.kv_heads;
    bool bad = false;

    // A sequence's units: those of all its rows' keys, for each kv head and row tile.
    const auto tiles_of = [&](const KvSeq& s) { return (s.t * int(a.group) + kStepRows - 1) / kStepRows; };
    const auto weight_of = [&](uint32_t b) -> uint64_t {
        const KvSeq s = load_seq(a.b, b);
        bad |= !s.ok;
        if (s.t == 0) return 0;
        return uint64_t(unit_count(visible(a, s, 0, s.t - 1), kUnit)) * kv_heads * uint32_t(tiles_of(s));
    };
    // Inclusive scan over the CTA's threads of one weight each; s_scan[kWarps]: the total.
    const auto scan = [&](uint64_t w) -> uint64_t {
        uint64_t x = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(~0u, x, d);
            if (int(lane) >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = x;
        __syncthreads();
        uint64_t before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < int(warp)) before += s_scan[i];
            total += s_scan[i];
        }
        __syncthreads();
        if (tid == 0) s_scan[kWarps] = total;
        return x + before;
    };
    uint64_t units = 0;
    for (uint32_t b0 = 0; b0 < a.b.batch; b0 += kWarps * 32) {
        scan(b0 + tid < a.b.batch ? weight_of(b0 + tid) : 0);
        __syncthreads();
        units += s_scan[kWarps];
    }
    const uint64_t most = (units + kMinUnits - 1) / kMinUnits;
    const uint32_t ctas = most < gridDim.x ? uint32_t(most) : gridDim.x;
    uint64_t u = 0, end = 0;
    if (blockIdx.x < ctas) {
        u = share_start(units, ctas, blockIdx.x);
        end = share_start(units, ctas, uint64_t(blockIdx.x) + 1);
    }
    // the sequence that holds unit u, and where its units begin
    uint32_t b = 0;
    uint64_t b_start = 0;
    if (u < end) {
        __shared__ uint32_t s_b;
        __shared__ uint64_t s_start;
        uint64_t base = 0;
        for (uint32_t b0 = 0; b0 < a.b.batch; b0 += kWarps * 32) {
            const uint64_t w = b0 + tid < a.b.batch ? weight_of(b0 + tid) : 0;
            const uint64_t upto = base + scan(w);
            if (w > 0 && u >= upto - w && u < upto) {
                s_b = b0 + tid;
                s_start = upto - w;
            }
            __syncthreads();
            base += s_scan[kWarps];
            if (base > u) break;
        }
        b = s_b;
        b_start = s_start;
    }

    while (u < end) {
        // the item that holds unit u
        const KvSeq s = load_seq(a.b, b);
        const KeyRange all = visible(a, s, 0, s.t > 0 ? s.t - 1 : 0);
        const int per_item = unit_count(all, kUnit);
        const uint64_t b_units = s.t == 0 ? 0 : uint64_t(per_item) * kv_heads * uint32_t(tiles_of(s));
        if (u >= b_start + b_units) {  // on to the next sequence
            b_start += b_units;
            ++b;
            continue;
        }
        const uint64_t item = (u - b_start) / uint32_t(per_item);
        const uint64_t item_start = b_start + item * uint32_t(per_item), item_end = item_start + uint32_t(per_item);
        const uint32_t head = uint32_t(item % kv_heads);
        const int row_first = int(item / kv_heads) * kStepRows;
        const int rows = min(kStepRows, s.t * int(a.group) - row_first);
        const uint64_t stop = item_end < end ? item_end : end;
        const int n_units = int(stop - u);
        const int i0 = row_first / int(a.group), i1 = (row_first + rows - 1) / int(a.group);
        const KeyRange keys = visible(a, s, i0, i1);
        const int base = (all.lo / kUnit + int(u - item_start)) * kUnit + int(warp) * kKeys;

        // queries, as the first operand of the products: rows g and g + 8
        uint32_t q[D / 16][4];
        KeyRange see[2];
#pragma unroll
        for (int r2 = 0; r2 < 2; ++r2) {
            const int r = g + 8 * r2;
            const bool there = r < rows;
            const int i = (row_first + (there ? r : 0)) / int(a.group);
            const uint32_t qh = head * a.group + uint32_t((row_first + (there ? r : 0)) % int(a.group));
            const uint16_t* src = a.q.d + uint64_t(s.row0 + i) * a.q.token_stride + uint64_t(qh) * a.q.head_stride;
            see[r2] = visible(a, s, i);
            if (!there) see[r2].hi = 0;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // FP8: dims are dealt so that a lane's share of a key is 16 contiguous bytes
                const int d0 = S::kFp8 ? (k / 4) * 64 + t4 * 16 + (k % 4) * 4 : k * 16 + 2 * t4;
                const int d1 = S::kFp8 ? d0 + 2 : d0 + 8;
                q[k][r2] = there ? *reinterpret_cast<const uint32_t*>(src + d0) : 0u;
                q[k][r2 + 2] = there ? *reinterpret_cast<const uint32_t*>(src + d1) : 0u;
            }
        }

        float o[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        // Lane i (mod 16) looks up key i of a stage: its page one stage ahead of
        // its copies, which start kStages - 1 stages ahead of their use.
        const int32_t* table = a.b.table + uint64_t(b) * a.b.table_stride;
        const uint32_t key = lane & 15u;
        const auto page_of = [&](int i) -> int32_t {
            const int pos = base + i * kUnit + int(key);
            if (i >= n_units || pos < keys.lo || pos >= keys.hi) return -1;
            const int32_t pg = table[uint32_t(pos) >> a.c.page_shift];
            if (pg < 0 || uint64_t(pg) >= a.c.pool_pages) {
                bad = true;
                return -1;
            }
            return pg;
        };
        const auto start_stage = [&](int i, int32_t page) {
            const int pos = base + i * kUnit + int(key);
            const uint32_t slot = uint32_t(pos) & ((1u << a.c.page_shift) - 1u);
            const int64_t off = page < 0 ? -1
                                         : int64_t(uint64_t(uint32_t(page)) * a.c.page_stride +
                                                   uint64_t(slot) * a.c.token_stride + uint64_t(head) * a.c.head_stride);
            const uint32_t stage = uint32_t(i) % S::kStages;
            const uint32_t dst = ring_u32 + stage * S::kStageBytes;
            if (i < n_units) {
#pragma unroll
                for (int j = 0; j < S::kCopies; ++j) {
                    const uint32_t r = uint32_t(j) * S::kRowsACopy + lane / S::kChunks, c = lane % S::kChunks;
                    const int64_t at = __shfl_sync(~0u, off, int(r));
                    const int64_t from = (at < 0 ? 0 : at) + int64_t(c) * 16;
                    copy16(dst + S::place_k(r, c), a.c.k + from, at >= 0);
                    copy16(dst + S::kSideBytes + S::place_v(r, c), a.c.v + from, at >= 0);
                }
                if (S::kFp8 && lane < 16)
                    scale_ring[stage * kKeys + key] =
                        page < 0 ? -1
                                 : int64_t(((uint64_t(uint32_t(page)) * kv_heads + head) << a.c.page_shift) + slot);
            }
            copy_commit();
        };
        // lanes 0 .. 15: K's scale of key `lane`; 16 .. 31: V's
        const auto scale_of = [&](int i) -> float {
            if (!S::kFp8 || i >= n_units) return 0.f;
            const int64_t at = scale_ring[uint32_t(i) % S::kStages * kKeys + key];
            return at < 0 ? 0.f : scale_value((lane < 16 ? a.c.k_scale : a.c.v_scale)[at]);
        };
        int32_t page = page_of(0);
        for (int i = 0; i < S::kStages - 1; ++i) {
            const int32_t next = page_of(i + 1);
            start_stage(i, page);
            page = next;
        }
        __syncwarp();
        float scale_next = scale_of(0);

        for (int i = 0; i < n_units; ++i) {
            copy_wait<S::kStages - 2>();
            __syncwarp();
            {
                const int32_t next = page_of(i + S::kStages);
                start_stage(i + S::kStages - 1, page);
                page = next;
            }
            __syncwarp();
            const float scale_now = scale_next;
            scale_next = scale_of(i + 1);
            uint8_t* stage = ring + uint32_t(i) % S::kStages * S::kStageBytes;
            uint8_t* v_stage = stage + S::kSideBytes;
            const uint32_t k_at = smem_u32(stage), v_at = smem_u32(v_stage);
            const int pos0 = base + i * kUnit;

            // scores of 16 rows by 16 keys
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            if (!S::kFp8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t kr[4];
                    ldmatrix4(kr, k_at + S::place_k((lane & 7u) + (lane >> 4) * 8u, 2u * k + ((lane >> 3) & 1u)));
                    mma_16816(H, sc[0], q[k], kr[0], kr[1]);
                    mma_16816(H, sc[1], q[k], kr[2], kr[3]);
                }
            } else {
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 w4 = *reinterpret_cast<const uint4*>(
                            stage + S::place_k(uint32_t(nb * 8 + g), uint32_t(c * 4 + t4)));
                        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t b0 = H ? fp8x2_to_half2<S::kE5M2>(w[j]) : fp8x2_to_bf16x2<S::kE5M2>(w[j]);
                            const uint32_t b1 =
                                H ? fp8x2_to_half2<S::kE5M2>(w[j] >> 16) : fp8x2_to_bf16x2<S::kE5M2>(w[j] >> 16);
                            mma_16816(H, sc[nb], q[c * 4 + j], b0, b1);
                        }
                    }
                }
            }
            float ks[4], vs[4];  // scales of the lane's four keys
            if (S::kFp8) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int src = (x >> 1) * 8 + 2 * t4 + (x & 1);
                    ks[x] = __shfl_sync(~0u, scale_now, src);
                    vs[x] = __shfl_sync(~0u, scale_now, src + 16);
                }
            }
            // scale, mask, running maximum
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int pos = pos0 + nb * 8 + 2 * t4 + (e & 1);
                    const KeyRange& r = see[e >> 1];
                    float x = sc[nb][e] * a.scale_log2;
                    if (S::kFp8) x *= ks[nb * 2 + (e & 1)];
                    x = pos >= r.lo && pos < r.hi ? x : -INFINITY;
                    sc[nb][e] = x;
                    top[e >> 1] = fmaxf(top[e >> 1], x);
                }
            bool grew = false;
            float low[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
                top[r] = fmaxf(top[r], m[r]);
                grew |= top[r] > m[r];
            }
            if (__any_sync(~0u, grew)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float f = top[r] == m[r] ? 1.f : exp2_fast(m[r] - top[r]);
                    l[r] *= f;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[j][2 * r] *= f;
                        o[j][2 * r + 1] *= f;
                    }
                    m[r] = top[r];
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) low[r] = m[r] == -INFINITY ? 0.f : m[r] - S::kShift;
            uint32_t p[4];
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[nb][e] = exp2_fast(sc[nb][e] - low[e >> 1]);
                    l[e >> 1] += sc[nb][e];
                    if (S::kFp8) sc[nb][e] *= vs[nb * 2 + (e & 1)];
                }
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    p[nb * 2 + r] = S::kPvHalf ? pack_half2(sc[nb][2 * r], sc[nb][2 * r + 1])
                                               : pack_bf16x2(sc[nb][2 * r], sc[nb][2 * r + 1]);
            }

            // A weight of 0 hides a finite value, not an infinity or a NaN.  Where some
            // row does not see all the keys of this stage, such values of V are
            // taken out and given to the rows that do see them.
            const int k0 = max(pos0, keys.lo), k1 = min(pos0 + kKeys, keys.hi);
            const bool partial = k0 < k1 && ((g < rows && (see[0].lo > k0 || see[0].hi < k1)) ||
                                             (g + 8 < rows && (see[1].lo > k0 || see[1].hi < k1)));
            if (__any_sync(~0u, partial)) {
                bool special = false;
#pragma unroll
                for (int j = 0; j < S::kCopies; ++j)
                    special |= special16<FMT, H>(
                        *reinterpret_cast<const uint4*>(v_stage + (uint32_t(j) * 32u + lane) * 16u));
                if (__any_sync(~0u, special)) {
                    for (int x = 0; x < kKeys; ++x) {
                        const int pos = pos0 + x;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t byte = uint32_t(S::out_dim(j, t4, e)) * (S::kFp8 ? 1u : 2u);
                                const uint8_t* at = v_stage + S::place_v(uint32_t(x), byte >> 4) + (byte & 15u);
                                float v;
                                if (S::kFp8)
                                    v = half2_to_float2(fp8x2_to_half2<S::kE5M2>(*at)).x;
                                else if (H)
                                    v = __half2float(*reinterpret_cast<const __half*>(at));
                                else
                                    v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at));
                                if (!(fabsf(v) < INFINITY)) {
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        if (pos >= see[r].lo && pos < see[r].hi) o[j][2 * r + e] += v;
                                }
                            }
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < S::kCopies; ++j) {
                        uint4* at = reinterpret_cast<uint4*>(v_stage + (uint32_t(j) * 32u + lane) * 16u);
                        uint32_t w[4] = {at->x, at->y, at->z, at->w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            if (!S::kFp8) {
                                constexpr uint32_t kInf = H ? 0x7C00u : 0x7F80u;
                                if ((w[y] & 0x7FFFu) >= kInf) w[y] &= 0xFFFF0000u;
                                if (((w[y] >> 16) & 0x7FFFu) >= kInf) w[y] &= 0x0000FFFFu;
                            } else {
                                for (int z = 0; z < 32; z += 8)
                                    if (((w[y] >> z) & 0x7Fu) >= (S::kE5M2 ? 0x7Cu : 0x7Fu)) w[y] &= ~(0xFFu << z);
                            }
                        }
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
                }
            }

            // weights times values
            if (!S::kFp8) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t vr[4];
                    ldmatrix4_trans(vr, v_at + S::place_v((lane & 7u) + ((lane >> 3) & 1u) * 8u, 2u * j + (lane >> 4)));
                    mma_16816(S::kPvHalf, o[2 * j], p, vr[0], vr[1]);
                    mma_16816(S::kPvHalf, o[2 * j + 1], p, vr[2], vr[3]);
                }
            } else {
                // the lane's D / 8 bytes of each of its four keys
                constexpr int W = D / 32;  // words
                uint32_t w[4][W];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t r = uint32_t((x >> 1) * 8 + 2 * t4 + (x & 1));
                    if (W == 4) {
                        const uint4 y = *reinterpret_cast<const uint4*>(v_stage + S::place_v(r, uint32_t(g)));
                        w[x][0] = y.x, w[x][1] = y.y, w[x][W - 2] = y.z, w[x][W - 1] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(v_stage + S::place_v(r, uint32_t(g) >> 1) +
                                                                        (uint32_t(g) & 1u) * 8u);
                        w[x][0] = y.x, w[x][1] = y.y;
                    }
                }
#pragma unroll
                for (int y = 0; y < W; ++y)
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        // bytes 2 h2 and 2 h2 + 1 of keys (0, 1) and of keys (2, 3), key pairs together
                        const uint32_t sel = h2 ? 0x7362u : 0x5140u;
                        const uint32_t ab = __byte_perm(w[0][y], w[1][y], sel);
                        const uint32_t cd = __byte_perm(w[2][y], w[3][y], sel);
                        mma_16816(S::kPvHalf, o[4 * y + 2 * h2], p, fp8x2_to_bf16x2<S::kE5M2>(ab),
                                  fp8x2_to_bf16x2<S::kE5M2>(cd));
                        mma_16816(S::kPvHalf, o[4 * y + 2 * h2 + 1], p, fp8x2_to_bf16x2<S::kE5M2>(ab >> 16),
                                  fp8x2_to_bf16x2<S::kE5M2>(cd >> 16));
                    }
            }
        }
        copy_wait<0>();

        // Join the four warps.  The sums l are still one quad lane's; m is the row's.
        __syncthreads();
        float* m_o = reinterpret_cast<float*>(smem);               // [warp][row][D]
        float* m_ml = m_o + kWarps * kStepRows * D;                // [warp][row][m, l]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(~0u, l[r], 1);
            l[r] += __shfl_xor_sync(~0u, l[r], 2);
            const int row = int(warp) * kStepRows + g + 8 * r;
            if (t4 == 0) {
                m_ml[2 * row] = m[r];
                m_ml[2 * row + 1] = l[r];
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) m_o[row * D + S::out_dim(j, t4, e)] = o[j][2 * r + e];
        }
        __syncthreads();
        // eight threads a row, D / 8 columns each
        constexpr int W = D / 8;
        const int row = int(tid >> 3), col = int(tid & 7u) * W;
        float mm = -INFINITY, ll = 0.f, acc[W];
#pragma unroll
        for (int x = 0; x < W; ++x) acc[x] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, m_ml[2 * (w * kStepRows + row)]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = m_ml[2 * (w * kStepRows + row)];
            const float f = mw == mm ? 1.f : exp2_fast(mw - mm);
            ll += f * m_ml[2 * (w * kStepRows + row) + 1];
#pragma unroll
            for (int x = 0; x < W; ++x) acc[x] += f * m_o[(w * kStepRows + row) * D + col + x];
        }
        bool write = true;
        if (u > item_start || stop < item_end) {
            // a part of the item
            const uint32_t first = share_of(units, ctas, item_start), last = share_of(units, ctas, item_end - 1);
            const auto slot = [&](uint32_t c) {
                return a.parts + (uint64_t(c) * 2 + (c == first ? 1 : 0)) * S::kPartFloats;
            };
            float* mine = slot(blockIdx.x);
            wait_predecessor();  // the counters are clear
            if (row < rows) {
                if (col == 0) {
                    mine[2 * row] = mm;
                    mine[2 * row + 1] = ll;
                }
#pragma unroll
                for (int x = 0; x < W; x += 4)
                    *reinterpret_cast<float4*>(mine + 2 * kStepRows + row * D + col + x) =
                        make_float4(acc[x], acc[x + 1], acc[x + 2], acc[x + 3]);
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(a.counters + first, 1u) == last - first;
            __syncthreads();
            write = s_last != 0;
            if (write && row < rows) {
                __threadfence();
                mm = -INFINITY;
                for (uint32_t c = first; c <= last; ++c) mm = fmaxf(mm, __ldcg(slot(c) + 2 * row));
                ll = 0.f;
#pragma unroll
                for (int x = 0; x < W; ++x) acc[x] = 0.f;
#pragma unroll 2
                for (uint32_t c = first; c <= last; ++c) {
                    const float* part = slot(c);
                    const float mw = __ldcg(part + 2 * row);
                    const float f = mw == mm ? 1.f : exp2_fast(mw - mm);
                    ll += f * __ldcg(part + 2 * row + 1);
#pragma unroll
                    for (int x = 0; x < W; x += 4) {
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(part + 2 * kStepRows + row * D + col + x));
                        acc[x] += f * y.x;
                        acc[x + 1] += f * y.y;
                        acc[x + 2] += f * y.z;
                        acc[x + 3] += f * y.w;
                    }
                }
            }
        }
        if (write && row < rows) {
            const int i = (row_first + row) / int(a.group);
            const uint32_t qh = head * a.group + uint32_t((row_first + row) % int(a.group));
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            uint16_t* dst = a.out.d + uint64_t(s.row0 + i) * a.out.token_stride + uint64_t(qh) * a.out.head_stride + col;
#pragma unroll
            for (int x = 0; x < W; x += 8) {
                uint32_t w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    w[y] = H ? pack_half2(acc[x + 2 * y] * inv, acc[x + 2 * y + 1] * inv)
                             : pack_bf16x2(acc[x + 2 * y] * inv, acc[x + 2 * y + 1] * inv);
                *reinterpret_cast<uint4*>(dst + x) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (a.lse && col == 0)
                a.lse[uint64_t(s.row0 + i) * a.q_heads + qh] =
                    ll == 0.f ? -INFINITY : (mm - S::kShift + log2f(ll)) * 0.693147180559945309f;
        }
        __syncthreads();  // the ring is free again
        u = stop;
    }
    wait_predecessor();  // the status word is clear
    if (bad) report(a.status, SPLITZIP_ERR_INVALID_ARG);
}

template <int FMT, bool H, int D>
int launch(const AttentionArgs& a, uint32_t ctas, cudaStream_t s) {
    using S = Step<FMT, H, D>;
    // every device once: the kernel's shared memory limit
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SPLITZIP_ERR_CUDA;
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        if (cudaFuncSetAttribute(kv_step_kernel<FMT, H, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
            cudaSuccess) {
            cudaGetLastError();
            return SPLITZIP_ERR_CUDA;
        }
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    ChainedLaunch l(dim3(ctas), dim3(kWarps * 32), S::kSmem, s);
    if (cudaLaunchKernelEx(&l.cfg, kv_step_kernel<FMT, H, D>, a) != cudaSuccess) {
        cudaGetLastError();
        return SPLITZIP_ERR_CUDA;
    }
    return SPLITZIP_OK;
}

template <int FMT, bool H>
int launch_dim(const AttentionArgs& a, uint32_t ctas, cudaStream_t s) {
    return a.c.head_dim == 128 ? launch<FMT, H, 128>(a, ctas, s) : launch<FMT, H, 64>(a, ctas, s);
}

}  // namespace

uint64_t step_part_floats(uint32_t head_dim) { return uint64_t(kStepRows) * (head_dim + 2); }

uint32_t step_ctas(uint64_t items_max, uint64_t keys_max) {
    const uint64_t units = items_max * ((keys_max + kUnit - 1) / kUnit + 1);
    return uint32_t(std::min<uint64_t>(kStepCtas, std::max<uint64_t>(1, (units + kMinUnits - 1) / kMinUnits)));
}

int launch_kv_step(const AttentionArgs& a, bool q_half, uint32_t ctas, cudaStream_t s) {
    switch (a.c.type) {
        case SPLITZIP_KV_FP8_E5M2: return q_half ? launch_dim<1, true>(a, ctas, s) : launch_dim<1, false>(a, ctas, s);
        case SPLITZIP_KV_FP8_E4M3: return q_half ? launch_dim<2, true>(a, ctas, s) : launch_dim<2, false>(a, ctas, s);
        default: return q_half ? launch_dim<0, true>(a, ctas, s) : launch_dim<0, false>(a, ctas, s);
    }
}

}  // namespace splitzip
