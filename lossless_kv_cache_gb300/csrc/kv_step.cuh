// Attention of few rows a sequence over a paged cache: decoding steps, one
// new token or a handful of drafted ones.
//
// Mathematics: one pass over the keys with a running maximum and sum (online
// softmax).  For each row m' = max(m, s), l' = l 2^(m-m') + sum 2^(s-m'),
// o' = o 2^(m-m') + sum 2^(s-m') v, in base 2 with the factor log2(e) in the
// score's scale; out = o / l.  Parts over different keys join by the same rule.
// FP8 values are exact in FP16 and are multiplied there without their scales:
// K's go to the scores, V's, 2^e, to the weights, and m is the maximum of s + e,
// so that the weights 2^(s+e-m) are at most 1 whatever the scales' range
// (l sums 2^(s-m), and the difference cancels in o / l).  That takes e for the
// size of the row, which it is as splitzip_kv_write stores it but for a row of
// zeros: those are looked for where they would raise m.  BF16 queries get a
// power of two for each row that brings them into FP16's range.
//
// What bounds it: HBM.  A tile of 16 rows does 64 operations a byte of a BF16
// cache, far below the ridge, so the layout is chosen for bytes in flight and
// few instructions a byte: a CTA is four warps, each with its own ring of
// stages of 16 keys (K and V) in shared memory filled by its own 16-byte
// cp.async copies, and no barrier between warps until an item ends.  The query
// heads that share a kv head are rows of one tile, so the cache is read once
// for all of them.  The products are S^T = K Q^T and O^T = V^T P^T, keys and
// dims along the 16 of an m16n8k16 and rows along its 8: a tile of 8 rows, the
// common one, wastes nothing, and P^T gets its place by transposing 8x8 blocks
// (movmatrix).  (With rows along the 16, a step of 8 rows took half as many
// products again, 48 more registers, and three CTAs an SM instead of four.)
//
// Roundings: weights to FP16, or to BF16 for a BF16 cache, whose V may be beyond
// FP16's range; BF16 queries over FP8 lose at most 2^-39 of a row's largest
// element; sums, maxima and parts are in 32 bits.
//
// One GB300, 32 query heads of 128 over 8, in a graph: 64 sequences of 8,192 E5M2
// tokens in 208 us (5.2 TB/s, 77 % of the measured copy rate; 186 to 211 on five of
// these GPUs), 512 of 1,024 in 218 us, one of 65,536 BF16 tokens in 49 us (5.4 TB/s,
// 80 %), four of 500 in 8.4 us, most of which is two launches, the scan and the
// first loads' latency.  Heads of 64, the first of these: 184 us (3.0 TB/s, 44 %).
#pragma once

#include <algorithm>
#include <atomic>

#include "kv_attention.cuh"
#include "tma_pipeline.cuh"

namespace splitzip {
namespace {

constexpr int kUnit = 64;      // keys of a unit: 16 for each of the four warps
constexpr int kWarps = 4;
constexpr int kKeys = 16;      // keys of a stage
constexpr int kMinUnits = 2;   // least share of a CTA (1,024 tokens: 8.2 us with 2, 9.4 with 4, 11.8 with 8)
constexpr uint32_t kStepCtas = 608;  // four on each of 152 SMs, at most

template <bool HALF>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (HALF)
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

// The transpose of an 8x8 matrix of 16-bit elements, two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// 16 bytes to shared memory, asynchronously; zeros where !there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// FMT 0: cache of the queries' 16-bit type (FP16 with H, else BF16), 1: E5M2,
// 2: E4M3 (queries of either type).  ROWS: rows of a tile, 8 or 16.
template <int FMT, bool H, int D, int ROWS>
struct Step {
    static constexpr bool kFp8 = FMT != 0;
    static constexpr bool kE5M2 = FMT == 1;
    static constexpr int kBlocks = ROWS / 8;           // of 8 rows
    static constexpr int kRowsLane = 2 * kBlocks;      // rows of a lane: 2 t, 2 t + 1 of each block
    static constexpr bool kHalf = kFp8 || H;           // products in FP16, else BF16
    // FP16 weights are 2^14 times the exponentials (at most 1), so that those
    // down to 2^-28 keep all bits; the factor cancels in o / l.
    static constexpr float kShift = kHalf ? 14.f : 0.f;
    static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
    static constexpr int kChunks = kRowBytes / 16;     // 16-byte pieces of a row
    static constexpr int kRowsACopy = 32 / kChunks;    // rows a warp copies with one instruction
    static constexpr int kCopies = kKeys / kRowsACopy;
    static constexpr int kSideBytes = kKeys * kRowBytes;
    static constexpr int kStageBytes = 2 * kSideBytes;
    // Bytes in flight: four CTAs an SM of 12 KB rings a warp, three of 16 KB where
    // four have not the registers, or (stages of 8 KB) two of 24 KB.
    static constexpr int kCtasPerSm = kStageBytes > 4096 ? 2 : ROWS == 16 && D == 128 ? 3 : 4;
    static constexpr int kStages = 49152 / kCtasPerSm / kStageBytes;
    static constexpr int kRing = kStages * kStageBytes;  // a warp's
    static constexpr int kScaleBytes = kFp8 ? kStages * 2 * kKeys : 0;  // of K and V for a stage's keys
    static constexpr int kMergeBytes = kWarps * ROWS * (D + 2) * 4;
    static constexpr int kRingBytes = kWarps * kRing > kMergeBytes ? kWarps * kRing : kMergeBytes;
    static constexpr int kJoinBytes = kWarps * int(kStepCtas) * 8;  // factor and sum of each part of a warp's row
    static constexpr int kSmem = kRingBytes + kWarps * kScaleBytes;
    static_assert(kRingBytes >= kJoinBytes, "join");

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
    // Column of the output that lane group g's accumulators c0, c1 (up 0) or c2,
    // c3 (up 1) of block j are of.
    static __device__ __forceinline__ int out_dim(int j, int g, int up) {
        return kFp8 ? (D / 8) * g + 2 * j + up : 16 * j + 8 * up + g;
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

template <int FMT, bool H, int D, int ROWS, bool TREE>
__global__ void __launch_bounds__(kWarps * 32, Step<FMT, H, D, ROWS>::kCtasPerSm)
    kv_step_kernel(const __grid_constant__ AttentionArgs a) {
    using S = Step<FMT, H, D, ROWS>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_scan[kWarps + 1];
    __shared__ uint32_t s_last;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const int g = int(lane >> 2), t4 = int(lane & 3u);
    uint8_t* ring = smem + warp * S::kRing;
    const uint32_t ring_u32 = smem_u32(ring);
    uint8_t* scale_ring = smem + S::kRingBytes + warp * S::kScaleBytes;
    const uint32_t kv_heads = a.c.kv_heads;
    // whether a stage's 16 keys are one page's (their rows a stride apart, their scales 16 bytes in a row)
    const bool one_page = a.c.page_shift >= 4 && (!S::kFp8 || ((reinterpret_cast<uintptr_t>(a.c.k_scale) |
                                                               reinterpret_cast<uintptr_t>(a.c.v_scale)) & 15u) == 0);
    bool bad = false;

    // A sequence's units: those of all its rows' keys, for each kv head and row tile.
    const auto tiles_of = [&](const KvSeq& s) { return (s.t * int(a.group) + ROWS - 1) / ROWS; };
    const auto weight_of = [&](uint32_t b) -> uint64_t {
        const KvSeq s = load_seq(a.b, b);
        bad |= !s.ok;
        if (s.t == 0) return 0;
        return uint64_t(unit_count(visible<TREE>(a, s, 0, s.t - 1), kUnit)) * kv_heads * uint32_t(tiles_of(s));
    };
    // As many CTAs as have kMinUnits each, but one for each item at least.  The
    // count of items, as far as it matters, rides above the units'.
    constexpr int kItemsAt = 38;
    const auto items_of = [&](uint32_t b) -> uint64_t {
        const KvSeq s = load_seq(a.b, b);
        return uint64_t(min(uint32_t(kStepCtas), uint32_t(tiles_of(s)) * kv_heads)) << kItemsAt;
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
    constexpr uint64_t kUnitsMask = (uint64_t(1) << kItemsAt) - 1;
    uint64_t units = 0, mine = 0, upto_mine = 0;  // mine: of the last round, the only one of up to 128 sequences
    for (uint32_t b0 = 0; b0 < a.b.batch; b0 += kWarps * 32) {
        mine = b0 + tid < a.b.batch ? weight_of(b0 + tid) : 0;
        upto_mine = scan(mine + (mine > 0 ? items_of(b0 + tid) : 0)) & kUnitsMask;
        __syncthreads();
        units += s_scan[kWarps];
    }
    const uint64_t items = units >> kItemsAt;
    units &= kUnitsMask;
    const uint64_t most = max(items, (units + kMinUnits - 1) / kMinUnits);
    uint32_t ctas = most < gridDim.x ? uint32_t(most) : gridDim.x;
    // Short shares that go past an item's end start, drain and join twice: as many for each
    // item then (2 trees of 8 tokens over 600: 64 items, 21 us with 304 CTAs, 14 with 256).
    if (TREE && most > ctas && items <= ctas && units <= uint64_t(ctas) * 8) ctas = ctas / uint32_t(items) * uint32_t(items);
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
            uint64_t w = mine, upto = upto_mine;
            if (a.b.batch > kWarps * 32) {
                w = b0 + tid < a.b.batch ? weight_of(b0 + tid) : 0;
                upto = base + scan(w);
            }
            if (w > 0 && u >= upto - w && u < upto) {
                s_b = b0 + tid;
                s_start = upto - w;
            }
            __syncthreads();
            if (a.b.batch > kWarps * 32) base += s_scan[kWarps];
            if (base > u) break;
        }
        b = s_b;
        b_start = s_start;
    }

    while (u < end) {
        // the item that holds unit u
        const KvSeq s = load_seq(a.b, b);
        const KeyRange all = visible<TREE>(a, s, 0, s.t > 0 ? s.t - 1 : 0);
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
        const int row_first = int(item / kv_heads) * ROWS;
        const int rows = min(ROWS, s.t * int(a.group) - row_first);
        const uint64_t stop = item_end < end ? item_end : end;
        const int n_units = int(stop - u);
        const int i0 = row_first / int(a.group), i1 = (row_first + rows - 1) / int(a.group);
        const KeyRange keys = visible<TREE>(a, s, i0, i1);
        const int base = (all.lo / kUnit + int(u - item_start)) * kUnit + int(warp) * kKeys;

        // Copies start kStages - 1 stages ahead of their use, and the page of a
        // stage's keys is looked up a stage before that: by lane i (mod 16) for key
        // i, or where a stage is one page's, by all lanes alike.
        const int32_t* table = a.b.table + uint64_t(b) * a.b.table_stride;
        const uint32_t key = lane & 15u, slots = (1u << a.c.page_shift) - 1u;
        const uint32_t copy_row = lane / S::kChunks, copy_col = lane % S::kChunks;
        const uint64_t copy_off = uint64_t(copy_row) * a.c.token_stride + copy_col * 16u;
        const uint64_t copy_step = uint64_t(S::kRowsACopy) * a.c.token_stride;
        const uint64_t head_off = uint64_t(head) * a.c.head_stride;
        const auto page_of = [&](int i) -> int32_t {
            const int pos = base + i * kUnit + (one_page ? 0 : int(key));
            if (i >= n_units || pos + (one_page ? kKeys : 1) <= keys.lo || pos >= keys.hi) return -1;
            const int32_t pg = __ldg(table + (uint32_t(pos) >> a.c.page_shift));
            if (pg < 0 || uint64_t(pg) >= a.c.pool_pages) {
                bad = true;
                return -1;
            }
            return pg;
        };
        // small pages: a key's scales, loaded with its copies and put into the ring a stage later
        uint32_t late_scale = 0, late_stage = 0;
        bool late = false;
        const auto start_stage = [&](int i, int32_t page) {
            const int pos0 = base + i * kUnit;
            const uint32_t stage = uint32_t(i) % S::kStages;
            const uint32_t dst = ring_u32 + stage * S::kStageBytes;
            if (i < n_units) {
                if (one_page) {
                    const uint64_t at = page < 0 ? 0
                                                 : uint64_t(uint32_t(page)) * a.c.page_stride +
                                                       uint64_t(uint32_t(pos0) & slots) * a.c.token_stride + head_off +
                                                       copy_off;
                    const uint8_t *k_from = a.c.k + at, *v_from = a.c.v + at;
                    if (page >= 0 && pos0 >= keys.lo && pos0 + kKeys <= keys.hi) {
#pragma unroll
                        for (int j = 0; j < S::kCopies; ++j) {
                            const uint32_t r = uint32_t(j) * S::kRowsACopy + copy_row;
                            copy16(dst + S::place_k(r, copy_col), k_from + uint64_t(j) * copy_step);
                            copy16(dst + S::kSideBytes + S::place_v(r, copy_col), v_from + uint64_t(j) * copy_step);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < S::kCopies; ++j) {
                            const uint32_t r = uint32_t(j) * S::kRowsACopy + copy_row;
                            const int pos = pos0 + int(r);
                            const bool there = page >= 0 && pos >= keys.lo && pos < keys.hi;
                            const uint64_t step = there ? uint64_t(j) * copy_step : 0;
                            copy16(dst + S::place_k(r, copy_col), k_from + step, there);
                            copy16(dst + S::kSideBytes + S::place_v(r, copy_col), v_from + step, there);
                        }
                    }
                    if (S::kFp8 && lane < 2) {
                        const uint64_t sc = page < 0 ? 0
                                                     : ((uint64_t(uint32_t(page)) * kv_heads + head) << a.c.page_shift) +
                                                           (uint32_t(pos0) & slots);
                        copy16(smem_u32(scale_ring) + (stage * 2 + lane) * kKeys, (lane ? a.c.v_scale : a.c.k_scale) + sc,
                               page >= 0);
                    }
                } else {
                    const uint32_t slot = uint32_t(pos0 + int(key)) & slots;
                    const int64_t off = page < 0 ? -1
                                                 : int64_t(uint64_t(uint32_t(page)) * a.c.page_stride +
                                                           uint64_t(slot) * a.c.token_stride + head_off);
#pragma unroll
                    for (int j = 0; j < S::kCopies; ++j) {
                        const uint32_t r = uint32_t(j) * S::kRowsACopy + copy_row;
                        const int64_t at = __shfl_sync(~0u, off, int(r));
                        const int64_t from = (at < 0 ? 0 : at) + int64_t(copy_col) * 16;
                        copy16(dst + S::place_k(r, copy_col), a.c.k + from, at >= 0);
                        copy16(dst + S::kSideBytes + S::place_v(r, copy_col), a.c.v + from, at >= 0);
                    }
                }
            }
            if (S::kFp8 && !one_page) {
                if (late) scale_ring[late_stage * 2 * kKeys + lane] = uint8_t(late_scale);
                late = i < n_units;
                late_stage = stage;
                late_scale = 0;
                if (page >= 0)
                    late_scale = (lane < 16 ? a.c.k_scale : a.c.v_scale)[((uint64_t(uint32_t(page)) * kv_heads + head)
                                                                          << a.c.page_shift) +
                                                                         (uint32_t(pos0 + int(key)) & slots)];
            }
            copy_commit();
        };
        int32_t page = page_of(0), page_next = page_of(1);
        for (int i = 0; i < S::kStages - 1; ++i) {
            start_stage(i, page);
            page = page_next;
            page_next = page_of(i + 2);
        }

        // queries, as the second operand: row g of each block
        uint32_t q[S::kBlocks][D / 16][2];
        float row_scale[S::kRowsLane];
#pragma unroll
        for (int nb = 0; nb < S::kBlocks; ++nb) {
            const int r = g + 8 * nb;
            const bool there = r < rows;
            const int i = (row_first + (there ? r : 0)) / int(a.group);
            const uint32_t qh = head * a.group + uint32_t((row_first + (there ? r : 0)) % int(a.group));
            const uint16_t* src = a.q.d + uint64_t(s.row0 + i) * a.q.token_stride + uint64_t(qh) * a.q.head_stride;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // FP8: dims are dealt so that a lane's share of a key is 16 contiguous bytes
                const int d0 = S::kFp8 ? (k / 4) * 64 + t4 * 16 + (k % 4) * 4 : k * 16 + 2 * t4;
                const int d1 = S::kFp8 ? d0 + 2 : d0 + 8;
                q[nb][k][0] = there ? *reinterpret_cast<const uint32_t*>(src + d0) : 0u;
                q[nb][k][1] = there ? *reinterpret_cast<const uint32_t*>(src + d1) : 0u;
            }
            float scale = a.scale_log2;
            if (S::kFp8 && !a.q_half) {
                // BF16 to FP16 by way of the power of two that brings the row's largest
                // finite element to [2^14, 2^15): what FP16 loses of the small ones is
                // below 2^-39 of it
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t lo = q[nb][k][y] & 0x7FFFu, hi = (q[nb][k][y] >> 16) & 0x7FFFu;
                        top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                    }
                top = max(top, __shfl_xor_sync(~0u, top, 1));
                top = max(top, __shfl_xor_sync(~0u, top, 2));
                // 2^up takes exponent e to 14, within what one normal factor can do
                const int e = int(top >> 7) - 127, up = min(126, 14 - e);
                const float f = __uint_as_float(uint32_t(127 + up) << 23);
                scale *= __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 v = bf16x2_to_float2(q[nb][k][y]);
                        q[nb][k][y] = pack_half2(v.x * f, v.y * f);
                    }
            }
            // the scores' rows are the lane's 2 t and 2 t + 1
            row_scale[2 * nb] = __shfl_sync(~0u, scale, 8 * t4);
            row_scale[2 * nb + 1] = __shfl_sync(~0u, scale, 8 * t4 + 4);
        }
        // what the lane's rows see: a range, and for a tree bits of its new tokens besides
        KeyRange see[S::kRowsLane];
        int mask_row[TREE ? S::kRowsLane : 1];  // -1: none
#pragma unroll
        for (int r = 0; r < S::kRowsLane; ++r) {
            const int row = 8 * (r >> 1) + 2 * t4 + (r & 1);
            const int i = (row_first + (row < rows ? row : 0)) / int(a.group);
            see[r] = TREE ? visible_before(a, s, i) : visible<false>(a, s, i);
            if (TREE) mask_row[TREE ? r : 0] = row < rows && s.n - s.t + i >= 0 ? s.row0 + i : -1;
            if (row >= rows) see[r].hi = 0;
        }
        // positions that every row of the tile sees
        const KeyRange each = TREE ? visible_to_all_before(a, s, i1)
                                   : KeyRange{visible<false>(a, s, i1).lo, visible<false>(a, s, i0).hi};
        uint32_t tree_sees[TREE ? S::kRowsLane : 1] = {};  // of a stage's keys
        const auto sees = [&](int r, int pos0, int key) -> bool {
            const int pos = pos0 + key;
            return (pos >= see[r].lo && pos < see[r].hi) || (TREE && (tree_sees[TREE ? r : 0] >> key & 1u));
        };

        float o[D / 16][S::kBlocks][4];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int nb = 0; nb < S::kBlocks; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][nb][e] = 0.f;
        float m[S::kRowsLane], l[S::kRowsLane];
#pragma unroll
        for (int r = 0; r < S::kRowsLane; ++r) m[r] = -INFINITY, l[r] = 0.f;

        for (int i = 0; i < n_units; ++i) {
            copy_wait<S::kStages - 2>();
            __syncwarp();
            start_stage(i + S::kStages - 1, page);
            page = page_next;
            page_next = page_of(i + S::kStages + 1);
            uint8_t* stage = ring + uint32_t(i) % S::kStages * S::kStageBytes;
            uint8_t* v_stage = stage + S::kSideBytes;
            const uint32_t k_at = smem_u32(stage), v_at = smem_u32(v_stage);
            const int pos0 = base + i * kUnit;

            // scores: keys g (c0, c1) and g + 8 (c2, c3) by rows 2 t and 2 t + 1 of each block
            float sc[S::kBlocks][4];
#pragma unroll
            for (int nb = 0; nb < S::kBlocks; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nb][e] = 0.f;
            if (!S::kFp8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t kr[4];
                    ldmatrix4(kr, k_at + S::place_k((lane & 7u) + ((lane >> 3) & 1u) * 8u, 2u * k + (lane >> 4)));
#pragma unroll
                    for (int nb = 0; nb < S::kBlocks; ++nb) mma_16816<S::kHalf>(sc[nb], kr, q[nb][k][0], q[nb][k][1]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint4 w0 = *reinterpret_cast<const uint4*>(stage + S::place_k(uint32_t(g), uint32_t(c * 4 + t4)));
                    const uint4 w8 =
                        *reinterpret_cast<const uint4*>(stage + S::place_k(uint32_t(g + 8), uint32_t(c * 4 + t4)));
                    const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, up[4] = {w8.x, w8.y, w8.z, w8.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t kr[4] = {fp8_pair_to_half2<S::kE5M2>(lo[j], 0), fp8_pair_to_half2<S::kE5M2>(up[j], 0),
                                                fp8_pair_to_half2<S::kE5M2>(lo[j], 1), fp8_pair_to_half2<S::kE5M2>(up[j], 1)};
#pragma unroll
                        for (int nb = 0; nb < S::kBlocks; ++nb)
                            mma_16816<S::kHalf>(sc[nb], kr, q[nb][c * 4 + j][0], q[nb][c * 4 + j][1]);
                    }
                }
            }
            // scales of the lane's two keys; V's also as exponents
            float ks[2], vs[2], ve[2];
            if (S::kFp8) {
                const uint8_t* at = scale_ring + uint32_t(i) % S::kStages * 2 * kKeys + g;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t kb = at[8 * x], vb = at[kKeys + 8 * x];
                    ks[x] = scale_value(kb);
                    vs[x] = scale_value(vb);
                    // at least -80, which bounds the sums of 2^(s-m)
                    ve[x] = __uint_as_float(0x4B000000u | max(vb, 47u)) - 8388735.f;
                }
            }
            // scale, mask, running maximum
            const bool masked = pos0 < each.lo || pos0 + kKeys > each.hi;
            if (TREE && masked) {
                const int left = s.n - pos0;
#pragma unroll
                for (int r = 0; r < S::kRowsLane; ++r) {
                    uint32_t& bits = tree_sees[TREE ? r : 0];
                    bits = 0;
                    if (left > 0 && mask_row[TREE ? r : 0] >= 0)
                        bits = mask_bits(a.mask + uint64_t(uint32_t(mask_row[TREE ? r : 0])) * a.words, a.words,
                                         pos0 - (s.n - s.t)) &
                               (left >= kKeys ? 0xFFFFu : (1u << left) - 1u);
                }
            }
            if (S::kFp8 && masked) {
                // a slot that nothing was written to may hold 255, and 0 times infinity is NaN
                vs[0] = fminf(vs[0], 1.7014118e38f);
                vs[1] = fminf(vs[1], 1.7014118e38f);
            }
#pragma unroll
            for (int r = 0; r < S::kRowsLane; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y = sc[r >> 1][2 * x + (r & 1)] * row_scale[r];
                    if (S::kFp8) y *= ks[x];
                    if (masked) y = sees(r, pos0, g + 8 * x) ? y : -INFINITY;
                    sc[r >> 1][2 * x + (r & 1)] = y;
                }
            float top[S::kRowsLane];
            // the rows' largest of the stage; whether some row's maximum grows
            const auto find_top = [&]() -> bool {
                bool grew = false;
#pragma unroll
                for (int r = 0; r < S::kRowsLane; ++r) {
                    top[r] = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float y = sc[r >> 1][2 * x + (r & 1)];
                        top[r] = fmaxf(top[r], S::kFp8 ? y + ve[x] : y);
                    }
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], d));
                    grew |= top[r] > m[r];
                }
                return __any_sync(~0u, grew);
            };
            bool grew = find_top();
            if (S::kFp8 && grew && __any_sync(~0u, vs[0] == 1.f || vs[1] == 1.f)) {
                // A row of zeros has the scale 2^0, which says nothing of its size: against a
                // maximum with that exponent the weights of rows of small scale, all of the
                // result, would lose bits or vanish.  It takes the least exponent instead, and
                // as its weight is then beyond FP16, the weight 0.
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t any = 0;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 w =
                            *reinterpret_cast<const uint4*>(v_stage + S::place_v(uint32_t(g + 8 * x), uint32_t(c * 4 + t4)));
                        any |= w.x | w.y | w.z | w.w;
                    }
                    any |= __shfl_xor_sync(~0u, any, 1);
                    any |= __shfl_xor_sync(~0u, any, 2);
                    if ((any & 0x7F7F7F7Fu) == 0) {
                        ve[x] = -80.f;
                        vs[x] = 0.f;
                    }
                }
                grew = find_top();
            }
            if (grew) {
                float f[S::kRowsLane];
#pragma unroll
                for (int r = 0; r < S::kRowsLane; ++r) {
                    const float now = fmaxf(top[r], m[r]);
                    f[r] = now == m[r] ? 1.f : exp2_fast(m[r] - now);
                    l[r] *= f[r];
                    m[r] = now;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int nb = 0; nb < S::kBlocks; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[j][nb][e] *= f[2 * nb + (e & 1)];
            }
            uint32_t p[S::kBlocks][2];
#pragma unroll
            for (int nb = 0; nb < S::kBlocks; ++nb) {
                float low[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) low[e] = m[2 * nb + e] == -INFINITY ? 0.f : m[2 * nb + e] - S::kShift;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float e0 = exp2_fast(sc[nb][2 * x] - low[0]), e1 = exp2_fast(sc[nb][2 * x + 1] - low[1]);
                    l[2 * nb] += e0;
                    l[2 * nb + 1] += e1;
                    if (S::kFp8) {
                        e0 *= vs[x];
                        e1 *= vs[x];
                    }
                    p[nb][x] = transpose8(S::kHalf ? pack_half2(e0, e1) : pack_bf16x2(e0, e1));
                }
            }

            // A weight of 0 hides a finite value, not an infinity or a NaN.  Where some
            // row does not see all the keys of this stage, such values of V are
            // taken out and given to the rows that do see them.
            const int k0 = max(pos0, keys.lo), k1 = min(pos0 + kKeys, keys.hi);
            if (masked && k0 < k1 && (each.lo > k0 || each.hi < k1)) {
                bool special = false;
#pragma unroll
                for (int j = 0; j < S::kCopies; ++j)
                    special |= special16<FMT, H>(
                        *reinterpret_cast<const uint4*>(v_stage + (uint32_t(j) * 32u + lane) * 16u));
                if (__any_sync(~0u, special)) {
#pragma unroll 1
                    for (int x = 0; x < kKeys; ++x) {
#pragma unroll
                        for (int j = 0; j < D / 16; ++j)
#pragma unroll
                            for (int up = 0; up < 2; ++up) {
                                const uint32_t byte = uint32_t(S::out_dim(j, g, up)) * (S::kFp8 ? 1u : 2u);
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
                                    for (int r = 0; r < S::kRowsLane; ++r)
                                        if (sees(r, pos0, x)) o[j][r >> 1][2 * up + (r & 1)] += v;
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

            // values times weights
            if (!S::kFp8) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t vr[4];
                    ldmatrix4_trans(vr, v_at + S::place_v((lane & 7u) + (lane >> 4) * 8u, 2u * j + ((lane >> 3) & 1u)));
#pragma unroll
                    for (int nb = 0; nb < S::kBlocks; ++nb) mma_16816<S::kHalf>(o[j][nb], vr, p[nb][0], p[nb][1]);
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
                for (int j = 0; j < D / 16; ++j) {
                    // bytes 2 j and 2 j + 1 of keys (0, 1) and of keys (2, 3), key pairs together
                    const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
                    const uint32_t ab = __byte_perm(w[0][j / 2], w[1][j / 2], sel);
                    const uint32_t cd = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
                    const uint32_t vr[4] = {fp8_pair_to_half2<S::kE5M2>(ab, 0), fp8_pair_to_half2<S::kE5M2>(ab, 1),
                                            fp8_pair_to_half2<S::kE5M2>(cd, 0), fp8_pair_to_half2<S::kE5M2>(cd, 1)};
#pragma unroll
                    for (int nb = 0; nb < S::kBlocks; ++nb) mma_16816<S::kHalf>(o[j][nb], vr, p[nb][0], p[nb][1]);
                }
            }
        }
        copy_wait<0>();

        // Join the four warps.  The sums l are still of the lane's keys; m is the row's.
        __syncthreads();
        float* m_o = reinterpret_cast<float*>(smem);      // [warp][row][D]
        float* m_ml = m_o + kWarps * ROWS * D;            // [warp][row][m, l]
#pragma unroll
        for (int r = 0; r < S::kRowsLane; ++r) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[r] += __shfl_xor_sync(~0u, l[r], d);
            const int row = int(warp) * ROWS + 8 * (r >> 1) + 2 * t4 + (r & 1);
            if (g == 0) {
                m_ml[2 * row] = m[r];
                m_ml[2 * row + 1] = l[r];
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int up = 0; up < 2; ++up) m_o[row * D + S::out_dim(j, g, up)] = o[j][r >> 1][2 * up + (r & 1)];
        }
        __syncthreads();
        const bool whole = u == item_start && stop == item_end;
        const uint32_t first = whole ? 0u : share_of(units, ctas, item_start);
        const uint32_t last = whole ? 0u : share_of(units, ctas, item_end - 1);
        const auto slot = [&](uint32_t c) {
            return a.parts + (uint64_t(c) * 2 + (c == first ? 1 : 0)) * uint32_t(ROWS * (D + 2));
        };
        // `n` (2 or 4) columns of a row's result from col
        const auto finish = [&](int row, int col, const float* acc, int n, float mm, float ll) {
            const int i = (row_first + row) / int(a.group);
            const uint32_t qh = head * a.group + uint32_t((row_first + row) % int(a.group));
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            uint16_t* dst = a.out.d + uint64_t(s.row0 + i) * a.out.token_stride + uint64_t(qh) * a.out.head_stride + col;
            const bool half = S::kFp8 ? a.q_half != 0 : H;
            for (int y = 0; y < n; y += 2)
                *reinterpret_cast<uint32_t*>(dst + y) =
                    half ? pack_half2(acc[y] * inv, acc[y + 1] * inv) : pack_bf16x2(acc[y] * inv, acc[y + 1] * inv);
            if (a.lse && col == 0)
                a.lse[uint64_t(s.row0 + i) * a.q_heads + qh] =
                    ll == 0.f ? -INFINITY : (mm - S::kShift + log2f(ll)) * 0.693147180559945309f;
        };
        // four columns a thread and turn, a row's on one after another
        if (!whole) wait_predecessor();  // the counters are clear
        for (int x = int(tid) * 4; x < rows * D; x += kWarps * 32 * 4) {
            const int row = x / D, col = x % D;
            float mm = -INFINITY, ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, m_ml[2 * (w * ROWS + row)]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = m_ml[2 * (w * ROWS + row)];
                const float f = mw == mm ? 1.f : exp2_fast(mw - mm);
                const float4 y = *reinterpret_cast<const float4*>(m_o + (w * ROWS + row) * D + col);
                ll += f * m_ml[2 * (w * ROWS + row) + 1];
                acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
            }
            if (whole) {
                const float four[4] = {acc.x, acc.y, acc.z, acc.w};
                finish(row, col, four, 4, mm, ll);
            } else {
                float* part = slot(blockIdx.x);
                if (col == 0) *reinterpret_cast<float2*>(part + 2 * row) = make_float2(mm, ll);
                *reinterpret_cast<float4*>(part + 2 * ROWS + x) = acc;
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(a.counters + first, 1u) == last - first;
            __syncthreads();
            if (s_last) {
                __threadfence();
                // a warp a row: the parts' factors, then its columns, D / 32 a lane
                const int parts = int(last - first) + 1;
                float* factor = reinterpret_cast<float*>(smem) + warp * 2 * kStepCtas;
                for (int row = int(warp); row < rows; row += kWarps) {
                    constexpr int W = D / 32, kAhead = 16;
                    const int col = int(lane) * W;
                    float acc[W], ahead[kAhead][W];
                    // the first columns are on their way while the factors are made
                    const auto load = [&](int c, float* to) {
                        const float* from = slot(first + uint32_t(c)) + 2 * ROWS + row * D + col;
                        if (W == 4) {
                            const float4 y = __ldcg(reinterpret_cast<const float4*>(from));
                            to[0] = y.x, to[1] = y.y, to[W - 2] = y.z, to[W - 1] = y.w;
                        } else {
                            const float2 y = __ldcg(reinterpret_cast<const float2*>(from));
                            to[0] = y.x, to[1] = y.y;
                        }
                    };
#pragma unroll
                    for (int c = 0; c < kAhead; ++c) load(min(c, parts - 1), ahead[c]);
                    float mm = -INFINITY, ll = 0.f;
                    for (int c = int(lane); c < parts; c += 32) {
                        const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot(first + uint32_t(c)) + 2 * row));
                        factor[c] = ml.x;
                        factor[kStepCtas + c] = ml.y;
                        mm = fmaxf(mm, ml.x);
                    }
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, d));
                    for (int c = int(lane); c < parts; c += 32) {
                        const float f = factor[c] == mm ? 1.f : exp2_fast(factor[c] - mm);
                        factor[c] = f;
                        ll += f * factor[kStepCtas + c];
                    }
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) ll += __shfl_xor_sync(~0u, ll, d);
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < W; ++y) acc[y] = 0.f;
                    for (int c0 = 0; c0 < parts; c0 += kAhead) {
#pragma unroll
                        for (int c = 0; c < kAhead; ++c)
                            if (c0 + c < parts) {
                                const float f = factor[c0 + c];
#pragma unroll
                                for (int y = 0; y < W; ++y) acc[y] += f * ahead[c][y];
                            }
                        if (c0 + kAhead < parts) {
#pragma unroll
                            for (int c = 0; c < kAhead; ++c) load(min(c0 + kAhead + c, parts - 1), ahead[c]);
                        }
                    }
                    finish(row, col, acc, W, mm, ll);
                    __syncwarp();
                }
            }
        }
        __syncthreads();  // the ring is free again
        u = stop;
    }
    wait_predecessor();  // the status word is clear
    if (bad) report(a.status, SPLITZIP_ERR_INVALID_ARG);
}

template <int FMT, bool H, int D, int ROWS, bool TREE>
int launch(const AttentionArgs& a, uint32_t ctas, cudaStream_t s) {
    using S = Step<FMT, H, D, ROWS>;
    // every device once: the kernel's shared memory limit
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SPLITZIP_ERR_CUDA;
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        if (cudaFuncSetAttribute(kv_step_kernel<FMT, H, D, ROWS, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return SPLITZIP_ERR_CUDA;
        }
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    // one wave: more CTAs would start when others end and have no even share
    ChainedLaunch l(dim3(std::min(ctas, uint32_t(S::kCtasPerSm) * 152u)), dim3(kWarps * 32), S::kSmem, s);
    if (cudaLaunchKernelEx(&l.cfg, kv_step_kernel<FMT, H, D, ROWS, TREE>, a) != cudaSuccess) {
        cudaGetLastError();
        return SPLITZIP_ERR_CUDA;
    }
    return SPLITZIP_OK;
}

template <int FMT, bool H, bool TREE>
int launch_shape(const AttentionArgs& a, uint32_t ctas, cudaStream_t s) {
    // Tiles of 8 rows where no sequence has more: half the products and registers.  64 sequences
    // of 8,192 E5M2 tokens and 4 rows take 204 us so and 253 with tiles of 16, four of 500 8.4 and 9.3.
    // So do trees over short contexts, whose parts' latency counts and whose keys the L2
    // holds for the next tile: 4 sequences of 500 with 16 rows 13 us so and 16 with tiles
    // of 16 rows, with 28 rows 15 and 17; 3 of 900 14 and 25, 15 and 18.
    const bool few = uint64_t(a.b.max_tokens) * a.group <= 8 || (TREE && short_tree(a.b));
    if (a.c.head_dim == 128) return few ? launch<FMT, H, 128, 8, TREE>(a, ctas, s) : launch<FMT, H, 128, 16, TREE>(a, ctas, s);
    return few ? launch<FMT, H, 64, 8, TREE>(a, ctas, s) : launch<FMT, H, 64, 16, TREE>(a, ctas, s);
}

template <bool TREE>
int launch_type(const AttentionArgs& a, uint32_t ctas, cudaStream_t s) {
    switch (a.c.type) {
        case SPLITZIP_KV_FP8_E5M2: return launch_shape<1, false, TREE>(a, ctas, s);
        case SPLITZIP_KV_FP8_E4M3: return launch_shape<2, false, TREE>(a, ctas, s);
        case SPLITZIP_KV_FP16: return launch_shape<0, true, TREE>(a, ctas, s);
        default: return launch_shape<0, false, TREE>(a, ctas, s);
    }
}

}  // namespace
}  // namespace splitzip
