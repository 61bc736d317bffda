// Attention of chunks of new tokens over a paged cache, on the fifth-generation
// tensor cores.
//
// Mathematics: as in kv_step.cuh, online softmax over units of 128 keys; the
// running maximum that the exponentials are taken against is allowed to lag
// the true one by a factor of 2^8, so that the sums o are rescaled only when
// it grows by more (the exact factor cancels in o / l).
//
// Three kernels: a plan (below) deals the work, this one does it, a last one
// joins the parts of items that several CTAs have a share of.
//
// Roundings: weights and V are in the queries' type for their product (see
// Chunk), everything else is in 32 bits.
//
// What bounds it: the tensor core, 4 * head_dim operations for each (row,
// key), with the exponentials next.  A CTA holds two tiles of 128 rows (new
// tokens by the query heads that share a kv head) and passes over the keys
// once for both.  Its warps:
//   softmax    0-3 and 4-7, one tile's each: a thread is a row; scores from
//              TMEM, exponentials back to TMEM as the first operand of the
//              product with V; rescaling and the final division are theirs too
//   loaders    K and V from their pages into swizzled shared memory.  16-bit
//              pages of eight tokens and more: warp 8, a box of a tensor map a
//              lane (twelve warps in all).  Otherwise 8-11, row by row with
//              cp.async (sixteen in all): smaller 16-bit pages in place, FP8 by
//              way of a staging buffer, converted by the thread that copied it
//   products   one warp (9 or 12) issues them, in the order
//              S0(j+1) | P1(j) V(j) | S1(j+1) | P0(j+1) V(j+1) | ...
//              so that each tile's softmax runs under the other's products
//   pieces     one thread of the next warp (10 or 13) walks the CTA's share and
//              describes its pieces
// TMEM: S0, S1 (128 columns each, the weights overwrite the scores), O0, O1.
// The tensor core executes a CTA's products in the order of issue, which is
// what lets S(j+1) overwrite the weights that P(j) V(j) reads.
//
// One GB300, 32 query heads of 128 over 8, in graphs: 2,048 new tokens over
// 32,768 of BF16 in 853 us (1.25 PFLOP/s, 65 % of the measured library product),
// a prompt of 8,192 tokens of FP16 in 445 us (1.24 PFLOP/s, 64 %), six chunks of
// up to 777 over up to 5,000 of E4M3 in 136 us (0.5 PFLOP/s); heads of 64, the
// first of these, 586 us (0.91 PFLOP/s, 47 %).  A unit of 256 rows by 128
// keys takes about 3,500 cycles of which the products are 2,048: a tile's next
// scores wait for its weights (its softmax takes 1,600 and its two hand-overs
// 650), and what K and V cost of the shared memory's bandwidth slows the
// products by 600.  FP8 takes about 6,000, bound by the conversion on the way
// into shared memory (its loaders share the issue slots with the softmax), and
// every row tile of a sequence converts all its keys again.  The kernels of
// sixteen warps have 128 registers a thread at launch and spill 204 bytes (FP16
// queries over FP8: 286 at 64 dims, 346 at 128); those of twelve spill none.
// Handing the weights over in halves, two threads a row, spinning waits and
// pipelined exponentials all measured the same or slower.
//
// Every wait is bounded.  A thread whose wait ran out stops waiting and
// working but walks its loops to the end, so that every barrier among threads
// is still reached, and SPLITZIP_ERR_TIMEOUT is reported.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "kv_attention.cuh"
#include "tma_pipeline.cuh"
#include "tcgen05.cuh"

namespace splitzip {
namespace {

constexpr int kUnit = 128;       // keys
constexpr int kTileRows = 128;   // rows of a softmax group
constexpr int kRows = 2 * kTileRows;
static_assert(kRows == kChunkRows, "rows of a part");
constexpr uint32_t kChunkCtas = 152;  // one on each SM
constexpr int kPlanThreads = 1024;
// What an item costs beside its keys (its rows of Q in and results out, the
// pipeline's start), in units: the plan counts that many before the item's own.
// The 8,192-token prompt took 596, 477, 449, 472 and 481 us with 4, 6, 8, 10 and
// 14; six ragged chunks over E4M3 164, 145, 136, 148 and 142.  Those two, of 128
// dims, are what it was chosen by.
constexpr int kItemCost = 8;

// How work is cut: rows of a tile, what an item costs beside its keys, and
// whether rows see a tree's masks.
struct CausalWork {
    static constexpr bool kTree = false;
    static constexpr int kTile = kRows, kCost = kItemCost;
};
struct TreeWork {
    static constexpr bool kTree = true;
    static constexpr int kTile = kRows, kCost = kItemCost;
};

// Tensor maps of K and V (unused by the kernels that copy rows themselves).
struct ChunkMaps {
    CUtensorMap k, v;
};

struct ChunkStart {
    uint32_t b, tile;
    uint64_t group_start;  // first unit of the (sequence, tile)'s kv heads
};

// The item that a CTA begins and others go on with: what the join of its parts
// has to know of it.  rows = 0: none.
struct alignas(16) ChunkSplit {
    int row0, row_first, rows;
    uint32_t head, last_cta;
};

struct ChunkPlan {
    uint64_t units;
    uint32_t ctas, pad;
    ChunkStart start[1];
};

template <class W>
__device__ __forceinline__ int tile_count(const AttentionArgs& a, const KvSeq& s) {
    return (s.t * int(a.group) + W::kTile - 1) / W::kTile;
}

struct Tile {
    int row_first, rows;
    KeyRange keys;
    int units;
};

template <class W>
__device__ __forceinline__ Tile tile_of(const AttentionArgs& a, const KvSeq& s, int tile) {
    Tile t;
    t.row_first = tile * W::kTile;
    t.rows = min(W::kTile, s.t * int(a.group) - t.row_first);
    t.keys = visible<W::kTree>(a, s, t.row_first / int(a.group), (t.row_first + t.rows - 1) / int(a.group));
    t.units = unit_count(t.keys, kUnit);
    return t;
}

// Deals the units of all items to the CTAs (see kv_attention.cuh) and clears
// the status word.  Items are in the order sequence, tile, kv
// head.  One CTA: sequences are dealt to its warps, a lane sums one of one or
// two tiles and the whole warp one of more; then a scan over the sequences, and
// where each CTA's share starts: by a search for the sequence and, where it has
// more tiles than two, the same walk again.
template <class W>
__global__ void __launch_bounds__(kPlanThreads) kv_chunk_plan_kernel(const __grid_constant__ AttentionArgs a,
                                                                     ChunkPlan* plan, uint32_t grid) {
    release_successor();
    constexpr uint32_t kPlanWarps = kPlanThreads / 32;
    __shared__ uint64_t s_upto[kPlanThreads];  // of a round's sequences: units through each
    __shared__ uint64_t s_warp[kPlanWarps];
    __shared__ int s_bad;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    const auto weight = [&](const KvSeq& s, int tile) -> uint64_t {
        return uint64_t(tile_of<W>(a, s, tile).units + W::kCost) * a.c.kv_heads;
    };
    // the lane's sequence of a round
    const uint32_t nth = lane * kPlanWarps + warp;
    const auto seq_at = [&](uint32_t b) -> KvSeq {
        KvSeq s{0, 0, 0, true};
        if (b < a.b.batch) {
            s = load_seq(a.b, b);
            if (!s.ok) s_bad = 1;
        }
        return s;
    };
    // Calls each(sequence, index in the round) by the whole warp for every sequence
    // of more than two tiles.
    const auto for_large = [&](const KvSeq& s, const auto& each) {
        uint32_t many = __ballot_sync(~0u, tile_count<W>(a, s) > 2);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            each(KvSeq{0, __shfl_sync(~0u, s.t, src), __shfl_sync(~0u, s.n, src), true},
                 uint32_t(src) * kPlanWarps + warp);
        }
    };
    // Units through each of the round's sequences into s_upto; returns the round's.
    const auto round_units = [&](const KvSeq& s) -> uint64_t {
        uint64_t w = 0;
        const int n = tile_count<W>(a, s);
        for (int i = 0; i < n && n <= 2; ++i) w += weight(s, i);
        __syncthreads();
        if (n <= 2) s_upto[nth] = w;
        for_large(s, [&](const KvSeq& o, uint32_t at) {
            uint64_t part = 0;
            for (int i = int(lane), tiles = tile_count<W>(a, o); i < tiles; i += 32) part += weight(o, i);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(~0u, part, d);
            if (lane == 0) s_upto[at] = part;
        });
        __syncthreads();
        uint64_t x = s_upto[tid];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(~0u, x, d);
            if (int(lane) >= d) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        uint64_t all = s_warp[lane];  // as many warps as lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(~0u, all, d);
            if (int(lane) >= d) all += y;
        }
        const uint64_t before = __shfl_sync(~0u, all, int(warp) - 1 + (warp == 0));
        s_upto[tid] = x + (warp == 0 ? 0 : before);
        const uint64_t total = __shfl_sync(~0u, all, 31);
        __syncthreads();
        return total;
    };
    static_assert(kPlanWarps == 32, "the scan over warps");
    uint64_t units = 0;
    KvSeq s{0, 0, 0, true};
    for (uint32_t b0 = 0; b0 < a.b.batch; b0 += kPlanThreads) {
        s = seq_at(b0 + nth);
        units += round_units(s);
    }
    const uint32_t ctas = uint32_t(min(uint64_t(grid), max(units, uint64_t(1))));
    uint64_t base = 0;
    for (uint32_t b0 = 0; b0 < a.b.batch; b0 += kPlanThreads) {
        uint64_t total = units;
        if (a.b.batch > kPlanThreads) {
            s = seq_at(b0 + nth);
            total = round_units(s);
        }
        // the CTAs whose share starts within [lo, hi); share_start(c) < hi without its division
        const auto starts = [&](uint32_t b, uint32_t tile, uint64_t lo, uint64_t hi) {
            for (uint64_t c = (lo * ctas + units - 1) / units; c < ctas && units * c < hi * ctas; ++c)
                plan->start[c] = ChunkStart{b, tile, lo};
        };
        const auto from_of = [&](uint32_t at) { return base + (at == 0 ? 0 : s_upto[at - 1]); };
        // shares that start in a sequence of one or two tiles: a lane each
        const uint64_t u = nth < ctas ? share_start(units, ctas, nth) : ~uint64_t(0);
        if (u >= base && u < base + total) {
            uint32_t at = 0, last = kPlanThreads - 1;
            while (at < last) {
                const uint32_t mid = (at + last) / 2;
                if (s_upto[mid] > u - base)
                    last = mid;
                else
                    at = mid + 1;
            }
            const KvSeq o = load_seq(a.b, b0 + at);
            const int n = tile_count<W>(a, o);
            if (n <= 2) {
                const uint64_t from = from_of(at), x = weight(o, 0);
                const uint32_t tile = n == 2 && u >= from + x ? 1 : 0;
                plan->start[nth] = ChunkStart{b0 + at, tile, from + tile * x};
            }
        }
        for_large(s, [&](const KvSeq& o, uint32_t at) {
            uint64_t from = from_of(at);
            for (int i0 = 0, tiles = tile_count<W>(a, o); i0 < tiles; i0 += 32) {
                const int i = i0 + int(lane);
                const uint64_t x = i < tiles ? weight(o, i) : 0;
                uint64_t y = x;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint64_t z = __shfl_up_sync(~0u, y, d);
                    if (int(lane) >= d) y += z;
                }
                if (x > 0) starts(b0 + at, uint32_t(i), from + y - x, from + y);
                from += __shfl_sync(~0u, y, 31);
            }
        });
        base += total;
    }
    __syncthreads();
    if (tid == 0) {
        plan->units = units;
        plan->ctas = ctas;
        *a.status = s_bad ? SPLITZIP_ERR_INVALID_ARG : SPLITZIP_OK;
    }
}

// One piece of a CTA's share: part or all of an item.
struct Segment {
    int row0, t, held;         // of the sequence: first packed row, new tokens, tokens held
    int row_first, rows;       // of the item: rows of the sequence
    int lo, hi;                // positions that some row of the item sees
    int first_unit, n;         // the piece's units; n = 0: no more pieces
    uint32_t b, head;
    uint32_t first_cta, last_cta;  // whose shares the item is in
};

constexpr int kSegments = 4;  // ring of pieces

// Weights are 2^shift times the exponentials: FP16 ones are then up to 2^8, the
// lag, above 2^7, within FP16's range, and those down to 2^-28 of the largest
// are not lost.
template <bool H>
__host__ __device__ constexpr float weight_shift() {
    return H ? 7.f : 0.f;
}

// FMT 0: cache of the queries' 16-bit type, 1: E5M2, 2: E4M3, 3: as 0, read
// through tensor maps (pages of 8 tokens and more).
template <int FMT, bool H, int D>
struct Chunk {
    static constexpr bool kTma = FMT == 3;
    static constexpr bool kFp8 = FMT == 1 || FMT == 2;
    static constexpr bool kE5M2 = FMT == 1;
    // Both products are in the queries' type.  BF16 holds FP8 values times their
    // scales exactly.  FP16 has not their range: there K goes without its scales,
    // which the scores' columns take, and V is held by halves, which the last
    // division makes good: what was written from FP16 can be 65,536 after its
    // rounding to FP8.  Up to 131,008 that is exact, but for a half of FP16's
    // least step below its normal numbers; larger values are infinite, as they
    // are for a read in FP16.
    static constexpr bool kPvHalf = H;
    static constexpr bool kScoreScale = kFp8 && H;
    static constexpr float kValueScale = kFp8 && H ? 0.5f : 1.f;
    static constexpr float kShift = weight_shift<H>();
    static constexpr int kHalves = D / 64;                 // blocks of 64 columns, 128 bytes a row
    static constexpr int kBlockBytes = 128 * 128;
    static constexpr int kTileBytes = kHalves * kBlockBytes;
    static constexpr int kStages = 131072 / kTileBytes;    // K and V tiles, alternating
    static constexpr int kDepth = kStages / 2;             // units in flight
    // warps: two softmax groups, then loaders, then products and pieces
    static constexpr int kThreads = kTma ? 384 : 512;
    static constexpr uint32_t kProductWarp = kTma ? 9 : 12, kSegmentWarp = kProductWarp + 1;
    static constexpr int kLagTiles = kFp8 ? 1 : 2;         // copies in flight ahead of their hand-over
    static constexpr int kRaw = kFp8 ? 2 : 0;              // FP8 staging buffers
    static constexpr int kRawBytes = 128 * D;
    static constexpr int kChunks = kFp8 ? D / 16 : D / 8;  // 16-byte pieces of a cache row
    static constexpr int kRowStep = 128 / kChunks;         // rows that the loaders copy at a time
    // Slots of the scores' factors, a unit each.  Nothing but the stages holds the
    // loaders back: unit u is described when K of unit u - 1 has a stage, so when the
    // scores of unit u - 1 - kDepth are done, and the softmax may still be about to
    // read the factors of that unit and of all after it.
    static constexpr uint32_t kFactors = kDepth > 2 ? 8 : 4;
    static_assert(kFactors >= kDepth + 2, "factors of units in flight");

    struct Shared {
        uint8_t q[2][kTileBytes];
        uint8_t stage[kStages][kTileBytes];
        uint8_t raw[kRaw > 0 ? kRaw : 1][kRaw > 0 ? kRawBytes : 16];
        // of a unit's keys: byte offset in the pools, or page (FP8, which has no room); -1: none
        std::conditional_t<kFp8, int32_t, int64_t> place[2][kTma ? 1 : kUnit];
        alignas(16) uint16_t k_factor[kScoreScale ? kFactors : 1][kScoreScale ? kUnit : 8];  // K's scales in BF16, for the scores
        uint8_t k_scale[4][kFp8 && !kScoreScale ? kUnit : 4], v_scale[4][kFp8 ? kUnit : 4];
        uint64_t kv_full[kStages];
        uint64_t freed[kDepth];          // K of unit u and V of unit u - 1 are no longer read
        uint64_t q_full[2], s_full[2], p_full[2], o_full[2], noted, drained;
        uint64_t seg_full[kSegments], seg_empty[kSegments];
        uint32_t tmem;
        Segment seg[kSegments];
    };
    static constexpr int kSmem = int(sizeof(Shared));
};

// Walks the CTA's share, whose first unit is `start`'s, and describes its
// pieces to the other roles (one thread, ahead of them by up to kSegments).
template <class W, class Shared>
__device__ __forceinline__ void walk_share(const AttentionArgs& a, Shared& sh, uint64_t units, uint32_t ctas,
                                           const ChunkStart& start, ChunkSplit* splits, bool& ok) {
    splits[blockIdx.x] = ChunkSplit{};
    uint64_t u = 0, end = 0, group_start = start.group_start;
    uint32_t b = start.b, tile = start.tile;
    if (blockIdx.x < ctas) {
        u = share_start(units, ctas, blockIdx.x);
        end = share_start(units, ctas, uint64_t(blockIdx.x) + 1);
    }
    for (uint32_t i = 0; ok; ++i) {
        Segment g{};
        while (g.n == 0 && u < end) {
            KvSeq s;
            Tile t;
            uint32_t size = 0;
            while (true) {
                s = load_seq(a.b, b);
                if (int(tile) >= tile_count<W>(a, s)) {
                    ++b;
                    tile = 0;
                    continue;
                }
                t = tile_of<W>(a, s, int(tile));
                size = uint32_t(t.units + W::kCost);
                if (u < group_start + uint64_t(size) * a.c.kv_heads) break;
                group_start += uint64_t(size) * a.c.kv_heads;
                ++tile;
            }
            const uint32_t head = uint32_t((u - group_start) / size);
            const uint64_t keys_start = group_start + uint64_t(head) * size + W::kCost;
            const uint64_t item_end = keys_start + uint32_t(t.units);
            const uint64_t from = max(u, keys_start), stop = min(item_end, end);
            if (from >= stop) {  // the share ends before the item's keys
                u = end;
                break;
            }
            u = stop;
            g.row0 = s.row0, g.t = s.t, g.held = s.n;
            g.row_first = t.row_first, g.rows = t.rows;
            g.lo = t.keys.lo, g.hi = t.keys.hi;
            g.first_unit = t.keys.lo / kUnit + int(from - keys_start);
            g.n = int(stop - from);
            g.b = b, g.head = head;
            g.first_cta = share_of(units, ctas, keys_start);
            g.last_cta = share_of(units, ctas, item_end - 1);
            if (g.first_cta == blockIdx.x && g.last_cta > g.first_cta)
                splits[blockIdx.x] = ChunkSplit{g.row0, g.row_first, g.rows, head, g.last_cta};
        }
        if (i >= uint32_t(kSegments)) ok = mbar_wait(&sh.seg_empty[i % kSegments], (i / kSegments - 1) & 1u);
        if (!ok) break;
        sh.seg[i % kSegments] = g;
        mbar_arrive(&sh.seg_full[i % kSegments]);
        if (g.n == 0) break;
    }
}

// The same with what the plan kernel found.
template <class W, class Shared>
__device__ __forceinline__ void segment_role(const AttentionArgs& a, Shared& sh, const ChunkPlan* plan, ChunkSplit* splits,
                                             bool& ok) {
    const uint64_t units = __ldcg(&plan->units);
    const uint32_t ctas = __ldcg(&plan->ctas);
    ChunkStart start{0, 0, 0};
    if (blockIdx.x < ctas && share_start(units, ctas, blockIdx.x) < share_start(units, ctas, uint64_t(blockIdx.x) + 1))
        start = ChunkStart{__ldcg(&plan->start[blockIdx.x].b), __ldcg(&plan->start[blockIdx.x].tile),
                           __ldcg(&plan->start[blockIdx.x].group_start)};
    walk_share<W>(a, sh, units, ctas, start, splits, ok);
}

// Waits until the stage of tile x (K of unit x / 2 where even, else V) can be
// overwritten.
template <class C>
__device__ __forceinline__ bool await_freed(typename C::Shared& sh, uint32_t x) {
    const int u = int(x >> 1) - C::kDepth + int(x & 1u);  // which release
    return u < 0 || mbar_wait(&sh.freed[u % C::kDepth], uint32_t(u / C::kDepth) & 1u);
}

template <int FMT, bool H, int D>
__device__ __forceinline__ void load_role(const AttentionArgs& a, typename Chunk<FMT, H, D>::Shared& sh,
                                          bool& ok, bool& bad) {
    using C = Chunk<FMT, H, D>;
    const uint32_t lt = threadIdx.x - 256u;
    const uint32_t c = lt % C::kChunks, r0 = lt / C::kChunks;
    uint32_t made = 0, handed = 0;  // tiles whose copies were started, and handed over

    const auto await_empty = [&](uint32_t x) {
        if (ok) ok = await_freed<C>(sh, x);
    };
    // Hands over tile `handed`, whose copies by this thread have landed.
    const auto hand_over = [&]() {
        const uint32_t x = handed++, st = x % C::kStages;
        if (C::kFp8) {
            await_empty(x);
            const bool is_v = x & 1u;
            const uint32_t ring = (x >> 1) & 3u;
            const uint8_t* scales = is_v || C::kScoreScale ? sh.v_scale[ring] : sh.k_scale[ring];
            if (ok) {
#pragma unroll
                for (int i0 = 0; i0 < C::kChunks; i0 += 4) {
                    // loads first: to the compiler the stores could be to the same memory
                    uint4 raw[4];
                    uint32_t scale[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        raw[i] = *reinterpret_cast<const uint4*>(sh.raw[x % 2] + (uint32_t(i0 + i) * 128u + lt) * 16u);
                        scale[i] = scales[r0 + uint32_t(i0 + i) * C::kRowStep];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t r = r0 + uint32_t(i0 + i) * C::kRowStep;
                        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                        uint32_t o[8];
                        if (C::kScoreScale && !is_v) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[j] = fp8_pair_to_half2<C::kE5M2>(w[j / 2], j & 1);
                        } else if (H) {
                            const float f = C::kValueScale * scale_value(scale[i]);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 v = half2_to_float2(fp8_pair_to_half2<C::kE5M2>(w[j / 2], j & 1));
                                const float2 z = mul2(v, make_float2(f, f));
                                o[j] = pack_half2(z.x, z.y);
                            }
                        } else {
                            // exact: BF16 holds the value and its product with a power of two
                            const uint32_t s16 = scale[i] * 0x00800080u;
                            const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&s16);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 f = half2_to_float2(fp8_pair_to_half2<C::kE5M2>(w[j / 2], j & 1));
                                const uint32_t v = pack_bf16x2(f.x, f.y);
                                const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), s2);
                                o[j] = *reinterpret_cast<const uint32_t*>(&z);
                            }
                        }
                        uint8_t* row = sh.stage[st] + (c >> 2) * C::kBlockBytes + r * 128u;
                        *reinterpret_cast<uint4*>(row + ((((2u * c) & 7u) ^ (r & 7u)) << 4)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(row + ((((2u * c + 1u) & 7u) ^ (r & 7u)) << 4)) =
                            make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
        }
        fence_async_proxy();
        __syncwarp();
        if ((lt & 31u) == 0) mbar_arrive(&sh.kv_full[st]);
    };

    for (uint32_t piece = 0;; ++piece) {
        const Segment& w = sh.seg[piece % kSegments];
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = named_barrier_and(1, 128, ok);
        if (!ok || w.n == 0) break;
        const int32_t* table = a.b.table + uint64_t(w.b) * a.b.table_stride;
        const auto page_of = [&](int j) -> int32_t {
            const int pos = (w.first_unit + j) * kUnit + int(lt);
            if (j >= w.n || pos < w.lo || pos >= w.hi) return -1;
            const int32_t pg = table[uint32_t(pos) >> a.c.page_shift];
            if (pg < 0 || uint64_t(pg) >= a.c.pool_pages) {
                bad = true;
                return -1;
            }
            return pg;
        };
        const uint32_t slots = (1u << a.c.page_shift) - 1u;
        // A unit's pages are looked up two units before it, its scales one, so that neither is
        // waited for (2,048 tokens over 8,192 of E4M3: 277 -> 261 us).
        const auto scales_at = [&](int j, int32_t pg, uint32_t& k, uint32_t& v) {
            k = v = 127;
            if (C::kFp8 && pg >= 0) {
                const uint32_t slot = (uint32_t(w.first_unit + j) * kUnit + lt) & slots;
                const uint64_t at = ((uint64_t(uint32_t(pg)) * a.c.kv_heads + w.head) << a.c.page_shift) + slot;
                k = __ldg(a.c.k_scale + at);
                v = __ldg(a.c.v_scale + at);
            }
        };
        int32_t page = page_of(0), next_page = page_of(1);
        uint32_t k_scale, v_scale;
        scales_at(0, page, k_scale, v_scale);
        for (int j = 0; j < w.n; ++j) {
            const uint32_t unit = made >> 1;  // of the share
            const int pos0 = (w.first_unit + j) * kUnit;
            {
                const uint32_t slot = (uint32_t(pos0) + lt) & slots;
                if (!C::kFp8) {
                    sh.place[unit & 1u][lt] = page < 0 ? -1
                                                       : int64_t(uint64_t(uint32_t(page)) * a.c.page_stride +
                                                                 uint64_t(slot) * a.c.token_stride);
                } else {
                    sh.place[unit & 1u][lt] = page;
                    if (C::kScoreScale)
                        sh.k_factor[unit % C::kFactors][lt] = uint16_t(k_scale << 7);
                    else
                        sh.k_scale[unit & 3u][lt] = uint8_t(k_scale);
                    sh.v_scale[unit & 3u][lt] = uint8_t(v_scale);
                }
            }
            page = next_page;
            next_page = page_of(j + 2);
            scales_at(j + 1, page, k_scale, v_scale);
            named_barrier(1, 128);
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const uint32_t x = made++;
                const uint8_t* pool = (side ? a.c.v : a.c.k) + uint64_t(w.head) * a.c.head_stride + c * 16u;
                if (!C::kFp8) await_empty(x);
                if (ok) {
                    const uint32_t dst = C::kFp8 ? smem_u32(sh.raw[x % 2])
                                                 : smem_u32(sh.stage[x % C::kStages]) + (c >> 3) * C::kBlockBytes;
#pragma unroll
                    for (int i0 = 0; i0 < C::kChunks; i0 += 8) {
                        // all places first: the copies are barriers to the compiler
                        int64_t pl[8];
#pragma unroll
                        for (int i = 0; i < 8 && i0 + i < C::kChunks; ++i)
                            pl[i] = sh.place[unit & 1u][r0 + uint32_t(i0 + i) * C::kRowStep];
#pragma unroll
                        for (int i = 0; i < 8 && i0 + i < C::kChunks; ++i) {
                            const uint32_t r = r0 + uint32_t(i0 + i) * C::kRowStep;
                            uint64_t off = uint64_t(max(pl[i], int64_t(0)));
                            if (C::kFp8)
                                off = off * a.c.page_stride + uint64_t((uint32_t(pos0) + r) & slots) * a.c.token_stride;
                            const uint32_t to = C::kFp8 ? dst + (uint32_t(i0 + i) * 128u + lt) * 16u
                                                        : dst + r * 128u + (((c & 7u) ^ (r & 7u)) << 4);
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(pool + off),
                                         "r"(pl[i] < 0 ? 0 : 16)
                                         : "memory");
                        }
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (made > uint32_t(C::kLagTiles)) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(C::kLagTiles) : "memory");
                    hand_over();
                }
            }
        }
        __syncwarp();
        if ((lt & 31u) == 0) mbar_arrive(&sh.seg_empty[piece % kSegments]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    while (handed < made) hand_over();
}

// The loader of a 16-bit cache whose pages are whole swizzle groups of eight
// tokens: one warp, a lane a box of up to 128 tokens by 64 columns.  Boxes that
// hold nothing an item sees lie past the last page, which reads as zeros.
template <class C>
__device__ __forceinline__ void load_tma_role(const AttentionArgs& a, typename C::Shared& sh, const CUtensorMap* k_map,
                                              const CUtensorMap* v_map, bool& ok, bool& bad) {
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t page_tokens = 1u << a.c.page_shift, box = min(page_tokens, uint32_t(kUnit));
    const uint32_t half = lane % C::kHalves, nth = lane / C::kHalves;  // of the lane's box: column block, box of the unit
    const bool mine = nth < kUnit / box;
    uint32_t made = 0, issued = 0;
    for (uint32_t piece = 0;; ++piece) {
        const Segment& w = sh.seg[piece % kSegments];
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = __all_sync(~0u, ok);
        if (!ok || w.n == 0) break;
        const int32_t* table = a.b.table + uint64_t(w.b) * a.b.table_stride;
        const auto page_of = [&](int j) -> int32_t {
            const int pos = (w.first_unit + j) * kUnit + int(nth * box);
            if (!mine || j >= w.n || pos + int(box) <= w.lo || pos >= w.hi) return -1;
            const int32_t pg = table[uint32_t(pos) >> a.c.page_shift];
            if (pg < 0 || uint64_t(pg) >= a.c.pool_pages) {
                bad = true;
                return -1;
            }
            return pg;
        };
        const int n = w.n, first_unit = w.first_unit;
        const int head = int(w.head);
        int32_t page = page_of(0);
        for (int j = 0; j < n; ++j) {
            const int token = ((first_unit + j) * kUnit + int(nth * box)) & int(page_tokens - 1u);
            const int32_t at = page < 0 ? int32_t(a.c.pool_pages) : page;
            page = page_of(j + 1);
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const uint32_t x = made++, st = x % C::kStages;
                if (ok) ok = await_freed<C>(sh, x);
                ok = __all_sync(~0u, ok);
                if (!ok) continue;
                issued = made;
                if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[st], C::kTileBytes);
                __syncwarp();
                if (mine)
                    tensor_load_4d(sh.stage[st] + half * C::kBlockBytes + nth * box * 128u, side ? v_map : k_map,
                                   int(half * 64u), head, token, at, &sh.kv_full[st]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[piece % kSegments]);
    }
    // no copy is in flight when the CTA ends
    for (uint32_t i = 0; i < uint32_t(C::kStages) && i < issued; ++i) {
        const uint32_t x = issued - 1 - i;
        if (!mbar_wait(&sh.kv_full[x % C::kStages], (x / C::kStages) & 1u)) ok = false;
    }
}

// One warp, converged, whose elected lane issues.  What lies between two
// steps' products counts, for the tensor core queues few of them: a wait of its
// own between them cost some 45 cycles of it.  So a step (a tile's weights
// times V, then its next scores) is asked for while the products before it are
// issued, and waited for only where it was not ready then.
template <int FMT, bool H, int D>
__device__ __forceinline__ void product_role(typename Chunk<FMT, H, D>::Shared& sh, uint32_t tmem, bool& ok) {
    using C = Chunk<FMT, H, D>;
    constexpr uint32_t kShapeS = tc_shape(!H, 128, 128, false);
    constexpr uint32_t kShapeO = tc_shape(!C::kPvHalf, 128, D, true);
    constexpr uint32_t kTileStep = C::kTileBytes >> 4, kBlockStep = C::kBlockBytes >> 4;  // in the descriptors' units
    const uint64_t q_operand = smem_operand(smem_u32(sh.q[0]), 16, 1024);
    const uint64_t k_operand = smem_operand(smem_u32(sh.stage[0]), 16, 1024);
    const uint64_t v_operand = smem_operand(smem_u32(sh.stage[1]), C::kBlockBytes, 1024);
    const bool leader = elect_lane();
    const auto scores = [&](int g, uint32_t stage) {
        const uint64_t q = q_operand + uint32_t(g) * kTileStep, kk = k_operand + stage * (2u * kTileStep);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = uint32_t(k / 4) * kBlockStep + uint32_t(k % 4) * 2u;
            tc_mma(leader && ok, tmem + uint32_t(g) * 128u, q + at, kk + at, kShapeS, k > 0);
        }
    };
    const auto sums = [&](int g, uint32_t stage, bool first) {
        const uint64_t v = v_operand + stage * (2u * kTileStep);
#pragma unroll
        for (int k = 0; k < kUnit / 16; ++k)
            tc_mma_ta(leader && ok, tmem + 256u + uint32_t(g) * 128u, tmem + uint32_t(g) * 128u + uint32_t(k) * 8u,
                      v + uint32_t(k) * (2048u >> 4), kShapeO, k > 0 || !first);
    };
    uint32_t unit = 0;  // of the share
    uint32_t segments[2] = {0, 0}, weights[2] = {0, 0};
    for (uint32_t piece = 0;; ++piece) {
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = __all_sync(~0u, ok);
        const int n = ok ? sh.seg[piece % kSegments].n : 0;
        if (n == 0) break;
        const bool two = sh.seg[piece % kSegments].rows > kTileRows;
        __syncwarp();
        if (leader) mbar_arrive(&sh.seg_empty[piece % kSegments]);
        // the first scores
        if (ok) ok = mbar_wait(&sh.kv_full[2u * (unit % C::kDepth)], (unit / C::kDepth) & 1u);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (g == 1 && !two) break;
            if (ok) ok = mbar_wait(&sh.q_full[g], segments[g]++ & 1u);
            tc_fence_after();
            scores(g, unit % C::kDepth);
            if (leader && ok) tc_commit(&sh.s_full[g]);
        }
        if (leader && ok) tc_commit(&sh.freed[unit % C::kDepth]);
        bool ready0 = false, ready1 = false;
        for (int j = 0; j < n; ++j, ++unit) {
            const bool last = j == n - 1;
            const uint32_t stage = unit % C::kDepth, phase = (unit / C::kDepth) & 1u;
            const uint32_t next = (unit + 1) % C::kDepth, next_phase = ((unit + 1) / C::kDepth) & 1u;
            const uint32_t turn0 = weights[0]++ & 1u, turn1 = weights[1] & 1u;
            if (!ready0) {
                if (ok) ok = mbar_wait(&sh.p_full[0], turn0);
                if (ok) ok = mbar_wait(&sh.kv_full[2u * stage + 1u], phase);
                if (ok && !last) ok = mbar_wait(&sh.kv_full[2u * next], next_phase);
            }
            tc_fence_after();
            sums(0, stage, j == 0);
            ready1 = two && mbar_try_wait(&sh.p_full[1], turn1);
            if (last) {
                if (leader && ok) tc_commit(&sh.o_full[0]);
            } else {
                scores(0, next);
                if (leader && ok) tc_commit(&sh.s_full[0]);
            }
            if (two) {
                ++weights[1];
                if (!ready1 && ok) ok = mbar_wait(&sh.p_full[1], turn1);
                tc_fence_after();
                sums(1, stage, j == 0);
                if (last) {
                    if (leader && ok) tc_commit(&sh.o_full[1]);
                } else {
                    scores(1, next);
                    if (leader && ok) tc_commit(&sh.s_full[1]);
                }
            }
            if (!last) {
                // the next unit's first tile: its weights, V, and the keys after
                const uint32_t after = (unit + 2) % C::kDepth, after_phase = ((unit + 2) / C::kDepth) & 1u;
                ready0 = mbar_try_wait(&sh.p_full[0], turn0 ^ 1u) & mbar_try_wait(&sh.kv_full[2u * next + 1u], next_phase);
                if (j + 2 < n) ready0 &= mbar_try_wait(&sh.kv_full[2u * after], after_phase);
                if (leader && ok) tc_commit(&sh.freed[next]);
            }
        }
    }
    // no product is in flight when the CTA gives its memory back
    if (leader) tc_commit(&sh.drained);
    __syncwarp();
    if (!mbar_wait(&sh.drained, 0)) ok = false;
}

// Columns of a row that an infinity or a NaN (both) of V reaches.
template <int D>
struct Reached {
    uint32_t plus[D / 32], minus[D / 32];
};

// The n lowest bits (none for n <= 0).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Which keys of a unit a row sees: from .. to - 1, or a bit for each.
struct SeenRange {
    int from, to;
    __device__ bool operator()(int key) const { return key >= from && key < to; }
};
struct SeenBits {
    uint32_t w[4];
    __device__ bool operator()(int key) const { return w[key >> 5] >> (key & 31) & 1u; }
};

// Notes the infinities and NaN of a V tile for a row.  Out of line: it hardly ever runs, and its registers are not
// to weigh on the loop around it.
template <bool H, int D, class Seen>
__device__ __noinline__ void note_special(const uint8_t* v, Seen seen, Reached<D>* reached) {
    constexpr uint32_t kInf = H ? 0x7C00u : 0x7F80u;
    for (int key = 0; key < kUnit; ++key) {
        const bool sees = seen(key);
        for (int k = 0; k < D / 2; ++k) {
            const uint32_t y = *reinterpret_cast<const uint32_t*>(
                v + (k >> 5) * (128 * 128) + key * 128 + ((((k >> 2) & 7) ^ (key & 7)) << 4) + (k & 3) * 4);
            for (int z = 0; z < 2; ++z) {
                const uint32_t bits = (y >> (16 * z)) & 0xFFFFu, mag = bits & 0x7FFFu, at = uint32_t(2 * k + z);
                if (mag >= kInf && sees) {
                    if (mag > kInf || !(bits & 0x8000u)) reached->plus[at >> 5] |= 1u << (at & 31u);
                    if (mag > kInf || (bits & 0x8000u)) reached->minus[at >> 5] |= 1u << (at & 31u);
                }
            }
        }
    }
}

// Where row `row` of a CTA's part of an item that CTA `first` begins is: columns
// o[0] .. o[D - 1], reference, sum, part_stride() floats apart.  A part lies in
// tiles of kTileRows rows, a tree's in a.part_blocks blocks of kFewRows, so that
// trees of few rows do with one.
template <bool TREE>
__device__ __forceinline__ constexpr int part_stride() {
    return TREE ? int(kFewRows) : kTileRows;
}

template <int D, bool TREE>
__device__ __forceinline__ float* part_at(const AttentionArgs& a, uint32_t cta, uint32_t first, uint32_t row,
                                          uint32_t blocks) {
    constexpr uint32_t kStride = part_stride<TREE>();
    const uint64_t slot = uint64_t(cta) * 2 + (cta == first ? 1 : 0);
    return a.parts + (slot * blocks + row / kStride) * (kStride * (D + 2)) + row % kStride;
}

// The natural logarithm of a row's sum of exponentials l against reference m.
__device__ __forceinline__ float log_sum(float m, float l, float scale, float shift) {
    return l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m * scale) - shift + log2f(l)) * 0.693147180559945309f;
}

template <int FMT, bool H, int D, bool TREE>
__device__ __forceinline__ void softmax_role(const AttentionArgs& a, typename Chunk<FMT, H, D>::Shared& sh,
                                             uint32_t tmem, bool& ok) {
    using C = Chunk<FMT, H, D>;
    const int g = int(threadIdx.x >> 7);
    const uint32_t row = threadIdx.x & 127u, lane = threadIdx.x & 31u, warp = row >> 5;
    const uint32_t lanes = (warp * 32u) << 16;
    const uint32_t s_at = tmem + lanes + uint32_t(g) * 128u, o_at = tmem + lanes + 256u + uint32_t(g) * 128u;
    const float scale = a.scale_log2;
    // A row of 16-bit elements is kLanes 16-byte pieces; a warp moves kMoves of
    // them for each of its rows, so that its accesses to memory are whole rows.
    constexpr uint32_t kLanes = D / 8;
    constexpr int kMoves = int(kLanes);
    const uint32_t piece_col = lane % kLanes, piece_row = lane / kLanes;
    // a row's piece in the group's part of sh.q, in the swizzle of the operands
    const auto staged = [&](uint32_t r, uint32_t c) {
        return reinterpret_cast<uint4*>(sh.q[g] + (c >> 3) * C::kBlockBytes + r * 128u + (((c & 7u) ^ (r & 7u)) << 4));
    };
    uint32_t segments = 0, units_done = 0, tile = 0, noted = 0;
    const auto await = [&](uint64_t* bar, uint32_t count) {
        if (ok) ok = mbar_wait(bar, count & 1u);
        ok = __all_sync(~0u, ok);
        tc_fence_after();
    };
    for (uint32_t piece = 0;; ++piece) {
        const Segment& w = sh.seg[piece % kSegments];
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = named_barrier_and(2 + uint32_t(g), 128, ok);
        if (!ok || w.n == 0) break;
        const auto leave = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.seg_empty[piece % kSegments]);
        };
        const int n = w.n;
        const uint32_t first_tile = tile;
        tile += 2u * uint32_t(n);
        if (g == 1 && w.rows <= kTileRows) {
            leave();
            continue;
        }
        // the thread's row: its packed row and head, -1 where there is none
        const auto place = [&](const KvRows& rows) -> int64_t {
            const int r = w.row_first + int(row) + g * kTileRows;  // of the sequence
            if (r >= w.row_first + w.rows) return -1;
            const int i = r / int(a.group);
            return int64_t(uint64_t(w.row0 + i) * rows.token_stride +
                           uint64_t(w.head * a.group + uint32_t(r - i * int(a.group))) * rows.head_stride);
        };
        KeyRange see, each;  // what the row sees, what every row of the item sees
        int mask_row = -1;   // a tree's row: with the bits of its mask besides
        {
            const KvSeq seq{w.row0, w.t, w.held, true};
            const int r = w.row_first + int(row) + g * kTileRows;
            const int i = r / int(a.group), i1 = (w.row_first + w.rows - 1) / int(a.group);
            const bool live = r < w.row_first + w.rows;
            if (TREE) {
                see = live ? visible_before(a, seq, i) : KeyRange{0, 0};
                if (live && w.held - w.t + i >= 0) mask_row = w.row0 + i;
                each = visible_to_all_before(a, seq, i1);
            } else {
                see = visible<false>(a, seq, i);
                if (!live) see.lo = see.hi = 0;
                each.hi = visible<false>(a, seq, w.row_first / int(a.group)).hi;
                each.lo = visible<false>(a, seq, i1).lo;
            }
        }
        {
            // the rows of Q, zeros where there is none; a negative scale's sign goes to Q
            const int64_t mine = place(a.q);
            const uint32_t flip = a.negate ? 0x80008000u : 0u;
            uint4 x[kMoves];
#pragma unroll
            for (int k = 0; k < kMoves; ++k) {
                const int64_t at = __shfl_sync(~0u, mine, k * int(32 / kLanes) + int(piece_row));
                x[k] = at < 0 ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4*>(a.q.d + at)[piece_col];
            }
#pragma unroll
            for (int k = 0; k < kMoves; ++k)
                *staged(warp * 32u + uint32_t(k) * (32 / kLanes) + piece_row, piece_col) =
                    make_uint4(x[k].x ^ flip, x[k].y ^ flip, x[k].z ^ flip, x[k].w ^ flip);
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[g]);
        }
        float low = -INFINITY;  // what exponentials are taken against, before the scale
        float sum = 0.f;
        Reached<D> reached;
        bool reaches = false;
        for (int j = 0; j < n; ++j) {
            const int pos0 = (w.first_unit + j) * kUnit;
            await(&sh.s_full[g], units_done++);
            uint32_t x[128];
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_load32(x + 32 * k, s_at + 32u * uint32_t(k));
            tmem_wait_load();
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_loaded32(x + 32 * k);
            if (C::kScoreScale) {
                const uint4* ks = reinterpret_cast<const uint4*>(sh.k_factor[((first_tile >> 1) + uint32_t(j)) % C::kFactors]);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint4 f8 = ks[k];
                    const uint32_t f[4] = {f8.x, f8.y, f8.z, f8.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int at = 8 * k + 2 * y;
                        const float2 z = mul2(make_float2(__uint_as_float(x[at]), __uint_as_float(x[at + 1])),
                                              bf16x2_to_float2(f[y]));
                        x[at] = __float_as_uint(z.x), x[at + 1] = __float_as_uint(z.y);
                    }
                }
            }
            const int from = see.lo - pos0, to = see.hi - pos0;
            std::conditional_t<TREE, SeenBits, SeenRange> seen;
            if constexpr (!TREE) {
                seen = SeenRange{from, to};
                if (!__all_sync(~0u, from <= 0 && to >= kUnit)) {
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k < from || k >= to) x[k] = 0xFF800000u;
                }
            } else {
                if (!__all_sync(~0u, from <= 0 && to >= kUnit)) {
                    const uint32_t* row = a.mask + uint64_t(uint32_t(max(mask_row, 0))) * a.words;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t bits = mask_row < 0 ? 0u : mask_bits(row, a.words, pos0 + 32 * y - (w.held - w.t));
                        // the range's keys, and of the new tokens those that there are
                        seen.w[y] = (low_bits(to - 32 * y) & ~low_bits(from - 32 * y)) |
                                    (bits & low_bits(w.held - pos0 - 32 * y));
                    }
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (!(seen.w[k >> 5] >> (k & 31) & 1u)) x[k] = 0xFF800000u;
                } else {
                    seen = SeenBits{{~0u, ~0u, ~0u, ~0u}};
                }
            }
            float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
            for (int k = 0; k < 128; k += 8) {
                m0 = max3(m0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                m1 = max3(m1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
                m2 = max3(m2, __uint_as_float(x[k + 4]), __uint_as_float(x[k + 5]));
                m3 = max3(m3, __uint_as_float(x[k + 6]), __uint_as_float(x[k + 7]));
            }
            const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
            const bool grew = top > low + a.lag;
            const float f = grew ? exp2_fast((low - top) * scale) : 1.f;
            if (grew) low = top;
            if (j > 0 && __any_sync(~0u, grew)) {
                // S(j) done means that the product before it is: o can be rescaled
#pragma unroll 1
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t o[16];
                    tmem_load16(o, o_at + 16u * uint32_t(k));
                    tmem_wait_load();
                    tmem_loaded16(o);
#pragma unroll
                    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                    tmem_store16(o_at + 16u * uint32_t(k), o);
                }
            }

            // A weight of 0 hides a finite value of V, not an infinity or a NaN: where
            // some row of the item does not see all of this unit's keys, such values
            // are noted for the rows that see them and taken out of V.
            const int k0 = max(pos0, w.lo), k1 = min(pos0 + kUnit, w.hi);
            if (k0 < k1 && (each.hi < k1 || each.lo > k0 || (C::kTma && (k0 > pos0 || k1 < pos0 + kUnit)))) {
                // the same in all rows' threads
                const uint32_t v_tile = first_tile + 2u * uint32_t(j) + 1u, st = v_tile % C::kStages;
                if (ok) ok = mbar_wait(&sh.kv_full[st], (v_tile / C::kStages) & 1u);
                uint8_t* v = sh.stage[st];
                constexpr uint32_t kInf = C::kPvHalf ? 0x7C00u : 0x7F80u;
                uint32_t most = 0;
                if (C::kTma && (k0 > pos0 || k1 < pos0 + kUnit)) {
                    // a page's tokens past the sequence's end came too: out of the
                    // products (group 1's are issued after group 0's), and of the search
                    const bool out = pos0 + int(row) < k0 || pos0 + int(row) >= k1;
                    if (g == 0 && out && ok) {
                        for (int k = 0; k < D / 8; ++k)
                            *reinterpret_cast<uint4*>(v + (k >> 3) * C::kBlockBytes + row * 128u + (k & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_async_proxy();
                }
#pragma unroll 8
                for (int k = 0; k < C::kTileBytes / 2048; ++k) {
                    const int key = pos0 + int((uint32_t(k) * 16u + (row >> 3)) & 127u);  // 8 pieces a row
                    if (C::kTma && (key < k0 || key >= k1)) continue;
                    const uint4 y = *reinterpret_cast<const uint4*>(v + (uint32_t(k) * 128u + row) * 16u);
                    most = __vmaxu2(most, __vmaxu2(__vmaxu2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu),
                                                   __vmaxu2(y.z & 0x7FFF7FFFu, y.w & 0x7FFF7FFFu)));
                }
                const bool special = (most & 0xFFFFu) >= kInf || (most >> 16) >= kInf;
                if (named_barrier_popc(2 + uint32_t(g), 128, special) > 0) {  // the same in both groups
                    if (!reaches) reached = Reached<D>{};
                    reaches = true;
                    note_special<C::kPvHalf, D>(v, seen, &reached);
                    // group 0 takes them out once both have noted them; group 1's product
                    // is issued after group 0's
                    if (g == 1) mbar_arrive(&sh.noted);
                    if (g == 0 && w.rows > kTileRows && ok) ok = mbar_wait(&sh.noted, noted++ & 1u);
                    if (g == 0) ok = named_barrier_and(2, 128, ok);  // nor does a warp of group 0 still look for them
                    if (g == 0 && ok) {
                        for (int k = 0; k < C::kTileBytes / 512; ++k) {
                            uint32_t* at = reinterpret_cast<uint32_t*>(v) + uint32_t(k) * 128u + row;
                            uint32_t y = *at;
                            if ((y & 0x7FFFu) >= kInf) y &= 0xFFFF0000u;
                            if (((y >> 16) & 0x7FFFu) >= kInf) y &= 0x0000FFFFu;
                            *at = y;
                        }
                        fence_async_proxy();
                    }
                }
            }
            const float ref = C::kShift - (low == -INFINITY ? 0.f : low * scale);
            const float2 scale2 = make_float2(scale, scale), ref2 = make_float2(ref, ref);
            float2 part[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 z = fma2(make_float2(__uint_as_float(x[32 * y + 2 * k]),
                                                      __uint_as_float(x[32 * y + 2 * k + 1])), scale2, ref2);
                    const float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
                    part[k & 3] = add2(part[k & 3], e);
                    p[k] = C::kPvHalf ? pack_half2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                }
                tmem_store16(s_at + uint32_t(16 * y), p);
            }
            tmem_wait_store();
            tc_fence_before();
            // one arrival a warp: 32 lanes' would be taken one after the other
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&sh.p_full[g]);
            part[0] = add2(add2(part[0], part[1]), add2(part[2], part[3]));
            sum = sum * f + (part[0].x + part[0].y);
        }

        // the piece's sums
        await(&sh.o_full[g], segments++);
        const uint32_t first = w.first_cta, last = w.last_cta;
        const bool whole = first == last;
        // 32 columns of the row, divided, to the stage
        const auto stage32 = [&](int k, const float* o, float f) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint32_t z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[e] = H ? pack_half2(o[8 * y + 2 * e] * f, o[8 * y + 2 * e + 1] * f)
                             : pack_bf16x2(o[8 * y + 2 * e] * f, o[8 * y + 2 * e + 1] * f);
                *staged(row, uint32_t(4 * k + y)) = make_uint4(z[0], z[1], z[2], z[3]);
            }
        };
        // the staged rows of the warp and their logarithms to memory
        const auto put = [&](float m, float l) {
            __syncwarp();
            const int64_t mine = place(a.out);
#pragma unroll
            for (int k = 0; k < kMoves; ++k) {
                const uint32_t r = uint32_t(k) * (32 / kLanes) + piece_row;
                const int64_t at = __shfl_sync(~0u, mine, int(r));
                const uint4 y = *staged(warp * 32u + r, piece_col);
                if (at >= 0) reinterpret_cast<uint4*>(a.out.d + at)[piece_col] = y;
            }
            if (a.lse && mine >= 0) {
                const int r = w.row_first + int(row) + g * kTileRows, i = r / int(a.group);
                a.lse[uint64_t(w.row0 + i) * a.q_heads + w.head * a.group + uint32_t(r - i * int(a.group))] =
                    log_sum(m, l, scale, C::kShift);
            }
        };
        // 32 columns of the row's sums
        const auto sums32 = [&](int k, float* o) {
            uint32_t bits[32];
            tmem_load32(bits, o_at + 32u * uint32_t(k));
            tmem_wait_load();
            tmem_loaded32(bits);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __uint_as_float(bits[y]);
            if (reaches) {
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                    if (reached.plus[k] >> y & 1u) o[y] += INFINITY;
                    if (reached.minus[k] >> y & 1u) o[y] += -INFINITY;
                }
            }
        };
        if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / (C::kValueScale * sum);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                float o[32];
                sums32(k, o);
                stage32(k, o, inv);
            }
            put(low, sum);
        } else {
            const bool live = int(row) + g * kTileRows < w.rows;
            constexpr int kStride = part_stride<TREE>();
            float* mine = part_at<D, TREE>(a, blockIdx.x, first, row + uint32_t(g) * kTileRows, TREE ? a.part_blocks : 2);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                float o[32];
                sums32(k, o);
                if (live) {
#pragma unroll
                    for (int y = 0; y < 32; ++y) mine[(32 * k + y) * kStride] = o[y];
                }
            }
            if (live) {
                mine[D * kStride] = low;
                mine[(D + 1) * kStride] = sum;
            }
        }
        // the loads of O are done before the next piece's product overwrites it
        tc_fence_before();
        leave();
    }
}

template <int FMT, bool H, int D, bool TREE>
__global__ void __launch_bounds__(Chunk<FMT, H, D>::kThreads, 1)
    kv_chunk_kernel(const __grid_constant__ AttentionArgs a, const ChunkPlan* plan, ChunkSplit* splits,
                    const __grid_constant__ ChunkMaps maps) {
    using C = Chunk<FMT, H, D>;
    extern __shared__ __align__(1024) uint8_t smem_chunk[];  // the swizzle goes by address bits below 1024
    auto& sh = *reinterpret_cast<typename C::Shared*>(smem_chunk);
    const uint32_t warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sh.kv_full[i], C::kTma ? 1 : 4);
        }
        for (int i = 0; i < C::kDepth; ++i) mbar_init(&sh.freed[i], 1);
        for (int g = 0; g < 2; ++g) {
            mbar_init(&sh.q_full[g], 4);
            mbar_init(&sh.s_full[g], 1);
            mbar_init(&sh.p_full[g], 4);
            mbar_init(&sh.o_full[g], 1);
        }
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], 8 + (C::kTma ? 1 : 4) + 1);  // warps of the softmax groups, loaders, products
        }
        mbar_init(&sh.noted, 128);
        mbar_init(&sh.drained, 1);
        mbar_init_fence();
    }
    if (warp == C::kProductWarp) tmem_alloc(smem_u32(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    wait_predecessor();  // the plan is written, the status clear
    release_successor();
    bool ok = true, bad = false;
    // registers of the launch: 384 threads of 168, 2 * 216 + 72 = 3 * 168, or 512 of 128,
    // 2 * 200 + 72 + 40 = 4 * 128
    if (warp < 8) {
        if (C::kTma)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        softmax_role<FMT, H, D, TREE>(a, sh, tmem, ok);
    } else if (C::kTma || warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if constexpr (!C::kTma) load_role<FMT, H, D>(a, sh, ok, bad);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    }
    if constexpr (C::kTma) {
        if (warp == 8) load_tma_role<C>(a, sh, &maps.k, &maps.v, ok, bad);
    }
    if (warp == C::kProductWarp) product_role<FMT, H, D>(sh, tmem, ok);
    if (threadIdx.x == C::kSegmentWarp * 32u) segment_role<std::conditional_t<TREE, TreeWork, CausalWork>>(a, sh, plan, splits, ok);
    if (bad) report(a.status, SPLITZIP_ERR_INVALID_ARG);
    if (!ok) report(a.status, SPLITZIP_ERR_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == C::kProductWarp) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

// Joins the parts of the item that CTA blockIdx.x of the kernel above began, if
// others went on with it.  A CTA has 32 rows, a lane a row; eight warps share
// the columns and two of each take every other part, joined in that order.
// A kernel of its own, since the parts of a long context (for one sequence and
// 8 kv heads 19 of up to 132 KB an item) are then read by many SMs, and not by
// the one that wrote the last of them.
constexpr int kJoinParts = 2, kJoinColumns = 8, kJoinThreads = kJoinParts * kJoinColumns * 32;

template <bool H, int D, bool TREE, int BLOCKS>
__global__ void __launch_bounds__(kJoinThreads)
    kv_chunk_join_kernel(const __grid_constant__ AttentionArgs a, const ChunkSplit* splits, float value_scale,
                         float scale, float shift) {
    constexpr int kColumns = D / kJoinColumns, kStride = part_stride<TREE>();
    __shared__ float s_o[D][32], s_l[kJoinColumns][32];
    wait_predecessor();
    const uint32_t first = blockIdx.x, lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const int part0 = int(warp / kJoinColumns), col0 = int(warp % kJoinColumns) * kColumns;
    const ChunkSplit w = splits[first];
    if (int(blockIdx.y) * 32 >= w.rows) return;
    const int row = int(blockIdx.y * 32u + lane);  // those past the last read what is there, and write nothing
    float m = -INFINITY, l = 0.f;
#pragma unroll 8
    for (uint32_t cta = first; cta <= w.last_cta; ++cta) m = fmaxf(m, part_at<D, TREE>(a, cta, first, uint32_t(row), BLOCKS)[D * kStride]);
    float o[kColumns];
#pragma unroll
    for (int y = 0; y < kColumns; ++y) o[y] = 0.f;
#pragma unroll 2
    for (uint32_t cta = first + uint32_t(part0); cta <= w.last_cta; cta += kJoinParts) {
        const float* part = part_at<D, TREE>(a, cta, first, uint32_t(row), BLOCKS);
        float x[kColumns];
#pragma unroll
        for (int y = 0; y < kColumns; ++y) x[y] = part[(col0 + y) * kStride];
        // parts of no reference (a scale of about zero leaves it there) count as they are
        const float mc = part[D * kStride], e = exp2_fast((mc - m) * scale), f = mc == m ? 1.f : e;
        l += f * part[(D + 1) * kStride];
#pragma unroll
        for (int y = 0; y < kColumns; ++y) o[y] += f * x[y];
    }
    if (part0 == 1) {
#pragma unroll
        for (int y = 0; y < kColumns; ++y) s_o[col0 + y][lane] = o[y];
        s_l[warp % kJoinColumns][lane] = l;
    }
    __syncthreads();
    if (part0 != 0 || row >= w.rows) return;
#pragma unroll
    for (int y = 0; y < kColumns; ++y) o[y] += s_o[col0 + y][lane];
    l += s_l[warp][lane];
    const float inv = l == 0.f ? 0.f : 1.f / (value_scale * l);
    const int r = w.row_first + row, i = r / int(a.group);
    const uint32_t head = w.head * a.group + uint32_t(r - i * int(a.group));
    uint16_t* out = a.out.d + uint64_t(w.row0 + i) * a.out.token_stride + uint64_t(head) * a.out.head_stride + col0;
#pragma unroll
    for (int k = 0; k < kColumns / 8; ++k) {
        uint32_t z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = o[8 * k + 2 * e] * inv, y = o[8 * k + 2 * e + 1] * inv;
            z[e] = H ? pack_half2(x, y) : pack_bf16x2(x, y);
        }
        reinterpret_cast<uint4*>(out)[k] = make_uint4(z[0], z[1], z[2], z[3]);
    }
    if (a.lse && col0 == 0) a.lse[uint64_t(w.row0 + i) * a.q_heads + head] = log_sum(m, l, scale, shift);
}

// Of the kernel above on `ctas` CTAs, whose items have up to `rows` rows.
template <bool H, int D, bool TREE>
cudaError_t launch_join(const AttentionArgs& a, uint32_t ctas, int rows, const ChunkSplit* splits, float value_scale,
                        float scale, float shift, cudaStream_t s) {
    ChainedLaunch l(dim3(ctas, uint32_t(rows) / 32), dim3(kJoinThreads), 0, s);
    if constexpr (TREE) {
        if (a.part_blocks == 1) {
            l.cfg.gridDim.y = 1;
            return cudaLaunchKernelEx(&l.cfg, kv_chunk_join_kernel<H, D, true, 1>, a, splits, value_scale, scale, shift);
        }
    }
    return cudaLaunchKernelEx(&l.cfg, kv_chunk_join_kernel<H, D, TREE, kRows / part_stride<TREE>()>, a, splits, value_scale,
                              scale, shift);
}

uint64_t plan_bytes(uint32_t ctas) { return sizeof(ChunkPlan) + uint64_t(ctas) * sizeof(ChunkStart); }

template <int FMT, bool H, int D, bool TREE>
int launch(const AttentionArgs& a, ChunkPlan* plan, const ChunkMaps& maps, uint32_t ctas, cudaStream_t s) {
    using C = Chunk<FMT, H, D>;
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SPLITZIP_ERR_CUDA;
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        if (cudaFuncSetAttribute(kv_chunk_kernel<FMT, H, D, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
            cudaSuccess) {
            cudaGetLastError();
            return SPLITZIP_ERR_CUDA;
        }
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    ChainedLaunch l(dim3(ctas), dim3(C::kThreads), C::kSmem, s);
    ChunkSplit* splits = reinterpret_cast<ChunkSplit*>(reinterpret_cast<uint8_t*>(plan) + plan_bytes(ctas));
    if (cudaLaunchKernelEx(&l.cfg, kv_chunk_kernel<FMT, H, D, TREE>, a, static_cast<const ChunkPlan*>(plan), splits, maps) !=
            cudaSuccess ||
        launch_join<H, D, TREE>(a, ctas, kRows, splits, C::kValueScale, a.scale_log2, C::kShift, s) != cudaSuccess) {
        cudaGetLastError();
        return SPLITZIP_ERR_CUDA;
    }
    return SPLITZIP_OK;
}

template <int FMT, bool TREE>
int launch_type(const AttentionArgs& a, bool half, ChunkPlan* plan, const ChunkMaps& maps, uint32_t ctas,
                cudaStream_t s) {
    if (a.c.head_dim == 128)
        return half ? launch<FMT, true, 128, TREE>(a, plan, maps, ctas, s) : launch<FMT, false, 128, TREE>(a, plan, maps, ctas, s);
    return half ? launch<FMT, true, 64, TREE>(a, plan, maps, ctas, s) : launch<FMT, false, 64, TREE>(a, plan, maps, ctas, s);
}

// Maps of the pools for boxes of 64 columns and up to 128 tokens of one head
// and page; false where the driver takes no such strides.
bool make_maps(const AttentionArgs& a, ChunkMaps* m) {
    const uint64_t dims[4] = {a.c.head_dim, a.c.kv_heads, uint64_t(1) << a.c.page_shift, a.c.pool_pages};
    const uint64_t strides[3] = {a.c.head_stride, a.c.token_stride, a.c.page_stride};
    const uint32_t box[4] = {64, 1, std::min<uint32_t>(1u << a.c.page_shift, kUnit), 1};
    return make_rows_map(a.c.k, 4, dims, strides, box, &m->k) && make_rows_map(a.c.v, 4, dims, strides, box, &m->v);
}

template <bool TREE>
int launch_chunk(const AttentionArgs& a, bool q_half, void* plan_at, uint32_t ctas, cudaStream_t s) {
    ChunkPlan* plan = static_cast<ChunkPlan*>(plan_at);
    kv_chunk_plan_kernel<std::conditional_t<TREE, TreeWork, CausalWork>><<<1, kPlanThreads, 0, s>>>(a, plan, ctas);
    if (cudaGetLastError() != cudaSuccess) return SPLITZIP_ERR_CUDA;
    ChunkMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    if (a.c.type == SPLITZIP_KV_FP8_E5M2) return launch_type<1, TREE>(a, q_half, plan, maps, ctas, s);
    if (a.c.type == SPLITZIP_KV_FP8_E4M3) return launch_type<2, TREE>(a, q_half, plan, maps, ctas, s);
    // By tensor maps where the pages allow it: a box's rows have to be whole groups of
    // eight for the swizzle.  2,048 tokens over 32,768 in pages of 16 took 835 us so, and
    // 1,104 with every row copied by the loaders' threads (in turn on one GPU).
    if (a.c.page_shift >= 3 && make_maps(a, &maps)) return launch_type<3, TREE>(a, q_half, plan, maps, ctas, s);
    return launch_type<0, TREE>(a, q_half, plan, maps, ctas, s);
}

}  // namespace
}  // namespace splitzip
