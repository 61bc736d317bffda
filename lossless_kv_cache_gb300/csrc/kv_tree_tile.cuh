// Attention of trees of up to 128 rows (drafted tokens by the query heads that
// share a kv head) a sequence over a paged cache, on the fifth-generation
// tensor cores.
//
// Mathematics: as in kv_chunk.cuh, with the scores of one tile of rows.  FP8
// values are multiplied in FP16.  A unit's keys hardly differ in their scales,
// so the converters bring K and V to the largest scale of the unit, 2^EK and 2^EV,
// which a row takes into the one factor of its scores and into its reference,
// the maximum of s + EV; its sums l are of 2^(s-ref).  FP16 holds what they make
// exactly (E5M2's elements are 2^-16 and more, 2^-22 with scales 2^kSpread apart).
// Where scales differ by more than 2^kSpread, EV from the piece's first by more
// than 2^30, or a row of V has the scale 2^0, which may be one of zeros, the keys
// keep scales of their own, as in kv_step.cuh: K's go to the scores, V's to the
// weights, and rows of zeros, whose scale says nothing of their size, count as
// e = -80 with the weight 0.  So no key takes precision from another.
//
// What bounds it: up to some 290 rows the bytes of the cache, so it is built to
// keep them coming.  A CTA's two softmax groups take every other unit of 128
// keys of the same rows, with sums of their own that are added up when the
// piece ends; a unit's softmax and products then run beside the next one's,
//   S(j+2) after P(j) V(j) | S(j+3) after P(j+1) V(j+1) | ...
// and K and V have rings of their own, K's ahead by a unit.
// (In kv_chunk.cuh the second group is a second tile of rows, which a tree
// does not have: its softmax, 3,300 cycles with its products, was all that ran.)
//   softmax    warps 0-3 even units, 4-7 odd ones; a thread is a row
//   copies     one warp, a box of a tensor map a lane (pages of eight tokens and
//              more): 16-bit K and V to where the products read them, FP8 to
//              staging buffers
//   scales     FP8: one warp looks up the keys' scales and makes the factors
//   converters FP8: eight warps, from the staging buffers to FP16 (for E5M2 a
//              permute of bytes and a product)
//   products   one warp; pieces one thread of another
// TMEM: S0, S1 (128 columns each, the weights overwrite the scores), O0, O1.
//
// Measured in a graph (32 query heads of 128 over 8, pages of 16): 32 trees of 16
// over 4,096 take 113 us over BF16 (4.9 TB/s, 73 % of a copy's rate) and 127 over
// E5M2 (kv_chunk.cuh's kernel with masks 210).  With 16 bits a unit takes about
// 1.3 us, which is HBM's; a CTA's first piece starts after 5 to 6 us, a piece's end
// costs 3 to 6.  With FP8 a unit takes 1.5 us, 2,900 cycles, half the bytes for
// nothing: a chain of conversion, scores, softmax and product in which neither the
// tensor pipe (24 %) nor the issue slots (40 %) nor shared memory is full.
// Roles stay small, with rolled loops and one place for each step: when their
// unrolled code did not fit the instruction caches together, every role was slow
// (262 us over E5M2).
//
// Every wait is bounded, as in kv_chunk.cuh.
#pragma once

#include "kv_chunk.cuh"

namespace splitzip {
namespace {

struct TileWork {
    static constexpr bool kTree = true;
    static constexpr int kTile = kTileRows;
    static constexpr int kCost = 5;  // what an item costs beside its keys, in units
};

// Up to so many sequences each CTA deals the units itself, a warp with a few
// sequences a lane, and no plan kernel runs before (16 trees of 16 tokens over 1,000
// 26.8 us and 28.9 with one, 120 of them 120.7 and 122.4).
constexpr uint32_t kPlanSequences = 128;

// The units of all items, and where this CTA's share of them starts (whole warp).
__device__ __forceinline__ uint64_t deal(const AttentionArgs& a, uint32_t* ctas, ChunkStart* start) {
    constexpr int kRounds = kPlanSequences / 32;
    const uint32_t lane = threadIdx.x & 31u;
    uint64_t mine[kRounds], units = 0;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const uint32_t b = uint32_t(i) * 32u + lane;
        mine[i] = 0;
        if (b < a.b.batch) {
            const KvSeq s = load_seq(a.b, b);
            if (s.t > 0) mine[i] = uint64_t(tile_of<TileWork>(a, s, 0).units + TileWork::kCost) * a.c.kv_heads;
        }
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) units += mine[i];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) units += __shfl_xor_sync(~0u, units, d);
    *ctas = uint32_t(min(uint64_t(gridDim.x), max(units, uint64_t(1))));
    *start = ChunkStart{0, 0, 0};
    if (blockIdx.x >= *ctas) return units;
    const uint64_t u = share_start(units, *ctas, blockIdx.x);
    uint64_t before = 0;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        uint64_t upto = mine[i];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(~0u, upto, d);
            if (int(lane) >= d) upto += y;
        }
        upto += before;
        const uint32_t holds = __ballot_sync(~0u, mine[i] > 0 && u >= upto - mine[i] && u < upto);
        if (holds) {
            const int src = __ffs(holds) - 1;
            *start = ChunkStart{uint32_t(i) * 32u + uint32_t(src), 0, __shfl_sync(~0u, upto - mine[i], src)};
        }
        before = __shfl_sync(~0u, upto, 31);
    }
    return units;
}

// What the rows have to know of a unit's scales.
struct UnitScales {
    float k;   // 2^EK
    float e;   // EV
    int own;   // the keys keep scales of their own
};

// FMT 0: cache of the queries' 16-bit type (FP16 with H, else BF16), 1: E5M2,
// 2: E4M3.
template <int FMT, bool H, int D>
struct TreeTile {
    static constexpr bool kFp8 = FMT != 0;
    static constexpr bool kE5M2 = FMT == 1;
    static constexpr bool kHalf = kFp8 || H;               // products in FP16
    static constexpr float kShift = weight_shift<kHalf>();
    static constexpr int kBlockBytes = 128 * 128;          // 64 columns
    static constexpr int kHalves = D / 64;
    static constexpr int kTileBytes = kHalves * kBlockBytes;
    // Tiles of K and V: what fits beside the rows of Q.  What counts is how much is on
    // its way from memory, 50 KB and more an SM: 16-bit tiles, or FP8 ones as they come,
    // and then as few converted ones as the products can do with.
    static constexpr int kKeys = kFp8 ? 2 : 98304 / kTileBytes, kValues = kFp8 ? 3 - kHalves : kKeys;
    // Barriers of V's tiles, two and more even for one tile: a group that looks at V before its
    // product is asked for knows that the tile two units before was there, and with one barrier
    // would take that tile's phase for its own.
    static constexpr int kValueBars = kValues > 1 ? kValues : 2;
    static constexpr int kConverters = kFp8 ? 8 : 0;       // warps
    static constexpr int kThreads = kFp8 ? 640 : 384;
    static constexpr uint32_t kProductWarp = 8 + kConverters, kSegmentWarp = kProductWarp + 1,
                              kCopyWarp = kProductWarp + 2, kScaleWarp = kProductWarp + 3;
    // FP8 tiles as they come: on their way, or being converted
    static constexpr int kRawBytes = 128 * D, kRaw = kFp8 ? (D == 128 ? 5 : 12) : 0;
    static constexpr int kChunks = D / 16;                 // their 16-byte pieces of a row
    static constexpr uint32_t kFactors = 4;                // slots of the keys' factors, a unit each
    static constexpr int kScaleUnits = 6;                  // units whose scales are on their way
    static constexpr int kSpread = 6;             // scales of a unit that are brought to the largest
    static constexpr int kRoom = kFp8 && !kE5M2 ? 7 : 0;  // E4M3's largest times 2^7 is in FP16's range

    struct Shared {
        uint8_t q[kTileBytes];
        uint8_t k[kKeys][kTileBytes];
        uint8_t v[kValues][kTileBytes];
        uint8_t raw[kFp8 ? kRaw : 1][kFp8 ? kRawBytes : 128];
        alignas(16) uint8_t raw_scale[kFp8 ? 8 : 1][2][kFp8 ? kUnit : 16];  // of K and V, 0: not there
        // of a unit's keys: what K and V are multiplied by as they are converted, 0: not there
        uint32_t k_times[kFp8 ? kFactors : 1][kFp8 ? kUnit : 1], v_times[kFp8 ? kFactors : 1][kFp8 ? kUnit : 1];
        // and where they keep scales of their own: K's, V's, and the exponents of V's
        float k_scale[kFp8 ? kFactors : 1][kFp8 ? kUnit : 1];
        float v_scale[kFp8 ? kFactors : 1][kFp8 ? kUnit : 1];
        float v_exp[kFp8 ? kFactors : 1][kFp8 ? kUnit : 1];
        UnitScales scales[kFp8 ? kFactors : 1];
        float2 group_ml[2][kTileRows];              // the groups' references and sums
        float row_scale[kFp8 ? kTileRows : 1];
        uint64_t k_full[kKeys], k_freed[kKeys], v_full[kValueBars], v_freed[kValues];
        uint64_t raw_full[kFp8 ? kRaw : 1], raw_freed[kFp8 ? kRaw : 1];
        uint64_t scale_full[kFp8 ? kFactors : 1], scale_freed[kFp8 ? kFactors : 1];
        uint64_t q_full, s_full[2], p_full[2], o_full[2], drained;
        uint64_t seg_full[kSegments], seg_empty[kSegments];
        uint32_t tmem;
        Segment seg[kSegments];
    };
    static constexpr int kSmem = int(sizeof(Shared));
    // warps that read a piece's description: softmax, converters, products, copies, scales
    static constexpr int kReaders = 8 + kConverters + 1 + 1 + (kFp8 ? 1 : 0);

    // Waits until slot u % N of a ring of N can be overwritten for the u-th time.
    template <uint32_t N>
    static __device__ __forceinline__ bool await(uint64_t* freed, uint32_t u) {
        return u < N || mbar_wait(&freed[u % N], (u / N - 1) & 1u);
    }
};

// One warp, a lane a box of up to 128 tokens: 64 columns of 16 bits, or whole
// rows of FP8.  Boxes that hold nothing an item sees lie past the last page,
// which reads as zeros.
template <class C>
__device__ __forceinline__ void copy_role(const AttentionArgs& a, typename C::Shared& sh, const CUtensorMap* k_map,
                                          const CUtensorMap* v_map, bool& ok, bool& bad) {
    constexpr uint32_t kBlocks = C::kFp8 ? 1 : C::kHalves;  // boxes beside one another
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t page_tokens = 1u << a.c.page_shift, box = min(page_tokens, uint32_t(kUnit));
    const uint32_t half = lane % kBlocks, nth = lane / kBlocks;  // of the lane's box: column block, box of the unit
    const bool mine = nth < kUnit / box;
    uint32_t unit = 0, issued[2] = {0, 0}, tiles = 0;  // units of the share; tiles of K and V, and of both, asked for
    for (uint32_t piece = 0;; ++piece) {
        const Segment& w = sh.seg[piece % kSegments];
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = __all_sync(~0u, ok);
        if (!ok || w.n == 0) break;
        const int32_t* table = a.b.table + uint64_t(w.b) * a.b.table_stride;
        const int n = w.n, first_unit = w.first_unit, head = int(w.head);
        // Looked up two units before its use, looked at one: it is not waited for.
        const auto sees = [&](int j) {
            const int pos = (first_unit + j) * kUnit + int(nth * box);
            return mine && j < n && pos + int(box) > w.lo && pos < w.hi;
        };
        const auto look_up = [&](int j) -> int32_t {
            return sees(j) ? table[uint32_t((first_unit + j) * kUnit + int(nth * box)) >> a.c.page_shift] : -1;
        };
        const auto checked = [&](int j, int32_t pg) -> int32_t {
            const bool good = pg >= 0 && uint64_t(pg) < a.c.pool_pages;
            if (sees(j) && !good) bad = true;
            return good ? pg : int32_t(a.c.pool_pages);
        };
        const auto ask = [&](int j, int32_t page, int side) {
            const uint32_t u = unit + uint32_t(j), slot = C::kFp8 ? tiles % (C::kFp8 ? C::kRaw : 1) : u % C::kKeys;
            if constexpr (C::kFp8) {
                if (ok) ok = C::template await<C::kRaw>(sh.raw_freed, tiles);
            } else {
                if (ok) ok = C::template await<C::kKeys>(side ? sh.v_freed : sh.k_freed, u);
            }
            ok = __all_sync(~0u, ok);
            if (!ok) return;
            uint64_t* full = C::kFp8 ? &sh.raw_full[slot] : side ? &sh.v_full[slot] : &sh.k_full[slot];
            uint8_t* to = C::kFp8 ? sh.raw[slot] + nth * box * (C::kRawBytes / 128u)
                                  : (side ? sh.v[slot] : sh.k[slot]) + half * C::kBlockBytes + nth * box * 128u;
            issued[side] = u + 1;
            ++tiles;
            if (lane == 0) mbar_arrive_expect_tx(full, C::kFp8 ? C::kRawBytes : C::kTileBytes);
            __syncwarp();
            if (mine) {
                const int token = ((first_unit + j) * kUnit + int(nth * box)) & int(page_tokens - 1u);
                tensor_load_4d(to, side ? v_map : k_map, int(half * 64u), head, token, page, full);
            }
        };
        int32_t page = checked(0, look_up(0)), found = look_up(1);
        ask(0, page, 0);
        for (int j = 0; j < n; ++j) {
            const int32_t next = checked(j + 1, found);
            found = look_up(j + 2);
            if (j + 1 < n) ask(j + 1, next, 0);
            ask(j, page, 1);
            page = next;
        }
        unit += uint32_t(n);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[piece % kSegments]);
    }
    // no copy is in flight when the CTA ends
    if constexpr (C::kFp8) {
        for (uint32_t i = 0; i < uint32_t(C::kRaw) && i < tiles; ++i) {
            const uint32_t x = tiles - 1 - i;
            if (!mbar_wait(&sh.raw_full[x % C::kRaw], (x / C::kRaw) & 1u)) ok = false;
        }
    } else {
        for (int side = 0; side < 2; ++side)
            for (uint32_t i = 0; i < uint32_t(C::kKeys) && i < issued[side]; ++i) {
                const uint32_t u = issued[side] - 1 - i;
                if (!mbar_wait(side ? &sh.v_full[u % C::kKeys] : &sh.k_full[u % C::kKeys], (u / C::kKeys) & 1u)) ok = false;
            }
    }
}

// One warp, four keys a lane: the scales of a unit's keys and what K and V are
// multiplied by.
template <class C>
__device__ __forceinline__ void scale_role(const AttentionArgs& a, typename C::Shared& sh, bool& ok) {
    const uint32_t lane = threadIdx.x & 31u, slots = (1u << a.c.page_shift) - 1u;
    uint32_t unit = 0;  // of the share
    for (uint32_t piece = 0;; ++piece) {
        const Segment& w = sh.seg[piece % kSegments];
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = __all_sync(~0u, ok);
        if (!ok || w.n == 0) break;
        const int n = w.n, first_unit = w.first_unit, lo = w.lo, hi = w.hi;
        const uint32_t head = w.head;
        const int32_t* table = a.b.table + uint64_t(w.b) * a.b.table_stride;
        // Scales come by copies of up to sixteen bytes, a lane's of one page each, units
        // ahead (bytes of DRAM that no other copy brings along); a unit's pages are looked
        // up one before they are asked for.
        const uint32_t run = min(1u << a.c.page_shift, 16u), runs = kUnit / run;
        const uint32_t side = lane / runs, key0 = lane % runs * run;
        const uint8_t* scales = side ? a.c.v_scale : a.c.k_scale;
        const auto sees = [&](int j) {
            const int pos = (first_unit + j) * kUnit + int(key0);
            return side < 2 && j < n && pos + int(run) > lo && pos < hi;
        };
        const auto look_up = [&](int j) -> int32_t {
            return sees(j) ? table[uint32_t((first_unit + j) * kUnit + int(key0)) >> a.c.page_shift] : -1;
        };
        const auto ask = [&](int j, int32_t page) {
            const bool there = page >= 0 && uint64_t(page) < a.c.pool_pages;
            const uint32_t slot = (uint32_t(first_unit + j) * kUnit + key0) & slots;
            const uint8_t* from =
                there ? scales + ((uint64_t(uint32_t(page)) * a.c.kv_heads + head) << a.c.page_shift) + slot : a.c.k_scale;
            if (side < 2 && j < n) {
                const uint32_t to = smem_u32(&sh.raw_scale[(unit + uint32_t(j)) % 8u][side][key0]);
                if (run == 16)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0)
                                 : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(there ? 8 : 0)
                                 : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int v_first = 127;
#pragma unroll 1
        for (int j = 0; j < C::kScaleUnits; ++j) ask(j, look_up(j));
        int32_t found = look_up(C::kScaleUnits);
        const uint32_t unit0 = unit;
        for (int j = 0; j < n; ++j) {
            const uint32_t u = unit0 + uint32_t(j), at = u % C::kFactors;
            ask(j + C::kScaleUnits, found);
            found = look_up(j + C::kScaleUnits + 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kScaleUnits) : "memory");
            __syncwarp();
            uint32_t k_now[4], v_now[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pos = (first_unit + j) * kUnit + 32 * i + int(lane);
                const bool in = pos >= lo && pos < hi;
                k_now[i] = in ? sh.raw_scale[u % 8u][0][32 * i + int(lane)] : 0u;
                v_now[i] = in ? sh.raw_scale[u % 8u][1][32 * i + int(lane)] : 0u;
            }
            // Of the keys that are there; rows of V with the scale 2^0, kv_write's for rows of zeros, count
            // as 2^-126, for they may have nothing of the size that it says.
            uint32_t most[2] = {0, 0}, least[2] = {~0u, ~0u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                most[0] = max(most[0], k_now[i]);
                most[1] = max(most[1], v_now[i]);
                least[0] = min(least[0], k_now[i] - 1u);
                least[1] = min(least[1], v_now[i] == 127u ? 0u : v_now[i] - 1u);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                most[i] = __reduce_max_sync(~0u, most[i]);
                least[i] = __reduce_min_sync(~0u, least[i]) + 1u;
                if (most[i] == 0) most[i] = least[i] = 127;
            }
            const int v_most = int(most[1]);
            if (j == 0) v_first = v_most;
            // a slot that nothing was written to may hold 255
            const bool own = most[0] > 254u || int(most[0] - least[0]) > C::kSpread ||
                             int(most[1] - least[1]) > C::kSpread || least[1] < 47u || most[1] > 237u ||
                             abs(v_most - v_first) > 30;
            if (ok) ok = C::template await<C::kFactors>(sh.scale_freed, u);
            ok = __all_sync(~0u, ok);
            if (ok) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t key = 32u * uint32_t(i) + lane;
                    // FP16 powers of two
                    const auto times = [&](uint32_t scale, uint32_t top) -> uint32_t {
                        return scale ? (15u + C::kRoom + (own ? 0u : scale - top)) * 0x04000400u : 0u;
                    };
                    sh.k_times[at][key] = times(k_now[i], most[0]);
                    sh.v_times[at][key] = times(v_now[i], most[1]);
                }
                if (own) {
                    // Keys that are not there have no part in anything.  Apart from the loop above, which
                    // is then small (64 trees of 8 tokens over 2,000 E5M2 139.5 -> 137.1 us).
#pragma unroll 1
                    for (uint32_t key = lane; key < uint32_t(kUnit); key += 32) {
                        const uint32_t v = sh.raw_scale[u % 8u][1][key];
                        sh.k_scale[at][key] = scale_value(sh.raw_scale[u % 8u][0][key]);
                        sh.v_scale[at][key] = scale_value(min(v, 254u));  // 0 times infinity is NaN
                        // at least -80, which bounds the sums of 2^(s-ref)
                        sh.v_exp[at][key] = float(int(max(v, 47u)) - 127);
                    }
                }
                if (lane == 0) sh.scales[at] = UnitScales{scale_value(most[0]), float(v_most - 127), own};
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.scale_full[at]);
            }
        }
        unit += uint32_t(n);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[piece % kSegments]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Eight warps, a 16-byte piece of every kRowStep-th row of a tile each thread, K a
// unit ahead of V.
template <class C>
__device__ __forceinline__ void convert_role(typename C::Shared& sh, bool& ok) {
    const uint32_t lt = threadIdx.x - 256u, lane = lt & 31u;
    constexpr uint32_t kRowStep = 32 * C::kConverters / C::kChunks;
    // Of a tile, and at a time: with four the code is larger and the kernel slower (32 trees
    // of 32 tokens over 4,096 E4M3 137.6 us, 133.5 with two, 138.4 with one).
    constexpr int kPieces = 128 / int(kRowStep), kOnce = 2;
    const uint32_t c = lt % C::kChunks, r0 = lt / C::kChunks;
    // a row's lanes of the two column blocks in turns: every bank once
    const bool swap = c & 4u;
    const uint32_t to = (c >> 2) * C::kBlockBytes + r0 * 128u +
                        ((((2u * c + (swap ? 1u : 0u)) & 7u) ^ (r0 & 7u)) << 4);  // kRowStep is a multiple of eight
    const int other = int(to ^ 16u) - int(to);  // the second half of the piece's 32 bytes
    uint32_t tiles = 0, unit = 0;
    const auto convert = [&](uint32_t u, bool is_v) {
        const uint32_t x = tiles++, slot = x % C::kRaw, at = u % C::kFactors;
        if (ok) ok = mbar_wait(&sh.scale_full[at], (u / C::kFactors) & 1u);
        if (ok) ok = mbar_wait(&sh.raw_full[slot], (x / C::kRaw) & 1u);
        if (ok) ok = is_v ? C::template await<C::kValues>(sh.v_freed, u) : C::template await<C::kKeys>(sh.k_freed, u);
        ok = __all_sync(~0u, ok);
        if (!ok) return;
        const uint8_t* raw = sh.raw[slot] + lt * 16u;
        const uint32_t* times = (is_v ? sh.v_times[at] : sh.k_times[at]) + r0;
        uint8_t* row = (is_v ? sh.v[u % C::kValues] : sh.k[u % C::kKeys]) + to;
        const bool zeros = is_v && sh.scales[at].own;  // are looked for
#pragma unroll 1
        for (int i0 = 0; i0 < kPieces; i0 += kOnce) {
            uint4 y[kOnce];
            uint32_t f[kOnce];
#pragma unroll
            for (int i = 0; i < kOnce; ++i) {
                y[i] = *reinterpret_cast<const uint4*>(raw + i * int(512 * C::kConverters));
                f[i] = times[uint32_t(i) * kRowStep];
            }
            raw += kOnce * 512 * C::kConverters;
            times += kOnce * kRowStep;
#pragma unroll
            for (int i = 0; i < kOnce; ++i) {
                if (f[i] == 0) y[i] = make_uint4(0, 0, 0, 0);  // whatever is there: 0 times NaN is NaN
                const uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
                if (zeros) {
                    const uint32_t any = __ballot_sync(~0u, ((w[0] | w[1] | w[2] | w[3]) & 0x7F7F7F7Fu) != 0);
                    if (c == 0 && (any >> lane & ((1u << C::kChunks) - 1u)) == 0) {
                        sh.v_scale[at][r0 + uint32_t(i0 + i) * kRowStep] = 0.f;
                        sh.v_exp[at][r0 + uint32_t(i0 + i) * kRowStep] = -80.f;
                    }
                }
                const __half2 f2 = *reinterpret_cast<const __half2*>(&f[i]);
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t h = fp8_pair_to_half2<C::kE5M2>(w[k / 2], k & 1);
                    const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&h), f2);
                    o[k] = *reinterpret_cast<const uint32_t*>(&z);
                }
                const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
                *reinterpret_cast<uint4*>(row) = swap ? hi : lo;
                *reinterpret_cast<uint4*>(row + other) = swap ? lo : hi;
                row += kRowStep * 128u;
            }
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&sh.raw_freed[slot]);
            mbar_arrive(is_v ? &sh.v_full[u % C::kValueBars] : &sh.k_full[u % C::kKeys]);
            if (is_v) mbar_arrive(&sh.scale_freed[at]);  // which the softmax may be done with before
        }
    };
    for (uint32_t piece = 0;; ++piece) {
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = __all_sync(~0u, ok);
        const int n = ok ? sh.seg[piece % kSegments].n : 0;
        if (n == 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[piece % kSegments]);
        // K 0, K 1, V 0, K 2, V 1 .. V n - 1
#pragma unroll 1
        for (int i = 0; i <= 2 * n; ++i) {
            const bool is_v = i > 0 && !(i & 1);
            const int j = is_v ? i / 2 - 1 : (i + 1) / 2;
            if (j < n) convert(unit + uint32_t(j), is_v);
        }
        unit += uint32_t(n);
    }
}

// One warp, converged, whose elected lane issues.
template <class C, int D>
__device__ __forceinline__ void tile_product_role(typename C::Shared& sh, uint32_t tmem, bool& ok) {
    constexpr uint32_t kShapeS = tc_shape(!C::kHalf, 128, 128, false);
    constexpr uint32_t kShapeO = tc_shape(!C::kHalf, 128, D, true);
    constexpr uint32_t kTileStep = C::kTileBytes >> 4, kBlockStep = C::kBlockBytes >> 4;  // in the descriptors' units
    const uint64_t q_operand = smem_operand(smem_u32(sh.q), 16, 1024);
    const uint64_t k_operand = smem_operand(smem_u32(sh.k[0]), 16, 1024);
    const uint64_t v_operand = smem_operand(smem_u32(sh.v[0]), C::kBlockBytes, 1024);
    const bool leader = elect_lane();
    uint32_t weights[2] = {0, 0};
    uint32_t unit = 0;  // of the share
    for (uint32_t piece = 0;; ++piece) {
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = __all_sync(~0u, ok);
        const int n = ok ? sh.seg[piece % kSegments].n : 0;
        if (n == 0) break;
        __syncwarp();
        if (leader) mbar_arrive(&sh.seg_empty[piece % kSegments]);
        if (ok) ok = mbar_wait(&sh.q_full, piece & 1u);
        // P(j - 2) V(j - 2), then S(j), both group j mod 2's
#pragma unroll 1
        for (int j = 0; j < n + 2; ++j) {
            const uint32_t g = uint32_t(j) & 1u;
            if (j >= 2) {
                const uint32_t u = unit + uint32_t(j - 2), stage = u % C::kValues;
                if (ok) ok = mbar_wait(&sh.p_full[g], weights[g]++ & 1u);
                if (ok) ok = mbar_wait(&sh.v_full[u % C::kValueBars], (u / C::kValueBars) & 1u);
                tc_fence_after();
                const uint64_t v = v_operand + stage * kTileStep;
#pragma unroll
                for (int k = 0; k < kUnit / 16; ++k)
                    tc_mma_ta(leader && ok, tmem + 256u + g * 128u, tmem + g * 128u + uint32_t(k) * 8u,
                              v + uint32_t(k) * (2048u >> 4), kShapeO, k > 0 || j >= 4);
                if (leader && ok) {
                    tc_commit(&sh.v_freed[stage]);
                    if (j >= n) tc_commit(&sh.o_full[g]);
                }
            }
            if (j < n) {
                const uint32_t u = unit + uint32_t(j), stage = u % C::kKeys;
                if (ok) ok = mbar_wait(&sh.k_full[stage], (u / C::kKeys) & 1u);
                tc_fence_after();
                const uint64_t kk = k_operand + stage * kTileStep;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = uint32_t(k / 4) * kBlockStep + uint32_t(k % 4) * 2u;
                    tc_mma(leader && ok, tmem + g * 128u, q_operand + at, kk + at, kShapeS, k > 0);
                }
                if (leader && ok) {
                    tc_commit(&sh.s_full[g]);
                    tc_commit(&sh.k_freed[stage]);
                }
            }
        }
        unit += uint32_t(n);
    }
    // no product is in flight when the CTA gives its memory back
    if (leader) tc_commit(&sh.drained);
    __syncwarp();
    if (!mbar_wait(&sh.drained, 0)) ok = false;
}

template <int FMT, bool H, int D>
__device__ __forceinline__ void tile_softmax_role(const AttentionArgs& a, typename TreeTile<FMT, H, D>::Shared& sh,
                                                  uint32_t tmem, bool& ok) {
    using C = TreeTile<FMT, H, D>;
    const int g = int(threadIdx.x >> 7);
    const uint32_t row = threadIdx.x & 127u, lane = threadIdx.x & 31u;
    const uint32_t lanes = ((row >> 5) * 32u) << 16;
    const uint32_t s_at = tmem + lanes + uint32_t(g) * 128u, o_at = tmem + lanes + 256u;
    // what references are times in base 2
    const float scale = C::kFp8 ? 1.f : a.scale_log2, lag = C::kFp8 ? 8.f : a.lag;
    const bool out_half = C::kFp8 ? a.q_half != 0 : H;
    // A row of 16-bit elements is kLanes 16-byte pieces; a warp moves sixteen of the
    // tile's rows, kRowsOnce at a time, so that its accesses to memory are whole rows.
    constexpr uint32_t kLanes = D / 8, kRowsOnce = 32 / kLanes;
    constexpr int kMoves = 16 / int(kRowsOnce);
    const uint32_t piece_col = lane % kLanes, piece_row = lane / kLanes, row0 = (threadIdx.x >> 5) * 16u;
    const auto staged = [&](uint32_t r, uint32_t c) {
        return reinterpret_cast<uint4*>(sh.q + (c >> 3) * C::kBlockBytes + r * 128u + (((c & 7u) ^ (r & 7u)) << 4));
    };
    uint32_t scored = 0, base = 0;  // scores that the group has taken; units of the share before the piece
    uint32_t pieces[2] = {0, 0};    // pieces that each group has had units of
    const auto await = [&](uint64_t* bar, uint32_t count) {
        if (ok) ok = mbar_wait(bar, count & 1u);
        ok = __all_sync(~0u, ok);
        tc_fence_after();
    };
    for (uint32_t piece = 0;; ++piece) {
        const Segment& w = sh.seg[piece % kSegments];
        if (ok) ok = mbar_wait(&sh.seg_full[piece % kSegments], (piece / kSegments) & 1u);
        ok = named_barrier_and(4, 256, ok);  // both groups go on or neither
        if (!ok || w.n == 0) break;
        const int n = w.n, piece_lo = w.lo, piece_hi = w.hi;
        // where the row of the warp's sixteen that is the lane's (mod 16) lies, -1 where there is none
        const auto place = [&](const KvRows& rows) -> int64_t {
            const int nth = int(row0 + lane % 16u), r = w.row_first + nth;  // of the sequence
            if (nth >= w.rows) return -1;
            const int i = r / int(a.group);
            return int64_t(uint64_t(w.row0 + i) * rows.token_stride +
                           uint64_t(w.head * a.group + uint32_t(r - i * int(a.group))) * rows.head_stride);
        };
        const bool warp_live = int(row & ~31u) < w.rows;  // a warp of no rows leaves its lanes as they are
        KeyRange see{0, 0};        // what the row sees before the tree
        int plain_from, plain_to;  // units of which every row sees all keys
        int mask_row = -1;         // and where the bits of the new tokens that it sees are
        {
            const KvSeq seq{w.row0, w.t, w.held, true};
            const int i = (w.row_first + int(row)) / int(a.group);
            if (int(row) < w.rows) {
                see = visible_before(a, seq, i);
                if (w.held - w.t + i >= 0) mask_row = w.row0 + i;
            }
            const KeyRange each = visible_to_all_before(a, seq, (w.row_first + w.rows - 1) / int(a.group));
            plain_from = (each.lo + kUnit - 1) / kUnit - w.first_unit;
            plain_to = each.hi / kUnit - w.first_unit;
        }
        {
            // the rows of Q, zeros where there is none; a negative scale's sign goes to Q
            const uint32_t flip = a.negate ? 0x80008000u : 0u;
            const int64_t mine = place(a.q);
            uint4 x[kMoves];
#pragma unroll
            for (int k = 0; k < kMoves; ++k) {
                const int64_t at = __shfl_sync(~0u, mine, k * int(kRowsOnce) + int(piece_row));
                x[k] = at < 0 ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4*>(a.q.d + at)[piece_col];
            }
#pragma unroll
            for (int k = 0; k < kMoves; ++k) {
                const uint32_t r = row0 + uint32_t(k) * kRowsOnce + piece_row;
                uint32_t y[4] = {x[k].x ^ flip, x[k].y ^ flip, x[k].z ^ flip, x[k].w ^ flip};
                if (C::kFp8) {
                    float down = 1.f;
                    if (!a.q_half) {
                        // BF16 to FP16 by way of the power of two that brings the row's largest
                        // finite element to [2^14, 2^15)
                        uint32_t top = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t lo = y[e] & 0x7FFFu, hi = (y[e] >> 16) & 0x7FFFu;
                            top = max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                        }
#pragma unroll
                        for (uint32_t d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
                        const int up = min(126, 14 - (int(top >> 7) - 127));
                        const float f = __uint_as_float(uint32_t(127 + up) << 23);
                        down = __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v = bf16x2_to_float2(y[e]);
                            y[e] = pack_half2(v.x * f, v.y * f);
                        }
                    }
                    if (piece_col == 0) sh.row_scale[r] = a.scale_log2 * down * (1.f / (1 << C::kRoom));
                }
                *staged(r, piece_col) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full);
        }
        float row_scale = 1.f;
        if (C::kFp8) {
            ok = named_barrier_and(4, 256, ok);
            row_scale = sh.row_scale[row];
        }
        float low = -INFINITY;  // what exponentials are taken against, before the scale
        float sum = 0.f;
        Reached<D> reached;
        bool reaches = false, begun = false;
        for (int j = g; j < n; j += 2, begun = true) {
            const uint32_t u = base + uint32_t(j), stage = u % C::kValues, factors = u % C::kFactors;
            const int pos0 = (w.first_unit + j) * kUnit;
            const bool all_seen = j >= plain_from && j < plain_to;  // by every row
            float unit_scale = scale, unit_e = 0.f;
            bool own = false;
            if (C::kFp8) {
                // made before the scores, so the wait for those covers the reading
                await(&sh.scale_full[factors], u / C::kFactors);
                const UnitScales us = sh.scales[factors];
                own = us.own;
                unit_scale = fmaxf(row_scale * us.k, 1.17549435e-38f);
                unit_e = us.e;
            }
            await(&sh.s_full[g], scored++);
            float f = 1.f;  // what the sums so far are multiplied by
            // a bit for each of 32 keys from column c on that the row sees
            const auto sees = [&](int c) -> uint32_t {
                const int at = pos0 + c;
                uint32_t bits = 0;
                if (mask_row >= 0)
                    bits = mask_bits(a.mask + uint64_t(uint32_t(mask_row)) * a.words, a.words, at - (w.held - w.t));
                // the range's keys, and of the new tokens those that there are
                return (low_bits(see.hi - at) & ~low_bits(see.lo - at)) | (bits & low_bits(w.held - at));
            };
            // a new reference, and what it makes of the sums so far
            const auto refer = [&](float top) {
                const bool grew = top > low + lag;
                f = grew ? exp2_fast((low - top) * scale) : 1.f;
                if (grew) low = top;
                if (begun && __any_sync(~0u, grew)) {
                    // S(j) done means that the group's product before it is: o can be rescaled
#pragma unroll 1
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t o[16];
                        tmem_load16(o, o_at + uint32_t(g) * 128u + 16u * uint32_t(k));
                        tmem_wait_load();
                        tmem_loaded16(o);
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                        tmem_store16(o_at + uint32_t(g) * 128u + 16u * uint32_t(k), o);
                    }
                }
            };
            // 32 columns of the row
            const auto take = [&](int c, uint32_t (&x)[32]) {
                tmem_load32(x, s_at + uint32_t(c));
                tmem_wait_load();
                tmem_loaded32(x);
            };
            const auto put = [&](int c, const uint32_t (&x)[32]) {
                tmem_store16(s_at + uint32_t(c), x);
                tmem_store16(s_at + uint32_t(c + 16), x + 16);
                tmem_wait_store();
            };
            if (C::kFp8 && own) await(&sh.v_full[u % C::kValueBars], u / C::kValueBars);  // which rows of V are zeros is known
            if (warp_live) {
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < kUnit; c += 32) {
                    uint32_t x[32];
                    take(c, x);
                    if (C::kFp8 && own) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            x[k] = __float_as_uint(__uint_as_float(x[k]) * row_scale * sh.k_scale[factors][c + k]);
                    }
                    if (!all_seen) {
                        const uint32_t bits = sees(c);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(bits >> k & 1u)) x[k] = 0xFF800000u;
                    }
                    if (!all_seen || own) put(c, x);
                    if (C::kFp8 && own) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) m0 = fmaxf(m0, __uint_as_float(x[k]) + sh.v_exp[factors][c + k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            m0 = max3(m0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                            m1 = max3(m1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
                        }
                    }
                }
                const float top = fmaxf(m0, m1);
                refer(C::kFp8 && !own ? fmaf(top, unit_scale, unit_e) : top);
            }

            // A weight of 0 hides a finite value of V, not an infinity or a NaN: where
            // some row does not see all of this unit's keys, such values are noted for
            // the rows that see them and taken out of V.
            const int k0 = max(pos0, piece_lo), k1 = min(pos0 + kUnit, piece_hi);
            if (!all_seen && k0 < k1) {
                const bool outside = !C::kFp8 && (k0 > pos0 || k1 < pos0 + kUnit);
                // the same in all of the group's threads
                if (ok) ok = mbar_wait(&sh.v_full[u % C::kValueBars], (u / C::kValueBars) & 1u);
                uint8_t* v = sh.v[stage];
                constexpr uint32_t kInf = C::kHalf ? 0x7C00u : 0x7F80u;
                if (outside) {
                    // a page's tokens past the sequence's end came too
                    if ((pos0 + int(row) < k0 || pos0 + int(row) >= k1) && ok) {
                        for (int k = 0; k < D / 8; ++k)
                            *reinterpret_cast<uint4*>(v + (k >> 3) * C::kBlockBytes + row * 128u + (k & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_async_proxy();
                }
                uint32_t most = 0;
#pragma unroll 8
                for (int k = 0; k < C::kTileBytes / 2048; ++k) {
                    const int key = pos0 + int((uint32_t(k) * 16u + (row >> 3)) & 127u);  // 8 pieces a row
                    if (!C::kFp8 && (key < k0 || key >= k1)) continue;
                    const uint4 y = *reinterpret_cast<const uint4*>(v + (uint32_t(k) * 128u + row) * 16u);
                    most = __vmaxu2(most, __vmaxu2(__vmaxu2(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu),
                                                   __vmaxu2(y.z & 0x7FFF7FFFu, y.w & 0x7FFF7FFFu)));
                }
                const bool special = (most & 0xFFFFu) >= kInf || (most >> 16) >= kInf;
                if (named_barrier_popc(2 + uint32_t(g), 128, special) > 0) {
                    if (!reaches) reached = Reached<D>{};
                    reaches = true;
                    note_special<C::kHalf, D>(v, SeenBits{{sees(0), sees(32), sees(64), sees(96)}}, &reached);
                    ok = named_barrier_and(2 + uint32_t(g), 128, ok);  // all have noted them
                    if (ok) {
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
            if (warp_live) {
                // FP8: the weights are 2^EV times what the sum takes; where keys have scales
                // of their own, 2^e of each
                const float shift = own ? ref : ref + unit_e, by = own ? 1.f : unit_scale;
                const float2 ref2 = make_float2(shift, shift), scale2 = make_float2(by, by);
                float2 part[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
                for (int c = 0; c < kUnit; c += 32) {
                    uint32_t x[32], p[16];
                    take(c, x);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 z = fma2(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])),
                                              scale2, ref2);
                        const float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
                        part[k & 1] = add2(part[k & 1], e);
                        x[2 * k] = __float_as_uint(e.x), x[2 * k + 1] = __float_as_uint(e.y);
                    }
                    if (C::kFp8 && own) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            x[k] = __float_as_uint(__uint_as_float(x[k]) * sh.v_scale[factors][c + k]);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        p[k] = C::kHalf ? pack_half2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]))
                                        : pack_bf16x2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
                    tmem_store16(s_at + uint32_t(c / 2), p);  // over scores that have been taken
                }
                part[0] = add2(part[0], part[1]);
                const float all = part[0].x + part[0].y;
                sum = sum * f + (C::kFp8 && !own ? all * exp2_fast(-unit_e) : all);
            }
            tmem_wait_store();
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) {
                mbar_arrive(&sh.p_full[g]);
                if (C::kFp8) mbar_arrive(&sh.scale_freed[factors]);
            }
        }
        base += uint32_t(n);

        // The piece's sums: both groups' of the row, a half of the columns a group.
        if (n > g) {
            await(&sh.o_full[g], pieces[g]);
            if (__any_sync(~0u, reaches)) {
#pragma unroll 1
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t o[16];
                    tmem_load16(o, o_at + uint32_t(g) * 128u + 16u * uint32_t(k));
                    tmem_wait_load();
                    tmem_loaded16(o);
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const int at = 16 * k + y;
                        float z = __uint_as_float(o[y]);
                        if (reaches && (reached.plus[at >> 5] >> (at & 31) & 1u)) z += INFINITY;
                        if (reaches && (reached.minus[at >> 5] >> (at & 31) & 1u)) z += -INFINITY;
                        o[y] = __float_as_uint(z);
                    }
                    tmem_store16(o_at + uint32_t(g) * 128u + 16u * uint32_t(k), o);
                }
                tmem_wait_store();
                tc_fence_before();
            }
        }
        sh.group_ml[g][row] = make_float2(low, sum);
        ok = named_barrier_and(4, 256, ok);
        if (n > (g ^ 1)) await(&sh.o_full[g ^ 1], pieces[g ^ 1]);
        tc_fence_after();
        ++pieces[0];
        if (n > 1) ++pieces[1];
        const float2 ml0 = sh.group_ml[0][row], ml1 = sh.group_ml[1][row];
        const float m = fmaxf(ml0.x, ml1.x);
        // groups of no reference (a scale of about zero leaves it there) count as they are
        const float f0 = ml0.x == m ? 1.f : exp2_fast((ml0.x - m) * scale);
        const float f1 = ml1.x == m ? 1.f : exp2_fast((ml1.x - m) * scale);
        const float l = f0 * ml0.y + f1 * ml1.y;
        const uint32_t first = w.first_cta, last = w.last_cta;
        const bool whole = first == last, live = int(row) < w.rows;
        const float inv = l == 0.f ? 0.f : 1.f / (l * (1 << C::kRoom));
        constexpr int kStride = part_stride<true>();
        float* part = part_at<D, true>(a, blockIdx.x, first, row, a.part_blocks);
        // an infinity or NaN stays one whatever the factor
        const auto times = [](float o, float f) { return fabsf(o) < INFINITY ? o * f : o; };
#pragma unroll 1
        for (int col = g * (D / 2); col < (g + 1) * (D / 2); col += 16) {
            uint32_t o0[16], o1[16];
            tmem_load16(o0, o_at + uint32_t(col));
            if (n > 1) tmem_load16(o1, o_at + 128u + uint32_t(col));
            tmem_wait_load();
            tmem_loaded16(o0);
            if (n > 1) tmem_loaded16(o1);
            float o[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                o[y] = times(__uint_as_float(o0[y]), f0);
                if (n > 1) o[y] += times(__uint_as_float(o1[y]), f1);
            }
            if (whole) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float lo = o[8 * y + 2 * e] * inv, hi = o[8 * y + 2 * e + 1] * inv;
                        z[e] = out_half ? pack_half2(lo, hi) : pack_bf16x2(lo, hi);
                    }
                    *staged(row, uint32_t(col / 8 + y)) = make_uint4(z[0], z[1], z[2], z[3]);
                }
            } else if (live) {
#pragma unroll
                for (int y = 0; y < 16; ++y) part[(col + y) * kStride] = o[y];
            }
        }
        if (!whole && live && g == 0) {
            part[D * kStride] = m;
            part[(D + 1) * kStride] = l;
        }
        if (whole) {
            ok = named_barrier_and(4, 256, ok);
            const int64_t mine = place(a.out);
#pragma unroll
            for (int k = 0; k < kMoves; ++k) {
                const uint32_t r = row0 + uint32_t(k) * kRowsOnce + piece_row;
                const int64_t at = __shfl_sync(~0u, mine, k * int(kRowsOnce) + int(piece_row));
                if (at >= 0) reinterpret_cast<uint4*>(a.out.d + at)[piece_col] = *staged(r, piece_col);
            }
            if (a.lse && g == 0 && live) {
                const int r = w.row_first + int(row), i = r / int(a.group);
                a.lse[uint64_t(w.row0 + i) * a.q_heads + w.head * a.group + uint32_t(r - i * int(a.group))] =
                    log_sum(m, l, scale, C::kShift);
            }
        }
        // the loads of O are done before the next piece's product overwrites it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.seg_empty[piece % kSegments]);
    }
}

template <int FMT, bool H, int D>
__global__ void __launch_bounds__(TreeTile<FMT, H, D>::kThreads, 1)
    kv_tree_tile_kernel(const __grid_constant__ AttentionArgs a, const ChunkPlan* plan, ChunkSplit* splits,
                        const __grid_constant__ ChunkMaps maps) {
    using C = TreeTile<FMT, H, D>;
    extern __shared__ __align__(1024) uint8_t smem_chunk[];  // the swizzle goes by address bits below 1024
    auto& sh = *reinterpret_cast<typename C::Shared*>(smem_chunk);
    const uint32_t warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kKeys; ++i) {
            mbar_init(&sh.k_full[i], C::kFp8 ? C::kConverters : 1);
            mbar_init(&sh.k_freed[i], 1);
        }
        for (int i = 0; i < C::kValueBars; ++i) mbar_init(&sh.v_full[i], C::kFp8 ? C::kConverters : 1);
        for (int i = 0; i < C::kValues; ++i) mbar_init(&sh.v_freed[i], 1);
        for (int i = 0; i < C::kRaw; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_freed[i], C::kConverters);
        }
        for (uint32_t i = 0; C::kFp8 && i < C::kFactors; ++i) {
            mbar_init(&sh.scale_full[i], 1);
            mbar_init(&sh.scale_freed[i], 4 + C::kConverters);  // of the unit's softmax, and of its V
        }
        mbar_init(&sh.q_full, 8);
        for (int g = 0; g < 2; ++g) {
            mbar_init(&sh.s_full[g], 1);
            mbar_init(&sh.p_full[g], 4);
            mbar_init(&sh.o_full[g], 1);
        }
        for (int i = 0; i < kSegments; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.seg_empty[i], C::kReaders);
        }
        mbar_init(&sh.drained, 1);
        mbar_init_fence();
    }
    if (warp == C::kProductWarp) tmem_alloc(smem_u32(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (plan) wait_predecessor();  // the plan is written
    release_successor();
    bool ok = true, bad = false;
    // registers of the launch: 384 threads of 168, 2 * 216 + 72 = 3 * 168, or 640 of 96,
    // 2 * 136 + 2 * 64 + 56 < 5 * 96
    if (warp < 8) {
        if (C::kFp8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        tile_softmax_role<FMT, H, D>(a, sh, tmem, ok);
    } else if (warp < C::kProductWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if constexpr (C::kFp8) convert_role<C>(sh, ok);
    } else if (C::kFp8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }
    if (warp == C::kCopyWarp) copy_role<C>(a, sh, &maps.k, &maps.v, ok, bad);
    if constexpr (C::kFp8) {
        if (warp == C::kScaleWarp) scale_role<C>(a, sh, ok);
    }
    if (warp == C::kProductWarp) tile_product_role<C, D>(sh, tmem, ok);
    if (warp == C::kSegmentWarp) {
        if (plan) {
            if ((threadIdx.x & 31u) == 0) segment_role<TileWork>(a, sh, plan, splits, ok);
        } else {
            uint32_t ctas;
            ChunkStart start;
            const uint64_t units = deal(a, &ctas, &start);
            if ((threadIdx.x & 31u) == 0) walk_share<TileWork>(a, sh, units, ctas, start, splits, ok);
        }
    }
    wait_predecessor();  // the status is clear
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

// Maps of FP8 pools for boxes of whole rows of up to 128 tokens of one head and
// page; false where the driver takes no such strides.
bool make_byte_maps(const AttentionArgs& a, ChunkMaps* m) {
    const uint64_t dims[4] = {a.c.head_dim, a.c.kv_heads, uint64_t(1) << a.c.page_shift, a.c.pool_pages};
    const uint64_t strides[3] = {a.c.head_stride, a.c.token_stride, a.c.page_stride};
    const uint32_t box[4] = {a.c.head_dim, 1, std::min<uint32_t>(1u << a.c.page_shift, kUnit), 1};
    return make_rows_map(a.c.k, 4, dims, strides, box, &m->k, true) &&
           make_rows_map(a.c.v, 4, dims, strides, box, &m->v, true);
}

template <int FMT, bool H, int D>
int launch_tile(const AttentionArgs& a, ChunkPlan* plan_at, const ChunkMaps& maps, uint32_t ctas, cudaStream_t s) {
    using C = TreeTile<FMT, H, D>;
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SPLITZIP_ERR_CUDA;
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        if (cudaFuncSetAttribute(kv_tree_tile_kernel<FMT, H, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
            cudaSuccess) {
            cudaGetLastError();
            return SPLITZIP_ERR_CUDA;
        }
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    }
    ChainedLaunch l(dim3(ctas), dim3(C::kThreads), C::kSmem, s);
    ChunkSplit* splits = reinterpret_cast<ChunkSplit*>(reinterpret_cast<uint8_t*>(plan_at) + plan_bytes(ctas));
    const ChunkPlan* plan = a.b.batch <= kPlanSequences ? nullptr : plan_at;
    const bool out_half = C::kFp8 ? a.q_half != 0 : H;
    const float scale = C::kFp8 ? 1.f : a.scale_log2, value_scale = float(1 << C::kRoom), shift = C::kShift;
    cudaError_t e = cudaLaunchKernelEx(&l.cfg, kv_tree_tile_kernel<FMT, H, D>, a, plan, splits, maps);
    if (e == cudaSuccess)
        e = out_half ? launch_join<true, D, true>(a, ctas, kTileRows, splits, value_scale, scale, shift, s)
                     : launch_join<false, D, true>(a, ctas, kTileRows, splits, value_scale, scale, shift, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? int(SPLITZIP_OK) : int(SPLITZIP_ERR_CUDA);
}

}  // namespace
}  // namespace splitzip
