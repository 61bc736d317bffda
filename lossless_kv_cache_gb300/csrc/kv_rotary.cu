// Rotary positions of the new tokens' queries and keys, with the write of keys
// and values into the pages (splitzip_kv_rotary_write).
//
// Mathematics: pair j of a row at position p is turned by p f_j turns.  f_j is a
// fraction of 2^64, so that the low 64 bits of the integer product p f_j are the
// fraction of a turn, exactly, at any position (in 32-bit floats position
// 1,000,000 would be off by 0.03 rad and more).  The upper 24 bits, signed, go to
// sincospi, the next 24 are a small turn after it, to first order.  The quantised
// write is kv_rw.cu's, of the 32-bit rotated row: one rounding, of what the cache
// keeps.  (One key element in two million comes out on the other side of a tie, as
// with sines, cosines and products rounded to 32 bits one after another.  Elements
// near a tie made again in 64 bits cost 9 to 16 % of the time.)
//
// What bounds it: HBM, mostly the queries (in and out).  A warp takes a token and
// some of its heads, 32 / LPR at a time: head_dim / 16 lanes a row, sixteen
// elements a lane, dealt so that a lane has both elements of its eight pairs
// whatever the layout and however much of the head is rotated.  The sines and
// cosines of those pairs are made once and serve all the warp's heads, of
// queries and keys.  32,768 tokens (32 query heads of 128 over 8) into BF16 pages
// with neighbours turned take 128 us, 94 % of a copy's rate; into E5M2 134 us, 82 %,
// where the arithmetic of the rounding counts too.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"

namespace splitzip {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kAhead = 2;  // units of rows on their way (32,768 tokens into E5M2: 149 us with one, 134)
constexpr int kMinCtas = 6;

struct RotaryArgs {
    KvCache c;
    KvBatch b;
    KvRows q, q_out, k, v;
    const uint64_t* turns;
    const int32_t* position;
    float magnitude;
    uint32_t q_heads, rot;
    // Heads are taken 32 / LPR at a time: `row_units` times for V, as often for K, then for Q; `per_warp` of them
    // by a warp, `warps` warps a token.
    uint32_t row_units, units, per_warp, warps;
    int* status;
};

// Sixteen floats of a row, quantised; LPR lanes hold the row.  Whole warp.
template <bool E5M2, int LPR>
__device__ __forceinline__ void quantise16(const float (&x)[16], uint2 (&out)[2], uint32_t* scale) {
    // largest finite magnitude; as integers, since the maximum of floats drops NaN
    uint32_t most = 0;
    bool special = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t m = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        special |= m >= 0x7F800000u;
        most = max(most, m);
    }
    if (__any_sync(~0u, special)) {
        most = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t m = __float_as_uint(x[i]) & 0x7FFFFFFFu;
            most = max(most, m < 0x7F800000u ? m : 0u);
        }
    }
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) most = max(most, __shfl_xor_sync(~0u, most, d));
    int k = int(most >> 23) - 127 - (E5M2 ? 15 : 8) + ((most & 0x7FFFFFu) > 0x600000u);
    k = most == 0 ? 0 : max(k, -126);
    *scale = uint32_t(k + 127);
    const float inv = __uint_as_float(uint32_t(127 - k) << 23);
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(inv, inv));
        q[i] = float2_to_fp8x2<E5M2>(f.x, f.y);
    }
    if (special) {  // the conversion saturates infinities
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t bits = __float_as_uint(x[i]);
            if ((bits & 0x7FFFFFFFu) == 0x7F800000u) {
                const uint32_t at = 8u * (i & 1), byte = (E5M2 ? 0x7Cu : 0x7Fu) | (bits >> 24 & 0x80u);
                q[i / 2] = (q[i / 2] & ~(0xFFu << at)) | byte << at;
            }
        }
    }
    out[0] = make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
    out[1] = make_uint2(__byte_perm(q[4], q[5], 0x5410), __byte_perm(q[6], q[7], 0x5410));
}

// Of an angle of `turn` / 2^64 turns, times the magnitude.
__device__ __forceinline__ void sine_cosine(uint64_t turn, float magnitude, float* s, float* c) {
    float s0, c0;
    sincospif(float(int32_t(turn >> 32) & ~0xFF) * 0x1p-31f, &s0, &c0);
    const float rest = float(uint32_t(turn >> 16) & 0xFFFFFFu) * (3.14159265358979f * 0x1p-47f);
    *c = fmaf(-s0, rest, c0) * magnitude;
    *s = fmaf(c0, rest, s0) * magnitude;
}

// FMT 0: 16-bit cache, 1: E5M2, 2: E4M3.  H: rows in FP16, else BF16.  LPR lanes
// hold a row.  INTER: pairs of neighbours, else of the two halves.
template <int FMT, bool H, int LPR, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, kMinCtas) kv_rotary_kernel(const __grid_constant__ RotaryArgs a) {
    constexpr uint32_t kHeads = 32 / LPR;
    const uint32_t lane = threadIdx.x & 31u, col = lane % LPR, nth = lane / LPR;
    const uint64_t warp = uint64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const uint64_t token = warp / a.warps;
    const uint32_t unit0 = uint32_t(warp - token * a.warps) * a.per_warp;
    const uint32_t unit1 = min(unit0 + a.per_warp, a.units);
    // the lane's two pieces of eight elements: pairs (piece, piece rot / 16 after it) of the halves, or any
    const uint32_t turned = a.rot / 16;  // lanes that rotate
    const bool rotates = col < turned;
    const uint32_t piece0 = INTER || !rotates ? 2 * col : col, piece1 = INTER || !rotates ? 2 * col + 1 : col + turned;
    bool bad = false;
    if (token < a.b.tokens && unit0 < unit1) {
        // the unit's rows: side 0 V, 1 K, 2 Q; false where the lane has no head
        const auto row_of = [&](uint32_t unit, int* side, uint32_t* head) -> bool {
            *side = unit < a.row_units ? 0 : unit < 2 * a.row_units ? 1 : 2;
            *head = (unit - uint32_t(*side) * a.row_units) * kHeads + nth;
            return *head < (*side == 2 ? a.q_heads : a.c.kv_heads);
        };
        const auto load = [&](uint32_t unit, uint4 (&x)[2]) {
            int side;
            uint32_t head;
            x[0] = x[1] = make_uint4(0, 0, 0, 0);
            if (unit < unit1 && row_of(unit, &side, &head)) {
                const KvRows& r = side == 0 ? a.v : side == 1 ? a.k : a.q;
                const uint4* from = reinterpret_cast<const uint4*>(r.d + token * r.token_stride + head * r.head_stride);
                x[0] = __ldcs(from + piece0);
                x[1] = __ldcs(from + piece1);
            }
        };
        // kAhead units on their way
        uint4 x[kAhead][2];
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) load(unit0 + i, x[i]);
        const KvPlace p = find_place(a.c, a.b, int(token), lane);
        bad = p.bad;
        if (p.mine && !(p.bad && unit1 <= 2 * a.row_units)) {
            // cosines and sines of the lane's eight pairs, two to a register pair
            float2 cs[4], sn[4];
            if (unit1 > a.row_units) {
                // a lane makes those of kMade pairs of the token's, for the rows of the warp
                // turn by the same angles
                constexpr uint32_t kMade = LPR * 8 / 32;
                const int64_t pos = a.position ? a.position[token] : p.pos;
                float c[kMade], s[kMade];
#pragma unroll
                for (uint32_t i = 0; i < kMade; ++i) {
                    c[i] = 1.f, s[i] = 0.f;
                    const uint32_t pair = lane * kMade + i;
                    if (2 * pair < a.rot) {
                        const uint64_t turn = __ldg(a.turns + pair) * uint64_t(pos);
                        sine_cosine(turn, a.magnitude, &s[i], &c[i]);
                    }
                }
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) {
                    const int from = int(col * (8 / kMade) + i / kMade);
                    (i & 1 ? cs[i / 2].y : cs[i / 2].x) = __shfl_sync(~0u, c[i % kMade], from);
                    (i & 1 ? sn[i / 2].y : sn[i / 2].x) = __shfl_sync(~0u, s[i % kMade], from);
                }
            }
#pragma unroll 1
            for (uint32_t base = unit0; base < unit1; base += kAhead)
#pragma unroll
            for (uint32_t slot = 0; slot < kAhead; ++slot) {
                const uint32_t unit = base + slot;
                if (unit >= unit1) break;
                const uint4 now[2] = {x[slot][0], x[slot][1]};
                load(unit + kAhead, x[slot]);
                int side;
                uint32_t head;
                const bool there = row_of(unit, &side, &head);
                const uint32_t w[8] = {now[0].x, now[0].y, now[0].z, now[0].w, now[1].x, now[1].y, now[1].z, now[1].w};
                float f[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 y = unpack16<H>(w[i]);
                    f[2 * i] = y.x, f[2 * i + 1] = y.y;
                }
                if (side != 0 && rotates) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (INTER) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float &e = f[4 * i + 2 * h], &o = f[4 * i + 2 * h + 1];
                                const float ch = h ? cs[i].y : cs[i].x, sh = h ? sn[i].y : sn[i].x;
                                const float t = e * ch - o * sh;
                                o = e * sh + o * ch;
                                e = t;
                            }
                        } else {
                            const float2 e = make_float2(f[2 * i], f[2 * i + 1]);
                            const float2 o = make_float2(f[2 * i + 8], f[2 * i + 9]);
                            const float2 t = fma2(e, cs[i], mul2(o, make_float2(-sn[i].x, -sn[i].y)));
                            const float2 z = fma2(e, sn[i], mul2(o, cs[i]));
                            f[2 * i] = t.x, f[2 * i + 1] = t.y;
                            f[2 * i + 8] = z.x, f[2 * i + 9] = z.y;
                        }
                    }
                }
                if (side == 2 || FMT == 0) {
                    uint4 y[2];
                    if (side == 0 || !rotates) {
                        y[0] = now[0], y[1] = now[1];  // as they are, NaN included
                    } else {
                        uint32_t z[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i] = pack16<H>(f[2 * i], f[2 * i + 1]);
                        y[0] = make_uint4(z[0], z[1], z[2], z[3]);
                        y[1] = make_uint4(z[4], z[5], z[6], z[7]);
                    }
                    if (side == 2) {
                        if (there) {
                            uint4* to = reinterpret_cast<uint4*>(a.q_out.d + token * a.q_out.token_stride +
                                                                 head * a.q_out.head_stride);
                            __stcs(to + piece0, y[0]);
                            __stcs(to + piece1, y[1]);
                        }
                    } else if (there && p.placed) {
                        uint4* to = reinterpret_cast<uint4*>((side ? a.c.k : a.c.v) + p.page * a.c.page_stride +
                                                             uint64_t(p.slot) * a.c.token_stride + head * a.c.head_stride);
                        to[piece0] = y[0];
                        to[piece1] = y[1];
                    }
                } else {
                    uint2 y[2];
                    uint32_t scale;
                    quantise16<FMT == 1, LPR>(f, y, &scale);
                    if (there && p.placed) {
                        uint2* to = reinterpret_cast<uint2*>((side ? a.c.k : a.c.v) + p.page * a.c.page_stride +
                                                             uint64_t(p.slot) * a.c.token_stride + head * a.c.head_stride);
                        to[piece0] = y[0];
                        to[piece1] = y[1];
                        if (col == 0)
                            (side ? a.c.k_scale : a.c.v_scale)[((p.page * a.c.kv_heads + head) << a.c.page_shift) +
                                                               p.slot] = uint8_t(scale);
                    }
                }
            }
        }
    }
    wait_predecessor();  // the status word has been cleared
    if (bad && lane == 0) report(a.status, SPLITZIP_ERR_INVALID_ARG);
}

// Heads that a warp takes for one set of sines and cosines, in units of 32 / LPR:
// all of them where tokens alone fill the GPU, fewer where the step is small and
// its latency counts.  64 tokens into E5M2 take 4.4 us with a unit a warp and 8.7
// with all; 4,096 tokens 34.8 and 23.6.  At this many warps the middle is as near:
// 512 tokens 6.0 (7.4 and 10.8), 2,048 14.7 (18.5 and 14.2).
constexpr uint64_t kWarpsWanted = 152 * 32;

template <int FMT, bool H>
cudaError_t launch_rotary(RotaryArgs& a, bool interleaved, cudaStream_t s) {
    const uint32_t lpr = a.c.head_dim / 16, heads = 32 / lpr;
    a.row_units = (a.c.kv_heads + heads - 1) / heads;
    a.units = 2 * a.row_units + (a.q_heads + heads - 1) / heads;
    const uint64_t split = std::max<uint64_t>(1, kWarpsWanted / a.b.tokens);
    a.per_warp = split >= a.units ? 1 : (a.units + uint32_t(split) - 1) / uint32_t(split);
    a.warps = (a.units + a.per_warp - 1) / a.per_warp;
    const uint64_t grid = (uint64_t(a.b.tokens) * a.warps + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
    ChainedLaunch l(dim3(uint32_t(grid)), dim3(kWarps * 32), 0, s);
    if (lpr == 8)
        return interleaved ? cudaLaunchKernelEx(&l.cfg, kv_rotary_kernel<FMT, H, 8, true>, a)
                           : cudaLaunchKernelEx(&l.cfg, kv_rotary_kernel<FMT, H, 8, false>, a);
    return interleaved ? cudaLaunchKernelEx(&l.cfg, kv_rotary_kernel<FMT, H, 4, true>, a)
                       : cudaLaunchKernelEx(&l.cfg, kv_rotary_kernel<FMT, H, 4, false>, a);
}

}  // namespace
}  // namespace splitzip

using namespace splitzip;

extern "C" int splitzip_kv_rotary_write(const splitzip_kv_cache_t* cache, const splitzip_kv_batch_t* batch,
                                        const splitzip_kv_rotary_t* rotary, const splitzip_kv_rows_t* q,
                                        const splitzip_kv_rows_t* q_out, uint32_t q_heads, const splitzip_kv_rows_t* k,
                                        const splitzip_kv_rows_t* v, int dtype, int* d_status, cudaStream_t stream) {
    RotaryArgs a;
    int st = check_kv(cache, batch, &a.c, &a.b, true);
    if (st != SPLITZIP_OK) return st;
    if (!rotary || !d_status || (reinterpret_cast<uintptr_t>(d_status) & 3u) || !kv_dtype_fits(a.c.type, dtype))
        return SPLITZIP_ERR_INVALID_ARG;
    if ((st = check_rows(k, a.b, a.c.kv_heads, a.c.head_dim, &a.k)) != SPLITZIP_OK) return st;
    if ((st = check_rows(v, a.b, a.c.kv_heads, a.c.head_dim, &a.v)) != SPLITZIP_OK) return st;
    if (!q != !q_out) return SPLITZIP_ERR_INVALID_ARG;
    a.q_heads = 0;
    a.q = a.q_out = KvRows{};
    if (q) {
        if (q_heads == 0) return SPLITZIP_ERR_INVALID_ARG;
        if (q_heads > 65536u) return SPLITZIP_ERR_UNSUPPORTED;
        if ((st = check_rows(q, a.b, q_heads, a.c.head_dim, &a.q)) != SPLITZIP_OK) return st;
        if ((st = check_rows(q_out, a.b, q_heads, a.c.head_dim, &a.q_out)) != SPLITZIP_OK) return st;
        a.q_heads = q_heads;
    }
    if (rotary->rotary_dim == 0 || rotary->rotary_dim % 16u || rotary->rotary_dim > a.c.head_dim ||
        !std::isfinite(rotary->magnitude) || !rotary->d_turns || (reinterpret_cast<uintptr_t>(rotary->d_turns) & 7u) ||
        (reinterpret_cast<uintptr_t>(rotary->d_position) & 3u))
        return SPLITZIP_ERR_INVALID_ARG;
    a.turns = rotary->d_turns;
    a.position = rotary->d_position;
    a.magnitude = rotary->magnitude;
    a.rot = rotary->rotary_dim;
    a.status = d_status;
    int sms;
    if ((st = device_sms(&sms)) != SPLITZIP_OK) return st;
    cudaError_t e = launch_kv_begin(a.b, d_status, nullptr, 0, stream);
    if (e == cudaSuccess && a.b.tokens > 0) {
        const bool h = dtype == SPLITZIP_FP16, pairs = rotary->interleaved != 0;
        if (a.c.type == SPLITZIP_KV_FP8_E5M2)
            e = h ? launch_rotary<1, true>(a, pairs, stream) : launch_rotary<1, false>(a, pairs, stream);
        else if (a.c.type == SPLITZIP_KV_FP8_E4M3)
            e = h ? launch_rotary<2, true>(a, pairs, stream) : launch_rotary<2, false>(a, pairs, stream);
        else
            e = h ? launch_rotary<0, true>(a, pairs, stream) : launch_rotary<0, false>(a, pairs, stream);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? SPLITZIP_OK : SPLITZIP_ERR_CUDA;
}
