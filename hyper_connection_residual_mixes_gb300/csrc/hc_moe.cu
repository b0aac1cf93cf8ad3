// hc_moe.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels, for
// GB300.
//
//   y[t] = sum over t's chosen experts e of  p[t, e] D[e] (silu(G[e] x[t]) * U[e] x[t])
// with the choice and its weights p made from the router's logits or given.
//
// A few tokens leave nothing but the reading of the chosen experts' weights.  They go
// past each SM once, in 8-row pieces of 128 bytes a row, straight to the lane that
// multiplies them: a lane copies (cp.async) 16 bytes of one row into a place of its own,
// a step ahead, and reads them from there, so that nothing but its own copies ever
// holds a warp up.  The products run on mma.sync m16n8k16 with 16 rows of weights on one side
// and 8 tokens on the other: a lane's 16 bytes are its operand as they lie, since the order of k within a
// piece is free as long as both operands share it, and 8 tokens waste the least of a
// tile.  The fifth-generation tensor cores would want the tokens padded to 16 columns at the
// least and the weights in swizzled tiles that all warps wait for; the products are not
// what takes time.
//
// Every block makes the choice and the lists of entries by expert for itself (some 3 us with 64 experts;
// a launch of its own would cost as much and have to be waited for).  First kernel: the rows of all
// chosen experts' G and U are dealt out evenly to the SMs, a block's warps share the contraction,
// and the products meet in shared memory: a = p silu(g) u, fp32, to the workspace.
// Second kernel: each SM has some rows of the output and all experts' D for them; tiles of 8 entries
// go round by round past its warps, which share the contraction, and each token's sum is kept
// in shared memory, experts in ascending order.  It is launched early and has made its lists and
// asked for its first weights when the first kernel ends.
//
// Measured (64 experts, 6 a token, 5,120 -> 2,048, 8-bit weights, bf16 outputs), in us, and of 6,767 GB/s for
// the chosen experts' weights: 16 tokens 309 (0.77), one token 55 (0.50), 64 tokens 597 (0.50); with the activation as
// one fp16 number, 11 bits of it, 290, 53 and 570.  fp16 outputs 307 and 589.  8 tokens, 2 of 8 experts, 16-bit
// weights, 79 (0.85; as two bf16 numbers 77.6).  37 tokens, 3 of 13 experts, 1,072 -> 336, 16-bit weights: 43 (bf16),
// 42 (fp16), latency: what of it the choices, the rounds and the two starts are has not been measured.
#include <atomic>

#include <cuda.h>

#include "hc_fp8.cuh"
#include "hc_pieces.cuh"
#include "hc_sublayer.h"
#include "hc_types.cuh"

namespace hc {

namespace moe {

constexpr int kMaxTokens = 64, kMaxTop = 16, kMaxExperts = 1024, kMaxEntries = kMaxTokens * kMaxTop;
constexpr int kUpWarps = 16, kUpPairs = 4;  // pairs of row tiles (of G and of U) of a unit
constexpr int kDownWarps = 16, kDownPairs = 3;  // ... of a pass
constexpr int kUpRing = kUpPairs * 2 * kCell, kDownRing = kDownPairs * 2 * kCell;  // of a warp: the pieces of a step
constexpr int kLows = 32 * kDownWarps * 64;  // bytes of k_moe_down's second numbers of a step

struct Args {
    const void *x;
    int64_t xs;
    int T, d, experts, inner, top;
    const float *logits;
    int sigmoid, normalise;
    float scale;
    int32_t *ids;
    float *p;
    const uint8_t *up, *down;
    Fp8Scales up_scales, down_scales;
    float *a;   // [T * top][inner]
    void *y;
    int64_t ys;
};

// The choice of experts, in shared memory.  Entry t * top + j is token t's j-th choice.
struct Lists {
    float p[kMaxEntries];
    int16_t id[kMaxEntries];         // the entry's expert, -1 for none
    uint16_t rank[kMaxEntries];      // ... and how many of its entries come before this one
    uint16_t list[kMaxEntries];      // entries by expert
    uint16_t active[kMaxExperts];    // experts with entries, ascending
    uint16_t first[kMaxExperts + 1]; // of the i-th of these: its first place in `list`
    uint16_t tiles[kMaxExperts + 1]; // ... and the tiles of 8 entries of those before it
    uint16_t of_tile[kMaxEntries];   // of a tile of 8 entries: which of these
    uint8_t token[kMaxEntries];      // of a place in `list`: its token
    int count[kMaxExperts];
    int n;                           // how many experts have entries
};

// A number whose order as an unsigned integer is that of the floats; 0 for -infinity and NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // (the two zeros are equal)
    return v > -INFINITY ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// A warp chooses a token's experts: the `top` largest logits, of equal ones the first.  Up to 256 are kept
// in registers, of more the ones behind the last choice are looked for in memory again.
constexpr int kKept = 8;
__device__ __forceinline__ void choose(const Args &a, Lists &l, int t, int lane, bool write) {
    const float *const lg = a.logits + (int64_t)t * a.experts;
    const bool kept = a.experts <= 32 * kKept;
    uint32_t keys[kKept];
#pragma unroll
    for (int i = 0; i < kKept; ++i) keys[i] = kept && lane + 32 * i < a.experts ? order_key(__ldg(lg + lane + 32 * i)) : 0u;
    float sum = 0.0f, best = 0.0f;
    if (!a.normalise && !a.sigmoid) {  // of the softmax over all experts
        uint32_t most = 0;
        if (kept) {
#pragma unroll
            for (int i = 0; i < kKept; ++i) most = keys[i] > most ? keys[i] : most;
        } else {
            for (int i = lane; i < a.experts; i += 32) most = max(most, order_key(__ldg(lg + i)));
        }
        best = of_key(__reduce_max_sync(0xffffffffu, most));
        for (int i = lane; i < a.experts; i += 32) {
            const float v = __ldg(lg + i);
            if (order_key(v) != 0u) sum += v == best ? 1.0f : expf(v - best);
        }
        sum = warp_sum(sum);
    }
    uint32_t last = 0xffffffffu;
    int last_e = -1, mine_e = -1;
    float mine = 0.0f, chosen = 0.0f, from = 0.0f;
    for (int j = 0; j < a.top; ++j) {
        uint32_t key = 0;
        int e = 0x7fffffff;
        if (kept) {
#pragma unroll
            for (int i = 0; i < kKept; ++i)
                if (keys[i] > key) key = keys[i], e = lane + 32 * i;
        } else {
            for (int i = lane; i < a.experts; i += 32) {
                const uint32_t k = order_key(__ldg(lg + i));
                if ((k < last || (k == last && i > last_e)) && k > key) key = k, e = i;
            }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, key);
        e = (int)__reduce_min_sync(0xffffffffu, key == top ? (uint32_t)e : 0x7fffffffu);
        if (top == 0u) break;  // nothing is left
        last = top, last_e = e;
#pragma unroll
        for (int i = 0; i < kKept; ++i)
            if (e == lane + 32 * i) keys[i] = 0u;
        const float v = of_key(top);
        if (j == 0) best = v, from = a.normalise && v < -20.0f ? v : 0.0f;
        // (below -20 the sigmoid is e^v to 2^-28 of itself; divided by the sum its largest may be taken out,
        // and has to be: below -87 the exponentials leave the normal numbers)
        const float s = a.sigmoid ? v < -20.0f ? expf(v - from) : 1.0f / (1.0f + expf(-v)) : v == best ? 1.0f : expf(v - best);
        chosen += s;
        if (lane == j) mine = s, mine_e = e;
    }
    const float by = a.normalise ? chosen : a.sigmoid ? 1.0f : sum;
    if (lane < a.top) {  // (top is at most 16)
        const int at = t * a.top + lane;
        const float p = by > 0.0f ? mine / by * a.scale : 0.0f;
        l.id[at] = (int16_t)mine_e, l.p[at] = p;
        if (write && blockIdx.x == 0) {
            if (a.ids) a.ids[at] = mine_e;
            if (a.p) a.p[at] = p;
        }
    }
}

// All threads: the choice and the lists by expert.  `write`: in the first kernel, which gives the choice to the
// caller too.
__device__ __forceinline__ void route(const Args &a, Lists &l, bool write) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int entries = a.T * a.top;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) l.count[e] = 0;
    if (a.logits) {
        for (int t = warp; t < a.T; t += nw) choose(a, l, t, lane, write);
    } else {
        // given: a place that names no expert has none; of an expert named twice the first place
        // gets both weights
        for (int i = threadIdx.x; i < entries; i += blockDim.x) {
            const int e = __ldg(a.ids + i);
            l.p[i] = __ldg(a.p + i);
            l.id[i] = (int16_t)(e < 0 || e >= a.experts ? -1 : e);
        }
        __syncthreads();
        const auto again = [&](int i) {  // whether an earlier place of the token names the same expert
            bool is = false;
            for (int j = i / a.top * a.top; j < i; ++j) is |= l.id[j] == l.id[i];
            return is && l.id[i] >= 0;
        };
        float p[kMaxEntries / 256];
        uint32_t twice = 0;
#pragma unroll
        for (int k = 0; k < kMaxEntries / 256; ++k) {
            const int i = threadIdx.x + k * blockDim.x;
            p[k] = 0.0f;
            if (i >= entries) break;
            p[k] = l.p[i];
            if (again(i)) twice |= 1u << k;
            else
                for (int j = i + 1; j < (i / a.top + 1) * a.top; ++j)
                    if (l.id[j] == l.id[i]) p[k] += l.p[j];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMaxEntries / 256; ++k) {
            const int i = threadIdx.x + k * blockDim.x;
            if (i >= entries) break;
            l.p[i] = p[k];
            if (twice >> k & 1u) l.id[i] = -1;
        }
    }
    __syncthreads();
    if (warp == 0) {
        // an expert's entries in their order (all blocks have to agree on which tile of 8 has one)
        for (int i0 = 0; i0 < entries; i0 += 32) {
            const int i = i0 + lane, e = i < entries ? l.id[i] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e), before = same & ((1u << lane) - 1u);
            if (e >= 0) l.rank[i] = (uint16_t)(l.count[e] + __popc(before));
            __syncwarp();
            if (e >= 0 && before == 0u) l.count[e] += __popc(same);
            __syncwarp();
        }
        int n = 0, at = 0, tiles = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane, c = e < a.experts ? l.count[e] : 0;
            int before = c, m = (c + 7) / 8;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, before, o), v = __shfl_up_sync(0xffffffffu, m, o);
                if (lane >= o) before += u, m += v;
            }
            const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
            if (c > 0) {
                const int i = n + __popc(some & ((1u << lane) - 1u));
                l.active[i] = (uint16_t)e, l.first[i] = (uint16_t)(at + before - c), l.tiles[i] = (uint16_t)(tiles + m - (c + 7) / 8);
                l.count[e] = at + before - c;  // from here on: the first place in `list`
            }
            n += __popc(some);
            at += __shfl_sync(0xffffffffu, before, 31);
            tiles += __shfl_sync(0xffffffffu, m, 31);
        }
        if (lane == 0) l.n = n, l.first[n] = (uint16_t)at, l.tiles[n] = (uint16_t)tiles;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < entries; i += blockDim.x)
        if (l.id[i] >= 0) {
            const int at = l.count[l.id[i]] + l.rank[i];
            l.list[at] = (uint16_t)i, l.token[at] = (uint8_t)(i / a.top);
        }
    for (int i = threadIdx.x; i < l.n; i += blockDim.x)
        for (int t = l.tiles[i]; t < l.tiles[i + 1]; ++t) l.of_tile[t] = (uint16_t)i;
    __syncthreads();
}

// fp16 copies of a token's values over a piece carry an even power of two that brings the
// largest to [2^13, 2^15): 11 bits of each value, of small ones 2^-38 of the largest.  Of that
// largest: the power, and the root of what undoes it.  One root goes to the sums (0 or from 2^-33 to 2^31), the
// other to the weights' scales, so that both stay normal numbers for scales from 2^-63 to 2^70 and any
// token, from 2^-100 for tokens of 2^-38 and more.  (Undone in one product with the scales, tokens of 2^-100 and
// scales of 2^-34, whose result scales of 2^100 bring back, had lost all their bits.)
__device__ __forceinline__ float power_of(float amax, float &root) {
    int b = (int)(__float_as_uint(amax) >> 23) | 1;
    b = b < 15 ? 15 : b;
    root = __uint_as_float((uint32_t)((b - 141) / 2 + 127) << 23);
    return __uint_as_float((uint32_t)(268 - b) << 23);
}

// ------------------------------------------------------------ G and U
// A unit: up to 32 rows (four tiles of 8) of one expert's G and U, for up to 8 entries.  An expert's
// rows are dealt out by what they cost, its number of such tiles of entries; these follow
// one another for the same rows, whose weights then come from L2.
struct Unit {
    int i, m, lo, hi;  // the expert (in `active`), tile of entries, rows
    int last, end;     // of this block: the last expert and the end of its rows
    __device__ __forceinline__ int limit(const Args &a) const { return i == last ? end : a.inner; }
    // The place of the weighted row `at`: the expert, and its row.
    static __device__ __forceinline__ void place(const Args &a, const Lists &l, int64_t at, int &i, int &row) {
        const int tile = (int)(at / a.inner);
        if (tile >= l.tiles[l.n]) i = l.n, row = 0;
        else i = l.of_tile[tile], row = (int)((at - (int64_t)l.tiles[i] * a.inner) / (l.tiles[i + 1] - l.tiles[i]));
    }
    __device__ __forceinline__ bool chunk(const Args &a, int row) {  // the unit that begins with a row, if there is one
        while (i < last && row >= a.inner) ++i, row = 0;
        if (i > last || (i == last && row >= end)) return false;
        m = 0, lo = row, hi = (row & ~7) + 8 * kUpPairs;
        if (hi > limit(a)) hi = limit(a);
        return true;
    }
    __device__ __forceinline__ bool next(const Args &a, const Lists &l) {
        if (++m < l.tiles[i + 1] - l.tiles[i]) return true;
        return chunk(a, hi);
    }
};

// Steps: a unit's pieces, one of 128 bytes of every row at a time, go round the warps.
template <typename TX, bool kF8>
__global__ void __launch_bounds__(32 * kUpWarps, 1) k_moe_up(const Args a) {
    constexpr int kBytes = kF8 ? 1 : 2, W = kUpWarps, kSums = kUpPairs * 128;
    constexpr int kPairs = kPairsOf<kF8>;
    extern __shared__ __align__(128) uint8_t smem[];
    float *const red = reinterpret_cast<float *>(smem + W * kUpRing);  // [2][warp][pair][4][lane]
    Lists &l = *reinterpret_cast<Lists *>(red + 2 * W * kSums);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    route(a, l, true);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t all = (int64_t)l.tiles[l.n] * a.inner;
    if (all == 0) return;
    Unit u;
    int row0;
    Unit::place(a, l, all * (blockIdx.x + 1) / gridDim.x, u.last, u.end);
    Unit::place(a, l, all * blockIdx.x / gridDim.x, u.i, row0);
    if (!u.chunk(a, row0)) return;
    const int row_bytes = a.d * kBytes, pieces = (row_bytes + 127) / 128;
    const int64_t matrix = (int64_t)a.inner * row_bytes;  // G or U of an expert
    const auto begin = [&](int n) {  // the warp's first piece of the n-th unit
        return (warp + n * (W - pieces % W)) % W;
    };

    // copies run a step ahead
    Unit ahead = u;
    bool more = true;
    int au = 0, ak = warp;
    uint32_t rows = 0;                // which of the unit's pairs of tiles have this lane's row
    const uint8_t *lane_row = a.up;   // this lane's row of the first tile
    const auto aim = [&]() {
        const int base = ahead.lo & ~7;
        lane_row = a.up + (int64_t)l.active[ahead.i] * 2 * matrix + (int64_t)(base + g) * row_bytes + t4 * 16;
        rows = 0;
#pragma unroll
        for (int j = 0; j < kUpPairs; ++j) rows |= (uint32_t)(base + 8 * j + g >= ahead.lo && base + 8 * j + g < ahead.hi) << j;
    };
    const auto settle = [&]() {  // to the unit that has a piece for this warp
        while (more && ak >= pieces) {
            more = ahead.next(a, l);
            if (more) aim(), ak = begin(++au);
        }
        if (!more) rows = 0;
    };
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kUpRing + lane * 16);
    const int64_t tile_bytes = 8 * (int64_t)row_bytes;
    const auto fetch = [&](int j) {
        const uint32_t to = ring + (uint32_t)(j * 2 * kCell);
        const uint8_t *const p = lane_row + (int64_t)j * tile_bytes + ak * 128;
        const bool there = rows >> j & 1u, first_half = there && ak * 128 + t4 * 16 < row_bytes,
                   second_half = there && ak * 128 + t4 * 16 + 64 < row_bytes;
        load_piece(to, p, first_half, second_half);
        load_piece(to + kCell, p + matrix, first_half, second_half);
        cp_async_commit();
    };
    const int row_blocks = (a.inner + kFp8Block - 1) / kFp8Block, col_blocks = (a.d + kFp8Block - 1) / kFp8Block;
    // ... and so do the tokens' values (token lane / 4 of the tile) and the scales (lane 2 j + (0: G, 1: U):
    // of pair j)
    uint4 raw[kPairs / 4];
    float scale_next = 1.0f;
    const auto load_tokens = [&]() {
        if (!more) return;
        const int entry = l.first[ahead.i] + 8 * ahead.m + g, base = ahead.lo & ~7;
        const bool has = entry < l.first[ahead.i + 1];
        const TX *const x = static_cast<const TX *>(a.x) + (has ? (int64_t)l.token[entry] * a.xs : 0);
#pragma unroll
        for (int s = 0; s < kPairs / 4; ++s) {
            const int c = kF8 ? ak * 128 + (s >> 1) * 64 + t4 * 16 + (s & 1) * 8 : ak * 64 + s * 32 + t4 * 8;
            raw[s] = make_uint4(0, 0, 0, 0);
            if (has && c < a.d) raw[s] = __ldg(reinterpret_cast<const uint4 *>(x + c));
        }
        if (kF8 && lane < 2 * kUpPairs && base + 8 * (lane >> 1) < ahead.hi)
            scale_next = a.up_scales.at((((int64_t)l.active[ahead.i] * 2 + (lane & 1)) * row_blocks + (base + 8 * (lane >> 1)) / kFp8Block) * col_blocks + ak);
    };
    aim();
    settle();
    load_tokens();
#pragma unroll
    for (int j = 0; j < kUpPairs; ++j) fetch(j);
    ak += W;
    settle();

    int buf = 0, un = 0;
    do {
        const int entry0 = l.first[u.i] + 8 * u.m, end = l.first[u.i + 1];
        const int base = u.lo & ~7, tiles = (u.hi - base + 7) / 8;
        float acc[kUpPairs][4];
#pragma unroll
        for (int j = 0; j < kUpPairs; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][k] = 0.0f;
        for (int k = begin(un); k < pieces; k += W) {
            uint32_t tok[kPairs];
            float root[2] = {1.0f, 1.0f};
            const float scale = scale_next;
#pragma unroll
            for (int s = 0; s < kPairs / 4; ++s) tok[4 * s] = raw[s].x, tok[4 * s + 1] = raw[s].y, tok[4 * s + 2] = raw[s].z, tok[4 * s + 3] = raw[s].w;
            if constexpr (kF8 && __is_same(TX, __nv_bfloat16)) {  // (the product with a power of two is exact in bf16)
                const auto pair_of = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
                __nv_bfloat162 top = __habs2(pair_of(tok[0]));
#pragma unroll
                for (int i = 1; i < kPairs; ++i) top = __hmax2(top, __habs2(pair_of(tok[i])));
                const float2 t = __bfloat1622float2(top);
                float amax = fmaxf(fmaxf(t.x, t.y), 0.0f), mine;
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const __nv_bfloat162 m = __float2bfloat162_rn(power_of(amax, mine));
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const __nv_bfloat162 p = __hmul2(pair_of(tok[i]), m);
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(&p);
                    tok[i] = half2_of(bf16lo(w), bf16hi(w));
                }
                root[0] = __shfl_sync(0xffffffffu, mine, 8 * t4), root[1] = __shfl_sync(0xffffffffu, mine, 8 * t4 + 4);
            }
            load_tokens();
#pragma unroll
            for (int j = 0; j < kUpPairs; ++j) {
                cp_async_wait<kUpPairs - 1>();
                const uint32_t here = ring + (uint32_t)(j * 2 * kCell);
                const Rows16<kF8> w(read_piece(here), read_piece(here + kCell));
                if (j < tiles) {
                    if constexpr (kF8) {
                        const float s0 = __shfl_sync(0xffffffffu, scale, 2 * j), s1 = __shfl_sync(0xffffffffu, scale, 2 * j + 1);
                        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        multiply<__half, true>(part, w, tok);
                        add_scaled(acc[j], part, s0, s1, root);
                    } else {
                        multiply<TX, false>(acc[j], w, tok);
                    }
                }
                fetch(j);
            }
            ak += W;
            settle();
        }
        // the warps' sums meet
        float *const sums = red + buf * W * kSums;
        if (begin(un) < pieces) {
#pragma unroll
            for (int j = 0; j < kUpPairs; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (j < tiles) sums[warp * kSums + (j * 4 + q) * 32 + lane] = acc[j][q];
        }
        __syncthreads();  // (two buffers: the next unit's sums are written while a slow warp still reads these)
        const int meet = pieces < W ? pieces : W, w0 = un * (pieces % W) % W;  // those that had a piece, in their order
        {
            const int j = threadIdx.x >> 6, q = threadIdx.x >> 5 & 1;
            const int row = base + 8 * j + g, entry = entry0 + 2 * t4 + q;
            if (j < tiles && row >= u.lo && row < u.hi && entry < end) {
                float gate = 0.0f, up = 0.0f;
                for (int i = 0, w = w0; i < meet; ++i) {
                    const float *const of_w = sums + w * kSums + (j * 4 + q) * 32 + lane;
                    gate += of_w[0], up += of_w[64];
                    if (++w == W) w = 0;
                }
                const int id = l.list[entry];
                a.a[(int64_t)id * a.inner + row] = gate / (1.0f + expf(-gate)) * up * l.p[id];
            }
        }
        ++un, buf ^= 1;
    } while (u.next(a, l));
    cp_async_wait<0>();
}

// ------------------------------------------------------------ D
// A block's rows of the output, in passes of kDownPairs pairs of tiles of 8 rows.  The tiles of 8
// entries follow one another in rounds: of a tile's contraction each warp has a piece, or several
// tiles share a round where pieces are few.  The warps' sums meet in shared memory, where each
// token's are added up expert by expert.
template <typename TX, bool kF8>
__global__ void __launch_bounds__(32 * kDownWarps, 1) k_moe_down(const Args a) {
    constexpr int kBytes = kF8 ? 1 : 2, W = kDownWarps, NP = kDownPairs, kPairs = kPairsOf<kF8>, kRows = 16 * NP;
    // a goes into the products as three bf16 numbers for bf16 weights (all 24 bits of it), else as two
    // fp16 numbers (22 bits)
    constexpr bool kBf16 = !kF8 && __is_same(TX, __nv_bfloat16);
    extern __shared__ __align__(128) uint8_t smem[];
    float *const red = reinterpret_cast<float *>(smem + W * kDownRing);  // [2][warp][pair][4][lane]
    float *const out = red + 2 * W * NP * 128;                           // [token][row]
    // The second numbers of a step of codes, [warp][4][lane], each read by the lane that wrote it: 16 registers
    // fewer, with which nothing spills (fp16, 16 tokens: 409 -> 337 us, with two chains of MMAs)
    uint4 *const lows = reinterpret_cast<uint4 *>(out + kMaxTokens * kRows) + (threadIdx.x & ~31u) * 4 + (threadIdx.x & 31u);
    Lists &l = *reinterpret_cast<Lists *>(out + kMaxTokens * kRows + (kF8 ? kLows / 4 : 0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    route(a, l, false);
    const int from = (int)((int64_t)a.d * blockIdx.x / gridDim.x), to = (int)((int64_t)a.d * (blockIdx.x + 1) / gridDim.x);
    const int row_bytes = a.inner * kBytes, pieces = (row_bytes + 127) / 128, all = l.tiles[l.n];
    const int row_blocks = (a.d + kFp8Block - 1) / kFp8Block, col_blocks = (a.inner + kFp8Block - 1) / kFp8Block;
    const int64_t matrix = (int64_t)a.d * row_bytes, tile_bytes = 8 * (int64_t)row_bytes;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kDownRing + lane * 16);
    // tiles of a round, this warp's among them and its first piece
    const int share = pieces <= W / 2 ? W / pieces : 1, mine = share > 1 ? warp / pieces : 0, k0 = share > 1 ? warp - mine * pieces : warp;
    const bool works = mine < share && k0 < pieces;
    bool waited = false;
    for (int base = from & ~7; base < to; base += kRows) {
        const int tiles = (to - base + 7) / 8 < 2 * NP ? (to - base + 7) / 8 : 2 * NP;
        uint32_t rows = 0;  // which tiles have this lane's row
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) rows |= (uint32_t)(base + 8 * i + g >= from && base + 8 * i + g < to) << i;
        for (int o = threadIdx.x; o < a.T * kRows; o += 32 * W) out[o] = 0.0f;
        // copies run a step ahead
        int ahead = works ? mine : all, ak = k0;
        uint32_t there = 0;
        const uint8_t *lane_row = a.down;
        const auto aim = [&]() {
            there = 0;
            if (ahead >= all) return;
            there = rows;
            lane_row = a.down + (int64_t)l.active[l.of_tile[ahead]] * matrix + (int64_t)(base + g) * row_bytes + ak * 128 + t4 * 16;
        };
        const auto fetch = [&](int j) {
            const uint32_t to_pair = ring + (uint32_t)(j * 2 * kCell);
            const bool first_half = ak * 128 + t4 * 16 < row_bytes, second_half = ak * 128 + t4 * 16 + 64 < row_bytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool is = there >> (2 * j + h) & 1u;
                load_piece(to_pair + h * kCell, lane_row + (2 * j + h) * tile_bytes, is && first_half, is && second_half);
            }
            cp_async_commit();
        };
        const auto advance = [&](int &tile, int &k) {  // this warp's next step
            k += W;
            if (k >= pieces) k = k0, tile += share;
        };
        aim();
#pragma unroll
        for (int j = 0; j < NP; ++j) fetch(j);
        advance(ahead, ak);
        aim();
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel's results are read from here on
        waited = true;
        // a step's activations (token lane / 4 of the tile) and scales (lane i: row tile i's), a step ahead too
        float4 raw[kPairs / 2];
        float scale_next = 1.0f;
        const auto load_tokens = [&](int tile, int k) {
            if (tile >= all) return;
            const int i = l.of_tile[tile], entry = l.first[i] + 8 * (tile - l.tiles[i]) + g;
            const bool has = entry < l.first[i + 1];
            const float *const p = a.a + (has ? (int64_t)l.list[entry] * a.inner : 0);
#pragma unroll
            for (int q = 0; q < kPairs / 2; ++q) {
                const int c = kF8 ? k * 128 + (q >> 2) * 64 + t4 * 16 + (q & 3) * 4 : k * 64 + (q >> 1) * 32 + t4 * 8 + (q & 1) * 4;
                raw[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (has && c < a.inner) raw[q] = __ldcg(reinterpret_cast<const float4 *>(p + c));
            }
            if (kF8 && lane < tiles) scale_next = a.down_scales.at(((int64_t)l.active[i] * row_blocks + (base + 8 * lane) / kFp8Block) * col_blocks + k);
        };
        int tile = works ? mine : all, k = k0, buf = 0;
        load_tokens(tile, k);
        for (int r0 = 0; r0 < all; r0 += share, buf ^= 1) {
            float *const sums = red + buf * W * NP * 128;
            if (tile < all) {
                float acc[NP][4];
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[j][q] = 0.0f;
                bool more = true;
                while (more) {
                    uint32_t tok[kPairs], low[kPairs], last[kBf16 ? kPairs : 1];
                    float root[2] = {1.0f, 1.0f};
                    const float *const f = reinterpret_cast<const float *>(raw);
                    if constexpr (kBf16) {  // (cut off after 8 bits each time, so that what is left is exact)
#pragma unroll
                        for (int q = 0; q < kPairs; ++q) {
                            tok[q] = cut_bf16x2(f[2 * q], f[2 * q + 1]);
                            const float a0 = f[2 * q] - bf16lo(tok[q]), a1 = f[2 * q + 1] - bf16hi(tok[q]);
                            low[q] = cut_bf16x2(a0, a1);
                            last[kBf16 ? q : 0] = cut_bf16x2(a0 - bf16lo(low[q]), a1 - bf16hi(low[q]));
                        }
                    } else {
                        float amax = 0.0f, own;
#pragma unroll
                        for (int q = 0; q < 2 * kPairs; ++q) amax = fmaxf(amax, fabsf(f[q]));
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                        const float m = power_of(amax, own);
#pragma unroll
                        for (int q = 0; q < kPairs; ++q) {
                            tok[q] = half2_of(f[2 * q] * m, f[2 * q + 1] * m);
                            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&tok[q]));
                            low[q] = half2_of(fmaf(f[2 * q], m, -h.x), fmaf(f[2 * q + 1], m, -h.y));
                        }
                        if constexpr (kF8) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) lows[32 * q] = make_uint4(low[4 * q], low[4 * q + 1], low[4 * q + 2], low[4 * q + 3]);
                        }
                        root[0] = __shfl_sync(0xffffffffu, own, 8 * t4), root[1] = __shfl_sync(0xffffffffu, own, 8 * t4 + 4);
                    }
                    const float scale = scale_next;
                    const int was = tile;
                    advance(tile, k);
                    load_tokens(tile, k);
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        cp_async_wait<NP - 1>();
                        if (2 * j < tiles) {
                            const uint32_t from_pair = ring + (uint32_t)(j * 2 * kCell);
                            const Rows16<kF8> w(read_piece(from_pair), read_piece(from_pair + kCell));
                            if constexpr (kBf16) {
                                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                multiply<TX, false>(part, w, last);
                                multiply_both<TX, false>(acc[j], w, tok, part, low);
#pragma unroll
                                for (int q = 0; q < 4; ++q) acc[j][q] += part[q];
                            } else {
                                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s0, s1;
                                if constexpr (kF8) {
                                    float more[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                                    for (int q = 0; q < 4; ++q) read16(low + 4 * q, smem_u32(lows + 32 * q));
                                    multiply_both<__half, kF8>(part, w, tok, more, low);
#pragma unroll
                                    for (int q = 0; q < 4; ++q) part[q] += more[q];
                                    s0 = __shfl_sync(0xffffffffu, scale, 2 * j), s1 = __shfl_sync(0xffffffffu, scale, 2 * j + 1);
                                } else {
                                    s0 = __shfl_sync(0xffffffffu, scale, 2 * j), s1 = __shfl_sync(0xffffffffu, scale, 2 * j + 1);
                                    multiply<__half, kF8>(part, w, low);
                                    multiply<__half, kF8>(part, w, tok);
                                }
                                add_scaled(acc[j], part, s0, s1, root);
                            }
                        }
                        fetch(j);
                    }
                    advance(ahead, ak);
                    aim();
                    more = tile == was;
                }
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) sums[(warp * NP + j) * 128 + q * 32 + lane] = acc[j][q];
            }
            __syncthreads();  // (two buffers: the next round's sums are written while a slow warp still reads these)
            // A thread has a row and every eighth token: nobody else adds to its sums.
            const int row = (int)threadIdx.x % kRows, eighth = (int)threadIdx.x / kRows;
            if (eighth < 8) {
                const int j = row >> 4, h = row >> 3 & 1;
                for (int t = 0; t < share && r0 + t < all; ++t) {
                    const int i = l.of_tile[r0 + t], entry0 = l.first[i] + 8 * (r0 + t - l.tiles[i]), n = l.first[i + 1] - entry0;
                    const int first = share > 1 ? t * pieces : 0, meet = share > 1 || pieces < W ? pieces : W;
                    for (int e = 0; e < 8 && e < n; ++e) {
                        const int token = l.token[entry0 + e];
                        if ((token & 7) != eighth) continue;
                        const float *const of_w = sums + (first * NP + j) * 128 + (2 * h + (e & 1)) * 32 + (row & 7) * 4 + (e >> 1);
                        float v = 0.0f;
                        for (int w = 0; w < meet; ++w) v += of_w[w * NP * 128];
                        out[token * kRows + row] += v;
                    }
                }
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        for (int o = threadIdx.x; o < a.T * kRows; o += 32 * W) {
            const int token = o / kRows, row = base + o - token * kRows;
            if (row >= from && row < to) static_cast<TX *>(a.y)[(int64_t)token * a.ys + row] = from_f<TX>(out[o]);
        }
        __syncthreads();
    }
}

constexpr int kDevices = 64;
constexpr int kUpSmem = kUpWarps * kUpRing + 2 * kUpWarps * kUpPairs * 128 * 4 + (int)sizeof(Lists);
template <bool kF8>
constexpr int kDownSmem = kDownWarps * kDownRing + 2 * kDownWarps * kDownPairs * 128 * 4 + kMaxTokens * 16 * kDownPairs * 4 + (int)sizeof(Lists) +
                          (kF8 ? kLows : 0);
static_assert(kUpSmem <= 227 * 1024 && kDownSmem<true> <= 227 * 1024, "an SM's memory");

// SMs of the current device; once per device allows the kernel its shared memory.
template <typename K>
cudaError_t allow(K k, int smem, std::atomic<int> (&sms)[kDevices], int &n) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    n = sms[dev].load(std::memory_order_acquire);
    if (n) return cudaSuccess;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    sms[dev].store(n, std::memory_order_release);  // (the attribute is set for whoever reads it)
    return cudaSuccess;
}

template <typename TX, bool kF8>
cudaError_t start_down(const Args &a, cudaStream_t s) {
    static std::atomic<int> sms[kDevices];
    const auto k = k_moe_down<TX, kF8>;
    int n = 0;
    const cudaError_t e = allow(k, kDownSmem<kF8>, sms, n);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const int most = (a.d + 7) / 8;
    cfg.gridDim = dim3((unsigned)(n < most ? n : most)), cfg.blockDim = dim3(32 * kDownWarps);
    cfg.dynamicSmemBytes = kDownSmem<kF8>, cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename TX, bool kF8>
cudaError_t start(const Args &a, cudaStream_t s) {
    static std::atomic<int> sms[kDevices];
    const auto k = k_moe_up<TX, kF8>;
    int n = 0;
    cudaError_t e = allow(k, kUpSmem, sms, n);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)n, 32 * kUpWarps, kUpSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return start_down<TX, kF8>(a, s);
}

}  // namespace moe

size_t moe_tokens_workspace_bytes(int T, int top_k, int inner) { return (size_t)T * top_k * inner * 4; }

cudaError_t launch_moe_tokens(const void *x, int64_t x_stride, hc_dtype type, int T, int d, int experts, int inner, int top_k,
                              const float *logits, bool sigmoid, bool normalise, float scale, int32_t *ids, float *p, const void *w_up,
                              const void *w_down, bool f8, const void *up_scales, const void *down_scales, bool scales_f32, void *y,
                              int64_t y_stride, void *workspace, cudaStream_t s) {
    const moe::Args a{x, x_stride, T, d, experts, inner, top_k, logits, sigmoid, normalise, scale, ids, p,
                      static_cast<const uint8_t *>(w_up), static_cast<const uint8_t *>(w_down), {up_scales, scales_f32},
                      {down_scales, scales_f32}, static_cast<float *>(workspace), y, y_stride};
    if (type == HC_BF16) return f8 ? moe::start<__nv_bfloat16, true>(a, s) : moe::start<__nv_bfloat16, false>(a, s);
    return f8 ? moe::start<__half, true>(a, s) : moe::start<__half, false>(a, s);
}

}  // namespace hc
