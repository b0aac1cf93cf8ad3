// hc_moe.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels, for
// GB300.
//
//   y[t] = sum over t's chosen experts e of  p[t, e] D[e] (silu(G[e] x[t]) * U[e] x[t])
// with the choice and its weights p made from the router's logits or given.
//
// A few tokens leave nothing but the reading of the chosen experts' weights.  They go
// past each SM once, in 8-row pieces of 128 bytes a row, straight to the lane that
// multiplies them: a lane copies (cp.async) 16 bytes of one row into a place of its own,
// many pieces ahead, and reads them from there, so that nothing but its own copies ever
// holds a warp up.  The products run on mma.sync m16n8k16 with the tokens on the 16
// side: they take a fraction of the time that the weights need to arrive, and the
// order of k within a piece is free as long as both operands share it, so a lane's 16
// bytes are its operand as they lie.
//
// First kernel: the rows of all chosen experts' G and U are dealt out evenly to the
// SMs, a block's warps share the contraction, and the products meet in shared memory:
// a = p silu(g) u, fp32, to the workspace.  Second kernel: each SM has some rows of the
// output and all experts' D for them, its warps share the experts and contraction,
// and sum over both.
#include <atomic>

#include <cuda.h>

#include "hc_fp8.cuh"
#include "hc_ptx.cuh"
#include "hc_sublayer.h"
#include "hc_types.cuh"

namespace hc {

namespace moe {

constexpr int kMaxTokens = 64, kMaxTop = 16, kMaxExperts = 1024, kMaxEntries = kMaxTokens * kMaxTop;
constexpr int kCell = 1024;       // bytes of a piece: 8 rows of 128 bytes
constexpr int kWarps = 8;
constexpr int kUpPairs = 4, kUpDeep = 2;      // pairs of row tiles (of G and of U) of a unit; steps whose pieces are under way
constexpr int kDownTiles = 6, kDownDeep = 4;  // row tiles of a pass; steps whose pieces are under way
constexpr int kUpRing = kUpDeep * kUpPairs * 2 * kCell, kDownRing = kDownDeep * kDownTiles * kCell;  // of a warp

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
    uint16_t tiles[kMaxExperts + 1]; // ... and the tiles of 16 entries of those before it
    uint64_t tokens[kMaxExperts];    // ... its tokens, as bits
    int count[kMaxExperts];
    int n;                           // how many experts have entries
};

// A number whose order as an unsigned integer is that of the floats; 0 for -infinity and NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // (the two zeros are equal)
    return v > -INFINITY ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// A warp chooses a token's experts: the `top` largest logits, of equal ones the first.
__device__ __forceinline__ void choose(const Args &a, Lists &l, int t, int lane) {
    const float *lg = a.logits + (int64_t)t * a.experts;
    uint32_t last = 0xffffffffu;
    int last_e = -1;
    float best = 0.0f, sum = 0.0f;
    for (int j = 0; j < a.top; ++j) {
        // the largest behind the one chosen last
        uint32_t key = 0;
        int e = 0x7fffffff;
        for (int i = lane; i < a.experts; i += 32) {
            const uint32_t k = order_key(__ldg(lg + i));
            if ((k < last || (k == last && i > last_e)) && k > key) key = k, e = i;
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, key);
        e = (int)__reduce_min_sync(0xffffffffu, key == top ? (uint32_t)e : 0x7fffffffu);
        last = top, last_e = e;
        float s = 0.0f;
        if (top != 0u) {
            const float v = of_key(top);
            if (j == 0) best = v;
            s = a.sigmoid ? 1.0f / (1.0f + expf(-v)) : v == best ? 1.0f : expf(v - best);
        }
        sum += s;
        if (lane == 0) {
            l.id[t * a.top + j] = (int16_t)(top != 0u ? e : -1);
            l.p[t * a.top + j] = s;
        }
        if (top == 0u) last = 0u, last_e = 0x7fffffff;  // nothing is left
    }
    if (!a.normalise) {
        if (!a.sigmoid) {  // over all experts
            sum = 0.0f;
            for (int i = lane; i < a.experts; i += 32) {
                const float v = __ldg(lg + i);
                if (order_key(v) != 0u) sum += v == best ? 1.0f : expf(v - best);
            }
            sum = warp_sum(sum);
        } else {
            sum = 1.0f;
        }
    }
    __syncwarp();
    for (int j = lane; j < a.top; j += 32) {
        float &p = l.p[t * a.top + j];
        p = sum > 0.0f ? p / sum * a.scale : 0.0f;
        if (blockIdx.x != 0) continue;
        if (a.ids) a.ids[t * a.top + j] = l.id[t * a.top + j];
        if (a.p) a.p[t * a.top + j] = p;
    }
}

// All threads: the choice and the lists by expert.  `write`: whether the choice goes to the caller too.
__device__ __forceinline__ void route(Args a, Lists &l, bool write) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (a.logits) {
        if (!write) a.ids = nullptr, a.p = nullptr;
        for (int t = warp; t < a.T; t += nw) choose(a, l, t, lane);
    } else {
        // given: a place that names no expert has none; of an expert named twice the first
        // place gets both weights
        for (int t = threadIdx.x; t < a.T; t += blockDim.x)
            for (int j = 0; j < a.top; ++j) {
                const int at = t * a.top + j;
                int e = __ldg(a.ids + at);
                float p = __ldg(a.p + at);
                if (e < 0 || e >= a.experts) e = -1;
                for (int i = t * a.top; e >= 0 && i < at; ++i)
                    if (l.id[i] == e) l.p[i] += p, e = -1;
                l.id[at] = (int16_t)e, l.p[at] = p;
            }
    }
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) l.count[e] = 0;
    __syncthreads();
    const int entries = a.T * a.top;
    if (warp == 0) {
        // an expert's entries in their order (all blocks have to agree on which tile of 16 has one)
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
            int before = c, m = (c + 15) / 16;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, before, o), v = __shfl_up_sync(0xffffffffu, m, o);
                if (lane >= o) before += u, m += v;
            }
            const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
            if (c > 0) {
                const int i = n + __popc(some & ((1u << lane) - 1u));
                l.active[i] = (uint16_t)e, l.first[i] = (uint16_t)(at + before - c), l.tiles[i] = (uint16_t)(tiles + m - (c + 15) / 16);
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
        if (l.id[i] >= 0) l.list[l.count[l.id[i]] + l.rank[i]] = (uint16_t)i;
    __syncthreads();
    for (int i = threadIdx.x; i < l.n; i += blockDim.x) {
        uint64_t m = 0;
        for (int j = l.first[i]; j < l.first[i + 1]; ++j) m |= (uint64_t)1 << (l.list[j] / a.top);
        l.tokens[i] = m;
    }
    __syncthreads();
}

// ------------------------------------------------------------ pieces
// A lane's share of a piece: 16 bytes at 16 (lane % 4) of the row lane / 4, and 64 bytes on.
// `there`: whether they are there, else zeros.
__device__ __forceinline__ void load_piece(uint32_t to, const uint8_t *from, bool there0, bool there1) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there0 ? 16 : 0) : "memory");
    asm volatile("cp.async.cg.shared.global.L2::128B [%0 + 512], [%1 + 64], 16, %2;" ::"r"(to), "l"(from), "r"(there1 ? 16 : 0) : "memory");
}
struct Piece {
    uint32_t w[8];
};
__device__ __forceinline__ Piece read_piece(uint32_t at) {
    Piece p;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(p.w[0]), "=r"(p.w[1]), "=r"(p.w[2]), "=r"(p.w[3]) : "r"(at) : "memory");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + 512];" : "=r"(p.w[4]), "=r"(p.w[5]), "=r"(p.w[6]), "=r"(p.w[7]) : "r"(at) : "memory");
    return p;
}
// four codes as two pairs of fp16
__device__ __forceinline__ void widen(uint32_t c, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The tokens' side of the MMAs over a piece: rows lane / 4 and + 8 of 16, this lane's
// values of k in pairs.  kF8: 16 of them per 16 bytes of codes (32 a piece), else 8 (16).
template <bool kF8>
struct Tokens {
    static constexpr int kPairs = kF8 ? 16 : 8;  // pairs of a row's values in a piece
    uint32_t v[2][kPairs];
    float unit[2];  // what a row's values were divided by

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            unit[r] = 1.0f;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) v[r][i] = 0;
        }
    }
    // A row's values -> fp16, the largest (over the piece: the lanes of four) brought to
    // [2^14, 2^15) by a power of two: 11 bits of each value, of small ones 2^-39 of the largest.
    // Of that largest: the power of two, and what it undoes.
    __device__ __forceinline__ float power(int r, float amax) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int b = (int)(__float_as_uint(amax) >> 23);
        b = b < 15 ? 15 : b;
        unit[r] = __uint_as_float((uint32_t)(b - 14) << 23);
        return __uint_as_float((uint32_t)(268 - b) << 23);
    }
    __device__ __forceinline__ void put_scaled(int r, const float (&f)[2 * kPairs]) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * kPairs; ++i) amax = fmaxf(amax, fabsf(f[i]));
        const float m = power(r, amax);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[r][i] = half2_of(f[2 * i] * m, f[2 * i + 1] * m);
    }
    // ... of bf16 values in pairs (the product with the power is exact in bf16)
    __device__ __forceinline__ void put_scaled(int r, const uint32_t (&w)[kPairs]) {
        const auto pair_of = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
        __nv_bfloat162 top = __habs2(pair_of(w[0]));
#pragma unroll
        for (int i = 1; i < kPairs; ++i) top = __hmax2(top, __habs2(pair_of(w[i])));
        const float2 t = __bfloat1622float2(top);
        const __nv_bfloat162 m = __float2bfloat162_rn(power(r, fmaxf(fmaxf(t.x, t.y), 0.0f)));
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const __nv_bfloat162 p = __hmul2(pair_of(w[i]), m);
            const uint32_t u = *reinterpret_cast<const uint32_t *>(&p);
            v[r][i] = half2_of(bf16lo(u), bf16hi(u));
        }
    }
};

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (__is_same(T, __nv_bfloat16)) mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
    else mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
}
// even, odd += a piece's products, every second step of k each (two chains of MMAs)
template <typename T, bool kF8>
__device__ __forceinline__ void multiply(float (&even)[4], float (&odd)[4], const Tokens<kF8> &x, const Piece &p) {
#pragma unroll
    for (int i = 0; i < Tokens<kF8>::kPairs; i += 2) {
        uint32_t b0, b1;
        if constexpr (kF8) widen(p.w[i / 2], b0, b1);
        else b0 = p.w[i], b1 = p.w[i + 1];
        mma<T>(i & 2 ? odd : even, x.v[0][i], x.v[1][i], x.v[0][i + 1], x.v[1][i + 1], b0, b1);
    }
}
// acc += a piece's products, scaled: by s (the block's) and what the tokens were divided by
template <bool kF8>
__device__ __forceinline__ void multiply_scaled(float (&acc)[4], const Tokens<kF8> &x, const Piece &p, float s) {
    float even[4] = {0.0f, 0.0f, 0.0f, 0.0f}, odd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    multiply<__half, kF8>(even, odd, x, p);
    const float u0 = s * x.unit[0], u1 = s * x.unit[1];
    acc[0] = fmaf(even[0] + odd[0], u0, acc[0]), acc[1] = fmaf(even[1] + odd[1], u0, acc[1]);
    acc[2] = fmaf(even[2] + odd[2], u1, acc[2]), acc[3] = fmaf(even[3] + odd[3], u1, acc[3]);
}

// ------------------------------------------------------------ G and U
// A unit: up to 32 rows (four tiles of 8) of one expert's G and U, for up to 16 entries.
struct Unit {
    int i, m, row, left;  // the expert (in `active`), tile of entries, next row; rows left of this block's
    int lo, hi;           // the unit's rows
    __device__ __forceinline__ bool next(const Args &a) {
        if (left <= 0) return false;
        lo = row, hi = (lo & ~7) + 8 * kUpPairs;
        if (hi > a.inner) hi = a.inner;
        if (hi - lo > left) hi = lo + left;
        left -= hi - lo, row = hi;
        return true;
    }
    // (after the unit's expert and tile have been looked at)
    __device__ __forceinline__ void step(const Args &a, const Lists &l) {
        if (row < a.inner) return;
        row = 0;
        if (++m >= l.tiles[i + 1] - l.tiles[i]) m = 0, ++i;
    }
};

// Steps: a unit's pieces, one of 128 bytes of every row at a time, go round the warps.
template <typename TX, bool kF8>
__global__ void __launch_bounds__(32 * kWarps, 1) k_moe_up(const Args a) {
    constexpr int kBytes = kF8 ? 1 : 2, kOut = kUpPairs * 128;  // kOut: rows by entries of a unit
    constexpr int kVecs = kF8 ? 4 : 2;  // 16-byte loads of a token's values of a piece
    extern __shared__ __align__(128) uint8_t smem[];
    float *const red = reinterpret_cast<float *>(smem + kWarps * kUpRing);  // [2][warp][G, U][kOut]
    Lists &l = *reinterpret_cast<Lists *>(red + 2 * kWarps * 2 * kOut);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    route(a, l, true);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t all = (int64_t)l.tiles[l.n] * a.inner;
    const int64_t from = all * blockIdx.x / gridDim.x, to = all * (blockIdx.x + 1) / gridDim.x;
    if (from == to) return;
    Unit first;
    {
        const int tile = (int)(from / a.inner);
        int lo = 0, hi = l.n;  // the expert whose tiles this one is of
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (l.tiles[mid] <= tile) lo = mid;
            else hi = mid;
        }
        first.i = lo, first.m = tile - l.tiles[lo], first.row = (int)(from - (int64_t)tile * a.inner), first.left = (int)(to - from);
    }
    const int row_bytes = a.d * kBytes, pieces = (row_bytes + 127) / 128;
    const int64_t matrix = (int64_t)a.inner * row_bytes;  // G or U of an expert
    const auto begin = [&](int u) {  // the warp's first piece of unit u
        return (warp + u * (kWarps - pieces % kWarps)) % kWarps;
    };

    // copies run kUpDeep steps ahead
    Unit ahead = first;
    bool more = ahead.next(a);
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
            ahead.step(a, l);
            more = ahead.next(a);
            if (more) aim(), ak = begin(++au);
        }
        if (!more) rows = 0;
    };
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kUpRing + lane * 16);
    const int64_t tile_bytes = 8 * (int64_t)row_bytes;
    const auto fetch = [&](uint32_t to, int j) {
        const uint8_t *const p = lane_row + (int64_t)j * tile_bytes + ak * 128;
        const bool there = rows >> j & 1u, first_half = there && ak * 128 + t4 * 16 < row_bytes,
                   second_half = there && ak * 128 + t4 * 16 + 64 < row_bytes;
        load_piece(to, p, first_half, second_half);
        load_piece(to + kCell, p + matrix, first_half, second_half);
        cp_async_commit();
    };
    if (more) aim();
    settle();
#pragma unroll
    for (int s = 0; s < kUpDeep; ++s) {
#pragma unroll
        for (int j = 0; j < kUpPairs; ++j) fetch(ring + (uint32_t)((s * kUpPairs + j) * 2 * kCell), j);
        ak += kWarps;
        settle();
    }

    const int row_blocks = (a.inner + kFp8Block - 1) / kFp8Block, col_blocks = (a.d + kFp8Block - 1) / kFp8Block;
    uint32_t at = ring;  // the step's place
    int buf = 0;
    Unit u = first;
    for (int un = 0; u.next(a); u.step(a, l), ++un, buf ^= 1) {
        // this lane's two tokens
        const int e = l.active[u.i], entry0 = l.first[u.i] + 16 * u.m, end = l.first[u.i + 1];
        const bool second = entry0 + 8 < end;  // (of the warp: whether there are more than eight)
        const TX *x[2];
        bool has[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            has[r] = entry0 + g + 8 * r < end;
            x[r] = static_cast<const TX *>(a.x) + (has[r] ? (int64_t)(l.list[entry0 + g + 8 * r] / a.top) * a.xs : 0);
        }
        const int base = u.lo & ~7, tiles = (u.hi - base + 7) / 8;
        // lane 2 j + (0: G, 1: U) looks after the scale of pair j
        int64_t scale_at = 0;
        if (kF8 && lane < 2 * tiles)
            scale_at = (((int64_t)e * 2 + (lane & 1)) * row_blocks + (base + 8 * (lane >> 1)) / kFp8Block) * col_blocks;
        uint4 raw[2][kVecs];
        float scale = 1.0f;
        const auto load_tokens = [&](int k) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int s = 0; s < kVecs; ++s) {
                    const int c = kF8 ? k * 128 + (s >> 1) * 64 + t4 * 16 + (s & 1) * 8 : k * 64 + s * 32 + t4 * 8;
                    raw[r][s] = make_uint4(0, 0, 0, 0);
                    if (has[r] && c < a.d) raw[r][s] = __ldg(reinterpret_cast<const uint4 *>(x[r] + c));
                }
            if (kF8 && lane < 2 * tiles) scale = a.up_scales.at(scale_at + k);
        };
        float acc[kUpPairs][2][4], odd[kF8 ? 1 : kUpPairs][2][4];
#pragma unroll
        for (int j = 0; j < kUpPairs; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[j][h][k] = 0.0f;
                    if (!kF8) odd[kF8 ? 0 : j][h][k] = 0.0f;
                }
        int k = begin(un);
        if (k < pieces) load_tokens(k);
        for (; k < pieces; k += kWarps) {
            Tokens<kF8> tok;
            tok.clear();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (r == 1 && !second) break;
                uint32_t w[Tokens<kF8>::kPairs];
#pragma unroll
                for (int s = 0; s < kVecs; ++s) w[4 * s] = raw[r][s].x, w[4 * s + 1] = raw[r][s].y, w[4 * s + 2] = raw[r][s].z, w[4 * s + 3] = raw[r][s].w;
                if constexpr (kF8 && __is_same(TX, __nv_bfloat16)) {
                    tok.put_scaled(r, w);
                } else {
#pragma unroll
                    for (int i = 0; i < Tokens<kF8>::kPairs; ++i) tok.v[r][i] = w[i];
                }
            }
            const float scales = scale;
            if (k + kWarps < pieces) load_tokens(k + kWarps);
#pragma unroll
            for (int j = 0; j < kUpPairs; ++j) {
                cp_async_wait<kUpDeep * kUpPairs - 1>();
                const uint32_t here = at + (uint32_t)(j * 2 * kCell);
                const Piece pg = read_piece(here), pu = read_piece(here + kCell);
                if (j < tiles) {
                    if constexpr (kF8) {
                        multiply_scaled<true>(acc[j][0], tok, pg, __shfl_sync(0xffffffffu, scales, 2 * j));
                        multiply_scaled<true>(acc[j][1], tok, pu, __shfl_sync(0xffffffffu, scales, 2 * j + 1));
                    } else {
                        multiply<TX, false>(acc[j][0], odd[kF8 ? 0 : j][0], tok, pg);
                        multiply<TX, false>(acc[j][1], odd[kF8 ? 0 : j][1], tok, pu);
                    }
                }
                fetch(here, j);
            }
            at = at == ring ? ring + kUpRing / kUpDeep : ring;
            static_assert(kUpDeep == 2, "two places");
            ak += kWarps;
            settle();
        }
        // the warps' sums meet
        float *const mine = red + ((buf * kWarps + warp) * 2) * kOut + lane;
        if (begin(un) < pieces) {
#pragma unroll
            for (int j = 0; j < kUpPairs; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (j < tiles && (q < 2 || second)) mine[h * kOut + (j * 4 + q) * 32] = acc[j][h][q] + (kF8 ? 0.0f : odd[kF8 ? 0 : j][h][q]);
        }
        __syncthreads();  // (two buffers: the next unit's sums are written while a slow warp still reads these)
        const int meet = pieces < kWarps ? pieces : kWarps, w0 = un * (pieces % kWarps) % kWarps;  // those that had a piece, in their order
        for (int o = threadIdx.x; o < kOut; o += 32 * kWarps) {
            const int j = o >> 7, q = o >> 5 & 3;  // (o % 32 is this lane)
            const int row = base + 8 * j + 2 * t4 + (q & 1), entry = entry0 + g + 8 * (q >> 1);
            if (j >= tiles || row < u.lo || row >= u.hi || entry >= end) continue;
            float gate = 0.0f, up = 0.0f;
            for (int i = 0, w = w0; i < meet; ++i) {
                const float *from_w = red + ((buf * kWarps + w) * 2) * kOut + o;
                gate += from_w[0], up += from_w[kOut];
                if (++w == kWarps) w = 0;
            }
            const int id = l.list[entry];
            a.a[(int64_t)id * a.inner + row] = gate / (1.0f + expf(-gate)) * up * l.p[id];
        }
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------ D
// A block's rows of the output, in passes of kDownTiles tiles of 8; MT tiles of 16 tokens.
// Steps: a piece of 128 bytes of every row of one expert; they go round the warps.
template <typename TX, bool kF8, int MT>
__global__ void __launch_bounds__(32 * kWarps, 1) k_moe_down(const Args a) {
    constexpr int kBytes = kF8 ? 1 : 2, NT = kDownTiles, V = 2 * Tokens<kF8>::kPairs;
    constexpr bool kSplit = !kF8 && __is_same(TX, __nv_bfloat16);  // a as two bf16 numbers
    static_assert(MT * NT * 4 * 32 * 4 <= kDownRing, "the sums meet where the pieces were");
    extern __shared__ __align__(128) uint8_t smem[];
    Lists &l = *reinterpret_cast<Lists *>(smem + kWarps * kDownRing);
    float *const red = reinterpret_cast<float *>(smem);  // [warp][tokens' tile][tile][4][lane]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    route(a, l, false);
    const int from = (int)((int64_t)a.d * blockIdx.x / gridDim.x), to = (int)((int64_t)a.d * (blockIdx.x + 1) / gridDim.x);
    const int row_bytes = a.inner * kBytes, pieces = (row_bytes + 127) / 128, all = l.n * pieces;
    const int row_blocks = (a.d + kFp8Block - 1) / kFp8Block, col_blocks = (a.inner + kFp8Block - 1) / kFp8Block;
    const int64_t matrix = (int64_t)a.d * row_bytes, tile_bytes = 8 * (int64_t)row_bytes;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kDownRing + lane * 16);
    bool waited = false;
    for (int base = from & ~7; base < to; base += 8 * NT) {
        const int tiles = (to - base + 7) / 8 < NT ? (to - base + 7) / 8 : NT;
        uint32_t rows = 0;  // which tiles have this lane's row
#pragma unroll
        for (int i = 0; i < NT; ++i) rows |= (uint32_t)(base + 8 * i + g >= from && base + 8 * i + g < to) << i;
        int ahead = warp, ai = warp / pieces, ak = warp - ai * pieces;
        const auto fetch = [&](uint32_t to_step) {  // a step's pieces
            if (ahead < all) {
                const uint8_t *const p = a.down + (int64_t)l.active[ai] * matrix + (int64_t)(base + g) * row_bytes + ak * 128 + t4 * 16;
                const bool first_half = ak * 128 + t4 * 16 < row_bytes, second_half = ak * 128 + t4 * 16 + 64 < row_bytes;
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    if (i < tiles) load_piece(to_step + (uint32_t)(i * kCell), p + i * tile_bytes, (rows >> i & 1u) && first_half, (rows >> i & 1u) && second_half);
            }
            cp_async_commit();
            ahead += kWarps, ak += kWarps;
            while (ak >= pieces) ak -= pieces, ++ai;
        };
#pragma unroll
        for (int s = 0; s < kDownDeep; ++s) fetch(ring + (uint32_t)(s * NT * kCell));
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel's results are read from here on
        waited = true;
        float acc[MT][NT][4], odd[kF8 || !kSplit ? 1 : MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[m][i][k] = 0.0f;
                    if (kSplit) odd[kSplit ? m : 0][i][k] = 0.0f;
                }
        // this lane's two tokens of a tile of 16: their activations for the expert
        const auto load_tokens = [&](int m, int i, int k, float4 (&raw)[2][V / 4]) {
            const uint64_t tokens = l.tokens[i];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (r == 1 && a.T <= 8) break;
                const int t = 16 * m + g + 8 * r;
                const bool has = tokens >> t & 1u;
                const float *from_a = a.a;
                if (has) from_a += (int64_t)l.list[l.first[i] + __popcll(tokens & (((uint64_t)1 << t) - 1))] * a.inner;
#pragma unroll
                for (int q = 0; q < V / 4; ++q) {
                    const int c = kF8 ? k * 128 + (q >> 2) * 64 + t4 * 16 + (q & 3) * 4 : k * 64 + (q >> 1) * 32 + t4 * 8 + (q & 1) * 4;
                    raw[r][q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (has && c < a.inner) raw[r][q] = __ldcg(reinterpret_cast<const float4 *>(from_a + c));
                }
            }
        };
        const auto load_scale = [&](int i, int k) {  // lane i: tile i's
            return kF8 && lane < tiles ? a.down_scales.at(((int64_t)l.active[i] * row_blocks + (base + 8 * lane) / kFp8Block) * col_blocks + k) : 1.0f;
        };
        float4 raw[2][V / 4];
        float scale = 1.0f;
        int bi = warp / pieces, bk = warp - bi * pieces, step = 0;
        if (warp < all) {
            if (MT == 1) load_tokens(0, bi, bk, raw);
            scale = load_scale(bi, bk);
        }
        for (int b = warp; b < all; b += kWarps) {
            const float scales = scale;
            int ni = bi, nk = bk + kWarps;
            while (nk >= pieces) nk -= pieces, ++ni;
            const uint64_t tokens = l.tokens[bi];
            const uint32_t here = ring + (uint32_t)(step * NT * kCell);
            cp_async_wait<kDownDeep - 1>();
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (MT > 1) {
                    if (!(tokens >> (16 * m) & 0xffffu)) continue;
                    load_tokens(m, bi, bk, raw);
                }
                Tokens<kF8> tok, low;
                tok.clear();
                if constexpr (kSplit) low.clear();
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (r == 1 && a.T <= 8) break;
                    float f[V];
#pragma unroll
                    for (int q = 0; q < V / 4; ++q) f[4 * q] = raw[r][q].x, f[4 * q + 1] = raw[r][q].y, f[4 * q + 2] = raw[r][q].z, f[4 * q + 3] = raw[r][q].w;
                    if constexpr (kSplit) {
#pragma unroll
                        for (int q = 0; q < V / 2; ++q) {
                            const uint32_t h = pack_bf16x2(f[2 * q], f[2 * q + 1]);
                            tok.v[r][q] = h;
                            low.v[r][q] = pack_bf16x2(f[2 * q] - bf16lo(h), f[2 * q + 1] - bf16hi(h));
                        }
                    } else {
                        tok.put_scaled(r, f);
                    }
                }
                if (MT == 1 && b + kWarps < all) {
                    load_tokens(0, ni, nk, raw);
                    scale = load_scale(ni, nk);
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (i >= tiles) continue;
                    const Piece p = read_piece(here + (uint32_t)(i * kCell));
                    if constexpr (kSplit) {
                        multiply<TX, false>(acc[m][i], odd[kSplit ? m : 0][i], tok, p);
                        multiply<TX, false>(acc[m][i], odd[kSplit ? m : 0][i], low, p);
                    } else {
                        multiply_scaled<kF8>(acc[m][i], tok, p, __shfl_sync(0xffffffffu, scales, i));
                    }
                }
            }
            if (MT > 1 && b + kWarps < all) scale = load_scale(ni, nk);
            bi = ni, bk = nk;
            if (++step == kDownDeep) step = 0;
            fetch(here);
        }
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    red[(((warp * MT + m) * NT + i) * 4 + k) * 32 + lane] = acc[m][i][k] + (kSplit ? odd[kSplit ? m : 0][i][k] : 0.0f);
        __syncthreads();
        const int meet = all < kWarps ? all : kWarps;
        for (int o = threadIdx.x; o < MT * NT * 128; o += 32 * kWarps) {
            const int m = o / (NT * 128), i = o / 128 % NT, k = o / 32 % 4;  // (o % 32 is this lane)
            const int tok = 16 * m + g + 8 * (k >> 1), row = base + 8 * i + 2 * t4 + (k & 1);
            if (tok >= a.T || row < from || row >= to) continue;
            float v = 0.0f;
            for (int w = 0; w < meet; ++w) v += red[w * MT * NT * 128 + o];
            static_cast<TX *>(a.y)[(int64_t)tok * a.ys + row] = from_f<TX>(v);
        }
        __syncthreads();
    }
}

constexpr int kDevices = 64;
constexpr int kUpSmem = kWarps * kUpRing + 2 * kWarps * 2 * kUpPairs * 128 * 4 + (int)sizeof(Lists);
constexpr int kDownSmem = kWarps * kDownRing + (int)sizeof(Lists);
static_assert(kUpSmem <= 227 * 1024 && kDownSmem <= 227 * 1024, "an SM's memory");

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

template <typename TX, bool kF8, int MT>
cudaError_t start_down(const Args &a, cudaStream_t s) {
    static std::atomic<int> sms[kDevices];
    const auto k = k_moe_down<TX, kF8, MT>;
    int n = 0;
    const cudaError_t e = allow(k, kDownSmem, sms, n);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const int most = (a.d + 7) / 8;
    cfg.gridDim = dim3((unsigned)(n < most ? n : most)), cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = kDownSmem, cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename TX, bool kF8>
cudaError_t start(const Args &a, cudaStream_t s) {
    static std::atomic<int> sms[kDevices];
    const auto k = k_moe_up<TX, kF8>;
    int n = 0;
    cudaError_t e = allow(k, kUpSmem, sms, n);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)n, 32 * kWarps, kUpSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (a.T <= 16) return start_down<TX, kF8, 1>(a, s);
    if (a.T <= 32) return start_down<TX, kF8, 2>(a, s);
    return start_down<TX, kF8, 4>(a, s);
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
