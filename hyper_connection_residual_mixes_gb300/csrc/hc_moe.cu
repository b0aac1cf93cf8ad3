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
constexpr int kUpWarps = 16, kUpCells = 8, kUpTiles = 8;  // warps, pieces each has under way, row tiles of a unit (4 of G, 4 of U)
constexpr int kDownCells = 192, kDownTiles = 6;           // pieces that a block has under way, row tiles of a pass

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
}

// ------------------------------------------------------------ pieces
// A lane's share of a piece: 16 bytes at 16 (lane % 4) and 64 more, of row lane / 4.
__device__ __forceinline__ void load_piece(uint32_t to, const uint8_t *row, bool is_there, int at, int row_bytes) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int off = at + 64 * s;
        const int bytes = is_there && off < row_bytes ? 16 : 0;
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to + 512 * s), "l"(bytes ? row + off : row), "r"(bytes)
                     : "memory");
    }
}
struct Piece {
    uint32_t w[8];
};
__device__ __forceinline__ Piece read_piece(uint32_t at) {
    Piece p;
#pragma unroll
    for (int s = 0; s < 2; ++s)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(p.w[4 * s]), "=r"(p.w[4 * s + 1]), "=r"(p.w[4 * s + 2]), "=r"(p.w[4 * s + 3])
                     : "r"(at + 512 * s)
                     : "memory");
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
    // values as they are
    __device__ __forceinline__ void put16(int r, int i, uint4 u) { v[r][i] = u.x, v[r][i + 1] = u.y, v[r][i + 2] = u.z, v[r][i + 3] = u.w; }
    // fp32 values -> fp16, the row's largest (over the piece: the lanes of four) brought to
    // [2^14, 2^15) by a power of two: 11 bits of each value, of small ones 2^-39 of the largest
    __device__ __forceinline__ void put_scaled(int r, const float (&f)[2 * kPairs]) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * kPairs; ++i) amax = fmaxf(amax, fabsf(f[i]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int b = (int)(__float_as_uint(amax) >> 23);
        b = b < 15 ? 15 : b;
        const float m = __uint_as_float((uint32_t)(268 - b) << 23);
        unit[r] = __uint_as_float((uint32_t)(b - 14) << 23);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[r][i] = half2_of(f[2 * i] * m, f[2 * i + 1] * m);
    }
};

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (__is_same(T, __nv_bfloat16)) mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
    else mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
}
// part += a piece's products
template <typename T, bool kF8>
__device__ __forceinline__ void multiply(float (&part)[4], const Tokens<kF8> &x, const Piece &p) {
#pragma unroll
    for (int i = 0; i < Tokens<kF8>::kPairs; i += 2) {
        uint32_t b0, b1;
        if constexpr (kF8) widen(p.w[i / 2], b0, b1);
        else b0 = p.w[i], b1 = p.w[i + 1];
        mma<T>(part, x.v[0][i], x.v[1][i], x.v[0][i + 1], x.v[1][i + 1], b0, b1);
    }
}

// ------------------------------------------------------------ G and U
// A unit: up to 32 rows (four tiles of 8) of one expert's G and U, for up to 16 entries.
struct Unit {
    int i, m, row, left;  // the expert (in `active`), tile of entries, next row; rows left of this block's
    int lo, hi;           // the unit's rows
    __device__ __forceinline__ bool next(const Args &a, const Lists &l) {
        if (left <= 0) return false;
        lo = row, hi = (lo & ~7) + 8 * (kUpTiles / 2);
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

template <typename TX, bool kF8>
__global__ void __launch_bounds__(32 * kUpWarps, 1) k_moe_up(const Args a) {
    constexpr int kBytes = kF8 ? 1 : 2;
    extern __shared__ __align__(128) uint8_t smem[];
    Lists &l = *reinterpret_cast<Lists *>(smem + kUpWarps * kUpCells * kCell + kUpWarps * kUpTiles * 4 * 32 * 4);
    float *const red = reinterpret_cast<float *>(smem + kUpWarps * kUpCells * kCell);  // [warp][tile][4][lane]
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

    // copies run ahead: unit by unit, piece by piece of this warp's, tile by tile
    Unit ahead = first;
    bool more = ahead.next(a, l);
    int au = 0, ak = warp, atile = 0, slot = 0;
    const uint8_t *abase = nullptr;
    const auto skip = [&](int u) {  // the warp's first piece of unit u: pieces go round the warps
        int k = (warp - u * pieces) % kUpWarps;
        return k < 0 ? k + kUpWarps : k;
    };
    const auto expert_base = [&](const Unit &u) { return a.up + (int64_t)l.active[u.i] * 2 * matrix; };
    if (more) abase = expert_base(ahead);
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kUpCells * kCell + lane * 16);
    const auto fetch = [&]() {
        while (more && ak >= pieces) {
            ahead.step(a, l);
            more = ahead.next(a, l);
            if (more) abase = expert_base(ahead), ak = skip(++au);
        }
        if (more) {
            const int row = (ahead.lo & ~7) + 8 * (atile >> 1) + g;
            load_piece(ring + (uint32_t)slot * kCell, abase + (atile & 1) * matrix + (int64_t)row * row_bytes,
                       row >= ahead.lo && row < ahead.hi, ak * 128 + t4 * 16, row_bytes);
            if (++atile == kUpTiles) atile = 0, ak += kUpWarps;
        }
        cp_async_commit();
        if (++slot == kUpCells) slot = 0;
    };
    for (int c = 0; c < kUpCells; ++c) fetch();

    const int row_blocks = (a.inner + kFp8Block - 1) / kFp8Block, col_blocks = (a.d + kFp8Block - 1) / kFp8Block;
    Unit u = first;
    for (int un = 0; u.next(a, l); u.step(a, l), ++un) {
        // this lane's two tokens
        const int e = l.active[u.i], at = l.first[u.i] + 16 * u.m + g, end = l.first[u.i + 1];
        const bool has[2] = {at < end, at + 8 < end};
        const bool second = l.first[u.i] + 16 * u.m + 8 < end;  // (of the warp: whether there are more than eight)
        const TX *x[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) x[r] = static_cast<const TX *>(a.x) + (has[r] ? (int64_t)(l.list[at + 8 * r] / a.top) * a.xs : 0);
        const int base = u.lo & ~7, tiles = (u.hi - base + 7) / 8;
        float acc[kUpTiles][4];
#pragma unroll
        for (int i = 0; i < kUpTiles; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
        for (int k = skip(un); k < pieces; k += kUpWarps) {
            Tokens<kF8> tok;
            tok.clear();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (r == 1 && !second) break;
                if constexpr (!kF8) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int c = k * 64 + s * 32 + t4 * 8;
                        if (has[r] && c < a.d) tok.put16(r, 4 * s, __ldg(reinterpret_cast<const uint4 *>(x[r] + c)));
                    }
                } else if constexpr (__is_same(TX, __half)) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int c = k * 128 + s * 64 + t4 * 16;
                        if (has[r] && c < a.d) {
                            tok.put16(r, 8 * s, __ldg(reinterpret_cast<const uint4 *>(x[r] + c)));
                            tok.put16(r, 8 * s + 4, __ldg(reinterpret_cast<const uint4 *>(x[r] + c + 8)));
                        }
                    }
                } else {
                    float f[32];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int c = k * 128 + (s >> 1) * 64 + t4 * 16 + (s & 1) * 8;
                        uint4 q = make_uint4(0, 0, 0, 0);
                        if (has[r] && c < a.d) q = __ldg(reinterpret_cast<const uint4 *>(x[r] + c));
                        f[8 * s] = bf16lo(q.x), f[8 * s + 1] = bf16hi(q.x), f[8 * s + 2] = bf16lo(q.y), f[8 * s + 3] = bf16hi(q.y);
                        f[8 * s + 4] = bf16lo(q.z), f[8 * s + 5] = bf16hi(q.z), f[8 * s + 6] = bf16lo(q.w), f[8 * s + 7] = bf16hi(q.w);
                    }
                    tok.put_scaled(r, f);
                }
            }
#pragma unroll
            for (int i = 0; i < kUpTiles; ++i) {
                cp_async_wait<kUpCells - 1>();
                const Piece p = read_piece(ring + (uint32_t)slot * kCell);
                if ((i >> 1) < tiles) {
                    if constexpr (kF8) {
                        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        multiply<__half, true>(part, tok, p);
                        // (a tile's rows are of one block of the scales)
                        const float s = a.up_scales.at((((int64_t)e * 2 + (i & 1)) * row_blocks + (base + 8 * (i >> 1)) / kFp8Block) * col_blocks + k);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float f = s * tok.unit[r];
                            acc[i][2 * r] = fmaf(part[2 * r], f, acc[i][2 * r]);
                            acc[i][2 * r + 1] = fmaf(part[2 * r + 1], f, acc[i][2 * r + 1]);
                        }
                    } else {
                        multiply<TX, false>(acc[i], tok, p);
                    }
                }
                fetch();
            }
        }
        // the warps' sums meet, those that had a piece in the order of their pieces
        const int from_warps = pieces < kUpWarps ? pieces : kUpWarps;
        if (skip(un) < pieces) {
#pragma unroll
            for (int i = 0; i < kUpTiles; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if ((i >> 1) < tiles && (k < 2 || second)) red[((warp * kUpTiles + i) * 4 + k) * 32 + lane] = acc[i][k];
        }
        __syncthreads();
        static_assert(kUpWarps * 32 == kUpTiles / 2 * 128, "a thread for each row and entry of a unit");
        {
            const int tile = threadIdx.x >> 7, k = threadIdx.x >> 5 & 3;
            const int row = base + 8 * tile + 2 * t4 + (k & 1), entry = l.first[u.i] + 16 * u.m + g + 8 * (k >> 1);
            if (tile < tiles && row >= u.lo && row < u.hi && entry < end) {
                float gate = 0.0f, up = 0.0f;
                for (int j = 0, w = un * pieces % kUpWarps; j < from_warps; ++j) {
                    gate += red[((w * kUpTiles + 2 * tile) * 4 + k) * 32 + lane];
                    up += red[((w * kUpTiles + 2 * tile + 1) * 4 + k) * 32 + lane];
                    if (++w == kUpWarps) w = 0;
                }
                const int id = l.list[entry];
                a.a[(int64_t)id * a.inner + row] = gate / (1.0f + expf(-gate)) * up * l.p[id];
            }
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------ D
// Rows [from, to) of the output; MT tiles of 16 tokens; kWarps warps share the experts and
// their contraction.
template <typename TX, bool kF8, int MT, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 1) k_moe_down(const Args a) {
    constexpr int kBytes = kF8 ? 1 : 2, kCells = kDownCells / kWarps, NT = kDownTiles;
    constexpr bool kSplit = !kF8 && __is_same(TX, __nv_bfloat16);  // a as two bf16 numbers
    static_assert(kWarps * MT * NT * 4 * 32 * 4 <= kDownCells * kCell && kCells % NT == 0 && kCells >= 2 * NT, "the sums meet where the pieces were");
    extern __shared__ __align__(128) uint8_t smem[];
    Lists &l = *reinterpret_cast<Lists *>(smem + kDownCells * kCell);
    float *const red = reinterpret_cast<float *>(smem);  // [warp][tokens' tile][tile][4][lane]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    route(a, l, false);
    const int from = (int)((int64_t)a.d * blockIdx.x / gridDim.x), to = (int)((int64_t)a.d * (blockIdx.x + 1) / gridDim.x);
    const int row_bytes = a.inner * kBytes, pieces = (row_bytes + 127) / 128, all = l.n * pieces;
    const int row_blocks = (a.d + kFp8Block - 1) / kFp8Block, col_blocks = (a.inner + kFp8Block - 1) / kFp8Block;
    const int64_t matrix = (int64_t)a.d * row_bytes;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kCells * kCell + lane * 16);
    bool waited = false;
    for (int base = from & ~7; base < to; base += 8 * NT) {
        const int tiles = (to - base + 7) / 8 < NT ? (to - base + 7) / 8 : NT;
        int ahead = warp, ai = warp / pieces, ak = warp - ai * pieces, slot = 0;
        const auto fetch = [&]() {  // a piece of every tile
            const uint8_t *const m = ahead < all ? a.down + (int64_t)l.active[ai] * matrix : nullptr;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int row = base + 8 * i + g;
                if (m && i < tiles)
                    load_piece(ring + (uint32_t)slot * kCell, m + (int64_t)row * row_bytes, row >= from && row < to, ak * 128 + t4 * 16, row_bytes);
                if (++slot == kCells) slot = 0;
            }
            cp_async_commit();
            ahead += kWarps, ak += kWarps;
            while (ak >= pieces) ak -= pieces, ++ai;
        };
        constexpr int kDeep = kCells / NT;
#pragma unroll
        for (int c = 0; c < kDeep; ++c) fetch();
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the first kernel's results are read from here on
        waited = true;
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[m][i][k] = 0.0f;
        int at = 0;  // the block of pieces in the ring
        for (int b = warp, bi = warp / pieces, bk = warp - bi * pieces; b < all; b += kWarps) {
            const int e = l.active[bi], first = l.first[bi], end = l.first[bi + 1];
            cp_async_wait<kDeep - 1>();
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                // this lane's two tokens: their entries for this expert
                int entry[2] = {-1, -1};
                bool some = false;
                for (int j = first; j < end; ++j) {
                    const int id = l.list[j], tok = id / a.top;
                    some |= tok >> 4 == m;
                    if (tok == 16 * m + g) entry[0] = id;
                    if (tok == 16 * m + g + 8) entry[1] = id;
                }
                if (!some) continue;
                Tokens<kF8> tok, low;
                tok.clear();
                if constexpr (kSplit) low.clear();
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    constexpr int V = 2 * Tokens<kF8>::kPairs;
                    float f[V];
#pragma unroll
                    for (int q = 0; q < V / 4; ++q) {
                        const int c = kF8 ? bk * 128 + (q >> 2) * 64 + t4 * 16 + (q & 3) * 4 : bk * 64 + (q >> 1) * 32 + t4 * 8 + (q & 1) * 4;
                        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (entry[r] >= 0 && c < a.inner) v = __ldcg(reinterpret_cast<const float4 *>(a.a + (int64_t)entry[r] * a.inner + c));
                        f[4 * q] = v.x, f[4 * q + 1] = v.y, f[4 * q + 2] = v.z, f[4 * q + 3] = v.w;
                    }
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
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (i >= tiles) continue;
                    const Piece p = read_piece(ring + (uint32_t)(at * NT + i) * kCell);
                    if constexpr (kSplit) {
                        multiply<TX, false>(acc[m][i], tok, p);
                        multiply<TX, false>(acc[m][i], low, p);
                    } else {
                        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        multiply<__half, kF8>(part, tok, p);
                        float s = 1.0f;
                        if constexpr (kF8) s = a.down_scales.at(((int64_t)e * row_blocks + (base + 8 * i) / kFp8Block) * col_blocks + bk);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float u = s * tok.unit[r];
                            acc[m][i][2 * r] = fmaf(part[2 * r], u, acc[m][i][2 * r]);
                            acc[m][i][2 * r + 1] = fmaf(part[2 * r + 1], u, acc[m][i][2 * r + 1]);
                        }
                    }
                }
            }
            if (++at == kDeep) at = 0;
            fetch();
            bk += kWarps;
            while (bk >= pieces) bk -= pieces, ++bi;
        }
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) red[(((warp * MT + m) * NT + i) * 4 + k) * 32 + lane] = acc[m][i][k];
        __syncthreads();
        const int warps = all < kWarps ? all : kWarps;
        for (int o = threadIdx.x; o < MT * NT * 128; o += 32 * kWarps) {
            const int m = o / (NT * 128), i = o / 128 % NT, k = o / 32 % 4;  // (o % 32 is this lane)
            const int tok = 16 * m + g + 8 * (k >> 1), row = base + 8 * i + 2 * t4 + (k & 1);
            if (tok >= a.T || row < from || row >= to) continue;
            float v = 0.0f;
            for (int w = 0; w < warps; ++w) v += red[w * MT * NT * 128 + o];
            static_cast<TX *>(a.y)[(int64_t)tok * a.ys + row] = from_f<TX>(v);
        }
        __syncthreads();
    }
}

constexpr int kDevices = 64;
constexpr int kUpSmem = kUpWarps * kUpCells * kCell + kUpWarps * kUpTiles * 4 * 32 * 4 + (int)sizeof(Lists);
constexpr int kDownSmem = kDownCells * kCell + (int)sizeof(Lists);
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

template <typename TX, bool kF8, int MT, int kWarps>
cudaError_t start_down(const Args &a, cudaStream_t s) {
    static std::atomic<int> sms[kDevices];
    const auto k = k_moe_down<TX, kF8, MT, kWarps>;
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
    k<<<(unsigned)n, 32 * kUpWarps, kUpSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (a.T <= 16) return start_down<TX, kF8, 1, 16>(a, s);
    if (a.T <= 32) return start_down<TX, kF8, 2, 16>(a, s);
    return start_down<TX, kF8, 4, 8>(a, s);
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
