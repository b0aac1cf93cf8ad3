// hc_grouped_mm.cu -- matrix products grouped by expert on the fifth-generation
// tensor cores, for GB300.
//
// Rows sorted by expert, offsets[e] <= r < offsets[e + 1] for expert e:
//   product   y[r][f] = sum_k x[r][k] w[e][f][k]          (or w[e][k][f])
//   weights'  g_w[e][c][f] = sum over e's rows of b[r][c] a[r][f]
// bf16 or fp16 operands, fp32 accumulation in tensor memory, one rounding.
//
// Both are D[f][c] = sum_k A[f][k] B[c][k] with f, the output's innermost
// index, on the MMA's M side (128 tensor-memory lanes) and c on its N side.
// The product puts the weights on M and the expert's rows on N: the weights'
// sizes are the same for every expert, and N may be any multiple of 16, so a
// ragged count of rows costs at most 15 columns of MMA work a tile.  An
// expert's rows are cut into tiles of equal length; the offsets are read on
// the device, so the host never waits for the router.
//
// CTAs walk the tiles, one or two an SM (Cfg::kPerSm; warp 0 loads by TMA, warp 1 issues
// tcgen05.mma, warps 2-9 write finished tiles, warp 10 clears the rows behind an
// expert's last one in the gradient's operands); two accumulators alternate, so
// that a tile is written while the next one's products run.  Where few tiles have
// long sums (a row of one wide expert, the gradient of few and long experts) these
// are made in slices, which a second launch adds up.  Where the tiles are
// large two CTAs work on one (cta_group::2: 256 of f, each CTA with half of A's
// rows and half of B's columns in its shared memory): an SM then loads 32 KB for a
// block of 64 of k instead of 48, and what L2 delivers to an SM (some 60 bytes a
// cycle) is what the products wait for otherwise.
//
// 49,152 rows of 64 experts, 2048 x 5120 bf16: 610 us in a burst, 1.69 PFLOP/s (0.88 of
// the measured burst rate); repeated until the board's power limits the clock, 735 us,
// 1.40 PFLOP/s (0.80 of the measured sustained rate).  The split into experts costs
// that last part, not the power alone: the same rows of one expert take 617 us (0.96),
// a library product of that size 609.  An expert of some 770 rows makes three or four
// row tiles, each of which reads all of its weights again, and the last round of
// tiles is not full.  768 rows of the same experts: 201 us, the weights at 0.98 of the
// measured copy rate.
#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hc_sublayer.h"
#include "hc_types.cuh"
#include "hc_umma.cuh"

namespace hc {

namespace gm {

constexpr int kM = 128;       // f per tile
constexpr int kBK = 64;       // k per block: one 128-byte swizzled row of 16-bit values
constexpr int kSub = 2;       // blocks per stage
constexpr int kGroup = 8;     // tiles of c that are walked together
constexpr int kEpilogue = 8;  // warps that write tiles: two for each quarter of the tensor memory's lanes
constexpr int kClear = 2 + kEpilogue, kThreads = 32 * (kClear + 1);
constexpr int kMaxExperts = 1024;
constexpr unsigned int kErrOffsets = 2u;  // device error bit: offsets out of order or out of range

template <int BN, bool kPair, bool kDeep>
struct Cfg {
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kTileF = kM * kCtas;           // f of a tile
    static constexpr int kOwn = BN / kCtas;             // columns whose B a CTA holds
    static constexpr int kGrain = 16 * kCtas;           // an MMA's columns come in these
    static constexpr int kRowBox = kOwn < 64 ? kOwn : 64;  // rows of a small box of B's (a large one holds kOwn)
    // A stage, what a full barrier stands for, is two blocks of k: waiting for one and
    // fencing takes the issuing warp some 300 cycles beside 60 an MMA, and four MMAs of 128
    // cycles do not cover that.  Its blocks are handed back one by one.  K-major
    // operands are loaded block by block as they come free, so that five of six are on
    // their way while one is multiplied; MN-major ones a stage at a time, because boxes
    // of 64 k load a fifth slower than boxes of 128 (both gradients 500 us against 455).
    static constexpr int kABytes = kSub * kM * kBK * 2, kBBytes = kSub * kOwn * kBK * 2, kStage = kABytes + kBBytes;
    // CTAs that share an SM.  Two, with half the stages each, even out the last round of
    // tiles (17 experts' 1224 x 6608: 52 us against 65 with one); but where every tile has
    // an SM to itself, all the stages do better (17 experts' 776 x 2096: 13 us against 16).
    static constexpr int kPerSm = kPair || kDeep ? 1 : 2;
    static constexpr int kStages = kPair ? 3 : kDeep ? 5 : 2;
    static constexpr int kTmemCols = 2 * BN;
    static constexpr int kSmem = kStages * kStage + 1024 + 3 * (kMaxExperts + 1) * 4;
    static_assert(kPerSm * (kSmem + 1024 + 512) <= 228 * 1024 && kPerSm * kTmemCols <= 512, "an SM's memory");
};

struct Args {
    const int32_t *offsets;
    int experts;
    int slices;         // the contraction is cut in so many; slice s goes to the s-th of so many outputs
    int64_t n;          // rows of the row operands
    int F, C, K;        // product: F outputs, K contraction; weights': F x C outputs
    void *out;
    int64_t out_stride; // between consecutive c (product: rows of y; weights': rows of g_w[e])
    int out_f32, fp16, zero_rest;
    int a_whole, b_whole; // whether an MN-major operand's stage comes in one box
};

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major: a block is rows of
// 128 bytes (64 k), 8-row groups 1024 bytes apart, 16 k = 32 bytes.  MN-major: a
// chunk of 64 f or c is rows of 128 bytes per k, 8 k = 1024 bytes, the stage's
// kSub * kBK of k; the next chunk follows; 16 k = 2048 bytes.
constexpr int kChunk = kSub * kBK * 128;
__device__ __forceinline__ uint64_t desc(uint32_t saddr, bool mn_major) {
    const uint64_t chunk = mn_major ? kChunk >> 4 : 1;
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (chunk << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint32_t idesc(bool fp16, bool a_mn, bool b_mn, int m, int n) {
    const uint32_t t = fp16 ? 0u : 1u;
    return (1u << 4) | (t << 7) | (t << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// One thread of the (converged) warp issues; the same one every time.  The other
// operands are the warp's common values, so that they can stay in uniform
// registers: issued from a branch for lane 0 alone an MMA took 150 cycles to
// issue, more than the 128 it runs.
template <bool kPair>
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id),
            "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id),
            "r"(accumulate)
            : "memory");
}
// The four MMAs of a block of 64 of k, their operands kStepA and kStepB (in
// descriptor units) apart, with one election.
template <bool kPair, uint32_t kStepA, uint32_t kStepB>
__device__ __forceinline__ void umma4(uint32_t d, uint64_t a0, uint64_t b0, uint32_t id, uint32_t accumulate) {
    static_assert(kBK == 64, "four MMAs of 16");
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d), "l"(a0), "l"(b0), "r"(id), "r"(accumulate), "n"(kStepA), "n"(kStepB)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d), "l"(a0), "l"(b0), "r"(id), "r"(accumulate), "n"(kStepA), "n"(kStepB)
            : "memory");
}
__device__ __forceinline__ void put(void *out, int64_t i, float v, int f32, int fp16) {
    if (f32) static_cast<float *>(out)[i] = v;
    else if (fp16) static_cast<__half *>(out)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
}

// 32 columns of a tile, `step` bytes apart in memory: column j of this lane's f at
// o + j * step, those below `cols`.  16-bit outputs in pairs of f where every pair
// is aligned: neighbouring lanes trade a column, so that each stores two f of one.
template <typename T>
__device__ __forceinline__ void put32(uint8_t *o, int64_t step, const uint32_t (&v)[32], int cols, bool in) {
#pragma unroll
    for (int j = 0; j < 32; ++j, o += step)
        if (in && j < cols) *reinterpret_cast<T *>(o) = from_f<T>(__uint_as_float(v[j]));
}
template <typename T>
__device__ __forceinline__ void put32_paired(uint8_t *o, int64_t step, const uint32_t (&v)[32], int cols, bool in, int lane) {
    const bool odd = lane & 1;
    if (odd) o += step - 2;
#pragma unroll
    for (int j = 0; j < 32; j += 2, o += 2 * step) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
        Vec<T, 2> p;
        put_pair(p, 0, odd ? f2_make(__uint_as_float(got), __uint_as_float(v[j + 1]))
                           : f2_make(__uint_as_float(v[j]), __uint_as_float(got)));
        if (in && j + odd < cols) *reinterpret_cast<Vec<T, 2> *>(o) = p;
    }
}

// The experts' row ranges and tiles, in shared memory.
struct Plan {
    const int *start, *end, *first;  // rows of expert e; its first tile (first[experts]: all tiles)
};
struct Tile {
    int e, slice;         // (weights': e counts through the slices' experts, their ranges are the slices' own)
    int f0, c0, cols;     // cols: columns of the tile that count (rows of the product)
    int k0, klen;         // contraction: rows [k0, k0 + klen) of the weights', [0, K) of the product
};
// An expert's tiles are walked in groups of kGroup tiles of c, through all of f
// before the next group: what the CTAs read at one time (some 80 tiles) is then
// about as wide as long, and stays in L2 where a long expert's rows do not.
__device__ __forceinline__ void place_of(int local, int ft, int ct, int &f, int &c) {
    const int g = local / (kGroup * ft), rest = local - g * (kGroup * ft);
    const int w = ct - g * kGroup < kGroup ? ct - g * kGroup : kGroup;
    f = rest / w;
    c = g * kGroup + rest - f * w;
}
template <int BN, bool kPair, bool kDeep, bool kWeights>
__device__ __forceinline__ Tile tile_of(const Args &a, const Plan &p, int tile, int &e) {
    while (tile >= p.first[e + 1]) ++e;
    const int local = tile - p.first[e];
    const int rows = p.end[e] - p.start[e];
    Tile t;
    t.e = kWeights ? e : e % a.experts;
    t.slice = kWeights ? 0 : e / a.experts;
    const int ft = (a.F + Cfg<BN, kPair, kDeep>::kTileF - 1) / Cfg<BN, kPair, kDeep>::kTileF;
    int f, c;
    if (kWeights) {
        place_of(local, ft, (a.C + BN - 1) / BN, f, c);
        t.c0 = c * BN;
        t.cols = a.C - t.c0 < BN ? a.C - t.c0 : BN;
        t.k0 = p.start[e];
        t.klen = rows;
    } else {
        const int nt = (rows + BN - 1) / BN;
        constexpr int kGrain = Cfg<BN, kPair, kDeep>::kGrain;
        const int per = ((rows + nt - 1) / nt + kGrain - 1) / kGrain * kGrain;
        place_of(local, ft, nt, f, c);
        const int at = c * per;
        t.c0 = p.start[e] + at;
        t.cols = rows - at < per ? rows - at : per;
        const int part = ((a.K + a.slices - 1) / a.slices + kSub * kBK - 1) / (kSub * kBK) * (kSub * kBK);  // whole stages
        t.k0 = t.slice * part < a.K ? t.slice * part : a.K;
        t.klen = a.K - t.k0 < part ? a.K - t.k0 : part;
    }
    t.f0 = f * Cfg<BN, kPair, kDeep>::kTileF;
    return t;
}

// Rows [s, t) of an expert; false, and none, for a range that is out of order or out
// of the n rows.
__device__ __forceinline__ bool range_of(const int32_t *offsets, int expert, int64_t n, int64_t &s, int64_t &t) {
    s = __ldg(offsets + expert), t = __ldg(offsets + expert + 1);
    if (s >= 0 && t >= s && t <= n) return true;
    s = t = 0;
    return false;
}
// Whether the (not empty) range keeps its rows where some ranges are out of order: it
// must not begin before the end of an earlier one that kept its own.
template <typename I>
__device__ __forceinline__ bool takes_rows(I s, I t, I &end) {
    if (s < end) return false;
    end = t;
    return true;
}

// Where the i-th stage of `stages` starts.  The gradient begins with an expert's
// last rows: their clearing then runs while the tile before is still multiplied.
template <bool kWeights>
__device__ __forceinline__ int stage_start(int i, int stages) {
    return kSub * kBK * (!kWeights ? i : i == 0 ? stages - 1 : i - 1);
}
// Whether the stage from k0 on ends among the rows of 16 that one MMA of the
// weights' gradient reads: the rows behind the expert's last, up to the next 16,
// are another expert's (or anything) and are made zero in both operands first.
__device__ __forceinline__ int rows_to_clear(int klen, int k0) {
    return klen - k0 <= kSub * kBK ? (16 - klen % 16) % 16 : 0;
}
// ... a warp clears them in a stage's `chunks` from `chunk0` on: its rows [left, left + rest).
__device__ __forceinline__ void clear_rows(uint32_t chunk0, int chunks, int left, int rest, int lane) {
    // eight lanes a row of 128 bytes, four rows at a time
    for (int ch = 0; ch < chunks; ++ch)
        for (int r = left + (lane >> 3); r < left + rest; r += 4)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(chunk0 + (uint32_t)(ch * kChunk + r * 128 + (lane & 7) * 16)),
                         "r"(0)
                         : "memory");
    fence_proxy_async_smem();
    __syncwarp();
}

// kAMn: the M side's operand lies MN-major in global memory (w[e][k][f], or the
// rows of the weights' gradient); kWeights: the weights' gradient (B is MN-major too).
// Of a pair the first CTA issues the MMAs and its barriers collect both CTAs'
// loads and both epilogues' arrivals; commits arrive at both CTAs' barriers.
template <int BN, bool kPair, bool kDeep, bool kAMn, bool kWeights>
__global__ void __launch_bounds__(kThreads, Cfg<BN, kPair, kDeep>::kPerSm)
k_grouped_mm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
             const __grid_constant__ CUtensorMap tm_small, const Args a) {
    using C = Cfg<BN, kPair, kDeep>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int *const s_start = reinterpret_cast<int *>(smem_raw + (sbase - smem_u32(smem_raw)) + S * C::kStage);
    int *const s_end = s_start + kMaxExperts, *const s_first = s_end + kMaxExperts;
    __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S * kSub], acc_full[2], acc_empty[2], done_bar;
    __shared__ __align__(8) uint64_t acc_read[2];  // of a pair's second CTA: an accumulator has been read
    __shared__ __align__(8) uint64_t clear_bar[kWeights ? S : 1];  // this CTA's loads of a stage to clear
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kPair ? (int)cluster_ctarank() : 0;
    const int worker = kPair ? (int)blockIdx.x >> 1 : (int)blockIdx.x, workers = kPair ? (int)gridDim.x >> 1 : (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full_bar[s]), C::kCtas);
        for (int s = 0; s < S * kSub; ++s) mbar_init(smem_u32(&empty_bar[s]), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), kEpilogue + (kPair ? 1 : 0));
            mbar_init(smem_u32(&acc_read[b]), kEpilogue);
        }
        if (kWeights)
            for (int s = 0; s < S; ++s) mbar_init(smem_u32(&clear_bar[s]), 1);
        mbar_init(smem_u32(&done_bar), 1);
        s_abort = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 1) tmem_get<kPair>(smem_u32(&s_tmem), C::kTmemCols);
    // (launched before the kernel in front of it has ended: from here on its results are read)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // every expert's rows and how many tiles they make; a range that is out of
    // order or out of the rows counts as empty and is reported
    const int parts = a.experts * a.slices;
    bool wrong = false;
    for (int e = threadIdx.x; e < parts; e += kThreads) {
        const int slice = e / a.experts, ex = e - slice * a.experts;
        int64_t s, t;
        if (!range_of(a.offsets, ex, a.n, s, t)) {
            if (blockIdx.x == 0) atomicOr(&g_device_error, kErrOffsets);
            wrong = true;
        }
        if (kWeights && a.slices > 1) {  // whole stages each, the last ones what is left
            const int64_t per = ((t - s + a.slices - 1) / a.slices + kSub * kBK - 1) / (kSub * kBK) * (kSub * kBK);
            const int64_t from = s + slice * per;
            s = from < t ? from : t;
            t = s + per < t ? s + per : t;
        }
        s_start[e] = (int)s, s_end[e] = (int)t;
        const int mt = (a.F + C::kTileF - 1) / C::kTileF;
        s_first[e + 1] = kWeights ? mt * ((a.C + BN - 1) / BN) : mt * (int)((t - s + BN - 1) / BN);
    }
    // Ranges all in order follow one another.  Where some are not, others may share rows:
    // two CTAs would write them, and the tiles' number, bounded for n rows, leave 32 bits.
    const bool disorder = __syncthreads_or(wrong);
    if (disorder) {
        if (threadIdx.x == 0) {
            int end = 0;
            for (int ex = 0; ex < a.experts; ++ex) {
                const int s = s_start[ex], t = s_end[(a.slices - 1) * a.experts + ex];  // (the last slice's end)
                if (s >= t || takes_rows(s, t, end)) continue;
                for (int e = ex; e < parts; e += a.experts) {
                    s_start[e] = s_end[e] = 0;
                    if (!kWeights) s_first[e + 1] = 0;
                }
            }
        }
        __syncthreads();
    }
    if (warp == 0) {  // running sum of the tile counts
        int carry = 0;
        if (lane == 0) s_first[0] = 0;
        for (int e0 = 0; e0 < parts; e0 += 32) {
            int v = e0 + lane < parts ? s_first[e0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (e0 + lane < parts) s_first[e0 + lane + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    if (kPair) cluster_sync_all();  // the other CTA's barriers and tensor memory are ready
    tmem_fence_after_sync();
    const uint32_t tbase = s_tmem;
    const Plan plan{s_start, s_end, s_first};
    const int tiles = s_first[parts];
    int e = 0;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&tm_a);
            prefetch_tmap(&tm_b);
        }
        __syncwarp();
        // (operands are read again by other tiles, outputs by none: 620 -> 613 us, 470 -> 453 us
        // for the prefill's product and the training batch's gradients.  What it costs the next
        // kernel: reading 64 MB, 96 MB takes it 14.0, 24.2 us after a decode batch's product,
        // 13.2, 20.3 after a plain read of as many bytes)
        const uint64_t pol = policy_evict_last();
        int slot = 0, issued = 0;
        uint32_t parity = 1;
        bool ok = true;
        for (int tile = worker; tile < tiles && ok; tile += workers) {
            Tile t = tile_of<BN, kPair, kDeep, kWeights>(a, plan, tile, e);
            // (one value for the warp: what the issuing thread reads stays in uniform registers)
            t.klen = __shfl_sync(0xffffffffu, t.klen, 0), t.k0 = __shfl_sync(0xffffffffu, t.k0, 0);
            t.f0 = __shfl_sync(0xffffffffu, t.f0, 0), t.c0 = __shfl_sync(0xffffffffu, t.c0, 0);
            t.cols = __shfl_sync(0xffffffffu, t.cols, 0), t.e = __shfl_sync(0xffffffffu, t.e, 0);
            // this CTA's columns of B
            const int own = (t.cols + C::kGrain - 1) / C::kGrain * 16;
            const int c0 = t.c0 + rank * own, f0 = t.f0 + rank * kM;
            const int chunks = (own + 63) / 64;
            // (of the product's rows a box for all that a CTA can hold, or a small one where it
            // holds them; a block's place is the same for both: the tiles follow one another in it)
            const bool small = own <= C::kRowBox;
            const CUtensorMap *tm_rows = small ? &tm_small : &tm_b;
            const bool b_whole = kWeights && a.b_whole && own == C::kOwn;  // (then c0 is a multiple of 64)
            constexpr bool kByStage = kAMn || kWeights;
            // bytes of a block (of an MN-major operand: of half a stage)
            const uint32_t bytes = (uint32_t)(kM * kBK * 2 + (kWeights ? chunks * kChunk / 2 : (small ? C::kRowBox : C::kOwn) * kBK * 2));
            const int stages = (t.klen + kSub * kBK - 1) / (kSub * kBK);
            for (int i = 0; i < stages && ok; ++i) {
                const int k0 = stage_start<kWeights>(i, stages);
                const int blocks = kByStage || t.klen - k0 > kBK ? kSub : 1;
                const uint32_t sa = sbase + (uint32_t)slot * C::kStage, sb = sa + C::kABytes;
                uint32_t bar = smem_u32(&full_bar[slot]);
                const int k = t.k0 + k0;
                for (int s = 0; s < blocks; ++s) {
                    if (!(ok = mbar_wait_warp<false>(smem_u32(&empty_bar[slot * kSub + s]), parity, &s_abort))) break;
                    if (s == 0) {
                        if (kWeights && rows_to_clear(t.klen, k0)) {
                            // the clearing warp passes the stage on to the (first CTA's) full barrier
                            bar = smem_u32(&clear_bar[slot]);
                            expect_bytes(bar, blocks * bytes);
                        } else if (rank == 0) {
                            expect_bytes(bar, C::kCtas * blocks * bytes);  // of a pair both CTAs' bytes
                        } else {
                            bar = mapa(bar, 0);
                            arrive_remote_relaxed(bar);
                        }
                        ++issued;
                    }
                    if (!kByStage) load_3d<kPair>(sa + s * (kM * kBK * 2), &tm_a, bar, k + s * kBK, f0, t.e, pol);
                    if (!kWeights) load_2d<kPair>(sb + s * (C::kBBytes / kSub), tm_rows, bar, k + s * kBK, c0, pol);
                }
                if (kByStage && ok) {
                    if (kWeights) {
                        if (a.a_whole) load_3d<kPair>(sa, &tm_a, bar, 0, k, f0 / 64, pol);
                        else
                            for (int j = 0; j < kM / 64; ++j) load_2d<kPair>(sa + j * kChunk, &tm_a, bar, f0 + j * 64, k, pol);
                        if (b_whole) load_3d<kPair>(sb, &tm_b, bar, 0, k, c0 / 64, pol);
                        else
                            for (int j = 0; j < chunks; ++j) load_2d<kPair>(sb + j * kChunk, &tm_small, bar, c0 + j * 64, k, pol);
                    } else if (a.a_whole) {
                        load_4d<kPair>(sa, &tm_a, bar, 0, k, f0 / 64, t.e, pol);
                    } else {
                        for (int j = 0; j < kM / 64; ++j) load_3d<kPair>(sa + j * kChunk, &tm_a, bar, f0 + j * 64, k, t.e, pol);
                    }
                }
                if (++slot == S) slot = 0, parity ^= 1u;
            }
        }
        // (this CTA needs nothing but its own: a kernel launched to follow may take its place)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        // the last stages issued must land before the CTA leaves (of a pair, the second
        // CTA's have when the MMAs have read them: its empty barriers say so)
        for (int k = 0; k < S && k < issued; ++k) {
            if (--slot < 0) slot = S - 1, parity ^= 1u;
            if (rank == 0) wait_exit(smem_u32(&full_bar[slot]), parity ^ 1u);
            else
                for (int s = 0; s < kSub; ++s) wait_exit(smem_u32(&empty_bar[slot * kSub + s]), parity ^ 1u);
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        int c = 0, slot = 0;
        uint32_t parity = 0;
        bool ok = true;
        // the first stage's descriptors; a stage and 16 of k are steps of their addresses
        const uint64_t da0 = desc(sbase, kAMn || kWeights), db0 = desc(sbase + C::kABytes, kWeights);
        constexpr uint32_t kStepA = (kAMn || kWeights ? 2048 : 32) >> 4, kStepB = (kWeights ? 2048 : 32) >> 4;
        for (int tile = worker; tile < tiles && ok; tile += workers) {
            const Tile t = tile_of<BN, kPair, kDeep, kWeights>(a, plan, tile, e);
            const int klen = __shfl_sync(0xffffffffu, t.klen, 0), cols = __shfl_sync(0xffffffffu, t.cols, 0);
            if (klen == 0) continue;  // an expert without rows: its gradient is zero
            const int b = c & 1;
            if (!(ok = mbar_wait_warp<kPair>(smem_u32(&acc_empty[b]), ((uint32_t)(c >> 1) & 1u) ^ 1u, &s_abort))) break;
            tmem_fence_after_sync();
            const uint32_t d = tbase + (uint32_t)(b * BN);
            const int n = (cols + C::kGrain - 1) / C::kGrain * C::kGrain;
            const uint32_t id = idesc(a.fp16, kAMn || kWeights, kWeights, C::kTileF, n);
            // bytes between the blocks of a stage
            constexpr int a_block = kAMn || kWeights ? kBK * 128 : kM * kBK * 2;
            constexpr int b_block = kWeights ? kBK * 128 : C::kBBytes / kSub;
            uint32_t accumulate = 0;
            const int stages = (klen + kSub * kBK - 1) / (kSub * kBK);
            for (int i = 0; i < stages; ++i) {
                const int k0 = stage_start<kWeights>(i, stages);
                // (the second CTA's clearing is seen by an acquire at cluster scope, too slow for every stage)
                if (kPair && kWeights && rows_to_clear(klen, k0))
                    ok = mbar_wait_warp<true>(smem_u32(&full_bar[slot]), parity, &s_abort);
                else
                    ok = mbar_wait_warp<false>(smem_u32(&full_bar[slot]), parity, &s_abort);
                if (!ok) break;
                tmem_fence_after_sync();
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    const int left = klen - k0 - s * kBK;
                    const uint64_t da = da0 + (uint32_t)(slot * C::kStage + s * a_block) / 16;
                    const uint64_t db = db0 + (uint32_t)(slot * C::kStage + s * b_block) / 16;
                    if (left >= kBK) {
                        umma4<kPair, kStepA, kStepB>(d, da, db, id, accumulate);
                    } else {
                        for (int ks = 0; ks * 16 < left; ++ks)
                            umma<kPair>(d, da + ks * kStepA, db + ks * kStepB, id, ks ? 1u : accumulate);
                    }
                    accumulate = 1;
                    // (also of a block that a last stage does not have, so that all barriers keep step)
                    umma_commit<kPair>(smem_u32(&empty_bar[slot * kSub + s]));
                }
                if (++slot == S) slot = 0, parity ^= 1u;
            }
            if (ok) umma_commit<kPair>(smem_u32(&acc_full[b]));
            ++c;
        }
        // every MMA issued has completed before the tensor memory is freed
        umma_commit<kPair>(smem_u32(&done_bar));
        wait_exit(smem_u32(&done_bar), 0u);
        __syncwarp();
    } else if (warp == 1) {
        // The second CTA of a pair passes on that its accumulators have been read.  An
        // arrival at the other CTA waits for what its thread has stored; this one's has
        // stored nothing, the writing warps' would wait for their tiles (1,500 cycles).
        int c = 0;
        for (int tile = worker; tile < tiles; tile += workers) {
            const Tile t = tile_of<BN, kPair, kDeep, kWeights>(a, plan, tile, e);
            if (t.klen == 0) continue;
            const int b = c & 1;
            if (!mbar_wait_warp<false>(smem_u32(&acc_read[b]), (uint32_t)(c >> 1) & 1u, &s_abort)) break;
            if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&acc_empty[b]), 0));
            __syncwarp();
            ++c;
        }
    } else if (warp == kClear) {
        if constexpr (kWeights) {
            int uses = 0;  // stages of the tiles before
            uint32_t parity = 0;
            bool ok = true;
            for (int tile = worker; tile < tiles && ok; tile += workers) {
                const Tile t = tile_of<BN, kPair, kDeep, kWeights>(a, plan, tile, e);
                const int stages = (t.klen + kSub * kBK - 1) / (kSub * kBK);
                const int slot = uses % S, k0 = stage_start<kWeights>(0, stages);
                uses += stages;
                if (stages == 0 || !rows_to_clear(t.klen, k0)) continue;
                if (!(ok = mbar_wait_warp<false>(smem_u32(&clear_bar[slot]), parity >> slot & 1u, &s_abort))) break;
                parity ^= 1u << slot;
                const int own = (t.cols + C::kGrain - 1) / C::kGrain * 16;
                clear_rows(sbase + (uint32_t)slot * C::kStage, kM / 64 + (own + 63) / 64, t.klen - k0, rows_to_clear(t.klen, k0),
                           lane);
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(smem_u32(&full_bar[slot]));
                    else mbar_arrive_remote(mapa(smem_u32(&full_bar[slot]), 0));
                }
                __syncwarp();
            }
        }
    } else {
        const int q = warp & 3, half = (warp - 2) / 4;  // the warp's quadrant of tensor-memory lanes; which of its two
        const int64_t esize = a.out_f32 ? 4 : 2;
        // (F is a multiple of 8, so pairs end with a row)
        const bool paired = a.out_stride % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0;
        if (!kWeights && a.zero_rest) {
            const auto clear = [&](int64_t from, int64_t to) {
                for (int64_t row = from + blockIdx.x; row < to; row += gridDim.x)
                    for (int f = threadIdx.x - 64; f < a.F; f += 32 * kEpilogue) put(a.out, row * a.out_stride + f, 0.0f, a.out_f32, a.fp16);
            };
            // rows of no expert: before the first one's and from the last one's end on, and
            // between the ranges that count where some are out of order
            if (!disorder) {
                clear(0, __ldg(a.offsets));
                clear(__ldg(a.offsets + a.experts), a.n);
            } else {
                int64_t end = 0;
                for (int ex = 0; ex < a.experts; ++ex)  // (one slice: the ranges ascend)
                    if (s_start[ex] < s_end[ex]) clear(end, s_start[ex]), end = s_end[ex];
                clear(end, a.n);
            }
        }
        int c = 0;
        for (int tile = worker; tile < tiles; tile += workers) {
            const Tile t = tile_of<BN, kPair, kDeep, kWeights>(a, plan, tile, e);
            const int f = t.f0 + rank * kM + q * 32 + lane;
            uint8_t *o = static_cast<uint8_t *>(a.out) +
                         ((kWeights ? (int64_t)t.e * a.C + t.c0 : t.slice * a.n + t.c0) * a.out_stride + f) * esize;
            const int64_t step = a.out_stride * esize;
            const bool in = f < a.F;
            if (t.klen == 0) {
                for (int j = half; j < t.cols; j += 2)
                    if (in) put(o + j * step, 0, 0.0f, a.out_f32, a.fp16);
                continue;
            }
            const int b = c & 1;
            if (!mbar_wait_warp<false>(smem_u32(&acc_full[b]), (uint32_t)(c >> 1) & 1u, &s_abort)) break;
            tmem_fence_after_sync();
            const uint32_t ta = tbase + (uint32_t)(b * BN) + ((uint32_t)(32 * q) << 16);
            o += half * 32 * step;
            for (int j0 = half * 32; j0 < t.cols; j0 += 64, o += 64 * step) {
                uint32_t v[32];
                tmem_ld32(ta + (uint32_t)j0, v);
                if (a.out_f32) put32<float>(o, step, v, t.cols - j0, in);
                else if (!paired) a.fp16 ? put32<__half>(o, step, v, t.cols - j0, in) : put32<__nv_bfloat16>(o, step, v, t.cols - j0, in);
                else if (a.fp16) put32_paired<__half>(o, step, v, t.cols - j0, in, lane);
                else put32_paired<__nv_bfloat16>(o, step, v, t.cols - j0, in, lane);
            }
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(rank == 0 ? &acc_empty[b] : &acc_read[b]));
            ++c;
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    if (kPair) cluster_sync_all();  // nothing of either CTA reaches into the other any more
    tmem_fence_after_sync();
    if (warp == 1) tmem_give_back<kPair>(tbase, C::kTmemCols);
}

// The sum over slices of the weights' gradient, one after the other (the same call
// gives the same bits), rounded to the output's type.  4 values a thread.
constexpr int kJoinThreads = 256;
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kJoinThreads) k_join_slices(const float *part, int64_t count, int slices, T *out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (i >= count) return;  // (count is a multiple of 64)
    float4 v = __ldcg(reinterpret_cast<const float4 *>(part + i));
    for (int s = 1; s < slices; ++s) {
        const float4 u = __ldcg(reinterpret_cast<const float4 *>(part + s * count + i));
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    Vec<T, 4> o;
    put_pair(o, 0, f2_make(v.x, v.y)), put_pair(o, 2, f2_make(v.z, v.w));
    if (kAligned) {
        *reinterpret_cast<Vec<T, 4> *>(out + i) = o;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) out[i + k] = o.v[k];
    }
}
template <typename T>
cudaError_t join_slices(const float *part, int64_t count, int slices, void *out, cudaStream_t s) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((count / 4 + kJoinThreads - 1) / kJoinThreads)), cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
    T *const o = static_cast<T *>(out);
    return reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0
               ? cudaLaunchKernelEx(&cfg, k_join_slices<T, true>, part, count, slices, o)
               : cudaLaunchKernelEx(&cfg, k_join_slices<T, false>, part, count, slices, o);
}

// The same for a product: a block adds up 4 * kJoinThreads outputs of a row, if the
// row is an expert's; others are zeroed (zero_rest) or left.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kJoinThreads)
k_join_rows(const float *part, const int32_t *offsets, int experts, int64_t n, int F, int slices, T *out, int64_t stride, int zero_rest) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x;
    bool mine = false, wrong = false;
    int64_t s, t;
    for (int e = threadIdx.x; e < experts; e += kJoinThreads) {
        wrong |= !range_of(offsets, e, n, s, t);
        mine |= s <= row && row < t;
    }
    bool has = __syncthreads_or(mine);
    if (__syncthreads_or(wrong)) {  // (as the kernel before gave out the rows)
        mine = false;
        if (threadIdx.x == 0) {
            int64_t end = 0;
            for (int e = 0; e < experts; ++e) {
                range_of(offsets, e, n, s, t);
                if (s < t && takes_rows(s, t, end)) mine |= s <= row && row < t;
            }
        }
        has = __syncthreads_or(mine);
    }
    const int f = (blockIdx.y * kJoinThreads + threadIdx.x) * 4;
    if (f >= F) return;  // (F is a multiple of 8)
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (has) {
        for (int k = 0; k < slices; ++k) {
            const float4 u = __ldcg(reinterpret_cast<const float4 *>(part + (k * n + row) * F + f));
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
    } else if (!zero_rest) {
        return;
    }
    T *o = out + row * stride + f;
    Vec<T, 4> r;
    put_pair(r, 0, f2_make(v.x, v.y)), put_pair(r, 2, f2_make(v.z, v.w));
    if (kAligned) {
        *reinterpret_cast<Vec<T, 4> *>(o) = r;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = r.v[k];
    }
}
template <typename T>
cudaError_t join_rows(const float *part, const Args &a, int slices, void *out, int64_t stride, int zero_rest, cudaStream_t s) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.n, (unsigned)((a.F / 4 + kJoinThreads - 1) / kJoinThreads)), cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
    T *const o = static_cast<T *>(out);
    return reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0 && stride % 4 == 0
               ? cudaLaunchKernelEx(&cfg, k_join_rows<T, true>, part, a.offsets, a.experts, a.n, a.F, slices, o, stride, zero_rest)
               : cudaLaunchKernelEx(&cfg, k_join_rows<T, false>, part, a.offsets, a.experts, a.n, a.F, slices, o, stride, zero_rest);
}

// SMs of the device that the rules below share work out for.  A constant: they decide
// the room that a workspace needs and the order of sums, which must not depend on the
// device that happens to be current when they are asked.  (A device with fewer SMs, or
// fewer pairs of them that can work together, takes another round of tiles.)
constexpr int kSms = 152;
// Whether a product takes the wide tiles: from some 40 rows an expert on they are
// the faster ones (us, narrow and wide, 16 experts of 2048 x 5120: 32 rows each 56
// and 60, 48 rows 64 and 60, 128 rows 102 and 64).  The host knows the mean alone: where
// few experts have all the rows, narrow tiles read those experts' weights once per 32
// of them (64 experts of 2048 x 5120: 768 rows evenly spread 206 us, all of one expert
// 44, 22 if the call names that one alone; 2,048 rows 209, 87 and 29).
bool wide_rows(int64_t n, int experts) { return n > 32 * (int64_t)experts; }
// Narrow tiles of a product at the most: one for each 128 outputs of each expert
// with rows (and of each 32 rows of one).
int64_t narrow_tiles(int64_t n, int experts, int N) { return (int64_t)(N + kM - 1) / kM * (n < experts ? n : experts + n / 32); }
// Slices of a product's contraction: where it is of 4,096 or more and the tiles leave
// half the kSms SMs (their pairs) without work, as many as there is room for, 512 of it
// each at the least (us, with slices and without: one row of one expert, 5120 x 4096
// 12.8 and 19.1, x 8192 19.6 and 34.3, x 2048 9.7 and 11.6, which the second launch
// takes back where the host is the slower one; three rows 3776 x 5936 13.4 and 26.1;
// 512 rows 1024 x 8192 16.7 and 40.2; slices of 1,024 at the least 0 to 10 % more).
int product_slices(int64_t n, int experts, int N, int K) {
    const int64_t tiles = wide_rows(n, experts) ? (N + 255) / 256 * (experts + n / 256) : narrow_tiles(n, experts, N);
    const int64_t room = (wide_rows(n, experts) ? kSms / 2 : kSms) / (tiles > 0 ? tiles : 1), s = room < K / 512 ? room : K / 512;
    return K < 4096 || s < 2 ? 1 : (int)(s * experts <= kMaxExperts ? s : 1);
}

// Slices of an expert's rows in the weights' gradient: where the tiles are at most
// half the pairs of CTAs of kSms SMs and experts have 2,048 rows or more, as many
// slices as the pairs have room for, each of 512 rows at the least (us, with slices
// and without: one expert, 2,048 rows 256 x 256 10.6 and 14.3, 12,733 rows 216 x 16
// 14.3 and 68.8, 41,907 rows 456 x 3296 120 and 225; eight experts 512 x 512, 8,192
// rows 12.6 and 10.7, 16,384 rows 14.9 and 15.2).  This too goes by the mean: of 16
// experts' 512 x 512 one with 30,000 rows and 15 with one take 133 us, the same rows
// evenly spread 17, that expert alone, in slices, 21; of 2048 x 1024 157, 83 and 82.
int slices_of(int64_t n, int experts, int N, int K) {
    const int64_t tiles = (int64_t)experts * ((N + 255) / 256) * ((K + 255) / 256);
    const int64_t room = kSms / 2 / tiles, rows = n / experts, s = room < rows / 512 ? room : rows / 512;
    return rows < 2048 || s < 2 ? 1 : (int)s;
}

bool encode(CUtensorMap *m, const void *base, bool fp16, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    const auto enc = encoder();
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return enc && enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                      const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A tensor of 16-bit values [d2][d1][d0] (d2 = 0: two axes), rows of d1 `stride1`
// values apart, boxes of b1 x 64 values, 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap *m, const void *base, bool fp16, int64_t d0, int64_t d1, int64_t stride1, int64_t d2, int b1) {
    const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    const cuuint64_t strides[2] = {(cuuint64_t)stride1 * 2, (cuuint64_t)stride1 * (cuuint64_t)d1 * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)b1, 1};
    return encode(m, base, fp16, d2 ? 3 : 2, dims, strides, box);
}
// An MN-major operand.  With d0 a multiple of 64 (*whole) it is an axis of its own of
// chunks of 64 between d1 and d2, and one box is a stage's `chunks` tiles of 64
// values by kSub * kBK of k, one after the other; else one box is one such tile.
bool make_operand_map(CUtensorMap *m, const void *base, bool fp16, int64_t d0, int64_t d1, int64_t stride1, int64_t d2,
                      int chunks, int *whole) {
    *whole = d0 % 64 == 0;
    if (!*whole) return make_map(m, base, fp16, d0, d1, stride1, d2, kSub * kBK);
    const cuuint64_t dims[4] = {64, (cuuint64_t)d1, (cuuint64_t)d0 / 64, (cuuint64_t)d2};
    const cuuint64_t strides[3] = {(cuuint64_t)stride1 * 2, 128, (cuuint64_t)stride1 * (cuuint64_t)d1 * 2};
    const cuuint32_t box[4] = {64, kSub * kBK, (cuuint32_t)chunks, 1};
    return encode(m, base, fp16, d2 ? 4 : 3, dims, strides, box);
}

constexpr int kDevices = 64;

int sm_count() {
    static std::atomic<int> sms[kDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return kSms;
    if ((n = sms[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return kSms;
    sms[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Launches on every SM (pairs: every two SMs that can work together), once per
// kernel and device finding out how many and allowing the shared memory.
template <int BN, bool kPair, bool kDeep, bool kAMn, bool kWeights>
cudaError_t launch(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &small, const Args &a, cudaStream_t s) {
    using C = Cfg<BN, kPair, kDeep>;
    const auto k = k_grouped_mm<BN, kPair, kDeep, kAMn, kWeights>;
    static std::atomic<int> ctas[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 2, attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads), cfg.dynamicSmemBytes = C::kSmem, cfg.stream = s;
    cfg.attrs = attrs, cfg.numAttrs = kPair ? 2 : 1;
    int grid = ctas[dev].load(std::memory_order_acquire);
    if (!grid) {
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&grid, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if (kPair) {
            int clusters = 0;
            cfg.gridDim = dim3((unsigned)grid / 2 * 2);
            if ((e = cudaOccupancyMaxActiveClusters(&clusters, k, &cfg)) != cudaSuccess) return e;
            if (clusters < 1) return cudaErrorLaunchOutOfResources;
            grid = grid / 2 < clusters ? grid / 2 * 2 : clusters * 2;
        }
        grid *= C::kPerSm;
        ctas[dev].store(grid, std::memory_order_release);  // (the attribute is set for whoever reads it)
    }
    cfg.gridDim = dim3((unsigned)grid);
    return cudaLaunchKernelEx(&cfg, k, ta, tb, small, a);
}

template <int BN, bool kPair, bool kDeep>
cudaError_t product(const void *x, int64_t x_stride, const void *w, bool w_kn, Args a, int64_t n, cudaStream_t s) {
    using C = Cfg<BN, kPair, kDeep>;
    CUtensorMap ta, tb, small;
    const bool ok = (w_kn ? make_operand_map(&ta, w, a.fp16, a.F, a.K, a.F, a.experts, kM / 64, &a.a_whole)
                          : make_map(&ta, w, a.fp16, a.K, a.F, a.K, a.experts, kM)) &&
                    make_map(&tb, x, a.fp16, a.K, n, x_stride, 0, C::kOwn) &&
                    make_map(&small, x, a.fp16, a.K, n, x_stride, 0, C::kRowBox);
    if (!ok) return cudaErrorInvalidValue;
    return w_kn ? launch<BN, kPair, kDeep, true, false>(ta, tb, small, a, s)
                : launch<BN, kPair, kDeep, false, false>(ta, tb, small, a, s);
}

}  // namespace gm

cudaError_t launch_grouped_mm(const void *x, int64_t x_stride, const void *w, bool w_kn, const int32_t *offsets, int64_t n,
                              int experts, int N, int K, bool fp16, void *y, int64_t y_stride, bool y_f32,
                              bool zero_rest, void *workspace, cudaStream_t s) {
    const int slices = gm::product_slices(n, experts, N, K);
    gm::Args a{offsets, experts, slices, n, N, 0, K, y, y_stride, y_f32, fp16, zero_rest, 0, 0};
    if (slices > 1) a.out = workspace, a.out_stride = N, a.out_f32 = 1, a.zero_rest = 0;
    cudaError_t e;
    // (few rows an expert: narrow row tiles leave room for more of the weights in flight)
    if (gm::wide_rows(n, experts)) e = gm::product<256, true, false>(x, x_stride, w, w_kn, a, n, s);
    else if (slices * gm::narrow_tiles(n, experts, N) <= gm::sm_count()) e = gm::product<32, false, true>(x, x_stride, w, w_kn, a, n, s);
    else e = gm::product<32, false, false>(x, x_stride, w, w_kn, a, n, s);
    if (e != cudaSuccess || slices == 1) return e;
    const float *const part = static_cast<const float *>(workspace);
    if (y_f32) return gm::join_rows<float>(part, a, slices, y, y_stride, zero_rest, s);
    return fp16 ? gm::join_rows<__half>(part, a, slices, y, y_stride, zero_rest, s)
                : gm::join_rows<__nv_bfloat16>(part, a, slices, y, y_stride, zero_rest, s);
}

size_t grouped_mm_workspace_bytes(int64_t n, int experts, int N, int K) {
    const int slices = gm::product_slices(n, experts, N, K);
    return slices == 1 ? 0 : (size_t)slices * n * N * 4;
}

cudaError_t launch_grouped_mm_weights(const void *b, int64_t b_stride, int C, const void *am, int64_t a_stride, int F,
                                      const int32_t *offsets, int64_t n, int experts, bool fp16, void *g_w,
                                      bool g_f32, void *workspace, cudaStream_t s) {
    using Cf = gm::Cfg<256, true, false>;
    const int slices = gm::slices_of(n, experts, C, F);
    void *const out = slices > 1 ? workspace : g_w;
    CUtensorMap ta, tb, chunk;
    gm::Args a{offsets, experts, slices, n, F, C, 0, out, F, g_f32 || slices > 1, fp16, false, 0, 0};
    if (!gm::make_operand_map(&ta, am, fp16, F, n, a_stride, 0, gm::kM / 64, &a.a_whole) ||
        !gm::make_operand_map(&tb, b, fp16, C, n, b_stride, 0, Cf::kOwn / 64, &a.b_whole) ||
        !gm::make_map(&chunk, b, fp16, C, n, b_stride, 0, gm::kSub * gm::kBK))
        return cudaErrorInvalidValue;
    const cudaError_t e = gm::launch<256, true, false, true, true>(ta, tb, chunk, a, s);
    if (e != cudaSuccess || slices == 1) return e;
    const float *const part = static_cast<const float *>(workspace);
    const int64_t count = (int64_t)experts * C * F;
    if (g_f32) return gm::join_slices<float>(part, count, slices, g_w, s);
    return fp16 ? gm::join_slices<__half>(part, count, slices, g_w, s) : gm::join_slices<__nv_bfloat16>(part, count, slices, g_w, s);
}

size_t grouped_mm_weights_workspace_bytes(int64_t n, int experts, int N, int K) {
    const int slices = gm::slices_of(n, experts, N, K);
    return slices == 1 ? 0 : (size_t)slices * experts * N * K * 4;
}

cudaError_t consume_grouped_mm_device_error(cudaStream_t s, unsigned int *flag) {
    cudaError_t e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
    unsigned int v = 0;
    e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
    if (e != cudaSuccess) return e;
    *flag = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
    }
    return e;
}

}  // namespace hc
