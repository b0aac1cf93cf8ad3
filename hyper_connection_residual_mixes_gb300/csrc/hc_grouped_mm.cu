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
// One CTA per SM walks the tiles (warp 0 loads by TMA, warp 1 issues
// tcgen05.mma, warps 2-5 write finished tiles); two accumulators alternate, so
// that a tile is written while the next one's products run.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "hc_ptx.cuh"
#include "hc_sublayer.h"

namespace hc {

namespace gm {

constexpr int kM = 128;       // f per tile
constexpr int kBK = 64;       // k per stage: one 128-byte swizzled row of 16-bit values
constexpr int kRowBox = 32;   // rows of a K-major B box
constexpr int kThreads = 192;
constexpr int kMaxExperts = 1024;
constexpr unsigned int kErrOffsets = 2u;  // device error bit: offsets out of order or out of range

template <int BN>
struct Cfg {
    static constexpr int kABytes = kM * kBK * 2, kBBytes = BN * kBK * 2, kStage = kABytes + kBBytes;
    static constexpr int kStages = BN >= 256 ? 4 : BN >= 128 ? 6 : BN >= 64 ? 8 : 10;
    static constexpr int kTmemCols = 2 * BN;
    static constexpr int kSmem = kStages * kStage + 1024 + 3 * (kMaxExperts + 1) * 4;
    static_assert(kSmem <= 227 * 1024 - 512, "shared memory");
};

struct Args {
    const int32_t *offsets;
    int experts;
    int64_t n;          // rows of the row operands
    int F, C, K;        // product: F outputs, K contraction; weights': F x C outputs
    void *out;
    int64_t out_stride; // between consecutive c (product: rows of y; weights': rows of g_w[e])
    int out_f32, fp16, zero_rest;
};

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major: rows of 128
// bytes (64 k), 8-row groups 1024 bytes apart, 16 k = 32 bytes.  MN-major: rows of
// 128 bytes (64 f or c) per k, 8 k = 1024 bytes, the next 64 f or c `chunk`
// bytes on, 16 k = 2048 bytes.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, bool mn_major) {
    const uint64_t chunk = mn_major ? (kBK * 128) >> 4 : 1;
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (chunk << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint32_t idesc(bool fp16, bool a_mn, bool b_mn, int n) {
    const uint32_t t = fp16 ? 0u : 1u;
    return (1u << 4) | (t << 7) | (t << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
}
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(id),
        "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, uint32_t bar, int c0, int c1, int c2,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}
// 16 columns of this lane, waited for in the same statement (no register copy
// can slip between the load and the wait).
__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(t)
        : "memory");
}
// On the way out: copies and MMAs already issued must land before the CTA
// leaves, whatever the abort flag says.
__device__ __forceinline__ void wait_exit(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        if (mbar_try_wait(bar, parity)) return;
        __nanosleep(128);
    }
    atomicOr(&g_device_error, kErrWaitTimeout);
}

__device__ __forceinline__ void put(void *out, int64_t i, float v, int f32, int fp16) {
    if (f32) static_cast<float *>(out)[i] = v;
    else if (fp16) static_cast<__half *>(out)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
}

// The experts' row ranges and tiles, in shared memory.
struct Plan {
    const int *start, *end, *first;  // rows of expert e; its first tile (first[experts]: all tiles)
};
struct Tile {
    int e, f0, c0, cols;  // cols: columns of the tile that count (rows of the product)
    int k0, klen;         // contraction: rows [k0, k0 + klen) of the weights', [0, K) of the product
};
template <int BN, bool kWeights>
__device__ __forceinline__ Tile tile_of(const Args &a, const Plan &p, int tile, int &e) {
    while (tile >= p.first[e + 1]) ++e;
    const int local = tile - p.first[e];
    const int rows = p.end[e] - p.start[e];
    Tile t;
    t.e = e;
    if (kWeights) {
        const int nc = (a.C + BN - 1) / BN;
        t.f0 = local / nc * kM;
        t.c0 = local % nc * BN;
        t.cols = a.C - t.c0 < BN ? a.C - t.c0 : BN;
        t.k0 = p.start[e];
        t.klen = rows;
    } else {
        const int nt = (rows + BN - 1) / BN;
        const int per = ((rows + nt - 1) / nt + 15) / 16 * 16;
        t.f0 = local / nt * kM;
        const int at = local % nt * per;
        t.c0 = p.start[e] + at;
        t.cols = rows - at < per ? rows - at : per;
        t.k0 = 0;
        t.klen = a.K;
    }
    return t;
}

// kAMn: the M side's operand lies MN-major in global memory (w[e][k][f], or the
// rows of the weights' gradient); kWeights: the weights' gradient (B is MN-major too).
template <int BN, bool kAMn, bool kWeights>
__global__ void __launch_bounds__(kThreads, 1)
k_grouped_mm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Args a) {
    using C = Cfg<BN>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int *const s_start = reinterpret_cast<int *>(smem_raw + (sbase - smem_u32(smem_raw)) + S * C::kStage);
    int *const s_end = s_start + kMaxExperts, *const s_first = s_end + kMaxExperts;
    __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], acc_full[2], acc_empty[2], done_bar;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full_bar[s]), 1), mbar_init(smem_u32(&empty_bar[s]), 1);
        for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&acc_full[b]), 1), mbar_init(smem_u32(&acc_empty[b]), 4);
        mbar_init(smem_u32(&done_bar), 1);
        s_abort = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), C::kTmemCols);
        tmem_relinquish();
    }
    // every expert's rows and how many tiles they make; a range that is out of
    // order or out of the rows counts as empty and is reported
    for (int e = threadIdx.x; e < a.experts; e += kThreads) {
        int64_t s = __ldg(a.offsets + e), t = __ldg(a.offsets + e + 1);
        if (s < 0 || t < s || t > a.n) {
            if (blockIdx.x == 0) atomicOr(&g_device_error, kErrOffsets);
            s = t = 0;
        }
        s_start[e] = (int)s, s_end[e] = (int)t;
        const int mt = (a.F + kM - 1) / kM;
        s_first[e + 1] = kWeights ? mt * ((a.C + BN - 1) / BN) : mt * (int)((t - s + BN - 1) / BN);
    }
    __syncthreads();
    if (warp == 0) {  // running sum of the tile counts
        int carry = 0;
        if (lane == 0) s_first[0] = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            int v = e0 + lane < a.experts ? s_first[e0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (e0 + lane < a.experts) s_first[e0 + lane + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tbase = s_tmem;
    const Plan plan{s_start, s_end, s_first};
    const int tiles = s_first[a.experts];
    int e = 0;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&tm_a);
            prefetch_tmap(&tm_b);
            const uint64_t pol = policy_evict_normal();
            int it = 0;
            for (int tile = blockIdx.x; tile < tiles && !s_abort; tile += gridDim.x) {
                const Tile t = tile_of<BN, kWeights>(a, plan, tile, e);
                const int nkb = (t.klen + kBK - 1) / kBK;
                const int boxes = kWeights ? (t.cols + 63) / 64 : (t.cols + kRowBox - 1) / kRowBox;
                constexpr int kBox = kWeights ? 64 * kBK * 2 : kRowBox * kBK * 2;
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int slot = it % S;
                    if (!mbar_wait<false>(smem_u32(&empty_bar[slot]), ((uint32_t)(it / S) & 1u) ^ 1u, &s_abort)) break;
                    const uint32_t sa = sbase + (uint32_t)slot * C::kStage, sb = sa + C::kABytes;
                    const uint32_t bar = smem_u32(&full_bar[slot]);
                    mbar_arrive_expect_tx(bar, (uint32_t)(C::kABytes + boxes * kBox));
                    const int k = t.k0 + kb * kBK;
                    if (kWeights) {
                        tma_load_2d(sa, &tm_a, bar, t.f0, k, pol);
                        tma_load_2d(sa + 64 * kBK * 2, &tm_a, bar, t.f0 + 64, k, pol);
                        for (int i = 0; i < boxes; ++i) tma_load_2d(sb + i * kBox, &tm_b, bar, t.c0 + i * 64, k, pol);
                    } else {
                        if (kAMn) {
                            tma_load_3d(sa, &tm_a, bar, t.f0, k, t.e, pol);
                            tma_load_3d(sa + 64 * kBK * 2, &tm_a, bar, t.f0 + 64, k, t.e, pol);
                        } else {
                            tma_load_3d(sa, &tm_a, bar, k, t.f0, t.e, pol);
                        }
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(sb + i * kBox, &tm_b, bar, k, t.c0 + i * kRowBox, pol);
                    }
                }
            }
            // the last stages issued must land before the CTA leaves
            for (int k = (it > S ? it - S : 0); k < it; ++k)
                wait_exit(smem_u32(&full_bar[k % S]), (uint32_t)(k / S) & 1u);
        }
    } else if (warp == 1) {
        int it = 0, c = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            const Tile t = tile_of<BN, kWeights>(a, plan, tile, e);
            if (t.klen == 0) continue;  // an expert without rows: its gradient is zero
            const int b = c & 1;
            if (!(ok = mbar_wait_warp<false>(smem_u32(&acc_empty[b]), ((uint32_t)(c >> 1) & 1u) ^ 1u, &s_abort))) break;
            tmem_fence_after_sync();
            const uint32_t d = tbase + (uint32_t)(b * BN);
            const uint32_t id = idesc(a.fp16, kAMn || kWeights, kWeights, (t.cols + 15) / 16 * 16);
            const int nkb = (t.klen + kBK - 1) / kBK;
            for (int kb = 0; kb < nkb; ++kb, ++it) {
                const int slot = it % S;
                if (!(ok = mbar_wait_warp<false>(smem_u32(&full_bar[slot]), (uint32_t)(it / S) & 1u, &s_abort))) break;
                const uint32_t sa = sbase + (uint32_t)slot * C::kStage, sb = sa + C::kABytes;
                const int left = t.klen - kb * kBK, steps = left >= kBK ? kBK / 16 : (left + 15) / 16;
                if (kWeights && left < steps * 16) {
                    // rows behind the expert's last, up to the next 16: another expert's (or
                    // anything), made zero in both operands before the MMA reads them
                    const int rest = steps * 16 - left, chunks = 2 + (t.cols + 63) / 64;
                    for (int i = lane; i < chunks * rest * 8; i += 32) {
                        const int ch = i / (rest * 8), r = left + i % (rest * 8) / 8;
                        const uint32_t p = sa + (uint32_t)(ch * 64 * kBK * 2 + r * 128 + (i & 7) * 16);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(p), "r"(0) : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tmem_fence_after_sync();
                if (lane == 0) {
                    for (int ks = 0; ks < steps; ++ks)
                        umma(d, desc(sa + (uint32_t)ks * (kAMn || kWeights ? 2048 : 32), kAMn || kWeights),
                             desc(sb + (uint32_t)ks * (kWeights ? 2048 : 32), kWeights), id, kb > 0 || ks > 0);
                    umma_commit(smem_u32(&empty_bar[slot]));
                }
                __syncwarp();
            }
            if (ok && lane == 0) umma_commit(smem_u32(&acc_full[b]));
            ++c;
        }
        // every MMA issued has completed before the tensor memory is freed
        if (lane == 0) {
            umma_commit(smem_u32(&done_bar));
            wait_exit(smem_u32(&done_bar), 0u);
        }
        __syncwarp();
    } else {
        const int q = warp & 3;  // the warp's quadrant of tensor-memory lanes
        const int64_t esize = a.out_f32 ? 4 : 2;
        if (!kWeights && a.zero_rest) {
            // rows of no expert: before offsets[0] and from offsets[experts] on
            int64_t lo = __ldg(a.offsets), hi = __ldg(a.offsets + a.experts);
            lo = lo < 0 ? 0 : lo > a.n ? a.n : lo;
            hi = hi < lo ? lo : hi > a.n ? a.n : hi;
            for (int64_t r = blockIdx.x; r < lo + (a.n - hi); r += gridDim.x) {
                const int64_t row = r < lo ? r : hi + (r - lo);
                for (int f = threadIdx.x - 64; f < a.F; f += 128) put(a.out, row * a.out_stride + f, 0.0f, a.out_f32, a.fp16);
            }
        }
        int c = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const Tile t = tile_of<BN, kWeights>(a, plan, tile, e);
            const int f = t.f0 + q * 32 + lane;
            uint8_t *o = static_cast<uint8_t *>(a.out) +
                         ((kWeights ? (int64_t)t.e * a.C + t.c0 : (int64_t)t.c0) * a.out_stride + f) * esize;
            const int64_t step = a.out_stride * esize;
            const bool in = f < a.F;
            if (t.klen == 0) {
                for (int j = 0; j < t.cols; ++j, o += step)
                    if (in) put(o, 0, 0.0f, a.out_f32, a.fp16);
                continue;
            }
            const int b = c & 1;
            if (!mbar_wait_warp<false>(smem_u32(&acc_full[b]), (uint32_t)(c >> 1) & 1u, &s_abort)) break;
            tmem_fence_after_sync();
            const uint32_t ta = tbase + (uint32_t)(b * BN) + ((uint32_t)(32 * q) << 16);
            for (int j0 = 0; j0 < t.cols; j0 += 16) {
                uint32_t v[16];
                tmem_ld16(ta + (uint32_t)j0, v);
#pragma unroll
                for (int j = 0; j < 16; ++j, o += step)
                    if (in && j0 + j < t.cols) put(o, 0, __uint_as_float(v[j]), a.out_f32, a.fp16);
            }
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&acc_empty[b]));
            ++c;
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (warp == 1) tmem_dealloc(tbase, C::kTmemCols);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
            qr != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A tensor of 16-bit values [d2][d1][d0] (d2 = 0: two axes), rows of d1 `stride1`
// values apart, boxes of b1 x 64 values, 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap *m, const void *base, bool fp16, int64_t d0, int64_t d1, int64_t stride1, int64_t d2, int b1) {
    const auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    cuuint64_t strides[2] = {(cuuint64_t)stride1 * 2, (cuuint64_t)stride1 * (cuuint64_t)d1 * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)b1, 1}, one[3] = {1, 1, 1};
    return enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 ? 3 : 2,
               const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 148;
    return sms;
}

template <int BN, bool kAMn, bool kWeights>
cudaError_t launch(const CUtensorMap &ta, const CUtensorMap &tb, const Args &a, cudaStream_t s) {
    const auto k = k_grouped_mm<BN, kAMn, kWeights>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN>::kSmem);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)sm_count(), kThreads, Cfg<BN>::kSmem, s>>>(ta, tb, a);
    return cudaGetLastError();
}

}  // namespace gm

cudaError_t launch_grouped_mm(const void *x, int64_t x_stride, const void *w, bool w_kn, const int32_t *offsets, int64_t n,
                              int experts, int N, int K, bool fp16, void *y, int64_t y_stride, bool y_f32,
                              bool zero_rest, cudaStream_t s) {
    CUtensorMap ta, tb;
    const bool ok = (w_kn ? gm::make_map(&ta, w, fp16, N, K, N, experts, gm::kBK)
                          : gm::make_map(&ta, w, fp16, K, N, K, experts, gm::kM)) &&
                    gm::make_map(&tb, x, fp16, K, n, x_stride, 0, gm::kRowBox);
    if (!ok) return cudaErrorInvalidValue;
    const gm::Args a{offsets, experts, n, N, 0, K, y, y_stride, y_f32, fp16, zero_rest};
    // Few rows an expert: narrow row tiles leave room for more stages of weights in flight.
    if (n <= 32 * (int64_t)experts)
        return w_kn ? gm::launch<32, true, false>(ta, tb, a, s) : gm::launch<32, false, false>(ta, tb, a, s);
    return w_kn ? gm::launch<256, true, false>(ta, tb, a, s) : gm::launch<256, false, false>(ta, tb, a, s);
}

cudaError_t launch_grouped_mm_weights(const void *b, int64_t b_stride, int C, const void *am, int64_t a_stride, int F,
                                      const int32_t *offsets, int64_t n, int experts, bool fp16, void *g_w,
                                      bool g_f32, cudaStream_t s) {
    CUtensorMap ta, tb;
    if (!gm::make_map(&ta, am, fp16, F, n, a_stride, 0, gm::kBK) || !gm::make_map(&tb, b, fp16, C, n, b_stride, 0, gm::kBK))
        return cudaErrorInvalidValue;
    const gm::Args a{offsets, experts, n, F, C, 0, g_w, F, g_f32, fp16, false};
    return gm::launch<256, true, true>(ta, tb, a, s);
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
