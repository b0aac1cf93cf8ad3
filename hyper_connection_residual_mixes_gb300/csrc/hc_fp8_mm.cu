// hc_fp8_mm.cu -- the matrix product of 8-bit numbers with a scale for each block of
// 128, on the fifth-generation tensor cores of GB300.
//
//   y[m][c] = sum over blocks b of 128:  sx[m][b] sw[c / 128][b]  sum over k in b  x[m][k] w[c][k]
// (transposed: w[k][c], sw[b][c / 128]), E4M3 codes x and w, scales sx of the rows'
// blocks and sw of the matrix's 128 x 128 blocks.
//
// A block's products are summed by tcgen05.mma (kind::f8f6f4, fp32 in tensor memory);
// every block's sums are then scaled and added to fp32 accumulators in registers,
// while the next block's products run into the other half of the tensor memory.  Rows
// lie on the MMA's M side, so that a thread, which holds a row, has one scale for all
// its columns of a block of the matrix.
#include <atomic>

#include <cuda.h>

#include "hc_fp8.cuh"
#include "hc_sublayer.h"
#include "hc_types.cuh"
#include "hc_umma.cuh"

namespace hc {

namespace f8 {

constexpr int kM = 128;   // rows per CTA
constexpr int kBK = 128;  // contraction per stage: one block of scales, one 128-byte swizzled row of codes
constexpr int kGroup = 8; // tiles of rows that are walked together
constexpr int kEpilogue = 8, kThreads = 32 * (kEpilogue + 4);  // (whole groups of four warps: registers are moved between these)
// Registers a thread: what a block of kThreads is launched with, and of that what the
// writing warps take (128 accumulators at BN = 256) and the others keep.
constexpr int kRegs = 168, kRegsWriting = 216, kRegsOther = 72;
static_assert(kEpilogue * kRegsWriting + 4 * kRegsOther <= (kEpilogue + 4) * kRegs, "the block's registers");

template <int BN, bool kPair>
struct Cfg {
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kTileM = kM * kCtas;
    static constexpr int kOwn = BN / kCtas;  // columns whose codes a CTA holds
    static constexpr int kABytes = kM * kBK, kBBytes = kOwn * kBK, kStage = kABytes + kBBytes;
    static constexpr int kStages = 6;
    static constexpr int kTmemCols = 2 * BN;
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr bool kMoved = BN == 256;  // registers are moved to the writing warps
    static_assert(kOwn == 128 && kSmem + 1024 <= 227 * 1024 && kTmemCols <= 512, "an SM's memory");
};

struct Args {
    Fp8Scales sx, sw;
    int64_t sw_col, sw_k;  // between scales of w for consecutive blocks of columns, of the contraction
    int64_t M;
    int C, L;              // columns of the output, length of the contraction
    void *y;
    int64_t ys;
    int y_type, y_wide;    // y_wide: rows take 16-byte stores
};

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major: rows of 128 codes, 8-row
// groups 1024 bytes apart, an MMA's 32 of k = 32 bytes.  MN-major: a row of 128 columns
// per k, 8 k = 1024 bytes, an MMA's 32 of k = 4096 bytes.
__device__ __forceinline__ uint64_t desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ constexpr uint32_t idesc(bool b_mn, int m, int n) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// The four MMAs of a block, operands kStepA and kStepB (in descriptor units) apart, the
// first one overwriting what tensor memory held; one election.
template <bool kPair, uint32_t kStepA, uint32_t kStepB>
__device__ __forceinline__ void umma_block(uint32_t d, uint64_t a0, uint64_t b0, uint32_t id) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, %4;\n\tadd.s64 b, %2, %5;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %4;\n\tadd.s64 b, b, %5;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %4;\n\tadd.s64 b, b, %5;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, t;\n\t}" ::"r"(d), "l"(a0), "l"(b0), "r"(id), "n"(kStepA), "n"(kStepB)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, %4;\n\tadd.s64 b, %2, %5;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %4;\n\tadd.s64 b, b, %5;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
            "add.s64 a, a, %4;\n\tadd.s64 b, b, %5;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t}" ::"r"(d), "l"(a0), "l"(b0), "r"(id), "n"(kStepA), "n"(kStepB)
            : "memory");
}

// 64 columns of this lane in pairs, waited for in the same statement (no register copy can
// slip between the loads and the wait).
__device__ __forceinline__ void tmem_ld64(uint32_t t, f32x2 (&v)[32]) {
    asm volatile(
        "{\n\t.reg .b32 r<64>;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {r0, r1, r2, r3, r4, r5, r6, r7, r8, r9, r10, r11, r12, r13, r14, r15, r16, r17, r18, r19, r20, r21, r22, r23, r24, r25, r26, r27, r28, r29, r30, r31, r32, r33, r34, r35, r36, r37, r38, r39, r40, r41, r42, r43, r44, r45, r46, r47, r48, r49, r50, r51, r52, r53, r54, r55, r56, r57, r58, r59, r60, r61, r62, r63}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "mov.b64 %0, {r0, r1};\n\tmov.b64 %1, {r2, r3};\n\tmov.b64 %2, {r4, r5};\n\tmov.b64 %3, {r6, r7};\n\tmov.b64 %4, {r8, r9};\n\tmov.b64 %5, {r10, r11};\n\tmov.b64 %6, {r12, r13};\n\tmov.b64 %7, {r14, r15};\n\tmov.b64 %8, {r16, r17};\n\tmov.b64 %9, {r18, r19};\n\tmov.b64 %10, {r20, r21};\n\tmov.b64 %11, {r22, r23};\n\tmov.b64 %12, {r24, r25};\n\tmov.b64 %13, {r26, r27};\n\tmov.b64 %14, {r28, r29};\n\tmov.b64 %15, {r30, r31};\n\tmov.b64 %16, {r32, r33};\n\tmov.b64 %17, {r34, r35};\n\tmov.b64 %18, {r36, r37};\n\tmov.b64 %19, {r38, r39};\n\tmov.b64 %20, {r40, r41};\n\tmov.b64 %21, {r42, r43};\n\tmov.b64 %22, {r44, r45};\n\tmov.b64 %23, {r46, r47};\n\tmov.b64 %24, {r48, r49};\n\tmov.b64 %25, {r50, r51};\n\tmov.b64 %26, {r52, r53};\n\tmov.b64 %27, {r54, r55};\n\tmov.b64 %28, {r56, r57};\n\tmov.b64 %29, {r58, r59};\n\tmov.b64 %30, {r60, r61};\n\tmov.b64 %31, {r62, r63};\n\t}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]), "=l"(v[12]), "=l"(v[13]), "=l"(v[14]), "=l"(v[15]), "=l"(v[16]), "=l"(v[17]), "=l"(v[18]), "=l"(v[19]), "=l"(v[20]), "=l"(v[21]), "=l"(v[22]), "=l"(v[23]), "=l"(v[24]), "=l"(v[25]), "=l"(v[26]), "=l"(v[27]), "=l"(v[28]), "=l"(v[29]), "=l"(v[30]), "=l"(v[31])
        : "r"(t)
        : "memory");
}

// 8 consecutive columns of a row
template <typename T>
__device__ __forceinline__ void put8(T *o, const f32x2 *v, int wide) {
    Vec<T, 8> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) put_pair(r, 2 * k, v[k]);
    if (wide) {
        constexpr int kParts = (int)sizeof(T) * 8 / 16;
        const Words<T, 8> &u = reinterpret_cast<const Words<T, 8> &>(r);
#pragma unroll
        for (int k = 0; k < kParts; ++k)
            reinterpret_cast<uint4 *>(o)[k] = make_uint4(u.w[4 * k], u.w[4 * k + 1], u.w[4 * k + 2], u.w[4 * k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = r.v[k];
    }
}
template <int NP>
__device__ __forceinline__ void put_row(const Args &a, int64_t row, int c, const f32x2 (&acc)[NP]) {
    if (row >= a.M) return;
#pragma unroll
    for (int j = 0; j < NP; j += 4) {
        if (c + 2 * j >= a.C) return;  // (C is a multiple of 16)
        const int64_t at = row * a.ys + c + 2 * j;
        if (a.y_type == HC_F32) put8(static_cast<float *>(a.y) + at, acc + j, a.y_wide);
        else if (a.y_type == HC_BF16) put8(static_cast<__nv_bfloat16 *>(a.y) + at, acc + j, a.y_wide);
        else put8(static_cast<__half *>(a.y) + at, acc + j, a.y_wide);
    }
}

// Tiles are walked in groups of kGroup tiles of rows, through all columns before the
// next group: what the CTAs read at one time is then about as wide as long.
__device__ __forceinline__ void place_of(int tile, int mt, int ct, int &m, int &c) {
    const int g = tile / (kGroup * ct), rest = tile - g * (kGroup * ct);
    const int w = mt - g * kGroup < kGroup ? mt - g * kGroup : kGroup;
    c = rest / w;
    m = g * kGroup + rest - c * w;
}

// kMn: w lies MN-major (transposed).  Of a pair the first CTA issues the MMAs; its
// barriers collect both CTAs' loads and both epilogues' arrivals; commits arrive at both.
template <int BN, bool kPair, bool kMn>
__global__ void __launch_bounds__(kThreads, 1)
k_fp8_mm(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Args a) {
    using C = Cfg<BN, kPair>;
    constexpr int S = C::kStages, NP = BN / 4;  // pairs of columns a writing thread holds
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t full_bar[S], empty_bar[S], acc_full[2], acc_empty[2], acc_read[2], done_bar;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kPair ? (int)cluster_ctarank() : 0;
    const int worker = kPair ? (int)blockIdx.x >> 1 : (int)blockIdx.x, workers = kPair ? (int)gridDim.x >> 1 : (int)gridDim.x;
    const int mt = (int)((a.M + C::kTileM - 1) / C::kTileM), ct = (a.C + BN - 1) / BN, tiles = mt * ct;
    const int blocks = (a.L + kBK - 1) / kBK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full_bar[s]), C::kCtas), mbar_init(smem_u32(&empty_bar[s]), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), kEpilogue + (kPair ? 1 : 0));
            mbar_init(smem_u32(&acc_read[b]), kEpilogue);
        }
        mbar_init(smem_u32(&done_bar), 1);
        s_abort = 0;
        fence_mbar_init_cluster();
    }
    if (warp == kEpilogue + 1) tmem_get<kPair>(smem_u32(&s_tmem), C::kTmemCols);
    tmem_fence_before_sync();
    __syncthreads();
    if (kPair) cluster_sync_all();  // the other CTA's barriers and tensor memory are ready
    tmem_fence_after_sync();
    const uint32_t tbase = s_tmem;
    // (launched before the kernel in front of it has ended: from here on its results are read)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp >= kEpilogue) {
        if constexpr (C::kMoved) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kEpilogue) {
            if (lane == 0) prefetch_tmap(&tm_x), prefetch_tmap(&tm_w);
            __syncwarp();
            const uint64_t pol = policy_evict_last();
            int slot = 0, issued = 0;
            uint32_t parity = 1;
            bool ok = true;
            for (int tile = worker; tile < tiles && ok; tile += workers) {
                int m, c;
                place_of(tile, mt, ct, m, c);
                m = __shfl_sync(0xffffffffu, m * C::kTileM + rank * kM, 0), c = __shfl_sync(0xffffffffu, c * BN + rank * C::kOwn, 0);
                for (int i = 0; i < blocks; ++i) {
                    if (!(ok = mbar_wait_warp<false>(smem_u32(&empty_bar[slot]), parity, &s_abort))) break;
                    const uint32_t sa = sbase + (uint32_t)slot * C::kStage;
                    uint32_t bar = smem_u32(&full_bar[slot]);
                    if (rank == 0) {
                        expect_bytes(bar, C::kCtas * C::kStage);  // of a pair both CTAs' bytes
                    } else {
                        bar = mapa(bar, 0);
                        arrive_remote_relaxed(bar);
                    }
                    ++issued;
                    load_2d<kPair>(sa, &tm_x, bar, i * kBK, m, pol);
                    if (kMn) load_2d<kPair>(sa + C::kABytes, &tm_w, bar, c, i * kBK, pol);
                    else load_2d<kPair>(sa + C::kABytes, &tm_w, bar, i * kBK, c, pol);
                    if (++slot == S) slot = 0, parity ^= 1u;
                }
            }
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            // the last stages issued must land before the CTA leaves (of a pair, the second
            // CTA's have when the MMAs have read them: its empty barriers say so)
            for (int k = 0; k < S && k < issued; ++k) {
                if (--slot < 0) slot = S - 1, parity ^= 1u;
                if (rank == 0) wait_exit(smem_u32(&full_bar[slot]), parity ^ 1u);
                else wait_exit(smem_u32(&empty_bar[slot]), parity ^ 1u);
            }
            __syncwarp();
        } else if (warp == kEpilogue + 1 && rank == 0) {
            int slot = 0;
            uint32_t parity = 0, use = 0;
            bool ok = true;
            const uint64_t da0 = desc(sbase), db0 = desc(sbase + C::kABytes);
            constexpr uint32_t kStepA = 32 >> 4, kStepB = (kMn ? 4096 : 32) >> 4, id = idesc(kMn, C::kTileM, BN);
            for (int tile = worker; tile < tiles && ok; tile += workers) {
                for (int i = 0; i < blocks; ++i, ++use) {
                    const uint32_t b = use & 1u;
                    // (what the other CTA passes on is that its loads from tensor memory have completed; no
                    // memory is handed over, so nothing is to be acquired from the cluster, block for block)
                    if (!(ok = mbar_wait_warp<false>(smem_u32(&acc_empty[b]), (use >> 1 & 1u) ^ 1u, &s_abort))) break;
                    if (!(ok = mbar_wait_warp<false>(smem_u32(&full_bar[slot]), parity, &s_abort))) break;
                    tmem_fence_after_sync();
                    const uint32_t at = (uint32_t)(slot * C::kStage) / 16;
                    umma_block<kPair, kStepA, kStepB>(tbase + b * BN, da0 + at, db0 + at, id);
                    umma_commit<kPair>(smem_u32(&empty_bar[slot]));
                    umma_commit<kPair>(smem_u32(&acc_full[b]));
                    if (++slot == S) slot = 0, parity ^= 1u;
                }
            }
            // every MMA issued has completed before the tensor memory is freed
            umma_commit<kPair>(smem_u32(&done_bar));
            wait_exit(smem_u32(&done_bar), 0u);
            __syncwarp();
        } else if (warp == kEpilogue + 1) {
            // The second CTA of a pair passes on that its accumulators have been read.  (From a warp of its
            // own and without a release: that would wait for what the writing warps have stored.)
            uint32_t use = 0;
            bool ok = true;
            for (int tile = worker; tile < tiles && ok; tile += workers) {
                for (int i = 0; i < blocks; ++i, ++use) {
                    const uint32_t b = use & 1u;
                    if (!(ok = mbar_wait_warp<false>(smem_u32(&acc_read[b]), use >> 1 & 1u, &s_abort))) break;
                    arrive_remote_relaxed(mapa(smem_u32(&acc_empty[b]), 0));
                }
            }
        }
    } else {
        if constexpr (C::kMoved) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWriting));
        const int q = warp & 3, half = warp >> 2;  // the warp's quadrant of tensor-memory lanes; which of its two
        uint32_t use = 0;
        bool ok = true;
        for (int tile = worker; tile < tiles && ok; tile += workers) {
            int m, c;
            place_of(tile, mt, ct, m, c);
            const int64_t row = (int64_t)m * C::kTileM + rank * kM + q * 32 + lane;
            const int c0 = c * BN + half * (BN / 2);
            // (rows and columns that are not there take a scale that is)
            const int64_t x_at = (row < a.M ? row : a.M - 1) * blocks;
            const int64_t w_at = (c0 < a.C ? c0 : a.C - 1) / kFp8Block * a.sw_col;
            uint32_t next_x = a.sx.raw(x_at), next_w = a.sw.raw(w_at);
            f32x2 acc[NP];
#pragma unroll
            for (int j = 0; j < NP; ++j) acc[j] = f2_dup(0.0f);
            for (int i = 0; i < blocks; ++i, ++use) {
                const uint32_t b = use & 1u;
                const f32x2 s = f2_dup(a.sx.value(next_x) * a.sw.value(next_w));
                if (i + 1 < blocks) next_x = a.sx.raw(x_at + i + 1), next_w = a.sw.raw(w_at + (i + 1) * a.sw_k);
                if (!(ok = mbar_wait_warp<false>(smem_u32(&acc_full[b]), use >> 1 & 1u, &s_abort))) break;
                tmem_fence_after_sync();
                const uint32_t ta = tbase + b * BN + (uint32_t)(half * (BN / 2)) + ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int j = 0; j < NP / 32; ++j) {
                    f32x2 v[32];
                    tmem_ld64(ta + 64 * j, v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) acc[32 * j + k] = f2_fma(v[k], s, acc[32 * j + k]);
                }
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(rank == 0 ? &acc_empty[b] : &acc_read[b]));
            }
            if (ok) put_row<NP>(a, row, c0, acc);
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    if (kPair) cluster_sync_all();  // nothing of either CTA reaches into the other any more
    tmem_fence_after_sync();
    if (warp == kEpilogue + 1) tmem_give_back<kPair>(tbase, C::kTmemCols);
}

// A matrix of codes [rows][width], rows `stride` bytes apart, boxes of 128 x 128, 128-byte
// swizzle, zeros outside.
bool make_map(CUtensorMap *m, const void *base, int64_t width, int64_t rows, int64_t stride) {
    const auto enc = encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {kBK, 128}, one[2] = {1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, one,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kDevices = 64;

// Launches on every SM (pairs: every two SMs that can work together), once per
// kernel and device finding out how many and allowing the shared memory.
template <int BN, bool kPair, bool kMn>
cudaError_t launch(const CUtensorMap &tx, const CUtensorMap &tw, const Args &a, cudaStream_t s) {
    using C = Cfg<BN, kPair>;
    const auto k = k_fp8_mm<BN, kPair, kMn>;
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
        cudaFuncAttributes is{};
        if ((e = cudaFuncGetAttributes(&is, k)) != cudaSuccess) return e;
        if (C::kMoved && is.numRegs != kRegs) return cudaErrorInvalidKernelImage;  // (the split would wait forever)
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&grid, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if (kPair) {
            int clusters = 0;
            cfg.gridDim = dim3((unsigned)grid / 2 * 2);
            if ((e = cudaOccupancyMaxActiveClusters(&clusters, k, &cfg)) != cudaSuccess) return e;
            if (clusters < 1) return cudaErrorLaunchOutOfResources;
            grid = grid / 2 < clusters ? grid / 2 * 2 : clusters * 2;
        }
        ctas[dev].store(grid, std::memory_order_release);  // (the attribute is set for whoever reads it)
    }
    const int64_t tiles = (a.M + C::kTileM - 1) / C::kTileM * ((a.C + BN - 1) / BN) * C::kCtas;
    cfg.gridDim = dim3((unsigned)(tiles < grid ? tiles : grid));
    return cudaLaunchKernelEx(&cfg, k, tx, tw, a);
}

}  // namespace f8

cudaError_t launch_fp8_mm(const uint8_t *x, int64_t x_stride, const void *x_scales, bool x_f32, const uint8_t *w,
                          const void *w_scales, bool w_f32, bool transposed, int64_t M, int N, int K, void *y, int64_t y_stride,
                          hc_dtype y_type, void *workspace, cudaStream_t s) {
    (void)workspace;
    const int C = transposed ? K : N, L = transposed ? N : K;
    const int64_t row = (K + kFp8Block - 1) / kFp8Block;  // scales of w in a row of blocks
    const int64_t size = y_type == HC_F32 ? 4 : 2;
    const f8::Args a{{x_scales, x_f32}, {w_scales, w_f32}, transposed ? 1 : row, transposed ? row : 1, M, C, L, y, y_stride,
                     y_type, reinterpret_cast<uintptr_t>(y) % 16 == 0 && y_stride * size % 16 == 0};
    CUtensorMap tx, tw;
    if (!f8::make_map(&tx, x, L, M, x_stride) || !f8::make_map(&tw, w, K, N, K)) return cudaErrorInvalidValue;
    const bool large = ((M + 255) / 256) * ((C + 255) / 256) > 38;
    if (large) return transposed ? f8::launch<256, true, true>(tx, tw, a, s) : f8::launch<256, true, false>(tx, tw, a, s);
    return transposed ? f8::launch<128, false, true>(tx, tw, a, s) : f8::launch<128, false, false>(tx, tw, a, s);
}

size_t fp8_mm_workspace_bytes(bool transposed, int64_t M, int N, int K) {
    (void)transposed, (void)M, (void)N, (void)K;
    return 0;
}

cudaError_t consume_fp8_mm_device_error(cudaStream_t s, unsigned int *flag) {
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
