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
//
// What bounds it: a block of 128 x 256 x 128 takes the tensor cores 512 cycles, but 1,050
// pass, in which the eight writing warps load 32,768 sums from tensor memory and add each to its
// accumulator (a packed FMA for two), on the same issue slots as all else.  16,384 x
// 10,240 x 5,120: 750 to 795 us, by the board's clocks, 2.16 to 2.29 PFLOP/s.  What other shapes of the same took beside 750, in us:
// pairs of CTAs on 256 x 256 787 (1,187 with a releasing arrival at the other CTA for each block), 128 x 128
// tiles 1,022 in four parts of columns, three issuing warps in turn 753, the next sums loaded
// between the FMAs of the last 772, MMAs held back to even the issue 768 and more.
// Small products are cut to fill the SMs (cut), up to 16 rows stream the matrix past mma.sync
// (k_fp8_few: 16 x 16,384 x 5,120 in 20 us, 0.62 of the copy rate, 1 x 512 x 1,024 in 3.1).
#include <algorithm>
#include <atomic>

#include <cuda.h>

#include "hc_fp8.cuh"
#include "hc_pieces.cuh"
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
// writing warps take (128 accumulators and 64 loaded sums at BN = 256) and the others keep.
constexpr int kRegs = 168, kRegsWriting = 216, kRegsOther = 72;
static_assert(kEpilogue * kRegsWriting + 4 * kRegsOther <= (kEpilogue + 4) * kRegs, "the block's registers");

template <int BN>
struct Cfg {
    static constexpr int kABytes = kM * kBK, kBBytes = BN * kBK, kStage = kABytes + kBBytes;
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr int kTmemCols = 2 * BN;  // two blocks' sums
    static constexpr int kSmem = kStages * kStage + 1024;
    static constexpr bool kMoved = BN == 256;  // registers are moved to the writing warps
    static_assert(BN % 128 == 0 && kSmem + 1024 <= 227 * 1024 && kTmemCols <= 512, "an SM's memory");
};

struct Args {
    Fp8Scales sx, sw;
    int64_t sw_col, sw_k;  // between scales of w for consecutive blocks of columns, of the contraction
    int64_t M;
    int C, L;              // columns of the output, length of the contraction
    void *y;
    int64_t ys;
    int y_type, y_wide;    // y_wide: rows take 16-byte stores
    int slices, per;       // (of a product that is cut: slices of the contraction, blocks of 128 in each)
    float *part;           // ... and its sums by slice: [slice][column / 4][row][column % 4], the order in which lanes have them
};

// Shared-memory matrix descriptors.  K-major, 128-byte swizzle: rows of 128 codes, 8-row
// groups 1024 bytes apart, an MMA's 32 of k = 32 bytes.  MN-major, 128-byte swizzle: rows of
// 128 columns, one per k; 8 k = 1024 bytes, an MMA's 32 of k = 4096 bytes, the next 128
// columns 16 KB on.
__device__ __forceinline__ uint64_t desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 * kBK >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ constexpr uint32_t idesc(bool b_mn, int m, int n) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// The four MMAs of a block, operands kStepA and kStepB (in descriptor units) apart, the
// first one overwriting what tensor memory held; one election of a thread of the
// converged warp.
template <uint32_t kStepA, uint32_t kStepB>
__device__ __forceinline__ void umma_block(uint32_t d, uint64_t a0, uint64_t b0, uint32_t id) {
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

// Whether a barrier's phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// 64 or 32 columns of this lane in pairs, waited for in the same statement (no register copy
// can slip between the load and the wait).
__device__ __forceinline__ void tmem_ld(uint32_t t, f32x2 (&v)[32]) {
    asm volatile(
        "{\n\t.reg .b32 r<64>;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {r0, r1, r2, r3, r4, r5, r6, r7, r8, r9, r10, r11, r12, r13, r14, r15, r16, r17, r18, r19, r20, r21, r22, r23, r24, r25, r26, r27, r28, r29, r30, r31, r32, r33, r34, r35, r36, r37, r38, r39, r40, r41, r42, r43, r44, r45, r46, r47, r48, r49, r50, r51, r52, r53, r54, r55, r56, r57, r58, r59, r60, r61, r62, r63}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "mov.b64 %0, {r0, r1};\n\tmov.b64 %1, {r2, r3};\n\tmov.b64 %2, {r4, r5};\n\tmov.b64 %3, {r6, r7};\n\tmov.b64 %4, {r8, r9};\n\tmov.b64 %5, {r10, r11};\n\tmov.b64 %6, {r12, r13};\n\tmov.b64 %7, {r14, r15};\n\tmov.b64 %8, {r16, r17};\n\tmov.b64 %9, {r18, r19};\n\tmov.b64 %10, {r20, r21};\n\tmov.b64 %11, {r22, r23};\n\tmov.b64 %12, {r24, r25};\n\tmov.b64 %13, {r26, r27};\n\tmov.b64 %14, {r28, r29};\n\tmov.b64 %15, {r30, r31};\n\tmov.b64 %16, {r32, r33};\n\tmov.b64 %17, {r34, r35};\n\tmov.b64 %18, {r36, r37};\n\tmov.b64 %19, {r38, r39};\n\tmov.b64 %20, {r40, r41};\n\tmov.b64 %21, {r42, r43};\n\tmov.b64 %22, {r44, r45};\n\tmov.b64 %23, {r46, r47};\n\tmov.b64 %24, {r48, r49};\n\tmov.b64 %25, {r50, r51};\n\tmov.b64 %26, {r52, r53};\n\tmov.b64 %27, {r54, r55};\n\tmov.b64 %28, {r56, r57};\n\tmov.b64 %29, {r58, r59};\n\tmov.b64 %30, {r60, r61};\n\tmov.b64 %31, {r62, r63};\n\t}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]), "=l"(v[12]), "=l"(v[13]), "=l"(v[14]), "=l"(v[15]), "=l"(v[16]), "=l"(v[17]), "=l"(v[18]), "=l"(v[19]), "=l"(v[20]), "=l"(v[21]), "=l"(v[22]), "=l"(v[23]), "=l"(v[24]), "=l"(v[25]), "=l"(v[26]), "=l"(v[27]), "=l"(v[28]), "=l"(v[29]), "=l"(v[30]), "=l"(v[31])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t t, f32x2 (&v)[16]) {
    asm volatile(
        "{\n\t.reg .b32 r<32>;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {r0, r1, r2, r3, r4, r5, r6, r7, r8, r9, r10, r11, r12, r13, r14, r15, r16, r17, r18, r19, r20, r21, r22, r23, r24, r25, r26, r27, r28, r29, r30, r31}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "mov.b64 %0, {r0, r1};\n\tmov.b64 %1, {r2, r3};\n\tmov.b64 %2, {r4, r5};\n\tmov.b64 %3, {r6, r7};\n\tmov.b64 %4, {r8, r9};\n\tmov.b64 %5, {r10, r11};\n\tmov.b64 %6, {r12, r13};\n\tmov.b64 %7, {r14, r15};\n\tmov.b64 %8, {r16, r17};\n\tmov.b64 %9, {r18, r19};\n\tmov.b64 %10, {r20, r21};\n\tmov.b64 %11, {r22, r23};\n\tmov.b64 %12, {r24, r25};\n\tmov.b64 %13, {r26, r27};\n\tmov.b64 %14, {r28, r29};\n\tmov.b64 %15, {r30, r31};\n\t}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]), "=l"(v[12]), "=l"(v[13]), "=l"(v[14]), "=l"(v[15])
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
template <int NP>
__device__ __forceinline__ void put_part(const Args &a, int slice, int64_t row, int c, const f32x2 (&acc)[NP]) {
    if (row >= a.M) return;
    float4 *const o = reinterpret_cast<float4 *>(a.part) + ((int64_t)slice * (a.C / 4) + c / 4) * a.M + row;
#pragma unroll
    for (int j = 0; j < NP; j += 2) {
        if (c + 2 * j >= a.C) return;
        float4 v;
        f2_split(acc[j], v.x, v.y), f2_split(acc[j + 1], v.z, v.w);
        o[j / 2 * a.M] = v;
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

// kMn: w lies MN-major (transposed).
template <int BN, bool kMn, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
k_fp8_mm(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, const Args a) {
    using C = Cfg<BN>;
    constexpr int S = C::kStages, NP = BN / 8;  // NP: pairs of columns a writing thread loads at a time, half of its own
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t full_bar[S], done_bar[S], acc_empty[2], exit_bar;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = (int)((a.M + kM - 1) / kM), ct = (a.C + BN - 1) / BN, of_slice = mt * ct, tiles = kSplit ? of_slice * a.slices : of_slice;
    const int blocks = (a.L + kBK - 1) / kBK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full_bar[s]), 1), mbar_init(smem_u32(&done_bar[s]), 1);
        for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&acc_empty[b]), kEpilogue);
        mbar_init(smem_u32(&exit_bar), 1);
        s_abort = 0;
        fence_mbar_init_cluster();
    }
    if (warp == kEpilogue + 1) tmem_get<false>(smem_u32(&s_tmem), C::kTmemCols);
    tmem_fence_before_sync();
    __syncthreads();
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
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                int m, c;
                const int slice = kSplit ? tile / of_slice : 0, i0 = kSplit ? slice * a.per : 0, i1 = kSplit && i0 + a.per < blocks ? i0 + a.per : blocks;
                place_of(tile - slice * of_slice, mt, ct, m, c);
                m = __shfl_sync(0xffffffffu, m * kM, 0), c = __shfl_sync(0xffffffffu, c * BN, 0);
                for (int i = i0; i < i1; ++i) {
                    if (!(ok = mbar_wait_warp<false>(smem_u32(&done_bar[slot]), parity, &s_abort))) break;
                    const uint32_t sa = sbase + (uint32_t)slot * C::kStage;
                    const uint32_t bar = smem_u32(&full_bar[slot]);
                    expect_bytes(bar, C::kStage);
                    ++issued;
                    load_2d<false>(sa, &tm_x, bar, i * kBK, m, pol);
#pragma unroll
                    for (int j = 0; j < BN; j += 128) {
                        if (kMn) load_2d<false>(sa + C::kABytes + j * kBK, &tm_w, bar, c + j, i * kBK, pol);
                        else load_2d<false>(sa + C::kABytes + j * kBK, &tm_w, bar, i * kBK, c + j, pol);
                    }
                    if (++slot == S) slot = 0, parity ^= 1u;
                }
            }
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            // the last stages issued must land before the CTA leaves
            for (int k = 0; k < S && k < issued; ++k) {
                if (--slot < 0) slot = S - 1, parity ^= 1u;
                wait_exit(smem_u32(&full_bar[slot]), parity ^ 1u);
            }
            __syncwarp();
        } else if (warp == kEpilogue + 1) {
            // One commit tells both that a stage is free and that a block's sums are there, and the
            // next barriers are looked at before the MMAs are issued (a look behind them waits for
            // their turn), and waited for only if they were not complete then.
            int slot = 0;
            uint32_t parity = 0, b = 0, b_parity = 1;
            bool ok = true, stage_ready = false, acc_ready = false;
            const uint64_t da0 = desc(sbase), db0 = desc(sbase + C::kABytes);
            constexpr uint32_t kStepA = 32 >> 4, kStepB = (kMn ? 4096 : 32) >> 4, id = idesc(kMn, kM, BN);
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                const int i0 = kSplit ? tile / of_slice * a.per : 0, i1 = kSplit && i0 + a.per < blocks ? i0 + a.per : blocks;
                for (int i = i0; i < i1; ++i) {
                    if (!__all_sync(0xffffffffu, stage_ready) && !(ok = mbar_wait_warp<false>(smem_u32(&full_bar[slot]), parity, &s_abort))) break;
                    if (!__all_sync(0xffffffffu, acc_ready) && !(ok = mbar_wait_warp<false>(smem_u32(&acc_empty[b]), b_parity, &s_abort))) break;
                    const uint32_t at = (uint32_t)(slot * C::kStage) / 16, d = tbase + b * BN, done = smem_u32(&done_bar[slot]);
                    if (++slot == S) slot = 0, parity ^= 1u;
                    if (b ^= 1u; b == 0) b_parity ^= 1u;
                    stage_ready = mbar_test(smem_u32(&full_bar[slot]), parity);
                    acc_ready = mbar_test(smem_u32(&acc_empty[b]), b_parity);
                    tmem_fence_after_sync();
                    umma_block<kStepA, kStepB>(d, da0 + at, db0 + at, id);
                    umma_commit<false>(done);
                }
            }
            // every MMA issued has completed before the tensor memory is freed
            umma_commit<false>(smem_u32(&exit_bar));
            wait_exit(smem_u32(&exit_bar), 0u);
            __syncwarp();
        }
    } else {
        if constexpr (C::kMoved) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWriting));
        const int q = warp & 3, half = warp >> 2;  // the warp's quadrant of tensor-memory lanes; which of its two
        uint32_t b = 0, parity = 0;
        int slot = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            int m, c;
            const int slice = kSplit ? tile / of_slice : 0, i0 = kSplit ? slice * a.per : 0, i1 = kSplit && i0 + a.per < blocks ? i0 + a.per : blocks;
            place_of(tile - slice * of_slice, mt, ct, m, c);
            const int64_t row = (int64_t)m * kM + q * 32 + lane;
            const int c0 = c * BN + half * (BN / 2);
            // (rows and columns that are not there take a scale that is)
            const int64_t x_at = (row < a.M ? row : a.M - 1) * blocks;
            const int64_t w_at = (c0 < a.C ? c0 : a.C - 1) / kFp8Block * a.sw_col;
            uint32_t next_x = a.sx.raw(x_at + i0), next_w = a.sw.raw(w_at + i0 * a.sw_k);
            f32x2 acc[2][NP];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < NP; ++j) acc[h][j] = f2_dup(0.0f);
            for (int i = i0; i < i1; ++i) {
                const f32x2 s = f2_dup(a.sx.value(next_x) * a.sw.value(next_w));
                if (i + 1 < i1) next_x = a.sx.raw(x_at + i + 1), next_w = a.sw.raw(w_at + (i + 1) * a.sw_k);
                if (!(ok = mbar_wait_warp<false>(smem_u32(&done_bar[slot]), parity, &s_abort))) break;
                if (++slot == S) slot = 0, parity ^= 1u;
                tmem_fence_after_sync();
                const uint32_t ta = tbase + b * BN + (uint32_t)(half * (BN / 2)) + ((uint32_t)(32 * q) << 16);
                f32x2 v[NP];
                tmem_ld(ta, v);
#pragma unroll
                for (int k = 0; k < NP; ++k) acc[0][k] = f2_fma(v[k], s, acc[0][k]);
                tmem_ld(ta + 2 * NP, v);
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&acc_empty[b]));
                __syncwarp();
                b ^= 1u;
#pragma unroll
                for (int k = 0; k < NP; ++k) acc[1][k] = f2_fma(v[k], s, acc[1][k]);
            }
            if (ok && kSplit) put_part<NP>(a, slice, row, c0, acc[0]), put_part<NP>(a, slice, row, c0 + 2 * NP, acc[1]);
            if (ok && !kSplit) put_row<NP>(a, row, c0, acc[0]), put_row<NP>(a, row, c0 + 2 * NP, acc[1]);
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (warp == kEpilogue + 1) tmem_give_back<false>(tbase, C::kTmemCols);
}

// ------------------------------------------------------------ up to 16 rows
// Few rows leave nothing but the reading of w: it goes past each SM once (hc_pieces.cuh), the SM's
// rows of w in chunks of 64; a chunk's pieces go round the warps, whose sums meet in
// shared memory.  NB tiles of 8 rows of x.
constexpr int kFewPairs = 4;  // pairs of row tiles of a chunk
template <int NB>
constexpr int kFewWarps = NB == 1 ? 16 : 12;  // (the sums of two tiles of x do not fit the registers of 16)
template <int NB>
constexpr int kFewSmem = kFewWarps<NB> * kFewPairs * (2 * kCell + NB * 128 * 4);

template <typename T>
__device__ __forceinline__ void put1(void *y, int64_t at, float v) {
    static_cast<T *>(y)[at] = from_f<T>(v);
}

template <int NB>
__global__ void __launch_bounds__(32 * kFewWarps<NB>, 1) k_fp8_few(const Args a, const uint8_t *__restrict__ x, int64_t xs, const uint8_t *__restrict__ w) {
    constexpr int W = kFewWarps<NB>, NP = kFewPairs, kRing = NP * 2 * kCell, kSums = NP * NB * 128;
    extern __shared__ __align__(128) uint8_t smem[];
    float *const red = reinterpret_cast<float *>(smem + W * kRing);  // [warp][pair][tile of x][4][lane]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int from = (int)((int64_t)a.C * blockIdx.x / gridDim.x), to = (int)((int64_t)a.C * (blockIdx.x + 1) / gridDim.x);
    const int pieces = (a.L + 127) / 128;
    const auto begin = [&](int n) { return (warp + n * (W - pieces % W)) % W; };  // the warp's first piece of the n-th chunk
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // copies, codes of x and scales run a step ahead: an: the chunk, ak: the piece
    int abase = from & ~7, an = 0, ak = warp;
    uint32_t rows = 0;  // which of the chunk's tiles have this lane's row
    const auto aim = [&]() {
        rows = 0;
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) rows |= (uint32_t)(abase + 8 * i + g >= from && abase + 8 * i + g < to) << i;
    };
    const auto settle = [&]() {
        while (abase < to && ak >= pieces) abase += 16 * NP, ak = begin(++an), aim();
    };
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kRing + lane * 16);
    const auto fetch = [&](int j) {
        const uint32_t at = ring + (uint32_t)(j * 2 * kCell);
        const uint8_t *const p = w + (int64_t)(abase + 16 * j + g) * a.L + ak * 128 + t4 * 16;
        const bool first_half = ak * 128 + t4 * 16 < a.L, second_half = ak * 128 + t4 * 16 + 64 < a.L;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool there = rows >> (2 * j + h) & 1u;
            load_piece(at + h * kCell, p + (int64_t)(8 * h) * a.L, there && first_half, there && second_half);
        }
        cp_async_commit();
    };
    uint4 raw[NB][2];
    uint32_t raw_x[NB], raw_w = 0;
    const auto load_rows = [&]() {
        if (abase >= to) return;
#pragma unroll
        for (int m = 0; m < NB; ++m) {
            const bool has = 8 * m + g < a.M;
            const int64_t row = has ? 8 * m + g : 0;
            raw_x[m] = a.sx.raw(row * pieces + ak);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int c = ak * 128 + s * 64 + t4 * 16;
                raw[m][s] = make_uint4(0, 0, 0, 0);
                if (has && c < a.L) raw[m][s] = __ldg(reinterpret_cast<const uint4 *>(x + row * xs + c));
            }
        }
        // (lane i: tile i's)
        if (lane < 2 * NP && abase + 8 * lane < to) raw_w = a.sw.raw((abase + 8 * lane) / kFp8Block * a.sw_col + ak * a.sw_k);
    };
    aim();
    settle();
    load_rows();
#pragma unroll
    for (int j = 0; j < NP; ++j) fetch(j);
    ak += W;
    settle();
    int n = 0;
    for (int base = from & ~7; base < to; base += 16 * NP, ++n) {
        float acc[NP][NB][4];
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int m = 0; m < NB; ++m)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[j][m][q] = 0.0f;
        for (int k = begin(n); k < pieces; k += W) {
            uint32_t tok[NB][16];
            float unit[NB][2];
#pragma unroll
            for (int m = 0; m < NB; ++m) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    widen(raw[m][s].x, tok[m][8 * s], tok[m][8 * s + 1]), widen(raw[m][s].y, tok[m][8 * s + 2], tok[m][8 * s + 3]);
                    widen(raw[m][s].z, tok[m][8 * s + 4], tok[m][8 * s + 5]), widen(raw[m][s].w, tok[m][8 * s + 6], tok[m][8 * s + 7]);
                }
                const float own = a.sx.value(raw_x[m]);
                unit[m][0] = __shfl_sync(0xffffffffu, own, 8 * t4), unit[m][1] = __shfl_sync(0xffffffffu, own, 8 * t4 + 4);
            }
            const float scale = a.sw.value(raw_w);
            load_rows();
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                cp_async_wait<NP - 1>();
                if (base + 16 * j < to) {
                    const uint32_t here = ring + (uint32_t)(j * 2 * kCell);
                    const Rows16<true> rows16(read_piece(here), read_piece(here + kCell));
                    const float s0 = __shfl_sync(0xffffffffu, scale, 2 * j), s1 = __shfl_sync(0xffffffffu, scale, 2 * j + 1);
#pragma unroll
                    for (int m = 0; m < NB; ++m) multiply_scaled<true>(acc[j][m], rows16, tok[m], s0, s1, unit[m]);
                }
                fetch(j);
            }
            ak += W;
            settle();
        }
        if (begin(n) < pieces) {
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int m = 0; m < NB; ++m)
#pragma unroll
                    for (int q = 0; q < 4; ++q) red[warp * kSums + ((j * NB + m) * 4 + q) * 32 + lane] = acc[j][m][q];
        }
        __syncthreads();
        const int meet = pieces < W ? pieces : W, w0 = n * (pieces % W) % W;  // the warps that had a piece, in their order
        for (int o = threadIdx.x; o < kSums; o += 32 * W) {
            const int j = o / (NB * 128), m = o / 128 % NB, q = o / 32 % 4;  // (o % 32 is this lane)
            const int row = 8 * m + 2 * t4 + (q & 1), col = base + 16 * j + 8 * (q >> 1) + g;
            if (row >= a.M || col < from || col >= to) continue;
            float v = 0.0f;
            for (int i = 0, f = w0; i < meet; ++i) {
                v += red[f * kSums + o];
                if (++f == W) f = 0;
            }
            const int64_t at = row * a.ys + col;
            if (a.y_type == HC_F32) put1<float>(a.y, at, v);
            else if (a.y_type == HC_BF16) put1<__nv_bfloat16>(a.y, at, v);
            else put1<__half>(a.y, at, v);
        }
        __syncthreads();
    }
    cp_async_wait<0>();
}

// A matrix of codes [rows][width], rows `stride` bytes apart, boxes of 128 x 128, 128-byte
// swizzle, zeros outside: the map names the rows and columns that are there and nothing else.  (Maps of less than
// 128 KB load slowly.  Maps with a third dimension that no load used, to reach that length, were followed by an illegal
// address in a captured product of 100 rows, in one of some six runs of the tests: the suspected cause is memory behind
// the matrix that such a map names.)
bool make_map(CUtensorMap *m, const void *base, int64_t width, int64_t rows, int64_t stride) {
    const auto enc = encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {kBK, 128}, one[2] = {1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, one,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kDevices = 64;

// Launches on every SM, once per kernel and device finding out how many there are and
// allowing the shared memory.
template <int BN, bool kMn, bool kSplit>
cudaError_t launch(const CUtensorMap &tx, const CUtensorMap &tw, const Args &a, cudaStream_t s) {
    using C = Cfg<BN>;
    const auto k = k_fp8_mm<BN, kMn, kSplit>;
    static std::atomic<int> ctas[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads), cfg.dynamicSmemBytes = C::kSmem, cfg.stream = s;
    cfg.attrs = &early, cfg.numAttrs = 1;
    int grid = ctas[dev].load(std::memory_order_acquire);
    if (!grid) {
        cudaFuncAttributes is{};
        if ((e = cudaFuncGetAttributes(&is, k)) != cudaSuccess) return e;
        if (C::kMoved && is.numRegs != kRegs) return cudaErrorInvalidKernelImage;  // (the split would wait forever)
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&grid, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        ctas[dev].store(grid, std::memory_order_release);  // (the attribute is set for whoever reads it)
    }
    const int64_t tiles = (a.M + kM - 1) / kM * ((a.C + BN - 1) / BN) * (kSplit ? a.slices : 1);
    cfg.gridDim = dim3((unsigned)(tiles < grid ? tiles : grid));
    return cudaLaunchKernelEx(&cfg, k, tx, tw, a);
}

// The sum over slices, one after the other (the same call gives the same bits), rounded to
// the output's type: 8 columns of a row a thread, 8 rows x 128 columns a block.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) k_join(const Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % 32, c = blockIdx.x * 128 + (threadIdx.x / 32 * 4 + lane / 8) * 8;
    const int64_t row = (int64_t)blockIdx.y * 8 + lane % 8;
    if (row >= a.M || c >= a.C) return;
    const float4 *p = reinterpret_cast<const float4 *>(a.part) + (int64_t)(c / 4) * a.M + row;
    const int64_t slice = (int64_t)(a.C / 4) * a.M;
    f32x2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = f2_dup(0.0f);
#pragma unroll 4
    for (int i = 0; i < a.slices; ++i, p += slice) {
        const float4 lo = __ldcg(p), hi = __ldcg(p + a.M);
        v[0] = f2_add(v[0], f2_make(lo.x, lo.y)), v[1] = f2_add(v[1], f2_make(lo.z, lo.w));
        v[2] = f2_add(v[2], f2_make(hi.x, hi.y)), v[3] = f2_add(v[3], f2_make(hi.z, hi.w));
    }
    const int64_t at = row * a.ys + c;
    if (a.y_type == HC_F32) put8(static_cast<float *>(a.y) + at, v, a.y_wide);
    else if (a.y_type == HC_BF16) put8(static_cast<__nv_bfloat16 *>(a.y) + at, v, a.y_wide);
    else put8(static_cast<__half *>(a.y) + at, v, a.y_wide);
}
cudaError_t join(const Args &a, cudaStream_t s) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.C + 127) / 128), (unsigned)((a.M + 7) / 8)), cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_join, a);
}

// How a product is cut: into tiles of 128 x bn and, where few tiles leave SMs idle, the
// contraction into slices of `per` blocks that k_join adds up.  The rule counts cycles:
// a block of 128 takes an SM some 1,050 with 256 columns and 860 with 128 (the signals and
// the sums, not the MMAs), but w comes in at 2,700 bytes a cycle at the most; the joining launch 1,500,
// a slice 1,500 more, and its sums 2.2 per 1,000 to write and read.  Measured with w in HBM, against the
// better of the whole contractions (us): 17 x 5,120 x 5,120 18.3 -> 12.4 (4 slices; 2: 15.0, 7: 13.2),
// 128 rows 20.0 -> 14.6 (4), 256 rows 20.6 -> 16.4 (3), 256 x 2,048 x 8,192 28.3 -> 15.3 (5); but
// 256 x 8,192 x 2,048 10.6 -> 13.6 (2) and 64 x 16,384 x 5,120 19.8 -> 21.9 (2), which the rule leaves
// whole.  A constant number of SMs: the cut decides the workspace and the order of the sums,
// which must not depend on the device.
constexpr int kSms = 152, kMostSlices = 32;
struct Cut {
    int bn, slices, per;
};
Cut cut(int64_t M, int C, int L) {
    const int64_t rows = (M + kM - 1) / kM, blocks = (L + kBK - 1) / kBK;
    const int64_t wide = rows * ((C + 255) / 256), narrow = rows * ((C + 127) / 128);
    Cut best{128, 1, (int)blocks};
    const double reading = (double)C * L / 2700;
    double least = std::max(reading, (double)((narrow + kSms - 1) / kSms * blocks) * 860);
    for (int64_t s = 1; s == 1 || (s <= kMostSlices && s <= blocks && wide * s <= kSms); ++s) {
        const int64_t per = (blocks + s - 1) / s;
        if ((blocks + per - 1) / per != s) continue;
        const double cycles = std::max(reading, (double)((wide * s + kSms - 1) / kSms * per) * 1050) +
                              (s == 1 ? 0 : 1500 + 1500 * (double)s + 0.0022 * (double)(s * M * C));
        if (cycles <= least) least = cycles, best = Cut{256, (int)s, (int)per};
    }
    return best;
}
bool few(bool transposed, int64_t M) { return !transposed && M <= 16; }

template <int NB>
cudaError_t launch_few(const Args &a, const uint8_t *x, int64_t xs, const uint8_t *w, cudaStream_t s) {
    const auto k = k_fp8_few<NB>;
    static std::atomic<int> sms[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    int n = sms[dev].load(std::memory_order_acquire);
    if (!n) {
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem<NB>)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        sms[dev].store(n, std::memory_order_release);  // (the attribute is set for whoever reads it)
    }
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.C / 8 < n ? a.C / 8 : n)), cfg.blockDim = dim3(32 * kFewWarps<NB>);
    cfg.dynamicSmemBytes = kFewSmem<NB>, cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a, x, xs, w);
}

}  // namespace f8

cudaError_t launch_fp8_mm(const uint8_t *x, int64_t x_stride, const void *x_scales, bool x_f32, const uint8_t *w,
                          const void *w_scales, bool w_f32, bool transposed, int64_t M, int N, int K, void *y, int64_t y_stride,
                          hc_dtype y_type, void *workspace, cudaStream_t s) {
    const int C = transposed ? K : N, L = transposed ? N : K;
    const int64_t row = (K + kFp8Block - 1) / kFp8Block;  // scales of w in a row of blocks
    const int64_t size = y_type == HC_F32 ? 4 : 2;
    const bool few = f8::few(transposed, M);
    const f8::Cut cut = few ? f8::Cut{0, 1, 0} : f8::cut(M, C, L);
    const f8::Args a{{x_scales, x_f32}, {w_scales, w_f32}, transposed ? 1 : row, transposed ? row : 1, M, C, L, y, y_stride,
                         y_type, reinterpret_cast<uintptr_t>(y) % 16 == 0 && y_stride * size % 16 == 0, cut.slices, cut.per,
                      static_cast<float *>(workspace)};
    if (few) return M <= 8 ? f8::launch_few<1>(a, x, x_stride, w, s) : f8::launch_few<2>(a, x, x_stride, w, s);
    CUtensorMap tx, tw;
    if (!f8::make_map(&tx, x, L, M, x_stride) || !f8::make_map(&tw, w, K, N, K)) return cudaErrorInvalidValue;
    if (cut.slices > 1) {
        const cudaError_t e = transposed ? f8::launch<256, true, true>(tx, tw, a, s) : f8::launch<256, false, true>(tx, tw, a, s);
        return e == cudaSuccess ? f8::join(a, s) : e;
    }
    if (cut.bn == 256) return transposed ? f8::launch<256, true, false>(tx, tw, a, s) : f8::launch<256, false, false>(tx, tw, a, s);
    return transposed ? f8::launch<128, true, false>(tx, tw, a, s) : f8::launch<128, false, false>(tx, tw, a, s);
}

size_t fp8_mm_workspace_bytes(bool transposed, int64_t M, int N, int K) {
    const int C = transposed ? K : N;
    if (f8::few(transposed, M)) return 0;
    const f8::Cut cut = f8::cut(M, C, transposed ? N : K);
    return cut.slices == 1 ? 0 : (size_t)cut.slices * M * C * 4;
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
