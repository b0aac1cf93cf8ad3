// hc_pieces.cuh -- products of a few tokens with matrices that are read once: the
// matrix goes past in pieces of 8 rows by 128 bytes, straight to the lane that multiplies
// them (cp.async into a place of the lane's own), and mma.sync m16n8k16 takes two of
// them as its 16 rows and 8 tokens as its columns.  The order of k within a piece is free as long
// as both operands share it, so a lane's 16 bytes are its operand as they lie.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hc_ptx.cuh"

namespace hc {

constexpr int kCell = 1024;  // bytes of a piece

// A lane's share of a piece: 16 bytes at 16 (lane % 4) of the row lane / 4, and 64 bytes on.
// `there`: whether they are there, else zeros.
__device__ __forceinline__ void load_piece(uint32_t to, const uint8_t *from, bool there0, bool there1) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there0 ? 16 : 0) : "memory");
    asm volatile("cp.async.cg.shared.global.L2::128B [%0 + 512], [%1 + 64], 16, %2;" ::"r"(to), "l"(from), "r"(there1 ? 16 : 0) : "memory");
}
// 16 bytes of shared memory
__device__ __forceinline__ void read16(uint32_t *w, uint32_t at) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}
struct Piece {
    uint32_t w[8];
};
__device__ __forceinline__ Piece read_piece(uint32_t at) {
    Piece p;
    read16(p.w, at), read16(p.w + 4, at + 512);
    return p;
}
// four codes as two pairs of fp16
__device__ __forceinline__ void widen(uint32_t c, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}
// two values cut off to bf16
__device__ __forceinline__ uint32_t cut_bf16x2(float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); }
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The tokens' side of the MMAs over a piece: token lane / 4 of 8, this lane's values of k in
// pairs.  kF8: 16 of them per 16 bytes of codes (32 a piece), else 8 (16).
template <bool kF8>
constexpr int kPairsOf = kF8 ? 16 : 8;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (__is_same(T, __nv_bfloat16)) mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
    else mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
}
// A pair of tiles (rows 0-7 of the MMA, rows 8-15) as its operand: four registers for each two
// pairs of k.
template <bool kF8>
struct Rows16 {
    uint32_t a[kPairsOf<kF8> / 2][4];
    __device__ __forceinline__ Rows16(const Piece &p, const Piece &q) {
#pragma unroll
        for (int i = 0; i < kPairsOf<kF8> / 2; ++i) {
            if constexpr (kF8) widen(p.w[i], a[i][0], a[i][2]), widen(q.w[i], a[i][1], a[i][3]);
            else a[i][0] = p.w[2 * i], a[i][2] = p.w[2 * i + 1], a[i][1] = q.w[2 * i], a[i][3] = q.w[2 * i + 1];
        }
    }
};
// acc += their products with the tokens
template <typename T, bool kF8>
__device__ __forceinline__ void multiply(float (&acc)[4], const Rows16<kF8> &w, const uint32_t (&x)[kPairsOf<kF8>]) {
#pragma unroll
    for (int i = 0; i < kPairsOf<kF8> / 2; ++i) mma<T>(acc, w.a[i][0], w.a[i][1], w.a[i][2], w.a[i][3], x[2 * i], x[2 * i + 1]);
}
// ... with two operands, in two chains of MMAs that do not wait for one another
template <typename T, bool kF8>
__device__ __forceinline__ void multiply_both(float (&acc)[4], const Rows16<kF8> &w, const uint32_t (&x)[kPairsOf<kF8>], float (&acc2)[4],
                                              const uint32_t (&x2)[kPairsOf<kF8>]) {
#pragma unroll
    for (int i = 0; i < kPairsOf<kF8> / 2; ++i) {
        mma<T>(acc2, w.a[i][0], w.a[i][1], w.a[i][2], w.a[i][3], x2[2 * i], x2[2 * i + 1]);
        mma<T>(acc, w.a[i][0], w.a[i][1], w.a[i][2], w.a[i][3], x[2 * i], x[2 * i + 1]);
    }
}
// acc += ..., times the scales of the two tiles' blocks and of the tokens' values
template <bool kF8>
__device__ __forceinline__ void multiply_scaled(float (&acc)[4], const Rows16<kF8> &w, const uint32_t (&x)[kPairsOf<kF8>], float s0,
                                                float s1, const float (&unit)[2]) {
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    multiply<__half, kF8>(part, w, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = fmaf(part[k], (k < 2 ? s0 : s1) * unit[k & 1], acc[k]);
}
// acc += sums of products, times the scales of the two tiles' blocks and the square of a power of two for each token
__device__ __forceinline__ void add_scaled(float (&acc)[4], const float (&part)[4], float s0, float s1, const float (&root)[2]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = fmaf(part[k] * root[k & 1], (k < 2 ? s0 : s1) * root[k & 1], acc[k]);
}

}  // namespace hc
