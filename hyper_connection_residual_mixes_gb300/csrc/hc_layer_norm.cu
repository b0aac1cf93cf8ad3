// hc_layer_norm.cu -- layer norm of sublayer inputs, forward and backward, for GB300.
//
// Forward, per row of d values:
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
//   y = (x - mean) rstd w + b.
// Backward, with xh = (x - mean) rstd and wg = g w:
//   g_x = rstd (wg - mean(wg) - xh mean(wg xh)),
//   g_w = sum over rows of g xh,  g_b = sum over rows of g.
// All sums run in fp32; y (and g_x) are rounded once, on the way out.
//
// Both directions move each row across HBM once and are bound by that.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hc_device.cuh"
#include "hc_ptx.cuh"
#include "hc_sublayer.h"

namespace hc {

namespace ln {

// ------------------------------------------------------------ element types
template <typename T>
__device__ __forceinline__ float to_f(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __half2float(v);
    else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {  // round to nearest even
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T v[VEC];
};

// a parameter value (norm_w, norm_b): fp32 or 16 bits, by its type code
__device__ __forceinline__ float param(const void *p, int type, int i) {
    if (type == HC_F32) return __ldg(static_cast<const float *>(p) + i);
    const uint16_t u = __ldg(static_cast<const uint16_t *>(p) + i);
    if (type == HC_BF16) return __uint_as_float((uint32_t)u << 16);
    return __half2float(__ushort_as_half(u));
}
template <int VEC>
__device__ __forceinline__ void params(const void *p, int type, int i, float (&o)[VEC]) {
    if constexpr (VEC >= 4) {
        if (type == HC_F32) {
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + k));
                o[k] = f.x, o[k + 1] = f.y, o[k + 2] = f.z, o[k + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k += 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i + k));
                if (type == HC_BF16) {
                    o[k] = bf16lo(u.x), o[k + 1] = bf16hi(u.x), o[k + 2] = bf16lo(u.y), o[k + 3] = bf16hi(u.y);
                } else {
                    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
                    const float2 c = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
                    o[k] = a.x, o[k + 1] = a.y, o[k + 2] = c.x, o[k + 3] = c.y;
                }
            }
        }
    } else {
        o[0] = param(p, type, i);
    }
}

// Read-only streaming load of a vector (each x, g value is read once per launch).
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_stream(const T *p) {
    Vec<T, VEC> r;
    if constexpr (sizeof(r) == 16) {
        uint4 u;
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(p));
        r = *reinterpret_cast<Vec<T, VEC> *>(&u);
    } else {
        r = *reinterpret_cast<const Vec<T, VEC> *>(p);
    }
    return r;
}

// Sum over the row's threads: the warp, or (tpr > 32) the whole block, whose
// warps meet in `red` (one slot per warp; each reduction of a row has its own).
__device__ __forceinline__ float team_sum(float v, int tpr, float *red) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = tpr >> 5;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? red[lane] : 0.0f);
}

// ------------------------------------------------------------ forward
// tpr threads hold a row in registers: thread t the vectors t + i * tpr.  With
// tpr == 32 each warp of the block has a row of its own, else the block has one.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(VEC > 1 && NV >= 8 ? 128 : 1024, 1)
k_layer_norm(const T *__restrict__ x, int64_t xs, const void *__restrict__ w, const void *__restrict__ b, int wt,
             int64_t n, int d, float eps, T *__restrict__ y, int64_t ys, float *__restrict__ mean_out,
             float *__restrict__ rstd_out, int tpr) {
    __shared__ float red[2][32];
    const int t = tpr == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = tpr == 32 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= n) return;  // whole warps; with tpr > 32 never (one block per row)
    const T *xr = x + row * xs;
    Vec<T, VEC> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
        if (c < d) v[i] = load_stream<T, VEC>(xr + c);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((t + i * tpr) * VEC >= d) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += to_f(v[i].v[k]);
    }
    const float mean = team_sum(sum, tpr, red[0]) / (float)d;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((t + i * tpr) * VEC >= d) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float c = to_f(v[i].v[k]) - mean;
            sq = fmaf(c, c, sq);
        }
    }
    const float rstd = 1.0f / sqrtf(team_sum(sq, tpr, red[1]) / (float)d + eps);
    T *yr = y + row * ys;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
        if (c >= d) continue;
        float wv[VEC], bv[VEC] = {};
        params<VEC>(w, wt, c, wv);
        if (b) params<VEC>(b, wt, c, bv);
        Vec<T, VEC> o;
#pragma unroll
        for (int k = 0; k < VEC; ++k) o.v[k] = from_f<T>(fmaf((to_f(v[i].v[k]) - mean) * rstd, wv[k], bv[k]));
        *reinterpret_cast<Vec<T, VEC> *>(yr + c) = o;
    }
    if (t == 0) {
        if (mean_out) mean_out[row] = mean;
        if (rstd_out) rstd_out[row] = rstd;
    }
}

// ------------------------------------------------------------ backward
// Each thread owns the same columns of every row its block takes, with their
// sums of g xh and g in registers; a block leaves one row of partial sums in
// the workspace, k_ln_columns adds the blocks' rows in a fixed order.
template <typename TX, typename TG, int VEC, int NV>
__global__ void __launch_bounds__(1024, 1)
k_ln_backward(const TG *__restrict__ gy, int64_t gs, const TX *__restrict__ x, int64_t xs,
              const void *__restrict__ w, int wt, const float *__restrict__ mean_in,
              const float *__restrict__ rstd_in, int64_t n, int d, TG *__restrict__ gx, int64_t gxs,
              float *__restrict__ part, int tpr) {
    extern __shared__ float s_cols[];  // several rows per block: [2][d] sums of the block
    __shared__ float red[2][2][32];
    const int teams = tpr == 32 ? (blockDim.x >> 5) : 1;
    const int team = tpr == 32 ? (threadIdx.x >> 5) : 0, t = tpr == 32 ? (threadIdx.x & 31) : threadIdx.x;
    const float inv_d = 1.0f / (float)d;
    float wv[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) wv[i][k] = aw[i][k] = ab[i][k] = 0.0f;
        if (c < d) params<VEC>(w, wt, c, wv[i]);
    }
    int buf = 0;
    for (int64_t row = (int64_t)blockIdx.x * teams + team; row < n; row += (int64_t)gridDim.x * teams, buf ^= 1) {
        const TX *xr = x + row * xs;
        const TG *gr = gy + row * gs;
        Vec<TX, VEC> xv[NV];
        Vec<TG, VEC> gv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c < d) {
                xv[i] = load_stream<TX, VEC>(xr + c);
                gv[i] = load_stream<TG, VEC>(gr + c);
            }
        }
        const float mean = __ldg(mean_in + row), rstd = __ldg(rstd_in + row);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((t + i * tpr) * VEC >= d) continue;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = (to_f(xv[i].v[k]) - mean) * rstd, g = to_f(gv[i].v[k]);
                const float wg = g * wv[i][k];
                s1 += wg;
                s2 = fmaf(wg, xh, s2);
                aw[i][k] = fmaf(g, xh, aw[i][k]);
                ab[i][k] += g;
            }
        }
        s1 = warp_sum(s1), s2 = warp_sum(s2);
        if (tpr > 32) {
            // (two buffers: a block writes the next row's sums while a slow warp still reads these)
            if ((threadIdx.x & 31) == 0) red[buf][0][threadIdx.x >> 5] = s1, red[buf][1][threadIdx.x >> 5] = s2;
            __syncthreads();
            const int lane = threadIdx.x & 31, nw = tpr >> 5;
            s1 = warp_sum(lane < nw ? red[buf][0][lane] : 0.0f);
            s2 = warp_sum(lane < nw ? red[buf][1][lane] : 0.0f);
        }
        const float m1 = s1 * inv_d, m2 = s2 * inv_d;
        TG *or_ = gx + row * gxs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c >= d) continue;
            Vec<TG, VEC> o;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = (to_f(xv[i].v[k]) - mean) * rstd;
                o.v[k] = from_f<TG>(rstd * (to_f(gv[i].v[k]) * wv[i][k] - m1 - xh * m2));
            }
            *reinterpret_cast<Vec<TG, VEC> *>(or_ + c) = o;
        }
    }
    float *pw = part + (int64_t)blockIdx.x * 2 * d, *pb = pw + d;
    if (teams == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int c = (t + i * tpr) * VEC + k;
                if (c < d) pw[c] = aw[i][k], pb[c] = ab[i][k];
            }
        return;
    }
    for (int m = 0; m < teams; ++m) {  // the warps add their columns in turn
        if (team == m) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const int c = (t + i * tpr) * VEC + k;
                    if (c < d) {
                        s_cols[c] = aw[i][k] + (m ? s_cols[c] : 0.0f);
                        s_cols[d + c] = ab[i][k] + (m ? s_cols[d + c] : 0.0f);
                    }
                }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) pw[c] = s_cols[c];
}

// g_w, g_b [d] from the blocks' partial rows [blocks][2][d]: 32 columns per
// block, the rows shared among 16 warps.
constexpr int kColWarps = 16;
__global__ void __launch_bounds__(32 * kColWarps)
k_ln_columns(const float *__restrict__ part, int blocks, int d, float *__restrict__ g_w, float *__restrict__ g_b) {
    __shared__ float s[kColWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (c < 2 * d)
        for (int r = warp; r < blocks; r += kColWarps) a += __ldcg(part + (int64_t)r * 2 * d + c);
    s[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < 2 * d) {
        for (int k = 1; k < kColWarps; ++k) a += s[k][lane];
        if (c < d) g_w[c] = a;
        else if (g_b) g_b[c - d] = a;
    }
}

int sm_count_of_device() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return sms;
}

bool aligned(const void *p, int64_t stride_bytes, size_t to) {
    return (reinterpret_cast<uintptr_t>(p) % to) == 0 && (uint64_t)stride_bytes % to == 0;
}

struct FwdCall {
    const void *x; int64_t xs; const void *w, *b; int wt; int64_t n; int d; float eps;
    void *y; int64_t ys; float *mean, *rstd; cudaStream_t s;
};

template <typename T, int VEC, int NV>
cudaError_t fwd_launch(const FwdCall &c, int tpr, int threads) {
    const int64_t per = tpr == 32 ? threads / 32 : 1;
    const int64_t blocks = (c.n + per - 1) / per;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    k_layer_norm<T, VEC, NV><<<(unsigned)blocks, threads, 0, c.s>>>(
        static_cast<const T *>(c.x), c.xs, c.w, c.b, c.wt, c.n, c.d, c.eps, static_cast<T *>(c.y), c.ys, c.mean,
        c.rstd, tpr);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t fwd_vec(const FwdCall &c) {
    const int vecs = (c.d + VEC - 1) / VEC;
    // A warp per row needs no block barrier and keeps the most bytes in flight;
    // it takes over once the rows fill the SMs with warps.
    const bool many = c.n >= 8 * (int64_t)sm_count_of_device();
    if (vecs <= 32) return fwd_launch<T, VEC, 1>(c, 32, 128);
    if (vecs <= 64) return fwd_launch<T, VEC, 2>(c, 32, 128);
    if (vecs <= 128) return fwd_launch<T, VEC, 4>(c, 32, 128);
    if constexpr (VEC > 1) if (many) {
        if (vecs <= 256) return fwd_launch<T, VEC, 8>(c, 32, 128);
        if (vecs <= 512) return fwd_launch<T, VEC, 16>(c, 32, 128);
        if (vecs <= 640) return fwd_launch<T, VEC, 20>(c, 32, 128);
    }
    const int tpr1 = (vecs + 31) / 32 * 32, tpr4 = (vecs + 127) / 128 * 32, tpr16 = (vecs + 511) / 512 * 32;
    if (vecs <= 1024) return fwd_launch<T, VEC, 1>(c, tpr1, tpr1);
    if (vecs <= 4096) return fwd_launch<T, VEC, 4>(c, tpr4, tpr4);
    return fwd_launch<T, 1, 16>(c, tpr16, tpr16);  // single values only: 4096 vectors hold the longest row
}

template <typename T>
cudaError_t fwd_type(const FwdCall &c) {
    constexpr int VEC = 16 / sizeof(T);
    const size_t pa = c.wt == HC_F32 ? 16 : 8;
    if (c.d % VEC == 0 && aligned(c.x, c.xs * (int64_t)sizeof(T), 16) && aligned(c.y, c.ys * (int64_t)sizeof(T), 16) &&
        aligned(c.w, 0, pa) && aligned(c.b, 0, pa))
        return fwd_vec<T, VEC>(c);
    return fwd_vec<T, 1>(c);
}

struct BwdCall {
    const void *gy; int64_t gs; const void *x; int64_t xs; const void *w; int wt; const float *mean, *rstd;
    int64_t n; int d; void *gx; int64_t gxs; float *part, *g_w, *g_b; cudaStream_t s;
};

// blocks of partial sums a launch may use
int64_t max_blocks(int d) { return d < 1024 ? 1216 : d <= 2048 ? 608 : 304; }

template <typename TX, typename TG, int VEC, int NV>
cudaError_t bwd_launch(const BwdCall &c, int tpr) {
    const int threads = tpr == 32 ? 256 : tpr;
    const int teams = tpr == 32 ? threads / 32 : 1;
    const size_t smem = teams > 1 ? (size_t)c.d * 8 : 0;
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_ln_backward<TX, TG, VEC, NV>, threads, smem);
    if (e != cudaSuccess) return e;
    int64_t blocks = (int64_t)(per_sm > 0 ? per_sm : 1) * sm_count_of_device();
    if (blocks > max_blocks(c.d)) blocks = max_blocks(c.d);
    if (blocks > (c.n + teams - 1) / teams) blocks = (c.n + teams - 1) / teams;
    k_ln_backward<TX, TG, VEC, NV><<<(unsigned)blocks, threads, smem, c.s>>>(
        static_cast<const TG *>(c.gy), c.gs, static_cast<const TX *>(c.x), c.xs, c.w, c.wt, c.mean, c.rstd, c.n, c.d,
        static_cast<TG *>(c.gx), c.gxs, c.part, tpr);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k_ln_columns<<<(unsigned)((2 * c.d + 31) / 32), 32 * kColWarps, 0, c.s>>>(c.part, (int)blocks, c.d, c.g_w, c.g_b);
    return cudaGetLastError();
}

template <typename TX, typename TG>
cudaError_t bwd_type(const BwdCall &c) {
    const size_t pa = c.wt == HC_F32 ? 16 : 8;
    const int d = c.d;
    if (d % 4 == 0 && d > 128 && aligned(c.x, c.xs * (int64_t)sizeof(TX), 4 * sizeof(TX)) &&
        aligned(c.gy, c.gs * (int64_t)sizeof(TG), 4 * sizeof(TG)) &&
        aligned(c.gx, c.gxs * (int64_t)sizeof(TG), 4 * sizeof(TG)) && aligned(c.w, 0, pa)) {
        if (d <= 256) return bwd_launch<TX, TG, 4, 2>(c, 32);
        if (d <= 8192) return bwd_launch<TX, TG, 4, 2>(c, (d + 255) / 256 * 32);
        return bwd_launch<TX, TG, 4, 4>(c, (d + 511) / 512 * 32);
    }
    if (d <= 128) return bwd_launch<TX, TG, 1, 4>(c, 32);
    if (d <= 8192) return bwd_launch<TX, TG, 1, 8>(c, (d + 255) / 256 * 32);
    return bwd_launch<TX, TG, 1, 16>(c, (d + 511) / 512 * 32);
}

}  // namespace ln

cudaError_t launch_layer_norm(const void *x, int64_t x_stride, hc_dtype x_type, const void *w, const void *b,
                              hc_dtype w_type, int64_t n, int d, float eps, void *y, int64_t y_stride,
                              float *mean, float *rstd, cudaStream_t s) {
    const ln::FwdCall c{x, x_stride, w, b, (int)w_type, n, d, eps, y, y_stride, mean, rstd, s};
    switch (x_type) {
        case HC_F32: return ln::fwd_type<float>(c);
        case HC_BF16: return ln::fwd_type<__nv_bfloat16>(c);
        case HC_F16: return ln::fwd_type<__half>(c);
    }
    return cudaErrorInvalidValue;
}

size_t layer_norm_backward_workspace_bytes(int64_t n, int d) {
    const int64_t blocks = n < ln::max_blocks(d) ? n : ln::max_blocks(d);
    return (size_t)blocks * 2 * (size_t)d * 4;
}

cudaError_t launch_layer_norm_backward(const void *g_y, int64_t g_stride, hc_dtype g_type, const void *x,
                                       int64_t x_stride, hc_dtype x_type, const void *w, hc_dtype w_type,
                                       const float *mean, const float *rstd, int64_t n, int d, void *g_x,
                                       int64_t gx_stride, float *g_w, float *g_b, void *workspace,
                                       cudaStream_t s) {
    const ln::BwdCall c{g_y, g_stride, x, x_stride, w, (int)w_type, mean, rstd, n, d, g_x, gx_stride,
                        static_cast<float *>(workspace), g_w, g_b, s};
    if (n == 0) {  // no rows: the sums over them are zero
        cudaError_t e = cudaMemsetAsync(g_w, 0, (size_t)d * 4, s);
        if (e == cudaSuccess && g_b) e = cudaMemsetAsync(g_b, 0, (size_t)d * 4, s);
        return e;
    }
    if (g_type == HC_F32) {
        if (x_type == HC_F32) return ln::bwd_type<float, float>(c);
        if (x_type == HC_BF16) return ln::bwd_type<__nv_bfloat16, float>(c);
        return ln::bwd_type<__half, float>(c);
    }
    if (x_type == HC_BF16) return ln::bwd_type<__nv_bfloat16, __nv_bfloat16>(c);
    return ln::bwd_type<__half, __half>(c);
}

}  // namespace hc
