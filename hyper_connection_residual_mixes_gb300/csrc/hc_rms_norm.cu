// hc_rms_norm.cu -- root-mean-square norm of a sublayer's input with the residual's
// addition in front and the cast to 8 bits behind it, its backward, and the casts
// by themselves, for GB300.
//
// Forward, per row of d values:
//   r = round(x + residual),  rstd = 1 / sqrt(sum r^2 / d + eps),  y = r rstd w,
//   codes, scales = the cast of y, unrounded, in groups of 128 (hc_fp8.cuh).
// Backward, with xh = r rstd and wg = g_y w:
//   g_x = g_r + rstd (wg - xh mean(wg xh)),  g_w = sum over rows of g_y xh.
// All sums run in fp32.
#include <atomic>

#include <cuda.h>

#include "hc_fp8.cuh"
#include "hc_ptx.cuh"
#include "hc_sublayer.h"
#include "hc_types.cuh"

namespace hc {

namespace rn {

// a weight value: fp32 or 16 bits, by its type code
__device__ __forceinline__ float param(const void *p, int type, int i) {
    if (type == HC_F32) return __ldg(static_cast<const float *>(p) + i);
    const uint16_t u = __ldg(static_cast<const uint16_t *>(p) + i);
    if (type == HC_BF16) return __uint_as_float((uint32_t)u << 16);
    return __half2float(__ushort_as_half(u));
}
template <int VEC>
__device__ __forceinline__ void params(const void *p, int type, int i, float (&o)[VEC]) {
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) {
            if (type == HC_F32) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + k));
                o[k] = f.x, o[k + 1] = f.y, o[k + 2] = f.z, o[k + 3] = f.w;
            } else {
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
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = param(p, type, i + k);
    }
}

// 1 / sqrt(a): the approximation and a Newton step, which leaves about a unit.
__device__ __forceinline__ float rsqrt_newton(float a) {
    const float r = rsqrtf(a);
    return r > 0.0f && r < INFINITY ? fmaf(r * 0.5f, fmaf(-a * r, r, 1.0f), r) : r;  // (0 and infinity stay)
}

__device__ __forceinline__ float largest(float amax, float v) { return fmaxf(amax, fabsf(v)); }  // (a NaN is passed over)
// ... over the lanes that hold a group of 128, VEC values each
template <int VEC>
__device__ __forceinline__ float largest_of_group(float amax) {
#pragma unroll
    for (int o = 64 / VEC; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    return amax;
}

struct Args {
    const void *x, *residual, *w;
    int64_t xs, res_s;
    int w_type;
    int64_t n;
    int d;
    float eps;
    void *r, *y;
    int64_t rs, ys;
    uint8_t *codes, *scales;
    int64_t cs;
    float *rstd;
    int codes_wide;  // whether VEC codes may be stored at once
};

// VEC codes of values already scaled
template <int VEC>
__device__ __forceinline__ void put_codes(uint8_t *o, const float (&v)[VEC], float inv, int wide) {
    if constexpr (VEC == 1) {
        *o = (uint8_t)fp8_codes(v[0] * inv, 0.0f);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int k = 0; k < VEC; k += 4)
            w[k / 4] = fp8_codes(v[k] * inv, v[k + 1] * inv) | fp8_codes(v[k + 2] * inv, v[k + 3] * inv) << 16;
        if (wide) {
            if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(o) = w[0];
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) o[k] = (uint8_t)(w[k / 4] >> (8 * (k & 3)));
        }
    }
}

// Sum over a row's threads: a warp, or (tpr > 32) the block.
__device__ __forceinline__ float team_sum(float v, int tpr, float *red) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < (tpr >> 5) ? red[lane] : 0.0f);
}

// ------------------------------------------------------------ forward
// A row held in registers by a team of tpr threads, thread t the vectors t + i * tpr:
// a warp a row (kWarps), or a block a row.
template <typename T, int VEC, int NV, bool kWarps>
__global__ void __launch_bounds__(kWarps ? 128 : 1024) k_rms_norm(const Args a) {
    __shared__ float red[32];
    __shared__ int s_amax[VEC == 1 && !kWarps ? 128 : 1];
    const int t = kWarps ? threadIdx.x & 31 : threadIdx.x, tpr = kWarps ? 32 : blockDim.x;
    const int64_t row = kWarps ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarps && row >= a.n) return;
    const int d = a.d;
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + row * a.res_s : nullptr;
    T *r = a.r ? static_cast<T *>(a.r) + row * a.rs : nullptr;
    T *y = a.y ? static_cast<T *>(a.y) + row * a.ys : nullptr;
    Vec<T, VEC> v[NV], u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
        if (c < d) {
            v[i] = *reinterpret_cast<const Vec<T, VEC> *>(x + c);
            if (res) u[i] = *reinterpret_cast<const Vec<T, VEC> *>(res + c);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
        if (c >= d) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            if (res) v[i].v[k] = from_f<T>(to_f(v[i].v[k]) + to_f(u[i].v[k]));
            const float f = to_f(v[i].v[k]);
            sum = fmaf(f, f, sum);
        }
        if (r) *reinterpret_cast<Vec<T, VEC> *>(r + c) = v[i];
    }
    const float rstd = rsqrt_newton(fmaf(team_sum(sum, tpr, red), 1.0f / (float)d, a.eps));
    if (t == 0 && a.rstd) a.rstd[row] = rstd;
    const int groups = (d + kFp8Block - 1) / kFp8Block;
    if (VEC == 1 && !kWarps && a.codes) {
        if (t < 128) s_amax[t] = 0;
        __syncthreads();
    }
    float keep[VEC == 1 ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
        const bool in = c < d;
        float f[VEC], w[VEC] = {}, amax = 0.0f;
        if (in) params<VEC>(a.w, a.w_type, c, w);
        Vec<T, VEC> o;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            f[k] = in ? to_f(v[i].v[k]) * rstd * w[k] : 0.0f;
            o.v[k] = from_f<T>(f[k]);
            amax = largest(amax, f[k]);
        }
        if (in && y) *reinterpret_cast<Vec<T, VEC> *>(y + c) = o;
        if (!a.codes) continue;
        if constexpr (VEC == 1) {
            keep[i] = f[0];
            if constexpr (!kWarps) {
                amax = largest_of_group<4>(amax);  // a warp's 32 columns are of one group
                if ((t & 31) == 0 && in) atomicMax(&s_amax[c / kFp8Block], __float_as_int(amax));
            }
        } else {
            const uint32_t byte = fp8_scale_byte(largest_of_group<VEC>(amax));
            if (in) {
                put_codes<VEC>(a.codes + row * a.cs + c, f, fp8_inverse(byte), a.codes_wide);
                if (c % kFp8Block == 0) a.scales[row * groups + c / kFp8Block] = (uint8_t)byte;
            }
        }
    }
    if constexpr (VEC == 1) {
        if (!a.codes) return;
        if (!kWarps) __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * tpr;
            float amax;
            if constexpr (kWarps) {  // a group: four vectors of one value of the warp
                amax = 0.0f;
#pragma unroll
                for (int j = i / 4 * 4; j < NV && j < i / 4 * 4 + 4; ++j) amax = largest(amax, keep[j]);
                amax = largest_of_group<4>(amax);
            } else {
                amax = c < d ? __int_as_float(s_amax[c / kFp8Block]) : 0.0f;
            }
            const uint32_t byte = fp8_scale_byte(amax);
            const float f[1] = {keep[i]};
            if (c < d) {
                put_codes<1>(a.codes + row * a.cs + c, f, fp8_inverse(byte), 0);
                if (c % kFp8Block == 0) a.scales[row * groups + c / kFp8Block] = (uint8_t)byte;
            }
        }
    }
}

template <typename T>
constexpr int kWide = 16 / (int)sizeof(T);  // values of a wide access

bool multiple(const void *p, int64_t stride, int64_t size, int64_t bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0 && stride * size % bytes == 0);
}

template <typename T, int VEC, int NV, bool kWarps>
cudaError_t start(const Args &a, int threads, cudaStream_t s) {
    k_rms_norm<T, VEC, NV, kWarps><<<(unsigned)(kWarps ? (a.n + 3) / 4 : a.n), kWarps ? 128 : threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward(Args a, cudaStream_t s) {
    constexpr int W = kWide<T>;
    const int64_t size = sizeof(T);
    const bool wide = a.d % W == 0 && multiple(a.x, a.xs, size, 16) && multiple(a.residual, a.res_s, size, 16) &&
                      multiple(a.r, a.rs, size, 16) && multiple(a.y, a.ys, size, 16) &&
                      multiple(a.w, 0, 1, a.w_type == HC_F32 ? 16 : 8);
    a.codes_wide = multiple(a.codes, a.cs, 1, W);
    // (threads of a block: whole groups of 128 values a pass)
    const int per = wide ? W : 1, need = (a.d + per - 1) / per;
    if (wide) {
        if (need <= 32) return start<T, W, 1, true>(a, 0, s);
        if (need <= 64) return start<T, W, 2, true>(a, 0, s);
        const int threads = need > 1024 ? 1024 : (need + 31) / 32 * 32;
        if (need <= 1024) return start<T, W, 1, false>(a, threads, s);
        if (need <= 2048) return start<T, W, 2, false>(a, threads, s);
        return start<T, W, 4, false>(a, threads, s);
    }
    if (need <= 128) return start<T, 1, 4, true>(a, 0, s);
    const int threads = need > 1024 ? 1024 : (need + 127) / 128 * 128;
    if (need <= 1024) return start<T, 1, 1, false>(a, threads, s);
    if (need <= 4096) return start<T, 1, 4, false>(a, threads, s);
    return start<T, 1, 16, false>(a, threads, s);
}

// ------------------------------------------------------------ backward
// A block walks over rows, its threads own columns and keep their sums of g xh; it
// leaves a row of partial sums in the workspace, k_columns adds these in a fixed
// order.  The second pass over a row reads it again, from L1 or L2.
struct BackArgs {
    const void *g, *gr, *r, *w;
    int64_t gs, grs, rs;
    int w_type;
    const float *rstd;
    int64_t n;
    int d;
    void *gx;
    int64_t gxs;
    float *part;
};

template <typename TX, typename TG, int VEC, int NV, bool kWarps>
__global__ void __launch_bounds__(kWarps ? 256 : 1024) k_rms_backward(const BackArgs a) {
    __shared__ float red[2][32];
    __shared__ float s_cols[kWarps ? 32 * VEC * NV : 1];
    const int t = kWarps ? threadIdx.x & 31 : threadIdx.x, tpr = kWarps ? 32 : blockDim.x;
    const int teams = kWarps ? 8 : 1, team = kWarps ? threadIdx.x >> 5 : 0;
    const float inv_d = 1.0f / (float)a.d;
    float aw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) aw[i][k] = 0.0f;
    int buf = 0;
    for (int64_t row = (int64_t)blockIdx.x * teams + team; row < a.n; row += (int64_t)gridDim.x * teams, buf ^= 1) {
        const TX *xr = static_cast<const TX *>(a.r) + row * a.rs;
        const TG *gr = static_cast<const TG *>(a.g) + row * a.gs;
        const TG *past = a.gr ? static_cast<const TG *>(a.gr) + row * a.grs : nullptr;
        const float rstd = __ldg(a.rstd + row);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c >= a.d) continue;
            const Vec<TX, VEC> xv = *reinterpret_cast<const Vec<TX, VEC> *>(xr + c);
            const Vec<TG, VEC> gv = *reinterpret_cast<const Vec<TG, VEC> *>(gr + c);
            float w[VEC];
            params<VEC>(a.w, a.w_type, c, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = to_f(xv.v[k]) * rstd, g = to_f(gv.v[k]);
                sum = fmaf(g * w[k], xh, sum);
                aw[i][k] = fmaf(g, xh, aw[i][k]);
            }
        }
        // (two buffers: a warp writes the next row's while a slow one still reads these)
        const float m = team_sum(sum, tpr, red[buf]) * inv_d;
        TG *o_row = static_cast<TG *>(a.gx) + row * a.gxs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c >= a.d) continue;
            const Vec<TX, VEC> xv = *reinterpret_cast<const Vec<TX, VEC> *>(xr + c);
            const Vec<TG, VEC> gv = *reinterpret_cast<const Vec<TG, VEC> *>(gr + c);
            Vec<TG, VEC> pv;
            if (past) pv = *reinterpret_cast<const Vec<TG, VEC> *>(past + c);
            float w[VEC];
            params<VEC>(a.w, a.w_type, c, w);
            Vec<TG, VEC> o;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = to_f(xv.v[k]) * rstd;
                const float g = rstd * fmaf(-xh, m, to_f(gv.v[k]) * w[k]);
                o.v[k] = from_f<TG>(past ? g + to_f(pv.v[k]) : g);
            }
            *reinterpret_cast<Vec<TG, VEC> *>(o_row + c) = o;
        }
    }
    float *pw = a.part + (int64_t)blockIdx.x * a.d;
    if constexpr (!kWarps) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int c = (t + i * tpr) * VEC + k;
                if (c < a.d) pw[c] = aw[i][k];
            }
    } else {
        for (int m = 0; m < teams; ++m) {  // the warps add their columns in turn
            if (team == m) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        const int c = (t + i * tpr) * VEC + k;
                        if (c < a.d) s_cols[c] = aw[i][k] + (m ? s_cols[c] : 0.0f);
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.d; c += blockDim.x) pw[c] = s_cols[c];
    }
}

// g_w: the blocks' partial sums added in a fixed order.  A block takes 32 columns;
// its 8 warps share the rows.
__global__ void __launch_bounds__(256) k_rms_columns(const float *__restrict__ part, int blocks, int d, float *__restrict__ gw) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < d)
        for (int b = warp; b < blocks; b += 8) v += part[(int64_t)b * d + c];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < d) {
#pragma unroll
        for (int k = 1; k < 8; ++k) v += s[k][lane];
        gw[c] = v;
    }
}

// blocks of the backward, and so rows of partial sums: by n alone
int back_blocks(int64_t n) { return (int)(n < 304 ? (n > 0 ? n : 1) : 304); }

template <typename TX, typename TG, int VEC, int NV, bool kWarps>
cudaError_t start_back(const BackArgs &a, int threads, float *gw, cudaStream_t s) {
    const int blocks = back_blocks(a.n);
    k_rms_backward<TX, TG, VEC, NV, kWarps><<<blocks, threads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_rms_columns<<<(a.d + 31) / 32, 256, 0, s>>>(a.part, blocks, a.d, gw);
    return cudaGetLastError();
}

template <typename TX, typename TG>
cudaError_t backward(const BackArgs &a, float *gw, cudaStream_t s) {
    constexpr int W = 16 / (int)(sizeof(TX) > sizeof(TG) ? sizeof(TX) : sizeof(TG));
    const bool wide = a.d % W == 0 && multiple(a.r, a.rs, sizeof(TX), W * sizeof(TX)) &&
                      multiple(a.g, a.gs, sizeof(TG), W * sizeof(TG)) && multiple(a.gr, a.grs, sizeof(TG), W * sizeof(TG)) &&
                      multiple(a.gx, a.gxs, sizeof(TG), W * sizeof(TG)) && multiple(a.w, 0, 1, a.w_type == HC_F32 ? 16 : 8);
    const int per = wide ? W : 1, need = (a.d + per - 1) / per;
    const int threads = need > 1024 ? 1024 : (need + 31) / 32 * 32;
    if (wide) {
        if (need <= 64) return start_back<TX, TG, W, 2, true>(a, 256, gw, s);
        if (need <= 1024) return start_back<TX, TG, W, 1, false>(a, threads, gw, s);
        if (need <= 2048) return start_back<TX, TG, W, 2, false>(a, threads, gw, s);
        return start_back<TX, TG, W, 4, false>(a, threads, gw, s);
    }
    if (need <= 128) return start_back<TX, TG, 1, 4, true>(a, 256, gw, s);
    if (need <= 1024) return start_back<TX, TG, 1, 1, false>(a, threads, gw, s);
    if (need <= 4096) return start_back<TX, TG, 1, 4, false>(a, threads, gw, s);
    return start_back<TX, TG, 1, 16, false>(a, threads, gw, s);
}

// ------------------------------------------------------------ casts
// Rows in groups of 128: VEC values a thread, 128 / VEC threads a group, kCastVectors
// groups a thread one after the other, their loads all under way at once.
constexpr int kCastThreads = 256, kCastVectors = 4;
template <typename T, int VEC>
__global__ void __launch_bounds__(kCastThreads)
k_fp8_cast(const T *__restrict__ x, int64_t xs, int64_t n, int d, int groups, uint8_t *__restrict__ codes, int64_t cs,
           uint8_t *__restrict__ scales, int wide) {
    constexpr int kTeam = kFp8Block / VEC, kTeams = kCastThreads / kTeam;
    const int t = threadIdx.x % kTeam;
    const int64_t first = (int64_t)blockIdx.x * (kTeams * kCastVectors) + threadIdx.x / kTeam, count = n * groups;
    Vec<T, VEC> v[kCastVectors];
#pragma unroll
    for (int i = 0; i < kCastVectors; ++i) {
        const int64_t g = first + i * kTeams, row = g / groups;
        const int c = (int)(g - row * groups) * kFp8Block + t * VEC;
        if (g < count && c < d) v[i] = *reinterpret_cast<const Vec<T, VEC> *>(x + row * xs + c);
    }
#pragma unroll
    for (int i = 0; i < kCastVectors; ++i) {
        const int64_t g = first + i * kTeams, row = g / groups;
        const int c = (int)(g - row * groups) * kFp8Block + t * VEC;
        const bool in = g < count && c < d;
        float f[VEC], amax = 0.0f;
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = in ? to_f(v[i].v[k]) : 0.0f, amax = largest(amax, f[k]);
        const uint32_t byte = fp8_scale_byte(largest_of_group<VEC>(amax));
        if (!in) continue;
        put_codes<VEC>(codes + row * cs + c, f, fp8_inverse(byte), wide);
        if (t == 0) scales[g] = (uint8_t)byte;
    }
}
// ... of rows that start anywhere: a warp a group, four values a lane, one by one
template <typename T>
__global__ void __launch_bounds__(kCastThreads)
k_fp8_cast_any(const T *__restrict__ x, int64_t xs, int64_t n, int d, int groups, uint8_t *__restrict__ codes, int64_t cs,
               uint8_t *__restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t g = (int64_t)blockIdx.x * (kCastThreads / 32) + (threadIdx.x >> 5), row = g / groups;
    if (row >= n) return;
    const int c0 = (int)(g - row * groups) * kFp8Block + lane;
    float f[4], amax = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = c0 + 32 * k < d ? to_f(x[row * xs + c0 + 32 * k]) : 0.0f, amax = largest(amax, f[k]);
    const uint32_t byte = fp8_scale_byte(largest_of_group<4>(amax));
    const float inv = fp8_inverse(byte);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (c0 + 32 * k < d) codes[row * cs + c0 + 32 * k] = (uint8_t)fp8_codes(f[k] * inv, 0.0f);
    if (lane == 0) scales[g] = (uint8_t)byte;
}

template <typename T>
cudaError_t cast(const void *x, int64_t xs, int64_t n, int d, uint8_t *codes, int64_t cs, uint8_t *scales, cudaStream_t s) {
    constexpr int W = kWide<T>;
    const int groups = (d + kFp8Block - 1) / kFp8Block;
    const int64_t count = n * groups;
    const T *const p = static_cast<const T *>(x);
    if (d % W == 0 && multiple(x, xs, sizeof(T), 16)) {
        constexpr int kEach = kCastThreads / (kFp8Block / W) * kCastVectors;
        k_fp8_cast<T, W><<<(unsigned)((count + kEach - 1) / kEach), kCastThreads, 0, s>>>(p, xs, n, d, groups, codes, cs, scales,
                                                                                         multiple(codes, cs, 1, W));
    } else {
        k_fp8_cast_any<T><<<(unsigned)((count + 7) / 8), kCastThreads, 0, s>>>(p, xs, n, d, groups, codes, cs, scales);
    }
    return cudaGetLastError();
}

// A matrix [N, K] in blocks of 128 x 128: a thread block each, thread t the columns
// 4 (t % 32) .. + 3 of the rows t / 32 + 8 i.
template <typename T, bool kVector>
__global__ void __launch_bounds__(256)
k_fp8_cast_weights(const T *__restrict__ w, int64_t N, int K, int64_t row_blocks, int col_blocks, uint8_t *__restrict__ codes,
                   uint8_t *__restrict__ scales) {
    __shared__ float red[8];
    const int64_t block = blockIdx.x, matrix = block / (row_blocks * col_blocks);
    const int64_t in = block - matrix * row_blocks * col_blocks, rb = in / col_blocks;
    const int c = (int)(in - rb * col_blocks) * kFp8Block + (threadIdx.x & 31) * 4;
    const int64_t r0 = rb * kFp8Block + (threadIdx.x >> 5), base = matrix * N * K;
    Vec<T, 4> v[16];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t at = base + (r0 + 8 * i) * K + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i].v[k] = from_f<T>(0.0f);
        if (r0 + 8 * i >= N) continue;
        if (kVector) {
            if (c < K) v[i] = *reinterpret_cast<const Vec<T, 4> *>(w + at);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < K) v[i].v[k] = w[at + k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) amax = largest(amax, to_f(v[i].v[k]));
    }
    amax = largest_of_group<4>(amax);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, red[k]);
    const uint32_t byte = fp8_scale_byte(amax);
    const float inv = fp8_inverse(byte);
    if (threadIdx.x == 0) scales[block] = (uint8_t)byte;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (r0 + 8 * i >= N || c >= K) continue;
        uint8_t *o = codes + base + (r0 + 8 * i) * K + c;
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = to_f(v[i].v[k]);
        if (kVector) {
            put_codes<4>(o, f, inv, 1);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < K) o[k] = (uint8_t)fp8_codes(f[k] * inv, 0.0f);
        }
    }
}

template <typename T>
cudaError_t cast_weights(const void *w, int64_t count, int64_t N, int K, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int64_t rb = (N + kFp8Block - 1) / kFp8Block;
    const int cb = (K + kFp8Block - 1) / kFp8Block;
    const unsigned grid = (unsigned)(count * rb * cb);
    const T *const p = static_cast<const T *>(w);
    if (K % 4 == 0 && multiple(w, 0, 1, 4 * sizeof(T)) && multiple(codes, 0, 1, 4))
        k_fp8_cast_weights<T, true><<<grid, 256, 0, s>>>(p, N, K, rb, cb, codes, scales);
    else
        k_fp8_cast_weights<T, false><<<grid, 256, 0, s>>>(p, N, K, rb, cb, codes, scales);
    return cudaGetLastError();
}

}  // namespace rn

cudaError_t launch_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride, hc_dtype type,
                            const void *w, hc_dtype w_type, int64_t n, int d, float eps, void *r, int64_t r_stride, void *y,
                            int64_t y_stride, uint8_t *codes, int64_t codes_stride, uint8_t *scales, float *rstd,
                            cudaStream_t s) {
    const rn::Args a{x, residual, w, x_stride, residual_stride, w_type, n, d, eps, r, y, r_stride, y_stride,
                     codes, scales, codes_stride, rstd, 0};
    if (type == HC_F32) return rn::forward<float>(a, s);
    return type == HC_BF16 ? rn::forward<__nv_bfloat16>(a, s) : rn::forward<__half>(a, s);
}

size_t rms_norm_backward_workspace_bytes(int64_t n, int d) { return (size_t)rn::back_blocks(n) * d * 4; }

cudaError_t launch_rms_norm_backward(const void *g_y, int64_t g_stride, const void *g_r, int64_t g_r_stride, hc_dtype g_type,
                                     const void *r, int64_t r_stride, hc_dtype type, const void *w, hc_dtype w_type,
                                     const float *rstd, int64_t n, int d, void *g_x, int64_t gx_stride, float *g_w,
                                     void *workspace, cudaStream_t s) {
    if (n == 0) return cudaMemsetAsync(g_w, 0, (size_t)d * 4, s);
    const rn::BackArgs a{g_y, g_r, r, w, g_stride, g_r_stride, r_stride, w_type, rstd, n, d, g_x, gx_stride,
                         static_cast<float *>(workspace)};
    if (type == HC_F32) return rn::backward<float, float>(a, g_w, s);
    if (type == HC_BF16)
        return g_type == HC_F32 ? rn::backward<__nv_bfloat16, float>(a, g_w, s) : rn::backward<__nv_bfloat16, __nv_bfloat16>(a, g_w, s);
    return g_type == HC_F32 ? rn::backward<__half, float>(a, g_w, s) : rn::backward<__half, __half>(a, g_w, s);
}

cudaError_t launch_fp8_cast(const void *x, int64_t x_stride, hc_dtype type, int64_t n, int d, uint8_t *codes, int64_t codes_stride,
                            uint8_t *scales, cudaStream_t s) {
    if (type == HC_F32) return rn::cast<float>(x, x_stride, n, d, codes, codes_stride, scales, s);
    return type == HC_BF16 ? rn::cast<__nv_bfloat16>(x, x_stride, n, d, codes, codes_stride, scales, s)
                           : rn::cast<__half>(x, x_stride, n, d, codes, codes_stride, scales, s);
}

cudaError_t launch_fp8_cast_weights(const void *w, hc_dtype type, int64_t count, int64_t N, int K, uint8_t *codes, uint8_t *scales,
                                    cudaStream_t s) {
    if (type == HC_F32) return rn::cast_weights<float>(w, count, N, K, codes, scales, s);
    return type == HC_BF16 ? rn::cast_weights<__nv_bfloat16>(w, count, N, K, codes, scales, s)
                           : rn::cast_weights<__half>(w, count, N, K, codes, scales, s);
}

}  // namespace hc
