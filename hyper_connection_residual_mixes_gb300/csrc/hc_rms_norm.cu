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
//
// Bound by HBM: each input is read once, each output written once, and a row stays in
// registers (forward) or in its slot of shared memory (backward, in the ring) between the sums and what
// needs them.  Long runs of rows come through a ring of bulk copies, short ones and rows that do not
// line up straight into registers; in the backward these, and rows of less than 1,024 or more than 8,192
// columns, are read twice, the second time from L1 or L2.  Measured, in us, and of 6,767 GB/s (a plain
// copy): forward of 65,536 x 5,120 bf16 with residual and 8-bit output 361 (0.96), backward of
// 8,192 x 5,120 with fp32 gradients 89 (0.97), 16 rows of 5,120 2.6 (one row's load, sum and write
// after another), 1,501 x 1,031 fp32 backward 12.  Rows that do not line up: 0.1 to 0.25, single
// values make too many loads.
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

// ------------------------------------------------------------ rows through a ring
// Many long rows: a block walks over rows that bulk copies bring into slots of shared
// memory ahead of it (one thread issues them; a block barrier of a row's reduction
// says that a slot has been read).
constexpr int kMostSlots = 6;
struct Ring {
    uint64_t full[kMostSlots];
    volatile int abort;
};
struct Place {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) slot = 0, parity ^= 1u;
    }
};
// All threads wait for a row; a wait that runs out is reported and the block goes on (its rows are
// then wrong, but every barrier is met).
__device__ __forceinline__ void ring_wait(Ring &r, const Place &p) { mbar_wait<false>(smem_u32(&r.full[p.slot]), p.parity, &r.abort); }
__device__ __forceinline__ void ring_init(Ring &r, int slots) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(smem_u32(&r.full[i]), 1);
        r.abort = 0;
        fence_mbar_init_cluster();
    }
    __syncthreads();
}
// After a wait that ran out: the copies still in flight must land before the block leaves.
__device__ __forceinline__ void ring_leave(Ring &r, int64_t its, int slots) {
    if (threadIdx.x == 0 && r.abort)
        for (int64_t k = its > slots ? its - slots : 0; k < its; ++k)
            for (uint32_t i = 0; i < (1u << 22); ++i) {
                if (mbar_try_wait(smem_u32(&r.full[k % slots]), (uint32_t)(k / slots) & 1u)) break;
                __nanosleep(128);
            }
}

// 16 columns a thread, in runs of 16 bytes.
template <typename T, int kMaxThreads, int kMinBlocks>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks) k_rms_norm_ring(const Args a, int slots) {
    constexpr int V = 16 / (int)sizeof(T), NV = 16 / V;
    extern __shared__ __align__(16) uint8_t s_rows[];
    __shared__ Ring ring;
    __shared__ float red[2][32];
    const int t = threadIdx.x, tpr = blockDim.x, warp = t >> 5, lane = t & 31, nw = tpr >> 5, d = a.d;
    const uint32_t row_bytes = (uint32_t)d * sizeof(T), slot_bytes = row_bytes * (a.residual ? 2 : 1);
    const int groups = (d + kFp8Block - 1) / kFp8Block;
    // (a block's rows lie together: 361 us for 65,536 rows of 5,120 bf16, for every gridDim-th row 368)
    const int64_t first = a.n * blockIdx.x / gridDim.x, rows = a.n * (blockIdx.x + 1) / gridDim.x - first;
    ring_init(ring, slots);
    const auto fetch = [&](int slot, int64_t it) {
        const uint32_t bar = smem_u32(&ring.full[slot]), to = smem_u32(s_rows) + (uint32_t)slot * slot_bytes;
        const int64_t row = first + it;
        mbar_arrive_expect_tx(bar, slot_bytes);
        bulk_load(to, static_cast<const T *>(a.x) + row * a.xs, row_bytes, bar);
        if (a.residual) bulk_load(to + row_bytes, static_cast<const T *>(a.residual) + row * a.res_s, row_bytes, bar);
    };
    if (t == 0)
        for (int it = 0; it < slots && it < rows; ++it) fetch(it, it);
    const float inv_d = 1.0f / (float)d;
    f32x2 w[NV][V / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[V] = {};
        if ((t + i * tpr) * V < d) params<V>(a.w, a.w_type, (t + i * tpr) * V, f);
#pragma unroll
        for (int k = 0; k < V; k += 2) w[i][k / 2] = f2_make(f[k], f[k + 1]);
    }
    Place place;
    int buf = 0;
    for (int64_t it = 0; it < rows; ++it, buf ^= 1) {
        const int64_t row = first + it;
        ring_wait(ring, place);
        const uint8_t *const slot = s_rows + (uint32_t)place.slot * slot_bytes;
        f32x2 v[NV][V / 2], acc = f2_dup(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * V;
#pragma unroll
            for (int k = 0; k < V / 2; ++k) v[i][k] = f2_dup(0.0f);
            if (c >= d) continue;
            Vec<T, V> x = *reinterpret_cast<const Vec<T, V> *>(slot + c * sizeof(T));
            if (a.residual) {
                const Vec<T, V> u = *reinterpret_cast<const Vec<T, V> *>(slot + row_bytes + c * sizeof(T));
#pragma unroll
                for (int k = 0; k < V; k += 2) put_pair(x, k, f2_add(pair(x, k), pair(u, k)));
                *reinterpret_cast<Vec<T, V> *>(static_cast<T *>(a.r) + row * a.rs + c) = x;
            }
#pragma unroll
            for (int k = 0; k < V; k += 2) v[i][k / 2] = pair(x, k), acc = f2_fma(v[i][k / 2], v[i][k / 2], acc);
        }
        const float sum = warp_sum(f2_hsum(acc));
        // (two buffers: a warp writes the next row's while a slow one still reads these)
        if (lane == 0) red[buf][warp] = sum;
        __syncthreads();
        if (t == 0 && it + slots < rows) fetch(place.slot, it + slots);  // every thread has read the slot
        place.next(slots);
        const float rstd = rsqrt_newton(fmaf(warp_sum(lane < nw ? red[buf][lane] : 0.0f), inv_d, a.eps));
        if (t == 0 && a.rstd) a.rstd[row] = rstd;
        const f32x2 rs = f2_dup(rstd);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * V;
#pragma unroll
            for (int k = 0; k < V / 2; ++k) v[i][k] = f2_mul(f2_mul(v[i][k], rs), w[i][k]);
            if (a.y && c < d) {
                Vec<T, V> o;
#pragma unroll
                for (int k = 0; k < V; k += 2) put_pair(o, k, v[i][k / 2]);
                *reinterpret_cast<Vec<T, V> *>(static_cast<T *>(a.y) + row * a.ys + c) = o;
            }
            if (!a.codes) continue;
            float f[V], amax = 0.0f;
#pragma unroll
            for (int k = 0; k < V; k += 2) f2_split(v[i][k / 2], f[k], f[k + 1]);
#pragma unroll
            for (int k = 0; k < V; ++k) amax = largest(amax, f[k]);
            const uint32_t byte = fp8_scale_byte(largest_of_group<V>(amax));
            if (c >= d) continue;
            put_codes<V>(a.codes + row * a.cs + c, f, fp8_inverse(byte), a.codes_wide);
            if (c % kFp8Block == 0) a.scales[row * groups + c / kFp8Block] = (uint8_t)byte;
        }
    }
    ring_leave(ring, rows, slots);
}

constexpr int kDevices = 64;
constexpr int kSmemBlock = 227 * 1024, kSmemSm = 228 * 1024;  // shared memory of a block, of an SM
int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kDevices ? dev : 0;
}
int sm_count() {
    static std::atomic<int> sms[kDevices];  // (any host thread may be the first to ask)
    const int dev = current_device();
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    sms[dev].store(n, std::memory_order_relaxed);
    return n;
}
// Slots of a ring and blocks of a launch: a grid that fills the SMs once (`most_per_sm` blocks
// each at the most), with as many slots as fit in `room` bytes of an SM, two where two fit
// (of fp32 rows of 16,384 with a residual one does).  What a kernel
// needs is asked for and set once per device.
template <auto kKernel>
cudaError_t ring_shape(int threads, int slot_bytes, int most_per_sm, int room, int64_t most, int *slots, int *blocks) {
    static std::atomic<int> regs[kDevices];
    const int dev = current_device();
    int r = regs[dev].load(std::memory_order_acquire);
    if (!r) {
        cudaFuncAttributes fa{};
        cudaError_t e = cudaFuncGetAttributes(&fa, kKernel);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBlock - (int)fa.sharedSizeBytes);
        if (e != cudaSuccess) return e;
        r = fa.numRegs;
        regs[dev].store(r, std::memory_order_release);  // (the attribute is set for whoever reads it)
    }
    const int warps = threads / 32, by_regs = 65536 / ((r * 32 + 255) / 256 * 256 * warps), by_threads = 64 / warps;
    int per_sm = by_regs < by_threads ? by_regs : by_threads;
    per_sm = per_sm < most_per_sm ? per_sm : most_per_sm;
    if (per_sm < 1) per_sm = 1;
    const int extra = 2048;  // a block's other shared memory
    while (per_sm > 1 && (kSmemSm / per_sm - extra) / slot_bytes < 2) --per_sm;
    const int fit = ((per_sm > 1 ? kSmemSm / per_sm : kSmemBlock) - extra) / slot_bytes;
    int n = room / per_sm / slot_bytes;
    n = n < 2 ? 2 : n > kMostSlots ? kMostSlots : n;
    *slots = n < fit ? n : fit;
    const int64_t grid = (int64_t)per_sm * sm_count();
    *blocks = (int)(grid < most ? grid : most);
    return cudaSuccess;
}
// (640 threads an SM and some 80 KB of rows on their way to it: of 65,536 rows of 5,120 bf16, to 8 bits,
// two blocks with two slots each 361 us, with three 405, five 417; three blocks with two 400.)
template <auto kKernel>
cudaError_t start_ring(const Args &a, int threads, int slot_bytes, cudaStream_t s) {
    int slots = 0, blocks = 0;
    const cudaError_t e = ring_shape<kKernel>(threads, slot_bytes, threads < 640 ? 640 / threads : 1, 84 * 1024, a.n, &slots, &blocks);
    if (e != cudaSuccess) return e;
    kKernel<<<blocks, threads, slots * slot_bytes, s>>>(a, slots);
    return cudaGetLastError();
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
    const int per = wide ? W : 1, need = (a.d + per - 1) / per;
    // (the ring for rows that fill it several times: 16,384 values an SM.  65,536 x 5,120 bf16: 361 us against
    // 417 of a block a row; for 16 rows of 5,120 a block a row 2.6 us, the ring's set-up alone takes 2)
    if (wide && a.d > 512 && a.n * a.d >= 16384 * (int64_t)sm_count()) {
        const int threads = (a.d + 511) / 512 * 32, slot = (int)(a.d * size) * (a.residual ? 2 : 1);
        if (threads <= 320) return start_ring<k_rms_norm_ring<T, 320, 2>>(a, threads, slot, s);
        return start_ring<k_rms_norm_ring<T, 1024, 1>>(a, threads, slot, s);
    }
    if (wide) {
        if (need <= 32) return start<T, W, 1, true>(a, 0, s);
        if (need <= 64) return start<T, W, 2, true>(a, 0, s);
        const int threads = need > 1024 ? 1024 : (need + 31) / 32 * 32;
        if (need <= 1024) return start<T, W, 1, false>(a, threads, s);
        if (need <= 2048) return start<T, W, 2, false>(a, threads, s);
        return start<T, W, 4, false>(a, threads, s);
    }
    if (need <= 128) return start<T, 1, 4, true>(a, 0, s);
    // (one by one: whole groups of 128 values a pass)
    const auto threads = [&](int each) { return (need + each * 128 - 1) / (each * 128) * 128; };
    if (need <= 1024) return start<T, 1, 4, false>(a, threads(4), s);
    if (need <= 8192) return start<T, 1, 8, false>(a, threads(8), s);
    return start<T, 1, 16, false>(a, 1024, s);
}

// ------------------------------------------------------------ backward
// A block walks over rows, its threads own columns and keep their sums of g xh; it
// leaves a row of partial sums in the workspace, k_rms_columns adds these in a fixed
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

// The same with the rows of r, g and g_r through a ring: 8 columns a thread in two runs of 4.
// Both passes over a row read it from its slot, which is filled again once the next
// row's barrier has passed.  8,192 x 5,120, fp32 gradients: 179 us with rows read twice through
// L2, 89 here.  A block has 1,024 threads at the most, so rows past 8,192 take the kernel above (0.53 of HBM).
template <typename TX, typename TG, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, 1) k_rms_backward_ring(const BackArgs a, int slots) {
    extern __shared__ __align__(16) uint8_t s_rows[];
    __shared__ Ring ring;
    __shared__ float red[2][32];
    const int t = threadIdx.x, tpr = blockDim.x, warp = t >> 5, lane = t & 31, nw = tpr >> 5, d = a.d;
    const uint32_t x_bytes = (uint32_t)d * sizeof(TX), g_bytes = (uint32_t)d * sizeof(TG), slot_bytes = x_bytes + g_bytes * (a.gr ? 2 : 1);
    const float inv_d = 1.0f / (float)d;
    const int64_t rows = (a.n - 1 - blockIdx.x) / gridDim.x + 1;
    ring_init(ring, slots);
    const auto fetch = [&](int slot, int64_t it) {
        const uint32_t bar = smem_u32(&ring.full[slot]), to = smem_u32(s_rows) + (uint32_t)slot * slot_bytes;
        const int64_t row = blockIdx.x + it * gridDim.x;
        mbar_arrive_expect_tx(bar, slot_bytes);
        bulk_load(to, static_cast<const TX *>(a.r) + row * a.rs, x_bytes, bar);
        bulk_load(to + x_bytes, static_cast<const TG *>(a.g) + row * a.gs, g_bytes, bar);
        if (a.gr) bulk_load(to + x_bytes + g_bytes, static_cast<const TG *>(a.gr) + row * a.grs, g_bytes, bar);
    };
    if (t == 0)
        for (int it = 0; it < slots && it < rows; ++it) fetch(it, it);
    f32x2 w[2][2], aw[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4] = {};
        if ((t + i * tpr) * 4 < d) params<4>(a.w, a.w_type, (t + i * tpr) * 4, f);
#pragma unroll
        for (int k = 0; k < 2; ++k) w[i][k] = f2_make(f[2 * k], f[2 * k + 1]), aw[i][k] = f2_dup(0.0f);
    }
    Place place;
    int before = 0, buf = 0;
    float rstd_next = __ldg(a.rstd + blockIdx.x);
    for (int64_t it = 0; it < rows; ++it, buf ^= 1) {
        const int64_t row = blockIdx.x + it * gridDim.x;
        const float rstd = rstd_next;
        if (it + 1 < rows) rstd_next = __ldg(a.rstd + row + gridDim.x);
        ring_wait(ring, place);
        const uint8_t *const slot = s_rows + (uint32_t)place.slot * slot_bytes;
        const f32x2 rs = f2_dup(rstd);
        f32x2 acc = f2_dup(0.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = (t + i * tpr) * 4;
            if (c >= d) continue;
            const Vec<TX, 4> x = *reinterpret_cast<const Vec<TX, 4> *>(slot + c * sizeof(TX));
            const Vec<TG, 4> g = *reinterpret_cast<const Vec<TG, 4> *>(slot + x_bytes + c * sizeof(TG));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x2 xh = f2_mul(pair(x, 2 * k), rs), gk = pair(g, 2 * k);
                acc = f2_fma(f2_mul(gk, w[i][k]), xh, acc);
                aw[i][k] = f2_fma(gk, xh, aw[i][k]);
            }
        }
        const float sum = warp_sum(f2_hsum(acc));
        // (two buffers: a warp writes the next row's while a slow one still reads these)
        if (lane == 0) red[buf][warp] = sum;
        __syncthreads();
        if (t == 0 && it > 0 && it - 1 + slots < rows) fetch(before, it - 1 + slots);  // every thread is done with the row before
        before = place.slot;
        place.next(slots);
        const f32x2 m = f2_dup(-warp_sum(lane < nw ? red[buf][lane] : 0.0f) * inv_d);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = (t + i * tpr) * 4;
            if (c >= d) continue;
            const Vec<TX, 4> x = *reinterpret_cast<const Vec<TX, 4> *>(slot + c * sizeof(TX));
            const Vec<TG, 4> g = *reinterpret_cast<const Vec<TG, 4> *>(slot + x_bytes + c * sizeof(TG));
            Vec<TG, 4> past, o;
            if (a.gr) past = *reinterpret_cast<const Vec<TG, 4> *>(slot + x_bytes + g_bytes + c * sizeof(TG));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f32x2 v = f2_mul(rs, f2_fma(f2_mul(pair(x, 2 * k), rs), m, f2_mul(pair(g, 2 * k), w[i][k])));
                if (a.gr) v = f2_add(v, pair(past, 2 * k));
                put_pair(o, 2 * k, v);
            }
            *reinterpret_cast<Vec<TG, 4> *>(static_cast<TG *>(a.gx) + row * a.gxs + c) = o;
        }
    }
    ring_leave(ring, rows, slots);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = (t + i * tpr) * 4;
        if (c >= d) continue;
        float f[4];
        f2_split(aw[i][0], f[0], f[1]), f2_split(aw[i][1], f[2], f[3]);
        *reinterpret_cast<float4 *>(a.part + (int64_t)blockIdx.x * d + c) = make_float4(f[0], f[1], f[2], f[3]);
    }
}

// g_w: the blocks' partial sums added in a fixed order.  A block takes 32 columns;
// its warps share the rows.
constexpr int kColumnWarps = 16;
__global__ void __launch_bounds__(32 * kColumnWarps) k_rms_columns(const float *__restrict__ part, int blocks, int d, float *__restrict__ gw) {
    __shared__ float s[kColumnWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.0f;
    if (c < d) {
#pragma unroll 10
        for (int b = warp; b < blocks; b += kColumnWarps) v += __ldcg(part + (int64_t)b * d + c);
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < d) {
        for (int k = 1; k < kColumnWarps; ++k) v += s[k][lane];
        gw[c] = v;
    }
}

// most blocks of the backward, and so rows of partial sums
int64_t most_blocks(int64_t n, int d) {
    const int64_t most = d < 1024 ? 1216 : d <= 2048 ? 608 : 304;
    return n < most ? n : most;
}

cudaError_t start_columns(const BackArgs &a, int blocks, float *gw, cudaStream_t s) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.d + 31) / 32)), cfg.blockDim = dim3(32 * kColumnWarps);
    cfg.stream = s, cfg.attrs = &early, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rms_columns, (const float *)a.part, blocks, a.d, gw);
}
template <typename TX, typename TG, int VEC, int NV, bool kWarps>
cudaError_t start_back(const BackArgs &a, int threads, float *gw, cudaStream_t s) {
    int64_t blocks = most_blocks(a.n, a.d);
    if (kWarps && blocks > (a.n + 7) / 8) blocks = (a.n + 7) / 8;
    k_rms_backward<TX, TG, VEC, NV, kWarps><<<(unsigned)blocks, threads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : start_columns(a, (int)blocks, gw, s);
}
template <auto kKernel>
cudaError_t start_back_ring(const BackArgs &a, int threads, int slot_bytes, float *gw, cudaStream_t s) {
    int slots = 0, blocks = 0;
    cudaError_t e = ring_shape<kKernel>(threads, slot_bytes, threads < 640 ? 640 / threads : 1, kSmemBlock, most_blocks(a.n, a.d), &slots, &blocks);
    if (e != cudaSuccess) return e;
    kKernel<<<blocks, threads, slots * slot_bytes, s>>>(a, slots);
    return (e = cudaGetLastError()) != cudaSuccess ? e : start_columns(a, blocks, gw, s);
}

template <typename TX, typename TG>
cudaError_t backward(const BackArgs &a, float *gw, cudaStream_t s) {
    constexpr int W = 16 / (int)(sizeof(TX) > sizeof(TG) ? sizeof(TX) : sizeof(TG));
    const bool wide = a.d % W == 0 && multiple(a.r, a.rs, sizeof(TX), W * sizeof(TX)) &&
                      multiple(a.g, a.gs, sizeof(TG), W * sizeof(TG)) && multiple(a.gr, a.grs, sizeof(TG), W * sizeof(TG)) &&
                      multiple(a.gx, a.gxs, sizeof(TG), W * sizeof(TG)) && multiple(a.w, 0, 1, a.w_type == HC_F32 ? 16 : 8);
    const bool bulk = wide && a.d * sizeof(TX) % 16 == 0 && a.d * sizeof(TG) % 16 == 0 && multiple(a.r, a.rs, sizeof(TX), 16) &&
                      multiple(a.g, a.gs, sizeof(TG), 16) && multiple(a.gr, a.grs, sizeof(TG), 16);
    if (bulk && a.d >= 1024 && a.d <= 8192) {
        const int threads = (a.d + 255) / 256 * 32, slot = a.d * (int)(sizeof(TX) + sizeof(TG) * (a.gr ? 2 : 1));
        if (threads <= 640) return start_back_ring<k_rms_backward_ring<TX, TG, 640>>(a, threads, slot, gw, s);
        return start_back_ring<k_rms_backward_ring<TX, TG, 1024>>(a, threads, slot, gw, s);
    }
    // (four vectors a thread where rows are long enough: more rows are under way then)
    const int per = wide ? W : 1, need = (a.d + per - 1) / per, threads = ((need + 3) / 4 + 31) / 32 * 32;
    if (wide) {
        if (need <= 64) return start_back<TX, TG, W, 2, true>(a, 256, gw, s);
        return start_back<TX, TG, W, 4, false>(a, threads, gw, s);
    }
    if (need <= 128) return start_back<TX, TG, 1, 4, true>(a, 256, gw, s);
    if (need <= 4096) return start_back<TX, TG, 1, 4, false>(a, threads, gw, s);
    return start_back<TX, TG, 1, 16, false>(a, 1024, gw, s);
}

// ------------------------------------------------------------ casts
// Rows in groups of 128: VEC values a thread, 128 / VEC threads a group, kCastVectors
// groups a thread one after the other, their loads all under way at once.  kFlat: dense rows of
// whole groups, whose places need no division.  8,192 x 10,240 bf16: 38 us, 0.98 of HBM.
constexpr int kCastThreads = 256, kCastVectors = 4;
template <typename T, int VEC, bool kFlat>
__global__ void __launch_bounds__(kCastThreads)
k_fp8_cast(const T *__restrict__ x, int64_t xs, int64_t n, int d, int groups, uint8_t *__restrict__ codes, int64_t cs,
           uint8_t *__restrict__ scales, int wide) {
    constexpr int kTeam = kFp8Block / VEC, kTeams = kCastThreads / kTeam;
    const int t = threadIdx.x % kTeam;
    const int64_t first = (int64_t)blockIdx.x * (kTeams * kCastVectors) + threadIdx.x / kTeam, count = n * groups;
    Vec<T, VEC> v[kCastVectors];
    bool in[kCastVectors];
    int64_t to[kCastVectors];
#pragma unroll
    for (int i = 0; i < kCastVectors; ++i) {
        const int64_t g = first + i * kTeams;
        int64_t from = to[i] = g * kFp8Block + t * VEC;
        in[i] = g < count;
        if (!kFlat) {
            // (a division of 32 bits where that will do)
            const int64_t row = count >> 31 ? g / groups : (int64_t)((uint32_t)g / (uint32_t)groups);
            const int c = (int)(g - row * groups) * kFp8Block + t * VEC;
            from = row * xs + c, to[i] = row * cs + c, in[i] &= c < d;
        }
        if (in[i]) v[i] = *reinterpret_cast<const Vec<T, VEC> *>(x + from);
    }
#pragma unroll
    for (int i = 0; i < kCastVectors; ++i) {
        float f[VEC], amax = 0.0f;
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = in[i] ? to_f(v[i].v[k]) : 0.0f, amax = largest(amax, f[k]);
        const uint32_t byte = fp8_scale_byte(largest_of_group<VEC>(amax));
        if (!in[i]) continue;
        put_codes<VEC>(codes + to[i], f, fp8_inverse(byte), wide);
        if (t == 0) scales[first + i * kTeams] = (uint8_t)byte;
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
        const unsigned grid = (unsigned)((count + kEach - 1) / kEach);
        const int codes_wide = multiple(codes, cs, 1, W);
        if (d % kFp8Block == 0 && (n == 1 || (xs == d && cs == d)))
            k_fp8_cast<T, W, true><<<grid, kCastThreads, 0, s>>>(p, xs, n, d, groups, codes, cs, scales, codes_wide);
        else
            k_fp8_cast<T, W, false><<<grid, kCastThreads, 0, s>>>(p, xs, n, d, groups, codes, cs, scales, codes_wide);
    } else {
        k_fp8_cast_any<T><<<(unsigned)((count + 7) / 8), kCastThreads, 0, s>>>(p, xs, n, d, groups, codes, cs, scales);
    }
    return cudaGetLastError();
}

// A matrix [N, K] in blocks of 128 x 128: a thread block each, thread t the columns
// 4 (t % 32) .. + 3 of the rows t / 32 + 8 i.  16,384 x 5,120: 178 us of bf16 (0.21 of HBM), 185 of fp32
// (0.33); one by one, 5,121 wide, 367 and 388.  Weights are cast once: nothing was done about it yet.
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

size_t rms_norm_backward_workspace_bytes(int64_t n, int d) { return (size_t)rn::most_blocks(n, d) * d * 4; }

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

cudaError_t consume_rms_norm_device_error(cudaStream_t s, unsigned int *flag) {
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
