// hc_adamw.cu -- one AdamW step over many tensors, for GB300.
//
// Per value, with t the step number:
//   g <- g * grad_scale                                  (when given)
//   m <- m beta1 + g (1 - beta1),   v <- v beta2 + g g (1 - beta2),
//   p <- p (1 - lr wd) - m / (sqrt(v) / sqrt(1 - beta2^t) + eps) * lr / (1 - beta1^t).
// Every operation is an fp32 operation rounded once, in the order written
// (no fused multiply-adds), so the result does not depend on how the tensors
// are laid out or split over launches; p is rounded once more to its own type.
//
// States are fp32, or 8 bits in the format of the MXFP8 cast: groups of 32
// values of a tensor share a power-of-two scale, each value is an E4M3 number
// times it.  m is held so, and of v its root r = sqrt(v), whose range is half
// as wide in powers of two; a positive r never becomes zero (it takes the
// smallest code instead), because m / (0 + eps) would throw a weight away.
// The update itself uses the unrounded m and v.
//
// The step reads and writes each value once and is bound by that: 28 bytes a
// value for fp32 parameters, gradients and states, 10.1 for bf16 parameters
// and gradients with 8-bit states.  All tensors of a call go in one launch
// (their descriptions are kernel parameters, 448 at the most).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "hc_device.cuh"
#include "hc_sublayer.h"

namespace hc {

namespace aw {

constexpr int kThreads = 256;
constexpr int kVec = 4;      // values a thread holds at a time: 16 bytes of fp32, an eighth of a group of 32
constexpr int kUnroll = 4;
constexpr int kChunk = kThreads * kVec * kUnroll;  // values per block

struct Desc {
    void *p;
    const void *g;
    void *m, *v;
    uint8_t *ms, *vs;  // null: fp32 states
    void *copy;
    int64_t numel;
    uint32_t first_block;
    uint8_t p_type, g_type, copy_type, vec;  // vec: every pointer takes kVec-wide accesses
};

template <int CAP>
struct Descs {
    Desc d[CAP];
};

struct Scalars {
    float beta1, rest1, beta2, rest2, eps;
    float decay, rate, root;            // used when neither lr nor step is on the device
    double log_beta1, log_beta2;
    float lr, wd;
    int64_t step;
    const float *lr_dev;
    const int64_t *step_dev;
    const float *grad_scale;
};

template <typename T>
__device__ __forceinline__ float to_f(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __half2float(v);
    else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}
template <typename T>
struct alignas(sizeof(T) * kVec) Vec {
    T v[kVec];
};

// values [i, i + kVec) of p, those below n (the others read as zero)
template <typename T>
__device__ __forceinline__ Vec<T> load(const void *p, int64_t i, int64_t n, bool vec) {
    const T *q = static_cast<const T *>(p) + i;
    Vec<T> r{};
    if (vec && i + kVec <= n) {
        r = *reinterpret_cast<const Vec<T> *>(q);
    } else {
#pragma unroll
        for (int k = 0; k < kVec; ++k)
            if (i + k < n) r.v[k] = q[k];
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store(void *p, int64_t i, int64_t n, bool vec, const Vec<T> &r) {
    T *q = static_cast<T *>(p) + i;
    if (vec && i + kVec <= n) {
        *reinterpret_cast<Vec<T> *>(q) = r;
    } else {
#pragma unroll
        for (int k = 0; k < kVec; ++k)
            if (i + k < n) q[k] = r.v[k];
    }
}

// ---- the 8-bit states
__device__ __forceinline__ float scale_of(uint32_t byte) {  // 2^(byte - 127)
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
__device__ __forceinline__ void decode(const Vec<uint8_t> &c, float s, float (&o)[kVec]) {
#pragma unroll
    for (int k = 0; k < kVec; k += 2) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c.v[k] | (uint32_t)c.v[k + 1] << 8), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        o[k] = __fmul_rn(f.x, s), o[k + 1] = __fmul_rn(f.y, s);
    }
}
// codes of a thread's four values; the eight threads of a group agree on its scale
template <bool kRoot>
__device__ __forceinline__ Vec<uint8_t> encode(const float (&x)[kVec], uint8_t &byte) {
    float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    // the smallest power of two at or above a / 448; no finite a needs one above 2^120
    const uint32_t bits = __float_as_uint(__fdiv_rn(a, 448.0f));
    int e = (int)(bits >> 23) + ((bits & 0x7fffffu) != 0);
    e = e < 1 ? 1 : e > 247 ? 247 : e;
    byte = (uint8_t)e;
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
    Vec<uint8_t> c;
#pragma unroll
    for (int k = 0; k < kVec; k += 2) {
        const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(x[k] * inv, x[k + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        c.v[k] = (uint8_t)(two & 0xffu), c.v[k + 1] = (uint8_t)(two >> 8);
    }
    if (kRoot) {
#pragma unroll
        for (int k = 0; k < kVec; ++k)
            if (c.v[k] == 0 && x[k] > 0.0f) c.v[k] = 1;
    }
    return c;
}

struct Rates {
    float decay, rate, root, gscale;
};

template <typename TP, typename TG, bool kPacked>
__device__ __forceinline__ void chunk(const Desc &d, int64_t base, const Scalars &c, const Rates &r, bool scaled) {
    const int64_t n = d.numel;
    const bool vec = d.vec;
    Vec<TP> pv[kUnroll];
    Vec<TG> gv[kUnroll];
    Vec<float> mv[kPacked ? 1 : kUnroll], vv[kPacked ? 1 : kUnroll];
    Vec<uint8_t> mc[kPacked ? kUnroll : 1], vc[kPacked ? kUnroll : 1];
    uint8_t mb[kPacked ? kUnroll : 1], vb[kPacked ? kUnroll : 1];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + (int64_t)(u * kThreads + (int)threadIdx.x) * kVec;
        pv[u] = load<TP>(d.p, i, n, vec);
        gv[u] = load<TG>(d.g, i, n, vec);
        if constexpr (kPacked) {
            mc[u] = load<uint8_t>(d.m, i, n, vec);
            vc[u] = load<uint8_t>(d.v, i, n, vec);
            mb[u] = i < n ? d.ms[i >> 5] : 0;
            vb[u] = i < n ? d.vs[i >> 5] : 0;
        } else {
            mv[u] = load<float>(d.m, i, n, vec);
            vv[u] = load<float>(d.v, i, n, vec);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + (int64_t)(u * kThreads + (int)threadIdx.x) * kVec;
        float m[kVec], v[kVec], root[kVec], p[kVec];
        if constexpr (kPacked) {
            decode(mc[u], scale_of(mb[u]), m);
            decode(vc[u], scale_of(vb[u]), v);
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = __fmul_rn(v[k], v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < kVec; ++k) m[k] = mv[u].v[k], v[k] = vv[u].v[k];
        }
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            float g = to_f(gv[u].v[k]);
            if (scaled) g = __fmul_rn(g, r.gscale);
            m[k] = __fadd_rn(__fmul_rn(m[k], c.beta1), __fmul_rn(g, c.rest1));
            v[k] = __fadd_rn(__fmul_rn(v[k], c.beta2), __fmul_rn(__fmul_rn(g, g), c.rest2));
            root[k] = __fsqrt_rn(v[k]);
            const float den = __fadd_rn(__fmul_rn(root[k], r.root), c.eps);
            p[k] = __fsub_rn(__fmul_rn(to_f(pv[u].v[k]), r.decay), __fmul_rn(__fdiv_rn(m[k], den), r.rate));
            pv[u].v[k] = from_f<TP>(p[k]);
        }
        if constexpr (kPacked) {
            // values behind the tensor's end read as zero and stay zero: they do not count in the group's scale
            uint8_t bm, br;
            const Vec<uint8_t> cm = encode<false>(m, bm), cr = encode<true>(root, br);
            if (i >= n) continue;
            store(d.m, i, n, vec, cm);
            store(d.v, i, n, vec, cr);
            if ((threadIdx.x & 7) == 0) d.ms[i >> 5] = bm, d.vs[i >> 5] = br;
        } else {
            if (i >= n) continue;
            Vec<float> om, ov;
#pragma unroll
            for (int k = 0; k < kVec; ++k) om.v[k] = m[k], ov.v[k] = v[k];
            store(d.m, i, n, vec, om);
            store(d.v, i, n, vec, ov);
        }
        store(d.p, i, n, vec, pv[u]);
        if (sizeof(TP) == 4 && d.copy) {
            if (d.copy_type == HC_BF16) {
                Vec<__nv_bfloat16> o;
#pragma unroll
                for (int k = 0; k < kVec; ++k) o.v[k] = __float2bfloat16_rn(p[k]);
                store(d.copy, i, n, vec, o);
            } else {
                Vec<__half> o;
#pragma unroll
                for (int k = 0; k < kVec; ++k) o.v[k] = __float2half_rn(p[k]);
                store(d.copy, i, n, vec, o);
            }
        }
    }
}

template <bool kPacked>
__device__ __forceinline__ void by_type(const Desc &d, int64_t base, const Scalars &c, const Rates &r, bool scaled) {
    if (d.p_type == HC_F32) chunk<float, float, kPacked>(d, base, c, r, scaled);
    else if (d.p_type == HC_BF16) {
        if (d.g_type == HC_F32) chunk<__nv_bfloat16, float, kPacked>(d, base, c, r, scaled);
        else chunk<__nv_bfloat16, __nv_bfloat16, kPacked>(d, base, c, r, scaled);
    } else {
        if (d.g_type == HC_F32) chunk<__half, float, kPacked>(d, base, c, r, scaled);
        else chunk<__half, __half, kPacked>(d, base, c, r, scaled);
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
k_adamw(const __grid_constant__ Descs<CAP> t, int count, const __grid_constant__ Scalars c) {
    // the last tensor whose first block is not behind this one
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.d[mid].first_block <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const Desc &d = t.d[lo];
    Rates r{c.decay, c.rate, c.root, 1.0f};
    if (c.lr_dev || c.step_dev) {
        const float lr = c.lr_dev ? __ldg(c.lr_dev) : c.lr;
        const int64_t st = c.step_dev ? __ldg(c.step_dev) : c.step;
        const double steps = (double)(st < 1 ? 1 : st);
        // 1 - beta^t = -expm1(t log beta), the product in 64 bits
        r.decay = 1.0f - lr * c.wd;
        r.rate = lr / -expm1f((float)(steps * c.log_beta1));
        r.root = 1.0f / sqrtf(-expm1f((float)(steps * c.log_beta2)));
    }
    const bool scaled = c.grad_scale != nullptr;
    if (scaled) r.gscale = __ldg(c.grad_scale);
    const int64_t base = (int64_t)(blockIdx.x - d.first_block) * kChunk;
    if (d.ms) by_type<true>(d, base, c, r, scaled);
    else by_type<false>(d, base, c, r, scaled);
}

bool vec_ok(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(bytes * kVec) == 0; }

Desc describe(const hc_adamw_tensor &t) {
    Desc d{};
    d.p = t.p, d.g = t.g, d.m = t.m, d.v = t.v, d.ms = t.m_scales, d.vs = t.v_scales, d.copy = t.p_copy;
    d.numel = t.numel;
    d.p_type = (uint8_t)t.p_type, d.g_type = (uint8_t)t.g_type, d.copy_type = (uint8_t)t.copy_type;
    const int64_t state = t.m_scales ? 1 : 4;
    d.vec = vec_ok(t.p, t.p_type == HC_F32 ? 4 : 2) && vec_ok(t.g, t.g_type == HC_F32 ? 4 : 2) && vec_ok(t.m, state) &&
            vec_ok(t.v, state) && (!t.p_copy || vec_ok(t.p_copy, 2));
    return d;
}

template <int CAP>
cudaError_t launch(const hc_adamw_tensor *t, int64_t count, const Scalars &c, cudaStream_t s) {
    static_assert(sizeof(Descs<CAP>) + sizeof(Scalars) + 16 <= 32764, "kernel parameters");
    Descs<CAP> ds;
    int64_t at = 0;
    while (at < count) {
        int k = 0;
        int64_t blocks = 0;
        for (; at < count && k < CAP; ++at) {
            if (t[at].numel == 0) continue;
            const int64_t b = (t[at].numel + kChunk - 1) / kChunk;
            if (blocks + b > INT32_MAX) break;
            ds.d[k] = describe(t[at]);
            ds.d[k++].first_block = (uint32_t)blocks;
            blocks += b;
        }
        if (k == 0) break;
        k_adamw<CAP><<<(unsigned)blocks, kThreads, 0, s>>>(ds, k, c);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace aw

cudaError_t launch_adamw(const hc_adamw_tensor *tensors, int64_t count, double lr, double beta1, double beta2,
                         double eps, double weight_decay, int64_t step, const float *lr_dev, const int64_t *step_dev,
                         const float *grad_scale, cudaStream_t s) {
    aw::Scalars c{};
    c.beta1 = (float)beta1, c.rest1 = (float)(1.0 - beta1), c.beta2 = (float)beta2, c.rest2 = (float)(1.0 - beta2);
    c.eps = (float)eps;
    c.decay = (float)(1.0 - lr * weight_decay);
    c.rate = (float)(lr / (1.0 - pow(beta1, (double)step)));
    c.root = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    c.log_beta1 = log(beta1), c.log_beta2 = log(beta2);
    c.lr = (float)lr, c.wd = (float)weight_decay, c.step = step;
    c.lr_dev = lr_dev, c.step_dev = step_dev, c.grad_scale = grad_scale;
    // (fewer parameter bytes for fewer tensors: they are copied with every launch)
    if (count <= 8) return aw::launch<8>(tensors, count, c, s);
    if (count <= 64) return aw::launch<64>(tensors, count, c, s);
    return aw::launch<448>(tensors, count, c, s);
}

}  // namespace hc
