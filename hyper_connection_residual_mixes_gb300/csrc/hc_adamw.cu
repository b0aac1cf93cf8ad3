// hc_adamw.cu -- one AdamW step over many tensors, for GB300.
//
// Per value, with t the step number:
//   g <- g * grad_scale                                  (when given)
//   m <- m beta1 + g (1 - beta1),   v <- v beta2 + g g (1 - beta2),
//   p <- p (1 - lr wd) - m / (sqrt(v) / sqrt(1 - beta2^t) + eps) * lr / (1 - beta1^t).
// With fp32 states every operation is an fp32 operation rounded once, in the
// order written (no fused multiply-adds); with 8-bit states products and sums
// are fused, and the root and the reciprocal of the denominator are the
// hardware's approximations (each within 2^-23 of its value, far below what the
// codes resolve): the exact ones made the step bound by its instructions.  The root
// is taken of subnormal v too (416 us for 252M values, 410 with those as zeros, which
// with a small eps threw weights away); of the denominator, positive as soon as v
// is, only an eps below 2^-126 can be subnormal, and counts as zero.
// Either way a value's result does not depend on how the tensors are laid out or
// split over launches.  p is rounded once more to its own type.
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
// and gradients with 8-bit states.  All tensors of a call with one kind of states
// go in one launch (their descriptions are kernel parameters, 448 at the most).
// 320 fp32 tensors of 39.7M values: 163 us, 0.99 of the measured copy rate; 252M
// bf16 values with 8-bit states: 416 us, 0.90 (some 43 instructions a value, which
// keep the issue slots 66 % busy).
#include <cuda_fp8.h>

#include "hc_sublayer.h"
#include "hc_types.cuh"

namespace hc {

namespace aw {

constexpr int kThreads = 256;
constexpr int kEach = 16;                 // values per thread and block
constexpr int kChunk = kThreads * kEach;  // values per block

struct Desc {
    void *p;
    const void *g;
    void *m, *v;
    uint8_t *ms, *vs;  // null: fp32 states
    void *copy;
    int64_t numel;
    uint32_t first_block;
    uint8_t p_type : 2, g_type : 2, copy_type : 2;
    uint8_t vec, head;  // vec: from value `head` on every pointer takes accesses of a thread's whole run
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

// Values a thread holds side by side: 16 bytes of the widest of p and g.
template <typename TP, typename TG>
constexpr int run_of() { return sizeof(TP) == 2 && sizeof(TG) == 2 ? 8 : 4; }

// values [i, i + V) of p, those below n (the others read as zero); kFull: all
// are there and aligned, so that the loads of a chunk go out together
template <bool kFull, typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const void *p, int64_t i, int64_t n) {
    const T *q = static_cast<const T *>(p) + i;
    Vec<T, V> r;
    if constexpr (kFull) {
        r = *reinterpret_cast<const Vec<T, V> *>(q);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) r.v[k] = i + k < n ? q[k] : T(0.0f);
    }
    return r;
}
template <bool kFull, typename T, int V>
__device__ __forceinline__ void store(void *p, int64_t i, int64_t n, const Vec<T, V> &r) {
    T *q = static_cast<T *>(p) + i;
    if constexpr (kFull) {
        *reinterpret_cast<Vec<T, V> *>(q) = r;
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (i + k < n) q[k] = r.v[k];
    }
}

// ---- the 8-bit states
__device__ __forceinline__ float scale_of(uint32_t byte) {  // 2^(byte - 127)
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
template <int V>
__device__ __forceinline__ f32x2 pair_of_codes(const Vec<uint8_t, V> &c, int k) {
    Words<uint8_t, V> u;
    u.v = c;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u.w[k / 4] >> (k % 4 * 8)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return f2_make(f.x, f.y);
}
// The larger of two numbers, a NaN if one is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}
// Codes of a thread's values; the 32 / V threads of a group agree on its scale,
// the smallest power of two at or above a / 448.  448 is 1.75 * 2^8, so with
// a = 1.f * 2^E that power is 2^(E - 8), or 2^(E - 7) where 1.f > 1.75: adding
// 0x1fffff to the bits carries into the exponent exactly then.  A NaN becomes
// E4M3's NaN and does not count in the scale.
template <bool kRoot, int V>
__device__ __forceinline__ Vec<uint8_t, V> encode(const f32x2 (&x)[V / 2], uint8_t &byte) {
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
        float x0, x1;
        f2_split(x[k], x0, x1);
        a = kRoot ? fmaxf(a, fmaxf(x0, x1)) : fmaxf(a, fmaxf(fabsf(x0), fabsf(x1)));
    }
#pragma unroll
    for (int o = 1; o < 32 / V; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    int e = (int)((__float_as_uint(a) + 0x1fffffu) >> 23) - 8;
    e = e < 1 ? 1 : e > 247 ? 247 : e;  // (247: an infinite a)
    byte = (uint8_t)e;
    const f32x2 inv = f2_dup(__uint_as_float((uint32_t)(254 - e) << 23));
    Words<uint8_t, V> u;
#pragma unroll
    for (int k = 0; k < V; k += 4) {
        uint32_t two[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float q0, q1;
            f2_split(f2_mul(x[k / 2 + h], inv), q0, q1);
            if (kRoot) {
                // the smallest code stands for 2^-9; x 2^110, cut off at 1, is 1 for every
                // positive root (they are at least 2^-75) and 0 for zero and NaN (whose code is q's, a NaN)
                float x0, x1;
                f2_split(x[k / 2 + h], x0, x1);
                q0 = max_or_nan(q0, __saturatef(x0 * 0x1p110f) * 0x1p-9f);
                q1 = max_or_nan(q1, __saturatef(x1 * 0x1p110f) * 0x1p-9f);
            }
            two[h] = __nv_cvt_float2_to_fp8x2(make_float2(q0, q1), __NV_SATFINITE, __NV_E4M3);
        }
        u.w[k / 4] = two[0] | two[1] << 16;
    }
    return u.v;
}
// Approximations of root and reciprocal, within 2^-23 of the value; the reciprocal
// takes numbers below 2^-126 as zero.
__device__ __forceinline__ f32x2 sqrt_approx(f32x2 x) {
    float a, b;
    f2_split(x, a, b);
    asm("sqrt.approx.f32 %0, %0;" : "+f"(a));
    asm("sqrt.approx.f32 %0, %0;" : "+f"(b));
    return f2_make(a, b);
}
__device__ __forceinline__ f32x2 rcp_approx(f32x2 x) {
    float a, b;
    f2_split(x, a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2_make(a, b);
}

struct Rates {
    float decay, rate, root, gscale;
};

template <typename TP, typename TG, bool kPacked, bool kFull>
__device__ __forceinline__ void chunk(const Desc &d, int64_t base, int64_t n, const Scalars &c, const Rates &r, bool scaled) {
    constexpr int V = run_of<TP, TG>(), U = kEach / V;
    Vec<TP, V> pv[U];
    Vec<TG, V> gv[U];
    Vec<float, V> mv[kPacked ? 1 : U], vv[kPacked ? 1 : U];
    Vec<uint8_t, V> mc[kPacked ? U : 1], vc[kPacked ? U : 1];
    uint8_t mb[kPacked ? U : 1], vb[kPacked ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + (u * kThreads + (int)threadIdx.x) * V;
        pv[u] = load<kFull, TP, V>(d.p, i, n);
        gv[u] = load<kFull, TG, V>(d.g, i, n);
        if constexpr (kPacked) {
            mc[u] = load<kFull, uint8_t, V>(d.m, i, n);
            vc[u] = load<kFull, uint8_t, V>(d.v, i, n);
            mb[u] = kFull || i < n ? d.ms[i >> 5] : 0;
            vb[u] = kFull || i < n ? d.vs[i >> 5] : 0;
        } else {
            mv[u] = load<kFull, float, V>(d.m, i, n);
            vv[u] = load<kFull, float, V>(d.v, i, n);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + (u * kThreads + (int)threadIdx.x) * V;
        float p[V];
        if constexpr (kPacked) {
            f32x2 m[V / 2], root[V / 2];
            const f32x2 ms = f2_dup(scale_of(mb[u])), rs = f2_dup(scale_of(vb[u]));
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const f32x2 g = f2_mul(pair(gv[u], 2 * k), f2_dup(r.gscale));
                const f32x2 r0 = f2_mul(pair_of_codes(vc[u], 2 * k), rs);
                m[k] = f2_fma(f2_mul(pair_of_codes(mc[u], 2 * k), ms), f2_dup(c.beta1), f2_mul(g, f2_dup(c.rest1)));
                root[k] = sqrt_approx(f2_fma(f2_mul(g, f2_dup(c.rest2)), g, f2_mul(f2_mul(r0, r0), f2_dup(c.beta2))));
                const f32x2 step = f2_mul(m[k], rcp_approx(f2_fma(root[k], f2_dup(r.root), f2_dup(c.eps))));
                const f32x2 q = f2_fma(step, f2_dup(-r.rate), f2_mul(pair(pv[u], 2 * k), f2_dup(r.decay)));
                put_pair(pv[u], 2 * k, q);
                f2_split(q, p[2 * k], p[2 * k + 1]);
            }
            // values behind the tensor's end read as zero and stay zero: they do not count in the group's scale
            uint8_t bm, br;
            const Vec<uint8_t, V> cm = encode<false, V>(m, bm), cr = encode<true, V>(root, br);
            if (kFull || i < n) {
                store<kFull>(d.m, i, n, cm);
                store<kFull>(d.v, i, n, cr);
                if (threadIdx.x % (32 / V) == 0) d.ms[i >> 5] = bm, d.vs[i >> 5] = br;
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float g = to_f(gv[u].v[k]);
                if (scaled) g = __fmul_rn(g, r.gscale);
                const float m = __fadd_rn(__fmul_rn(mv[u].v[k], c.beta1), __fmul_rn(g, c.rest1));
                const float v = __fadd_rn(__fmul_rn(vv[u].v[k], c.beta2), __fmul_rn(__fmul_rn(g, g), c.rest2));
                const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v), r.root), c.eps);
                p[k] = __fsub_rn(__fmul_rn(to_f(pv[u].v[k]), r.decay), __fmul_rn(__fdiv_rn(m, den), r.rate));
                mv[u].v[k] = m, vv[u].v[k] = v;
                pv[u].v[k] = from_f<TP>(p[k]);
            }
            store<kFull>(d.m, i, n, mv[u]);
            store<kFull>(d.v, i, n, vv[u]);
        }
        store<kFull>(d.p, i, n, pv[u]);
        if (sizeof(TP) == 4 && d.copy) {
            if (d.copy_type == HC_BF16) {
                Vec<__nv_bfloat16, V> o;
#pragma unroll
                for (int k = 0; k < V; ++k) o.v[k] = __float2bfloat16_rn(p[k]);
                store<kFull>(d.copy, i, n, o);
            } else {
                Vec<__half, V> o;
#pragma unroll
                for (int k = 0; k < V; ++k) o.v[k] = __float2half_rn(p[k]);
                store<kFull>(d.copy, i, n, o);
            }
        }
    }
}

template <typename TP, typename TG, bool kPacked>
__device__ __forceinline__ void whole_or_end(const Desc &d, int64_t base, const Scalars &c, const Rates &r, bool scaled) {
    if (!kPacked && d.head && base == d.head) chunk<TP, TG, kPacked, false>(d, 0, d.head, c, r, scaled);
    if (d.vec && base + kChunk <= d.numel) chunk<TP, TG, kPacked, true>(d, base, d.numel, c, r, scaled);
    else chunk<TP, TG, kPacked, false>(d, base, d.numel, c, r, scaled);
}

// One kernel per kind of states: the 8-bit step needs half the registers, and
// with four blocks on an SM instead of two its loads hide behind one another (at 64
// registers it spills 224 bytes a thread).
template <int CAP, bool kPacked>
__global__ void __launch_bounds__(kThreads, kPacked ? 4 : 2)
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
    const int64_t base = (kPacked ? 0 : d.head) + (int64_t)(blockIdx.x - d.first_block) * kChunk;
    if (d.p_type == HC_F32) whole_or_end<float, float, kPacked>(d, base, c, r, scaled);
    else if (d.p_type == HC_BF16) {
        if (d.g_type == HC_F32) whole_or_end<__nv_bfloat16, float, kPacked>(d, base, c, r, scaled);
        else whole_or_end<__nv_bfloat16, __nv_bfloat16, kPacked>(d, base, c, r, scaled);
    } else {
        if (d.g_type == HC_F32) whole_or_end<__half, float, kPacked>(d, base, c, r, scaled);
        else whole_or_end<__half, __half, kPacked>(d, base, c, r, scaled);
    }
}

// Values of `bytes` each to pass before a run is aligned.
int values_to_run(const void *p, int64_t bytes, int run) {
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(p) % (uintptr_t)(bytes * run));
    return (int)((run - off / bytes) % run);
}

Desc describe(const hc_adamw_tensor &t) {
    Desc d{};
    d.p = t.p, d.g = t.g, d.m = t.m, d.v = t.v, d.ms = t.m_scales, d.vs = t.v_scales, d.copy = t.p_copy;
    d.numel = t.numel;
    d.p_type = (uint8_t)t.p_type & 3, d.g_type = (uint8_t)t.g_type & 3, d.copy_type = (uint8_t)t.copy_type & 3;
    const int64_t pb = t.p_type == HC_F32 ? 4 : 2, gb = t.g_type == HC_F32 ? 4 : 2, state = t.m_scales ? 1 : 4;
    const int run = pb == 2 && gb == 2 ? 8 : 4;  // run_of
    // Tensors cut out of flat buffers at the same odd place are aligned again after the
    // same few values, which the first block takes one by one (with 8-bit states the
    // groups begin with the tensor, so only a tensor that is aligned itself will do).
    const int head = values_to_run(t.p, pb, run);
    d.vec = head == values_to_run(t.g, gb, run) && head == values_to_run(t.m, state, run) &&
            head == values_to_run(t.v, state, run) && (!t.p_copy || head == values_to_run(t.p_copy, 2, run)) &&
            (head == 0 || !t.m_scales) && head <= t.numel;
    d.head = d.vec ? (uint8_t)head : 0;
    return d;
}

template <int CAP, bool kPacked>
cudaError_t launch(const hc_adamw_tensor *t, int64_t count, const Scalars &c, cudaStream_t s) {
    static_assert(sizeof(Descs<CAP>) + sizeof(Scalars) + 16 <= 32764, "kernel parameters");
    Descs<CAP> ds;
    int64_t at = 0;
    while (at < count) {
        int k = 0;
        int64_t blocks = 0;
        for (; at < count && k < CAP; ++at) {
            if (t[at].numel == 0 || (t[at].m_scales != nullptr) != kPacked) continue;
            const Desc d = describe(t[at]);
            const int64_t rest = d.numel - d.head, b = rest > kChunk ? (rest + kChunk - 1) / kChunk : 1;
            if (blocks + b > INT32_MAX) break;
            ds.d[k] = d;
            ds.d[k++].first_block = (uint32_t)blocks;
            blocks += b;
        }
        if (k == 0) break;
        k_adamw<CAP, kPacked><<<(unsigned)blocks, kThreads, 0, s>>>(ds, k, c);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <bool kPacked>
cudaError_t launch_kind(const hc_adamw_tensor *t, int64_t count, const Scalars &c, cudaStream_t s) {
    // (fewer parameter bytes for fewer tensors: they are copied with every launch)
    if (count <= 8) return launch<8, kPacked>(t, count, c, s);
    if (count <= 64) return launch<64, kPacked>(t, count, c, s);
    return launch<448, kPacked>(t, count, c, s);
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
    int64_t packed = 0;
    for (int64_t i = 0; i < count; ++i) packed += tensors[i].m_scales != nullptr;
    if (packed < count) {
        const cudaError_t e = aw::launch_kind<false>(tensors, count, c, s);
        if (e != cudaSuccess) return e;
    }
    return packed ? aw::launch_kind<true>(tensors, count, c, s) : cudaSuccess;
}

}  // namespace hc
