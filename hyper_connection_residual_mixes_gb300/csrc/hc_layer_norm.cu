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
// Both directions move each row across HBM once and are bound by that: 65,536 rows
// of 5,120 bf16 take 208 us forward (0.95 of the measured copy rate), 8,192 rows
// with fp32 gradients 70 us backward (0.89; 4 of them for the column sums), replayed as
// a graph.  Rows that
// start anywhere take the same way, with accesses of one or two values: 65,536 rows of
// 5,119 bf16 395 us, bound by the loads' and stores' issue.
#include <atomic>

#include <cuda.h>

#include "hc_ptx.cuh"
#include "hc_sublayer.h"
#include "hc_types.cuh"

namespace hc {

namespace ln {
constexpr int kSlots = 6;  // most ring slots (the backward at 5120 columns, bf16 with fp32 gradients: 4 80, 6 69.5, 7, all that fit, 70.4 us)

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
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = param(p, type, i + k);
    }
}

// Read-only streaming load of a vector (each x, g value is read once per launch),
// volatile so that a load for the next row stays in front of this row's work.
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_stream(const T *p) {
    constexpr int kBytes = sizeof(T) * VEC;
    union {
        Vec<T, VEC> v;
        uint4 u4;
        uint2 u2;
        uint32_t u1;
        uint16_t h;
    } r;
    if constexpr (kBytes == 16)
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.u4.x), "=r"(r.u4.y), "=r"(r.u4.z), "=r"(r.u4.w)
                     : "l"(p));
    else if constexpr (kBytes == 8)
        asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(r.u2.x), "=r"(r.u2.y) : "l"(p));
    else if constexpr (kBytes == 4)
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r.u1) : "l"(p));
    else
        asm volatile("ld.global.nc.b16 %0, [%1];" : "=h"(r.h) : "l"(p));
    static_assert(kBytes == 16 || kBytes == 8 || kBytes == 4 || kBytes == 2, "loads of 2 to 16 bytes");
    return r.v;
}

__device__ __forceinline__ float f2_lo(f32x2 v) {
    float a, b;
    f2_split(v, a, b);
    return a;
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

// 1 / sqrt(a): the approximation and a Newton step, which leaves about a unit.
__device__ __forceinline__ float rsqrt_newton(float a) {
    const float r = rsqrtf(a);
    return r > 0.0f && r < INFINITY ? fmaf(r * 0.5f, fmaf(-a * r, r, 1.0f), r) : r;  // (0 and infinity stay)
}

// ------------------------------------------------------------ forward
// A row whose values a team of tpr threads holds in registers, thread t the
// vectors t + i * tpr: statistics and output.
template <typename T, int VEC, int NV>
struct Row {
    Vec<T, VEC> v[NV];
    __device__ __forceinline__ void load(const T *x, int t, int tpr, int d) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c < d) v[i] = load_stream<T, VEC>(x + c);
        }
    }
    __device__ __forceinline__ void statistics(int t, int tpr, int d, float eps, float (*red)[32], float &mean,
                                               float &rstd) const {
        const float inv_d = 1.0f / (float)d;
        f32x2 sum = f2_dup(0.0f), sq = f2_dup(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((t + i * tpr) * VEC >= d) continue;
#pragma unroll
            for (int k = 0; k < VEC; k += 2) sum = f2_add(sum, at(i, k));
        }
        mean = team_sum(f2_hsum(sum), tpr, red[0]) * inv_d;
        const f32x2 neg = f2_dup(-mean);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((t + i * tpr) * VEC >= d) continue;
#pragma unroll
            for (int k = 0; k < VEC; k += 2) {
                f32x2 c = f2_add(at(i, k), neg);
                if (VEC == 1) c = f2_make(f2_lo(c), 0.0f);
                sq = f2_fma(c, c, sq);
            }
        }
        rstd = rsqrt_newton(fmaf(team_sum(f2_hsum(sq), tpr, red[1]), inv_d, eps));
    }
    // values k, k + 1 of vector i (of single values: the value and 0)
    __device__ __forceinline__ f32x2 at(int i, int k) const {
        if constexpr (VEC == 1) return f2_make(to_f(v[i].v[0]), 0.0f);
        else return pair(v[i], k);
    }
    __device__ __forceinline__ Vec<T, VEC> normed(int i, float mean, float rstd, const float (&w)[VEC],
                                                  const float (&b)[VEC]) const {
        Vec<T, VEC> o;
        if constexpr (VEC == 1) {
            o.v[0] = from_f<T>(fmaf((to_f(v[i].v[0]) - mean) * rstd, w[0], b[0]));
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k += 2)
                put_pair(o, k, f2_fma(f2_mul(f2_add(pair(v[i], k), f2_dup(-mean)), f2_dup(rstd)), f2_make(w[k], w[k + 1]),
                                      f2_make(b[k], b[k + 1])));
        }
        return o;
    }
};

// One block per row.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024, 1)
k_layer_norm(const T *__restrict__ x, int64_t xs, const void *__restrict__ w, const void *__restrict__ b, int wt,
             int64_t n, int d, float eps, T *__restrict__ y, int64_t ys, float *__restrict__ mean_out,
             float *__restrict__ rstd_out) {
    __shared__ float red[2][32];
    const int t = threadIdx.x, tpr = blockDim.x;
    const int64_t row = blockIdx.x;
    Row<T, VEC, NV> r;
    r.load(x + row * xs, t, tpr, d);
    // (a thread's only vector: its weights come while the row does)
    float w0[VEC] = {}, b0[VEC] = {};
    if (NV == 1 && t * VEC < d) {
        params<VEC>(w, wt, t * VEC, w0);
        if (b) params<VEC>(b, wt, t * VEC, b0);
    }
    float mean, rstd;
    r.statistics(t, tpr, d, eps, red, mean, rstd);
    T *yr = y + row * ys;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * VEC;
        if (c >= d) continue;
        if (NV > 1) {
            params<VEC>(w, wt, c, w0);
            if (b) params<VEC>(b, wt, c, b0);
        }
        *reinterpret_cast<Vec<T, VEC> *>(yr + c) = r.normed(i, mean, rstd, w0, b0);
    }
    if (t == 0) {
        if (mean_out) mean_out[row] = mean;
        if (rstd_out) rstd_out[row] = rstd;
    }
}

// Short rows: a warp per row, which keeps its columns' weights and walks over rows,
// the next one on its way while this one is worked on.
constexpr int kWarpRowThreads = 128;
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kWarpRowThreads)
k_layer_norm_warps(const T *__restrict__ x, int64_t xs, const void *__restrict__ w, const void *__restrict__ b, int wt,
                   int64_t n, int d, float eps, T *__restrict__ y, int64_t ys, float *__restrict__ mean_out,
                   float *__restrict__ rstd_out) {
    const int t = threadIdx.x & 31;
    const int64_t first = (int64_t)blockIdx.x * (kWarpRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t step = (int64_t)gridDim.x * (kWarpRowThreads / 32);
    Row<T, VEC, NV> next;
    if (first < n) next.load(x + first * xs, t, 32, d);
    float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + 32 * i) * VEC;
#pragma unroll
        for (int k = 0; k < VEC; ++k) wv[i][k] = bv[i][k] = 0.0f;
        if (c >= d) continue;
        params<VEC>(w, wt, c, wv[i]);
        if (b) params<VEC>(b, wt, c, bv[i]);
    }
    for (int64_t row = first; row < n; row += step) {
        const Row<T, VEC, NV> r = next;
        if (row + step < n) next.load(x + (row + step) * xs, t, 32, d);
        float mean, rstd;
        r.statistics(t, 32, d, eps, nullptr, mean, rstd);
        T *yr = y + row * ys;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + 32 * i) * VEC;
            if (c < d) *reinterpret_cast<Vec<T, VEC> *>(yr + c) = r.normed(i, mean, rstd, wv[i], bv[i]);
        }
        if (t == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
    }
}

// ------------------------------------------------------------ rows through a ring
// Long rows, many of them: a block keeps its columns' weights in registers and
// walks over rows, which bulk copies bring into a ring of shared-memory slots
// ahead of it (one thread issues them; the block barrier of a row's reduction
// says that a slot has been read).
struct Ring {
    uint64_t full[kSlots];
    volatile int abort;
};
// Where a row of the block stands in the ring.
struct Place {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) slot = 0, parity ^= 1u;
    }
};
// All threads wait for a row; a wait that runs out is reported and the block
// goes on (its rows are then wrong, but every barrier is met).
__device__ __forceinline__ void ring_wait(Ring &r, const Place &p) {
    mbar_wait<false>(smem_u32(&r.full[p.slot]), p.parity, &r.abort);
}
__device__ __forceinline__ void ring_init(Ring &r, int slots) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(smem_u32(&r.full[i]), 1);
        r.abort = 0;
        fence_mbar_init_cluster();
    }
    __syncthreads();
}
// A kernel launched to follow this one may start its blocks now (it waits for
// this grid's end, and so for its writes, before it reads anything).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_grid_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// After a wait that ran out: the copies still in flight must land before the block leaves.
__device__ __forceinline__ void ring_leave(Ring &r, int64_t its, int slots) {
    if (threadIdx.x == 0 && r.abort)
        for (int64_t k = its > slots ? its - slots : 0; k < its; ++k)
            for (uint32_t i = 0; i < (1u << 22); ++i) {
                if (mbar_try_wait(smem_u32(&r.full[k % slots]), (uint32_t)(k / slots) & 1u)) break;
                __nanosleep(128);
            }
}

// Room of a row of d values of `size` bytes in a slot.  Bulk copies move whole
// blocks of 16 bytes; a row that starts anywhere is copied with the blocks it
// begins and ends in.
__host__ __device__ constexpr uint32_t room_of(int d, int size, bool anywhere) {
    return anywhere ? ((uint32_t)(d * size) + 15u & ~15u) + 16u : (uint32_t)(d * size);
}
// The rows of a tensor, from the first value of the first row to the last of the last.
template <typename T, bool kAnywhere>
struct Rows {
    const T *x;
    int64_t stride, n;
    int d;
    // A row's copy: whole blocks [from, from + bytes), `skip` bytes into the slot.
    struct Copy {
        const uint8_t *from;
        uint32_t bytes, skip;
    };
    __device__ __forceinline__ const T *row(int64_t r) const { return x + r * stride; }
    // the row where it lies in its slot
    __device__ __forceinline__ const T *in(const uint8_t *slot, int64_t r) const {
        return reinterpret_cast<const T *>(slot + (kAnywhere ? reinterpret_cast<uintptr_t>(row(r)) & 15u : 0u));
    }
    // Nothing before the first row's start or behind the last one's end is read: the
    // values of the blocks that reach there are fetched one by one, here.
    __device__ __forceinline__ Copy copy(int64_t r, uint8_t *slot) const {
        const uintptr_t first = reinterpret_cast<uintptr_t>(row(r)), end = first + (uint32_t)d * sizeof(T);
        if (!kAnywhere) return Copy{reinterpret_cast<const uint8_t *>(first), (uint32_t)d * (uint32_t)sizeof(T), 0u};
        const uintptr_t base = first & ~(uintptr_t)15;
        uintptr_t lo = base, hi = (end + 15) & ~(uintptr_t)15;
        if (lo < reinterpret_cast<uintptr_t>(x)) {
            lo += 16;
            for (uintptr_t q = first; q < lo; q += sizeof(T))
                *reinterpret_cast<T *>(slot + (q - base)) = *reinterpret_cast<const T *>(q);
        }
        if (hi > reinterpret_cast<uintptr_t>(row(n - 1) + d)) {
            hi -= 16;
            for (uintptr_t q = hi; q < end; q += sizeof(T))
                *reinterpret_cast<T *>(slot + (q - base)) = *reinterpret_cast<const T *>(q);
        }
        return Copy{reinterpret_cast<const uint8_t *>(lo), (uint32_t)(hi - lo), (uint32_t)(lo - base)};
    }
};

// A thread's share of a row: NV runs of V values, run i from column (t + i tpr) V
// on, worked on in pieces of Q pairs: a run, or with V = 1 two runs, of which the
// second may be behind the row.  kFull: the block's threads hold exactly d columns.
// kSelect (V = 1): no branch around a piece that is behind the row, its values read
// as zero and are not stored (20,000 rows of 12,287 bf16 forward 428 us, with the
// branch 671; 6,705 rows of 5,983 fp32 backward 113 us, with the branch 88).
template <int V, int NV, bool kFull, bool kSelect>
struct Share {
    static constexpr int Q = V == 1 ? 1 : V / 2, kPieces = V * NV / 2 / Q;
    int t, tpr, d;
    // the share's first column, a piece's distance from it and a piece's first column
    __device__ __forceinline__ int start() const { return t * V; }
    __device__ __forceinline__ int ahead(int i) const { return V == 1 ? 2 * i * tpr : i * tpr * V; }
    __device__ __forceinline__ int column(int i) const { return start() + ahead(i); }
    __device__ __forceinline__ bool has(int i) const { return kFull || (kSelect && V == 1) || column(i) < d; }
    __device__ __forceinline__ bool first(int i) const { return !kSelect || column(i) < d; }
    __device__ __forceinline__ bool second(int i) const { return column(i) + tpr < d; }
    // a piece that is there; `mine` is the share's start in the row
    template <typename T>
    __device__ __forceinline__ void load(const T *mine, int i, f32x2 *o) const {
        const T *q = mine + ahead(i);
        if constexpr (V == 1) {
            o[0] = f2_make(first(i) ? to_f(q[0]) : 0.0f, second(i) ? to_f(q[tpr]) : 0.0f);
        } else {
            const Vec<T, V> u = *reinterpret_cast<const Vec<T, V> *>(q);
#pragma unroll
            for (int k = 0; k < Q; ++k) o[k] = pair(u, 2 * k);
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *mine, int i, const f32x2 *o) const {
        T *q = mine + ahead(i);
        if constexpr (V == 1) {
            float a, b;
            f2_split(o[0], a, b);
            if (first(i)) q[0] = from_f<T>(a);
            if (second(i)) q[tpr] = from_f<T>(b);
        } else {
            Vec<T, V> u;
#pragma unroll
            for (int k = 0; k < Q; ++k) put_pair(u, 2 * k, o[k]);
            *reinterpret_cast<Vec<T, V> *>(q) = u;
        }
    }
    __device__ __forceinline__ void weights(const void *w, int type, f32x2 *o) const {  // of all pieces
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int c = column(i);
            if constexpr (V == 1) {
                o[i] = f2_make(c < d ? param(w, type, c) : 0.0f, second(i) ? param(w, type, c + tpr) : 0.0f);
            } else {
                float f[V] = {};
                if (has(i)) params<V>(w, type, c, f);
#pragma unroll
                for (int k = 0; k < Q; ++k) o[i * Q + k] = f2_make(f[2 * k], f[2 * k + 1]);
            }
        }
    }
    // v, with zeros for absent values
    __device__ __forceinline__ f32x2 keep(int i, f32x2 v) const {
        if (kFull || V > 1) return v;
        float a, b;
        f2_split(v, a, b);
        return f2_make(first(i) ? a : 0.0f, second(i) ? b : 0.0f);
    }
    // how many columns of the row a warp has
    __device__ __forceinline__ float of_warp(int warp) const {
        if (kFull) return (float)(32 * V * NV);
        int c = 0;
        for (int i = 0; i < NV; ++i) {
            const int left = d - (i * tpr + 32 * warp) * V;
            c += left < 0 ? 0 : left > 32 * V ? 32 * V : left;
        }
        return (float)c;
    }
};

// 16 columns a thread, in runs of V: 16 bytes, or (rows that start anywhere) one or
// two values.  R rows go through a pass together, so that their reductions overlap
// and share the barrier.  Mean and sum of squares are taken per warp first (about
// the warp's own mean), then joined over the warps, so that a pass costs one block
// barrier:
//   mean = sum c_w m_w / d,  M2 = sum M2_w + c_w (m_w - mean)^2.
template <typename T, int V, int R, bool kFull, int kMaxThreads, int kMinBlocks>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks)
k_layer_norm_ring(const T *__restrict__ x, int64_t xs, const void *__restrict__ w, const void *__restrict__ b, int wt,
                  int64_t n, int d, float eps, T *__restrict__ y, int64_t ys, float *__restrict__ mean_out,
                  float *__restrict__ rstd_out, int slots) {
    constexpr bool kAnywhere = V * sizeof(T) < 16;
    constexpr int P = 8;
    extern __shared__ __align__(16) uint8_t s_rows[];
    __shared__ Ring ring;
    __shared__ float2 red[2][R][32];
    const int t = threadIdx.x, tpr = blockDim.x, warp = t >> 5, lane = t & 31, nw = tpr >> 5;
    using Own = Share<V, 16 / V, kFull, true>;
    constexpr int Q = Own::Q, kPieces = Own::kPieces;
    const Own own{t, tpr, d};
    const Rows<T, kAnywhere> in{x, xs, n, d};
    const uint32_t slot_bytes = room_of(d, sizeof(T), kAnywhere);
    ring_init(ring, slots);
    const int64_t rows = (n - 1 - blockIdx.x) / gridDim.x + 1;  // of this block (the grid has at most n)
    const auto fetch = [&](int slot, int64_t it) {
        const uint32_t bar = smem_u32(&ring.full[slot]);
        uint8_t *at = s_rows + (uint32_t)slot * slot_bytes;
        const auto c = in.copy(blockIdx.x + it * gridDim.x, at);
        mbar_arrive_expect_tx(bar, c.bytes);
        bulk_load(smem_u32(at) + c.skip, c.from, c.bytes, bar);
    };
    if (t == 0)
        for (int it = 0; it < slots && it < rows; ++it) fetch(it, it);
    const float inv_d = 1.0f / (float)d;
    const float mine = own.of_warp(warp), inv_mine = mine > 0.0f ? 1.0f / mine : 0.0f;
    const float weight = lane < nw ? own.of_warp(lane) : 0.0f;  // what lane w weighs warp w's mean with
    f32x2 wv[P], bv[P];
    own.weights(w, wt, wv);
#pragma unroll
    for (int p = 0; p < P; ++p) bv[p] = f2_dup(0.0f);
    if (b) own.weights(b, wt, bv);
    Place place;
    T *yr = y + blockIdx.x * ys + own.start();
    int buf = 0;
    for (int64_t it = 0; it < rows; it += R, buf ^= 1) {
        f32x2 v[R][P];
        float m_w[R], m2_w[R];
        const Place first = place;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m_w[r] = m2_w[r] = 0.0f;
            if (it + r >= rows) break;  // the block's last pass
            ring_wait(ring, place);
            const T *xr = in.in(s_rows + (uint32_t)place.slot * slot_bytes, blockIdx.x + (it + r) * gridDim.x) + own.start();
            place.next(slots);
            f32x2 acc = f2_dup(0.0f);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (!own.has(i)) continue;
                own.load(xr, i, v[r] + i * Q);
#pragma unroll
                for (int p = i * Q; p < (i + 1) * Q; ++p) acc = f2_add(acc, v[r][p]);
            }
            m_w[r] = f2_hsum(acc);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) m_w[r] = warp_sum(m_w[r]) * inv_mine;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const f32x2 neg = f2_dup(-m_w[r]);
            f32x2 acc = f2_dup(0.0f);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (!own.has(i)) continue;
#pragma unroll
                for (int p = i * Q; p < (i + 1) * Q; ++p) {
                    v[r][p] = f2_add(v[r][p], neg);
                    const f32x2 c = own.keep(i, v[r][p]);
                    acc = f2_fma(c, c, acc);
                }
            }
            m2_w[r] = f2_hsum(acc);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) m2_w[r] = warp_sum(m2_w[r]);
        // (two buffers: a warp writes the next pass's while a slow one still reads these)
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) red[buf][r][warp] = make_float2(m_w[r], m2_w[r]);
        __syncthreads();
        if (t == 0) {  // every thread has read the slots: they can be filled again
            Place p = first;
#pragma unroll
            for (int r = 0; r < R; ++r, p.next(slots))
                if (it + r + slots < rows) fetch(p.slot, it + r + slots);
        }
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 q = lane < nw ? red[buf][r][lane] : make_float2(0.0f, 0.0f);
            mean[r] = warp_sum(weight * q.x) * inv_d;
            const float off = q.x - mean[r];
            rstd[r] = rsqrt_newton(fmaf(warp_sum(fmaf(weight * off, off, q.y)), inv_d, eps));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (it + r >= rows) break;
            const f32x2 rs = f2_dup(rstd[r]), shift = f2_dup((m_w[r] - mean[r]) * rstd[r]);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (!own.has(i)) continue;
#pragma unroll
                for (int p = i * Q; p < (i + 1) * Q; ++p) v[r][p] = f2_fma(f2_fma(v[r][p], rs, shift), wv[p], bv[p]);
                own.store(yr, i, v[r] + i * Q);
            }
            yr += gridDim.x * ys;
            if (t == 0) {
                const int64_t row = blockIdx.x + (it + r) * gridDim.x;
                if (mean_out) mean_out[row] = mean[r];
                if (rstd_out) rstd_out[row] = rstd[r];
            }
        }
    }
    ring_leave(ring, rows, slots);
}

// ------------------------------------------------------------ backward
// Each thread owns the same columns of every row its block takes, with their
// sums of g xh and g in registers; a block leaves one row of partial sums in
// the workspace, k_ln_columns adds the blocks' rows in a fixed order.
template <typename TX, typename TG, int VEC, int NV>
__global__ void __launch_bounds__(512, 1)
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
    // the next row's values are on their way while this one is worked on
    Vec<TX, VEC> xn[NV];
    Vec<TG, VEC> gn[NV];
    float mean_next = 0.0f, rstd_next = 0.0f;
    const int64_t first = (int64_t)blockIdx.x * teams + team, step = (int64_t)gridDim.x * teams;
    const auto fetch = [&](int64_t row) {
        const TX *xr = x + row * xs;
        const TG *gr = gy + row * gs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c < d) {
                xn[i] = load_stream<TX, VEC>(xr + c);
                gn[i] = load_stream<TG, VEC>(gr + c);
            }
        }
        mean_next = __ldg(mean_in + row), rstd_next = __ldg(rstd_in + row);
    };
    if (first < n) fetch(first);
    int buf = 0;
    for (int64_t row = first; row < n; row += step, buf ^= 1) {
        Vec<TX, VEC> xv[NV];
        Vec<TG, VEC> gv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) xv[i] = xn[i], gv[i] = gn[i];
        const float mean = mean_next, rstd = rstd_next;
        if (row + step < n) fetch(row + step);
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
                // (the product rounded as in the sums: with d = 1 the gradient is 0)
                const float wg = __fmul_rn(to_f(gv[i].v[k]), wv[i][k]);
                o.v[k] = from_f<TG>(rstd * (wg - m1 - xh * m2));
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

// Rows too long for that: the second pass over a row reads it (and the weights)
// again, from L2, so that the registers hold the column sums alone.
template <typename TX, typename TG, int VEC, int NV>
__global__ void __launch_bounds__(1024, 1)
k_ln_backward_wide(const TG *__restrict__ gy, int64_t gs, const TX *__restrict__ x, int64_t xs,
                   const void *__restrict__ w, int wt, const float *__restrict__ mean_in,
                   const float *__restrict__ rstd_in, int64_t n, int d, TG *__restrict__ gx, int64_t gxs,
                   float *__restrict__ part) {
    __shared__ float2 red[2][32];
    const int t = threadIdx.x, tpr = blockDim.x, warp = t >> 5, lane = t & 31, nw = tpr >> 5;
    const float inv_d = 1.0f / (float)d;
    float aw[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) aw[i][k] = ab[i][k] = 0.0f;
    int buf = 0;
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x, buf ^= 1) {
        const TX *xr = x + row * xs;
        const TG *gr = gy + row * gs;
        const float mean = __ldg(mean_in + row), rstd = __ldg(rstd_in + row);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c >= d) continue;
            const Vec<TX, VEC> xv = *reinterpret_cast<const Vec<TX, VEC> *>(xr + c);
            const Vec<TG, VEC> gv = *reinterpret_cast<const Vec<TG, VEC> *>(gr + c);
            float wv[VEC];
            params<VEC>(w, wt, c, wv);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = (to_f(xv.v[k]) - mean) * rstd, g = to_f(gv.v[k]), wg = g * wv[k];
                s1 += wg;
                s2 = fmaf(wg, xh, s2);
                aw[i][k] = fmaf(g, xh, aw[i][k]);
                ab[i][k] += g;
            }
        }
        s1 = warp_sum(s1), s2 = warp_sum(s2);
        if (lane == 0) red[buf][warp] = make_float2(s1, s2);
        __syncthreads();
        const float2 r = lane < nw ? red[buf][lane] : make_float2(0.0f, 0.0f);
        const float m1 = warp_sum(r.x) * inv_d, m2 = warp_sum(r.y) * inv_d;
        TG *o_row = gx + row * gxs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * VEC;
            if (c >= d) continue;
            const Vec<TX, VEC> xv = *reinterpret_cast<const Vec<TX, VEC> *>(xr + c);
            const Vec<TG, VEC> gv = *reinterpret_cast<const Vec<TG, VEC> *>(gr + c);
            float wv[VEC];
            params<VEC>(w, wt, c, wv);
            Vec<TG, VEC> o;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float xh = (to_f(xv.v[k]) - mean) * rstd;
                o.v[k] = from_f<TG>(rstd * (to_f(gv.v[k]) * wv[k] - m1 - xh * m2));
            }
            *reinterpret_cast<Vec<TG, VEC> *>(o_row + c) = o;
        }
    }
    float *pw = part + (int64_t)blockIdx.x * 2 * d, *pb = pw + d;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const int c = (t + i * tpr) * VEC + k;
            if (c < d) pw[c] = aw[i][k], pb[c] = ab[i][k];
        }
}

// The same with the rows of x and g through a ring: 8 columns a thread in runs of V
// (4 where rows take bulk copies as they are, else 1 or 2), R rows a pass.  Both
// passes over a row read it from its slot, which is filled again once the next
// pass's barrier has passed.
template <typename TX, typename TG, int V, int R, bool kFull, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, 1)
k_ln_backward_ring(const TG *__restrict__ gy, int64_t gs, const TX *__restrict__ x, int64_t xs,
                   const void *__restrict__ w, int wt, const float *__restrict__ mean_in,
                   const float *__restrict__ rstd_in, int64_t n, int d, TG *__restrict__ gx, int64_t gxs,
                   float *__restrict__ part, int slots) {
    constexpr bool kAnywhere = V < 4;
    constexpr int P = 4;
    extern __shared__ __align__(16) uint8_t s_rows[];
    __shared__ Ring ring;
    __shared__ float2 red[2][R][32];
    const int t = threadIdx.x, tpr = blockDim.x, warp = t >> 5, lane = t & 31, nw = tpr >> 5;
    using Own = Share<V, 8 / V, kFull, false>;
    constexpr int Q = Own::Q, kPieces = Own::kPieces;
    const Own own{t, tpr, d};
    const Rows<TX, kAnywhere> xin{x, xs, n, d};
    const Rows<TG, kAnywhere> gin{gy, gs, n, d};
    const uint32_t x_room = room_of(d, sizeof(TX), kAnywhere), slot_bytes = x_room + room_of(d, sizeof(TG), kAnywhere);
    const float inv_d = 1.0f / (float)d;
    ring_init(ring, slots);
    const int64_t rows = (n - 1 - blockIdx.x) / gridDim.x + 1;
    const auto fetch = [&](int slot, int64_t it) {
        const uint32_t bar = smem_u32(&ring.full[slot]);
        uint8_t *at = s_rows + (uint32_t)slot * slot_bytes;
        const int64_t row = blockIdx.x + it * gridDim.x;
        const auto a = xin.copy(row, at);
        const auto g = gin.copy(row, at + x_room);
        mbar_arrive_expect_tx(bar, a.bytes + g.bytes);
        bulk_load(smem_u32(at) + a.skip, a.from, a.bytes, bar);
        bulk_load(smem_u32(at) + x_room + g.skip, g.from, g.bytes, bar);
    };
    if (t == 0)
        for (int it = 0; it < slots && it < rows; ++it) fetch(it, it);
    Place place, before;
    f32x2 wv[P], aw[P], ab[P];
    own.weights(w, wt, wv);
#pragma unroll
    for (int p = 0; p < P; ++p) aw[p] = ab[p] = f2_dup(0.0f);
    float mean_next[R], rstd_next[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        mean_next[r] = rstd_next[r] = 0.0f;
        if (r < rows) mean_next[r] = __ldg(mean_in + blockIdx.x + r * gridDim.x), rstd_next[r] = __ldg(rstd_in + blockIdx.x + r * gridDim.x);
    }
    int buf = 0;
    for (int64_t it = 0; it < rows; it += R, buf ^= 1) {
        float mean[R], rstd[R], s1[R], s2[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = mean_next[r], rstd[r] = rstd_next[r];
            const int64_t next = blockIdx.x + (it + R + r) * gridDim.x;
            if (it + R + r < rows) mean_next[r] = __ldg(mean_in + next), rstd_next[r] = __ldg(rstd_in + next);
        }
        const Place first = place;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s1[r] = s2[r] = 0.0f;
            if (it + r >= rows) break;  // the block's last pass
            ring_wait(ring, place);
            const uint8_t *slot = s_rows + (uint32_t)place.slot * slot_bytes;
            const int64_t row = blockIdx.x + (it + r) * gridDim.x;
            place.next(slots);
            const TX *xr = xin.in(slot, row) + own.start();
            const TG *gr = gin.in(slot + x_room, row) + own.start();
            f32x2 a1 = f2_dup(0.0f), a2 = f2_dup(0.0f);
            const f32x2 neg = f2_dup(-mean[r]), rs = f2_dup(rstd[r]);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (!own.has(i)) continue;
                f32x2 xv[Q], gv[Q];
                own.load(xr, i, xv);
                own.load(gr, i, gv);
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const int p = i * Q + k;
                    const f32x2 xh = own.keep(i, f2_mul(f2_add(xv[k], neg), rs)), wg = f2_mul(gv[k], wv[p]);
                    a1 = f2_add(a1, wg);
                    a2 = f2_fma(wg, xh, a2);
                    aw[p] = f2_fma(gv[k], xh, aw[p]);
                    ab[p] = f2_add(ab[p], gv[k]);
                }
            }
            s1[r] = f2_hsum(a1), s2[r] = f2_hsum(a2);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) s1[r] = warp_sum(s1[r]), s2[r] = warp_sum(s2[r]);
        // (two buffers: a warp writes the next pass's sums while a slow one still reads these)
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) red[buf][r][warp] = make_float2(s1[r], s2[r]);
        __syncthreads();
        if (t == 0 && it > 0) {  // every thread is done with the rows before: their slots can be filled again
            Place q = before;
#pragma unroll
            for (int r = 0; r < R; ++r, q.next(slots))
                if (it - R + r + slots < rows) fetch(q.slot, it - R + r + slots);
        }
        before = first;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 q = lane < nw ? red[buf][r][lane] : make_float2(0.0f, 0.0f);
            s1[r] = warp_sum(q.x), s2[r] = warp_sum(q.y);
        }
        Place here = first;
#pragma unroll
        for (int r = 0; r < R; ++r, here.next(slots)) {
            if (it + r >= rows) break;
            const uint8_t *slot = s_rows + (uint32_t)here.slot * slot_bytes;
            const int64_t row = blockIdx.x + (it + r) * gridDim.x;
            const TX *xr = xin.in(slot, row) + own.start();
            const TG *gr = gin.in(slot + x_room, row) + own.start();
            TG *o_row = gx + row * gxs + own.start();
            const f32x2 neg = f2_dup(-mean[r]), rs = f2_dup(rstd[r]);
            const f32x2 m1 = f2_dup(-s1[r] * inv_d), m2 = f2_dup(-s2[r] * inv_d);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (!own.has(i)) continue;
                f32x2 xv[Q], gv[Q];
                own.load(xr, i, xv);
                own.load(gr, i, gv);
#pragma unroll
                for (int k = 0; k < Q; ++k)
                    gv[k] = f2_mul(rs, f2_fma(f2_mul(f2_add(xv[k], neg), rs), m2, f2_fma(gv[k], wv[i * Q + k], m1)));
                own.store(o_row, i, gv);
            }
        }
    }
    ring_leave(ring, rows, slots);
    launch_dependents();
    float *pw = part + (int64_t)blockIdx.x * 2 * d + own.start();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        if (!own.has(i)) continue;
        own.store(pw, i, aw + i * Q);
        own.store(pw + d, i, ab + i * Q);
    }
}

// g_w, g_b [d] from the blocks' partial rows [blocks][2][d]: 32 columns per
// block, the rows shared among 16 warps.
constexpr int kColWarps = 16;
__global__ void __launch_bounds__(32 * kColWarps)
k_ln_columns(const float *__restrict__ part, int blocks, int d, float *__restrict__ g_w, float *__restrict__ g_b) {
    __shared__ float s[kColWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    wait_for_grid_before();
    float a = 0.0f;
    if (c < 2 * d) {
#pragma unroll 10
        for (int r = warp; r < blocks; r += kColWarps) a += __ldcg(part + (int64_t)r * 2 * d + c);
    }
    s[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < 2 * d) {
        for (int k = 1; k < kColWarps; ++k) a += s[k][lane];
        if (c < d) g_w[c] = a;
        else if (g_b) g_b[c - d] = a;
    }
}

constexpr int kDevices = 64;
constexpr int kSmemBlock = 227 * 1024, kSmemSm = 228 * 1024;  // shared memory of a block, of an SM

int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kDevices ? dev : 0;
}
int sm_count_of_device() {
    static std::atomic<int> sms[kDevices];  // (any host thread may be the first to ask)
    const int dev = current_device();
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    sms[dev].store(n, std::memory_order_relaxed);
    return n;
}
// Blocks of a kernel that an SM holds by its threads and registers (handed out to
// warps in units of 256), and the most dynamic shared memory allowed to it; asked
// for and set once per kernel and device.
template <auto kKernel>
cudaError_t blocks_per_sm(int threads, int *per_sm) {
    static std::atomic<int> regs[kDevices];
    const int dev = current_device();
    int r = regs[dev].load(std::memory_order_acquire);
    if (!r) {
        cudaFuncAttributes fa{};
        cudaError_t e = cudaFuncGetAttributes(&fa, kKernel);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSmemBlock - (int)fa.sharedSizeBytes);
        if (e != cudaSuccess) return e;
        r = fa.numRegs;
        regs[dev].store(r, std::memory_order_release);  // (the attribute is set for whoever reads it)
    }
    const int warps = threads / 32, by_regs = 65536 / ((r * 32 + 255) / 256 * 256 * warps), by_threads = 64 / warps;
    *per_sm = by_regs < by_threads ? by_regs : by_threads;
    if (*per_sm < 1) *per_sm = 1;
    return cudaSuccess;
}

bool aligned(const void *p, int64_t stride_bytes, size_t to) {
    return (reinterpret_cast<uintptr_t>(p) % to) == 0 && (uint64_t)stride_bytes % to == 0;
}

struct FwdCall {
    const void *x; int64_t xs; const void *w, *b; int wt; int64_t n; int d; float eps;
    void *y; int64_t ys; float *mean, *rstd; cudaStream_t s;
};

template <typename T, int VEC, int NV>
cudaError_t fwd_warps(const FwdCall &c) {
    constexpr auto kKernel = k_layer_norm_warps<T, VEC, NV>;
    int per_sm = 0;
    const cudaError_t e = blocks_per_sm<kKernel>(kWarpRowThreads, &per_sm);
    if (e != cudaSuccess) return e;
    const int64_t need = (c.n + kWarpRowThreads / 32 - 1) / (kWarpRowThreads / 32);
    const int64_t most = (int64_t)per_sm * sm_count_of_device();
    kKernel<<<(unsigned)(need < most ? need : most), kWarpRowThreads, 0, c.s>>>(
        static_cast<const T *>(c.x), c.xs, c.w, c.b, c.wt, c.n, c.d, c.eps, static_cast<T *>(c.y), c.ys, c.mean, c.rstd);
    return cudaGetLastError();
}
template <typename T, int VEC, int NV>
cudaError_t fwd_blocks(const FwdCall &c, int threads) {
    k_layer_norm<T, VEC, NV><<<(unsigned)c.n, threads, 0, c.s>>>(
        static_cast<const T *>(c.x), c.xs, c.w, c.b, c.wt, c.n, c.d, c.eps, static_cast<T *>(c.y), c.ys, c.mean, c.rstd);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t fwd_vec(const FwdCall &c) {
    const int vecs = (c.d + VEC - 1) / VEC;
    if (vecs <= 32) return fwd_warps<T, VEC, 1>(c);
    if (vecs <= 64) return fwd_warps<T, VEC, 2>(c);
    if (vecs <= 128) return fwd_warps<T, VEC, 4>(c);
    if (vecs <= 1024) return fwd_blocks<T, VEC, 1>(c, (vecs + 31) / 32 * 32);
    if (vecs <= 4096) return fwd_blocks<T, VEC, 4>(c, (vecs + 127) / 128 * 32);
    return fwd_blocks<T, VEC < 4 ? VEC : 1, 16>(c, (vecs + 511) / 512 * 32);  // (runs of 4 and 8 never are so many)
}

// Slots of a ring and blocks of a launch: as many slots as fit beside the SM's
// other blocks, and a grid that fills the SMs once.
template <auto kKernel>
cudaError_t ring_shape(int threads, int slot_bytes, int least, int best, int64_t rows, int64_t most, int *slots, int *blocks) {
    int per_sm = 0;
    const cudaError_t e = blocks_per_sm<kKernel>(threads, &per_sm);
    if (e != cudaSuccess) return e;
    const int extra = 2048;  // a block's other shared memory
    while (per_sm > 1 && (kSmemSm / per_sm - extra) / slot_bytes < least) --per_sm;
    const int room = (per_sm > 1 ? kSmemSm / per_sm : kSmemBlock) - extra;
    *slots = room / slot_bytes < best ? room / slot_bytes : best;
    int64_t grid = (int64_t)per_sm * sm_count_of_device();
    if (grid > most) grid = most;
    if (grid > rows) grid = rows;
    *blocks = (int)grid;
    return cudaSuccess;
}

template <auto kKernel, typename T>
cudaError_t fwd_ring_launch(const FwdCall &c, int threads, int room) {
    int slots = 0, blocks = 0;
    const cudaError_t e = ring_shape<kKernel>(threads, room, 3, 4, c.n, INT32_MAX, &slots, &blocks);
    if (e != cudaSuccess) return e;
    kKernel<<<blocks, threads, slots * room, c.s>>>(static_cast<const T *>(c.x), c.xs, c.w, c.b, c.wt, c.n, c.d, c.eps,
                                                    static_cast<T *>(c.y), c.ys, c.mean, c.rstd, slots);
    return cudaGetLastError();
}
template <typename T, int V>
cudaError_t fwd_ring(const FwdCall &c) {
    const int threads = (c.d + 511) / 512 * 32, room = (int)room_of(c.d, sizeof(T), V * sizeof(T) < 16);
    if (threads <= 320) {
        if constexpr (V * sizeof(T) == 16)
            if (c.d == threads * 16) return fwd_ring_launch<k_layer_norm_ring<T, V, 2, true, 320, 2>, T>(c, threads, room);
        return fwd_ring_launch<k_layer_norm_ring<T, V, 2, false, 320, 2>, T>(c, threads, room);
    }
    if (threads <= 704) return fwd_ring_launch<k_layer_norm_ring<T, V, 2, false, 704, 1>, T>(c, threads, room);
    return fwd_ring_launch<k_layer_norm_ring<T, V, 1, false, 1024, 1>, T>(c, threads, room);
}

template <typename T>
cudaError_t fwd_type(const FwdCall &c) {
    constexpr int VEC = 16 / sizeof(T);
    const size_t pa = c.wt == HC_F32 ? 16 : 8;
    // The ring from 16,384 values an SM on (us, ring and without: 304 rows of 5,120 3.7 and 3.3, 608 rows 4.2
    // and 5.4, 4,864 rows 17.8 and 35.4; 608 rows of 1,024 3.0 and 2.6, 4,864 rows 5.8 and 6.2; 2,048
    // rows of 520 4.7 and 3.7, 65,536 rows 49 and 65, of 264 39 and 30; in any place 65,536 rows of 5,119
    // 390 and 1,046, of 257 53 and 89, 20,000 rows of 12,287 428 and 1,013).
    const bool many = c.n * c.d >= 16384 * (int64_t)sm_count_of_device();
    if (c.d % VEC == 0 && aligned(c.x, c.xs * (int64_t)sizeof(T), 16) && aligned(c.y, c.ys * (int64_t)sizeof(T), 16) &&
        aligned(c.w, 0, pa) && aligned(c.b, 0, pa)) {
        if (c.d > 512 && many) return fwd_ring<T, VEC>(c);
        return fwd_vec<T, VEC>(c);
    }
    // (16-bit rows of even width and spacing: two values at a time)
    if constexpr (sizeof(T) == 2)
        if (c.d % 2 == 0 && aligned(c.x, c.xs * 2, 4) && aligned(c.y, c.ys * 2, 4)) {
            if (c.d > 256 && many) return fwd_ring<T, 2>(c);
            return fwd_vec<T, 2>(c);
        }
    if (c.d > 128 && many) return fwd_ring<T, 1>(c);
    return fwd_vec<T, 1>(c);
}

struct BwdCall {
    const void *gy; int64_t gs; const void *x; int64_t xs; const void *w; int wt; const float *mean, *rstd;
    int64_t n; int d; void *gx; int64_t gxs; float *part, *g_w, *g_b; cudaStream_t s;
};

// blocks of partial sums a launch may use
int64_t max_blocks(int d) { return d < 1024 ? 1216 : d <= 2048 ? 608 : 304; }

// The second launch starts while the first one's last blocks run (its blocks are
// small, and wait for the first grid's end themselves).
cudaError_t launch_columns(const BwdCall &c, int blocks) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((2 * c.d + 31) / 32)), cfg.blockDim = dim3(32 * kColWarps);
    cfg.stream = c.s, cfg.attrs = &early, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_ln_columns, (const float *)c.part, blocks, c.d, c.g_w, c.g_b);
}

template <typename TX, typename TG, int VEC, int NV>
cudaError_t bwd_launch(const BwdCall &c, int tpr) {
    constexpr auto kKernel = k_ln_backward<TX, TG, VEC, NV>;
    const int threads = tpr == 32 ? 256 : tpr;
    const int teams = tpr == 32 ? threads / 32 : 1;
    const size_t smem = teams > 1 ? (size_t)c.d * 8 : 0;
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<kKernel>(threads, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t blocks = (int64_t)per_sm * sm_count_of_device();
    if (blocks > max_blocks(c.d)) blocks = max_blocks(c.d);
    if (blocks > (c.n + teams - 1) / teams) blocks = (c.n + teams - 1) / teams;
    kKernel<<<(unsigned)blocks, threads, smem, c.s>>>(
        static_cast<const TG *>(c.gy), c.gs, static_cast<const TX *>(c.x), c.xs, c.w, c.wt, c.mean, c.rstd, c.n, c.d,
        static_cast<TG *>(c.gx), c.gxs, c.part, tpr);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_columns(c, (int)blocks);
}

template <typename TX, typename TG, int VEC, int NV>
cudaError_t bwd_wide(const BwdCall &c, int threads) {
    constexpr auto kKernel = k_ln_backward_wide<TX, TG, VEC, NV>;
    int per_sm = 0;
    cudaError_t e = blocks_per_sm<kKernel>(threads, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t blocks = (int64_t)per_sm * sm_count_of_device();
    if (blocks > max_blocks(c.d)) blocks = max_blocks(c.d);
    if (blocks > c.n) blocks = c.n;
    kKernel<<<(unsigned)blocks, threads, 0, c.s>>>(
        static_cast<const TG *>(c.gy), c.gs, static_cast<const TX *>(c.x), c.xs, c.w, c.wt, c.mean, c.rstd, c.n, c.d,
        static_cast<TG *>(c.gx), c.gxs, c.part);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_columns(c, (int)blocks);
}

template <auto kKernel, typename TX, typename TG>
cudaError_t bwd_ring_launch(const BwdCall &c, int threads, int room, int least) {
    int slots = 0, blocks = 0;
    cudaError_t e = ring_shape<kKernel>(threads, room, least, kSlots, c.n, max_blocks(c.d), &slots, &blocks);
    if (e != cudaSuccess) return e;
    kKernel<<<blocks, threads, slots * room, c.s>>>(
        static_cast<const TG *>(c.gy), c.gs, static_cast<const TX *>(c.x), c.xs, c.w, c.wt, c.mean, c.rstd, c.n, c.d,
        static_cast<TG *>(c.gx), c.gxs, c.part, slots);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_columns(c, blocks);
}
template <typename TX, typename TG, int V>
cudaError_t bwd_ring(const BwdCall &c) {
    const int threads = (c.d + 255) / 256 * 32;
    const int room = (int)(room_of(c.d, sizeof(TX), V < 4) + room_of(c.d, sizeof(TG), V < 4));
    if (threads > 768) return bwd_ring_launch<k_ln_backward_ring<TX, TG, V, 1, false, 1024>, TX, TG>(c, threads, room, 2);
    if (threads > 640) return bwd_ring_launch<k_ln_backward_ring<TX, TG, V, 1, false, 768>, TX, TG>(c, threads, room, 2);
    if constexpr (V == 4) {
        // (us, two rows a pass and one: 8,192 rows of 5,120 with fp32 gradients 70 and 73, all bf16 16,384 rows
        // 114 and 124, of 4,096 97 and 106, 32,768 rows of 2,560 118 and 122, of 2,048 100 and 96)
        if (c.d >= 2560) {
            if (c.d % 256 == 0) return bwd_ring_launch<k_ln_backward_ring<TX, TG, V, 2, true, 640>, TX, TG>(c, threads, room, 4);
            return bwd_ring_launch<k_ln_backward_ring<TX, TG, V, 2, false, 640>, TX, TG>(c, threads, room, 4);
        }
        if (c.d % 256 == 0) return bwd_ring_launch<k_ln_backward_ring<TX, TG, V, 1, true, 640>, TX, TG>(c, threads, room, 2);
    }
    return bwd_ring_launch<k_ln_backward_ring<TX, TG, V, 1, false, 640>, TX, TG>(c, threads, room, 2);
}

template <typename TX, typename TG>
cudaError_t bwd_type(const BwdCall &c) {
    const size_t pa = c.wt == HC_F32 ? 16 : 8;
    const int d = c.d;
    if (d % 4 == 0 && d > 128 && aligned(c.x, c.xs * (int64_t)sizeof(TX), 4 * sizeof(TX)) &&
        aligned(c.gy, c.gs * (int64_t)sizeof(TG), 4 * sizeof(TG)) &&
        aligned(c.gx, c.gxs * (int64_t)sizeof(TG), 4 * sizeof(TG)) && aligned(c.w, 0, pa)) {
        // (us, ring and plain loads: 76 rows of 5,120 6.6 and 9.4, 4,864 rows 45.6 and 84.3; of 1,024
        // columns 4.5 and 4.9, 13.8 and 15.2; 53,310 rows of 520 fp32 98 and 77; in any place 41,791 rows
        // of 1,435 fp16 165 and 211, 6,705 of 5,983 fp32 88 and 311, 53,310 of 519 fp32 128 and 104, in pairs 65,536 of 770 bf16 138 and 216)
        const bool bulk = (int64_t)d * sizeof(TX) % 16 == 0 && (int64_t)d * sizeof(TG) % 16 == 0 &&
                          aligned(c.x, c.xs * (int64_t)sizeof(TX), 16) && aligned(c.gy, c.gs * (int64_t)sizeof(TG), 16);
        if (bulk && d >= 1024 && d <= 8192) return bwd_ring<TX, TG, 4>(c);
        if (d <= 256) return bwd_launch<TX, TG, 4, 2>(c, 32);
        if (d < 1024) return bwd_launch<TX, TG, 4, 2>(c, (d + 255) / 256 * 32);
        if (d > 8192) return bwd_wide<TX, TG, 4, 4>(c, (d + 511) / 512 * 32);
    }
    // (16-bit rows of even width and spacing: two values at a time)
    if constexpr (sizeof(TX) == 2)
        if (d % 2 == 0 && d > 256 && aligned(c.x, c.xs * 2, 4) && aligned(c.gy, c.gs * (int64_t)sizeof(TG), 2 * sizeof(TG)) &&
            aligned(c.gx, c.gxs * (int64_t)sizeof(TG), 2 * sizeof(TG))) {
            if (d < 512) return bwd_launch<TX, TG, 2, 4>(c, (d + 255) / 256 * 32);
            if (d <= 8192) return bwd_ring<TX, TG, 2>(c);
            return bwd_wide<TX, TG, 2, 8>(c, (d + 511) / 512 * 32);
        }
    if (d <= 128) return bwd_launch<TX, TG, 1, 4>(c, 32);
    if (d < 1024) return bwd_launch<TX, TG, 1, 8>(c, (d + 255) / 256 * 32);
    if (d <= 8192) return bwd_ring<TX, TG, 1>(c);
    return bwd_wide<TX, TG, 1, 16>(c, (d + 511) / 512 * 32);
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

cudaError_t consume_layer_norm_device_error(cudaStream_t s, unsigned int *flag) {
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
