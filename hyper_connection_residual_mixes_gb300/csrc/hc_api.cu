// hc_api.cu -- the C ABI of libhc: host-side validation, then dispatch to the
// kernels.  Nothing here allocates device memory; every launch goes on the
// caller's stream.  See include/hc.h for the contract of each entry point.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/hc.h"
#include "hc_backward_generic.h"
#include "hc_launch.h"
#include "hc_sublayer.h"

namespace {

thread_local int g_last_cuda_error = 0;

constexpr int kMaxD = 16384;

struct Span {
    uintptr_t lo, hi;  // [lo, hi); empty when lo == hi
};

Span span(const void *p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

bool overlaps(Span a, Span b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool finite_nonneg(float v) { return std::isfinite(v) && v >= 0.0f; }

hc_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return HC_OK;
    g_last_cuda_error = (int)e;
    return HC_ERR_CUDA;
}

// Shape checks shared by the entry points.  n == 0 is valid (no work).
hc_status check_shape(int64_t n, int hc, int d, bool uses_d) {
    if (n < 0) return HC_ERR_INVALID_ARG;
    if (hc <= 0) return HC_ERR_INVALID_ARG;
    if (hc != 2 && hc != 4 && hc != 8) return HC_ERR_UNSUPPORTED;  // the compiled stream counts
    if (uses_d) {
        if (d <= 0) return HC_ERR_INVALID_ARG;
        if (d % 64 != 0 || d > kMaxD) return HC_ERR_UNSUPPORTED;
        // n * hc * d elements must be addressable with 64-bit byte offsets
        if (n > (INT64_MAX / 8) / ((int64_t)hc * d)) return HC_ERR_INVALID_ARG;
    } else if (n > INT64_MAX / 1024) {
        return HC_ERR_INVALID_ARG;
    }
    return HC_OK;
}

// Every output span must be disjoint from every input span and from the other outputs.
hc_status check_alias(const Span *outs, int n_out, const Span *ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlaps(outs[i], ins[j])) return HC_ERR_ALIAS;
        for (int j = i + 1; j < n_out; ++j)
            if (overlaps(outs[i], outs[j])) return HC_ERR_ALIAS;
    }
    return HC_OK;
}

// ---- sublayer operators: typed rows with a stride
bool known(hc_dtype t) { return t == HC_F32 || t == HC_BF16 || t == HC_F16; }

int64_t size_of(hc_dtype t) { return t == HC_F32 ? 4 : 2; }

bool aligned_to(const void *p, int64_t bytes) { return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes) == 0; }

// n rows of d elements, `stride` elements apart
Span rows_span(const void *p, int64_t n, int64_t d, int64_t stride, hc_dtype t) {
    return span(p, n > 0 ? ((n - 1) * stride + d) * size_of(t) : 0);
}

// rows whose extent in bytes stays far inside 64 bits
bool rows_fit(int64_t n, int64_t d, int64_t stride) {
    return stride >= 0 && n <= INT64_MAX / 64 / (stride > d ? stride : d > 0 ? d : 1);
}

// A range of memory that a call reads or writes, for checks over many tensors.
struct Use {
    uintptr_t lo, hi;
    bool written;
};

// Whether a written range meets any other range.  u holds `runs` runs of ranges
// (run r ends before at[r]), each most often ascending already, as tensors made one
// after the other are: only those that are not get sorted, then the runs are
// merged pairwise (`spare` has room for all).  In order of their starts each
// range is compared with the furthest end so far, of the written ones or (if it
// is written itself) of all.
bool any_overlap(Use *u, Use *spare, int64_t *at, int runs) {
    const auto before = [](const Use &a, const Use &b) { return a.lo < b.lo; };
    for (int r = 0; r < runs; ++r) {
        Use *first = u + (r ? at[r - 1] : 0), *last = u + at[r];
        if (!std::is_sorted(first, last, before)) std::sort(first, last, before);
    }
    for (; runs > 1; runs = (runs + 1) / 2, std::swap(u, spare)) {
        for (int r = 0; r < runs; r += 2) {
            Use *first = u + (r ? at[r - 1] : 0), *mid = u + at[r], *last = r + 1 < runs ? u + at[r + 1] : mid;
            std::merge(first, mid, mid, last, spare + (first - u), before);
        }
        for (int r = 0; r < (runs + 1) / 2; ++r) at[r] = at[2 * r + 1 < runs ? 2 * r + 1 : 2 * r];
    }
    const int64_t n = at[0];
    uintptr_t written_end = 0, end = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (u[i].lo < (u[i].written ? end : written_end)) return true;
        if (u[i].hi > end) end = u[i].hi;
        if (u[i].written && u[i].hi > written_end) written_end = u[i].hi;
    }
    return false;
}

hc_status check_adamw_tensor(const hc_adamw_tensor &t) {
    const hc_dtype pt = (hc_dtype)t.p_type, gt = (hc_dtype)t.g_type, ct = (hc_dtype)t.copy_type;
    if (t.numel < 0 || t.numel > (int64_t)1 << 42 || !known(pt) || !known(gt)) return HC_ERR_INVALID_ARG;
    if (!t.m_scales != !t.v_scales) return HC_ERR_INVALID_ARG;
    if (gt != HC_F32 && gt != pt) return HC_ERR_UNSUPPORTED;
    if (t.p_copy && (pt != HC_F32 || (ct != HC_BF16 && ct != HC_F16))) return HC_ERR_UNSUPPORTED;
    if (t.numel == 0) return HC_OK;
    if (!t.p || !t.g || !t.m || !t.v) return HC_ERR_INVALID_ARG;
    const int64_t state = t.m_scales ? 1 : 4;
    if (!aligned_to(t.p, size_of(pt)) || !aligned_to(t.g, size_of(gt)) || !aligned_to(t.m, state) ||
        !aligned_to(t.v, state) || !aligned_to(t.p_copy, 2))
        return HC_ERR_MISALIGNED;
    return HC_OK;
}

hc_status check_grouped(int64_t n, int experts, int N, int K, hc_dtype type, hc_dtype out_type) {
    if (n < 0 || experts <= 0 || N <= 0 || K <= 0 || !known(type) || !known(out_type)) return HC_ERR_INVALID_ARG;
    if (type == HC_F32 || (out_type != HC_F32 && out_type != type) || experts > 1024 || N % 8 || K % 8 ||
        n > INT32_MAX - 4096 || N > INT32_MAX - 4096 || K > INT32_MAX - 4096)  // (a tile's last row and column fit 32 bits)
        return HC_ERR_UNSUPPORTED;
    // sizes that no device memory holds (and whose tile counts would not fit 32 bits)
    const int64_t most = (int64_t)1 << 40;
    if (n * N > most || n * K > most || (int64_t)N * K > most / experts) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

hc_status check_norm(int64_t n, int d, hc_dtype x_type, hc_dtype w_type) {
    if (n < 0 || d <= 0 || !known(x_type) || !known(w_type)) return HC_ERR_INVALID_ARG;
    if (d > kMaxD || n > INT32_MAX || (w_type != HC_F32 && w_type != x_type)) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

}  // namespace

extern "C" {

const char *hc_status_string(hc_status status) {
    switch (status) {
        case HC_OK: return "HC_OK";
        case HC_ERR_INVALID_ARG: return "HC_ERR_INVALID_ARG: null pointer, bad size or bad scalar";
        case HC_ERR_UNSUPPORTED: return "HC_ERR_UNSUPPORTED: a size or type that this entry point does not serve";
        case HC_ERR_MISALIGNED: return "HC_ERR_MISALIGNED: a pointer without the alignment that this entry point needs";
        case HC_ERR_ALIAS: return "HC_ERR_ALIAS: an output overlaps an input or another output";
        case HC_ERR_CUDA: return "HC_ERR_CUDA: a CUDA call failed (see hc_last_cuda_error)";
        case HC_ERR_TIMEOUT: return "HC_ERR_TIMEOUT: a kernel gave up waiting on a barrier";
    }
    return "unknown hc_status";
}

int hc_last_cuda_error(void) { return g_last_cuda_error; }

int hc_version(void) { return 200; }

hc_status hc_consume_device_error(cudaStream_t stream) {
    unsigned int flag = 0, flag_chain = 0, flag_bwd = 0, flag_proj = 0, flag_grouped = 0, flag_norm = 0;
    hc_status st = cuda_status(hc::consume_device_error(stream, &flag));
    if (st != HC_OK) return st;
    st = cuda_status(hc::consume_slices_device_error(stream, &flag_chain));
    if (st != HC_OK) return st;
    st = cuda_status(hc::consume_backward_device_error(stream, &flag_bwd));
    if (st != HC_OK) return st;
    st = cuda_status(hc::consume_proj_device_error(stream, &flag_proj));
    if (st != HC_OK) return st;
    st = cuda_status(hc::consume_grouped_mm_device_error(stream, &flag_grouped));
    if (st != HC_OK) return st;
    st = cuda_status(hc::consume_layer_norm_device_error(stream, &flag_norm));
    if (st != HC_OK) return st;
    // (bit 0 of each: a wait ran out; bit 1 of the grouped products': bad offsets)
    if (flag | flag_norm | flag_chain | flag_bwd | flag_proj | (flag_grouped & 1u)) return HC_ERR_TIMEOUT;
    return flag_grouped ? HC_ERR_INVALID_ARG : HC_OK;
}

hc_status hc_selftest_barrier_timeout(cudaStream_t stream) {
    return cuda_status(hc::launch_selftest_wait(stream));
}

hc_status hc_split_sinkhorn(const float *mixes, const float *hc_scale, const float *hc_base,
                            int64_t n, int hc, int sinkhorn_iters, float eps, float *pre,
                            float *post, float *comb, cudaStream_t stream) {
    hc_status st = check_shape(n, hc, 0, false);
    if (st != HC_OK) return st;
    if (sinkhorn_iters < 1 || !finite_nonneg(eps)) return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!mixes || !hc_scale || !hc_base || !pre || !post || !comb) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {mixes, hc_scale, hc_base, pre, post, comb};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    const int64_t mix = (int64_t)(2 + hc) * hc;
    const Span ins[] = {span(mixes, n * mix * 4), span(hc_scale, 12), span(hc_base, mix * 4)};
    const Span outs[] = {span(pre, n * hc * 4), span(post, n * hc * 4), span(comb, n * hc * hc * 4)};
    if ((st = check_alias(outs, 3, ins, 3)) != HC_OK) return st;
    return cuda_status(hc::launch_split_sinkhorn(mixes, hc_scale, hc_base, n, hc, sinkhorn_iters, eps,
                                                 pre, post, comb, stream));
}

hc_status hc_mixes(const uint16_t *x, const float *hc_fn, const float *hc_scale,
                   const float *hc_base, int64_t n, int hc, int d, int sinkhorn_iters,
                   float eps, float norm_eps, float *pre, float *post, float *comb,
                   float *mixes_out, cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (sinkhorn_iters < 1 || !finite_nonneg(eps) || !finite_nonneg(norm_eps))
        return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!x || !hc_fn || !hc_scale || !hc_base || !pre || !post || !comb) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {x, hc_fn, hc_scale, hc_base, pre, post, comb};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    if (mixes_out && !aligned16(mixes_out)) return HC_ERR_MISALIGNED;
    const int64_t mix = (int64_t)(2 + hc) * hc, K = (int64_t)hc * d;
    const Span ins[] = {span(x, n * K * 2), span(hc_fn, mix * K * 4), span(hc_scale, 12),
                        span(hc_base, mix * 4)};
    const Span outs[] = {span(pre, n * hc * 4), span(post, n * hc * 4),
                         span(comb, n * hc * hc * 4), span(mixes_out, mixes_out ? n * mix * 4 : 0)};
    if ((st = check_alias(outs, 4, ins, 4)) != HC_OK) return st;
    if (hc == 4 && hc::cluster_path_supported(d))
        return cuda_status(hc::launch_block_cluster(x, nullptr, nullptr, hc_fn, hc_scale, hc_base,
                                                    nullptr, n, d, sinkhorn_iters, eps, norm_eps,
                                                    nullptr, nullptr, pre, post, comb, mixes_out,
                                                    stream));
    return cuda_status(hc::launch_tokens_simple(x, nullptr, nullptr, hc_fn, hc_scale, hc_base,
                                                nullptr, n, hc, d, sinkhorn_iters, eps, norm_eps,
                                                nullptr, nullptr, pre, post, comb, mixes_out,
                                                stream));
}

hc_status hc_pre_norm(const uint16_t *x, const float *pre_mix, const float *norm_w, int64_t n,
                      int hc, int d, float norm_eps, uint16_t *out, cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (!finite_nonneg(norm_eps)) return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!x || !pre_mix || !norm_w || !out) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {x, pre_mix, norm_w, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    const Span ins[] = {span(x, n * hc * d * 2), span(pre_mix, n * hc * 4), span(norm_w, d * 4)};
    const Span outs[] = {span(out, n * d * 2)};
    if ((st = check_alias(outs, 1, ins, 3)) != HC_OK) return st;
    return cuda_status(hc::launch_pre_norm(x, pre_mix, norm_w, n, hc, d, norm_eps, out, stream));
}

size_t hc_block_step_backward_workspace_bytes(int64_t n, int hc, int d) {
    if (check_shape(n, hc, d, true) != HC_OK) return 0;
    return hc == 4 ? hc::backward_workspace_bytes(n, d) : hc::backward_generic_workspace_bytes(n, hc, d);
}

hc_status hc_block_step_backward(const uint16_t *x, const float *pre_mix, const uint16_t *f,
                                 const float *hc_fn, const float *hc_scale, const float *hc_base,
                                 const float *norm_w, int64_t n, int hc, int d, int sinkhorn_iters,
                                 float eps, float norm_eps, const float *g_h_norm, const float *g_y,
                                 const float *g_pre, float *g_x, float *g_pre_mix, float *g_f,
                                 float *g_hc_fn, float *g_hc_scale, float *g_hc_base,
                                 float *g_norm_w, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (sinkhorn_iters < 1 || sinkhorn_iters > 128 || !finite_nonneg(eps) || !finite_nonneg(norm_eps))
        return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!x || !pre_mix || !f || !hc_fn || !hc_scale || !hc_base || !norm_w || !g_h_norm || !g_y ||
        !g_x || !g_pre_mix || !g_f || !g_hc_fn || !g_hc_scale || !g_hc_base || !g_norm_w || !workspace)
        return HC_ERR_INVALID_ARG;
    if (workspace_bytes < hc_block_step_backward_workspace_bytes(n, hc, d)) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {x, pre_mix, f, hc_fn, hc_scale, hc_base, norm_w, g_h_norm, g_y, g_x,
                          g_pre_mix, g_f, g_hc_fn, g_hc_scale, g_hc_base, g_norm_w, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    if (g_pre && !aligned16(g_pre)) return HC_ERR_MISALIGNED;
    const int64_t mix = (int64_t)(2 + hc) * hc, K = (int64_t)hc * d;
    const Span ins[] = {span(x, n * K * 2), span(pre_mix, n * hc * 4), span(f, n * d * 2),
                        span(hc_fn, mix * K * 4), span(hc_scale, 12), span(hc_base, mix * 4),
                        span(norm_w, d * 4), span(g_h_norm, n * d * 4), span(g_y, n * K * 4),
                        span(g_pre, g_pre ? n * hc * 4 : 0)};
    const Span outs[] = {span(g_x, n * K * 4), span(g_pre_mix, n * hc * 4), span(g_f, n * d * 4),
                         span(g_hc_fn, mix * K * 4), span(g_hc_scale, 12), span(g_hc_base, mix * 4),
                         span(g_norm_w, d * 4), span(workspace, (int64_t)workspace_bytes)};
    if ((st = check_alias(outs, 8, ins, 10)) != HC_OK) return st;
    if (hc != 4)  // two or eight streams: the plain kernels of hc_backward_generic.cu
        return cuda_status(hc::launch_block_step_backward_generic(
            hc, x, pre_mix, f, hc_fn, hc_scale, hc_base, norm_w, n, d, sinkhorn_iters, eps, norm_eps,
            g_h_norm, g_y, g_pre, g_x, g_pre_mix, g_f, g_hc_fn, g_hc_scale, g_hc_base, g_norm_w,
            workspace, stream));
    return cuda_status(hc::launch_block_step_backward(
        x, pre_mix, f, hc_fn, hc_scale, hc_base, norm_w, n, d, sinkhorn_iters, eps, norm_eps,
        g_h_norm, g_y, g_pre, g_x, g_pre_mix, g_f, g_hc_fn, g_hc_scale, g_hc_base, g_norm_w,
        workspace, stream));
}

hc_status hc_block_step_backward_no_workspace(
    const uint16_t *x, const float *pre_mix, const uint16_t *f, const float *hc_fn,
    const float *hc_scale, const float *hc_base, const float *norm_w, int64_t n, int hc, int d,
    int sinkhorn_iters, float eps, float norm_eps, const float *g_h_norm, const float *g_y,
    const float *g_pre, float *g_x, float *g_pre_mix, float *g_f, float *g_hc_fn, float *g_hc_scale,
    float *g_hc_base, float *g_norm_w, cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (hc != 4 || hc::backward_workspace_bytes(n, d) > hc::backward_static_scratch_bytes())
        return HC_ERR_UNSUPPORTED;
    if (n == 0) return HC_OK;
    void *scratch = nullptr;
    if ((st = cuda_status(hc::backward_static_scratch(&scratch))) != HC_OK) return st;
    return hc_block_step_backward(x, pre_mix, f, hc_fn, hc_scale, hc_base, norm_w, n, hc, d,
                                  sinkhorn_iters, eps, norm_eps, g_h_norm, g_y, g_pre, g_x,
                                  g_pre_mix, g_f, g_hc_fn, g_hc_scale, g_hc_base, g_norm_w, scratch,
                                  hc::backward_static_scratch_bytes(), stream);
}

hc_status hc_mxfp8_cast(const uint16_t *in, int64_t rows, int d, uint8_t *codes, uint8_t *scales,
                        cudaStream_t stream) {
    if (rows < 0 || d <= 0) return HC_ERR_INVALID_ARG;
    if (d % 32 != 0) return HC_ERR_UNSUPPORTED;
    if (rows > (INT64_MAX / 8) / d) return HC_ERR_INVALID_ARG;
    if (rows == 0) return HC_OK;
    if (!in || !codes || !scales) return HC_ERR_INVALID_ARG;
    if (!aligned16(in) || !aligned16(codes)) return HC_ERR_MISALIGNED;
    const Span ins[] = {span(in, rows * d * 2)};
    const Span outs[] = {span(codes, rows * d), span(scales, rows * (d / 32))};
    hc_status st = check_alias(outs, 2, ins, 1);
    if (st != HC_OK) return st;
    return cuda_status(hc::launch_mxfp8_cast(in, rows, d, codes, scales, stream));
}

hc_status hc_pre_norm_mxfp8(const uint16_t *x, const float *pre_mix, const float *norm_w, int64_t n,
                            int hc, int d, float norm_eps, uint16_t *h_norm_out, uint8_t *codes,
                            uint8_t *scales, cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (!finite_nonneg(norm_eps)) return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!x || !pre_mix || !norm_w || !codes || !scales) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {x, pre_mix, norm_w, codes};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    if (h_norm_out && !aligned16(h_norm_out)) return HC_ERR_MISALIGNED;
    const Span ins[] = {span(x, n * hc * d * 2), span(pre_mix, n * hc * 4), span(norm_w, d * 4)};
    const Span outs[] = {span(codes, n * d), span(scales, n * (d / 32)),
                         span(h_norm_out, h_norm_out ? n * d * 2 : 0)};
    if ((st = check_alias(outs, 3, ins, 3)) != HC_OK) return st;
    return cuda_status(hc::launch_pre_norm_mxfp8(x, pre_mix, norm_w, n, hc, d, norm_eps, h_norm_out,
                                                 codes, scales, stream));
}

hc_status hc_post(const uint16_t *f, const uint16_t *residual, const float *post,
                  const float *comb, int64_t n, int hc, int d, uint16_t *y,
                  cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (n == 0) return HC_OK;
    if (!f || !residual || !post || !comb || !y) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {f, residual, post, comb, y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    const Span ins[] = {span(f, n * d * 2), span(residual, n * hc * d * 2), span(post, n * hc * 4),
                        span(comb, n * hc * hc * 4)};
    const Span outs[] = {span(y, n * hc * d * 2)};
    if ((st = check_alias(outs, 1, ins, 4)) != HC_OK) return st;
    return cuda_status(hc::launch_post(f, residual, post, comb, n, hc, d, y, stream));
}

hc_status hc_block_step(const uint16_t *x, const float *pre_mix, const uint16_t *f,
                        const float *hc_fn, const float *hc_scale, const float *hc_base,
                        const float *norm_w, int64_t n, int hc, int d, int sinkhorn_iters,
                        float eps, float norm_eps, uint16_t *h_norm, uint16_t *y,
                        float *pre_out, float *post_out, float *comb_out,
                        cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (sinkhorn_iters < 1 || !finite_nonneg(eps) || !finite_nonneg(norm_eps))
        return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!x || !pre_mix || !f || !hc_fn || !hc_scale || !hc_base || !norm_w || !h_norm || !y ||
        !pre_out)
        return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {x, pre_mix, f, hc_fn, hc_scale, hc_base, norm_w, h_norm, y, pre_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    if ((post_out && !aligned16(post_out)) || (comb_out && !aligned16(comb_out)))
        return HC_ERR_MISALIGNED;
    const int64_t mix = (int64_t)(2 + hc) * hc, K = (int64_t)hc * d;
    const Span ins[] = {span(x, n * K * 2),        span(pre_mix, n * hc * 4), span(f, n * d * 2),
                        span(hc_fn, mix * K * 4),  span(hc_scale, 12),        span(hc_base, mix * 4),
                        span(norm_w, d * 4)};
    const Span outs[] = {span(h_norm, n * d * 2), span(y, n * K * 2), span(pre_out, n * hc * 4),
                         span(post_out, post_out ? n * hc * 4 : 0),
                         span(comb_out, comb_out ? n * hc * hc * 4 : 0)};
    if ((st = check_alias(outs, 5, ins, 7)) != HC_OK) return st;
    if (hc == 4 && hc::cluster_path_supported(d))
        return cuda_status(hc::launch_block_cluster(x, pre_mix, f, hc_fn, hc_scale, hc_base, norm_w,
                                                    n, d, sinkhorn_iters, eps, norm_eps, h_norm, y,
                                                    pre_out, post_out, comb_out, nullptr, stream));
    return cuda_status(hc::launch_tokens_simple(x, pre_mix, f, hc_fn, hc_scale, hc_base, norm_w, n,
                                                hc, d, sinkhorn_iters, eps, norm_eps, h_norm, y,
                                                pre_out, post_out, comb_out, nullptr, stream));
}

size_t hc_chain_state_bytes(int64_t n, int hc, int d) {
    if (check_shape(n, hc, d, true) != HC_OK || hc != 4 || !hc::slices_supported(d)) return 0;
    return hc::chain_state_bytes(n);
}

hc_status hc_chain_begin(const uint16_t *x, const float *pre_mix, const float *hc_fn,
                         const float *hc_scale, const float *hc_base, int64_t n, int hc, int d,
                         int sinkhorn_iters, float eps, float norm_eps, float *state_out,
                         size_t state_bytes, float *pre_out, uint16_t *h_pre_out,
                         cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (sinkhorn_iters < 1 || !finite_nonneg(eps) || !finite_nonneg(norm_eps))
        return HC_ERR_INVALID_ARG;
    if (hc != 4 || !hc::slices_supported(d)) return HC_ERR_UNSUPPORTED;
    if (n == 0) return HC_OK;
    if (!x || !pre_mix || !hc_fn || !hc_scale || !hc_base || !state_out) return HC_ERR_INVALID_ARG;
    if (state_bytes < hc::chain_state_bytes(n)) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {x, pre_mix, hc_fn, hc_scale, hc_base, state_out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    if ((pre_out && !aligned16(pre_out)) || (h_pre_out && !aligned16(h_pre_out))) return HC_ERR_MISALIGNED;
    const int64_t mix = (int64_t)(2 + hc) * hc, K = (int64_t)hc * d;
    const Span ins[] = {span(x, n * K * 2), span(pre_mix, n * hc * 4), span(hc_fn, mix * K * 4),
                        span(hc_scale, 12), span(hc_base, mix * 4)};
    const Span outs[] = {span(state_out, (int64_t)state_bytes), span(pre_out, pre_out ? n * hc * 4 : 0),
                         span(h_pre_out, h_pre_out ? n * d * 2 : 0)};
    if ((st = check_alias(outs, 3, ins, 5)) != HC_OK) return st;
    return cuda_status(hc::launch_slices_begin(x, pre_mix, hc_fn, hc_scale, hc_base, n, d,
                                               sinkhorn_iters, eps, norm_eps, state_out, pre_out,
                                               h_pre_out, stream));
}

hc_status hc_chain_side(const uint16_t *x, const uint16_t *f, const float *state_in,
                        const float *norm_w, const float *hc_fn_next, const float *hc_scale_next,
                        const float *hc_base_next, int64_t n, int hc, int d, int sinkhorn_iters,
                        float eps, float norm_eps, uint16_t *h_norm, uint16_t *y,
                        float *state_out, size_t state_bytes, float *pre_out, uint16_t *h_pre_out,
                        cudaStream_t stream) {
    hc_status st = check_shape(n, hc, d, true);
    if (st != HC_OK) return st;
    if (sinkhorn_iters < 1 || !finite_nonneg(eps) || !finite_nonneg(norm_eps))
        return HC_ERR_INVALID_ARG;
    if (hc != 4 || !hc::slices_supported(d)) return HC_ERR_UNSUPPORTED;
    if (n == 0) return HC_OK;
    const bool next = hc_fn_next != nullptr;
    if (!x || !f || !state_in || !norm_w || !y) return HC_ERR_INVALID_ARG;
    // the next side's weights come all together, with a state to write, or not at all
    if (next != (hc_scale_next != nullptr) || next != (hc_base_next != nullptr)) return HC_ERR_INVALID_ARG;
    if (next && (!state_out || state_bytes < hc::chain_state_bytes(n))) return HC_ERR_INVALID_ARG;
    // the next side's bf16 h needs a next side; it and this side's h_norm are one or the other
    if (h_pre_out && (!next || h_norm)) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {x, f, state_in, norm_w, y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    if ((h_norm && !aligned16(h_norm)) || (h_pre_out && !aligned16(h_pre_out))) return HC_ERR_MISALIGNED;
    if (next) {
        const void *nptrs[] = {hc_fn_next, hc_scale_next, hc_base_next, state_out};
        for (const void *p : nptrs)
            if (!aligned16(p)) return HC_ERR_MISALIGNED;
    }
    if (pre_out && !aligned16(pre_out)) return HC_ERR_MISALIGNED;
    const int64_t mix = (int64_t)(2 + hc) * hc, K = (int64_t)hc * d;
    const Span ins[] = {span(x, n * K * 2),
                        span(f, n * d * 2),
                        span(state_in, n * HC_STATE_FLOATS * 4),
                        span(norm_w, d * 4),
                        span(hc_fn_next, next ? mix * K * 4 : 0),
                        span(hc_scale_next, next ? 12 : 0),
                        span(hc_base_next, next ? mix * 4 : 0)};
    const Span outs[] = {span(h_norm, h_norm ? n * d * 2 : 0), span(y, n * K * 2),
                         span(state_out, next ? (int64_t)state_bytes : 0),
                         span(pre_out, (next && pre_out) ? n * hc * 4 : 0),
                         span(h_pre_out, h_pre_out ? n * d * 2 : 0)};
    if ((st = check_alias(outs, 5, ins, 7)) != HC_OK) return st;
    return cuda_status(hc::launch_slices_side(x, f, state_in, norm_w, hc_fn_next, hc_scale_next,
                                              hc_base_next, n, d, sinkhorn_iters, eps, norm_eps,
                                              h_norm, y, next ? state_out : nullptr,
                                              next ? pre_out : nullptr, h_pre_out, stream));
}

hc_status hc_chain_norm(const uint16_t *h_pre, const float *state, const float *norm_w, int64_t n,
                        int d, uint16_t *h_norm, uint8_t *codes, uint8_t *scales,
                        cudaStream_t stream) {
    if (n < 0 || d <= 0) return HC_ERR_INVALID_ARG;
    if (d % 64 != 0 || d > kMaxD) return HC_ERR_UNSUPPORTED;
    if (n > (INT64_MAX / 8) / d) return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!h_pre || !state || !norm_w) return HC_ERR_INVALID_ARG;
    if ((codes == nullptr) != (scales == nullptr) || (!h_norm && !codes)) return HC_ERR_INVALID_ARG;
    const void *ptrs[] = {h_pre, state, norm_w};
    for (const void *p : ptrs)
        if (!aligned16(p)) return HC_ERR_MISALIGNED;
    if ((h_norm && !aligned16(h_norm)) || (codes && !aligned16(codes))) return HC_ERR_MISALIGNED;
    const Span ins[] = {span(h_pre, n * d * 2), span(state, n * HC_STATE_FLOATS * 4), span(norm_w, d * 4)};
    const Span outs[] = {span(h_norm, h_norm ? n * d * 2 : 0), span(codes, codes ? n * d : 0),
                         span(scales, scales ? n * (d / 32) : 0)};
    hc_status st = check_alias(outs, 3, ins, 3);
    if (st != HC_OK) return st;
    return cuda_status(hc::launch_chain_norm(h_pre, state, norm_w, n, d, h_norm, codes, scales, stream));
}

hc_status hc_layer_norm(const void *x, int64_t x_stride, hc_dtype x_type, const void *norm_w,
                        const void *norm_b, hc_dtype w_type, int64_t n, int d, float eps, void *y,
                        int64_t y_stride, float *mean, float *rstd, cudaStream_t stream) {
    hc_status st = check_norm(n, d, x_type, w_type);
    if (st != HC_OK) return st;
    if (!finite_nonneg(eps) || !rows_fit(n, d, x_stride) || !rows_fit(n, d, y_stride) || (n > 1 && y_stride < d))
        return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!x || !norm_w || !y) return HC_ERR_INVALID_ARG;
    const int64_t xb = size_of(x_type), wb = size_of(w_type);
    if (!aligned_to(x, xb) || !aligned_to(y, xb) || !aligned_to(norm_w, wb) || !aligned_to(norm_b, wb) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return HC_ERR_MISALIGNED;
    const Span ins[] = {rows_span(x, n, d, x_stride, x_type), span(norm_w, d * wb), span(norm_b, norm_b ? d * wb : 0)};
    const Span outs[] = {rows_span(y, n, d, y_stride, x_type), span(mean, mean ? n * 4 : 0),
                         span(rstd, rstd ? n * 4 : 0)};
    if ((st = check_alias(outs, 3, ins, 3)) != HC_OK) return st;
    return cuda_status(hc::launch_layer_norm(x, x_stride, x_type, norm_w, norm_b, w_type, n, d, eps, y, y_stride,
                                             mean, rstd, stream));
}

size_t hc_layer_norm_backward_workspace_bytes(int64_t n, int d) {
    if (check_norm(n, d, HC_F32, HC_F32) != HC_OK) return 0;
    return hc::layer_norm_backward_workspace_bytes(n, d);
}

hc_status hc_layer_norm_backward(const void *g_y, int64_t g_stride, hc_dtype g_type, const void *x,
                                 int64_t x_stride, hc_dtype x_type, const void *norm_w,
                                 hc_dtype w_type, const float *mean, const float *rstd, int64_t n,
                                 int d, void *g_x, int64_t gx_stride, float *g_norm_w,
                                 float *g_norm_b, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
    hc_status st = check_norm(n, d, x_type, w_type);
    if (st != HC_OK) return st;
    if (!known(g_type)) return HC_ERR_INVALID_ARG;
    if (g_type != HC_F32 && g_type != x_type) return HC_ERR_UNSUPPORTED;
    if (!rows_fit(n, d, x_stride) || !rows_fit(n, d, g_stride) || !rows_fit(n, d, gx_stride) ||
        (n > 1 && gx_stride < d) || !g_norm_w)
        return HC_ERR_INVALID_ARG;
    if (n > 0 && (!g_y || !x || !norm_w || !mean || !rstd || !g_x || !workspace ||
                  workspace_bytes < hc_layer_norm_backward_workspace_bytes(n, d)))
        return HC_ERR_INVALID_ARG;
    const int64_t xb = size_of(x_type), gb = size_of(g_type), wb = size_of(w_type);
    if (!aligned_to(g_y, gb) || !aligned_to(x, xb) || !aligned_to(norm_w, wb) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4) || !aligned_to(g_x, gb) || !aligned_to(g_norm_w, 4) || !aligned_to(g_norm_b, 4) ||
        (n > 0 && !aligned16(workspace)))
        return HC_ERR_MISALIGNED;
    const Span ins[] = {rows_span(g_y, n, d, g_stride, g_type), rows_span(x, n, d, x_stride, x_type),
                        span(norm_w, n > 0 ? d * wb : 0), span(mean, n * 4), span(rstd, n * 4)};
    const Span outs[] = {rows_span(g_x, n, d, gx_stride, g_type), span(g_norm_w, (int64_t)d * 4),
                         span(g_norm_b, g_norm_b ? (int64_t)d * 4 : 0),
                         span(workspace, (int64_t)hc_layer_norm_backward_workspace_bytes(n, d))};
    if ((st = check_alias(outs, 4, ins, 5)) != HC_OK) return st;
    return cuda_status(hc::launch_layer_norm_backward(g_y, g_stride, g_type, x, x_stride, x_type, norm_w, w_type,
                                                      mean, rstd, n, d, g_x, gx_stride, g_norm_w, g_norm_b,
                                                      workspace, stream));
}

hc_status hc_adamw_step(const hc_adamw_tensor *tensors, int64_t count, double lr, double beta1,
                        double beta2, double eps, double weight_decay, int64_t step,
                        const float *lr_dev, const int64_t *step_dev, const float *grad_scale,
                        cudaStream_t stream) {
    const bool beta_ok = beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0;
    if (count < 0 || count > (1 << 24) || !beta_ok || step < 1 || !(std::isfinite(lr) && lr >= 0.0) ||
        !(std::isfinite(eps) && eps >= 0.0) || !(std::isfinite(weight_decay) && weight_decay >= 0.0))
        return HC_ERR_INVALID_ARG;
    if (count == 0) return HC_OK;
    if (!tensors) return HC_ERR_INVALID_ARG;
    if (!aligned_to(lr_dev, 4) || !aligned_to(step_dev, 8) || !aligned_to(grad_scale, 4)) return HC_ERR_MISALIGNED;
    for (int64_t i = 0; i < count; ++i) {
        const hc_status st = check_adamw_tensor(tensors[i]);
        if (st != HC_OK) return st;
    }
    const int64_t most = 7 * count + 3;
    Use few[128];
    Use *const use = 2 * most <= 128 ? few : new (std::nothrow) Use[2 * most];
    if (!use) return cuda_status(cudaErrorMemoryAllocation);
    int64_t k = 0, at[8];
    const auto add = [&](const void *p, int64_t bytes, bool written) {
        if (!p || bytes <= 0) return;
        const Span r = span(p, bytes);
        use[k++] = Use{r.lo, r.hi, written};
    };
    const hc_adamw_tensor *const end = tensors + count;
    const auto state = [](const hc_adamw_tensor &t) { return t.m_scales ? t.numel : t.numel * 4; };
    for (auto t = tensors; t != end; ++t) add(t->p, t->numel * size_of((hc_dtype)t->p_type), true);
    at[0] = k;
    for (auto t = tensors; t != end; ++t) add(t->g, t->numel * size_of((hc_dtype)t->g_type), false);
    at[1] = k;
    for (auto t = tensors; t != end; ++t) add(t->m, state(*t), true);
    at[2] = k;
    for (auto t = tensors; t != end; ++t) add(t->v, state(*t), true);
    at[3] = k;
    for (auto t = tensors; t != end; ++t) add(t->m_scales, (t->numel + 31) / 32, true);
    at[4] = k;
    for (auto t = tensors; t != end; ++t) add(t->v_scales, (t->numel + 31) / 32, true);
    at[5] = k;
    for (auto t = tensors; t != end; ++t) add(t->p_copy, t->numel * 2, true);
    at[6] = k;
    add(lr_dev, 4, false);
    add(step_dev, 8, false);
    add(grad_scale, 4, false);
    at[7] = k;
    const bool clash = any_overlap(use, use + most, at, 8);
    if (use != few) delete[] use;
    if (clash) return HC_ERR_ALIAS;
    return cuda_status(hc::launch_adamw(tensors, count, lr, beta1, beta2, eps, weight_decay, step, lr_dev, step_dev,
                                        grad_scale, stream));
}

size_t hc_grouped_mm_workspace_bytes(int64_t n, int experts, int N, int K) {
    if (check_grouped(n, experts, N, K, HC_BF16, HC_F32) != HC_OK) return 0;
    return hc::grouped_mm_workspace_bytes(n, experts, N, K);
}

hc_status hc_grouped_mm(const void *x, int64_t x_stride, const void *w, int transposed,
                        const int32_t *offsets, int64_t n, int experts, int N, int K, hc_dtype type,
                        void *y, int64_t y_stride, hc_dtype y_type, int zero_rest,
                        void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    hc_status st = check_grouped(n, experts, N, K, type, y_type);
    if (st != HC_OK) return st;
    if (x_stride < K || y_stride < N || !rows_fit(n, K, x_stride) || !rows_fit(n, N, y_stride)) return HC_ERR_INVALID_ARG;
    if (n == 0) return HC_OK;
    if (!x || !w || !offsets || !y) return HC_ERR_INVALID_ARG;
    if (x_stride % 8 || x_stride >= (int64_t)1 << 38) return HC_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(w) || !aligned_to(offsets, 4) || !aligned_to(y, size_of(y_type)))
        return HC_ERR_MISALIGNED;
    const Span ins[] = {rows_span(x, n, K, x_stride, type), span(w, (int64_t)experts * N * K * 2),
                        span(offsets, ((int64_t)experts + 1) * 4)};
    const size_t need = hc::grouped_mm_workspace_bytes(n, experts, N, K);
    if (need && (!workspace || workspace_bytes < need)) return HC_ERR_INVALID_ARG;
    if (need && !aligned16(workspace)) return HC_ERR_MISALIGNED;
    const Span outs[] = {rows_span(y, n, N, y_stride, y_type), span(need ? workspace : nullptr, (int64_t)need)};
    if ((st = check_alias(outs, 2, ins, 3)) != HC_OK) return st;
    return cuda_status(hc::launch_grouped_mm(x, x_stride, w, transposed != 0, offsets, n, experts, N, K, type == HC_F16, y,
                                             y_stride, y_type == HC_F32, zero_rest != 0, workspace, stream));
}

size_t hc_grouped_mm_weights_workspace_bytes(int64_t n, int experts, int N, int K) {
    if (check_grouped(n, experts, N, K, HC_BF16, HC_F32) != HC_OK) return 0;
    return hc::grouped_mm_weights_workspace_bytes(n, experts, N, K);
}

hc_status hc_grouped_mm_weights(const void *g_y, int64_t g_stride, const void *x, int64_t x_stride,
                                const int32_t *offsets, int64_t n, int experts, int N, int K,
                                hc_dtype type, void *g_w, int transposed, hc_dtype g_type,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    hc_status st = check_grouped(n, experts, N, K, type, g_type);
    if (st != HC_OK) return st;
    if (x_stride < K || g_stride < N || !rows_fit(n, K, x_stride) || !rows_fit(n, N, g_stride)) return HC_ERR_INVALID_ARG;
    if (!g_w || (n > 0 && (!g_y || !x || !offsets))) return HC_ERR_INVALID_ARG;
    if (x_stride % 8 || g_stride % 8 || x_stride >= (int64_t)1 << 38 || g_stride >= (int64_t)1 << 38)
        return HC_ERR_UNSUPPORTED;
    if (!aligned16(g_y) || !aligned16(x) || !aligned_to(offsets, 4) || !aligned_to(g_w, size_of(g_type)))
        return HC_ERR_MISALIGNED;
    const int64_t bytes = (int64_t)experts * N * K * size_of(g_type);
    const size_t need = hc::grouped_mm_weights_workspace_bytes(n, experts, N, K);
    if (need && (!workspace || workspace_bytes < need)) return HC_ERR_INVALID_ARG;
    if (need && !aligned16(workspace)) return HC_ERR_MISALIGNED;
    if (n == 0) return cuda_status(cudaMemsetAsync(g_w, 0, (size_t)bytes, stream));  // sums over no rows
    const Span ins[] = {rows_span(g_y, n, N, g_stride, type), rows_span(x, n, K, x_stride, type),
                        span(offsets, ((int64_t)experts + 1) * 4)};
    const Span outs[] = {span(g_w, bytes), span(need ? workspace : nullptr, (int64_t)need)};
    if ((st = check_alias(outs, 2, ins, 3)) != HC_OK) return st;
    // the innermost axis of g_w goes on the MMA's M side
    const bool f16 = type == HC_F16, f32 = g_type == HC_F32;
    return cuda_status(transposed
                           ? hc::launch_grouped_mm_weights(x, x_stride, K, g_y, g_stride, N, offsets, n, experts, f16, g_w, f32,
                                                             workspace, stream)
                           : hc::launch_grouped_mm_weights(g_y, g_stride, N, x, x_stride, K, offsets, n, experts, f16, g_w, f32,
                                                             workspace, stream));
}

}  // extern "C"
