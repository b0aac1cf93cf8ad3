// hc_sublayer.h -- internal launcher prototypes of the sublayer operators
// (layer norm, experts' matrix products, AdamW).  Arguments have been
// validated by hc_api.cu before any of these is called.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/hc.h"

namespace hc {

// ------------------------------------------------------------ layer norm (hc_layer_norm.cu)
cudaError_t launch_layer_norm(const void *x, int64_t x_stride, hc_dtype x_type, const void *w, const void *b,
                              hc_dtype w_type, int64_t n, int d, float eps, void *y, int64_t y_stride,
                              float *mean, float *rstd, cudaStream_t s);

size_t layer_norm_backward_workspace_bytes(int64_t n, int d);
cudaError_t launch_layer_norm_backward(const void *g_y, int64_t g_stride, hc_dtype g_type, const void *x,
                                       int64_t x_stride, hc_dtype x_type, const void *w, hc_dtype w_type,
                                       const float *mean, const float *rstd, int64_t n, int d, void *g_x,
                                       int64_t gx_stride, float *g_w, float *g_b, void *workspace,
                                       cudaStream_t s);

// ------------------------------------------------------------ AdamW (hc_adamw.cu)
cudaError_t launch_adamw(const hc_adamw_tensor *tensors, int64_t count, double lr, double beta1, double beta2,
                         double eps, double weight_decay, int64_t step, const float *lr_dev, const int64_t *step_dev,
                         const float *grad_scale, cudaStream_t s);

// as the other files' (hc_launch.h)
cudaError_t consume_layer_norm_device_error(cudaStream_t s, unsigned int *flag);

// ------------------------------------------------------------ experts' products (hc_grouped_mm.cu)
// y [n, N] = x [n, K] w[e]^T, w [experts][N][K] (w_kn: [experts][K][N]).
cudaError_t launch_grouped_mm(const void *x, int64_t x_stride, const void *w, bool w_kn, const int32_t *offsets, int64_t n,
                              int experts, int N, int K, bool fp16, void *y, int64_t y_stride, bool y_f32,
                              bool zero_rest, void *workspace, cudaStream_t s);
size_t grouped_mm_workspace_bytes(int64_t n, int experts, int N, int K);
// g_w [experts][C][F] = sum over the expert's rows of b[r][c] a[r][f].
cudaError_t launch_grouped_mm_weights(const void *b, int64_t b_stride, int C, const void *a, int64_t a_stride, int F,
                                      const int32_t *offsets, int64_t n, int experts, bool fp16, void *g_w,
                                      bool g_f32, void *workspace, cudaStream_t s);
size_t grouped_mm_weights_workspace_bytes(int64_t n, int experts, int N, int K);
// as the other files' (hc_launch.h); bit 1 (value 2): offsets out of order or out of range
cudaError_t consume_grouped_mm_device_error(cudaStream_t s, unsigned int *flag);

}  // namespace hc
