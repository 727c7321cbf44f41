// layer_norm.cuh -- layer norm of token rows and its backward pass (layer_norm.cu).
#pragma once
#include "common.cuh"

namespace vae {

constexpr int kLayerNormMaxC = 8192;

// y = gamma (x - mean) rstd + beta; stats [rows][2] (mean, rstd) where not NULL.
int layer_norm(const void *x, int dtype, long long rows, int c, float eps, const float *gamma,
               const float *beta, void *y, float *stats, cudaStream_t s);

size_t layer_norm_backward_ws_bytes(long long rows, int c);
int layer_norm_backward(const void *dy, const void *x, int dtype, const float *stats,
                        long long rows, int c, const float *gamma, const void *dres, void *dx,
                        float *dgamma, float *dbeta, void *ws, cudaStream_t s);

}  // namespace vae
