// gn_train.cuh -- GroupNorm(+SiLU) that keeps 8-bit checkpoints, and its
// backward pass (gn_train.cu).
#pragma once
#include "ckpt.cuh"

namespace vae {

// Room for the statistics, their partials and the per-channel sums.
size_t gn_ckpt_ws_bytes(int n, int c, long long spatial, int groups);
size_t gn_backward_ws_bytes(int n, int c, long long spatial, int groups);

// y = act(GroupNorm(x)); stats [n][groups] (mean, 1 / sqrt(var + eps));
// x_ckpt / y_ckpt: views with q == nullptr are not written.
int gn_ckpt(const float *x, int n, int c, long long spatial, int nhwc, int groups, float eps,
            const float *gamma, const float *beta, int silu, float *y, CkptView x_ckpt,
            CkptView y_ckpt, float *stats, void *ws, cudaStream_t s);

int gn_backward(const float *dy, CkptView x_ckpt, const float *stats, int n, int c,
                long long spatial, int nhwc, int groups, const float *gamma, const float *beta,
                int silu, const float *dres, float *dx, float *dgamma, float *dbeta, void *ws,
                cudaStream_t s);

}  // namespace vae
