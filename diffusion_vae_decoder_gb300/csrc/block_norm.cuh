// block_norm.cuh -- the token norm around a block (block_norm.cu).
#pragma once
#include "ckpt.cuh"

namespace vae {

constexpr int kBlockNormMaxC = 4096;

struct BlockNormArgs {
  int n;             // samples (rows of gate)
  long long tokens;  // tokens per sample
  int c;
  const float *w_post, *gate, *scale, *w_pre;  // gate, scale, w_pre may be NULL
};

// h = x + gate scale (u / rms(u)) w_post, y = h / rms(h) w_pre; with u_ckpt.q
// also the checkpoints of u (and of h when w_pre) and rstd [2][rows].
int block_norm(const BlockNormArgs &a, const float *u, const float *x, float eps, float *h,
               float *y, CkptView u_ckpt, CkptView h_ckpt, float *rstd, cudaStream_t s);

size_t block_norm_backward_ws_bytes(const BlockNormArgs &a);
int block_norm_backward(const BlockNormArgs &a, const float *dy, const float *dh, CkptView u_ckpt,
                        CkptView h_ckpt, const float *rstd, float *du, float *dx, float *dw_post,
                        float *dgate, float *dscale, float *dw_pre, void *ws, cudaStream_t s);

}  // namespace vae
