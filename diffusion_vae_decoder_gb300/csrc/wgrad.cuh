// wgrad.cuh -- weight gradient of the stride-1 convs from an 8-bit checkpoint
// of the conv's input (wgrad.cu).
#pragma once
#include "ckpt.cuh"

namespace vae {

size_t wgrad_ws_bytes(int n, int cin, int h, int w, int cout, int k);
int wgrad(const float *dy, CkptView x_ckpt, int n, int cin, int h, int w, int nhwc, int cout,
          int k, float *dw, float *dbias, void *ws, cudaStream_t s);

}  // namespace vae
