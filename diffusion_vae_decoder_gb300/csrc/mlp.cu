// mlp.cu -- the C-ABI entry points of a transformer MLP's operators: argument
// checks, then the kernels of layer_norm.cu, dropout.cu and linear.cu.
#include <cmath>

#include "dropout.cuh"
#include "layer_norm.cuh"
#include "linear.cuh"
#include "tokens.cuh"

using namespace vae;

namespace {

constexpr long long kMaxRows = 0x7ffffe00ll;  // tokens of one call

template <class... T>
bool all_aligned(T... p) {
  return ((reinterpret_cast<uintptr_t>(p) % 16 == 0) && ...);
}

int norm_args_ok(long long rows, int c) {
  if (rows <= 0 || c <= 0) return VAE_EINVAL;
  if (rows > kMaxRows || c % 4 || c > kLayerNormMaxC) return VAE_EUNSUPPORTED;
  return VAE_OK;
}
int linear_args_ok(int dtype, long long rows, int n, int k) {
  if (!dtype_ok(dtype) || rows <= 0 || n <= 0 || k <= 0) return VAE_EINVAL;
  if (rows > kMaxRows || n % 8 || k % 8 || n > 65536 || k > 65536) return VAE_EUNSUPPORTED;
  return VAE_OK;
}
// Whether `out` is one of the arrays that a product reads while it writes.
template <class... T>
bool one_of(const void *out, T... in) {
  return out && ((out == static_cast<const void *>(in)) || ...);
}
bool act_ok(int act) { return act == VAE_ACT_NONE || act == VAE_ACT_SILU || act == VAE_ACT_GELU; }
int workspace_ok(const void *ws, size_t ws_bytes, size_t need) {
  if (!need) return VAE_OK;
  if (!ws) return VAE_EINVAL;
  return ws_bytes < need ? VAE_EWORKSPACE : VAE_OK;
}
cudaStream_t cu(vae_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

// ------------------------------------------------------------------ layer norm
int vae_layer_norm(const void *x, int dtype, long long rows, int c, float eps, const float *gamma,
                   const float *beta, void *y, float *stats, vae_stream_t stream) {
  if (!x || !gamma || !y || !dtype_ok(dtype)) return VAE_EINVAL;
  VAE_TRY(norm_args_ok(rows, c));
  if (!all_aligned(x, gamma, beta, y, stats)) return VAE_EINVAL;
  return layer_norm(x, dtype, rows, c, eps, gamma, beta, y, stats, cu(stream));
}

size_t vae_layer_norm_backward_workspace_size(long long rows, int c) {
  return norm_args_ok(rows, c) == VAE_OK ? layer_norm_backward_ws_bytes(rows, c) : 0;
}

int vae_layer_norm_backward(const void *dy, const void *x, int dtype, const float *stats,
                            long long rows, int c, const float *gamma, const void *dres, void *dx,
                            float *dgamma, float *dbeta, void *ws, size_t ws_bytes,
                            vae_stream_t stream) {
  if (!dy || !x || !stats || !gamma || !dx || !dtype_ok(dtype)) return VAE_EINVAL;
  VAE_TRY(norm_args_ok(rows, c));
  if (!all_aligned(dy, x, stats, gamma, dres, dx, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, layer_norm_backward_ws_bytes(rows, c)));
  return layer_norm_backward(dy, x, dtype, stats, rows, c, gamma, dres, dx, dgamma, dbeta, ws,
                             cu(stream));
}

// ------------------------------------------------------------------ dropout
int vae_dropout(const void *x, int dtype, long long count, double p, unsigned long long seed,
                unsigned long long offset, const long long *state, const void *residual, void *y,
                vae_stream_t stream) {
  if (!x || !y || !dtype_ok(dtype) || count <= 0 || !(p >= 0.0 && p <= 1.0)) return VAE_EINVAL;
  if (!all_aligned(x, residual, y) || reinterpret_cast<uintptr_t>(state) % 8) return VAE_EINVAL;
  return dropout(x, dtype, count, static_cast<uint32_t>(std::floor(65536.0 * p + 0.5)), seed,
                 offset, state, residual, y, cu(stream));
}

// ------------------------------------------------------------------ linear
size_t vae_linear_workspace_size(int dtype, long long rows, int n, int k) {
  return linear_args_ok(dtype, rows, n, k) == VAE_OK ? linear_ws_bytes(dtype, rows, n, k) : 0;
}

int vae_linear(const void *x, int dtype, long long rows, int k, const void *w, const float *bias,
               int n, int act, const void *residual, void *y, void *z, void *ws, size_t ws_bytes,
               vae_stream_t stream) {
  if (!x || !w || !y || !act_ok(act) || one_of(y, x, w) || one_of(z, x, w, y, residual))
    return VAE_EINVAL;
  VAE_TRY(linear_args_ok(dtype, rows, n, k));
  if (!all_aligned(x, w, bias, residual, y, z, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, linear_ws_bytes(dtype, rows, n, k)));
  return linear(x, dtype, rows, k, w, bias, n, act, residual, y, z, ws, cu(stream));
}

size_t vae_linear_dgrad_workspace_size(int dtype, long long rows, int n, int k) {
  return linear_args_ok(dtype, rows, n, k) == VAE_OK ? linear_dgrad_ws_bytes(dtype, rows, n, k) : 0;
}

int vae_linear_dgrad(const void *dy, int dtype, long long rows, int n, const void *w, int k,
                     int act, const void *z, void *dx, void *ws, size_t ws_bytes,
                     vae_stream_t stream) {
  if (!dy || !w || !dx || !act_ok(act) || (act != VAE_ACT_NONE) != (z != nullptr) ||
      one_of(dx, dy, w))
    return VAE_EINVAL;
  VAE_TRY(linear_args_ok(dtype, rows, n, k));
  if (!all_aligned(dy, w, z, dx, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, linear_dgrad_ws_bytes(dtype, rows, n, k)));
  return linear_dgrad(dy, dtype, rows, n, w, k, act, z, dx, ws, cu(stream));
}

size_t vae_linear_wgrad_workspace_size(int dtype, long long rows, int n, int k) {
  return linear_args_ok(dtype, rows, n, k) == VAE_OK ? linear_wgrad_ws_bytes(dtype, rows, n, k) : 0;
}

int vae_linear_wgrad(const void *dy, const void *x, int dtype, long long rows, int n, int k,
                     float *dw, float *dbias, void *ws, size_t ws_bytes, vae_stream_t stream) {
  if (!dy || !x || !dw || one_of(dw, dy, x) || one_of(dbias, dy, x, dw)) return VAE_EINVAL;
  VAE_TRY(linear_args_ok(dtype, rows, n, k));
  if (!all_aligned(dy, x, dw, dbias, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, linear_wgrad_ws_bytes(dtype, rows, n, k)));
  return linear_wgrad(dy, x, dtype, rows, n, k, dw, dbias, ws, cu(stream));
}

}  // extern "C"
