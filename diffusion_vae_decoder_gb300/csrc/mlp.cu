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
// Whether two arrays have memory in common: what a product writes with what it reads.
// partly: and are not the same one, which operators that go through both number by number
// write over.
bool meet(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
  const auto p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p && q && p < q + b_bytes && q < p + a_bytes;
}
bool partly(const void *a, const void *b, size_t bytes) { return a != b && meet(a, bytes, b, bytes); }
size_t bytes_of(int dtype, long long rows, long long c) {
  return static_cast<size_t>(rows) * c * dtype_bytes(dtype);
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
  if (partly(y, x, bytes_of(dtype, rows, c))) return VAE_EINVAL;
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
  const size_t size = bytes_of(dtype, rows, c);
  if (partly(dx, dy, size) || partly(dx, x, size) || partly(dx, dres, size)) return VAE_EINVAL;
  return layer_norm_backward(dy, x, dtype, stats, rows, c, gamma, dres, dx, dgamma, dbeta, ws,
                             cu(stream));
}

// ------------------------------------------------------------------ dropout
int vae_dropout(const void *x, int dtype, long long count, double p, unsigned long long seed,
                unsigned long long offset, const long long *state, const void *residual, void *y,
                vae_stream_t stream) {
  if (!x || !y || !dtype_ok(dtype) || count <= 0 || !(p >= 0.0 && p <= 1.0)) return VAE_EINVAL;
  if (!all_aligned(x, residual, y) || reinterpret_cast<uintptr_t>(state) % 8) return VAE_EINVAL;
  const size_t size = bytes_of(dtype, count, 1);
  if (partly(y, x, size) || partly(y, residual, size)) return VAE_EINVAL;
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
  if (!x || !w || !y || !act_ok(act)) return VAE_EINVAL;
  VAE_TRY(linear_args_ok(dtype, rows, n, k));
  if (!all_aligned(x, w, bias, residual, y, z, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, linear_ws_bytes(dtype, rows, n, k)));
  const size_t xs = bytes_of(dtype, rows, k), wsz = bytes_of(dtype, n, k),
               ys = bytes_of(dtype, rows, n);
  if (meet(y, ys, x, xs) || meet(y, ys, w, wsz) || partly(y, residual, ys) || meet(z, ys, x, xs) ||
      meet(z, ys, w, wsz) || meet(z, ys, y, ys) || meet(z, ys, residual, ys))
    return VAE_EINVAL;
  return linear(x, dtype, rows, k, w, bias, n, act, residual, y, z, ws, cu(stream));
}

size_t vae_linear_dgrad_workspace_size(int dtype, long long rows, int n, int k) {
  return linear_args_ok(dtype, rows, n, k) == VAE_OK ? linear_dgrad_ws_bytes(dtype, rows, n, k) : 0;
}

int vae_linear_dgrad(const void *dy, int dtype, long long rows, int n, const void *w, int k,
                     int act, const void *z, void *dx, void *ws, size_t ws_bytes,
                     vae_stream_t stream) {
  if (!dy || !w || !dx || !act_ok(act) || (act != VAE_ACT_NONE) != (z != nullptr))
    return VAE_EINVAL;
  VAE_TRY(linear_args_ok(dtype, rows, n, k));
  if (!all_aligned(dy, w, z, dx, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, linear_dgrad_ws_bytes(dtype, rows, n, k)));
  const size_t size = bytes_of(dtype, rows, k);
  if (meet(dx, size, dy, bytes_of(dtype, rows, n)) || meet(dx, size, w, bytes_of(dtype, n, k)) ||
      partly(dx, z, size))
    return VAE_EINVAL;
  return linear_dgrad(dy, dtype, rows, n, w, k, act, z, dx, ws, cu(stream));
}

size_t vae_linear_wgrad_workspace_size(int dtype, long long rows, int n, int k) {
  return linear_args_ok(dtype, rows, n, k) == VAE_OK ? linear_wgrad_ws_bytes(dtype, rows, n, k) : 0;
}

int vae_linear_wgrad(const void *dy, const void *x, int dtype, long long rows, int n, int k,
                     float *dw, float *dbias, void *ws, size_t ws_bytes, vae_stream_t stream) {
  if (!dy || !x || !dw) return VAE_EINVAL;
  VAE_TRY(linear_args_ok(dtype, rows, n, k));
  if (!all_aligned(dy, x, dw, dbias, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, linear_wgrad_ws_bytes(dtype, rows, n, k)));
  const size_t ds = bytes_of(dtype, rows, n), xs = bytes_of(dtype, rows, k),
               dws = bytes_of(VAE_F32, n, k), dbs = bytes_of(VAE_F32, 1, n);
  if (meet(dw, dws, dy, ds) || meet(dw, dws, x, xs) || meet(dbias, dbs, dy, ds) ||
      meet(dbias, dbs, x, xs) || meet(dbias, dbs, dw, dws))
    return VAE_EINVAL;
  return linear_wgrad(dy, x, dtype, rows, n, k, dw, dbias, ws, cu(stream));
}

}  // extern "C"
