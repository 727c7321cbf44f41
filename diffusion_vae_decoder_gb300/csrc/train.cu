// train.cu -- the C-ABI entry points of the training operators: argument
// checks, then the kernels of ckpt.cu, gn_train.cu, wgrad.cu and block_norm.cu.
#include "block_norm.cuh"
#include "ckpt.cuh"
#include "gn_train.cuh"
#include "wgrad.cuh"

using namespace vae;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
template <class... T>
bool all_aligned(T... p) {
  return (aligned16(p) && ...);
}

constexpr long long kMaxRows = 0x7fffffffll;  // pixels or tokens of one call
constexpr int kMaxSamples = 65535;            // a grid dimension

// An optional checkpoint's two arrays: both or none.
bool pair(const void *q, const void *scale) { return (q != nullptr) == (scale != nullptr); }

// A workspace of `need` bytes (none: ws may be NULL).
int workspace_ok(const void *ws, size_t ws_bytes, size_t need) {
  if (!need) return VAE_OK;
  if (!ws) return VAE_EINVAL;
  return ws_bytes < need ? VAE_EWORKSPACE : VAE_OK;
}

int act_args_ok(int n, int c, long long spatial, int layout) {
  if (n <= 0 || c <= 0 || spatial <= 0) return VAE_EINVAL;
  if (layout != VAE_NCHW && layout != VAE_NHWC) return VAE_EINVAL;
  if (n > kMaxSamples || spatial > kMaxRows / n) return VAE_EUNSUPPORTED;
  return VAE_OK;
}

int gn_args_ok(int n, int c, long long spatial, int layout, int groups) {
  VAE_TRY(act_args_ok(n, c, spatial, layout));
  if (groups <= 0) return VAE_EINVAL;
  if (c % groups || c % 4 || c > 1024) return VAE_EUNSUPPORTED;
  return VAE_OK;
}

int block_norm_args_ok(int n, long long tokens, int c) {
  if (n <= 0 || tokens <= 0 || c <= 0) return VAE_EINVAL;
  if (c % 4 || c > kBlockNormMaxC || n > kMaxSamples || tokens > kMaxRows / n)
    return VAE_EUNSUPPORTED;
  return VAE_OK;
}

int wgrad_args_ok(int n, int cin, int h, int w, int layout, int cout, int k) {
  if (n <= 0 || cin <= 0 || h <= 0 || w <= 0 || cout <= 0) return VAE_EINVAL;
  if (layout != VAE_NCHW && layout != VAE_NHWC) return VAE_EINVAL;
  if (k != 1 && k != 3) return VAE_EUNSUPPORTED;
  if (cin > 4096 || cout > 4096 || h > 65535 || w > 65535) return VAE_EUNSUPPORTED;
  // the reduction walks rows of w + 1 positions with 32-bit indexes
  if (static_cast<long long>(h) * (w + 1ll) > kMaxRows / 2 / n) return VAE_EUNSUPPORTED;
  if (layout == VAE_NHWC && cout % 4) return VAE_EUNSUPPORTED;
  return VAE_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ checkpoints
size_t vae_ckpt_bytes(long long rows, int c) {
  if (rows <= 0 || c <= 0 || rows > kMaxRows || c > 65536) return 0;
  return ckpt_bytes(rows, c);
}

int vae_ckpt_pack(const float *x, int n, int c, long long spatial, int layout, void *q,
                  void *scale, vae_stream_t stream) {
  if (!x || !q || !scale) return VAE_EINVAL;
  VAE_TRY(act_args_ok(n, c, spatial, layout));
  if (c > 65536) return VAE_EUNSUPPORTED;
  if (!all_aligned(x, q, scale)) return VAE_EINVAL;
  return ckpt_pack(x, n, c, spatial, layout == VAE_NHWC, ckpt_view(q, scale),
                   reinterpret_cast<cudaStream_t>(stream));
}

int vae_ckpt_unpack(const void *q, const void *scale, int n, int c, long long spatial, int layout,
                    float *x, vae_stream_t stream) {
  if (!x || !q || !scale) return VAE_EINVAL;
  VAE_TRY(act_args_ok(n, c, spatial, layout));
  if (c > 65536) return VAE_EUNSUPPORTED;
  if (!all_aligned(x, q, scale)) return VAE_EINVAL;
  return ckpt_unpack(ckpt_view(q, scale), n, c, spatial, layout == VAE_NHWC, x,
                     reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ GroupNorm + SiLU
size_t vae_groupnorm_silu_ckpt_workspace_size(int n, int c, long long spatial, int layout,
                                              int groups) {
  return gn_args_ok(n, c, spatial, layout, groups) == VAE_OK
             ? gn_ckpt_ws_bytes(n, c, spatial, layout == VAE_NHWC, groups) : 0;
}

int vae_groupnorm_silu_ckpt(const float *x, int n, int c, long long spatial, int layout,
                            int groups, float eps, const float *gamma, const float *beta,
                            int apply_silu, float *y, void *x_q, void *x_scale, void *y_q,
                            void *y_scale, float *stats, void *ws, size_t ws_bytes,
                            vae_stream_t stream) {
  if (!x || !gamma || !beta || !y || !stats || !pair(x_q, x_scale) || !pair(y_q, y_scale))
    return VAE_EINVAL;
  VAE_TRY(gn_args_ok(n, c, spatial, layout, groups));
  if (!all_aligned(x, y, x_q, x_scale, y_q, y_scale, stats, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, gn_ckpt_ws_bytes(n, c, spatial, layout == VAE_NHWC, groups)));
  return gn_ckpt(x, n, c, spatial, layout == VAE_NHWC, groups, eps, gamma, beta, apply_silu != 0,
                 y, ckpt_view(x_q, x_scale), ckpt_view(y_q, y_scale), stats, ws,
                 reinterpret_cast<cudaStream_t>(stream));
}

size_t vae_groupnorm_silu_backward_workspace_size(int n, int c, long long spatial, int layout,
                                                  int groups) {
  return gn_args_ok(n, c, spatial, layout, groups) == VAE_OK
             ? gn_backward_ws_bytes(n, c, spatial, layout == VAE_NHWC, groups) : 0;
}

int vae_groupnorm_silu_backward(const float *dy, const void *x_q, const void *x_scale,
                                const float *stats, int n, int c, long long spatial, int layout,
                                int groups, const float *gamma, const float *beta,
                                int apply_silu, const float *dres, float *dx, float *dgamma, float *dbeta,
                                void *ws, size_t ws_bytes, vae_stream_t stream) {
  if (!dy || !x_q || !x_scale || !stats || !gamma || !beta || !dx) return VAE_EINVAL;
  VAE_TRY(gn_args_ok(n, c, spatial, layout, groups));
  if (!all_aligned(dy, x_q, x_scale, stats, dres, dx, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes,
                       gn_backward_ws_bytes(n, c, spatial, layout == VAE_NHWC, groups)));
  return gn_backward(dy, ckpt_view(x_q, x_scale), stats, n, c, spatial,
                     layout == VAE_NHWC, groups, gamma, beta, apply_silu != 0, dres, dx, dgamma,
                     dbeta, ws, reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ conv weight gradient
size_t vae_conv2d_wgrad_workspace_size(int n, int cin, int h, int w, int layout, int cout,
                                       int k) {
  return wgrad_args_ok(n, cin, h, w, layout, cout, k) == VAE_OK
             ? wgrad_ws_bytes(n, cin, h, w, cout, k) : 0;
}

int vae_conv2d_wgrad(const float *dy, const void *x_q, const void *x_scale, int n, int cin, int h,
                     int w, int layout, int cout, int k, float *dw, float *dbias, void *ws,
                     size_t ws_bytes, vae_stream_t stream) {
  if (!dy || !x_q || !x_scale || !dw) return VAE_EINVAL;
  VAE_TRY(wgrad_args_ok(n, cin, h, w, layout, cout, k));
  if (!all_aligned(dy, x_q, x_scale, ws)) return VAE_EINVAL;
  VAE_TRY(workspace_ok(ws, ws_bytes, wgrad_ws_bytes(n, cin, h, w, cout, k)));
  return wgrad(dy, ckpt_view(x_q, x_scale), n, cin, h, w, layout == VAE_NHWC, cout, k, dw,
               dbias, ws, reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------ block norm
int vae_block_norm(const float *u, const float *x, int n, long long tokens, int c, float eps,
                   const float *w_post, const float *gate, const float *scale,
                   const float *w_pre, float *h, float *y, void *u_q, void *u_scale, void *h_q,
                   void *h_scale, float *rstd, vae_stream_t stream) {
  if (!u || !x || !w_post || !h) return VAE_EINVAL;
  if ((w_pre != nullptr) != (y != nullptr)) return VAE_EINVAL;
  // keeping: u's checkpoint and rstd, and h's exactly where there is a norm of h
  if (!pair(u_q, u_scale) || !pair(h_q, h_scale) || (u_q != nullptr) != (rstd != nullptr))
    return VAE_EINVAL;
  if ((h_q != nullptr) != (u_q && w_pre)) return VAE_EINVAL;
  VAE_TRY(block_norm_args_ok(n, tokens, c));
  if (!all_aligned(u, x, w_post, gate, scale, w_pre, h, y, u_q, u_scale, h_q, h_scale))
    return VAE_EINVAL;
  const BlockNormArgs a{n, tokens, c, w_post, gate, scale, w_pre};
  return block_norm(a, u, x, eps, h, y, ckpt_view(u_q, u_scale), ckpt_view(h_q, h_scale), rstd,
                    reinterpret_cast<cudaStream_t>(stream));
}

size_t vae_block_norm_backward_workspace_size(int n, long long tokens, int c, int has_gate) {
  if (block_norm_args_ok(n, tokens, c) != VAE_OK) return 0;
  BlockNormArgs a{n, tokens, c, nullptr, nullptr, nullptr, nullptr};
  static const float present = 0.f;
  if (has_gate) a.gate = &present;
  return block_norm_backward_ws_bytes(a);
}

int vae_block_norm_backward(const float *dy, const float *dh, const void *u_q,
                            const void *u_scale, const void *h_q, const void *h_scale,
                            const float *rstd, int n, long long tokens, int c,
                            const float *w_post, const float *gate, const float *scale,
                            const float *w_pre, float *du, float *dx, float *dw_post,
                            float *dgate, float *dscale, float *dw_pre, void *ws, size_t ws_bytes,
                            vae_stream_t stream) {
  if (!u_q || !u_scale || !rstd || !w_post || !du || !dx || !pair(h_q, h_scale))
    return VAE_EINVAL;
  if ((w_pre != nullptr) != (dy != nullptr) || (w_pre != nullptr) != (h_q != nullptr))
    return VAE_EINVAL;
  if (!dy && !dh) return VAE_EINVAL;
  if ((dgate && !gate) || (dscale && !scale) || (dw_pre && !w_pre)) return VAE_EINVAL;
  VAE_TRY(block_norm_args_ok(n, tokens, c));
  if (!all_aligned(dy, dh, u_q, u_scale, h_q, h_scale, w_post, gate, scale, w_pre, du, dx, ws))
    return VAE_EINVAL;
  const BlockNormArgs a{n, tokens, c, w_post, gate, scale, w_pre};
  VAE_TRY(workspace_ok(ws, ws_bytes, block_norm_backward_ws_bytes(a)));
  return block_norm_backward(a, dy, dh, ckpt_view(u_q, u_scale),
                             ckpt_view(h_q, h_scale), rstd, du, dx, dw_post, dgate,
                             dscale, dw_pre, ws, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
