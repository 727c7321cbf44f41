// block_norm.cu -- the norms before and after a transformer block, fused with
// the block's gate, residual scale and residual sum, and their backward pass
// from 8-bit checkpoints. Token-major rows of c channels.
//
// Forward, per row of sample n, with rms(v) = sqrt(mean(v^2) + eps):
//   m = 1 / rms(u), uh = u m       h = x + gate[n] scale w_post uh
//   r = 1 / rms(h), hh = h r       y = w_pre hh
// Backward, uh and hh from the checkpoints' u~, h~ and the saved m, r:
//   dH = dh + r (w_pre dy - hh mean(hh w_pre dy));        dx = dH
//   t = gate scale w_post dH;   du = m (t - uh mean(uh t))
//   S[n][c] = sum over n's rows of dH uh, from which
//   dgate[n] = scale w_post S[n], dscale = sum_n gate w_post S[n],
//   dw_post = sum_n gate scale S[n];   dw_pre = sum over all rows of dy hh
// (the three gradients share one column sum: their factors do not depend on
// the row).
//
// A row stays in the registers of W warps, four channels at a time, so each
// tensor moves once: 16 bytes per element forward (18.06 with checkpoints),
// 18.06 backward; HBM bounds both, launch latency a single token. Column sums
// run in registers over the rows of a block and meet in a fixed order.
#include <type_traits>

#include "block_norm.cuh"

namespace vae {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBwdBlocks = 2 * 152;

// Sum over the W warps of a row; `buf` holds kWarps floats and alternates
// between two calls, so one barrier per call is enough.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += buf[warp / W * W + i];
  }
  return v;
}

__device__ __forceinline__ float4 ld4(const float *p) {
  return __ldg(reinterpret_cast<const float4 *>(p));
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z),
                     fmaf(a.w, b.w, c.w));
}
__device__ __forceinline__ float4 mul4s(float4 a, float b) {
  return make_float4(a.x * b, a.y * b, a.z * b, a.w * b);
}

// Channels of thread `tid` of a row's W warps: quad i starts at 4 (i T + tid).
template <int W, int NV, bool KEEP>
__global__ void __launch_bounds__(kThreads)
    block_norm_fwd(const float *u, const float *x, unsigned rows, unsigned tokens, int c,
                   float eps, const float *__restrict__ w_post, const float *__restrict__ gate,
                   const float *__restrict__ scale, const float *__restrict__ w_pre, float *h,
                   float *y, CkptView ku, CkptView kh, float *__restrict__ rstd) {
  constexpr int T = 32 * W, R = kWarps / W;  // threads per row, rows per block
  __shared__ float buf[2][kWarps];
  const int tid = threadIdx.x % T, cp = (c + 31) & ~31;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f), one = make_float4(1.f, 1.f, 1.f, 1.f);
  float4 f[NV], wp[NV];  // w_post scale; w_pre
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = 4 * (i * T + tid);
    f[i] = ch < c ? ld4(w_post + ch) : zero;
    if (scale && ch < c) f[i] = mul4(f[i], ld4(scale + ch));
    wp[i] = w_pre && ch < c ? ld4(w_pre + ch) : zero;
  }
  for (unsigned r0 = blockIdx.x * R; r0 < rows; r0 += gridDim.x * R) {
    const unsigned row = r0 + threadIdx.x / T;
    const bool live = row < rows;
    const size_t at = static_cast<size_t>(row) * c;
    const float *g = gate && live ? gate + static_cast<size_t>(row / tokens) * c : nullptr;
    float4 v[NV], xv[NV];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 4 * (i * T + tid);
      const bool in = live && ch < c;
      v[i] = in ? __ldcs(reinterpret_cast<const float4 *>(u + at + ch)) : zero;
      xv[i] = in ? __ldcs(reinterpret_cast<const float4 *>(x + at + ch)) : zero;
      ss += dot4(v[i], v[i]);
    }
    const float m = rsqrtf(row_sum<W>(ss, buf[0]) / c + eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 4 * (i * T + tid);
      if (KEEP) {
        uint32_t byte;
        const uint32_t b = octet_quantise(v[i], &byte);
        if (live && ch < cp) {
          __stcs(reinterpret_cast<uint32_t *>(ku.q + static_cast<size_t>(row) * cp + ch), b);
          if ((tid & 7) == 0)
            ku.scale[static_cast<size_t>(row) * (cp >> 5) + (ch >> 5)] =
                static_cast<uint8_t>(byte);
        }
      }
      const float4 gf = mul4(f[i], g && ch < c ? ld4(g + ch) : one);
      v[i] = fma4(gf, mul4s(v[i], m), xv[i]);
      if (live && ch < c) __stcs(reinterpret_cast<float4 *>(h + at + ch), v[i]);
      ss += dot4(v[i], v[i]);
    }
    if (KEEP && live && tid == 0) rstd[row] = m;
    if (!w_pre) {
      if (W > 1) __syncthreads();  // buf[0] is free for the next row
      continue;
    }
    const float r = rsqrtf(row_sum<W>(ss, buf[1]) / c + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 4 * (i * T + tid);
      if (KEEP) {
        uint32_t byte;
        const uint32_t b = octet_quantise(v[i], &byte);
        if (live && ch < cp) {
          __stcs(reinterpret_cast<uint32_t *>(kh.q + static_cast<size_t>(row) * cp + ch), b);
          if ((tid & 7) == 0)
            kh.scale[static_cast<size_t>(row) * (cp >> 5) + (ch >> 5)] =
                static_cast<uint8_t>(byte);
        }
      }
      if (live && ch < c)
        __stcs(reinterpret_cast<float4 *>(y + at + ch), mul4(mul4s(v[i], r), wp[i]));
    }
    if (KEEP && live && tid == 0) rstd[rows + row] = r;
  }
}

// grid (slabs, n): a block takes rows [tokens s / slabs, tokens (s + 1) / slabs)
// of one sample. part [n][slabs][c] float2: sums of dH uh and dy hh.
template <int W, int NV>
__global__ void __launch_bounds__(kThreads)
    block_norm_bwd(const float *dy, const float *dh, CkptView ku, CkptView kh,
                   const float *__restrict__ rstd, unsigned rows, unsigned tokens, int c,
                   const float *__restrict__ w_post, const float *__restrict__ gate,
                   const float *__restrict__ scale, const float *__restrict__ w_pre, float *du,
                   float *dx, float2 *__restrict__ part) {
  constexpr int T = 32 * W, R = kWarps / W;
  __shared__ float buf[2][kWarps];
  __shared__ float4 red[R > 1 ? kThreads * NV : 1][2];
  const int tid = threadIdx.x % T, grp = threadIdx.x / T, cp = (c + 31) & ~31;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 f[NV], wp[NV], su[NV], sh[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = 4 * (i * T + tid);
    const bool in = ch < c;
    f[i] = in ? ld4(w_post + ch) : zero;
    if (scale && in) f[i] = mul4(f[i], ld4(scale + ch));
    if (gate && in) f[i] = mul4(f[i], ld4(gate + static_cast<size_t>(blockIdx.y) * c + ch));
    wp[i] = w_pre && in ? ld4(w_pre + ch) : zero;
    su[i] = sh[i] = zero;
  }
  const unsigned t0 = static_cast<unsigned>(static_cast<unsigned long long>(tokens) * blockIdx.x /
                                            gridDim.x),
                 t1 = static_cast<unsigned>(static_cast<unsigned long long>(tokens) *
                                            (blockIdx.x + 1) / gridDim.x);
  for (unsigned tk = t0; tk < t1; tk += R) {
    const bool live = tk + grp < t1;
    const size_t row = static_cast<size_t>(blockIdx.y) * tokens + tk + grp;
    const size_t at = row * c;
    const float m = live ? rstd[row] : 0.f, r = live && w_pre ? rstd[rows + row] : 0.f;
    float4 g[NV], b[NV];   // dh, later dH; dy w_pre
    uint32_t qu[NV];
    float4 hh[NV];
    float uscale[NV];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 4 * (i * T + tid);
      const bool in = live && ch < c;
      g[i] = in && dh ? __ldcs(reinterpret_cast<const float4 *>(dh + at + ch)) : zero;
      qu[i] = in ? __ldcs(reinterpret_cast<const uint32_t *>(ku.q + row * cp + ch)) : 0u;
      uscale[i] = in ? ckpt_scale(__ldg(ku.scale + row * (cp >> 5) + (ch >> 5))) : 0.f;
      b[i] = hh[i] = zero;
      if (w_pre && in) {
        b[i] = __ldcs(reinterpret_cast<const float4 *>(dy + at + ch));
        hh[i] = unpack_e4m3x4(__ldcs(reinterpret_cast<const uint32_t *>(kh.q + row * cp + ch)),
                              ckpt_scale(__ldg(kh.scale + row * (cp >> 5) + (ch >> 5))));
      }
    }
    if (w_pre) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        hh[i] = mul4s(hh[i], r);
        sh[i] = fma4(b[i], hh[i], sh[i]);
        b[i] = mul4(b[i], wp[i]);
        dot += dot4(b[i], hh[i]);
      }
      const float k = row_sum<W>(dot, buf[0]) / c;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        g[i].x += r * fmaf(-hh[i].x, k, b[i].x);
        g[i].y += r * fmaf(-hh[i].y, k, b[i].y);
        g[i].z += r * fmaf(-hh[i].z, k, b[i].z);
        g[i].w += r * fmaf(-hh[i].w, k, b[i].w);
      }
    }
    dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 4 * (i * T + tid);
      if (live && ch < c) __stcs(reinterpret_cast<float4 *>(dx + at + ch), g[i]);
      hh[i] = mul4s(unpack_e4m3x4(qu[i], uscale[i]), m);  // uh
      su[i] = fma4(g[i], hh[i], su[i]);
      g[i] = mul4(g[i], f[i]);
      dot += dot4(g[i], hh[i]);
    }
    const float k = row_sum<W>(dot, buf[1]) / c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 4 * (i * T + tid);
      if (live && ch < c)
        __stcs(reinterpret_cast<float4 *>(du + at + ch),
               make_float4(m * fmaf(-hh[i].x, k, g[i].x), m * fmaf(-hh[i].y, k, g[i].y),
                           m * fmaf(-hh[i].z, k, g[i].z), m * fmaf(-hh[i].w, k, g[i].w)));
    }
    if (W > 1 && !w_pre) __syncthreads();  // one barrier per row would let buf[1] be overwritten
  }
  float4 *o = reinterpret_cast<float4 *>(
      part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * c);
  if (R > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      red[grp * T * NV + i * T + tid][0] = su[i];
      red[grp * T * NV + i * T + tid][1] = sh[i];
    }
    __syncthreads();
  }
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 4 * (i * T + tid);
      if (ch >= c) continue;
      float4 a = su[i], b = sh[i];
      for (int k = 1; k < R; ++k) {
        const float4 p = red[k * T * NV + i * T + tid][0], q = red[k * T * NV + i * T + tid][1];
        a = make_float4(a.x + p.x, a.y + p.y, a.z + p.z, a.w + p.w);
        b = make_float4(b.x + q.x, b.y + q.y, b.z + q.z, b.w + q.w);
      }
      o[ch / 2] = make_float4(a.x, b.x, a.y, b.y);
      o[ch / 2 + 1] = make_float4(a.z, b.z, a.w, b.w);
    }
  }
}

// Block b: channels [32 b, 32 b + 32); lanes are channels, warps stride over
// the slabs, samples in order.
__global__ void __launch_bounds__(1024)
    block_norm_merge(const float2 *__restrict__ part, int n, int slabs, int c,
                     const float *__restrict__ w_post, const float *__restrict__ gate,
                     const float *__restrict__ scale, float *__restrict__ dw_post,
                     float *__restrict__ dgate, float *__restrict__ dscale,
                     float *__restrict__ dw_pre) {
  __shared__ float2 red[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = 32 * blockIdx.x + lane;
  const float wpo = ch < c ? w_post[ch] : 0.f, sc = scale && ch < c ? scale[ch] : 1.f;
  float sum_s = 0.f, sum_p = 0.f;  // sum of gate S; sum of dy hh
  for (int i = 0; i < n; ++i) {
    float2 t = make_float2(0.f, 0.f);
    if (ch < c)
      for (int s = warp; s < slabs; s += 32) {
        const float2 v = part[(static_cast<size_t>(i) * slabs + s) * c + ch];
        t.x += v.x;
        t.y += v.y;
      }
    red[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && ch < c) {
      for (int w = 1; w < 32; ++w) {
        t.x += red[w][lane].x;
        t.y += red[w][lane].y;
      }
      if (dgate) dgate[static_cast<size_t>(i) * c + ch] = sc * wpo * t.x;
      sum_s = fmaf(gate ? gate[static_cast<size_t>(i) * c + ch] : 1.f, t.x, sum_s);
      sum_p += t.y;
    }
    __syncthreads();
  }
  if (warp == 0 && ch < c) {
    if (dw_post) dw_post[ch] = sc * sum_s;
    if (dscale) dscale[ch] = wpo * sum_s;
    if (dw_pre) dw_pre[ch] = sum_p;
  }
}

// Rows of up to 512 channels take a warp; wider rows two, four or eight
// warps, so that a thread never holds more than four quads of each tensor.
template <class F>
int by_width(int c, F &&f) {
  const int cp = ckpt_cp(c);
  if (cp <= 128) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  if (cp <= 256) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
  if (cp <= 512) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  if (cp <= 1024) return f(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
  if (cp <= 2048) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
}

// Samples matter only to the gate: without one all rows are one sample.
struct Shape {
  unsigned rows, tokens;
  int n;
};
Shape shape_of(const BlockNormArgs &a) {
  const unsigned rows = static_cast<unsigned>(a.n * a.tokens);
  if (!a.gate) return {rows, rows, 1};
  return {rows, static_cast<unsigned>(a.tokens), a.n};
}
int bwd_slabs(const Shape &sh) {
  const long long most = std::max(1, kBwdBlocks / sh.n);
  return static_cast<int>(std::max(1ll, std::min<long long>(most, (sh.tokens + 7) / 8)));
}

}  // namespace

int block_norm(const BlockNormArgs &a, const float *u, const float *x, float eps, float *h,
               float *y, CkptView ku, CkptView kh, float *rstd, cudaStream_t s) {
  const Shape sh = shape_of(a);
  return by_width(a.c, [&](auto w, auto nv) -> int {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value, R = kWarps / W;
    const unsigned grid = static_cast<unsigned>(
        std::min<long long>((static_cast<long long>(sh.rows) + R - 1) / R, 8ll * num_sms()));
    if (ku.q)
      block_norm_fwd<W, NV, true><<<grid, kThreads, 0, s>>>(
          u, x, sh.rows, sh.tokens, a.c, eps, a.w_post, a.gate, a.scale, a.w_pre, h, y, ku, kh,
          rstd);
    else
      block_norm_fwd<W, NV, false><<<grid, kThreads, 0, s>>>(
          u, x, sh.rows, sh.tokens, a.c, eps, a.w_post, a.gate, a.scale, a.w_pre, h, y, ku, kh,
          rstd);
    VAE_LAUNCH_CHECK();
    count_launches(1);
    return VAE_OK;
  });
}

size_t block_norm_backward_ws_bytes(const BlockNormArgs &a) {
  const Shape sh = shape_of(a);
  Carver cv(nullptr, 0);
  cv.take<float2>(static_cast<size_t>(sh.n) * bwd_slabs(sh) * a.c);
  return cv.used;
}

int block_norm_backward(const BlockNormArgs &a, const float *dy, const float *dh, CkptView ku,
                        CkptView kh, const float *rstd, float *du, float *dx, float *dw_post,
                        float *dgate, float *dscale, float *dw_pre, void *ws, cudaStream_t s) {
  const Shape sh = shape_of(a);
  const int slabs = bwd_slabs(sh);
  Carver cv(ws, ~size_t(0));
  float2 *part = cv.take<float2>(static_cast<size_t>(sh.n) * slabs * a.c);
  VAE_TRY(by_width(a.c, [&](auto w, auto nv) -> int {
    constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
    block_norm_bwd<W, NV><<<dim3(slabs, sh.n), kThreads, 0, s>>>(
        dy, dh, ku, kh, rstd, sh.rows, sh.tokens, a.c, a.w_post, a.gate, a.scale, a.w_pre, du, dx,
        part);
    VAE_LAUNCH_CHECK();
    return VAE_OK;
  }));
  block_norm_merge<<<ceil_div(a.c, 32), 1024, 0, s>>>(part, sh.n, slabs, a.c, a.w_post, a.gate,
                                                      a.scale, dw_post, dgate, dscale, dw_pre);
  VAE_LAUNCH_CHECK();
  count_launches(2);
  return VAE_OK;
}

}  // namespace vae
