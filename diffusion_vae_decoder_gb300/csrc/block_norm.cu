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
// A row stays in the registers of T threads, eight channels each in packed
// pairs, and the next row's loads are issued before a row is worked on, so each
// tensor moves once: 16 bytes per element forward (18.06 with checkpoints),
// 18.06 backward. HBM bounds both, launch latency a single token. Column sums run
// in registers over the rows of a block and meet in a fixed order. Measured:
// forward 16384 x 512 with checkpoints 25.9 us (5.9 TB/s), one token 2.7 us;
// backward 4 x 4096 x 1024 53 us, 45 of it the rows (6.7 TB/s), 1024 x 512 8.0 us.
#include <type_traits>

#include "block_norm.cuh"
#include "gn_train.cuh"
#include "ptx.cuh"

namespace vae {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBwdBlocks = 2 * 152;

// Sum over the T threads of a row. Rows wider than a warp meet in `buf` (kWarps
// floats; two calls alternate between two of them, so that one barrier of the
// row's warps per call is enough).
template <int T>
__device__ __forceinline__ float row_sum(float v, float *buf) {
#pragma unroll
  for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    named_barrier_sync(1 + warp / W, T);
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += buf[first + i];
  }
  return v;
}
__device__ __forceinline__ float total(uint64_t pair) { return lo2(pair) + hi2(pair); }
__device__ __forceinline__ uint64_t both(float v) { return pk2(v, v); }

// Eight channels of a row of weights (`other` without one); zeros past c.
__device__ __forceinline__ Oct load_or(const float *p, int ch, int c, float other) {
  if (p) return load_oct<false, false>(p + ch, c - ch);
  const float4 a = ch < c ? make_float4(other, other, other, other) : make_float4(0, 0, 0, 0);
  const float4 b = ch + 4 < c ? make_float4(other, other, other, other) : make_float4(0, 0, 0, 0);
  return oct_of(a, b);
}
__device__ __forceinline__ Oct times(const Oct &a, const Oct &b) {
  Oct o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o.v[j] = mul2(a.v[j], b.v[j]);
  return o;
}
__device__ __forceinline__ void keep_oct(CkptView k, unsigned row, int cp, int ch, bool in,
                                         const Oct &v) {
  uint32_t byte;
  const uint2 q = quad_quantise(v, &byte);
  if (!in) return;
  __stcs(reinterpret_cast<uint2 *>(k.q + static_cast<size_t>(row) * cp + ch), q);
  if ((ch & 31) == 0)
    k.scale[static_cast<size_t>(row) * (cp >> 5) + (ch >> 5)] = static_cast<uint8_t>(byte);
}

// Oct i of a row's thread `tid` starts at channel 8 (i T + tid).
template <int T, int NV, bool KEEP, bool WIDE>
__global__ void __launch_bounds__(kThreads, NV == 1 ? 3 : 2)
    block_norm_fwd(const float *u, const float *x, unsigned rows, unsigned tokens, int c,
                   float eps, const float *__restrict__ w_post, const float *__restrict__ gate,
                   const float *__restrict__ scale, const float *__restrict__ w_pre, float *h,
                   float *y, CkptView ku, CkptView kh, float *__restrict__ rstd) {
  constexpr int R = kThreads / T;  // rows of a block
  __shared__ float buf[2][kWarps];
  const int tid = threadIdx.x % T, cp = (c + 31) & ~31;
  const unsigned step = gridDim.x * R;
  unsigned row = blockIdx.x * R + threadIdx.x / T;
  Oct un[NV], xn[NV];
  auto fetch = [&](unsigned r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid), left = r < rows ? c - ch : 0;
      const size_t at = static_cast<size_t>(r) * c + ch;
      un[i] = load_oct<WIDE, true>(u + at, left);
      xn[i] = load_oct<WIDE, true>(x + at, left);
    }
  };
  fetch(row);
  Oct f[NV], gf[NV], wp[NV];  // w_post scale; times the sample's gate; w_pre
  unsigned sample = ~0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = 8 * (i * T + tid);
    f[i] = times(load_or(w_post, ch, c, 1.f), load_or(scale, ch, c, 1.f));
    gf[i] = f[i];
    wp[i] = load_or(w_pre, ch, c, 0.f);
  }
  // whole blocks leave the loop together: every lane takes part in the shuffles
  for (unsigned r0 = blockIdx.x * R; r0 < rows; r0 += step, row += step) {
    const bool live = row < rows;
    if (gate && live && row / tokens != sample) {
      sample = row / tokens;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        gf[i] = times(f[i], load_or(gate + static_cast<size_t>(sample) * c, 8 * (i * T + tid), c,
                                    1.f));
    }
    Oct v[NV], xv[NV];
    uint64_t ss = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = un[i];
      xv[i] = xn[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2(v[i].v[j], v[i].v[j], ss);
    }
    if (r0 + step < rows) fetch(row + step);
    const float m = rsqrtf(row_sum<T>(total(ss), buf[0]) / c + eps);
    ss = 0;
    const uint64_t m2 = both(m);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid);
      if (KEEP) keep_oct(ku, row, cp, ch, live && ch < cp, v[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i].v[j] = fma2(gf[i].v[j], mul2(v[i].v[j], m2), xv[i].v[j]);
        ss = fma2(v[i].v[j], v[i].v[j], ss);
      }
      store_oct<WIDE>(h + static_cast<size_t>(row) * c + ch, live ? c - ch : 0, v[i]);
    }
    if (KEEP && live && tid == 0) rstd[row] = m;
    if (!w_pre) {
      if (T > 32) named_barrier_sync(1 + threadIdx.x / T, T);  // buf[0] is free for the next row
      continue;
    }
    const float r = rsqrtf(row_sum<T>(total(ss), buf[1]) / c + eps);
    const uint64_t r2 = both(r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid);
      if (KEEP) keep_oct(kh, row, cp, ch, live && ch < cp, v[i]);
      Oct o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.v[j] = mul2(mul2(v[i].v[j], r2), wp[i].v[j]);
      store_oct<WIDE>(y + static_cast<size_t>(row) * c + ch, live ? c - ch : 0, o);
    }
    if (KEEP && live && tid == 0) rstd[rows + row] = r;
  }
}

// grid (slabs, n): a block takes every gridDim.x-th run of R rows of one sample,
// so that the grid sweeps side by side. part [n][slabs][c] float2: sums of dH uh
// and dy hh.
template <int T, int NV, bool WIDE>
__global__ void __launch_bounds__(kThreads, NV == 1 ? 2 : 1)
    block_norm_bwd(const float *dy, const float *dh, CkptView ku, CkptView kh,
                   const float *__restrict__ rstd, unsigned rows, unsigned tokens, int c,
                   const float *__restrict__ w_post, const float *__restrict__ gate,
                   const float *__restrict__ scale, const float *__restrict__ w_pre, float *du,
                   float *dx, float2 *__restrict__ part) {
  constexpr int R = kThreads / T;
  __shared__ float buf[2][kWarps];
  __shared__ float4 red[R > 1 ? kThreads * NV : 1][4];
  grid_release();
  const int tid = threadIdx.x % T, grp = threadIdx.x / T, cp = (c + 31) & ~31;
  const unsigned row0 = blockIdx.y * tokens, step = gridDim.x * R;
  Oct gn[NV], bn[NV];
  uint2 qun[NV], qhn[NV];
  uint32_t sun[NV], shn[NV];
  float mn, rn;
  auto fetch = [&](unsigned tk) {
    const bool live = tk < tokens;
    const size_t row = row0 + tk;
    mn = live ? rstd[row] : 0.f;
    rn = live && w_pre ? rstd[rows + row] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid), left = live ? c - ch : 0;
      const size_t at = row * c + ch, aq = row * cp + ch, as = row * (cp >> 5) + (ch >> 5);
      gn[i] = load_oct<WIDE, true>(dh + at, dh ? left : 0);
      bn[i] = load_oct<WIDE, true>(dy + at, w_pre ? left : 0);
      qun[i] = qhn[i] = make_uint2(0, 0);
      sun[i] = shn[i] = 0;
      if (left > 0) {
        qun[i] = __ldcs(reinterpret_cast<const uint2 *>(ku.q + aq));
        sun[i] = __ldg(ku.scale + as);
        if (w_pre) {
          qhn[i] = __ldcs(reinterpret_cast<const uint2 *>(kh.q + aq));
          shn[i] = __ldg(kh.scale + as);
        }
      }
    }
  };
  unsigned tk = blockIdx.x * R + grp;
  fetch(tk);
  Oct f[NV], wp[NV], su[NV], sh[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int ch = 8 * (i * T + tid);
    f[i] = times(load_or(w_post, ch, c, 1.f), load_or(scale, ch, c, 1.f));
    if (gate) f[i] = times(f[i], load_or(gate + static_cast<size_t>(blockIdx.y) * c, ch, c, 1.f));
    wp[i] = load_or(w_pre, ch, c, 0.f);
    su[i] = sh[i] = {{0, 0, 0, 0}};
  }
  for (unsigned t0 = blockIdx.x * R; t0 < tokens; t0 += step, tk += step) {
    const bool live = tk < tokens;
    Oct g[NV], b[NV], hh[NV], uh[NV];
    const float m = mn, r = rn;
    uint64_t dot = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      g[i] = gn[i];
      hh[i] = unpack_oct(qhn[i], ckpt_scale(shn[i]));
      uh[i] = unpack_oct(qun[i], ckpt_scale(sun[i]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        hh[i].v[j] = mul2(hh[i].v[j], both(r));
        sh[i].v[j] = fma2(bn[i].v[j], hh[i].v[j], sh[i].v[j]);
        b[i].v[j] = mul2(bn[i].v[j], wp[i].v[j]);
        dot = fma2(b[i].v[j], hh[i].v[j], dot);
      }
    }
    if (t0 + step < tokens) fetch(tk + step);
    if (w_pre) {
      const uint64_t k = both(-row_sum<T>(total(dot), buf[0]) / c);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          g[i].v[j] = fma2(both(r), fma2(hh[i].v[j], k, b[i].v[j]), g[i].v[j]);
    }
    dot = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid);
      store_oct<WIDE>(dx + static_cast<size_t>(row0 + tk) * c + ch, live ? c - ch : 0, g[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uh[i].v[j] = mul2(uh[i].v[j], both(m));
        su[i].v[j] = fma2(g[i].v[j], uh[i].v[j], su[i].v[j]);
        g[i].v[j] = mul2(g[i].v[j], f[i].v[j]);
        dot = fma2(g[i].v[j], uh[i].v[j], dot);
      }
    }
    const uint64_t k = both(-row_sum<T>(total(dot), buf[1]) / c);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid);
      Oct o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.v[j] = mul2(both(m), fma2(uh[i].v[j], k, g[i].v[j]));
      store_oct<WIDE>(du + static_cast<size_t>(row0 + tk) * c + ch, live ? c - ch : 0, o);
    }
    // (one barrier per row would let the next row overwrite buf[1])
    if (T > 32 && !w_pre) named_barrier_sync(1 + threadIdx.x / T, T);
  }
  float4 *o = reinterpret_cast<float4 *>(
      part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * c);
  if (R > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float4 *e = red[(grp * NV + i) * T + tid];
      e[0] = oct_lo(su[i]);
      e[1] = oct_hi(su[i]);
      e[2] = oct_lo(sh[i]);
      e[3] = oct_hi(sh[i]);
    }
    __syncthreads();
  }
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid);
      for (int k = 1; k < R; ++k) {
        const float4 *e = red[(k * NV + i) * T + tid];
        const Oct p = oct_of(e[0], e[1]), q = oct_of(e[2], e[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          su[i].v[j] = add2(su[i].v[j], p.v[j]);
          sh[i].v[j] = add2(sh[i].v[j], q.v[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ch + 2 * j < c)  // (c is a multiple of four)
          o[ch / 2 + j] = make_float4(lo2(su[i].v[j]), lo2(sh[i].v[j]), hi2(su[i].v[j]),
                                      hi2(sh[i].v[j]));
    }
  }
}

// Block b: channels [32 b, 32 b + 32); lanes are channels. The 32 warps split
// the samples (up to 32 at a time) and their slabs; fixed order. (Eight loads in
// flight: four take 1.3 us longer for 4 x 76 slabs, ten and more keep fetching
// instructions, 2.7 us longer.)
__global__ void __launch_bounds__(1024)
    block_norm_merge(const float2 *part, int n, int slabs, int c,
                     const float *__restrict__ w_post, const float *__restrict__ gate,
                     const float *__restrict__ scale, float *dw_post, float *dgate, float *dscale,
                     float *dw_pre) {
  __shared__ float2 red[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = 32 * blockIdx.x + lane;
  const float wpo = ch < c ? w_post[ch] : 0.f, sc = scale && ch < c ? scale[ch] : 1.f;
  const int per = 32 / min(n, 32);  // warps of a sample
  float sum_s = 0.f, sum_p = 0.f;   // sum of gate S; sum of dy hh
  grid_wait();
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + warp / per;
    float2 t = make_float2(0.f, 0.f);
    if (ch < c && i < min(n, i0 + 32)) {
      const float2 *e = part + static_cast<size_t>(i) * slabs * c + ch;
#pragma unroll 8
      for (int s = warp % per; s < slabs; s += per) {
        const float2 v = e[static_cast<size_t>(s) * c];
        t.x += v.x;
        t.y += v.y;
      }
    }
    red[warp][lane] = t;
    __syncthreads();
    const int j = i0 + warp;  // one warp per sample adds its warps' sums
    const bool mine = ch < c && j < min(n, i0 + 32);
    if (mine) {
      t = red[warp * per][lane];
#pragma unroll 4
      for (int w = 1; w < per; ++w) {
        t.x += red[warp * per + w][lane].x;
        t.y += red[warp * per + w][lane].y;
      }
      const size_t at = static_cast<size_t>(j) * c + ch;
      if (dgate) dgate[at] = sc * wpo * t.x;
      if (gate) t.x *= gate[at];
    }
    __syncthreads();
    red[warp][lane] = mine ? t : make_float2(0.f, 0.f);
    __syncthreads();
    if (warp == 0)
#pragma unroll 4
      for (int w = 0; w < min(32, n - i0); ++w) {
        sum_s += red[w][lane].x;
        sum_p += red[w][lane].y;
      }
    __syncthreads();
  }
  if (warp == 0 && ch < c) {
    if (dw_post) dw_post[ch] = sc * sum_s;
    if (dscale) dscale[ch] = wpo * sum_s;
    if (dw_pre) dw_pre[ch] = sum_p;
  }
}

// Threads of a row: the fewest of these that hold it with eight channels each,
// up to a block's 256; rows over 2048 channels take two octs a thread.
template <class F>
int by_width(int c, F &&f) {
  using std::integral_constant;
  const int octs = ckpt_cp(c) / 8;
  if (octs <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (octs <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (octs <= 64) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (octs <= 128) return f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  if (octs <= 256) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
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
int bwd_slabs(const Shape &sh, int c) {
  const int octs = ckpt_cp(c) / 8;
  const int r = octs <= 8 ? 32 : octs <= 32 ? 8 : octs <= 64 ? 4 : octs <= 128 ? 2 : 1;
  const long long most = std::max(1, kBwdBlocks / sh.n);
  return static_cast<int>(std::max(1ll, std::min<long long>(most, (sh.tokens + r - 1) / r)));
}

}  // namespace

int block_norm(const BlockNormArgs &a, const float *u, const float *x, float eps, float *h,
               float *y, CkptView ku, CkptView kh, float *rstd, cudaStream_t s) {
  const Shape sh = shape_of(a);
  const bool wide = y ? wide_ok(a.c, u, x, h, y) : wide_ok(a.c, u, x, h);
  return by_width(a.c, [&](auto t, auto nv) -> int {
    constexpr int T = decltype(t)::value, NV = decltype(nv)::value, R = kThreads / T;
    const unsigned grid = static_cast<unsigned>(std::min<long long>(
        (static_cast<long long>(sh.rows) + R - 1) / R, (NV == 1 ? 3ll : 2ll) * num_sms()));
    auto kernel = ku.q ? (wide ? block_norm_fwd<T, NV, true, true>
                               : block_norm_fwd<T, NV, true, false>)
                       : (wide ? block_norm_fwd<T, NV, false, true>
                               : block_norm_fwd<T, NV, false, false>);
    kernel<<<grid, kThreads, 0, s>>>(u, x, sh.rows, sh.tokens, a.c, eps, a.w_post, a.gate, a.scale,
                                     a.w_pre, h, y, ku, kh, rstd);
    VAE_LAUNCH_CHECK();
    count_launches(1);
    return VAE_OK;
  });
}

size_t block_norm_backward_ws_bytes(const BlockNormArgs &a) {
  const Shape sh = shape_of(a);
  Carver cv(nullptr, 0);
  cv.take<float2>(static_cast<size_t>(sh.n) * bwd_slabs(sh, a.c) * a.c);
  return cv.used;
}

int block_norm_backward(const BlockNormArgs &a, const float *dy, const float *dh, CkptView ku,
                        CkptView kh, const float *rstd, float *du, float *dx, float *dw_post,
                        float *dgate, float *dscale, float *dw_pre, void *ws, cudaStream_t s) {
  const Shape sh = shape_of(a);
  const int slabs = bwd_slabs(sh, a.c);
  Carver cv(ws, ~size_t(0));
  float2 *part = cv.take<float2>(static_cast<size_t>(sh.n) * slabs * a.c);
  const bool wide = (!dy || wide_ok(a.c, dy)) && (!dh || wide_ok(a.c, dh)) && wide_ok(a.c, du, dx);
  VAE_TRY(by_width(a.c, [&](auto t, auto nv) -> int {
    constexpr int T = decltype(t)::value, NV = decltype(nv)::value;
    auto kernel = wide ? block_norm_bwd<T, NV, true> : block_norm_bwd<T, NV, false>;
    kernel<<<dim3(slabs, sh.n), kThreads, 0, s>>>(dy, dh, ku, kh, rstd, sh.rows, sh.tokens, a.c,
                                                  a.w_post, a.gate, a.scale, a.w_pre, du, dx, part);
    VAE_LAUNCH_CHECK();
    return VAE_OK;
  }));
  VAE_CUDA_TRY(launch_after(block_norm_merge, ceil_div(a.c, 32), 1024, 0, s, part, sh.n, slabs,
                            a.c, a.w_post, a.gate, a.scale, dw_post, dgate, dscale, dw_pre));
  count_launches(2);
  return VAE_OK;
}

}  // namespace vae
