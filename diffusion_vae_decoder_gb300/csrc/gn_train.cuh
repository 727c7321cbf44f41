// gn_train.cuh -- GroupNorm(+SiLU) that keeps 8-bit checkpoints, and its
// backward pass (gn_train.cu).
#pragma once
#include "ckpt.cuh"
#include "gn_stats.cuh"

namespace vae {

// Room for the partial statistics and the per-channel sums; 0 where one launch
// of clusters needs none.
size_t gn_ckpt_ws_bytes(int n, int c, long long spatial, int nhwc, int groups);
size_t gn_backward_ws_bytes(int n, int c, long long spatial, int nhwc, int groups);

// y = act(GroupNorm(x)); stats [n][groups] (mean, 1 / sqrt(var + eps));
// x_ckpt / y_ckpt: views with q == nullptr are not written.
int gn_ckpt(const float *x, int n, int c, long long spatial, int nhwc, int groups, float eps,
            const float *gamma, const float *beta, int silu, float *y, CkptView x_ckpt,
            CkptView y_ckpt, float *stats, void *ws, cudaStream_t s);

int gn_backward(const float *dy, CkptView x_ckpt, const float *stats, int n, int c,
                long long spatial, int nhwc, int groups, const float *gamma, const float *beta,
                int silu, const float *dres, float *dx, float *dgamma, float *dbeta, void *ws,
                cudaStream_t s);

// The same in one launch of thread-block clusters that hold a (sample, channel
// slab) on chip between the reduction and the elementwise pass
// (gn_resident.cu); VAE_EUNSUPPORTED, with nothing launched, for sizes that
// gn_resident does not take.
bool gn_resident(int n, int c, long long spatial, int nhwc, int groups);
int gn_ckpt_resident(const float *x, int n, int c, long long spatial, int nhwc, int groups,
                     float eps, const float *gamma, const float *beta, int silu, float *y,
                     CkptView x_ckpt, CkptView y_ckpt, float *stats, cudaStream_t s);
// sums: [n][c] float2 for (sum dz, sum dz xh), written when n > 1 (dgamma and
// dbeta are written here for n == 1).
int gn_backward_resident(const float *dy, CkptView x_ckpt, const float *stats, int n, int c,
                         long long spatial, int nhwc, int groups, const float *gamma,
                         const float *beta, int silu, const float *dres, float *dx,
                         float *dgamma, float *dbeta, float2 *sums, cudaStream_t s);

// ------------------------------------------------------------- device pieces
// Eight channels of a pixel, in packed pairs: z = (x - mean) scale + beta with
// scale = rstd gamma.
struct Affine8 {
  uint64_t nmean[4], scale[4], beta[4];
  uint64_t low[4];  // what rounding dropped of scale; forward only
};
// What rounding dropped of a b (nothing where that is not finite).
__device__ __forceinline__ float dropped(float a, float b) {
  const float p = a * b;
  return isfinite(p) ? fmaf(a, b, -p) : 0.f;
}
__device__ __forceinline__ Affine8 affine_of(const float (&mean)[8], const float (&rstd)[8],
                                             const float (&gamma)[8], const float (&beta)[8]) {
  Affine8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.nmean[j] = pk2(-mean[2 * j], -mean[2 * j + 1]);
    f.scale[j] = pk2(rstd[2 * j] * gamma[2 * j], rstd[2 * j + 1] * gamma[2 * j + 1]);
    f.beta[j] = pk2(beta[2 * j], beta[2 * j + 1]);
    f.low[j] = pk2(dropped(rstd[2 * j], gamma[2 * j]), dropped(rstd[2 * j + 1], gamma[2 * j + 1]));
  }
  return f;
}
// 1 / sqrt(v + eps) of v = m2 / n, rounded once: the error of a group's rstd is
// every output's. One Newton step from r = 1 / sqrtf, its residual 1 - v r^2 with
// the parts that rounding drops.
__device__ __forceinline__ float precise_rstd(float m2, float m2_low, float n, float eps) {
  if (!(n > 0.f)) return 1.0f / sqrtf(eps);
  const float q = m2 / n, q_low = (fmaf(-q, n, m2) + m2_low) / n;
  const float v = q + eps, v_low = (eps - (v - q)) + (q - (v - (v - q))) + q_low;
  const float r = 1.0f / sqrtf(v), t = v * r;
  const float e = fmaf(-t, r, 1.f) - (fmaf(v, r, -t) + v_low * r) * r;
  return isfinite(e) ? fmaf(0.5f * r, e, r) : r;
}
__device__ __forceinline__ uint64_t rcp2(uint64_t a) {
  float x, y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(lo2(a)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(hi2(a)));
  return pk2(x, y);
}
// 1 / (1 + e^-z), from the exp2 and reciprocal units (e^-z overflows to infinity for
// z < -88, whose reciprocal is 0). The product with log2 e is rounded: e^-z is off by
// up to |z| half-steps. That is for the backward pass alone, where SiLU's derivative,
// under |z| e^z there, is off by 0.6 half-steps of 1 at most; the precise form costs
// 3 % of it NHWC (256 channels at 256^2: 46.5 to 47.8 us) and 5 % NCHW.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z) {
  const uint64_t t = mul2(z, pk2(-1.4426950408889634f, -1.4426950408889634f));
  return rcp2(add2(pk2(ex2_approx(lo2(t)), ex2_approx(hi2(t))), pk2(1.f, 1.f)));
}
// The same with e^-z to the unit's own precision, for y and its checkpoint: with t the
// rounded product, e^-z = 2^t (1 - w), w = z + t ln 2. y is off by 3.9 half-steps at
// most for |z| < 12, where the form above measured 14.5. 1/2 - w is held to [0, 1]: for
// |z| over 1e6, where e^-z is 0 or infinity, w may be anything, and with an infinite z
// a NaN. (128 channels at 512^2: 81.3 us with either form, HBM bounds the pass.)
__device__ __forceinline__ uint64_t sigmoid2_precise(uint64_t z) {
  const uint64_t t = mul2(z, pk2(-1.4426950408889634f, -1.4426950408889634f));
  const uint64_t w = fma2(t, pk2(0.6931471805599453f, 0.6931471805599453f), z);
  const uint64_t q = add2(pk2(__saturatef(0.5f - lo2(w)), __saturatef(0.5f - hi2(w))),
                          pk2(0.5f, 0.5f));
  return rcp2(fma2(pk2(ex2_approx(lo2(t)), ex2_approx(hi2(t))), q, pk2(1.f, 1.f)));
}
template <bool SILU>
__device__ __forceinline__ Oct forward8(const Oct &x, const Affine8 &f) {
  Oct o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t d = add2(x.v[j], f.nmean[j]);
    const uint64_t z = fma2(d, f.scale[j], fma2(d, f.low[j], f.beta[j]));
    o.v[j] = SILU ? mul2(z, sigmoid2_precise(z)) : z;
  }
  return o;
}
// dz of eight elements; dev receives x - mean.
template <bool SILU>
__device__ __forceinline__ Oct grad8(const Oct &dy, const Oct &x, const Affine8 &f, Oct *dev) {
  Oct o;
  const uint64_t one = pk2(1.f, 1.f), minus = pk2(-1.f, -1.f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    dev->v[j] = add2(x.v[j], f.nmean[j]);
    o.v[j] = dy.v[j];
    if (SILU) {
      const uint64_t z = fma2(dev->v[j], f.scale[j], f.beta[j]);
      const uint64_t s = sigmoid2(z);
      o.v[j] = mul2(dy.v[j], mul2(s, fma2(z, fma2(s, minus, one), one)));
    }
  }
  return o;
}

// ------------------------------------------------------------- NCHW pieces
// 32 channels of one pixel in a thread's registers, packed pairs; a warp's lanes
// are 32 neighbouring pixels (a "run"), so that the planes are read and written
// coalesced and a checkpoint block is one thread's.
struct Row32 {
  uint64_t v[16];
};
// Per pair of channels: the affine of Affine8, and for the backward pass the
// group means of dx = scale dz + (k1 + dev k2); forward, k1 is Affine8's low.
struct PairAffine {
  uint64_t nmean, scale, beta, k1, k2;
};
__device__ __forceinline__ Row32 load_planes(const float *p, long long plane, int left) {
  Row32 r;
  float v[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = j < left ? __ldcs(p + j * plane) : 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) r.v[j] = pk2(v[2 * j], v[2 * j + 1]);
  return r;
}
__device__ __forceinline__ void store_planes(float *p, long long plane, int left,
                                             const Row32 &r) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (2 * j < left) __stcs(p + (2 * j) * plane, lo2(r.v[j]));
    if (2 * j + 1 < left) __stcs(p + (2 * j + 1) * plane, hi2(r.v[j]));
  }
}
__device__ __forceinline__ void keep_row32(const Row32 &r, CkptView k, long long row, int cp,
                                           int cb) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = max_abs3(m, lo2(r.v[j]), hi2(r.v[j]));
  const uint32_t byte = ckpt_scale_byte(__float_as_uint(m));
  const float inv = ckpt_inv_scale(byte);
  const uint64_t i2 = pk2(inv, inv);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint64_t a = mul2(r.v[2 * j], i2), b = mul2(r.v[2 * j + 1], i2);
    w[j] = pack_e4m3x4(lo2(a), hi2(a), lo2(b), hi2(b));
  }
  uint4 *dst = reinterpret_cast<uint4 *>(k.q + row * cp + 32 * cb);
  __stcs(dst, make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(dst + 1, make_uint4(w[4], w[5], w[6], w[7]));
  k.scale[row * (cp >> 5) + cb] = static_cast<uint8_t>(byte);
}
__device__ __forceinline__ Row32 read_row32(CkptView k, long long row, int cp, int cb) {
  const uint4 *src = reinterpret_cast<const uint4 *>(k.q + row * cp + 32 * cb);
  const uint4 a = __ldg(src), b = __ldg(src + 1);
  const float sc = ckpt_scale(__ldg(k.scale + row * (cp >> 5) + cb));
  const Oct o[4] = {unpack_oct(make_uint2(a.x, a.y), sc), unpack_oct(make_uint2(a.z, a.w), sc),
                    unpack_oct(make_uint2(b.x, b.y), sc), unpack_oct(make_uint2(b.z, b.w), sc)};
  Row32 r;
#pragma unroll
  for (int j = 0; j < 16; ++j) r.v[j] = o[j / 4].v[j % 4];
  return r;
}
// The affines of the 32-channel block that starts at channel ch0, zeros past c,
// by the block's first 16 threads.
__device__ __forceinline__ void load_pairs(PairAffine *out, const float2 *stats,
                                           const float *gamma, const float *beta, int ch0, int c,
                                           int cg, int t) {
  float m[2], s[2], b[2], low[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int ch = ch0 + 2 * t + h;
    const bool in = ch < c;
    const float2 st = in ? stats[ch / cg] : make_float2(0.f, 0.f);
    m[h] = -st.x;
    s[h] = in ? st.y * gamma[ch] : 0.f;
    low[h] = in ? dropped(st.y, gamma[ch]) : 0.f;
    b[h] = in ? beta[ch] : 0.f;
  }
  out[t].nmean = pk2(m[0], m[1]);
  out[t].scale = pk2(s[0], s[1]);
  out[t].beta = pk2(b[0], b[1]);
  out[t].k1 = pk2(low[0], low[1]);
}
__device__ __forceinline__ Row32 forward32(const Row32 &x, const PairAffine *f, int silu) {
  Row32 o;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint64_t d = add2(x.v[j], f[j].nmean);
    const uint64_t z = fma2(d, f[j].scale, fma2(d, f[j].k1, f[j].beta));
    o.v[j] = silu ? mul2(z, sigmoid2_precise(z)) : z;
  }
  return o;
}
// dz of 32 elements; dev receives x - mean.
__device__ __forceinline__ Row32 grad32(const Row32 &dy, const Row32 &x, const PairAffine *f,
                                        int silu, Row32 *dev) {
  Row32 o;
  const uint64_t one = pk2(1.f, 1.f), minus = pk2(-1.f, -1.f);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    dev->v[j] = add2(x.v[j], f[j].nmean);
    o.v[j] = dy.v[j];
    if (silu) {
      const uint64_t z = fma2(dev->v[j], f[j].scale, f[j].beta);
      const uint64_t s = sigmoid2(z);
      o.v[j] = mul2(dy.v[j], mul2(s, fma2(z, fma2(s, minus, one), one)));
    }
  }
  return o;
}
// dx of 32 elements from dz, in place of dz.
__device__ __forceinline__ Row32 dx32(const Row32 &dz, const Row32 &dev, const PairAffine *f) {
  Row32 o;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    o.v[j] = fma2(f[j].scale, dz.v[j], fma2(dev.v[j], f[j].k2, f[j].k1));
  return o;
}

// Sums of 32 values over a warp, value j to lane j: 31 shuffles; each step
// halves the values a lane still carries. The order is fixed.
__device__ __forceinline__ float reduce_scatter32(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < o) {
        const float keep = up ? v[j + o] : v[j], send = up ? v[j] : v[j + o];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
  }
  return v[0];
}
__device__ __forceinline__ float sum_to_lane(const Row32 &r, int lane) {
  float v[32];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    v[2 * j] = lo2(r.v[j]);
    v[2 * j + 1] = hi2(r.v[j]);
  }
  return reduce_scatter32(v, lane);
}
// (sum dz, sum dz dev) of a run, channel j to lane j.
__device__ __forceinline__ float2 run_sums(const Row32 &dz, const Row32 &dev, int lane) {
  Row32 t;
#pragma unroll
  for (int j = 0; j < 16; ++j) t.v[j] = mul2(dz.v[j], dev.v[j]);
  const float a = sum_to_lane(dz, lane);
  return make_float2(a, sum_to_lane(t, lane));
}
// The triple of a run's `count` leading lanes, channel j to lane j: deviations
// from lane 0's values.
__device__ __forceinline__ Triple run_triple(const Row32 &x, int count, int lane) {
  Row32 d, q;
  float first = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float a = __shfl_sync(0xffffffffu, lo2(x.v[j]), 0);
    const float b = __shfl_sync(0xffffffffu, hi2(x.v[j]), 0);
    if (lane == 2 * j) first = a;
    if (lane == 2 * j + 1) first = b;
    d.v[j] = lane < count ? add2(x.v[j], pk2(-a, -b)) : 0;
    q.v[j] = mul2(d.v[j], d.v[j]);
  }
  const float s = sum_to_lane(d, lane), ss = sum_to_lane(q, lane);
  if (count <= 0) return {0.f, 0.f, 0.f};
  const float m = s / count;
  return {static_cast<float>(count), first + m, fmaxf(ss - s * m, 0.f)};
}

}  // namespace vae
