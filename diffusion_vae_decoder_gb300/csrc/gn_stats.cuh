// gn_stats.cuh -- GroupNorm statistics shared by the inference kernels
// (groupnorm.cu) and the ones that keep checkpoints (gn_train.cu).
#pragma once
#include <cuda_runtime.h>

namespace vae {

constexpr int kStatThreads = 256;

// (count, mean, M2) of a set of values; merged with the parallel-variance
// combination, which works on deviations from the means (no cancellation of
// large raw sums). FP32 arithmetic: FP64 throughput on this part is low.
struct Triple {
  float n, mean, m2;
};

__device__ __forceinline__ Triple merge(Triple a, Triple b) {
  if (a.n == 0.f) return b;
  if (b.n == 0.f) return a;
  const float n = a.n + b.n;
  const float wb = __fdividef(b.n, n);
  const float d = b.mean - a.mean;
  return {n, fmaf(d, wb, a.mean), a.m2 + b.m2 + d * d * a.n * wb};
}

// Fixed-order merge of the 32 lanes' triples (xor butterfly: at each level a
// lane merges the lower-lane operand first); every lane returns the total,
// bit-identical to lane 0's.
__device__ __forceinline__ Triple warp_merge(Triple acc) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Triple other{__shfl_xor_sync(0xffffffffu, acc.n, o),
                       __shfl_xor_sync(0xffffffffu, acc.mean, o),
                       __shfl_xor_sync(0xffffffffu, acc.m2, o)};
    acc = (threadIdx.x & o) ? merge(other, acc) : merge(acc, other);
  }
  return acc;
}

// NHWC: x[n][spatial][c]. Block `blk` of `nblk` of sample n reduces its slab
// of pixels into partials [n][groups][nblk] (count, mean, M2); sm holds
// 3 * kStatThreads * 4 floats.
template <class P>
__device__ __forceinline__ void stats_slab_nhwc(const float *__restrict__ x, int c,
                                                long long spatial, int groups, int nblk, int n,
                                                int blk, float *sm, P *__restrict__ part) {
  const int tpp = c >> 2;
  const int ppi = kStatThreads / tpp;
  const int tid = threadIdx.x;
  const int lc = tid % tpp, pl = tid / tpp;
  const long long p0 = spatial * blk / nblk, p1 = spatial * (blk + 1) / nblk;
  float k[4] = {0, 0, 0, 0}, s[4] = {0, 0, 0, 0}, ss[4] = {0, 0, 0, 0};
  int cnt = 0;
  if (pl < ppi) {
    const float *base = x + (static_cast<long long>(n) * spatial) * c + 4 * lc;
    long long pix = p0 + pl;
    if (pix < p1) {  // shift every sum by the first value this thread sees
      const float4 v = __ldg(reinterpret_cast<const float4 *>(base + pix * c));
      k[0] = v.x;
      k[1] = v.y;
      k[2] = v.z;
      k[3] = v.w;
    }
    // four independent loads in flight per iteration
    for (; pix + 3 * ppi < p1; pix += 4 * ppi) {
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = __ldg(reinterpret_cast<const float4 *>(base + (pix + u * ppi) * c));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float a[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float d = a[j] - k[j];
          s[j] += d;
          ss[j] = fmaf(d, d, ss[j]);
        }
      }
      cnt += 4;
    }
    for (; pix < p1; pix += ppi) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(base + pix * c));
      const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = a[j] - k[j];
        s[j] += d;
        ss[j] = fmaf(d, d, ss[j]);
      }
      ++cnt;
    }
    float *e = sm + (static_cast<long long>(pl) * c + 4 * lc) * 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float mean_d = cnt ? s[j] / cnt : 0.f;
      e[3 * j + 0] = static_cast<float>(cnt);
      e[3 * j + 1] = k[j] + mean_d;
      e[3 * j + 2] = cnt ? fmaxf(ss[j] - s[j] * mean_d, 0.f) : 0.f;
    }
  }
  __syncthreads();
  const int cg = c / groups;
  for (int g = tid; g < groups; g += kStatThreads) {
    Triple acc{0.f, 0.f, 0.f};
    for (int l = 0; l < ppi; ++l)
      for (int ch = g * cg; ch < (g + 1) * cg; ++ch) {
        const float *e = sm + (static_cast<long long>(l) * c + ch) * 3;
        acc = merge(acc, Triple{e[0], e[1], e[2]});
      }
    P *o = part + ((static_cast<long long>(n) * groups + g) * nblk + blk) * 3;
    o[0] = acc.n;
    o[1] = acc.mean;
    o[2] = acc.m2;
  }
}

// NCHW: group (n, g) is the contiguous segment of cg * spatial floats.
// Block `blk` of `nblk` of segment ng reduces its share into partials
// [n * groups][nblk] (count, mean, M2).
template <class P>
__device__ __forceinline__ void stats_segment_nchw(const float *__restrict__ x, int c,
                                                   long long spatial, int groups, int nblk,
                                                   int ng, int blk, float (*red)[3],
                                                   P *__restrict__ part) {
  const int cg = c / groups;
  const long long seg = static_cast<long long>(cg) * spatial;
  const float *base = x + static_cast<long long>(ng) * seg;
  const long long e0 = seg * blk / nblk, e1 = seg * (blk + 1) / nblk;
  float k = 0.f, s = 0.f, ss = 0.f;
  int cnt = 0;
  for (long long i = e0 + threadIdx.x; i < e1; i += kStatThreads) {
    const float v = __ldg(base + i);
    if (cnt == 0) k = v;
    const float d = v - k;
    s += d;
    ss = fmaf(d, d, ss);
    ++cnt;
  }
  const float md = cnt ? s / cnt : 0.f;
  red[threadIdx.x][0] = cnt;
  red[threadIdx.x][1] = k + md;
  red[threadIdx.x][2] = cnt ? fmaxf(ss - s * md, 0.f) : 0.f;
  __syncthreads();
  for (int w = kStatThreads / 2; w > 0; w >>= 1) {
    if (threadIdx.x < w) {
      const Triple a{red[threadIdx.x][0], red[threadIdx.x][1], red[threadIdx.x][2]};
      const Triple b{red[threadIdx.x + w][0], red[threadIdx.x + w][1], red[threadIdx.x + w][2]};
      const Triple r = merge(a, b);
      red[threadIdx.x][0] = r.n;
      red[threadIdx.x][1] = r.mean;
      red[threadIdx.x][2] = r.m2;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    P *o = part + (static_cast<long long>(ng) * nblk + blk) * 3;
    o[0] = red[0][0];
    o[1] = red[0][1];
    o[2] = red[0][2];
  }
}

// SiLU with the fast exponential and division: their few-ulp error sits far
// below the TF32 rounding applied to the result before the next conv.
// (v < -88: exp overflows to inf and the quotient is -0, SiLU's limit.)
__device__ __forceinline__ float act(float v, int silu) {
  return silu ? __fdividef(v, 1.0f + __expf(-v)) : v;
}

}  // namespace vae
