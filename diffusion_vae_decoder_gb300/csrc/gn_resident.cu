// gn_resident.cu -- GroupNorm(+SiLU) with checkpoints and its backward pass in
// one launch, for tensors whose (sample, channel slab) pieces fit the shared
// memory of a thread-block cluster.
//
// A slab is the smallest run of channels made of whole groups and whole
// 32-channel checkpoint blocks (lcm(32, c / groups); every channel when c is
// not a multiple of 32). A cluster of up to 16 blocks splits its pixels, keeps
// them in shared memory, reduces, exchanges the partial sums of the blocks
// through distributed shared memory (every block adds them in rank order, so
// all get the same bits) and writes the results: each tensor moves once, and
// the three launches with two passes over HBM of gn_train.cu become one. These
// are the launch-bound sizes: at [1, 512, 64, 64] NHWC the forward takes one
// launch instead of 9.1 + 5.1 + 10.9 us of kernels.
#include "gn_train.cuh"
#include "ptx.cuh"

namespace vae {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr size_t kMaxSmem = 227 * 1024 - 1024;

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

struct ResArgs {
  const float *x;      // forward: x; backward: dy
  CkptView kx, ky;
  int c, groups, slab;  // slab: channels, a multiple of 32
  long long spatial;
  int per;              // pixels of a block
  const float *gamma, *beta;
  int silu;
  float eps;            // forward
  float *y;             // forward
  float2 *stats;        // [n][groups] (mean, rstd): written forward, read backward
  const float *dres;    // backward
  float *dx, *dgamma, *dbeta;
  float2 *sums;
};

// Shared memory in front of the pixels: per channel of the slab an affine
// (mean, rstd, gamma, beta), per channel or group a triple, per channel a pair.
__host__ __device__ constexpr size_t head_floats(int slab) {
  return static_cast<size_t>(slab) * 9;
}
// Scratch of the block's channel sums: a pair per (pixel lane, channel).
constexpr size_t kRedFloats = kThreads * 4 * 2;

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t v;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(v));
  return v;
}

// No block leaves while another may read its shared memory.
__device__ __forceinline__ void leave() {
  if (cluster_size() > 1) cluster_sync();
}

// gamma and beta of the slab's channels into the affines (loaded while the
// pixels are on their way).
__device__ __forceinline__ void load_gamma(const ResArgs &a, float4 *aff, int ch0) {
  for (int ch = threadIdx.x; ch < a.slab; ch += kThreads) {
    const bool in = ch0 + ch < a.c;
    aff[ch].z = in ? a.gamma[ch0 + ch] : 0.f;
    aff[ch].w = in ? a.beta[ch0 + ch] : 0.f;
  }
}

// Channel sums of a block whose threads hold four channels each (quad q of the
// slab, pixel lane pl of ppi): out[channel] = (sum s, sum t). Lanes of a warp
// that share a quad first, then the rows of `red` in order.
__device__ __forceinline__ void channel_sums(float (&s)[4], float (&t)[4], int slab, int q,
                                             int pl, int ppi, float2 *red, float2 *out) {
  const int quads = slab >> 2;
  const bool folds = 32 % quads == 0;
  int rows = ppi, row = pl;
  if (folds) {
    for (int o = quads; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
        t[j] += __shfl_xor_sync(0xffffffffu, t[j], o);
      }
    rows = kWarps;
    row = threadIdx.x >> 5;
  }
  if (folds ? (threadIdx.x & 31) < quads : pl < ppi)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[row * slab + 4 * q + j] = make_float2(s[j], t[j]);
  __syncthreads();
  for (int ch = threadIdx.x; ch < slab; ch += kThreads) {
    float2 v = red[ch];
#pragma unroll 8
    for (int l = 1; l < rows; ++l) {
      v.x += red[l * slab + ch].x;
      v.y += red[l * slab + ch].y;
    }
    out[ch] = v;
  }
  __syncthreads();
}

// Merges the group triples of the cluster's blocks (lane r reads rank r's),
// writes stats and completes the slab's affines. tri: this block's [groups of
// the slab][3]; gst: a pair per group.
__device__ __forceinline__ void finish_stats(const ResArgs &a, float *tri, float2 *gst,
                                             float4 *aff, int g0, int ng, int n) {
  const uint32_t nctas = cluster_size(), rank = cluster_ctarank();
  const uint32_t lane = threadIdx.x & 31;
  const int cg = a.c / a.groups;
  if (nctas > 1)
    cluster_sync();
  else
    __syncthreads();
  for (int g = threadIdx.x >> 5; g < ng; g += kWarps) {
    Triple t{0.f, 0.f, 0.f};
    if (nctas > 1) {
      if (lane < nctas) {
        const uint32_t src = mapa_rank(tri + 3 * g, lane);
        t = Triple{ld_cluster(src), ld_cluster(src + 4), ld_cluster(src + 8)};
      }
      t = warp_merge(t);
    } else {
      t = Triple{tri[3 * g], tri[3 * g + 1], tri[3 * g + 2]};
    }
    if (lane == 0) {
      const float var = t.n > 0.f ? t.m2 / t.n : 0.f;
      const float2 st = make_float2(t.mean, 1.0f / sqrtf(var + a.eps));
      gst[g] = st;
      if (rank == 0) a.stats[n * a.groups + g0 + g] = st;
    }
  }
  __syncthreads();
  for (int ch = threadIdx.x; ch < ng * cg; ch += kThreads) {
    const float2 st = gst[ch / cg];
    aff[ch].x = st.x;
    aff[ch].y = st.y;
  }
  __syncthreads();
}

// grid (cluster, slabs, n).
__global__ void __launch_bounds__(kThreads) gn_res_fwd_nhwc(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float *tri = sm + 4 * a.slab;
  float2 *sums = reinterpret_cast<float2 *>(sm + 7 * a.slab);
  float2 *red = reinterpret_cast<float2 *>(sm + head_floats(a.slab));
  float4 *data = reinterpret_cast<float4 *>(sm + head_floats(a.slab) + kRedFloats);
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  const int quads = a.slab >> 2, ppi = kThreads / quads;
  const int q = threadIdx.x % quads, pl = threadIdx.x / quads, ch = ch0 + 4 * q;
  const bool real = ch < a.c, live = pl < ppi;
  const long long p0 = static_cast<long long>(blockIdx.x) * a.per;
  const int count = static_cast<int>(max(0ll, min(static_cast<long long>(a.per), a.spatial - p0)));
  const long long row0 = n * a.spatial + p0;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  load_gamma(a, aff, ch0);
  const float *src = a.x + row0 * a.c + ch;
  // Sums of deviations from the piece's first pixel (the block's pixel lanes
  // share it, so that they add up).
  const float4 first =
      real && count ? __ldg(reinterpret_cast<const float4 *>(src)) : zero;
  const float k[4] = {first.x, first.y, first.z, first.w};
  float s[4] = {0, 0, 0, 0}, ss[4] = {0, 0, 0, 0};
  if (live) {
    auto add = [&](float4 v) {
      const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = e[j] - k[j];
        s[j] += d;
        ss[j] = fmaf(d, d, ss[j]);
      }
    };
    int p = pl, i = threadIdx.x;
    for (; p + 7 * ppi < count; p += 8 * ppi, i += 8 * kThreads) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = real ? __ldcs(reinterpret_cast<const float4 *>(
                          src + static_cast<long long>(p + u * ppi) * a.c)) : zero;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        data[i + u * kThreads] = v[u];
        add(v[u]);
      }
    }
    for (; p < count; p += ppi, i += kThreads) {
      const float4 v =
          real ? __ldcs(reinterpret_cast<const float4 *>(src + static_cast<long long>(p) * a.c))
               : zero;
      data[i] = v;
      add(v);
    }
  }
  channel_sums(s, ss, a.slab, q, pl, ppi, red, sums);
  const int cg = a.c / a.groups, g0 = ch0 / cg;
  const int ng = min(a.slab, a.c - ch0) / cg;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = warp; g < ng; g += kWarps) {
    Triple t{0.f, 0.f, 0.f};
    for (int i = lane; i < cg; i += 32) {
      const float2 v = sums[g * cg + i];
      const float m = count ? v.x / count : 0.f;
      const float shift = count ? __ldg(a.x + row0 * a.c + ch0 + g * cg + i) : 0.f;
      t = merge(t, Triple{static_cast<float>(count), shift + m, fmaxf(v.y - v.x * m, 0.f)});
    }
    t = warp_merge(t);
    if (lane == 0) {
      tri[3 * g] = t.n;
      tri[3 * g + 1] = t.mean;
      tri[3 * g + 2] = t.m2;
    }
  }
  finish_stats(a, tri, sums, aff, g0, ng, n);
  if (live) {
    float4 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = real ? aff[4 * q + j] : zero;
    const uint32_t mask = octet_mask();
#pragma unroll 2
    for (int p = pl, i = threadIdx.x; p < count; p += ppi, i += kThreads) {
      const long long row = row0 + p;
      const float4 v = data[i];
      float4 o;
      o.x = act(fmaf((v.x - f[0].x) * f[0].y, f[0].z, f[0].w), a.silu);
      o.y = act(fmaf((v.y - f[1].x) * f[1].y, f[1].z, f[1].w), a.silu);
      o.z = act(fmaf((v.z - f[2].x) * f[2].y, f[2].z, f[2].w), a.silu);
      o.w = act(fmaf((v.w - f[3].x) * f[3].y, f[3].z, f[3].w), a.silu);
      if (real) __stcs(reinterpret_cast<float4 *>(a.y + row * a.c + ch), o);
      uint32_t byte;
      if (a.kx.q) {
        const uint32_t b = octet_quantise(v, mask, &byte);
        __stcs(reinterpret_cast<uint32_t *>(a.kx.q + row * cp + ch), b);
        if ((q & 7) == 0) a.kx.scale[row * (cp >> 5) + (ch >> 5)] = static_cast<uint8_t>(byte);
      }
      if (a.ky.q) {
        const uint32_t b = octet_quantise(o, mask, &byte);
        __stcs(reinterpret_cast<uint32_t *>(a.ky.q + row * cp + ch), b);
        if ((q & 7) == 0) a.ky.scale[row * (cp >> 5) + (ch >> 5)] = static_cast<uint8_t>(byte);
      }
    }
  }
  leave();
}

// Pixels of a channel row in shared memory: a.per rounded up to 32.
__global__ void __launch_bounds__(kThreads) gn_res_fwd_nchw(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float *tri = sm + 4 * a.slab, *chs = tri;  // channel triples first, group triples over them
  float *data = sm + head_floats(a.slab);
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  const int chans = min(a.slab, a.c - ch0), ld = (a.per + 31) & ~31;
  const long long p0 = static_cast<long long>(blockIdx.x) * a.per;
  const int count = static_cast<int>(max(0ll, min(static_cast<long long>(a.per), a.spatial - p0)));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float *src = a.x + (static_cast<long long>(n) * a.c + ch0) * a.spatial + p0;
  load_gamma(a, aff, ch0);
  // a warp per channel: load it, then its triple from shared memory, two passes
  for (int ch = warp; ch < chans; ch += kWarps) {
    const float *s = src + ch * a.spatial;
    float *d = data + ch * ld;
    float sum = 0.f;
    int p = lane;
    for (; p + 480 < count; p += 512) {
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = __ldcs(s + p + 32 * u);
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        d[p + 32 * u] = v[u];
        sum += v[u];
      }
    }
#pragma unroll 4
    for (; p < count; p += 32) {
      const float v = __ldcs(s + p);
      d[p] = v;
      sum += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float mean = count ? sum / count : 0.f;
    float m2 = 0.f, rest = 0.f;  // the mean's own rounding is corrected by the rest
    for (int i = lane; i < count; i += 32) {
      const float e = d[i] - mean;
      rest += e;
      m2 = fmaf(e, e, m2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m2 += __shfl_xor_sync(0xffffffffu, m2, o);
      rest += __shfl_xor_sync(0xffffffffu, rest, o);
    }
    if (lane == 0) {
      const float fix = count ? rest / count : 0.f;
      chs[3 * ch] = static_cast<float>(count);
      chs[3 * ch + 1] = mean + fix;
      chs[3 * ch + 2] = count ? fmaxf(m2 - rest * fix, 0.f) : 0.f;
    }
  }
  __syncthreads();
  const int cg = a.c / a.groups, g0 = ch0 / cg, ng = chans / cg;
  // (group g's triple replaces that of channel g <= g cg: merged by one thread
  // in order, after every thread has read its channels)
  Triple t[2];
  int at = 0;
  for (int g = threadIdx.x; g < ng; g += kThreads, ++at) {
    t[at] = Triple{0.f, 0.f, 0.f};
    for (int j = 0; j < cg; ++j) {
      const float *e = chs + 3 * (g * cg + j);
      t[at] = merge(t[at], Triple{e[0], e[1], e[2]});
    }
  }
  __syncthreads();
  at = 0;
  for (int g = threadIdx.x; g < ng; g += kThreads, ++at) {
    tri[3 * g] = t[at].n;
    tri[3 * g + 1] = t[at].mean;
    tri[3 * g + 2] = t[at].m2;
  }
  finish_stats(a, tri, reinterpret_cast<float2 *>(sm + 7 * a.slab), aff, g0, ng, n);
  float *ys = a.y + (static_cast<long long>(n) * a.c + ch0) * a.spatial + p0;
  const int blocks = (chans + 31) / 32;
  for (int item = threadIdx.x; item < blocks * ld; item += kThreads) {
    const int cb = item / ld, p = item - cb * ld;
    if (p >= count) continue;
    const long long row = n * a.spatial + p0 + p;
    const int in = min(32, chans - 32 * cb);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = j < in ? data[(32 * cb + j) * ld + p] : 0.f;
    if (a.kx.q) keep_row32(v, a.kx, row, cp, ch0 / 32 + cb);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < in) {
        const float4 f = aff[32 * cb + j];
        v[j] = act(fmaf((v[j] - f.x) * f.y, f.z, f.w), a.silu);
        __stcs(ys + static_cast<long long>(32 * cb + j) * a.spatial + p, v[j]);
      }
    if (a.ky.q) keep_row32(v, a.ky, row, cp, ch0 / 32 + cb);
  }
  leave();
}

// ------------------------------------------------------------- backward
// Fills the slab's affines from the saved statistics.
__device__ __forceinline__ void load_affine(const ResArgs &a, float4 *aff, int n, int ch0) {
  const int cg = a.c / a.groups;
  for (int ch = threadIdx.x; ch < a.slab; ch += kThreads) {
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ch0 + ch < a.c) {
      const float2 st = a.stats[n * a.groups + (ch0 + ch) / cg];
      f = make_float4(st.x, st.y, a.gamma[ch0 + ch], a.beta[ch0 + ch]);
    }
    aff[ch] = f;
  }
}

// mine: this block's per-channel (sum dz, sum dz xh). Adds the cluster's
// blocks' in rank order, leaves per channel (k1, k2) of its group in `km`, and
// has rank 0 write the channel sums out.
__device__ __forceinline__ void finish_sums(const ResArgs &a, const float2 *mine, float2 *km,
                                            const float4 *aff, int n, int ch0) {
  const uint32_t nctas = cluster_size(), rank = cluster_ctarank();
  const int chans = min(a.slab, a.c - ch0), cg = a.c / a.groups;
  if (nctas > 1)
    cluster_sync();
  else
    __syncthreads();
  for (int ch = threadIdx.x; ch < chans; ch += kThreads) {
    float2 t = make_float2(0.f, 0.f);
    if (nctas > 1) {
      float2 part[16];
#pragma unroll
      for (uint32_t r = 0; r < 16; ++r)
        if (r < nctas) {
          const uint32_t src = mapa_rank(mine + ch, r);
          part[r] = make_float2(ld_cluster(src), ld_cluster(src + 4));
        }
#pragma unroll
      for (uint32_t r = 0; r < 16; ++r)
        if (r < nctas) {
          t.x += part[r].x;
          t.y += part[r].y;
        }
    } else {
      t = mine[ch];
    }
    km[ch] = t;
    if (rank == 0) {
      if (a.sums) {
        a.sums[static_cast<size_t>(n) * a.c + ch0 + ch] = t;
      } else {
        if (a.dbeta) a.dbeta[ch0 + ch] = t.x;
        if (a.dgamma) a.dgamma[ch0 + ch] = t.y;
      }
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = warp; g < chans / cg; g += kWarps) {
    float u = 0.f, v = 0.f;
    for (int j = lane; j < cg; j += 32) {
      const float ga = aff[g * cg + j].z;
      u = fmaf(ga, km[g * cg + j].x, u);
      v = fmaf(ga, km[g * cg + j].y, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      u += __shfl_xor_sync(0xffffffffu, u, o);
      v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    const float f = aff[g * cg].y / (static_cast<float>(cg) * a.spatial);
    for (int j = lane; j < cg; j += 32) km[g * cg + j] = make_float2(u * f, v * f);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) gn_res_bwd_nhwc(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float2 *mine = reinterpret_cast<float2 *>(sm + 4 * a.slab);
  float2 *km = reinterpret_cast<float2 *>(sm + 7 * a.slab);
  float2 *red = reinterpret_cast<float2 *>(sm + head_floats(a.slab));
  float4 *data = reinterpret_cast<float4 *>(sm + head_floats(a.slab) + kRedFloats);
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  const int quads = a.slab >> 2, ppi = kThreads / quads;
  const int q = threadIdx.x % quads, pl = threadIdx.x / quads, ch = ch0 + 4 * q;
  const bool live = pl < ppi && ch < a.c;
  const long long p0 = static_cast<long long>(blockIdx.x) * a.per;
  const int count = static_cast<int>(max(0ll, min(static_cast<long long>(a.per), a.spatial - p0)));
  const long long row0 = n * a.spatial + p0;
  load_affine(a, aff, n, ch0);
  __syncthreads();
  float4 f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = aff[4 * q + j];
  const uint8_t *qs = a.kx.q + row0 * cp + ch, *bs = a.kx.scale + row0 * (cp >> 5) + (ch >> 5);
  auto value = [&](int p) {
    return unpack_e4m3x4(
        __ldg(reinterpret_cast<const uint32_t *>(qs + static_cast<long long>(p) * cp)),
        ckpt_scale(__ldg(bs + static_cast<long long>(p) * (cp >> 5))));
  };
  float s[4] = {0, 0, 0, 0}, t[4] = {0, 0, 0, 0};
  if (live) {
    const float *src = a.x + row0 * a.c + ch;
    auto add = [&](float4 g, float4 v, int i) {
      const float gv[4] = {g.x, g.y, g.z, g.w}, xv[4] = {v.x, v.y, v.z, v.w};
      float dz[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float xh;
        dz[j] = grad_z(gv[j], xv[j], f[j].x, f[j].y, f[j].z, f[j].w, a.silu, &xh);
        s[j] += dz[j];
        t[j] = fmaf(dz[j], xh, t[j]);
      }
      data[i] = make_float4(dz[0], dz[1], dz[2], dz[3]);
    };
    int p = pl, i = threadIdx.x;
    for (; p + 3 * ppi < count; p += 4 * ppi, i += 4 * kThreads) {
      float4 g[4], v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        g[u] = __ldcs(reinterpret_cast<const float4 *>(src + static_cast<long long>(p + u * ppi) *
                                                                 a.c));
        v[u] = value(p + u * ppi);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) add(g[u], v[u], i + u * kThreads);
    }
    for (; p < count; p += ppi, i += kThreads)
      add(__ldcs(reinterpret_cast<const float4 *>(src + static_cast<long long>(p) * a.c)),
          value(p), i);
  }
  channel_sums(s, t, a.slab, q, pl, ppi, red, mine);
  finish_sums(a, mine, km, aff, n, ch0);
  if (live) {
    float2 kk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = km[4 * q + j];
#pragma unroll 4
    for (int p = pl, i = threadIdx.x; p < count; p += ppi, i += kThreads) {
      const float4 v = value(p), z = data[i];
      const size_t at = (row0 + p) * a.c + ch;
      const float dz[4] = {z.x, z.y, z.z, z.w}, xv[4] = {v.x, v.y, v.z, v.w};
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = fmaf(f[j].y * f[j].z, dz[j],
                    -fmaf((xv[j] - f[j].x) * f[j].y, kk[j].y, kk[j].x));
      if (a.dres) {
        const float4 r = __ldcs(reinterpret_cast<const float4 *>(a.dres + at));
        o[0] += r.x;
        o[1] += r.y;
        o[2] += r.z;
        o[3] += r.w;
      }
      __stcs(reinterpret_cast<float4 *>(a.dx + at), make_float4(o[0], o[1], o[2], o[3]));
    }
  }
  leave();
}

__global__ void __launch_bounds__(kThreads, 1) gn_res_bwd_nchw(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float2 *mine = reinterpret_cast<float2 *>(sm + 4 * a.slab);
  float2 *km = reinterpret_cast<float2 *>(sm + 7 * a.slab);
  float2 *red = reinterpret_cast<float2 *>(sm + head_floats(a.slab));  // [warps][32]
  float *data = sm + head_floats(a.slab) + kRedFloats;
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  const int chans = min(a.slab, a.c - ch0), ld = (a.per + 31) & ~31;
  const long long p0 = static_cast<long long>(blockIdx.x) * a.per;
  const int count = static_cast<int>(max(0ll, min(static_cast<long long>(a.per), a.spatial - p0)));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long base = (static_cast<long long>(n) * a.c + ch0) * a.spatial + p0;
  load_affine(a, aff, n, ch0);
  __syncthreads();
  // Warps take a 32-channel block and every `stride`th run of 32 pixels of it;
  // a run's channel sums go to the lanes right away.
  const int blocks = (chans + 31) / 32;
  const int stride = blocks < kWarps ? kWarps / blocks : 1;
  for (int cb0 = 0; cb0 < blocks; cb0 += kWarps) {
    const int cb = cb0 + warp % min(blocks, kWarps), run0 = warp / min(blocks, kWarps);
    float2 sum = make_float2(0.f, 0.f);
    if (cb < blocks && run0 < stride) {
      const int in = min(32, chans - 32 * cb);
      const float *src = a.x + base + static_cast<long long>(32 * cb) * a.spatial;
      for (int p0w = 32 * run0; p0w < count; p0w += 32 * stride) {
        const int p = p0w + lane;
        const bool here = p < count;
        float v[32], g[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          g[j] = j < in && here ? __ldcs(src + j * a.spatial + p) : 0.f;
          v[j] = 0.f;
        }
        if (here) read_row32(v, a.kx, n * a.spatial + p0 + p, cp, ch0 / 32 + cb);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float4 f = aff[32 * cb + j];
          float xh;
          g[j] = grad_z(g[j], v[j], f.x, f.y, f.z, f.w, a.silu, &xh);
          if (j < in && here) data[(32 * cb + j) * ld + p] = g[j];
          v[j] = g[j] * xh;
        }
        sum.x += reduce_scatter32(g, lane);
        sum.y += reduce_scatter32(v, lane);
      }
    }
    red[warp * 32 + lane] = sum;
    __syncthreads();
    if (run0 == 0 && cb < blocks) {  // one warp per block adds its runs in order
      float2 v = sum;
      for (int r = 1; r < stride; ++r) {
        const float2 w = red[(warp + r * blocks) * 32 + lane];
        v.x += w.x;
        v.y += w.y;
      }
      mine[32 * cb + lane] = v;
    }
    __syncthreads();
  }
  finish_sums(a, mine, km, aff, n, ch0);
  for (int item = threadIdx.x; item < blocks * ld; item += kThreads) {
    const int cb = item / ld, p = item - cb * ld;
    if (p >= count) continue;
    const int in = min(32, chans - 32 * cb);
    float v[32];
    read_row32(v, a.kx, n * a.spatial + p0 + p, cp, ch0 / 32 + cb);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < in) {
        const int ch = 32 * cb + j;
        const float4 f = aff[ch];
        const float2 m = km[ch];
        const long long at = base + static_cast<long long>(ch) * a.spatial + p;
        float o = fmaf(f.y * f.z, data[ch * ld + p], -fmaf((v[j] - f.x) * f.y, m.y, m.x));
        if (a.dres) o += __ldcs(a.dres + at);
        __stcs(a.dx + at, o);
      }
  }
  leave();
}

// ------------------------------------------------------------- launch
int slab_channels(int c, int groups) {
  const int cg = c / groups;
  if (c % 32) return ckpt_cp(c);
  int l = cg;
  while (l % 32) l += cg;
  return l;  // divides c
}

// Blocks of a cluster: as few as fit, up to 8 until the launch has a block per
// SM or a block under 256 pixels; 16 (not portable) only to fit. 0: no fit.
int cluster_blocks(int n, int c, long long spatial, int slab, size_t fixed, int *per,
                   size_t *smem, bool nhwc) {
  const int pieces = n * ((c + slab - 1) / slab);
  const int quads = slab / 4, ppi = kThreads / quads;
  for (int cl = 1; cl <= 16; cl *= 2) {
    const long long pp = (spatial + cl - 1) / cl;
    if (pp > 65536) continue;
    // NHWC: slots of one pixel per pixel lane; NCHW: rows of pixels rounded up to 32
    const size_t bytes = nhwc ? static_cast<size_t>((pp + ppi - 1) / ppi) * kThreads * 16
                              : static_cast<size_t>((pp + 31) / 32 * 32) * slab * 4;
    const size_t total = fixed + bytes;
    if (total > kMaxSmem) continue;
    if (cl < 8 && static_cast<long long>(pieces) * cl < 152 && pp >= 256) continue;
    *per = static_cast<int>(pp);
    *smem = total;
    return cl;
  }
  return 0;
}

template <class Kernel>
int launch(Kernel kernel, const ResArgs &a, int cl, int n, size_t smem, cudaStream_t s) {
  VAE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kMaxSmem)));
  if (cl > 8)
    VAE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cl, (a.c + a.slab - 1) / a.slab, n);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cl;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cl > 8) {  // a cluster of 16 needs 16 SMs of one partition
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters < 1) {
      (void)cudaGetLastError();
      return VAE_EUNSUPPORTED;
    }
  }
  VAE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a));
  VAE_LAUNCH_CHECK();
  count_launches(1);
  return VAE_OK;
}

}  // namespace

int gn_ckpt_resident(const float *x, int n, int c, long long spatial, int nhwc, int groups,
                     float eps, const float *gamma, const float *beta, int silu, float *y,
                     CkptView kx, CkptView ky, float *stats, cudaStream_t s) {
  ResArgs a{};
  a.slab = slab_channels(c, groups);
  const size_t fixed = (head_floats(a.slab) + (nhwc ? kRedFloats : 0)) * sizeof(float);
  size_t smem = 0;
  const int cl = cluster_blocks(n, c, spatial, a.slab, fixed, &a.per, &smem, nhwc);
  if (!cl) return VAE_EUNSUPPORTED;
  a.x = x;
  a.kx = kx;
  a.ky = ky;
  a.c = c;
  a.groups = groups;
  a.spatial = spatial;
  a.gamma = gamma;
  a.beta = beta;
  a.silu = silu;
  a.eps = eps;
  a.y = y;
  a.stats = reinterpret_cast<float2 *>(stats);
  return nhwc ? launch(gn_res_fwd_nhwc, a, cl, n, smem, s)
              : launch(gn_res_fwd_nchw, a, cl, n, smem, s);
}

int gn_backward_resident(const float *dy, CkptView kx, const float *stats, int n, int c,
                         long long spatial, int nhwc, int groups, const float *gamma,
                         const float *beta, int silu, const float *dres, float *dx,
                         float *dgamma, float *dbeta, float2 *sums, cudaStream_t s) {
  ResArgs a{};
  a.slab = slab_channels(c, groups);
  const size_t fixed = (head_floats(a.slab) + kRedFloats) * sizeof(float);
  size_t smem = 0;
  const int cl = cluster_blocks(n, c, spatial, a.slab, fixed, &a.per, &smem, nhwc);
  if (!cl) return VAE_EUNSUPPORTED;
  a.x = dy;
  a.kx = kx;
  a.c = c;
  a.groups = groups;
  a.spatial = spatial;
  a.gamma = gamma;
  a.beta = beta;
  a.silu = silu;
  a.stats = reinterpret_cast<float2 *>(const_cast<float *>(stats));
  a.dres = dres;
  a.dx = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.sums = n > 1 ? sums : nullptr;
  return nhwc ? launch(gn_res_bwd_nhwc, a, cl, n, smem, s)
              : launch(gn_res_bwd_nchw, a, cl, n, smem, s);
}

}  // namespace vae
