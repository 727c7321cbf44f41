// gn_resident.cu -- GroupNorm(+SiLU) with checkpoints and its backward pass in
// one launch, for tensors whose (sample, channel slab) pieces fit the shared
// memory of a thread-block cluster.
//
// A slab is the smallest run of channels made of whole groups and whole
// 32-channel checkpoint blocks (lcm(32, c / groups); every channel when c is
// not a multiple of 32). A cluster of up to 8 blocks splits its pixels, keeps
// them in shared memory, reduces, exchanges the partial sums of the blocks
// through distributed shared memory (every block adds them in rank order, so
// all get the same bits) and writes the results: each tensor moves once, and
// the three launches with two passes over HBM of gn_train.cu become one. These
// are the launch-bound sizes: at [1, 512, 64, 64] NHWC the forward takes 13 us of the
// GPU instead of 15, the backward 12 instead of 18, and a call of the binding in a
// bare loop on the same tensors, which the host bounds, 24 and 17 instead of 31 and
// 25. On the GPU it is one block's chain of launch, load, two cluster barriers and
// store.
#include "gn_train.cuh"
#include "ptx.cuh"

namespace vae {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr size_t kMaxHeld = 64 * 1024;  // of a block's pixels
constexpr int kMaxCluster = 8;

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
constexpr size_t kRedFloats = kThreads * 8 * 2;

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
// pixels are on their way). Behind channel c everything is zero: finish_stats
// completes real channels only, and the padding's share of a checkpoint block
// must not come from what an earlier kernel left here.
__device__ __forceinline__ void load_gamma(const ResArgs &a, float4 *aff, int ch0) {
  for (int ch = threadIdx.x; ch < a.slab; ch += kThreads) {
    const bool in = ch0 + ch < a.c;
    aff[ch] = make_float4(0.f, 0.f, in ? a.gamma[ch0 + ch] : 0.f, in ? a.beta[ch0 + ch] : 0.f);
  }
}

// Channel sums of a block whose threads hold eight channels each (oct o of the
// slab, pixel lane pl of ppi): out[channel] = (sum s, sum t). Lanes of a warp
// that share an oct first, then the rows of `red` in order.
__device__ __forceinline__ void channel_sums(uint64_t (&s)[4], uint64_t (&t)[4], int slab, int o,
                                             int pl, int ppi, float2 *red, float2 *out) {
  const int octs = slab >> 3;
  const bool folds = 32 % octs == 0;
  int rows = ppi, row = pl;
  if (folds) {
    for (int d = octs; d < 32; d <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = add2(s[j], __shfl_xor_sync(0xffffffffu, s[j], d));
        t[j] = add2(t[j], __shfl_xor_sync(0xffffffffu, t[j], d));
      }
    rows = kWarps;
    row = threadIdx.x >> 5;
  }
  if (folds ? (threadIdx.x & 31) < octs : pl < ppi)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[row * slab + 8 * o + 2 * j] = make_float2(lo2(s[j]), lo2(t[j]));
      red[row * slab + 8 * o + 2 * j + 1] = make_float2(hi2(s[j]), hi2(t[j]));
    }
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

// The packed affine of eight channels.
__device__ __forceinline__ Affine8 affine8(const float4 *aff) {
  float m[8], r[8], ga[8], be[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 a = aff[j];
    m[j] = a.x;
    r[j] = a.y;
    ga[j] = a.z;
    be[j] = a.w;
  }
  return affine_of(m, r, ga, be);
}

// NCHW: room for the slab's channel pairs, or before them for a triple per warp
// and lane.
__host__ __device__ constexpr size_t pair_floats(int slab) {
  const size_t a = static_cast<size_t>(slab) / 2 * (sizeof(PairAffine) / 4);
  const size_t b = kWarps * 32 * 3;
  return a > b ? a : b;
}
__device__ __forceinline__ void pair_up(const ResArgs &a, const float4 *aff, PairAffine *pairs,
                                        int chans) {
  for (int t = threadIdx.x; t < a.slab / 2; t += kThreads) {
    float4 f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      f[h] = 2 * t + h < chans ? aff[2 * t + h] : make_float4(0.f, 0.f, 0.f, 0.f);
    pairs[t].nmean = pk2(-f[0].x, -f[1].x);
    pairs[t].scale = pk2(f[0].y * f[0].z, f[1].y * f[1].z);
    pairs[t].beta = pk2(f[0].w, f[1].w);
    pairs[t].k1 = pk2(dropped(f[0].y, f[0].z), dropped(f[1].y, f[1].z));
  }
  __syncthreads();
}

// Where a thread stands in a block's piece of an NHWC tensor.
struct Piece {
  int o, pl, ppi, ch, left, count;
  long long row0;
  __device__ Piece(const ResArgs &a) {
    const int octs = a.slab >> 3, ch0 = blockIdx.y * a.slab;
    ppi = kThreads / octs;
    o = threadIdx.x % octs;
    pl = threadIdx.x / octs;
    ch = ch0 + 8 * o;
    left = pl < ppi ? a.c - ch : 0;
    const long long p0 = static_cast<long long>(blockIdx.x) * a.per;
    count = static_cast<int>(max(0ll, min(static_cast<long long>(a.per), a.spatial - p0)));
    row0 = blockIdx.z * a.spatial + p0;
  }
};

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
      const float2 st = make_float2(t.mean, precise_rstd(t.m2, 0.f, t.n, a.eps));
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
template <bool SILU, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) gn_res_fwd_nhwc(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float *tri = sm + 4 * a.slab;
  float2 *sums = reinterpret_cast<float2 *>(sm + 7 * a.slab);
  float2 *red = reinterpret_cast<float2 *>(sm + head_floats(a.slab));
  float4 *data = reinterpret_cast<float4 *>(sm + head_floats(a.slab) + kRedFloats);
  const Piece pc(a);
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  load_gamma(a, aff, ch0);
  const float *src = a.x + pc.row0 * a.c + pc.ch;
  // Sums of deviations from the piece's first pixel (the block's pixel lanes
  // share it, so that they add up).
  Oct k = load_oct<WIDE, true>(src, pc.count ? pc.left : 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) k.v[j] = mul2(k.v[j], pk2(-1.f, -1.f));
  uint64_t s[4] = {0, 0, 0, 0}, ss[4] = {0, 0, 0, 0};
  if (pc.pl < pc.ppi) {
    constexpr int U = 4;
    for (int p = pc.pl, i = threadIdx.x; p < pc.count; p += U * pc.ppi, i += 2 * U * kThreads) {
      Oct v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = load_oct<WIDE, true>(src + static_cast<long long>(p + u * pc.ppi) * a.c,
                        p + u * pc.ppi < pc.count ? pc.left : 0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p + u * pc.ppi >= pc.count) break;
        data[i + 2 * u * kThreads] = oct_lo(v[u]);
        data[i + (2 * u + 1) * kThreads] = oct_hi(v[u]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t d = add2(v[u].v[j], k.v[j]);
          s[j] = add2(s[j], d);
          ss[j] = fma2(d, d, ss[j]);
        }
      }
    }
  }
  channel_sums(s, ss, a.slab, pc.o, pc.pl, pc.ppi, red, sums);
  const int cg = a.c / a.groups, g0 = ch0 / cg;
  const int ng = min(a.slab, a.c - ch0) / cg;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = warp; g < ng; g += kWarps) {
    Triple t{0.f, 0.f, 0.f};
    for (int i = lane; i < cg; i += 32) {
      const float2 v = sums[g * cg + i];
      const float m = pc.count ? v.x / pc.count : 0.f;
      const float shift = pc.count ? a.x[pc.row0 * a.c + ch0 + g * cg + i] : 0.f;
      t = merge(t, Triple{static_cast<float>(pc.count), shift + m, fmaxf(v.y - v.x * m, 0.f)});
    }
    t = warp_merge(t);
    if (lane == 0) {
      tri[3 * g] = t.n;
      tri[3 * g + 1] = t.mean;
      tri[3 * g + 2] = t.m2;
    }
  }
  finish_stats(a, tri, sums, aff, g0, ng, n);
  const Affine8 f = affine8(aff + 8 * pc.o);
#pragma unroll 2
  for (int p0 = 0, i = threadIdx.x; p0 < pc.count; p0 += pc.ppi, i += 2 * kThreads) {
    const long long row = pc.row0 + p0 + pc.pl;
    const bool in = p0 + pc.pl < pc.count && pc.pl < pc.ppi;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const Oct v = oct_of(in ? data[i] : zero, in ? data[i + kThreads] : zero);
    const Oct o = forward8<SILU>(v, f);
    store_oct<WIDE>(a.y + row * a.c + pc.ch, in ? pc.left : 0, o);
    uint32_t byte;
    if (a.kx.q) {
      const uint2 q = quad_quantise(v, &byte);
      if (in) {
        __stcs(reinterpret_cast<uint2 *>(a.kx.q + row * cp + pc.ch), q);
        if ((pc.o & 3) == 0)
          a.kx.scale[row * (cp >> 5) + (pc.ch >> 5)] = static_cast<uint8_t>(byte);
      }
    }
    if (a.ky.q) {
      const uint2 q = quad_quantise(o, &byte);
      if (in) {
        __stcs(reinterpret_cast<uint2 *>(a.ky.q + row * cp + pc.ch), q);
        if ((pc.o & 3) == 0)
          a.ky.scale[row * (cp >> 5) + (pc.ch >> 5)] = static_cast<uint8_t>(byte);
      }
    }
  }
  leave();
}

// Warps of an NCHW block take a 32-channel block of the slab and every
// `stride`th run of 32 pixels of it; more blocks than warps go in rounds.
struct Runs {
  int blocks, width, stride, first;
  __device__ Runs(int chans) {
    const int warp = threadIdx.x >> 5;
    blocks = (chans + 31) / 32;
    width = min(blocks, kWarps);
    stride = kWarps / width;
    first = warp / width;  // `stride` and above: idle
  }
  __device__ int block(int round) const { return round + (threadIdx.x >> 5) % width; }
};

// Shared memory of a block: per run of 32 pixels the channels of the slab, 32
// pixels each ([run][channel][32]).
__global__ void __launch_bounds__(kThreads, 2) gn_res_fwd_nchw(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float *tri = sm + 4 * a.slab, *chs = tri;  // channel triples, then group triples over them
  PairAffine *pairs = reinterpret_cast<PairAffine *>(sm + head_floats(a.slab));
  Triple *red = reinterpret_cast<Triple *>(pairs);  // [warps][32], before the pairs
  float *data = sm + head_floats(a.slab) + pair_floats(a.slab);
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  const int chans = min(a.slab, a.c - ch0), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long p0 = static_cast<long long>(blockIdx.x) * a.per;
  const int count = static_cast<int>(max(0ll, min(static_cast<long long>(a.per), a.spatial - p0)));
  const long long base = (static_cast<long long>(n) * a.c + ch0) * a.spatial + p0;
  load_gamma(a, aff, ch0);
  const Runs rn(chans);
  for (int round = 0; round < rn.blocks; round += rn.width) {
    const int cb = rn.block(round);
    Triple t{0.f, 0.f, 0.f};
    if (cb < rn.blocks && rn.first < rn.stride)
      for (int r = rn.first; 32 * r < count; r += rn.stride) {
        const int p = 32 * r + lane, left = chans - 32 * cb;
        const Row32 v = load_planes(a.x + base + static_cast<long long>(32 * cb) * a.spatial + p,
                                    a.spatial, p < count ? left : 0);
        float *d = data + (static_cast<size_t>(r) * a.slab + 32 * cb) * 32 + lane;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          d[64 * j] = lo2(v.v[j]);
          d[64 * j + 32] = hi2(v.v[j]);
        }
        t = merge(t, run_triple(v, min(32, count - 32 * r), lane));
      }
    red[warp * 32 + lane] = t;
    __syncthreads();
    if (rn.first == 0 && cb < rn.blocks) {
      for (int r = 1; r < rn.stride; ++r) t = merge(t, red[(warp + r * rn.width) * 32 + lane]);
      float *e = chs + 3 * (32 * cb + lane);
      e[0] = t.n;
      e[1] = t.mean;
      e[2] = t.m2;
    }
    __syncthreads();
  }
  const int cg = a.c / a.groups, g0 = ch0 / cg, ng = chans / cg;
  // (group g's triple replaces that of channel g <= g cg: merged by one thread
  // in order, after every thread has read its channels)
  Triple t[1024 / kThreads];
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
  pair_up(a, aff, pairs, chans);
  for (int round = 0; round < rn.blocks; round += rn.width) {
    const int cb = rn.block(round);
    if (cb >= rn.blocks || rn.first >= rn.stride) continue;
    const int left = chans - 32 * cb;
    for (int r = rn.first; 32 * r < count; r += rn.stride) {
      const int p = 32 * r + lane;
      if (p >= count) continue;
      const float *d = data + (static_cast<size_t>(r) * a.slab + 32 * cb) * 32 + lane;
      Row32 v;
#pragma unroll
      for (int j = 0; j < 16; ++j) v.v[j] = pk2(d[64 * j], d[64 * j + 32]);
      const long long row = n * a.spatial + p0 + p;
      if (a.kx.q) keep_row32(v, a.kx, row, cp, ch0 / 32 + cb);
      const Row32 o = forward32(v, pairs + 16 * cb, a.silu);
      store_planes(a.y + base + static_cast<long long>(32 * cb) * a.spatial + p, a.spatial, left,
                   o);
      if (a.ky.q) keep_row32(o, a.ky, row, cp, ch0 / 32 + cb);
    }
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
      float2 part[kMaxCluster];
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r)
        if (r < nctas) {
          const uint32_t src = mapa_rank(mine + ch, r);
          part[r] = make_float2(ld_cluster(src), ld_cluster(src + 4));
        }
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r)
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

template <bool SILU, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) gn_res_bwd_nhwc(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float2 *mine = reinterpret_cast<float2 *>(sm + 4 * a.slab);
  float2 *km = reinterpret_cast<float2 *>(sm + 7 * a.slab);
  float2 *red = reinterpret_cast<float2 *>(sm + head_floats(a.slab));
  float4 *data = reinterpret_cast<float4 *>(sm + head_floats(a.slab) + kRedFloats);
  const Piece pc(a);
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  load_affine(a, aff, n, ch0);
  __syncthreads();
  const Affine8 f = affine8(aff + 8 * pc.o);
  const uint8_t *qs = a.kx.q + pc.row0 * cp + pc.ch,
                *bs = a.kx.scale + pc.row0 * (cp >> 5) + (pc.ch >> 5);
  uint64_t s[4] = {0, 0, 0, 0}, t[4] = {0, 0, 0, 0};
  if (pc.pl < pc.ppi) {
    const float *src = a.x + pc.row0 * a.c + pc.ch;
    constexpr int U = 2;
    for (int p = pc.pl, i = threadIdx.x; p < pc.count; p += U * pc.ppi, i += 2 * U * kThreads) {
      Oct g[U];
      uint2 q[U];
      uint32_t sb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long pp = p + u * pc.ppi;
        const bool in = pp < pc.count;
        g[u] = load_oct<WIDE, true>(src + pp * a.c, in ? pc.left : 0);
        q[u] = in ? __ldg(reinterpret_cast<const uint2 *>(qs + pp * cp)) : make_uint2(0, 0);
        sb[u] = in ? __ldg(bs + pp * (cp >> 5)) : 0u;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p + u * pc.ppi >= pc.count) break;
        Oct dev;
        const Oct dz = grad8<SILU>(g[u], unpack_oct(q[u], ckpt_scale(sb[u])), f, &dev);
        data[i + 2 * u * kThreads] = oct_lo(dz);
        data[i + (2 * u + 1) * kThreads] = oct_hi(dz);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[j] = add2(s[j], dz.v[j]);
          t[j] = fma2(dz.v[j], dev.v[j], t[j]);
        }
      }
    }
  }
  float rstd[8];  // dev rstd = xh
#pragma unroll
  for (int j = 0; j < 8; ++j) rstd[j] = aff[8 * pc.o + j].y;
#pragma unroll
  for (int j = 0; j < 4; ++j) t[j] = mul2(t[j], pk2(rstd[2 * j], rstd[2 * j + 1]));
  channel_sums(s, t, a.slab, pc.o, pc.pl, pc.ppi, red, mine);
  finish_sums(a, mine, km, aff, n, ch0);
  if (pc.left > 0) {
    uint64_t k1[4], k2[4];  // dx = scale dz + (k1 + dev k2), both means negated
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = km[8 * pc.o + 2 * j], v = km[8 * pc.o + 2 * j + 1];
      const bool in = 2 * j < pc.left;  // (left is a multiple of four)
      k1[j] = in ? pk2(-u.x, -v.x) : 0;
      k2[j] = in ? pk2(-u.y * rstd[2 * j], -v.y * rstd[2 * j + 1]) : 0;
    }
#pragma unroll 2
    for (int p = pc.pl, i = threadIdx.x; p < pc.count; p += pc.ppi, i += 2 * kThreads) {
      const Oct x = unpack_oct(
          __ldg(reinterpret_cast<const uint2 *>(qs + static_cast<long long>(p) * cp)),
          ckpt_scale(__ldg(bs + static_cast<long long>(p) * (cp >> 5))));
      const Oct dz = oct_of(data[i], data[i + kThreads]);
      const size_t at = (pc.row0 + p) * a.c + pc.ch;
      Oct o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o.v[j] = fma2(f.scale[j], dz.v[j], fma2(add2(x.v[j], f.nmean[j]), k2[j], k1[j]));
      if (a.dres) {
        const Oct r = load_oct<WIDE, true>(a.dres + at, pc.left);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = add2(o.v[j], r.v[j]);
      }
      store_oct<WIDE>(a.dx + at, pc.left, o);
    }
  }
  leave();
}

__global__ void __launch_bounds__(kThreads, 2) gn_res_bwd_nchw(const ResArgs a) {
  extern __shared__ __align__(16) float sm[];
  float4 *aff = reinterpret_cast<float4 *>(sm);
  float2 *mine = reinterpret_cast<float2 *>(sm + 4 * a.slab);
  float2 *km = reinterpret_cast<float2 *>(sm + 7 * a.slab);
  PairAffine *pairs = reinterpret_cast<PairAffine *>(sm + head_floats(a.slab));
  float2 *red = reinterpret_cast<float2 *>(sm + head_floats(a.slab) + pair_floats(a.slab));
  float *data = sm + head_floats(a.slab) + pair_floats(a.slab) + kWarps * 32 * 2;
  const int n = blockIdx.z, ch0 = blockIdx.y * a.slab, cp = (a.c + 31) & ~31;
  const int chans = min(a.slab, a.c - ch0), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long p0 = static_cast<long long>(blockIdx.x) * a.per;
  const int count = static_cast<int>(max(0ll, min(static_cast<long long>(a.per), a.spatial - p0)));
  const long long base = (static_cast<long long>(n) * a.c + ch0) * a.spatial + p0;
  load_affine(a, aff, n, ch0);
  __syncthreads();
  pair_up(a, aff, pairs, chans);
  const Runs rn(chans);
  for (int round = 0; round < rn.blocks; round += rn.width) {
    const int cb = rn.block(round);
    float2 sum = make_float2(0.f, 0.f);
    if (cb < rn.blocks && rn.first < rn.stride)
      for (int r = rn.first; 32 * r < count; r += rn.stride) {
        const int p = 32 * r + lane;
        const bool here = p < count;  // (elsewhere dy = 0, which adds nothing)
        const Row32 g =
            load_planes(a.x + base + static_cast<long long>(32 * cb) * a.spatial + p, a.spatial,
                        here ? chans - 32 * cb : 0);
        const Row32 v =
            read_row32(a.kx, n * a.spatial + p0 + (here ? p : 0), cp, ch0 / 32 + cb);
        Row32 dev;
        const Row32 dz = grad32(g, v, pairs + 16 * cb, a.silu, &dev);
        float *d = data + (static_cast<size_t>(r) * a.slab + 32 * cb) * 32 + lane;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          d[64 * j] = lo2(dz.v[j]);
          d[64 * j + 32] = hi2(dz.v[j]);
        }
        const float2 t = run_sums(dz, dev, lane);
        sum.x += t.x;
        sum.y += t.y;
      }
    red[warp * 32 + lane] = sum;
    __syncthreads();
    if (rn.first == 0 && cb < rn.blocks) {  // one warp per block adds its runs in order
      for (int r = 1; r < rn.stride; ++r) {
        const float2 w = red[(warp + r * rn.width) * 32 + lane];
        sum.x += w.x;
        sum.y += w.y;
      }
      sum.y *= aff[32 * cb + lane].y;  // dev rstd = xh
      mine[32 * cb + lane] = sum;
    }
    __syncthreads();
  }
  finish_sums(a, mine, km, aff, n, ch0);
  for (int t = threadIdx.x; t < a.slab / 2; t += kThreads) {
    float2 m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ch = 2 * t + h;
      m[h] = ch < chans ? make_float2(-km[ch].x, -km[ch].y * aff[ch].y) : make_float2(0.f, 0.f);
    }
    pairs[t].k1 = pk2(m[0].x, m[1].x);
    pairs[t].k2 = pk2(m[0].y, m[1].y);
  }
  __syncthreads();
  for (int round = 0; round < rn.blocks; round += rn.width) {
    const int cb = rn.block(round);
    if (cb >= rn.blocks || rn.first >= rn.stride) continue;
    const int left = chans - 32 * cb;
    for (int r = rn.first; 32 * r < count; r += rn.stride) {
      const int p = 32 * r + lane;
      if (p >= count) continue;
      const float *d = data + (static_cast<size_t>(r) * a.slab + 32 * cb) * 32 + lane;
      Row32 dz, dev = read_row32(a.kx, n * a.spatial + p0 + p, cp, ch0 / 32 + cb);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        dz.v[j] = pk2(d[64 * j], d[64 * j + 32]);
        dev.v[j] = add2(dev.v[j], pairs[16 * cb + j].nmean);
      }
      Row32 o = dx32(dz, dev, pairs + 16 * cb);
      const long long at = base + static_cast<long long>(32 * cb) * a.spatial + p;
      if (a.dres) {
        const Row32 res = load_planes(a.dres + at, a.spatial, left);
#pragma unroll
        for (int j = 0; j < 16; ++j) o.v[j] = add2(o.v[j], res.v[j]);
      }
      store_planes(a.dx + at, a.spatial, left, o);
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

// Shared memory besides the pixels.
size_t fixed_bytes(int slab, bool nhwc, bool backward) {
  const size_t red = nhwc ? kRedFloats
                          : pair_floats(slab) + (backward ? kWarps * 32 * 2 : 0);
  return (head_floats(slab) + red) * sizeof(float);
}

constexpr size_t kMaxSmem =
    kMaxHeld + (head_floats(1024) + std::max(kRedFloats, pair_floats(1024) + kWarps * 32 * 2)) * 4;
static_assert(kMaxSmem <= 227 * 1024, "the widest slab (c <= 1024) fits an SM");

// Blocks of a cluster; 0: the three launches of gn_train.cu. As few blocks as
// hold the pixels, up to 8 until the launch has a block per SM or a block under 256
// (NHWC) or 128 pixels.
//
// A block takes about 8 us and 0.7 (forward; backward 0.5) per 1024 numbers that it
// holds, three launches 8 to 14 us in all, but 10 us more of the host's time when
// they are called one by one. Measured, GPU (calls in a loop), us:
//   numbers a block          one launch           three launches
//   4096  (1, 64, 1024)      10.5 (23)  7.8 (17)  8.8 (31)  12.5 (25)  NCHW
//   16384 (1, 256, 4096)     11.1 (24)  9.4 (18)  12.3 (31) 15.0 (25)  NHWC
//   16384 (1, 256, 4096)     16.0 (23)  12.7 (17) 10.9 (31) 13.1 (25)  NCHW
//   23500 (2, 96, 1961)                 21.0 (27)           12.2 (26)  NCHW
//   49152 (1, 96, 4096)      41.3 (43)  33.3 (35) 8.7 (33)  12.5 (26)  NCHW
//   twice 16384 (4, 512, 4096) 72 (73)  58 (60)   30 (33)   54 (58)    NCHW
// so one launch up to 16384 numbers, counting the rounds that the SMs take.
int cluster_blocks(int n, int c, long long spatial, int slab, int *per, size_t *bytes,
                   bool nhwc) {
  const int pieces = n * ((c + slab - 1) / slab);
  const int ppi = kThreads / (slab / 8);
  for (int cl = 1; cl <= kMaxCluster; cl *= 2) {
    const long long pp = (spatial + cl - 1) / cl;
    if (pp > 65536) continue;
    // NHWC: slots of one pixel per pixel lane; NCHW: rows of pixels rounded up to 32
    const size_t held = nhwc ? static_cast<size_t>((pp + ppi - 1) / ppi) * kThreads * 32
                             : static_cast<size_t>((pp + 31) / 32 * 32) * slab * 4;
    const long long blocks = static_cast<long long>(pieces) * cl, rounds = (blocks + 255) / 256;
    if (held * rounds > kMaxHeld) continue;
    if (cl < kMaxCluster && blocks < 152 && pp >= (nhwc ? 256 : 128)) continue;
    *per = static_cast<int>(pp);
    *bytes = held;
    return cl;
  }
  return 0;
}

template <class Kernel>
int launch(Kernel kernel, const ResArgs &a, int cl, int n, size_t smem, cudaStream_t s) {
  if (smem > 48 * 1024)
    VAE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(kMaxSmem)));
  if (cl == 1) {  // (a launch with a cluster attribute costs the host more)
    kernel<<<dim3(1, (a.c + a.slab - 1) / a.slab, n), kThreads, smem, s>>>(a);
    VAE_LAUNCH_CHECK();
    count_launches(1);
    return VAE_OK;
  }
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
  VAE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a));
  VAE_LAUNCH_CHECK();
  count_launches(1);
  return VAE_OK;
}

}  // namespace

bool gn_resident(int n, int c, long long spatial, int nhwc, int groups) {
  int per = 0;
  size_t held = 0;
  return cluster_blocks(n, c, spatial, slab_channels(c, groups), &per, &held, nhwc) > 0;
}

int gn_ckpt_resident(const float *x, int n, int c, long long spatial, int nhwc, int groups,
                     float eps, const float *gamma, const float *beta, int silu, float *y,
                     CkptView kx, CkptView ky, float *stats, cudaStream_t s) {
  ResArgs a{};
  a.slab = slab_channels(c, groups);
  size_t held = 0;
  const int cl = cluster_blocks(n, c, spatial, a.slab, &a.per, &held, nhwc);
  if (!cl) return VAE_EUNSUPPORTED;
  const size_t smem = fixed_bytes(a.slab, nhwc, false) + held;
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
  if (!nhwc) return launch(gn_res_fwd_nchw, a, cl, n, smem, s);
  return launch(wide_ok(c, x, y) ? (silu ? gn_res_fwd_nhwc<true, true> : gn_res_fwd_nhwc<false, true>)
                                 : (silu ? gn_res_fwd_nhwc<true, false>
                                         : gn_res_fwd_nhwc<false, false>),
                a, cl, n, smem, s);
}

int gn_backward_resident(const float *dy, CkptView kx, const float *stats, int n, int c,
                         long long spatial, int nhwc, int groups, const float *gamma,
                         const float *beta, int silu, const float *dres, float *dx,
                         float *dgamma, float *dbeta, float2 *sums, cudaStream_t s) {
  ResArgs a{};
  a.slab = slab_channels(c, groups);
  size_t held = 0;
  const int cl = cluster_blocks(n, c, spatial, a.slab, &a.per, &held, nhwc);
  if (!cl) return VAE_EUNSUPPORTED;
  const size_t smem = fixed_bytes(a.slab, nhwc, true) + held;
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
  if (!nhwc) return launch(gn_res_bwd_nchw, a, cl, n, smem, s);
  const bool wide = dres ? wide_ok(c, dy, dx, dres) : wide_ok(c, dy, dx);
  return launch(wide ? (silu ? gn_res_bwd_nhwc<true, true> : gn_res_bwd_nhwc<false, true>)
                     : (silu ? gn_res_bwd_nhwc<true, false> : gn_res_bwd_nhwc<false, false>),
                a, cl, n, smem, s);
}

}  // namespace vae
