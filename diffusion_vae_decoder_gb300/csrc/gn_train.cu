// gn_train.cu -- GroupNorm(+SiLU) that keeps 8-bit checkpoints of its input
// and output, and the backward pass that reads the input's checkpoint.
//
// Forward, per (sample, group): mean, biased variance, rstd = 1/sqrt(var +
// eps); y = act((x - mean) rstd gamma + beta); x_ckpt = Q(x), y_ckpt = Q(y)
// (ckpt.cuh). Backward, with xh = (x~ - mean) rstd of the checkpoint's x~,
// z = xh gamma + beta and s = 1 / (1 + e^-z):
//   dz = dy s (1 + z (1 - s)) (dy without SiLU)
//   dbeta = sum dz, dgamma = sum dz xh       (samples and pixels)
//   dx = rstd (gamma dz - mean_g(gamma dz) - xh mean_g(gamma dz xh)) (+ dres)
//
// Both need a sum over the whole (sample, group) before the first output
// element, so both are a reducing pass, a small merge and an elementwise pass.
// The first walks the pixels forwards, the second backwards, and outputs are
// stored evict-first, so that the second pass finds in L2 what the first one
// read last.
//
// NHWC: a thread owns eight channels, in packed pairs (these sweeps are bound
// by issued instructions before HBM); the four lanes of a 32-channel block share
// its scale by shuffles. NCHW: a thread owns one pixel and 32 channels,
// so every load and store of the planes is coalesced over pixels and a
// checkpoint block is one thread's registers.
//
// Measured: forward [1, 512, 512, 128] NHWC 82 us, statistics 25 (134 MB, 5.4
// TB/s), merge 3, apply 52 (336 MB, 6.5 TB/s; 1 us of it for the low part of the
// scale, without which y is off by 1.0e-7 rms instead of 0.7e-7); backward [1, 256, 256, 256] 49 us,
// sums 21 (84 MB), merge 4, dx 25 (151 MB, some of it from L2). The sums' pass is
// short: coefficients before it, exp and reciprocal in it and the reduction
// behind it are a third of its time; 2 to 4 pixels in flight measure the same,
// three blocks an SM at 80 registers 59 to 69 us.
#include "gn_stats.cuh"
#include "gn_train.cuh"
#include "ptx.cuh"

namespace vae {

namespace {

constexpr int kThreads = 256;      // NHWC kernels
constexpr int kPixThreads = 128;   // NCHW kernels: one pixel per thread
constexpr int kBlocks = 2 * 152;   // NHWC: the resident blocks, two per SM
constexpr int kPixBlocks = 8 * 152;
constexpr int kMergeThreads = 320;  // a block's slabs in one round

constexpr long long kMostInARow = 4096;

// Blocks (slabs of pixels) per sample. A thread adds up kMostInARow numbers in a row
// at most: step i of a sum of like numbers is off by up to i half-steps of one, and a
// plane of 2^23 pixels in sums of 32768 had its mean off by 4e-4. More blocks than
// are resident are whole rounds of them: from 5 GB on NHWC, and the NCHW statistics of
// many samples from 0.6.
int slabs_nhwc(int n, int c, long long spatial) {
  const int ppi = kThreads / (ckpt_cp(c) / 8);
  const long long most = std::max(1, kBlocks / n);
  const long long rounds = (spatial - 1) / (kMostInARow * ppi * most) + 1;
  return static_cast<int>(std::max(1ll, std::min(rounds * most, spatial / (4 * ppi))));
}
int slabs_nchw(int n, int c, long long spatial) {
  const long long most = std::max(1, kPixBlocks / (n * (ckpt_cp(c) / 32)));
  const long long rounds = (spatial - 1) / (kMostInARow * kPixThreads * most) + 1;
  return static_cast<int>(std::min(rounds * most, (spatial + kPixThreads - 1) / kPixThreads));
}
int slabs_stats_nchw(int ng, long long seg) {  // (a grid's y)
  const long long most = std::max(1, kBlocks / ng);
  const long long rounds = (seg - 1) / (kMostInARow * kStatThreads * most) + 1;
  return static_cast<int>(
      std::max(1ll, std::min({65535ll, rounds * most, seg / (kStatThreads * 8)})));
}

// ------------------------------------------------------------- statistics
__global__ void __launch_bounds__(kStatThreads)
    ckpt_stats_nchw(const float *__restrict__ x, int c, long long spatial, int groups,
                    float *__restrict__ part) {
  __shared__ float red[kStatThreads][3];
  grid_release();
  stats_segment_nchw(x, c, spatial, groups, gridDim.y, blockIdx.x, blockIdx.y, red, part);
}

// A Triple whose mean and M2 carry what rounding dropped of them (Knuth's two-sum):
// a (sample, group) merges 300 of them, and the error of the total is every
// output's. (Before: rstd off by 6e-8 rms, the mean by 3e-8 of the deviation.)
struct Wide {
  float n, mean, m2, mean_low, m2_low;
};
__device__ __forceinline__ float two_sum(float a, float b, float *low) {
  const float s = a + b, c = s - a;
  *low += (a - (s - c)) + (b - c);
  return s;
}
__device__ __forceinline__ Wide merge(const Wide &a, const Wide &b) {
  if (a.n == 0.f) return b;
  if (b.n == 0.f) return a;
  Wide r{a.n + b.n, 0.f, 0.f, a.mean_low, a.m2_low + b.m2_low};
  const float w = b.n / r.n, d = (b.mean - a.mean) + (b.mean_low - a.mean_low);
  r.mean = two_sum(a.mean, d * w, &r.mean_low);
  r.m2 = two_sum(a.m2, b.m2, &r.m2_low);
  r.m2 = two_sum(r.m2, d * d * a.n * w, &r.m2_low);
  return r;
}

// One block per (sample, group): merges its partials in a fixed order. (Little
// code: a kernel this short is bound by fetching its instructions.)
__global__ void __launch_bounds__(kMergeThreads)
    ckpt_stats_merge(const float *part, int slabs, float eps, float2 *stats) {
  __shared__ Wide red[kMergeThreads / 32];
  grid_release();
  grid_wait();
  const float *e = part + static_cast<size_t>(blockIdx.x) * slabs * 3;
  Wide acc{0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int b = threadIdx.x; b < slabs; b += kMergeThreads)
    acc = merge(acc, Wide{e[3 * b], e[3 * b + 1], e[3 * b + 2], 0.f, 0.f});
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {  // (a lane merges the lower lane's first)
    const Wide other{__shfl_xor_sync(0xffffffffu, acc.n, o),
                     __shfl_xor_sync(0xffffffffu, acc.mean, o),
                     __shfl_xor_sync(0xffffffffu, acc.m2, o),
                     __shfl_xor_sync(0xffffffffu, acc.mean_low, o),
                     __shfl_xor_sync(0xffffffffu, acc.m2_low, o)};
    const bool upper = threadIdx.x & o;
    acc = merge(upper ? other : acc, upper ? acc : other);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int w = 1; w < kMergeThreads / 32; ++w) acc = merge(acc, red[w]);
    stats[blockIdx.x] = make_float2(acc.mean + acc.mean_low,
                                    precise_rstd(acc.m2, acc.m2_low, acc.n, eps));
  }
}

// ------------------------------------------------------------- NHWC pieces
// A thread owns channels 8 o .. 8 o + 7 of its pixels; at any time the grid
// works on one contiguous run of pixels. Blocks are walked by whole iterations,
// so that every lane takes part in the shuffles of a checkpoint block.

struct Sweep {
  int o, pl, ppi, ch, left, iters;
  unsigned first, step, spatial;
  long long row0;  // the sample's first pixel
  __device__ Sweep(int c, long long pixels) {
    const int octs = ((c + 31) & ~31) >> 3;
    ppi = kThreads / octs;
    o = threadIdx.x % octs;
    pl = threadIdx.x / octs;
    ch = 8 * o;
    left = pl < ppi ? c - ch : 0;
    spatial = static_cast<unsigned>(pixels);  // (below 2^31)
    first = blockIdx.x * ppi + pl;
    step = gridDim.x * ppi;
    iters = static_cast<int>((spatial + step - 1) / step);
    row0 = static_cast<long long>(blockIdx.y) * pixels;
  }
  __device__ unsigned pixel(int i) const { return first + static_cast<unsigned>(i) * step; }
  // (pixels past the last sweep are outside; those before the first wrap round)
  __device__ bool in(unsigned p) const { return p < spatial; }
};

// base + p * stride, one 32 x 32 -> 64 bit multiply-add.
template <class T>
__device__ __forceinline__ T *row_at(T *base, unsigned p, unsigned stride) {
  return base + static_cast<unsigned long long>(p) * stride;
}

// Statistics: part [n][groups][gridDim.x] triples. Sums of deviations from the
// block's first pixel, which its pixel lanes share.
template <bool WIDE>
__global__ void __launch_bounds__(kThreads, 2)
    ckpt_stats_nhwc(const float *__restrict__ x, int c, long long spatial, int groups,
                    float *__restrict__ part) {
  __shared__ float2 red[kThreads * 8];
  __shared__ float shift[1024];
  grid_release();
  const Sweep sw(c, spatial);
  const int cp = (c + 31) & ~31;
  x += sw.row0 * c;
  const unsigned origin = blockIdx.x * sw.ppi;  // (every block has a pixel)
  const float *src = x + sw.ch;
  constexpr int D = 6;  // loads in flight
  Oct k = load_oct<WIDE, false>(row_at(src, origin, c), sw.left), v[D];
  auto fetch = [&](int i) {
    const unsigned p = sw.pixel(i);
    return load_oct<WIDE, false>(row_at(src, p, c), sw.in(p) ? sw.left : 0);
  };
#pragma unroll
  for (int u = 0; u < D; ++u) v[u] = fetch(u);
  if (sw.pl == 0)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (2 * j < sw.left) {
        shift[sw.ch + 2 * j] = lo2(k.v[j]);
        shift[sw.ch + 2 * j + 1] = hi2(k.v[j]);
      }
#pragma unroll
  for (int j = 0; j < 4; ++j) k.v[j] = mul2(k.v[j], pk2(-1.f, -1.f));
  uint64_t a[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
  if (sw.pl < sw.ppi) {
#pragma unroll 1
    for (int i = 0; i < sw.iters; i += D)
#pragma unroll
      for (int u = 0; u < D; ++u) {
        const Oct x8 = v[u];
        v[u] = fetch(i + u + D);
        if (sw.in(sw.pixel(i + u))) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t d = add2(x8.v[j], k.v[j]);
            a[j] = add2(a[j], d);
            b[j] = fma2(d, d, b[j]);
          }
        }
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[sw.pl * cp + sw.ch + 2 * j] = make_float2(lo2(a[j]), lo2(b[j]));
      red[sw.pl * cp + sw.ch + 2 * j + 1] = make_float2(hi2(a[j]), hi2(b[j]));
    }
  }
  __syncthreads();
  // pixels of the block: a full ppi per iteration but for the last
  const unsigned last = (sw.iters - 1) * sw.step + origin;
  const float total = static_cast<float>(
      static_cast<long long>(sw.iters - 1) * sw.ppi +
      (last < sw.spatial ? min(static_cast<unsigned>(sw.ppi), sw.spatial - last) : 0u));
  for (int i = threadIdx.x; i < c; i += kThreads) {
    float2 t = red[i];
#pragma unroll 8
    for (int l = 1; l < sw.ppi; ++l) {
      t.x += red[l * cp + i].x;
      t.y += red[l * cp + i].y;
    }
    red[i] = t;  // (column i is this thread's)
  }
  __syncthreads();
  const int cg = c / groups, lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
    Triple t{0.f, 0.f, 0.f};
    for (int i = lane; i < cg; i += 32) {
      const float2 v = red[g * cg + i];
      const float m = v.x / total;
      t = merge(t, Triple{total, shift[g * cg + i] + m, fmaxf(v.y - v.x * m, 0.f)});
    }
    t = warp_merge(t);
    if (lane == 0) {
      float *o =
          part + ((static_cast<size_t>(blockIdx.y) * groups + g) * gridDim.x + blockIdx.x) * 3;
      o[0] = t.n;
      o[1] = t.mean;
      o[2] = t.m2;
    }
  }
}

__device__ __forceinline__ Affine8 load_affine8(const Sweep &sw, int c, int groups,
                                                const float2 *__restrict__ stats,
                                                const float *__restrict__ gamma,
                                                const float *__restrict__ beta) {
  const int cg = c / groups;
  float m[8], r[8], ga[8], be[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = j < sw.left;
    const float2 st = in ? stats[blockIdx.y * groups + (sw.ch + j) / cg] : make_float2(0.f, 0.f);
    m[j] = st.x;
    r[j] = st.y;
    ga[j] = in ? gamma[sw.ch + j] : 0.f;
    be[j] = in ? beta[sw.ch + j] : 0.f;
  }
  return affine_of(m, r, ga, be);
}

// k: the checkpoint from the sample's first row on.
__device__ __forceinline__ void keep_oct(CkptView k, unsigned p, int cp, int ch, bool in,
                                         const Oct &v) {
  uint32_t byte;
  const uint2 q = quad_quantise(v, &byte);
  if (!in) return;
  __stcs(reinterpret_cast<uint2 *>(row_at(k.q + ch, p, cp)), q);
  if ((ch & 31) == 0) *row_at(k.scale + (ch >> 5), p, cp >> 5) = static_cast<uint8_t>(byte);
}
__device__ __forceinline__ CkptView from_row(CkptView k, long long row, int cp) {
  if (k.q) {
    k.q += row * cp;
    k.scale += row * (cp >> 5);
  }
  return k;
}

// ------------------------------------------------------------- forward apply
// grid (blocks, n). From the end to the start.
template <bool SILU, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2)
    ckpt_apply_nhwc(const float *x, int c, long long spatial, int groups,
                    const float2 *stats, const float *__restrict__ gamma,
                    const float *__restrict__ beta, float *y, CkptView kx, CkptView ky) {
  const Sweep sw(c, spatial);
  const int cp = (c + 31) & ~31;
  const float *src = x + sw.row0 * c + sw.ch;
  float *dst = y + sw.row0 * c + sw.ch;
  kx = from_row(kx, sw.row0, cp);
  ky = from_row(ky, sw.row0, cp);
  constexpr int D = 4;  // loads in flight
  Oct v[D];
  auto fetch = [&](int i) {
    const unsigned p = sw.pixel(i);
    return load_oct<WIDE, true>(row_at(src, p, c), sw.in(p) ? sw.left : 0);
  };
#pragma unroll
  for (int u = 0; u < D; ++u) v[u] = fetch(sw.iters - 1 - u);
  grid_wait();
  const Affine8 f = load_affine8(sw, c, groups, stats, gamma, beta);
#pragma unroll 1
  for (int top = sw.iters - 1; top >= 0; top -= D)
#pragma unroll
    for (int u = 0; u < D; ++u) {
      const int i = top - u;
      const unsigned p = sw.pixel(i);
      const bool in = sw.in(p) && sw.pl < sw.ppi;
      const Oct x8 = v[u];
      v[u] = fetch(i - D);
      if (kx.q) keep_oct(kx, p, cp, sw.ch, in, x8);
      const Oct o = forward8<SILU>(x8, f);
      store_oct<WIDE>(row_at(dst, p, c), in ? sw.left : 0, o);
      if (ky.q) keep_oct(ky, p, cp, sw.ch, in, o);
    }
}

// grid (slabs, cp / 32, n): a thread per pixel and 32 channels.
__global__ void __launch_bounds__(kPixThreads)
    ckpt_apply_nchw(const float *x, int c, long long spatial, int groups,
                    const float2 *stats, const float *__restrict__ gamma,
                    const float *__restrict__ beta, int silu, float *y, CkptView kx,
                    CkptView ky) {
  __shared__ PairAffine aff[16];
  grid_wait();
  const int n = blockIdx.z, cb = blockIdx.y, cp = (c + 31) & ~31;
  if (threadIdx.x < 16)
    load_pairs(aff, stats + n * groups, gamma, beta, 32 * cb, c, c / groups, threadIdx.x);
  __syncthreads();
  const long long p0 = spatial * blockIdx.x / gridDim.x,
                  p1 = spatial * (blockIdx.x + 1) / gridDim.x;
  const long long base = (static_cast<long long>(n) * c + 32 * cb) * spatial;
  for (long long p = p1 - 1 - threadIdx.x; p >= p0; p -= kPixThreads) {
    const long long row = static_cast<long long>(n) * spatial + p;
    const Row32 v = load_planes(x + base + p, spatial, c - 32 * cb);
    if (kx.q) keep_row32(v, kx, row, cp, cb);
    const Row32 o = forward32(v, aff, silu);
    store_planes(y + base + p, spatial, c - 32 * cb, o);
    if (ky.q) keep_row32(o, ky, row, cp, cb);
  }
}

// ------------------------------------------------------------- backward
// Per-(slab, channel) sums of dz and dz xh: part [n][slabs][c] float2. grid (slabs, n).
template <bool SILU, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2)
    ckpt_sums_nhwc(const float *__restrict__ dy, CkptView k, int c, long long spatial, int groups,
                   const float2 *__restrict__ stats, const float *__restrict__ gamma,
                   const float *__restrict__ beta, float2 *__restrict__ part) {
  __shared__ float2 red[kThreads * 8];
  grid_release();
  const Sweep sw(c, spatial);
  const int cp = (c + 31) & ~31;
  uint64_t a[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
  if (sw.pl < sw.ppi) {
    const float *src = dy + sw.row0 * c + sw.ch;
    const CkptView kv = from_row(k, sw.row0, cp);
    constexpr int D = 3;  // pixels in flight
    Oct g[D];
    uint2 q[D];
    uint32_t sb[D];
    auto fetch = [&](int i, int u) {
      const unsigned p = sw.pixel(i);
      const bool in = sw.in(p);
      g[u] = load_oct<WIDE, false>(row_at(src, p, c), in ? sw.left : 0);
      q[u] = make_uint2(0, 0);
      sb[u] = 0;
      if (in) {
        q[u] = __ldg(reinterpret_cast<const uint2 *>(row_at(kv.q + sw.ch, p, cp)));
        sb[u] = __ldg(row_at(kv.scale + (sw.ch >> 5), p, cp >> 5));
      }
    };
#pragma unroll
    for (int u = 0; u < D; ++u) fetch(u, u);
    const Affine8 f = load_affine8(sw, c, groups, stats, gamma, beta);
#pragma unroll 1
    for (int i = 0; i < sw.iters; i += D)
#pragma unroll
      for (int u = 0; u < D; ++u) {  // (a pixel outside has dy = 0 and adds nothing)
        const Oct dy8 = g[u], x8 = unpack_oct(q[u], ckpt_scale(sb[u]));
        fetch(i + u + D, u);
        Oct dev;
        const Oct dz = grad8<SILU>(dy8, x8, f, &dev);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[j] = add2(a[j], dz.v[j]);
          b[j] = fma2(dz.v[j], dev.v[j], b[j]);
        }
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[sw.pl * cp + sw.ch + 2 * j] = make_float2(lo2(a[j]), lo2(b[j]));
      red[sw.pl * cp + sw.ch + 2 * j + 1] = make_float2(hi2(a[j]), hi2(b[j]));
    }
  }
  __syncthreads();
  float2 *o = part + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * c;
  for (int i = threadIdx.x; i < c; i += kThreads) {
    float2 t = red[i];
#pragma unroll 8
    for (int l = 1; l < sw.ppi; ++l) {
      t.x += red[l * cp + i].x;
      t.y += red[l * cp + i].y;
    }
    t.y *= stats[blockIdx.y * groups + i / (c / groups)].y;  // dev rstd = xh
    o[i] = t;
  }
}

// grid (slabs, cp / 32, n).
__global__ void __launch_bounds__(kPixThreads)
    ckpt_sums_nchw(const float *__restrict__ dy, CkptView k, int c, long long spatial, int groups,
                   const float2 *__restrict__ stats, const float *__restrict__ gamma,
                   const float *__restrict__ beta, int silu, float2 *__restrict__ part) {
  __shared__ PairAffine aff[16];
  __shared__ float2 red[kPixThreads / 32][32];
  grid_release();
  const int n = blockIdx.z, cb = blockIdx.y, cp = (c + 31) & ~31, cg = c / groups;
  if (threadIdx.x < 16)
    load_pairs(aff, stats + n * groups, gamma, beta, 32 * cb, c, cg, threadIdx.x);
  __syncthreads();
  const int left = c - 32 * cb, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long p0 = spatial * blockIdx.x / gridDim.x,
                  p1 = spatial * (blockIdx.x + 1) / gridDim.x;
  const float *src = dy + (static_cast<long long>(n) * c + 32 * cb) * spatial;
  float2 sum = make_float2(0.f, 0.f);  // of channel `lane`
  for (long long pw = p0 + 32 * warp; pw < p1; pw += kPixThreads) {
    const long long p = pw + lane;
    const bool here = p < p1;  // (elsewhere dy = 0, which adds nothing)
    const Row32 g = load_planes(src + p, spatial, here ? left : 0);
    const Row32 v = read_row32(k, static_cast<long long>(n) * spatial + (here ? p : p0), cp, cb);
    Row32 dev;
    const Row32 dz = grad32(g, v, aff, silu, &dev);
    const float2 t = run_sums(dz, dev, lane);
    sum.x += t.x;
    sum.y += t.y;
  }
  red[warp][lane] = sum;
  __syncthreads();
  if (threadIdx.x < 32 && threadIdx.x < left) {
    float2 t = red[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kPixThreads / 32; ++w) {
      t.x += red[w][threadIdx.x].x;
      t.y += red[w][threadIdx.x].y;
    }
    const int ch = 32 * cb + threadIdx.x;
    t.y *= stats[n * groups + ch / cg].y;  // dev rstd = xh
    part[(static_cast<size_t>(n) * gridDim.x + blockIdx.x) * c + ch] = t;
  }
}

// Block (b, i): channels [32 b, 32 b + 32) of sample i; lanes are channels, warps
// stride over the slabs; fixed order.
__global__ void __launch_bounds__(1024)
    ckpt_sums_merge(const float2 *part, int slabs, int c, float2 *sums) {
  __shared__ float2 red[32][32];
  grid_release();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = 32 * blockIdx.x + lane;
  const float2 *e = part + static_cast<size_t>(blockIdx.y) * slabs * c + ch;
  float2 t = make_float2(0.f, 0.f);
  if (ch < c)
#pragma unroll 8
    for (int s = warp; s < slabs; s += 32) {
      const float2 v = e[static_cast<size_t>(s) * c];
      t.x += v.x;
      t.y += v.y;
    }
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && ch < c) {
#pragma unroll 4
    for (int w = 1; w < 32; ++w) {
      t.x += red[w][lane].x;
      t.y += red[w][lane].y;
    }
    sums[static_cast<size_t>(blockIdx.y) * c + ch] = t;
  }
}

// dbeta and dgamma of channels [first, last): sums over the samples, in order.
__device__ __forceinline__ void param_grads(const float2 *sums, int n, int c, int first, int last,
                                            float *dgamma, float *dbeta) {
  for (int ch = first + threadIdx.x; ch < last; ch += blockDim.x) {
    float2 t = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float2 v = sums[static_cast<size_t>(i) * c + ch];
      t.x += v.x;
      t.y += v.y;
    }
    if (dbeta) dbeta[ch] = t.x;
    if (dgamma) dgamma[ch] = t.y;
  }
}
__global__ void __launch_bounds__(128)
    ckpt_param_grads(const float2 *sums, int n, int c, float *dgamma, float *dbeta) {
  grid_wait();
  const int first = blockIdx.x * blockDim.x;
  param_grads(sums, n, c, first, min(c, first + static_cast<int>(blockDim.x)), dgamma, dbeta);
}

// k1[g] = rstd mean_g(gamma dz), k2[g] = rstd mean_g(gamma dz xh) of sample n
// for groups [g0, g1), into shared memory; a warp per group.
__device__ __forceinline__ void group_means(float2 *km, const float2 *sums, int n, int c,
                                            int groups, long long spatial,
                                            const float2 *__restrict__ stats,
                                            const float *__restrict__ gamma, int g0, int g1) {
  const int cg = c / groups, lane = threadIdx.x & 31;
  for (int g = g0 + (threadIdx.x >> 5); g < g1; g += blockDim.x >> 5) {
    float a = 0.f, b = 0.f;
    for (int j = lane; j < cg; j += 32) {
      const float2 t = sums[static_cast<size_t>(n) * c + g * cg + j];
      const float ga = gamma[g * cg + j];
      a = fmaf(ga, t.x, a);
      b = fmaf(ga, t.y, b);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane == 0) {
      const float f = stats[n * groups + g].y / (static_cast<float>(cg) * spatial);
      km[g - g0] = make_float2(a * f, b * f);
    }
  }
  __syncthreads();
}

// grid (slabs, n).
template <bool SILU, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2)
    ckpt_dx_nhwc(const float *dy, CkptView k, int c, long long spatial, int groups,
                 const float2 *__restrict__ stats, const float *__restrict__ gamma,
                 const float *__restrict__ beta, const float2 *sums, const float *dres, float *dx,
                 float *dgamma, float *dbeta) {
  __shared__ float2 km[1024];
  const Sweep sw(c, spatial);
  const int cp = (c + 31) & ~31, cg = c / groups;
  const float *src = dy + sw.row0 * c + sw.ch, *res = dres ? dres + sw.row0 * c + sw.ch : nullptr;
  float *dst = dx + sw.row0 * c + sw.ch;
  const CkptView kv = from_row(k, sw.row0, cp);
  constexpr int D = 3;  // pixels in flight
  Oct g[D];
  uint2 q[D];
  uint32_t sb[D];
  auto fetch = [&](int i, int u) {
    const unsigned p = sw.pixel(i);
    const bool in = sw.in(p);
    g[u] = load_oct<WIDE, true>(row_at(src, p, c), in ? sw.left : 0);
    q[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (in) {
      q[u] = __ldcs(reinterpret_cast<const uint2 *>(row_at(kv.q + sw.ch, p, cp)));
      sb[u] = __ldg(row_at(kv.scale + (sw.ch >> 5), p, cp >> 5));
    }
  };
#pragma unroll
  for (int u = 0; u < D; ++u) fetch(sw.iters - 1 - u, u);
  grid_wait();
  group_means(km, sums, blockIdx.y, c, groups, spatial, stats, gamma, 0, groups);
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0)
    param_grads(sums, gridDim.y, c, 0, c, dgamma, dbeta);
  if (sw.pl >= sw.ppi) return;
  const Affine8 f = load_affine8(sw, c, groups, stats, gamma, beta);
  // dx = scale dz + (k1 + dev k2): both means negated, k2 with the rstd of xh
  uint64_t k1[4], k2[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = make_float2(0.f, 0.f);
      if (2 * j + h < sw.left) {
        const int g = (sw.ch + 2 * j + h) / cg;
        m[h] = make_float2(-km[g].x, -km[g].y * stats[blockIdx.y * groups + g].y);
      }
    }
    k1[j] = pk2(m[0].x, m[1].x);
    k2[j] = pk2(m[0].y, m[1].y);
  }
#pragma unroll 1
  for (int top = sw.iters - 1; top >= 0; top -= D)
#pragma unroll
    for (int u = 0; u < D; ++u) {
      const int i = top - u;
      const unsigned p = sw.pixel(i);
      const int left = sw.in(p) ? sw.left : 0;
      const Oct dy8 = g[u], x8 = unpack_oct(q[u], ckpt_scale(sb[u]));
      Oct dev, o, r = {{0, 0, 0, 0}};
      if (res) r = load_oct<WIDE, true>(row_at(res, p, c), left);
      fetch(i - D, u);
      const Oct dz = grad8<SILU>(dy8, x8, f, &dev);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o.v[j] = fma2(f.scale[j], dz.v[j], fma2(dev.v[j], k2[j], k1[j]));
        o.v[j] = add2(o.v[j], r.v[j]);
      }
      store_oct<WIDE>(row_at(dst, p, c), left, o);
    }
}

// grid (slabs, cp / 32, n).
__global__ void __launch_bounds__(kPixThreads)
    ckpt_dx_nchw(const float *dy, CkptView k, int c, long long spatial, int groups,
                 const float2 *__restrict__ stats, const float *__restrict__ gamma,
                 const float *__restrict__ beta, int silu, const float2 *sums, const float *dres,
                 float *dx, float *dgamma, float *dbeta) {
  __shared__ PairAffine aff[16];
  __shared__ float2 km[32];
  const int n = blockIdx.z, cb = blockIdx.y, cp = (c + 31) & ~31, cg = c / groups;
  const int left = c - 32 * cb, chans = min(32, left);
  if (threadIdx.x < 16)
    load_pairs(aff, stats + n * groups, gamma, beta, 32 * cb, c, cg, threadIdx.x);
  const int g0 = 32 * cb / cg, g1 = (32 * cb + chans - 1) / cg + 1;
  grid_wait();
  group_means(km, sums, n, c, groups, spatial, stats, gamma, g0, g1);
  if (threadIdx.x < 16) {
    float2 m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ch = 2 * threadIdx.x + h, g = (32 * cb + ch) / cg;
      m[h] = ch < chans ? make_float2(-km[g - g0].x, -km[g - g0].y * stats[n * groups + g].y)
                        : make_float2(0.f, 0.f);
    }
    aff[threadIdx.x].k1 = pk2(m[0].x, m[1].x);
    aff[threadIdx.x].k2 = pk2(m[0].y, m[1].y);
  }
  __syncthreads();
  const long long p0 = spatial * blockIdx.x / gridDim.x,
                  p1 = spatial * (blockIdx.x + 1) / gridDim.x;
  const long long base = (static_cast<long long>(n) * c + 32 * cb) * spatial;
  for (long long p = p1 - 1 - threadIdx.x; p >= p0; p -= kPixThreads) {
    const Row32 g = load_planes(dy + base + p, spatial, left);
    const Row32 v = read_row32(k, static_cast<long long>(n) * spatial + p, cp, cb);
    Row32 dev;
    const Row32 dz = grad32(g, v, aff, silu, &dev);
    Row32 o = dx32(dz, dev, aff);
    if (dres) {
      const Row32 r = load_planes(dres + base + p, spatial, left);
#pragma unroll
      for (int j = 0; j < 16; ++j) o.v[j] = add2(o.v[j], r.v[j]);
    }
    store_planes(dx + base + p, spatial, left, o);
  }
  if (blockIdx.x == 0 && n == 0)
    param_grads(sums, gridDim.z, c, 32 * cb, 32 * cb + chans, dgamma, dbeta);
}

// ------------------------------------------------------------- workspaces
struct CkptWs {
  float *part;   // statistics partials [n][groups][slabs] x 3, or float2 sums [n][slabs][c]
  float2 *sums;  // [n][c]
};

CkptWs carve_forward(Carver &cv, int n, int c, long long spatial, int groups) {
  CkptWs w{};
  const long long ng = static_cast<long long>(n) * groups;
  const size_t a = static_cast<size_t>(ng) * slabs_nhwc(n, c, spatial);
  const size_t b = static_cast<size_t>(ng) *
                   slabs_stats_nchw(static_cast<int>(ng), spatial * (c / groups));
  w.part = cv.take<float>(3 * std::max(a, b));
  return w;
}
CkptWs carve_backward(Carver &cv, int n, int c, long long spatial) {
  CkptWs w{};
  const size_t slabs = std::max(slabs_nhwc(n, c, spatial), slabs_nchw(n, c, spatial));
  w.part = cv.take<float>(2 * static_cast<size_t>(n) * slabs * c);
  w.sums = cv.take<float2>(static_cast<size_t>(n) * c);
  return w;
}

}  // namespace

size_t gn_ckpt_ws_bytes(int n, int c, long long spatial, int nhwc, int groups) {
  if (gn_resident(n, c, spatial, nhwc, groups)) return 0;
  Carver cv(nullptr, 0);
  carve_forward(cv, n, c, spatial, groups);
  return cv.used;
}
size_t gn_backward_ws_bytes(int n, int c, long long spatial, int nhwc, int groups) {
  if (n == 1 && gn_resident(n, c, spatial, nhwc, groups)) return 0;
  Carver cv(nullptr, 0);
  carve_backward(cv, n, c, spatial);
  return cv.used;
}

int gn_ckpt(const float *x, int n, int c, long long spatial, int nhwc, int groups, float eps,
            const float *gamma, const float *beta, int silu, float *y, CkptView kx, CkptView ky,
            float *stats, void *ws, cudaStream_t s) {
  const int rc = gn_ckpt_resident(x, n, c, spatial, nhwc, groups, eps, gamma, beta, silu, y, kx,
                                  ky, stats, s);
  if (rc != VAE_EUNSUPPORTED) return rc;
  Carver cv(ws, ~size_t(0));
  const CkptWs w = carve_forward(cv, n, c, spatial, groups);
  float2 *st = reinterpret_cast<float2 *>(stats);
  const int ng = n * groups;
  const bool wide = wide_ok(c, x, y);
  int slabs;
  if (nhwc) {
    slabs = slabs_nhwc(n, c, spatial);
    (wide ? ckpt_stats_nhwc<true> : ckpt_stats_nhwc<false>)<<<dim3(slabs, n), kThreads, 0, s>>>(
        x, c, spatial, groups, w.part);
  } else {
    slabs = slabs_stats_nchw(ng, spatial * (c / groups));
    ckpt_stats_nchw<<<dim3(ng, slabs), kStatThreads, 0, s>>>(x, c, spatial, groups, w.part);
  }
  VAE_LAUNCH_CHECK();
  VAE_CUDA_TRY(launch_after(ckpt_stats_merge, ng, kMergeThreads, 0, s, w.part, slabs, eps, st));
  if (nhwc)
    VAE_CUDA_TRY(launch_after(
        wide ? (silu ? ckpt_apply_nhwc<true, true> : ckpt_apply_nhwc<false, true>)
             : (silu ? ckpt_apply_nhwc<true, false> : ckpt_apply_nhwc<false, false>),
        dim3(slabs, n), kThreads, 0, s, x, c, spatial, groups, st, gamma, beta, y, kx, ky));
  else
    VAE_CUDA_TRY(launch_after(ckpt_apply_nchw,
                              dim3(slabs_nchw(n, c, spatial), ckpt_cp(c) / 32, n), kPixThreads, 0,
                              s, x, c, spatial, groups, st, gamma, beta, silu, y, kx, ky));
  count_launches(3);
  return VAE_OK;
}

int gn_backward(const float *dy, CkptView k, const float *stats, int n, int c, long long spatial,
                int nhwc, int groups, const float *gamma, const float *beta, int silu,
                const float *dres, float *dx, float *dgamma, float *dbeta, void *ws,
                cudaStream_t s) {
  Carver cv(ws, ~size_t(0));
  const CkptWs w = carve_backward(cv, n, c, spatial);
  const float2 *st = reinterpret_cast<const float2 *>(stats);
  float2 *part = reinterpret_cast<float2 *>(w.part);
  const bool wide = dres ? wide_ok(c, dy, dx, dres) : wide_ok(c, dy, dx);
  const int rc = gn_backward_resident(dy, k, stats, n, c, spatial, nhwc, groups, gamma, beta,
                                      silu, dres, dx, dgamma, dbeta, w.sums, s);
  if (rc == VAE_OK && n > 1 && (dgamma || dbeta)) {
    VAE_CUDA_TRY(
        launch_after(ckpt_param_grads, ceil_div(c, 128), 128, 0, s, w.sums, n, c, dgamma, dbeta));
    count_launches(1);
  }
  if (rc != VAE_EUNSUPPORTED) return rc;
  const int slabs = nhwc ? slabs_nhwc(n, c, spatial) : slabs_nchw(n, c, spatial);
  const dim3 grid = nhwc ? dim3(slabs, n) : dim3(slabs, ckpt_cp(c) / 32, n);
  if (nhwc)
    (wide ? (silu ? ckpt_sums_nhwc<true, true> : ckpt_sums_nhwc<false, true>)
          : (silu ? ckpt_sums_nhwc<true, false> : ckpt_sums_nhwc<false, false>))<<<grid, kThreads, 0,
                                                                          s>>>(
        dy, k, c, spatial, groups, st, gamma, beta, part);
  else
    ckpt_sums_nchw<<<grid, kPixThreads, 0, s>>>(dy, k, c, spatial, groups, st, gamma, beta, silu,
                                                part);
  VAE_LAUNCH_CHECK();
  VAE_CUDA_TRY(launch_after(ckpt_sums_merge, dim3(ckpt_cp(c) / 32, n), 1024, 0, s, part, slabs, c,
                            w.sums));
  if (nhwc)
    VAE_CUDA_TRY(launch_after(
        wide ? (silu ? ckpt_dx_nhwc<true, true> : ckpt_dx_nhwc<false, true>)
             : (silu ? ckpt_dx_nhwc<true, false> : ckpt_dx_nhwc<false, false>),
        grid, kThreads, 0, s, dy, k, c, spatial, groups, st, gamma, beta, w.sums, dres, dx, dgamma,
        dbeta));
  else
    VAE_CUDA_TRY(launch_after(ckpt_dx_nchw, grid, kPixThreads, 0, s, dy, k, c, spatial, groups, st,
                              gamma, beta, silu, w.sums, dres, dx, dgamma, dbeta));
  count_launches(3);
  return VAE_OK;
}

}  // namespace vae
