// layer_norm.cu -- layer norm of token rows [rows][c] and its backward pass.
//
// Forward, per row: mean = sum x / c, rstd = 1 / sqrt(sum (x - mean)^2 / c + eps),
//   y = gamma (x - mean) rstd + beta
// Backward, with xh = (x - mean) rstd and t = gamma dy:
//   dx = rstd (t - mean(t) - xh mean(t xh)) + dres
//   dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
//
// A row stays in the registers of T threads, eight numbers each in packed pairs of
// floats, whatever the type in memory: x is read once and the squares are of
// deviations from the mean, so that a mean far from zero costs nothing. The next
// rows' loads are issued before a row is worked on (kAhead). The column sums of the backward
// pass run in registers over the rows of a block (a thread adds up rows / blocks
// numbers) and meet in a second, short kernel in a fixed order. Few rows take one
// launch and no workspace: further blocks of it read the rows once more, column by
// column, from L2 (small_columns).
//
// HBM bounds both, latency and the launch small calls. Measured, forward: 65536 x 1024
// bf16 50 us (5.4 TB/s), float 81 us (6.7 TB/s), 16384 x 512 bf16 7.4 us (from L2), one
// float row of 512 1.7 us.
// Backward with dres: 16384 x 1024 bf16 28 us (4.7 TB/s; 33 us with one row's loads
// under way), float 45 us (5.9 TB/s); three blocks an SM instead of two 35 and 52 us.
#include <cmath>

#include "layer_norm.cuh"
#include "ptx.cuh"
#include "tokens.cuh"

namespace vae {

namespace {

// Blocks of the backward pass: two on each SM of a GB300, and as many elsewhere, so that
// the size of the workspace and the order of the sums do not depend on the device.
constexpr int kBwdBlocks = 2 * 152;

// Rows whose loads are under way while one is worked on: of 16-bit numbers two, as many
// bytes as one of floats, and forward three (65536 x 1024 50 us instead of 52); one
// where the registers hold two octs a thread.
template <class D, int NV, int MOST>
constexpr int kAhead = sizeof(D) == 4 || NV > 1 ? 1 : MOST;

template <int T>
constexpr int block_threads() { return T > 256 ? T : 256; }

// Sum of both halves of `v` over the T threads of a row. Rows wider than a warp
// meet in `buf` (one entry a warp); calls in a row alternate between two of them,
// so that the one barrier of a call is enough.
template <int T>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 *buf) {
#pragma unroll
  for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    named_barrier_sync(1 + warp / W, T);
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v.x += buf[first + i].x;
      v.y += buf[first + i].y;
    }
  }
  return v;
}
template <int T>
__device__ __forceinline__ float row_sum(float v, float2 *buf) {
  return row_sum2<T>(make_float2(v, 0.f), buf).x;
}
__device__ __forceinline__ float total(uint64_t pair) { return lo2(pair) + hi2(pair); }
__device__ __forceinline__ uint64_t both(float v) { return pk2(v, v); }

// Oct i of a row's thread `tid` starts at channel 8 (i T + tid).
template <class D, int T, int NV, bool WIDE>
__global__ void __launch_bounds__(block_threads<T>())
    layer_norm_fwd(const D *x, unsigned rows, int c, float eps, const float *__restrict__ gamma,
                   const float *__restrict__ beta, D *y, float *__restrict__ stats) {
  constexpr int R = block_threads<T>() / T;  // rows of a block
  __shared__ float2 buf[2][block_threads<T>() / 32];
  const int tid = threadIdx.x % T;
  const unsigned step = gridDim.x * R;
  unsigned row = blockIdx.x * R + threadIdx.x / T;
  constexpr int P = kAhead<D, NV, 3>;
  Raw<D> next[P][NV];
  auto fetch = [&](unsigned r, int slot) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid);
      next[slot][i] = load_raw<D, WIDE>(x + static_cast<size_t>(r) * c + ch, r < rows ? c - ch : 0);
    }
  };
#pragma unroll
  for (int q = 0; q < P; ++q) fetch(row + q * step, q);
  Oct g[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    g[i] = param_oct(gamma, 8 * (i * T + tid), c, 1.f);
    b[i] = param_oct(beta, 8 * (i * T + tid), c, 0.f);
  }
  const float inv_c = 1.f / c;
  // whole blocks leave the loop together: every lane takes part in the shuffles
  for (unsigned long long r0 = blockIdx.x * R; r0 < rows; r0 += P * step) {
#pragma unroll
    for (int q = 0; q < P; ++q, row += step) {
      if (q && r0 + q * step >= rows) break;
      const bool live = row < rows;
      Oct v[NV];
      uint64_t sum = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = oct_of(next[q][i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = add2(sum, v[i].v[j]);
      }
      if (r0 + (q + P) * step < rows) fetch(row + P * step, q);
      const float mean = row_sum<T>(total(sum), buf[0]) * inv_c;
      uint64_t ss = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int left = c - 8 * (i * T + tid);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i].v[j] = add2(v[i].v[j], both(-mean));
          if (2 * j < left) ss = fma2(v[i].v[j], v[i].v[j], ss);  // (c is a multiple of four)
        }
      }
      const float rstd = 1.f / sqrtf(row_sum<T>(total(ss), buf[1]) * inv_c + eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int ch = 8 * (i * T + tid);
        Oct o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = fma2(mul2(v[i].v[j], both(rstd)), g[i].v[j], b[i].v[j]);
        store_raw<D, WIDE>(y + static_cast<size_t>(row) * c + ch, live ? c - ch : 0, raw_of<D>(o));
      }
      if (stats && live && tid == 0)
        *reinterpret_cast<float2 *>(stats + 2 * static_cast<size_t>(row)) = make_float2(mean, rstd);
    }
  }
}

// One or two numbers, as floats.
__device__ __forceinline__ float2 load_word(const float *p) { return make_float2(*p, 0.f); }
template <class D>
__device__ __forceinline__ float2 load_word(const D *p) {
  const uint64_t v = unpack2(*reinterpret_cast<const uint32_t *>(p), D{});
  return make_float2(lo2(v), hi2(v));
}
// dgamma and dbeta of a block's 32 bytes of channels: eight lanes are neighbouring
// words, and all threads / 8 rows at a time, eight loads in flight each, meet in a
// fixed order.
template <class D, int THREADS>
__device__ __forceinline__ void small_columns(const D *dy, const D *x, const float *stats,
                                              unsigned rows, int c, int block, float *dgamma,
                                              float *dbeta, float4 *red) {
  constexpr int N = 4 / sizeof(D), G = THREADS / 8;  // channels of a word; rows at a time
  const int ch = (block * 8 + (threadIdx.x & 7)) * N;
  const unsigned first = threadIdx.x >> 3;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);  // dy xh of both, dy of both
  if (ch < c) {
#pragma unroll 8
    for (unsigned r = first; r < rows; r += G) {
      const size_t at = static_cast<size_t>(r) * c + ch;
      const float2 d = load_word(dy + at), v = load_word(x + at);
      const float2 s = __ldg(reinterpret_cast<const float2 *>(stats) + r);
      sum.x = fmaf(d.x, (v.x - s.x) * s.y, sum.x);
      sum.z += d.x;
      if (N > 1) {
        sum.y = fmaf(d.y, (v.y - s.x) * s.y, sum.y);
        sum.w += d.y;
      }
    }
  }
  red[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x < 8 && ch < c) {
#pragma unroll 4
    for (int g = 1; g < G; ++g) {
      const float4 o = red[8 * g + threadIdx.x];
      sum.x += o.x;
      sum.y += o.y;
      sum.z += o.z;
      sum.w += o.w;
    }
    if (dgamma) dgamma[ch] = sum.x;
    if (dbeta) dbeta[ch] = sum.z;
    if (N > 1) {  // (c is a multiple of four)
      if (dgamma) dgamma[ch + 1] = sum.y;
      if (dbeta) dbeta[ch + 1] = sum.w;
    }
  }
}

// part [blocks][c] float2: sums of dy xh and dy over the block's rows. Without it (few
// rows) blocks from `row_blocks` on take columns.
template <class D, int T, int NV, bool WIDE, bool SMALL>
__global__ void __launch_bounds__(block_threads<T>())
    layer_norm_bwd(const D *dy, const D *x, const float *__restrict__ stats, unsigned rows, int c,
                   const float *__restrict__ gamma, const D *dres, D *dx, float2 *part,
                   unsigned row_blocks, float *dgamma, float *dbeta) {
  constexpr int R = block_threads<T>() / T;
  __shared__ float2 buf[2][block_threads<T>() / 32];
  __shared__ float4 red[SMALL ? block_threads<T>() / 4 : R > 1 ? block_threads<T>() * NV : 1][4];
  if (SMALL && blockIdx.x >= row_blocks)
    return small_columns<D, block_threads<T>()>(dy, x, stats, rows, c, blockIdx.x - row_blocks,
                                                dgamma, dbeta, &red[0][0]);
  if (!SMALL) grid_release();
  const int tid = threadIdx.x % T, grp = threadIdx.x / T;
  const unsigned step = row_blocks * R;
  unsigned row = blockIdx.x * R + grp;
  constexpr int P = kAhead<D, NV, 2>;
  Raw<D> xn[P][NV], dn[P][NV], rn[P][NV];
  float2 sn[P];
  auto fetch = [&](unsigned r, int slot) {
    const bool live = r < rows;
    sn[slot] = live ? __ldg(reinterpret_cast<const float2 *>(stats) + r) : make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid), left = live ? c - ch : 0;
      const size_t at = static_cast<size_t>(r) * c + ch;
      xn[slot][i] = load_raw<D, WIDE>(x + at, left);
      dn[slot][i] = load_raw<D, WIDE>(dy + at, left);
      if (dres) rn[slot][i] = load_raw<D, WIDE>(dres + at, left);
    }
  };
#pragma unroll
  for (int q = 0; q < P; ++q) fetch(row + q * step, q);
  Oct g[NV], sg[NV], sb[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    g[i] = param_oct(gamma, 8 * (i * T + tid), c, 1.f);
    sg[i] = sb[i] = {{0, 0, 0, 0}};
  }
  const float inv_c = 1.f / c;
  int turn = 0;
  for (unsigned long long r0 = blockIdx.x * R; r0 < rows; r0 += P * step) {
#pragma unroll
    for (int q = 0; q < P; ++q, row += step) {
      if (q && r0 + q * step >= rows) break;
      const bool live = row < rows;
      Oct xh[NV], t[NV], res[NV];
      const float mean = sn[q].x, rstd = sn[q].y;
      uint64_t st = 0, sx = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xh[i] = oct_of(xn[q][i]);
        t[i] = oct_of(dn[q][i]);
        if (dres) res[i] = oct_of(rn[q][i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xh[i].v[j] = mul2(add2(xh[i].v[j], both(-mean)), both(rstd));
          if (!SMALL) {
            sg[i].v[j] = fma2(t[i].v[j], xh[i].v[j], sg[i].v[j]);
            sb[i].v[j] = add2(t[i].v[j], sb[i].v[j]);
          }
          t[i].v[j] = mul2(t[i].v[j], g[i].v[j]);  // (zero past c, as dy is)
          st = add2(st, t[i].v[j]);
          sx = fma2(t[i].v[j], xh[i].v[j], sx);
        }
      }
      if (r0 + (q + P) * step < rows) fetch(row + P * step, q);
      const float2 s = row_sum2<T>(make_float2(total(st), total(sx)), buf[turn]);
      turn ^= 1;
      const uint64_t m1 = both(-s.x * inv_c), m2 = both(-s.y * inv_c), r2 = both(rstd);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int ch = 8 * (i * T + tid);
        Oct o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t d = fma2(xh[i].v[j], m2, add2(t[i].v[j], m1));
          o.v[j] = dres ? fma2(d, r2, res[i].v[j]) : mul2(d, r2);
        }
        store_raw<D, WIDE>(dx + static_cast<size_t>(row) * c + ch, live ? c - ch : 0, raw_of<D>(o));
      }
    }
  }
  if (SMALL) return;
  if (R > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float4 *e = red[(grp * NV + i) * T + tid];
      e[0] = oct_lo(sg[i]);
      e[1] = oct_hi(sg[i]);
      e[2] = oct_lo(sb[i]);
      e[3] = oct_hi(sb[i]);
    }
    __syncthreads();
  }
  if (grp == 0) {
    float4 *out = reinterpret_cast<float4 *>(part + static_cast<size_t>(blockIdx.x) * c);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = 8 * (i * T + tid);
      for (int k = 1; k < R; ++k) {
        const float4 *e = red[(k * NV + i) * T + tid];
        const Oct p = oct_of(e[0], e[1]), q = oct_of(e[2], e[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sg[i].v[j] = add2(sg[i].v[j], p.v[j]);
          sb[i].v[j] = add2(sb[i].v[j], q.v[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ch + 2 * j < c)
          out[ch / 2 + j] =
              make_float4(lo2(sg[i].v[j]), lo2(sb[i].v[j]), hi2(sg[i].v[j]), hi2(sb[i].v[j]));
    }
  }
}

// Block b: channels [32 b, 32 b + 32), lanes are channels; the 32 warps split the
// blocks' sums, eight loads in flight each, and meet in a fixed order.
__global__ void __launch_bounds__(1024)
    layer_norm_merge(const float2 *part, int blocks, int c, float *dgamma, float *dbeta) {
  __shared__ float2 red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = 32 * blockIdx.x + lane;
  float2 t = make_float2(0.f, 0.f);
  grid_wait();
  if (ch < c) {
#pragma unroll 8
    for (int s = warp; s < blocks; s += 32) {
      const float2 v = part[static_cast<size_t>(s) * c + ch];
      t.x += v.x;
      t.y += v.y;
    }
  }
  red[warp][lane] = t;
  __syncthreads();
  // warp w adds up channel w's 32 sums by a tree over the lanes
  t = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
  }
  const int mine = 32 * blockIdx.x + warp;
  if (lane == 0 && mine < c) {
    if (dgamma) dgamma[mine] = t.x;
    if (dbeta) dbeta[mine] = t.y;
  }
}

// Threads of a row: the fewest of these that hold it with eight numbers each, up to
// 256; two octs a thread up to 4096 channels, and 512 threads up to 8192.
template <class F>
int by_width(int c, F &&f) {
  using std::integral_constant;
  const int octs = ceil_div(c, 8);
  if (octs <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (octs <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (octs <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (octs <= 64) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (octs <= 128) return f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  if (octs <= 256) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (octs <= 512) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
}
int bwd_blocks(long long rows, int c) {
  const int octs = ceil_div(c, 8);
  const int r = octs <= 8    ? 32
                : octs <= 16  ? 16
                : octs <= 32  ? 8
                : octs <= 64  ? 4
                : octs <= 128 ? 2
                              : 1;
  // (two octs a thread: one block an SM; a second round of them costs 5 %)
  return static_cast<int>(std::min<long long>(octs > 256 ? kBwdBlocks / 2 : kBwdBlocks,
                                              (rows + r - 1) / r));
}

}  // namespace

int layer_norm(const void *x, int dtype, long long rows, int c, float eps, const float *gamma,
               const float *beta, void *y, float *stats, cudaStream_t s) {
  return by_dtype(dtype, [&](auto d) -> int {
    using D = decltype(d);
    return by_width(c, [&](auto t, auto nv) -> int {
      constexpr int T = decltype(t)::value, NV = decltype(nv)::value, R = block_threads<T>() / T;
      const long long most = (T > 256 ? 1ll : NV > 1 ? 2ll : 4ll) * num_sms();
      const unsigned grid = static_cast<unsigned>(std::min<long long>((rows + R - 1) / R, most));
      auto kernel = raw_wide<D>(c, x, y) ? layer_norm_fwd<D, T, NV, true>
                                         : layer_norm_fwd<D, T, NV, false>;
      kernel<<<grid, block_threads<T>(), 0, s>>>(static_cast<const D *>(x),
                                                 static_cast<unsigned>(rows), c, eps, gamma, beta,
                                                 static_cast<D *>(y), stats);
      VAE_LAUNCH_CHECK();
      count_launches(1);
      return VAE_OK;
    });
  });
}

// Whether further blocks that read the rows again cost less than a second launch: 2048
// x 512 bf16 5.9 us where 2049 rows take 6.8, 1024 x 1024 4.4 where 1025 take 6.8, and
// 1221 x 700 float 5.6 where both launches took 6.9.
static bool few_rows(long long rows, int c) { return rows <= 2048 && rows * c <= 1 << 20; }

size_t layer_norm_backward_ws_bytes(long long rows, int c) {
  return few_rows(rows, c) ? 0 : static_cast<size_t>(bwd_blocks(rows, c)) * c * sizeof(float2);
}

int layer_norm_backward(const void *dy, const void *x, int dtype, const float *stats,
                        long long rows, int c, const float *gamma, const void *dres, void *dx,
                        float *dgamma, float *dbeta, void *ws, cudaStream_t s) {
  const unsigned blocks = bwd_blocks(rows, c);
  const bool small = few_rows(rows, c);
  float2 *part = static_cast<float2 *>(ws);
  VAE_TRY(by_dtype(dtype, [&](auto d) -> int {
    using D = decltype(d);
    return by_width(c, [&](auto t, auto nv) -> int {
      constexpr int T = decltype(t)::value, NV = decltype(nv)::value;
      const bool wide = raw_wide<D>(c, dy, x, dres, dx);
      auto launch = [&](auto kernel, unsigned row_blocks, unsigned col_blocks) -> int {
        kernel<<<row_blocks + col_blocks, block_threads<T>(), 0, s>>>(
            static_cast<const D *>(dy), static_cast<const D *>(x), stats,
            static_cast<unsigned>(rows), c, gamma, static_cast<const D *>(dres),
            static_cast<D *>(dx), part, row_blocks, dgamma, dbeta);
        VAE_LAUNCH_CHECK();
        count_launches(1);
        return VAE_OK;
      };
      if (!small)
        return launch(wide ? layer_norm_bwd<D, T, NV, true, false>
                           : layer_norm_bwd<D, T, NV, false, false>, blocks, 0);
      auto kernel = wide ? layer_norm_bwd<D, T, NV, true, true>
                         : layer_norm_bwd<D, T, NV, false, true>;
      const unsigned cols = dgamma || dbeta ? ceil_div(c * sizeof(D), 32) : 0;
      if (dx != dy && dx != x) return launch(kernel, blocks, cols);
      // the columns are read before the rows are overwritten
      if (cols) VAE_TRY(launch(kernel, 0, cols));
      return launch(kernel, blocks, 0);
    });
  }));
  if (small) return VAE_OK;
  VAE_CUDA_TRY(launch_after(layer_norm_merge, ceil_div(c, 32), 1024, 0, s, part,
                            static_cast<int>(blocks), c, dgamma, dbeta));
  count_launches(1);
  return VAE_OK;
}

}  // namespace vae
