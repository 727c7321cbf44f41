// gemv.cu -- a linear layer for up to eight rows (single tokens in serving).
//
// The weights are read once, and that bounds it: a warp takes four of w's rows, its
// lanes eight numbers of each at a time, and multiplies them with the same numbers of
// every row of x, in FP32, whatever the type. Long reductions are split over the warps
// of a block, whose sums meet in shared memory in a fixed order; one thread then
// finishes four neighbouring results. No tensor core: a 128-row tile would multiply
// 120 rows of zeros, and its copies, barriers and tensor memory take 5.5 us where this
// takes 2.3 (512 -> 2048, one row).
#include "linear_epilogue.cuh"

namespace vae {

namespace {

constexpr int kWarps = 4;
constexpr int kCols = 4;  // of a warp

template <class D, int ROWS>
__global__ void __launch_bounds__(32 * kWarps)
    few_rows(const D *__restrict__ x, int rows, int k, const D *__restrict__ w, int n, int along,
             int kind, GemmEpilogue e) {
  __shared__ float4 sums[kWarps][ROWS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % along;  // of the reduction
  const int group = blockIdx.x * (kWarps / along) + warp / along;
  const int col = kCols * group;
  uint64_t acc[ROWS][kCols];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[r][c] = 0;
  if (col < n) {
    const D *wc = w + static_cast<size_t>(col) * k;
#pragma unroll 2
    for (int at = 8 * (32 * part + lane); at < k; at += 256 * along) {
      Raw<D> wr[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        wr[c] = load_raw<D, sizeof(D) == 2>(wc + static_cast<size_t>(c) * k + at, 8);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const Oct xo = oct_of(load_raw<D, sizeof(D) == 2>(x + static_cast<size_t>(r) * k + at,
                                                         r < rows ? 8 : 0));
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const Oct wo = oct_of(wr[c]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][c] = fma2(xo.v[j], wo.v[j], acc[r][c]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    float v[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      v[c] = lo2(acc[r][c]) + hi2(acc[r][c]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], o);
    }
    if (lane == 0) sums[warp][r] = make_float4(v[0], v[1], v[2], v[3]);
  }
  __syncthreads();
  const int r = lane;
  if (part || r >= rows || col >= n) return;
  Quad sum = {{0, 0}}, bias = sum, aux = sum, z, y;
  for (int i = 0; i < along; ++i) {
    const float4 s = sums[warp + i][r];
    sum.v[0] = add2(sum.v[0], pk2(s.x, s.y));
    sum.v[1] = add2(sum.v[1], pk2(s.z, s.w));
  }
  const size_t to = static_cast<size_t>(r) * n + col;
  if (e.bias) bias = load_quad(e.bias + col);
  if (e.aux) aux = load_quad(static_cast<const D *>(e.aux) + to);
  by_kind(kind, [&](auto kd) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      y.v[j] = finish2<decltype(kd)::value, sizeof(D) == 4>(sum.v[j], bias.v[j], aux.v[j], &z.v[j]);
  });
  store_quad(static_cast<D *>(e.out) + to, y);
  if (e.keep) store_quad(static_cast<D *>(e.keep) + to, z);
}

}  // namespace

int linear_few(const void *x, int dtype, int rows, int k, const void *w, int n,
               const GemmEpilogue &e, cudaStream_t s) {
  // a warp's share of the reduction is 512 numbers, two loads of each row, where k has them
  const int along = k >= 2048 ? 4 : k >= 1024 ? 2 : 1;
  const unsigned grid = static_cast<unsigned>(ceil_div(n, kCols * (kWarps / along)));
  const int kind = kind_of(e);
  return by_dtype(dtype, [&](auto d) -> int {
    using D = decltype(d);
    auto kernel = rows == 1   ? few_rows<D, 1>
                  : rows == 2 ? few_rows<D, 2>
                  : rows <= 4 ? few_rows<D, 4>
                              : few_rows<D, 8>;
    kernel<<<grid, 32 * kWarps, 0, s>>>(static_cast<const D *>(x), rows, k,
                                        static_cast<const D *>(w), n, along, kind, e);
    VAE_LAUNCH_CHECK();
    count_launches(1);
    return VAE_OK;
  });
}

}  // namespace vae
