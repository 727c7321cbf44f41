// linear.cu -- a linear layer on token rows, and its gradients.
//
//   z = x w^T + b, y = act(z) + residual       x [rows][k], w [n][k]
//   dx = (dy w) act'(z)                        z [rows][k] of the layer that made x
//   dw = dy^T x, db = sum over rows of dy
// The products run on the tensor cores (gemm.cu); floats go in as three bf16 parts,
// which a pass of its own writes (6 bytes a number).
#include "linear.cuh"
#include "tokens.cuh"

namespace vae {

namespace {

// x = h + m + l exactly, each the nearest bf16 of what is left: 8 significant bits
// and a sign, so that |m| <= 2^-8 |x| and |l| <= 2^-17 |x| (what lies below the
// smallest bf16 is dropped). A finite x that would round to infinity is cut, and no h
// but zero's is zero (m takes it back). A NaN is h. An infinity is l, beside h = 1 of its
// sign: of the products that are added up l enters the one with the other number's h
// alone, so that each of them is infinite with the right sign, finite, or NaN where
// infinity times x is (an infinite h would meet zeros and other signs in m and l).
__device__ __forceinline__ uint32_t nearest_bf16(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__device__ __forceinline__ void split3(float x, uint32_t *h, uint32_t *m, uint32_t *l) {
  const uint32_t bits = __float_as_uint(x), mag = bits & 0x7fffffffu;
  if (mag >= 0x7f800000u) {
    const bool infinite = mag == 0x7f800000u;
    *h = infinite ? (bits >> 16 & 0x8000u) | 0x3f80u : nearest_bf16(x);
    *m = 0;
    *l = infinite ? bits >> 16 : 0;
    return;
  }
  *h = mag >= 0x7f7f8000u ? bits >> 16 : nearest_bf16(x);
  if (mag && !(*h & 0x7fffu)) *h |= 1u;
  const float r = x - __uint_as_float(*h << 16);
  *m = nearest_bf16(r);
  *l = nearest_bf16(r - __uint_as_float(*m << 16));
}

// Two tensors at once: parts of a [na] behind one another at da, of b [nb] at db.
__global__ void __launch_bounds__(256)
    split_kernel(const float *__restrict__ a, long long na, uint16_t *da,
                 const float *__restrict__ b, long long nb, uint16_t *db) {
  grid_release();
  const long long step = 8ll * gridDim.x * 256;
  for (long long at = 8ll * (blockIdx.x * 256ll + threadIdx.x); at < na + nb; at += step) {
    const bool second = at >= na;
    const long long i = second ? at - na : at, n = second ? nb : na;
    const float *src = (second ? b : a) + i;
    uint16_t *dst = (second ? db : da) + i;
    const Raw<float> r = load_raw<float, false>(src, 8);
    const uint32_t *v = reinterpret_cast<const uint32_t *>(r.v);
    uint32_t w[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h0, m0, l0, h1, m1, l1;
      split3(__uint_as_float(v[2 * j]), &h0, &m0, &l0);
      split3(__uint_as_float(v[2 * j + 1]), &h1, &m1, &l1);
      w[0][j] = h0 | h1 << 16;
      w[1][j] = m0 | m1 << 16;
      w[2][j] = l0 | l1 << 16;
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint4 *>(dst + q * n) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
  }
}

// Operands a [na], b [nb] of type `dtype`: as they are, or floats' parts in `ws`.
size_t parts_bytes(int dtype, long long na, long long nb) {
  return dtype == VAE_F32 ? 6 * static_cast<size_t>(na + nb) : 0;
}
int operands(GemmDesc *d, int dtype, const void *a, long long na, const void *b, long long nb,
             void *ws, cudaStream_t s) {
  d->a.p = a;
  d->b.p = b;
  d->dtype = dtype;
  d->f16 = dtype == VAE_F16;
  if (dtype != VAE_F32) return VAE_OK;
  uint16_t *pa = static_cast<uint16_t *>(ws), *pb = pa + 3 * na;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>((na + nb + 2047) / 2048, 8ll * num_sms()));
  split_kernel<<<grid, 256, 0, s>>>(static_cast<const float *>(a), na, pa,
                                    static_cast<const float *>(b), nb, pb);
  VAE_LAUNCH_CHECK();
  count_launches(1);
  d->a.p = pa;
  d->b.p = pb;
  d->parts = 3;
  d->wait = true;
  return VAE_OK;
}

// dw [count], the sums of `slices` arrays (blocks before `sum_blocks`, 1024 numbers
// each), and dbias [n], of `columns` rows (32 numbers a block, the others); both in a
// fixed order.
__global__ void __launch_bounds__(256)
    merge_sums(const float *part, int slices, long long count, float *__restrict__ dw,
               unsigned sum_blocks, const float *cols, int columns, int n,
               float *__restrict__ dbias) {
  __shared__ float red[8][32];
  grid_wait();
  if (blockIdx.x < sum_blocks) {
    const long long i = 4 * (blockIdx.x * 256ll + threadIdx.x);
    if (i >= count) return;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < slices; ++s) {
      const float4 v = *reinterpret_cast<const float4 *>(part + s * count + i);
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
    *reinterpret_cast<float4 *>(dw + i) = t;
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = 32 * (blockIdx.x - sum_blocks) + lane;
  float t = 0.f;
  if (ch < n)
#pragma unroll 8
    for (int s = warp; s < columns; s += 8) t += cols[static_cast<size_t>(s) * n + ch];
  red[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && ch < n) {
#pragma unroll
    for (int w = 1; w < 8; ++w) t += red[w][lane];
    dbias[ch] = t;
  }
}

}  // namespace

// ------------------------------------------------------------------ operators
// Few rows are multiplied on the FP32 cores: up to four, whose weights' bytes bound both
// ways (one row 512 -> 2048 2.3 us, in a tile 5.5; four rows 4096 -> 4096 7.9, 9.1), and
// up to eight of smaller weights (eight rows 2048 -> 1024 4.3 us, in a tile 6.2; 2048 ->
// 4096 9.1, 6.9) or of floats, whose weights a tile would need split (2048 -> 4096 16.2,
// 25.6).
static bool takes_few(int dtype, long long rows, int n, int k) {
  if (rows > kFewRows) return false;
  return rows <= 4 || dtype == VAE_F32 || static_cast<long long>(n) * k < 4 << 20;
}

size_t linear_ws_bytes(int dtype, long long rows, int n, int k) {
  return takes_few(dtype, rows, n, k) ? 0 : parts_bytes(dtype, rows * k, static_cast<long long>(n) * k);
}

int linear(const void *x, int dtype, long long rows, int k, const void *w, const float *bias,
           int n, int act, const void *residual, void *y, void *z, void *ws, cudaStream_t s) {
  if (takes_few(dtype, rows, n, k))
    return linear_few(x, dtype, static_cast<int>(rows), k, w, n, {bias, residual, y, z, act, false},
                      s);
  GemmDesc d;
  VAE_TRY(operands(&d, dtype, x, rows * k, w, static_cast<long long>(n) * k, ws, s));
  d.m = rows;
  d.n = n;
  d.k = k;
  d.epi = {bias, residual, y, z, act, false};
  d.plan = gemm_plan(d.m, d.n, d.k, d.parts, false);
  return gemm(d, s);
}

size_t linear_dgrad_ws_bytes(int dtype, long long rows, int n, int k) {
  return parts_bytes(dtype, rows * n, static_cast<long long>(n) * k);
}

int linear_dgrad(const void *dy, int dtype, long long rows, int n, const void *w, int k, int act,
                 const void *z, void *dx, void *ws, cudaStream_t s) {
  GemmDesc d;
  VAE_TRY(operands(&d, dtype, dy, rows * n, w, static_cast<long long>(n) * k, ws, s));
  d.b.k_major = false;
  d.m = rows;
  d.n = k;
  d.k = n;
  d.epi = {nullptr, z, dx, nullptr, act, true};
  d.plan = gemm_plan(d.m, d.n, d.k, d.parts, false);
  return gemm(d, s);
}

size_t linear_wgrad_ws_bytes(int dtype, long long rows, int n, int k) {
  const GemmPlan plan = gemm_plan(n, k, rows, dtype == VAE_F32 ? 3 : 1, true);
  Carver cv(nullptr, 0);
  cv.take<char>(parts_bytes(dtype, rows * n, rows * k));
  if (plan.slices > 1) cv.take<float>(static_cast<size_t>(plan.slices) * n * k);
  if (plan.columns > 1) cv.take<float>(static_cast<size_t>(plan.columns) * n);
  return cv.used;
}

int linear_wgrad(const void *dy, const void *x, int dtype, long long rows, int n, int k, float *dw,
                 float *dbias, void *ws, cudaStream_t s) {
  Carver cv(ws, ~size_t(0));
  void *parts = cv.take<char>(parts_bytes(dtype, rows * n, rows * k));
  GemmDesc d;
  VAE_TRY(operands(&d, dtype, dy, rows * n, x, rows * k, parts, s));
  d.plan = gemm_plan(n, k, rows, d.parts, true);
  const long long count = static_cast<long long>(n) * k;
  const int slices = d.plan.slices, columns = d.plan.columns;
  float *sums = slices > 1 ? cv.take<float>(static_cast<size_t>(slices) * count) : dw;
  float *cols = columns > 1 ? cv.take<float>(static_cast<size_t>(columns) * n) : dbias;
  d.dtype = VAE_F32;
  d.a.k_major = d.b.k_major = false;
  d.m = n;
  d.n = k;
  d.k = rows;
  d.epi = {nullptr, nullptr, sums, nullptr, VAE_ACT_NONE, true};
  if (dbias) d.cols = {dy, dtype, rows, cols};
  VAE_TRY(gemm(d, s));
  const unsigned sum_blocks = slices > 1 ? ceil_div(count, 1024) : 0;
  const unsigned col_blocks = dbias && columns > 1 ? ceil_div(n, 32) : 0;
  if (sum_blocks + col_blocks == 0) return VAE_OK;
  VAE_CUDA_TRY(launch_after(merge_sums, sum_blocks + col_blocks, 256, 0, s, sums, slices, count, dw,
                            sum_blocks, cols, columns, n, dbias));
  count_launches(1);
  return VAE_OK;
}

}  // namespace vae
