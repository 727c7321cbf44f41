// dropout.cu -- dropout from a counter-based generator: the mask is a function of
// (seed, offset, element) and is computed where it is needed, forward and backward.
//
// Philox 4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as
// 1, 2, 3", 2011) with the seed as its key and offset + i / 8 as the low 64 bits of
// its counter gives 128 bits, 16 for each of eight elements. An element is dropped
// where its bits are below T = floor(65536 p + 1/2); the others are scaled by
// 65536 / (65536 - T), the inverse of the probability that T stands for, so that the
// expectation is x's. 16 bits and not 32: a block of ten rounds (20 wide products
// and 20 three-input operations) is shared by eight elements instead of four, which
// keeps the kernel below HBM's time in the 16-bit types (4 bytes an element). HBM
// bounds it: 16384 x 2048 bf16 with a residual 30 us (6.7 TB/s), without 26 us.
#include "dropout.cuh"
#include "tokens.cuh"

namespace vae {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 philox(uint64_t counter, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32);
  uint32_t c2 = 0, c3 = 0;
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Two elements (low half of `bits` first): kept ones scaled, dropped ones 0
// whatever they hold, plus the residual's.
__device__ __forceinline__ uint64_t drop2(uint64_t x, uint32_t bits, uint32_t threshold,
                                          uint64_t scale, uint64_t residual) {
  const uint64_t s = fma2(x, scale, residual);
  return pk2((bits & 0xffffu) >= threshold ? lo2(s) : lo2(residual),
             (bits >> 16) >= threshold ? hi2(s) : hi2(residual));
}

template <class D, bool RES, bool WIDE>
__global__ void __launch_bounds__(kThreads)
    dropout_kernel(const D *x, long long octs, int tail, uint32_t threshold, float scale,
                   uint64_t seed, uint64_t offset, const long long *__restrict__ state,
                   const D *residual, D *y) {
  if (state) {
    seed = static_cast<uint64_t>(__ldg(state));
    offset += static_cast<uint64_t>(__ldg(state + 1));
  }
  const uint64_t scale2 = pk2(scale, scale);
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  // the last, partial oct: one number at a time
  if (i == 0 && tail) {
    const uint4 w = philox(offset + static_cast<uint64_t>(octs), seed);
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    for (int j = 0; j < tail; ++j) {
      const long long at = 8 * octs + j;
      const float r = RES ? static_cast<float>(residual[at]) : 0.f;
      const uint32_t bits = words[j >> 1] >> (16 * (j & 1)) & 0xffffu;
      y[at] = static_cast<D>(bits >= threshold ? fmaf(static_cast<float>(x[at]), scale, r) : r);
    }
  }
  for (; i < octs; i += step) {
    const Raw<D> xr = load_raw<D, WIDE>(x + 8 * i, 8);
    Raw<D> rr;
    if (RES) rr = load_raw<D, WIDE>(residual + 8 * i, 8);
    const uint4 w = philox(offset + static_cast<uint64_t>(i), seed);
    const Oct v = oct_of(xr);
    Oct r = {{0, 0, 0, 0}}, o;
    if (RES) r = oct_of(rr);
    o.v[0] = drop2(v.v[0], w.x, threshold, scale2, r.v[0]);
    o.v[1] = drop2(v.v[1], w.y, threshold, scale2, r.v[1]);
    o.v[2] = drop2(v.v[2], w.z, threshold, scale2, r.v[2]);
    o.v[3] = drop2(v.v[3], w.w, threshold, scale2, r.v[3]);
    store_raw<D, WIDE>(y + 8 * i, 8, raw_of<D>(o));
  }
}

}  // namespace

int dropout(const void *x, int dtype, long long count, uint32_t threshold, uint64_t seed,
            uint64_t offset, const long long *state, const void *residual, void *y,
            cudaStream_t s) {
  return by_dtype(dtype, [&](auto d) -> int {
    using D = decltype(d);
    const long long octs = count / 8;
    const float scale =
        threshold < 65536 ? static_cast<float>(65536.0 / (65536.0 - threshold)) : 0.f;
    const bool wide = raw_wide<D>(8, x, residual, y);
    auto kernel = residual ? wide ? dropout_kernel<D, true, true> : dropout_kernel<D, true, false>
                  : wide   ? dropout_kernel<D, false, true>
                           : dropout_kernel<D, false, false>;
    const unsigned grid = static_cast<unsigned>(std::max<long long>(
        1, std::min<long long>((octs + kThreads - 1) / kThreads, 8ll * num_sms())));
    kernel<<<grid, kThreads, 0, s>>>(static_cast<const D *>(x), octs, static_cast<int>(count % 8),
                                     threshold, scale, seed, offset, state,
                                     static_cast<const D *>(residual), static_cast<D *>(y));
    VAE_LAUNCH_CHECK();
    count_launches(1);
    return VAE_OK;
  });
}

}  // namespace vae
