// ckpt.cu -- packing a tensor into an 8-bit activation checkpoint and reading
// one back (format: ckpt.cuh). Both are one sweep over the tensor, bound by
// HBM: 5.03 bytes per element. Measured, [1, 512, 512, 128]: pack 25 us (6.7 TB/s;
// with four channels a thread 36), unpack 30 (34); NCHW 30 and 29 us.
#include "ckpt.cuh"

namespace vae {

namespace {

constexpr int kThreads = 256;

// NHWC, c a multiple of four: a thread per eight channels, the blocks sweep the
// rows side by side. A block's threads all take part in every step (shuffles).
struct Octets {
  int octs, o, step_o;
  long long row, step_row;
  int count;  // steps of this block
  __device__ Octets(long long rows, int cp) : octs(cp >> 3) {
    const unsigned step = gridDim.x * kThreads;
    const long long first = static_cast<long long>(blockIdx.x) * kThreads, i = first + threadIdx.x;
    row = i / octs;
    o = static_cast<int>(i - row * octs);
    step_row = step / octs;
    step_o = static_cast<int>(step % octs);
    count = static_cast<int>((rows * octs - first + step - 1) / step);
  }
  __device__ __forceinline__ void next() {
    row += step_row;
    o += step_o;
    if (o >= octs) {
      o -= octs;
      ++row;
    }
  }
};

template <bool WIDE>
__global__ void __launch_bounds__(kThreads)
    pack_octets(const float *__restrict__ x, long long rows, int c, CkptView k) {
  constexpr int D = 4;  // loads in flight
  const int cp = (c + 31) & ~31;
  Octets at(rows, cp), ahead = at;
  Oct v[D];
  auto fetch = [&]() {
    const Oct r = load_oct<WIDE, true>(x + ahead.row * c + 8 * ahead.o,
                                       ahead.row < rows ? c - 8 * ahead.o : 0);
    ahead.next();
    return r;
  };
#pragma unroll
  for (int u = 0; u < D; ++u) v[u] = fetch();
#pragma unroll 1
  for (int i = 0; i < at.count; i += D)
#pragma unroll
    for (int u = 0; u < D; ++u) {
      uint32_t byte;
      const uint2 q = quad_quantise(v[u], &byte);
      v[u] = fetch();
      if (at.row < rows) {
        __stcs(reinterpret_cast<uint2 *>(k.q + at.row * cp + 8 * at.o), q);
        if ((at.o & 3) == 0)
          k.scale[at.row * (cp >> 5) + (at.o >> 2)] = static_cast<uint8_t>(byte);
      }
      at.next();
    }
}

template <bool WIDE>
__global__ void __launch_bounds__(kThreads)
    unpack_octets(CkptView k, long long rows, int c, float *__restrict__ x) {
  constexpr int D = 4;
  const int cp = (c + 31) & ~31;
  Octets at(rows, cp), ahead = at;
  uint2 q[D];
  uint32_t sc[D];
  auto fetch = [&](int u) {
    q[u] = make_uint2(0, 0);
    sc[u] = 0;
    if (ahead.row < rows) {
      q[u] = __ldcs(reinterpret_cast<const uint2 *>(k.q + ahead.row * cp + 8 * ahead.o));
      sc[u] = __ldg(k.scale + ahead.row * (cp >> 5) + (ahead.o >> 2));
    }
    ahead.next();
  };
#pragma unroll
  for (int u = 0; u < D; ++u) fetch(u);
#pragma unroll 1
  for (int i = 0; i < at.count; i += D)
#pragma unroll
    for (int u = 0; u < D; ++u) {
      const Oct v = unpack_oct(q[u], ckpt_scale(sc[u]));
      fetch(u);
      store_oct<WIDE>(x + at.row * c + 8 * at.o, at.row < rows ? c - 8 * at.o : 0, v);
      at.next();
    }
}

// NHWC, any c: a thread per four channels of a row.
__global__ void __launch_bounds__(kThreads)
    pack_rows(const float *__restrict__ x, long long rows, int c, CkptView k) {
  const int cp = (c + 31) & ~31, quads = cp >> 2;
  const long long total = rows * quads;  // a multiple of 8: octets stay whole
  for (long long i0 = blockIdx.x * static_cast<long long>(kThreads); i0 < total;
       i0 += static_cast<long long>(gridDim.x) * kThreads) {
    const long long i = i0 + threadIdx.x, row = i / quads;
    const int q = static_cast<int>(i - row * quads), ch = 4 * q;
    const bool in = i < total;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      if (ch < c) v.x = x[row * c + ch];
      if (ch + 1 < c) v.y = x[row * c + ch + 1];
      if (ch + 2 < c) v.z = x[row * c + ch + 2];
      if (ch + 3 < c) v.w = x[row * c + ch + 3];
    }
    uint32_t byte;
    const uint32_t b = octet_quantise(v, &byte);
    if (!in) continue;
    *reinterpret_cast<uint32_t *>(k.q + row * cp + ch) = b;
    if ((q & 7) == 0) k.scale[row * (cp >> 5) + (q >> 3)] = static_cast<uint8_t>(byte);
  }
}

__global__ void __launch_bounds__(kThreads)
    unpack_rows(CkptView k, long long rows, int c, float *__restrict__ x) {
  const int cp = (c + 31) & ~31, quads = (c + 3) >> 2;
  const long long total = rows * quads;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long row = i / quads;
    const int q = static_cast<int>(i - row * quads), ch = 4 * q;
    const float4 v = unpack_e4m3x4(
        __ldcs(reinterpret_cast<const uint32_t *>(k.q + row * cp + ch)),
        ckpt_scale(__ldg(k.scale + row * (cp >> 5) + (q >> 3))));
    const float f[4] = {v.x, v.y, v.z, v.w};
    for (int j = 0; j < 4 && ch + j < c; ++j) x[row * c + ch + j] = f[j];
  }
}

// NCHW: a warp per (32 pixels, 32 channels); lanes are pixels. grid (pixel
// blocks, cp / 32, n).
__global__ void __launch_bounds__(128)
    pack_planes(const float *__restrict__ x, int c, long long spatial, CkptView k) {
  const int cp = (c + 31) & ~31, cb = blockIdx.y, n = blockIdx.z, chans = min(32, c - 32 * cb);
  const float *xs = x + (static_cast<long long>(n) * c + 32 * cb) * spatial;
  for (long long p = blockIdx.x * 128ll + threadIdx.x; p < spatial; p += gridDim.x * 128ll) {
    const long long row = static_cast<long long>(n) * spatial + p;
    float v[32];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = j < chans ? __ldcs(xs + j * spatial + p) : 0.f;
      m = max(m, abs_bits(v[j]));
    }
    const uint32_t byte = ckpt_scale_byte(m);
    const float inv = ckpt_inv_scale(byte);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = pack_e4m3x4(v[4 * j] * inv, v[4 * j + 1] * inv, v[4 * j + 2] * inv,
                         v[4 * j + 3] * inv);
    uint4 *dst = reinterpret_cast<uint4 *>(k.q + row * cp + 32 * cb);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    k.scale[row * (cp >> 5) + cb] = static_cast<uint8_t>(byte);
  }
}

__global__ void __launch_bounds__(128)
    unpack_planes(CkptView k, int c, long long spatial, float *__restrict__ x) {
  const int cp = (c + 31) & ~31, cb = blockIdx.y, n = blockIdx.z, chans = min(32, c - 32 * cb);
  float *xs = x + (static_cast<long long>(n) * c + 32 * cb) * spatial;
  for (long long p = blockIdx.x * 128ll + threadIdx.x; p < spatial; p += gridDim.x * 128ll) {
    const long long row = static_cast<long long>(n) * spatial + p;
    const uint4 *src = reinterpret_cast<const uint4 *>(k.q + row * cp + 32 * cb);
    const float sc = ckpt_scale(__ldg(k.scale + row * (cp >> 5) + cb));
    const uint4 lo = __ldcs(src), hi = __ldcs(src + 1);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 v = unpack_e4m3x4(w[j], sc);
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * j + i < chans) __stcs(xs + (4 * j + i) * spatial + p, f[i]);
    }
  }
}

int sweep_blocks(long long items, int per_block) {
  return static_cast<int>(
      std::max(1ll, std::min<long long>(16ll * num_sms(), (items + per_block - 1) / per_block)));
}
// Four blocks an SM, which are resident together.
int octet_blocks(long long rows, int cp) {
  return static_cast<int>(
      std::min<long long>(4ll * num_sms(), (rows * (cp / 8) + kThreads - 1) / kThreads));
}

}  // namespace

int ckpt_pack(const float *x, int n, int c, long long spatial, int nhwc, CkptView k,
              cudaStream_t s) {
  const int cp = ckpt_cp(c);
  if (nhwc) {
    const long long rows = static_cast<long long>(n) * spatial;
    if (c % 4 == 0)
      (wide_ok(c, x) ? pack_octets<true> : pack_octets<false>)<<<octet_blocks(rows, cp), kThreads,
                                                                 0, s>>>(x, rows, c, k);
    else
      pack_rows<<<sweep_blocks(rows * (cp / 4), kThreads), kThreads, 0, s>>>(x, rows, c, k);
  } else {
    pack_planes<<<dim3(sweep_blocks(spatial, 128), cp / 32, n), 128, 0, s>>>(x, c, spatial, k);
  }
  VAE_LAUNCH_CHECK();
  count_launches(1);
  return VAE_OK;
}

int ckpt_unpack(CkptView k, int n, int c, long long spatial, int nhwc, float *x, cudaStream_t s) {
  if (nhwc) {
    const long long rows = static_cast<long long>(n) * spatial;
    if (c % 4 == 0)
      (wide_ok(c, x) ? unpack_octets<true> : unpack_octets<false>)<<<
          octet_blocks(rows, ckpt_cp(c)), kThreads, 0, s>>>(k, rows, c, x);
    else
      unpack_rows<<<sweep_blocks(rows * ((c + 3) / 4), kThreads), kThreads, 0, s>>>(k, rows, c, x);
  } else {
    unpack_planes<<<dim3(sweep_blocks(spatial, 128), ckpt_cp(c) / 32, n), 128, 0, s>>>(k, c,
                                                                                     spatial, x);
  }
  VAE_LAUNCH_CHECK();
  count_launches(1);
  return VAE_OK;
}

}  // namespace vae
