// ckpt.cuh -- 8-bit activation checkpoints: the format (include/vae.h,
// vae_ckpt_bytes) and the device code that writes and reads it.
//
// Rows (pixels or tokens) of c channels, c padded to cp = 32 ceil(c / 32). A
// block of 32 consecutive channels of a row shares one power-of-two scale 2^e,
// e the smallest integer >= -127 with max|v| <= 448 * 2^e (448 is the largest
// e4m3 number), and holds q = e4m3(v * 2^-e), rounded to nearest even. The
// rounding to 4 significand bits is the point of the format (a quarter of the
// bytes); everything around it is exact: v * 2^-e changes only the exponent,
// and q * 2^e fits bf16. A block with an infinity or NaN has the scale byte
// 255 and reads back as NaN throughout.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "silu.cuh"

namespace vae {

struct CkptView {
  uint8_t *q = nullptr;      // [rows][cp] e4m3
  uint8_t *scale = nullptr;  // [rows][cp / 32] e + 127
};

inline int ckpt_cp(int c) { return (c + 31) / 32 * 32; }
inline size_t ckpt_scale_offset(long long rows, int c) {
  return align_up(static_cast<size_t>(rows) * ckpt_cp(c), 256);
}
inline size_t ckpt_bytes(long long rows, int c) {
  return ckpt_scale_offset(rows, c) + static_cast<size_t>(rows) * (ckpt_cp(c) / 32);
}
inline CkptView ckpt_view(const void *q, const void *scale) {
  CkptView v;
  v.q = static_cast<uint8_t *>(const_cast<void *>(q));
  v.scale = static_cast<uint8_t *>(const_cast<void *>(scale));
  return v;
}

// Scale byte of a block from the largest bit pattern of its |v| (unsigned
// order is the order of magnitudes, with infinity and NaN on top).
// 448 = 1.75 * 2^8, so e = exponent - 8, one more when the significand is
// above 1.75: when adding 0x1fffff to its 23 bits carries.
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t amax_bits) {
  const int b = max(static_cast<int>((amax_bits + 0x1fffffu) >> 23) - 8, 0);
  return amax_bits >= 0x7f800000u ? 255u : static_cast<uint32_t>(b);
}
// 2^-e as a float (a normal number for every byte below 255); NaN for 255.
__device__ __forceinline__ float ckpt_inv_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : (254u - byte) << 23);
}
// 2^e as a float; byte 255 gives infinity, whose product with the stored NaNs is NaN.
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// max(|a|, |b|, |c|), NaN when one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Four values (already times 2^-e) -> four e4m3 bytes, the first lowest.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
// Two e4m3 bytes -> two halves (exact).
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return *reinterpret_cast<__half2 *>(&r);
}
__device__ __forceinline__ float4 unpack_e4m3x4(uint32_t q, float scale) {
  const float2 a = __half22float2(e4m3x2_half2(q & 0xffffu));
  const float2 b = __half22float2(e4m3x2_half2(q >> 16));
  return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

// A block spread over the eight lanes of an aligned octet, four values each:
// quantises them, returns this lane's four bytes and the block's scale byte.
// Every lane of the warp calls.
__device__ __forceinline__ uint32_t octet_quantise(float4 v, uint32_t *byte) {
  float m = max_abs3(max_abs3(v.x, v.y, v.z), v.w, v.w);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, m, o);
    m = max_abs3(m, w, w);
  }
  *byte = ckpt_scale_byte(__float_as_uint(m));
  const float inv = ckpt_inv_scale(*byte);
  return pack_e4m3x4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
}

// Eight consecutive channels as packed pairs, for the two-wide FP32 pipe.
struct Oct {
  uint64_t v[4];
};
__device__ __forceinline__ Oct oct_of(float4 a, float4 b) {
  return {{pk2(a.x, a.y), pk2(a.z, a.w), pk2(b.x, b.y), pk2(b.z, b.w)}};
}
__device__ __forceinline__ float4 oct_lo(const Oct &o) {
  return make_float4(lo2(o.v[0]), hi2(o.v[0]), lo2(o.v[1]), hi2(o.v[1]));
}
__device__ __forceinline__ float4 oct_hi(const Oct &o) {
  return make_float4(lo2(o.v[2]), hi2(o.v[2]), lo2(o.v[3]), hi2(o.v[3]));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight channels in one 256-bit access where rows and pointers are 32-byte
// aligned (WIDE: c a multiple of eight), else in two of 128 bits: with 32 bytes
// between lanes the halves of a sector would pass L2 twice. Those past c (a
// multiple of four), from `left` on, are zeros. LAST: the data is not needed in
// L2 any more (evict first), and stores never are.
template <bool WIDE, bool LAST>
__device__ __forceinline__ Oct load_oct(const float *p, int left) {
  if (WIDE) {
    Oct o = {{0, 0, 0, 0}};
    if (left > 0) {
      if (LAST)
        asm volatile("ld.global.L1::no_allocate.L2::evict_first.v4.b64 {%0, %1, %2, %3}, [%4];"
                     : "=l"(o.v[0]), "=l"(o.v[1]), "=l"(o.v[2]), "=l"(o.v[3])
                     : "l"(p)
                     : "memory");
      else
        asm volatile("ld.global.L1::no_allocate.v4.b64 {%0, %1, %2, %3}, [%4];"
                     : "=l"(o.v[0]), "=l"(o.v[1]), "=l"(o.v[2]), "=l"(o.v[3])
                     : "l"(p)
                     : "memory");
    }
    return o;
  }
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  return oct_of(left > 0 ? *reinterpret_cast<const float4 *>(p) : zero,
                left > 4 ? *(reinterpret_cast<const float4 *>(p) + 1) : zero);
}
template <bool WIDE>
__device__ __forceinline__ void store_oct(float *p, int left, const Oct &o) {
  if (WIDE) {
    if (left > 0)
      asm volatile("st.global.L2::evict_first.v4.b64 [%4], {%0, %1, %2, %3};" ::"l"(o.v[0]),
                   "l"(o.v[1]), "l"(o.v[2]), "l"(o.v[3]), "l"(p)
                   : "memory");
    return;
  }
  if (left > 0) __stcs(reinterpret_cast<float4 *>(p), oct_lo(o));
  if (left > 4) __stcs(reinterpret_cast<float4 *>(p) + 1, oct_hi(o));
}
// Whether all of these tensors of c channels a pixel take 256-bit accesses.
template <class... T>
inline bool wide_ok(int c, const T *...p) {
  return c % 8 == 0 && (((reinterpret_cast<uintptr_t>(p) & 31) == 0) && ...);
}

// octet_quantise for a block spread over four aligned lanes, eight values each.
__device__ __forceinline__ uint2 quad_quantise(const Oct &x, uint32_t *byte) {
  float m = max_abs3(lo2(x.v[0]), hi2(x.v[0]), lo2(x.v[1]));
  m = max_abs3(m, hi2(x.v[1]), lo2(x.v[2]));
  m = max_abs3(m, hi2(x.v[2]), lo2(x.v[3]));
  m = max_abs3(m, hi2(x.v[3]), __shfl_xor_sync(0xffffffffu, max_abs3(m, hi2(x.v[3]), m), 1));
  m = max_abs3(m, m, __shfl_xor_sync(0xffffffffu, m, 2));
  *byte = ckpt_scale_byte(__float_as_uint(m));
  const float inv = ckpt_inv_scale(*byte);
  const uint64_t i2 = pk2(inv, inv);
  uint64_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = mul2(x.v[j], i2);
  return make_uint2(pack_e4m3x4(lo2(q[0]), hi2(q[0]), lo2(q[1]), hi2(q[1])),
                    pack_e4m3x4(lo2(q[2]), hi2(q[2]), lo2(q[3]), hi2(q[3])));
}
__device__ __forceinline__ Oct unpack_oct(uint2 q, float scale) {
  const uint64_t s2 = pk2(scale, scale);
  const float2 a = __half22float2(e4m3x2_half2(q.x & 0xffffu));
  const float2 b = __half22float2(e4m3x2_half2(q.x >> 16));
  const float2 c = __half22float2(e4m3x2_half2(q.y & 0xffffu));
  const float2 d = __half22float2(e4m3x2_half2(q.y >> 16));
  return {{mul2(pk2(a.x, a.y), s2), mul2(pk2(b.x, b.y), s2), mul2(pk2(c.x, c.y), s2),
           mul2(pk2(d.x, d.y), s2)}};
}

// Pack / unpack a float tensor (ckpt.cu); x in either layout.
int ckpt_pack(const float *x, int n, int c, long long spatial, int nhwc, CkptView out,
              cudaStream_t s);
int ckpt_unpack(CkptView in, int n, int c, long long spatial, int nhwc, float *x, cudaStream_t s);

}  // namespace vae
