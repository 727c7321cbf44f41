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
inline CkptView ckpt_view(const void *p, long long rows, int c) {
  CkptView v;
  if (!p) return v;
  v.q = static_cast<uint8_t *>(const_cast<void *>(p));
  v.scale = v.q + ckpt_scale_offset(rows, c);
  return v;
}

// Scale byte of a block from the largest bit pattern of its |v| (unsigned
// order is the order of magnitudes, with infinity and NaN on top).
// 448 = 1.75 * 2^8, so e = exponent - 8, one more when the significand is
// above 1.75.
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int b = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return b > 0 ? static_cast<uint32_t>(b) : 0u;
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
// `mask` names the octet's lanes (octet_mask), all of which have to call.
__device__ __forceinline__ uint32_t octet_mask() { return 0xffu << (threadIdx.x & 24); }
__device__ __forceinline__ uint32_t octet_max(uint32_t m, uint32_t mask) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
  return m;
}
__device__ __forceinline__ uint32_t octet_quantise(float4 v, uint32_t mask, uint32_t *byte) {
  const uint32_t m =
      max(max(abs_bits(v.x), abs_bits(v.y)), max(abs_bits(v.z), abs_bits(v.w)));
  *byte = ckpt_scale_byte(octet_max(m, mask));
  const float inv = ckpt_inv_scale(*byte);
  return pack_e4m3x4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
}

// Pack / unpack a float tensor (ckpt.cu); x in either layout.
int ckpt_pack(const float *x, int n, int c, long long spatial, int nhwc, CkptView out,
              cudaStream_t s);
int ckpt_unpack(CkptView in, int n, int c, long long spatial, int nhwc, float *x, cudaStream_t s);

}  // namespace vae
