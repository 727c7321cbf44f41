// tokens.cuh -- token rows in float32, bfloat16 or float16: the numbers of a row
// in memory (T) and in registers (packed pairs of floats, eight to an Oct).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ckpt.cuh"

namespace vae {

using bf16 = __nv_bfloat16;

// f(T{}) with the type that `dtype` names.
template <class F>
int by_dtype(int dtype, F &&f) {
  if (dtype == VAE_BF16) return f(bf16{});
  if (dtype == VAE_F16) return f(__half{});
  return f(float{});
}
inline bool dtype_ok(int dtype) {
  return dtype == VAE_F32 || dtype == VAE_BF16 || dtype == VAE_F16;
}
inline size_t dtype_bytes(int dtype) { return dtype == VAE_F32 ? 4 : 2; }

// Eight numbers as they lie in memory.
template <class T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};

__device__ __forceinline__ uint64_t unpack2(uint32_t w, bf16) {
  return pk2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint64_t unpack2(uint32_t w, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return pk2(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, bf16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <class T>
__device__ __forceinline__ Oct oct_of(const Raw<T> &r) {
  if constexpr (sizeof(T) == 4) {
    auto two = [](uint32_t a, uint32_t b) { return a | static_cast<uint64_t>(b) << 32; };
    return {{two(r.v[0].x, r.v[0].y), two(r.v[0].z, r.v[0].w), two(r.v[1].x, r.v[1].y),
             two(r.v[1].z, r.v[1].w)}};
  } else {
    return {{unpack2(r.v[0].x, T{}), unpack2(r.v[0].y, T{}), unpack2(r.v[0].z, T{}),
             unpack2(r.v[0].w, T{})}};
  }
}
template <class T>
__device__ __forceinline__ Raw<T> raw_of(const Oct &o) {
  Raw<T> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      r.v[h] = make_uint4(__float_as_uint(lo2(o.v[2 * h])), __float_as_uint(hi2(o.v[2 * h])),
                          __float_as_uint(lo2(o.v[2 * h + 1])),
                          __float_as_uint(hi2(o.v[2 * h + 1])));
  } else {
    r.v[0] = make_uint4(pack2(lo2(o.v[0]), hi2(o.v[0]), T{}), pack2(lo2(o.v[1]), hi2(o.v[1]), T{}),
                        pack2(lo2(o.v[2]), hi2(o.v[2]), T{}), pack2(lo2(o.v[3]), hi2(o.v[3]), T{}));
  }
  return r;
}

// The eight numbers at p, of which `left` (a multiple of four, or more than eight)
// are the row's; zeros for the others. WIDE: rows and pointers are aligned to
// eight numbers, and one access takes them (of 32 bytes for float: with two of 16
// the halves of a sector would pass L2 twice). Plain loads, in program order with
// the stores: an output may be the input.
template <class T, bool WIDE>
__device__ __forceinline__ Raw<T> load_raw(const T *p, int left) {
  Raw<T> r;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if constexpr (sizeof(T) == 4) {
    r.v[0] = r.v[1] = zero;
    if (WIDE) {
      if (left > 0)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.v[0].x), "=r"(r.v[0].y), "=r"(r.v[0].z), "=r"(r.v[0].w),
                       "=r"(r.v[1].x), "=r"(r.v[1].y), "=r"(r.v[1].z), "=r"(r.v[1].w)
                     : "l"(p)
                     : "memory");
      return r;
    }
    if (left > 0) r.v[0] = *reinterpret_cast<const uint4 *>(p);
    if (left > 4) r.v[1] = *reinterpret_cast<const uint4 *>(p + 4);
  } else {
    r.v[0] = zero;
    if (WIDE) {
      if (left > 0) r.v[0] = *reinterpret_cast<const uint4 *>(p);
      return r;
    }
    if (left > 0) {
      const uint2 a = *reinterpret_cast<const uint2 *>(p);
      r.v[0].x = a.x;
      r.v[0].y = a.y;
    }
    if (left > 4) {
      const uint2 b = *reinterpret_cast<const uint2 *>(p + 4);
      r.v[0].z = b.x;
      r.v[0].w = b.y;
    }
  }
  return r;
}
template <class T, bool WIDE>
__device__ __forceinline__ void store_raw(T *p, int left, const Raw<T> &r) {
  if constexpr (sizeof(T) == 4) {
    if (WIDE) {
      if (left > 0)
        asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r.v[0].x),
                     "r"(r.v[0].y), "r"(r.v[0].z), "r"(r.v[0].w), "r"(r.v[1].x), "r"(r.v[1].y),
                     "r"(r.v[1].z), "r"(r.v[1].w), "l"(p)
                     : "memory");
      return;
    }
    if (left > 0) *reinterpret_cast<uint4 *>(p) = r.v[0];
    if (left > 4) *reinterpret_cast<uint4 *>(p + 4) = r.v[1];
  } else {
    if (WIDE) {
      if (left > 0) *reinterpret_cast<uint4 *>(p) = r.v[0];
      return;
    }
    if (left > 0) *reinterpret_cast<uint2 *>(p) = make_uint2(r.v[0].x, r.v[0].y);
    if (left > 4) *reinterpret_cast<uint2 *>(p + 4) = make_uint2(r.v[0].z, r.v[0].w);
  }
}
// Whether rows of c numbers at these addresses take whole-oct accesses.
template <class T, class... P>
inline bool raw_wide(int c, P... p) {
  return c % 8 == 0 && ((reinterpret_cast<uintptr_t>(p) % (8 * sizeof(T)) == 0) && ...);
}

// Eight floats of a parameter row at channel ch, for a row of c (a multiple of
// four); `other` without one, zeros past c. 16-byte aligned.
__device__ __forceinline__ Oct param_oct(const float *p, int ch, int c, float other) {
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 o = make_float4(other, other, other, other);
  const float4 a = ch >= c ? zero : p ? __ldg(reinterpret_cast<const float4 *>(p + ch)) : o;
  const float4 b = ch + 4 >= c ? zero : p ? __ldg(reinterpret_cast<const float4 *>(p + ch + 4)) : o;
  return oct_of(a, b);
}

}  // namespace vae
