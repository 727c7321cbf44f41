// linear_epilogue.cuh -- what follows a linear layer's sums: bias, activation and
// residual, or the derivative of the activation before it.
#pragma once
#include "gn_train.cuh"
#include "linear.cuh"
#include "tokens.cuh"

namespace vae {

// What becomes of a sum: KIND of an activation, or of its derivative at aux.
enum Kind { kNone, kSilu, kGelu, kSiluSlope, kGeluSlope };
inline int kind_of(const GemmEpilogue &e) {
  if (e.act == VAE_ACT_NONE) return kNone;
  const bool silu = e.act == VAE_ACT_SILU;
  return e.derivative ? (silu ? kSiluSlope : kGeluSlope) : (silu ? kSilu : kGelu);
}
// f(integral_constant) with the launch's kind: one branch around a block of results,
// where branches in it cost a third of a tile's time.
template <class F>
__device__ __forceinline__ void by_kind(int kind, F &&f) {
  switch (kind) {
    case kSilu: return f(std::integral_constant<int, kSilu>{});
    case kGelu: return f(std::integral_constant<int, kGelu>{});
    case kSiluSlope: return f(std::integral_constant<int, kSiluSlope>{});
    case kGeluSlope: return f(std::integral_constant<int, kGeluSlope>{});
    default: return f(std::integral_constant<int, kNone>{});
  }
}

// max and min that give a NaN for one.
__device__ __forceinline__ uint64_t at_least2(uint64_t z, float low) {
  float a, b;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(lo2(z)), "f"(low));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(hi2(z)), "f"(low));
  return pk2(a, b);
}
__device__ __forceinline__ uint64_t at_most2(uint64_t z, float high) {
  float a, b;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(lo2(z)), "f"(high));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(b) : "f"(hi2(z)), "f"(high));
  return pk2(a, b);
}

// The activations are z sigmoid(v), v = z for SiLU and z (a + b z^2) for GELU in its
// tanh form, a = sqrt(8 / pi), b = 0.044715 a. Beyond kFar both they and their
// derivatives are, to far below float's resolution, what they are there on the
// negative side (sigmoid 1e-38), and z and 1 on the positive one; z is held inside
// (activations: on the negative side), so that no product of a large and a vanishing
// number is formed. A NaN stays one.
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.071354816f;
template <int KIND>
constexpr bool is_gelu = KIND == kGelu || KIND == kGeluSlope;
template <int KIND>
constexpr float kFar = is_gelu<KIND> ? 10.f : 87.f;
// s = 1 / (1 + e) with e = e^-v, for v >= -87.4, by the exp2 and reciprocal units, to
// 2^-21 and the rounding of v log2 e (2^-23 |v|), which PRECISE puts back for results
// that are floats (v at most 128 there: the rest of an infinite product is a NaN, and
// e is 0 long before). (The reciprocal by Newton steps from an integer seed instead, for a
// unit that takes a warp eight clocks: 33 us instead of 31 for 16384 x 512 -> 2048.)
template <bool PRECISE>
__device__ __forceinline__ uint64_t sigmoid_of(uint64_t v, uint64_t *e) {
  const uint64_t t = mul2(v, pk2(-1.4426950408889634f, -1.4426950408889634f));
  *e = pk2(ex2_approx(lo2(t)), ex2_approx(hi2(t)));
  if constexpr (PRECISE) {  // e^-v = 2^t (1 - w)
    const uint64_t w = fma2(t, pk2(0.6931471805599453f, 0.6931471805599453f), v);
    *e = fma2(mul2(*e, w), pk2(-1.f, -1.f), *e);
  }
  return rcp2(add2(*e, pk2(1.f, 1.f)));
}
template <int KIND, bool PRECISE>
__device__ __forceinline__ uint64_t act2(uint64_t z) {
  const uint64_t h = at_least2(z, -kFar<KIND>);
  uint64_t v = h, e;
  if (is_gelu<KIND>)
    v = mul2(h, fma2(mul2(h, h), pk2(kGeluB, kGeluB), pk2(kGeluA, kGeluA)));
  if (PRECISE) v = at_most2(v, 128.f);
  return mul2(h, sigmoid_of<PRECISE>(v, &e));
}
// act'(z) = s + z v' s (1 - s), with 1 - s = e s, which loses nothing where s is near 1.
template <int KIND, bool PRECISE>
__device__ __forceinline__ uint64_t act_slope2(uint64_t z) {
  const uint64_t h = at_most2(at_least2(z, -kFar<KIND>), kFar<KIND>);
  uint64_t v = h, w = h, e;  // w = z v'
  if (is_gelu<KIND>) {
    const uint64_t q = mul2(h, h), a = pk2(kGeluA, kGeluA);
    v = mul2(h, fma2(q, pk2(kGeluB, kGeluB), a));
    w = mul2(h, fma2(q, pk2(3.f * kGeluB, 3.f * kGeluB), a));
  }
  const uint64_t s = sigmoid_of<PRECISE>(v, &e);
  return mul2(s, fma2(w, mul2(e, s), pk2(1.f, 1.f)));
}

// Two neighbouring sums of a row -> out, and z.
template <int KIND, bool PRECISE>
__device__ __forceinline__ uint64_t finish2(uint64_t sum, uint64_t bias, uint64_t aux,
                                            uint64_t *z) {
  if constexpr (KIND == kSiluSlope || KIND == kGeluSlope) {
    return mul2(sum, act_slope2<KIND, PRECISE>(aux));
  } else {
    *z = add2(sum, bias);
    if constexpr (KIND == kNone) return add2(*z, aux);
    else return add2(act2<KIND, PRECISE>(*z), aux);
  }
}

// Four numbers of type T, as two pairs.
struct Quad {
  uint64_t v[2];
};
template <class T>
__device__ __forceinline__ Quad load_quad(const T *p) {
  if constexpr (sizeof(T) == 4) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    return {{pk2(f.x, f.y), pk2(f.z, f.w)}};
  } else {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return {{unpack2(u.x, T{}), unpack2(u.y, T{})}};
  }
}
template <class T>
__device__ __forceinline__ void store_quad(T *p, const Quad &q) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4 *>(p) =
        make_float4(lo2(q.v[0]), hi2(q.v[0]), lo2(q.v[1]), hi2(q.v[1]));
  else
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(pack2(lo2(q.v[0]), hi2(q.v[0]), T{}), pack2(lo2(q.v[1]), hi2(q.v[1]), T{}));
}

}  // namespace vae
