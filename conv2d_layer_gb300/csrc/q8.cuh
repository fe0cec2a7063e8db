// q8.cuh - element types of the residual block's kernels: 16-byte vectors,
// conversions, and the 8-bit format (e4m3 values, one power-of-two scale byte
// for each group of columns of a row).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

namespace c2d {

constexpr int kQ8Group = 32;  // columns that share a scale, when not a whole row

template <typename T>
__device__ __forceinline__ float to_f(T v) { return static_cast<float>(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
// Decoded values, clamped to T's largest finite one: e4m3 rounding may carry a value close to it up to the
// next power of two, which T does not hold. NaN passes.
template <typename T>
__device__ __forceinline__ T from_q8(float v) {
  constexpr float top = sizeof(T) == 4 ? 3.402823466e38f : (std::is_same<T, __half>::value ? 65504.f : 3.3895313892515355e38f);
  return from_f<T>(v > top ? top : (v < -top ? -top : v));
}

// The largest scale whose values (448 times it at most) T holds without clamping.
template <typename T>
__device__ __forceinline__ constexpr float q8_safe_scale() {
  return std::is_same<T, __half>::value ? 128.f : 6.6461399789245794e35f;  // 2^7, 2^119
}

// 32 bytes at once (32-byte aligned): a whole sector a thread.
__device__ __forceinline__ void ld_32b(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void st_32b(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// V consecutive elements; V * sizeof(T) = 32 or 16 bytes (aligned to as much) or V = 1.
template <typename T, int V>
__device__ __forceinline__ void ld_vec(const T* p, T (&e)[V]) {
  if constexpr (V == 1) {
    e[0] = *p;
  } else if constexpr (sizeof(T) * V == 32) {
    uint32_t w[8];
    ld_32b(p, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) reinterpret_cast<uint32_t*>(e)[i] = w[i];
  } else {
    static_assert(sizeof(T) * V == 16, "16- or 32-byte vectors");
    *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
  }
}
template <typename T, int V>
__device__ __forceinline__ void st_vec(T* p, const T (&e)[V]) {
  if constexpr (V == 1) {
    *p = e[0];
  } else if constexpr (sizeof(T) * V == 32) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = reinterpret_cast<const uint32_t*>(e)[i];
    st_32b(p, w);
  } else {
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
  }
}

// Magnitude bits of a finite value, 0 for infinities and NaN: ordered like the magnitudes.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// Scale byte (e + 127) of a group whose largest finite magnitude has these bits: the smallest e in
// [-126, 127] with amax <= 448 * 2^e, 448 = 1.75 * 2^8; e = 0 for an empty or zero group.
__device__ __forceinline__ uint32_t q8_scale_byte(uint32_t amax_bits) {
  if (amax_bits == 0u) return 127u;
  const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(e < 1 ? 1 : e);
}
__device__ __forceinline__ float q8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }  // 2^(byte - 127)
// The scale of byte b in two factors, which are applied before and after another scale: for a product's sum v (0, or
// 2^-18 to 2^46 in magnitude: e4m3 products, 2^28 of them at most) no step of v * f.x * q8_scale(a) * f.y overflows or
// underflows where the result does not (one after the other, 2^111 and 2^-125 took a sum of 2^18 to infinity). f.y is 1
// for scales of 2^-100 to 2^80; one beyond that comes in two halves of the same sign.
__device__ __forceinline__ float2 q8_factors(uint32_t b) {
  const uint32_t x = b < 27u ? 64u : (b > 207u ? 191u : b);
  return make_float2(q8_scale(x), q8_scale(b - x + 127u));
}
__device__ __forceinline__ float q8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// Two values, already divided by their scale, to e4m3 (a in the low byte). The conversion saturates, so
// an infinity is turned into NaN first: t * 0 + t.
__device__ __forceinline__ uint32_t q8_pack2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(__fmaf_rn(b, 0.f, b)), "f"(__fmaf_rn(a, 0.f, a)));
  return r;
}
// The same without infinities among the values (NaN converts to NaN).
__device__ __forceinline__ uint32_t q8_pack2_finite(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// The two e4m3 values of the low 16 bits.
__device__ __forceinline__ float2 q8_unpack2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t q8_pack4(const float* v, float inv, bool finite) {
  return finite ? q8_pack2_finite(v[0] * inv, v[1] * inv) | q8_pack2_finite(v[2] * inv, v[3] * inv) << 16
                : q8_pack2(v[0] * inv, v[1] * inv) | q8_pack2(v[2] * inv, v[3] * inv) << 16;
}
// Stores V e4m3 bytes of v[] * inv; finite: no infinity among them.
template <int V>
__device__ __forceinline__ void q8_store(uint8_t* p, const float (&v)[V], float inv, bool finite) {
  if constexpr (V == 1) {
    *p = static_cast<uint8_t>(q8_pack2(v[0] * inv, 0.f));
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(p) = q8_pack4(v, inv, finite);
  } else if constexpr (V == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(q8_pack4(v, inv, finite), q8_pack4(v + 4, inv, finite));
  } else {
    static_assert(V == 16, "V is 1, 4, 8 or 16");
    *reinterpret_cast<uint4*>(p) = make_uint4(q8_pack4(v, inv, finite), q8_pack4(v + 4, inv, finite),
                                              q8_pack4(v + 8, inv, finite), q8_pack4(v + 12, inv, finite));
  }
}
// V e4m3 bytes as they lie in memory, and their values times scale.
template <int V>
struct Q8Raw {
  uint32_t w[V < 4 ? 1 : V / 4];
};
template <int V>
__device__ __forceinline__ Q8Raw<V> q8_load(const uint8_t* p) {
  Q8Raw<V> r;
  if constexpr (V == 1) r.w[0] = *p;
  else if constexpr (V == 4) r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (V == 8) *reinterpret_cast<uint2*>(r.w) = *reinterpret_cast<const uint2*>(p);
  else *reinterpret_cast<uint4*>(r.w) = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <int V>
__device__ __forceinline__ void q8_values(const Q8Raw<V>& r, float (&v)[V], float scale) {
  if constexpr (V == 1) {
    v[0] = q8_unpack2(r.w[0]).x * scale;
  } else {
    const uint32_t* w = r.w;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = q8_unpack2(w[i / 2] >> (16 * (i & 1)));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
}

// ---------------------------------------------------------------- activations of the dense layer
// In fp32 to about 1e-6 relative (1e-5 where |z| is in the tens and the result tiny), in the forms that lose
// nothing near zero or in the tails: the outputs are rounded to 16 bits, but the bias gradient sums the
// derivatives in fp32.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2/pi)

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 rcp_2(float2 x) { return make_float2(rcp(x.x), rcp(x.y)); }
// x within [-b, b]; NaN passes.
__device__ __forceinline__ float clamp_nan(float x, float b) {
  float y;
  asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}" : "=f"(y) : "f"(x), "f"(b), "f"(-b));
  return y;
}
__device__ __forceinline__ float2 clamp_nan(float2 x, float b) { return make_float2(clamp_nan(x.x, b), clamp_nan(x.y, b)); }

// Two values at a time: the multiplications and additions go in packed f32x2 instructions.
template <int A>
__device__ __forceinline__ float2 dense_act(float2 z) {
  if constexpr (A == 1) {  // NaN passes
    return make_float2(z.x > 0.f ? z.x : (z.x <= 0.f ? 0.f : z.x), z.y > 0.f ? z.y : (z.y <= 0.f ? 0.f : z.y));
  } else if constexpr (A == 2) {
    // tanh z = z (1 - z^2/3 + 2 z^4/15 - 17 z^6/315) below 1/4 (the next term is under 4e-7 of z), else
    // (1 - e) / (1 + e) with e = exp(-2|z|) and z's sign
    const float2 a = make_float2(fabsf(z.x), fabsf(z.y)), s = __fmul2_rn(z, z);
    const float2 e = ex2_2(__fmul2_rn(a, splat(-2.f * kLog2e)));
    const float2 big = __fmul2_rn(__ffma2_rn(e, splat(-1.f), splat(1.f)), rcp_2(__fadd2_rn(e, splat(1.f))));
    float2 p = __ffma2_rn(s, splat(-17.f / 315.f), splat(2.f / 15.f));
    p = __ffma2_rn(s, p, splat(-1.f / 3.f));
    p = __fmul2_rn(z, __ffma2_rn(s, p, splat(1.f)));
    return make_float2(a.x < 0.25f ? p.x : copysignf(big.x, z.x), a.y < 0.25f ? p.y : copysignf(big.y, z.y));
  } else if constexpr (A == 3) {
    return rcp_2(__fadd2_rn(ex2_2(__fmul2_rn(z, splat(-kLog2e))), splat(1.f)));
  } else if constexpr (A == 4) {
    // z/2 (1 + tanh u) = z / (1 + exp(-2u)); past |z| = 16 the factor is 0 or 1 to fp32 (clamped, so that
    // u does not overflow)
    const float2 c = clamp_nan(z, 16.f);
    const float2 u = __fmul2_rn(c, __ffma2_rn(__fmul2_rn(c, c), splat(-kLog2e * kGelu2 * 0.044715f), splat(-kLog2e * kGelu2)));
    return __fmul2_rn(z, rcp_2(__fadd2_rn(ex2_2(u), splat(1.f))));
  } else if constexpr (A == 5) {
    return __fmul2_rn(z, rcp_2(__fadd2_rn(ex2_2(__fmul2_rn(z, splat(-kLog2e))), splat(1.f))));
  } else {
    return z;
  }
}
template <int A>
__device__ __forceinline__ float2 dense_dact(float2 z) {
  if constexpr (A == 1) {
    return make_float2(z.x > 0.f ? 1.f : (z.x <= 0.f ? 0.f : z.x), z.y > 0.f ? 1.f : (z.y <= 0.f ? 0.f : z.y));
  } else if constexpr (A == 2 || A == 3) {
    // tanh: 1 - tanh^2 = 4 e / (1 + e)^2, e = exp(-2|z|); sigmoid: s (1 - s) = e / (1 + e)^2, e = exp(-|z|)
    const float2 e = ex2_2(__fmul2_rn(make_float2(fabsf(z.x), fabsf(z.y)), splat(A == 2 ? -2.f * kLog2e : -kLog2e)));
    const float2 r = rcp_2(__fadd2_rn(e, splat(1.f)));
    return __fmul2_rn(__fmul2_rn(A == 2 ? __fmul2_rn(e, splat(4.f)) : e, r), r);
  } else if constexpr (A == 4 || A == 5) {
    // s + z s (1 - s) w, w = d(2u)/dz (gelu) or 1 (silu)
    const float2 c = clamp_nan(z, A == 4 ? 16.f : 88.f);
    float2 u, w;
    if constexpr (A == 4) {
      const float2 q = __fmul2_rn(c, c);
      u = __fmul2_rn(c, __ffma2_rn(q, splat(-kLog2e * kGelu2 * 0.044715f), splat(-kLog2e * kGelu2)));
      w = __fmul2_rn(c, __ffma2_rn(q, splat(3.f * 0.044715f * kGelu2), splat(kGelu2)));
    } else {
      u = __fmul2_rn(c, splat(-kLog2e));
      w = c;
    }
    const float2 s = rcp_2(__fadd2_rn(ex2_2(u), splat(1.f)));
    return __ffma2_rn(__fmul2_rn(s, w), __ffma2_rn(s, splat(-1.f), splat(1.f)), s);
  } else {
    return splat(1.f);
  }
}
template <int A>
struct DAct {
  static constexpr int value = A;
};
template <typename F>
__device__ __forceinline__ void with_dense_act(int act, F&& f) {
  switch (act) {
    case 1: f(DAct<1>{}); break;
    case 2: f(DAct<2>{}); break;
    case 3: f(DAct<3>{}); break;
    case 4: f(DAct<4>{}); break;
    case 5: f(DAct<5>{}); break;
    default: f(DAct<0>{}); break;
  }
}

}  // namespace c2d
