// Shared by the trend-network operators (affine.cu, norm.cu, scan.cu): element types,
// activations, and the guards of their C entries.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <new>

#include "common.cuh"

namespace cr {

cr_status fail_literal(cr_status code, const char* msg);

// Sticky word in mapped host memory that a kernel sets when one of its bounded waits runs out;
// the next operator call reports and clears it.  Reading it costs no synchronisation.
cr_status wait_word(int** d_word);

// Tensor map of a 2-D operand (inner contiguous, leading dimension ld) for 128-byte swizzled boxes.
cr_status make_tensor_map_2d(CUtensorMap* tm, int type, const void* base, int inner, int outer, int ld, int box_inner,
                             int box_outer);

// The same without a swizzle, for tiles that threads read.
cr_status make_tensor_map_2d_plain(CUtensorMap* tm, int type, const void* base, int inner, int outer, int ld, int box_inner,
                                   int box_outer);

// total[D] = the sum of the rows of part (rows x D, row-major), in a fixed order.
cr_status add_rows(const float* part, int rows, int D, float* total, cudaStream_t stream);

// C++ exceptions end at the C entries.
#define CR_ENTRY_BEGIN try {
#define CR_ENTRY_END(what)                                                                    \
  }                                                                                           \
  catch (const std::bad_alloc&) { return ::cr::fail_literal(CR_ERR_NOMEM, what ": host memory"); } \
  catch (...) { return ::cr::fail_literal(CR_ERR_STATE, what ": unexpected host exception"); }

#define CR_REQUIRE(cond, msg) \
  do {                        \
    if (!(cond)) return ::cr::fail_literal(CR_ERR_ARG, msg); \
  } while (0)

// ---------------------------------------------------------------- element types
template <class T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_float<__nv_fp8_e4m3>(__nv_fp8_e4m3 x) { return float(x); }

template <class T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __nv_fp8_e4m3 from_float<__nv_fp8_e4m3>(float x) { return __nv_fp8_e4m3(x); }

inline int type_bytes(int type) {
  return type == CR_TYPE_F32 ? 4 : type == CR_TYPE_E4M3 ? 1 : 2;
}

// Calls f(T{}) with the element type of `type`, one of FP32, FP16, BF16 (checked before).
template <class F>
cr_status with_type(int type, F&& f) {
  if (type == CR_TYPE_F32) return f(float{});
  if (type == CR_TYPE_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

// ---------------------------------------------------------------- activations
// e = exp(-|x|) never overflows; sigmoid of both signs without cancellation.
__device__ __forceinline__ void sigmoid_pair(float x, float& p, float& q) {   // p = sigmoid(x), q = sigmoid(-x)
  const float e = expf(-fabsf(x));
  const float big = __fdividef(1.0f, 1.0f + e), small = e * big;
  p = x >= 0.0f ? big : small;
  q = x >= 0.0f ? small : big;
  if (x != x) p = q = x;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == CR_ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays
  if (ACT == CR_ACT_SILU) {
    // z e^z -> -0 as z -> -inf, where z sigmoid(z) would be inf * 0
    float p, q;
    sigmoid_pair(z, p, q);
    return z == -INFINITY ? -0.0f : z * p;
  }
  if (ACT == CR_ACT_GELU) return z == -INFINITY ? -0.0f : 0.5f * z * erfcf(-z * 0.70710678118654752f);
  return z;
}

template <int ACT>
__device__ __forceinline__ float activation_slope(float z) {
  if (ACT == CR_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if (ACT == CR_ACT_SILU) {
    float p, q;
    sigmoid_pair(z, p, q);
    return fabsf(z) == INFINITY ? p : p * fmaf(z, q, 1.0f);
  }
  if (ACT == CR_ACT_GELU) {
    const float cdf = 0.5f * erfcf(-z * 0.70710678118654752f);
    return fabsf(z) == INFINITY ? cdf : fmaf(z * 0.39894228040143268f, expf(-0.5f * z * z), cdf);
  }
  return 1.0f;
}

// v[] = act(v[]) with one test of `act` for all of them.
template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  if (act == CR_ACT_RELU) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = activate<CR_ACT_RELU>(v[q]);
  } else if (act == CR_ACT_SILU) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = activate<CR_ACT_SILU>(v[q]);
  } else if (act == CR_ACT_GELU) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = activate<CR_ACT_GELU>(v[q]);
  }
}

template <class F>
cr_status with_act(int act, F&& f) {
  switch (act) {
    case CR_ACT_RELU: return f(std::integral_constant<int, CR_ACT_RELU>{});
    case CR_ACT_SILU: return f(std::integral_constant<int, CR_ACT_SILU>{});
    case CR_ACT_GELU: return f(std::integral_constant<int, CR_ACT_GELU>{});
    default: return f(std::integral_constant<int, CR_ACT_NONE>{});
  }
}

// ---------------------------------------------------------------- gates
// h_t = a h_{t-1} + c x_t.  Products that feed a sum are written as fmaf or __fmul_rn, so that every
// variant of a kernel rounds alike.
template <int VEC>
struct alignas(4 * VEC) Floats {   // one float, or two in the halves of a register pair
  float x[VEC];
};
__device__ __forceinline__ uint64_t pair_of(const Floats<2>& v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x[0]), "f"(v.x[1]));
  return r;
}
__device__ __forceinline__ Floats<2> floats_of(uint64_t p) {
  Floats<2> v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x[0]), "=f"(v.x[1]) : "l"(p));
  return v;
}
// Rounded to nearest, two at a time in one instruction.
__device__ __forceinline__ Floats<1> mul(Floats<1> a, Floats<1> b) { return {{__fmul_rn(a.x[0], b.x[0])}}; }
__device__ __forceinline__ Floats<1> add(Floats<1> a, Floats<1> b) { return {{__fadd_rn(a.x[0], b.x[0])}}; }
__device__ __forceinline__ Floats<1> fma(Floats<1> a, Floats<1> b, Floats<1> c) { return {{fmaf(a.x[0], b.x[0], c.x[0])}}; }
__device__ __forceinline__ Floats<2> mul(Floats<2> a, Floats<2> b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)));
  return floats_of(r);
}
__device__ __forceinline__ Floats<2> add(Floats<2> a, Floats<2> b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)));
  return floats_of(r);
}
__device__ __forceinline__ Floats<2> fma(Floats<2> a, Floats<2> b, Floats<2> c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)), "l"(pair_of(c)));
  return floats_of(r);
}
template <int VEC>
__device__ __forceinline__ Floats<VEC> all_of(float x) {
  Floats<VEC> v;
#pragma unroll
  for (int q = 0; q < VEC; ++q) v.x[q] = x;
  return v;
}

template <int VEC>
struct GateParts {
  Floats<VEC> a, rest;   // sigmoid(g) and sigmoid(-g); coefficient gate: g and 1
};
// sigmoid(g) = 1 / (1 + e^-g) and sigmoid(-g) = e^-g / (1 + e^-g), which has no cancellation.  e^-g is kept
// below 2^125.5 so that it stays finite (sigmoid(g) is then 1e-38); NaN stays.  The hardware's 2^x
// and reciprocal err by about 2^-22, and g log2(e) rounds to 2^-24 of itself: 2^-20 in all for |g| < 16.
template <int GATE, int VEC>
__device__ __forceinline__ GateParts<VEC> gate_parts(Floats<VEC> g) {
  if (GATE == CR_GATE_COEFF) return {g, all_of<VEC>(1.0f)};
  Floats<VEC> e = mul(g, all_of<VEC>(-1.4426950408889634f));
#pragma unroll
  for (int q = 0; q < VEC; ++q) {
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(e.x[q]) : "f"(125.5f));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x[q]));
  }
  Floats<VEC> r = add(e, all_of<VEC>(1.0f));
#pragma unroll
  for (int q = 0; q < VEC; ++q) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r.x[q]));
  return {r, mul(e, r)};
}
template <int VEC>
__device__ __forceinline__ Floats<VEC> sqrt_of(Floats<VEC> v) {
#pragma unroll
  for (int q = 0; q < VEC; ++q) asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(v.x[q]));
  return v;
}
template <int GATE, int VEC>
__device__ __forceinline__ Floats<VEC> gate_input(const GateParts<VEC>& p) {   // c; 1 - a^2 = rest (1 + a)
  return GATE == CR_GATE_VARIANCE ? sqrt_of(mul(p.rest, add(p.a, all_of<VEC>(1.0f)))) : p.rest;
}
// h' da/dg + x dc/dg.  Variance gate: dc/dg = -a (a rest) / c = -a^2 sqrt(rest / (1 + a)), finite at a = 1.
template <int GATE, int VEC>
__device__ __forceinline__ Floats<VEC> gate_slope(const GateParts<VEC>& p, Floats<VEC> before, Floats<VEC> x) {
  if (GATE == CR_GATE_COEFF) return before;
  const Floats<VEC> minus = all_of<VEC>(-1.0f);
  if (GATE == CR_GATE_CONVEX) return mul(mul(p.a, p.rest), fma(x, minus, before));
  Floats<VEC> s = add(p.a, all_of<VEC>(1.0f));
#pragma unroll
  for (int q = 0; q < VEC; ++q) s.x[q] = __fdividef(p.rest.x[q], s.x[q]);
  return mul(p.a, fma(before, p.rest, mul(mul(mul(x, minus), p.a), sqrt_of(s))));
}

}  // namespace cr
