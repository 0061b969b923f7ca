// Shared by the trend-network operators (affine.cu, norm.cu, scan.cu): element types,
// activations, and the guards of their C entries.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <initializer_list>
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

// Number of SMs of the current device.
int sm_count();

// Lets a kernel have `bytes` of dynamic shared memory, the same number at every call: once per kernel (which `done`
// belongs to) and device, so that host threads do not take it from one another.  large_clusters: clusters of more than 8 too.
cr_status allow_shared(const void* kernel, int bytes, std::atomic<uint64_t>& done, bool large_clusters = false);

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

// Sizes of the operators end 2^16 before 2^31: indices that run past them by a tile, a warp or the step of a
// grid-wide loop stay below 2^31.
constexpr int MAXSIZE = 0x7fffffff - 0xffff;
#define CR_REQUIRE_SIZES(what, ...) \
  CR_REQUIRE(::cr::largest({__VA_ARGS__}) <= ::cr::MAXSIZE, what ": sizes end at 2^31 - 2^16")
inline int largest(std::initializer_list<int> sizes) {
  int m = 0;
  for (int s : sizes) m = s > m ? s : m;
  return m;
}

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

// Two neighbours at a time: one conversion instruction, where element by element each needs one and
// the halves have to be put together.
__device__ __forceinline__ float2 widen2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ float2 widen2(uint32_t w, __nv_bfloat16) {   // BF16 is the upper half of FP32
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, __nv_fp8_e4m3) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// 8 consecutive elements as they are in memory.
template <class T>
struct alignas(sizeof(T) == 1 ? 8 : 16) Eight {
  uint32_t w[2 * sizeof(T)];
};
template <class T>
__device__ __forceinline__ void widen8(const Eight<T>& p, float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = widen2(p.w[q], T{});
    v[2 * q] = f.x;
    v[2 * q + 1] = f.y;
  }
}
__device__ __forceinline__ void widen8(const Eight<float>& p, float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(p.w[q]);
}
template <class T>
__device__ __forceinline__ Eight<T> narrow8(const float* v) {
  Eight<T> p;
#pragma unroll
  for (int q = 0; q < 4; ++q) p.w[q] = narrow2(v[2 * q], v[2 * q + 1], T{});
  return p;
}
template <>
__device__ __forceinline__ Eight<__nv_fp8_e4m3> narrow8<__nv_fp8_e4m3>(const float* v) {
  Eight<__nv_fp8_e4m3> p;
#pragma unroll
  for (int q = 0; q < 2; ++q)
    p.w[q] = narrow2(v[4 * q], v[4 * q + 1], __nv_fp8_e4m3{}) | narrow2(v[4 * q + 2], v[4 * q + 3], __nv_fp8_e4m3{}) << 16;
  return p;
}
template <>
__device__ __forceinline__ Eight<float> narrow8<float>(const float* v) {
  Eight<float> p;
#pragma unroll
  for (int q = 0; q < 8; ++q) p.w[q] = __float_as_uint(v[q]);
  return p;
}

inline int type_bytes(int type) {
  return type == CR_TYPE_F32 ? 4 : type == CR_TYPE_E4M3 ? 1 : 2;
}

// Launches a kernel that may be set up (barriers, tensor memory, its first instructions) while the
// stream's previous kernel finishes, and calls wait_for_previous() before it touches memory.
template <class... Par, class... Arg>
cudaError_t launch_after(void (*kernel)(Par...), unsigned grid, unsigned block, size_t smem, int cluster, cudaStream_t stream, Arg&&... arg) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, Par(arg)...);
}

// Calls f(T{}) with the element type of `type`, one of FP32, FP16, BF16 (checked before).
template <class F>
cr_status with_type(int type, F&& f) {
  if (type == CR_TYPE_F32) return f(float{});
  if (type == CR_TYPE_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

// ---------------------------------------------------------------- one float, or two
// Products that feed a sum are written as fmaf or __fmul_rn, so that every variant of a kernel rounds alike.
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

// ---------------------------------------------------------------- activations
// Written from the hardware's 2^x and reciprocal (each within about 2^-22), because a product's
// epilogue shares the SM's issue slots and power with the MMAs: the K = 4096, N = 16384, M = 8192 BF16
// product with silu took 666 us with expf and 634 us with these.  Arguments are clamped where
// the function has reached its limit, so that infinities give limits; NaN stays.
__device__ __forceinline__ float clamp_low(float x, float low) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(low));
  return x;
}
__device__ __forceinline__ float clamp_high(float x, float high) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(high));
  return x;
}
__device__ __forceinline__ float exp2_fast(float x) {
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ float rcp_fast(float x) {
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
constexpr float LOG2E = 1.4426950408889634f;

template <int VEC>
__device__ __forceinline__ Floats<VEC> exp2_fast(Floats<VEC> x) {
#pragma unroll
  for (int q = 0; q < VEC; ++q) x.x[q] = exp2_fast(x.x[q]);
  return x;
}
template <int VEC>
__device__ __forceinline__ Floats<VEC> rcp_fast(Floats<VEC> x) {
#pragma unroll
  for (int q = 0; q < VEC; ++q) x.x[q] = rcp_fast(x.x[q]);
  return x;
}

// Phi(a) - 1 for a >= 0, and g = e^(-a^2 / 2): erfc by Hastings' rational-exponential formula (Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26; its coefficients here times -1/2), absolute error 7.5e-8.  t is the
// reciprocal of tail_denominator(a).
template <int VEC>
__device__ __forceinline__ Floats<VEC> tail_denominator(Floats<VEC> a) {
  return fma(a, all_of<VEC>(0.3275911f * 0.70710678118654752f), all_of<VEC>(1.0f));
}
template <int VEC>
__device__ __forceinline__ Floats<VEC> minus_tail(Floats<VEC> a, Floats<VEC> t, Floats<VEC>& g) {
  const auto k = [](float x) { return all_of<VEC>(x); };
  g = exp2_fast(mul(mul(a, a), k(-0.5f * LOG2E)));
  Floats<VEC> p = fma(t, k(-0.5f * 1.061405429f), k(0.5f * 1.453152027f));
  p = fma(t, p, k(-0.5f * 1.421413741f));
  p = fma(t, p, k(0.5f * 0.284496736f));
  p = fma(t, p, k(-0.5f * 0.254829592f));
  return mul(mul(t, p), g);
}
template <int VEC>
__device__ __forceinline__ Floats<VEC> minus_tail(Floats<VEC> a, Floats<VEC>& g) {
  return minus_tail(a, rcp_fast(tail_denominator(a)), g);
}

template <int ACT, int VEC>
__device__ __forceinline__ Floats<VEC> activate(Floats<VEC> z) {
  if (ACT == CR_ACT_RELU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) z.x[q] = clamp_low(z.x[q], 0.0f);
  }
  if (ACT == CR_ACT_SILU) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) z.x[q] = clamp_low(z.x[q], -88.0f);   // e^88 is finite, and its reciprocal flushed to 0
    return mul(z, rcp_fast(add(exp2_fast(mul(z, all_of<VEC>(-LOG2E))), all_of<VEC>(1.0f))));
  }
  if (ACT == CR_ACT_GELU) {   // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|))
    Floats<VEC> a, g;
#pragma unroll
    for (int q = 0; q < VEC; ++q) {
      a.x[q] = clamp_high(fabsf(z.x[q]), 30.0f);
      z.x[q] = clamp_low(z.x[q], 0.0f);
    }
    return fma(a, minus_tail(a, g), z);
  }
  return z;
}

template <int ACT>
__device__ __forceinline__ float activation_slope(float z) {
  if (ACT == CR_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if (ACT == CR_ACT_SILU) {
    z = clamp_high(clamp_low(z, -88.0f), 88.0f);
    const float e = exp2_fast(z * -LOG2E), p = rcp_fast(1.0f + e);
    return p * fmaf(z, e * p, 1.0f);
  }
  if (ACT == CR_ACT_GELU) {
    z = clamp_high(clamp_low(z, -30.0f), 30.0f);
    Floats<1> g;
    const float m = minus_tail(Floats<1>{{fabsf(z)}}, g).x[0];
    return fmaf(z * 0.39894228040143268f, g.x[0], z < 0.0f ? -m : 1.0f + m);
  }
  return 1.0f;
}

// v[] = act(v[]) with one test of `act` for all of them, two at a time.
template <int ACT, int N>
__device__ __forceinline__ void activate_each(float* v) {
  constexpr int VEC = N % 2 == 0 ? 2 : 1;
#pragma unroll
  for (int q = 0; q < N; q += VEC) {
    Floats<VEC> z;
#pragma unroll
    for (int x = 0; x < VEC; ++x) z.x[x] = v[q + x];
    z = activate<ACT, VEC>(z);
#pragma unroll
    for (int x = 0; x < VEC; ++x) v[q + x] = z.x[x];
  }
}
template <int N>
__device__ __forceinline__ void activate_all(float* v, int act) {
  if (act == CR_ACT_RELU) activate_each<CR_ACT_RELU, N>(v);
  else if (act == CR_ACT_SILU) activate_each<CR_ACT_SILU, N>(v);
  else if (act == CR_ACT_GELU) activate_each<CR_ACT_GELU, N>(v);
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
// h_t = a h_{t-1} + c x_t.
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
  Floats<VEC> e = mul(g, all_of<VEC>(-LOG2E));
#pragma unroll
  for (int q = 0; q < VEC; ++q) {
    e.x[q] = exp2_fast(clamp_high(e.x[q], 125.5f));
  }
  Floats<VEC> r = add(e, all_of<VEC>(1.0f));
#pragma unroll
  for (int q = 0; q < VEC; ++q) r.x[q] = rcp_fast(r.x[q]);
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
// h' da/dg + x dc/dg from a and c.  Convex gate: c = 1 - a.  Variance gate: 1 - a = c^2 / (1 + a) gives
// da/dg = a c^2 / (1 + a) and dc/dg = -a^2 c / (1 + a), finite at a = 1.
template <int GATE, int VEC>
__device__ __forceinline__ Floats<VEC> gate_slope(Floats<VEC> a, Floats<VEC> c, Floats<VEC> before, Floats<VEC> x) {
  if (GATE == CR_GATE_COEFF) return before;
  const Floats<VEC> minus = all_of<VEC>(-1.0f);
  if (GATE == CR_GATE_CONVEX) return mul(mul(a, c), fma(x, minus, before));
  Floats<VEC> r = add(a, all_of<VEC>(1.0f));
#pragma unroll
  for (int q = 0; q < VEC; ++q) r.x[q] = rcp_fast(r.x[q]);
  return mul(mul(mul(a, c), r), fma(before, c, mul(mul(x, minus), a)));
}

}  // namespace cr
