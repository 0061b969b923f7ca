// Root-mean-square norm of columns with the residual's addition and an optional e4m3 output,
// and its gradient (cr_rmsnorm, cr_rmsnorm_backward).
#include <type_traits>

#include "ops.cuh"

namespace cr {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) s += red[w];
  return s;
}
// maximum that keeps NaN
__device__ __forceinline__ float nan_max(float a, float b) { return (a != a || a > b) ? a : b; }
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = nan_max(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) s = nan_max(s, red[w]);
  return s;
}

// One block per column, the column read once for each of its reductions.
template <class T, class O>
__global__ void __launch_bounds__(NT) k_rmsnorm(const T* X, int ldx, const T* R, int ldr, const float* gamma, int D,
                                                float eps, T* H, int ldh, O* Y, int ldy, float* scale) {
  __shared__ float red[NT / 32];
  const size_t t = blockIdx.x;
  const T* x = X + t * ldx;
  const T* r = R ? R + t * ldr : nullptr;
  float ss = 0.0f;
  for (int i = threadIdx.x; i < D; i += NT) {
    const float h = to_float(x[i]) + (r ? to_float(r[i]) : 0.0f);
    ss = fmaf(h, h, ss);
  }
  const float rs = 1.0f / sqrtf(block_sum(ss, red) / (float)D + eps);
  float inv = 1.0f;
  if (std::is_same<O, __nv_fp8_e4m3>::value) {
    float mx = 0.0f;
    for (int i = threadIdx.x; i < D; i += NT) {
      const float h = to_float(x[i]) + (r ? to_float(r[i]) : 0.0f);
      mx = nan_max(fabsf(h * rs * gamma[i]), mx);
    }
    mx = block_max(mx, red);
    const float s = nan_max(mx, 0x1p-100f) / 448.0f;
    if (threadIdx.x == 0) scale[t] = s;
    inv = 1.0f / s;
  }
  for (int i = threadIdx.x; i < D; i += NT) {
    const float h = to_float(x[i]) + (r ? to_float(r[i]) : 0.0f);
    Y[t * ldy + i] = from_float<O>(h * rs * gamma[i] * inv);
    if (H) H[t * ldh + i] = from_float<T>(h);
  }
}

template <class T>
__global__ void __launch_bounds__(NT) k_rmsnorm_dx(const T* H, int ldh, const float* gamma, const T* dY, int lddy,
                                                   const T* dH, int lddh, int D, float eps, T* dX, int lddx, float* rs_out) {
  __shared__ float red[NT / 32];
  const size_t t = blockIdx.x;
  float ss = 0.0f, dot = 0.0f;
  for (int i = threadIdx.x; i < D; i += NT) {
    const float h = to_float(H[t * ldh + i]);
    ss = fmaf(h, h, ss);
    dot = fmaf(__fmul_rn(gamma[i], to_float(dY[t * lddy + i])), h, dot);
  }
  const float rs = 1.0f / sqrtf(block_sum(ss, red) / (float)D + eps);
  const float m = block_sum(dot, red) / (float)D * rs * rs * rs;
  if (threadIdx.x == 0) rs_out[t] = rs;
  if (!dX) return;
  for (int i = threadIdx.x; i < D; i += NT) {
    const float h = to_float(H[t * ldh + i]);
    float d = fmaf(-h, m, __fmul_rn(rs, __fmul_rn(gamma[i], to_float(dY[t * lddy + i]))));
    if (dH) d += to_float(dH[t * lddh + i]);
    dX[t * lddx + i] = from_float<T>(d);
  }
}

template <class T>
__global__ void __launch_bounds__(NT) k_rmsnorm_dgamma(const T* H, int ldh, const T* dY, int lddy, const float* rs, int D,
                                                       int T_, float* dgamma) {
  const int i = blockIdx.x * NT + threadIdx.x;
  if (i >= D) return;
  float s = 0.0f;
  for (size_t t = 0; t < (size_t)T_; ++t) s = fmaf(__fmul_rn(to_float(dY[t * lddy + i]), to_float(H[t * ldh + i])), rs[t], s);
  dgamma[i] = s;
}

bool float_type(int t) { return t == CR_TYPE_F32 || t == CR_TYPE_F16 || t == CR_TYPE_BF16; }

}  // namespace
}  // namespace cr

using namespace cr;

extern "C" cr_status cr_rmsnorm(int type, const void* d_X, int ldx, const void* d_R, int ldr, const float* d_gamma, int D,
                                int T, double eps, void* d_H, int ldh, int out_type, void* d_Y, int ldy, float* d_scale,
                                cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(float_type(type), "cr_rmsnorm: type must be FP32, FP16 or BF16");
  CR_REQUIRE(out_type == type || out_type == CR_TYPE_E4M3, "cr_rmsnorm: out_type must be type or e4m3");
  CR_REQUIRE(D >= 1 && T >= 0, "cr_rmsnorm: D >= 1, T >= 0");
  CR_REQUIRE(eps >= 0.0 && eps < 1e30, "cr_rmsnorm: eps must be finite and not negative");
  CR_REQUIRE(ldx >= D && ldy >= D && (!d_R || ldr >= D) && (!d_H || ldh >= D), "cr_rmsnorm: leading dimension below D");
  CR_REQUIRE((out_type == CR_TYPE_E4M3) == (d_scale != nullptr) || T == 0, "cr_rmsnorm: d_scale belongs to the e4m3 output");
  if (T == 0) return CR_OK;
  CR_REQUIRE(d_X && d_gamma && d_Y, "cr_rmsnorm: NULL argument");
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    if (out_type == CR_TYPE_E4M3)
      k_rmsnorm<E, __nv_fp8_e4m3><<<T, NT, 0, stream>>>((const E*)d_X, ldx, (const E*)d_R, ldr, d_gamma, D, (float)eps, (E*)d_H,
                                                        ldh, (__nv_fp8_e4m3*)d_Y, ldy, d_scale);
    else
      k_rmsnorm<E, E><<<T, NT, 0, stream>>>((const E*)d_X, ldx, (const E*)d_R, ldr, d_gamma, D, (float)eps, (E*)d_H, ldh,
                                            (E*)d_Y, ldy, nullptr);
    CR_CHECK_LAUNCH("k_rmsnorm");
    return CR_OK;
  });
  CR_ENTRY_END("cr_rmsnorm")
}

extern "C" cr_status cr_rmsnorm_backward(int type, const void* d_H, int ldh, const float* d_gamma, const void* d_dY, int lddy,
                                         const void* d_dH, int lddh, int D, int T, double eps, void* d_dX, int lddx,
                                         float* d_dgamma, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(float_type(type), "cr_rmsnorm_backward: type must be FP32, FP16 or BF16");
  CR_REQUIRE(D >= 1 && T >= 0, "cr_rmsnorm_backward: D >= 1, T >= 0");
  CR_REQUIRE(eps >= 0.0 && eps < 1e30, "cr_rmsnorm_backward: eps must be finite and not negative");
  CR_REQUIRE(ldh >= D && lddy >= D && (!d_dH || lddh >= D) && (!d_dX || lddx >= D),
             "cr_rmsnorm_backward: leading dimension below D");
  if (T == 0) {
    if (d_dgamma) CR_CUDA(cudaMemsetAsync(d_dgamma, 0, (size_t)D * sizeof(float), stream));
    return CR_OK;
  }
  CR_REQUIRE(d_H && d_gamma && d_dY, "cr_rmsnorm_backward: NULL argument");
  float* rs = nullptr;
  CR_CUDA(scratch_alloc((void**)&rs, (size_t)T * sizeof(float), stream));
  const cr_status st = with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    // dgamma first: dX may overwrite dY, so the columns' r are found without writing dX, then dX
    k_rmsnorm_dx<E><<<T, NT, 0, stream>>>((const E*)d_H, ldh, d_gamma, (const E*)d_dY, lddy, nullptr, 0, D, (float)eps, nullptr, 0, rs);
    CR_CHECK_LAUNCH("k_rmsnorm_dx");
    if (d_dgamma) {
      k_rmsnorm_dgamma<E><<<(D + NT - 1) / NT, NT, 0, stream>>>((const E*)d_H, ldh, (const E*)d_dY, lddy, rs, D, T, d_dgamma);
      CR_CHECK_LAUNCH("k_rmsnorm_dgamma");
    }
    if (d_dX) {
      k_rmsnorm_dx<E><<<T, NT, 0, stream>>>((const E*)d_H, ldh, d_gamma, (const E*)d_dY, lddy, (const E*)d_dH, lddh, D,
                                            (float)eps, (E*)d_dX, lddx, rs);
      CR_CHECK_LAUNCH("k_rmsnorm_dx");
    }
    return CR_OK;
  });
  scratch_free(rs, stream);
  return st;
  CR_ENTRY_END("cr_rmsnorm_backward")
}
