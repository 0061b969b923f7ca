// Gated recurrence along time over packed series, its gradient and its single step
// (cr_gated_scan, cr_gated_scan_backward, cr_gated_step).
#include <type_traits>

#include "ops.cuh"

namespace cr {
namespace {

constexpr int NT = 128;
constexpr int BLOCK = 64;   // steps between saved states

struct Series {
  int beg, end;
};
// Column range of series s, clamped so that a bad offset stays in bounds.
__device__ __forceinline__ Series series_of(const int32_t* off, int s, int T) {
  if (!off) return {0, T};
  const int b = min(max(off[s], 0), T), e = min(max(off[s + 1], b), T);
  return {b, e};
}

// One thread per feature and series, step by step.
template <class T, int GATE>
__global__ void __launch_bounds__(NT) k_scan_fwd(const T* G, int ldg, const T* X, int ldx, int D, int n, const int32_t* off,
                                                 const float* h0, int ldh0, T* H, int ldh, float* hT, int ldhT, float* saved) {
  const int d = blockIdx.x * NT + threadIdx.x;
  if (d >= D) return;
  const Series sr = series_of(off, blockIdx.y, n);
  float h = h0 ? h0[(size_t)blockIdx.y * ldh0 + d] : 0.0f;
  for (int t = sr.beg; t < sr.end; ++t) {
    if (saved && t % BLOCK == 0) saved[(size_t)(t / BLOCK) * D + d] = h;
    const Gate g = gate_of<GATE>(to_float(G[(size_t)t * ldg + d]));
    h = fmaf(g.a, h, __fmul_rn(g.c, to_float(X[(size_t)t * ldx + d])));
    if (H) H[(size_t)t * ldh + d] = from_float<T>(h);
  }
  if (hT) hT[(size_t)blockIdx.y * ldhT + d] = h;
}

// Backwards, block by block: the states inside a block are recomputed from the saved one.
template <class T, int GATE>
__global__ void __launch_bounds__(NT) k_scan_bwd(const T* G, int ldg, const T* X, int ldx, const T* dH, int lddh, int D, int n,
                                                 const int32_t* off, const float* h0, int ldh0, const float* dhT, int lddhT,
                                                 const float* saved, T* dG, int lddg, T* dX, int lddx, float* dh0, int lddh0) {
  const int d = blockIdx.x * NT + threadIdx.x;
  if (d >= D) return;
  const Series sr = series_of(off, blockIdx.y, n);
  float carry = dhT ? dhT[(size_t)blockIdx.y * lddhT + d] : 0.0f;
  float prev[BLOCK];
  for (int hi = sr.end; hi > sr.beg;) {
    const int lo = max(sr.beg, (hi - 1) / BLOCK * BLOCK);
    float h = lo % BLOCK == 0 && lo > sr.beg ? saved[(size_t)(lo / BLOCK) * D + d]
                                             : (h0 ? h0[(size_t)blockIdx.y * ldh0 + d] : 0.0f);
    for (int t = lo; t < hi; ++t) {
      prev[t - lo] = h;
      const Gate g = gate_of<GATE>(to_float(G[(size_t)t * ldg + d]));
      h = fmaf(g.a, h, __fmul_rn(g.c, to_float(X[(size_t)t * ldx + d])));
    }
    for (int t = hi - 1; t >= lo; --t) {
      const float gl = to_float(G[(size_t)t * ldg + d]), x = to_float(X[(size_t)t * ldx + d]);
      const Gate g = gate_of<GATE>(gl), sl = gate_slope<GATE>(gl);
      const float q = __fadd_rn(to_float(dH[(size_t)t * lddh + d]), carry);
      if (dX) dX[(size_t)t * lddx + d] = from_float<T>(__fmul_rn(g.c, q));
      if (dG) dG[(size_t)t * lddg + d] = from_float<T>(__fmul_rn(q, fmaf(prev[t - lo], sl.a, __fmul_rn(x, sl.c))));
      carry = __fmul_rn(g.a, q);
    }
    hi = lo;
  }
  if (dh0) dh0[(size_t)blockIdx.y * lddh0 + d] = carry;
}

template <class T, int GATE>
__global__ void __launch_bounds__(NT) k_scan_step(const T* G, int ldg, const T* X, int ldx, const float* h, int ldh, int D, T* H,
                                                  int ldo, float* hn, int ldn) {
  const int d = blockIdx.x * NT + threadIdx.x;
  if (d >= D) return;
  const size_t b = blockIdx.y;
  const Gate g = gate_of<GATE>(to_float(G[b * ldg + d]));
  const float v = fmaf(g.a, h[b * ldh + d], __fmul_rn(g.c, to_float(X[b * ldx + d])));
  hn[b * ldn + d] = v;
  if (H) H[b * ldo + d] = from_float<T>(v);
}

bool float_type(int t) { return t == CR_TYPE_F32 || t == CR_TYPE_F16 || t == CR_TYPE_BF16; }

template <class F>
cr_status with_gate(int gate, F&& f) {
  switch (gate) {
    case CR_GATE_COEFF: return f(std::integral_constant<int, CR_GATE_COEFF>{});
    case CR_GATE_CONVEX: return f(std::integral_constant<int, CR_GATE_CONVEX>{});
    default: return f(std::integral_constant<int, CR_GATE_VARIANCE>{});
  }
}

}  // namespace
}  // namespace cr

using namespace cr;

extern "C" cr_status cr_gated_scan_saved(int D, int T, size_t* count) {
  CR_REQUIRE(D >= 1 && T >= 0 && count, "cr_gated_scan_saved: D >= 1, T >= 0, count");
  *count = (size_t)D * (size_t)(((long long)T + BLOCK - 1) / BLOCK);
  return CR_OK;
}

extern "C" cr_status cr_gated_scan(int type, int gate, const void* d_G, int ldg, const void* d_X, int ldx, int D, int T,
                                   const int32_t* d_off, int n_seq, const float* d_h0, int ldh0, void* d_H, int ldh,
                                   float* d_hT, int ldhT, float* d_saved, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(float_type(type), "cr_gated_scan: type must be FP32, FP16 or BF16");
  CR_REQUIRE(gate >= CR_GATE_COEFF && gate <= CR_GATE_VARIANCE, "cr_gated_scan: unknown gate");
  CR_REQUIRE(D >= 1 && T >= 0 && n_seq >= 0 && n_seq <= 65535, "cr_gated_scan: D >= 1, T >= 0, 0 <= n_seq <= 65535");
  CR_REQUIRE(d_off || n_seq == 1, "cr_gated_scan: without offsets there is one series");
  CR_REQUIRE(n_seq > 0 || T == 0, "cr_gated_scan: columns without a series");
  CR_REQUIRE((T == 0 || (d_G && d_X && ldg >= D && ldx >= D)) && (!d_H || ldh >= D), "cr_gated_scan: NULL argument or leading dimension below D");
  CR_REQUIRE((!d_h0 || ldh0 >= D) && (!d_hT || ldhT >= D), "cr_gated_scan: leading dimension below D");
  if (n_seq == 0) return CR_OK;
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    return with_gate(gate, [&](auto g0) -> cr_status {
      k_scan_fwd<E, decltype(g0)::value><<<dim3((D + NT - 1) / NT, n_seq), NT, 0, stream>>>(
          (const E*)d_G, ldg, (const E*)d_X, ldx, D, T, d_off, d_h0, ldh0, (E*)d_H, ldh, d_hT, ldhT, d_saved);
      CR_CHECK_LAUNCH("k_scan_fwd");
      return CR_OK;
    });
  });
  CR_ENTRY_END("cr_gated_scan")
}

extern "C" cr_status cr_gated_scan_backward(int type, int gate, const void* d_G, int ldg, const void* d_X, int ldx,
                                            const void* d_dH, int lddh, int D, int T, const int32_t* d_off, int n_seq,
                                            const float* d_h0, int ldh0, const float* d_dhT, int lddhT, const float* d_saved,
                                            void* d_dG, int lddg, void* d_dX, int lddx, float* d_dh0, int lddh0,
                                            cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(float_type(type), "cr_gated_scan_backward: type must be FP32, FP16 or BF16");
  CR_REQUIRE(gate >= CR_GATE_COEFF && gate <= CR_GATE_VARIANCE, "cr_gated_scan_backward: unknown gate");
  CR_REQUIRE(D >= 1 && T >= 0 && n_seq >= 0 && n_seq <= 65535, "cr_gated_scan_backward: D >= 1, T >= 0, 0 <= n_seq <= 65535");
  CR_REQUIRE(d_off || n_seq == 1, "cr_gated_scan_backward: without offsets there is one series");
  CR_REQUIRE(n_seq > 0 || T == 0, "cr_gated_scan_backward: columns without a series");
  CR_REQUIRE(T == 0 || (d_G && d_X && d_dH && ldg >= D && ldx >= D && lddh >= D),
             "cr_gated_scan_backward: NULL argument or leading dimension below D");
  CR_REQUIRE((!d_h0 || ldh0 >= D) && (!d_dhT || lddhT >= D) && (!d_dG || lddg >= D) && (!d_dX || lddx >= D) &&
                 (!d_dh0 || lddh0 >= D), "cr_gated_scan_backward: leading dimension below D");
  if (n_seq == 0) return CR_OK;
  float* own = nullptr;
  if (!d_saved && T > 0) {
    size_t count = 0;
    CR_TRY(cr_gated_scan_saved(D, T, &count));
    CR_CUDA(scratch_alloc((void**)&own, count * sizeof(float), stream));
    const cr_status st = cr_gated_scan(type, gate, d_G, ldg, d_X, ldx, D, T, d_off, n_seq, d_h0, ldh0, nullptr, 0, nullptr, 0, own, stream);
    if (st != CR_OK) {
      scratch_free(own, stream);
      return st;
    }
    d_saved = own;
  }
  const cr_status st = with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    return with_gate(gate, [&](auto g0) -> cr_status {
      k_scan_bwd<E, decltype(g0)::value><<<dim3((D + NT - 1) / NT, n_seq), NT, 0, stream>>>(
          (const E*)d_G, ldg, (const E*)d_X, ldx, (const E*)d_dH, lddh, D, T, d_off, d_h0, ldh0, d_dhT, lddhT, d_saved,
          (E*)d_dG, lddg, (E*)d_dX, lddx, d_dh0, lddh0);
      CR_CHECK_LAUNCH("k_scan_bwd");
      return CR_OK;
    });
  });
  scratch_free(own, stream);
  return st;
  CR_ENTRY_END("cr_gated_scan_backward")
}

extern "C" cr_status cr_gated_step(int type, int gate, const void* d_G, int ldg, const void* d_X, int ldx, const float* d_h,
                                   int ldh, int D, int B, void* d_H, int ldo, float* d_hnext, int ldn, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(float_type(type), "cr_gated_step: type must be FP32, FP16 or BF16");
  CR_REQUIRE(gate >= CR_GATE_COEFF && gate <= CR_GATE_VARIANCE, "cr_gated_step: unknown gate");
  CR_REQUIRE(D >= 1 && B >= 0 && B <= 65535, "cr_gated_step: D >= 1, 0 <= B <= 65535");
  if (B == 0) return CR_OK;
  CR_REQUIRE(d_G && d_X && d_h && d_hnext, "cr_gated_step: NULL argument");
  CR_REQUIRE(ldg >= D && ldx >= D && ldh >= D && ldn >= D && (!d_H || ldo >= D), "cr_gated_step: leading dimension below D");
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    return with_gate(gate, [&](auto g0) -> cr_status {
      k_scan_step<E, decltype(g0)::value><<<dim3((D + NT - 1) / NT, B), NT, 0, stream>>>(
          (const E*)d_G, ldg, (const E*)d_X, ldx, d_h, ldh, D, (E*)d_H, ldo, d_hnext, ldn);
      CR_CHECK_LAUNCH("k_scan_step");
      return CR_OK;
    });
  });
  CR_ENTRY_END("cr_gated_step")
}
