// Affine product with bias, activation and residual in its epilogue, and its gradient
// (cr_affine, cr_affine_backward).
#include <type_traits>

#include "ops.cuh"

namespace cr {
namespace {

constexpr int NT = 256;

// C(i, j) = epilogue(sum_k A(i, k) B(j, k)), C column-major: i runs along C's columns.  Element
// (i, k) of A is at i * ai + k * ak, element (j, k) of B at j * bj + k * bk.
template <class E, class O>
struct Prod {
  const E *A, *B;
  long long ai, ak, bj, bk;
  int I, J, K;
  const float *iscale, *jscale, *bias;
  const O* R;
  int ldr;
  O* Z;
  int ldz;
  O* C;
  int ldc;
};

// 64 x 64 outputs per block, 4 x 4 per thread, operands through shared memory in FP32.
template <class E, class O, int ACT>
__global__ void __launch_bounds__(NT) k_prod(const Prod<E, O> p) {
  __shared__ float sa[16][65], sb[16][65];
  const int i0 = blockIdx.x * 64, j0 = blockIdx.y * 64;
  const int ti = threadIdx.x % 16, tj = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += 16) {
    for (int e = threadIdx.x; e < 64 * 16; e += NT) {
      const int k = p.ak == 1 ? e % 16 : e / 64, i = p.ak == 1 ? e / 16 : e % 64;
      const bool in = i0 + i < p.I && k0 + k < p.K;
      sa[k][i] = in ? to_float(p.A[(i0 + i) * p.ai + (k0 + k) * p.ak]) : 0.0f;
    }
    for (int e = threadIdx.x; e < 64 * 16; e += NT) {
      const int k = p.bk == 1 ? e % 16 : e / 64, j = p.bk == 1 ? e / 16 : e % 64;
      const bool in = j0 + j < p.J && k0 + k < p.K;
      sb[k][j] = in ? to_float(p.B[(j0 + j) * p.bj + (k0 + k) * p.bk]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(sa[k][ti + 16 * a], sb[k][tj + 16 * b], acc[a][b]);
    __syncthreads();
  }
  for (int a = 0; a < 4; ++a)
    for (int b = 0; b < 4; ++b) {
      const int i = i0 + ti + 16 * a, j = j0 + tj + 16 * b;
      if (i >= p.I || j >= p.J) continue;
      float z = acc[a][b];
      if (p.iscale) z *= p.iscale[i];
      if (p.jscale) z *= p.jscale[j];
      if (p.bias) z += p.bias[i];
      if (p.Z) p.Z[(size_t)j * p.ldz + i] = from_float<O>(z);
      float y = activate<ACT>(z);
      if (p.R) y += to_float(p.R[(size_t)j * p.ldr + i]);
      p.C[(size_t)j * p.ldc + i] = from_float<O>(y);
    }
}

// G = dY .* act'(Z), and the row sums of its unrounded values; one block per 32 features.
template <class E, int ACT>
__global__ void __launch_bounds__(NT) k_affine_g(const E* dY, int lddy, const E* Z, int ldz, int N, int M, E* G, int ldg, float* db) {
  __shared__ float red[NT / 32][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < N)
    for (int j = w; j < M; j += NT / 32) {
      float g = to_float(dY[(size_t)j * lddy + i]);
      if (ACT != CR_ACT_NONE) g = __fmul_rn(g, activation_slope<ACT>(to_float(Z[(size_t)j * ldz + i])));
      s += g;
      if (G) G[(size_t)j * ldg + i] = from_float<E>(g);
    }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && i < N && db) {
    for (int v = 1; v < NT / 32; ++v) s += red[v][lane];
    db[i] = s;
  }
}

template <class E, class O>
cr_status product(const Prod<E, O>& p, int act, cudaStream_t stream) {
  return with_act(act, [&](auto a0) -> cr_status {
    k_prod<E, O, decltype(a0)::value><<<dim3((p.I + 63) / 64, (p.J + 63) / 64), NT, 0, stream>>>(p);
    CR_CHECK_LAUNCH("k_prod");
    return CR_OK;
  });
}

}  // namespace
}  // namespace cr

using namespace cr;

extern "C" cr_status cr_affine(int type, const void* d_W, int ldw, const void* d_X, int ldx, int K, int N, int M,
                               const float* d_wscale, const float* d_xscale, const float* d_bias, int act, int out_type,
                               const void* d_R, int ldr, void* d_Z, int ldz, void* d_Y, int ldy, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(type == CR_TYPE_F16 || type == CR_TYPE_BF16 || type == CR_TYPE_E4M3, "cr_affine: type must be FP16, BF16 or e4m3");
  CR_REQUIRE(out_type == CR_TYPE_F32 || out_type == CR_TYPE_F16 || out_type == CR_TYPE_BF16,
             "cr_affine: out_type must be FP32, FP16 or BF16");
  CR_REQUIRE(act >= CR_ACT_NONE && act <= CR_ACT_GELU, "cr_affine: unknown activation");
  CR_REQUIRE(type == CR_TYPE_E4M3 || (!d_wscale && !d_xscale), "cr_affine: scales belong to e4m3");
  CR_REQUIRE(K >= 1 && N >= 1 && M >= 0, "cr_affine: K >= 1, N >= 1, M >= 0");
  CR_REQUIRE(ldw >= K && ldx >= K && ldy >= N && (!d_R || ldr >= N) && (!d_Z || ldz >= N), "cr_affine: leading dimension too small");
  if (M == 0) return CR_OK;
  CR_REQUIRE(d_W && d_X && d_Y, "cr_affine: NULL argument");
  const auto go = [&](auto e0, auto o0) -> cr_status {
    using E = decltype(e0);
    using O = decltype(o0);
    const Prod<E, O> p{(const E*)d_W, (const E*)d_X, ldw, 1, ldx, 1, N, M, K, d_wscale, d_xscale, d_bias,
                       (const O*)d_R, ldr, (O*)d_Z, ldz, (O*)d_Y, ldy};
    return product(p, act, stream);
  };
  return with_type(out_type, [&](auto o0) -> cr_status {
    if (type == CR_TYPE_F16) return go(__half{}, o0);
    if (type == CR_TYPE_BF16) return go(__nv_bfloat16{}, o0);
    return go(__nv_fp8_e4m3{}, o0);
  });
  CR_ENTRY_END("cr_affine")
}

extern "C" cr_status cr_affine_backward(int type, const void* d_W, int ldw, const void* d_X, int ldx, const void* d_dY,
                                        int lddy, const void* d_Z, int ldz, int K, int N, int M, int act, void* d_dX, int lddx,
                                        int dw_type, void* d_dW, int lddw, float* d_db, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(type == CR_TYPE_F16 || type == CR_TYPE_BF16, "cr_affine_backward: type must be FP16 or BF16");
  CR_REQUIRE(act >= CR_ACT_NONE && act <= CR_ACT_GELU, "cr_affine_backward: unknown activation");
  CR_REQUIRE(!d_dW || dw_type == type || dw_type == CR_TYPE_F32, "cr_affine_backward: dw_type must be type or FP32");
  CR_REQUIRE(K >= 1 && N >= 1 && M >= 0, "cr_affine_backward: K >= 1, N >= 1, M >= 0");
  CR_REQUIRE((!d_dX || (ldw >= K && lddx >= K)) && (!d_dW || (ldx >= K && lddw >= K)) && lddy >= N &&
                 (act == CR_ACT_NONE || ldz >= N), "cr_affine_backward: leading dimension too small");
  CR_REQUIRE(M == 0 || (d_dY && (act == CR_ACT_NONE || d_Z) && (!d_dX || d_W) && (!d_dW || d_X)), "cr_affine_backward: NULL argument");
  if (M == 0) {
    if (d_db) CR_CUDA(cudaMemsetAsync(d_db, 0, (size_t)N * sizeof(float), stream));
    if (d_dW) CR_CUDA(cudaMemset2DAsync(d_dW, (size_t)lddw * type_bytes(dw_type), 0, (size_t)K * type_bytes(dw_type), N, stream));
    return CR_OK;
  }
  void* own = nullptr;
  if (act != CR_ACT_NONE && (d_dX || d_dW)) CR_CUDA(scratch_alloc(&own, (size_t)N * M * 2, stream));
  const auto go = [&](auto e0) -> cr_status {
    using E = decltype(e0);
    const E* G = own ? (const E*)own : (const E*)d_dY;
    const int ldg = own ? N : lddy;
    if (own || d_db)
      CR_TRY(with_act(act, [&](auto a0) -> cr_status {
        k_affine_g<E, decltype(a0)::value><<<(N + 31) / 32, NT, 0, stream>>>((const E*)d_dY, lddy, (const E*)d_Z, ldz, N, M,
                                                                            (E*)own, N, d_db);
        CR_CHECK_LAUNCH("k_affine_g");
        return CR_OK;
      }));
    if (d_dX) {   // dX(i, j) = sum_n W(i, n) G(n, j)
      const Prod<E, E> p{(const E*)d_W, G, 1, ldw, ldg, 1, K, M, N, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, (E*)d_dX, lddx};
      CR_TRY(product(p, CR_ACT_NONE, stream));
    }
    if (d_dW) {   // dW(i, n) = sum_j X(i, j) G(n, j)
      if (dw_type == CR_TYPE_F32) {
        const Prod<E, float> p{(const E*)d_X, G, 1, ldx, 1, ldg, K, N, M, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, (float*)d_dW, lddw};
        CR_TRY(product(p, CR_ACT_NONE, stream));
      } else {
        const Prod<E, E> p{(const E*)d_X, G, 1, ldx, 1, ldg, K, N, M, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, (E*)d_dW, lddw};
        CR_TRY(product(p, CR_ACT_NONE, stream));
      }
    }
    return CR_OK;
  };
  const cr_status st = type == CR_TYPE_F16 ? go(__half{}) : go(__nv_bfloat16{});
  scratch_free(own, stream);
  return st;
  CR_ENTRY_END("cr_affine_backward")
}
