// Affine product with bias, activation and residual in its epilogue, and its gradient
// (cr_affine, cr_affine_backward).
#include "product.cuh"

namespace cr {
namespace {

// G = dY .* act'(Z), and the row sums of its unrounded values: a block takes 32 V features and every
// gridDim.y-th 8 columns, a thread V features of a column (V = 8: 16-byte accesses), and leaves its sums
// in part[blockIdx.y][N].  Bound by HBM (dY and Z read, G written): N = 8192, M = 2048 BF16
// silu 18 us, 5.5 TB/s.
template <class E, int ACT, int V>
__global__ void __launch_bounds__(NT) k_affine_g(const E* dY, int lddy, const E* Z, int ldz, int N, int M, E* G, int ldg, float* part) {
  __shared__ float red[NT / 32][32 * V + V];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i = (blockIdx.x * 32 + lane) * V;
  float s[V] = {};
  if (i < N) {
#pragma unroll 4
    for (int j = blockIdx.y * (NT / 32) + w; j < M; j += gridDim.y * (NT / 32)) {
      const E *dy = dY + (size_t)j * lddy + i, *zz = Z + (size_t)j * ldz + i;
      float g[V], z[V];
      if constexpr (V == 8) {
        widen8(*reinterpret_cast<const Eight<E>*>(dy), g);
        if (ACT != CR_ACT_NONE) widen8(*reinterpret_cast<const Eight<E>*>(zz), z);
      } else {
        g[0] = to_float(*dy);
        if (ACT != CR_ACT_NONE) z[0] = to_float(*zz);
      }
#pragma unroll
      for (int q = 0; q < V; ++q) {
        if (ACT != CR_ACT_NONE) g[q] = __fmul_rn(g[q], activation_slope<ACT>(z[q]));
        s[q] += g[q];
      }
      if (G) {
        if constexpr (V == 8) *reinterpret_cast<Eight<E>*>(G + (size_t)j * ldg + i) = narrow8<E>(g);
        else G[(size_t)j * ldg + i] = from_float<E>(g[0]);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < V; ++q) red[w][lane * V + q] = s[q];
  __syncthreads();
  for (int x = threadIdx.x; x < 32 * V; x += NT) {
    const int f = blockIdx.x * 32 * V + x;
    float t = red[0][x];
    for (int y = 1; y < NT / 32; ++y) t += red[y][x];
    if (f < N) part[(size_t)blockIdx.y * N + f] = t;
  }
}

template <class E, int V>
cr_status gradient_at_z(const E* dY, int lddy, const E* Z, int ldz, int N, int M, int act, E* G, int ldg, float* db, cudaStream_t stream) {
  const int bx = (N + 32 * V - 1) / (32 * V), by = std::max(1, std::min({(M + 7) / 8, 4 * sm_count() / bx, 65535}));
  float* part = nullptr;
  if (db) CR_CUDA(scratch_alloc((void**)&part, (size_t)by * N * sizeof(float), stream));
  cr_status st = with_act(act, [&](auto a0) -> cr_status {
    TimedScope ts("k_affine_g", stream);
    k_affine_g<E, decltype(a0)::value, V><<<dim3(bx, by), NT, 0, stream>>>(dY, lddy, Z, ldz, N, M, G, ldg, part);
    CR_CHECK_LAUNCH("k_affine_g");
    return CR_OK;
  });
  if (st == CR_OK && db) st = add_rows(part, by, N, db, stream);
  scratch_free(part, stream);
  return st;
}

}  // namespace

cr_status affine_product(Operand P, Operand Q, int type, int K, int out_type, const Epilogue& e, int* err, cudaStream_t stream, First* first) {
  return product<AFFINE>(P, Q, type, K, out_type, e, err, stream, first);
}

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
  CR_REQUIRE_SIZES("cr_affine", K, N, M);
  CR_REQUIRE(ldw >= K && ldx >= K && ldy >= N && (!d_R || ldr >= N) && (!d_Z || ldz >= N), "cr_affine: leading dimension too small");
  if (M == 0) return CR_OK;
  CR_REQUIRE(d_W && d_X && d_Y, "cr_affine: NULL argument");
  int* err = nullptr;
  CR_TRY(wait_word(&err));
  const Epilogue e{d_wscale, d_xscale, d_bias, act, d_R, ldr, d_Z, ldz, d_Y, ldy};
  return affine_product(Operand{d_W, N, ldw, true}, Operand{d_X, M, ldx, true}, type, K, out_type, e, err, stream);
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
  CR_REQUIRE_SIZES("cr_affine_backward", K, N, M);
  CR_REQUIRE((!d_dX || (ldw >= K && lddx >= K)) && (!d_dW || (ldx >= K && lddw >= K)) && lddy >= N &&
                 (act == CR_ACT_NONE || ldz >= N), "cr_affine_backward: leading dimension too small");
  CR_REQUIRE(M == 0 || (d_dY && (act == CR_ACT_NONE || d_Z) && (!d_dX || d_W) && (!d_dW || d_X)), "cr_affine_backward: NULL argument");
  if (M == 0) {
    if (d_db) CR_CUDA(cudaMemsetAsync(d_db, 0, (size_t)N * sizeof(float), stream));
    if (d_dW) CR_CUDA(cudaMemset2DAsync(d_dW, (size_t)lddw * type_bytes(dw_type), 0, (size_t)K * type_bytes(dw_type), N, stream));
    return CR_OK;
  }
  if (!d_dX && !d_dW && !d_db) return CR_OK;
  int* err = nullptr;
  CR_TRY(wait_word(&err));
  void* own = nullptr;
  const int ldown = (N + 7) & ~7;   // columns on 16-byte boundaries
  if (act != CR_ACT_NONE && (d_dX || d_dW)) CR_CUDA(scratch_alloc(&own, (size_t)ldown * M * 2, stream));
  const auto go = [&](auto e0) -> cr_status {
    using E = decltype(e0);
    const E* G = own ? (const E*)own : (const E*)d_dY;
    const int ldg = own ? ldown : lddy;
    if (own || d_db) {
      const auto ok16 = [](const void* q, int ld) { return ((uintptr_t)q & 15) == 0 && ld % 8 == 0; };
      const bool vec = N % 8 == 0 && ok16(d_dY, lddy) && (act == CR_ACT_NONE || ok16(d_Z, ldz));
      if (vec) CR_TRY((gradient_at_z<E, 8>((const E*)d_dY, lddy, (const E*)d_Z, ldz, N, M, act, (E*)own, ldown, d_db, stream)));
      else CR_TRY((gradient_at_z<E, 1>((const E*)d_dY, lddy, (const E*)d_Z, ldz, N, M, act, (E*)own, ldown, d_db, stream)));
    }
    First first;
    for (int part = 0; part < 2; ++part) {
      if ((part == 0) == (N >= M)) {   // the one with the longer sums first
        if (!d_dX) continue;           // dX(i, j) = sum_n W(i, n) G(n, j)
        const Epilogue e{nullptr, nullptr, nullptr, CR_ACT_NONE, nullptr, 0, nullptr, 0, d_dX, lddx};
        CR_TRY(affine_product(Operand{d_W, K, ldw, false}, Operand{G, M, ldg, true}, type, N, type, e, err, stream, &first));
      } else {
        if (!d_dW) continue;           // dW(i, n) = sum_j X(i, j) G(n, j)
        const Epilogue e{nullptr, nullptr, nullptr, CR_ACT_NONE, nullptr, 0, nullptr, 0, d_dW, lddw};
        CR_TRY(affine_product(Operand{d_X, K, ldx, false}, Operand{G, N, ldg, false}, type, M, dw_type, e, err, stream, &first));
      }
    }
    return CR_OK;
  };
  const cr_status st = type == CR_TYPE_F16 ? go(__half{}) : go(__nv_bfloat16{});
  scratch_free(own, stream);
  return st;
  CR_ENTRY_END("cr_affine_backward")
}
