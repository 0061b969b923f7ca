// Gated affine product (two projections of the same columns, the first one's activation times the second one), and
// its gradient (cr_gated_affine, cr_gated_affine_backward).
//
// The product is product.cuh's GATED form: both halves of W in one tile, so that X is read once for both and no sum leaves
// the SM.  Bound by the tensor cores or by reading W like the affine product: K = N = M = 4096 BF16 with bias and silu 140 us,
// 1.96 PFLOP/s, e4m3 78 us (in a row, under the power limit, 151 to 162 and 82 to 87); K = 4096, N = 12288, M = 24 FP16 36 us, 5.6 TB/s;
// K = N = 2048, M = 1 BF16 5.3 us.
#include "product.cuh"

namespace cr {
namespace {

// G = [dY .* Zu .* act'(Zg); dY .* act(Zg)] for Z = [Zg; Zu], and the row sums of its unrounded values: a block takes
// 32 V outputs and every gridDim.y-th 8 columns, a thread V outputs of a column (V = 8: 16-byte accesses), and leaves
// its sums in part[blockIdx.y][2 N].  Bound by HBM: dY and Z read, G written (N = 8192, M = 4099 BF16 silu 54 us, 6.2 TB/s).
template <class E, int ACT, int V>
__global__ void __launch_bounds__(NT) k_gated_g(const E* dY, int lddy, const E* Z, int ldz, int N, int M, E* G, int ldg, float* part) {
  __shared__ float red[2][NT / 32][32 * V + V];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i = (blockIdx.x * 32 + lane) * V;
  float sg[V] = {}, su[V] = {};
  if (i < N) {
#pragma unroll 2
    for (int j = blockIdx.y * (NT / 32) + w; j < M; j += gridDim.y * (NT / 32)) {
      const E *dy = dY + (size_t)j * lddy + i, *zz = Z + (size_t)j * ldz + i;
      float d[V], g[V], u[V];
      if constexpr (V == 8) {
        widen8(*reinterpret_cast<const Eight<E>*>(dy), d);
        widen8(*reinterpret_cast<const Eight<E>*>(zz), g);
        widen8(*reinterpret_cast<const Eight<E>*>(zz + N), u);
      } else {
        d[0] = to_float(*dy);
        g[0] = to_float(*zz);
        u[0] = to_float(zz[N]);
      }
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float a = activate<ACT, 1>(Floats<1>{{g[q]}}).x[0];
        g[q] = __fmul_rn(__fmul_rn(d[q], u[q]), activation_slope<ACT>(g[q]));
        u[q] = __fmul_rn(d[q], a);
        sg[q] += g[q];
        su[q] += u[q];
      }
      if (G) {
        E* out = G + (size_t)j * ldg + i;
        if constexpr (V == 8) {
          *reinterpret_cast<Eight<E>*>(out) = narrow8<E>(g);
          *reinterpret_cast<Eight<E>*>(out + N) = narrow8<E>(u);
        } else {
          out[0] = from_float<E>(g[0]);
          out[N] = from_float<E>(u[0]);
        }
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < V; ++q) {
    red[0][w][lane * V + q] = sg[q];
    red[1][w][lane * V + q] = su[q];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < 64 * V; x += NT) {
    const int h = x / (32 * V), c = x % (32 * V), f = blockIdx.x * 32 * V + c;
    float t = red[h][0][c];
    for (int y = 1; y < NT / 32; ++y) t += red[h][y][c];
    if (f < N) part[(size_t)blockIdx.y * 2 * N + (size_t)h * N + f] = t;
  }
}

template <class E, int V>
cr_status gradient_at_z(const E* dY, int lddy, const E* Z, int ldz, int N, int M, int act, E* G, int ldg, float* db, cudaStream_t stream) {
  const int bx = (N + 32 * V - 1) / (32 * V), by = std::max(1, std::min({(M + 7) / 8, 4 * sm_count() / bx, 65535}));
  float* part = nullptr;
  if (db) CR_CUDA(scratch_alloc((void**)&part, (size_t)by * 2 * N * sizeof(float), stream));
  cr_status st = with_act(act, [&](auto a0) -> cr_status {
    TimedScope ts("k_gated_g", stream);
    k_gated_g<E, decltype(a0)::value, V><<<dim3(bx, by), NT, 0, stream>>>(dY, lddy, Z, ldz, N, M, G, ldg, part);
    CR_CHECK_LAUNCH("k_gated_g");
    return CR_OK;
  });
  if (st == CR_OK && db) st = add_rows(part, by, 2 * N, db, stream);
  scratch_free(part, stream);
  return st;
}

}  // namespace
}  // namespace cr

using namespace cr;

extern "C" cr_status cr_gated_affine(int type, const void* d_W, int ldw, const void* d_X, int ldx, int K, int N, int M,
                                     const float* d_wscale, const float* d_xscale, const float* d_bias, int act, int out_type,
                                     void* d_Z, int ldz, void* d_Y, int ldy, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(type == CR_TYPE_F16 || type == CR_TYPE_BF16 || type == CR_TYPE_E4M3, "cr_gated_affine: type must be FP16, BF16 or e4m3");
  CR_REQUIRE(out_type == CR_TYPE_F32 || out_type == CR_TYPE_F16 || out_type == CR_TYPE_BF16,
             "cr_gated_affine: out_type must be FP32, FP16 or BF16");
  CR_REQUIRE(act >= CR_ACT_NONE && act <= CR_ACT_GELU, "cr_gated_affine: unknown activation");
  CR_REQUIRE(type == CR_TYPE_E4M3 || (!d_wscale && !d_xscale), "cr_gated_affine: scales belong to e4m3");
  CR_REQUIRE(K >= 1 && N >= 1 && M >= 0, "cr_gated_affine: K >= 1, N >= 1, M >= 0");
  CR_REQUIRE(N <= MAXSIZE / 2, "cr_gated_affine: 2 N ends at 2^31 - 2^16");
  CR_REQUIRE_SIZES("cr_gated_affine", K, N, M);
  CR_REQUIRE(ldw >= K && ldx >= K && ldy >= N && (!d_Z || ldz >= 2 * N), "cr_gated_affine: leading dimension too small");
  if (M == 0) return CR_OK;
  CR_REQUIRE(d_W && d_X && d_Y, "cr_gated_affine: NULL argument");
  int* err = nullptr;
  CR_TRY(wait_word(&err));
  const Epilogue e{d_wscale, d_xscale, d_bias, act, nullptr, 0, d_Z, ldz, d_Y, ldy};
  return product<GATED>(Operand{d_W, 2 * N, ldw, true}, Operand{d_X, M, ldx, true}, type, K, out_type, e, err, stream);
  CR_ENTRY_END("cr_gated_affine")
}

extern "C" cr_status cr_gated_affine_backward(int type, const void* d_W, int ldw, const void* d_X, int ldx, const void* d_dY,
                                              int lddy, const void* d_Z, int ldz, int K, int N, int M, int act, void* d_dX,
                                              int lddx, int dw_type, void* d_dW, int lddw, float* d_db, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(type == CR_TYPE_F16 || type == CR_TYPE_BF16, "cr_gated_affine_backward: type must be FP16 or BF16");
  CR_REQUIRE(act >= CR_ACT_NONE && act <= CR_ACT_GELU, "cr_gated_affine_backward: unknown activation");
  CR_REQUIRE(!d_dW || dw_type == type || dw_type == CR_TYPE_F32, "cr_gated_affine_backward: dw_type must be type or FP32");
  CR_REQUIRE(K >= 1 && N >= 1 && M >= 0, "cr_gated_affine_backward: K >= 1, N >= 1, M >= 0");
  CR_REQUIRE(N <= MAXSIZE / 2, "cr_gated_affine_backward: 2 N ends at 2^31 - 2^16");
  CR_REQUIRE_SIZES("cr_gated_affine_backward", K, N, M);
  CR_REQUIRE((!d_dX || (ldw >= K && lddx >= K)) && (!d_dW || (ldx >= K && lddw >= K)) && lddy >= N && ldz >= 2 * N,
             "cr_gated_affine_backward: leading dimension too small");
  CR_REQUIRE(M == 0 || (d_dY && d_Z && (!d_dX || d_W) && (!d_dW || d_X)), "cr_gated_affine_backward: NULL argument");
  if (M == 0) {
    if (d_db) CR_CUDA(cudaMemsetAsync(d_db, 0, (size_t)2 * N * sizeof(float), stream));
    if (d_dW) CR_CUDA(cudaMemset2DAsync(d_dW, (size_t)lddw * type_bytes(dw_type), 0, (size_t)K * type_bytes(dw_type), (size_t)2 * N, stream));
    return CR_OK;
  }
  if (!d_dX && !d_dW && !d_db) return CR_OK;
  int* err = nullptr;
  CR_TRY(wait_word(&err));
  void* own = nullptr;
  const int two = 2 * N, ldown = (two + 7) & ~7;   // columns on 16-byte boundaries
  if (d_dX || d_dW) CR_CUDA(scratch_alloc(&own, (size_t)ldown * M * 2, stream));
  const auto go = [&](auto e0) -> cr_status {
    using E = decltype(e0);
    const auto ok16 = [](const void* q, int ld) { return ((uintptr_t)q & 15) == 0 && ld % 8 == 0; };
    const E *dY = (const E*)d_dY, *Z = (const E*)d_Z;
    if (N % 8 == 0 && ok16(d_dY, lddy) && ok16(d_Z, ldz)) CR_TRY((gradient_at_z<E, 8>(dY, lddy, Z, ldz, N, M, act, (E*)own, ldown, d_db, stream)));
    else CR_TRY((gradient_at_z<E, 1>(dY, lddy, Z, ldz, N, M, act, (E*)own, ldown, d_db, stream)));
    First first;
    for (int part = 0; part < 2; ++part) {
      if ((part == 0) == (two >= M)) {   // the one with the longer sums first
        if (!d_dX) continue;             // dX(i, j) = sum_n W(i, n) G(n, j)
        const Epilogue e{nullptr, nullptr, nullptr, CR_ACT_NONE, nullptr, 0, nullptr, 0, d_dX, lddx};
        CR_TRY(affine_product(Operand{d_W, K, ldw, false}, Operand{own, M, ldown, true}, type, two, type, e, err, stream, &first));
      } else {
        if (!d_dW) continue;             // dW(i, n) = sum_j X(i, j) G(n, j)
        const Epilogue e{nullptr, nullptr, nullptr, CR_ACT_NONE, nullptr, 0, nullptr, 0, d_dW, lddw};
        CR_TRY(affine_product(Operand{d_X, K, ldx, false}, Operand{own, two, ldown, false}, type, M, dw_type, e, err, stream, &first));
      }
    }
    return CR_OK;
  };
  const cr_status st = type == CR_TYPE_F16 ? go(__half{}) : go(__nv_bfloat16{});
  scratch_free(own, stream);
  return st;
  CR_ENTRY_END("cr_gated_affine_backward")
}
