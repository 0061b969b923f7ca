// Orthogonalised update of a weight matrix by Newton-Schulz products (cr_orthogonalize).
//
// X = G / |G|_F, then X <- a X + (b A + c A^2) X with A = X X^T (X^T X for more rows than columns), `steps` times.  Every
// matrix between two products is FP16 with FP32 sums: 1024 times its value, which keeps entries of up to 64 finite and
// of 2^-24 with 11 bits (X's are about 1 / sqrt(K N)).  FP16 holds three bits more than a BF16 output; for FP16 and FP32
// outputs each matrix is a sum of two FP16 ones (22 bits), and a product three (the one of the two small parts is below
// 2^-22 of it).  A and b A + c A^2 are symmetric: the wide kernel forms half of their tiles and stores them twice.
#include <cmath>

#include "product.cuh"

namespace cr {
namespace {

constexpr float UNIT = 1024.0f;   // the matrices hold UNIT times their values
constexpr int MAXPART = 1024;

// Sums of squares of a block's elements to part[block]: of those above 2^50 and below 2^-50 scaled by 2^-90 and 2^90, so
// that no square overflows or underflows.
struct Squares {
  double big, mid, small;
};
template <class T, int V>
__global__ void __launch_bounds__(NT) k_ortho_norm(const T* G, int ld, int K, int N, Squares* part) {
  __shared__ Squares red[NT / 32];
  float big = 0.0f, mid = 0.0f, small = 0.0f;
  const int per = (K + V - 1) / V;
  const long long total = (long long)per * N;
#pragma unroll 4
  for (long long e = (long long)blockIdx.x * NT + threadIdx.x; e < total; e += (long long)gridDim.x * NT) {
    const int col = e >> 32 ? (int)(e / per) : (int)((uint32_t)e / (uint32_t)per), i = (int)(e - (long long)col * per) * V;
    const T* from = G + (size_t)col * ld + i;
    float x[V];
    if constexpr (V == 8) widen8(*reinterpret_cast<const Eight<T>*>(from), x);
    else x[0] = to_float(from[0]);
#pragma unroll
    for (int q = 0; q < V; ++q) {
      const float a = fabsf(x[q]);
      const bool high = a > 0x1p50f, low = a < 0x1p-50f;
      const float y = high ? a * 0x1p-90f : low ? a * 0x1p90f : a;
      if (high) big = fmaf(y, y, big);
      else if (low) small = fmaf(y, y, small);
      else mid = fmaf(y, y, mid);
    }
  }
  Squares s = {big, mid, small};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.big += __shfl_xor_sync(0xffffffffu, s.big, o);
    s.mid += __shfl_xor_sync(0xffffffffu, s.mid, o);
    s.small += __shfl_xor_sync(0xffffffffu, s.small, o);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < NT / 32; ++w) {
      s.big += red[w].big;
      s.mid += red[w].mid;
      s.small += red[w].small;
    }
    part[blockIdx.x] = s;
  }
}

// X = UNIT G / |G|_F, zero for a zero matrix and NaN where |G|_F is not finite, as FP16 with the rest after it in X2 (may
// be NULL).  UNIT / |G|_F is m 2^e, and 2^e is applied in two halves that are normal numbers.
template <class T, int V>
__global__ void __launch_bounds__(NT) k_ortho_scale(const T* G, int ld, int K, int N, const Squares* part, int parts, __half* X, __half* X2, int ldx) {
  __shared__ float factor[3];
  if (threadIdx.x < 32) {
    Squares s = {0.0, 0.0, 0.0};
    for (int q = threadIdx.x; q < parts; q += 32) {
      s.big += part[q].big;
      s.mid += part[q].mid;
      s.small += part[q].small;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s.big += __shfl_xor_sync(0xffffffffu, s.big, o);
      s.mid += __shfl_xor_sync(0xffffffffu, s.mid, o);
      s.small += __shfl_xor_sync(0xffffffffu, s.small, o);
    }
    if (threadIdx.x == 0) {
      const double norm = sqrt(s.big * 0x1p180 + s.mid + s.small * 0x1p-180);
      int e = 0;
      double m = 0.0;
      if (norm > 0.0 && norm < 1e300) m = frexp((double)UNIT / norm, &e);
      else if (norm != 0.0) m = norm - norm;   // NaN
      factor[0] = (float)m;
      factor[1] = (float)ldexp(1.0, e / 2);
      factor[2] = (float)ldexp(1.0, e - e / 2);
    }
  }
  __syncthreads();
  const float m = factor[0], p1 = factor[1], p2 = factor[2];
  const int per = ldx / 8;
  const long long total = (long long)per * N;
  for (long long e = (long long)blockIdx.x * NT + threadIdx.x; e < total; e += (long long)gridDim.x * NT) {
    const int col = e >> 32 ? (int)(e / per) : (int)((uint32_t)e / (uint32_t)per), i = (int)(e - (long long)col * per) * 8;
    const T* from = G + (size_t)col * ld + i;
    float x[8];
    if constexpr (V == 8) {
      widen8(*reinterpret_cast<const Eight<T>*>(from), x);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = i + q < K ? to_float(from[q]) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = x[q] * p1 * p2 * m;
    const Eight<__half> hi = narrow8<__half>(x);
    *reinterpret_cast<Eight<__half>*>(X + (size_t)col * ldx + i) = hi;
    if (X2) {
      float h[8];
      widen8(hi, h);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] -= h[q];
      *reinterpret_cast<Eight<__half>*>(X2 + (size_t)col * ldx + i) = narrow8<__half>(x);
    }
  }
}

// O = (X + X2) / UNIT in FP32.
__global__ void __launch_bounds__(NT) k_ortho_join(const __half* X, const __half* X2, int ldx, int K, int N, float* O, int ldo) {
  let_next_start();
  wait_for_previous();
  const int per = (K + 3) / 4;
  const long long total = (long long)per * N;
  const bool vec = ((uintptr_t)O & 15) == 0 && ldo % 4 == 0;
  for (long long e = (long long)blockIdx.x * NT + threadIdx.x; e < total; e += (long long)gridDim.x * NT) {
    const int col = e >> 32 ? (int)(e / per) : (int)((uint32_t)e / (uint32_t)per), i = (int)(e - (long long)col * per) * 4;
    const uint2 a = *reinterpret_cast<const uint2*>(X + (size_t)col * ldx + i), b = *reinterpret_cast<const uint2*>(X2 + (size_t)col * ldx + i);
    const float2 a0 = widen2(a.x, __half{}), a1 = widen2(a.y, __half{}), b0 = widen2(b.x, __half{}), b1 = widen2(b.y, __half{});
    const float v[4] = {(a0.x + b0.x) / UNIT, (a0.y + b0.y) / UNIT, (a1.x + b1.x) / UNIT, (a1.y + b1.y) / UNIT};
    float* to = O + (size_t)col * ldo + i;
    if (vec && i + 4 <= K) *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
    else
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + q < K) to[q] = v[q];
  }
}

// An FP16 matrix of the library's, or a sum of two.
struct Split {
  __half *hi, *lo;
  int ld;
};

// C = alpha P Q^T + beta R (R may be missing), C rows x cols; the last product's C is the caller's, of out_type.
struct Step {
  Split P, Q, R, C;
  int I, J, K;
  bool p_major, q_major;   // k contiguous
  bool symmetric;
  float alpha, beta;
  void* out;               // instead of C
  int out_type, ldout;
};
cr_status step_product(const Step& s, int* err, cudaStream_t stream) {
  Params p = {};
  p.err = err;
  p.limit = option_wait_ns();
  p.I = s.I;
  p.J = s.J;
  p.pk = s.p_major;
  p.qk = s.q_major;
  p.segments = s.P.lo ? 3 : 1;
  p.kblocks = (s.K + 63) / 64 * p.segments;
  p.alpha = s.alpha;
  p.beta = s.beta;
  p.e.R = s.R.hi;
  p.e.ldr = s.R.ld;
  p.R2 = s.R.lo;
  p.e.C = s.out ? s.out : s.C.hi;
  p.e.ldc = s.out ? s.ldout : s.C.ld;
  p.C2 = s.out ? nullptr : s.C.lo;
  const int out_type = s.out ? s.out_type : CR_TYPE_F16;
  p.tma_c = ((uintptr_t)p.e.C & 15) == 0 && p.e.ldc % 8 == 0;
  const Choice ch = choose<STEP>(s.I, s.J, p.kblocks, s.q_major, s.symmetric);
  p.triangle = ch.wide && s.symmetric;
  p.bn = ch.bn;
  p.ti = ch.wide ? (s.I + 255) / 256 : (s.I + 127) / 128;
  p.tj = ch.wide ? (s.J + 255) / 256 : (s.J + p.bn - 1) / p.bn;
  p.idesc = ch.wide ? idesc_of(256, 256, false, !p.qk, !p.pk) : idesc_of(128, p.bn, false, !p.pk, !p.qk);
  p.stages = WSTAGES - 1;   // two output buffers per warp
  const auto maps_of = [&](CUtensorMap* m, CUtensorMap* m2, const Split& x, int rows, bool major, int box) -> cr_status {
    CR_TRY(map_of(m, Operand{x.hi, rows, x.ld, major}, CR_TYPE_F16, s.K, box));
    return x.lo ? map_of(m2, Operand{x.lo, rows, x.ld, major}, CR_TYPE_F16, s.K, box) : CR_OK;
  };
  const auto go = [&](auto o0) -> cr_status {
    using O = decltype(o0);
    if (!ch.wide) {
      ThinMaps maps = {};
      CR_TRY(maps_of(&maps.P, &maps.P2, s.P, s.I, s.p_major, 128));
      CR_TRY(maps_of(&maps.Q, &maps.Q2, s.Q, s.J, s.q_major, p.bn));
      return launch_thin<STEP, false, O>(maps, p, ch.split, ch.stages, stream);
    }
    Maps<STEP> maps = {};
    CR_TRY(maps_of(&maps.P, &maps.P2, s.P, s.I, s.p_major, 128));
    CR_TRY(maps_of(&maps.Q, &maps.Q2, s.Q, s.J, s.q_major, 128));
    const auto tile = [&](CUtensorMap* m, const void* x, int type, int ld) { return make_tensor_map_2d(m, type, x, s.I, s.J, ld, 64, 32); };
    if (p.tma_c) CR_TRY(tile(&maps.C, p.e.C, out_type, p.e.ldc));
    if (p.C2) CR_TRY(tile(&maps.C2, p.C2, CR_TYPE_F16, p.e.ldc));
    if (s.R.hi) CR_TRY(tile(&maps.R, s.R.hi, CR_TYPE_F16, s.R.ld));
    if (s.R.lo) CR_TRY(tile(&maps.R2, s.R.lo, CR_TYPE_F16, s.R.ld));
    if (p.triangle) {
      CR_TRY(make_tensor_map_2d_plain(&maps.T, CR_TYPE_F16, p.e.C, s.J, s.I, p.e.ldc, 32, 64));
      if (p.C2) CR_TRY(make_tensor_map_2d_plain(&maps.T2, CR_TYPE_F16, p.C2, s.J, s.I, p.e.ldc, 32, 64));
    }
    const long long n = p.tj;
    return launch_wide<STEP, false, O>(maps, p, p.triangle ? n * (n + 1) / 2 : (long long)p.ti * p.tj, stream);
  };
  return out_type == CR_TYPE_BF16 ? go(__nv_bfloat16{}) : go(__half{});
}

template <class T>
cr_status start(const T* G, int ld, int K, int N, Squares* part, const Split& X, cudaStream_t stream) {
  const bool vec = ((uintptr_t)G & 15) == 0 && (long long)ld * sizeof(T) % 16 == 0 && K % 8 == 0;
  const long long items = (long long)(vec ? K / 8 : K) * N;
  const int blocks = (int)std::max<long long>(1, std::min<long long>({(items + 2 * NT - 1) / (2 * NT), 4ll * sm_count(), MAXPART}));
  const auto go = [&](auto v0) -> cr_status {
    constexpr int V = decltype(v0)::value;
    {
      TimedScope ts("k_ortho_norm", stream);
      k_ortho_norm<T, V><<<blocks, NT, 0, stream>>>(G, ld, K, N, part);
      CR_CHECK_LAUNCH("k_ortho_norm");
    }
    const long long words = (long long)X.ld / 8 * N;
    TimedScope ts("k_ortho_scale", stream);
    k_ortho_scale<T, V><<<(unsigned)std::min<long long>((words + NT - 1) / NT, 8ll * sm_count()), NT, 0, stream>>>(
        G, ld, K, N, part, blocks, X.hi, X.lo, X.ld);
    CR_CHECK_LAUNCH("k_ortho_scale");
    return CR_OK;
  };
  return vec ? go(std::integral_constant<int, 8>{}) : go(std::integral_constant<int, 1>{});
}

}  // namespace
}  // namespace cr

using namespace cr;

extern "C" cr_status cr_orthogonalize(int type, const void* d_G, int ldg, int K, int N, int steps, double a, double b, double c,
                                      int out_type, void* d_O, int ldo, cr_stream stream) {
  CR_ENTRY_BEGIN
  const auto known = [](int t) { return t == CR_TYPE_F32 || t == CR_TYPE_F16 || t == CR_TYPE_BF16; };
  CR_REQUIRE(known(type) && known(out_type), "cr_orthogonalize: types are FP32, FP16 and BF16");
  CR_REQUIRE(K >= 1 && N >= 1, "cr_orthogonalize: K >= 1, N >= 1");
  CR_REQUIRE_SIZES("cr_orthogonalize", K, N);
  CR_REQUIRE(steps >= 1 && steps <= 100, "cr_orthogonalize: 1 to 100 steps");
  CR_REQUIRE(std::abs(a) <= 64.0 && std::abs(b) <= 64.0 && std::abs(c) <= 64.0, "cr_orthogonalize: coefficients are finite, up to 64");
  CR_REQUIRE(ldg >= K && ldo >= K, "cr_orthogonalize: leading dimension below K");
  CR_REQUIRE(d_G && d_O, "cr_orthogonalize: NULL argument");
  int* err = nullptr;
  CR_TRY(wait_word(&err));
  const bool two = out_type != CR_TYPE_BF16, wide = K <= N;
  const int s = wide ? K : N, ld = (K + 7) & ~7, lds = (s + 7) & ~7;
  const auto bytes = [](long long l, long long n) { return (size_t)((l * n * 2 + 255) & ~255ll); };
  const size_t bx = bytes(ld, N), bs = bytes(lds, s);
  uint8_t* own = nullptr;
  CR_CUDA(scratch_alloc((void**)&own, MAXPART * sizeof(Squares) + (two ? 2 : 1) * 2 * (bx + bs), stream));
  uint8_t* next = own + MAXPART * sizeof(Squares);
  const auto take = [&](size_t n, int l) {
    Split x = {(__half*)next, two ? (__half*)(next + n) : nullptr, l};
    next += two ? 2 * n : n;
    return x;
  };
  Split X = take(bx, ld), Y = take(bx, ld), A = take(bs, lds), B = take(bs, lds);
  const auto all = [&]() -> cr_status {
    if (type == CR_TYPE_F32) CR_TRY(start((const float*)d_G, ldg, K, N, (Squares*)own, X, stream));
    else if (type == CR_TYPE_F16) CR_TRY(start((const __half*)d_G, ldg, K, N, (Squares*)own, X, stream));
    else CR_TRY(start((const __nv_bfloat16*)d_G, ldg, K, N, (Squares*)own, X, stream));
    const float unit = 1.0f / UNIT;
    for (int q = 0; q < steps; ++q) {
      const bool last = q + 1 == steps;
      Step m = {};
      m.P = m.Q = X;   // A(i, j) = sum of X X^T over columns, or of X^T X over rows
      m.C = A;
      m.I = m.J = s;
      m.K = wide ? N : K;
      m.p_major = m.q_major = !wide;
      m.symmetric = true;
      m.alpha = unit;
      CR_TRY(step_product(m, err, stream));
      m.P = m.Q = m.R = A;   // B = b A + c A A
      m.C = B;
      m.K = s;
      m.p_major = m.q_major = true;
      m.alpha = (float)c * unit;
      m.beta = (float)b;
      CR_TRY(step_product(m, err, stream));
      m.R = X;   // a X + B X, or a X + X B
      m.C = Y;
      m.I = K;
      m.J = N;
      m.P = wide ? B : X;
      m.p_major = wide;
      m.Q = wide ? X : B;
      m.q_major = true;
      m.symmetric = false;
      m.alpha = unit;
      m.beta = (float)a;
      if (last && out_type != CR_TYPE_F32) {
        m.out = d_O;
        m.out_type = out_type;
        m.ldout = ldo;
        m.alpha *= unit;
        m.beta *= unit;
      }
      CR_TRY(step_product(m, err, stream));
      std::swap(X, Y);
    }
    if (out_type == CR_TYPE_F32) {
      const long long words = (long long)((K + 3) / 4) * N;
      TimedScope ts("k_ortho_join", stream);
      CR_CUDA(launch_after(k_ortho_join, (unsigned)std::min<long long>((words + NT - 1) / NT, 8ll * sm_count()), NT, 0, 1, stream, X.hi, X.lo,
                           X.ld, K, N, (float*)d_O, ldo));
      CR_CHECK_LAUNCH("k_ortho_join");
    }
    return CR_OK;
  };
  const cr_status st = all();
  scratch_free(own, stream);
  return st;
  CR_ENTRY_END("cr_orthogonalize")
}
