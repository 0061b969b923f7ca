// Orthogonalised update of a weight matrix by Newton-Schulz products (cr_orthogonalize).
//
// X = G / |G|_F, then X <- a X + (b A + c A^2) X with A = X X^T (X^T X for more rows than columns), `steps` times.  Every
// matrix between two products is FP16 with FP32 sums: 1024 times its value, which keeps entries of up to 64 finite and
// of 2^-24 with 11 bits (X's are about 1 / sqrt(K N)).  FP16 holds three bits more than a BF16 output; for FP16 and FP32
// outputs each matrix is a sum of two FP16 ones (22 bits), and a product three (the one of the two small parts is below
// 2^-22 of it).  A and b A + c A^2 are symmetric: the wide kernel forms half of their tiles and stores them twice.
// Bound by the tensor cores where the matrices are large (4096 x 8192 BF16, five steps: 1510 to 1665 us as the power limit has it,
// 1.6 to 1.45 PFLOP/s with symmetric products counted by half), by the chain of 15 dependent products where they are not (512 x 512 115 us, 2048 x 2048 254 us).
#include <cmath>

#include "product.cuh"

namespace cr {
namespace {

constexpr float UNIT = 1024.0f;   // the matrices hold UNIT times their values
constexpr int MAXPART = 1024;

// Sums of squares of a block's elements to part[block]: of those above 2^48 and below 2^-50 scaled by 2^-90 and 2^90, so
// that no square overflows or underflows, nor 2^31 of them.
struct Squares {
  float big, mid, small;
};
__device__ __forceinline__ void add_square(float x, float& big, float& mid, float& small) {
  const float a = fabsf(x);
  const bool high = a > 0x1p48f, low = a < 0x1p-50f;
  const float b = high ? a * 0x1p-90f : 0.0f, m = high || low ? 0.0f : a, s = low ? a * 0x1p90f : 0.0f;   // NaN goes to the middle
  big = fmaf(b, b, big);
  mid = fmaf(m, m, mid);
  small = fmaf(s, s, small);
}
// n elements: where the largest lies well inside the middle range the others may be added there too, because those that are too
// small for it are below 2^-12 of the largest.
template <int n>
__device__ __forceinline__ void add_squares(const float* x, float& big, float& mid, float& small) {
  float most = fabsf(x[0]);
#pragma unroll
  for (int q = 1; q < n; ++q) most = fmaxf(most, fabsf(x[q]));
  if (most <= 0x1p48f && most >= 0x1p-38f) {
#pragma unroll
    for (int q = 0; q < n; ++q) mid = fmaf(x[q], x[q], mid);
  } else {
#pragma unroll
    for (int q = 0; q < n; ++q) add_square(x[q], big, mid, small);
  }
}
__device__ __forceinline__ Squares warp_sum(Squares s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.big += __shfl_xor_sync(0xffffffffu, s.big, o);
    s.mid += __shfl_xor_sync(0xffffffffu, s.mid, o);
    s.small += __shfl_xor_sync(0xffffffffu, s.small, o);
  }
  return s;
}
// X = ((g f[1]) f[2]) f[0] is UNIT g / |G|_F, zero for a zero matrix and NaN where |G|_F is not finite.  The sum is t 2^U for the
// highest range that holds anything (what is below it by more than FP32's digits drops out), and UNIT / |G|_F is f[0] times a
// power of two that is applied in two halves, which are normal numbers.
__device__ __forceinline__ void scale_of(const Squares& s, float* f) {
  const bool high = s.big != 0.0f, mid = s.mid != 0.0f;
  const float t = high ? s.big + (s.mid * 0x1p-90f) * 0x1p-90f : mid ? s.mid + (s.small * 0x1p-90f) * 0x1p-90f : s.small;
  const int U = high ? 180 : mid ? 0 : -180;
  const int bits = __float_as_int(t), e = ((bits >> 23) - 127) & ~1;   // t / 2^e in [1, 4)
  const float m = __int_as_float(bits - (e << 23));
  f[0] = t == 0.0f ? 0.0f : t - t + 1.0f / sqrtf(m);   // infinity and NaN: NaN
  const int E = 10 - (e + U) / 2, h = E / 2;           // UNIT = 2^10
  f[1] = __int_as_float((h + 127) << 23);
  f[2] = __int_as_float((E - h + 127) << 23);
}
// V elements: 16 bytes, or one.
template <class T, int V>
__device__ __forceinline__ void load_some(const T* p, float* v) {
  if constexpr (V == 1) {
    v[0] = to_float(p[0]);
  } else if constexpr (sizeof(T) == 4) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x;
    v[1] = w.y;
    v[2] = w.z;
    v[3] = w.w;
  } else {
    float w[8];
    widen8(*reinterpret_cast<const Eight<T>*>(p), w);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = w[q];
  }
}
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
    load_some<T, V>(from, x);
    add_squares<V>(x, big, mid, small);
  }
  Squares s = warp_sum(Squares{big, mid, small});
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

// X = UNIT G / |G|_F as FP16 with the rest after it in X2 (may be NULL).
template <class T, int V>
__global__ void __launch_bounds__(NT) k_ortho_scale(const T* G, int ld, int K, int N, const Squares* part, int parts, __half* X, __half* X2, int ldx) {
  __shared__ float factor[3];
  if (threadIdx.x < 32) {
    Squares s = {0.0f, 0.0f, 0.0f};
    for (int q = threadIdx.x; q < parts; q += 32) {
      s.big += part[q].big;
      s.mid += part[q].mid;
      s.small += part[q].small;
    }
    s = warp_sum(s);
    if (threadIdx.x == 0) scale_of(s, factor);
  }
  __syncthreads();
  const float m = factor[0], p1 = factor[1], p2 = factor[2];
  const int per = ldx / 8;
  const long long total = (long long)per * N;
  for (long long e = (long long)blockIdx.x * NT + threadIdx.x; e < total; e += (long long)gridDim.x * NT) {
    const int col = e >> 32 ? (int)(e / per) : (int)((uint32_t)e / (uint32_t)per), i = (int)(e - (long long)col * per) * 8;
    const T* from = G + (size_t)col * ld + i;
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; q += V) {
      if (i + q < K) load_some<T, V>(from + q, x + q);
      else
#pragma unroll
        for (int r = 0; r < V; ++r) x[q + r] = 0.0f;
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

// C = alpha (sum of the parts) + beta R for 32 x 32 outputs, four to a thread, to FP16 with the rest after it in C2 (may be NULL), or
// to the caller's matrix; TRI: C is symmetric, parts hold the 256-wide tiles ti <= tj, and C(j, i) is stored too.  Bound by
// latency and L2: all parts of an output are on their way at once.
constexpr int JTILE = 32;
template <class O>
struct alignas(4 * sizeof(O)) FourOf {
  O x[4];
};
// Four elements of a column from `at` on, the first `n` of them if they are fewer.
template <class O>
__device__ __forceinline__ void put4(O* C, O* C2, size_t at, int n, bool vec, const float (&v)[4]) {
  FourOf<O> o, rest;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    o.x[q] = from_float<O>(v[q]);
    rest.x[q] = from_float<O>(v[q] - to_float(o.x[q]));
  }
  if (vec && n >= 4) {
    *reinterpret_cast<FourOf<O>*>(C + at) = o;
    if (C2) *reinterpret_cast<FourOf<O>*>(C2 + at) = rest;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < n) {
        C[at + q] = o.x[q];
        if (C2) C2[at + q] = rest.x[q];
      }
  }
}
template <class O, bool TRI>
__global__ void __launch_bounds__(NT) k_ortho_sum(const float* part, int parts, int ldp, int jpad, int I, int J, const __half* R, const __half* R2,
                                                  int ldr, float alpha, float beta, O* C, O* C2, int ldc, int vec) {
  __shared__ float turned[TRI ? JTILE : 1][JTILE + 1];
  const int across = (I + JTILE - 1) / JTILE, i0 = (int)(blockIdx.x % across) * JTILE, j0 = (int)(blockIdx.x / across) * JTILE;
  let_next_start();
  wait_for_previous();
  if (TRI && i0 / 256 > j0 / 256) return;
  const int x = threadIdx.x % 8 * 4, y = threadIdx.x / 8, i = i0 + x, j = j0 + y;
  float v[4] = {};
  if (j < J && i < I) {
    const float* from = part + (size_t)j * ldp + i;
    const size_t step = (size_t)jpad * ldp;
    uint2 r = make_uint2(0, 0), r2 = make_uint2(0, 0);
    if (R) r = *reinterpret_cast<const uint2*>(R + (size_t)j * ldr + i);
    if (R2) r2 = *reinterpret_cast<const uint2*>(R2 + (size_t)j * ldr + i);
    float4 z = *reinterpret_cast<const float4*>(from);
#pragma unroll 8
    for (int q = 1; q < parts; ++q) {
      const float4 w = *reinterpret_cast<const float4*>(from + q * step);
      z.x += w.x;
      z.y += w.y;
      z.z += w.z;
      z.w += w.w;
    }
    const float2 a = widen2(r.x, __half{}), b = widen2(r.y, __half{}), c = widen2(r2.x, __half{}), d = widen2(r2.y, __half{});
    v[0] = fmaf(beta, a.x + c.x, z.x * alpha);
    v[1] = fmaf(beta, a.y + c.y, z.y * alpha);
    v[2] = fmaf(beta, b.x + d.x, z.z * alpha);
    v[3] = fmaf(beta, b.y + d.y, z.w * alpha);
    put4(C, C2, (size_t)j * ldc + i, I - i, vec, v);
  }
  if constexpr (!TRI) return;
  if (i0 / 256 == j0 / 256) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) turned[x + q][y] = v[q];
  __syncthreads();
  const int col = i0 + y, row = j0 + x;   // C(row .. row + 3, col)
  if (col < I && row < J) {
    const float t[4] = {turned[y][x], turned[y][x + 1], turned[y][x + 2], turned[y][x + 3]};
    put4(C, C2, (size_t)col * ldc + row, J - row, vec, t);
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
  p.tma_c = ((uintptr_t)p.e.C & 15) == 0 && p.e.ldc % 8 == 0;   // STEP's wide outputs are of 16 bits
  p.vec4 = ((uintptr_t)p.e.C & (4 * type_bytes(out_type) - 1)) == 0 && p.e.ldc % 4 == 0;
  // With two parts a sum has to keep FP32's digits, and the tensor cores' adders cut off what they cannot hold: of the products of two
  // first parts they sum up 3 k-blocks (12 additions) by themselves (2500 x 1001 FP32, five steps: relative error 1.5e-5 with whole
  // sums; by 3 k-blocks 4.4e-6 in 346 us, by 2 3.0e-6 in 371; FP32 products 3.7e-6).  Reading an accumulator out takes about
  // 2 us from its last MMA to its next one, twice as long as three k-blocks' MMAs, and there are two of them.
  const Choice ch = choose<STEP>(s.I, s.J, p.kblocks, s.q_major, s.symmetric, s.P.lo != nullptr);
  p.parts = ch.parts;
  p.chunk = s.P.lo ? 3 : p.kblocks;
  p.jpad = (s.J + 255) / 256 * 256;
  p.triangle = ch.wide && s.symmetric;
  p.bn = ch.bn;
  p.ti = ch.wide ? (s.I + 255) / 256 : (s.I + 127) / 128;
  p.tj = ch.wide ? (s.J + 255) / 256 : (s.J + p.bn - 1) / p.bn;
  p.idesc = ch.wide ? idesc_of(256, 256, false, !p.qk, !p.pk) : idesc_of(128, p.bn, false, !p.pk, !p.qk);
  p.stages = ch.parts ? WSTAGES - 1 : WSTAGES;   // SUMS: twice as many output buffers
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
    const long long n = p.tj, tiles = p.triangle ? n * (n + 1) / 2 : (long long)p.ti * p.tj;
    if (p.parts > 0) {
      Maps<SUMS> maps = {};
      CR_TRY(maps_of(&maps.P, &maps.P2, s.P, s.I, s.p_major, 128));
      CR_TRY(maps_of(&maps.Q, &maps.Q2, s.Q, s.J, s.q_major, 128));
      if (p.parts == 1 && !p.triangle) {   // finished in the kernel
        const auto tile = [&](CUtensorMap* m, const void* x, int type, int ld) {
          return make_tensor_map_2d(m, type, x, s.I, s.J, ld, OROW / type_bytes(type), 32);
        };
        p.tma_c = ((uintptr_t)p.e.C & 15) == 0 && (long long)p.e.ldc * sizeof(O) % 16 == 0;
        if (p.tma_c) CR_TRY(tile(&maps.C, p.e.C, out_type, p.e.ldc));
        if (p.C2) CR_TRY(tile(&maps.C2, p.C2, CR_TYPE_F16, p.e.ldc));
        if (s.R.hi) CR_TRY(tile(&maps.R, s.R.hi, CR_TYPE_F16, s.R.ld));
        if (s.R.lo) CR_TRY(tile(&maps.R2, s.R.lo, CR_TYPE_F16, s.R.ld));
        return launch_wide<SUMS, false, O>(maps, p, tiles, stream);
      }
      const int ldp = (s.I + 3) & ~3;
      float* part = nullptr;
      CR_CUDA(scratch_alloc((void**)&part, (size_t)p.parts * p.jpad * ldp * sizeof(float), stream));
      const auto run = [&]() -> cr_status {
        CR_TRY(make_tensor_map_2d(&maps.C, CR_TYPE_F32, part, s.I, p.parts * p.jpad, ldp, 32, 32));
        CR_TRY((launch_wide<SUMS, false, O>(maps, p, tiles * p.parts, stream)));
        TimedScope ts("k_ortho_sum", stream);
        const int vec = ((uintptr_t)p.e.C & (4 * sizeof(O) - 1)) == 0 && p.e.ldc % 4 == 0;
        const unsigned grid = (unsigned)((long long)((s.I + JTILE - 1) / JTILE) * ((s.J + JTILE - 1) / JTILE));
        const auto sum = [&](auto tri) {
          return launch_after(k_ortho_sum<O, decltype(tri)::value>, grid, NT, 0, 1, stream, part, p.parts, ldp, p.jpad, s.I, s.J, (const __half*)p.e.R,
                              (const __half*)p.R2, s.R.ld, p.alpha, p.beta, (O*)p.e.C, (O*)p.C2, p.e.ldc, vec);
        };
        CR_CUDA(p.triangle ? sum(std::true_type{}) : sum(std::false_type{}));
        CR_CHECK_LAUNCH("k_ortho_sum");
        return CR_OK;
      };
      const cr_status st = run();
      scratch_free(part, stream);
      return st;
    }
    if constexpr (sizeof(O) == 2) {
      Maps<STEP> maps = {};
      CR_TRY(map_of(&maps.P, Operand{s.P.hi, s.I, s.P.ld, s.p_major}, CR_TYPE_F16, s.K, 128));
      CR_TRY(map_of(&maps.Q, Operand{s.Q.hi, s.J, s.Q.ld, s.q_major}, CR_TYPE_F16, s.K, 128));
      if (p.tma_c) CR_TRY(make_tensor_map_2d(&maps.C, out_type, p.e.C, s.I, s.J, p.e.ldc, 64, 32));
      if (s.R.hi) CR_TRY(make_tensor_map_2d(&maps.R, CR_TYPE_F16, s.R.hi, s.I, s.J, s.R.ld, 64, 32));
      if (p.triangle) CR_TRY(make_tensor_map_2d_plain(&maps.T, CR_TYPE_F16, p.e.C, s.J, s.I, p.e.ldc, 32, 64));
      return launch_wide<STEP, false, O>(maps, p, tiles, stream);
    }
    return fail_literal(CR_ERR_STATE, "cr_orthogonalize: FP32 comes from the sums");
  };
  return out_type == CR_TYPE_F32 ? go(float{}) : out_type == CR_TYPE_BF16 ? go(__nv_bfloat16{}) : go(__half{});
}

template <class T>
cr_status start(const T* G, int ld, int K, int N, Squares* part, const Split& X, cudaStream_t stream) {
  constexpr int W = 16 / (int)sizeof(T);
  const bool vec = ((uintptr_t)G & 15) == 0 && ld % W == 0 && K % W == 0;
  const long long items = (long long)(vec ? K / W : K) * N;
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
  return vec ? go(std::integral_constant<int, W>{}) : go(std::integral_constant<int, 1>{});
}

// ---------------------------------------------------------------- small matrices
// Up to 128 rows on the short side: one cluster does all steps.  Each CTA keeps a slab of the long side's columns n of X (L,
// a multiple of 128) in shared memory, [i / 64][n][i % 64] in the 128-byte swizzle, which the tensor cores read as rows i with
// k = n (A = X X^T) and as rows n with k = i (X^T B).  The CTAs' parts of A are joined through shared memory of the cluster, in
// the order of the CTAs: each sums the rows that it owns and hands them to all.  B takes A's place, X' X's.  B has two parts for a BF16
// output too: its rounding is a third of the error where one side is much longer than the other, and eight more MMAs are
// little here (the second part takes the place of the sums, which have been read).
// Bound by the chain of products, exchanges and barriers: 128 x 128 to BF16 25 us, 3 us a step, to FP32 43 us; 128 x 2048, by 16
// CTAs, 51 to 55 us, 8.5 us a step.  Launched separately, the 17 kernels of 128 x 128 took 166 us.
constexpr int SROWS = 128, STHREADS = 256, SCLUSTER = 16;
constexpr int SA = SROWS * SROWS * 2;   // bytes of A's FP16 part, [j / 64][i][j % 64]
constexpr int SSUMS = SROWS * SROWS * 4;   // the CTA's sums for A
struct SmallBars {
  uint64_t product, block[4];
  uint32_t tmem;
  float sums[SCLUSTER][3], warps[STHREADS / 32][3];
  float factor[3];
};
struct Small {
  const void* G;
  int ldg, K, N, steps, L, ncta;
  int alias;   // the sums in A's two parts, where there is no room beside them: one more barrier per step
  float a, b, c;
  void* O;
  int ldo;
  unsigned long long limit;
  int* err;
};
__host__ __device__ constexpr int small_smem(int L, bool pairs, bool alias) {
  return 1024 + (L * SROWS * 2 + (alias ? 0 : SA)) * (pairs ? 2 : 1) + SSUMS + (int)sizeof(SmallBars);
}
constexpr bool small_alias(int L, bool pairs) { return small_smem(L, pairs, false) > 227 * 1024; }

__device__ __forceinline__ void fence_proxies() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_cluster2(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
// Descriptor of a rows-contiguous operand whose 64-row blocks are `stride` bytes apart (tile_desc's are ATOM apart).
__device__ __forceinline__ uint64_t rows_desc(uint32_t saddr, int stride) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(stride >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Byte of element col (a multiple of 8 for 16-byte accesses) of a 64-element row in the 128-byte swizzle.
__device__ __forceinline__ int swizzled(int row, int col) { return row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2; }

// v to FP16, what is left to a second one.
template <bool PAIRS>
__device__ __forceinline__ void put8(uint8_t* hi, int lo, int at, float (&v)[8]) {
  const Eight<__half> h = narrow8<__half>(v);
  *reinterpret_cast<Eight<__half>*>(hi + at) = h;
  if (PAIRS) {
    float w[8];
    widen8(h, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] -= w[q];
    *reinterpret_cast<Eight<__half>*>(hi + lo + at) = narrow8<__half>(v);
  }
}
template <bool PAIRS>
__device__ __forceinline__ void get8(const uint8_t* hi, int lo, int at, float (&v)[8]) {
  widen8(*reinterpret_cast<const Eight<__half>*>(hi + at), v);
  if (PAIRS) {
    float w[8];
    widen8(*reinterpret_cast<const Eight<__half>*>(hi + lo + at), w);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += w[q];
  }
}

template <class T, class O, bool PAIRS>
__global__ void __launch_bounds__(STHREADS, 1) k_ortho_small(const Small p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int L = p.L, half = L * 128, xlo = 2 * half;   // bytes of 64 rows of X, of a part of X
  uint8_t *X = smem, *A = X + (PAIRS ? 2 : 1) * xlo, *P = p.alias ? A : A + (PAIRS ? 2 : 1) * SA;   // P: this CTA's sums for A
  SmallBars* bars = reinterpret_cast<SmallBars*>(P + SSUMS);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = p.ncta > 1 ? (int)cluster_rank() : 0;
  const bool wide = p.K <= p.N;
  const int s = wide ? p.K : p.N, l = wide ? p.N : p.K, n0 = rank * L, cols = max(0, min(L, l - n0));
  // PAIRS: two accumulators for each sum, the second half of the large products in the second one: half as long a chain of the
  // tensor cores' additions, which cut off what they cannot hold
  const uint32_t second = L <= 128 ? 128 : 256, tcols = PAIRS ? 2 * second : L <= 128 ? 128 : L <= 256 ? 256 : 512;
  if (threadIdx.x == 0) {
    mbar_init(&bars->product, 1);
    for (int m = 0; m < 4; ++m) mbar_init(&bars->block[m], 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars->tmem, tcols);
  if (p.ncta > 1) cluster_arrive_relaxed();   // waited for before the first access to another CTA
  for (int e = threadIdx.x; e < (PAIRS ? 2 : 1) * xlo / 16; e += STHREADS) reinterpret_cast<uint4*>(X)[e] = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);
  wait_for_previous();
  let_next_start();
  const auto together = [&] {   // all threads of the cluster
    if (p.ncta > 1) cluster_sync_all();
    else __syncthreads();
  };

  // G's elements of the slab, 128 x 128 at a time: lanes along its columns, warps across them, all of a thread's on their way at
  // once.  The last ones stay in registers, the others come a second time from L2.
  const T* G = (const T*)p.G + (wide ? (size_t)n0 * p.ldg : n0);
  const int inner = wide ? s : cols, outer = wide ? cols : s;
  {
    float g[4][16];
    const auto load = [&](int x0, int y0) {
#pragma unroll
      for (int b = 0; b < 16; ++b)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int x = x0 + 32 * a + lane, y = y0 + 8 * b + warp;
          g[a][b] = x < inner && y < outer ? to_float(G[(size_t)y * p.ldg + x]) : 0.0f;
        }
    };
    float big = 0.0f, mid = 0.0f, small = 0.0f;
    int lx = -1, ly = -1;   // what is in g
    for (int y0 = 0; y0 < outer; y0 += 128)
      for (int x0 = 0; x0 < inner; x0 += 128) {
        load(x0, y0);
        lx = x0;
        ly = y0;
#pragma unroll
        for (int a = 0; a < 4; ++a) add_squares<16>(g[a], big, mid, small);
      }
    Squares sum = warp_sum(Squares{big, mid, small});
    if (lane == 0) {
      bars->warps[warp][0] = sum.big;
      bars->warps[warp][1] = sum.mid;
      bars->warps[warp][2] = sum.small;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
      float x = 0.0f;
      for (int w = 0; w < STHREADS / 32; ++w) x += bars->warps[w][threadIdx.x];
      bars->sums[rank][threadIdx.x] = x;
    }
    if (p.ncta > 1) {
      cluster_wait();
      __syncthreads();
      if ((int)threadIdx.x < 3 * p.ncta) {   // to every CTA
        const float x = bars->sums[rank][threadIdx.x % 3];
        const uint32_t to = cluster_addr(smem_u32(&bars->sums[rank][threadIdx.x % 3]), threadIdx.x / 3);
        if ((int)threadIdx.x / 3 != rank) store_cluster(to, __float_as_uint(x));
      }
    }
    together();
    if (threadIdx.x == 0) {
      Squares all = {0.0f, 0.0f, 0.0f};
      for (int r = 0; r < p.ncta; ++r) {
        all.big += bars->sums[r][0];
        all.mid += bars->sums[r][1];
        all.small += bars->sums[r][2];
      }
      scale_of(all, bars->factor);
    }
    __syncthreads();
    const float m = bars->factor[0], p1 = bars->factor[1], p2 = bars->factor[2];
    for (int y0 = ly; y0 >= 0; y0 -= 128)
      for (int x0 = lx; x0 >= 0; x0 -= 128) {
        if (x0 != lx || y0 != ly) load(x0, y0);
#pragma unroll
        for (int b = 0; b < 16; ++b)
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const int x = x0 + 32 * a + lane, y = y0 + 8 * b + warp;
            if (x < inner && y < outer) {
              const float v = g[a][b] * p1 * p2 * m;
              const int i = wide ? x : y, n = wide ? y : x, at = i / 64 * half + swizzled(n, i % 64);
              const __half hi = __float2half_rn(v);
              *reinterpret_cast<__half*>(X + at) = hi;
              if (PAIRS) *reinterpret_cast<__half*>(X + xlo + at) = __float2half_rn(v - __half2float(hi));
            }
          }
      }
  }
  fence_proxies();
  __syncthreads();

  const uint32_t rows_id = idesc_of(128, 128, false, true, true), k_id = idesc_of(128, 128, false, false, false);
  const uint32_t sx = smem_u32(X), sa = smem_u32(A), sums = smem_u32(P);
  constexpr int SEGS = PAIRS ? 3 : 1;
  // parts of the first and second operand, the small products first
  const auto first_lo = [](int seg) { return PAIRS && seg == 1; };
  const auto second_lo = [](int seg) { return PAIRS && seg == 0; };
  uint32_t turn = 0;
  const auto landed = [&](uint64_t* bar, uint32_t parity) {   // MMAs need nobody's help: late ones are reported, and waited for
    if (!mbar_wait(bar, parity, p.limit)) {
      *(volatile int*)p.err = 1;
      __threadfence_system();
      mbar_wait(bar, parity, LANDING_NS);
    }
    tc_fence_after();
    __syncwarp();
  };
  const float unit = 1.0f / UNIT;
  const int quad = warp & 3, side = warp >> 2, row = quad * 32 + lane;   // TMEM lane, and which 64 columns
  const auto sums_of = [&](int col, bool two, float (&v)[64]) {   // this thread's 64 columns of an accumulator, or of both
    const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + col + side * 64;
    uint32_t u[2][32];
    tmem_ld32(from, u[0]);
    tmem_ld32(from + 32, u[1]);
    tmem_ld_wait();
#pragma unroll
    for (int x = 0; x < 64; ++x) v[x] = __uint_as_float(u[x / 32][x % 32]);
    if (PAIRS && two) {
#pragma unroll
      for (int y = 0; y < 64; y += 16) {
        float w[16];
        tmem_ld16(from + second + y, w);
#pragma unroll
        for (int x = 0; x < 16; ++x) v[y + x] += w[x];
      }
    }
  };
  for (int step = 0; step < p.steps; ++step) {
    // A's part of this slab
    if (warp == 0 && elect_one()) {
      const uint64_t d0 = rows_desc(sx, half);
      const int ks = max(1, (cols + 15) / 16);   // columns that are not there are zero
      for (int seg = 0; seg < SEGS; ++seg) {
        const uint64_t da = d0 + (first_lo(seg) ? xlo >> 4 : 0), db = d0 + (second_lo(seg) ? xlo >> 4 : 0);
        for (int k = 0; k < ks; ++k) {
          const bool late = PAIRS && seg == 2 && k >= (ks + 1) / 2;
          mma_any<false, false>(late ? tmem + second : tmem, da + k * 128, db + k * 128, rows_id, late ? k > (ks + 1) / 2 : (seg | k) != 0);
        }
      }
      mma_commit(&bars->product);
    }
    __syncwarp();
    landed(&bars->product, turn);
    turn ^= 1;
    {
      float v[64];
      sums_of(0, (cols + 15) / 16 >= 2, v);
      if (p.ncta == 1) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float w[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) w[x] = v[8 * q + x] * unit;
          put8<PAIRS>(A, SA, side * SA / 2 + swizzled(row, 8 * q), w);
        }
      } else {   // 16-byte word w of row i at w ^ (i & 31)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          *reinterpret_cast<float4*>(P + row * 512 + (((side * 16 + q) ^ (row & 31)) << 4)) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    }
    if (p.ncta > 1) {
      cluster_sync_all();
      const auto exchange = [&](auto nc) {   // 16 words of 16 bytes from other CTAs to a thread, all on their way at once
        constexpr int NC = decltype(nc)::value, OWN = SROWS / NC, WORDS = 16 / NC;
        float4 x[WORDS][NC];
#pragma unroll
        for (int q = 0; q < WORDS; ++q) {
          const int e = threadIdx.x + q * STHREADS, i = rank * OWN + e / 32;
#pragma unroll
          for (int r = 0; r < NC; ++r) x[q][r] = load_cluster4(cluster_addr(sums + i * 512 + ((e % 32 ^ (i & 31)) << 4), r));
        }
        if (p.alias) cluster_sync_all();   // the sums have been read: A may take their place
#pragma unroll
        for (int q = 0; q < WORDS; ++q) {
          float4 z = x[q][0];
#pragma unroll
          for (int r = 1; r < NC; ++r) {
            z.x += x[q][r].x;
            z.y += x[q][r].y;
            z.z += x[q][r].z;
            z.w += x[q][r].w;
          }
          const int e = threadIdx.x + q * STHREADS, i = rank * OWN + e / 32, j = e % 32 * 4, at = j / 64 * (SA / 2) + swizzled(i, j % 64);
          const float v[4] = {z.x * unit, z.y * unit, z.z * unit, z.w * unit};
          const uint32_t h0 = narrow2(v[0], v[1], __half{}), h1 = narrow2(v[2], v[3], __half{});
          uint32_t l0 = 0, l1 = 0;
          if (PAIRS) {
            const float2 f0 = widen2(h0, __half{}), f1 = widen2(h1, __half{});
            l0 = narrow2(v[0] - f0.x, v[1] - f0.y, __half{});
            l1 = narrow2(v[2] - f1.x, v[3] - f1.y, __half{});
          }
#pragma unroll
          for (int r = 0; r < NC; ++r) {
            store_cluster2(cluster_addr(sa + at, r), h0, h1);
            if (PAIRS) store_cluster2(cluster_addr(sa + SA + at, r), l0, l1);
          }
        }
      };
      if (p.ncta == 2) exchange(std::integral_constant<int, 2>{});
      else if (p.ncta == 4) exchange(std::integral_constant<int, 4>{});
      else if (p.ncta == 8) exchange(std::integral_constant<int, 8>{});
      else exchange(std::integral_constant<int, 16>{});
    }
    fence_proxies();
    tc_fence_before();
    together();
    tc_fence_after();
    fence_proxies();
    // A A
    if (warp == 0 && elect_one()) {
      const uint64_t d0 = tile_desc(sa, true);
      for (int seg = 0; seg < SEGS; ++seg) {
        const uint64_t da = d0 + (first_lo(seg) ? SA >> 4 : 0), db = d0 + (second_lo(seg) ? SA >> 4 : 0);
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = (k / 4 * (SA / 2) >> 4) + k % 4 * 2;
          const bool late = PAIRS && seg == 2 && k >= 4;
          mma_any<false, false>(late ? tmem + second : tmem, da + at, db + at, k_id, late ? k > 4 : (seg | k) != 0);
        }
      }
      mma_commit(&bars->product);
    }
    __syncwarp();
    landed(&bars->product, turn);
    turn ^= 1;
    {   // B in A's place
      float v[64];
      sums_of(0, true, v);
      const float c = p.c * unit;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float w[8];
        const int at = side * SA / 2 + swizzled(row, 8 * q);
        get8<PAIRS>(A, SA, at, w);
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] = fmaf(p.b, w[x], c * v[8 * q + x]);
        put8<true>(A, SA, at, w);
      }
    }
    fence_proxies();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // X^T B, 128 columns of X at a time
    const int blocks = max(1, (cols + 127) / 128);
    if (warp == 0 && elect_one()) {
      const uint64_t dx = tile_desc(sx, true), d0 = tile_desc(sa, true);
      for (int m = 0; m < blocks; ++m) {
        for (int seg = 0; seg < (PAIRS ? 3 : 2); ++seg) {
          const uint64_t da = dx + (first_lo(seg) ? xlo >> 4 : 0) + m * (128 * 128 >> 4), db = d0 + (seg == 0 ? SA >> 4 : 0);
          for (int k = 0; k < 8; ++k) {
            const bool late = PAIRS && seg == 2 && k >= 4;
            mma_any<false, false>((late ? tmem + second : tmem) + m * 128, da + (k / 4 * half >> 4) + k % 4 * 2,
                                  db + (k / 4 * (SA / 2) >> 4) + k % 4 * 2, k_id, late ? k > 4 : (seg | k) != 0);
          }
        }
        mma_commit(&bars->block[m]);
      }
    }
    __syncwarp();
    const bool last = step + 1 == p.steps;
    for (int m = 0; m < blocks; ++m) {
      landed(&bars->block[m], step & 1);
      float v[64];
      sums_of(m * 128, true, v);
      const int n = m * 128 + row;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float w[8];
        const int at = side * half + swizzled(n, 8 * q);
        get8<PAIRS>(X, xlo, at, w);
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] = fmaf(p.a, w[x], unit * v[8 * q + x]);
        if (!last) {
          put8<PAIRS>(X, xlo, at, w);
        } else if (!wide) {
          if (n < cols) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const int i = side * 64 + 8 * q + x;
              if (i < s) ((O*)p.O)[(size_t)i * p.ldo + n0 + n] = from_float<O>(w[x] * unit);
            }
          }
        } else {   // to X's place, FP32 in halves, and from there with lanes along the columns
          uint32_t hi[4], lo[4] = {};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if constexpr (sizeof(O) == 4) {
              const uint32_t f0 = __float_as_uint(w[2 * x] * unit), f1 = __float_as_uint(w[2 * x + 1] * unit);
              hi[x] = f0 >> 16 | (f1 & 0xffff0000u);
              lo[x] = (f0 & 0xffffu) | f1 << 16;
            } else {
              hi[x] = narrow2(w[2 * x] * unit, w[2 * x + 1] * unit, O{});
            }
          }
          *reinterpret_cast<uint4*>(X + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if (sizeof(O) == 4) *reinterpret_cast<uint4*>(X + xlo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    }
    fence_proxies();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (wide)
#pragma unroll 4
    for (int n = warp; n < cols; n += STHREADS / 32)
#pragma unroll
      for (int k = 0; k < SROWS / 32; ++k) {
        const int i = lane + 32 * k, at = i / 64 * half + swizzled(n, i % 64);
        if (i >= s) continue;
        O* to = (O*)p.O + (size_t)(n0 + n) * p.ldo + i;
        if constexpr (sizeof(O) == 4)
          *to = __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(X + at) << 16 | *reinterpret_cast<const uint16_t*>(X + xlo + at));
        else *to = *reinterpret_cast<const O*>(X + at);
      }
  if (warp == 1) tmem_dealloc(tmem, tcols);
}

// The largest cluster that the current device can run with a CTA of this kernel per SM (16 is not portable; 8 is).
int largest_cluster() {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::atomic<int>& k = known[dev & 63];
  if (k.load(std::memory_order_relaxed) == 0) {
    const auto kernel = k_ortho_small<float, __nv_bfloat16, false>;
    cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = SCLUSTER;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(SCLUSTER);
    cfg.blockDim = dim3(STHREADS);
    cfg.dynamicSmemBytes = 227 * 1024;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) cudaGetLastError();
    k.store(n > 0 ? SCLUSTER : SCLUSTER / 2, std::memory_order_relaxed);
  }
  return k.load(std::memory_order_relaxed);
}

template <class T, class O, bool PAIRS>
cr_status launch_small(const Small& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  CR_TRY(allow_shared((const void*)k_ortho_small<T, O, PAIRS>, 227 * 1024, done, true));
  TimedScope ts("k_ortho_small", stream);
  CR_CUDA(launch_after(k_ortho_small<T, O, PAIRS>, p.ncta, STHREADS, small_smem(p.L, PAIRS, p.alias), p.ncta, stream, p));
  CR_CHECK_LAUNCH("k_ortho_small");
  return CR_OK;
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
  const int across = std::min(K, N), along = std::max(K, N);
  if (across <= SROWS && along <= largest_cluster() * (two ? 256 : 512)) {
    Small p = {d_G, ldg, K, N, steps, 0, 1, 0, (float)a, (float)b, (float)c, d_O, ldo, option_wait_ns(), err};
    while (p.ncta < largest_cluster() && along > 128 * p.ncta) p.ncta *= 2;
    p.L = ((along + p.ncta - 1) / p.ncta + 127) / 128 * 128;
    p.alias = small_alias(p.L, two);
    return with_type(type, [&](auto t0) -> cr_status {
      using T = decltype(t0);
      if (out_type == CR_TYPE_F32) return launch_small<T, float, true>(p, stream);
      if (out_type == CR_TYPE_F16) return launch_small<T, __half, true>(p, stream);
      return launch_small<T, __nv_bfloat16, false>(p, stream);
    });
  }
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
      if (last) {
        m.out = d_O;
        m.out_type = out_type;
        m.ldout = ldo;
        m.alpha *= unit;
        m.beta *= unit;
      }
      CR_TRY(step_product(m, err, stream));
      std::swap(X, Y);
    }
    return CR_OK;
  };
  const cr_status st = all();
  scratch_free(own, stream);
  return st;
  CR_ENTRY_END("cr_orthogonalize")
}
