// Group norm over packed fields with an activation, and its gradient (cr_group_norm, cr_group_norm_backward).
//
// A group of a field is the field's columns times the group's consecutive features.  Two kernels: the first leaves each
// tile's share of every group's mean and sum of squared deviations (each formed about the share's own mean, so that a
// large common value costs no digits), the second joins the shares of the groups that its tile needs, in a fixed order,
// and goes over the tile again.  The gradient does the same with its two sums.  Bound by HBM, X read twice where it does not
// stay in L2, and by 4 us of each launch's set-up and joins: 8 fields of 16384 x 1024 BF16 with silu 142 us; 37 ragged
// fields of 50021 x 512 FP16 with gelu 43 us; the gradient of 11 fields of 40963 x 640 BF16
// with silu 63 us.  Fewer and larger tiles than one round of resident blocks leave SMs idle, more and smaller ones pay the set-up
// again (the first case by 256-column tiles 168 us).
#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "ptx.cuh"

namespace cr {
namespace {

constexpr int NT = 256;
constexpr float FINITE = 3.402823466e38f;   // the largest
constexpr int SMALL = 12;   // k_gnorm_small: accesses of a thread, if one field had all columns
// Blocks that share an SM, and columns of a batch: forward two with 6 (8 fields of 16384 x 1024 BF16 silu, 4 of FP32, 37 ragged fields of
// 50021 x 512 FP16 gelu, 20000 x 96 FP16: 142, 130, 45, 15 us; three with 4 163, 136, 51, 17; two with 4 147, 139, 47, 14; two with
// 8 143, 129, 51, 15).  Backward two with 6 (4 of FP32), in tiles of whole pairs: 131072 x 1024 BF16 silu 248 us, 40963 x 640 60,
// 20000 x 96 15, 30000 x 320 FP16 in 200 fields 44; three with 4 (2), in tiles of whole batches, 263, 67, 17, 46; two with 6 in
// tiles of whole batches 249, 62, 18, 50.
constexpr int FORWARD = 2, BATCH = 6, BACKWARD = 2;
template <class T>
constexpr int BACKWARD_BATCH = sizeof(T) == 2 ? 6 : 4;

// Tile (fb, t): features fb * TX * V on, columns t * cols on.  Threads: TX along features, V consecutive ones each
// (V = 8: 16-byte accesses for 16-bit types), NT / TX along columns.
struct Fields {
  const int32_t* off;   // NULL: one field of T columns
  int n, T;
  int D, group, groups;   // features; of a group
  int cols, tiles, blocks;   // columns of a tile, tiles along columns and along features
};
__device__ __forceinline__ int field_begin(const Fields& p, int f) {   // clamped: no offset leads out of the matrix
  return p.off ? min(max(p.off[f], 0), p.T) : f == 0 ? 0 : p.T;
}
// The first field that ends at c or later; by all threads of the block.
__device__ int first_field(const Fields& p, int c) {
  if (!p.off) return 0;
  int lo = 0, hi = p.n;
  while (hi > lo) {
    const int step = (hi - lo + NT - 1) / NT;
    const long long at = lo + (threadIdx.x + 1ll) * step - 1;
    const int k = __syncthreads_count(at < hi && field_begin(p, (int)at + 1) < c);
    lo += k * step;
    if (step == 1) break;
    hi = min(hi, lo + step);
  }
  return lo;
}
// The tile's share of field f is slot (t + f), that of group g in feature block fb slot (fb + g): both pairs only go up.
__device__ __forceinline__ size_t share(const Fields& p, int t, int f, int fb, int g) {
  return (size_t)(t + f) * ((size_t)p.blocks + p.groups) + fb + g;
}
size_t shares(const Fields& p) { return (size_t)(p.tiles + p.n) * ((size_t)p.blocks + p.groups); }

// V elements as they are in memory.  They are loaded in batches of columns before any is used or stored: the compiler may not
// move a load of X above a store to Y, which may be the same matrix.
template <class T, int V>
struct alignas(V * sizeof(T)) Raw {
  uint32_t w[V * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T* p) { *this = *reinterpret_cast<const Raw*>(p); }
  __device__ __forceinline__ void widen(float (&v)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 f = widen2(w[e / 2], T{});
        v[e] = f.x;
        v[e + 1] = f.y;
      }
    }
  }
};
template <class T>
struct Raw<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void widen(float (&v)[1]) const { v[0] = to_float(w); }
};
template <class T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    p[0] = from_float<T>(v[0]);
  } else {
    Raw<T, V> o;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < V; ++e) o.w[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 2) o.w[e / 2] = narrow2(v[e], v[e + 1], T{});
    }
    *reinterpret_cast<Raw<T, V>*>(p) = o;
  }
}
template <class T, int V>
struct Pair {
  Raw<T, V> x, d;
};
// The thread's columns a, a + TY, .. < b in batches of B, each loaded before the one before it is used: load(buffer, elements past
// the first column's), use(batch, column, how many).
template <int B, int TY, class Buf, class L, class U>
__device__ __forceinline__ void in_batches(int a, int b, L&& load, U&& use) {
  const int count = a < b ? (b - a + TY - 1) / TY : 0, full = count / B;
  Buf now[B], next[B];
  if (full > 0) {
#pragma unroll
    for (int q = 0; q < B; ++q) load(now[q], q * TY);
  }
#pragma unroll 2
  for (int k = 1; k <= full; ++k) {
    if (k < full) {
#pragma unroll
      for (int q = 0; q < B; ++q) load(next[q], (k * B + q) * TY);
    }
    use(now, (k - 1) * B * TY, std::integral_constant<int, B>{});
#pragma unroll
    for (int q = 0; q < B; ++q) now[q] = next[q];
  }
  const int left = count - full * B, at = full * B * TY;
#pragma unroll
  for (int q = 0; q < B - 1; ++q)
    if (q < left) load(now[q], at + q * TY);
#pragma unroll
  for (int q = 0; q < B - 1; ++q)
    if (q < left) use(reinterpret_cast<const Buf(&)[1]>(now[q]), at + q * TY, std::integral_constant<int, 1>{});
}
template <int V>
__device__ __forceinline__ Floats<V == 1 ? 1 : 2> pair_at(const float (&v)[V], int e) {
  if constexpr (V == 1) return {{v[0]}};
  else return {{v[e], v[e + 1]}};
}

// A block's groups g0 .. g1 are reduced by as many threads each as there are, 8 to 32: use(g, lane, lanes), all threads of a warp
// together; g may pass g1 in the last turn.
__device__ __forceinline__ float lanes_sum(float x, int lanes) {
  if (lanes > 16) x += __shfl_xor_sync(0xffffffffu, x, 16);
  if (lanes > 8) x += __shfl_xor_sync(0xffffffffu, x, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <class U>
__device__ __forceinline__ void each_group(int g0, int g1, U&& use) {
  const int shift = g1 - g0 < NT / 32 ? 5 : g1 - g0 < NT / 16 ? 4 : 3, lanes = 1 << shift, lane = threadIdx.x & (lanes - 1);
  for (int g = g0 + ((int)threadIdx.x >> shift); g - ((int)(threadIdx.x & 31) >> shift) <= g1; g += NT >> shift) use(g, lane, lanes);
}
// The groups of V features from i on.
template <int V, class U>
__device__ __forceinline__ void each_feature(const Fields& p, int i, U&& use) {
  int g = i / p.group, r = i - g * p.group;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    use(e, g);
    if (++r == p.group) {
      r = 0;
      ++g;
    }
  }
}

// Calls run(f, a, b, begin, end) for the columns a .. b - 1 inside the tile of field f, begin .. end - 1, and none(f) for empty fields, each by one tile.
template <class R, class E>
__device__ __forceinline__ void each_field(const Fields& p, int t, R&& run, E&& none) {
  const int c0 = t * p.cols, c1 = min(p.T, c0 + p.cols);
  const bool last = t + 1 == p.tiles;
  for (int f = first_field(p, c0); f < p.n; ++f) {
    const int begin = field_begin(p, f), end = field_begin(p, f + 1);
    if (begin >= c1 && !last) break;
    const int a = max(begin, c0), b = min(end, c1);
    if (a < b) run(f, a, b, begin, end);
    else if (begin >= end && begin >= c0) none(f);
  }
}

// To [-high, high] in one instruction; NaN stays, or becomes high.
template <bool NAN_STAYS>
__device__ __forceinline__ float clamp_both(float x, float high) {
  if (NAN_STAYS) asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(x) : "f"(high));
  else asm("min.xorsign.abs.f32 %0, %0, %1;" : "+f"(x) : "f"(high));
  return x;
}
// Activations (SLOPE: their slopes) as in ops.cuh from one reciprocal each: denominator(z) gives what result() needs the reciprocal
// of.  So that the product of two denominators does not overflow, silu's are 1 + e^-|z|, with
// silu(z) = max(z, 0) - |z| e^-|z| / (1 + e^-|z|); where e^-|z| is flushed to 0 the function has reached its limit.
template <int ACT, bool SLOPE, int P>
struct Curve {
  Floats<P> z, w;   // z, or max(z, 0); silu: e^-|z|, or -|z| e^-|z|; gelu: |z|
  __device__ __forceinline__ Floats<P> denominator(Floats<P> x) {
    if constexpr (ACT == CR_ACT_SILU) {
      Floats<P> c;   // the argument, clamped; a value's NaN is in z alone, so that the other value does not meet it
#pragma unroll
      for (int o = 0; o < P; ++o) c.x[o] = clamp_both<SLOPE>(x.x[o], 88.0f);
      w = mul(c, all_of<P>(LOG2E));
#pragma unroll
      for (int o = 0; o < P; ++o) {
        w.x[o] = exp2_fast(-fabsf(w.x[o]));
        z.x[o] = SLOPE ? c.x[o] : clamp_low(x.x[o], 0.0f);
      }
      const Floats<P> d = add(w, all_of<P>(1.0f));
      if (!SLOPE) {
#pragma unroll
        for (int o = 0; o < P; ++o) w.x[o] = __fmul_rn(w.x[o], -fabsf(c.x[o]));
      }
      return d;
    } else {
      if (SLOPE) {
#pragma unroll
        for (int o = 0; o < P; ++o) {
          z.x[o] = clamp_both<true>(x.x[o], 30.0f);
          w.x[o] = fabsf(z.x[o]);
        }
      } else {   // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|))
#pragma unroll
        for (int o = 0; o < P; ++o) {
          w.x[o] = fminf(fabsf(x.x[o]), 30.0f);
          z.x[o] = clamp_low(x.x[o], 0.0f);
        }
      }
      return tail_denominator(w);
    }
  }
  __device__ __forceinline__ Floats<P> result(Floats<P> t) const {
    if constexpr (ACT == CR_ACT_SILU) {
      if constexpr (SLOPE) {
        Floats<P> top;   // of sigmoid(z) = top / (1 + e^-|z|)
#pragma unroll
        for (int o = 0; o < P; ++o) top.x[o] = z.x[o] < 0.0f ? w.x[o] : 1.0f;
        return mul(t, fma(z, mul(w, t), top));
      } else {
        return fma(w, t, z);
      }
    } else {
      Floats<P> g;
      const Floats<P> m = minus_tail(w, t, g);
      if constexpr (SLOPE) {
        Floats<P> phi;
#pragma unroll
        for (int o = 0; o < P; ++o) phi.x[o] = z.x[o] < 0.0f ? -m.x[o] : 1.0f + m.x[o];
        return fma(mul(z, all_of<P>(0.39894228040143268f)), g, phi);
      } else {
        return fma(w, m, z);
      }
    }
  }
};
// z = act(z), or its slope, for P features of C columns.  Reciprocals of two values come from one instruction, whose throughput
// (one warp in 8 cycles and SM quarter, like 2^x's) bounds kernels that do little else: 1/x = y / (x y), within about 2^-22.  The two
// are a feature's in two columns of a field: neighbouring features may be of different groups, which know nothing of
// one another, not even a NaN.  In a thread of ONE_GROUP they are the features', each NaN kept to its own.
template <int ACT, bool SLOPE, bool ONE_GROUP, int P, int C>
__device__ __forceinline__ void curve(Floats<P> (&z)[C]) {
  static_assert(C == 1 || (C == 2 && !ONE_GROUP), "one or two columns");
  if constexpr (ACT == CR_ACT_SILU || ACT == CR_ACT_GELU) {
    Curve<ACT, SLOPE, P> k[C];
    Floats<P> d[C];
#pragma unroll
    for (int c = 0; c < C; ++c) d[c] = k[c].denominator(z[c]);
    if constexpr (C == 2) {
      const Floats<P> r = rcp_fast(mul(d[0], d[1]));
      z[0] = k[0].result(mul(r, d[1]));
      z[1] = k[1].result(mul(r, d[0]));
    } else if constexpr (P == 2 && ONE_GROUP) {
      const float a = fmaxf(d[0].x[0], 1.0f), b = fmaxf(d[0].x[1], 1.0f), r = rcp_fast(__fmul_rn(a, b));   // 1 for NaN, which z keeps
      z[0] = k[0].result(Floats<P>{{__fmul_rn(r, b), __fmul_rn(r, a)}});
    } else {
      z[0] = k[0].result(rcp_fast(d[0]));
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (!SLOPE) z[c] = activate<ACT, P>(z[c]);
      else
#pragma unroll
        for (int o = 0; o < P; ++o) z[c].x[o] = activation_slope<ACT>(z[c].x[o]);
    }
  }
}

// ---------------------------------------------------------------- forward
template <class T, int TX, int V>
__global__ void __launch_bounds__(NT, FORWARD) k_gnorm_stats(const T* X, int ldx, const Fields p, float2* part) {
  constexpr int TY = NT / TX, FW = TX * V;
  __shared__ float2 red[TY][FW];   // of a thread's features
  __shared__ float2 feature[FW];
  const int fb = blockIdx.x % p.blocks, t = blockIdx.x / p.blocks;
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, i0 = fb * FW, i = i0 + tx * V;
  const int width = min(FW, p.D - i0);
  let_next_start();
  wait_for_previous();
  each_field(p, t, [&](int f, int a, int b, int begin, int end) {
    float mean[V] = {}, m2[V] = {}, n = 0.0f;
    if (i < p.D) {
      constexpr int B = BATCH, P = V > 1 ? 2 : 1;
      const T* from = X + (size_t)(a + ty) * ldx + i;
      in_batches<B, TY, Raw<T, V>>(a + ty, b, [&](Raw<T, V>& raw, int j) { raw.load(from + (size_t)j * ldx); },
                                   [&](const auto& raw, int, auto count) {   // the batch's own mean and deviations, joined to what is there
        constexpr int C = decltype(count)::value;
        float x[C][V];
#pragma unroll
        for (int q = 0; q < C; ++q) raw[q].widen(x[q]);
        const float w = __fdividef(C, n + C), nw = n * w;
        n += C;
#pragma unroll
        for (int e = 0; e < V; e += P) {
          Floats<P> d2 = all_of<P>(0.0f), minus = mul(pair_at(x[0], e), all_of<P>(-1.0f));   // the batch's mean, negative
          if constexpr (C > 1) {
            Floats<P> m[C];
#pragma unroll
            for (int q = 0; q < C; ++q) m[q] = pair_at(x[q], e);
#pragma unroll
            for (int h = 1; h < C; h *= 2)
#pragma unroll
              for (int q = 0; q + h < C; q += 2 * h) m[q] = add(m[q], m[q + h]);
            minus = mul(m[0], all_of<P>(-1.0f / C));
#pragma unroll
            for (int q = 0; q < C; ++q) {
              const Floats<P> d = add(pair_at(x[q], e), minus);
              d2 = fma(d, d, d2);
            }
          }
          const Floats<P> old = pair_at(mean, e), dev = add(minus, old), up = fma(dev, all_of<P>(-w), old);
          const Floats<P> t = add(pair_at(m2, e), fma(mul(dev, all_of<P>(nw)), dev, d2));
#pragma unroll
          for (int o = 0; o < P; ++o) {
            mean[e + o] = up.x[o];
            m2[e + o] = t.x[o];
          }
        }
      });
    }
    __syncthreads();   // the last field's sums have been read
#pragma unroll
    for (int e = 0; e < V; ++e) red[ty][tx * V + e] = make_float2(mean[e], m2[e]);
    __syncthreads();
    for (int x = threadIdx.x; x < width; x += NT) {   // about the first thread's mean, which is no further off than a TY-th of the columns
      const float at = red[0][x].x, n = (float)(b - a), one = 1.0f / n;
      float s = 0.0f, s2 = red[0][x].y;
#pragma unroll
      for (int y = 1; y < TY; ++y) {
        const float cols = (float)((max(b - a - y, 0) + TY - 1) / TY), d = red[y][x].x - at;
        if (cols > 0.0f) {
          s = fmaf(d, cols * one, s);   // by shares of 1: a sum of deviations times columns may overflow where the mean does not
          s2 += fmaf(d * cols, d, red[y][x].y);
        }
      }
      feature[x] = make_float2(at + s, s2 <= FINITE ? clamp_low(fmaf(-s * n, s, s2), 0.0f) : s2);
    }
    __syncthreads();
    // features of a group have the same number of columns: their mean, and their deviations about it
    each_group(i0 / p.group, (i0 + width - 1) / p.group, [&](int g, int lane, int lanes) {
      const int x0 = max(0, g * p.group - i0), x1 = min(width, (g + 1) * p.group - i0);
      float s = 0.0f, d2 = 0.0f;
      const float at = x0 < x1 ? feature[x0].x : 0.0f;
      const float one = 1.0f / (float)(x1 - x0);
      for (int x = x0 + lane; x < x1; x += lanes) s = fmaf(feature[x].x - at, one, s);
      const float m = at + lanes_sum(s, lanes);
      for (int x = x0 + lane; x < x1; x += lanes) {
        const float d = feature[x].x - m;
        d2 += fmaf(d * (float)(b - a), d, feature[x].y);
      }
      d2 = lanes_sum(d2, lanes);
      if (lane == 0 && x0 < x1) part[share(p, t, f, fb, g)] = make_float2(m, d2);
    });
  }, [](int) {});
}

// The tiles and feature blocks that group g of the field in columns begin .. end - 1 is spread over, by `lanes` threads:
// get(share, columns, features).
template <int FW, class G>
__device__ __forceinline__ void each_share(const Fields& p, int f, int begin, int end, int t0, int t1, int g, int lane, int lanes, G&& get) {
  const int i0 = g * p.group, i1 = i0 + p.group, b0 = i0 / FW, nb = (i1 - 1) / FW - b0 + 1;
  for (int fb = b0; fb < b0 + nb; ++fb) {
    const int features = min(i1, (fb + 1) * FW) - max(i0, fb * FW);
#pragma unroll 4
    for (int t = t0 + lane; t <= t1; t += lanes)
      get(share(p, t, f, fb, g), min(end, (t + 1) * p.cols) - max(begin, t * p.cols), features);
  }
}

// Columns are t * cols + cols <= T + cols < 2^31.
template <class T, int TX, int V, int ACT>
__global__ void __launch_bounds__(NT, FORWARD) k_gnorm_apply(const T* X, int ldx, const Fields p, const float2* part, const float* gamma,
                                                    const float* beta, float eps, T* Y, int ldy, float* mean_out, float* rstd_out, int lds) {
  constexpr int TY = NT / TX, FW = TX * V;
  __shared__ float2 stat[FW];   // by group of the block
  const int fb = blockIdx.x % p.blocks, t = blockIdx.x / p.blocks;
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, i0 = fb * FW, i = i0 + tx * V;
  const int width = min(FW, p.D - i0), g0 = i0 / p.group, g1 = (i0 + width - 1) / p.group;
  let_next_start();
  wait_for_previous();
  float gm[V], bt[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    gm[e] = gamma && i < p.D ? gamma[i + e] : 1.0f;
    bt[e] = beta && i < p.D ? beta[i + e] : 0.0f;
  }
  each_field(p, t, [&](int f, int a, int b, int begin, int end) {
    __syncthreads();
    const int t0 = begin / p.cols, t1 = (end - 1) / p.cols;
    each_group(g0, g1, [&](int g, int lane, int lanes) {
      // the mean about one share's mean, then the deviations about it
      const bool there = g <= g1;
      const float n = (float)(end - begin) * (float)p.group, one = 1.0f / n;
      const float at = there ? part[share(p, t0, f, g * p.group / FW, g)].x : 0.0f;
      float s = 0.0f, d2 = 0.0f;
      if (there)
        each_share<FW>(p, f, begin, end, t0, t1, g, lane, lanes,
                       [&](size_t k, int cols, int features) { s = fmaf(part[k].x - at, (float)cols * (float)features * one, s); });
      const float mean = at + lanes_sum(s, lanes);
      if (there)
        each_share<FW>(p, f, begin, end, t0, t1, g, lane, lanes, [&](size_t k, int cols, int features) {
          const float2 w = part[k];
          const float d = w.x - mean;
          d2 += fmaf(d * ((float)cols * (float)features), d, w.y);
        });
      d2 = lanes_sum(d2, lanes);
      if (there && lane == 0) {
        const float r = 1.0f / sqrtf(d2 / n + eps);
        stat[g - g0] = make_float2(mean, r);
        if (mean_out && a == begin && g * p.group >= i0) {   // the tile with the group's first element
          mean_out[(size_t)f * lds + g] = mean;
          rstd_out[(size_t)f * lds + g] = r;
        }
      }
    });
    __syncthreads();
    if (i < p.D) {
      float m[V], s[V];
      each_feature<V>(p, i, [&](int e, int g) {
        const float2 st = stat[min(g, g1) - g0];
        m[e] = -st.x;
        s[e] = st.y * gm[e];
      });
      constexpr int B = BATCH, P = V > 1 ? 2 : 1;
      // from the last column to the first: the last ones that the first look read are the likeliest to be in L2 still
      const int last = a + ty < b ? b - 1 - (b - 1 - a - ty) % TY : 0;
      const T* from = X + (size_t)last * ldx + i;
      T* to = Y + (size_t)last * ldy + i;
      in_batches<B, TY, Raw<T, V>>(a + ty, b, [&](Raw<T, V>& raw, int j) { raw.load(from - (size_t)j * ldx); },
                                   [&](const auto& raw, int j, auto count) {
        constexpr int C = decltype(count)::value > 1 ? 2 : 1;   // columns at a time
        static_assert(decltype(count)::value % C == 0, "batches of whole pairs");
#pragma unroll
        for (int q = 0; q < decltype(count)::value; q += C) {
          float x[C][V];
#pragma unroll
          for (int c = 0; c < C; ++c) raw[q + c].widen(x[c]);
#pragma unroll
          for (int e = 0; e < V; e += P) {   // m is minus the mean
            Floats<P> z[C];
#pragma unroll
            for (int c = 0; c < C; ++c) z[c] = fma(add(pair_at(x[c], e), pair_at(m, e)), pair_at(s, e), pair_at(bt, e));
            curve<ACT, false, false>(z);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
              for (int o = 0; o < P; ++o) x[c][e + o] = z[c].x[o];
          }
#pragma unroll
          for (int c = 0; c < C; ++c) store<T, V>(to - (size_t)(j + (q + c) * TY) * ldy, x[c]);
        }
      });
    }
  }, [&](int f) {
    if (!mean_out) return;
    for (int g = g0 + (int)threadIdx.x; g <= g1; g += NT)
      if (g * p.group >= i0) mean_out[(size_t)f * lds + g] = rstd_out[(size_t)f * lds + g] = 0.0f;
  });
}

// A block per field and group, where one that had all T columns would be small (12 accesses a thread: 1024 x 256 BF16 in groups of 8
// 5.7 us, by tiles 8.4; 4096 x 256 13.5 and 11.6): one launch, and the second look at X finds it in L1 or L2.  Threads: TX = group / V along features, the others along columns.
template <class T, int V, int ACT>
__global__ void __launch_bounds__(NT) k_gnorm_small(const T* X, int ldx, const Fields p, const float* gamma, const float* beta, float eps, T* Y,
                                                    int ldy, float* mean_out, float* rstd_out, int lds) {
  __shared__ float red[2][NT / 32];
  let_next_start();
  wait_for_previous();
  const int g = blockIdx.x % p.groups, f = blockIdx.x / p.groups, i0 = g * p.group;
  const int begin = field_begin(p, f), end = field_begin(p, f + 1), TX = p.group / V;
  if (begin >= end) {
    if (mean_out && threadIdx.x == 0) mean_out[(size_t)f * lds + g] = rstd_out[(size_t)f * lds + g] = 0.0f;
    return;
  }
  const int total = (end - begin) * TX, step = NT / TX * TX;   // a thread keeps its features
  const int tx = threadIdx.x % TX, first = threadIdx.x < step ? (int)threadIdx.x : total;
  const auto at = [&](int e) { return (size_t)(begin + e / TX); };
  const auto block_sum = [&](float x, int k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) red[k][threadIdx.x >> 5] = x;
    __syncthreads();
    x = red[k][0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) x += red[k][w];
    return x;
  };
  const float shift = to_float(X[(size_t)begin * ldx + i0]), n = (float)(end - begin) * (float)p.group, one = 1.0f / n;
  float s = 0.0f, d2 = 0.0f;
#pragma unroll 4
  for (int e = first; e < total; e += step) {
    Raw<T, V> raw;
    raw.load(X + at(e) * ldx + i0 + tx * V);
    float x[V];
    raw.widen(x);
#pragma unroll
    for (int q = 0; q < V; ++q) s = fmaf(x[q] - shift, one, s);
  }
  const float mean = shift + block_sum(s, 0);
#pragma unroll 4
  for (int e = first; e < total; e += step) {
    Raw<T, V> raw;
    raw.load(X + at(e) * ldx + i0 + tx * V);
    float x[V];
    raw.widen(x);
#pragma unroll
    for (int q = 0; q < V; ++q) d2 = fmaf(x[q] - mean, x[q] - mean, d2);
  }
  const float r = 1.0f / sqrtf(block_sum(d2, 1) / n + eps);
  if (mean_out && threadIdx.x == 0) {
    mean_out[(size_t)f * lds + g] = mean;
    rstd_out[(size_t)f * lds + g] = r;
  }
  float sc[V], bt[V];
#pragma unroll
  for (int q = 0; q < V; ++q) {
    const int i = i0 + tx * V + q;
    sc[q] = gamma ? r * gamma[i] : r;
    bt[q] = beta ? beta[i] : 0.0f;
  }
  constexpr int B = 4;
  for (int e = first; e < total; e += B * step) {
    Raw<T, V> raw[B];
#pragma unroll
    for (int k = 0; k < B; ++k)
      if (e + k * step < total) raw[k].load(X + at(e + k * step) * ldx + i0 + tx * V);
#pragma unroll
    for (int k = 0; k < B; ++k)
      if (e + k * step < total) {
        float x[V];
        raw[k].widen(x);
#pragma unroll
        for (int q = 0; q < V; ++q) x[q] = fmaf(x[q] - mean, sc[q], bt[q]);
        constexpr int P = V > 1 ? 2 : 1;
#pragma unroll
        for (int q = 0; q < V; q += P) {
          Floats<P> z[1] = {pair_at(x, q)};
          curve<ACT, false, true>(z);
#pragma unroll
          for (int o = 0; o < P; ++o) x[q + o] = z[0].x[o];
        }
        store<T, V>(Y + at(e + k * step) * ldy + i0 + tx * V, x);
      }
  }
}

// ---------------------------------------------------------------- backward
// h = (x - mean) r and dz = dY act'(gamma h + beta) of a batch's columns, two at a time: use(column, feature, h, dz) for all features of a
// column, then done(column).  m is minus the mean.
template <int ACT, int V, class T, int N, class U, class D>
__device__ __forceinline__ void each_slope(const Pair<T, V> (&raw)[N], const float (&m)[V], const float (&r)[V], const float (&gm)[V],
                                           const float (&bt)[V], U&& use, D&& done) {
  constexpr int P = V > 1 ? 2 : 1, C = N > 1 ? 2 : 1;
  static_assert(N % C == 0, "batches of whole pairs");
#pragma unroll
  for (int q = 0; q < N; q += C) {
    float x[C][V], d[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      raw[q + c].x.widen(x[c]);
      raw[q + c].d.widen(d[c]);
    }
#pragma unroll
    for (int e = 0; e < V; e += P) {
      Floats<P> h[C], z[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        h[c] = mul(add(pair_at(x[c], e), pair_at(m, e)), pair_at(r, e));
        z[c] = fma(h[c], pair_at(gm, e), pair_at(bt, e));
      }
      if constexpr (ACT != CR_ACT_NONE) curve<ACT, true, false>(z);
#pragma unroll
      for (int c = 0; c < C; ++c) use(q + c, e, h[c], ACT != CR_ACT_NONE ? mul(pair_at(d[c], e), z[c]) : pair_at(d[c], e));
    }
#pragma unroll
    for (int c = 0; c < C; ++c) done(q + c);
  }
}

// With h = (x - mean) r, dz = dY act'(gamma h + beta): a feature's sums over the tile of dz h and dz go to
// psum[t][2 D], and the groups' shares of sum gamma dz and sum gamma dz h to part.
template <class T, int TX, int V, int ACT>
__global__ void __launch_bounds__(NT, BACKWARD) k_gnorm_sums(const T* X, int ldx, const T* dY, int lddy, const Fields p, const float* gamma,
                                                   const float* beta, const float* mean, const float* rstd, int lds, float2* part, float* pgamma,
                                                   float* pbeta) {
  constexpr int TY = NT / TX, FW = TX * V;
  __shared__ float2 red[TY][FW];
  __shared__ float2 feature[FW], all[FW];
  const int fb = blockIdx.x % p.blocks, t = blockIdx.x / p.blocks;
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, i0 = fb * FW, i = i0 + tx * V;
  const int width = min(FW, p.D - i0);
  let_next_start();
  for (int x = threadIdx.x; x < FW; x += NT) all[x] = make_float2(0.0f, 0.0f);
  wait_for_previous();
  float gm[V], bt[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    gm[e] = gamma && i < p.D ? gamma[i + e] : 1.0f;
    bt[e] = beta && i < p.D ? beta[i + e] : 0.0f;
  }
  each_field(p, t, [&](int f, int a, int b, int begin, int end) {
    float sb[V] = {}, sg[V] = {};
    if (i < p.D) {
      float m[V], r[V];
      each_feature<V>(p, i, [&](int e, int g) {
        const size_t at = (size_t)f * lds + min(g, p.groups - 1);
        m[e] = -mean[at];
        r[e] = rstd[at];
      });
      constexpr int B = BACKWARD_BATCH<T>, P = V > 1 ? 2 : 1;
      const T *xs = X + (size_t)(a + ty) * ldx + i, *ds = dY + (size_t)(a + ty) * lddy + i;
      in_batches<B, TY, Pair<T, V>>(a + ty, b, [&](Pair<T, V>& raw, int j) {
        raw.x.load(xs + (size_t)j * ldx);
        raw.d.load(ds + (size_t)j * lddy);
      }, [&](const auto& raw, int, auto) {
        each_slope<ACT, V>(raw, m, r, gm, bt, [&](int, int e, Floats<P> h, Floats<P> dz) {
          const Floats<P> b1 = add(pair_at(sb, e), dz), g1 = fma(dz, h, pair_at(sg, e));
#pragma unroll
          for (int o = 0; o < P; ++o) {
            sb[e + o] = b1.x[o];
            sg[e + o] = g1.x[o];
          }
        }, [](int) {});
      });
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) red[ty][tx * V + e] = make_float2(sb[e], sg[e]);
    __syncthreads();
    for (int x = threadIdx.x; x < width; x += NT) {
      float2 s = red[0][x];
      for (int y = 1; y < TY; ++y) {
        s.x += red[y][x].x;
        s.y += red[y][x].y;
      }
      feature[x] = s;
      all[x].x += s.x;
      all[x].y += s.y;
    }
    __syncthreads();
    if (part) {
      each_group(i0 / p.group, (i0 + width - 1) / p.group, [&](int g, int lane, int lanes) {
        const int x0 = max(0, g * p.group - i0), x1 = min(width, (g + 1) * p.group - i0);
        float2 s = make_float2(0.0f, 0.0f);
        for (int x = x0 + lane; x < x1; x += lanes) {
          const float w = gamma ? gamma[i0 + x] : 1.0f;
          s.x = fmaf(w, feature[x].x, s.x);
          s.y = fmaf(w, feature[x].y, s.y);
        }
        s.x = lanes_sum(s.x, lanes);
        s.y = lanes_sum(s.y, lanes);
        if (lane == 0 && x0 < x1) part[share(p, t, f, fb, g)] = s;
      });
    }
  }, [](int) {});
  __syncthreads();
  for (int x = threadIdx.x; x < width; x += NT) {
    if (pgamma) pgamma[(size_t)t * p.D + i0 + x] = all[x].y;
    if (pbeta) pbeta[(size_t)t * p.D + i0 + x] = all[x].x;
  }
}

// total[D] = the sum of the rows of part (rows x D) for 32 features from i0 on, in a fixed order, by a block.
__device__ __forceinline__ void sum_rows(const float* part, int rows, int D, int i0, float* total, float (&red)[NT / 32][33]) {
  const int i = i0 + threadIdx.x % 32, w = threadIdx.x / 32;
  float s = 0.0f;
  if (i < D) {
#pragma unroll 8
    for (int r = w; r < rows; r += NT / 32) s += part[(size_t)r * D + i];
  }
  red[w][threadIdx.x % 32] = s;
  __syncthreads();
  if (w == 0 && i < D) {
    for (int y = 1; y < NT / 32; ++y) s += red[y][threadIdx.x];
    total[i] = s;
  }
}

// dX = r (gamma dz - mean(gamma dz) - h mean(gamma dz h)), means over the group, by the first `tiles` blocks (0: not wanted); the
// others sum up the parts of dgamma and dbeta (rows of them), 32 features each.
template <class T, int TX, int V, int ACT>
__global__ void __launch_bounds__(NT, BACKWARD) k_gnorm_dx(const T* X, int ldx, const T* dY, int lddy, const Fields p, const float2* part,
                                                 const float* gamma, const float* beta, const float* mean, const float* rstd, int lds, T* dX,
                                                 int lddx, unsigned tiles, int rows, const float* pgamma, const float* pbeta, float* dgamma,
                                                 float* dbeta) {
  constexpr int TY = NT / TX, FW = TX * V;
  __shared__ float2 stat[FW];
  __shared__ float red[NT / 32][33];
  if (blockIdx.x >= tiles) {
    let_next_start();
    wait_for_previous();
    const unsigned b = blockIdx.x - tiles, per = (p.D + 31) / 32;
    const bool second = !dgamma || b >= per;
    sum_rows(second ? pbeta : pgamma, rows, p.D, (int)(b % per) * 32, second ? dbeta : dgamma, red);
    return;
  }
  const int fb = blockIdx.x % p.blocks, t = blockIdx.x / p.blocks;
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, i0 = fb * FW, i = i0 + tx * V;
  const int width = min(FW, p.D - i0), g0 = i0 / p.group, g1 = (i0 + width - 1) / p.group;
  let_next_start();
  wait_for_previous();
  float gm[V], bt[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    gm[e] = gamma && i < p.D ? gamma[i + e] : 1.0f;
    bt[e] = beta && i < p.D ? beta[i + e] : 0.0f;
  }
  each_field(p, t, [&](int f, int a, int b, int begin, int end) {
    __syncthreads();
    const int t0 = begin / p.cols, t1 = (end - 1) / p.cols;
    each_group(g0, g1, [&](int g, int lane, int lanes) {
      float2 s = make_float2(0.0f, 0.0f);
      if (g <= g1)
        each_share<FW>(p, f, begin, end, t0, t1, g, lane, lanes, [&](size_t k, int, int) {
          const float2 w = part[k];
          s.x += w.x;
          s.y += w.y;
        });
      s.x = lanes_sum(s.x, lanes);
      s.y = lanes_sum(s.y, lanes);
      const float n = (float)(end - begin) * (float)p.group;
      if (lane == 0 && g <= g1) stat[g - g0] = make_float2(s.x / n, s.y / n);
    });
    __syncthreads();
    if (i < p.D) {
      float m[V], r[V], c1[V], c2[V];
      each_feature<V>(p, i, [&](int e, int g) {
        const int k = min(g, g1);
        const size_t at = (size_t)f * lds + k;
        m[e] = -mean[at];
        r[e] = rstd[at];
        c1[e] = -r[e] * stat[k - g0].x;
        c2[e] = -r[e] * stat[k - g0].y;
      });
      constexpr int B = BACKWARD_BATCH<T>, P = V > 1 ? 2 : 1;
      const int last = a + ty < b ? b - 1 - (b - 1 - a - ty) % TY : 0;   // from the last column to the first, as k_gnorm_apply
      const T *xs = X + (size_t)last * ldx + i, *ds = dY + (size_t)last * lddy + i;
      T* to = dX + (size_t)last * lddx + i;
      in_batches<B, TY, Pair<T, V>>(a + ty, b, [&](Pair<T, V>& raw, int j) {
        raw.x.load(xs - (size_t)j * ldx);
        raw.d.load(ds - (size_t)j * lddy);
      }, [&](const auto& raw, int j, auto) {
        float y[2][V];
        each_slope<ACT, V>(raw, m, r, gm, bt, [&](int q, int e, Floats<P> h, Floats<P> dz) {   // c1 and c2 are the sums times -r
          const Floats<P> v = fma(h, pair_at(c2, e), fma(mul(dz, pair_at(gm, e)), pair_at(r, e), pair_at(c1, e)));
#pragma unroll
          for (int o = 0; o < P; ++o) y[q % 2][e + o] = v.x[o];
        }, [&](int q) { store<T, V>(to - (size_t)(j + q * TY) * lddx, y[q % 2]); });
      });
    }
  }, [](int) {});
}

// Small fields as in k_gnorm_small: a block per field and group forms both its sums and its dX, and leaves its features' sums for
// dgamma and dbeta in pgamma[field][D] and pbeta[field][D].
template <class T, int V, int ACT>
__global__ void __launch_bounds__(NT) k_gnorm_small_bwd(const T* X, int ldx, const T* dY, int lddy, const Fields p, const float* gamma,
                                                        const float* beta, const float* mean, const float* rstd, int lds, T* dX, int lddx,
                                                        float* pgamma, float* pbeta) {
  __shared__ float red[2][NT / 32];
  __shared__ float2 feature[NT * V];
  constexpr int P = V > 1 ? 2 : 1;
  let_next_start();
  wait_for_previous();
  const int g = blockIdx.x % p.groups, f = blockIdx.x / p.groups, i0 = g * p.group;
  const int begin = field_begin(p, f), end = max(begin, field_begin(p, f + 1)), TX = p.group / V, TY = NT / TX;
  const int total = (end - begin) * TX, step = TY * TX;   // a thread keeps its features
  const int tx = threadIdx.x % TX, first = threadIdx.x < step ? (int)threadIdx.x : total;
  const float minus = begin < end ? -mean[(size_t)f * lds + g] : 0.0f, r = begin < end ? rstd[(size_t)f * lds + g] : 0.0f;
  const float n = (float)(end - begin) * (float)p.group;
  float gm[V], bt[V], sb[V] = {}, sg[V] = {};
#pragma unroll
  for (int q = 0; q < V; ++q) {
    gm[q] = gamma ? gamma[i0 + tx * V + q] : 1.0f;
    bt[q] = beta ? beta[i0 + tx * V + q] : 0.0f;
  }
  const auto look = [&](int e, auto&& use) {   // use(q, h, dz), P features at a time
    Pair<T, V> raw;
    const size_t j = (size_t)(begin + e / TX);
    raw.x.load(X + j * ldx + i0 + tx * V);
    raw.d.load(dY + j * lddy + i0 + tx * V);
    float x[V], d[V];
    raw.x.widen(x);
    raw.d.widen(d);
#pragma unroll
    for (int q = 0; q < V; q += P) {
      const Floats<P> h = mul(add(pair_at(x, q), all_of<P>(minus)), all_of<P>(r));
      Floats<P> dz = pair_at(d, q);
      if (ACT != CR_ACT_NONE) {
        Floats<P> z[1] = {fma(h, pair_at(gm, q), pair_at(bt, q))};
        curve<ACT, true, true>(z);
        dz = mul(dz, z[0]);
      }
      use(q, h, dz);
    }
  };
#pragma unroll 2
  for (int e = first; e < total; e += step)
    look(e, [&](int q, Floats<P> h, Floats<P> dz) {
      const Floats<P> b = add(pair_at(sb, q), dz), c = fma(dz, h, pair_at(sg, q));
#pragma unroll
      for (int o = 0; o < P; ++o) {
        sb[q + o] = b.x[o];
        sg[q + o] = c.x[o];
      }
    });
  float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
  for (int q = 0; q < V; ++q) {
    feature[threadIdx.x * V + q] = make_float2(sb[q], sg[q]);   // [ty][feature] of the step's threads
    c1 = fmaf(gm[q], sb[q], c1);
    c2 = fmaf(gm[q], sg[q], c2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    c1 += __shfl_xor_sync(0xffffffffu, c1, o);
    c2 += __shfl_xor_sync(0xffffffffu, c2, o);
  }
  if ((threadIdx.x & 31) == 0) {
    red[0][threadIdx.x >> 5] = c1;
    red[1][threadIdx.x >> 5] = c2;
  }
  __syncthreads();
  c1 = red[0][0];
  c2 = red[1][0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) {
    c1 += red[0][w];
    c2 += red[1][w];
  }
  for (int x = threadIdx.x; x < p.group; x += NT) {
    float2 t = feature[x];
    for (int y = 1; y < TY; ++y) {
      t.x += feature[y * p.group + x].x;
      t.y += feature[y * p.group + x].y;
    }
    if (pgamma) pgamma[(size_t)f * p.D + i0 + x] = t.y;
    if (pbeta) pbeta[(size_t)f * p.D + i0 + x] = t.x;
  }
  if (!dX || begin == end) return;
  const Floats<P> m1 = all_of<P>(-r * (c1 / n)), m2 = all_of<P>(-r * (c2 / n));
#pragma unroll 2
  for (int e = first; e < total; e += step) {
    float y[V];
    look(e, [&](int q, Floats<P> h, Floats<P> dz) {
      const Floats<P> v = fma(h, m2, fma(mul(dz, pair_at(gm, q)), all_of<P>(r), m1));
#pragma unroll
      for (int o = 0; o < P; ++o) y[q + o] = v.x[o];
    });
    store<T, V>(dX + (size_t)(begin + e / TX) * lddx + i0 + tx * V, y);
  }
}

// Columns of 16-bit types on 8- or 16-byte boundaries (bytes), of FP32 on 16-byte ones.
bool aligned(const void* p, int ld, int eb, int bytes) { return ((uintptr_t)p & (bytes - 1)) == 0 && (long long)ld * eb % bytes == 0; }

// Calls f(TX, V) for a matrix of D features, V of them to a thread (1 where 16-byte or, for V = 4 of 16-bit types, 8-byte accesses do
// not apply): the widest of 32, 16 and 8 threads along them that leaves little unused (64 and 128 threads,
// which read whole rows, are no faster: 142 to 148 us for eight fields of 16384 x 1024).
template <int V, class F>
cr_status with_tile(int D, bool vec, F&& f) {
  using std::integral_constant;
  if (!vec) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  const auto padded = [&](int w) { return (D + w * V - 1) / (w * V) * (w * V); };
  const int best = padded(8);
  if (4ll * padded(32) <= 5ll * best) return f(integral_constant<int, 32>{}, integral_constant<int, V>{});
  if (padded(16) == best) return f(integral_constant<int, 16>{}, integral_constant<int, V>{});
  return f(integral_constant<int, 8>{}, integral_constant<int, V>{});
}

// Tiles that are resident at once, of a multiple of `unit` columns to a thread: a tile's set-up and its groups' sums cost about as much as
// 64 KB of columns.
Fields make_fields(const int32_t* off, int n, int T, int D, int groups, int width, int rows, int resident, int unit) {
  Fields p = {};
  p.off = off;
  p.n = off ? n : 1;
  p.T = T;
  p.D = D;
  p.groups = groups;
  p.group = D / groups;
  p.blocks = (D + width - 1) / width;
  const long long want = std::max(1, resident * sm_count() / p.blocks), per = (T + want - 1) / want, whole = unit * rows;
  p.cols = (int)((per + whole - 1) / whole * whole);
  p.tiles = (T + p.cols - 1) / p.cols;
  return p;
}

cr_status check(const char* what, int type, int D, int T, int groups, const int32_t* off, int n) {
  if (type != CR_TYPE_F32 && type != CR_TYPE_F16 && type != CR_TYPE_BF16) return fail(CR_ERR_ARG, std::string(what) + ": type must be FP32, FP16 or BF16");
  if (D < 1 || T < 0 || (off && n < 0)) return fail(CR_ERR_ARG, std::string(what) + ": D >= 1, T >= 0, n_field >= 0");
  if (std::max({D, T, off ? n : 0}) > MAXSIZE) return fail(CR_ERR_ARG, std::string(what) + ": sizes end at 2^31 - 2^16");
  if (groups < 1 || groups > D || D % groups) return fail(CR_ERR_ARG, std::string(what) + ": groups must divide D");
  return CR_OK;
}

}  // namespace
}  // namespace cr

using namespace cr;

extern "C" cr_status cr_group_norm(int type, const void* d_X, int ldx, int D, int T, int groups, const int32_t* d_off, int n_field,
                                   const float* d_gamma, const float* d_beta, double eps, int act, void* d_Y, int ldy, float* d_mean,
                                   float* d_rstd, int lds, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_TRY(check("cr_group_norm", type, D, T, groups, d_off, n_field));
  CR_REQUIRE(act >= CR_ACT_NONE && act <= CR_ACT_GELU, "cr_group_norm: unknown activation");
  CR_REQUIRE(eps >= 0.0 && eps < 1e30, "cr_group_norm: eps must be finite and not negative");
  CR_REQUIRE(ldx >= D && ldy >= D, "cr_group_norm: leading dimension below D");
  CR_REQUIRE((d_mean == nullptr) == (d_rstd == nullptr), "cr_group_norm: d_mean and d_rstd belong together");
  CR_REQUIRE(!d_mean || lds >= groups, "cr_group_norm: leading dimension below groups");
  const int n = d_off ? n_field : 1;
  if (T == 0 || n == 0) {
    if (d_mean && n > 0) {
      CR_CUDA(cudaMemset2DAsync(d_mean, (size_t)lds * 4, 0, (size_t)groups * 4, n, stream));
      CR_CUDA(cudaMemset2DAsync(d_rstd, (size_t)lds * 4, 0, (size_t)groups * 4, n, stream));
    }
    return CR_OK;
  }
  CR_REQUIRE(d_X && d_Y, "cr_group_norm: NULL argument");
  int* err = nullptr;   // these kernels wait for nobody, but report what an earlier call's did
  CR_TRY(wait_word(&err));
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    constexpr int EB = sizeof(E), W = 16 / EB;
    const bool vec = D % W == 0 && aligned(d_X, ldx, EB, 16) && aligned(d_Y, ldy, EB, 16);
    const int group = D / groups;
    if ((long long)T * (vec && group % W == 0 ? group / W : group) <= SMALL * NT && (long long)n * groups <= 128 * sm_count() && group <= NT) {
      Fields p = {};
      p.off = d_off;
      p.n = n;
      p.T = T;
      p.D = D;
      p.groups = groups;
      p.group = D / groups;
      return with_act(act, [&](auto a0) -> cr_status {
        constexpr int ACT = decltype(a0)::value;
        TimedScope ts("k_gnorm_small", stream);
        const auto go = [&](auto v0) {
          return launch_after(k_gnorm_small<E, decltype(v0)::value, ACT>, (unsigned)(n * groups), NT, 0, 1, stream, (const E*)d_X, ldx, p, d_gamma,
                              d_beta, (float)eps, (E*)d_Y, ldy, d_mean, d_rstd, lds);
        };
        CR_CUDA(vec && p.group % W == 0 ? go(std::integral_constant<int, W>{}) : go(std::integral_constant<int, 1>{}));
        CR_CHECK_LAUNCH("k_gnorm_small");
        return CR_OK;
      });
    }
    return with_tile<W>(D, vec, [&](auto tx0, auto v0) -> cr_status {
      constexpr int TX = decltype(tx0)::value, V = decltype(v0)::value;
      const Fields p = make_fields(d_off, n_field, T, D, groups, TX * V, NT / TX, FORWARD, BATCH);
      const unsigned grid = (unsigned)((long long)p.tiles * p.blocks);
      float2* part = nullptr;
      CR_CUDA(scratch_alloc((void**)&part, shares(p) * sizeof(float2), stream));
      const auto run = [&]() -> cr_status {
        {
          TimedScope ts("k_gnorm_stats", stream);
          CR_CUDA(launch_after(k_gnorm_stats<E, TX, V>, grid, NT, 0, 1, stream, (const E*)d_X, ldx, p, part));
          CR_CHECK_LAUNCH("k_gnorm_stats");
        }
        return with_act(act, [&](auto a0) -> cr_status {
          TimedScope ts("k_gnorm_apply", stream);
          CR_CUDA(launch_after(k_gnorm_apply<E, TX, V, decltype(a0)::value>, grid, NT, 0, 1, stream, (const E*)d_X, ldx, p, part, d_gamma, d_beta,
                               (float)eps, (E*)d_Y, ldy, d_mean, d_rstd, lds));
          CR_CHECK_LAUNCH("k_gnorm_apply");
          return CR_OK;
        });
      };
      const cr_status st = run();
      scratch_free(part, stream);
      return st;
    });
  });
  CR_ENTRY_END("cr_group_norm")
}

extern "C" cr_status cr_group_norm_backward(int type, const void* d_X, int ldx, int D, int T, int groups, const int32_t* d_off,
                                            int n_field, const float* d_gamma, const float* d_beta, const void* d_dY, int lddy,
                                            const float* d_mean, const float* d_rstd, int lds, int act, void* d_dX, int lddx,
                                            float* d_dgamma, float* d_dbeta, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_TRY(check("cr_group_norm_backward", type, D, T, groups, d_off, n_field));
  CR_REQUIRE(act >= CR_ACT_NONE && act <= CR_ACT_GELU, "cr_group_norm_backward: unknown activation");
  CR_REQUIRE(ldx >= D && lddy >= D && (!d_dX || lddx >= D) && lds >= groups, "cr_group_norm_backward: leading dimension too small");
  const int n = d_off ? n_field : 1;
  if (T == 0 || n == 0) {
    if (d_dgamma) CR_CUDA(cudaMemsetAsync(d_dgamma, 0, (size_t)D * sizeof(float), stream));
    if (d_dbeta) CR_CUDA(cudaMemsetAsync(d_dbeta, 0, (size_t)D * sizeof(float), stream));
    return CR_OK;
  }
  CR_REQUIRE(d_X && d_dY && d_mean && d_rstd, "cr_group_norm_backward: NULL argument");
  if (!d_dX && !d_dgamma && !d_dbeta) return CR_OK;
  int* err = nullptr;
  CR_TRY(wait_word(&err));
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    const int group = D / groups;
    constexpr int WS = 16 / (int)sizeof(E);
    const bool wide = group % WS == 0 && D % WS == 0 && aligned(d_X, ldx, sizeof(E), 16) && aligned(d_dY, lddy, sizeof(E), 16) &&
                      (!d_dX || aligned(d_dX, lddx, sizeof(E), 16));
    if ((long long)T * (wide ? group / WS : group) <= SMALL * NT && (long long)n * groups <= 128 * sm_count() && group <= NT) {
      Fields p = {};
      p.off = d_off;
      p.n = n;
      p.T = T;
      p.D = D;
      p.groups = groups;
      p.group = group;
      float* part = nullptr;
      const size_t rows = (size_t)n * D;
      if (d_dgamma || d_dbeta) CR_CUDA(scratch_alloc((void**)&part, 2 * rows * sizeof(float), stream));
      const auto run = [&]() -> cr_status {
        CR_TRY(with_act(act, [&](auto a0) -> cr_status {
          constexpr int ACT = decltype(a0)::value;
          TimedScope ts("k_gnorm_small", stream);
          const auto go = [&](auto v0) {
            return launch_after(k_gnorm_small_bwd<E, decltype(v0)::value, ACT>, (unsigned)(n * groups), NT, 0, 1, stream, (const E*)d_X, ldx,
                                (const E*)d_dY, lddy, p, d_gamma, d_beta, d_mean, d_rstd, lds, (E*)d_dX, lddx, d_dgamma ? part : nullptr,
                                d_dbeta ? part + rows : nullptr);
          };
          CR_CUDA(wide ? go(std::integral_constant<int, WS>{}) : go(std::integral_constant<int, 1>{}));
          CR_CHECK_LAUNCH("k_gnorm_small_bwd");
          return CR_OK;
        }));
        if (!part) return CR_OK;
        const unsigned sums = (unsigned)((D + 31) / 32) * ((d_dgamma ? 1 : 0) + (d_dbeta ? 1 : 0));
        CR_CUDA(launch_after(k_gnorm_dx<E, 32, 1, CR_ACT_NONE>, sums, NT, 0, 1, stream, (const E*)d_X, ldx, (const E*)d_dY, lddy, p,
                             (const float2*)nullptr, d_gamma, d_beta, d_mean, d_rstd, lds, (E*)nullptr, D, 0u, n, part, part + rows, d_dgamma, d_dbeta));
        CR_CHECK_LAUNCH("k_gnorm_dx");
        return CR_OK;
      };
      const cr_status st = run();
      scratch_free(part, stream);
      return st;
    }
    // four features to a thread: with eight, their six constants each do not fit into registers beside the columns on their way
    constexpr int EB = sizeof(E), W = 4;
    const bool vec = D % W == 0 && aligned(d_X, ldx, EB, W * EB) && aligned(d_dY, lddy, EB, W * EB) && (!d_dX || aligned(d_dX, lddx, EB, W * EB));
    return with_tile<W>(D, vec, [&](auto tx0, auto v0) -> cr_status {
      constexpr int TX = decltype(tx0)::value, V = decltype(v0)::value;
      const Fields p = make_fields(d_off, n_field, T, D, groups, TX * V, NT / TX, BACKWARD, 2);
      const unsigned grid = (unsigned)((long long)p.tiles * p.blocks);
      const size_t rows = (size_t)p.tiles * D;
      float2* part = nullptr;
      CR_CUDA(scratch_alloc((void**)&part, shares(p) * sizeof(float2) + 2 * rows * sizeof(float), stream));
      float *pgamma = (float*)(part + shares(p)), *pbeta = pgamma + rows;
      const auto run = [&]() -> cr_status {
        CR_TRY(with_act(act, [&](auto a0) -> cr_status {
          constexpr int ACT = decltype(a0)::value;
          {
            TimedScope ts("k_gnorm_sums", stream);
            CR_CUDA(launch_after(k_gnorm_sums<E, TX, V, ACT>, grid, NT, 0, 1, stream, (const E*)d_X, ldx, (const E*)d_dY, lddy, p, d_gamma, d_beta,
                                 d_mean, d_rstd, lds, d_dX ? part : nullptr, d_dgamma ? pgamma : nullptr, d_dbeta ? pbeta : nullptr));
            CR_CHECK_LAUNCH("k_gnorm_sums");
          }
          TimedScope ts("k_gnorm_dx", stream);
          const unsigned sums = (unsigned)((D + 31) / 32) * ((d_dgamma ? 1 : 0) + (d_dbeta ? 1 : 0)), tiles = d_dX ? grid : 0;
          CR_CUDA(launch_after(k_gnorm_dx<E, TX, V, ACT>, tiles + sums, NT, 0, 1, stream, (const E*)d_X, ldx, (const E*)d_dY, lddy, p, part, d_gamma,
                               d_beta, d_mean, d_rstd, lds, (E*)d_dX, lddx, tiles, p.tiles, pgamma, pbeta, d_dgamma, d_dbeta));
          CR_CHECK_LAUNCH("k_gnorm_dx");
          return CR_OK;
        }));
        return CR_OK;
      };
      const cr_status st = run();
      scratch_free(part, stream);
      return st;
    });
  });
  CR_ENTRY_END("cr_group_norm_backward")
}
