// Group norm over packed fields with an activation, and its gradient (cr_group_norm, cr_group_norm_backward).
//
// A group of a field is the field's columns times the group's consecutive features.  Two kernels: the first leaves each
// tile's share of every group's mean and sum of squared deviations (each formed about the share's own mean, so that a
// large common value costs no digits), the second joins the shares of the groups that its tile needs, in a fixed order,
// and goes over the tile again.  The gradient does the same with its two sums.
#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "ptx.cuh"

namespace cr {
namespace {

constexpr int NT = 256;

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
  return (size_t)(t + f) * (p.blocks + p.groups) + fb + g;
}
size_t shares(const Fields& p) { return (size_t)(p.tiles + p.n) * (p.blocks + p.groups); }

template <class T, int V>
__device__ __forceinline__ void load(const T* p, float (&v)[V]) {
  if constexpr (V == 8) widen8(*reinterpret_cast<const Eight<T>*>(p), v);
  else v[0] = to_float(p[0]);
}
template <class T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
  if constexpr (V == 8) *reinterpret_cast<Eight<T>*>(p) = narrow8<T>(v);
  else p[0] = from_float<T>(v[0]);
}

// n values of mean and sum of squared deviations m2; joined with those of m others (Chan, Golub and LeVeque's update).
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments join(Moments a, Moments b) {
  const float n = a.n + b.n;
  if (b.n == 0.0f) return a;
  const float d = b.mean - a.mean, w = b.n / n;
  return {n, fmaf(d, w, a.mean), a.m2 + fmaf(d * a.n * w, d, b.m2)};
}

// Calls run(f, a, b) for the fields' columns a .. b - 1 inside the tile, and none(f) for empty fields, each by one tile.
template <class R, class E>
__device__ __forceinline__ void each_field(const Fields& p, int t, R&& run, E&& none) {
  const int c0 = t * p.cols, c1 = min(p.T, c0 + p.cols);
  const bool last = t + 1 == p.tiles;
  for (int f = first_field(p, c0); f < p.n; ++f) {
    const int begin = field_begin(p, f), end = field_begin(p, f + 1);
    if (begin >= c1 && !last) break;
    const int a = max(begin, c0), b = min(end, c1);
    if (a < b) run(f, a, b);
    else if (begin >= end && begin >= c0) none(f);
  }
}

// ---------------------------------------------------------------- forward
template <class T, int TX, int V>
__global__ void __launch_bounds__(NT) k_gnorm_stats(const T* X, int ldx, const Fields p, float2* part) {
  constexpr int TY = NT / TX, FW = TX * V;
  __shared__ float2 red[TY][FW];   // of a thread's features
  __shared__ float2 feature[FW];
  const int fb = blockIdx.x % p.blocks, t = blockIdx.x / p.blocks;
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, i0 = fb * FW, i = i0 + tx * V;
  const int width = min(FW, p.D - i0);
  let_next_start();
  wait_for_previous();
  each_field(p, t, [&](int f, int a, int b) {
    float mean[V] = {}, m2[V] = {}, n = 0.0f;
    if (i < p.D) {
      int j = a + ty;
      for (; j + 3 * TY < b; j += 4 * TY) {   // four columns: their own mean and deviations, joined to what is there
        float x[4][V];
#pragma unroll
        for (int q = 0; q < 4; ++q) load<T, V>(X + (size_t)(j + q * TY) * ldx + i, x[q]);
        const float w = 4.0f / (n + 4.0f), nw = n * w;
        n += 4.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float m = ((x[0][e] + x[1][e]) + (x[2][e] + x[3][e])) * 0.25f;
          float s = 0.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q) s = fmaf(x[q][e] - m, x[q][e] - m, s);
          const float d = m - mean[e];
          mean[e] = fmaf(d, w, mean[e]);
          m2[e] += fmaf(d * nw, d, s);
        }
      }
      for (; j < b; j += TY) {
        float x[V];
        load<T, V>(X + (size_t)j * ldx + i, x);
        const float w = 1.0f / (n + 1.0f), nw = n * w;
        n += 1.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = x[e] - mean[e];
          mean[e] = fmaf(d, w, mean[e]);
          m2[e] = fmaf(d * nw, d, m2[e]);
        }
      }
    }
    __syncthreads();   // the last field's sums have been read
#pragma unroll
    for (int e = 0; e < V; ++e) red[ty][tx * V + e] = make_float2(mean[e], m2[e]);
    __syncthreads();
    for (int x = threadIdx.x; x < width; x += NT) {
      Moments m = {0.0f, 0.0f, 0.0f};
      for (int y = 0; y < TY; ++y) {
        const int cols = b - a > y ? (b - a - y + TY - 1) / TY : 0;
        m = join(m, Moments{(float)cols, red[y][x].x, red[y][x].y});
      }
      feature[x] = make_float2(m.mean, m.m2);
    }
    __syncthreads();
    // features of a group have the same number of columns: their mean, and their deviations about it
    const int lane = threadIdx.x & 31, g0 = i0 / p.group, g1 = (i0 + width - 1) / p.group;
    for (int g = g0 + ((int)threadIdx.x >> 5); g <= g1; g += NT / 32) {
      const int x0 = max(0, g * p.group - i0), x1 = min(width, (g + 1) * p.group - i0);
      float s = 0.0f, d2 = 0.0f;
      const float at = feature[x0].x;
      for (int x = x0 + lane; x < x1; x += 32) s += feature[x].x - at;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float m = at + s / (float)(x1 - x0);
      for (int x = x0 + lane; x < x1; x += 32) {
        const float d = feature[x].x - m;
        d2 += fmaf(d * (float)(b - a), d, feature[x].y);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d2 += __shfl_xor_sync(0xffffffffu, d2, o);
      if (lane == 0) part[share(p, t, f, fb, g)] = make_float2(m, d2);
    }
  }, [](int) {});
}

// The feature blocks and tiles that field f's group g is spread over, visited by a warp: get(share, columns, features).
template <int FW, class G>
__device__ __forceinline__ void each_share(const Fields& p, int f, int g, G&& get) {
  const int begin = field_begin(p, f), end = field_begin(p, f + 1);
  const int t0 = begin / p.cols, nt = (end - 1) / p.cols - t0 + 1;
  const int i0 = g * p.group, i1 = i0 + p.group, b0 = i0 / FW, nb = (i1 - 1) / FW - b0 + 1;
  const long long total = (long long)nt * nb;
  for (long long e = threadIdx.x & 31; e < total; e += 32) {
    const int t = t0 + (int)(e / nb), fb = b0 + (int)(e % nb);
    const int cols = min(end, (t + 1) * p.cols) - max(begin, t * p.cols), features = min(i1, (fb + 1) * FW) - max(i0, fb * FW);
    get(share(p, t, f, fb, g), cols, features);
  }
}

// Columns are t * cols + cols <= T + cols < 2^31.
template <class T, int TX, int V, int ACT>
__global__ void __launch_bounds__(NT) k_gnorm_apply(const T* X, int ldx, const Fields p, const float2* part, const float* gamma,
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
  each_field(p, t, [&](int f, int a, int b) {
    __syncthreads();
    for (int g = g0 + ((int)threadIdx.x >> 5); g <= g1; g += NT / 32) {
      Moments m = {0.0f, 0.0f, 0.0f};
      each_share<FW>(p, f, g, [&](size_t s, int cols, int features) { m = join(m, Moments{(float)cols * (float)features, part[s].x, part[s].y}); });
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Moments other = {__shfl_down_sync(0xffffffffu, m.n, o), __shfl_down_sync(0xffffffffu, m.mean, o), __shfl_down_sync(0xffffffffu, m.m2, o)};
        if (m.n == 0.0f) m = other;
        else m = join(m, other);
      }
      if ((threadIdx.x & 31) == 0) {
        const float r = 1.0f / sqrtf(m.m2 / m.n + eps);
        stat[g - g0] = make_float2(m.mean, r);
        if (mean_out && a == field_begin(p, f) && g * p.group >= i0) {   // the tile with the group's first element
          mean_out[(size_t)f * lds + g] = m.mean;
          rstd_out[(size_t)f * lds + g] = r;
        }
      }
    }
    __syncthreads();
    if (i < p.D) {
      float m[V], s[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 st = stat[(i + e) / p.group - g0];
        m[e] = st.x;
        s[e] = st.y * gm[e];
      }
#pragma unroll 4
      for (int j = a + ty; j < b; j += TY) {
        float x[V];
        load<T, V>(X + (size_t)j * ldx + i, x);
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = fmaf(x[e] - m[e], s[e], bt[e]);
        activate_each<ACT, V>(x);
        store<T, V>(Y + (size_t)j * ldy + i, x);
      }
    }
  }, [&](int f) {
    if (!mean_out) return;
    for (int g = g0 + (int)threadIdx.x; g <= g1; g += NT)
      if (g * p.group >= i0) mean_out[(size_t)f * lds + g] = rstd_out[(size_t)f * lds + g] = 0.0f;
  });
}

// ---------------------------------------------------------------- backward
// With h = (x - mean) r, dz = dY act'(gamma h + beta): a feature's sums over the tile of dz h and dz go to
// psum[t][2 D], and the groups' shares of sum gamma dz and sum gamma dz h to part.
template <class T, int TX, int V, int ACT>
__global__ void __launch_bounds__(NT) k_gnorm_sums(const T* X, int ldx, const T* dY, int lddy, const Fields p, const float* gamma,
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
  each_field(p, t, [&](int f, int a, int b) {
    float sb[V] = {}, sg[V] = {};
    if (i < p.D) {
      float m[V], r[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const size_t at = (size_t)f * lds + (i + e) / p.group;
        m[e] = mean[at];
        r[e] = rstd[at];
      }
#pragma unroll 2
      for (int j = a + ty; j < b; j += TY) {
        float x[V], d[V];
        load<T, V>(X + (size_t)j * ldx + i, x);
        load<T, V>(dY + (size_t)j * lddy + i, d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float h = __fmul_rn(x[e] - m[e], r[e]);
          if (ACT != CR_ACT_NONE) d[e] = __fmul_rn(d[e], activation_slope<ACT>(fmaf(h, gm[e], bt[e])));
          sb[e] += d[e];
          sg[e] = fmaf(d[e], h, sg[e]);
        }
      }
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
      const int lane = threadIdx.x & 31, g0 = i0 / p.group, g1 = (i0 + width - 1) / p.group;
      for (int g = g0 + ((int)threadIdx.x >> 5); g <= g1; g += NT / 32) {
        const int x0 = max(0, g * p.group - i0), x1 = min(width, (g + 1) * p.group - i0);
        float2 s = make_float2(0.0f, 0.0f);
        for (int x = x0 + lane; x < x1; x += 32) {
          const float w = gamma ? gamma[i0 + x] : 1.0f;
          s.x = fmaf(w, feature[x].x, s.x);
          s.y = fmaf(w, feature[x].y, s.y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
          s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
        }
        if (lane == 0) part[share(p, t, f, fb, g)] = s;
      }
    }
  }, [](int) {});
  __syncthreads();
  for (int x = threadIdx.x; x < width; x += NT) {
    if (pgamma) pgamma[(size_t)t * p.D + i0 + x] = all[x].y;
    if (pbeta) pbeta[(size_t)t * p.D + i0 + x] = all[x].x;
  }
}

// dX = r (gamma dz - mean(gamma dz) - h mean(gamma dz h)), means over the group.
template <class T, int TX, int V, int ACT>
__global__ void __launch_bounds__(NT) k_gnorm_dx(const T* X, int ldx, const T* dY, int lddy, const Fields p, const float2* part,
                                                 const float* gamma, const float* beta, const float* mean, const float* rstd, int lds, T* dX,
                                                 int lddx) {
  constexpr int TY = NT / TX, FW = TX * V;
  __shared__ float2 stat[FW];
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
  each_field(p, t, [&](int f, int a, int b) {
    __syncthreads();
    for (int g = g0 + ((int)threadIdx.x >> 5); g <= g1; g += NT / 32) {
      float2 s = make_float2(0.0f, 0.0f);
      each_share<FW>(p, f, g, [&](size_t k, int, int) {
        s.x += part[k].x;
        s.y += part[k].y;
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
      }
      const float n = (float)(field_begin(p, f + 1) - field_begin(p, f)) * (float)p.group;
      if ((threadIdx.x & 31) == 0) stat[g - g0] = make_float2(s.x / n, s.y / n);
    }
    __syncthreads();
    if (i < p.D) {
      float m[V], r[V], c1[V], c2[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int g = (i + e) / p.group;
        const size_t at = (size_t)f * lds + g;
        m[e] = mean[at];
        r[e] = rstd[at];
        c1[e] = stat[g - g0].x;
        c2[e] = stat[g - g0].y;
      }
#pragma unroll 2
      for (int j = a + ty; j < b; j += TY) {
        float x[V], d[V];
        load<T, V>(X + (size_t)j * ldx + i, x);
        load<T, V>(dY + (size_t)j * lddy + i, d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float h = __fmul_rn(x[e] - m[e], r[e]);
          if (ACT != CR_ACT_NONE) d[e] = __fmul_rn(d[e], activation_slope<ACT>(fmaf(h, gm[e], bt[e])));
          x[e] = __fmul_rn(r[e], fmaf(-h, c2[e], fmaf(d[e], gm[e], -c1[e])));
        }
        store<T, V>(dX + (size_t)j * lddx + i, x);
      }
    }
  }, [](int) {});
}

bool ok16(const void* p, int ld, int eb) { return ((uintptr_t)p & 15) == 0 && (long long)ld * eb % 16 == 0; }

// Calls f(TX, V) for a matrix of D features: the widest of 256, 128 and 64 features that leaves least unused.
template <class F>
cr_status with_tile(int D, bool vec, F&& f) {
  using std::integral_constant;
  if (!vec) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  const auto padded = [&](int w) { return (D + w - 1) / w * w; };
  const int best = std::min({padded(256), padded(128), padded(64)});
  if (padded(256) == best) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (padded(128) == best) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
}

// Columns of a tile: about four tiles to an SM, and 16 columns to a thread's lane of them at most.
Fields make_fields(const int32_t* off, int n, int T, int D, int groups, int width, int rows) {
  Fields p = {};
  p.off = off;
  p.n = off ? n : 1;
  p.T = T;
  p.D = D;
  p.groups = groups;
  p.group = D / groups;
  p.blocks = (D + width - 1) / width;
  const long long want = std::max(1ll, 4ll * sm_count() / p.blocks);
  const long long per = (T + want - 1) / want;
  p.cols = (int)std::min<long long>(std::max<long long>((per + 4 * rows - 1) / (4 * rows), 1) * 4 * rows, 32 * rows);
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
    const bool vec = D % 8 == 0 && ok16(d_X, ldx, sizeof(E)) && ok16(d_Y, ldy, sizeof(E));
    return with_tile(D, vec, [&](auto tx0, auto v0) -> cr_status {
      constexpr int TX = decltype(tx0)::value, V = decltype(v0)::value;
      const Fields p = make_fields(d_off, n_field, T, D, groups, TX * V, NT / TX);
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
    const bool vec = D % 8 == 0 && ok16(d_X, ldx, sizeof(E)) && ok16(d_dY, lddy, sizeof(E)) && (!d_dX || ok16(d_dX, lddx, sizeof(E)));
    return with_tile(D, vec, [&](auto tx0, auto v0) -> cr_status {
      constexpr int TX = decltype(tx0)::value, V = decltype(v0)::value;
      const Fields p = make_fields(d_off, n_field, T, D, groups, TX * V, NT / TX);
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
          if (!d_dX) return CR_OK;
          TimedScope ts("k_gnorm_dx", stream);
          CR_CUDA(launch_after(k_gnorm_dx<E, TX, V, ACT>, grid, NT, 0, 1, stream, (const E*)d_X, ldx, (const E*)d_dY, lddy, p, part, d_gamma, d_beta,
                               d_mean, d_rstd, lds, (E*)d_dX, lddx));
          CR_CHECK_LAUNCH("k_gnorm_dx");
          return CR_OK;
        }));
        if (d_dgamma) CR_TRY(add_rows(pgamma, p.tiles, D, d_dgamma, stream));
        if (d_dbeta) CR_TRY(add_rows(pbeta, p.tiles, D, d_dbeta, stream));
        return CR_OK;
      };
      const cr_status st = run();
      scratch_free(part, stream);
      return st;
    });
  });
  CR_ENTRY_END("cr_group_norm_backward")
}
