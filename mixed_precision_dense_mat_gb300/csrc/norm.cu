// Root-mean-square norm of columns with the residual's addition and an optional e4m3 output,
// and its gradient (cr_rmsnorm, cr_rmsnorm_backward).
#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "ptx.cuh"

namespace cr {
namespace {

// Both are bound by HBM: the forward pass reads X and R and writes H and Y, the backward reads H, dY
// and dH and writes dX.  A group of G threads holds one column in registers (8 VPT elements per
// thread), so that memory is read once, and needs one exchange among its threads: the sum of squares
// together with max|h gamma| (max|y| is that times r), or with the sum of u h.  Blocks are
// resident and go from column to column with gamma in registers.  Each group has a ring of columns in
// shared memory, filled by bulk copies several columns ahead: loads into registers, one column
// ahead, kept too few bytes in flight (4096 x 32768 BF16 to e4m3 with residual: 264 us,
// with the ring 147 us, 6.4 TB/s).
constexpr int NT = 256;
constexpr int MAXD = 16384;   // longer columns: the kernels that go over memory again

// maximum that keeps NaN
__device__ __forceinline__ float nan_max(float a, float b) { return clamp_low(a, b); }

// Two values reduced over the group: x by sum, y by sum or by maximum.  `red` is used alternately
// (turn) so that one barrier per column is enough.
// G = 8, 16 or 32: threads of a warp; G = 0: the block.
template <int G>
__device__ __forceinline__ int group_size() { return G ? G : (int)blockDim.x; }
template <int G>
__device__ __forceinline__ int in_group() { return G ? (int)threadIdx.x % G : (int)threadIdx.x; }
template <int G, bool MAX>
__device__ __forceinline__ void reduce2(float& x, float& y, float2 (*red)[32], int turn) {
#pragma unroll
  for (int o = G ? G / 2 : 16; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    const float z = __shfl_xor_sync(0xffffffffu, y, o);
    y = MAX ? nan_max(y, z) : y + z;
  }
  if (G) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[turn][warp] = make_float2(x, y);
  __syncthreads();
  x = red[turn][0].x;
  y = red[turn][0].y;
  for (int w = 1; w < (int)blockDim.x / 32; ++w) {
    x += red[turn][w].x;
    y = MAX ? nan_max(y, red[turn][w].y) : y + red[turn][w].y;
  }
}

// The thread's elements of a column: 8 consecutive ones VPT times (VEC: 16-byte accesses), or single
// ones G apart.
template <int G, int VPT, bool VEC>
__device__ __forceinline__ int element(int v, int e) {
  const int t = in_group<G>(), n = group_size<G>();
  return VEC ? (v * n + t) * 8 + e : t + n * (v * 8 + e);
}
template <class T, int G, int VPT, bool VEC>
__device__ __forceinline__ void load_col(const T* p, int D, float (&h)[VPT][8]) {
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (VEC) {
      const int i = element<G, VPT, VEC>(v, 0);
      Eight<T> w = {};
      if (i < D) w = *reinterpret_cast<const Eight<T>*>(p + i);
      widen8(w, h[v]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = element<G, VPT, VEC>(v, e);
        h[v][e] = i < D ? to_float(p[i]) : 0.0f;
      }
    }
  }
}
template <class O, int G, int VPT, bool VEC>
__device__ __forceinline__ void store8(O* p, int D, int v, const float (&y)[8]) {
  if (VEC) {
    const int i = element<G, VPT, VEC>(v, 0);
    if (i < D) *reinterpret_cast<Eight<O>*>(p + i) = narrow8<O>(y);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = element<G, VPT, VEC>(v, e);
      if (i < D) p[i] = from_float<O>(y[e]);
    }
  }
}
template <int G, int VPT, bool VEC>
__device__ __forceinline__ void load_gamma(const float* gamma, int D, float (&g)[VPT][8]) {
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = element<G, VPT, VEC>(v, e);
      g[v][e] = i < D ? gamma[i] : 0.0f;
    }
}

// Elements go through the arithmetic in pairs, two to an instruction (one by one: 150 us and 66 us where the kernels
// below take 147 and 62).
__device__ __forceinline__ Floats<2> two(const float* p) { return {{p[0], p[1]}}; }
__device__ __forceinline__ void put(float* p, Floats<2> v) {
  p[0] = v.x[0];
  p[1] = v.x[1];
}

// Columns of up to 256 features are read directly: a block has many of them in flight anyway (256 x 262144 BF16
// with residual: 90 us, by the ring 102; backward 84 us, 103; only to e4m3 the ring is ahead, 83 us for 86).
template <int G, int VPT, bool VEC>
__host__ __device__ constexpr bool uses_ring() { return VEC && (G == 0 || VPT > 1); }

// The group's ring: `stages` stages of the NIN inputs' columns, in the block's dynamic shared memory
// after the barriers.  The group's first thread refills the stage of the column before the present
// one, after the exchange that all threads reach only when they are done with that column.
struct Wait {
  unsigned long long limit;
  int* err;
};
// When a wait's limit runs out that is reported, and the copies, which need nobody's help, are waited for all the
// same, up to `upto`: stages are refilled and left only with nothing in flight to them.  Were they not to land even
// so, nothing more is filled or waited for (upto = 0).  Times in units of 1024 ns: 32 bits are enough, and with 64 the
// backward pass loses 1 to 3 %.
__device__ __forceinline__ uint32_t coarse(unsigned long long ns) { return (uint32_t)(ns >> 10); }
__device__ __forceinline__ void landed(uint64_t* full, uint32_t ph, const Wait& w, uint32_t& upto) {
  uint32_t t0 = 0;
  while (!mbar_try_wait(full, ph)) {
    const uint32_t t = coarse(global_timer_ns()) | 1u;
    if (t0 == 0) t0 = t;
    if (t - t0 > coarse(w.limit)) *(volatile int*)w.err = 1;
    if (t - t0 > upto) {
      upto = 0;
      return;
    }
  }
}
template <class T, int G, int NIN>
struct Ring {
  uint64_t* full;
  uint8_t* mem;
  int stages, bytes, st = 0;   // bytes of one column
  uint32_t ph = 0;
  uint32_t upto;
  __device__ Ring(uint8_t* smem, int stages_, int D, const Wait& w)
      : stages(stages_), bytes(D * (int)sizeof(T)), upto(coarse(w.limit + LANDING_NS)) {
    const int group = G ? threadIdx.x / 32 : 0, groups = G ? blockDim.x / 32 : 1;
    full = reinterpret_cast<uint64_t*>(smem) + group * stages;
    mem = smem + (groups * stages * 8 + 127) / 128 * 128 + (size_t)group * stages * NIN * bytes;
    if (in_group<G>() == 0) {
      for (int q = 0; q < stages; ++q) mbar_init(&full[q], 1);
      fence_mbar_init();
    }
    if (G == 32) __syncwarp();
    else __syncthreads();
  }
  __device__ void fill(int stage, const T* const (&col)[NIN]) {   // by the group's first thread; NULL: not there
    if (upto == 0) return;
    uint32_t n = 0;
#pragma unroll
    for (int q = 0; q < NIN; ++q)
      if (col[q]) n += bytes;
    mbar_arrive_expect_tx(&full[stage], n);
#pragma unroll
    for (int q = 0; q < NIN; ++q)
      if (col[q]) bulk_load(mem + ((size_t)stage * NIN + q) * bytes, col[q], bytes, &full[stage]);
  }
  // Waits for the current stage.
  __device__ const T* take(int q, const Wait& w) {
    if (q == 0) landed(&full[st], ph, w, upto);
    return reinterpret_cast<const T*>(mem + ((size_t)st * NIN + q) * bytes);
  }
  __device__ void next() {
    if (++st == stages) st = 0, ph ^= 1u;
  }
};

// h = x + residual, y = h r gamma with r = 1 / sqrt(mean h^2 + eps); to e4m3, divided by its column's scale max|y| / 448.
template <class T, class O, int G, int VPT, bool VEC>
__global__ void __launch_bounds__(G ? NT : 512)
    k_rmsnorm(const T* X, int ldx, const T* R, int ldr, const float* gamma, int D, int n, float eps, T* H, int ldh, O* Y, int ldy,
              float* scale, int stages, const Wait wait) {
  constexpr bool Q = std::is_same<O, __nv_fp8_e4m3>::value, RING = uses_ring<G, VPT, VEC>();
  constexpr int PER = G ? NT / G : 1;   // columns per block at a time
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][32];
  Ring<T, G, 2> ring(smem, RING ? stages : 0, D, wait);
  let_next_start();
  wait_for_previous();
  float g[VPT][8];
  const int step = gridDim.x * PER, t0 = blockIdx.x * PER + (G ? threadIdx.x / G : 0), sub = G ? threadIdx.x % 32 / G : 0;
  const auto fill = [&](int stage, long long t) {
    if (t < n) ring.fill(stage, {X + (size_t)t * ldx, R ? R + (size_t)t * ldr : nullptr});
  };
  if (RING && in_group<G>() == 0)
    for (int q = 0; q < stages - 1; ++q) fill(q, t0 + (long long)q * step);
  load_gamma<G, VPT, VEC>(gamma, D, g);
  for (int t = t0, turn = 0; t - sub < n; t += step, turn ^= 1) {   // the groups of a warp stay together
    const bool live = G == 0 || G == 32 || t < n;
    const size_t c = live ? t : n - 1;
    float h[VPT][8], mx = 0.0f;
    Floats<2> s2 = all_of<2>(0.0f);
    load_col<T, G, VPT, VEC>(RING ? ring.take(0, wait) : X + c * ldx, D, h);
    if (R) {
      float r[VPT][8];
      load_col<T, G, VPT, VEC>(RING ? ring.take(1, wait) : R + c * ldr, D, r);
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int e = 0; e < 8; e += 2) put(&h[v][e], add(two(&h[v][e]), two(&r[v][e])));
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (H && live) store8<T, G, VPT, VEC>(H + c * ldh, D, v, h[v]);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const Floats<2> x = two(&h[v][e]);
        s2 = fma(x, x, s2);
        put(&h[v][e], mul(x, two(&g[v][e])));
        if (Q) mx = nan_max(nan_max(mx, fabsf(h[v][e])), fabsf(h[v][e + 1]));
      }
    }
    float ss = s2.x[0] + s2.x[1];
    reduce2<G, true>(ss, mx, red, turn);
    if (RING) {
      if (G == 32) __syncwarp();
      if (in_group<G>() == 0) fill((ring.st ? ring.st : stages) - 1, t + (long long)(stages - 1) * step);
      ring.next();
    }
    const float rs = 1.0f / sqrtf(ss / (float)D + eps);
    float f = rs;
    if (Q) {
      const float s = nan_max(mx * rs, 0x1p-100f) / 448.0f;
      if (in_group<G>() == 0 && live) scale[c] = s;
      f = clamp_high(rs * (1.0f / s), 3.0e38f);   // kept finite, for columns of zeros
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) put(&h[v][e], mul(two(&h[v][e]), all_of<2>(f)));
      if (live) store8<O, G, VPT, VEC>(Y + c * ldy, D, v, h[v]);
    }
  }
}

// dX = r (u - h r^2 mean(u h)) + dH with u = gamma dY, dgamma = sum dY h r.  The block's sums for dgamma go to
// part[block][D], to be added by k_add_rows (2560 x 16411 BF16 with dH: 62 us in all, 5.4 TB/s).
template <class T, int G, int VPT, bool VEC>
__global__ void __launch_bounds__(G ? NT : 512)
    k_rmsnorm_bwd(const T* H, int ldh, const float* gamma, const T* dY, int lddy, const T* dH, int lddh, int D, int n, float eps, T* dX,
                  int lddx, float* part, int stages, const Wait wait) {
  constexpr bool RING = uses_ring<G, VPT, VEC>();
  constexpr int PER = G ? NT / G : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][32];
  Ring<T, G, 3> ring(smem, RING ? stages : 0, D, wait);
  let_next_start();
  wait_for_previous();
  float g[VPT][8], dg[VPT][8] = {};
  const int step = gridDim.x * PER, t0 = blockIdx.x * PER + (G ? threadIdx.x / G : 0), sub = G ? threadIdx.x % 32 / G : 0;
  const auto fill = [&](int stage, long long t) {
    if (t < n) ring.fill(stage, {H + (size_t)t * ldh, dY + (size_t)t * lddy, dH ? dH + (size_t)t * lddh : nullptr});
  };
  if (RING && in_group<G>() == 0)
    for (int q = 0; q < stages - 1; ++q) fill(q, t0 + (long long)q * step);
  load_gamma<G, VPT, VEC>(gamma, D, g);
  for (int t = t0, turn = 0; t - sub < n; t += step, turn ^= 1) {
    const bool live = G == 0 || G == 32 || t < n;
    const size_t c = live ? t : n - 1;
    const T *ch = RING ? ring.take(0, wait) : H + c * ldh, *cd = RING ? ring.take(1, wait) : dY + c * lddy;
    float h[VPT][8], d[VPT][8];
    Floats<2> s2 = all_of<2>(0.0f), dot2 = all_of<2>(0.0f);
    load_col<T, G, VPT, VEC>(ch, D, h);
    load_col<T, G, VPT, VEC>(cd, D, d);
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const Floats<2> x = two(&h[v][e]);
        s2 = fma(x, x, s2);
        dot2 = fma(mul(two(&g[v][e]), two(&d[v][e])), x, dot2);
      }
    float ss = s2.x[0] + s2.x[1], dot = dot2.x[0] + dot2.x[1];
    const T* cr = !dH ? nullptr : RING ? ring.take(2, wait) : dH + c * lddh;
    reduce2<G, false>(ss, dot, red, turn);
    if (RING) {
      if (G == 32) __syncwarp();
      if (in_group<G>() == 0) fill((ring.st ? ring.st : stages) - 1, t + (long long)(stages - 1) * step);
    }
    const float rs = 1.0f / sqrtf(ss / (float)D + eps), m = dot / (float)D * rs * rs * rs;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float o[8] = {};
      if (cr) {
        if (VEC) {
          const int i = element<G, VPT, VEC>(v, 0);
          Eight<T> w = {};
          if (i < D) w = *reinterpret_cast<const Eight<T>*>(cr + i);
          widen8(w, o);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = element<G, VPT, VEC>(v, e);
            o[e] = i < D ? to_float(cr[i]) : 0.0f;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const Floats<2> x = two(&h[v][e]), y = two(&d[v][e]);
        if (live) put(&dg[v][e], fma(mul(y, x), all_of<2>(rs), two(&dg[v][e])));
        put(&o[e], add(two(&o[e]), fma(x, all_of<2>(-m), mul(all_of<2>(rs), mul(two(&g[v][e]), y)))));
      }
      if (dX && live) store8<T, G, VPT, VEC>(dX + c * lddx, D, v, o);
    }
    if (RING) ring.next();
  }
  if (!part) return;
  float* out = part + (size_t)blockIdx.x * D;
  if (G == 0) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = element<G, VPT, VEC>(v, e);
        if (i < D) out[i] = dg[v][e];
      }
  } else {   // the block's columns, one after the other
    __shared__ float sum[NT / 32][33];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float own = dg[v][e];
#pragma unroll
        for (int o = 16; o >= G && o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);   // the warp's groups
        __syncthreads();
        sum[threadIdx.x >> 5][threadIdx.x & 31] = own;
        __syncthreads();
        const int i = element<G, VPT, VEC>(v, e);
        if (threadIdx.x < G && i < D) {
          float x = 0.0f;
          for (int w = 0; w < NT / 32; ++w) x += sum[w][threadIdx.x];
          out[i] = x;
        }
      }
  }
}

// The sum of `rows` partial vectors (gradients of vectors), in a fixed order: 32 features per block, 32 threads each.
// Latency (456 rows of 2560: 7.6 us cold).
__global__ void __launch_bounds__(1024) k_add_rows(const float* part, int rows, int D, float* total) {
  __shared__ float sum[32][33];
  let_next_start();
  wait_for_previous();
  const int i = blockIdx.x * 32 + threadIdx.x % 32, y0 = threadIdx.x / 32;
  float s = 0.0f;
  if (i < D)
    for (int r = y0; r < rows; r += 32) s += part[(size_t)r * D + i];
  sum[y0][threadIdx.x % 32] = s;
  __syncthreads();
  if (y0 == 0 && i < D) {
    for (int y = 1; y < 32; ++y) s += sum[y][threadIdx.x];
    total[i] = s;
  }
}

// ---------------------------------------------------------------- columns longer than MAXD
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

// One block per column, the column read once for each of its reductions: bound by HBM and L2 (20000 x 4096 BF16 with
// residual 254 us, to e4m3 270 us).
template <class T, class O>
__global__ void __launch_bounds__(NT) k_rmsnorm_long(const T* X, int ldx, const T* R, int ldr, const float* gamma, int D,
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
__global__ void __launch_bounds__(NT) k_rmsnorm_dx_long(const T* H, int ldh, const float* gamma, const T* dY, int lddy,
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

// A feature per thread and part blockIdx.y of the columns, to part[blockIdx.y][D]; k_add_rows adds the parts.
// Bound by HBM once enough parts keep loads in flight (20000 x 4096 BF16, the whole backward pass: 437 us, in one
// part 1689 us).
template <class T>
__global__ void __launch_bounds__(NT) k_rmsnorm_dgamma_long(const T* H, int ldh, const T* dY, int lddy, const float* rs, int D,
                                                            int T_, int per, float* part) {
  const int i = blockIdx.x * NT + threadIdx.x;
  if (i >= D) return;
  const int t0 = blockIdx.y * per, t1 = min(T_, t0 + per);
  float s = 0.0f;
#pragma unroll 4
  for (int t = t0; t < t1; ++t)
    s = fmaf(__fmul_rn(to_float(dY[(size_t)t * lddy + i]), to_float(H[(size_t)t * ldh + i])), rs[t], s);
  part[(size_t)blockIdx.y * D + i] = s;
}

// Calls f(group, vectors per thread, 16-byte accesses) as integral constants for columns of D: 8 or 16
// threads per column up to 64 and 128 (64 x 1048576 BF16 with residual: 90 us, a warp per column 260 us), a warp
// per column up to 1024, then a block of as many warps as the column fills.
template <class F>
cr_status with_split(int D, bool vec, F&& f) {
  const auto go = [&](auto g, auto v) -> cr_status {
    return vec ? f(g, v, std::true_type{}) : f(g, v, std::false_type{});
  };
  using std::integral_constant;
  if (D <= 64) return go(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (D <= 128) return go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (D <= 256) return go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (!vec && D <= 1024) return f(integral_constant<int, 0>{}, integral_constant<int, 1>{}, std::false_type{});
  if (D <= 512) return go(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  if (D <= 768) return go(integral_constant<int, 32>{}, integral_constant<int, 3>{});
  if (D <= 1024) return go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  if (D <= 4096) return go(integral_constant<int, 0>{}, integral_constant<int, 1>{});
  if (D <= 8192) return go(integral_constant<int, 0>{}, integral_constant<int, 2>{});
  return go(integral_constant<int, 0>{}, integral_constant<int, 4>{});
}
constexpr int threads_for(int G, int VPT, int D) { return G ? NT : (D + 256 * VPT - 1) / (256 * VPT) * 32; }

// Whether two stages of a column's inputs fit; longer ones are read directly.
bool ring_fits(int nin, int D, int eb) { return 2ll * nin * D * eb <= 200 * 1024; }
constexpr int MAXSHARED = 224 * 1024;   // of the rings, next to at most 2 KB of static shared memory
// Blocks for n columns, `per` at a time each, stages of their rings and shared memory: about 50 KB,
// so that several blocks share an SM; no more stages than a block has columns.
struct Plan {
  int blocks = 0, stages = 0;
  size_t smem = 0;
};
template <class K>
cr_status make_plan(Plan& plan, K kernel, int threads, int n, int per, bool ring, int nin, int D, int eb) {
  const int items = (n + per - 1) / per;
  const size_t stage = (size_t)per * nin * D * eb;
  if (ring) {
    plan.stages = (int)std::min<size_t>(8, std::max<size_t>(2, (size_t)50 * 1024 / stage));
    if (items <= sm_count()) plan.stages = 2;
    plan.smem = ((size_t)per * plan.stages * 8 + 127) / 128 * 128 + plan.stages * stage;
  }
  plan.blocks = items;
  if (items <= sm_count()) return CR_OK;   // one each
  int b = 0;
  CR_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, kernel, threads, plan.smem));
  plan.blocks = std::min(items, std::max(b, 1) * sm_count());
  return CR_OK;
}

struct Fwd {
  const void *X, *R;
  int ldx, ldr;
  const float* gamma;
  int D, n;
  float eps;
  void *H, *Y;
  int ldh, ldy;
  float* scale;
  Wait wait;
};
template <class T, class O, int G, int VPT, bool VEC>
cr_status launch_fwd(const Fwd& p, cudaStream_t stream) {
  constexpr int PER = G ? NT / G : 1;
  const int TH = threads_for(G, VPT, p.D);
  static std::atomic<uint64_t> done{0};
  CR_TRY(allow_shared((const void*)k_rmsnorm<T, O, G, VPT, VEC>, MAXSHARED, done));
  Plan plan;
  CR_TRY(make_plan(plan, k_rmsnorm<T, O, G, VPT, VEC>, TH, p.n, PER, uses_ring<G, VPT, VEC>(), 2, p.D, sizeof(T)));
  TimedScope ts("k_rmsnorm", stream);
  CR_CUDA(launch_after(k_rmsnorm<T, O, G, VPT, VEC>, plan.blocks, TH, plan.smem, 1, stream, (const T*)p.X, p.ldx, (const T*)p.R, p.ldr,
                       p.gamma, p.D, p.n, p.eps, (T*)p.H, p.ldh, (O*)p.Y, p.ldy, p.scale, plan.stages, p.wait));
  CR_CHECK_LAUNCH("k_rmsnorm");
  return CR_OK;
}

struct Bwd {
  const void *H, *dY, *dH;
  int ldh, lddy, lddh;
  const float* gamma;
  int D, n;
  float eps;
  void* dX;
  int lddx;
  float* dgamma;
  Wait wait;
};
template <class T, int G, int VPT, bool VEC>
cr_status launch_bwd(const Bwd& p, cudaStream_t stream) {
  constexpr int PER = G ? NT / G : 1;
  const int TH = threads_for(G, VPT, p.D);
  static std::atomic<uint64_t> done{0};
  CR_TRY(allow_shared((const void*)k_rmsnorm_bwd<T, G, VPT, VEC>, MAXSHARED, done));
  Plan plan;
  CR_TRY(make_plan(plan, k_rmsnorm_bwd<T, G, VPT, VEC>, TH, p.n, PER, uses_ring<G, VPT, VEC>(), 3, p.D, sizeof(T)));
  const int blocks = plan.blocks;
  float* part = nullptr;
  if (p.dgamma) CR_CUDA(scratch_alloc((void**)&part, (size_t)blocks * p.D * sizeof(float), stream));
  cudaError_t e;
  {
    TimedScope ts("k_rmsnorm_bwd", stream);
    e = launch_after(k_rmsnorm_bwd<T, G, VPT, VEC>, blocks, TH, plan.smem, 1, stream, (const T*)p.H, p.ldh, p.gamma, (const T*)p.dY, p.lddy,
                     (const T*)p.dH, p.lddh, p.D, p.n, p.eps, (T*)p.dX, p.lddx, part, plan.stages, p.wait);
    count_launch();
  }
  const cr_status st = e != cudaSuccess ? cuda_fail(e, "k_rmsnorm_bwd") : p.dgamma ? add_rows(part, blocks, p.D, p.dgamma, stream) : CR_OK;
  scratch_free(part, stream);
  return st;
}

bool ok16(const void* p, int ld, int eb) { return !p || (((uintptr_t)p & 15) == 0 && (long long)ld * eb % 16 == 0); }

bool float_type(int t) { return t == CR_TYPE_F32 || t == CR_TYPE_F16 || t == CR_TYPE_BF16; }

}  // namespace

cr_status add_rows(const float* part, int rows, int D, float* total, cudaStream_t stream) {
  CR_CUDA(launch_after(k_add_rows, (unsigned)((D + 31) / 32), 1024, 0, 1, stream, part, rows, D, total));
  CR_CHECK_LAUNCH("k_add_rows");
  return CR_OK;
}

}  // namespace cr

using namespace cr;

extern "C" cr_status cr_rmsnorm(int type, const void* d_X, int ldx, const void* d_R, int ldr, const float* d_gamma, int D,
                                int T, double eps, void* d_H, int ldh, int out_type, void* d_Y, int ldy, float* d_scale,
                                cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(float_type(type), "cr_rmsnorm: type must be FP32, FP16 or BF16");
  CR_REQUIRE(out_type == type || out_type == CR_TYPE_E4M3, "cr_rmsnorm: out_type must be type or e4m3");
  CR_REQUIRE(D >= 1 && T >= 0, "cr_rmsnorm: D >= 1, T >= 0");
  CR_REQUIRE_SIZES("cr_rmsnorm", D, T);
  CR_REQUIRE(eps >= 0.0 && eps < 1e30, "cr_rmsnorm: eps must be finite and not negative");
  CR_REQUIRE(ldx >= D && ldy >= D && (!d_R || ldr >= D) && (!d_H || ldh >= D), "cr_rmsnorm: leading dimension below D");
  CR_REQUIRE((out_type == CR_TYPE_E4M3) == (d_scale != nullptr) || T == 0, "cr_rmsnorm: d_scale belongs to the e4m3 output");
  if (T == 0) return CR_OK;
  CR_REQUIRE(d_X && d_gamma && d_Y, "cr_rmsnorm: NULL argument");
  Wait wait = {option_wait_ns(), nullptr};
  CR_TRY(wait_word(&wait.err));
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    const int eb = sizeof(E);
    const auto run = [&](auto o0) -> cr_status {
      using O = decltype(o0);
      if (D > MAXD) {
        k_rmsnorm_long<E, O><<<T, NT, 0, stream>>>((const E*)d_X, ldx, (const E*)d_R, ldr, d_gamma, D, (float)eps, (E*)d_H, ldh,
                                                   (O*)d_Y, ldy, d_scale);
        CR_CHECK_LAUNCH("k_rmsnorm_long");
        return CR_OK;
      }
      const bool vec = D % 8 == 0 && ring_fits(2, D, eb) && ok16(d_X, ldx, eb) && ok16(d_R, ldr, eb) && ok16(d_H, ldh, eb) &&
                       (sizeof(O) == 1 ? ((uintptr_t)d_Y & 7) == 0 && ldy % 8 == 0 : ok16(d_Y, ldy, sizeof(O)));
      return with_split(D, vec, [&](auto g, auto v, auto w) -> cr_status {
        return launch_fwd<E, O, decltype(g)::value, decltype(v)::value, decltype(w)::value>(
            Fwd{d_X, d_R, ldx, ldr, d_gamma, D, T, (float)eps, d_H, d_Y, ldh, ldy, d_scale, wait}, stream);
      });
    };
    return out_type == CR_TYPE_E4M3 ? run(__nv_fp8_e4m3{}) : run(t0);
  });
  CR_ENTRY_END("cr_rmsnorm")
}

extern "C" cr_status cr_rmsnorm_backward(int type, const void* d_H, int ldh, const float* d_gamma, const void* d_dY, int lddy,
                                         const void* d_dH, int lddh, int D, int T, double eps, void* d_dX, int lddx,
                                         float* d_dgamma, cr_stream stream) {
  CR_ENTRY_BEGIN
  CR_REQUIRE(float_type(type), "cr_rmsnorm_backward: type must be FP32, FP16 or BF16");
  CR_REQUIRE(D >= 1 && T >= 0, "cr_rmsnorm_backward: D >= 1, T >= 0");
  CR_REQUIRE_SIZES("cr_rmsnorm_backward", D, T);
  CR_REQUIRE(eps >= 0.0 && eps < 1e30, "cr_rmsnorm_backward: eps must be finite and not negative");
  CR_REQUIRE(ldh >= D && lddy >= D && (!d_dH || lddh >= D) && (!d_dX || lddx >= D),
             "cr_rmsnorm_backward: leading dimension below D");
  if (T == 0) {
    if (d_dgamma) CR_CUDA(cudaMemsetAsync(d_dgamma, 0, (size_t)D * sizeof(float), stream));
    return CR_OK;
  }
  CR_REQUIRE(d_H && d_gamma && d_dY, "cr_rmsnorm_backward: NULL argument");
  if (!d_dX && !d_dgamma) return CR_OK;
  Wait wait = {option_wait_ns(), nullptr};
  CR_TRY(wait_word(&wait.err));
  float* mem = nullptr;
  const cr_status st = with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    if (D > MAXD) {
      const int bx = (D + NT - 1) / NT, per = std::max(8, (int)(((long long)T * bx + 8 * sm_count() - 1) / (8 * sm_count())));
      const int by = (int)(((long long)T + per - 1) / per);
      CR_CUDA(scratch_alloc((void**)&mem, ((size_t)T + (d_dgamma ? (size_t)by * D : 0)) * sizeof(float), stream));
      if (d_dgamma) {   // first, since dX may overwrite dY: the columns' r, without writing dX, then the sums
        k_rmsnorm_dx_long<E><<<T, NT, 0, stream>>>((const E*)d_H, ldh, d_gamma, (const E*)d_dY, lddy, nullptr, 0, D, (float)eps, nullptr, 0, mem);
        CR_CHECK_LAUNCH("k_rmsnorm_dx_long");
        k_rmsnorm_dgamma_long<E><<<dim3(bx, by), NT, 0, stream>>>((const E*)d_H, ldh, (const E*)d_dY, lddy, mem, D, T, per, mem + T);
        CR_CHECK_LAUNCH("k_rmsnorm_dgamma_long");
        CR_TRY(add_rows(mem + T, by, D, d_dgamma, stream));
      }
      if (d_dX) {
        k_rmsnorm_dx_long<E><<<T, NT, 0, stream>>>((const E*)d_H, ldh, d_gamma, (const E*)d_dY, lddy, (const E*)d_dH, lddh, D,
                                                   (float)eps, (E*)d_dX, lddx, mem);
        CR_CHECK_LAUNCH("k_rmsnorm_dx_long");
      }
      return CR_OK;
    }
    const int eb = sizeof(E);
    const bool vec = D % 8 == 0 && ring_fits(3, D, eb) && ok16(d_H, ldh, eb) && ok16(d_dY, lddy, eb) && ok16(d_dH, lddh, eb) && ok16(d_dX, lddx, eb);
    return with_split(D, vec, [&](auto g, auto v, auto w) -> cr_status {
      return launch_bwd<E, decltype(g)::value, decltype(v)::value, decltype(w)::value>(
          Bwd{d_H, d_dY, d_dH, ldh, lddy, lddh, d_gamma, D, T, (float)eps, d_dX, lddx, d_dgamma, wait}, stream);
    });
  });
  scratch_free(mem, stream);
  return st;
  CR_ENTRY_END("cr_rmsnorm_backward")
}
