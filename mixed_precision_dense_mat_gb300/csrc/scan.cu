// Gated recurrence along time over packed series, its gradient and its single step
// (cr_gated_scan, cr_gated_scan_backward, cr_gated_step).
#include <limits.h>

#include <type_traits>

#include "ops.cuh"
#include "ptx.cuh"

namespace cr {
namespace {

// How the scan is split.  A block owns 32 VEC features and CH consecutive steps (a chunk); each of its
// 8 warps owns SUB of the steps, each thread VEC features of them, in registers, so that G and X
// are read once and H is written once.  The map of a run of steps on the state is h -> A h + B,
// and such maps compose; "start from h0" is the map A = 0, B = h0, so that packed series need
// no other care (A = 0 is taken as "forget", not multiplied, so that nothing crosses into the
// next series).  Warps join their maps in shared memory, chunks through global memory in two
// levels: a chunk composes the maps of the earlier chunks of its group, and takes the state
// before the group from the group's predecessor.  Every composition has a fixed order, so results
// do not depend on which block is done first.  Blocks take their place from a counter: whatever a
// block waits for was taken earlier and is running.
constexpr int WARPS = 8, NT = 32 * WARPS;
constexpr int FSUB = 16, BSUB = 8;        // steps per thread, forward and backward
constexpr int BLOCK = WARPS * BSUB;       // steps between saved states: a chunk of the backward pass
constexpr int MAXGROUP = 64;

struct Lookback {
  int chunks, tiles, group;
  int* flags;      // counter, then [tile][chunk] map written, then [tile][group] state written
  float2* maps;    // [chunk][feature]
  float* states;   // [group][feature]: the state that the group hands on
  unsigned long long limit;
  int* err;
};

__device__ __forceinline__ void forget_or(float& A, float& B, float a, float b) {   // (a, b) after (A, B)
  B = a == 0.0f ? b : fmaf(a, B, b);
  A = a == 0.0f ? 0.0f : A * a;
}
__device__ __forceinline__ float apply_map(float A, float B, float h) { return A == 0.0f ? B : fmaf(A, h, B); }

__device__ __forceinline__ int ld_flag(const int* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Marks data that the warp's lanes have stored as readable.
__device__ __forceinline__ void raise_flag(int* p) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    __threadfence();
    asm volatile("st.relaxed.gpu.global.s32 [%0], 1;" ::"l"(p) : "memory");
  }
}
// Waits until flags[0 .. n) are raised (n <= 32, one per lane); false when the limit runs out.
__device__ __forceinline__ bool wait_flags(const int* flags, int n, const Lookback& lb) {
  const int lane = threadIdx.x & 31;
  unsigned long long t0 = 0;
  while (true) {
    const bool up = lane >= n || ld_flag(flags + lane) != 0;
    if (__all_sync(0xffffffffu, up)) break;
    const unsigned long long t = global_timer_ns();
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, t - t0 > lb.limit)) {
      *(volatile int*)lb.err = 1;
      __threadfence_system();
      return false;
    }
  }
  __threadfence();
  return true;
}

// First s in [0, n] with off[s] >= t, found by the 32 lanes together.
__device__ __forceinline__ int first_at_least(const int32_t* off, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5, p = lo + (lane + 1) * step - 1;
    const bool less = p < hi && off[p] < t;
    const int c = __popc(__ballot_sync(0xffffffffu, less)), nlo = lo + c * step;
    if (step == 1) return nlo;
    hi = min(hi, nlo + step - 1);
    lo = nlo;
  }
  return lo;
}

// Series that start or end in the chunk [t0, t0 + len): first[t - t0], last[t - t0] = the series or -1.
// empty(s) is called (by a whole warp) for the empty series that belong to the chunk.
template <class F>
__device__ __forceinline__ void mark_series(const int32_t* off, int n, int t0, int len, int T, int* first, int* last, F&& empty) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int q = threadIdx.x; q < len; q += NT) {
    first[q] = !off && t0 + q == 0 ? 0 : -1;
    last[q] = !off && t0 + q == T - 1 ? 0 : -1;
  }
  if (!off) return;
  const int lo = first_at_least(off, n, t0);
  const bool final = t0 + len >= T;   // empty series at T belong to the last chunk
  __syncthreads();
  for (int base = max(lo - 1, 0) + warp * 32; base < n; base += NT) {
    const int s = base + lane;
    const int b = s < n ? off[s] : INT_MAX, e = s < n ? off[s + 1] : INT_MAX;
    const bool in = s < n && (b < t0 + len || final);
    if (in && e > b) {
      if (b >= t0 && b < t0 + len) first[b - t0] = s;
      if (e - 1 >= t0 && e - 1 < t0 + len) last[e - 1 - t0] = s;
    }
    uint32_t none = __ballot_sync(0xffffffffu, in && s >= lo && e <= b);
    for (; none; none &= none - 1) empty(base + __ffs(none) - 1);
    if (!__any_sync(0xffffffffu, in)) break;
  }
}

// The state that enters this block's chunk k of its tile, for the features f .. f + VEC - 1 of the
// thread: (A, B) is the chunk's own map, the same in all warps.  fold and state are shared memory.
// All threads call it; false when a wait ran out.
template <int VEC>
__device__ __forceinline__ bool state_in(const Lookback& lb, int tile, int k, int f, int D, const float (&A)[VEC], const float (&B)[VEC],
                                         float2 (*fold)[32 * VEC], float* state, int* bad, float (&h)[VEC]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = k / lb.group, in = k % lb.group, c0 = g * lb.group;
  int* flags = lb.flags + 1 + (size_t)tile * lb.chunks;
  int* gflags = lb.flags + 1 + (size_t)lb.tiles * lb.chunks + (size_t)tile * ((lb.chunks + lb.group - 1) / lb.group);
  const bool lastin = in == lb.group - 1;
  if (warp == 0 && !lastin && k + 1 < lb.chunks) {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      if (f + v < D) lb.maps[(size_t)k * D + f + v] = make_float2(A[v], B[v]);
    raise_flag(flags + k);
  }
  // the earlier chunks of the group, a fixed part of them per warp
  const int per = lb.group / WARPS, c1 = min(in, (warp + 1) * per);
  float FA[VEC], FB[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) FA[v] = 1.0f, FB[v] = 0.0f;
  bool ok = true;
  if (warp * per < c1) {
    ok = wait_flags(flags + c0 + warp * per, c1 - warp * per, lb);
    if (ok) {
      float2 m[MAXGROUP / WARPS][VEC];
#pragma unroll
      for (int q = 0; q < MAXGROUP / WARPS; ++q)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          m[q][v] = warp * per + q < c1 && f + v < D ? __ldcg(lb.maps + (size_t)(c0 + warp * per + q) * D + f + v) : make_float2(1.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < MAXGROUP / WARPS; ++q)
#pragma unroll
        for (int v = 0; v < VEC; ++v) forget_or(FA[v], FB[v], m[q][v].x, m[q][v].y);
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) fold[warp][lane * VEC + v] = make_float2(FA[v], FB[v]);
  if (warp == 0) {
    if (g > 0) ok = wait_flags(gflags + g - 1, 1, lb) && ok;
#pragma unroll
    for (int v = 0; v < VEC; ++v) state[lane * VEC + v] = g > 0 && ok && f + v < D ? __ldcg(lb.states + (size_t)(g - 1) * D + f + v) : 0.0f;
  }
  if (!ok) *bad = 1;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    h[v] = state[lane * VEC + v];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 m = fold[w][lane * VEC + v];
      h[v] = apply_map(m.x, m.y, h[v]);
    }
  }
  if (warp == 0 && lastin && k + 1 < lb.chunks) {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      if (f + v < D) lb.states[(size_t)g * D + f + v] = apply_map(A[v], B[v], h[v]);
    raise_flag(gflags + g);
  }
  return *(volatile int*)bad == 0;
}

template <class T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T x[VEC];
};

// The features' h0 (or its gradient's seed) of series s.
template <int VEC>
__device__ __forceinline__ void load_state(const float* h0, int ld, int s, int f, int D, float (&h)[VEC]) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) h[v] = h0 && f + v < D ? h0[(size_t)s * ld + f + v] : 0.0f;
}
template <int VEC>
__device__ __forceinline__ void store_state(float* hT, int ld, int s, int f, int D, const float (&h)[VEC]) {
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    if (hT && f + v < D) hT[(size_t)s * ld + f + v] = h[v];
}

template <class T>
struct FwdArgs {
  const T *G, *X;
  int ldg, ldx, D, n;   // n columns
  const int32_t* off;
  int series;
  const float* h0;
  int ldh0;
  T* H;
  int ldh;
  float* hT;
  int ldhT;
  float* saved;
};

// Forward scan.  Bound by HBM (G and X read, H written).
template <class T, int GATE, int VEC>
__global__ void __launch_bounds__(NT, 2) k_scan_fwd(const FwdArgs<T> p, const Lookback lb) {
  constexpr int CH = WARPS * FSUB, W = 32 * VEC;
  __shared__ int first[CH], last[CH], s_place, s_bad;
  __shared__ float2 maps[WARPS][W], fold[WARPS][W];
  __shared__ float state[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    s_place = lb.chunks > 1 ? atomicAdd(lb.flags, 1) : (int)blockIdx.x;
    s_bad = 0;
  }
  __syncthreads();
  const int k = s_place / lb.tiles, tile = s_place % lb.tiles, t0 = k * CH + warp * FSUB, f = tile * W + lane * VEC;
  const bool on = f < p.D;
  Pack<T, VEC> rg[FSUB], rx[FSUB];
#pragma unroll
  for (int i = 0; i < FSUB; ++i)
    if (on && t0 + i < p.n) {
      rg[i] = *reinterpret_cast<const Pack<T, VEC>*>(p.G + (size_t)(t0 + i) * p.ldg + f);
      rx[i] = *reinterpret_cast<const Pack<T, VEC>*>(p.X + (size_t)(t0 + i) * p.ldx + f);
    }
  mark_series(p.off, p.series, k * CH, CH, p.n, first, last, [&](int s) {
    float h[VEC];
    load_state<VEC>(p.h0, p.ldh0, s, f, p.D, h);
    store_state<VEC>(p.hT, p.ldhT, s, f, p.D, h);
  });
  __syncthreads();
  const uint32_t starts = __ballot_sync(0xffffffffu, lane < FSUB && first[warp * FSUB + (lane & (FSUB - 1))] >= 0);
  const uint32_t ends = __ballot_sync(0xffffffffu, lane < FSUB && last[warp * FSUB + (lane & (FSUB - 1))] >= 0);

  float a[FSUB][VEC], b[FSUB][VEC], A[VEC], B[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) A[v] = 1.0f, B[v] = 0.0f;
#pragma unroll
  for (int i = 0; i < FSUB; ++i) {
    if (starts >> i & 1u) {
      load_state<VEC>(p.h0, p.ldh0, first[warp * FSUB + i], f, p.D, B);
#pragma unroll
      for (int v = 0; v < VEC; ++v) A[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const bool in = on && t0 + i < p.n;
      const Gate g = gate_of<GATE>(in ? to_float(rg[i].x[v]) : 0.0f);
      a[i][v] = in ? g.a : 1.0f;
      b[i][v] = in ? __fmul_rn(g.c, to_float(rx[i].x[v])) : 0.0f;
      A[v] *= a[i][v];
      B[v] = fmaf(a[i][v], B[v], b[i][v]);
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) maps[warp][lane * VEC + v] = make_float2(A[v], B[v]);
  __syncthreads();
  // the map of the warps before this one, and the whole chunk's
  float PA[VEC], PB[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    A[v] = PA[v] = 1.0f, B[v] = PB[v] = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 m = maps[w][lane * VEC + v];
      forget_or(A[v], B[v], m.x, m.y);
      if (w < warp) PA[v] = A[v], PB[v] = B[v];
    }
  }
  float h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) h[v] = 0.0f;
  if (lb.chunks > 1 && !state_in<VEC>(lb, tile, k, f, p.D, A, B, fold, state, &s_bad, h)) return;
#pragma unroll
  for (int v = 0; v < VEC; ++v) h[v] = apply_map(PA[v], PB[v], h[v]);
  if (p.saved && warp * FSUB % BLOCK == 0 && t0 < p.n) store_state<VEC>(p.saved, p.D, t0 / BLOCK, f, p.D, h);
#pragma unroll
  for (int i = 0; i < FSUB; ++i) {
    if (starts >> i & 1u) load_state<VEC>(p.h0, p.ldh0, first[warp * FSUB + i], f, p.D, h);
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = fmaf(a[i][v], h[v], b[i][v]);
    if (p.H && on && t0 + i < p.n) {
      Pack<T, VEC> o;
#pragma unroll
      for (int v = 0; v < VEC; ++v) o.x[v] = from_float<T>(h[v]);
      *reinterpret_cast<Pack<T, VEC>*>(p.H + (size_t)(t0 + i) * p.ldh + f) = o;
    }
    if (ends >> i & 1u) store_state<VEC>(p.hT, p.ldhT, last[warp * FSUB + i], f, p.D, h);
  }
}

template <class T>
struct BwdArgs {
  const T *G, *X, *dH;
  int ldg, ldx, lddh, D, n;
  const int32_t* off;
  int series;
  const float *h0, *dhT, *saved;
  int ldh0, lddhT;
  T *dG, *dX;
  int lddg, lddx;
  float* dh0;
  int lddh0;
};

// Backward scan, from the last chunk to the first: r_t = a_t q_t, q_t = dh_t + r_{t+1}, with "take dhT" at
// a series' last step.  The states inside a chunk are recomputed from the saved one before
// it, which reads G and X (needed anyway) in place of H.  Bound by HBM (G, X, dH read, dG, dX written).
template <class T, int GATE, int VEC>
__global__ void __launch_bounds__(NT, 2) k_scan_bwd(const BwdArgs<T> p, const Lookback lb) {
  constexpr int CH = BLOCK, SUB = BSUB, W = 32 * VEC;
  __shared__ int first[CH], last[CH], s_place, s_bad;
  __shared__ float2 maps[WARPS][W], back[WARPS][W], fold[WARPS][W];
  __shared__ float state[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    s_place = lb.chunks > 1 ? atomicAdd(lb.flags, 1) : (int)blockIdx.x;
    s_bad = 0;
  }
  __syncthreads();
  const int k = s_place / lb.tiles, tile = s_place % lb.tiles, chunk = lb.chunks - 1 - k;
  const int t0 = chunk * CH + warp * SUB, f = tile * W + lane * VEC;
  const bool on = f < p.D;
  Pack<T, VEC> rg[SUB], rx[SUB], rd[SUB];
#pragma unroll
  for (int i = 0; i < SUB; ++i)
    if (on && t0 + i < p.n) {
      rg[i] = *reinterpret_cast<const Pack<T, VEC>*>(p.G + (size_t)(t0 + i) * p.ldg + f);
      rx[i] = *reinterpret_cast<const Pack<T, VEC>*>(p.X + (size_t)(t0 + i) * p.ldx + f);
      rd[i] = *reinterpret_cast<const Pack<T, VEC>*>(p.dH + (size_t)(t0 + i) * p.lddh + f);
    }
  float h[VEC];
  load_state<VEC>(p.saved, p.D, chunk, f, p.D, h);
  mark_series(p.off, p.series, chunk * CH, CH, p.n, first, last, [&](int s) {
    float q[VEC];
    load_state<VEC>(p.dhT, p.lddhT, s, f, p.D, q);
    store_state<VEC>(p.dh0, p.lddh0, s, f, p.D, q);
  });
  __syncthreads();
  const uint32_t starts = __ballot_sync(0xffffffffu, lane < SUB && first[warp * SUB + (lane & (SUB - 1))] >= 0);
  const uint32_t ends = __ballot_sync(0xffffffffu, lane < SUB && last[warp * SUB + (lane & (SUB - 1))] >= 0);

  float a[SUB][VEC], b[SUB][VEC], A[VEC], B[VEC], RA[VEC], RB[VEC];   // b: c x, then the state before the step
#pragma unroll
  for (int v = 0; v < VEC; ++v) A[v] = RA[v] = 1.0f, B[v] = RB[v] = 0.0f;
#pragma unroll
  for (int i = 0; i < SUB; ++i) {
    if (starts >> i & 1u) {
      load_state<VEC>(p.h0, p.ldh0, first[warp * SUB + i], f, p.D, B);
#pragma unroll
      for (int v = 0; v < VEC; ++v) A[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const bool in = on && t0 + i < p.n;
      const Gate g = gate_of<GATE>(in ? to_float(rg[i].x[v]) : 0.0f);
      a[i][v] = in ? g.a : 1.0f;
      b[i][v] = in ? __fmul_rn(g.c, to_float(rx[i].x[v])) : 0.0f;
      A[v] *= a[i][v];
      B[v] = fmaf(a[i][v], B[v], b[i][v]);
    }
  }
#pragma unroll
  for (int i = SUB - 1; i >= 0; --i) {
    if (ends >> i & 1u) {
      load_state<VEC>(p.dhT, p.lddhT, last[warp * SUB + i], f, p.D, RB);
#pragma unroll
      for (int v = 0; v < VEC; ++v) RA[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float d = on && t0 + i < p.n ? to_float(rd[i].x[v]) : 0.0f;
      RB[v] = __fmul_rn(a[i][v], __fadd_rn(d, RB[v]));
      RA[v] *= a[i][v];
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    maps[warp][lane * VEC + v] = make_float2(A[v], B[v]);
    back[warp][lane * VEC + v] = make_float2(RA[v], RB[v]);
  }
  __syncthreads();
  float PA[VEC], PB[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 m = maps[w][lane * VEC + v];
      if (w < warp) h[v] = apply_map(m.x, m.y, h[v]);
    }
    RA[v] = PA[v] = 1.0f, RB[v] = PB[v] = 0.0f;
#pragma unroll
    for (int w = WARPS - 1; w >= 0; --w) {
      const float2 m = back[w][lane * VEC + v];
      forget_or(RA[v], RB[v], m.x, m.y);
      if (w > warp) PA[v] = RA[v], PB[v] = RB[v];
    }
  }
#pragma unroll
  for (int i = 0; i < SUB; ++i) {
    if (starts >> i & 1u) load_state<VEC>(p.h0, p.ldh0, first[warp * SUB + i], f, p.D, h);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float next = fmaf(a[i][v], h[v], b[i][v]);
      b[i][v] = h[v];
      h[v] = next;
    }
  }
  float r[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) r[v] = 0.0f;
  if (lb.chunks > 1 && !state_in<VEC>(lb, tile, k, f, p.D, RA, RB, fold, state, &s_bad, r)) return;
#pragma unroll
  for (int v = 0; v < VEC; ++v) r[v] = apply_map(PA[v], PB[v], r[v]);
#pragma unroll
  for (int i = SUB - 1; i >= 0; --i) {
    if (ends >> i & 1u) load_state<VEC>(p.dhT, p.lddhT, last[warp * SUB + i], f, p.D, r);
    if (on && t0 + i < p.n) {
      Pack<T, VEC> og, ox;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float gl = to_float(rg[i].x[v]), x = to_float(rx[i].x[v]);
        const Gate g = gate_of<GATE>(gl), sl = gate_slope<GATE>(gl);
        const float q = __fadd_rn(to_float(rd[i].x[v]), r[v]);
        ox.x[v] = from_float<T>(__fmul_rn(g.c, q));
        og.x[v] = from_float<T>(__fmul_rn(q, fmaf(b[i][v], sl.a, __fmul_rn(x, sl.c))));
        r[v] = __fmul_rn(a[i][v], q);
      }
      if (p.dX) *reinterpret_cast<Pack<T, VEC>*>(p.dX + (size_t)(t0 + i) * p.lddx + f) = ox;
      if (p.dG) *reinterpret_cast<Pack<T, VEC>*>(p.dG + (size_t)(t0 + i) * p.lddg + f) = og;
    }
    if (starts >> i & 1u) store_state<VEC>(p.dh0, p.lddh0, first[warp * SUB + i], f, p.D, r);
  }
}

// No columns: every series is empty.
__global__ void __launch_bounds__(NT) k_scan_states(const float* from, int ldf, float* to, int ldt, int D) {
  for (int d = blockIdx.x * NT + threadIdx.x; d < D; d += gridDim.x * NT)
    to[(size_t)blockIdx.y * ldt + d] = from ? from[(size_t)blockIdx.y * ldf + d] : 0.0f;
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

// Scratch of one scan over `chunks` chunks of `tiles` feature tiles, freed in stream order.
struct Scratch {
  Lookback lb = {};
  void* mem = nullptr;
  cudaStream_t stream = nullptr;
  ~Scratch() { scratch_free(mem, stream); }
  cr_status make(int T, int chunk, int tiles, int D, cudaStream_t s) {
    CR_TRY(wait_word(&lb.err));
    lb.limit = option_wait_ns();
    lb.chunks = (int)(((long long)T + chunk - 1) / chunk);
    lb.tiles = tiles;
    // Groups: few hand-overs along the series against few maps to compose per chunk.
    lb.group = lb.chunks <= 256 ? 16 : lb.chunks <= 1024 ? 32 : MAXGROUP;
    if (lb.chunks <= 1) return CR_OK;
    const size_t groups = ((size_t)lb.chunks + lb.group - 1) / lb.group;
    const size_t flags = (1 + (size_t)tiles * (lb.chunks + groups)) * sizeof(int), up = (flags + 255) / 256 * 256;
    const size_t maps = (size_t)lb.chunks * D * sizeof(float2);
    stream = s;
    CR_CUDA(scratch_alloc(&mem, up + maps + groups * D * sizeof(float), s));
    lb.flags = (int*)mem;
    lb.maps = (float2*)((char*)mem + up);
    lb.states = (float*)((char*)mem + up + maps);
    CR_CUDA(cudaMemsetAsync(mem, 0, flags, s));
    return CR_OK;
  }
};

// Two features per thread where every matrix allows accesses of two elements.
struct Pairs {
  size_t bytes;
  bool ok;
  Pairs(int D, size_t eb) : bytes(2 * eb), ok(D % 2 == 0) {}
  Pairs& with(const void* p, int ld) {
    if (p && ((uintptr_t)p % bytes || ld % 2)) ok = false;
    return *this;
  }
};

cr_status states_only(const float* from, int ldf, float* to, int ldt, int D, int n, cudaStream_t stream) {
  if (!to || n == 0) return CR_OK;
  k_scan_states<<<dim3((D + NT - 1) / NT, n), NT, 0, stream>>>(from, ldf, to, ldt, D);
  CR_CHECK_LAUNCH("k_scan_states");
  return CR_OK;
}

template <class E, int GATE>
cr_status forward(const FwdArgs<E>& p, cudaStream_t stream) {
  const bool two = Pairs(p.D, sizeof(E)).with(p.G, p.ldg).with(p.X, p.ldx).with(p.H, p.ldh).ok;
  const int w = two ? 64 : 32, tiles = (p.D + w - 1) / w;
  Scratch sc;
  CR_TRY(sc.make(p.n, WARPS * FSUB, tiles, p.D, stream));
  const long long blocks = (long long)sc.lb.chunks * tiles;
  CR_REQUIRE(blocks < INT_MAX, "cr_gated_scan: more than 2^31 blocks");
  TimedScope ts("k_scan_fwd", stream);
  if (two) k_scan_fwd<E, GATE, 2><<<(unsigned)blocks, NT, 0, stream>>>(p, sc.lb);
  else k_scan_fwd<E, GATE, 1><<<(unsigned)blocks, NT, 0, stream>>>(p, sc.lb);
  CR_CHECK_LAUNCH("k_scan_fwd");
  return CR_OK;
}

template <class E, int GATE>
cr_status backward(const BwdArgs<E>& p, cudaStream_t stream) {
  const bool two = Pairs(p.D, sizeof(E)).with(p.G, p.ldg).with(p.X, p.ldx).with(p.dH, p.lddh).with(p.dG, p.lddg).with(p.dX, p.lddx).ok;
  const int w = two ? 64 : 32, tiles = (p.D + w - 1) / w;
  Scratch sc;
  CR_TRY(sc.make(p.n, BLOCK, tiles, p.D, stream));
  const long long blocks = (long long)sc.lb.chunks * tiles;
  CR_REQUIRE(blocks < INT_MAX, "cr_gated_scan_backward: more than 2^31 blocks");
  TimedScope ts("k_scan_bwd", stream);
  if (two) k_scan_bwd<E, GATE, 2><<<(unsigned)blocks, NT, 0, stream>>>(p, sc.lb);
  else k_scan_bwd<E, GATE, 1><<<(unsigned)blocks, NT, 0, stream>>>(p, sc.lb);
  CR_CHECK_LAUNCH("k_scan_bwd");
  return CR_OK;
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
  if (T == 0) return states_only(d_h0, ldh0, d_hT, ldhT, D, n_seq, stream);
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    return with_gate(gate, [&](auto g0) -> cr_status {
      return forward<E, decltype(g0)::value>(
          FwdArgs<E>{(const E*)d_G, (const E*)d_X, ldg, ldx, D, T, d_off, n_seq, d_h0, ldh0, (E*)d_H, ldh, d_hT, ldhT, d_saved}, stream);
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
  if (T == 0) return states_only(d_dhT, lddhT, d_dh0, lddh0, D, n_seq, stream);
  float* own = nullptr;
  if (!d_saved) {
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
      return backward<E, decltype(g0)::value>(
          BwdArgs<E>{(const E*)d_G, (const E*)d_X, (const E*)d_dH, ldg, ldx, lddh, D, T, d_off, n_seq, d_h0, d_dhT, d_saved, ldh0, lddhT,
                     (E*)d_dG, (E*)d_dX, lddg, lddx, d_dh0, lddh0}, stream);
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
