// Gated recurrence along time over packed series, its gradient and its single step
// (cr_gated_scan, cr_gated_scan_backward, cr_gated_step).
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "ops.cuh"
#include "ptx.cuh"

namespace cr {
namespace {

// How the scan is split.  A work item is a chunk of consecutive steps by a tile of W features (128
// bytes of each column).  Resident blocks take items in order of time from a counter: whatever an
// item waits for was taken earlier and is being worked on.  Warp 8 of a block takes the items and
// loads them by TMA into stages while the other 8 warps work; each of these owns SUB of the
// chunk's steps and each of its lanes VEC features.  They go over the tile in shared memory twice,
// for its map and, once the state before it is known, for the outputs, so that HBM is read once
// and few registers are held meanwhile: several blocks fit on an SM, which covers the time that
// a block waits for its predecessors.
// The map of a run of steps on the state is h -> A h + B, and such maps compose; a run in which a
// series starts has a mark of its own in place of A, so that nothing crosses into the next series and
// everything else, NaN and infinities too, goes on.  Warps join their maps in
// shared memory, chunks through global memory in two levels: a chunk composes the maps of the
// earlier chunks of its group, and takes the state before the group from the group's
// predecessor.  Every composition has a fixed order, so results do not depend on timing.
constexpr int WARPS = 8, NT = 32 * (WARPS + 1);
constexpr int FSUB = 16, BSUB = 8;        // steps per warp, forward and backward
constexpr int BLOCK = BSUB;               // steps between saved states: a warp's part of a backward chunk
// Stages per block and blocks per SM.  More blocks hide the waits for predecessors, more stages the
// loads; forward 2048 x 65536 BF16: 1 and 5 186 us, 1 and 4 192 us, 2 and 3 195 us, 3 and 2 245 us;
// backward 1536 x 50021 FP16, variance gate: 1 and 4 225 us, 2 and 3 210 us.
constexpr int FSTAGES = 1, FBLOCKS = 5, BSTAGES = 2, BBLOCKS = 3;
constexpr int MAXGROUP = 64;
constexpr int ROW = 128;                  // bytes of a column in a tile
template <class T>
constexpr int vec_of() { return 4 / (int)sizeof(T); }

// What chunks tell each other, cleared before the call.  Every entry is one 64-bit word, written
// and read whole, that is 0 until it is there, so that no fence stands between data and flag: a
// map is A in the low half, with +0 written as -0, and B in the high one; a state has 1 in the low half.
typedef unsigned long long Word;
struct Lookback {
  int chunks, tiles, group, width;   // width: features rounded up to whole tiles
  int* counter;
  Word* maps;      // [chunk][feature]
  Word* states;    // [group][feature]: the state that the group hands on
  unsigned long long limit;
  int* err;
};

__device__ __forceinline__ void post(Word* p, Word w) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}
__device__ __forceinline__ Word peek(const Word* p) {
  Word w;
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(w) : "l"(p) : "memory");
  return w;
}
// A of a map: 0, a series starts in the run and the state before it does not count; ZERO, one of the run's
// coefficients is 0; +-TINY, their product underflowed; else the product, which may be infinite.  ZERO and TINY leave
// nothing of a finite state, but infinities and NaN go on.  With sigmoids for coefficients there is no ZERO and
// nothing grows, so that maps are multiply-adds throughout.  With coefficients of any size a state that is not
// finite, and a map that makes it so, go by the rules of through_exactly: an infinite A leaves a state of exactly
// zero alone, since the product may only have overflowed (a coefficient that is infinite or NaN is in B already).
// Watching for that costs the coefficient gate 5 % (2048 x 65536 BF16: 175 us, without 166).
constexpr float ZERO = 0x1p-149f, TINY = 0x1p-148f;
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }
__device__ __forceinline__ float through_exactly(float2 m, float h) {   // the state after map m
  const float a = fabsf(m.x);
  if (a == 0.0f || h == 0.0f || (a <= TINY && is_finite(h))) return m.y;
  return fmaf(a == ZERO ? 0.0f : m.x, h, m.y);
}
__device__ __forceinline__ float2 then_exactly(float2 m, float2 n) {   // n after m
  const float B = through_exactly(n, m.y), p = m.x * n.x, low = fminf(fabsf(m.x), fabsf(n.x));
  if (low == 0.0f) return make_float2(0.0f, B);
  if (low == ZERO) return make_float2(is_finite(p) ? ZERO : p * 0.0f, B);
  return make_float2(fabsf(p) <= TINY || (low == TINY && is_finite(p)) ? copysignf(TINY, p) : p, B);
}
// n maps in a row, `step` apart, of shared memory or of the words of chunks; and a state through n maps, with the
// states before them left in before[k * step].x (NULL: not wanted).  Calls, to cost the usual path no registers.
__device__ __noinline__ float2 joined_exactly(const float2* maps, int step, int n) {
  float2 m = make_float2(1.0f, 0.0f);
  for (int k = 0; k < n; ++k) m = then_exactly(m, maps[k * step]);
  return m;
}
__device__ __noinline__ float2 joined_exactly(const Word* maps, size_t step, int n) {
  float2 m = make_float2(1.0f, 0.0f);
  for (int k = 0; k < n; ++k) {
    const Word w = peek(maps + k * step);
    m = then_exactly(m, make_float2(__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))));
  }
  return m;
}
__device__ __noinline__ float carried_exactly(const float2* maps, int step, int n, float h, float2* before) {
  for (int k = 0; k < n; ++k) {
    if (before) before[k * step].x = h;
    h = through_exactly(maps[k * step], h);
  }
  return h;
}
// Maps in a row as multiply-adds; exact(): no rule of then_exactly says anything else.
template <int GATE>
struct Joined {
  static constexpr bool ANY = GATE == CR_GATE_COEFF;
  float A = 1.0f, B = 0.0f, low = 1.0f, odd = 0.0f;
  __device__ __forceinline__ void add(float a, float b) {
    B = fabsf(a) <= (ANY ? TINY : 0.0f) ? b : fmaf(a, B, b);
    A *= a;
    low = fminf(low, fabsf(a));
    if (ANY) odd = fmaf(B, 0.0f, odd);   // NaN from the first B on that is not finite
  }
  __device__ __forceinline__ bool exact() const { return !ANY || odd == 0.0f; }
  __device__ __forceinline__ float2 map() const {
    if (ANY) return make_float2(low <= TINY ? copysignf(low, A) : fabsf(A) <= TINY ? copysignf(TINY, A) : A, B);
    return make_float2(low == 0.0f ? 0.0f : fmaxf(A, TINY), B);
  }
};
// A state through maps as multiply-adds; exact(): it was finite before and after each.
template <int GATE>
struct Carried {
  static constexpr bool ANY = GATE == CR_GATE_COEFF;
  float h, odd;
  __device__ __forceinline__ Carried(float h0) : h(h0), odd(ANY ? h0 * 0.0f : 0.0f) {}
  __device__ __forceinline__ void go(float2 m) {
    h = fabsf(m.x) <= (ANY ? TINY : 0.0f) ? m.y : fmaf(m.x, h, m.y);
    if (ANY) odd = fmaf(h, 0.0f, odd);
  }
  __device__ __forceinline__ bool exact() const { return !ANY || odd == 0.0f; }
};
// A of a run of steps from the product of its coefficients, zero(v) saying whether one of them is 0.
template <int GATE, int VEC, class Zero>
__device__ __forceinline__ void mark_product(Floats<VEC>& A, bool start, Zero&& zero) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    if (start) A.x[v] = 0.0f;
    else if (GATE != CR_GATE_COEFF) A.x[v] = fmaxf(A.x[v], TINY);   // (NaN is in B too)
    else if (!(fabsf(A.x[v]) > TINY)) A.x[v] = zero(v) ? ZERO : A.x[v] == A.x[v] ? copysignf(TINY, A.x[v]) : A.x[v];
  }
}

__device__ __forceinline__ Word map_word(float2 m) {
  return (Word)__float_as_uint(m.y) << 32 | __float_as_uint(m.x == 0.0f ? -0.0f : m.x);
}
// Reads N words, `stride` apart, of which the first n are waited for (the others stay 0); false when
// the limit runs out.
template <int N>
__device__ __forceinline__ bool await(const Word* p, size_t stride, int n, const Lookback& lb, Word (&w)[N]) {
#pragma unroll
  for (int q = 0; q < N; ++q) w[q] = 0;
  unsigned long long t0 = 0;
  while (true) {
    bool there = true;
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (q < n && w[q] == 0) w[q] = peek(p + q * stride);
#pragma unroll
    for (int q = 0; q < N; ++q) there = there && (q >= n || w[q] != 0);
    if (there) return true;
    const unsigned long long t = global_timer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > lb.limit) {
      *(volatile int*)lb.err = 1;
      __threadfence_system();
      return false;
    }
  }
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

// By one warp: series that start or end in the chunk [t0, t0 + len): first[t - t0], last[t - t0] = the
// series or -1.  empty(s) is called for the empty series that belong to the chunk.
template <class F>
__device__ __forceinline__ void mark_series(const int32_t* off, int n, int t0, int len, int T, int* first, int* last, F&& empty) {
  const int lane = threadIdx.x & 31;
  for (int q = lane; q < len; q += 32) {
    first[q] = !off && t0 + q == 0 ? 0 : -1;
    last[q] = !off && t0 + q == T - 1 ? 0 : -1;
  }
  if (!off) return;
  const int lo = first_at_least(off, n, t0);
  const bool final = t0 + len >= T;   // empty series at T belong to the last chunk
  __syncwarp();
  for (int base = max(lo - 1, 0); base < n; base += 32) {
    const int s = base + lane;
    const int b = s < n ? off[s] : INT_MAX, e = s < n ? off[s + 1] : INT_MAX;
    const bool in = s < n && (b < t0 + len || final);
    if (in && e > b) {
      if (b >= t0 && b < t0 + len) first[b - t0] = s;
      if (e - 1 >= t0 && e - 1 < t0 + len) last[e - 1 - t0] = s;
    }
    uint32_t none = __ballot_sync(0xffffffffu, in && s >= lo && e <= b);
    for (; none; none &= none - 1) empty(base + __ffs(none) - 1);
    if (!__all_sync(0xffffffffu, in)) break;
  }
  __syncwarp();
}

// The features' h0 (or its gradient's seed) of series s.
template <int VEC>
__device__ __forceinline__ void load_state(const float* h0, int ld, int s, int f, int D, Floats<VEC>& h) {
#pragma unroll
  for (int v = 0; v < VEC; ++v) h.x[v] = h0 && f + v < D ? h0[(size_t)s * ld + f + v] : 0.0f;
}
template <int VEC>
__device__ __forceinline__ void store_state(float* hT, int ld, int s, int f, int D, const Floats<VEC>& h) {
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    if (hT && f + v < D) hT[(size_t)s * ld + f + v] = h.x[v];
}

__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Shared memory of a block: ring of stages of NIN input tiles, then this.
template <int CH, int W, int STAGES>
struct Shared {
  uint64_t full[STAGES], empty[STAGES];
  int place[STAGES];
  int first[STAGES][CH], last[STAGES][CH];
  float2 maps[WARPS][W], fold[WARPS][W];   // fold[.].x: then the states that enter the warps
  float2 total[W];                         // the chunk's map, kept by a group's last chunk
  int bad;
};

struct Input {
  const void* p;
  int ld;
};

// Warp 8: takes work items and fills stages.  item(place, tile, t0) gives an item's tile and first
// step, empty(tile, s) handles an empty series.
template <class T, int CH, int NIN, int W, int STAGES, class Item, class Empty>
__device__ __forceinline__ void feed(const Lookback& lb, Shared<CH, W, STAGES>* sh, uint8_t* ring, const CUtensorMap* const (&tm)[NIN], bool tma,
                                     const int32_t* off, int series, int n, Item&& item, Empty&& empty) {
  const int lane = threadIdx.x & 31, total = lb.chunks * lb.tiles;
  int it = 0;
  bool done = false;
  for (;; ++it) {
    const int st = it % STAGES;
    const bool go = mbar_wait(&sh->empty[st], ((uint32_t)(it / STAGES) & 1u) ^ 1u, lb.limit) && !*(volatile int*)&sh->bad;
    if (!__all_sync(0xffffffffu, go)) break;   // the lanes' clocks and reads differ: they leave together
    int place = 0;   // taken late: an item held back here holds up the blocks that wait for its map
    if (lane == 0) place = lb.chunks > 1 ? atomicAdd(lb.counter, 1) : (int)blockIdx.x + it * (int)gridDim.x;
    place = __shfl_sync(0xffffffffu, place, 0);
    if (place >= total) {
      if (lane == 0) {
        sh->place[st] = -1;
        mbar_arrive(&sh->full[st]);
      }
      done = true;
      break;
    }
    int tile, t0;
    item(place, tile, t0);
    if (lane == 0) {
      sh->place[st] = place;
      if (tma) {
        mbar_expect_tx(&sh->full[st], NIN * CH * ROW);
#pragma unroll
        for (int q = 0; q < NIN; ++q) tma_load_2d(ring + (st * NIN + q) * CH * ROW, tm[q], &sh->full[st], tile * W, t0);
      }
    }
    mark_series(off, series, t0, CH, n, sh->first[st], sh->last[st], [&](int s) { empty(tile, s); });
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->full[st]);
  }
  // Copies in flight land before the block leaves, whatever became of the workers.  (When all items are taken, the one
  // before in the last stage is done with, and its barrier has gone on.)
  __syncwarp();
  if (lane == 0) {
    if (!done) {
      *(volatile int*)lb.err = 1;
      __threadfence_system();
    }
    for (int q = 1; tma && q <= STAGES - (done ? 1 : 0) && q <= it; ++q)
      mbar_wait(&sh->full[(it - q) % STAGES], (uint32_t)((it - q) / STAGES) & 1u, LANDING_NS);
  }
}

// Without TMA (a matrix whose columns are not on 16-byte boundaries): each warp copies its own rows, eight
// rows' loads in flight at once (2047 x 32768 BF16 forward: 186 us, one after the other 384 us, by TMA 2048 108 us).
// A call: inlined, its registers cost the TMA path 1 %.
template <class T, int W, int ROWS>
__device__ __noinline__ void copy_rows(Input in, uint8_t* tile, int row0, int f0, int t0, int D, int n) {
  constexpr int BATCH = 8, PER = W / 32;
  const int lane = threadIdx.x & 31;
  T* to = reinterpret_cast<T*>(tile) + row0 * W + lane;
  const T* from = (const T*)in.p + (size_t)t0 * in.ld + f0 + lane;
#pragma unroll
  for (int r0 = 0; r0 < ROWS; r0 += BATCH) {
    T v[BATCH][PER];
#pragma unroll
    for (int r = 0; r < BATCH; ++r)
#pragma unroll
      for (int x = 0; x < PER; ++x)
        v[r][x] = f0 + lane + 32 * x < D && t0 + r0 + r < n ? from[(size_t)(r0 + r) * in.ld + 32 * x] : from_float<T>(0.0f);
#pragma unroll
    for (int r = 0; r < BATCH; ++r)
#pragma unroll
      for (int x = 0; x < PER; ++x) to[(r0 + r) * W + 32 * x] = v[r][x];
  }
}

// The item in the stage of round `it`; -1 when there is none or the wait for it ran out.  sh->bad is
// written before a barrier of the workers and read before the next, so that they agree.
template <int STAGES, class S>
__device__ __forceinline__ int next_item(const Lookback& lb, S* sh, int it) {
  if (!mbar_wait(&sh->full[it % STAGES], (uint32_t)(it / STAGES) & 1u, lb.limit)) {
    *(volatile int*)&sh->bad = 1;
    *(volatile int*)lb.err = 1;
    __threadfence_system();
  }
  workers_sync();
  return *(volatile int*)&sh->bad ? -1 : sh->place[it % STAGES];
}

// Joins the workers' maps (A, B) of a chunk (position k in the order of work): the state that enters the
// part of each warp, in sh->fold[warp][feature].x.  Warps compose in the order 0 .. 7, or 7 .. 0 with REVERSE.  All
// workers call it; meanwhile() runs between posting the chunk's map and waiting for others; false when a
// wait ran out.
template <int GATE, bool REVERSE, int VEC, int W, class S, class Meanwhile>
__device__ __forceinline__ bool join(const Lookback& lb, S* sh, int tile, int k, const Floats<VEC>& A, const Floats<VEC>& B,
                                     Meanwhile&& meanwhile) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int v = 0; v < VEC; ++v) sh->maps[warp][lane * VEC + v] = make_float2(A.x[v], B.x[v]);
  workers_sync();
  const int g = k / lb.group, in = k % lb.group, c0 = g * lb.group;
  const bool more = k + 1 < lb.chunks, lastin = in == lb.group - 1;
  // one thread per feature: the chunk's map
  const int x = threadIdx.x, fx = tile * W + x;
  constexpr int STEP = REVERSE ? -W : W;   // from one warp's maps to the next's
  const int w0 = REVERSE ? WARPS - 1 : 0;
  if (x < W) {
    Joined<GATE> all;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 m = sh->maps[REVERSE ? WARPS - 1 - w : w][x];
      all.add(m.x, m.y);
    }
    const float2 total = all.exact() ? all.map() : joined_exactly(&sh->maps[w0][x], STEP, WARPS);
    if (lastin) sh->total[x] = total;
    else if (more) post(lb.maps + (size_t)k * lb.width + fx, map_word(total));
  }
  meanwhile();
  bool fine = true;
  float h = 0.0f;
  if (lb.chunks > 1) {
    // the earlier chunks of the group, a fixed part of them per warp
    const int per = lb.group / WARPS, q0 = warp * per, n = min(in - q0, per);
    bool ok = true;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      Joined<GATE> all;
      for (int q = 0; q < n; q += 4) {
        Word w[4];
        ok = await(lb.maps + (size_t)(c0 + q0 + q) * lb.width + tile * W + 32 * v + lane, lb.width, n - q, lb, w) && ok;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (q + y < n) all.add(__uint_as_float((uint32_t)w[y]), __uint_as_float((uint32_t)(w[y] >> 32)));
      }
      sh->fold[warp][32 * v + lane] = all.exact() ? all.map() : joined_exactly(lb.maps + (size_t)(c0 + q0) * lb.width + tile * W + 32 * v + lane, lb.width, n);
    }
    if (x < W && g > 0) {
      Word w[1];
      ok = await(lb.states + (size_t)(g - 1) * lb.width + fx, 0, 1, lb, w) && ok;
      h = __uint_as_float((uint32_t)(w[0] >> 32));
    }
    if (!ok) *(volatile int*)&sh->bad = 1;
    workers_sync();
    fine = *(volatile int*)&sh->bad == 0;
  }
  if (x < W) {
    if (lb.chunks > 1) {
      Carried<GATE> state(h);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) state.go(sh->fold[w][x]);
      h = state.exact() ? state.h : carried_exactly(&sh->fold[0][x], W, WARPS, h, nullptr);
      if (lastin && more) {
        Carried<GATE> next(h);
        next.go(sh->total[x]);
        if (!next.exact()) next.h = through_exactly(sh->total[x], h);
        post(lb.states + (size_t)g * lb.width + fx, (Word)__float_as_uint(next.h) << 32 | 1u);
      }
    }
    Carried<GATE> state(h);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const int u = REVERSE ? WARPS - 1 - w : w;
      sh->fold[u][x].x = state.h;
      if (w + 1 < WARPS) state.go(sh->maps[u][x]);
    }
    if (!state.exact()) carried_exactly(&sh->maps[w0][x], STEP, WARPS, h, &sh->fold[w0][x]);
  }
  workers_sync();
  return fine;
}

template <class T>
struct FwdArgs {
  Input G, X;
  int D, n;   // n columns
  const int32_t* off;
  int series;
  const float* h0;
  int ldh0;
  T* H;
  int ldh;
  float* hT;
  int ldhT;
  float* saved;
  int tma, pairs;   // inputs by TMA; H takes accesses of VEC elements
};

// VEC consecutive elements in FP32.
template <class T, int VEC>
__device__ __forceinline__ Floats<VEC> widened(const uint8_t* at);
template <>
__device__ __forceinline__ Floats<1> widened<float, 1>(const uint8_t* at) { return {{*reinterpret_cast<const float*>(at)}}; }
template <>
__device__ __forceinline__ Floats<2> widened<__half, 2>(const uint8_t* at) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(at));
  return {{f.x, f.y}};
}
template <>
__device__ __forceinline__ Floats<2> widened<__nv_bfloat16, 2>(const uint8_t* at) {   // BF16 is the upper half of FP32
  const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
  return {{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}};
}
__device__ __forceinline__ void put_all(float* o, const Floats<1>& v) { *o = v.x[0]; }
__device__ __forceinline__ void put_all(__half* o, const Floats<2>& v) {
  *reinterpret_cast<__half2*>(o) = __floats2half2_rn(v.x[0], v.x[1]);
}
__device__ __forceinline__ void put_all(__nv_bfloat16* o, const Floats<2>& v) {
  *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(v.x[0], v.x[1]);
}

template <class T, int VEC>
__device__ __forceinline__ void put(T* out, int ld, int t, int f, int D, bool vec, const Floats<VEC>& v) {
  T* o = out + (size_t)t * ld + f;
  if (vec) {
    put_all(o, v);
  } else {
#pragma unroll
    for (int q = 0; q < VEC; ++q)
      if (f + q < D) o[q] = from_float<T>(v.x[q]);
  }
}

// Forward scan.  HBM (G and X read, H written) would take 119 us for 2048 x 65536 BF16; it takes 175 us with
// coefficients, 196 with the convex gate, 222 with the variance gate: the gates' 2^x, reciprocal and square
// root, made twice, and the waits for the chunks before.  Kept in registers and shared memory between the two passes
// they cost more (204 us, convex): fewer blocks fit.  Steps past the end and features past D hold
// zeros: their states are never used.
template <class T, int GATE>
__global__ void __launch_bounds__(NT, FBLOCKS)
    k_scan_fwd(const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmX, const FwdArgs<T> p, const Lookback lb) {
  constexpr int CH = WARPS * FSUB, VEC = vec_of<T>(), W = 32 * VEC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~(uintptr_t)127);
  auto* sh = reinterpret_cast<Shared<CH, W, FSTAGES>*>(ring + FSTAGES * 2 * CH * ROW);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int q = 0; q < FSTAGES; ++q) {
      mbar_init(&sh->full[q], 1);
      mbar_init(&sh->empty[q], WARPS);
    }
    sh->bad = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == WARPS) {
    const CUtensorMap* const tm[2] = {&tmG, &tmX};
    feed<T, CH, 2, W>(
        lb, sh, ring, tm, p.tma, p.off, p.series, p.n,
        [&](int place, int& tile, int& t0) {
          tile = place % lb.tiles;
          t0 = place / lb.tiles * CH;
        },
        [&](int tile, int s) {
          Floats<VEC> h;
          load_state<VEC>(p.h0, p.ldh0, s, tile * W + lane * VEC, p.D, h);
          store_state<VEC>(p.hT, p.ldhT, s, tile * W + lane * VEC, p.D, h);
        });
    return;
  }
  for (int it = 0;; ++it) {
    const int st = it % FSTAGES;
    const int place = next_item<FSTAGES>(lb, sh, it);
    if (place < 0) break;
    const int k = place / lb.tiles, tile = place % lb.tiles, t0 = k * CH + warp * FSUB, f = tile * W + lane * VEC;
    uint8_t* in = ring + st * 2 * CH * ROW;
    if (!p.tma) {
      copy_rows<T, W, FSUB>(p.G, in, warp * FSUB, tile * W, t0, p.D, p.n);
      copy_rows<T, W, FSUB>(p.X, in + CH * ROW, warp * FSUB, tile * W, t0, p.D, p.n);
      __syncwarp();
    }
    const int* first = sh->first[st] + warp * FSUB;
    const int* last = sh->last[st] + warp * FSUB;
    const uint32_t starts = __ballot_sync(0xffffffffu, lane < FSUB && first[lane & (FSUB - 1)] >= 0);
    const uint32_t ends = __ballot_sync(0xffffffffu, lane < FSUB && last[lane & (FSUB - 1)] >= 0);
    const uint8_t* row = in + warp * FSUB * ROW + lane * 4;

    const auto step = [&](int i, Floats<VEC>& a, Floats<VEC>& b) {   // h -> a h + b
      const auto c = gate_parts<GATE>(widened<T, VEC>(row + i * ROW));
      a = c.a;
      b = mul(gate_input<GATE>(c), widened<T, VEC>(row + CH * ROW + i * ROW));
    };
    Floats<VEC> A = all_of<VEC>(1.0f), B = all_of<VEC>(0.0f), a, b;
    if (!starts) {   // without branches, so that steps overlap
#pragma unroll 4
      for (int i = 0; i < FSUB; ++i) {
        step(i, a, b);
        A = mul(A, a);
        B = fma(a, B, b);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < FSUB; ++i) {
        if (starts >> i & 1u) load_state<VEC>(p.h0, p.ldh0, first[i], f, p.D, B);
        step(i, a, b);
        B = fma(a, B, b);
      }
    }
    mark_product<GATE>(A, starts != 0, [&](int v) {
      bool zero = false;
      for (int i = 0; i < FSUB; ++i) zero = zero || widened<T, VEC>(row + i * ROW).x[v] == 0.0f;
      return zero;
    });
    if (!join<GATE, false, VEC, W>(lb, sh, tile, k, A, B, [] {})) return;
    Floats<VEC> h;
#pragma unroll
    for (int v = 0; v < VEC; ++v) h.x[v] = sh->fold[warp][lane * VEC + v].x;
    if (!(starts | ends) && p.H && p.pairs && p.n - t0 >= FSUB) {   // inside a series
      if (f < p.D) {
        T* o = p.H + (size_t)t0 * p.ldh + f;
#pragma unroll 4
        for (int i = 0; i < FSUB; ++i, o += p.ldh) {
          if (i % BLOCK == 0) store_state<VEC>(p.saved, p.D, (t0 + i) / BLOCK, f, p.D, h);
          step(i, a, b);
          h = fma(a, h, b);
          put_all(o, h);
        }
      }
    } else {
      const int steps = f < p.D ? p.n - t0 : 0;
#pragma unroll 1
      for (int i = 0; i < FSUB; ++i) {
        if (i % BLOCK == 0 && i < steps) store_state<VEC>(p.saved, p.D, (t0 + i) / BLOCK, f, p.D, h);
        if (starts >> i & 1u) load_state<VEC>(p.h0, p.ldh0, first[i], f, p.D, h);
        step(i, a, b);
        h = fma(a, h, b);
        if (p.H && i < steps) put<T, VEC>(p.H, p.ldh, t0 + i, f, p.D, p.pairs, h);
        if (ends >> i & 1u) store_state<VEC>(p.hT, p.ldhT, last[i], f, p.D, h);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->empty[st]);
  }
}

template <class T>
struct BwdArgs {
  Input G, X, dH;
  int D, n;
  const int32_t* off;
  int series;
  const float *h0, *dhT, *saved;
  int ldh0, lddhT;
  T *dG, *dX;
  int lddg, lddx;
  float* dh0;
  int lddh0;
  int tma, pairs;
};

// Backward scan, from the last chunk to the first: r_t = a_t q_t, q_t = dh_t + r_{t+1}, with "take dhT" at
// a series' last step.  Each warp recomputes the states of its steps from the one saved before
// them, which reads G and X (needed anyway) in place of H: 0.5 bytes per element (one state in
// 8 steps) against H's 2 or 4 and its rounding.  The states and the slopes dg / q need no later step: they are
// made between posting the chunk's map and waiting for the later chunks', and the slopes take the
// inputs' place in shared memory, so that after the wait a step is four multiply-adds (all of it after the
// wait: 289 us where this takes 210, 1536 x 50021 FP16, variance gate).  Bound by HBM (G, X, dH read, dG,
// dX written) and, beyond it, by the wait for the chunks after it.
template <class T, int GATE>
__global__ void __launch_bounds__(NT, BBLOCKS)
    k_scan_bwd(const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmD,
               const BwdArgs<T> p, const Lookback lb) {
  constexpr int CH = WARPS * BSUB, SUB = BSUB, VEC = vec_of<T>(), W = 32 * VEC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~(uintptr_t)127);
  auto* sh = reinterpret_cast<Shared<CH, W, BSTAGES>*>(ring + BSTAGES * 3 * CH * ROW);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int q = 0; q < BSTAGES; ++q) {
      mbar_init(&sh->full[q], 1);
      mbar_init(&sh->empty[q], WARPS);
    }
    sh->bad = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == WARPS) {
    const CUtensorMap* const tm[3] = {&tmG, &tmX, &tmD};
    feed<T, CH, 3, W>(
        lb, sh, ring, tm, p.tma, p.off, p.series, p.n,
        [&](int place, int& tile, int& t0) {
          tile = place % lb.tiles;
          t0 = (lb.chunks - 1 - place / lb.tiles) * CH;
        },
        [&](int tile, int s) {
          Floats<VEC> q;
          load_state<VEC>(p.dhT, p.lddhT, s, tile * W + lane * VEC, p.D, q);
          store_state<VEC>(p.dh0, p.lddh0, s, tile * W + lane * VEC, p.D, q);
        });
    return;
  }
  for (int it = 0;; ++it) {
    const int st = it % BSTAGES;
    const int place = next_item<BSTAGES>(lb, sh, it);
    if (place < 0) break;
    const int k = place / lb.tiles, tile = place % lb.tiles, chunk = lb.chunks - 1 - k;
    const int t0 = chunk * CH + warp * SUB, f = tile * W + lane * VEC;
    uint8_t* in = ring + st * 3 * CH * ROW;
    Floats<VEC> h;
    load_state<VEC>(p.saved, p.D, t0 / BLOCK, f, t0 < p.n ? p.D : 0, h);
    if (!p.tma) {
      copy_rows<T, W, SUB>(p.G, in, warp * SUB, tile * W, t0, p.D, p.n);
      copy_rows<T, W, SUB>(p.X, in + CH * ROW, warp * SUB, tile * W, t0, p.D, p.n);
      copy_rows<T, W, SUB>(p.dH, in + 2 * CH * ROW, warp * SUB, tile * W, t0, p.D, p.n);
      __syncwarp();
    }
    const int* first = sh->first[st] + warp * SUB;
    const int* last = sh->last[st] + warp * SUB;
    const uint32_t starts = __ballot_sync(0xffffffffu, lane < SUB && first[lane & (SUB - 1)] >= 0);
    const uint32_t ends = __ballot_sync(0xffffffffu, lane < SUB && last[lane & (SUB - 1)] >= 0);
    uint8_t* row = in + warp * SUB * ROW + lane * 4;

    Floats<VEC> RA = all_of<VEC>(1.0f), RB = all_of<VEC>(0.0f), a[SUB], c[SUB];
    const auto gates = [&](int i) {
      const auto parts = gate_parts<GATE>(widened<T, VEC>(row + i * ROW));
      a[i] = parts.a;
      c[i] = parts.rest;
      RB = mul(a[i], add(widened<T, VEC>(row + 2 * CH * ROW + i * ROW), RB));
      RA = mul(RA, a[i]);
    };
    const auto states = [&](int i) {
      c[i] = gate_input<GATE>(GateParts<VEC>{a[i], c[i]});
      const Floats<VEC> x = widened<T, VEC>(row + CH * ROW + i * ROW), slope = gate_slope<GATE>(a[i], c[i], h, x);
      h = fma(a[i], h, mul(c[i], x));
#pragma unroll
      for (int v = 0; v < VEC; ++v) *reinterpret_cast<float*>(row + v * CH * ROW + i * ROW) = slope.x[v];
    };
    if (!ends) {   // without branches, so that steps overlap
#pragma unroll
      for (int i = SUB - 1; i >= 0; --i) gates(i);
    } else {
#pragma unroll
      for (int i = SUB - 1; i >= 0; --i) {
        if (ends >> i & 1u) load_state<VEC>(p.dhT, p.lddhT, last[i], f, p.D, RB);
        gates(i);
      }
    }
    mark_product<GATE>(RA, ends != 0, [&](int v) {
      bool zero = false;
#pragma unroll
      for (int i = 0; i < SUB; ++i) zero = zero || a[i].x[v] == 0.0f;
      return zero;
    });
    const bool fine = join<GATE, true, VEC, W>(lb, sh, tile, k, RA, RB, [&] {
      if (!starts) {
#pragma unroll
        for (int i = 0; i < SUB; ++i) states(i);
      } else {
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
          if (starts >> i & 1u) load_state<VEC>(p.h0, p.ldh0, first[i], f, p.D, h);
          states(i);
        }
      }
    });
    if (!fine) return;
    Floats<VEC> q;
#pragma unroll
    for (int v = 0; v < VEC; ++v) q.x[v] = sh->fold[warp][lane * VEC + v].x;
    const auto step = [&](int i, Floats<VEC>& dx, Floats<VEC>& dg) {   // gradients of step i; q passes on
      q = add(widened<T, VEC>(row + 2 * CH * ROW + i * ROW), q);
      dx = mul(c[i], q);
#pragma unroll
      for (int v = 0; v < VEC; ++v) dg.x[v] = *reinterpret_cast<const float*>(row + v * CH * ROW + i * ROW);
      dg = mul(q, dg);
      q = mul(a[i], q);
    };
    Floats<VEC> dx, dg;
    if (!(starts | ends) && p.dX && p.dG && p.pairs && p.n - t0 >= SUB) {   // inside a series
      if (f < p.D) {
        T* ox = p.dX + (size_t)(t0 + SUB - 1) * p.lddx + f;
        T* og = p.dG + (size_t)(t0 + SUB - 1) * p.lddg + f;
#pragma unroll
        for (int i = SUB - 1; i >= 0; --i, ox -= p.lddx, og -= p.lddg) {
          step(i, dx, dg);
          put_all(ox, dx);
          put_all(og, dg);
        }
      }
    } else {
      const int steps = f < p.D ? p.n - t0 : 0;
#pragma unroll
      for (int i = SUB - 1; i >= 0; --i) {
        if (ends >> i & 1u) load_state<VEC>(p.dhT, p.lddhT, last[i], f, p.D, q);
        step(i, dx, dg);
        if (i < steps) {
          if (p.dX) put<T, VEC>(p.dX, p.lddx, t0 + i, f, p.D, p.pairs, dx);
          if (p.dG) put<T, VEC>(p.dG, p.lddg, t0 + i, f, p.D, p.pairs, dg);
        }
        if (starts >> i & 1u) store_state<VEC>(p.dh0, p.lddh0, first[i], f, p.D, q);
      }
    }
    fence_smem_to_tma();   // the slopes were written where the next copy goes
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->empty[st]);
  }
}

// No columns: every series is empty.
__global__ void __launch_bounds__(256) k_scan_states(const float* from, int ldf, float* to, int ldt, int D, int n) {
  for (int s = blockIdx.x; s < n; s += gridDim.x)
    for (int d = threadIdx.x; d < D; d += 256) to[(size_t)s * ldt + d] = from ? from[(size_t)s * ldf + d] : 0.0f;
}

// One step: V consecutive features of one series per thread (V = 4: aligned matrices).  Bound by HBM
// for many series (4096 x 8192 BF16 73 us, 6.4 TB/s), by the launch for few (4096 x 64: 5 us).
template <class T, int GATE, int V>
__global__ void __launch_bounds__(256) k_scan_step(const T* G, int ldg, const T* X, int ldx, const float* h, int ldh, int D, int B, T* H,
                                                   int ldo, float* hn, int ldn) {
  struct alignas(sizeof(T) * V) Elements {
    T x[V];
  };
  struct alignas(sizeof(float) * V) States {
    float x[V];
  };
  let_next_start();
  wait_for_previous();
  const int per = (D + V - 1) / V;
  for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < (long long)per * B; e += (long long)gridDim.x * 256) {
    const size_t b = (size_t)(e / per);
    const int d = (int)(e % per) * V;
    const Elements g = *reinterpret_cast<const Elements*>(G + b * ldg + d), x = *reinterpret_cast<const Elements*>(X + b * ldx + d);
    States s = *reinterpret_cast<const States*>(h + b * ldh + d);
    Elements o;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      const auto c = gate_parts<GATE>(Floats<1>{{to_float(g.x[q])}});
      s.x[q] = fmaf(c.a.x[0], s.x[q], __fmul_rn(gate_input<GATE>(c).x[0], to_float(x.x[q])));
      o.x[q] = from_float<T>(s.x[q]);
    }
    *reinterpret_cast<States*>(hn + b * ldn + d) = s;
    if (H) *reinterpret_cast<Elements*>(H + b * ldo + d) = o;
  }
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
  cr_status make(int T, int chunk, int tiles, int w, cudaStream_t s) {
    CR_TRY(wait_word(&lb.err));
    lb.limit = option_wait_ns();
    lb.chunks = (int)(((long long)T + chunk - 1) / chunk);
    lb.tiles = tiles;
    lb.width = tiles * w;
    // Groups: few hand-overs along the series against few maps to compose per chunk.  Groups of 16, 32 and 64, BF16, convex
    // gate, backward: 64 chunks of 2048 features (4096 steps) 32.7, 32.1 and 34.5 us; 1024 chunks 332, 317 and 357; 4096
    // chunks of 64 features 159, 91 and 81.
    lb.group = lb.chunks <= 256 ? 16 : lb.chunks <= 1024 ? 32 : MAXGROUP;
    if (lb.chunks <= 1) return CR_OK;
    const size_t groups = ((size_t)lb.chunks + lb.group - 1) / lb.group;
    const size_t maps = (size_t)lb.chunks * lb.width, bytes = 256 + (maps + groups * lb.width) * sizeof(Word);
    stream = s;
    CR_CUDA(scratch_alloc(&mem, bytes, s));
    lb.counter = (int*)mem;
    lb.maps = (Word*)((char*)mem + 256);
    lb.states = lb.maps + maps;
    CR_CUDA(cudaMemsetAsync(mem, 0, bytes, s));
    return CR_OK;
  }
};

template <class T>
bool tma_ok(const Input& in) { return ((uintptr_t)in.p & 15) == 0 && (long long)in.ld * (int)sizeof(T) % 16 == 0; }
template <class T>
bool vec_ok(const void* p, int ld, int D) {
  return !p || ((uintptr_t)p % (vec_of<T>() * sizeof(T)) == 0 && ld % vec_of<T>() == 0 && D % vec_of<T>() == 0);
}
template <class T>
constexpr int type_of() { return std::is_same<T, float>::value ? CR_TYPE_F32 : std::is_same<T, __half>::value ? CR_TYPE_F16 : CR_TYPE_BF16; }
template <class T>
cr_status map_in(CUtensorMap* tm, const Input& in, int D, int n, int steps) {
  return make_tensor_map_2d_plain(tm, type_of<T>(), in.p, D, n, in.ld, ROW / (int)sizeof(T), steps);
}

cr_status states_only(const float* from, int ldf, float* to, int ldt, int D, int n, cudaStream_t stream) {
  if (!to || n == 0) return CR_OK;
  k_scan_states<<<std::min(n, 16 * sm_count()), 256, 0, stream>>>(from, ldf, to, ldt, D, n);
  CR_CHECK_LAUNCH("k_scan_states");
  return CR_OK;
}

template <class E, int GATE>
cr_status forward(FwdArgs<E> p, cudaStream_t stream) {
  constexpr int CH = WARPS * FSUB, W = 32 * vec_of<E>(), SMEM = FSTAGES * 2 * CH * ROW + sizeof(Shared<CH, W, FSTAGES>) + 128;
  const int tiles = (p.D + W - 1) / W;
  Scratch sc;
  CR_TRY(sc.make(p.n, CH, tiles, W, stream));
  CR_REQUIRE((long long)sc.lb.chunks * tiles < INT_MAX / 2, "cr_gated_scan: more than 2^30 work items");
  static std::atomic<uint64_t> done{0};
  CR_TRY(allow_shared((const void*)k_scan_fwd<E, GATE>, SMEM, done));
  p.tma = tma_ok<E>(p.G) && tma_ok<E>(p.X);
  p.pairs = vec_ok<E>(p.H, p.ldh, p.D);
  CUtensorMap tmG = {}, tmX = {};
  if (p.tma) {
    CR_TRY(map_in<E>(&tmG, p.G, p.D, p.n, CH));
    CR_TRY(map_in<E>(&tmX, p.X, p.D, p.n, CH));
  }
  TimedScope ts("k_scan_fwd", stream);
  k_scan_fwd<E, GATE><<<std::min(FBLOCKS * sm_count(), sc.lb.chunks * tiles), NT, SMEM, stream>>>(tmG, tmX, p, sc.lb);
  CR_CHECK_LAUNCH("k_scan_fwd");
  return CR_OK;
}

template <class E, int GATE>
cr_status backward(BwdArgs<E> p, cudaStream_t stream) {
  constexpr int W = 32 * vec_of<E>(), CH = WARPS * BSUB, SMEM = BSTAGES * 3 * CH * ROW + sizeof(Shared<CH, W, BSTAGES>) + 128;
  const int tiles = (p.D + W - 1) / W;
  Scratch sc;
  CR_TRY(sc.make(p.n, CH, tiles, W, stream));
  CR_REQUIRE((long long)sc.lb.chunks * tiles < INT_MAX / 2, "cr_gated_scan_backward: more than 2^30 work items");
  static std::atomic<uint64_t> done{0};
  CR_TRY(allow_shared((const void*)k_scan_bwd<E, GATE>, SMEM, done));
  p.tma = tma_ok<E>(p.G) && tma_ok<E>(p.X) && tma_ok<E>(p.dH);
  p.pairs = vec_ok<E>(p.dG, p.lddg, p.D) && vec_ok<E>(p.dX, p.lddx, p.D);
  CUtensorMap tmG = {}, tmX = {}, tmD = {};
  if (p.tma) {
    CR_TRY(map_in<E>(&tmG, p.G, p.D, p.n, CH));
    CR_TRY(map_in<E>(&tmX, p.X, p.D, p.n, CH));
    CR_TRY(map_in<E>(&tmD, p.dH, p.D, p.n, CH));
  }
  TimedScope ts("k_scan_bwd", stream);
  k_scan_bwd<E, GATE><<<std::min(BBLOCKS * sm_count(), sc.lb.chunks * tiles), NT, SMEM, stream>>>(tmG, tmX, tmD, p, sc.lb);
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
  CR_REQUIRE(D >= 1 && T >= 0 && n_seq >= 0, "cr_gated_scan: D >= 1, T >= 0, n_seq >= 0");
  CR_REQUIRE_SIZES("cr_gated_scan", D, T, n_seq);
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
          FwdArgs<E>{{d_G, ldg}, {d_X, ldx}, D, T, d_off, n_seq, d_h0, ldh0, (E*)d_H, ldh, d_hT, ldhT, d_saved, 0, 0}, stream);
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
  CR_REQUIRE(D >= 1 && T >= 0 && n_seq >= 0, "cr_gated_scan_backward: D >= 1, T >= 0, n_seq >= 0");
  CR_REQUIRE_SIZES("cr_gated_scan_backward", D, T, n_seq);
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
          BwdArgs<E>{{d_G, ldg}, {d_X, ldx}, {d_dH, lddh}, D, T, d_off, n_seq, d_h0, d_dhT, d_saved, ldh0, lddhT, (E*)d_dG,
                     (E*)d_dX, lddg, lddx, d_dh0, lddh0, 0, 0}, stream);
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
  CR_REQUIRE(D >= 1 && B >= 0, "cr_gated_step: D >= 1, B >= 0");
  CR_REQUIRE_SIZES("cr_gated_step", D, B);
  if (B == 0) return CR_OK;
  CR_REQUIRE(d_G && d_X && d_h && d_hnext, "cr_gated_step: NULL argument");
  CR_REQUIRE(ldg >= D && ldx >= D && ldh >= D && ldn >= D && (!d_H || ldo >= D), "cr_gated_step: leading dimension below D");
  int* word = nullptr;   // waits for nothing itself, but reports an earlier call
  CR_TRY(wait_word(&word));
  return with_type(type, [&](auto t0) -> cr_status {
    using E = decltype(t0);
    return with_gate(gate, [&](auto g0) -> cr_status {
      constexpr int GATE = decltype(g0)::value;
      const auto ok4 = [](const void* p, int ld, size_t eb) { return !p || ((uintptr_t)p % (4 * eb) == 0 && ld % 4 == 0); };
      const bool four = D % 4 == 0 && ok4(d_G, ldg, sizeof(E)) && ok4(d_X, ldx, sizeof(E)) && ok4(d_H, ldo, sizeof(E)) &&
                        ok4(d_h, ldh, 4) && ok4(d_hnext, ldn, 4);
      const long long items = (long long)(four ? D / 4 : D) * B;
      const unsigned grid = (unsigned)std::min<long long>((items + 255) / 256, 16 * sm_count());
      if (four)
        CR_CUDA(launch_after(k_scan_step<E, GATE, 4>, grid, 256, 0, 1, stream, (const E*)d_G, ldg, (const E*)d_X, ldx, d_h, ldh, D, B, (E*)d_H, ldo, d_hnext, ldn));
      else
        CR_CUDA(launch_after(k_scan_step<E, GATE, 1>, grid, 256, 0, 1, stream, (const E*)d_G, ldg, (const E*)d_X, ldx, d_h, ldh, D, B, (E*)d_H, ldo, d_hnext, ldn));
      CR_CHECK_LAUNCH("k_scan_step");
      return CR_OK;
    });
  });
  CR_ENTRY_END("cr_gated_step")
}
