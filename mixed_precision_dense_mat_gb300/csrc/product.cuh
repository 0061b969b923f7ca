// Products on the tensor cores with the operators' epilogues: the affine product (affine.cu), the gated one
// (gated.cu) and the steps of the orthogonalised update (ortho.cu).  Each of these files instantiates its own form.
#pragma once
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "ops.cuh"
#include "ptx.cuh"

namespace cr {

// A product C(i, j) = epilogue(sum_k P(i, k) Q(j, k)), C column-major: i runs along C's columns.
// P and Q are matrices in memory of which k or the row is the contiguous index.
struct Operand {
  const void* ptr;
  int rows, ld;
  bool k_major;   // k contiguous, rows ld apart; otherwise rows contiguous, k ld apart
};
struct Epilogue {
  const float *iscale, *jscale, *bias;
  int act;
  const void* R;
  int ldr;
  void* Z;
  int ldz;
  void* C;
  int ldc;
};

// A wide product that another one may follow which does not depend on it: its tiles and their length.  In
// its last round some pairs are free, and the second product starts there (K = 2048, N = 8192, M = 4096 BF16,
// dX and dW: 128 tiles of 128 k-blocks and 256 of 64 on 76 pairs, 7 rounds of 64 k-blocks for 4 + 4).
struct First {
  long long tiles = 0;
  int kblocks = 0;
};

// The affine form's product (affine.cu).  err: the wait word, which the entry has asked for before any of its work.
cr_status affine_product(Operand P, Operand Q, int type, int K, int out_type, const Epilogue& e, int* err, cudaStream_t stream, First* first = nullptr);

namespace {

constexpr int NT = 256;

// Forms.  AFFINE: C = act(sum + bias) + R.  GATED: P has two halves of I rows, C = act(first half's sum) times the
// second half's sum.  STEP: C = alpha sum + beta R, all matrices FP16, or, in the thin kernel, sums of two (the second one
// small); C symmetric where the wide kernel's tiles say so.  SUMS (wide): STEP with sums of two, or the sums alone, in FP32.
enum Form { AFFINE, GATED, STEP, SUMS };

struct Params {
  int I, J, kblocks;     // GATED: I of each half
  int pk, qk;            // operand P, Q is k-major
  uint32_t idesc;        // MMA instruction descriptor
  int ti, tj;            // output tiles
  int bn;                // thin kernel: columns j of its tile
  int stages;            // wide kernel
  int second;            // wide kernel: follows another product of the call that it does not depend on
  int early, ahead;      // then: pairs that are free before the others, and tiles that they can take until then
  int tma_c, tma_z;      // C, Z can be stored by TMA
  int vec_r;             // R allows 16-byte accesses
  int tma_r;             // wide kernel: R comes by TMA into the output buffers (16-bit outputs)
  int vec4;              // four consecutive i of everything in the epilogue can be accessed at once
  // STEP and SUMS
  int segments;          // 1, or 3: the products of P's and Q's first parts and of each one's first with the other's second part
  int triangle;          // C symmetric: tiles ti <= tj alone are formed (STEP stores them at (tj, ti) too; wide kernel)
  int parts;             // SUMS: tiles over as many parts of k, one matrix of jpad rows below the other
  int jpad;
  int chunk;             // SUMS: k-blocks of two first parts that the tensor cores sum up by themselves; such sums are added in registers
  float alpha, beta;
  void *C2, *R2;         // second parts (NULL: none), laid out like C and R
  Epilogue e;
  unsigned long long limit;
  int* err;
};

constexpr int KBYTES = 128;                      // one stage holds 128 bytes of k per row
constexpr int ATOM = 64 * 128;                   // rows-contiguous operand: 64 rows x 64 k
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool bf16, bool a_rows, bool b_rows) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_rows ? 1u : 0u) << 15) |
         ((b_rows ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Shared-memory descriptor of an operand tile in the 128-byte swizzle.  k-major: rows of 128 bytes
// in 8-row groups 1024 apart.  Rows contiguous: 64-row blocks 8192 bytes apart, each 64 k of 128
// bytes in 8-k groups 1024 apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, bool k_major) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
  return d | (uint64_t)(k_major ? 1 : ATOM >> 4) << 16;
}
// From one MMA's k to the next inside a stage, in descriptor units of 16 bytes: 32 bytes along k,
// or 16 k of 128 bytes.
__device__ __forceinline__ uint32_t desc_step(bool k_major) { return k_major ? 2 : 128; }

__device__ __forceinline__ void gave_up(const Params& p, volatile int* abort) {
  *abort = 1;
  *(volatile int*)p.err = 1;
  __threadfence_system();
}

constexpr int OROW = 128, WBUF = 32 * OROW;      // an epilogue warp's rows on their way out: one tile of 128-byte rows

// z (a finished sum) to the output (i, j).
template <class O>
__device__ __forceinline__ void finish(const Params& p, int i, int j, float z) {
  if (p.e.iscale) z *= p.e.iscale[i];
  if (p.e.jscale) z *= p.e.jscale[j];
  if (p.e.bias) z += p.e.bias[i];
  if (p.e.Z) ((O*)p.e.Z)[(size_t)j * p.e.ldz + i] = from_float<O>(z);
  float v[1] = {z};
  activate_all<1>(v, p.e.act);
  if (p.e.R) v[0] += to_float(((const O*)p.e.R)[(size_t)j * p.e.ldr + i]);
  ((O*)p.e.C)[(size_t)j * p.e.ldc + i] = from_float<O>(v[0]);
}

// Four consecutive i of column j.
template <class O>
__device__ __forceinline__ void thin_finish4(const Params& p, int i, int j, float (&v)[4]) {
  const Epilogue& e = p.e;
  if (!p.vec4 || i + 4 > p.I) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < p.I) finish<O>(p, i + q, j, v[q]);
    return;
  }
  const float js = e.jscale ? e.jscale[j] : 1.0f;
  float4 is = make_float4(1, 1, 1, 1), b = make_float4(0, 0, 0, 0);
  if (e.iscale) is = *reinterpret_cast<const float4*>(e.iscale + i);
  if (e.bias) b = *reinterpret_cast<const float4*>(e.bias + i);
  v[0] = fmaf(v[0] * is.x, js, b.x);
  v[1] = fmaf(v[1] * is.y, js, b.y);
  v[2] = fmaf(v[2] * is.z, js, b.z);
  v[3] = fmaf(v[3] * is.w, js, b.w);
  struct alignas(4 * sizeof(O)) Four {
    O x[4];
  };
  const auto put = [&](void* out, int ld) {
    Four o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o.x[q] = from_float<O>(v[q]);
    *reinterpret_cast<Four*>((O*)out + (size_t)j * ld + i) = o;
  };
  if (e.Z) put(e.Z, e.ldz);
  activate_all<4>(v, e.act);
  if (e.R) {
    const Four r = *reinterpret_cast<const Four*>((const O*)e.R + (size_t)j * e.ldr + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] += to_float(r.x[q]);
  }
  put(e.C, e.ldc);
}

// One i and 16 columns from j0.
template <class O>
__device__ __forceinline__ void thin_store16(const Params& p, int i, int j0, float (&v)[16]) {
  const int n = min(16, p.J - j0);
  const float is = p.e.iscale ? p.e.iscale[i] : 1.0f, b = p.e.bias ? p.e.bias[i] : 0.0f;
#pragma unroll
  for (int q = 0; q < 16; ++q)
    if (q < n) {
      v[q] = fmaf(v[q] * is, p.e.jscale ? p.e.jscale[j0 + q] : 1.0f, b);
      if (p.e.Z) ((O*)p.e.Z)[(size_t)(j0 + q) * p.e.ldz + i] = from_float<O>(v[q]);
    }
  activate_all<16>(v, p.e.act);
#pragma unroll
  for (int q = 0; q < 16; ++q)
    if (q < n) {
      if (p.e.R) v[q] += to_float(((const O*)p.e.R)[(size_t)(j0 + q) * p.e.ldr + i]);
      ((O*)p.e.C)[(size_t)(j0 + q) * p.e.ldc + i] = from_float<O>(v[q]);
    }
}

// gate and up (finished sums) to the output (i, j).
template <class O>
__device__ __forceinline__ void finish_gated(const Params& p, int i, int j, float g, float u) {
  const Epilogue& e = p.e;
  if (e.iscale) g *= e.iscale[i], u *= e.iscale[p.I + i];
  if (e.jscale) g *= e.jscale[j], u *= e.jscale[j];
  if (e.bias) g += e.bias[i], u += e.bias[p.I + i];
  if (e.Z) {
    ((O*)e.Z)[(size_t)j * e.ldz + i] = from_float<O>(g);
    ((O*)e.Z)[(size_t)j * e.ldz + p.I + i] = from_float<O>(u);
  }
  float v[1] = {g};
  activate_all<1>(v, e.act);
  ((O*)e.C)[(size_t)j * e.ldc + i] = from_float<O>(__fmul_rn(v[0], u));
}

// Four consecutive i of column j.
template <class O>
__device__ __forceinline__ void finish_gated4(const Params& p, int i, int j, float (&g)[4], float (&u)[4]) {
  const Epilogue& e = p.e;
  if (!p.vec4 || i + 4 > p.I) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < p.I) finish_gated<O>(p, i + q, j, g[q], u[q]);
    return;
  }
  const float js = e.jscale ? e.jscale[j] : 1.0f;
  struct alignas(4 * sizeof(O)) Four {
    O x[4];
  };
  const auto half = [&](int row, float (&v)[4]) {
    float4 is = make_float4(1, 1, 1, 1), b = make_float4(0, 0, 0, 0);
    if (e.iscale) is = *reinterpret_cast<const float4*>(e.iscale + row);
    if (e.bias) b = *reinterpret_cast<const float4*>(e.bias + row);
    v[0] = fmaf(v[0] * is.x, js, b.x);
    v[1] = fmaf(v[1] * is.y, js, b.y);
    v[2] = fmaf(v[2] * is.z, js, b.z);
    v[3] = fmaf(v[3] * is.w, js, b.w);
    if (e.Z) {
      Four o;
#pragma unroll
      for (int q = 0; q < 4; ++q) o.x[q] = from_float<O>(v[q]);
      *reinterpret_cast<Four*>((O*)e.Z + (size_t)j * e.ldz + row) = o;
    }
  };
  half(i, g);
  half(p.I + i, u);
  activate_all<4>(g, e.act);
  Four o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o.x[q] = from_float<O>(__fmul_rn(g[q], u[q]));
  *reinterpret_cast<Four*>((O*)e.C + (size_t)j * e.ldc + i) = o;
}

// STEP: four consecutive i of column j (R, R2 and C2 are the library's own matrices, with columns on 16-byte boundaries).
struct StepR {
  uint2 hi, lo;
};
__device__ __forceinline__ StepR step_r(const Params& p, int i, int j) {
  StepR r = {make_uint2(0, 0), make_uint2(0, 0)};
  const size_t at = (size_t)j * p.e.ldr + i;
  if (p.e.R && i < p.I) r.hi = *reinterpret_cast<const uint2*>((const __half*)p.e.R + at);
  if (p.R2 && i < p.I) r.lo = *reinterpret_cast<const uint2*>((const __half*)p.R2 + at);
  return r;
}
template <class O>
__device__ __forceinline__ void finish_step4(const Params& p, int i, int j, const StepR& r, float (&v)[4]) {
  if (i >= p.I) return;
  const size_t c = (size_t)j * p.e.ldc + i;
  const float2 a = widen2(r.hi.x, __half{}), b = widen2(r.hi.y, __half{}), x = widen2(r.lo.x, __half{}), y = widen2(r.lo.y, __half{});
  v[0] = fmaf(p.beta, a.x + x.x, v[0] * p.alpha);
  v[1] = fmaf(p.beta, a.y + x.y, v[1] * p.alpha);
  v[2] = fmaf(p.beta, b.x + y.x, v[2] * p.alpha);
  v[3] = fmaf(p.beta, b.y + y.y, v[3] * p.alpha);
  struct alignas(4 * sizeof(O)) Four {
    O x[4];
  } o, rest;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    o.x[q] = from_float<O>(v[q]);
    rest.x[q] = from_float<O>(v[q] - to_float(o.x[q]));
  }
  if (p.vec4 && i + 4 <= p.I) {
    *reinterpret_cast<Four*>((O*)p.e.C + c) = o;
    if (p.C2) *reinterpret_cast<Four*>((O*)p.C2 + c) = rest;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < p.I) {
        ((O*)p.e.C)[c + q] = o.x[q];
        if (p.C2) ((O*)p.C2)[c + q] = rest.x[q];
      }
  }
}

// A float vector's N entries from i0 on, spread over the warp's lanes (0 past the end): entry q is w[q / 32] of
// lane q % 32, and every_entry gives it to all lanes.  Loaded ahead and handed round by shuffles: as loads of
// the same address by all lanes, bias alone took 2.5 us per 256 x 256 tile.
template <int N>
__device__ __forceinline__ void load_row(const float* x, int i0, int I, float (&w)[N / 32]) {
  const int i = i0 + (threadIdx.x & 31);
#pragma unroll
  for (int q = 0; q < N / 32; ++q) w[q] = x && i + 32 * q < I ? x[i + 32 * q] : 0.0f;
}
template <int N>
__device__ __forceinline__ float every_entry(const float (&w)[N], int q) { return __shfl_sync(0xffffffffu, w[q / 32], q % 32); }

// A warp's 32 rows j of N = OROW / sizeof(O) values from (i0, j0) live in its buffer as rows of 128 bytes in the
// 128-byte swizzle: 16-byte word q of row r is at word q ^ (r & 7).
template <class O>
__device__ __forceinline__ O* at_in(uint8_t* buf, int row, int col) {
  const int byte = col * (int)sizeof(O);
  return reinterpret_cast<O*>(buf + row * OROW + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15));
}

// To memory: through the buffer and by TMA, or, where TMA cannot address the output, with each row's
// elements stored by neighbouring lanes.  `ready`: the buffer's last tile has been read.
template <class O, int N>
__device__ __forceinline__ void put_rows(const CUtensorMap* tm, int tma, O* out, int ld, int I, int J, int i0, int j0, uint8_t* buf,
                                         bool ready, const float* v) {
  const int lane = threadIdx.x & 31;
  if (!ready && lane == 0) tma_store_wait_read();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {
    const Eight<O> w = narrow8<O>(v + 8 * q);
#pragma unroll
    for (int x = 0; x < (int)sizeof(O) / 2; ++x)
      *reinterpret_cast<uint4*>(buf + lane * OROW + (((int)sizeof(O) / 2 * q + x) ^ (lane & 7)) * 16) =
          make_uint4(w.w[4 * x], w.w[4 * x + 1], w.w[4 * x + 2], w.w[4 * x + 3]);
  }
  if (tma) {
    fence_smem_to_tma();
    __syncwarp();
    if (lane == 0 && j0 < J) {
      tma_store_2d(tm, buf, i0, j0);
      tma_store_commit();
    }
  } else {
    __syncwarp();
    for (int r = 0; r < 32 && j0 + r < J; ++r)
#pragma unroll
      for (int c = lane; c < N; c += 32)
        if (i0 + c < I) out[(size_t)(j0 + r) * ld + i0 + c] = *at_in<O>(buf, r, c);
    fence_smem_to_tma();   // the next R may come into the buffer by TMA
    __syncwarp();
  }
}
// From memory, added to v, where TMA cannot address the matrix.
template <class O, int N>
__device__ __forceinline__ void add_rows_of(const O* in, int ld, int I, int J, int i0, int j0, uint8_t* buf, float* v) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) tma_store_wait_read();
  __syncwarp();
  for (int r0 = 0; r0 < 32; r0 += 8) {   // the loads of 8 rows in flight at once
    O w[8][N / 32];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < N / 32; ++c)
        if (j0 + r0 + r < J && i0 + lane + 32 * c < I) w[r][c] = in[(size_t)(j0 + r0 + r) * ld + i0 + lane + 32 * c];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < N / 32; ++c) *at_in<O>(buf, r0 + r, lane + 32 * c) = w[r][c];
  }
  __syncwarp();
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] += to_float(*at_in<O>(buf, lane, q));
  __syncwarp();
}

// Epilogue of the warp's 32 rows j and N columns i; v holds the sums.
template <class O, int N>
__device__ __forceinline__ void wide_finish(const Params& p, const CUtensorMap* tmC, const CUtensorMap* tmZ, int i0, int j0, float js,
                                            const float (&is)[N / 32], const float (&bias)[N / 32], uint8_t* buf, const uint8_t* rows, float* v) {
  const Epilogue& e = p.e;
  const int j = j0 + (threadIdx.x & 31);
  if (e.iscale) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] *= every_entry(is, q);
  }
  if (e.jscale) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] *= js;
  }
  if (e.bias) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] += every_entry(bias, q);
  }
  if (e.Z) put_rows<O, N>(tmZ, p.tma_z, (O*)e.Z, e.ldz, p.I, p.J, i0, j0, buf, false, v);
  activate_all<N>(v, e.act);
  if (rows) {   // R in the output buffer
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
      float w[8];
      widen8(*reinterpret_cast<const Eight<O>*>(rows + lane * OROW + ((q ^ (lane & 7)) << 4)), w);
#pragma unroll
      for (int x = 0; x < 8; ++x) v[8 * q + x] += w[x];
    }
  } else if (e.R && p.vec_r && i0 + N <= p.I) {
    if (j < p.J) {
      const O* r = (const O*)e.R + (size_t)j * e.ldr + i0;
#pragma unroll
      for (int q = 0; q < N; q += 8) {
        float w[8];
        widen8(*reinterpret_cast<const Eight<O>*>(r + q), w);
#pragma unroll
        for (int x = 0; x < 8; ++x) v[q + x] += w[x];
      }
    }
  } else if (e.R) {
    add_rows_of<O, N>((const O*)e.R, e.ldr, p.I, p.J, i0, j0, buf, v);
  }
  __syncwarp();
  put_rows<O, N>(tmC, p.tma_c, (O*)e.C, e.ldc, p.I, p.J, i0, j0, buf, rows != nullptr, v);
}

// ---------------------------------------------------------------- wide kernel
// 256 x 256 outputs per CTA pair (cta_group::2): the pair's MMA has M = 256 rows j (128 per CTA, its
// operand A = Q) and N = 256 columns i (operand B = P, half of it in each CTA; N = 128 takes as long per
// k-block, 0.27 us).  Bound by the tensor cores: K = 4096, N = 8192, M = 4096 BF16 with bias and silu 149 us,
// 1.84 PFLOP/s, the tensor pipe active 83 % of the time; e4m3 75 us, 3.64 PFLOP/s.  Persistent; warp 0
// loads by TMA into a ring of stages, warp 1 of the first CTA issues the MMAs, warps 2-9 take the
// accumulator (two of them in TMEM, so the epilogue of one tile overlaps the next tile's products)
// through the epilogue: a thread holds one j and 32 consecutive i.
constexpr int WSTAGES = 6;                       // 5 with two output buffers per warp
constexpr int WTILE = 128 * KBYTES;              // one operand's half tile of a stage, 16 KB
constexpr int WSTAGE = 2 * WTILE;
constexpr int WEPI = 8;                          // epilogue warps
constexpr int epilogue_warps(int form) { return form == SUMS ? 2 * WEPI : WEPI; }   // SUMS: half the columns each, held in registers
constexpr int wide_threads(int form) { return 64 + 32 * epilogue_warps(form); }
struct WideBars {
  uint64_t full[WSTAGES], empty[WSTAGES], tfull[2], tempty[2], rows[WEPI][2], settled;
  uint32_t tmem;
  int abort;
  int issued[2];   // in the first CTA: stages that the two CTAs' loaders have filled in all
};
constexpr int WSMEM = WSTAGES * WSTAGE + WEPI * WBUF + 1024 + 384;
static_assert(WSTAGE == WEPI * WBUF, "a stage's memory is a second set of output buffers");
static_assert(sizeof(WideBars) <= 384, "barrier area");

// What the wide kernel reads and writes by TMA.  AFFINE: R is the residual; GATED: Z2 is Z's second half; STEP: T
// is C's store of transposed tiles; SUMS: P and Q have second parts.
template <int FORM>
struct Maps {
  CUtensorMap P, Q, C, Z, R;
};
template <>
struct Maps<GATED> {
  CUtensorMap P, Q, C, Z, Z2;
};
template <>
struct Maps<STEP> {
  CUtensorMap P, Q, C, R, T;
};
template <>
struct Maps<SUMS> {
  CUtensorMap P, Q, P2, Q2, C, C2, R, R2;   // C alone with parts: their FP32 matrices
};

// Tile t of the triangle i <= j, column by column.
__device__ __forceinline__ void triangle_tile(int t, int& i, int& j) {
  j = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((long long)j * (j + 1) / 2 > t) --j;
  while ((long long)(j + 1) * (j + 2) / 2 <= t) ++j;
  i = t - (int)((long long)j * (j + 1) / 2);
}

// Tile t: column tiles j in groups of 16 and all row tiles i inside a group, so that the tiles in
// flight share operands in L2 (K = 4096, N = 16384, M = 8192 BF16: groups of 1 674 us, 4 592, 8 564, 16 555, 32 583).
__device__ __forceinline__ void wide_tile(const Params& p, int t, int& i, int& j) {
  constexpr int GROUP = 16;
  const int per = GROUP * p.ti, g = t / per, gj = min(GROUP, p.tj - g * GROUP), r = t - g * per;
  i = r / gj;
  j = g * GROUP + r % gj;
}

// The i-th tile of pair cl of n.  The first `early` pairs take `ahead` tiles each before all pairs take turns.
__device__ __forceinline__ int wide_turn(const Params& p, int cl, int n, int i) {
  if (cl >= p.early) return p.early * p.ahead + i * n + cl;
  return i < p.ahead ? i * p.early + cl : p.early * p.ahead + (i - p.ahead) * n + cl;
}

// GATED: the warp's 32 rows j and N outputs i from the sums of both halves (K = 4096, N = M = 8192 e4m3: 280 us with this
// epilogue behind the next tile's products, 3.9 PFLOP/s).
template <class O, int N>
__device__ __forceinline__ void gated_finish(const Params& p, const Maps<GATED>& maps, int i0, int j0, float js, const float (&gs)[N / 32],
                                             const float (&ws)[N / 32], const float (&gb)[N / 32], const float (&wb)[N / 32], uint8_t* buf,
                                             float* g, float* w) {
  const Epilogue& e = p.e;
  if (e.iscale) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      g[q] *= every_entry(gs, q);
      w[q] *= every_entry(ws, q);
    }
  }
  if (e.jscale) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      g[q] *= js;
      w[q] *= js;
    }
  }
  if (e.bias) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      g[q] += every_entry(gb, q);
      w[q] += every_entry(wb, q);
    }
  }
  if (e.Z) {
    put_rows<O, N>(&maps.Z, p.tma_z, (O*)e.Z, e.ldz, p.I, p.J, i0, j0, buf, false, g);
    put_rows<O, N>(&maps.Z2, p.tma_z, (O*)e.Z + p.I, e.ldz, p.I, p.J, i0, j0, buf, false, w);
  }
  activate_all<N>(g, e.act);
#pragma unroll
  for (int q = 0; q < N; ++q) g[q] = __fmul_rn(g[q], w[q]);
  put_rows<O, N>(&maps.C, p.tma_c, (O*)e.C, e.ldc, p.I, p.J, i0, j0, buf, false, g);
}

// STEP: the warp's 32 rows j and N = 64 columns i; R is in buf (with_r).  A tile off the diagonal of a symmetric C goes out
// a second time, transposed: 64 rows of 32 elements.
template <class O, int N>
__device__ __forceinline__ void step_finish(const Params& p, const Maps<STEP>& maps, int i0, int j0, bool twice, uint8_t* buf, bool with_r, float* v) {
  static_assert(N == 64, "16-bit outputs");
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] *= p.alpha;
  if (with_r) {
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
      float r[8];
      widen8(*reinterpret_cast<const Eight<__half>*>(buf + lane * OROW + ((q ^ (lane & 7)) << 4)), r);
#pragma unroll
      for (int x = 0; x < 8; ++x) v[8 * q + x] = fmaf(p.beta, r[x], v[8 * q + x]);
    }
  } else if (lane == 0) {
    tma_store_wait_read();
  }
  __syncwarp();
  put_rows<O, N>(&maps.C, p.tma_c, (O*)p.e.C, p.e.ldc, p.I, p.J, i0, j0, buf, true, v);
  if (!twice) return;
  if (lane == 0) tma_store_wait_read();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < N; ++q) reinterpret_cast<O*>(buf)[q * 32 + lane] = from_float<O>(v[q]);
  fence_smem_to_tma();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&maps.T, buf, j0, i0);
    tma_store_commit();
  }
}

template <int FORM, bool F8, class O>
__global__ void __launch_bounds__(wide_threads(FORM), 1) k_wide(const __grid_constant__ Maps<FORM> maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  WideBars* bars = reinterpret_cast<WideBars*>(smem + WSTAGES * WSTAGE + WEPI * WBUF);
  volatile int* abort_flag = &bars->abort;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform: the loops below keep their state in uniform registers
  const uint32_t rank = cluster_rank();
  const bool triangle = (FORM == STEP || FORM == SUMS) && p.triangle;
  const int tiles = triangle ? (int)((long long)p.tj * (p.tj + 1) / 2) : p.ti * p.tj, ncl = gridDim.x >> 1, cl = blockIdx.x >> 1;
  const int ntiles = FORM == SUMS ? tiles * p.parts : tiles;
  // SUMS: all tiles of a part of k before the next part
  const auto tile_at = [&](int t, int& i, int& j) {
    if (FORM == SUMS) t %= tiles;
    if (triangle) triangle_tile(t, i, j);
    else wide_tile(p, t, i, j);
  };
  // SUMS: where the tensor cores' sum that begins at kb ends.  What products with a small part lose is below 2^-11 of what the others do.
  const auto run_end = [&](int kb, int kb1) {
    const int small = p.kblocks / p.segments * (p.segments - 1);
    return min(kb1, kb < small ? small : kb + p.chunk);
  };
  const auto k_range = [&](int t, int& k0, int& k1) {
    const int part = FORM == SUMS ? t / tiles : 0;
    k0 = FORM == SUMS ? (int)((long long)p.kblocks * part / p.parts) : 0;
    k1 = FORM == SUMS ? (int)((long long)p.kblocks * (part + 1) / p.parts) : p.kblocks;
  };
  constexpr int KE = F8 ? 128 : 64;   // k elements per stage

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->tfull[b], 1);
      mbar_init(&bars->tempty[b], 2 * epilogue_warps(FORM));   // one arrival per epilogue warp of the pair
      for (int x = 0; x < WEPI; ++x) mbar_init(&bars->rows[x][b], 1);
    }
    mbar_init(&bars->settled, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&bars->tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);
  // The kernel before a second product is the first one, which lets this one start only after its own
  // wait: the inputs are there.  It is waited for at the end, so that later kernels need not.
  if (!p.second) wait_for_previous();
  let_next_start();
  const auto give_up = [&] {   // both CTAs leave their loops at the flag
    gave_up(p, abort_flag);
    store_cluster(cluster_addr(smem_u32(&bars->abort), rank ^ 1u), 1);
  };

  if (warp == 0) {
    if (elect_one()) {
      prefetch_tmap(&maps.P);
      prefetch_tmap(&maps.Q);
    }
    uint32_t st = 0, ph = 0;
    int issued = 0;
    const int per = FORM == SUMS ? p.kblocks / p.segments : p.kblocks;   // k-blocks of a segment
    bool ok = true;
    const uint32_t full0 = cluster_addr(smem_u32(&bars->full[0]), 0);
    for (int u = 0, t; ok && (t = wide_turn(p, cl, ncl, u)) < ntiles; ++u) {
      int ti, tj;
      tile_at(t, ti, tj);
      // GATED: the second CTA's half of operand B is the same rows of P's second half
      const int i0 = FORM == GATED ? ti * 128 + (int)rank * p.I : ti * 256 + (int)rank * 128, j0 = tj * 256 + (int)rank * 128;
      const CUtensorMap *tmP = &maps.P, *tmQ = &maps.Q;
      int kb0, kb1;
      k_range(t, kb0, kb1);
      for (int kb = kb0, kx = FORM == SUMS ? kb0 % per : 0; kb < kb1; ++kb, ++kx) {
        if constexpr (FORM == SUMS) {   // the small products first
          if (kx == per) kx = 0;
          if (p.segments == 3) {
            tmP = kb / per == 1 ? &maps.P2 : &maps.P;
            tmQ = kb < per ? &maps.Q2 : &maps.Q;
          }
        }
        ok = mbar_wait_warp(&bars->empty[st], ph ^ 1u, p.limit);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* sa = smem + st * WSTAGE;
          uint8_t* sb = sa + WTILE;
          if (rank == 0) mbar_arrive_expect_tx(&bars->full[st], 2 * WSTAGE);
          const uint32_t bar = full0 + 8 * st;
          const int k0 = kx * KE;
          if (p.qk) {
            tma_load_2d_pair(sa, tmQ, bar, k0, j0);
          } else {
            tma_load_2d_pair(sa, tmQ, bar, j0, k0);
            tma_load_2d_pair(sa + ATOM, tmQ, bar, j0 + 64, k0);
          }
          if (p.pk) {
            tma_load_2d_pair(sb, tmP, bar, k0, i0);
          } else {
            tma_load_2d_pair(sb, tmP, bar, i0, k0);
            tma_load_2d_pair(sb + ATOM, tmP, bar, i0 + 64, k0);
          }
        }
        ++issued;
        if (++st == (uint32_t)p.stages) st = 0, ph ^= 1u;
      }
    }
    for (int q = min(issued, p.stages); ok && q > 0; --q) {   // the stages' last arrivals come before the CTA leaves
      const int n = issued - q;
      ok = mbar_wait_warp(&bars->empty[n % p.stages], (uint32_t)(n / p.stages) & 1u, p.limit);
    }
    if (lane == 0) {
      if (!ok) give_up();
      store_cluster(cluster_addr(smem_u32(&bars->issued[rank]), 0), (uint32_t)issued);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      uint32_t st = 0, ph = 0;
      bool ok = true;
      const uint32_t ps = desc_step(p.pk), qs = desc_step(p.qk), s0 = smem_u32(smem);
      const uint64_t da0 = tile_desc(s0, p.qk), db0 = tile_desc(s0 + WTILE, p.pk);
      if constexpr (FORM == SUMS) {
        uint32_t run = 0;   // accumulators filled
        for (int u = 0, t; ok && (t = wide_turn(p, cl, ncl, u)) < ntiles; ++u) {
          int kb0, kb1;
          k_range(t, kb0, kb1);
          for (int kb = kb0, begin = kb0; kb < kb1; ++kb) {
            const uint32_t b = run & 1u;
            if (kb == begin) {
              ok = mbar_wait_warp(&bars->tempty[b], (run >> 1 & 1u) ^ 1u, p.limit);
              if (!ok) break;
              tc_fence_after();
            }
            ok = mbar_wait_warp(&bars->full[st], ph, p.limit);
            if (!ok) break;
            tc_fence_after();
            const bool end = kb + 1 == run_end(begin, kb1);
            if (elect_one()) {
              const uint64_t da = da0 + st * (WSTAGE >> 4), db = db0 + st * (WSTAGE >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_any<true, F8>(tmem + b * 256, da + kk * qs, db + kk * ps, p.idesc, kb != begin || kk != 0);
              mma_commit_pair(&bars->empty[st]);
              if (end) mma_commit_pair(&bars->tfull[b]);
            }
            __syncwarp();
            if (end) begin = kb + 1;
            run += end;
            if (++st == (uint32_t)p.stages) st = 0, ph ^= 1u;
          }
        }
      } else
      for (int u = 0; ok && wide_turn(p, cl, ncl, u) < ntiles; ++u) {
        const int b = u & 1;
        ok = mbar_wait_warp(&bars->tempty[b], ((uint32_t)(u >> 1) & 1u) ^ 1u, p.limit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(b * 256);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          ok = mbar_wait_warp(&bars->full[st], ph, p.limit);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t da = da0 + st * (WSTAGE >> 4), db = db0 + st * (WSTAGE >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_any<true, F8>(acc, da + kk * qs, db + kk * ps, p.idesc, (kb | kk) != 0);
            mma_commit_pair(&bars->empty[st]);
            if (kb + 1 == p.kblocks) mma_commit_pair(&bars->tfull[b]);
          }
          __syncwarp();
          if (++st == (uint32_t)p.stages) st = 0, ph ^= 1u;
        }
      }
      if (!ok && lane == 0) give_up();
      __syncwarp();
      if (elect_one()) mma_commit_own(&bars->settled);   // whoever gave up: MMAs in flight end before tensor memory is freed
      mbar_wait_warp(&bars->settled, 0, LANDING_NS);
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* buf = smem + p.stages * WSTAGE + (warp - 2) * WBUF;   // AFFINE with R: a second one WSTAGE further
    const uint32_t tempty[2] = {cluster_addr(smem_u32(&bars->tempty[0]), 0), cluster_addr(smem_u32(&bars->tempty[1]), 0)};
    uint32_t nrows = 0;   // parity of the two buffers' next R
    uint32_t run = 0;     // SUMS: accumulators read
    for (int u = 0, t; (t = wide_turn(p, cl, ncl, u)) < ntiles; ++u) {
      const int b = u & 1;
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
      int ti, tj;
      tile_at(t, ti, tj);
      const int j0 = tj * 256 + (int)rank * 128 + quad * 32, ibase = FORM == GATED ? ti * 128 + half * 64 : ti * 256 + half * (FORM == SUMS ? 64 : 128);
      constexpr int N = OROW / (int)sizeof(O);
      const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(b * 256 + half * (FORM == GATED ? 64 : 128));
      const auto accumulator_read = [&] {   // the next tile but one may have it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty[b]);
      };
      if constexpr (FORM == GATED) {
        if (!mbar_wait_warp(&bars->tfull[b], (uint32_t)(u >> 1) & 1u, p.limit)) {
          if (lane == 0) give_up();
          break;
        }
        tc_fence_after();
        const float js = p.e.jscale && j0 + lane < p.J ? p.e.jscale[j0 + lane] : 1.0f;
        for (int c = 0; c < 64; c += N) {
          uint32_t g[N / 32][32], w[N / 32][32];
          float gs[N / 32], ws[N / 32], gb[N / 32], wb[N / 32];
          load_row<N>(p.e.iscale, ibase + c, p.I, gs);
          load_row<N>(p.e.iscale ? p.e.iscale + p.I : nullptr, ibase + c, p.I, ws);
          load_row<N>(p.e.bias, ibase + c, p.I, gb);
          load_row<N>(p.e.bias ? p.e.bias + p.I : nullptr, ibase + c, p.I, wb);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < N / 32; ++q) {
            tmem_ld32(tq + (uint32_t)(c + 32 * q), g[q]);
            tmem_ld32(tq + (uint32_t)(128 + c + 32 * q), w[q]);
          }
          tmem_ld_wait();
          if (c + N == 64) accumulator_read();
          if (ibase + c >= p.I) continue;
          gated_finish<O, N>(p, maps, ibase + c, j0, js, gs, ws, gb, wb, buf, reinterpret_cast<float*>(g), reinterpret_cast<float*>(w));
        }
      } else if constexpr (FORM == SUMS) {
        int kb0, kb1;
        k_range(t, kb0, kb1);
        // With one part of k the tile is finished here: R's first part is asked for before the products, the second one after.
        const bool here = j0 < p.J && ibase < p.I, direct = p.parts == 1 && !triangle && here;
        uint64_t* rbar = &bars->rows[(warp - 2) % WEPI][(warp - 2) / WEPI];
        const auto ask = [&](const CUtensorMap* m) {
          if (lane == 0) {
            tma_store_wait_read();
            mbar_arrive_expect_tx(rbar, WBUF);
            tma_load_2d(buf, m, rbar, ibase, j0);
          }
        };
        const bool with_r = direct && p.e.R;
        if (with_r) ask(&maps.R);
        float sum[64];
#pragma unroll
        for (int q = 0; q < 64; ++q) sum[q] = 0.0f;
        bool lost = false;
#pragma unroll 1
        for (int kb = kb0; kb < kb1; kb = run_end(kb, kb1), ++run) {
          const uint32_t acc = run & 1u;
          if (!mbar_wait_warp(&bars->tfull[acc], run >> 1 & 1u, p.limit)) {
            if (lane == 0) give_up();
            lost = true;
            break;
          }
          tc_fence_after();
          const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + acc * 256 + (uint32_t)(half * 64);
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            float v[16];
            tmem_ld16(from + (uint32_t)c, v);
#pragma unroll
            for (int q = 0; q < 16; ++q) sum[c + q] += v[q];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty[acc]);
        }
        if (lost) {
          if (with_r) mbar_wait_warp(rbar, nrows & 1u, LANDING_NS);
          break;
        }
        if (!here) continue;
        if (!direct) {
#pragma unroll
          for (int c = 0; c < 64; c += 32)
            if (ibase + c < p.I) put_rows<float, 32>(&maps.C, 1, nullptr, 0, 0, 0x7fffffff, ibase + c, t / tiles * p.jpad + j0, buf, false, sum + c);
          continue;
        }
#pragma unroll
        for (int q = 0; q < 64; ++q) sum[q] *= p.alpha;
        const auto add_r = [&] {
          const bool there = mbar_wait_warp(rbar, nrows & 1u, p.limit);
          if (!there) {
            if (lane == 0) give_up();   // it goes on with what lands, and leaves at the next tile
            mbar_wait_warp(rbar, nrows & 1u, LANDING_NS);
          }
          nrows ^= 1u;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float r[8];
            widen8(*reinterpret_cast<const Eight<__half>*>(buf + lane * OROW + ((q ^ (lane & 7)) << 4)), r);
#pragma unroll
            for (int x = 0; x < 8; ++x) sum[8 * q + x] = fmaf(p.beta, r[x], sum[8 * q + x]);
          }
          fence_smem_to_tma();
          __syncwarp();
        };
        if (with_r) {
          add_r();
          if (p.R2) {
            ask(&maps.R2);
            add_r();
          }
        }
#pragma unroll
        for (int c = 0; c < 64; c += N)
          if (ibase + c < p.I) put_rows<O, N>(&maps.C, p.tma_c, (O*)p.e.C, p.e.ldc, p.I, p.J, ibase + c, j0, buf, false, sum + c);
        if (p.C2) {
#pragma unroll
          for (int q = 0; q < 64; ++q) sum[q] -= to_float(from_float<O>(sum[q]));
#pragma unroll
          for (int c = 0; c < 64; c += N)
            if (ibase + c < p.I) put_rows<O, N>(&maps.C2, 1, (O*)p.C2, p.e.ldc, p.I, p.J, ibase + c, j0, buf, false, sum + c);
        }
      } else if constexpr (FORM == STEP) {
        const auto there = [&](int c) { return j0 < p.J && ibase + c < p.I; };
        bool pending = false;   // R of the columns at c is on its way
        const auto ask = [&](int c) {
          pending = p.e.R && there(c);
          if (pending && lane == 0) {
            tma_store_wait_read();
            mbar_arrive_expect_tx(&bars->rows[warp - 2][0], WBUF);
            tma_load_2d(buf, &maps.R, &bars->rows[warp - 2][0], ibase + c, j0);
          }
        };
        ask(0);
        if (!mbar_wait_warp(&bars->tfull[b], (uint32_t)(u >> 1) & 1u, p.limit)) {
          if (lane == 0) give_up();
          if (pending) mbar_wait_warp(&bars->rows[warp - 2][0], nrows & 1u, LANDING_NS);
          break;
        }
        tc_fence_after();
        bool lost = false;
        for (int c = 0; c < 128 && !lost; c += N) {
          uint32_t v[N / 32][32];
          if (c > 0) ask(c);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < N / 32; ++q) tmem_ld32(tq + (uint32_t)(c + 32 * q), v[q]);
          tmem_ld_wait();
          if (c + N == 128) accumulator_read();
          if (!there(c)) continue;
          if (pending) {
            if (!mbar_wait_warp(&bars->rows[warp - 2][0], nrows & 1u, p.limit)) {
              if (lane == 0) give_up();   // it goes on with what lands, and leaves at the next tile
              lost = !mbar_wait_warp(&bars->rows[warp - 2][0], nrows & 1u, LANDING_NS);
              if (lost) continue;
            }
            nrows ^= 1u;
          }
          step_finish<O, N>(p, maps, ibase + c, j0, triangle && ti != tj, buf, pending, reinterpret_cast<float*>(v));
        }
        if (lost) break;
      } else {
        // R of the chunk at buffer x or after it that has been asked for lands, so that the warp can leave
        const auto r_landed = [&](int x) {
          bool ok = true;
          for (; p.tma_r && j0 < p.J && x < 2; ++x)
            if (ibase + x * N < p.I) ok = mbar_wait_warp(&bars->rows[warp - 2][x], (nrows >> x) & 1u, LANDING_NS) && ok;
          return ok;
        };
        if (p.tma_r && j0 < p.J) {   // both chunks' R, before the wait for the products
          if (lane == 0) {
            tma_store_wait_read();
            for (int c = 0; c < 2; ++c)
              if (ibase + c * N < p.I) {
                mbar_arrive_expect_tx(&bars->rows[warp - 2][c], WBUF);
                tma_load_2d(buf + c * WSTAGE, &maps.R, &bars->rows[warp - 2][c], ibase + c * N, j0);
              }
          }
        }
        if (!mbar_wait_warp(&bars->tfull[b], (uint32_t)(u >> 1) & 1u, p.limit)) {
          if (lane == 0) give_up();
          r_landed(0);
          break;
        }
        tc_fence_after();
        const float js = p.e.jscale && j0 + lane < p.J ? p.e.jscale[j0 + lane] : 1.0f;
        for (int c = 0; c < 128; c += N) {
          uint32_t v[N / 32][32];
          float is[N / 32], bias[N / 32];
          load_row<N>(p.e.iscale, ibase + c, p.I, is);
          load_row<N>(p.e.bias, ibase + c, p.I, bias);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < N / 32; ++q) tmem_ld32(tq + (uint32_t)(c + 32 * q), v[q]);
          tmem_ld_wait();
          if (c + N == 128) accumulator_read();
          if (ibase + c >= p.I) continue;
          uint8_t* out = buf;
          const uint8_t* rows = nullptr;
          if (p.tma_r && j0 < p.J) {
            const int x = c / N;
            rows = out = buf + x * WSTAGE;
            if (!mbar_wait_warp(&bars->rows[warp - 2][x], (nrows >> x) & 1u, p.limit)) {
              if (lane == 0) give_up();   // it goes on with what lands, and leaves at the next tile
              if (!r_landed(x)) break;
            }
            nrows ^= 1u << x;
          }
          wide_finish<O, N>(p, &maps.C, &maps.Z, ibase + c, j0, js, is, bias, out, rows, reinterpret_cast<float*>(v));
        }
      }
    }
    if (lane == 0) tma_store_wait_read();
  }
  if (p.second) wait_for_previous();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // neither CTA leaves while the other's MMAs, copies or arrivals may reach it
  if (*abort_flag) {    // the same in both: operands in flight land too
    if (rank == 0 && warp == 0) {
      const int n0 = *(volatile int*)&bars->issued[0], n1 = *(volatile int*)&bars->issued[1], last = max(n0, n1);
      for (int n = max(last - p.stages, 0); n < last; ++n) {
        uint64_t* full = &bars->full[n % p.stages];
        if (lane == 0) {   // a stage that only one of the two has filled: the barrier waits for its half
          if (n >= n0) mbar_arrive_expect_tx(full, WSTAGE);
          else if (n >= n1) mbar_complete_tx(full, WSTAGE);
        }
        __syncwarp();
        mbar_wait_warp(full, (uint32_t)(n / p.stages) & 1u, LANDING_NS);
      }
    }
    __syncwarp();
    cluster_sync_all();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- thin kernel
// 128 outputs i x bn columns j per cluster (operand A = P, B = Q): few columns, where the product is
// bound by reading P (K = 4096, N = 12288, M = 16 FP16: 20 us, 5.0 TB/s).  The CTAs of a cluster take equal
// parts of k.  Each finishes 128 / split of the i: the others copy their partial sums for these into
// its shared memory in bulk, and it adds them in the order of the parts.
constexpr int TTHREADS = 192;
constexpr int TMAXSTAGES = 8;
struct ThinBars {
  uint64_t full[TMAXSTAGES], empty[TMAXSTAGES], done, got;
  uint32_t tmem;
  int abort;
};

// GATED: 64 outputs, the first 64 rows of the tile from P's first half and the others from its second; both sums of an
// output meet in shared memory.  STEP goes through it too, for accesses of four elements.
struct ThinMaps {
  CUtensorMap P, Q, P2, Q2;   // P2, Q2: STEP's second parts
};
template <int FORM, bool F8, class O>
__global__ void __launch_bounds__(TTHREADS) k_thin(const __grid_constant__ ThinMaps maps, const Params p, int split, int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int qbytes = p.qk ? p.bn * KBYTES : (p.bn + 63) / 64 * ATOM;
  const int stage_bytes = WTILE + qbytes;
  ThinBars* bars = reinterpret_cast<ThinBars*>(smem + stages * stage_bytes);
  volatile int* abort_flag = &bars->abort;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split, tile = blockIdx.x / split;
  constexpr int OUT = FORM == GATED ? 64 : 128;   // outputs i of a tile
  const int i0 = tile / p.tj * OUT, j0 = tile % p.tj * p.bn;
  const int kb0 = (int)((long long)p.kblocks * rank / split), kb1 = (int)((long long)p.kblocks * (rank + 1) / split);
  // STEP with two parts: four k-blocks at most to an accumulator, and two of them, so that the tensor cores' chains stay short
  const uint32_t bcols = p.bn <= 32 ? 32 : p.bn <= 64 ? 64 : p.bn <= 128 ? 128 : 256;
  const bool two_sums = FORM == STEP && p.segments == 3;
  const uint32_t cols = two_sums ? 2 * bcols : bcols;
  const int ncols = min(p.bn, p.J - j0);
  constexpr int KE = F8 ? 128 : 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->done, 1);
    mbar_init(&bars->got, 1);
    bars->abort = 0;
    fence_mbar_init();
    if (split > 1) mbar_arrive_expect_tx(&bars->got, 512u * (uint32_t)ncols);
  }
  if (warp == 1) tmem_alloc(&bars->tmem, cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);
  let_next_start();
  wait_for_previous();
  if (split > 1) cluster_arrive_relaxed();   // waited for before the first copy to another CTA
  // Partial sums in blocks of sb consecutive i, [block][column][sb]: this CTA's own ones in the
  // stages' memory once its MMAs are done, those that it receives, [part of k] of them, after the
  // barriers, because other CTAs may be done before this one's last MMA.
  // GATED: a CTA finishes OUT / split outputs, and has `own` sums for them.
  const int own = 128 / split, outs = OUT / split, sb = min(outs, 32);
  float* sent = reinterpret_cast<float*>(smem);
  float* received = reinterpret_cast<float*>(smem + stages * stage_bytes + 256);

  if (warp == 0) {
    if (elect_one()) {
      prefetch_tmap(&maps.P);
      prefetch_tmap(&maps.Q);
    }
    int st = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int per = FORM == STEP ? p.kblocks / p.segments : p.kblocks;   // k-blocks of a segment
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = mbar_wait_warp(&bars->empty[st], ph ^ 1u, p.limit);
      if (!ok) break;
      if (elect_one()) {
        uint8_t* sp = smem + st * stage_bytes;
        uint8_t* sq = sp + WTILE;
        mbar_arrive_expect_tx(&bars->full[st], stage_bytes);
        int kx = kb;
        const CUtensorMap *tmP = &maps.P, *tmQ = &maps.Q;
        if (FORM == STEP && p.segments == 3) {   // the small products first
          const int seg = kb / per;
          kx = kb - seg * per;
          if (seg == 1) tmP = &maps.P2;
          if (seg == 0) tmQ = &maps.Q2;
        }
        const int k0 = kx * KE;
        if (FORM == GATED) {
          tma_load_2d(sp, tmP, &bars->full[st], k0, i0);
          tma_load_2d(sp + ATOM, tmP, &bars->full[st], k0, p.I + i0);
        } else if (p.pk) {
          tma_load_2d(sp, tmP, &bars->full[st], k0, i0);
        } else {
          tma_load_2d(sp, tmP, &bars->full[st], i0, k0);
          tma_load_2d(sp + ATOM, tmP, &bars->full[st], i0 + 64, k0);
        }
        if (p.qk) {
          tma_load_2d(sq, tmQ, &bars->full[st], k0, j0);
        } else {
          for (int h = 0; h < qbytes / ATOM; ++h) tma_load_2d(sq + h * ATOM, tmQ, &bars->full[st], j0 + h * 64, k0);
        }
      }
      ++issued;
      if (++st == stages) st = 0, ph ^= 1u;
    }
    if (!ok && lane == 0) gave_up(p, abort_flag);
    for (int q = min(issued, stages); q > 0; --q) {   // copies land before the CTA leaves, whoever gave up
      const int n = issued - q;
      mbar_wait(&bars->full[n % stages], (uint32_t)(n / stages) & 1u, LANDING_NS);
    }
    __syncwarp();
    if (split > 1) cluster_wait();
  } else if (warp == 1) {
    if (kb1 > kb0) {
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint32_t ps = desc_step(p.pk), qs = desc_step(p.qk), s0 = smem_u32(smem);
      const uint64_t da0 = tile_desc(s0, p.pk), db0 = tile_desc(s0 + WTILE, p.qk);
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        ok = mbar_wait_warp(&bars->full[st], ph, p.limit);
        tc_fence_after();
        if (elect_one()) {
          if (ok) {
            const uint64_t da = da0 + (uint32_t)(st * stage_bytes >> 4), db = db0 + (uint32_t)(st * stage_bytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_any<false, F8>(two_sums && kb >= kb0 + 4 ? tmem + bcols : tmem, da + kk * ps, db + kk * qs, p.idesc,
                                 (kb != kb0 && !(two_sums && kb == kb0 + 4)) || kk != 0);
            mma_commit(&bars->empty[st]);
          }
          if (kb + 1 == kb1 || !ok) mma_commit(&bars->done);   // after giving up too: it completes once the issued MMAs have
        }
        __syncwarp();
        if (++st == stages) st = 0, ph ^= 1u;
      }
      if (!ok && lane == 0) gave_up(p, abort_flag);
    }
    __syncwarp();
    if (split > 1) cluster_wait();
  } else {
    const int f = (warp & 3) * 32 + lane, i = i0 + f;
    bool ok = true;
    if (kb1 > kb0) {
      ok = mbar_wait(&bars->done, 0, p.limit);
      if (!ok) {
        gave_up(p, abort_flag);
        mbar_wait(&bars->done, 0, LANDING_NS);   // MMAs in flight read the stages and write tensor memory
      }
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    if (split > 1) cluster_wait();
    const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float* to = sent + (size_t)(f / sb * ncols) * sb + f % sb;
    for (int c = 0; c < ncols; c += 16) {
      float v[16];
      __syncwarp();
      if (kb1 > kb0 && ok) {
        tmem_ld16(tq + (uint32_t)c, v);
        if (two_sums && kb1 > kb0 + 4) {
          float w[16];
          tmem_ld16(tq + bcols + (uint32_t)c, w);
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] += w[q];
        }
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = 0.0f;
      }
      if (FORM != AFFINE || split > 1) {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (c + q < ncols) to[(c + q) * sb] = v[q];
      } else if (i < p.I) {
        thin_store16<O>(p, i, j0 + c, v);
      }
    }
    if (split > 1) {
      fence_smem_to_tma();
      __syncwarp();
      const int f0 = (warp & 3) * 32 + lane * sb;   // lanes 0 .. 32 / sb - 1 send one block each
      if (lane < 32 / sb) {
        const int side = f0 / OUT * outs, g0 = f0 % OUT;   // GATED: after the first half's sums, the second half's
        const uint32_t owner = (uint32_t)(g0 / outs), bytes = 4u * (uint32_t)(ncols * sb);
        const uint32_t at = (uint32_t)(rank * own + side + g0 % outs) / (uint32_t)sb * bytes;
        copy_to_cluster(cluster_addr(smem_u32(received), owner) + at, sent + (size_t)(f0 / sb * ncols) * sb, bytes,
                        cluster_addr(smem_u32(&bars->got), owner));
      }
    }
  }
  if (FORM != AFFINE || split > 1) {
    bool got = true;
    const float* parts = received;
    if (split > 1) {
      got = mbar_wait(&bars->got, 0, p.limit);
      if (!got) {
        gave_up(p, abort_flag);
        mbar_wait(&bars->got, 0, LANDING_NS);   // every CTA of the cluster sends, whatever became of its sums
      }
    } else {
      parts = sent;
      __syncthreads();
    }
    const int total = ncols * own, outputs = ncols * outs;
    const auto joined = [&](int e) {
      float4 z = *reinterpret_cast<const float4*>(parts + e);
      for (int r = 1; r < split; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(parts + r * total + e);
        z.x += x.x;
        z.y += x.y;
        z.z += x.z;
        z.w += x.w;
      }
      return z;
    };
    const auto place = [&](int e, int& i, int& j) {
      const int block = e / (ncols * sb), in = e - block * ncols * sb;
      i = i0 + rank * outs + block * sb + in % sb;
      j = j0 + in / sb;
    };
    if constexpr (FORM == STEP) {   // R of four outputs' eights on its way at once: stores to C hold up later loads
      constexpr int U = 4;
      for (int e0 = 4 * (int)threadIdx.x; got && e0 < outputs; e0 += U * 4 * TTHREADS) {
        StepR r[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int e = e0 + k * 4 * TTHREADS;
          int i, j;
          place(e, i, j);
          if (e < outputs) r[k] = step_r(p, i, j);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int e = e0 + k * 4 * TTHREADS;
          if (e >= outputs) break;
          int i, j;
          place(e, i, j);
          const float4 z = joined(e);
          float v[4] = {z.x, z.y, z.z, z.w};
          finish_step4<O>(p, i, j, r[k], v);
        }
      }
    } else {
      for (int e = 4 * (int)threadIdx.x; got && e < outputs; e += 4 * TTHREADS) {
        const float4 z = joined(e);
        int i, j;
        place(e, i, j);
        float v[4] = {z.x, z.y, z.z, z.w};
        if constexpr (FORM == GATED) {
          const float4 y = joined(outputs + e);
          float w[4] = {y.x, y.y, y.z, y.w};
          finish_gated4<O>(p, i, j, v, w);
        } else {
          thin_finish4<O>(p, i, j, v);
        }
      }
    }
    __syncwarp();
    if (split > 1) cluster_sync_all();   // copies read this CTA's memory until their receivers have them
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

// ---------------------------------------------------------------- one column
// One warp per output i, one column: P is read once, straight into registers, with no shared-memory
// pipeline, tensor memory or cluster to set up (K = N = 2048 BF16: 3.6 us a call in a row, the thin kernel
// 4.3 us; launched to overlap with the previous kernel it takes 6.6 us).  With two columns reading Q again
// for each output costs more than that (5.1 us), and with more outputs than resident warps a
// second round does (K = 4096, N = 12288: 28.6 us, the thin kernel 18.3 us).  V = 16 / sizeof(E)
// elements at a time where P and Q are aligned, else one.
template <class E, int V>
__device__ __forceinline__ void widen(const E* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_float(*p);
  } else if constexpr (sizeof(E) == 2) {
    widen8(*reinterpret_cast<const Eight<E>*>(p), v);
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[q / 2] >> (16 * (q & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * q] = f.x;
      v[2 * q + 1] = f.y;
    }
  }
}
template <int FORM, class E, class O, int V>
__global__ void __launch_bounds__(NT) k_one(const E* P, int ldp, const E* Q, int K, const Params p) {
  const int lane = threadIdx.x & 31, i = blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
  if (i >= p.I) return;
  const E* row = P + (size_t)i * ldp;
  const E* row2 = FORM == GATED ? row + (size_t)p.I * ldp : nullptr;
  float s = 0.0f, s2 = 0.0f;
#pragma unroll 4
  for (int k = lane * V; k < K; k += 32 * V) {
    float w[V], w2[V], x[V];
    widen<E, V>(row + k, w);
    if (FORM == GATED) widen<E, V>(row2 + k, w2);
    widen<E, V>(Q + k, x);
#pragma unroll
    for (int q = 0; q < V; ++q) {
      s = fmaf(w[q], x[q], s);
      if (FORM == GATED) s2 = fmaf(w2[q], x[q], s2);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    if (FORM == GATED) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
  }
  if (lane == 0) {
    if (FORM == GATED) finish_gated<O>(p, i, 0, s, s2);
    else finish<O>(p, i, 0, s);
  }
}

// Copies a matrix whose columns of n elements start at any address into columns ld apart on 16-byte
// boundaries: a thread stores 16 bytes at once (elements past n are zero).  It reads them as the 4-byte words
// that they lie in, shifted into place, and element by element where a word would reach past the column's end
// or the matrix's ends.  Bound by the narrow loads and the copy's own traffic: K = 4095, N = 8192, M = 4096 BF16
// takes 183 us, K = 4096 138 us (element by element 190 us).
template <class E>
__global__ void __launch_bounds__(NT) k_pack(const E* src, int lds, int n, int m, E* dst, int ld) {
  constexpr int V = 16 / (int)sizeof(E);
  struct alignas(16) Word {
    E x[V];
  };
  const int per = ld / V;
  const uintptr_t begin = (uintptr_t)src, end = (uintptr_t)(src + (size_t)(m - 1) * lds + n);
  for (long long e = (long long)blockIdx.x * NT + threadIdx.x; e < (long long)per * m; e += (long long)gridDim.x * NT) {
    const size_t c = e >> 32 ? (size_t)(e / per) : (uint32_t)e / (uint32_t)per;
    const int i = (int)(e - (long long)c * per) * V;
    const E* from = src + c * lds + i;
    const uintptr_t a = (uintptr_t)from, first = a & ~(uintptr_t)3;
    if (i + V <= n && first >= begin && first + 20 <= end) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(first);
      uint32_t w[5];
#pragma unroll
      for (int q = 0; q < 5; ++q) w[q] = p[q];
      const uint32_t shift = (uint32_t)(a & 3) * 8;
      *reinterpret_cast<uint4*>(dst + c * ld + i) =
          make_uint4(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift), __funnelshift_r(w[2], w[3], shift),
                     __funnelshift_r(w[3], w[4], shift));
    } else {
      Word w;
#pragma unroll
      for (int q = 0; q < V; ++q) w.x[q] = i + q < n ? from[q] : E(0);
      *reinterpret_cast<Word*>(dst + c * ld + i) = w;
    }
  }
}

// An operand as TMA can read it: a 16-byte aligned base and leading dimension, copied into
// scratch where the caller's is not.
struct Packed {
  void* own = nullptr;
  cudaStream_t stream = nullptr;
  ~Packed() { scratch_free(own, stream); }
  cr_status make(Operand& o, int type, int K, cudaStream_t s) {
    const int eb = type_bytes(type);
    if (((uintptr_t)o.ptr & 15) == 0 && (long long)o.ld * eb % 16 == 0) return CR_OK;
    stream = s;
    const int n = o.k_major ? K : o.rows, m = o.k_major ? o.rows : K;
    const int ld = (int)(((long long)n * eb + 15) / 16 * 16 / eb);
    CR_CUDA(scratch_alloc(&own, (size_t)ld * m * eb, s));
    const long long words = (long long)ld * eb / 16 * m;
    const unsigned grid = (unsigned)std::min<long long>((words + NT - 1) / NT, 8 * sm_count());
    if (eb == 2) k_pack<uint16_t><<<grid, NT, 0, s>>>((const uint16_t*)o.ptr, o.ld, n, m, (uint16_t*)own, ld);
    else k_pack<uint8_t><<<grid, NT, 0, s>>>((const uint8_t*)o.ptr, o.ld, n, m, (uint8_t*)own, ld);
    CR_CHECK_LAUNCH("k_pack");
    o.ptr = own;
    o.ld = ld;
    return CR_OK;
  }
};

cr_status map_of(CUtensorMap* tm, const Operand& o, int type, int K, int rows_per_box) {
  if (o.k_major) return make_tensor_map_2d(tm, type, o.ptr, K, o.rows, o.ld, KBYTES / type_bytes(type), rows_per_box);
  return make_tensor_map_2d(tm, type, o.ptr, o.rows, K, o.ld, 64, 64);
}

template <int FORM>
struct Names {
  static constexpr const char* wide = FORM == AFFINE ? "k_affine_wide" : FORM == GATED ? "k_gated_wide" : "k_ortho_wide";
  static constexpr const char* thin = FORM == AFFINE ? "k_affine_thin" : FORM == GATED ? "k_gated_thin" : "k_ortho_thin";
  static constexpr const char* one = FORM == GATED ? "k_gated_one" : "k_affine_one";
};

template <int FORM, bool F8, class O>
cr_status launch_wide(const Maps<FORM>& maps, const Params& p, long long tiles, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  CR_TRY(allow_shared((const void*)k_wide<FORM, F8, O>, WSMEM, done));
  const int pairs = std::min((long long)sm_count() / 2, tiles);
  TimedScope ts(Names<FORM>::wide, stream);
  CR_CUDA(launch_after(k_wide<FORM, F8, O>, 2 * pairs, wide_threads(FORM), WSMEM, 2, stream, maps, p));
  CR_CHECK_LAUNCH(Names<FORM>::wide);
  return CR_OK;
}

template <int FORM, bool F8, class O>
cr_status launch_thin(const ThinMaps& maps, const Params& p, int split, int stages, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  CR_TRY(allow_shared((const void*)k_thin<FORM, F8, O>, 227 * 1024, done));
  const int stage = WTILE + (p.qk ? p.bn * KBYTES : (p.bn + 63) / 64 * ATOM);
  const size_t smem = (size_t)stages * stage + 1024 + 256 + (split > 1 ? 512 * p.bn : 0);
  TimedScope ts(Names<FORM>::thin, stream);
  CR_CUDA(launch_after(k_thin<FORM, F8, O>, (unsigned)((long long)p.ti * p.tj * split), TTHREADS, smem, split, stream, maps, p, split,
                       stages));
  CR_CHECK_LAUNCH(Names<FORM>::thin);
  return CR_OK;
}

// Clusters of s CTAs that are resident at once with c CTAs per SM: fewer than SMs x c / s (15 of 8, 36 of 4
// on a GB300's 152 SMs), because a cluster's CTAs share a GPC.
template <int FORM>
int resident_clusters(int s, int c) {
  struct Table {
    std::once_flag once;
    int n[4] = {};
    void fill() {
      const auto kernel = k_thin<FORM, false, __half>;
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
      for (int e = 0; e < 4; ++e) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 1 << e;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(4096 << e);
        cfg.blockDim = dim3(TTHREADS);
        cfg.dynamicSmemBytes = 200 * 1024;   // one CTA per SM
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n[e], kernel, &cfg) != cudaSuccess) {
          cudaGetLastError();
          n[e] = sm_count() / (1 << e);
        }
      }
    }
  };
  static Table tables[64];   // by device
  int dev = 0;
  cudaGetDevice(&dev);
  Table& table = tables[dev & 63];
  std::call_once(table.once, [&] { table.fill(); });
  return c * table.n[s == 1 ? 0 : s == 2 ? 1 : s == 4 ? 2 : 3];
}

// Which kernel, with which tiles.  Times in microseconds from the rates measured on GB300 (K = 1024 to
// 8192, N = 1024 to 16384, M = 1 to 8192); the choice only has to be right where they differ.
struct Choice {
  bool wide;
  int bn, split, stages;
  double us;
  int parts = 0;   // wide, of the FORM STEP: by way of SUMS, over so many parts of k
};
// sums: a STEP with two parts, whose wide form is SUMS and whose thin one is for short sums.
template <int FORM>
Choice choose(int I, int J, int kblocks, bool qk, bool triangle = false, bool sums = false) {
  Choice best = {false, 0, 1, 0, 1e30};
  const int sms = sm_count();
  const auto tiles = [](int n, int t) { return (n + t - 1) / t; };
  // Wide: rounds of tiles over the CTA pairs, 0.27 to 0.3 us per k-block, or the epilogue of a tile.
  if (J > 128 || sums) {
    const long long n = tiles(J, 256), t = triangle ? n * (n + 1) / 2 : tiles(I, 256) * n, rounds = (t + sms / 2 - 1) / (sms / 2);
    best = {true, 0, 1, 0, 6.5 + rounds * std::max(kblocks * 0.29 + 0.6, 3.3)};
    // By way of SUMS: tiles over parts of k, which cost a launch and the way of every part's sums through L2.
    for (int parts = 1; FORM == STEP && parts <= 16 && (parts == 1 || kblocks >= 4 * parts); ++parts) {
      const double r = (double)((t * parts + sms / 2 - 1) / (sms / 2));
      const bool joined = parts > 1 || triangle;
      const double us = (joined ? 11.0 : 8.0) + r * std::max(tiles(kblocks, parts) * 0.29 + 0.6, 2.0) +
                        (joined ? 1.2e-6 * parts * I * J * (triangle ? 0.5 : 1.0) : 0.0);
      if (us < best.us || (sums && parts == 1)) best = {true, 0, 1, 0, us, parts};
    }
  }
  // Thin: parts of k for which all clusters are resident at once, with three stages or more and two
  // k-blocks or more for each CTA; a second wave of CTAs costs more than longer parts (K = 4096,
  // N = 12288, M = 16 FP16: 96 CTAs with 8 stages 23.5 us, 192 with 4 22.2 us, 384 with 3 20.8 us, 384
  // with 4, no longer resident at once, 25.8 us).  An SM takes in about 100 KB per microsecond, HBM
  // gives less to fewer CTAs, joining the parts costs 1 us at 16 columns, 5 at 128, and so, nearly, does
  // the epilogue of each tile that has to wait for an SM (K = 64, N = 8192, M = 4096 BF16 with
  // bias and silu: thin 59 us, wide 34 us).
  for (int bn = J <= 16 ? 16 : J <= 32 ? 32 : 64; bn <= (J > 64 ? 128 : 64); bn *= 2) {
    const int stage = WTILE + (qk ? bn * KBYTES : (bn + 63) / 64 * ATOM);
    const long long t = (long long)tiles(I, 128) * tiles(J, bn);
    for (int split = 8; split >= 1; split /= 2) {
      if (split > 1 && kblocks < 2 * split) continue;
      if (sums && tiles(kblocks, split) > 8) continue;
      int per = 1;
      while (per < 3 && t > resident_clusters<FORM>(split, per)) ++per;
      if (t > resident_clusters<FORM>(split, per)) {
        if (split > 1) continue;
        per = 2;
      }
      const int received = split > 1 ? 512 * bn : 0;
      const int stages = std::min(TMAXSTAGES, (227 * 1024 / per - 3584 - received) / stage);
      if (stages < (split > 1 ? 3 : 2) || (split > 1 && stages * stage < received)) continue;
      const double ctas = (double)t * split;
      const double waves = std::max(1.0, ctas / sms);
      const double hbm = (double)I * kblocks * KBYTES / 5.5e6 * (1.0 + 0.25 * std::max(0.0, 1.0 - ctas / (2.5 * sms)));
      const double later = std::max(0.0, ctas / sms - per) * 0.025 * bn;   // epilogues of tiles after the resident ones
      // STEP: a CTA's outputs by four, R read with them, are what takes long (five steps of 1400 x 1400 without this term 293 us,
      // 238 with it; 700 x 2500 175 and 152; 512 x 512 124 and 114; 1000 x 1000 177 and 203).
      const double ends = FORM == STEP ? 0.047 * bn / split + (split > 1 ? 0.02 * bn : 0.0) : split > 1 ? 0.3 + 0.04 * bn : 0.0;
      const double us = 5.0 + later + ends + std::max(waves * tiles(kblocks, split) * stage / 100e3, hbm);
      if (us < best.us) best = {false, bn, split, stages, us};
    }
    if (J <= 64) break;
  }
  return best;
}

template <int FORM, class E, class O>
cr_status one_column(const Operand& P, const Operand& Q, int K, const Params& p, cudaStream_t stream) {
  const E *a = (const E*)P.ptr, *b = (const E*)Q.ptr;
  constexpr int V = 16 / (int)sizeof(E);
  const bool vec = (((uintptr_t)a | (uintptr_t)b) & 15) == 0 && P.ld % V == 0 && K % V == 0;
  const unsigned grid = (unsigned)((p.I + NT / 32 - 1) / (NT / 32));
  TimedScope ts(Names<FORM>::one, stream);
  if (vec) k_one<FORM, E, O, V><<<grid, NT, 0, stream>>>(a, P.ld, b, K, p);
  else k_one<FORM, E, O, 1><<<grid, NT, 0, stream>>>(a, P.ld, b, K, p);
  CR_CHECK_LAUNCH(Names<FORM>::one);
  return CR_OK;
}

// The AFFINE and GATED forms' product; GATED: P has 2 I rows.
template <int FORM>
cr_status product(Operand P, Operand Q, int type, int K, int out_type, const Epilogue& e, int* err, cudaStream_t stream, First* first = nullptr) {
  static_assert(FORM == AFFINE || FORM == GATED, "");
  Params p = {};
  p.err = err;
  p.limit = option_wait_ns();
  p.I = FORM == GATED ? P.rows / 2 : P.rows;
  p.J = Q.rows;
  p.e = e;
  p.pk = P.k_major;
  p.qk = Q.k_major;
  p.segments = 1;
  const int ke = KBYTES / type_bytes(type), ob = type_bytes(out_type);
  p.kblocks = (K + ke - 1) / ke;
  const auto ok16 = [&](const void* q, int ld) { return !q || (((uintptr_t)q & 15) == 0 && (long long)ld * ob % 16 == 0); };
  p.tma_c = ok16(e.C, e.ldc);
  p.tma_z = ok16(e.Z, e.ldz) && (FORM == AFFINE || (long long)p.I * ob % 16 == 0);
  p.vec_r = ok16(e.R, e.ldr);
  const auto ok4 = [&](const void* q, int ld) { return !q || (((uintptr_t)q & (4 * ob - 1)) == 0 && ld % 4 == 0); };
  p.vec4 = (((uintptr_t)e.bias | (uintptr_t)e.iscale) & 15) == 0 && ok4(e.C, e.ldc) && ok4(e.R, e.ldr) && ok4(e.Z, e.ldz) &&
           (FORM == AFFINE || p.I % 4 == 0);
  if (p.J == 1 && p.pk && p.qk && p.I <= 64 * sm_count())   // one round of warps
    return with_type(out_type, [&](auto o0) -> cr_status {
      using O = decltype(o0);
      if (type == CR_TYPE_F16) return one_column<FORM, __half, O>(P, Q, K, p, stream);
      if (type == CR_TYPE_BF16) return one_column<FORM, __nv_bfloat16, O>(P, Q, K, p, stream);
      return one_column<FORM, __nv_fp8_e4m3, O>(P, Q, K, p, stream);
    });
  Packed ownP, ownQ;
  CR_TRY(ownP.make(P, type, K, stream));
  CR_TRY(ownQ.make(Q, type, K, stream));
  const Choice ch = choose<FORM>(P.rows, p.J, p.kblocks, p.qk);
  const bool wide = ch.wide, bf16 = type == CR_TYPE_BF16;
  const int rows = (FORM == GATED ? 64 : 128) * (wide ? 2 : 1);   // outputs i of a tile
  p.bn = ch.bn;
  p.ti = (p.I + rows - 1) / rows;
  p.tj = wide ? (p.J + 255) / 256 : (p.J + p.bn - 1) / p.bn;
  p.idesc = wide ? idesc_of(256, 256, bf16, !p.qk, !p.pk) : idesc_of(128, p.bn, bf16, !p.pk, !p.qk);
  p.tma_r = wide && e.R && ob == 2 && p.tma_c && !e.Z && p.vec_r;   // with Z the buffer is in use before R is added
  p.stages = p.tma_r ? WSTAGES - 1 : WSTAGES;
  if (first) {
    const bool alone = wide && !ownP.own && !ownQ.own;   // nothing runs between the two
    const long long pairs = sm_count() / 2, tiles = (long long)p.ti * p.tj;
    p.second = alone && first->tiles > 0;
    if (p.second) {
      p.early = (int)std::min({(pairs - first->tiles % pairs) % pairs, pairs, tiles});
      p.ahead = (2 * first->kblocks + p.kblocks) / (2 * p.kblocks);   // to the nearest
    }
    *first = {alone ? tiles : 0, p.kblocks};
  }
  if (!wide) {
    ThinMaps maps = {};
    CR_TRY(map_of(&maps.P, P, type, K, FORM == GATED ? 64 : 128));
    CR_TRY(map_of(&maps.Q, Q, type, K, p.bn));
    return with_type(out_type, [&](auto o0) -> cr_status {
      using O = decltype(o0);
      return type == CR_TYPE_E4M3 ? launch_thin<FORM, true, O>(maps, p, ch.split, ch.stages, stream)
                                  : launch_thin<FORM, false, O>(maps, p, ch.split, ch.stages, stream);
    });
  }
  Maps<FORM> maps = {};
  CR_TRY(map_of(&maps.P, P, type, K, 128));
  CR_TRY(map_of(&maps.Q, Q, type, K, 128));
  if (p.tma_c) CR_TRY(make_tensor_map_2d(&maps.C, out_type, e.C, p.I, p.J, e.ldc, OROW / ob, 32));
  if (e.Z && p.tma_z) CR_TRY(make_tensor_map_2d(&maps.Z, out_type, e.Z, p.I, p.J, e.ldz, OROW / ob, 32));
  if constexpr (FORM == AFFINE) {
    if (p.tma_r) CR_TRY(make_tensor_map_2d(&maps.R, out_type, e.R, p.I, p.J, e.ldr, KBYTES / ob, 32));
  } else {
    if (e.Z && p.tma_z) CR_TRY(make_tensor_map_2d(&maps.Z2, out_type, (const uint8_t*)e.Z + (size_t)p.I * ob, p.I, p.J, e.ldz, OROW / ob, 32));
  }
  return with_type(out_type, [&](auto o0) -> cr_status {
    using O = decltype(o0);
    const long long tiles = (long long)p.ti * p.tj;
    return type == CR_TYPE_E4M3 ? launch_wide<FORM, true, O>(maps, p, tiles, stream) : launch_wide<FORM, false, O>(maps, p, tiles, stream);
  });
}

}  // namespace
}  // namespace cr
