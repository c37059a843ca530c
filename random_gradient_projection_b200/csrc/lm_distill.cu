// Distillation from a teacher's top logits, loss and gradient in one pass over the student's
// logits.  Per row n with student logits z (V of them) and the teacher's entries (idx_k, val_k):
//
//   q   = softmax over the row's entries with idx in [0, V) of val / tau
//   p   = softmax over V of z / tau
//   l_n = w_n tau^2 sum_k q_k (log q_k - log p_{idx_k})
//   Gout_nv = dl_n / dz_v = w_n tau (p_v - sum_{k : idx_k = v} q_k)
//
// Bound by memory where it is fast: z is read from DRAM once and Gout written once (2 V elements a
// row).  Statistics are fp32: each thread keeps a running maximum and sum, joined over the CTA once;
// Gout is rounded once, as it is written.  Gout may be the logits themselves: every thread rewrites
// only what it has read, and the teacher's entries are read before the first store of their row.
// Two kernels: distill_kernel, a row per CTA, which holds the first part of its row in registers
// between the statistics and the gradient and takes the rest again from L2; and, for long rows,
// distill_rows_kernel, which streams rows through shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "lm.h"
#include "lm_launch.h"
#include "lm_ptx.cuh"

namespace grape {
namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <class T>
struct Unit;   // one 16-byte load
template <>
struct Unit<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Unit<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void put_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A running maximum m and the sum s of 2^((x - m) scale) over the values x so far.  Differences are
// taken before they are scaled: a logit at the type's lowest value stays finite.  The reference
// of a sum whose values are all -inf is 0, so that they count 0 rather than NaN.
struct Running {
  float m = -INFINITY, s = 0.0f;
  static __device__ __forceinline__ float ref(float m) { return m == -INFINITY ? 0.0f : m; }
  __device__ __forceinline__ void join(float m2, float s2, float scale) {
    const float mm = fmaxf(m, m2), r = ref(mm);
    // an empty side has s = 0 and m = -inf: 2^(-inf) = 0
    s = s * ex2((m - r) * scale) + s2 * ex2((m2 - r) * scale);
    m = mm;
  }
};

// Two floats in a register pair, and the instructions that work on both: the arithmetic on rows is
// bound by instruction issue.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t r) {
  float2 x;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(r));
  return x;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^((v - ref) scale) of the elements of a unit, as pairs.  The difference comes first, as everywhere
// in this file: it is exact for logits near their reference however large both are, and the same for
// every exponent that meets another one (fma(v, scale, -ref scale) saves an instruction a pair, but
// leaves the rounding of ref scale in every exponent: 4e-5 relative at |ref| / tau = 1000, and
// NaN at 1e10).
template <class T>
__device__ __forceinline__ void exps(const uint4& raw, float ref, float scale, uint64_t (&e)[Unit<T>::kN / 2]) {
  float v[Unit<T>::kN];
  Unit<T>::get(raw, v);
  const uint64_t c = pair(scale, scale), r = pair(-ref, -ref);
#pragma unroll
  for (int i = 0; i < Unit<T>::kN / 2; ++i) {
    const float2 x = unpair(mul2(add2(pair(v[2 * i], v[2 * i + 1]), r), c));
    e[i] = pair(ex2(x.x), ex2(x.y));
  }
}
template <class T>
__device__ __forceinline__ float sum_of(uint64_t (&e)[Unit<T>::kN / 2]) {
#pragma unroll
  for (int o = 1; o < Unit<T>::kN / 2; o <<= 1)
#pragma unroll
    for (int i = 0; i + o < Unit<T>::kN / 2; i += 2 * o) e[i] = add2(e[i], e[i + o]);
  const float2 x = unpair(e[0]);
  return x.x + x.y;
}
// f times the pairs, as a unit.
template <class T>
__device__ __forceinline__ uint4 scaled(const uint64_t (&e)[Unit<T>::kN / 2], float f) {
  float v[Unit<T>::kN];
#pragma unroll
  for (int i = 0; i < Unit<T>::kN / 2; ++i) {
    const float2 x = unpair(mul2(e[i], pair(f, f)));
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
  return Unit<T>::put(v);
}
// The largest element of a unit.
__device__ __forceinline__ float unit_max(const uint4& r, float) {
  return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
}
__device__ __forceinline__ float unit_max(const uint4& r, __nv_bfloat16) {
  auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  const __nv_bfloat162 m = __hmax2(__hmax2(h(r.x), h(r.y)), __hmax2(h(r.z), h(r.w)));
  return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
}
// A unit of nothing but -inf.
__device__ __forceinline__ uint4 unit_of(uint32_t w) { return make_uint4(w, w, w, w); }
__device__ __forceinline__ uint4 unit_none(float) { return unit_of(0xff800000u); }
__device__ __forceinline__ uint4 unit_none(__nv_bfloat16) { return unit_of(0xff80ff80u); }

struct DistillParams {
  const void* idx;
  const void* val;
  const float* weights;
  float* loss;
  int64_t N;
  int V, K, id_bytes, val_f32;
  float tau, scale;   // scale = log2(e) / tau: exponents are taken in base 2
};

// CACHE 16-byte units per thread stay in registers.
template <class T, int THREADS, int CACHE, int MINB>
__global__ void __launch_bounds__(THREADS, MINB) distill_kernel(const DistillParams p, const T* logits, T* Gout) {
  constexpr int kN = Unit<T>::kN, kWarps = THREADS / 32;
  extern __shared__ float dyn[];   // [K] q (then the summed mass), [K] z, [K] idx
  __shared__ float red[kWarps][4];
  __shared__ float kl_red[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* sq = dyn;
  float* sz = dyn + p.K;
  int* si = reinterpret_cast<int*>(dyn + 2 * p.K);

  const int64_t row = blockIdx.x;
  const T* z = logits + row * p.V;
  T* g = Gout + row * p.V;
  const float w = p.weights ? p.weights[row] : 1.0f;
  // 16-byte units [a, b) of the row; `head` elements before them and `rest` after (a row of an odd
  // length starts anywhere; Gout has the same alignment, both bases being 16-byte aligned)
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
  const int head = min(p.V, mis ? kN - mis : 0);
  const int units = (p.V - head) / kN;
  const int rest0 = head + units * kN;
  // the elements outside the units: at most one per thread
  const int edge = tid < head ? tid : (tid >= 32 && rest0 + tid - 32 < p.V ? rest0 + tid - 32 : -1);
  const uint4* zu = reinterpret_cast<const uint4*>(z + head);
  uint4* gu = reinterpret_cast<uint4*>(g + head);

  // the teacher's entries
  Running t;
  if (w != 0.0f)
    for (int k = tid; k < p.K; k += THREADS) {
      const int64_t at = row * p.K + k;
      const int64_t i = p.id_bytes == 8 ? static_cast<const long long*>(p.idx)[at]
                                        : static_cast<int64_t>(static_cast<const int*>(p.idx)[at]);
      const bool in = i >= 0 && i < p.V;
      const float v = in ? (p.val_f32 ? static_cast<const float*>(p.val)[at]
                                      : as_f32(static_cast<const __nv_bfloat16*>(p.val)[at]))
                         : -INFINITY;
      si[k] = in ? static_cast<int>(i) : -1;
      sq[k] = v;
      sz[k] = in ? as_f32(z[i]) : 0.0f;
      if (in) t.join(v, v == -INFINITY ? 0.0f : 1.0f, p.scale);
    }
  if (__syncthreads_or(w != 0.0f && t.s != 0.0f) == 0) {
    // no weight, or no teacher: the row has no loss (its logits may hold anything)
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int u = tid; u < units; u += THREADS) gu[u] = zero;
    if (edge >= 0) put_f32(g + edge, 0.0f);
    if (tid == 0) p.loss[row] = 0.0f;
    return;
  }

  // ---- statistics of the student's row ------------------------------------------------------------
  uint4 cache[CACHE];
  const float ze = edge >= 0 ? as_f32(z[edge]) : -INFINITY;
#pragma unroll
  for (int c = 0; c < CACHE; ++c) {
    const int u = tid + c * THREADS;
    if (u < units) cache[c] = zu[u];
  }
  Running st;
  {
    float m = ze;
#pragma unroll
    for (int c = 0; c < CACHE; ++c)
      if (tid + c * THREADS < units) {
        float v[kN];
        Unit<T>::get(cache[c], v);
#pragma unroll
        for (int i = 0; i < kN; ++i) m = fmaxf(m, v[i]);
      }
    const float r = Running::ref(m);
    float s = ex2((ze - r) * p.scale);
#pragma unroll
    for (int c = 0; c < CACHE; ++c)
      if (tid + c * THREADS < units) {
        float v[kN];
        Unit<T>::get(cache[c], v);
#pragma unroll
        for (int i = 0; i < kN; ++i) s += ex2((v[i] - r) * p.scale);
      }
    st.m = m;
    st.s = s;
  }
  for (int u = tid + CACHE * THREADS; u < units; u += THREADS) {
    float v[kN];
    Unit<T>::get(zu[u], v);
    float m = v[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) m = fmaxf(m, v[i]);
    const float r = Running::ref(m);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) s += ex2((v[i] - r) * p.scale);
    st.join(m, s, p.scale);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    st.join(__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o), p.scale);
    t.join(__shfl_xor_sync(0xffffffffu, t.m, o), __shfl_xor_sync(0xffffffffu, t.s, o), p.scale);
  }
  if (lane == 0) {
    red[warp][0] = st.m;
    red[warp][1] = st.s;
    red[warp][2] = t.m;
    red[warp][3] = t.s;
  }
  __syncthreads();
  Running a, b;   // the row's student and teacher, the same in every thread
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    a.join(red[k][0], red[k][1], p.scale);
    b.join(red[k][2], red[k][3], p.scale);
  }
  const float ra = a.m;   // -inf for a row of -inf only, which gives NaN as the formula does
  const float gs = w * p.tau, f = gs / a.s;

  // ---- the gradient without the teacher's mass ---------------------------------------------------
  auto grad = [&](float x) { return f * ex2((x - ra) * p.scale); };
#pragma unroll
  for (int c = 0; c < CACHE; ++c) {
    const int u = tid + c * THREADS;
    if (u < units) {
      float v[kN];
      Unit<T>::get(cache[c], v);
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = grad(v[i]);
      gu[u] = Unit<T>::put(v);
    }
  }
  for (int u = tid + CACHE * THREADS; u < units; u += THREADS) {
    float v[kN];
    Unit<T>::get(zu[u], v);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = grad(v[i]);
    gu[u] = Unit<T>::put(v);
  }
  if (edge >= 0) put_f32(g + edge, grad(ze));

  // ---- the teacher's entries: loss, and their places of the gradient ------------------------------
  const float lse2 = log2f(a.s), tb = Running::ref(b.m), tl = log2f(b.s);
  float kl = 0.0f;
  for (int k = tid; k < p.K; k += THREADS) {
    const float lq = (sq[k] - tb) * p.scale - tl;   // log2 q
    const float q = si[k] >= 0 ? ex2(lq) : 0.0f;
    if (!(q == 0.0f)) kl += q * (lq - ((sz[k] - ra) * p.scale - lse2));
    sq[k] = q;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) kl += __shfl_xor_sync(0xffffffffu, kl, o);
  if (lane == 0) kl_red[warp] = kl;
  __syncthreads();   // also: the stores above come before those below
  for (int k = tid; k < p.K; k += THREADS) {
    const int i = si[k];
    if (i < 0) continue;
    float mass = 0.0f;
    bool mine = true;   // the first of equal indices writes, with the mass of all of them
    for (int j = 0; j < p.K; ++j)
      if (si[j] == i) {
        mass += sq[j];
        mine = mine && j >= k;
      }
    if (mine) put_f32(g + i, gs * (ex2((sz[k] - ra) * p.scale) / a.s - mass));
  }
  if (tid == 0) {
    float tot = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) tot += kl_red[k];
    p.loss[row] = w * p.tau * p.tau * 0.69314718055994531f * tot;
  }
}

// ---- long rows: streamed through shared memory ------------------------------------------------
// A CTA takes rows in turn and moves them through a ring of slots of 16 or 24 KB in shared memory, one
// bulk copy per slot each way.  Sixteen or twenty-four warps do the arithmetic in place, in two
// passes over the row's chunks: maximum and sum as they arrive, then the gradient, chunk by chunk,
// after which a chunk is stored and its slot loaded with the next row's data.  So memory does not wait for the
// exponentials (two per element: for bf16 their unit alone takes 0.8 of the row's time on the bus)
// nor for the reductions.  Bound by instruction issue (2.7 a cycle of an SM), next to memory: 4096 x
// 50265 bf16 takes 170 us (4.8 TB/s), 8192 x 128000 850-870 (4.9 TB/s), 4096 x 50265 fp32 288-299
// (5.6 TB/s).  A row longer than the ring has its first chunks loaded twice, the second time from
// L2; otherwise DRAM and L2 see every logit once and every gradient once.
// Rows are dealt out by their number, whatever their weights: where many have none, the CTA with the
// most live rows decides (4096 x 50265 with 15 / 50 / 90 % of the rows masked at random: 167 / 140 / 98 us).
// Four warps work on the teacher's entries: they prepare the next row's while a row is summed, and put
// their mass into each finished chunk before it is stored.  Two threads issue the copies, each those
// of every other slot: waiting until a slot has been read out takes a microsecond, which one thread
// alone could not hide.
//
// Chunks of a row in the order of their slots: its n chunks, then (n > kSlots) the first
// over = n - kSlots of them again.  Slots come free in the same order: an `over` chunk after the
// first pass, every other one when its gradient has been stored.
constexpr int kTeachThreads = 128, kCopyWarps = 2;
constexpr int kRowTeacher = kTeachThreads;   // entries of a row at most: one per thread
constexpr int kStatRing = 16;
constexpr uint64_t kWaitNs = 4000000000ull;
// MINB CTAs on an SM: threads that do the arithmetic, 16-byte units of a chunk (two per thread), slots.
template <int MINB>
struct RowCfg {
  static constexpr int kThreads = MINB == 1 ? 768 : 512;
  static constexpr int kBlock = kThreads + kTeachThreads + 32 * kCopyWarps;
  static constexpr int kChunk = 2 * kThreads, kChunkBytes = kChunk * 16;
  static constexpr int kSlots = (MINB == 1 ? 216 : 96) * 1024 / kChunkBytes;
  static_assert(kTeachThreads == 128 && kSlots < kStatRing, "a row's statistics outlive its slots");
};

template <int ID, int N>
__device__ __forceinline__ void bar_sync() { asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory"); }
constexpr int kBarRow = 1, kBarTeach = 2;

// The 16-byte units of a row, its elements outside them, and its chunks.
template <class T, class CFG>
struct RowGeo {
  int head, rest0, units;   // elements before the units, first element after them; units
  int n, over;              // chunks; those that are loaded twice
  __device__ __forceinline__ RowGeo(const T* z, int V) {
    constexpr int kN = Unit<T>::kN;
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    head = min(V, mis ? kN - mis : 0);
    units = (V - head) / kN;
    rest0 = head + units * kN;
    n = (units + CFG::kChunk - 1) / CFG::kChunk;
    over = max(0, n - CFG::kSlots);
  }
  // chunk of the e-th slot of the row, and whether its gradient is stored from there
  __device__ __forceinline__ int chunk(int e) const { return e < n ? e : e - n; }
  __device__ __forceinline__ bool stored(int e) const { return e >= over; }
  __device__ __forceinline__ uint32_t bytes(int c) const {
    return static_cast<uint32_t>(min(CFG::kChunk, units - c * CFG::kChunk)) * 16;
  }
};

// The next row (itself included) with a weight; its weight in *w (1 without weights), N if none.
__device__ __forceinline__ int64_t next_row(const DistillParams& p, int64_t row, int64_t step, float* w) {
  *w = 1.0f;
  if (p.weights)
    for (; row < p.N; row += step) {
      *w = p.weights[row];
      if (*w != 0.0f) break;
    }
  return row;
}

template <class T, int MINB>
__global__ void __launch_bounds__(RowCfg<MINB>::kBlock, MINB)
    distill_rows_kernel(const DistillParams p, const T* logits, T* Gout) {
  using Cfg = RowCfg<MINB>;
  constexpr int kRowThreads = Cfg::kThreads, kRowBlock = Cfg::kBlock, kChunk = Cfg::kChunk;
  constexpr int kChunkBytes = Cfg::kChunkBytes, kSlots = Cfg::kSlots;
  constexpr int kN = Unit<T>::kN, kWarps = kRowThreads / 32;
  using Geo = RowGeo<T, Cfg>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kSlots], computed[kSlots], patched[kSlots], ready[2];
  __shared__ float2 red[2][kWarps], stats[kStatRing];
  __shared__ __align__(16) int ti[2][kRowTeacher];
  __shared__ float tv[2][kRowTeacher], tred[2][kTeachThreads / 32];
  __shared__ int has_teacher[2], gave_up;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t first = blockIdx.x, step = gridDim.x;

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&computed[s], kWarps);
      ptx::mbar_init(&patched[s], kTeachThreads / 32);
    }
    ptx::mbar_init(&ready[0], 1);
    ptx::mbar_init(&ready[1], 1);
    gave_up = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort = &gave_up;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return ptx::mbar_wait_pause_or_abort(bar, parity, kWaitNs, abort, tid < kRowThreads ? 20 : 100);
  };
  // slot and phase of the ring's L-th use
  auto slot_of = [](uint32_t L) { return L % kSlots; };
  auto phase_of = [](uint32_t L) { return (L / kSlots) & 1; };

  if (warp >= kRowBlock / 32 - kCopyWarps) {
    // ---------------- copies ----------------
    if (lane == 0) {
      const uint32_t me = warp - (kRowBlock / 32 - kCopyWarps);
      struct Walk {   // over the slots' uses, row by row
        int64_t row;
        int e;
        Geo g;
      };
      float w;
      const int64_t row0 = next_row(p, first, step, &w);
      Walk in{row0, 0, Geo(logits + row0 * p.V, p.V)}, out = in;
      auto advance = [&](Walk& x) {
        if (++x.e == x.g.n + x.g.over) {
          x.row = next_row(p, x.row + step, step, &w);
          x.e = 0;
          x.g = Geo(logits + x.row * p.V, p.V);
        }
      };
      uint32_t L = 0, F = 0;
      auto release = [&]() {   // the next slot in order comes free
        if (slot_of(F) % kCopyWarps == me) {
          wait(&patched[slot_of(F)], phase_of(F));
          if (out.g.stored(out.e)) {
            const int c = out.g.chunk(out.e);
            ptx::bulk_store(
                reinterpret_cast<uint8_t*>(Gout + out.row * p.V + out.g.head) + static_cast<int64_t>(c) * kChunkBytes,
                ring + slot_of(F) * kChunkBytes, out.g.bytes(c));
            ptx::bulk_commit_group();
            ptx::bulk_wait_group_read0();   // the slot has been read out
          }
        }
        ++F;
        advance(out);
      };
      while (in.row < p.N && !*abort) {
        if (L >= kSlots) release();
        const int c = in.g.chunk(in.e), s = slot_of(L);
        if (s % kCopyWarps == me) {
          const uint32_t bytes = in.g.bytes(c);
          ptx::mbar_arrive_expect_tx(&full[s], bytes);
          ptx::bulk_load(
              ring + s * kChunkBytes,
              reinterpret_cast<const uint8_t*>(logits + in.row * p.V + in.g.head) + static_cast<int64_t>(c) * kChunkBytes,
              bytes, &full[s]);
        }
        ++L;
        advance(in);
      }
      while (F < L && !*abort) release();
      ptx::bulk_wait_group0();
    }
  } else if (tid >= kRowThreads) {
    // ---------------- the teacher's entries ----------------
    const int t0 = tid - kRowThreads;
    // This thread's entry of the row at work, and of the next one.
    int idx = -1, nidx = -1;
    float val = -INFINITY, nval = -INFINITY, zk = 0.0f;
    T nz = static_cast<T>(0.0f);   // (as it lies in memory, so that nothing waits for it early)
    float lq = 0.0f, q = 0.0f, mass = 0.0f;
    bool mine = false, live = false;
    auto fetch = [&](int64_t row) {
      nidx = -1;
      nval = -INFINITY;
      if (t0 < p.K && row < p.N) {
        const int64_t at = row * p.K + t0;
        if (p.id_bytes == 8) {
          const int64_t id = static_cast<const long long*>(p.idx)[at];
          nidx = id >= 0 && id < p.V ? static_cast<int>(id) : -1;
        } else {
          nidx = static_cast<const int*>(p.idx)[at];
        }
        nval = p.val_f32 ? static_cast<const float*>(p.val)[at] : as_f32(static_cast<const __nv_bfloat16*>(p.val)[at]);
      }
    };
    auto gather = [&](int64_t row) {   // the fetched entry's logit
      if (nidx >= 0 && nidx < p.V) nz = logits[row * p.V + nidx];
    };
    // Takes the fetched row, the j-th at work: whether it has entries, its q (every warp computes the
    // softmax over all of them), and for the first of equal indices the mass of all of them.
    auto take = [&](uint32_t j) {
      const bool in = nidx >= 0 && nidx < p.V;
      idx = in ? nidx : -1;
      val = in ? nval : -INFINITY;
      zk = as_f32(nz);
      ti[j & 1][t0] = idx;
      tv[j & 1][t0] = val;
      bar_sync<kBarTeach, kTeachThreads>();
      const float* v = tv[j & 1];
      float x[kRowTeacher / 32], m = -INFINITY, s = 0.0f;
#pragma unroll
      for (int k = 0; k < kRowTeacher / 32; ++k) {
        x[k] = v[32 * k + lane];
        m = fmaxf(m, x[k]);
      }
      const float ref = Running::ref(ptx::warp_max(m));
#pragma unroll
      for (int k = 0; k < kRowTeacher / 32; ++k) s += ex2((x[k] - ref) * p.scale);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      live = s != 0.0f;
      if (t0 == 0) {
        has_teacher[j & 1] = live;
        ptx::mbar_arrive(&ready[j & 1]);
      }
      const float l = log2f(s);
      lq = (val - ref) * p.scale - l;   // log2 q
      q = mass = idx >= 0 ? ex2(lq) : 0.0f;
      mine = idx >= 0;
      // equal indices are rare: counted without branches (in the warp, then against the other warps),
      // and summed entry by entry where there are any
      int equal = __popc(__match_any_sync(0xffffffffu, mine ? idx : -1 - lane)) - 1;
      const int4* all = reinterpret_cast<const int4*>(ti[j & 1]);
      const int quads = (p.K + 3) / 4;   // (past K: -1)
      if (p.K > 32)
#pragma unroll 4
        for (int k = 0; k < quads; ++k) {
          const int4 i4 = all[k];
          const int n = (i4.x == idx) + (i4.y == idx) + (i4.z == idx) + (i4.w == idx);
          equal += (k >> 3) == (t0 >> 5) ? 0 : n;
        }
      if (mine && equal > 0)
        for (int k2 = 0; k2 < p.K; ++k2) {
          if (ti[j & 1][k2] != idx || k2 == t0) continue;
          if (k2 < t0)
            mine = false;
          else
            mass += ex2((v[k2] - ref) * p.scale - l);
        }
    };
    float w = 0.0f, nw = 0.0f;
    int64_t row = next_row(p, first, step, &w);
    uint32_t L = 0, j = 0;
    if (row < p.N) {
      fetch(row);
      gather(row);
      take(0);
    }
    while (row < p.N) {
      const int64_t nrow = next_row(p, row + step, step, &nw);
      fetch(nrow);   // arrives while this row is worked on
      const Geo g(logits + row * p.V, p.V);
      const float gs = w * p.tau;
      const bool loss_live = live;
      float kl = 0.0f, grad = 0.0f;
      const int uses = g.n + g.over;
      for (int e = 0; e < uses; ++e, ++L) {
        const int s = slot_of(L);
        wait(&computed[s], phase_of(L));
        if (e == 0 && nrow < p.N) gather(nrow);
        if (g.stored(e) && live) {
          if (e == g.over) {   // the row's statistics are there
            const float2 st = stats[j % kStatRing];
            const float lp = (zk - st.x) * p.scale;   // log2 p, not normalised
            if (!(q == 0.0f)) kl = q * (lq - (lp - log2f(st.y)));
            grad = gs * (ex2(lp) / st.y - mass);
            if (mine && (idx < g.head || idx >= g.rest0)) put_f32(Gout + row * p.V + idx, grad);
          }
          const int c = g.chunk(e), e0 = g.head + c * kChunk * kN, e1 = min(g.rest0, e0 + kChunk * kN);
          if (mine && idx >= e0 && idx < e1) put_f32(reinterpret_cast<T*>(ring + s * kChunkBytes) + (idx - e0), grad);
        }
        ptx::fence_proxy_async_smem();   // the chunk, as computed and patched, is read by a bulk store next
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&patched[s]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) kl += __shfl_xor_sync(0xffffffffu, kl, o);
      if (lane == 0) tred[j & 1][t0 >> 5] = kl;
      if (nrow < p.N)
        take(j + 1);   // (with a barrier, after which `tred` can be read)
      else
        bar_sync<kBarTeach, kTeachThreads>();
      if (t0 == 0) {
        const float* r = tred[j & 1];
        p.loss[row] = loss_live ? gs * p.tau * 0.69314718055994531f * ((r[0] + r[1]) + (r[2] + r[3])) : 0.0f;
      }
      row = nrow;
      w = nw;
      ++j;
    }
    // Where a wait gave up, a gradient may be missing or wrong in any of this CTA's rows, the finished
    // ones included (their last chunks are stored late): none of their losses stands.  (This thread
    // writes the losses, and every wait of the others is for chunks that have passed through here.)
    if (t0 == 0 && *abort)
      for (row = first; row < p.N; row += step) p.loss[row] = __int_as_float(0x7fc00000);
  } else {
    // ---------------- arithmetic ----------------
    uint32_t j = 0;
    int slot = 0, phase = 0;   // of the row's first chunk
    // (the fence between this thread's accesses and the bulk copies is the teacher's, on the way
    // from here to the copying thread: one per chunk instead of one per thread and chunk)
    auto release = [&](int s) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&computed[s]);
    };
    float w = 1.0f;
    if (p.weights && first < p.N) w = p.weights[first];
    // the elements of a row outside its units: at most one per thread
    auto edge_of = [&](const Geo& g) {
      return tid < g.head ? tid : (tid >= 32 && g.rest0 + tid - 32 < p.V ? g.rest0 + tid - 32 : -1);
    };
    auto edge_at = [&](int64_t row) {   // not converted here: the load need not have arrived yet
      T x = static_cast<T>(-INFINITY);
      const int e = row < p.N ? edge_of(Geo(logits + row * p.V, p.V)) : -1;
      if (e >= 0) x = logits[row * p.V + e];
      return x;
    };
    T nze = edge_at(first);
    for (int64_t row = first; row < p.N; row += step) {
      T* gz = Gout + row * p.V;
      const Geo g(logits + row * p.V, p.V);
      const int edge = edge_of(g);
      const float ze = as_f32(nze);
      nze = edge_at(row + step);   // the next row's, and its weight, arrive meanwhile
      const float nw = p.weights && row + step < p.N ? p.weights[row + step] : 1.0f;
      if (w == 0.0f) {   // no loss: nothing of the row is read
        uint4* gu = reinterpret_cast<uint4*>(gz + g.head);
        for (int u = tid; u < g.units; u += kRowThreads) gu[u] = make_uint4(0, 0, 0, 0);
        if (edge >= 0) put_f32(gz + edge, 0.0f);
        if (tid == 0) p.loss[row] = 0.0f;
        w = nw;
        continue;
      }
      // ---- maximum and sum ----
      float m = ze, s = ze == -INFINITY ? 0.0f : ze - ze + 1.0f;   // (NaN and inf: NaN)
      int sl = slot, ph = phase;   // slot and phase of the chunk at hand
      for (int c = 0; c < g.n; ++c) {
        wait(&full[sl], ph);
        const uint4* buf = reinterpret_cast<const uint4*>(ring + sl * kChunkBytes);
        const int left = g.units - c * kChunk;   // units of this chunk and the ones after it
        if (left >= kChunk) {
          const uint4 x0 = buf[tid], x1 = buf[tid + kRowThreads];
          const float m0 = m;
          m = fmaxf(m, fmaxf(unit_max(x0, T()), unit_max(x1, T())));
          const float ref = Running::ref(m);
          s *= ex2((m0 - ref) * p.scale);
          uint64_t e0[kN / 2], e1[kN / 2];
          exps<T>(x0, ref, p.scale, e0);
          exps<T>(x1, ref, p.scale, e1);
#pragma unroll
          for (int i = 0; i < kN / 2; ++i) e0[i] = add2(e0[i], e1[i]);
          s += sum_of<T>(e0);
        } else {   // the row's last chunk: warps past its end do nothing
          for (int u = tid; (u & ~31) < left; u += kRowThreads) {
            const uint4 x = u < left ? buf[u] : unit_none(T());
            const float m0 = m;
            m = fmaxf(m, unit_max(x, T()));
            const float ref = Running::ref(m);
            s *= ex2((m0 - ref) * p.scale);
            uint64_t e[kN / 2];
            exps<T>(x, ref, p.scale, e);
            s += sum_of<T>(e);
          }
        }
        if (c < g.over) release(sl);
        if (++sl == kSlots) sl = 0, ph ^= 1;
      }
      {
        const float m0 = m;
        m = ptx::warp_max(m);
        s *= ex2((m0 - Running::ref(m)) * p.scale);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      }
      if (lane == 0) red[j & 1][warp] = make_float2(m, s);
      bar_sync<kBarRow, kRowThreads>();
      {   // of the CTA, a lane per warp; the same in every thread
        const float2 x = lane < kWarps ? red[j & 1][lane] : make_float2(-INFINITY, 0.0f);
        m = ptx::warp_max(x.x);
        s = x.y * ex2((x.x - Running::ref(m)) * p.scale);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      }
      if (tid == 0) stats[j % kStatRing] = make_float2(m, s);

      // ---- the gradient, in place, without the teacher's mass ----
      wait(&ready[j & 1], (j >> 1) & 1);
      const bool live = has_teacher[j & 1] != 0;
      const float f = w * p.tau / s;
      if (edge >= 0) put_f32(gz + edge, live ? f * ex2((ze - m) * p.scale) : 0.0f);
      // (from slot `over` of the row on)
      sl = slot + g.over;
      ph = phase;
      while (sl >= kSlots) sl -= kSlots, ph ^= 1;
      for (int e = g.over; e < g.n + g.over; ++e) {
        const int c = g.chunk(e);
        if (e >= g.n) wait(&full[sl], ph);
        uint4* buf = reinterpret_cast<uint4*>(ring + sl * kChunkBytes);
        const int left = g.units - c * kChunk;
        if (live && left >= kChunk) {
          const uint4 x0 = buf[tid], x1 = buf[tid + kRowThreads];
          uint64_t e0[kN / 2], e1[kN / 2];
          exps<T>(x0, m, p.scale, e0);
          exps<T>(x1, m, p.scale, e1);
          buf[tid] = scaled<T>(e0, f);
          buf[tid + kRowThreads] = scaled<T>(e1, f);
        } else {
          for (int u = tid; u < min(left, kChunk); u += kRowThreads) {
            uint64_t x[kN / 2];
            exps<T>(buf[u], m, p.scale, x);
            buf[u] = live ? scaled<T>(x, f) : make_uint4(0, 0, 0, 0);
          }
        }
        release(sl);
        if (++sl == kSlots) sl = 0, ph ^= 1;
      }
      slot = sl;
      phase = ph;
      ++j;
      w = nw;
    }
  }
  if (*abort) {   // let copies in flight land before the CTA leaves
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 20000000ull) __nanosleep(1000);
  }
}

template <class T, int THREADS, int CACHE, int MINB>
cudaError_t run(const DistillParams& p, const void* logits, void* Gout, cudaStream_t st) {
  distill_kernel<T, THREADS, CACHE, MINB>
      <<<static_cast<unsigned>(p.N), THREADS, static_cast<size_t>(p.K) * 12, st>>>(
          p, static_cast<const T*>(logits), static_cast<T*>(Gout));
  return cudaGetLastError();
}

template <class T, int MINB>
cudaError_t run_rows(const DistillParams& p, const void* logits, void* Gout, cudaStream_t st) {
  using Cfg = RowCfg<MINB>;
  const int smem = Cfg::kSlots * Cfg::kChunkBytes;
  cudaError_t e = lm_configure_kernel(reinterpret_cast<const void*>(distill_rows_kernel<T, MINB>), smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(p.N, static_cast<int64_t>(MINB) * lm_sm_count());
  distill_rows_kernel<T, MINB><<<static_cast<unsigned>(grid), Cfg::kBlock, smem, st>>>(
      p, static_cast<const T*>(logits), static_cast<T*>(Gout));
  return cudaGetLastError();
}

// Which kernel, from the bytes of a row (us at N = 8192, measured):
//  - up to 32 KB, 128 threads a row and eight rows an SM, the part of a row beyond their registers
//    coming from L2 a second time (bf16 V = 4000: 46 against 80 for the ring; V = 8192: 72 against 91; V =
//    16000: 129 against 139; V = 20000, beyond: 153 against 161; V = 32000: 284 against 218);
//  - beyond, the ring, with two CTAs on an SM up to 64 KB (bf16 V = 32000: 218 against 243 with one; bf16
//    V = 50265, beyond: 168 at N = 4096 against 170) and one from there on, with half as many
//    threads again (bf16 V = 128000: 861 against 921 with two; fp32 V = 32000: 354 against 380);
//  - long rows with more than 128 teacher entries: 512 threads and two rows an SM, otherwise as
//    the first (bf16 V = 128000: 1100).
constexpr int64_t kShortUpTo = 32768, kTwoUpTo = 65536;
template <class T>
cudaError_t pick(const DistillParams& p, const void* logits, void* Gout, cudaStream_t st) {
  const int64_t bytes = static_cast<int64_t>(p.V) * sizeof(T);
  if (bytes <= kShortUpTo) return run<T, 128, 4, 8>(p, logits, Gout, st);
  if (p.K <= kRowTeacher)
    return bytes <= kTwoUpTo ? run_rows<T, 2>(p, logits, Gout, st) : run_rows<T, 1>(p, logits, Gout, st);
  return run<T, 512, 8, 2>(p, logits, Gout, st);
}

}  // namespace

cudaError_t distill_loss(const void* logits, int dtype, int64_t N, int V, const void* idx, int id_bytes,
                         const void* val, int val_dtype, int K, const float* weights, float tau, float* loss,
                         void* Gout, cudaStream_t st) {
  if (N == 0) return cudaSuccess;
  DistillParams p{};
  p.idx = idx;
  p.val = val;
  p.weights = weights;
  p.loss = loss;
  p.N = N;
  p.V = V;
  p.K = K;
  p.id_bytes = id_bytes;
  p.val_f32 = val_dtype == GRAPE_F32;
  p.tau = tau;
  p.scale = static_cast<float>(1.4426950408889634 / tau);
  return dtype == GRAPE_F32 ? pick<float>(p, logits, Gout, st) : pick<__nv_bfloat16>(p, logits, Gout, st);
}

}  // namespace grape
