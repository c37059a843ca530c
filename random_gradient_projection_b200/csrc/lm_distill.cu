// Distillation from a teacher's top logits, loss and gradient in one pass over the student's
// logits.  Per row n with student logits z (V of them) and the teacher's entries (idx_k, val_k):
//
//   q   = softmax over the row's entries with idx in [0, V) of val / tau
//   p   = softmax over V of z / tau
//   l_n = w_n tau^2 sum_k q_k (log q_k - log p_{idx_k})
//   Gout_nv = dl_n / dz_v = w_n tau (p_v - sum_{k : idx_k = v} q_k)
//
// Bound by memory: z is read from DRAM once and Gout written once (2 V elements a row); the
// kernel holds the first part of a row in registers between the statistics and the gradient and
// takes the rest again from L2, where the rows in flight (one per resident CTA) fit.  Statistics
// are fp32: each thread keeps a running maximum and sum, joined over the CTA once; Gout is
// rounded once, as it is written.  Gout may be the logits themselves: every thread rewrites
// only what it has read, and the teacher's entries are read before the first store.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "lm.h"

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

template <class T, int THREADS, int CACHE, int MINB>
cudaError_t run(const DistillParams& p, const void* logits, void* Gout, cudaStream_t st) {
  distill_kernel<T, THREADS, CACHE, MINB>
      <<<static_cast<unsigned>(p.N), THREADS, static_cast<size_t>(p.K) * 12, st>>>(
          p, static_cast<const T*>(logits), static_cast<T*>(Gout));
  return cudaGetLastError();
}

template <class T>
cudaError_t pick(const DistillParams& p, const void* logits, void* Gout, cudaStream_t st) {
  // Short rows: a small CTA holds the whole row and several rows share an SM.
  if (static_cast<int64_t>(p.V) * sizeof(T) <= 128 * 16 * 4) return run<T, 128, 4, 8>(p, logits, Gout, st);
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
