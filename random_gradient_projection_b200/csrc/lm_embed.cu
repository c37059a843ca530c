// Token embedding of a language model: lookup with scaling, and the gradient of the table
// in the per-sample form that private training needs.
//
//   out_n   = scale E[id_n]                                   (zero row: id outside [0, vocab))
//   G_i[v]  = scale sum_{t : id_it = v} g_it                  sample i's table gradient (never formed)
//   sq_i    = sum_v ||G_i[v]||^2                              its squared norm, for the joint clip
//   dE      = sum_i c_i G_i                                   the clipped sum
//
// The method clips every sample's gradient over all its parameters before the sum
// ("Metodologia: DP-GRAPE", design choice 2, technical summary of "Memory-Efficient
// Differentially Private Training with Gradient Random Projection"); the table's gradient is
// a sum over tokens like a linear layer's, with one-hot rows in the place of A.
//
// Nothing here does arithmetic to speak of: every kernel is bound by the bytes it moves.
// Both reductions run over the tokens sorted by (token, position), so that every sum has a
// fixed order and needs no floating-point atomics: results are the same bits every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "lm.h"
#include "lm_launch.h"
#include "lm_ptx.cuh"

namespace grape {
namespace {

template <class T>
struct Vec8;   // eight consecutive elements as fp32
template <>
struct Vec8<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { raw = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Token number j, or `vocab` where it lies outside [0, vocab).
__device__ __forceinline__ int token_at(const void* ids, int id_bytes, int64_t j, int vocab) {
  const int64_t v = id_bytes == 8 ? __ldg(static_cast<const long long*>(ids) + j)
                                  : static_cast<int64_t>(__ldg(static_cast<const int*>(ids) + j));
  return v >= 0 && v < vocab ? static_cast<int>(v) : vocab;
}

// ---- lookup ------------------------------------------------------------------------------
// A CTA takes 512 consecutive units of the output (a unit: eight elements of a row, or one
// where a row's pitch is no multiple of eight), two per thread, both rows' loads issued before the
// first store; eight CTAs an SM overlap their two round trips, to the id and to its row (8192 x
// 4096 fp32 rows to bf16: 26.5 us; four units a thread 28.8, eight 35).
constexpr int kLookupThreads = 256, kLookupPer = 2;

template <class TT, class TO, bool VEC>
__global__ void __launch_bounds__(kLookupThreads, 8) embed_kernel(const TT* __restrict__ table, const void* ids,
                                                               int id_bytes, int64_t n, int vocab, int d, float scale,
                                                               TO* out) {
  const int units = VEC ? d / 8 : d;   // per row
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kLookupThreads * kLookupPer);
  const int64_t row0 = base / units;
  const uint32_t off0 = static_cast<uint32_t>(base % units);
  int64_t row[kLookupPer];
  int col[kLookupPer], tok[kLookupPer];
#pragma unroll
  for (int k = 0; k < kLookupPer; ++k) {
    const uint32_t o = off0 + k * kLookupThreads + threadIdx.x;
    row[k] = row0 + o / units;
    col[k] = static_cast<int>(o % units) * (VEC ? 8 : 1);
    tok[k] = row[k] < n ? token_at(ids, id_bytes, row[k], vocab) : vocab;
  }
  if (VEC) {
    Vec8<TT> v[kLookupPer];
#pragma unroll
    for (int k = 0; k < kLookupPer; ++k)
      if (tok[k] < vocab)
        v[k].load(table + static_cast<int64_t>(tok[k]) * d + col[k]);
      else
        v[k].zero();
#pragma unroll
    for (int k = 0; k < kLookupPer; ++k)
      if (row[k] < n) {
        float f[8];
        v[k].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = tok[k] < vocab ? f[i] * scale : 0.0f;
        store8(out + row[k] * d + col[k], f);
      }
  } else {
    float f[kLookupPer];
#pragma unroll
    for (int k = 0; k < kLookupPer; ++k)
      f[k] = tok[k] < vocab ? to_f32(table[static_cast<int64_t>(tok[k]) * d + col[k]]) * scale : 0.0f;
#pragma unroll
    for (int k = 0; k < kLookupPer; ++k)
      if (row[k] < n) from_f32(out + row[k] * d + col[k], f[k]);
  }
}

// ---- order by (token, position) ---------------------------------------------------------------
// A stable least-significant-digit radix sort of the token numbers by one cluster, whose
// CTAs exchange their digit counts through distributed shared memory: no launch per pass,
// and the lists stay in L2.  A warp owns consecutive items, so counting them
// in item order makes the placement stable.  Items outside [0, vocab) get the key
// `vocab` and so end up last.  Digits have 8 bits at most: two passes up to 65535 tokens.
// Up to kSortHeld items a CTA (131072 ids), a pass puts its items in order in shared memory first, so
// that they are written as runs (scattered 4-byte stores made up half of the kernel); beyond, they
// are scattered.  Latency bound: a pass is one round trip to L2 and two cluster barriers.
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortBins = 256, kSortCluster = 16, kSortRounds = 8;
constexpr int kSortHeld = kSortThreads * kSortRounds;

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// The lanes with this lane's digit (0 .. kSortBins, the last for no item), by one vote per bit.
__device__ __forceinline__ uint32_t equal_digits(int digit) {
  uint32_t same = 0xffffffffu;
#pragma unroll
  for (int b = 0; b <= 8; ++b) {
    const bool bit = (digit >> b) & 1;
    const uint32_t v = __ballot_sync(0xffffffffu, bit);
    same &= bit ? v : ~v;
  }
  return same;
}

__global__ void __launch_bounds__(kSortThreads) embed_order_kernel(const void* ids, int id_bytes, int n, int vocab,
                                                                   int passes, int digit_bits, int* positions,
                                                                   int* tokens, int* tmp_positions, int* tmp_tokens,
                                                                   uint32_t* present) {
  __shared__ uint32_t cnt[kSortWarps][kSortBins];
  __shared__ uint32_t tot[kSortBins], base[kSortBins], lbase[kSortBins], wsum[kSortBins / 32], lsum[kSortBins / 32];
  extern __shared__ int held[];   // keys, then positions (kSortHeld each)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = gridDim.x, rank = blockIdx.x;   // the grid is one cluster
  const uint32_t lt = (1u << lane) - 1;

  for (int w = rank * kSortThreads + tid; w < (vocab + 31) / 32; w += ctas * kSortThreads) present[w] = 0;

  // this warp's items [w0, w1): whole rounds of 32, kSortRounds of them at a time in registers
  const int64_t per = ((static_cast<int64_t>(n) + ctas * kSortThreads - 1) / (ctas * kSortThreads)) * 32;
  const int64_t first = (static_cast<int64_t>(rank) * kSortWarps + warp) * per;
  const int w0 = static_cast<int>(first < n ? first : n);
  const int w1 = static_cast<int>(first + per < n ? first + per : n);
  const int mask = (1 << digit_bits) - 1;
  const bool hold = per <= 32 * kSortRounds;   // all of a CTA's items fit
  const int64_t cta0 = static_cast<int64_t>(rank) * kSortWarps * per;
  const int mine = static_cast<int>(cta0 >= n ? 0 : min(static_cast<int64_t>(n) - cta0, kSortWarps * per));

  for (int p = 0; p < passes; ++p) {
    const int shift = p * digit_bits;
    const bool to_final = ((passes - 1 - p) & 1) == 0;
    const int* src_pos = to_final ? tmp_positions : positions;
    const int* src_tok = to_final ? tmp_tokens : tokens;
    int* dst_pos = to_final ? positions : tmp_positions;
    int* dst_tok = to_final ? tokens : tmp_tokens;
    int key[kSortRounds], pos[kSortRounds];
    auto load = [&](int j0) {   // all rounds' loads in flight; -1: no item
      if (p > 0) {
#pragma unroll
        for (int k = 0; k < kSortRounds; ++k) {
          const int j = j0 + 32 * k + lane;
          key[k] = -1;
          if (j < w1) {
            key[k] = __ldcg(src_tok + j);
            pos[k] = __ldcg(src_pos + j);
          }
        }
        return;
      }
      if (id_bytes == 8) {
        int64_t id[kSortRounds];
#pragma unroll
        for (int k = 0; k < kSortRounds; ++k) {
          const int j = j0 + 32 * k + lane;
          id[k] = j < w1 ? __ldg(static_cast<const long long*>(ids) + j) : 0;
        }
#pragma unroll
        for (int k = 0; k < kSortRounds; ++k) key[k] = id[k] >= 0 && id[k] < vocab ? static_cast<int>(id[k]) : vocab;
      } else {
#pragma unroll
        for (int k = 0; k < kSortRounds; ++k) {
          const int j = j0 + 32 * k + lane;
          key[k] = j < w1 ? __ldg(static_cast<const int*>(ids) + j) : 0;
        }
#pragma unroll
        for (int k = 0; k < kSortRounds; ++k) key[k] = key[k] >= 0 && key[k] < vocab ? key[k] : vocab;
      }
#pragma unroll
      for (int k = 0; k < kSortRounds; ++k) {
        pos[k] = j0 + 32 * k + lane;
        if (pos[k] >= w1) key[k] = -1;
      }
    };
    auto digit_of = [&](int k) { return k < 0 ? kSortBins : (k >> shift) & mask; };   // no item: a bin of its own

    for (int i = tid; i < kSortWarps * kSortBins; i += kSortThreads) (&cnt[0][0])[i] = 0;
    if (w0 < w1) load(w0);
    __syncthreads();
    for (int j0 = w0; j0 < w1; j0 += 32 * kSortRounds) {
      if (j0 > w0) load(j0);
#pragma unroll
      for (int k = 0; k < kSortRounds; ++k) {
        if (j0 + 32 * k >= w1) break;
        const int digit = digit_of(key[k]);
        const uint32_t same = equal_digits(digit);
        if (digit < kSortBins && (same & lt) == 0) cnt[warp][digit] += __popc(same);
        __syncwarp();
      }
    }
    if (!hold && w0 < w1) load(w0);   // the placement starts over (otherwise they are still here)
    __syncthreads();
    if (tid < kSortBins) {   // items of bin `tid` in the warps before each warp
      uint32_t run = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = cnt[w][tid];
        cnt[w][tid] = run;
        run += c;
      }
      tot[tid] = run;
    }
    if (ctas > 1)
      ptx::cluster_sync();
    else
      __syncthreads();
    if (tid < kSortBins) {
      uint32_t all = 0, before = 0, x[kSortCluster];
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c)
        x[c] = c >= ctas ? 0 : ctas == 1 ? tot[tid] : ld_dsmem_u32(ptx::cluster_addr(&tot[tid], c));
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        before += c < rank ? x[c] : 0;
        all += x[c];
      }
      uint32_t incl = all, lincl = tot[tid];   // scans over the bins: of the cluster, of this CTA
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o), z = __shfl_up_sync(0xffffffffu, lincl, o);
        if (lane >= o) incl += y, lincl += z;
      }
      if (lane == 31) wsum[warp] = incl, lsum[warp] = lincl;
      base[tid] = incl - all + before;
      lbase[tid] = lincl - tot[tid];
    }
    __syncthreads();
    if (tid < kSortBins) {
      uint32_t add = 0, ladd = 0;
      for (int w = 0; w < warp; ++w) add += wsum[w], ladd += lsum[w];
      base[tid] += add;
      lbase[tid] += ladd;
    }
    __syncthreads();
    if (hold) {
#pragma unroll
      for (int k = 0; k < kSortRounds; ++k) {
        if (w0 + 32 * k >= w1) break;
        const int digit = digit_of(key[k]);
        const uint32_t same = equal_digits(digit);
        uint32_t at = 0;
        if (digit < kSortBins) at = lbase[digit] + cnt[warp][digit] + __popc(same & lt);
        __syncwarp();
        if (digit < kSortBins) {
          if ((same & lt) == 0) cnt[warp][digit] += __popc(same);
          held[at] = key[k];
          held[kSortHeld + at] = pos[k];
        }
        __syncwarp();
      }
      __syncthreads();
      for (int i = tid; i < mine; i += kSortThreads) {
        const int k = held[i], digit = digit_of(k);
        const uint32_t at = base[digit] + (i - lbase[digit]);
        dst_pos[at] = held[kSortHeld + i];
        dst_tok[at] = k;
        // last pass: these items are in the order of their whole keys now
        if (p == passes - 1 && k < vocab && (i == 0 || held[i - 1] != k)) atomicOr(present + (k >> 5), 1u << (k & 31));
      }
      __syncthreads();   // `held` and the counts may be written again
    } else {
      for (int j0 = w0; j0 < w1; j0 += 32 * kSortRounds) {
        if (j0 > w0) load(j0);
#pragma unroll
        for (int k = 0; k < kSortRounds; ++k) {
          if (j0 + 32 * k >= w1) break;
          const int digit = digit_of(key[k]);
          const uint32_t same = equal_digits(digit);
          uint32_t at = 0;
          if (digit < kSortBins) at = base[digit] + cnt[warp][digit] + __popc(same & lt);
          __syncwarp();
          if (digit < kSortBins) {
            if ((same & lt) == 0) cnt[warp][digit] += __popc(same);
            dst_pos[at] = pos[k];
            dst_tok[at] = key[k];
          }
          __syncwarp();
        }
      }
    }
    // the lists are read by other threads (and CTAs) next
    __threadfence();
    if (ctas > 1)
      ptx::cluster_sync();
    else
      __syncthreads();
  }
  // which tokens occur at all: their rows of the gradient are written by the sums, the others zeroed
  if (hold) return;
  for (int j = rank * kSortThreads + tid; j < n; j += ctas * kSortThreads) {
    const int t = __ldcg(tokens + j);
    if (t < vocab && (j == 0 || __ldcg(tokens + j - 1) != t)) atomicOr(present + (t >> 5), 1u << (t & 31));
  }
}

// ---- sums over runs of the sorted list ----------------------------------------------------------
// A run is a maximal stretch of equal keys in the sorted list: a token (gradient), or a token
// within a sample (norms; within a token the positions, so the samples, ascend).  A warp takes a
// chunk of up to 32 consecutive items and 256 columns of G, eight per lane, and walks the items
// with the rows of the next eight in flight.  Runs inside the chunk are finished there; the first
// and the last may go on in the chunks around, so their sums go to part[chunk][0] (a run that
// began earlier) or part[chunk][1] (one that begins here), and a second, short launch adds those in
// chunk order.  So a token that fills half the batch is spread over as many warps as any other.
// Bound by memory: 16 x 512 tokens, d = 4096, vocab 32000, bf16: the gradient with its zero rows and
// joins 102 us (591 MB, 5.8 TB/s), the norms with theirs 21 us (67 MB, 3.2 TB/s).
struct SegParams {
  const int* positions;
  const int* tokens;
  int n, T, vocab, d;
  int R, chunks, tiles;     // items per chunk, chunks, 256-column tiles
  float scale;
  const float* weights;     // per sample; null: 1 (gradient only)
  float* part;              // [chunk][2][tiles * 256]
  float* grad;              // vocab x d
  float* slots;             // [tile][n] (norms)
  const uint32_t* present;
  int seg_blocks;           // gradient: blocks beyond these zero the rows of absent tokens
};
constexpr int kSegWarps = 4, kSegAhead = 8;

__device__ __forceinline__ float* part_at(const SegParams& p, int chunk, int which, int tile, int lane) {
  return p.part + ((static_cast<size_t>(chunk) * 2 + which) * p.tiles + tile) * 256 + lane * 8;
}

template <class TG, bool VEC>
struct RowPiece {   // this lane's eight columns of a row of G
  Vec8<TG> v;
  float s[8];
  __device__ __forceinline__ void load(const TG* row, int col, int d) {
    if (VEC) {
      if (col < d)
        v.load(row + col);
      else
        v.zero();
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = col + 32 * i < d ? to_f32(row[col + 32 * i]) : 0.0f;
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if (VEC) {
      v.get(f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = s[i];
    }
  }
};

// First column of this lane in its tile; its eight are consecutive (VEC) or 32 apart.
template <bool VEC>
__device__ __forceinline__ int lane_col(int tile, int lane) { return tile * 256 + (VEC ? lane * 8 : lane); }

template <bool VEC>
__device__ __forceinline__ void store_grad(const SegParams& p, int t, int col, const float (&acc)[8]) {
  float* g = p.grad + static_cast<size_t>(t) * p.d + col;
  if (VEC) {
    if (col < p.d) store8(g, acc);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + 32 * i < p.d) g[32 * i] = acc[i];
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// NORMS: runs are (token, sample) and give ||sum||^2 per tile into slots[tile][position of the
// run's first item] (zero at every other position), which sample_sums_kernel adds per sample.
// Otherwise runs are tokens and give the rows of grad, weighted per sample.
template <class TG, bool VEC, bool NORMS>
__global__ void __launch_bounds__(32 * kSegWarps) segment_kernel(const SegParams p, const TG* __restrict__ G) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!NORMS && static_cast<int>(blockIdx.x) >= p.seg_blocks) {
    // rows of absent tokens
    const int nw = (gridDim.x - p.seg_blocks) * kSegWarps;
    for (int v = (blockIdx.x - p.seg_blocks) * kSegWarps + warp; v < p.vocab; v += nw) {
      if ((__ldg(p.present + (v >> 5)) >> (v & 31)) & 1u) continue;
      float* g = p.grad + static_cast<size_t>(v) * p.d;
      if (VEC) {
        for (int c = lane * 4; c < p.d; c += 128) *reinterpret_cast<float4*>(g + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        for (int c = lane; c < p.d; c += 32) g[c] = 0.0f;
      }
    }
    return;
  }
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kSegWarps + warp;
  const int chunk = static_cast<int>(job / p.tiles), tile = static_cast<int>(job % p.tiles);
  if (chunk >= p.chunks) return;
  const int c0 = chunk * p.R, len = min(p.R, p.n - c0);
  int tok = p.vocab, pos = 0;
  if (lane < len) {
    tok = __ldg(p.tokens + c0 + lane);
    pos = __ldg(p.positions + c0 + lane);
  }
  const int count = __popc(__ballot_sync(0xffffffffu, tok < p.vocab));   // dropped items are last
  const int sample = NORMS || p.weights ? pos / p.T : 0;
  const float c = !NORMS && p.weights && lane < count ? __ldg(p.weights + sample) : 1.0f;
  const float w = p.scale * c;
  const uint32_t out = NORMS ? 0u : __ballot_sync(0xffffffffu, c == 0.0f);   // their rows are not read
  // does the run of the first item begin earlier, does that of the last item go on?
  bool head = false, tail = false;
  if (count > 0) {
    if (c0 > 0 && lane == 0) {
      head = __ldg(p.tokens + c0 - 1) == tok;
      if (NORMS && head) head = __ldg(p.positions + c0 - 1) / p.T == sample;
    }
    head = __shfl_sync(0xffffffffu, head, 0);
    if (count == len && c0 + len < p.n && lane == len - 1) {
      tail = __ldg(p.tokens + c0 + len) == tok;
      if (NORMS && tail) tail = __ldg(p.positions + c0 + len) / p.T == sample;
    }
    tail = __shfl_sync(0xffffffffu, tail, len - 1);
  }
  // lanes whose item ends its run in this chunk
  const int next_tok = __shfl_down_sync(0xffffffffu, tok, 1), next_sample = __shfl_down_sync(0xffffffffu, sample, 1);
  const bool last = lane == count - 1 ? !tail : (next_tok != tok || (NORMS && next_sample != sample));
  const uint32_t ends = __ballot_sync(0xffffffffu, lane < count && last);

  const int col = lane_col<VEC>(tile, lane);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float slot = 0.0f;
  int run_first = 0;
  for (int j0 = 0; j0 < count; j0 += kSegAhead) {
    RowPiece<TG, VEC> x[kSegAhead];
#pragma unroll
    for (int k = 0; k < kSegAhead; ++k) {
      const int row = __shfl_sync(0xffffffffu, pos, min(j0 + k, 31));
      if (j0 + k < count && !((out >> (j0 + k)) & 1u)) x[k].load(G + static_cast<size_t>(row) * p.d, col, p.d);
    }
#pragma unroll
    for (int k = 0; k < kSegAhead; ++k) {
      const int j = j0 + k;
      const float wj = __shfl_sync(0xffffffffu, w, min(j, 31));
      const int tj = __shfl_sync(0xffffffffu, tok, min(j, 31));
      if (j < count) {
        if (!((out >> j) & 1u)) {
          float f[8];
          x[k].get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
        }
        if ((ends >> j) & 1u) {
          if (head) {
            store8(part_at(p, chunk, 0, tile, lane), acc);
          } else if (NORMS) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(acc[i], acc[i], ss);
            ss = warp_sum(ss);
            if (lane == run_first) slot = ss;
          } else {
            store_grad<VEC>(p, tj, col, acc);
          }
          head = false;
          run_first = j + 1;
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        }
      }
    }
  }
  if (tail) store8(part_at(p, chunk, head ? 0 : 1, tile, lane), acc);
  if (NORMS && lane < len) p.slots[static_cast<size_t>(tile) * p.n + pos] = slot;
}

// The runs that begin in a chunk and go on in the next ones: their partial sums, added in a fixed
// order.  A CTA looks at eight chunks, one per warp, in one 256-column tile.  A run over few chunks is
// added by its warp; a longer one by all eight warps, an eighth of its chunks each (from 4 / 16 / 64
// chunks on, us: norms of 16 x 512 x 1024 14.3 / 12.9 / 12.9, gradient 33.3 / 33.3 / 35.6, gradient of 8 x
// 8192 x 1024 68.2 / 68.2 / 70.6).
constexpr int kJoinWarps = 8, kJoinAlone = 16;

__device__ __forceinline__ void add_parts(const SegParams& p, int c0, int c1, int tile, int lane, float (&acc)[8]) {
#pragma unroll 1
  for (int c = c0; c < c1; c += 4) {   // four in flight
    float4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c + u < c1) {
        const float4* q = reinterpret_cast<const float4*>(part_at(p, c + u, 0, tile, lane));
        a[u] = __ldcg(q);
        b[u] = __ldcg(q + 1);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c + u < c1) {
        acc[0] += a[u].x, acc[1] += a[u].y, acc[2] += a[u].z, acc[3] += a[u].w;
        acc[4] += b[u].x, acc[5] += b[u].y, acc[6] += b[u].z, acc[7] += b[u].w;
      }
  }
}

template <bool VEC, bool NORMS>
__global__ void __launch_bounds__(32 * kJoinWarps) segment_join_kernel(const SegParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  __shared__ int long_more[kJoinWarps];
  __shared__ float sums[kJoinWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x / p.tiles * kJoinWarps, tile = blockIdx.x % p.tiles;
  const int chunk = first + warp, c0 = chunk * p.R, c1 = c0 + p.R;
  // does a run begin in this chunk and go on, and through how many chunks after it?
  int t = p.vocab, sample = 0, more = 0;
  auto same = [&](int j) {
    return __ldg(p.tokens + j) == t && (!NORMS || __ldg(p.positions + j) / p.T == sample);
  };
  if (chunk < p.chunks && c1 < p.n) {
    t = __ldg(p.tokens + c1 - 1);
    if (NORMS) sample = __ldg(p.positions + c1 - 1) / p.T;
    if (t < p.vocab && same(c1) && !(same(c0) && c0 > 0 && same(c0 - 1))) {
      more = 1;   // all but the last of these chunks are full of the run
      while (true) {
        const int64_t e = static_cast<int64_t>(chunk + more + lane + 1) * p.R;   // end of the chunk `more + lane` after
        const bool on = e < p.n && same(static_cast<int>(e) - 1) && same(static_cast<int>(e));
        const uint32_t m = __ballot_sync(0xffffffffu, on);
        more += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        if (m != 0xffffffffu) break;
      }
    }
  }
  if (lane == 0) long_more[warp] = more > kJoinAlone ? more : 0;
  __syncthreads();

  auto finish = [&](float (&acc)[8]) {   // by the run's warp
    if (NORMS) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(acc[i], acc[i], ss);
      ss = warp_sum(ss);
      // the run's first item in this chunk
      const uint32_t m = __ballot_sync(0xffffffffu, lane < p.R && same(c0 + lane));   // a suffix of the chunk's lanes
      if (lane == 0) p.slots[static_cast<size_t>(tile) * p.n + __ldg(p.positions + c0 + __ffs(m) - 1)] = ss;
    } else {
      store_grad<VEC>(p, t, lane_col<VEC>(tile, lane), acc);
    }
  };
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto begin = [&]() {
    const float4* q = reinterpret_cast<const float4*>(part_at(p, chunk, 1, tile, lane));
    const float4 a = __ldcg(q), b = __ldcg(q + 1);
    acc[0] = a.x, acc[1] = a.y, acc[2] = a.z, acc[3] = a.w, acc[4] = b.x, acc[5] = b.y, acc[6] = b.z, acc[7] = b.w;
  };
  if (more > 0 && more <= kJoinAlone) {
    begin();
    add_parts(p, chunk + 1, chunk + 1 + more, tile, lane, acc);
    finish(acc);
  }
  for (int k = 0; k < kJoinWarps; ++k) {   // the long ones, one after another
    const int n = long_more[k];
    if (n == 0) continue;
    const int from = first + k + 1;
    float part[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_parts(p, from + static_cast<int>(static_cast<int64_t>(n) * warp / kJoinWarps),
              from + static_cast<int>(static_cast<int64_t>(n) * (warp + 1) / kJoinWarps), tile, lane, part);
    store8(&sums[warp][lane * 8], part);
    __syncthreads();
    if (warp == k) {
      begin();
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += sums[w][lane * 8 + i];
      finish(acc);
    }
    __syncthreads();
  }
}

// sq[b] = sum of the slots of sample b over all tiles, in a fixed order.  A sample with many slots is
// summed by a cluster of CTAs, whose sums its first one adds.
constexpr int kSumThreads = 1024, kSumCluster = 8;
__global__ void __launch_bounds__(kSumThreads) sample_sums_kernel(const float* slots, int n, int T, int tiles, int parts,
                                                                  float* sq) {
  ptx::griddep_wait();
  __shared__ float red[kSumThreads / 32], sum;
  const int b = blockIdx.x / parts, part = blockIdx.x % parts;
  float s = 0.0f;
  const float* q = slots + static_cast<size_t>(b) * T;
  const int64_t total = static_cast<int64_t>(T) * tiles;
  const int64_t end = total * (part + 1) / parts;
  for (int64_t i0 = total * part / parts + threadIdx.x; i0 < end; i0 += 8 * kSumThreads) {   // eight in flight
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t i = i0 + u * kSumThreads;
      // (64-bit divisions would take longer than the loads)
      const int64_t tile = total <= 0xffffffffll ? static_cast<uint32_t>(i) / static_cast<uint32_t>(T) : i / T;
      x[u] = i < end ? __ldcg(q + tile * n + (i - tile * T)) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) s += x[u];
  }
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = warp_sum(red[threadIdx.x]);
    if (threadIdx.x == 0) {
      sum = s;
      if (parts == 1) sq[b] = s;
    }
  }
  if (parts == 1) return;
  __syncthreads();
  ptx::cluster_sync();   // every CTA's sum is there
  if (part == 0 && threadIdx.x == 0) {
    float tot = 0.0f;
    for (int c = 0; c < parts; ++c) tot += __uint_as_float(ld_dsmem_u32(ptx::cluster_addr(&sum, c)));
    sq[b] = tot;
  }
  __syncthreads();
  ptx::cluster_sync();   // and none leaves before it has been read
}

cudaError_t launch_sums(const SegParams& p, int B, float* sq, cudaStream_t st) {
  // one round of eight values a thread is enough for one CTA
  const int parts = static_cast<int64_t>(p.T) * p.tiles > 8 * kSumThreads ? kSumCluster : 1;
  if (static_cast<int64_t>(B) * parts > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * parts);
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = st;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = parts;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_sums_kernel, static_cast<const float*>(p.slots), p.n, p.T, p.tiles, parts, sq);
}

int tiles_of(int d) { return (d + 255) / 256; }

// Items per chunk: 32 (a lane each) once that gives every SM 16 warps, else 8, so that a short
// batch still spreads over the machine.  (8 against 32, us, norms and gradient: 1 x 512 x 256 10.0 and 5.7
// / 13.4 and 8.8, 16 x 512 x 1024 12.9 and 33.3 / 16.5 and 31.6, 16 x 512 x 4096 29.3 and 106 / 21.2 and
// 102, 8 x 8192 x 1024 60 and 94 / 43 and 68.)
constexpr int kPlanSms = 148;   // of a B200 (workspaces are sized without asking a device)
int chunk_items(int64_t n, int d) { return n * tiles_of(d) / 32 >= kPlanSms * 16 ? 32 : 8; }

SegParams seg_params(const void* order, int B, int T, int vocab, int d, float scale, void* ws) {
  const int64_t n = static_cast<int64_t>(B) * T;
  const EmbedOrderLayout lay(n, vocab);
  const char* o = static_cast<const char*>(order);
  SegParams p{};
  p.positions = reinterpret_cast<const int*>(o + lay.positions);
  p.tokens = reinterpret_cast<const int*>(o + lay.tokens);
  p.present = reinterpret_cast<const uint32_t*>(o + lay.present);
  p.n = static_cast<int>(n);
  p.T = T;
  p.vocab = vocab;
  p.d = d;
  p.R = chunk_items(n, d);
  p.chunks = static_cast<int>((n + p.R - 1) / p.R);
  p.tiles = tiles_of(d);
  p.scale = scale;
  p.part = static_cast<float*>(ws);
  p.slots = p.part + static_cast<size_t>(p.chunks) * 2 * p.tiles * 256;
  return p;
}

unsigned join_blocks(const SegParams& p) {
  return static_cast<unsigned>((p.chunks + kJoinWarps - 1) / kJoinWarps) * static_cast<unsigned>(p.tiles);
}

template <class TG, bool VEC>
cudaError_t run_sqnorms(const SegParams& p, int B, const TG* G, float* sq, cudaStream_t st) {
  const int64_t jobs = static_cast<int64_t>(p.chunks) * p.tiles;
  const unsigned blocks = static_cast<unsigned>((jobs + kSegWarps - 1) / kSegWarps);
  cudaError_t e = lm_launch(false, segment_kernel<TG, VEC, true>, dim3(blocks), 32 * kSegWarps, 0, st, p, G);
  if (e == cudaSuccess)
    e = lm_launch(true, segment_join_kernel<VEC, true>, dim3(join_blocks(p)), 32 * kJoinWarps, 0, st, p);
  if (e == cudaSuccess) e = launch_sums(p, B, sq, st);
  return e;
}

template <class TG, bool VEC>
cudaError_t run_grad(SegParams p, const TG* G, cudaStream_t st) {
  const int64_t jobs = static_cast<int64_t>(p.chunks) * p.tiles;
  const unsigned blocks = static_cast<unsigned>((jobs + kSegWarps - 1) / kSegWarps);
  const unsigned zero = static_cast<unsigned>(std::min<int64_t>((p.vocab + kSegWarps - 1) / kSegWarps, kPlanSms * 8));
  p.seg_blocks = static_cast<int>(blocks);
  cudaError_t e = lm_launch(false, segment_kernel<TG, VEC, false>, dim3(blocks + zero), 32 * kSegWarps, 0, st, p, G);
  if (e == cudaSuccess && blocks > 0)
    e = lm_launch(true, segment_join_kernel<VEC, false>, dim3(join_blocks(p)), 32 * kJoinWarps, 0, st, p);
  return e;
}

template <class TT, class TO>
cudaError_t run_lookup(const void* table, const void* ids, int id_bytes, int64_t n, int vocab, int d, float scale,
                       void* out, cudaStream_t st) {
  const TT* t = static_cast<const TT*>(table);
  TO* o = static_cast<TO*>(out);
  const bool vec = d % 8 == 0;
  const int64_t units = n * (vec ? d / 8 : d), per = kLookupThreads * kLookupPer;
  const int64_t grid = (units + per - 1) / per;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (vec)
    embed_kernel<TT, TO, true><<<static_cast<unsigned>(grid), kLookupThreads, 0, st>>>(t, ids, id_bytes, n, vocab, d,
                                                                                       scale, o);
  else
    embed_kernel<TT, TO, false><<<static_cast<unsigned>(grid), kLookupThreads, 0, st>>>(t, ids, id_bytes, n, vocab, d,
                                                                                        scale, o);
  return cudaGetLastError();
}

// Whether the current device can run a cluster of sixteen of the order's CTAs (asked once per device).
bool sixteen_fit(int smem) {
  static std::atomic<int> known[64];   // 0: not asked yet, 1: yes, 2: no
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  int k = known[dev].load(std::memory_order_relaxed);
  if (k == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kSortCluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = kSortCluster;
    a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok = cudaFuncSetAttribute(reinterpret_cast<const void*>(embed_order_kernel),
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, embed_order_kernel, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();
    k = ok ? 1 : 2;
    known[dev].store(k, std::memory_order_relaxed);
  }
  return k == 1;
}

}  // namespace

cudaError_t embed_forward(const void* table, int table_dtype, const void* ids, int id_bytes, int64_t n, int vocab,
                          int d, float scale, int out_dtype, void* out, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  const bool tf = table_dtype == GRAPE_F32, of = out_dtype == GRAPE_F32;
  if (tf && of) return run_lookup<float, float>(table, ids, id_bytes, n, vocab, d, scale, out, st);
  if (tf) return run_lookup<float, __nv_bfloat16>(table, ids, id_bytes, n, vocab, d, scale, out, st);
  if (of) return run_lookup<__nv_bfloat16, float>(table, ids, id_bytes, n, vocab, d, scale, out, st);
  return run_lookup<__nv_bfloat16, __nv_bfloat16>(table, ids, id_bytes, n, vocab, d, scale, out, st);
}

cudaError_t embed_order(const void* ids, int id_bytes, int64_t n, int vocab, void* order, cudaStream_t st) {
  const EmbedOrderLayout lay(n, vocab);
  char* o = static_cast<char*>(order);
  int bits = 1;
  while (vocab >> bits) ++bits;   // keys 0 .. vocab
  const int passes = (bits + 7) / 8, digit_bits = (bits + passes - 1) / passes;
  const int smem = 2 * kSortHeld * 4;
  cudaError_t e = lm_configure_kernel(reinterpret_cast<const void*>(embed_order_kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  // one CTA for a short list, the portable eight, and sixteen where each still has a round for every
  // warp and the device can hold such a cluster (65536 ids: 25 us against 34 with eight)
  const int ctas = n > 32768 && sixteen_fit(smem) ? kSortCluster : n > 2048 ? 8 : 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = ctas;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, embed_order_kernel, ids, id_bytes, static_cast<int>(n), vocab, passes, digit_bits,
                            reinterpret_cast<int*>(o + lay.positions), reinterpret_cast<int*>(o + lay.tokens),
                            reinterpret_cast<int*>(o + lay.tmp_positions), reinterpret_cast<int*>(o + lay.tmp_tokens),
                            reinterpret_cast<uint32_t*>(o + lay.present));
}

size_t embed_workspace_bytes(int64_t n, int d) {
  const int64_t R = chunk_items(n, d), chunks = (n + R - 1) / R;
  return lm_round256(static_cast<size_t>(chunks) * 2 * tiles_of(d) * 256 * 4 +
                     static_cast<size_t>(tiles_of(d)) * n * 4 + 256);
}

cudaError_t embed_sqnorms(const void* order, int B, int T, int vocab, int d, const void* G, int dtype, float scale,
                          void* ws, float* sqnorms, cudaStream_t st) {
  if (B == 0) return cudaSuccess;
  if (T == 0) return cudaMemsetAsync(sqnorms, 0, static_cast<size_t>(B) * 4, st);
  const SegParams p = seg_params(order, B, T, vocab, d, scale, ws);
  const bool vec = d % 8 == 0;
  if (dtype == GRAPE_F32)
    return vec ? run_sqnorms<float, true>(p, B, static_cast<const float*>(G), sqnorms, st)
               : run_sqnorms<float, false>(p, B, static_cast<const float*>(G), sqnorms, st);
  return vec ? run_sqnorms<__nv_bfloat16, true>(p, B, static_cast<const __nv_bfloat16*>(G), sqnorms, st)
             : run_sqnorms<__nv_bfloat16, false>(p, B, static_cast<const __nv_bfloat16*>(G), sqnorms, st);
}

cudaError_t embed_grad(const void* order, int B, int T, int vocab, int d, const void* G, int dtype, float scale,
                       const float* weights, void* ws, float* grad, cudaStream_t st) {
  SegParams p = seg_params(order, B, T, vocab, d, scale, ws);
  p.weights = weights;
  p.grad = grad;
  const bool vec = d % 8 == 0;
  if (dtype == GRAPE_F32)
    return vec ? run_grad<float, true>(p, static_cast<const float*>(G), st)
               : run_grad<float, false>(p, static_cast<const float*>(G), st);
  return vec ? run_grad<__nv_bfloat16, true>(p, static_cast<const __nv_bfloat16*>(G), st)
             : run_grad<__nv_bfloat16, false>(p, static_cast<const __nv_bfloat16*>(G), st);
}

}  // namespace grape
