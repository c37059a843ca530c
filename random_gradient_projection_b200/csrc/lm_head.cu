// Softmax cross entropy of a vocabulary head, with gradients, that never holds the logits:
//
//   z_nv = h_n . W_v                     N live rows, V vocabulary rows, d wide
//   l_n  = w_n (lse_v z_nv - z_{n,label})
//   g_nv = w_n (exp(z_nv - lse_n) - [v = label_n])
//   dH_n = sum_v g_nv W_v,   dW_v = sum_n g_nv h_n
//
// Four contractions on one warp-specialised kernel, head_gemm_kernel<EPI, PLANES>:
//
//   STATS  z over the whole vocabulary, reduced in the epilogue to a maximum and a sum of
//          exponentials per row and 128 columns (and the label's logit)
//   GRAD   z again for one piece of the vocabulary; the epilogue writes g (bf16) for the piece
//   DH     dH (+)= g W over the piece          (K = the piece's columns, split when rows are few)
//   DW     dW of the piece = g^T H             (K = rows)
//
// so the memory is one piece of g, at most kPieceBytes (or 4096 columns), whatever V is.  The price
// is the second product z: 6 (8) N V d flops for dH (and dW) where keeping the logits takes 4 (6).
//
// Rows without a loss (label outside [0, V), or weight 0) are dropped first: the live rows are
// gathered in order into a compact H, so masked rows cost nothing, and whatever they hold (NaN
// included) reaches no sum.  The number of live rows is known on the device only; every kernel
// reads it there.
//
// Precision.  bf16 inputs: products are exact in the tensor core and accumulate in fp32; g is
// rounded once to bf16 as the operand of the second product (relative 2^-8 at most per element,
// independent from element to element, so it averages out in the sums), as the method's own
// step does with AP.  fp32 inputs (PLANES = 3): each operand is split into three bf16 planes
// x = x0 + x1 + x2 (24 bits together) and the six products of order up to 2^-16 are accumulated,
// smallest first; the three dropped ones are below 2^-24 relative.  Six tensor-core products
// run several times faster than one on the fp32 cores.
//
// The kernel: a cluster of two CTAs (one tile of 256 x 256, cta_group::2), each CTA with half of
// A's rows and half of B's columns in its ring of shared-memory stages.  Warps 0 and 10-12 of each
// CTA load by TMA, warp 1 of CTA 0 issues the MMAs for both, warps 2-9 are the epilogue of their
// CTA's 128 rows; two 256-column accumulators in TMEM let it overlap the next tile.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "lm.h"
#include "tc.h"
#include "tc_ptx.cuh"

namespace grape {
namespace {

constexpr int kTile = 256;            // rows and columns of a tile
constexpr int kHalf = 128;            // of a CTA
constexpr int kBK = 64;
constexpr int kStages = 6;
constexpr int kStage = 2 * kHalf * kBK * 2;   // A half and B half: 32 KB
constexpr int kEpiWarps = 8;
constexpr int kProducers = 4;
constexpr int kThreads = 32 * (2 + kEpiWarps + kProducers - 1);
constexpr int kBox = 32 * 128;        // an epilogue warp's staging box: 32 rows x 128 bytes
constexpr int kBarOff = kStages * kStage;
constexpr int kBoxOff = kBarOff + 1024;
constexpr int kSmem = kBoxOff + kEpiWarps * kBox + 1024;   // + alignment slack
static_assert(kProducers <= kStages, "parity waits need at most as many producers as stages");
static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
constexpr int kGroupM = 8;            // row tiles that share a column of B tiles in L2
constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr uint64_t kDrainNs = 20000000ull;
constexpr size_t kPieceBytes = size_t(128) << 20;
constexpr int kErrTimeout = 1;
#ifdef GRAPE_CHECKED
constexpr int kErrBounds = 8;   // a TMA box off the 16-byte rule or at a negative coordinate (skipped)
#endif

enum Epi : int { STATS = 0, GRAD = 1, DH = 2, DW = 3 };

// Device words at the start of the workspace.
struct HeadState {
  int err;
  int n_live;
};

struct HeadGemm {
  CUtensorMap mapA, mapB;
  HeadState* state;
  int m_tiles;          // DW: vocabulary tiles of the piece; otherwise from n_live
  int n_tiles, splits;  // column tiles; parts of the K extent (DH)
  int kblocks;          // K extent in blocks of 64 (DW: from n_live)
  int planeA, planeB;   // elements from one plane of an operand to the next
  int v0, V, d;         // first vocabulary row of the piece; sizes
  int64_t n_pad;        // rows of the compact buffers
  const int* labels;    // compact rows
  const float* weights;
  const float* lse;
  float2* parts;        // STATS: [128-column slot][n_pad] (maximum, sum of exponentials)
  float* target;        // STATS: the label's logit
  __nv_bfloat16* g;     // GRAD: [n_pad][ldg]
  int64_t ldg;
  int planeG;           // GRAD: elements from one plane of g to the next
  float* acc;           // DH: [split][n_pad][ldacc] fp32 (several pieces or splits)
  int64_t ldacc;
  int add, last;        // DH: add to acc; write the result (no later piece, no splits)
  const int* rows;      // compact row -> row of H
  void* out;            // dH or dW, dtype of H
  float* poison;        // loss: set to NaN if a wait gives up
  int64_t n_rows;
};

__device__ __forceinline__ void fail(const HeadGemm& p, int bit) {
  atomicOr(&p.state->err, bit);
  for (int64_t i = 0; i < p.n_rows; ++i) p.poison[i] = __int_as_float(0x7fc00000);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// The products of the planes of A and B that are kept, smallest first.
__device__ __forceinline__ void plane_pair(int planes, int prod, int* a, int* b) {
  if (planes == 1) {
    *a = *b = 0;
  } else {
    // (2,0) (0,2) (1,1) (1,0) (0,1) (0,0)
    *a = (0x001102 >> (4 * prod)) & 0xf;
    *b = (0x010120 >> (4 * prod)) & 0xf;
  }
}

struct Tile {
  int m, n, s, kb0, kb1;
};

// Tiles in the order the CTA pairs take them: groups of kGroupM row tiles, column by column, so
// that the pairs at work share a few row and column panels in L2.
__device__ __forceinline__ Tile tile_at(int t, int mt, int nt, int splits, int kblocks) {
  Tile c;
  const int per = mt * nt;
  c.s = t / per;
  const int r = t - c.s * per;
  const int g = r / (kGroupM * nt), m0 = g * kGroupM;
  const int gs = min(kGroupM, mt - m0), q = r - m0 * nt;
  c.m = m0 + q % gs;
  c.n = q / gs;
  c.kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * c.s / splits);
  c.kb1 = static_cast<int>(static_cast<int64_t>(kblocks) * (c.s + 1) / splits);
  return c;
}

template <int EPI, int PLANES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    head_gemm_kernel(const __grid_constant__ HeadGemm p) {
  constexpr bool kAMn = EPI == DW, kBMn = EPI == DH || EPI == DW;
  constexpr int kProds = PLANES == 1 ? 1 : 6;
  constexpr uint32_t kIdesc = ptx::idesc_bf16(kTile, kTile, kAMn, kBMn);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);   // [kStages], of CTA 0
  uint64_t* empty = full + kStages;                               // [kStages], of each CTA
  uint64_t* accfull = empty + kStages;                            // [2], of each CTA
  uint64_t* accempty = accfull + 2;                               // [2], of CTA 0
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return ptx::mbar_wait_or_abort(bar, parity, kWaitLimitNs, abort_flag);
  };

  ptx::griddep_launch_dependents();
  if (warp == 0 && lane == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 2);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&accfull[b], 1);
      ptx::mbar_init(&accempty[b], 2 * kEpiWarps);
    }
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.mapA);
    ptx::prefetch_tmap(&p.mapB);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_slot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything read below (the live rows, and what the previous kernels wrote) is complete now
  ptx::griddep_wait();

  const int n_live = __ldcg(&p.state->n_live);
  const int mt = EPI == DW ? p.m_tiles : (n_live + kTile - 1) / kTile;
  const int kblocks = EPI == DW ? (n_live + kBK - 1) / kBK : p.kblocks;
  const int tiles = mt * p.n_tiles * p.splits;

  const int producer = warp == 0 ? 0 : (warp >= 2 + kEpiWarps ? warp - (1 + kEpiWarps) : -1);
  if (producer >= 0) {
    // ---------------- TMA producers ----------------
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      uint32_t full0[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) full0[s] = ptx::cluster_addr(&full[s], 0);
      for (int t = pair; ok && t < tiles; t += pairs) {
        const Tile c = tile_at(t, mt, p.n_tiles, p.splits, kblocks);
        const int am = c.m * kTile + static_cast<int>(rank) * kHalf;
        const int bn = c.n * kTile + static_cast<int>(rank) * kHalf;
        for (int prod = 0; ok && prod < kProds; ++prod) {
          int pa, pb;
          plane_pair(PLANES, prod, &pa, &pb);
          const int ax = pa * p.planeA, bx = pb * p.planeB;
          for (int kb = c.kb0; kb < c.kb1; ++kb, ++it) {
            if (static_cast<int>(it % kProducers) != producer) continue;
            const int s = it % kStages;
            const uint32_t use = it / kStages;
            if (use > 0 && !wait(&empty[s], (use - 1) & 1)) {
              fail(p, kErrTimeout);
              ok = false;
              break;
            }
            uint8_t* sa = smem + s * kStage;
            uint8_t* sb = sa + kStage / 2;
            const int k = kb * kBK;
            const uint32_t bar = ptx::cluster_addr(&full[s], 0);
#ifdef GRAPE_CHECKED
            const int xa = kAMn ? ax + am : ax + k, xb = kBMn ? bx + bn : bx + k;
            if (xa < 0 || xb < 0 || xa % 8 || xb % 8 || k < 0 || am < 0 || bn < 0) {
              atomicOr(&p.state->err, kErrBounds);
              continue;   // the stage never completes, and the bounded waits end the kernel
            }
#endif
            ptx::mbar_arrive_expect_tx_cluster(bar, kStage);
            if (kAMn) {
              ptx::tma_load_2d_pair(sa, &p.mapA, bar, ax + am, k);
              ptx::tma_load_2d_pair(sa + 8192, &p.mapA, bar, ax + am + 64, k);
            } else {
              ptx::tma_load_2d_pair(sa, &p.mapA, bar, ax + k, am);
            }
            if (kBMn) {
              const int y = EPI == DH ? p.v0 + k : k;
              ptx::tma_load_2d_pair(sb, &p.mapB, bar, bx + bn, y);
              ptx::tma_load_2d_pair(sb + 8192, &p.mapB, bar, bx + bn + 64, y);
            } else {
              ptx::tma_load_2d_pair(sb, &p.mapB, bar, bx + k, p.v0 + bn);
            }
          }
        }
      }
      // Neither CTA may leave while the pair's MMAs still signal its barriers: wait until the
      // last use of every stage of this producer is released.
      if (ok && !*abort_flag) {
        for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
          if (static_cast<int>(k % kProducers) == producer && !wait(&empty[k % kStages], (k / kStages) & 1)) {
            fail(p, kErrTimeout);
            break;
          }
      }
      if (*abort_flag) {   // let loads in flight land before the CTA leaves
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < kDrainNs) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ---------------- UMMA issuer (CTA 0) ----------------
    if (rank == 0 && lane == 0) {
      uint32_t it = 0, tc = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs, ++tc) {
        const Tile c = tile_at(t, mt, p.n_tiles, p.splits, kblocks);
        const int b = tc & 1;
        const uint32_t use = tc >> 1;
        if (use > 0 && !wait(&accempty[b], (use - 1) & 1)) {
          fail(p, kErrTimeout);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t dacc = tmem + b * kTile;
        const int steps = kProds * (c.kb1 - c.kb0);
        for (int i = 0; i < steps; ++i, ++it) {
          const int s = it % kStages;
          if (!wait(&full[s], (it / kStages) & 1)) {
            fail(p, kErrTimeout);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a_base = ptx::smem_u32(smem + s * kStage), b_base = a_base + kStage / 2;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            const uint64_t ad = kAMn ? ptx::desc_sw128(a_base + k * 2048, 8192, 1024)
                                     : ptx::desc_sw128(a_base + k * 32, 16, 1024);
            const uint64_t bd = kBMn ? ptx::desc_sw128(b_base + k * 2048, 8192, 1024)
                                     : ptx::desc_sw128(b_base + k * 32, 16, 1024);
            ptx::umma_bf16_pair(dacc, ad, bd, kIdesc, (i > 0 || k > 0) ? 1u : 0u);
          }
          ptx::umma_commit_pair(&empty[s]);
        }
        ptx::umma_commit_pair(&accfull[b]);
      }
    }
  } else {
    // ---------------- epilogue: warps 2..9 ----------------
    const int ew = warp - 2, q = warp & 3, h = ew >> 2;
    uint8_t* box = smem + kBoxOff + ew * kBox;
    uint4* box4 = reinterpret_cast<uint4*>(box);
    uint32_t tc = 0;
    for (int t = pair; t < tiles; t += pairs, ++tc) {
      const Tile c = tile_at(t, mt, p.n_tiles, p.splits, kblocks);
      const int b = tc & 1;
      const bool got = wait(&accfull[b], (tc >> 1) & 1);
      if (!got && lane == 0) fail(p, kErrTimeout);
      ptx::tc_fence_after();
      const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * kTile + h * kHalf;
      const int row0 = c.m * kTile + static_cast<int>(rank) * kHalf + q * 32;   // this warp's first row
      const int row = row0 + lane;
      const int col0 = c.n * kTile + h * kHalf;                                 // and column of the tile grid

      if (EPI == STATS) {
        const int label = row < n_live ? __ldcg(p.labels + row) : -1;
        float m = -INFINITY, s = 0.0f;
#pragma unroll 1
        for (int cc = 0; cc < kHalf; cc += 32) {
          float v[32];
          ptx::tmem_ld32(tbase + cc, v);
          const int c0 = col0 + cc;
          if (c0 + 32 > p.V) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c0 + j >= p.V) v[j] = -INFINITY;
          }
          if (label >= c0 && label < c0 + 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (label == c0 + j) p.target[row] = v[j];
          }
          float mm = m;
#pragma unroll
          for (int j = 0; j < 32; ++j) mm = fmaxf(mm, v[j]);
          const float r = mm == -INFINITY ? 0.0f : mm;   // nothing but -inf so far: sums stay 0
          s *= ex2((m - r) * kLog2e);
#pragma unroll
          for (int j = 0; j < 32; ++j) s += ex2((v[j] - r) * kLog2e);
          m = mm;
        }
        if (row < n_live) p.parts[static_cast<int64_t>(2 * c.n + h) * p.n_pad + row] = make_float2(m, s);
      } else if (EPI == GRAD) {
        const bool live = row < n_live;
        const int label = live ? __ldcg(p.labels + row) - p.v0 : -1;
        const float w = live ? __ldcg(p.weights + row) : 0.0f;
        const float lse = live ? __ldcg(p.lse + row) : 0.0f;
#pragma unroll 1
        for (int cc = 0; cc < kHalf; cc += 64) {
          float v[64];
          ptx::tmem_ld64(tbase + cc, v);
          const int c0 = col0 + cc;
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = w * ex2((v[j] - lse) * kLog2e);
          if (label >= c0 && label < c0 + 64) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (label == c0 + j) v[j] -= w;
          }
          if (!live || p.v0 + c0 + 64 > p.V) {   // rows and columns that only fill up the tile
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (!live || p.v0 + c0 + j >= p.V) v[j] = 0.0f;
          }
#pragma unroll
          for (int pl = 0; pl < PLANES; ++pl) {
            // the warp's 32 rows x 64 columns through its box, so that whole 128-byte lines are
            // written: unit u of row r sits at u ^ (r & 7)
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              uint4 x;
              x.x = pack2(v[8 * u + 0], v[8 * u + 1]);
              x.y = pack2(v[8 * u + 2], v[8 * u + 3]);
              x.z = pack2(v[8 * u + 4], v[8 * u + 5]);
              x.w = pack2(v[8 * u + 6], v[8 * u + 7]);
              box4[lane * 8 + (u ^ (lane & 7))] = x;
            }
            if (pl + 1 < PLANES) {
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] -= __bfloat162float(__float2bfloat16_rn(v[j]));
            }
            __syncwarp();
            const int u = lane & 7;
            __nv_bfloat16* dst = p.g + static_cast<int64_t>(row0) * p.ldg +
                                 static_cast<int64_t>(pl) * p.planeG + c0 + 8 * u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 4 * i + (lane >> 3);
              *reinterpret_cast<uint4*>(dst + rr * p.ldg) = box4[rr * 8 + (u ^ (rr & 7))];
            }
          }
        }
      } else {   // DH, DW: 32 columns at a time through the box
        const bool have = c.kb1 > c.kb0;
        const int M = EPI == DH ? n_live : p.V - p.v0;   // rows that exist
        float* acc = EPI == DH && p.acc ? p.acc + static_cast<int64_t>(c.s) * p.n_pad * p.ldacc : nullptr;
#pragma unroll 1
        for (int cc = 0; cc < kHalf; cc += 32) {
          float v[32];
          ptx::tmem_ld32(tbase + cc, v);
          const int c0 = col0 + cc;
          if (c0 >= p.d) continue;
          __syncwarp();
          float4* f4 = reinterpret_cast<float4*>(box);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            f4[lane * 8 + (u ^ (lane & 7))] = have ? make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3])
                                                   : make_float4(0.f, 0.f, 0.f, 0.f);
          __syncwarp();
          const int u = lane & 7, col = c0 + 4 * u;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), r = row0 + rr;
            if (r >= M || col >= p.d) continue;
            float4 x = f4[rr * 8 + (u ^ (rr & 7))];
            if (EPI == DH && acc) {
              float4* a = reinterpret_cast<float4*>(acc + r * p.ldacc + col);
              if (p.add) {
                const float4 y = *a;
                x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
              }
              if (!p.last) {
                *a = x;
                continue;
              }
            }
            const int64_t orow = EPI == DH ? __ldcg(p.rows + r) : p.v0 + r;
            if (PLANES == 3) {
              float* o = static_cast<float*>(p.out) + orow * p.d + col;
              if (p.d % 4 == 0) {
                *reinterpret_cast<float4*>(o) = x;
              } else {
                const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (col + k < p.d) o[k] = e[k];
              }
            } else {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + orow * p.d + col;
              if (p.d % 4 == 0) {
                *reinterpret_cast<uint2*>(o) = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
              } else {
                const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (col + k < p.d) o[k] = __float2bfloat16_rn(e[k]);
              }
            }
          }
        }
      }
      // this accumulator may be overwritten by the tile after next
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(ptx::cluster_addr(&accempty[b], 0));
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // the peer's arrivals on this CTA's barriers are in
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ---- the small kernels around the products -----------------------------------------------------

__device__ __forceinline__ int label_at(const void* labels, int id_bytes, int64_t n, int V) {
  const int64_t v = id_bytes == 8 ? static_cast<const long long*>(labels)[n]
                                  : static_cast<int64_t>(static_cast<const int*>(labels)[n]);
  return v >= 0 && v < V ? static_cast<int>(v) : -1;
}

// The live rows in order, then the dropped ones from the end backwards: rows[0 .. n_live) and
// rows[N-1], rows[N-2], ...  One CTA; dropped rows' losses are zeroed here.
__global__ void __launch_bounds__(1024) head_rows_kernel(const void* labels, int id_bytes, const float* weights,
                                                         int N, int V, HeadState* state, int* rows, int* lab, float* wgt,
                                                         float* loss) {
  ptx::griddep_launch_dependents();
  __shared__ int wtot[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int done = 0;   // live rows so far
  for (int n0 = 0; n0 < N; n0 += 1024) {
    const int n = n0 + tid;
    int label = -1;
    float w = 0.0f;
    if (n < N) {
      label = label_at(labels, id_bytes, n, V);
      w = weights ? weights[n] : 1.0f;
    }
    const bool live = label >= 0 && w != 0.0f;
    const uint32_t m = __ballot_sync(0xffffffffu, live);
    if (lane == 0) wtot[warp] = __popc(m);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      before += k < warp ? wtot[k] : 0;
      all += wtot[k];
    }
    const int at = done + before + __popc(m & ((1u << lane) - 1));
    if (live) {
      rows[at] = n;
      lab[at] = label;
      wgt[at] = w;
    } else if (n < N) {
      rows[N - 1 - (n - at)] = n;   // n - at dropped rows come before this one
      loss[n] = 0.0f;
    }
    done += all;
    __syncthreads();
  }
  if (tid == 0) {
    state->err = 0;
    state->n_live = done;
  }
}

// Row r of the compact H (bf16, or three planes of fp32), a CTA per row: the live rows, then zero
// rows up to a whole tile.  Dropped rows of dH are zeroed.
template <class T, int PLANES>
__global__ void __launch_bounds__(128) head_gather_kernel(const T* H, int d, int64_t N, const HeadState* state,
                                                          const int* rows, __nv_bfloat16* Hc, int plane, T* dH) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t r = blockIdx.x;
  const int n_live = __ldcg(&state->n_live);
  const int64_t fill = (static_cast<int64_t>(n_live) + kTile - 1) / kTile * kTile;
  __nv_bfloat16* dst = Hc + r * plane * PLANES;
  if (r < n_live) {
    const T* src = H + static_cast<int64_t>(__ldcg(rows + r)) * d;
    if (PLANES == 1 && d % 8 == 0) {
      for (int c = threadIdx.x; c < d / 8; c += 128)
        reinterpret_cast<uint4*>(dst)[c] = reinterpret_cast<const uint4*>(src)[c];
    } else {
      for (int c = threadIdx.x; c < plane; c += 128) {
        float x = c < d ? static_cast<float>(src[c]) : 0.0f;
#pragma unroll
        for (int k = 0; k < PLANES; ++k) {
          const __nv_bfloat16 b = __float2bfloat16_rn(x);
          dst[k * plane + c] = b;
          x -= __bfloat162float(b);
        }
      }
    }
    return;
  }
  if (r < fill)
    for (int c = threadIdx.x; c < plane * PLANES / 8; c += 128) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
  if (r < N && dH) {
    T* o = dH + static_cast<int64_t>(__ldcg(rows + r)) * d;
    for (int c = threadIdx.x; c < d; c += 128) o[c] = static_cast<T>(0.0f);
  }
}

// A copy of W that the tensor maps can address: rows padded to a multiple of eight, or three
// planes of an fp32 W.
template <class T, int PLANES>
__global__ void __launch_bounds__(128) head_weights_kernel(const T* W, int d, __nv_bfloat16* Wc, int plane) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t r = blockIdx.x;
  for (int c = threadIdx.x; c < plane; c += 128) {
    float x = c < d ? static_cast<float>(W[r * d + c]) : 0.0f;
#pragma unroll
    for (int k = 0; k < PLANES; ++k) {
      const __nv_bfloat16 b = __float2bfloat16_rn(x);
      Wc[(r * PLANES + k) * plane + c] = b;
      x -= __bfloat162float(b);
    }
  }
}

// lse and loss of 32 rows per CTA: eight threads share a row's partial sums, joined in order.
__global__ void __launch_bounds__(256) head_loss_kernel(const HeadState* state, const float2* parts, int slots,
                                                        int64_t n_pad, const float* target, const float* weights,
                                                        const int* rows, float* lse, float* loss) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  __shared__ float2 red[8][32];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int n_live = __ldcg(&state->n_live);
  const int row = blockIdx.x * 32 + lane;
  if (blockIdx.x * 32 >= n_live) return;
  float m = -INFINITY, s = 0.0f;
  auto join = [&](float m2, float s2) {
    const float mm = fmaxf(m, m2), r = mm == -INFINITY ? 0.0f : mm;
    s = s * ex2((m - r) * kLog2e) + s2 * ex2((m2 - r) * kLog2e);
    m = mm;
  };
  if (row < n_live)
    for (int k = part; k < slots; k += 8) {
      const float2 x = __ldcg(parts + k * n_pad + row);
      join(x.x, x.y);
    }
  red[part][lane] = make_float2(m, s);
  __syncthreads();
  if (part == 0 && row < n_live) {
    m = -INFINITY;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) join(red[k][lane].x, red[k][lane].y);
    const float l = m + logf(s);
    lse[row] = l;
    // log(s) - (target - m) rather than lse - target: the difference of the two large ones is exact
    float x = __ldcg(weights + row) * (logf(s) - (__ldcg(target + row) - m));
    if (__ldcg(&state->err)) x = __int_as_float(0x7fc00000);
    loss[__ldcg(rows + row)] = x;
  }
}

// dH from the splits of the vocabulary, added in order.
template <class T>
__global__ void __launch_bounds__(256) head_join_kernel(const HeadState* state, const float* acc, int splits,
                                                        int64_t n_pad, int64_t ldacc, int d, const int* rows, T* dH) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int n_live = __ldcg(&state->n_live);
  for (int64_t r = blockIdx.y; r < n_live; r += gridDim.y) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d) continue;
    float x = 0.0f;
    for (int s = 0; s < splits; ++s) x += __ldcg(acc + (s * n_pad + r) * ldacc + c);
    dH[static_cast<int64_t>(__ldcg(rows + r)) * d + c] = static_cast<T>(x);
  }
}

// ---- host ---------------------------------------------------------------------------------------

struct HeadPlan {
  int planes, plane;       // bf16 planes of an operand; elements of a plane's row
  bool copy_W;
  int64_t n_pad;
  int slots;               // 128-column slots of the vocabulary
  int piece, pieces;       // columns of a piece (a multiple of 256), pieces
  int splits;              // of DH
  bool acc;                // DH goes through fp32 memory
  int64_t ldacc;
  size_t o_rows, o_labels, o_weights, o_lse, o_target, o_parts, o_H, o_W, o_g, o_acc, bytes;

  explicit HeadPlan(const HeadShape& s) {
    planes = s.dtype == GRAPE_F32 ? 3 : 1;
    // three planes lie side by side, and a block of 64 must not reach into the next one
    plane = planes == 3 ? (s.d + 63) / 64 * 64 : (s.d + 7) / 8 * 8;
    copy_W = planes == 3 || plane != s.d;
    n_pad = (s.N + kTile - 1) / kTile * kTile;
    slots = (s.V + kTile - 1) / kTile * 2;
    const int64_t vmax = (static_cast<int64_t>(s.V) + kTile - 1) / kTile * kTile;
    int64_t cols = static_cast<int64_t>(kPieceBytes / (std::max<int64_t>(n_pad, 1) * 2 * planes)) / kTile * kTile;
    cols = std::min(std::max<int64_t>(cols, 4096), vmax);
    pieces = static_cast<int>((vmax + cols - 1) / cols);
    piece = static_cast<int>(((vmax + pieces - 1) / pieces + kTile - 1) / kTile * kTile);
    pieces = static_cast<int>((vmax + piece - 1) / piece);
    // few tiles of dH: its long sum over the vocabulary is split over the CTA pairs, at least
    // eight blocks of 64 each
    const int64_t out_tiles = n_pad / kTile * ((s.d + kTile - 1) / kTile);
    splits = 1;
    if (s.dH && pieces == 1 && out_tiles > 0 && out_tiles < 74)
      splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(74 / out_tiles, piece / kBK / 8)));
    acc = s.dH && (pieces > 1 || splits > 1);
    ldacc = (s.d + 3) / 4 * 4;
    size_t o = 256;
    auto take = [&](size_t b) {
      const size_t at = o;
      o += lm_round256(b);
      return at;
    };
    const size_t np = static_cast<size_t>(n_pad);
    const bool grads = s.dH || s.dW;
    o_rows = take(np * 4);
    o_labels = take(np * 4);
    o_weights = take(np * 4);
    o_lse = take(np * 4);
    o_target = take(np * 4);
    o_parts = take(np * slots * 8);
    o_H = take(np * plane * planes * 2);
    o_W = take(copy_W ? static_cast<size_t>(s.V) * plane * planes * 2 : 0);
    o_g = take(grads ? np * piece * planes * 2 : 0);
    o_acc = take(acc ? np * ldacc * splits * 4 : 0);
    bytes = o;
  }
};

template <class Kern, class... Args>
cudaError_t launch(bool pdl, Kern kernel, dim3 grid, unsigned block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int EPI, int PLANES>
cudaError_t run_gemm(const HeadGemm& p, int64_t max_tiles, cudaStream_t st) {
  const void* k = reinterpret_cast<const void*>(head_gemm_kernel<EPI, PLANES>);
  cudaError_t e = tc_configure_kernel(k, kSmem, kThreads);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tc_sm_count() / 2, max_tiles));
  return launch(true, head_gemm_kernel<EPI, PLANES>, dim3(static_cast<unsigned>(2 * pairs)), kThreads, kSmem, st, p);
}

template <class T, int PLANES>
cudaError_t run_head(const HeadShape& s, const T* H, const T* W, const void* labels, int id_bytes,
                     const float* weights, char* ws, float* loss, T* dH, T* dW, cudaStream_t st) {
  const HeadPlan pl(s);
  HeadState* state = reinterpret_cast<HeadState*>(ws);
  int* rows = reinterpret_cast<int*>(ws + pl.o_rows);
  int* lab = reinterpret_cast<int*>(ws + pl.o_labels);
  float* wgt = reinterpret_cast<float*>(ws + pl.o_weights);
  float* lse = reinterpret_cast<float*>(ws + pl.o_lse);
  float* target = reinterpret_cast<float*>(ws + pl.o_target);
  float2* parts = reinterpret_cast<float2*>(ws + pl.o_parts);
  __nv_bfloat16* Hc = reinterpret_cast<__nv_bfloat16*>(ws + pl.o_H);
  __nv_bfloat16* Wc = pl.copy_W ? reinterpret_cast<__nv_bfloat16*>(ws + pl.o_W)
                                : const_cast<__nv_bfloat16*>(reinterpret_cast<const __nv_bfloat16*>(W));
  __nv_bfloat16* g = reinterpret_cast<__nv_bfloat16*>(ws + pl.o_g);
  const int wide = pl.plane * PLANES;
  const int64_t gw = static_cast<int64_t>(pl.piece) * PLANES;

  cudaError_t e = launch(false, head_rows_kernel, dim3(1), 1024, 0, st, labels, id_bytes, weights,
                         static_cast<int>(s.N), s.V, state, rows, lab, wgt, loss);
  if (e == cudaSuccess && s.N > 0)
    e = launch(true, head_gather_kernel<T, PLANES>, dim3(static_cast<unsigned>(pl.n_pad)), 128, 0, st, H, s.d, s.N,
               static_cast<const HeadState*>(state), static_cast<const int*>(rows), Hc, pl.plane, dH);
  if (e == cudaSuccess && pl.copy_W)
    e = launch(true, head_weights_kernel<T, PLANES>, dim3(s.V), 128, 0, st, W, s.d, Wc, pl.plane);
  if (e != cudaSuccess) return e;
  if (s.N == 0) return dW ? cudaMemsetAsync(dW, 0, static_cast<size_t>(s.V) * s.d * sizeof(T), st) : cudaSuccess;

  // operand views: K-major boxes of 64 x 128 rows, M/N-major boxes of 64 x 64
  CUtensorMap H_k, H_mn, W_k, W_mn, g_k, g_mn;
  if (!tc_map_2d(&H_k, Hc, pl.n_pad, wide, wide, kBK, kHalf) || !tc_map_2d(&W_k, Wc, s.V, wide, wide, kBK, kHalf))
    return cudaErrorInvalidValue;
  HeadGemm p;
  std::memset(&p, 0, sizeof(p));
  p.state = state;
  p.V = s.V;
  p.d = s.d;
  p.n_pad = pl.n_pad;
  p.labels = lab;
  p.weights = wgt;
  p.lse = lse;
  p.parts = parts;
  p.target = target;
  p.g = g;
  p.ldg = gw;
  p.planeG = pl.piece;
  p.rows = rows;
  p.poison = loss;
  p.n_rows = s.N;
  p.splits = 1;

  const int64_t mt = pl.n_pad / kTile;
  p.mapA = H_k;
  p.mapB = W_k;
  p.planeA = p.planeB = pl.plane;
  p.kblocks = (pl.plane + kBK - 1) / kBK;
  p.n_tiles = pl.slots / 2;
  e = run_gemm<STATS, PLANES>(p, mt * p.n_tiles, st);
  if (e == cudaSuccess)
    e = launch(true, head_loss_kernel, dim3(static_cast<unsigned>((s.N + 31) / 32)), 256, 0, st,
               static_cast<const HeadState*>(state), static_cast<const float2*>(parts), pl.slots, pl.n_pad,
               static_cast<const float*>(target), static_cast<const float*>(wgt), static_cast<const int*>(rows), lse,
               loss);
  if (e != cudaSuccess || (!s.dH && !s.dW)) return e;

  if (!tc_map_2d(&H_mn, Hc, pl.n_pad, wide, wide, 64, kBK) || !tc_map_2d(&W_mn, Wc, s.V, wide, wide, 64, kBK) ||
      !tc_map_2d(&g_k, g, pl.n_pad, gw, gw, kBK, kHalf) || !tc_map_2d(&g_mn, g, pl.n_pad, gw, gw, 64, kBK))
    return cudaErrorInvalidValue;
  const int dt = (s.d + kTile - 1) / kTile;
  for (int i = 0; i < pl.pieces; ++i) {
    const int v0 = i * pl.piece, cols = std::min(pl.piece, s.V - v0), vt = (cols + kTile - 1) / kTile;
    HeadGemm q = p;
    q.v0 = v0;
    q.n_tiles = vt;
    e = run_gemm<GRAD, PLANES>(q, mt * vt, st);
    if (e != cudaSuccess) return e;
    if (s.dH) {
      HeadGemm y = q;
      y.mapA = g_k;
      y.mapB = W_mn;
      y.planeA = pl.piece;
      y.kblocks = (cols + kBK - 1) / kBK;
      y.n_tiles = dt;
      y.splits = pl.splits;
      y.acc = pl.acc ? reinterpret_cast<float*>(ws + pl.o_acc) : nullptr;
      y.ldacc = pl.ldacc;
      y.add = i > 0;
      y.last = i + 1 == pl.pieces && pl.splits == 1;
      y.out = dH;
      e = run_gemm<DH, PLANES>(y, mt * dt * pl.splits, st);
      if (e != cudaSuccess) return e;
    }
    if (s.dW) {
      HeadGemm x = q;
      x.mapA = g_mn;
      x.mapB = H_mn;
      x.planeA = pl.piece;
      x.m_tiles = vt;
      x.n_tiles = dt;
      x.out = dW;
      e = run_gemm<DW, PLANES>(x, static_cast<int64_t>(vt) * dt, st);
      if (e != cudaSuccess) return e;
    }
  }
  if (s.dH && pl.splits > 1)
    e = launch(true, head_join_kernel<T>, dim3((s.d + 255) / 256, static_cast<unsigned>(std::min<int64_t>(s.N, 4096))), 256,
               0, st, static_cast<const HeadState*>(state), reinterpret_cast<const float*>(ws + pl.o_acc), pl.splits,
               pl.n_pad, pl.ldacc, s.d, static_cast<const int*>(rows), dH);
  return e;
}

}  // namespace

size_t head_workspace_bytes(const HeadShape& s) { return HeadPlan(s).bytes; }

cudaError_t head_loss(const HeadShape& s, const void* H, const void* W, const void* labels, int id_bytes,
                      const float* weights, void* ws, float* loss, void* dH, void* dW, cudaStream_t st) {
  char* w = static_cast<char*>(ws);
  if (s.dtype == GRAPE_F32)
    return run_head<float, 3>(s, static_cast<const float*>(H), static_cast<const float*>(W), labels, id_bytes, weights,
                              w, loss, static_cast<float*>(dH), static_cast<float*>(dW), st);
  return run_head<__nv_bfloat16, 1>(s, static_cast<const __nv_bfloat16*>(H), static_cast<const __nv_bfloat16*>(W),
                                    labels, id_bytes, weights, w, loss, static_cast<__nv_bfloat16*>(dH),
                                    static_cast<__nv_bfloat16*>(dW), st);
}

}  // namespace grape
