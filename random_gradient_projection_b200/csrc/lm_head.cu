// Softmax cross entropy of a vocabulary head, with gradients, that never holds the logits:
//
//   z_nv = h_n . W_v                     N live rows, V vocabulary rows, d wide
//   l_n  = w_n (lse_v z_nv - z_{n,label})
//   g_nv = w_n (exp(z_nv - lse_n) - [v = label_n])
//   dH_n = sum_v g_nv W_v,   dW_v = sum_n g_nv h_n
//
// The contractions run on one warp-specialised kernel, head_gemm_kernel<EPI, PLANES>:
//
//   STATS  z over the whole vocabulary, reduced in the epilogue to a maximum and a sum of
//          exponentials per row and tile, and the label's logit beside them
//   GRAD   z again for one piece of the vocabulary; the epilogue writes g for the piece
//   EXP    z once for one piece; the epilogue writes e_nv = exp(z_nv - r_n) and its row sums,
//          with a reference r_n that is known beforehand
//   DH     dH (+)= g W, or e W, over the piece (K = the piece's columns, split when rows are few)
//   DW     dW of the piece = g^T H             (K = rows)
//
// so the memory is one piece of g (at most kPieceBytes, or 4096 columns), whatever V is.
//
// With dW, or for a small problem, STATS comes first and GRAD recomputes z: 6 (8) N V d flops for
// dH (and dW), where keeping the logits takes 4 (6).  With dH alone the recomputation is not needed:
// softmax times W can be summed before the softmax is normalised,
//
//   dH_n = w_n (sum_{v != label} e_nv W_v / s_n - (1 - p_n) W_label),   s_n = sum_v e_nv,
//
// and the label's own logit, one short dot product per row, is a reference r_n that keeps every
// e_nv at most exp(l_n) and s_n at least 1.  So EXP overflows only where a row's loss passes 60;
// an epilogue that sees this sets `retry`, and the two-pass kernels, which are launched behind
// and otherwise leave at once, compute the call anew: one such row makes the whole call take 2.4 times
// as long (8192 x 4096 x 32000: 3.5 -> 8.4 ms).
//
// Both ways leave the label's column out of the sum s'_n, so that what is small for a row that is
// sure of its label never is a difference of large numbers: 1 - p_n = s'_n / s_n with s_n = s'_n +
// e_label, l_n = log1p(s'_n / e_label), and g's entry at the label is -w_n s'_n / s_n (from p_n - 1
// it would be off by 2^-24 of the largest logit, all of it at 1 - p_n = 1e-6).
//
// Rows without a loss (label outside [0, V), or weight 0) are dropped first: where there are any,
// the live rows are gathered in order into a compact H, so masked rows enter no product, and whatever
// they hold (NaN included) reaches no sum.  The number of live rows is known on the device only;
// every kernel reads it there.  (The plan - pieces, splits, one pass or two - and the workspace are
// made for all N rows, so a call with few live ones fills the machine less well: 8192 x 1024 x
// 32000 dH takes 1005 us, with half of the rows masked 540, with 90 % 278.)
//
// Precision.  bf16 inputs: products are exact in the tensor core and accumulate in fp32; g (or e) is
// rounded once to bf16 as the operand of the second product (relative 2^-8 at most per element,
// independent from element to element, so it averages out in the sums), as the method's own
// step does with AP.  fp32 inputs (PLANES = 3): each operand is split into three bf16 planes
// x = x0 + x1 + x2 (24 bits together) and the six products of order up to 2^-16 are accumulated,
// smallest first; the three dropped ones are below 2^-24 relative.  Six tensor-core products
// run several times faster than one on the fp32 cores.  The tensor core's accumulator truncates at
// every step (measured: logits of one sign come out low by 1.7e-8 per step of K = 16, 4.2e-6 at
// d = 4096), so sums that end in an fp32 result leave TMEM every kChunk blocks and are added,
// rounded to nearest, in registers.
//
// The kernel: a cluster of two CTAs (one tile of 256 x 256, cta_group::2), each CTA with half of
// A's rows and half of B's columns in its ring of shared-memory stages.  Warp 17 of each
// CTA loads by TMA, warp 16 of CTA 0 issues the MMAs for both, warps 0-15 are the epilogue of their
// CTA's 128 rows (each 32 rows x 64 columns, in registers); two 256-column accumulators in TMEM
// let it overlap the next sums.  Bound by the tensor pipe where d is large: at 8192 x 4096 x 32000 EXP
// runs at 1547 and DH at 1564 TFLOP/s in bursts (a library product of that size: 1596), both at 1262
// under the power cap (library 1376); with d of a few hundred the epilogue's exponentials bound it.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "lm.h"
#include "lm_launch.h"
#include "lm_ptx.cuh"

namespace grape {
namespace {

constexpr int kTile = 256;            // rows and columns of a tile
constexpr int kHalf = 128;            // of a CTA
constexpr int kBK = 64;
constexpr int kStages = 6;
constexpr int kStage = 2 * kHalf * kBK * 2;   // A half and B half: 32 KB
constexpr int kEpiWarps = 16;
constexpr int kCols = 64;             // columns of an epilogue warp
constexpr int kMmaWarp = kEpiWarps, kLoadWarp = kEpiWarps + 1;   // of a fifth warpgroup
constexpr int kThreads = 32 * (kEpiWarps + 4);
// Registers per thread: 640 threads are launched with 96 each (61440); the epilogue's 512 take
// 112, the other 128 keep 32 (61440 again; without this the epilogues spill).
constexpr int kRegsLaunch = 96, kRegsEpi = 112, kRegsOther = 32;
static_assert(kThreads == 640 && 512 * kRegsEpi + 128 * kRegsOther <= kThreads * kRegsLaunch, "register split");
constexpr int kBox = 32 * 64;         // an epilogue warp's staging box: 32 rows x 64 bytes
constexpr int kBarOff = kStages * kStage;
constexpr int kBoxOff = kBarOff + 1024;
constexpr int kSmem = kBoxOff + kEpiWarps * kBox + 1024;   // + alignment slack
static_assert(kBoxOff % 1024 == 0, "boxes are aligned");
static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
// Blocks of 64 of a split of DH at least: a block is 8.4 MFLOP, 0.38 us at a pair's share of the
// measured rate, and joining the splits takes 3 us.  (dH with 6 / 24 / 96, us: 64 x 256 x 1000 31 / 33 /
// 33, 64 x 1024 x 32000 57 / 57 / 73, 512 x 1024 x 32000 88 / 88 / 98, 2048 x 1024 x 32000 255 / 246 / 261.)
constexpr int kSplitBlocks = 24;
// Row tiles that share a column of B tiles in L2 (4 / 8 / 16: 2048 x 1024 x 50265 399-421 / 395-400 /
// 397 us, 8192 x 4096 x 32000 3536-3609 / 3464-3535 / 3481-3517).
constexpr int kGroupM = 8;
constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr uint64_t kDrainNs = 20000000ull;
constexpr size_t kPieceBytes = size_t(256) << 20;
constexpr float kExpLimit = 1e26f;     // exp(60): sums of 2^17 such terms, times W, stay in fp32
constexpr int kErrTimeout = 1;
#ifdef GRAPE_CHECKED
constexpr int kErrBounds = 8;   // a TMA box off the 16-byte rule or at a negative coordinate (skipped)
#endif

enum Epi : int { STATS = 0, GRAD = 1, EXP = 2, DH = 3, DW = 4 };

// Blocks of 64 that stay in the tensor core's accumulator at most.
template <int EPI, int PLANES>
struct Chunk {
  static constexpr int kBlocks = PLANES == 3 ? 8 : (EPI == STATS || EPI == EXP) ? 16 : 1 << 30;
};

// Device words at the start of the workspace.
struct HeadState {
  int err;
  int n_live;
  int retry;   // EXP met a row whose loss is too large for its reference
};

struct HeadGemm {
  CUtensorMap mapA, mapB;
  CUtensorMap mapH;     // H itself in place of its compact copy, when every row is live
  int direct;           // mapH may be used: 1 for A, 2 for B
  HeadState* state;
  int only_retry;       // leave at once unless state->retry
  int m_tiles;          // DW: vocabulary tiles of the piece; otherwise from n_live
  int n_tiles, splits;  // column tiles; parts of the K extent (DH)
  int kblocks;          // K extent in blocks of 64 (DW: from n_live)
  int planeA, planeB;   // elements from one plane of an operand to the next
  int v0, V, d;         // first vocabulary row of the piece; sizes
  int64_t n_pad;        // rows of the compact buffers
  const int* labels;    // compact rows
  const float* ref;     // EXP: r_n; GRAD: the row's largest logit
  const float2* scale;  // GRAD: w / s and w s' / s
  float2* parts;        // STATS: [tile][n_pad] (maximum, sum of exponentials), the label's column
                        // left out; EXP: (sum, unused)
  float* target;        // STATS: the label's logit; EXP: less r_n
  __nv_bfloat16* g;     // GRAD, EXP: [n_pad][ldg]
  int64_t ldg;
  int planeG;           // elements from one plane of g to the next
  float* acc;           // DH: [split][n_pad][ldacc] fp32 (several pieces or splits)
  int64_t ldacc;
  int add, last;        // DH: add to acc; write the result (no later piece, no splits)
  const float2* coef;   // DH after EXP: w / s and w s' / s; null after GRAD
  const void* W;        // DH after EXP: W as given, for the label's row
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

__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory"); }

template <int PLANES>
struct HeadType {
  using T = __nv_bfloat16;
};
template <>
struct HeadType<3> {
  using T = float;
};

// Four consecutive results of a row, from column `col` on; those from d on do not exist.
__device__ __forceinline__ void store4(float* o, const float (&x)[4], int col, int d) {
  if (d % 4 == 0) {
    *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k < d) o[k] = x[k];
  }
}
__device__ __forceinline__ void store4(__nv_bfloat16* o, const float (&x)[4], int col, int d) {
  if (d % 4 == 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k < d) o[k] = __float2bfloat16_rn(x[k]);
  }
}

template <int EPI, int PLANES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    head_gemm_kernel(const __grid_constant__ HeadGemm p) {
  constexpr bool kAMn = EPI == DW, kBMn = EPI == DH || EPI == DW;
  constexpr int kProds = PLANES == 1 ? 1 : 6;
  constexpr int kChunk = Chunk<EPI, PLANES>::kBlocks;
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
    return ptx::mbar_wait_suspend_or_abort(bar, parity, kWaitLimitNs, abort_flag);
  };

  ptx::griddep_launch_dependents();
  if (p.only_retry) {
    ptx::griddep_wait();
    if (__ldcg(&p.state->retry) == 0) return;   // the same in every thread of the grid
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
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
  if (warp == kMmaWarp) {
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

  if (warp >= kMmaWarp) {
    ptx::setmaxnreg_dec<kRegsOther>();   // the whole warpgroup, one instruction
    if (warp == kLoadWarp) {
      // ---------------- TMA producer ----------------
      if (lane == 0) {
        const bool all_live = n_live == p.n_rows;
        const CUtensorMap* mapA = p.direct == 1 && all_live ? &p.mapH : &p.mapA;
        const CUtensorMap* mapB = p.direct == 2 && all_live ? &p.mapH : &p.mapB;
        uint32_t it = 0;
        bool ok = true;
        for (int t = pair; ok && t < tiles; t += pairs) {
          const Tile c = tile_at(t, mt, p.n_tiles, p.splits, kblocks);
          const int am = c.m * kTile + static_cast<int>(rank) * kHalf;
          const int bn = c.n * kTile + static_cast<int>(rank) * kHalf;
          for (int prod = 0; ok && prod < kProds; ++prod) {
            int pa, pb;
            plane_pair(PLANES, prod, &pa, &pb);
            const int ax = pa * p.planeA, bx = pb * p.planeB;
            for (int kb = c.kb0; kb < c.kb1; ++kb, ++it) {
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
              // CTA 0 announces the bytes of both (those of CTA 1 may land first: the phase still waits for
              // this one arrival).  With a remote arrival of CTA 1's own one loading thread fed 780
              // TFLOP/s, so 1435.
              if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * kStage);
              if (kAMn) {
                ptx::tma_load_2d_pair(sa, mapA, bar, ax + am, k);
                ptx::tma_load_2d_pair(sa + 8192, mapA, bar, ax + am + 64, k);
              } else {
                ptx::tma_load_2d_pair(sa, mapA, bar, ax + k, am);
              }
              if (kBMn) {
                const int y = EPI == DH ? p.v0 + k : k;
                ptx::tma_load_2d_pair(sb, mapB, bar, bx + bn, y);
                ptx::tma_load_2d_pair(sb + 8192, mapB, bar, bx + bn + 64, y);
              } else {
                ptx::tma_load_2d_pair(sb, mapB, bar, bx + k, p.v0 + bn);
              }
            }
          }
        }
        // Neither CTA may leave while the pair's MMAs still signal its barriers: wait until the
        // last use of every stage is released.
        if (ok && !*abort_flag) {
          for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
            if (!wait(&empty[k % kStages], (k / kStages) & 1)) {
              fail(p, kErrTimeout);
              break;
            }
        }
        if (*abort_flag) {   // let loads in flight land before the CTA leaves
          const uint64_t t0 = ptx::globaltimer_ns();
          while (ptx::globaltimer_ns() - t0 < kDrainNs) __nanosleep(1000);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------- UMMA issuer (CTA 0) ----------------
      if (rank == 0 && lane == 0) {
        uint32_t it = 0, ch = 0;   // stage uses, accumulator uses
        bool ok = true;
        for (int t = pair; ok && t < tiles; t += pairs) {
          const Tile c = tile_at(t, mt, p.n_tiles, p.splits, kblocks);
          const int steps = kProds * (c.kb1 - c.kb0);
          int i = 0;
          do {
            const int b = ch & 1;
            const uint32_t use = ch >> 1;
            if (use > 0 && !wait(&accempty[b], (use - 1) & 1)) {
              fail(p, kErrTimeout);
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t dacc = tmem + b * kTile;
            const int i0 = i, i1 = steps - i > kChunk ? i + kChunk : steps;
            for (; i < i1; ++i, ++it) {
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
                ptx::umma_bf16_pair(dacc, ad, bd, kIdesc, (i > i0 || k > 0) ? 1u : 0u);
              }
              ptx::umma_commit_pair(&empty[s]);
            }
            ptx::umma_commit_pair(&accfull[b]);
            ++ch;
          } while (ok && i < steps);
        }
      }
    }
  } else {
    // ---------------- epilogue: warps 0..15 ----------------
    // Warp w: TMEM lanes 32 (w % 4).. (a hardware rule) and 64 of the tile's columns.
    ptx::setmaxnreg_inc<kRegsEpi>();
    const int q = warp & 3, h = warp >> 2;
    uint8_t* box = smem + kBoxOff + warp * kBox;
    // this lane's two values in the box of the warp with this lane quarter and columns h2 (STATS, which
    // stages nothing in the boxes, has two places in turn)
    auto part_of = [&](int h2, uint32_t turn) {
      return reinterpret_cast<float2*>(smem + kBoxOff + (4 * h2 + q) * kBox) + lane + (EPI == STATS ? 32 * (turn & 1) : 0);
    };
    uint32_t turn = 0;
    uint32_t ch = 0;
    auto release = [&]() {   // this accumulator may be overwritten
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(ptx::cluster_addr(&accempty[ch & 1], 0));
      ++ch;
    };
    for (int t = pair; t < tiles; t += pairs) {
      const Tile c = tile_at(t, mt, p.n_tiles, p.splits, kblocks);
      const int steps = kProds * (c.kb1 - c.kb0);
      const int row0 = c.m * kTile + static_cast<int>(rank) * kHalf + q * 32;   // this warp's first row
      const int row = row0 + lane;
      const int col0 = c.n * kTile + h * kCols;   // and column, within the piece

      // the sum of the chunks (every warp walks all of them even after a failed wait, whose
      // successors then return at once, so that the barriers below are reached by all)
      // (bf16 results of one chunk are read out 16 columns at a time further down instead)
      constexpr bool kStream = (EPI == DH || EPI == DW) && PLANES == 1;
      float v[kCols];
      int i = 0;
      do {
        const int b = ch & 1;
        const bool got = wait(&accfull[b], (ch >> 1) & 1);
        if (!got && lane == 0) fail(p, kErrTimeout);
        ptx::tc_fence_after();
        if (kStream) break;
        const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * kTile + h * kCols;
        if (i == 0) {
          ptx::tmem_ld64(tbase, v);
        } else {
#pragma unroll
          for (int cc = 0; cc < kCols; cc += 8) {
            float x[8];
            ptx::tmem_ld8(tbase + cc, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[cc + j] += x[j];
          }
        }
        release();
        i = steps - i > kChunk ? i + kChunk : steps;
      } while (i < steps);

      if (EPI == STATS || EPI == EXP || EPI == GRAD) {
        const bool live = row < n_live;
        const int label = live ? __ldcg(p.labels + row) - p.v0 : -1;
        const int left = p.V - p.v0 - col0;   // columns of this warp that exist
        float2 part = make_float2(0.0f, 0.0f);
        if (EPI == STATS) {
          if (left < kCols) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (j >= left) v[j] = -INFINITY;
          }
          if (label >= col0 && label < col0 + kCols) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (label == col0 + j) {
                p.target[row] = v[j];
                v[j] = -INFINITY;   // left out of the sums
              }
          }
          float m = v[0];
#pragma unroll
          for (int j = 1; j < kCols; ++j) m = fmaxf(m, v[j]);
          const float r = m == -INFINITY ? 0.0f : m;   // nothing but -inf: the sum stays 0
          float s = 0.0f;
#pragma unroll
          for (int j = 0; j < kCols; ++j) s += ex2((v[j] - r) * kLog2e);
          part = make_float2(m, s);
        } else {
          const float2 w = EPI == GRAD && live ? __ldcg(p.scale + row) : make_float2(1.0f, 0.0f);
          const float r = live ? __ldcg(p.ref + row) : 0.0f;
          if (EPI == EXP && label >= col0 && label < col0 + kCols) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (label == col0 + j) {
                // (the reference is this logit up to rounding: far off it, nothing below would hold)
                if (!(fabsf(v[j] - r) < 60.0f)) atomicOr(&p.state->retry, 1);
                p.target[row] = v[j] - r;
                v[j] = -INFINITY;   // left out of the sums
              }
          }
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] = w.x * ex2((v[j] - r) * kLog2e);
          if (EPI == GRAD && label >= col0 && label < col0 + kCols) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (label == col0 + j) v[j] = -w.y;
          }
          if (!live || left < kCols) {   // rows and columns that only fill up the tile
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (!live || j >= left) v[j] = 0.0f;
          }
          if (EPI == EXP) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < kCols; ++j) s += v[j];
            if (s > kExpLimit) atomicOr(&p.state->retry, 1);
            part = make_float2(s, 0.0f);
          }
#pragma unroll
          for (int pl = 0; pl < PLANES; ++pl) {
#pragma unroll
            for (int half = 0; half < kCols; half += 32) {
              // the warp's 32 rows x 32 columns through its box, so that pieces of 64 bytes are
              // written: unit u of row r sits at u ^ (r / 2 % 4)
              uint4* box4 = reinterpret_cast<uint4*>(box);
              __syncwarp();
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int j = half + 8 * u;
                box4[lane * 4 + (u ^ ((lane >> 1) & 3))] =
                    make_uint4(pack2(v[j], v[j + 1]), pack2(v[j + 2], v[j + 3]), pack2(v[j + 4], v[j + 5]),
                               pack2(v[j + 6], v[j + 7]));
              }
              __syncwarp();
              const int u = lane & 3;
              __nv_bfloat16* dst = p.g + static_cast<int64_t>(row0) * p.ldg + static_cast<int64_t>(pl) * p.planeG + col0 +
                                   half + 8 * u;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int rr = 8 * k + (lane >> 2);
                *reinterpret_cast<uint4*>(dst + rr * p.ldg) = box4[rr * 4 + (u ^ ((rr >> 1) & 3))];
              }
            }
            if (pl + 1 < PLANES) {
#pragma unroll
              for (int j = 0; j < kCols; ++j) v[j] -= __bfloat162float(__float2bfloat16_rn(v[j]));
            }
          }
        }
        if (EPI != GRAD) {
          // the row's four parts, one per warp of its lane quarter, joined in order
          __syncwarp();   // the box has been read out
          *part_of(h, turn) = part;
          epi_bar();
          if (h == 0 && live) {
            float2 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = *part_of(k, turn);
            float2 y;
            if (EPI == EXP) {
              y = make_float2(((x[0].x + x[1].x) + x[2].x) + x[3].x, 0.0f);
            } else {
              const float m = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
              const float r = m == -INFINITY ? 0.0f : m;
              float s = 0.0f;
#pragma unroll
              for (int k = 0; k < 4; ++k) s += x[k].y * ex2((x[k].x - r) * kLog2e);
              y = make_float2(m, s);
            }
            p.parts[static_cast<int64_t>(p.v0 / kTile + c.n) * p.n_pad + row] = y;
          }
          if (EPI != STATS) epi_bar();   // the boxes may be written again
          ++turn;
        }
      } else {   // DH, DW: 16 columns at a time through the box
        using T = typename HeadType<PLANES>::T;
        const bool have = steps > 0;
        const int M = EPI == DH ? n_live : p.V - p.v0;   // rows that exist
        float* acc = EPI == DH && p.acc ? p.acc + static_cast<int64_t>(c.s) * p.n_pad * p.ldacc : nullptr;
        float4* f4 = reinterpret_cast<float4*>(box);
        auto put16 = [&](int cc, const float* x16) {
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 4; ++u)
            f4[lane * 4 + (u ^ ((lane >> 1) & 3))] =
                have ? make_float4(x16[4 * u], x16[4 * u + 1], x16[4 * u + 2], x16[4 * u + 3])
                     : make_float4(0.f, 0.f, 0.f, 0.f);
          __syncwarp();
          const int u = lane & 3, col = col0 + cc + 4 * u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = 8 * k + (lane >> 2), r = row0 + rr;
            if (r >= M || col >= p.d) continue;
            const float4 x4 = f4[rr * 4 + (u ^ ((rr >> 1) & 3))];
            float x[4] = {x4.x, x4.y, x4.z, x4.w};
            if (EPI == DH && acc) {
              float4* a = reinterpret_cast<float4*>(acc + r * p.ldacc + col);
              if (p.add) {
                const float4 y = *a;
                x[0] += y.x, x[1] += y.y, x[2] += y.z, x[3] += y.w;
              }
              if (!p.last) {
                *a = make_float4(x[0], x[1], x[2], x[3]);
                continue;
              }
            }
            if (EPI == DH && p.coef) {
              const float2 co = __ldcg(p.coef + r);
              const T* wl = static_cast<const T*>(p.W) + static_cast<int64_t>(__ldcg(p.labels + r)) * p.d + col;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + e < p.d) x[e] = co.x * x[e] - co.y * static_cast<float>(wl[e]);
            }
            const int64_t orow = EPI == DH ? __ldcg(p.rows + r) : p.v0 + r;
            store4(static_cast<T*>(p.out) + orow * p.d + col, x, col, p.d);
          }
        };
        if (kStream) {
          const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + (ch & 1) * kTile + h * kCols;
#pragma unroll 1
          for (int cc = 0; cc < kCols; cc += 16) {
            float x[16];
            ptx::tmem_ld16(tbase + cc, x);
            if (col0 + cc < p.d) put16(cc, x);
          }
          release();
        } else {
#pragma unroll
          for (int cc = 0; cc < kCols; cc += 16)
            if (col0 + cc < p.d) put16(cc, v + cc);
        }
      }
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // the peer's arrivals on this CTA's barriers are in
  if (warp == kMmaWarp) {
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
// rows[N-1], rows[N-2], ...  One CTA, 8192 rows at a time with all their loads in flight; dropped
// rows' losses are zeroed here.
constexpr int kRowsPer = 8;
__global__ void __launch_bounds__(1024) head_rows_kernel(const void* labels, int id_bytes, const float* weights,
                                                         int N, int V, HeadState* state, int* rows, int* lab, float* wgt,
                                                         float* loss) {
  ptx::griddep_launch_dependents();
  __shared__ int tot[kRowsPer * 32], scan[kRowsPer * 32 + 1], wsum[kRowsPer];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int done = 0;   // live rows so far
  for (int n0 = 0; n0 < N; n0 += 1024 * kRowsPer) {
    int label[kRowsPer];
    float w[kRowsPer];
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      const int n = n0 + k * 1024 + tid;
      label[k] = n < N ? label_at(labels, id_bytes, n, V) : -1;
      w[k] = n < N && weights ? weights[n] : 1.0f;
    }
    uint32_t m[kRowsPer];
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      m[k] = __ballot_sync(0xffffffffu, label[k] >= 0 && w[k] != 0.0f);
      if (lane == 0) tot[k * 32 + warp] = __popc(m[k]);
    }
    __syncthreads();
    if (tid < kRowsPer * 32) {   // exclusive scan of the 256 counts
      const int x = tot[tid];
      int incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      scan[tid] = incl - x;
      if (lane == 31) wsum[warp] = incl;
    }
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      const int n = n0 + k * 1024 + tid;
      const int at = done + all + scan[k * 32 + warp] + __popc(m[k] & ((1u << lane) - 1));
      if (label[k] >= 0 && w[k] != 0.0f) {
        rows[at] = n;
        lab[at] = label[k];
        wgt[at] = w[k];
      } else if (n < N) {
        rows[N - 1 - (n - at)] = n;   // n - at dropped rows come before this one
        loss[n] = 0.0f;
      }
      all += wsum[k];
    }
    done += all;
    __syncthreads();
  }
  if (tid == 0) {
    state->err = 0;
    state->n_live = done;
    state->retry = 0;
  }
}

// Row r of the compact H (bf16, or three planes of fp32), a CTA per row: the live rows, then zero
// rows up to a whole tile; nothing where the products can read H itself (`direct` and every row
// live).  Dropped rows of dH are zeroed.  ref (not null): the label's logit of each live row.
// With few rows (FEW: at most kFewRows) there is no launch of head_rows_kernel before: every CTA counts
// the live rows itself, and writes its own row's entry of what that kernel writes (512 x 256 x 1000: 35.8
// us, with the launch 37.5; the two meet at 1024 rows, 38.4 and 38.8).
constexpr int kFewRows = 1024, kFewPer = kFewRows / 128;
struct FewRows {
  const void* labels;
  int id_bytes, V;
  const float* weights;
  float* wgt;
  float* loss;
};
template <class T, int PLANES, bool FEW>
__global__ void __launch_bounds__(128) head_gather_kernel(const T* H, int d, int64_t N, HeadState* state, int* rows,
                                                          __nv_bfloat16* Hc, int plane, T* dH, int direct, const T* W,
                                                          int* labels, float* ref, const FewRows few) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  __shared__ float red[4];
  const int64_t r = blockIdx.x;
  int n_live, row = -1, label = 0;
  if (FEW) {
    __shared__ int count[4], found[2];
    const int tid = threadIdx.x, n0 = tid * kFewPer;   // a thread's rows are consecutive
    int lab[kFewPer];
    float w[kFewPer];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kFewPer; ++k) {
      lab[k] = n0 + k < N ? label_at(few.labels, few.id_bytes, n0 + k, few.V) : -1;
      w[k] = n0 + k < N && few.weights ? few.weights[n0 + k] : 1.0f;
    }
#pragma unroll
    for (int k = 0; k < kFewPer; ++k) {
      if (w[k] == 0.0f) lab[k] = -1;
      mine += lab[k] >= 0;
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if ((tid & 31) >= o) before += y;
    }
    if ((tid & 31) == 31) count[tid >> 5] = before;
    __syncthreads();
    before -= mine;
    for (int k = 0; k < tid >> 5; ++k) before += count[k];
    n_live = count[0] + count[1] + count[2] + count[3];
    // the r-th live row, or from the end backwards the dropped ones
#pragma unroll
    for (int k = 0; k < kFewPer; ++k) {
      const int n = n0 + k;
      const int at = lab[k] >= 0 ? before : static_cast<int>(N) - 1 - (n - before);
      if (n < N && at == r) {
        found[0] = n;
        found[1] = lab[k];
        rows[r] = n;
        if (lab[k] >= 0) {
          labels[r] = lab[k];
          few.wgt[r] = w[k];
        } else {
          few.loss[n] = 0.0f;
        }
      }
      before += lab[k] >= 0;
    }
    if (r == 0 && tid == 0) {
      state->err = 0;
      state->n_live = n_live;
      state->retry = 0;
    }
    __syncthreads();
    if (r < N) {
      row = found[0];
      label = found[1];
    }
  } else {
    n_live = __ldcg(&state->n_live);
    if (r < N) row = __ldcg(rows + r);
    if (ref && r < n_live) label = __ldcg(labels + r);
  }
  const int64_t fill = (static_cast<int64_t>(n_live) + kTile - 1) / kTile * kTile;
  const bool copy = !(direct && n_live == N);
  __nv_bfloat16* dst = Hc + r * plane * PLANES;
  if (r < n_live) {
    const T* src = H + static_cast<int64_t>(row) * d;
    const T* wl = ref ? W + static_cast<int64_t>(label) * d : nullptr;
    float dot = 0.0f;
    if (PLANES == 1 && d % 8 == 0) {
      for (int c = threadIdx.x; c < d / 8; c += 128) {
        const uint4 x = reinterpret_cast<const uint4*>(src)[c];
        if (copy) reinterpret_cast<uint4*>(dst)[c] = x;
        if (ref) {
          const uint4 y = reinterpret_cast<const uint4*>(wl)[c];
          const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            dot = fmaf(__uint_as_float(a[k] << 16), __uint_as_float(b[k] << 16), dot);
            dot = fmaf(__uint_as_float(a[k] & 0xffff0000u), __uint_as_float(b[k] & 0xffff0000u), dot);
          }
        }
      }
    } else {
      for (int c = threadIdx.x; c < plane; c += 128) {
        float x = c < d ? static_cast<float>(src[c]) : 0.0f;
        if (ref && c < d) dot = fmaf(x, static_cast<float>(wl[c]), dot);
#pragma unroll
        for (int k = 0; k < PLANES; ++k) {
          const __nv_bfloat16 b = __float2bfloat16_rn(x);
          dst[k * plane + c] = b;
          x -= __bfloat162float(b);
        }
      }
    }
    if (ref) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) ref[r] = (red[0] + red[1]) + (red[2] + red[3]);
    }
    return;
  }
  if (copy && r < fill)
    for (int c = threadIdx.x; c < plane * PLANES / 8; c += 128) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
  if (r < N && dH) {
    T* o = dH + static_cast<int64_t>(row) * d;
    for (int c = threadIdx.x; c < d; c += 128) o[c] = static_cast<T>(0.0f);
  }
}

// A copy of W that the tensor maps can address: rows padded to a multiple of eight, or three
// planes of an fp32 W.  Four columns a thread where W's rows allow it (10007 x 764 fp32: 13 us, 20 a column at a time).
template <class T, int PLANES>
__global__ void __launch_bounds__(128) head_weights_kernel(const T* W, int d, __nv_bfloat16* Wc, int plane) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t r = blockIdx.x;
  if (PLANES == 3 && d % 4 == 0) {
    for (int c = 4 * threadIdx.x; c < plane; c += 512) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (c < d) {
        const float4 y = *reinterpret_cast<const float4*>(W + r * d + c);
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
      }
#pragma unroll
      for (int k = 0; k < PLANES; ++k) {
        alignas(8) __nv_bfloat16 b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          b[e] = __float2bfloat16_rn(x[e]);
          x[e] -= __bfloat162float(b[e]);
        }
        *reinterpret_cast<uint2*>(Wc + (r * PLANES + k) * plane + c) = *reinterpret_cast<const uint2*>(b);
      }
    }
    return;
  }
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

// The losses, from the rows' partial sums, 32 rows per CTA: eight threads share a row's parts, eight
// loads of each in flight, joined in a fixed order.  After STATS (EXPS false): loss, the row's largest
// logit and the coefficients of g (w / s, w s' / s).  After EXP: loss, and the same coefficients of dH.
template <bool EXPS>
__global__ void __launch_bounds__(256) head_loss_kernel(const HeadState* state, int only_retry, const float2* parts,
                                                        int slots, int64_t n_pad, const float* target,
                                                        const float* weights, const int* rows, float* top,
                                                        float2* coef, float* loss) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (only_retry && __ldcg(&state->retry) == 0) return;
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
    for (int k0 = part; k0 < slots; k0 += 64) {
      float2 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        x[u] = k0 + 8 * u < slots ? __ldcg(parts + (k0 + 8 * u) * n_pad + row)
                                  : make_float2(EXPS ? 0.0f : -INFINITY, 0.0f);
      if (EXPS) {
#pragma unroll
        for (int u = 0; u < 8; ++u) s += x[u].x;
      } else {
        float mm = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) mm = fmaxf(mm, x[u].x);
        const float r = mm == -INFINITY ? 0.0f : mm;
        s *= ex2((m - r) * kLog2e);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += x[u].y * ex2((x[u].x - r) * kLog2e);
        m = mm;
      }
    }
  red[part][lane] = make_float2(m, s);
  __syncthreads();
  if (part == 0 && row < n_live) {
    const float w = __ldcg(weights + row), t = __ldcg(target + row);
    float x;
    if (EXPS) {
      s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += red[k][lane].y;
      const float el = ex2(t * kLog2e), inv = 1.0f / (s + el);
      coef[row] = make_float2(w * inv, w * (s * inv));
      x = w * log1pf(s / el);
    } else {
      m = -INFINITY;
      s = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) join(red[k][lane].x, red[k][lane].y);
      // the label's term joins the others', each relative to the largest logit
      const float mm = fmaxf(m, t), el = ex2((t - mm) * kLog2e);
      s *= ex2((m - mm) * kLog2e);
      const float inv = 1.0f / (s + el);
      top[row] = mm;
      coef[row] = make_float2(w * inv, w * (s * inv));
      x = w * (t >= m ? log1pf(s) : logf(s + el) - (t - mm));   // (t >= m: el = 1)
    }
    if (__ldcg(&state->err)) x = __int_as_float(0x7fc00000);
    loss[__ldcg(rows + row)] = x;
  }
}

// dH from the splits of the vocabulary, added in order (and, after EXP, the coefficients applied).  A
// thread takes four columns, eight splits' values in flight; at most kJoinBlocks CTAs, four an SM, so
// that a launch that leaves at once costs little (512 x 1024 x 32000 with 148 / 592 / 2368: 106 / 88 / 85
// us, 64 x 256 x 1000 33.6 / 33.2 / 33.2).
constexpr int kJoinThreads = 128, kJoinBlocks = 592;
template <class T>
__global__ void __launch_bounds__(kJoinThreads) head_join_kernel(const HeadState* state, int only_retry,
                                                                 const float* acc, int splits, int64_t n_pad,
                                                                 int64_t ldacc, int d, const int* rows,
                                                                 const float2* coef, const int* labels, const T* W,
                                                                 T* dH) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (only_retry && __ldcg(&state->retry) == 0) return;
  const int n_live = __ldcg(&state->n_live);
  const int c = 4 * (blockIdx.x * kJoinThreads + threadIdx.x);
  if (c >= d) return;
  for (int64_t r = blockIdx.y; r < n_live; r += gridDim.y) {
    const int64_t row = __ldcg(rows + r);
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < splits; s0 += 8) {
      float4 y[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        y[u] = s0 + u < splits ? __ldcg(reinterpret_cast<const float4*>(acc + ((s0 + u) * n_pad + r) * ldacc + c))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) x[0] += y[u].x, x[1] += y[u].y, x[2] += y[u].z, x[3] += y[u].w;
    }
    if (coef) {
      const float2 co = __ldcg(coef + r);
      const T* wl = W + static_cast<int64_t>(__ldcg(labels + r)) * d + c;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k < d) x[k] = co.x * x[k] - co.y * static_cast<float>(wl[k]);
    }
    store4(dH + row * d + c, x, c, d);
  }
}

// ---- host ---------------------------------------------------------------------------------------

// From this many multiplications (rows in whole tiles) x d x V on, dH alone takes one pass: the product
// it saves is worth more than the launches behind it that leave at once, 2 us each (one pass against
// two, us: 256 x 256 x 30000, 2.0e9, 52 / 53; 512 x 512 x 16000, 4.2e9, 51 / 53; 512 x 512 x 32000 70 / 75;
// 64 x 1024 x 128000, 3.4e10 in whole tiles, 153 / 191).
constexpr double kOnePassWork = 4.0e9;
constexpr int kPlanPairs = 74;         // pairs of SMs of a B200 (a plan is made without asking a device)

struct HeadPlan {
  int planes, plane;       // bf16 planes of an operand; elements of a plane's row
  bool copy_W;
  int64_t n_pad;
  int slots;               // tiles of the vocabulary: one partial sum per row each
  int piece, pieces;       // columns of a piece (a multiple of 256), pieces
  int splits;              // of DH
  bool acc;                // DH goes through fp32 memory
  int64_t ldacc;
  bool one_pass;           // EXP
  size_t o_rows, o_labels, o_weights, o_ref, o_coef, o_target, o_parts, o_H, o_W, o_g, o_acc, bytes;

  explicit HeadPlan(const HeadShape& s) {
    planes = s.dtype == GRAPE_F32 ? 3 : 1;
    // three planes lie side by side, and a block of 64 must not reach into the next one
    plane = planes == 3 ? (s.d + 63) / 64 * 64 : (s.d + 7) / 8 * 8;
    copy_W = planes == 3 || plane != s.d;
    n_pad = (s.N + kTile - 1) / kTile * kTile;
    slots = (s.V + kTile - 1) / kTile;
    one_pass = s.dH && !s.dW && static_cast<double>(n_pad) * s.d * s.V >= kOnePassWork;
    const int64_t vmax = (static_cast<int64_t>(s.V) + kTile - 1) / kTile * kTile;
    int64_t cols = static_cast<int64_t>(kPieceBytes / (std::max<int64_t>(n_pad, 1) * 2 * planes)) / kTile * kTile;
    cols = std::min(std::max<int64_t>(cols, 4096), vmax);
    pieces = static_cast<int>((vmax + cols - 1) / cols);
    piece = static_cast<int>(((vmax + pieces - 1) / pieces + kTile - 1) / kTile * kTile);
    pieces = static_cast<int>((vmax + piece - 1) / piece);
    // few tiles of dH: its long sum over the vocabulary is split over the CTA pairs, at least
    // kSplitBlocks blocks of 64 (of every kept product) each
    const int64_t out_tiles = n_pad / kTile * ((s.d + kTile - 1) / kTile);
    splits = 1;
    if (s.dH && out_tiles > 0 && out_tiles < kPlanPairs)
      splits = static_cast<int>(std::max<int64_t>(
          1, std::min<int64_t>(kPlanPairs / out_tiles, piece / kBK * (planes == 3 ? 6 : 1) / kSplitBlocks)));
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
    o_ref = take(np * 4);
    o_target = take(np * 4);
    o_coef = take(np * 8);
    o_parts = take(np * slots * 8);
    o_H = take(np * plane * planes * 2);
    o_W = take(copy_W ? static_cast<size_t>(s.V) * plane * planes * 2 : 0);
    o_g = take(grads ? np * piece * planes * 2 : 0);
    o_acc = take(acc ? np * ldacc * splits * 4 : 0);
    bytes = o;
  }
};

template <int EPI, int PLANES>
cudaError_t run_gemm(const HeadGemm& p, int64_t max_tiles, cudaStream_t st) {
  const void* k = reinterpret_cast<const void*>(head_gemm_kernel<EPI, PLANES>);
  cudaError_t e = lm_configure_kernel(k, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(lm_sm_count() / 2, max_tiles));
  return lm_launch(true, head_gemm_kernel<EPI, PLANES>, dim3(static_cast<unsigned>(2 * pairs)), kThreads, kSmem, st, p);
}

template <class T, int PLANES>
cudaError_t run_head(const HeadShape& s, const T* H, const T* W, const void* labels, int id_bytes,
                     const float* weights, char* ws, float* loss, T* dH, T* dW, cudaStream_t st) {
  const HeadPlan pl(s);
  HeadState* state = reinterpret_cast<HeadState*>(ws);
  int* rows = reinterpret_cast<int*>(ws + pl.o_rows);
  int* lab = reinterpret_cast<int*>(ws + pl.o_labels);
  float* wgt = reinterpret_cast<float*>(ws + pl.o_weights);
  float* ref = reinterpret_cast<float*>(ws + pl.o_ref);
  float* target = reinterpret_cast<float*>(ws + pl.o_target);
  float2* parts = reinterpret_cast<float2*>(ws + pl.o_parts);
  __nv_bfloat16* Hc = reinterpret_cast<__nv_bfloat16*>(ws + pl.o_H);
  __nv_bfloat16* Wc = pl.copy_W ? reinterpret_cast<__nv_bfloat16*>(ws + pl.o_W)
                                : const_cast<__nv_bfloat16*>(reinterpret_cast<const __nv_bfloat16*>(W));
  __nv_bfloat16* g = reinterpret_cast<__nv_bfloat16*>(ws + pl.o_g);
  const int wide = pl.plane * PLANES;
  const int64_t gw = static_cast<int64_t>(pl.piece) * PLANES;

  float2* coef = reinterpret_cast<float2*>(ws + pl.o_coef);
  const int direct = PLANES == 1 && !pl.copy_W;   // H itself can be an operand when every row is live

  if (s.N == 0) return dW ? cudaMemsetAsync(dW, 0, static_cast<size_t>(s.V) * s.d * sizeof(T), st) : cudaSuccess;
  cudaError_t e = cudaSuccess;
  const bool few = s.N <= kFewRows;
  if (!few)
    e = lm_launch(false, head_rows_kernel, dim3(1), 1024, 0, st, labels, id_bytes, weights, static_cast<int>(s.N), s.V,
                  state, rows, lab, wgt, loss);
  if (e == cudaSuccess) {
    auto gather = [&](auto kernel) {
      return lm_launch(!few, kernel, dim3(static_cast<unsigned>(pl.n_pad)), 128, 0, st, H, s.d, s.N, state, rows, Hc,
                       pl.plane, dH, direct, W, lab, pl.one_pass ? ref : nullptr,
                       FewRows{labels, id_bytes, s.V, weights, wgt, loss});
    };
    e = few ? gather(head_gather_kernel<T, PLANES, true>) : gather(head_gather_kernel<T, PLANES, false>);
  }
  if (e == cudaSuccess && pl.copy_W)
    e = lm_launch(true, head_weights_kernel<T, PLANES>, dim3(s.V), 128, 0, st, W, s.d, Wc, pl.plane);
  if (e != cudaSuccess) return e;

  // operand views: K-major boxes of 64 x 128 rows, M/N-major boxes of 64 x 64
  const bool grads = s.dH || s.dW;
  CUtensorMap H_k, H_mn, W_k, W_mn, g_k, g_mn, X_k, X_mn;
  std::memset(&X_k, 0, sizeof(X_k));
  std::memset(&X_mn, 0, sizeof(X_mn));
  bool ok = lm_map_2d(&H_k, Hc, pl.n_pad, wide, wide, kBK, kHalf) && lm_map_2d(&W_k, Wc, s.V, wide, wide, kBK, kHalf);
  if (ok && direct) ok = lm_map_2d(&X_k, H, s.N, wide, wide, kBK, kHalf) && lm_map_2d(&X_mn, H, s.N, wide, wide, 64, kBK);
  if (ok && grads)
    ok = lm_map_2d(&H_mn, Hc, pl.n_pad, wide, wide, 64, kBK) && lm_map_2d(&W_mn, Wc, s.V, wide, wide, 64, kBK) &&
         lm_map_2d(&g_k, g, pl.n_pad, gw, gw, kBK, kHalf) && lm_map_2d(&g_mn, g, pl.n_pad, gw, gw, 64, kBK);
  if (!ok) return cudaErrorInvalidValue;

  HeadGemm base;
  std::memset(&base, 0, sizeof(base));
  base.state = state;
  base.V = s.V;
  base.d = s.d;
  base.n_pad = pl.n_pad;
  base.labels = lab;
  base.ref = ref;
  base.scale = coef;
  base.parts = parts;
  base.target = target;
  base.g = g;
  base.ldg = gw;
  base.planeG = pl.piece;
  base.rows = rows;
  base.poison = loss;
  base.n_rows = s.N;
  base.splits = 1;
  const int64_t mt = pl.n_pad / kTile;
  const int dt = (s.d + kTile - 1) / kTile;

  // z of the vocabulary rows from v0 on (`cols` of them)
  auto logits = [&](int v0, int cols) {
    HeadGemm p = base;
    p.mapA = H_k;
    p.mapB = W_k;
    p.mapH = X_k;
    p.direct = direct;
    p.planeA = p.planeB = pl.plane;
    p.kblocks = (pl.plane + kBK - 1) / kBK;
    p.v0 = v0;
    p.n_tiles = (cols + kTile - 1) / kTile;
    return p;
  };
  auto losses = [&](bool exps, int only_retry) {
    const dim3 grid(static_cast<unsigned>((s.N + 31) / 32));
    auto go = [&](auto kernel) {
      return lm_launch(true, kernel, grid, 256, 0, st, static_cast<const HeadState*>(state), only_retry,
                    static_cast<const float2*>(parts), pl.slots, pl.n_pad, static_cast<const float*>(target),
                    static_cast<const float*>(wgt), static_cast<const int*>(rows), ref, coef, loss);
    };
    return exps ? go(head_loss_kernel<true>) : go(head_loss_kernel<false>);
  };
  auto input_grad = [&](int i, int v0, int cols, bool exps, int only_retry) {
    HeadGemm p = base;
    p.only_retry = only_retry;
    p.mapA = g_k;
    p.mapB = W_mn;
    p.planeA = pl.piece;
    p.planeB = pl.plane;
    p.kblocks = (cols + kBK - 1) / kBK;
    p.v0 = v0;
    p.n_tiles = dt;
    p.splits = pl.splits;
    p.acc = pl.acc ? reinterpret_cast<float*>(ws + pl.o_acc) : nullptr;
    p.ldacc = pl.ldacc;
    p.add = i > 0;
    p.last = i + 1 == pl.pieces && pl.splits == 1;
    p.coef = exps ? coef : nullptr;
    p.W = W;
    p.out = dH;
    cudaError_t e2 = run_gemm<DH, PLANES>(p, mt * dt * pl.splits, st);
    if (e2 == cudaSuccess && i + 1 == pl.pieces && pl.splits > 1) {
      const unsigned gx = static_cast<unsigned>((s.d + 4 * kJoinThreads - 1) / (4 * kJoinThreads));
      const unsigned gy = static_cast<unsigned>(std::min<int64_t>(s.N, std::max<int64_t>(1, kJoinBlocks / gx)));
      e2 = lm_launch(true, head_join_kernel<T>, dim3(gx, gy), kJoinThreads, 0, st, static_cast<const HeadState*>(state),
                     only_retry, reinterpret_cast<const float*>(ws + pl.o_acc), pl.splits, pl.n_pad, pl.ldacc, s.d,
                     static_cast<const int*>(rows), p.coef, static_cast<const int*>(lab), W, dH);
    }
    return e2;
  };

  if (pl.one_pass) {
    for (int i = 0; i < pl.pieces; ++i) {
      const int v0 = i * pl.piece, cols = std::min(pl.piece, s.V - v0);
      HeadGemm p = logits(v0, cols);
      e = run_gemm<EXP, PLANES>(p, mt * p.n_tiles, st);
      if (e == cudaSuccess && i + 1 == pl.pieces) e = losses(true, 0);
      if (e == cudaSuccess) e = input_grad(i, v0, cols, true, 0);
      if (e != cudaSuccess) return e;
    }
  }
  // two passes; after EXP they leave at once unless it asked for them
  const int retry = pl.one_pass ? 1 : 0;
  HeadGemm p = logits(0, s.V);
  p.only_retry = retry;
  e = run_gemm<STATS, PLANES>(p, mt * p.n_tiles, st);
  if (e == cudaSuccess) e = losses(false, retry);
  for (int i = 0; grads && e == cudaSuccess && i < pl.pieces; ++i) {
    const int v0 = i * pl.piece, cols = std::min(pl.piece, s.V - v0);
    p = logits(v0, cols);
    p.only_retry = retry;
    e = run_gemm<GRAD, PLANES>(p, mt * p.n_tiles, st);
    if (e == cudaSuccess && s.dH) e = input_grad(i, v0, cols, false, retry);
    if (e == cudaSuccess && s.dW) {
      HeadGemm x = base;
      x.mapA = g_mn;
      x.mapB = H_mn;
      x.mapH = X_mn;
      x.direct = direct ? 2 : 0;
      x.planeA = pl.piece;
      x.planeB = pl.plane;
      x.v0 = v0;
      x.m_tiles = p.n_tiles;
      x.n_tiles = dt;
      x.out = dW;
      e = run_gemm<DW, PLANES>(x, static_cast<int64_t>(x.m_tiles) * dt, st);
    }
  }
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
