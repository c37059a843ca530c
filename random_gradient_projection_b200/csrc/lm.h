// Internal interface of the operators at the two ends of a language model's stack of
// linear layers: token embedding, vocabulary head with its loss, distillation.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "../../include/grape.h"

namespace grape {

// Records `msg` for grape_global_error and returns `code` (api.cu).
int fail_global(int code, const std::string& msg);

inline size_t lm_round256(size_t b) { return (b + 255) & ~size_t(255); }

// ---- embedding: lm_embed.cu ------------------------------------------------------------
cudaError_t embed_forward(const void* table, int table_dtype, const void* ids, int id_bytes, int64_t n, int vocab,
                          int d, float scale, int out_dtype, void* out, cudaStream_t st);

// The caller-owned buffer of grape_embed_order: byte offsets of its parts.
struct EmbedOrderLayout {
  size_t positions = 0, tokens, tmp_positions, tmp_tokens, present, bytes;
  EmbedOrderLayout(int64_t n, int vocab) {
    const size_t list = lm_round256(static_cast<size_t>(n) * 4);
    tokens = list;
    tmp_positions = 2 * list;
    tmp_tokens = 3 * list;
    present = 4 * list;
    bytes = present + lm_round256((static_cast<size_t>(vocab) + 31) / 32 * 4);
  }
};
cudaError_t embed_order(const void* ids, int id_bytes, int64_t n, int vocab, void* order, cudaStream_t st);

size_t embed_workspace_bytes(int64_t n, int d);
cudaError_t embed_sqnorms(const void* order, int B, int T, int vocab, int d, const void* G, int dtype, float scale,
                          void* ws, float* sqnorms, cudaStream_t st);
cudaError_t embed_grad(const void* order, int B, int T, int vocab, int d, const void* G, int dtype, float scale,
                       const float* weights, void* ws, float* grad, cudaStream_t st);

// ---- distillation: lm_distill.cu ----------------------------------------------------------
constexpr int kMaxTeacher = 1024;
cudaError_t distill_loss(const void* logits, int dtype, int64_t N, int V, const void* idx, int id_bytes,
                         const void* val, int val_dtype, int K, const float* weights, float tau, float* loss,
                         void* Gout, cudaStream_t st);

// ---- vocabulary head: lm_head.cu -----------------------------------------------------------
struct HeadShape {
  int64_t N;
  int d, V, dtype;
  bool dH, dW;
};
size_t head_workspace_bytes(const HeadShape& s);
cudaError_t head_loss(const HeadShape& s, const void* H, const void* W, const void* labels, int id_bytes,
                      const float* weights, void* ws, float* loss, void* dH, void* dW, cudaStream_t st);

}  // namespace grape
