// C entry points of the language-model operators (see include/grape.h): argument checks, all
// made before anything is launched, and the calls into the kernel files.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <new>
#include <string>

#include "lm.h"
#include "tc.h"

namespace {

using grape::fail_global;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
bool dtype_ok(int32_t t) { return t == GRAPE_F32 || t == GRAPE_BF16; }
int einval(const char* msg) { return fail_global(GRAPE_EINVAL, msg); }

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// The kernels are built for sm_100a only.  A device's answer is kept: it cannot change.
int check_device(bool tensor_maps) {
  constexpr int kDevices = 64;
  static std::atomic<int> fits[kDevices];   // 0: not asked yet, 1: yes, 2: no
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  int known = e == cudaSuccess && dev < kDevices ? fits[dev].load(std::memory_order_relaxed) : 0;
  if (e == cudaSuccess && known == 0) {
    int major = 0, minor = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    known = major == 10 && minor == 0 ? 1 : 2;
    if (e == cudaSuccess && dev < kDevices) fits[dev].store(known, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail_global(GRAPE_ECUDA, std::string("device query: ") + cudaGetErrorString(e));
  }
  if (known != 1) return fail_global(GRAPE_EUNSUPPORTED, "needs an sm_100a device (B200)");
  if (tensor_maps && !grape::tc_tensor_maps_available())
    return fail_global(GRAPE_EUNSUPPORTED, "cuTensorMapEncodeTiled is not available from the driver");
  return GRAPE_OK;
}

int done(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return GRAPE_OK;
  cudaGetLastError();
  return fail_global(GRAPE_ECUDA, std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
}

// Runs `f`; a C caller sees no exception.
template <class F>
int guarded(const char* name, F&& f) {
  try {
    NvtxRange r(name);
    return f();
  } catch (const std::bad_alloc&) {
    return GRAPE_ENOMEM;
  } catch (...) {
    return GRAPE_ECUDA;
  }
}

constexpr int64_t kMaxIds = int64_t(1) << 30;
constexpr int32_t kMaxVocab = 1 << 30, kMaxWidth = 1 << 20;
const char* const kVocabRange = "vocab must lie in [1, 2^30]";
const char* const kWidthRange = "d must lie in [1, 2^20]";

const char* ids_problem(const void* ids, int32_t id_bytes, int64_t n, int32_t vocab) {
  if (id_bytes != 4 && id_bytes != 8) return "id_bytes must be 4 or 8";
  if (n < 0 || n > kMaxIds) return "the number of ids must lie in [0, 2^30]";
  if (vocab < 1 || vocab > kMaxVocab) return kVocabRange;
  if (n > 0 && !ids) return "ids must not be null";
  if (!aligned(ids, static_cast<size_t>(id_bytes))) return "ids must be aligned to their element size";
  return nullptr;
}

const char* batch_problem(int32_t B, int32_t T, int32_t vocab, int32_t d) {
  if (B < 0 || T < 0 || static_cast<int64_t>(B) * T > kMaxIds) return "need B, T >= 0 and B*T <= 2^30";
  if (vocab < 1 || vocab > kMaxVocab) return kVocabRange;
  if (d < 1 || d > kMaxWidth) return kWidthRange;
  return nullptr;
}

const char* head_problem(int64_t N, int32_t d, int32_t vocab, int32_t dtype) {
  if (N < 0 || N > kMaxIds) return "N must lie in [0, 2^30]";
  if (vocab < 1 || vocab > kMaxVocab) return kVocabRange;
  if (d < 1 || d > kMaxWidth) return kWidthRange;
  if (!dtype_ok(dtype)) return "dtype must be GRAPE_F32 or GRAPE_BF16";
  if ((N / 256 + 1) * (static_cast<int64_t>(vocab) / 256 + 1) > 0x7fffffff ||
      (N / 256 + 1) * (static_cast<int64_t>(d) / 256 + 1) > 0x7fffffff)
    return "N * vocab too large";
  return nullptr;
}

}  // namespace

extern "C" {

int grape_embed(const void* table, int32_t table_dtype, const void* ids, int32_t id_bytes, int64_t n_ids,
                int32_t vocab, int32_t d, double scale, int32_t out_dtype, void* out, void* stream) {
  return guarded("grape_embed", [&]() -> int {
    if (const char* m = ids_problem(ids, id_bytes, n_ids, vocab)) return einval(m);
    if (d < 1 || d > kMaxWidth) return einval(kWidthRange);
    if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype)) return einval("dtypes must be GRAPE_F32 or GRAPE_BF16");
    if (!std::isfinite(static_cast<float>(scale))) return einval("scale must be finite in fp32");
    if (n_ids == 0) return GRAPE_OK;
    if (!table || !out) return einval("table and out must not be null");
    if (!aligned16(table) || !aligned16(out)) return einval("table and out must be 16-byte aligned");
    if (int rc = check_device(false)) return rc;
    return done(grape::embed_forward(table, table_dtype, ids, id_bytes, n_ids, vocab, d, static_cast<float>(scale),
                                     out_dtype, out, static_cast<cudaStream_t>(stream)),
                "embed");
  });
}

int grape_embed_order_bytes(int64_t n_ids, int32_t vocab, uint64_t* bytes) {
  if (!bytes) return einval("bytes must not be null");
  if (const char* m = ids_problem(bytes, 8, n_ids, vocab)) return einval(m);
  *bytes = grape::EmbedOrderLayout(n_ids, vocab).bytes;
  return GRAPE_OK;
}

int grape_embed_order(const void* ids, int32_t id_bytes, int64_t n_ids, int32_t vocab, void* order, void* stream) {
  return guarded("grape_embed_order", [&]() -> int {
    if (const char* m = ids_problem(ids, id_bytes, n_ids, vocab)) return einval(m);
    if (!order || !aligned16(order)) return einval("order must be a 16-byte aligned device buffer");
    if (int rc = check_device(false)) return rc;
    return done(grape::embed_order(ids, id_bytes, n_ids, vocab, order, static_cast<cudaStream_t>(stream)),
                "embed order");
  });
}

int grape_embed_workspace_bytes(int32_t B, int32_t T, int32_t vocab, int32_t d, uint64_t* bytes) {
  if (!bytes) return einval("bytes must not be null");
  if (const char* m = batch_problem(B, T, vocab, d)) return einval(m);
  *bytes = grape::embed_workspace_bytes(static_cast<int64_t>(B) * T, d);
  return GRAPE_OK;
}

int grape_embed_sqnorms(const void* order, int32_t B, int32_t T, int32_t vocab, int32_t d, const void* Gout,
                        int32_t dtype, double scale, void* workspace, float* sqnorms, void* stream) {
  return guarded("grape_embed_sqnorms", [&]() -> int {
    if (const char* m = batch_problem(B, T, vocab, d)) return einval(m);
    if (!dtype_ok(dtype)) return einval("dtype must be GRAPE_F32 or GRAPE_BF16");
    if (!std::isfinite(static_cast<float>(scale))) return einval("scale must be finite in fp32");
    if (!order || !aligned16(order) || !workspace || !aligned16(workspace))
      return einval("order and workspace must be 16-byte aligned device buffers");
    if (B > 0 && (!sqnorms || !aligned(sqnorms, 4))) return einval("sqnorms must not be null");
    if (static_cast<int64_t>(B) * T > 0 && (!Gout || !aligned16(Gout)))
      return einval("Gout must not be null and must be 16-byte aligned");
    if (int rc = check_device(false)) return rc;
    return done(grape::embed_sqnorms(order, B, T, vocab, d, Gout, dtype, static_cast<float>(scale), workspace, sqnorms,
                                     static_cast<cudaStream_t>(stream)),
                "embed sqnorms");
  });
}

int grape_embed_grad(const void* order, int32_t B, int32_t T, int32_t vocab, int32_t d, const void* Gout,
                     int32_t dtype, double scale, const float* weights, void* workspace, float* grad, void* stream) {
  return guarded("grape_embed_grad", [&]() -> int {
    if (const char* m = batch_problem(B, T, vocab, d)) return einval(m);
    if (!dtype_ok(dtype)) return einval("dtype must be GRAPE_F32 or GRAPE_BF16");
    if (!std::isfinite(static_cast<float>(scale))) return einval("scale must be finite in fp32");
    if (!order || !aligned16(order) || !workspace || !aligned16(workspace))
      return einval("order and workspace must be 16-byte aligned device buffers");
    if (!grad || !aligned16(grad)) return einval("grad must not be null and must be 16-byte aligned");
    if (!aligned(weights, 4)) return einval("weights must be aligned to their element size");
    if (static_cast<int64_t>(B) * T > 0 && (!Gout || !aligned16(Gout)))
      return einval("Gout must not be null and must be 16-byte aligned");
    if (int rc = check_device(false)) return rc;
    return done(grape::embed_grad(order, B, T, vocab, d, Gout, dtype, static_cast<float>(scale), weights, workspace,
                                  grad, static_cast<cudaStream_t>(stream)),
                "embed grad");
  });
}

int grape_head_loss_bytes(int64_t N, int32_t d, int32_t vocab, int32_t dtype, int32_t want_dH, int32_t want_dW,
                          uint64_t* bytes) {
  if (!bytes) return einval("bytes must not be null");
  if (const char* m = head_problem(N, d, vocab, dtype)) return einval(m);
  *bytes = grape::head_workspace_bytes(grape::HeadShape{N, d, vocab, dtype, want_dH != 0, want_dW != 0});
  return GRAPE_OK;
}

int grape_head_loss(const void* H, const void* W, const void* labels, int32_t id_bytes, const float* weights,
                    int64_t N, int32_t d, int32_t vocab, int32_t dtype, void* workspace, float* loss, void* dH,
                    void* dW, void* stream) {
  return guarded("grape_head_loss", [&]() -> int {
    if (const char* m = head_problem(N, d, vocab, dtype)) return einval(m);
    if (const char* m = ids_problem(labels, id_bytes, N, vocab)) return einval(m);
    if (!W || !aligned16(W)) return einval("W must not be null and must be 16-byte aligned");
    if (N > 0 && (!H || !loss)) return einval("H and loss must not be null");
    if (!aligned16(H) || !aligned16(dH) || !aligned16(dW)) return einval("H, dH and dW must be 16-byte aligned");
    if (!aligned(loss, 4) || !aligned(weights, 4)) return einval("loss and weights must be aligned to their element size");
    if (!workspace || !aligned16(workspace)) return einval("workspace must be a 16-byte aligned device buffer");
    if (int rc = check_device(true)) return rc;
    return done(grape::head_loss(grape::HeadShape{N, d, vocab, dtype, dH != nullptr, dW != nullptr}, H, W, labels,
                                 id_bytes, weights, workspace, loss, dH, dW, static_cast<cudaStream_t>(stream)),
                "head loss");
  });
}

int grape_distill_loss(const void* logits, int32_t dtype, int64_t N, int32_t vocab, const void* indices,
                       int32_t id_bytes, const void* values, int32_t value_dtype, int32_t K, const float* weights,
                       double temperature, float* loss, void* Gout, void* stream) {
  return guarded("grape_distill_loss", [&]() -> int {
    if (!dtype_ok(dtype) || !dtype_ok(value_dtype)) return einval("dtypes must be GRAPE_F32 or GRAPE_BF16");
    if (id_bytes != 4 && id_bytes != 8) return einval("id_bytes must be 4 or 8");
    if (N < 0 || N > 0x7fffffff) return einval("N must lie in [0, 2^31 - 1]");
    if (vocab < 1 || vocab > kMaxVocab) return einval(kVocabRange);
    if (K < 1 || K > grape::kMaxTeacher) return einval("K must lie in [1, 1024]");
    // (so that log2(e) / temperature and temperature^2 are finite and normal in fp32)
    if (!(temperature >= 0x1p-60 && temperature <= 0x1p60)) return einval("temperature must lie in [2^-60, 2^60]");
    if (N == 0) return GRAPE_OK;
    if (!logits || !indices || !values || !loss || !Gout)
      return einval("logits, indices, values, loss and Gout must not be null");
    if (!aligned16(logits) || !aligned16(Gout)) return einval("logits and Gout must be 16-byte aligned");
    if (!aligned(indices, static_cast<size_t>(id_bytes)) || !aligned(values, value_dtype == GRAPE_F32 ? 4 : 2) ||
        !aligned(loss, 4) || !aligned(weights, 4))
      return einval("indices, values, loss and weights must be aligned to their element size");
    if (int rc = check_device(false)) return rc;
    return done(grape::distill_loss(logits, dtype, N, vocab, indices, id_bytes, values, value_dtype, K, weights,
                                    static_cast<float>(temperature), loss, Gout, static_cast<cudaStream_t>(stream)),
                "distill loss");
  });
}

}  // extern "C"
