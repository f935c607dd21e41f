// C ABI entry points of the page planner and of the rotary positions.
#include <cuda_runtime.h>

#include <cstdint>
#include <new>
#include <string>

#include "kernels.h"
#include "spectra_internal.h"

using namespace spectra;

struct spectra_planner {
  int page_tokens = 0;
  int device = 0;
  int32_t* err = nullptr;  // device error word
};

namespace {

#define CUDA_TRY(expr)                                                                        \
  do {                                                                                        \
    cudaError_t e_ = (expr);                                                                  \
    if (e_ != cudaSuccess)                                                                    \
      return fail(SPECTRA_ERR_CUDA, std::string(#expr) + ": " + cudaGetErrorString(e_));     \
  } while (0)

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

spectra_status check_device(const spectra_planner* p) {
  int dev = -1;
  CUDA_TRY(cudaGetDevice(&dev));
  if (dev != p->device) return fail(SPECTRA_ERR_INVALID, "planner belongs to another CUDA device");
  return SPECTRA_OK;
}

spectra_status check_batch(const spectra_planner* p, int32_t batch, int32_t n_prefix, int32_t max_pages) {
  if (batch <= 0) return fail(SPECTRA_ERR_INVALID, "batch must be positive");
  if (batch > kPlanMaxBatch) return fail(SPECTRA_ERR_UNSUPPORTED, "at most 16384 sequences");
  if (max_pages <= 0) return fail(SPECTRA_ERR_INVALID, "max_pages_per_seq must be positive");
  if (n_prefix < 0 || n_prefix > max_pages)
    return fail(SPECTRA_ERR_INVALID, "n_prefix must be in [0, max_pages_per_seq]");
  return check_device(p);
}

// Tensors of one call: the same heads; in place, or elsewhere; output rows apart.
spectra_status check_heads(const spectra_heads* in, const spectra_heads* out, int32_t d_head, int64_t T, int esz) {
  if (!out) return fail(SPECTRA_ERR_INVALID, "an input without its output");
  if (in->n_heads < 0 || in->n_heads > 65536 || in->n_heads != out->n_heads)
    return fail(SPECTRA_ERR_INVALID, "input and output need the same head count, at most 65536");
  if (in->n_heads == 0 || T == 0) return SPECTRA_OK;
  if (!in->data || !out->data) return fail(SPECTRA_ERR_INVALID, "null pointer");
  if (!aligned(in->data, esz) || !aligned(out->data, esz)) return fail(SPECTRA_ERR_INVALID, "misaligned tensor");
  if (in->token_stride < 0 || in->head_stride < 0 || out->token_stride < 0 || out->head_stride < 0)
    return fail(SPECTRA_ERR_INVALID, "negative stride");
  const int64_t big = (int64_t)1 << 40;  // keeps every product below within 63 bits
  if (in->token_stride > big || in->head_stride > big || out->token_stride > big || out->head_stride > big)
    return fail(SPECTRA_ERR_INVALID, "stride too large");
  // output rows must not overlap: tokens apart with heads inside, or the reverse
  // (a single token or head leaves its own stride open)
  const int64_t H = out->n_heads, ts = out->token_stride, hs = out->head_stride, d = d_head;
  const bool heads_inside = (H == 1 || hs >= d) && (T == 1 || ts >= (H > 1 ? (H - 1) * hs : 0) + d);
  const bool tokens_inside = (T == 1 || ts >= d) && (H == 1 || hs / d >= 1) &&
                             (H == 1 || T == 1 || (ts <= (hs - d) / (T - 1)));
  if (!heads_inside && !tokens_inside) return fail(SPECTRA_ERR_INVALID, "output rows overlap");
  if (in->data == out->data && ((T > 1 && in->token_stride != ts) || (H > 1 && in->head_stride != hs)))
    return fail(SPECTRA_ERR_INVALID, "an output in its input's place needs the same strides");
  return SPECTRA_OK;
}

}  // namespace

extern "C" {

spectra_status spectra_planner_create(int32_t page_tokens, spectra_planner** out) {
  return guarded([&]() -> spectra_status {
    if (!out) return fail(SPECTRA_ERR_INVALID, "null pointer");
    *out = nullptr;
    if (page_tokens < 32 || page_tokens > 1024 || page_tokens % 32 != 0)
      return fail(SPECTRA_ERR_INVALID, "page_tokens must be a multiple of 32 in 32..1024");
    spectra_planner* p = new (std::nothrow) spectra_planner();
    if (!p) return fail(SPECTRA_ERR_INVALID, "out of host memory");
    p->page_tokens = page_tokens;
    cudaError_t e = cudaGetDevice(&p->device);
    if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&p->err), 256);
    if (e == cudaSuccess) e = cudaMemset(p->err, 0, 256);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);  // (the planner's streams may not wait for it)
    if (e != cudaSuccess) {
      spectra_planner_destroy(p);
      return fail(SPECTRA_ERR_CUDA, std::string("planner: ") + cudaGetErrorString(e));
    }
    *out = p;
    return SPECTRA_OK;
  });
}

void spectra_planner_destroy(spectra_planner* p) {
  if (!p) return;
  if (p->err) cudaFree(p->err);
  delete p;
}

spectra_status spectra_plan_append(const spectra_planner* p, int32_t batch, const int32_t* lengths,
                                   const int32_t* new_tokens, const int32_t* prefix_pages, int32_t n_prefix,
                                   const int32_t* free_pages, const int32_t* n_free, int32_t* n_free_out,
                                   int32_t* page_table, int32_t max_pages_per_seq, int64_t max_tokens,
                                   int32_t* seq_ids, int32_t* positions, int64_t* slots, int32_t* offsets,
                                   void* stream) {
  return spectra_plan_append_ex(p, batch, lengths, new_tokens, prefix_pages, n_prefix, free_pages, INT32_MAX, n_free,
                                n_free_out, page_table, max_pages_per_seq, max_tokens, seq_ids, positions, slots,
                                offsets, stream);
}

spectra_status spectra_plan_append_ex(const spectra_planner* p, int32_t batch, const int32_t* lengths,
                                      const int32_t* new_tokens, const int32_t* prefix_pages, int32_t n_prefix,
                                      const int32_t* free_pages, int64_t free_capacity, const int32_t* n_free,
                                      int32_t* n_free_out, int32_t* page_table, int32_t max_pages_per_seq,
                                      int64_t max_tokens, int32_t* seq_ids, int32_t* positions, int64_t* slots,
                                      int32_t* offsets, void* stream) {
  return guarded([&]() -> spectra_status {
    if (!p || !lengths || !new_tokens || !free_pages || !n_free || !n_free_out || !page_table || !offsets)
      return fail(SPECTRA_ERR_INVALID, "null pointer");
    if (free_capacity < 0 || free_capacity > INT32_MAX) return fail(SPECTRA_ERR_INVALID, "free_capacity out of range");
    if (max_tokens < 0 || max_tokens > (1 << 24)) return fail(SPECTRA_ERR_INVALID, "max_tokens out of range");
    if (max_tokens > 0 && !seq_ids) return fail(SPECTRA_ERR_INVALID, "null pointer");
    if (n_prefix > 0 && !prefix_pages) return fail(SPECTRA_ERR_INVALID, "null pointer");
    if (!aligned(lengths, 4) || !aligned(new_tokens, 4) || !aligned(prefix_pages, 4) || !aligned(free_pages, 4) ||
        !aligned(n_free, 4) || !aligned(n_free_out, 4) || !aligned(page_table, 4) || !aligned(seq_ids, 4) ||
        !aligned(positions, 4) || !aligned(slots, 8) || !aligned(offsets, 4))
      return fail(SPECTRA_ERR_INVALID, "misaligned buffer");
    const spectra_status s = check_batch(p, batch, n_prefix, max_pages_per_seq);
    if (s != SPECTRA_OK) return s;
    CUDA_TRY(launch_plan_append(p->page_tokens, p->err, batch, lengths, new_tokens, prefix_pages, n_prefix, free_pages,
                                free_capacity, n_free, n_free_out, page_table, max_pages_per_seq, max_tokens, seq_ids, positions,
                                slots, offsets, static_cast<cudaStream_t>(stream)));
    return SPECTRA_OK;
  });
}

spectra_status spectra_release_pages(const spectra_planner* p, int32_t batch, const int32_t* finished,
                                     int32_t* lengths, int32_t n_prefix, const int32_t* page_table,
                                     int32_t max_pages_per_seq, int32_t* free_pages, int64_t free_capacity,
                                     int32_t* n_free, void* stream) {
  return guarded([&]() -> spectra_status {
    if (!p || !finished || !lengths || !page_table || !free_pages || !n_free)
      return fail(SPECTRA_ERR_INVALID, "null pointer");
    if (free_capacity < 0 || free_capacity > INT32_MAX) return fail(SPECTRA_ERR_INVALID, "free_capacity out of range");
    if (!aligned(finished, 4) || !aligned(lengths, 4) || !aligned(page_table, 4) || !aligned(free_pages, 4) ||
        !aligned(n_free, 4))
      return fail(SPECTRA_ERR_INVALID, "misaligned buffer");
    const spectra_status s = check_batch(p, batch, n_prefix, max_pages_per_seq);
    if (s != SPECTRA_OK) return s;
    CUDA_TRY(launch_release_pages(p->page_tokens, p->err, batch, finished, lengths, n_prefix, page_table,
                                  max_pages_per_seq, free_pages, free_capacity, n_free,
                                  static_cast<cudaStream_t>(stream)));
    return SPECTRA_OK;
  });
}

spectra_status spectra_planner_status(const spectra_planner* p, void* stream) {
  return guarded([&]() -> spectra_status {
    if (!p) return fail(SPECTRA_ERR_INVALID, "null planner");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // in `stream` alone, and cleared before the return: a later call's error in another stream stays
    int32_t v = 0;
    CUDA_TRY(cudaMemcpyAsync(&v, p->err, 4, cudaMemcpyDeviceToHost, st));
    CUDA_TRY(cudaMemsetAsync(p->err, 0, 4, st));
    CUDA_TRY(cudaStreamSynchronize(st));
    if (v == 0) return SPECTRA_OK;
    return fail(static_cast<spectra_status>(v), v == SPECTRA_ERR_CAPACITY
                                                    ? "too few free pages, table entries or token slots"
                                                    : "a sequence's length or token count is not valid");
  });
}

spectra_status spectra_rope_frequencies(const spectra_rope* rope, int32_t d_head, double* freq, double* magnitude) {
  return guarded([&]() -> spectra_status {
    if (!rope) return fail(SPECTRA_ERR_INVALID, "null pointer");
    RopeFreq f;
    std::string why;
    if (!rope_frequencies(*rope, d_head, &f, &why)) return fail(SPECTRA_ERR_INVALID, why);
    if (freq)
      for (int i = 0; i < f.rot / 2; ++i) freq[i] = f.freq[i];
    if (magnitude) *magnitude = f.magnitude;
    return SPECTRA_OK;
  });
}

spectra_status spectra_rope_apply(const spectra_rope* rope, int32_t dtype, int32_t d_head, const int32_t* positions,
                                  int64_t n_tokens, const spectra_heads* q, const spectra_heads* q_out,
                                  const spectra_heads* k, const spectra_heads* k_out, int32_t inverse,
                                  void* stream) {
  return guarded([&]() -> spectra_status {
    if (!rope || !q) return fail(SPECTRA_ERR_INVALID, "null pointer");
    if (dtype != SPECTRA_F32 && dtype != SPECTRA_BF16) return fail(SPECTRA_ERR_INVALID, "dtype must be F32 or BF16");
    if (n_tokens < 0 || n_tokens > INT32_MAX) return fail(SPECTRA_ERR_INVALID, "n_tokens out of range");
    if (n_tokens > 0 && !positions) return fail(SPECTRA_ERR_INVALID, "null pointer");
    if (!aligned(positions, 4)) return fail(SPECTRA_ERR_INVALID, "misaligned positions");
    RopeFreq f;
    std::string why;
    if (!rope_frequencies(*rope, d_head, &f, &why)) return fail(SPECTRA_ERR_INVALID, why);
    if (k_out && !k) return fail(SPECTRA_ERR_INVALID, "an output without its input");
    const int esz = dtype == SPECTRA_BF16 ? 2 : 4;
    spectra_status s = check_heads(q, q_out, d_head, n_tokens, esz);
    if (s == SPECTRA_OK && k) s = check_heads(k, k_out, d_head, n_tokens, esz);
    if (s != SPECTRA_OK) return s;
    const spectra_heads* const in[2] = {q, k};
    const spectra_heads* const out[2] = {q_out, k_out};
    CUDA_TRY(launch_rope(f, dtype == SPECTRA_BF16, d_head, positions, n_tokens, in, out, inverse != 0,
                         static_cast<cudaStream_t>(stream)));
    return SPECTRA_OK;
  });
}

}  // extern "C"
