// extern "C" entry points of the serving operators beside the decode step: norms with rotation and
// append, window and tree attention, page bookkeeping, row compaction.  Argument validation
// and launches, as in hata_api.cu.
#include <algorithm>
#include <cmath>

#include "hata_kernels.cuh"

using namespace hata;

namespace {

bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool null_or4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether two int32 arrays share memory (a null array: no).
bool overlap(const int32_t* a, size_t n_a, const int32_t* b, size_t n_b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && a0 < b0 + 4 * n_b && b0 < a0 + 4 * n_a;
}

hata_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return HATA_OK;
  return e == cudaErrorNotSupported ? HATA_ERR_UNSUPPORTED : HATA_ERR_CUDA;
}

bool make_paged(const hata_dims_t& d, const int32_t* table, int block_size, int n_blocks, PagedCache* pg) {
  if (!ok4(table) || block_size < 16 || block_size > 65536 || (block_size & (block_size - 1)) || n_blocks < 1)
    return false;
  if ((long long)n_blocks * d.n_kv_heads * block_size > 0x7fffffffLL) return false;
  pg->block_table = table;
  pg->block_shift = 0;
  while ((1 << pg->block_shift) < block_size) ++pg->block_shift;
  pg->n_blocks = n_blocks;
  pg->max_blocks = (int)(((long long)d.max_seq + block_size - 1) / block_size);
  return true;
}

hata_status_t norm_rope(const hata_dims_t* dims, const RopeArgs& a, const PagedCache* pg, void* ws, size_t ws_bytes,
                        void* stream) {
  const hata_dims_t& d = *dims;
  const long long unit = d.dtype == HATA_BF16 ? 8 : 4;  // elements of 16 bytes
  if (!ok16(a.q_in) || !ok16(a.k_in) || !ok16(a.v_in) || !ok16(a.q_out) || !ok16(a.K) || !ok16(a.V))
    return HATA_ERR_INVALID_ARG;
  if (!ok4(a.seq_lens) || !null_or4(a.n_new) || !null_or4(a.positions) || !null_or4(a.q_weight) ||
      !null_or4(a.k_weight))
    return HATA_ERR_INVALID_ARG;
  if (a.n_tok < 1) return HATA_ERR_INVALID_ARG;
  const long long q_row = (long long)d.n_q_heads * d.head_dim, kv_row = (long long)d.n_kv_heads * d.head_dim;
  if (a.q_stride < q_row || a.k_stride < kv_row || a.v_stride < kv_row || a.q_stride % unit || a.k_stride % unit ||
      a.v_stride % unit)
    return HATA_ERR_INVALID_ARG;
  if (!(a.eps > 0.f) || !std::isfinite(a.eps)) return HATA_ERR_INVALID_ARG;
  if (a.rot < 0 || a.rot > d.head_dim || a.rot % 2) return HATA_ERR_INVALID_ARG;
  if (a.rot % 16) return HATA_ERR_UNSUPPORTED;
  if (a.rot > 0 && (!ok16(a.table) || a.n_pos < 1)) return HATA_ERR_INVALID_ARG;
  if (!ok16(ws) || ws_bytes < kStatusBytes) return HATA_ERR_WORKSPACE;
  return status_of(launch_norm_rope(d, a, pg, static_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

hata_status_t span_call(const hata_dims_t* dims, SpanArgs a, const PagedCache* pg, void* ws, size_t ws_bytes,
                        void* stream) {
  const hata_dims_t& d = *dims;
  if (!ok16(a.q) || !ok16(a.K) || !ok16(a.V) || !ok16(a.out) || !ok4(a.seq_lens) || !null_or4(a.n_new) ||
      !null_or4(a.mask))
    return HATA_ERR_INVALID_ARG;
  if (!std::isfinite(a.scale)) return HATA_ERR_INVALID_ARG;
  if (!ok16(ws) || ws_bytes < span_ws_bytes(d, a.n_tok)) return HATA_ERR_WORKSPACE;
  if (a.scale <= 0.f) a.scale = 1.0f / std::sqrt((float)d.head_dim);
  return status_of(launch_span(d, a, pg, static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

hata_status_t hata_rope_table(float* table, int n_pos, int rot_dim, double theta, void* stream) {
  if (!ok16(table) || n_pos < 1 || rot_dim < 2 || rot_dim > kHeadDim || rot_dim % 2 || !(theta > 0.0) ||
      !std::isfinite(theta))
    return HATA_ERR_INVALID_ARG;
  if (rot_dim % 16) return HATA_ERR_UNSUPPORTED;
  return status_of(launch_rope_table(table, n_pos, rot_dim, theta, static_cast<cudaStream_t>(stream)));
}

hata_status_t hata_norm_rope(const hata_dims_t* dims, int n_tok, const void* q_in, long long q_stride,
                             const void* k_in, long long k_stride, const void* v_in, long long v_stride,
                             const float* q_weight, const float* k_weight, float eps, const float* table, int n_pos,
                             int rot_dim, int interleaved, const int32_t* n_new, const int32_t* positions,
                             const int32_t* seq_lens, void* q_out, void* K, void* V, void* workspace,
                             size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  const RopeArgs a{q_in,     k_in,  v_in,      q_stride, k_stride, v_stride, q_weight, k_weight, table, n_new,
                   positions, seq_lens, q_out, K,        V,        eps,      n_tok,    n_pos,    rot_dim, interleaved};
  return norm_rope(dims, a, nullptr, workspace, workspace_bytes, stream);
}

hata_status_t hata_norm_rope_paged(const hata_dims_t* dims, int n_tok, const void* q_in, long long q_stride,
                                   const void* k_in, long long k_stride, const void* v_in, long long v_stride,
                                   const float* q_weight, const float* k_weight, float eps, const float* table,
                                   int n_pos, int rot_dim, int interleaved, const int32_t* n_new,
                                   const int32_t* positions, const int32_t* seq_lens, void* q_out, void* K_pool,
                                   void* V_pool, const int32_t* block_table, int block_size, int n_blocks,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  PagedCache pg;
  if (!make_paged(*dims, block_table, block_size, n_blocks, &pg)) return HATA_ERR_INVALID_ARG;
  const RopeArgs a{q_in,     k_in,  v_in,      q_stride, k_stride, v_stride, q_weight, k_weight, table, n_new,
                   positions, seq_lens, q_out, K_pool,   V_pool,   eps,      n_tok,    n_pos,    rot_dim, interleaved};
  return norm_rope(dims, a, &pg, workspace, workspace_bytes, stream);
}

hata_status_t hata_span_workspace_size(const hata_dims_t* dims, int n_tok, size_t* bytes) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  if (!bytes || n_tok < 1) return HATA_ERR_INVALID_ARG;
  if (n_tok > kMaxTreeTokens) return HATA_ERR_UNSUPPORTED;
  *bytes = span_ws_bytes(*dims, n_tok);
  return HATA_OK;
}

hata_status_t hata_window_decode(const hata_dims_t* dims, const void* q, const void* K, const void* V,
                                 const int32_t* seq_lens, int window, int n_sink, float scale, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  if (window < 1 || n_sink < 0) return HATA_ERR_INVALID_ARG;
  const SpanArgs a{q, K, V, seq_lens, nullptr, nullptr, out, scale, 1, window, n_sink};
  return span_call(dims, a, nullptr, workspace, workspace_bytes, stream);
}

hata_status_t hata_window_decode_paged(const hata_dims_t* dims, const void* q, const void* K_pool, const void* V_pool,
                                       const int32_t* block_table, int block_size, int n_blocks,
                                       const int32_t* seq_lens, int window, int n_sink, float scale, void* out,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  PagedCache pg;
  if (window < 1 || n_sink < 0 || !make_paged(*dims, block_table, block_size, n_blocks, &pg))
    return HATA_ERR_INVALID_ARG;
  const SpanArgs a{q, K_pool, V_pool, seq_lens, nullptr, nullptr, out, scale, 1, window, n_sink};
  return span_call(dims, a, &pg, workspace, workspace_bytes, stream);
}

hata_status_t hata_window_prefill(const hata_dims_t* dims, const void* q, const void* K, const void* V,
                                  const int32_t* seq_lens, int window, int n_sink, float scale, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  if (dims->dtype != HATA_BF16) return HATA_ERR_UNSUPPORTED;
  if (!ok16(q) || !ok16(K) || !ok16(V) || !ok16(out) || !ok4(seq_lens)) return HATA_ERR_INVALID_ARG;
  if (window < 1 || n_sink < 0 || !std::isfinite(scale)) return HATA_ERR_INVALID_ARG;
  if (!ok16(workspace) || workspace_bytes < kStatusBytes) return HATA_ERR_WORKSPACE;
  if (scale <= 0.f) scale = 1.0f / std::sqrt((float)dims->head_dim);
  return status_of(launch_window_prefill(*dims, q, K, V, seq_lens, window, n_sink, scale, out,
                                         static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

hata_status_t hata_tree_attention(const hata_dims_t* dims, int n_tok, const void* q, const void* K, const void* V,
                                  const int32_t* seq_lens, const int32_t* n_new, const uint32_t* mask, float scale,
                                  void* out, void* workspace, size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  if (n_tok < 1) return HATA_ERR_INVALID_ARG;
  if (n_tok > kMaxTreeTokens) return HATA_ERR_UNSUPPORTED;
  const SpanArgs a{q, K, V, seq_lens, n_new, mask, out, scale, n_tok, 0, 0};
  return span_call(dims, a, nullptr, workspace, workspace_bytes, stream);
}

hata_status_t hata_tree_attention_paged(const hata_dims_t* dims, int n_tok, const void* q, const void* K_pool,
                                        const void* V_pool, const int32_t* block_table, int block_size, int n_blocks,
                                        const int32_t* seq_lens, const int32_t* n_new, const uint32_t* mask,
                                        float scale, void* out, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  PagedCache pg;
  if (n_tok < 1 || !make_paged(*dims, block_table, block_size, n_blocks, &pg)) return HATA_ERR_INVALID_ARG;
  if (n_tok > kMaxTreeTokens) return HATA_ERR_UNSUPPORTED;
  const SpanArgs a{q, K_pool, V_pool, seq_lens, n_new, mask, out, scale, n_tok, 0, 0};
  return span_call(dims, a, &pg, workspace, workspace_bytes, stream);
}

hata_status_t hata_pages_workspace_size(const hata_dims_t* dims, size_t* bytes) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  if (!bytes) return HATA_ERR_INVALID_ARG;
  if (dims->batch > kMaxPageRows) return HATA_ERR_UNSUPPORTED;
  *bytes = pages_ws_bytes(dims->batch);
  return HATA_OK;
}

hata_status_t hata_pages_fork(const hata_dims_t* dims, const int32_t* parent, int32_t* block_table, int block_size,
                              int n_blocks, int32_t* seq_lens, int32_t* ref_count, void* workspace,
                              size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  PagedCache pg;
  if (!ok4(parent) || !ok4(seq_lens) || !ok4(ref_count) || !make_paged(*dims, block_table, block_size, n_blocks, &pg))
    return HATA_ERR_INVALID_ARG;
  if (dims->batch > kMaxPageRows) return HATA_ERR_UNSUPPORTED;
  if (!ok16(workspace) || workspace_bytes < pages_ws_bytes(dims->batch)) return HATA_ERR_WORKSPACE;
  return status_of(launch_pages_fork(*dims, parent, block_table, pg.max_blocks, n_blocks, seq_lens, ref_count,
                                     static_cast<uint32_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

hata_status_t hata_pages_resize(const hata_dims_t* dims, const int32_t* new_lens, void* K_pool, void* V_pool,
                                void* codes_pool, int32_t* block_table, int block_size, int n_blocks,
                                int32_t* seq_lens, int32_t* ref_count, void* workspace, size_t workspace_bytes,
                                void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  PagedCache pg;
  if (!ok4(new_lens) || !ok4(seq_lens) || !ok4(ref_count) || !ok16(K_pool) || !ok16(V_pool) ||
      (codes_pool && !ok16(codes_pool)) || !make_paged(*dims, block_table, block_size, n_blocks, &pg))
    return HATA_ERR_INVALID_ARG;
  if (dims->batch > kMaxPageRows) return HATA_ERR_UNSUPPORTED;
  if (!ok16(workspace) || workspace_bytes < pages_ws_bytes(dims->batch)) return HATA_ERR_WORKSPACE;
  return status_of(launch_pages_resize(*dims, new_lens, K_pool, V_pool, codes_pool, pg, block_table, seq_lens,
                                       ref_count, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)));
}

static hata_status_t compact(const hata_dims_t* dims, int n_tok, const int32_t* keep, const int32_t* n_keep,
                             const int32_t* n_new, const int32_t* seq_lens, void* K, void* V, void* codes,
                             const PagedCache* pg, int32_t* new_lens, void* ws, size_t ws_bytes, void* stream) {
  if (!ok4(keep) || !ok4(n_keep) || !null_or4(n_new) || !ok4(seq_lens) || !ok16(K) || !ok16(V) ||
      (codes && !ok16(codes)) || !null_or4(new_lens) || new_lens == seq_lens)
    return HATA_ERR_INVALID_ARG;
  if (n_tok < 1 || n_tok > dims->max_seq) return HATA_ERR_INVALID_ARG;
  if (!ok16(ws) || ws_bytes < kStatusBytes) return HATA_ERR_WORKSPACE;
  // new_lens is written while other CTAs of the sequence may still read the call's int32 inputs
  const size_t B = (size_t)dims->batch;
  if (overlap(new_lens, B, keep, B * (size_t)n_tok) || overlap(new_lens, B, n_keep, B) || overlap(new_lens, B, n_new, B) ||
      overlap(new_lens, B, seq_lens, B) || (pg && overlap(new_lens, B, pg->block_table, B * (size_t)pg->max_blocks)))
    return HATA_ERR_INVALID_ARG;
  return status_of(launch_compact(*dims, n_tok, keep, n_keep, n_new, seq_lens, K, V, codes, pg, new_lens,
                                  static_cast<uint32_t*>(ws), static_cast<cudaStream_t>(stream)));
}

hata_status_t hata_compact_kv(const hata_dims_t* dims, int n_tok, const int32_t* keep, const int32_t* n_keep,
                              const int32_t* n_new, const int32_t* seq_lens, void* K, void* V, void* codes,
                              int32_t* new_lens, void* workspace, size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  return compact(dims, n_tok, keep, n_keep, n_new, seq_lens, K, V, codes, nullptr, new_lens, workspace,
                 workspace_bytes, stream);
}

hata_status_t hata_compact_kv_paged(const hata_dims_t* dims, int n_tok, const int32_t* keep, const int32_t* n_keep,
                                    const int32_t* n_new, const int32_t* seq_lens, void* K_pool, void* V_pool,
                                    void* codes_pool, const int32_t* block_table, int block_size, int n_blocks,
                                    int32_t* new_lens, void* workspace, size_t workspace_bytes, void* stream) {
  hata_status_t s = check_dims(dims);
  if (s != HATA_OK) return s;
  PagedCache pg;
  if (!make_paged(*dims, block_table, block_size, n_blocks, &pg)) return HATA_ERR_INVALID_ARG;
  return compact(dims, n_tok, keep, n_keep, n_new, seq_lens, K_pool, V_pool, codes_pool, &pg, new_lens, workspace,
                 workspace_bytes, stream);
}

}  // extern "C"
