// Internal launchers of libhata's kernels (host side).  Arguments are already
// validated by hata_api.cu; every launcher returns cudaGetLastError().
#pragma once

#include "hata_common.cuh"

namespace hata {

// status: the caller's device status word (a bounded wait that runs out is recorded there)
cudaError_t launch_encode(const hata_dims_t& d, const void* x, int x_heads, int x_len, int n_tok,
                          const int32_t* seq_end, const float* W, uint32_t* codes, int codes_len, uint32_t* status,
                          cudaStream_t stream);

size_t prefill_ws_bytes(const hata_dims_t& d);
cudaError_t launch_prefill(const hata_dims_t& d, const void* q, const void* K, const void* V, const float* W,
                           void* codes, const int32_t* seq_lens, float scale, void* out, char* ws,
                           cudaStream_t stream);
cudaError_t launch_hamming(const hata_dims_t& d, const uint32_t* qcode, const uint32_t* codes,
                           const int32_t* seq_lens, int32_t* scores, cudaStream_t stream);

cudaError_t launch_topk(const hata_dims_t& d, const WsLayout& L, const int32_t* scores, const int32_t* seq_lens,
                        int k, int32_t* idx, int32_t* n_sel, char* ws, cudaStream_t stream);

cudaError_t launch_sparse_decode(const hata_dims_t& d, const WsLayout& L, const void* q, const void* K,
                                 const void* V, const int32_t* idx, int k, float scale, void* out, char* ws,
                                 cudaStream_t stream);

// Whether the fused decode-step kernel covers these dims and budget.
bool fused_step_applies(const hata_dims_t& d, int k);
// Fused decode step: bytes of workspace its plan needs (0 if it does not apply)
size_t fused_step_ws_bytes(const hata_dims_t& d, int k);
cudaError_t launch_encode_mma(const hata_dims_t& d, const void* x, int x_heads, int x_len, int n_tok,
                              const int32_t* seq_end, const float* W, uint32_t* codes, int codes_len,
                              cudaStream_t stream);
// Prefill encode on tcgen05 tensor cores (bf16 keys, r <= 128; else cudaErrorNotSupported).
cudaError_t launch_encode_tc(const hata_dims_t& d, const void* x, int x_heads, int x_len, int n_tok,
                             const int32_t* seq_end, const float* W, uint32_t* codes, int codes_len,
                             uint32_t* status, cudaStream_t stream);
size_t dense_ws_bytes(const hata_dims_t& d);
cudaError_t launch_dense_decode(const hata_dims_t& d, const void* q, const void* K, const void* V,
                                const int32_t* seq_lens, float scale, void* out, char* ws, cudaStream_t stream);
// Returns cudaErrorNotSupported when the fused kernel does not apply to these dims.
// Paged cache: K, V and codes are pools [n_blocks][Hkv][1 << block_shift][...] and
// block_table [B][max_blocks] maps each sequence's logical blocks to pool blocks.
struct PagedCache {
  const int32_t* block_table;
  int block_shift, n_blocks, max_blocks;
};

// pg: paged pools (the layout of the paged step), or null for [B][Hkv][max_seq][d] caches
cudaError_t launch_append_kv(const hata_dims_t& d, const void* new_k, const void* new_v, void* K, void* V,
                             const int32_t* seq_lens, const PagedCache* pg, cudaStream_t stream);

// Launches a kernel that may be set up while the one before it on the stream still runs: the kernel waits for that
// one to end (griddepcontrol.wait) before it reads what that one may have written, and before it writes anything.
// A kernel that comes next waits for this grid alone, so this grid must not end before the ones ahead of it have: at
// least one CTA waits whatever the inputs are, and a thread that returns without waiting has touched nothing that those
// kernels touch but their common inputs.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*k)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                         const Args&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, Params(args)...);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// Norms, position rotation and cache append (hata_rope.cu).
struct RopeArgs {
  const void *q_in, *k_in, *v_in;
  long long q_stride, k_stride, v_stride;
  const float *q_weight, *k_weight, *table;
  const int32_t *n_new, *positions, *seq_lens;
  void *q_out, *K, *V;
  float eps;
  int n_tok, n_pos, rot, interleaved;
};
cudaError_t launch_norm_rope(const hata_dims_t& d, const RopeArgs& a, const PagedCache* pg, uint32_t* status,
                             cudaStream_t stream);
cudaError_t launch_rope_table(float* table, int n_pos, int rot, double theta, cudaStream_t stream);

// Window decode (window > 0, n_tok = 1) and tree attention (window = 0) (hata_span.cu).
struct SpanArgs {
  const void *q, *K, *V;
  const int32_t *seq_lens, *n_new;
  const uint32_t* mask;
  void* out;
  float scale;
  int n_tok, window, sink;
};
constexpr int kMaxTreeTokens = 128;  // new tokens per sequence of one call
size_t span_ws_bytes(const hata_dims_t& d, int n_tok);
cudaError_t launch_span(const hata_dims_t& d, const SpanArgs& a, const PagedCache* pg, char* ws, cudaStream_t stream);
int span_sms();  // SMs of the current device, found once per device
// Prefill with a sliding window and sinks (hata_span_tc.cu).
cudaError_t launch_window_prefill(const hata_dims_t& d, const void* q, const void* K, const void* V,
                                  const int32_t* seq_lens, int window, int sink, float scale, void* out,
                                  uint32_t* status, cudaStream_t stream);

// Page bookkeeping and row compaction (hata_pages.cu).
constexpr int kMaxPageRows = 1024;  // sequences of one call
size_t pages_ws_bytes(int batch);
cudaError_t launch_pages_fork(const hata_dims_t& d, const int32_t* parent, int32_t* table, int max_blocks,
                              int n_blocks, int32_t* seq_lens, int32_t* ref, uint32_t* status, cudaStream_t stream);
cudaError_t launch_pages_resize(const hata_dims_t& d, const int32_t* new_lens, void* K, void* V, void* codes,
                                const PagedCache& pg, int32_t* table, int32_t* seq_lens, int32_t* ref, char* ws,
                                cudaStream_t stream);
cudaError_t launch_compact(const hata_dims_t& d, int n_tok, const int32_t* keep, const int32_t* n_keep,
                           const int32_t* n_new, const int32_t* seq_lens, void* K, void* V, void* codes,
                           const PagedCache* pg, int32_t* new_lens, uint32_t* status, cudaStream_t stream);

// Wk: separate key encoder, or equal to W (one encoder for queries and keys).
// pg: paged cache, or null for [B][Hkv][max_seq][...] slabs.
cudaError_t launch_fused_step(const hata_dims_t& d, const WsLayout& L, const void* q, const void* K,
                              const void* V, const float* W, const float* Wk, uint32_t* codes,
                              const int32_t* seq_lens, int k, float scale, void* out, uint32_t* qcode_out,
                              int32_t* idx_out, const PagedCache* pg, char* ws, cudaStream_t stream);

// Decode step as a scan kernel over all SMs plus a per-unit tail kernel (hata_fused.cu).
bool split_step_applies(const hata_dims_t& d, int k);
size_t split_step_ws_bytes(const hata_dims_t& d, int k);
cudaError_t launch_split_step(const hata_dims_t& d, const WsLayout& L, const void* q, const void* K,
                              const void* V, const float* W, const float* Wk, uint32_t* codes,
                              const int32_t* seq_lens, int k, float scale, void* out, uint32_t* qcode_out,
                              int32_t* idx_out, const PagedCache* pg, char* ws, cudaStream_t stream);

}  // namespace hata
