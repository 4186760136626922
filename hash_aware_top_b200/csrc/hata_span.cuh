// Attention of a few query rows over a span of a cache, split over all SMs: what the kernels for
// window decode and tree attention share (arguments, the split of the work).
//
// A unit is (sequence b, KV head g, tile of query rows).  The rows of a unit are the G * T (query
// head of the group, new token) pairs, which lie next to each other in q and out.  Its keys are a
// list of tiles of kSpanTile cache slots: all of [0, L) for a tree; the tiles that hold sinks, then
// those that hold the window, for a window.  The tiles of all units, in the order (b, row tile, g, tile), are
// cut into equal runs, one per CTA, so ragged lengths keep every SM busy to the end; a CTA's run may
// end one unit and begin the next.  A unit that one CTA covers is written at once.  Otherwise each of
// its CTAs leaves a partial (row maximum, row sum, weighted values; fp32) in the workspace, and a second kernel,
// launched early (programmatic dependent launch), joins them in the order of the split.  Joining them in
// the last CTA to arrive was slower: one SM then reads all partials of a unit (15 us for 32 rows and 19 runs).
#pragma once

#include "hata_kernels.cuh"

namespace hata {
namespace span {

constexpr int kSpanTile = 128;  // cache slots of a tile

struct Params {
  const void *q, *K, *V;
  void* out;
  float* part;  // partials
  uint32_t* status;
  const int32_t *seq_lens, *n_new;
  const uint32_t* mask;  // [B][T][ceil(T / 32)], or null: token i sees tokens j <= i
  const int32_t* block_table;
  int block_shift, n_blocks, max_blocks;
  int B, Hq, Hkv, G, T, R, max_seq, mask_words;  // R = G * T
  int row_tiles;                                 // tiles of query rows per (b, g)
  int window, sink;                              // window > 0: window decode (T = 1)
  float scale_log2;
};

// One sequence's share of the work.
struct Seq {
  int L;      // visible slots end here
  int ctx;    // tree: slots before the new tokens
  int n_b;    // new tokens
  int sink_tiles, win_tile;  // window: list index j < sink_tiles is tile j, else tile win_tile + j - sink_tiles
  int tiles;  // tiles of each unit of this sequence; 0: nothing to do or write
  bool bad;   // lengths out of range: flagged, rows left as they were (tree) or clamped (window)
};

__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
  Seq s;
  int L = p.seq_lens[b];
  s.bad = false;
  if (p.window > 0) {
    if (L > p.max_seq) {
      s.bad = true;
      L = p.max_seq;
    }
    L = max(L, 0);
    s.n_b = 1;
    s.ctx = L;
    const int all = (L + kSpanTile - 1) / kSpanTile;
    const int w0 = max(0, L - min(p.window, L));
    s.win_tile = w0 / kSpanTile;
    s.sink_tiles = (min(p.sink, L) + kSpanTile - 1) / kSpanTile;
    if (s.sink_tiles >= s.win_tile) s.sink_tiles = s.win_tile;  // the two runs meet: tiles 0 .. all - 1
    s.tiles = max(1, s.sink_tiles + all - s.win_tile);          // at least one, so an empty row is written as zeros
  } else {
    const int n = p.n_new ? p.n_new[b] : p.T;
    s.bad = n < 0 || n > p.T || L < n || L > p.max_seq;
    s.n_b = s.bad ? 0 : n;
    s.ctx = L - s.n_b;
    s.sink_tiles = s.win_tile = 0;
    s.tiles = s.n_b > 0 ? (L + kSpanTile - 1) / kSpanTile : 0;
  }
  s.L = L;
  return s;
}

// Where a CTA stands in the list of tiles (the same in every thread of a warp).
struct Cursor {
  int b;                // sequence
  Seq seq;
  long long seq_start;  // first tile of the sequence in the list of all tiles
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Tiles of all units, and of the units of sequences before b.  All lanes of a warp; every warp that needs them
// computes them, 32 sequences at a time, so no barrier is needed.
__device__ __forceinline__ void count_tiles(const Params& p, int lane, int b, bool flag, long long* total,
                                            long long* before) {
  const long long per_tile = (long long)p.Hkv * p.row_tiles;
  *total = *before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    long long n = 0;
    if (b0 + lane < p.B) {
      const Seq s = seq_of(p, b0 + lane);
      n = s.tiles * per_tile;
      if (s.bad && flag) set_status(p.status, HATA_ERR_INVALID_ARG);
    }
    if (b0 < b) *before += warp_sum(b0 + lane < b ? n : 0);
    *total += warp_sum(n);
  }
}

// This CTA's run [*at, *end) of the list of all tiles, each CTA's length *per, and the sequence it begins in.
// False: the CTA has none.
__device__ __forceinline__ bool my_run(const Params& p, int lane, bool flag, long long* at, long long* end,
                                       long long* per, Cursor* c) {
  long long total, before;
  count_tiles(p, lane, 0, flag, &total, &before);
  *per = max(1LL, (total + gridDim.x - 1) / gridDim.x);
  *at = (long long)blockIdx.x * *per;
  *end = min(total, *at + *per);
  if (*at >= *end) return false;
  c->b = 0;
  c->seq_start = 0;
  const long long per_tile = (long long)p.Hkv * p.row_tiles;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    long long n = 0;
    if (b0 + lane < p.B) n = seq_of(p, b0 + lane).tiles * per_tile;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, c->seq_start + incl > *at);
    if (past) {
      const int l = __ffs(past) - 1;
      c->b = b0 + l;
      c->seq_start += __shfl_sync(0xffffffffu, incl - n, l);
      break;
    }
    c->seq_start += __shfl_sync(0xffffffffu, incl, 31);
  }
  c->seq = seq_of(p, c->b);
  return true;
}

// Whether new token i sees slot s, a slot that some token may see.
__device__ __forceinline__ bool sees(const Params& p, const Seq& q, int b, int i, int s) {
  const int j = s - q.ctx;
  if (j < 0) return true;
  if (!p.mask) return j <= i;
  return (p.mask[((size_t)b * p.T + i) * p.mask_words + (j >> 5)] >> (j & 31)) & 1u;
}

// The n lowest bits (none below 1, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// A slot that no token sees may hold anything (a value row that is not finite would turn 0 * V into NaN), so
// it is read as zeros.  Bit k of the answer: some token sees slot s0 + k (k < 16).  All lanes of a warp.
__device__ __forceinline__ unsigned seen_by_any16(const Params& p, const Seq& q, int b, int s0, int lane) {
  if (p.window <= 0 && s0 + 16 <= q.ctx) return 0xffffu;
  unsigned in = low_bits(min(16, q.L - s0));
  if (p.window > 0) in &= low_bits(p.sink - s0) | ~low_bits(q.L - min(p.window, q.L) - s0);
  if (s0 + 16 <= q.ctx || !p.mask || !in) return in;
  unsigned any = 0;
  for (int i = lane; i < q.n_b; i += 32)
    for (int k = max(0, q.ctx - s0); k < 16; ++k)
      if ((in >> k) & 1u) any |= sees(p, q, b, i, s0 + k) ? 1u << k : 0u;
  any = __reduce_or_sync(0xffffffffu, any);
  return in & (any | low_bits(q.ctx - s0));  // slots before the new tokens are seen by all
}

}  // namespace span

// Launches a kernel that may be set up while the one before it on the stream runs (and waits for it with
// griddepcontrol.wait before it reads anything).
template <typename... Args>
cudaError_t launch_early(void (*k)(Args...), dim3 grid, unsigned threads, cudaStream_t st, Args... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// Tensor-core form of tree attention (hata_span_tc.cu): bf16, any number of rows.
size_t span_tc_part_bytes(const hata_dims_t& d, int n_tok);
cudaError_t launch_span_tc(const hata_dims_t& d, const span::Params& s, const PagedCache* pg, cudaStream_t stream);

}  // namespace hata
