// Attention of a few query rows over a span of a cache, split over all SMs: what the kernels for
// window decode and tree attention share (arguments, the split of the work).
//
// A unit is (sequence b, KV head g, tile of query rows).  The rows of a unit are the G * T (query
// head of the group, new token) pairs, which lie next to each other in q and out.  Its keys are a
// list of tiles of kSpanTile cache slots: all of [0, L) for a tree; the tiles that hold sinks, then
// those that hold the window, for a window.  The tiles of all units, in the order (b, row tile, g, tile), are
// shared out over the CTAs (Split below), so ragged lengths keep every SM busy to the end.  A unit that one CTA
// covers is written at once.  Otherwise each of
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

// How the tiles are shared out.  Two ways, and every warp that needs to know works out the same one:
//   flat     CTA c takes tiles c * per .. of the list of all tiles; a run may end one unit and begin another, which
//            costs about kSwitchTiles tiles of time (the pipeline drains, rows are written, queries are loaded)
//   aligned  each unit of sequence b gets k_b CTAs of its own, in proportion to its tiles (1 + its share of
//            the CTAs that are more than units), so no run changes its unit, but some CTAs are idle
// Aligned is taken when its longest run is no longer than a flat one and a change of unit: 8 units of 256 tiles
// on 148 SMs take 14.2 tiles each, 8 x 18 runs of 14.2 against 148 runs of 13.8 tiles, most with a change.
constexpr int kSwitchTiles = 3;

struct Split {
  int total;     // tiles of all units
  int per;       // flat: tiles of a run
  int units;     // of sequences with tiles
  int my_tiles;  // with at most 32 sequences: of sequence `lane`
  bool aligned;
};

// a / b.  A 32-bit division takes over a hundred cycles, and every CTA does several before it can load anything; below
// 2^22 the quotient of the floats is off by one at most.
__device__ __forceinline__ unsigned quotient(unsigned a, unsigned b) {
  if (a >= (1u << 22)) return a / b;
  const unsigned q = __float2uint_rz(__fdividef((float)a, (float)b));
  const int r = (int)(a - q * b);
  return r < 0 ? q - 1 : (unsigned)r >= b ? q + 1 : q;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// aligned: CTAs of a unit.  32-bit: a unit has at most 2^24 tiles, a GPU at most 255 SMs (both checked on the host).
__device__ __forceinline__ int ctas_of(const Split& sp, int tiles, int grid) {
  return tiles == 0 ? 0 : min(tiles, 1 + (int)quotient((unsigned)tiles * (unsigned)(grid - sp.units), (unsigned)sp.total));
}

// Tiles of each unit of sequence b0 + lane.
__device__ __forceinline__ int tiles_at(const Params& p, const Split& sp, int b0, int lane) {
  if (p.B <= 32) return sp.my_tiles;
  return b0 + lane < p.B ? seq_of(p, b0 + lane).tiles : 0;
}

// All lanes of a warp.  The number of all tiles fits an int (checked on the host).
__device__ __forceinline__ Split split_of(const Params& p, int lane, int grid, bool flag) {
  Split sp;
  sp.total = sp.units = sp.my_tiles = 0;
  const int upt = p.Hkv * p.row_tiles;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int n = 0;
    if (b0 + lane < p.B) {
      const Seq s = seq_of(p, b0 + lane);
      n = s.tiles;
      if (s.bad && flag) set_status(p.status, HATA_ERR_INVALID_ARG);
    }
    sp.my_tiles = n;
    sp.total += warp_sum(n) * upt;
    sp.units += __popc(__ballot_sync(0xffffffffu, n > 0)) * upt;
  }
  sp.per = max(1, (int)quotient((unsigned)(sp.total + grid - 1), (unsigned)grid));
  sp.aligned = false;
  if (sp.units > 0 && sp.units <= grid) {
    int longest = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int tiles = tiles_at(p, sp, b0, lane), k = ctas_of(sp, tiles, grid);
      longest = max(longest, __reduce_max_sync(0xffffffffu, k ? (int)quotient((unsigned)(tiles + k - 1), (unsigned)k) : 0));
    }
    sp.aligned = longest <= sp.per + kSwitchTiles;
  }
  return sp;
}

// Sum over the sequences before b of their tiles (flat) or CTAs (aligned).
__device__ __forceinline__ int before(const Params& p, const Split& sp, int lane, int grid, int b) {
  int sum = 0;
  const int upt = p.Hkv * p.row_tiles;
  for (int b0 = 0; b0 < b; b0 += 32) {
    const int tiles = tiles_at(p, sp, b0, lane);
    sum += warp_sum(b0 + lane < b ? (sp.aligned ? ctas_of(sp, tiles, grid) : tiles) * upt : 0);
  }
  return sum;
}

// A run of one unit's tiles.
struct Piece {
  int b, in_seq;  // sequence, unit within it
  Seq seq;
  int j0, j1;     // of the unit's list of tiles
  int cta;        // this CTA
  bool whole;     // all of the unit
  int slot;       // of its partial: a CTA continues one unit at most (2 cta), and leaves one at most (2 cta + 1)
};

// The runs of this CTA, one after another.  All lanes of a warp.
struct Walker {
  Split sp;
  int at, end;  // flat: of the list of all tiles
  int b, base;  // sequence, and its first tile (flat)
  Seq seq;
  bool one;     // aligned: a run is left
  Piece only;

  __device__ __forceinline__ void begin(const Params& p, int lane, bool flag) {
    const int grid = (int)gridDim.x, cta = (int)blockIdx.x, upt = p.Hkv * p.row_tiles;
    sp = split_of(p, lane, grid, flag);
    one = false;
    at = sp.aligned ? cta : cta * sp.per;  // cta * per < total + per * grid
    end = sp.aligned ? 0 : min(sp.total, at + sp.per);
    if (!sp.aligned && at >= end) return;
    // the sequence that holds tile (or CTA) `at`
    b = base = 0;
    bool found = false;
    for (int b0 = 0; b0 < p.B && !found; b0 += 32) {
      const int tiles = tiles_at(p, sp, b0, lane);
      const int n = (sp.aligned ? ctas_of(sp, tiles, grid) : tiles) * upt;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + incl > at);
      if (past) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        base += __shfl_sync(0xffffffffu, incl - n, l);
        found = true;
      } else {
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (!found) {  // aligned: more CTAs than runs
      end = at;
      return;
    }
    seq = seq_of(p, b);
    if (sp.aligned) {
      const unsigned k = (unsigned)ctas_of(sp, seq.tiles, grid), unit = quotient((unsigned)(at - base), k);
      const unsigned part = (unsigned)(at - base) - unit * k;
      only.b = b;
      only.in_seq = (int)unit;
      only.seq = seq;
      only.j0 = (int)quotient((unsigned)seq.tiles * part, k);
      only.j1 = (int)quotient((unsigned)seq.tiles * (part + 1), k);
      only.cta = cta;
      only.whole = k == 1;
      only.slot = 2 * cta;
      one = true;
      end = at;
    }
  }

  __device__ __forceinline__ bool next(const Params& p, Piece& s) {
    if (one) {
      s = only;
      one = false;
      return true;
    }
    if (at >= end) return false;
    const int upt = p.Hkv * p.row_tiles;
    while (at >= base + seq.tiles * upt) {
      base += seq.tiles * upt;
      seq = seq_of(p, ++b);
    }
    s.b = b;
    s.seq = seq;
    s.in_seq = (int)quotient((unsigned)(at - base), (unsigned)seq.tiles);
    const int u0 = base + s.in_seq * seq.tiles;
    s.j0 = at - u0;
    s.j1 = min(end - u0, seq.tiles);
    s.cta = (int)blockIdx.x;
    s.whole = s.j0 == 0 && s.j1 == seq.tiles;
    s.slot = 2 * s.cta + (s.j0 > 0 ? 0 : 1);
    at = u0 + s.j1;
    return true;
  }
};

// The runs of a unit, for the kernel that joins them: run i is CTA cta0 + i's, its partial in slot(i).
struct Runs {
  int cta0, n;
  bool aligned;
  int per, u0;
  __device__ __forceinline__ int slot(int i) const {
    const int c = cta0 + i;
    return 2 * c + (aligned || c * per > u0 ? 0 : 1);
  }
};

__device__ __forceinline__ Runs runs_of(const Params& p, int lane, int grid, int b, int in_seq, const Seq& seq) {
  const Split sp = split_of(p, lane, grid, false);
  const int first = before(p, sp, lane, grid, b);
  Runs r;
  r.aligned = sp.aligned;
  r.per = sp.per;
  r.u0 = first + in_seq * seq.tiles;
  if (sp.aligned) {
    r.n = ctas_of(sp, seq.tiles, grid);
    r.cta0 = first + in_seq * r.n;
  } else {
    r.cta0 = r.u0 / sp.per;
    r.n = (r.u0 + seq.tiles - 1) / sp.per - r.cta0 + 1;
  }
  return r;
}

// The n lowest bits (none below 1, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Bit k: new token i sees slot s0 + k (k < 32), of those that some token may see.
__device__ __forceinline__ uint32_t row_bits(const Params& p, const Seq& q, int b, int i, int s0) {
  const int j0 = s0 - q.ctx;  // the new token that slot s0 holds; before 0: context, seen by all
  if (!p.mask) return low_bits(i + 1 - j0);
  const uint32_t* row = p.mask + ((size_t)b * p.T + i) * p.mask_words;
  const int w = j0 >> 5;
  const uint32_t lo = w < 0 ? 0xffffffffu : w < p.mask_words ? __ldg(row + w) : 0u;
  const uint32_t hi = w + 1 < 0 ? 0xffffffffu : w + 1 < p.mask_words ? __ldg(row + w + 1) : 0u;
  return __funnelshift_r(lo, hi, j0 & 31);
}

// A slot that no token sees may hold anything (a value row that is not finite would turn 0 * V into NaN), so
// it is read as zeros.  Bit k of the answer: some token sees slot s0 + k (k < 16).  All lanes of a warp.
__device__ __forceinline__ unsigned seen_by_any16(const Params& p, const Seq& q, int b, int s0, int lane) {
  if (p.window <= 0 && s0 + 16 <= q.ctx) return 0xffffu;
  unsigned in = low_bits(min(16, q.L - s0));
  if (p.window > 0) in &= low_bits(p.sink - s0) | ~low_bits(q.L - min(p.window, q.L) - s0);
  if (s0 + 16 <= q.ctx || !p.mask || !in) return in;
  unsigned any = 0;
  for (int i = lane; i < q.n_b; i += 32) any |= row_bits(p, q, b, i, s0);
  return in & __reduce_or_sync(0xffffffffu, any);
}

}  // namespace span

// Whether the counts of the split fit their types.
inline bool span_fits(const span::Params& p, long long units) {
  return p.max_seq <= 0x7fffff00 && span_sms() <= 255 &&
         units * ((p.max_seq + span::kSpanTile - 1LL) / span::kSpanTile) <= 0x3fffffffLL;
}

// Tensor-core form of tree attention (hata_span_tc.cu): bf16, any number of rows.
size_t span_tc_part_bytes(const hata_dims_t& d, int n_tok);
cudaError_t launch_span_tc(const hata_dims_t& d, const span::Params& s, const PagedCache* pg, cudaStream_t stream);

}  // namespace hata
