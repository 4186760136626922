// Bookkeeping of a paged cache on the device, so that a whole serving step (roll back, fork, grow,
// append, attend, accept) is enqueued without a host round trip and can be captured in a graph:
//   fork     row b takes the pages of row parent[b], all rows read before any is written
//   resize   every row to its new length: pages past the end freed, a shared partial last page copied
//            (copy on write) before the row may append to it, new pages allocated
//   compact  accepted rows of the newest tokens moved to the front of them (K, V and codes)
// A page is free when its reference count is zero, and the j-th page needed is the j-th lowest free page, so
// there is no list of free pages to keep, and the result does not depend on the order of threads.
//
// Bound: latency.  The tables and counts are a few hundred KB, read and written once; resize's
// decisions are one CTA (a prefix sum over rows and two passes over the counts, kept in shared memory), its copies and
// compact's moves spread over all SMs as 16-byte vectors.  The kernels are launched early, so a
// launch overlaps the kernel before it.  Measured on B200: a beam step of 32 sequences over 256-page
// rows (roll back, fork 8 into 24, grow with 24 copies on write: five kernels) 19-21 us, of which each
// resize's decisions are about 5; compacting 16 sequences' trees of 64 tokens 3.0-3.4 us.
#include <algorithm>
#include <map>
#include <mutex>

#include "hata_kernels.cuh"
#include "hata_ptx.cuh"

namespace hata {

namespace {

constexpr int kPgThreads = 1024;
constexpr int kPgWarps = kPgThreads / 32;
constexpr int kForkCols = 8;  // table columns of one fork CTA
constexpr int kFreeBatch = 8;  // entries a lane frees at a time: a round trip to a count takes about a microsecond

// ---- fork: a CTA owns 8 columns of the table: it reads them for every row, then writes them
__global__ void __launch_bounds__(256)
    pages_fork_kernel(const int32_t* __restrict__ parent, int32_t* table, int32_t* seq_lens, int32_t* ref, int B,
                      int max_blocks, int n_blocks, uint32_t* status) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  extern __shared__ int32_t fork_old[];  // [B][kForkCols], then for CTA 0 the lengths [B]
  const int c0 = (int)blockIdx.x * kForkCols, tid = threadIdx.x;
  for (int e = tid; e < B * kForkCols; e += blockDim.x) {
    const int c = c0 + e % kForkCols;
    fork_old[e] = c < max_blocks ? table[(size_t)(e / kForkCols) * max_blocks + c] : -1;
  }
  int32_t* lens = fork_old + (size_t)B * kForkCols;
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += blockDim.x) lens[b] = seq_lens[b];
  __syncthreads();
  for (int e = tid; e < B * kForkCols; e += blockDim.x) {
    const int b = e / kForkCols, c = c0 + e % kForkCols, pa = parent[b];
    if (pa < 0 || pa >= B || pa == b) continue;
    const int was = fork_old[e], now = fork_old[pa * kForkCols + e % kForkCols];
    if (c >= max_blocks || was == now) continue;  // the same page (or none) on both sides
    if (was >= 0 && was < n_blocks) atomicSub(&ref[was], 1);
    if (now >= 0 && now < n_blocks) atomicAdd(&ref[now], 1);
    table[(size_t)b * max_blocks + c] = now;
  }
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += blockDim.x) {
      const int pa = parent[b];
      if (pa >= B) set_status(status, HATA_ERR_INVALID_ARG);
      if (pa >= 0 && pa < B && pa != b) seq_lens[b] = lens[pa];
    }
}

// ---- resize: the decisions, by one CTA
struct ResizeParams {
  const int32_t* new_lens;
  int32_t *table, *seq_lens, *ref;
  int32_t* copies;  // workspace: per row (source page, target page, rows), source -1: nothing to copy
  int B, max_seq, max_blocks, n_blocks, block_shift;
  uint32_t* status;
};

// LOCAL: the counts are brought into shared memory first and written back at the end.  Freeing the 4800 entries of 24 rows
// takes 4800 atomics, at one SM's rate of about one scattered atomic per cycle and 1.7 cycles each 4 us in L2.  Pools whose
// counts do not fit (about 50,000 pages) do it there.
template <bool LOCAL>
__global__ void __launch_bounds__(kPgThreads) pages_resize_kernel(const ResizeParams p) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  extern __shared__ int32_t rs_smem[];
  int32_t* s_old = rs_smem;         // length before, -1: the row stays out of it
  int32_t* s_new = s_old + p.B;     // length after
  int32_t* s_tail = s_new + p.B;    // page a growing row would write into, else -1
  int32_t* s_first = s_tail + p.B;  // first column that gets a page
  int32_t* s_pre = s_first + p.B;   // pages needed by earlier rows; [B]: by all
  int32_t* s_ref = s_pre + p.B + 1;  // LOCAL: the counts
  __shared__ int32_t scan_sum[kPgWarps], free_sum[kPgWarps];
  __shared__ int32_t s_free;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.B;
  const int bs = 1 << p.block_shift;
  auto pages_of = [&](int len) { return (int)(((long long)len + bs - 1) >> p.block_shift); };
  auto count = [&](int q) -> int {
    if constexpr (LOCAL) return s_ref[q];
    else return __ldcg(&p.ref[q]);
  };
  auto add = [&](int q, int n) -> int {  // the count before
    if constexpr (LOCAL) return atomicAdd(&s_ref[q], n);
    else return atomicAdd(&p.ref[q], n);
  };
  if constexpr (LOCAL) {
#pragma unroll 8
    for (int q = tid; q < p.n_blocks; q += kPgThreads) s_ref[q] = p.ref[q];
  }
  for (int b = tid; b < B; b += kPgThreads) {
    const int old = p.seq_lens[b], nw = p.new_lens[b];
    const bool ok = old >= 0 && old <= p.max_seq, ok_new = nw >= 0 && nw <= p.max_seq;
    if (!ok || !ok_new) set_status(p.status, HATA_ERR_INVALID_ARG);
    s_old[b] = ok ? old : -1;
    s_new[b] = ok_new ? nw : old;  // a new length out of range leaves the row as it is
    p.copies[3 * b] = -1;
  }
  __syncthreads();
  // the last pages of growing rows that are partly filled
  for (int b = tid; b < B; b += kPgThreads) {
    const int old = s_old[b];
    int tail = -1;
    if (old >= 0 && s_new[b] > old && (old & (bs - 1))) {
      tail = p.table[(size_t)b * p.max_blocks + pages_of(old) - 1];
      if (tail < 0 || tail >= p.n_blocks) {
        tail = -1;
        set_status(p.status, HATA_ERR_INVALID_ARG);
      }
    }
    s_tail[b] = tail;
  }
  // frees: a warp per row
  for (int b = warp; b < B; b += kPgWarps) {
    const int old = s_old[b];
    if (old < 0) continue;
    const int n_new = pages_of(s_new[b]), n_old = pages_of(old);
    int32_t* row = p.table + (size_t)b * p.max_blocks;
    for (int c0 = n_new + lane; c0 < n_old; c0 += 32 * kFreeBatch) {
      int page[kFreeBatch], held[kFreeBatch];
#pragma unroll
      for (int k = 0; k < kFreeBatch; ++k) page[k] = c0 + 32 * k < n_old ? row[c0 + 32 * k] : INT32_MIN;
#pragma unroll
      for (int k = 0; k < kFreeBatch; ++k) {
        if (page[k] != INT32_MIN) row[c0 + 32 * k] = -1;
        held[k] = page[k] >= 0 && page[k] < p.n_blocks ? add(page[k], -1) : 1;
      }
#pragma unroll
      for (int k = 0; k < kFreeBatch; ++k) {
        if (page[k] == INT32_MIN) continue;
        if (held[k] <= 0) add(page[k], 1);  // counted less often than it is used
        if (held[k] <= 0 || page[k] < 0 || page[k] >= p.n_blocks) set_status(p.status, HATA_ERR_INVALID_ARG);
      }
    }
  }
  __syncthreads();
  // each warp counts the free pages of its share of them
  const int per = ((p.n_blocks + kPgWarps - 1) / kPgWarps + 31) / 32 * 32;
  const int p0 = min(p.n_blocks, warp * per), p1 = min(p.n_blocks, p0 + per);
  int mine = 0;
#pragma unroll 8
  for (int q = p0 + lane; q < p1; q += 32) mine += count(q) == 0;
  // needs: of the rows that share a tail page and grow, the earlier ones copy it and, when nobody else holds
  // it, the last one keeps it (what rows handled one after another would do)
  for (int b = tid; b < B; b += kPgThreads) {
    const int old = s_old[b];
    int need = 0, first = 0;
    if (old >= 0) {
      const int nw = s_new[b], n_old = pages_of(old);
      int copy = 0;
      if (nw > old) {
        if (s_tail[b] >= 0) {
          const int held = count(s_tail[b]);
          if (held > 1) {
            int earlier = 0;
            for (int o = 0; o < b; ++o) earlier += s_tail[o] == s_tail[b];
            copy = held - earlier > 1;
          }
        }
        need = pages_of(nw) - n_old + copy;
      }
      first = n_old - copy;
    }
    s_first[b] = first;
    s_pre[b] = need;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) free_sum[warp] = mine;
  __syncthreads();
  // exclusive prefix of the needs over rows
  int carry = 0;
  for (int b0 = 0; b0 < B; b0 += kPgThreads) {
    const int v = b0 + tid < B ? s_pre[b0 + tid] : 0;
    int tot = 0;
    const int x = block_exclusive_scan<kPgThreads>(v, scan_sum, &tot);
    if (b0 + tid < B) s_pre[b0 + tid] = carry + x;
    carry += tot;
  }
  if (tid == 0) s_pre[B] = carry;
  const int total = carry;
  if (warp == 0) {
    int x = free_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_free = x;
    free_sum[lane] = x;
  }
  __syncthreads();
  const bool enough = s_free >= total;
  if (!enough && tid == 0) set_status(p.status, HATA_ERR_NO_PAGES);
  if (enough && total > 0) {
    int rank = free_sum[warp] - mine;  // free pages before this warp's share
    for (int q0 = p0; q0 < p1 && rank < total; q0 += 32) {
      const int q = q0 + lane;
      const bool is_free = q < p1 && count(q) == 0;
      const unsigned m = __ballot_sync(0xffffffffu, is_free);
      const int r = rank + __popc(m & ((1u << lane) - 1u));
      if (is_free && r < total) {
        int lo = 0, hi = B;  // the row b with s_pre[b] <= r < s_pre[b + 1]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_pre[mid] <= r) lo = mid;
          else hi = mid;
        }
        p.table[(size_t)lo * p.max_blocks + s_first[lo] + (r - s_pre[lo])] = q;
        add(q, 1);
        if (r == s_pre[lo] && s_first[lo] < pages_of(s_old[lo])) {  // takes the place of a shared last page
          p.copies[3 * lo + 1] = q;
          p.copies[3 * lo + 2] = s_old[lo] & (bs - 1);
          p.copies[3 * lo] = s_tail[lo];
        }
      }
      rank += __popc(m);
    }
  }
  __syncthreads();
  for (int b = tid; b < B; b += kPgThreads) {
    const int old = s_old[b], nw = s_new[b];
    if (old < 0 || (nw > old && !enough)) continue;  // too few pages: no row grows
    if (nw > old && s_first[b] < pages_of(old)) add(s_tail[b], -1);
    p.seq_lens[b] = nw;
  }
  if constexpr (LOCAL) {
    __syncthreads();
#pragma unroll 8
    for (int q = tid; q < p.n_blocks; q += kPgThreads) p.ref[q] = s_ref[q];
  }
}

// Shared memory that counts may take, and the kernel's attribute for it, set once per device under a mutex.
constexpr size_t kLocalBytes = 220 * 1024;
cudaError_t configure_local() {
  static std::mutex mu;
  static std::map<int, cudaError_t> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  auto it = done.find(dev);
  if (it != done.end()) return it->second;
  e = cudaFuncSetAttribute(pages_resize_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLocalBytes);
  if (e != cudaSuccess) (void)cudaGetLastError();
  done[dev] = e;
  return e;
}

// ---- copies: one CTA per (row, KV head, piece) and tensor; a page's rows of one head are contiguous
__global__ void __launch_bounds__(256)
    pages_copy_kernel(const int32_t* copies, unsigned char* K, unsigned char* V, unsigned char* codes,
                      int hkv, int bs, int row_bytes, int code_bytes, int n_piece) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int b = blockIdx.y;
  const int src = copies[3 * b];
  if (src < 0) return;
  const int dst = copies[3 * b + 1], rows = copies[3 * b + 2];
  int x = (int)blockIdx.x;
  const int piece = x % n_piece;
  x /= n_piece;
  const int g = x % hkv, t = x / hkv;
  unsigned char* base = t == 0 ? K : t == 1 ? V : codes;
  const int rb = t < 2 ? row_bytes : code_bytes;
  unsigned char* from = base + ((size_t)src * hkv + g) * bs * rb;
  unsigned char* to = base + ((size_t)dst * hkv + g) * bs * rb;
  const size_t bytes = (size_t)rows * rb, nv = bytes / 16;
  for (size_t e = (size_t)piece * 256 + threadIdx.x; e < nv; e += (size_t)n_piece * 256)
    reinterpret_cast<uint4*>(to)[e] = reinterpret_cast<const uint4*>(from)[e];
  if (piece == 0) {  // the last bytes of narrow codes
    const size_t e = nv * 16 + 2 * threadIdx.x;
    if (e < bytes) *reinterpret_cast<uint16_t*>(to + e) = *reinterpret_cast<const uint16_t*>(from + e);
  }
}

// ---- compact: row base + keep[j] to row base + j, j < n_keep, keep ascending.  A target row j is never the
// source of a later chunk (source j' >= j'), so a CTA that owns some heads of (b, tensor) loads a
// chunk of rows, waits for all of it, stores it and goes on.
struct CompactParams {
  const int32_t *keep, *n_keep, *n_new, *seq_lens;
  unsigned char *K, *V, *codes;
  int32_t* new_lens;
  const int32_t* block_table;
  uint32_t* status;
  int B, n_tok, Hkv, max_seq, row_shift, code_shift;  // log2 of 16-byte pieces of a row; of pieces of a code
  int code_bytes;
  int head_shift, head_groups;  // log2 of the heads of a CTA, CTAs of a tensor
  int block_shift, n_blocks, max_blocks;
};

constexpr int kCpThreads = 256;
constexpr int kCpBatch = 4;  // pieces a thread holds between load and store

// Rows of `heads` KV heads (a power of two) from g0 on.
template <typename E, bool PAGED>
__device__ __forceinline__ void compact_rows(const CompactParams& p, E* base, int row_shift, int b, int g0, int start,
                                             int n_keep) {
  // pieces of type E: 1 << row_shift of them make a row, and consecutive threads take consecutive pieces
  const int32_t* keep = p.keep + (size_t)b * p.n_tok;
  auto row_of = [&](int t, int g, bool& ok) -> size_t {
    if constexpr (PAGED) {
      const int blk = p.block_table[(size_t)b * p.max_blocks + (t >> p.block_shift)];
      if (blk < 0 || blk >= p.n_blocks) {
        ok = false;
        return 0;
      }
      return (((size_t)blk * p.Hkv + g) << p.block_shift) + (size_t)(t & ((1 << p.block_shift) - 1));
    } else {
      return ((size_t)b * p.Hkv + g) * p.max_seq + t;
    }
  };
  const int j_shift = row_shift + p.head_shift, row_mask = (1 << row_shift) - 1, head_mask = (1 << p.head_shift) - 1;
  const long long n = (long long)n_keep << j_shift;
  for (long long e0 = 0; e0 < n; e0 += kCpThreads * kCpBatch) {
    E v[kCpBatch];
    size_t to[kCpBatch];
    bool moves[kCpBatch];
#pragma unroll
    for (int u = 0; u < kCpBatch; ++u) {
      const long long e = e0 + u * kCpThreads + threadIdx.x;
      moves[u] = false;
      const int g = g0 + ((int)(e >> row_shift) & head_mask);
      if (e >= n || g >= p.Hkv) continue;
      const int j = (int)(e >> j_shift), c = (int)e & row_mask;
      const int k = keep[j];
      if (k == j) continue;
      bool ok = true;
      const size_t from = row_of(start + k, g, ok);
      const size_t dst = row_of(start + j, g, ok);
      if (!ok) {
        set_status(p.status, HATA_ERR_INVALID_ARG);
        continue;
      }
      moves[u] = true;
      to[u] = (dst << row_shift) + c;
      v[u] = base[(from << row_shift) + c];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCpBatch; ++u)
      if (moves[u]) base[to[u]] = v[u];
    __syncthreads();
  }
}

// The end of the slots in [start, end) of sequence b that another sequence holds too, in a page that both have in the
// same column (as hata_pages_fork leaves them); 0 if there are none.  This thread's share of the other rows and columns.
__device__ __forceinline__ int shared_end(const CompactParams& p, int b, int start, int end) {
  int top = 0;
  if (start >= end) return top;
  const int c1 = ((end - 1) >> p.block_shift) + 1;
  const int across = p.B <= 32 ? 32 : kCpThreads;  // threads side by side on the rows of one column
  for (int c = (start >> p.block_shift) + (int)threadIdx.x / across; c < c1; c += kCpThreads / across) {
    const int page = p.block_table[(size_t)b * p.max_blocks + c];
#pragma unroll 4
    for (int o = (int)threadIdx.x % across; o < p.B; o += across) {
      const int held = min(min(p.seq_lens[o], end), (int)min((long long)(c + 1) << p.block_shift, 0x7fffffffLL));
      const int other = p.block_table[(size_t)o * p.max_blocks + c];
      if (o != b && page == other && page >= 0 && page < p.n_blocks && held > c << p.block_shift) top = max(top, held);
    }
  }
  return top;
}

template <bool PAGED>
__global__ void __launch_bounds__(kCpThreads) compact_kernel(const CompactParams p) {
  const int b = blockIdx.y, t = (int)blockIdx.x / p.head_groups, tid = threadIdx.x;
  const int g = ((int)blockIdx.x - t * p.head_groups) << p.head_shift;
  const int L = p.seq_lens[b], n_b = p.n_new ? p.n_new[b] : p.n_tok, n_keep = p.n_keep[b];
  bool bad = n_b < 0 || n_b > p.n_tok || L < n_b || L > p.max_seq || n_keep < 0 || n_keep > n_b;
  if (!bad) {
    const int32_t* keep = p.keep + (size_t)b * p.n_tok;
    int wrong = 0, moved = n_keep;  // first row that moves: keep ascends, so all later ones do too
    int k = tid < n_keep ? keep[tid] : 0, before = tid > 0 && tid < n_keep ? keep[tid - 1] : -1;
    int top = 0;
    if constexpr (PAGED) top = shared_end(p, b, L - n_b, L - n_b + n_keep);  // its loads and those of keep go out together
    for (int j = tid; j < n_keep;) {
      wrong |= k < 0 || k >= n_b || before >= k;
      if (k != j) moved = min(moved, j);
      if ((j += kCpThreads) < n_keep) {
        k = keep[j];
        before = keep[j - 1];
      }
    }
    if constexpr (PAGED) {
      // Rows that another sequence holds must not move under it.  Every CTA of the sequence finds the same answer.
      __shared__ int s_moved[kCpThreads / 32], s_top[kCpThreads / 32];
      top = __reduce_max_sync(0xffffffffu, top);
      moved = __reduce_min_sync(0xffffffffu, moved);
      if ((tid & 31) == 0) {
        s_moved[tid >> 5] = moved;
        s_top[tid >> 5] = top;
      }
      bad = __syncthreads_or(wrong) != 0;
      int first = n_keep, end = 0;
#pragma unroll
      for (int w = 0; w < kCpThreads / 32; ++w) {
        first = min(first, s_moved[w]);
        end = max(end, s_top[w]);
      }
      bad |= end > L - n_b + first;
    } else {
      bad = __syncthreads_or(wrong) != 0;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) set_status(p.status, HATA_ERR_INVALID_ARG);
    if (p.new_lens) p.new_lens[b] = bad ? L : L - n_b + n_keep;
  }
  if (bad) return;
  if (t < 2) {
    compact_rows<uint4, PAGED>(p, reinterpret_cast<uint4*>(t == 0 ? p.K : p.V), p.row_shift, b, g, L - n_b, n_keep);
  } else if (p.code_bytes == 2) {
    compact_rows<uint16_t, PAGED>(p, reinterpret_cast<uint16_t*>(p.codes), 0, b, g, L - n_b, n_keep);
  } else {
    compact_rows<uint32_t, PAGED>(p, reinterpret_cast<uint32_t*>(p.codes), p.code_shift, b, g, L - n_b, n_keep);
  }
}

}  // namespace

size_t pages_ws_bytes(int batch) { return align_up(kStatusBytes, 16) + align_up((size_t)batch * 12, 16); }

cudaError_t launch_pages_fork(const hata_dims_t& d, const int32_t* parent, int32_t* table, int max_blocks,
                              int n_blocks, int32_t* seq_lens, int32_t* ref, uint32_t* status, cudaStream_t st) {
  const unsigned grid = (unsigned)((max_blocks + kForkCols - 1) / kForkCols);
  const size_t smem = (size_t)d.batch * (kForkCols + 1) * 4;  // at most 36 KB: d.batch <= kMaxPageRows
  return launch_early(pages_fork_kernel, dim3(grid), 256, smem, st, parent, table, seq_lens, ref, d.batch, max_blocks, n_blocks,
                      status);
}

cudaError_t launch_pages_resize(const hata_dims_t& d, const int32_t* new_lens, void* K, void* V, void* codes,
                                const PagedCache& pg, int32_t* table, int32_t* seq_lens, int32_t* ref, char* ws,
                                cudaStream_t st) {
  ResizeParams p;
  p.new_lens = new_lens;
  p.table = table;
  p.seq_lens = seq_lens;
  p.ref = ref;
  p.copies = reinterpret_cast<int32_t*>(ws + kStatusBytes);
  p.B = d.batch;
  p.max_seq = d.max_seq;
  p.max_blocks = pg.max_blocks;
  p.n_blocks = pg.n_blocks;
  p.block_shift = pg.block_shift;
  p.status = reinterpret_cast<uint32_t*>(ws);
  const size_t rows = (size_t)(5 * d.batch + 1) * 4, local = rows + (size_t)pg.n_blocks * 4;
  cudaError_t e;
  if (local <= kLocalBytes) {
    if ((e = configure_local()) != cudaSuccess) return e;
    e = launch_early(pages_resize_kernel<true>, dim3(1), kPgThreads, local, st, p);
  } else {
    e = launch_early(pages_resize_kernel<false>, dim3(1), kPgThreads, rows, st, p);  // at most 21 KB
  }
  if (e != cudaSuccess) return e;
  const int bs = 1 << pg.block_shift, row_bytes = kHeadDim * (d.dtype == HATA_BF16 ? 2 : 4);
  const int n_piece = std::max(1, std::min(64, bs / 64));  // 16-32 KB of a K page per CTA
  const int tensors = codes ? 3 : 2;
  return launch_early(pages_copy_kernel, dim3((unsigned)(tensors * d.n_kv_heads * n_piece), (unsigned)d.batch), 256, 0, st,
                      p.copies, static_cast<unsigned char*>(K), static_cast<unsigned char*>(V),
                      static_cast<unsigned char*>(codes), d.n_kv_heads, bs, row_bytes, d.hash_bits / 8, n_piece);
}

cudaError_t launch_compact(const hata_dims_t& d, int n_tok, const int32_t* keep, const int32_t* n_keep,
                           const int32_t* n_new, const int32_t* seq_lens, void* K, void* V, void* codes,
                           const PagedCache* pg, int32_t* new_lens, uint32_t* status, cudaStream_t st) {
  CompactParams p{};
  p.keep = keep;
  p.n_keep = n_keep;
  p.n_new = n_new;
  p.seq_lens = seq_lens;
  p.K = static_cast<unsigned char*>(K);
  p.V = static_cast<unsigned char*>(V);
  p.codes = static_cast<unsigned char*>(codes);
  p.new_lens = new_lens;
  p.status = status;
  p.B = d.batch;
  p.n_tok = n_tok;
  p.Hkv = d.n_kv_heads;
  p.max_seq = d.max_seq;
  p.row_shift = d.dtype == HATA_BF16 ? 4 : 5;
  p.code_bytes = d.hash_bits / 8;
  while ((4 << p.code_shift) < p.code_bytes) ++p.code_shift;
  if (pg) {
    p.block_table = pg->block_table;
    p.block_shift = pg->block_shift;
    p.n_blocks = pg->n_blocks;
    p.max_blocks = pg->max_blocks;
  }
  if (d.batch > 65535) return cudaErrorNotSupported;
  // A CTA takes several heads where the CTAs left still are four per SM: each looks through its page's column of the
  // table (256 sequences, 8 heads, 5 rows kept of 64: 22 us with one head, 6 with eight).
  const int tensors = codes ? 3 : 2;
  auto groups = [&](int shift) { return (d.n_kv_heads + (1 << shift) - 1) >> shift; };
  while ((1 << p.head_shift) < d.n_kv_heads && (long long)d.batch * tensors * groups(p.head_shift + 1) >= 4 * span_sms())
    ++p.head_shift;
  p.head_groups = groups(p.head_shift);
  const dim3 grid((unsigned)(p.head_groups * tensors), (unsigned)d.batch);
  if (pg) compact_kernel<true><<<grid, kCpThreads, 0, st>>>(p);
  else compact_kernel<false><<<grid, kCpThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace hata
