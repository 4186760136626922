// Attention on the 5th-generation tensor cores where many query rows share their keys: prefill with a
// sliding window and sinks, and tree attention when a KV head has many (query head, token) rows.
//
// A CTA (twelve warps, two idle; one per SM, persistent) runs two streams.  A stream is 128 query rows with their
// own scores S and output O in TMEM (128 columns each) and a warpgroup whose thread owns one row:
//   S = Q K^T (tcgen05.mma, M = N = 128)  ->  p = 2^(s c - m), c = scale log2 e, in registers  ->  P as bf16 over
//   the first half of S  ->  O += P V (P from TMEM, V as an MN-major operand)
// While one stream's warpgroup computes its exponentials, the tensor core works for the other.  K and V tiles of
// 128 slots come through one ring of five 32 KB stages (four for a prefill) (TMA; a page of fewer than 128 slots is a box of its own);
// one warp loads, one lane of another issues the MMAs.  The running maximum m moves only when a row's maximum
// passes it by more than 2^8; O is then rescaled in TMEM, which is safe once S has arrived, since the MMAs run in
// order and PV of the tile before was issued first.
//
// The two streams take
//   * prefill: 256 rows = P heads of one group x 256 / P positions, P the largest power of two in G (at most
//     16), so a window's ragged ends cost 256 / P rows, not 256; their keys are the sinks' rows and the window's,
//     packed into tiles together;
//   * tree, more than 128 rows: two tiles of rows, every key tile read by both;
//   * tree, up to 128 rows: the same rows, even key tiles for one stream, odd ones for the other.
// Prefill writes its rows.  Tree attention splits the key tiles of all units evenly over the CTAs (hata_span.cuh);
// each run of a unit leaves (maximum, sum, O) in fp32 in the workspace, and span_merge_kernel joins them in
// the order of the split.
//
// Bound by the chain of a stream: about 2400 cycles of a row's warpgroup per tile (the exponentials alone are 1024 at the
// 8 cycles that an SMSP needs for a warp's ex2) and 1060 from P to the next S (768 of MMAs, the rest handing over), while
// the two streams' MMAs take 2048 of the 3550 that a pair of tiles costs.  Measured on B200: prefill of 8192 positions,
// window 1024, 4 sinks, 32 / 8 heads 147 us (0.54 of the measured bf16 burst rate over the visible pairs; 164 us, 0.49,
// when it runs for seconds); 256 rows over 4 x 57K slots 227-236 us (0.61-0.63 of a copy's bandwidth; 286-291 us, 0.50, for
// seconds on end); 64 rows over 4 x 32K slots 110 us (0.75).
// Slower than the 154 us that the prefill took then: sixteen row warps with half of the columns each (166 us); half tiles of
// N = 64, so that scores come while the other half is turned (179 us: twice the handing over, and N = 64 MMAs at two
// thirds of the rate).
// P is rounded to bf16, the type of V, with which it shares an MMA; the row sums take it unrounded, in fp32.
//
// Every wait is bounded; on expiry HATA_ERR_TIMEOUT goes to the status word, and the CTA stops issuing,
// waits (bounded) for its copies and MMAs, frees its TMEM and returns.
#include <algorithm>
#include <map>
#include <mutex>

#include "hata_ptx.cuh"
#include "hata_span.cuh"
#include "hata_tc.cuh"

namespace hata {

namespace {

using span::Params;

constexpr int kTcThreads = 384;  // two warpgroups of rows, one of loader, MMA issue and two idle warps
// Registers of a thread: 152 at launch, then 192 for the rows' warpgroups (a row's 128 scores stay in registers) and
// 72 for the other (256 x 192 + 128 x 72 = 384 x 152); the rest of the SM's leaves room for a merging CTA.
constexpr int kTcRegs = 152, kTcRowRegs = 192, kTcIssueRegs = 72;
static_assert(256 * kTcRowRegs + 128 * kTcIssueRegs == kTcThreads * kTcRegs, "registers of the launch");
constexpr int kTcMmaWarp = 8, kTcTmaWarp = 9;
constexpr int kTcTile = 128;
static_assert(kTcTile == span::kSpanTile, "the split of the work counts these tiles");
constexpr int kTcTileB = kTcTile * kHeadDim * 2;  // 32 KB
constexpr int kTcStages = 5;  // of the ring; a prefill uses the last one to write its rows out
constexpr uint32_t kTcQ = 0;                      // two tiles of query rows
constexpr uint32_t kTcRing = 2 * kTcTileB;
constexpr uint32_t kTcOut = kTcRing + (kTcStages - 1) * kTcTileB;  // per stream 128 rows x 64 columns of output, 16 KB
constexpr int kTcSmem = (2 + kTcStages) * kTcTileB + 1024;         // + alignment to 1024 bytes
constexpr uint32_t kTcTmemCols = 512;             // S of the streams at 0 and 128, O at 256 and 384
constexpr uint32_t kTcTries = 1u << 22, kTcTestTries = 1u << 10;
constexpr float kTcSlack = 8.f;  // log2 units: p <= 2^8 between rescales
constexpr int kPartFloats = kTcTile * (kHeadDim + 2);  // a stream's partial: m [128], l [128], O [32][128][4]

struct TcParams {
  Params s;
  int prefill_heads;  // P: heads of a prefill CTA
  int pos_block;      // prefill: positions of a CTA (256 / P)
  int pos_shift;      // prefill: log2 of the rows of one head in a stream
  int n_blocks_pos;   // prefill: blocks of positions
  int rows_of_items;  // prefill: CTAs' items per block of positions, B * Hq / P
  int pair;           // tree: two tiles of rows (else one, its key tiles shared out)
  int box_rows;       // rows of a K / V box
  int q_box;          // rows of a Q box
  int test_expire;
};

// The MMAs of K = 16 that make one 128 x 128 x 128 product, issued by one elected lane of a warp whose lanes all
// call this together with the same arguments: descriptors then stay in uniform registers.  Issued under `if (lane ==
// 0)` the same eight took 730 to 1050 cycles, against the 512 that the tensor core needs.
// S = Q K^T: both operands K-major, four steps of 32 bytes in each half of 64 columns
__device__ __forceinline__ void mma8_s(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 1024;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 1026;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 1028;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 1030;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
      "l"(q), "l"(k), "r"(idesc)
      : "memory");
}
// Half of O (+)= P V, 64 slots: P in TMEM (8 columns per step), V MN-major (2048 bytes per step); `more`: add to O
__device__ __forceinline__ void mma4_pv(uint32_t d, uint32_t pa, uint64_t v, uint32_t idesc, uint32_t more) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t}\n" ::"r"(d),
      "r"(pa), "l"(v), "r"(idesc), "r"(more)
      : "memory");
}
// tc::commit by the lane that issues the MMAs
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(tc::smem_u32(bar))
      : "memory");
}

// One CTA's next piece of work: a run of key tiles for its two streams.
struct Seg {
  int b, g;
  int L, ctx, n_b;
  int sr, base;              // key row r of the run's list is slot r for r < sr, else slot r + base
  int j0, j1;                // tiles of 128 key rows
  int row0;                  // tree: first row; prefill: first position
  int head0;                 // prefill: first query head
  long long slot;            // tree: partial
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
// 16 consecutive 32-bit columns written to this thread's TMEM lane
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Walks the pieces of work of a CTA.  All lanes of a warp call it together; every warp walks alike.
template <bool TREE>
struct Walk {
  const TcParams& p;
  int lane;
  int at, end, per;  // prefill: items of this CTA
  span::Walker runs;

  __device__ __forceinline__ Walk(const TcParams& prm, int ln, bool flag) : p(prm), lane(ln) {
    if constexpr (TREE) {
      runs.begin(p.s, lane, flag);
    } else {
      if (flag)
        for (int b = lane; b < p.s.B; b += 32)
          if (p.s.seq_lens[b] > p.s.max_seq) set_status(p.s.status, HATA_ERR_INVALID_ARG);
      per = gridDim.x;
      at = blockIdx.x;
      end = p.n_blocks_pos * p.rows_of_items;
    }
  }

  __device__ __forceinline__ bool next(Seg& s) {
    if constexpr (TREE) {
      span::Piece pc;
      if (!runs.next(p.s, pc)) return false;
      s.b = pc.b;
      s.g = pc.in_seq % p.s.Hkv;
      s.L = pc.seq.L;
      s.ctx = pc.seq.ctx;
      s.n_b = pc.seq.n_b;
      s.sr = s.base = 0;
      s.j0 = pc.j0;
      s.j1 = pc.j1;
      s.row0 = pc.in_seq / p.s.Hkv * (p.pair ? 2 * kTcTile : kTcTile);
      s.head0 = 0;
      // unit + CTA grows along the runs, so no two share it
      s.slot = (long long)pc.b * p.s.Hkv * p.s.row_tiles + pc.in_seq + pc.cta;
      return true;
    } else {
      for (; at < end; at += per) {
        const unsigned blk_up = (unsigned)at / (unsigned)p.rows_of_items, rest = (unsigned)at % (unsigned)p.rows_of_items;
        const unsigned hb = (unsigned)(p.rows_of_items / p.s.B);
        const int blk = p.n_blocks_pos - 1 - (int)blk_up;  // the longest rows first
        s.b = (int)(rest / hb);
        s.head0 = (int)(rest % hb) * p.prefill_heads;
        s.g = s.head0 / p.s.G;
        int L = p.s.seq_lens[s.b];
        L = max(0, min(L, p.s.max_seq));
        s.row0 = blk * p.pos_block;
        if (s.row0 >= L) continue;
        s.L = s.ctx = L;
        s.n_b = 0;
        const int t_hi = min(s.row0 + p.pos_block, L) - 1;
        // The sinks' rows (to a multiple of 8), then the rows from the first one that the block's window
        // reaches, packed into tiles without the gap between them.
        const int w0 = max(0, s.row0 - min(p.s.window, s.row0 + 1) + 1), sinks = (min(p.s.sink, t_hi + 1) + 7) / 8 * 8;
        const bool gap = w0 > sinks;
        s.sr = gap ? sinks : 0;
        s.base = gap ? w0 - sinks : 0;
        s.j0 = 0;
        s.j1 = (t_hi - s.base) / kTcTile + 1;
        s.slot = 0;
        at += per;
        return true;
      }
      return false;
    }
  }
};

// Visibility words of new tokens, 128 bits in four registers; bit j: token j is seen.
struct Bits128 {
  uint32_t w0, w1, w2, w3;
  __device__ __forceinline__ uint32_t word(int i) const {  // ones below (the context), zeros above
    return i < 0 ? 0xffffffffu : i == 0 ? w0 : i == 1 ? w1 : i == 2 ? w2 : i == 3 ? w3 : 0u;
  }
  // bits j0 .. j0 + 31, where negative indices are slots before the new tokens
  __device__ __forceinline__ uint32_t at(int j0) const {
    const int i = j0 >> 5;  // floor
    return __funnelshift_r(word(i), word(i + 1), j0 & 31);
  }
};

template <bool TREE, bool PAGED>
__global__ void __maxnreg__(kTcRegs)
    span_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap kmap8,
                   const __grid_constant__ CUtensorMap vmap8, const TcParams p) {
  constexpr uint32_t kStages = TREE ? kTcStages : kTcStages - 1;
  extern __shared__ __align__(1024) unsigned char tc_smem[];
  __shared__ __align__(8) uint64_t q_full, q_free, full[kStages], freed[kStages], s_full[2], p_half[2], p_full[2],
      o_full[2], drain, never;
  __shared__ uint32_t tmem_s;
  __shared__ volatile int abort_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (tc::smem_u32(tc_smem) + 1023u) & ~1023u;
  // What came before on the stream has ended, before TMEM is taken: its CTAs may need TMEM of this SM.
  ptx::pdl_wait();
  if (warp == 0) tc::tmem_alloc(&tmem_s, kTcTmemCols);
  if (tid == 256) {
    tc::mbar_init(&q_full, 1);
    tc::mbar_init(&q_free, 1);
    for (uint32_t i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&freed[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(&s_full[w], 1);
      tc::mbar_init(&p_half[w], kTcTile);
      tc::mbar_init(&p_full[w], kTcTile);
      tc::mbar_init(&o_full[w], 1);
    }
    tc::mbar_init(&drain, 1);
    tc::mbar_init(&never, 1);
    tc::mbar_init_fence();
    abort_s = 0;
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_s;

  auto wait_ok = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (tc::mbar_wait(bar, parity, 1)) return true;
    for (uint32_t it = 0; it < kTcTries; it += 64) {
      if (abort_s) return false;
      if (tc::mbar_wait(bar, parity, 64)) return true;
    }
    set_status(p.s.status, HATA_ERR_TIMEOUT);
    abort_s = 1;
    return false;
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {  // the same answer in every lane
    const bool r = wait_ok(bar, parity);
    return __all_sync(0xffffffffu, r);
  };
  // The ring holds K and V tiles in the order of `item` numbers.  Pair: K_j, V_j, K_{j+1}, ...  Shared out: the K
  // tiles of both streams, then their V tiles, and so on; an odd last tile has no second stream.
  const bool pair = !TREE || p.pair;
  auto streams_in = [&](int n, int i) { return pair ? 1 : (2 * i + 1 < n ? 2 : 1); };  // tiles of step i (pair: one)
  auto steps_of = [&](int n) { return pair ? n : (n + 1) / 2; };
  // items of a step i of a run of n tiles, counted from the run's first item: K of stream w, V of stream w
  auto item_k = [&](int i, int w) { return pair ? 2 * i : 4 * i + w; };
  auto item_v = [&](int n, int i, int w) { return pair ? 2 * i + 1 : 4 * i + streams_in(n, i) + w; };

  if constexpr (TREE) ptx::pdl_launch_dependents();  // the merge may be set up; it waits for this kernel to end
  Walk<TREE> walk(p, lane, blockIdx.x == 0 && warp == 0);
  Seg sg;

  if (warp >= kTcMmaWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kTcIssueRegs));
  if (warp == kTcTmaWarp) {
    // ---------------- loader: lane l issues box l ----------------
    uint32_t item = 0;  // ring items issued
    uint32_t n_q = 0;   // Q loads issued
    bool ok = true;
    while (ok && walk.next(sg)) {
      if (n_q > 0 && !(ok = wait_warp(&q_free, (n_q - 1) & 1))) break;
      ++n_q;
      if constexpr (TREE) {
        const int rows = pair ? 2 : 1;
        if (lane == 0) tc::mbar_expect(&q_full, (uint32_t)(rows * kTcTileB));
        __syncwarp();
        const int y = (p.s.Hq * sg.b + sg.g * p.s.G) * p.s.T + sg.row0;
        if (lane < 2 * rows)
          tc::tma_load_2d(base + kTcQ + (uint32_t)lane * (kTcTileB / 2), &qmap, 64 * (lane & 1),
                          y + kTcTile * (lane >> 1), &q_full);
      } else {
        if (lane == 0) tc::mbar_expect(&q_full, (uint32_t)(2 * kTcTileB));
        __syncwarp();
        // 256 rows as boxes of q_box rows: consecutive heads, or (P = 1) consecutive positions of one head
        const int boxes = 2 * kTcTile / p.q_box;
        if (lane < 2 * boxes) {
          const int bx = lane >> 1, r = bx * p.q_box;  // row of the 256
          const int head = p.prefill_heads == 1 ? sg.head0 : sg.head0 + bx;
          const int pos = p.prefill_heads == 1 ? sg.row0 + r : sg.row0;
          tc::tma_load_2d(base + kTcQ + (uint32_t)(r / kTcTile) * kTcTileB + (uint32_t)(lane & 1) * (kTcTileB / 2) +
                              (uint32_t)(r % kTcTile) * 128u,
                          &qmap, 64 * (lane & 1), (p.s.Hq * sg.b + head) * p.s.max_seq + pos, &q_full);
        }
      }
      auto load = [&](const CUtensorMap* map, const CUtensorMap* map8, int tile) -> bool {  // the next ring item
        const uint32_t st = item % kStages, round = item / kStages;
        if (round > 0 && !wait_warp(&freed[st], (round - 1) & 1)) return false;
        const uint32_t dst = base + kTcRing + st * kTcTileB;
        const int s0 = tile * kTcTile;
        if constexpr (PAGED) {
          // boxes of the pages that hold slots below L; the rows of the others are masked (K) or zeroed (V)
          const int br = p.box_rows, n_box = min(kTcTile / br, (sg.L - s0 + br - 1) / br);
          if (lane == 0) tc::mbar_expect(&full[st], (uint32_t)(n_box * br * kHeadDim * 2));
          __syncwarp();
          if (lane < 2 * n_box) {
            const int r = (lane >> 1) * br, s = s0 + r;
            int blk = p.s.block_table[(size_t)sg.b * p.s.max_blocks + (s >> p.s.block_shift)];
            if (blk < 0 || blk >= p.s.n_blocks) {
              set_status(p.s.status, HATA_ERR_INVALID_ARG);
              blk = 0;
            }
            const int y = ((blk * p.s.Hkv + sg.g) << p.s.block_shift) + (s & ((1 << p.s.block_shift) - 1));
            tc::tma_load_2d(dst + (uint32_t)(lane & 1) * (kTcTileB / 2) + (uint32_t)r * 128u, map, 64 * (lane & 1), y,
                            &full[st]);
          }
        } else {
          if (lane == 0) tc::mbar_expect(&full[st], (uint32_t)kTcTileB);
          __syncwarp();
          const int kv = (p.s.Hkv * sg.b + sg.g) * p.s.max_seq;
          if (s0 >= sg.sr || s0 + kTcTile <= sg.sr) {
            if (lane < 2)
              tc::tma_load_2d(dst + (uint32_t)lane * (kTcTileB / 2), map, 64 * lane, kv + s0 + (s0 >= sg.sr ? sg.base : 0),
                              &full[st]);
          } else {  // the tile where the sinks end: boxes of 8 rows
            const int r = (lane >> 1) * 8, row = s0 + r;
            tc::tma_load_2d(dst + (uint32_t)(lane & 1) * (kTcTileB / 2) + (uint32_t)r * 128u, map8, 64 * (lane & 1),
                            kv + row + (row >= sg.sr ? sg.base : 0), &full[st]);
          }
        }
        ++item;
        return true;
      };
      const int n = sg.j1 - sg.j0, steps = steps_of(n);
      for (int i = 0; ok && i < steps; ++i) {
        const int m = streams_in(n, i);
        for (int w = 0; ok && w < m; ++w) ok = load(&kmap, &kmap8, sg.j0 + (pair ? i : 2 * i + w));
        for (int w = 0; ok && w < m; ++w) ok = load(&vmap, &vmap8, sg.j0 + (pair ? i : 2 * i + w));
      }
    }
    // every copy still in flight lands before the CTA leaves
    for (uint32_t it = item > kStages ? item - kStages : 0; it < item; ++it)
      tc::mbar_wait(&full[it % kStages], (it / kStages) & 1, kTcTries);
    if (n_q > 0) tc::mbar_wait(&q_full, (n_q - 1) & 1, kTcTries);
  } else if (warp == kTcMmaWarp) {
    // ---------------- MMA issue: every lane runs this, one elected lane issues ----------------
    bool ok = true;
    if (p.test_expire && !tc::mbar_wait(&never, 0, kTcTestTries)) {  // test hook: this wait runs out
      if (lane == 0) set_status(p.s.status, HATA_ERR_TIMEOUT);
      abort_s = 1;
      ok = false;
    }
    constexpr uint32_t idS = tc::idesc_bf16(kTcTile, kTcTile, false);
    constexpr uint32_t idPV = tc::idesc_bf16(kTcTile, kHeadDim, true);
    uint32_t item0 = 0;         // first ring item of the run
    uint32_t done0 = 0, done1 = 0;  // tiles whose P the streams have delivered
    for (int n_seg = 0; ok && walk.next(sg); ++n_seg) {
      const int n = __shfl_sync(0xffffffffu, sg.j1 - sg.j0, 0), steps = steps_of(n);
      ok = wait_warp(&q_full, (uint32_t)(n_seg & 1));
      auto slot_of = [&](int k) { return (item0 + (uint32_t)k) % kStages; };
      auto wait_item = [&](int k) {
        const uint32_t it = item0 + (uint32_t)k;
        return wait_warp(&full[it % kStages], (it / kStages) & 1);
      };
      const uint64_t q_desc[2] = {tc::desc_kmajor_sw128(base + kTcQ),
                                  tc::desc_kmajor_sw128(base + kTcQ + (pair ? (uint32_t)kTcTileB : 0u))};
      auto k_desc = [&](uint32_t slot) { return tc::desc_kmajor_sw128(base + kTcRing + slot * kTcTileB); };
      const int s0n = pair ? 2 : streams_in(n, 0);  // streams of the first step
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!ok || w >= s0n) break;
        if ((!pair || w == 0) && !(ok = wait_item(item_k(0, w)))) break;
        const uint32_t ks = slot_of(item_k(0, w));
        tc::fence_after();
        mma8_s(tmem + (uint32_t)w * kTcTile, q_desc[w], k_desc(ks), idS);
        commit_elected(&s_full[w]);
        if (!pair || w == 1) commit_elected(&freed[ks]);
      }
      if (ok && steps == 1) commit_elected(&q_free);
#pragma unroll 1
      for (int i = 0; ok && i < steps; ++i) {
        const int m = pair ? 2 : streams_in(n, i);
        const int m_next = i + 1 < steps ? (pair ? 2 : streams_in(n, i + 1)) : 0;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!ok || w >= m) break;
          // the tiles first: when P comes, its PV and the next S go out at once
          if ((!pair || w == 0) && !(ok = wait_item(item_v(n, i, w)))) break;
          if ((!pair || w == 0) && w < m_next && !(ok = wait_item(item_k(i + 1, w)))) break;
          const uint32_t vs = slot_of(item_v(n, i, w)), ks = slot_of(item_k(i + 1, w));
          const uint64_t vd = tc::desc_mnmajor_sw128(base + kTcRing + vs * kTcTileB, (uint32_t)(kTcTileB / 2));
          const uint64_t kd = k_desc(ks);
          uint32_t& done = w ? done1 : done0;
          const uint32_t o = tmem + 256u + (uint32_t)w * kHeadDim, sp = tmem + (uint32_t)(w * kTcTile);
          if (!(ok = wait_warp(&p_half[w], done & 1))) break;
          tc::fence_after();
          mma4_pv(o, sp, vd, idPV, i > 0 ? 1u : 0u);
          if (!(ok = wait_warp(&p_full[w], done & 1))) break;
          ++done;
          tc::fence_after();
          mma4_pv(o, sp + 32u, vd + 512u, idPV, 1u);
          if (w < m_next) {
            mma8_s(sp, q_desc[w], kd, idS);
            commit_elected(&s_full[w]);
            if (!pair || w == 1) commit_elected(&freed[ks]);
            if (i + 2 == steps && w == m_next - 1) commit_elected(&q_free);
          } else {
            commit_elected(&o_full[w]);  // the stream's last PV
          }
          if (!pair || w == 1) commit_elected(&freed[vs]);
        }
      }
      item0 += (uint32_t)(2 * n);
    }
    commit_elected(&drain);  // every MMA issued above completes before the CTA leaves
    tc::mbar_wait(&drain, 0, kTcTries);
    __syncwarp();
  }
  } else {
    // ---------------- a stream's warpgroup: row m of its 128 ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kTcRowRegs));
    const int w = warp >> 2, m = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t sa = lane_base + (uint32_t)(w * kTcTile), oa = lane_base + 256u + (uint32_t)(w * kHeadDim);
    const float c = p.s.scale_log2;
    uint32_t item0 = 0, tiles = 0, outs = 0;  // ring items, score tiles and outputs so far
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int n = sg.j1 - sg.j0, steps = steps_of(n);
      const int mine = pair ? steps : (n + 1 - w) / 2;  // steps of this stream
      // what this row sees
      int t = 0, row = 0, t_lo = 0, t_hi = 0;
      bool live;
      Bits128 seen{0u, 0u, 0u, 0u}, any{0u, 0u, 0u, 0u};
      const bool has_new = TREE && sg.j1 * kTcTile > sg.ctx;  // the run reaches the new tokens
      if constexpr (TREE) {
        row = sg.row0 + (pair ? w * kTcTile : 0) + m;
        const int i = row % p.s.T;
        live = row < p.s.R && i < sg.n_b;
        if (has_new) {
          if (p.s.mask) {
            const uint32_t* mw = p.s.mask + ((size_t)sg.b * p.s.T + i) * p.s.mask_words;
            seen.w0 = mw[0];
            if (p.s.mask_words > 1) seen.w1 = mw[1];
            if (p.s.mask_words > 2) seen.w2 = mw[2];
            if (p.s.mask_words > 3) seen.w3 = mw[3];
          } else {
            seen.w0 = span::low_bits(i + 1);
            seen.w1 = span::low_bits(i - 31);
            seen.w2 = span::low_bits(i - 63);
            seen.w3 = span::low_bits(i - 95);
          }
          seen.w0 &= span::low_bits(sg.n_b);
          seen.w1 &= span::low_bits(sg.n_b - 32);
          seen.w2 &= span::low_bits(sg.n_b - 64);
          seen.w3 &= span::low_bits(sg.n_b - 96);
          // the new tokens that any token sees
          any = {0u, 0u, 0u, 0u};
          for (int j = lane; p.s.mask && j < sg.n_b; j += 32) {
            const uint32_t* mw = p.s.mask + ((size_t)sg.b * p.s.T + j) * p.s.mask_words;
            any.w0 |= mw[0];
            if (p.s.mask_words > 1) any.w1 |= mw[1];
            if (p.s.mask_words > 2) any.w2 |= mw[2];
            if (p.s.mask_words > 3) any.w3 |= mw[3];
          }
          any.w0 = __reduce_or_sync(0xffffffffu, p.s.mask ? any.w0 : 0xffffffffu) & span::low_bits(sg.n_b);
          any.w1 = __reduce_or_sync(0xffffffffu, p.s.mask ? any.w1 : 0xffffffffu) & span::low_bits(sg.n_b - 32);
          any.w2 = __reduce_or_sync(0xffffffffu, p.s.mask ? any.w2 : 0xffffffffu) & span::low_bits(sg.n_b - 64);
          any.w3 = __reduce_or_sync(0xffffffffu, p.s.mask ? any.w3 : 0xffffffffu) & span::low_bits(sg.n_b - 96);
        }
      } else {
        t = p.prefill_heads == 1 ? sg.row0 + w * kTcTile + m : sg.row0 + (m & (p.q_box - 1));
        live = t < sg.L;
        // the stream's positions, for the test whether a tile lies at an edge of what they see
        t_lo = p.prefill_heads == 1 ? sg.row0 + w * kTcTile : sg.row0;
        t_hi = t_lo + min(p.pos_block, kTcTile) - 1;
      }
      float m_used = -INFINITY, l = 0.f;
      for (int i = 0; i < mine; ++i) {
        // first key row of the tile, and the slot of that row but for the sinks'
        const int r0 = (sg.j0 + (pair ? i : 2 * i + w)) * kTcTile, s0 = r0 + sg.base;
        if (!(ok = wait_warp(&s_full[w], tiles & 1))) break;
        ++tiles;
        tc::fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::ld32_nowait(sa + 32 * k, x[k]);
        tc::ld_wait();
        // Tiles at an edge of what the rows see: visibility words of this row, 32 slots each.  Chunks that every row of
        // the warp sees need no masking, and those that none sees (bit k of `none`) no exponentials.
        const uint32_t ninf = 0xff800000u;
        unsigned none = 0;
        bool edge;
        if constexpr (TREE) {
          edge = s0 + kTcTile > sg.ctx;
        } else {
          edge = r0 < sg.sr ? r0 + kTcTile > p.s.sink
                            : s0 + kTcTile > t_lo + 1 || (s0 <= t_hi - p.s.window && s0 + kTcTile > p.s.sink);
        }
        if (edge) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v;
            if constexpr (TREE) {
              v = seen.at(s0 + 32 * k - sg.ctx);
            } else {
              const int e0 = s0 + 32 * k;
              v = span::low_bits(t + 1 - e0) &
                  (~span::low_bits(t - min(p.s.window, t + 1) + 1 - e0) | span::low_bits(min(p.s.sink, sg.L) - e0));
              const int r = r0 + 32 * k;
              if (r < sg.sr) v = (v & ~span::low_bits(sg.sr - r)) | span::low_bits(min(p.s.sink, sg.sr) - r);
            }
            if (!__any_sync(0xffffffffu, v != 0u)) none |= 1u << k;
            if (__any_sync(0xffffffffu, v != 0xffffffffu)) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[k][e] = (v >> e) & 1u ? x[k][e] : ninf;
            }
          }
        }
        float mx;
        {
          float m8[8];
#pragma unroll
          for (int h = 0; h < 8; ++h) m8[h] = fmax3(__uint_as_float(x[0][h]), __uint_as_float(x[0][h + 8]), __uint_as_float(x[0][h + 16]));
#pragma unroll
          for (int e = 24; e < 120; e += 16)
#pragma unroll
            for (int h = 0; h < 8; ++h)
              m8[h] = fmax3(m8[h], __uint_as_float(x[(e + h) >> 5][(e + h) & 31]), __uint_as_float(x[(e + 8 + h) >> 5][(e + 8 + h) & 31]));
#pragma unroll
          for (int h = 0; h < 8; ++h) m8[h] = fmaxf(m8[h], __uint_as_float(x[3][24 + h]));
          mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
        }
        const float m_tile = mx * c;
        if (i == 0) {
          m_used = m_tile;
        } else if (__any_sync(0xffffffffu, m_tile > m_used + kTcSlack)) {
          const float m_new = fmaxf(m_used, m_tile);
          const float alpha = m_new == -INFINITY ? 1.f : ex2(m_used - m_new);
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tc::ld32(oa + 32 * k, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st32(oa + 32 * k, o);
          }
          l *= alpha;
          m_used = m_new;
        }
        // value rows that nobody sees (possibly not finite) are zeroed, so that 0 * V stays 0; in a pair the
        // first stream does it for both, since its PV is issued first
        if ((!pair || w == 0) && s0 + kTcTile > sg.ctx) {
          const uint32_t it = item0 + (uint32_t)item_v(n, i, w);
          if (!(ok = wait_warp(&full[it % kStages], (it / kStages) & 1))) break;
          bool drop = s0 + m >= sg.L;
          if constexpr (TREE) {
            const int j = s0 + m - sg.ctx;
            if (!drop && j >= 0) drop = !(any.at(j) & 1u);
          }
          if (drop) {
            unsigned char* vrow = tc_smem + (base - tc::smem_u32(tc_smem)) + kTcRing + (it % kStages) * kTcTileB +
                                  (m >> 3) * 1024 + (m & 7) * 128;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              *reinterpret_cast<uint4*>(vrow + q * 16) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(vrow + kTcTileB / 2 + q * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          tc::fence_async_smem();
        }
        // p = 2^(x c - m) and its sum, two at a time; each half of P is handed over as soon as it is stored, so that
        // its PV runs while the other half is computed
        const float mr = m_used == -INFINITY ? 0.f : m_used;  // nothing seen yet: p = 2^-inf = 0
        const uint64_t c2 = pack2(c, c), mr2 = pack2(-mr, -mr);
        uint64_t sum2[2] = {0ull, 0ull};
        auto chunk = [&](int k, uint32_t (&pk)[16]) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, d;
            unpack2(fma2(pack2(__uint_as_float(x[k][2 * e]), __uint_as_float(x[k][2 * e + 1])), c2, mr2), a, d);
            a = ex2(a);
            d = ex2(d);
            sum2[e & 1] = add2(sum2[e & 1], pack2(a, d));
            pk[e] = bf16x2(a, d);
          }
        };
        if (none == 0) {
          uint32_t pk[4][16];
          chunk(0, pk[0]);
          st16(sa, pk[0]);
          chunk(1, pk[1]);
          st16(sa + 16, pk[1]);
          chunk(2, pk[2]);
          tc::st_wait();  // the stores of chunks 0 and 1 are done by now
          tc::fence_before();
          tc::mbar_arrive(&p_half[w]);
          st16(sa + 32, pk[2]);
          chunk(3, pk[3]);
          st16(sa + 48, pk[3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t pk[16];
            if ((none >> k) & 1u) {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            } else {
              chunk(k, pk);
            }
            st16(sa + 16 * k, pk);
            if (k == 1) {
              tc::st_wait();
              tc::fence_before();
              tc::mbar_arrive(&p_half[w]);
            }
          }
        }
        {
          float a, d, e, f;
          unpack2(sum2[0], a, d);
          unpack2(sum2[1], e, f);
          l += (a + d) + (e + f);
        }
        tc::st_wait();
        tc::fence_before();
        tc::mbar_arrive(&p_full[w]);
      }
      item0 += (uint32_t)(2 * n);
      if (!ok) break;
      if (mine > 0) {
        if (!(ok = wait_warp(&o_full[w], outs & 1))) break;
        ++outs;
        tc::fence_after();
      }
      if constexpr (TREE) {
        float* part = p.s.part + ((size_t)sg.slot * 2 + w) * kPartFloats;
        part[m] = m_used;
        part[kTcTile + m] = l;
        if (mine > 0) {
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t o[32];
            tc::ld32(oa + 32 * k, o);
            float4* dst = reinterpret_cast<float4*>(part + 2 * kTcTile) + (size_t)(8 * k) * kTcTile + m;
            if (live)
#pragma unroll
              for (int q = 0; q < 8; ++q)
                dst[q * kTcTile] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                               __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
          }
        }
      } else {
        // Rows through shared memory, 64 columns at a time: a warp's 32 rows of 128 bytes (piece q of row r at q ^ (r
        // & 7)), then eight lanes per row, so a store covers four rows of 128 bytes instead of 32 of 16.
        const float inv = l == 0.f ? 0.f : 1.f / l;
        unsigned char* stage = tc_smem + (base - tc::smem_u32(tc_smem)) + kTcOut + (uint32_t)warp * 4096u;
        // 16 rows that begin at a multiple of 16 are one head's: this lane's row and piece of the first and second 16
        int pos[2];
        __nv_bfloat16* out[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int mr = (warp & 3) * 32 + 16 * k + (lane >> 3);
          const int head = sg.head0 + (p.prefill_heads == 1 ? 0 : w * (p.prefill_heads >> 1) + (mr >> p.pos_shift));
          pos[k] = t_lo + (mr & (p.q_box - 1));
          out[k] = static_cast<__nv_bfloat16*>(p.s.out) +
                   ((size_t)(sg.b * p.s.Hq + head) * p.s.max_seq + pos[k]) * kHeadDim + 8 * (lane & 7);
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          __syncwarp();  // the other half's rows have been read
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t o[32];
            tc::ld32(oa + 64 * half + 32 * k, o);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = bf16x2(__uint_as_float(o[8 * q + 2 * e]) * inv, __uint_as_float(o[8 * q + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * k + q) ^ (lane & 7)) << 4)) =
                  make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = 4 * e + (lane >> 3), q = lane & 7;  // row of the warp, piece
            const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((q ^ (r & 7)) << 4));
            if (pos[e >> 2] + 4 * (e & 3) < sg.L)
              *reinterpret_cast<uint4*>(out[e >> 2] + 4 * (e & 3) * kHeadDim + 64 * half) = v;
          }
        }
      }
      tc::fence_before();  // O has been read: the next run's first P allows its overwriting
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, kTcTmemCols);
  }
}

// Joins the partials of a unit in the order of the split: thread (row, 4 columns).  The partials were just written by
// other SMs: six of them are under way at a time (one after another, 36 partials of a unit took 25 us).
// grid = (units, 32, row tiles of a unit).
constexpr int kMergeBatch = 6;
constexpr int kMergeRegs = 56;  // 128 threads of these fit beside the main kernel's CTA
__global__ void __maxnreg__(kMergeRegs) span_merge_kernel(const TcParams p, int grid_tc, int rows_per_unit) {
  const int lane = threadIdx.x & 31;
  const int upt = p.s.Hkv * p.s.row_tiles, unit = (int)blockIdx.x, b = unit / upt, in_seq = unit % upt;
  // the lengths are the call's inputs: where the partials lie is found while the main kernel still runs
  const span::Seq sq = span::seq_of(p.s, b);
  const span::Runs runs = sq.tiles > 0 ? span::runs_of(p.s, lane, grid_tc, b, in_seq, sq) : span::Runs{};
  const int g = in_seq % p.s.Hkv, half = blockIdx.z;  // half: of a pair, the row tile
  const int m = threadIdx.x, q4 = (int)blockIdx.y;
  const int row = in_seq / p.s.Hkv * rows_per_unit + half * kTcTile + m;
  // a row's partials: one per run and, if its key tiles were shared out over both streams, stream
  const int n_str = p.pair ? 1 : 2, n = runs.n * n_str;
  const float* first = p.s.part + ((size_t)(unit + runs.cta0) * 2 + (p.pair ? half : 0)) * kPartFloats + m;
  const size_t step = (size_t)kPartFloats * (p.pair ? 2 : 1);
  ptx::pdl_wait();  // also where there is nothing to join: what comes next on the stream waits for this grid alone
  if (sq.tiles == 0 || row >= p.s.R || row % p.s.T >= sq.n_b) return;
  float M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += kMergeBatch) {
    float mi[kMergeBatch], li[kMergeBatch];
    float4 v[kMergeBatch];
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) {
      const float* pp = first + (size_t)(i0 + k) * step;
      const bool in = i0 + k < n;
      mi[k] = in ? __ldcg(pp) : -INFINITY;
      li[k] = in ? __ldcg(pp + kTcTile) : 0.f;
      v[k] = in ? __ldcg(reinterpret_cast<const float4*>(pp + 2 * kTcTile - m) + (size_t)q4 * kTcTile + m)
                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m_new = M;
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) m_new = fmaxf(m_new, mi[k]);
    const float back = m_new == -INFINITY ? 1.f : exp2f(M - m_new);
    M = m_new;
    l *= back;
    o.x *= back;
    o.y *= back;
    o.z *= back;
    o.w *= back;
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k) {
      if (mi[k] == -INFINITY) continue;  // nothing seen in this run (or the stream had no tile: O was not written)
      const float f = exp2f(mi[k] - M);
      l = fmaf(li[k], f, l);
      o.x = fmaf(v[k].x, f, o.x);
      o.y = fmaf(v[k].y, f, o.y);
      o.z = fmaf(v[k].z, f, o.z);
      o.w = fmaf(v[k].w, f, o.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.s.out) +
                       (((size_t)b * p.s.Hq + (size_t)g * p.s.G) * p.s.T + row) * kHeadDim + 4 * q4;
  *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
}

template <bool TREE, bool PAGED>
cudaError_t configure_tc() {
  static std::mutex mu;
  static std::map<int, cudaError_t> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  auto it = done.find(dev);
  if (it != done.end()) return it->second;
  e = cudaFuncSetAttribute(span_tc_kernel<TREE, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
  if (e != cudaSuccess) (void)cudaGetLastError();
  done[dev] = e;
  return e;
}

}  // namespace

size_t span_tc_part_bytes(const hata_dims_t& d, int n_tok) {
  const long long R = (long long)(d.n_q_heads / d.n_kv_heads) * n_tok;
  const long long rows = R > kTcTile ? 2 * kTcTile : kTcTile;
  const size_t units = (size_t)d.batch * d.n_kv_heads * (size_t)((R + rows - 1) / rows);
  return (units + (size_t)span_sms()) * 2 * kPartFloats * 4;
}

cudaError_t launch_span_tc(const hata_dims_t& d, const span::Params& s, const PagedCache* pg, cudaStream_t st) {
  const int sms = span_sms();
  TcParams p{};
  p.s = s;
  p.pair = s.R > kTcTile ? 1 : 0;
  const int rows = p.pair ? 2 * kTcTile : kTcTile;
  p.s.row_tiles = (s.R + rows - 1) / rows;
  p.test_expire = (d.flags & HATA_FLAG_TEST_EXPIRE_WAIT) ? 1 : 0;
  CUtensorMap qm, km, vm;
  p.box_rows = pg ? std::min(1 << pg->block_shift, kTcTile) : kTcTile;
  const long long kv_rows =
      pg ? ((long long)pg->n_blocks * d.n_kv_heads) << pg->block_shift : (long long)d.batch * d.n_kv_heads * d.max_seq;
  const long long q_rows = (long long)d.batch * d.n_q_heads * s.T;
  const long long units = (long long)d.batch * d.n_kv_heads * p.s.row_tiles;
  if (!span_fits(p.s, units)) return cudaErrorNotSupported;
  if (kv_rows + kTcTile > 0x7fffffffLL || q_rows + 2 * kTcTile > 0x7fffffffLL) return cudaErrorNotSupported;
  if (!make_bf16_rows_map(&qm, s.q, q_rows, kTcTile) || !make_bf16_rows_map(&km, s.K, kv_rows, p.box_rows) ||
      !make_bf16_rows_map(&vm, s.V, kv_rows, p.box_rows))
    return cudaErrorNotSupported;
  cudaError_t e = pg ? configure_tc<true, true>() : configure_tc<true, false>();
  if (e != cudaSuccess) return e;
  e = launch_early(pg ? span_tc_kernel<true, true> : span_tc_kernel<true, false>, dim3((unsigned)sms), kTcThreads, kTcSmem, st,
                   qm, km, vm, km, vm, p);
  if (e != cudaSuccess) return e;
  return launch_early(span_merge_kernel, dim3((unsigned)units, kHeadDim / 4, p.pair ? 2 : 1), kTcTile, 0, st, p, sms, rows);
}

cudaError_t launch_window_prefill(const hata_dims_t& d, const void* q, const void* K, const void* V,
                                  const int32_t* seq_lens, int window, int sink, float scale, void* out,
                                  uint32_t* status, cudaStream_t st) {
  TcParams p{};
  p.s.q = q;
  p.s.K = K;
  p.s.V = V;
  p.s.out = out;
  p.s.status = status;
  p.s.seq_lens = seq_lens;
  p.s.B = d.batch;
  p.s.Hq = d.n_q_heads;
  p.s.Hkv = d.n_kv_heads;
  p.s.G = d.n_q_heads / d.n_kv_heads;
  p.s.max_seq = d.max_seq;
  p.s.window = window;
  p.s.sink = sink;
  p.s.scale_log2 = scale * 1.4426950408889634f;
  p.test_expire = (d.flags & HATA_FLAG_TEST_EXPIRE_WAIT) ? 1 : 0;
  p.prefill_heads = p.s.G & -p.s.G;  // a power of two, at most 16 (G <= 16)
  p.pos_block = 2 * kTcTile / p.prefill_heads;
  p.q_box = std::min(p.pos_block, kTcTile);
  while ((1 << p.pos_shift) < p.q_box) ++p.pos_shift;
  p.n_blocks_pos = (d.max_seq + p.pos_block - 1) / p.pos_block;
  p.rows_of_items = d.batch * (d.n_q_heads / p.prefill_heads);
  p.box_rows = kTcTile;
  const long long q_rows = (long long)d.batch * d.n_q_heads * d.max_seq, kv_rows = (long long)d.batch * d.n_kv_heads * d.max_seq;
  if (q_rows + 2 * kTcTile > 0x7fffffffLL) return cudaErrorNotSupported;
  CUtensorMap qm, km, vm, km8, vm8;
  if (!make_bf16_rows_map(&qm, q, q_rows, p.q_box) || !make_bf16_rows_map(&km, K, kv_rows, kTcTile) ||
      !make_bf16_rows_map(&vm, V, kv_rows, kTcTile) || !make_bf16_rows_map(&km8, K, kv_rows, 8) ||
      !make_bf16_rows_map(&vm8, V, kv_rows, 8))
    return cudaErrorNotSupported;
  cudaError_t e = configure_tc<false, false>();
  if (e != cudaSuccess) return e;
  const long long items = (long long)p.n_blocks_pos * p.rows_of_items;
  if (items > 0x3fffffffLL) return cudaErrorNotSupported;
  const unsigned grid = (unsigned)std::min<long long>(items, span_sms());
  return launch_early(span_tc_kernel<false, false>, dim3(grid), kTcThreads, kTcSmem, st, qm, km, vm, km8, vm8, p);
}

}  // namespace hata
