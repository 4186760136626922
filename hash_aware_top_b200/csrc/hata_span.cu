// Window decode and tree attention: softmax(scale * q . K) V of the new tokens' rows over the visible slots
// of a contiguous or paged cache (hata_span.cuh has the split of the work).
//
// span_mma_kernel (bf16, tiles of up to 32 rows per KV head): eight warps, each with 16 slots of a 128-slot tile, on its own: it
// streams its rows of K and V through three shared-memory stages (cp.async, 16-byte pieces swizzled so that the eight
// rows of a fragment lie in distinct banks), computes S on m16n8k16 tiles with the query rows as M, turns S
// into P in place (the accumulator of S has the layout of the A operand of P.V), and adds P.V to its own running
// output.  No barrier inside a run of tiles.  The warps meet once per unit.  Bound by memory: at 6.5 TB/s an SM
// receives a warp's 8 KB step every 364 cycles, and 128 KB are in flight.  Measured on B200: 16 ragged sequences of
// 8207 visible slots, 32 / 8 heads, paged, 87-91 us (0.91-0.94 of a copy's bandwidth); 8 x 64K slots 329 us (1.00); 28 rows over
// 29K slots 30-33 us (0.55-0.59: 3 us of launches, 2 us to find the run, 2 us to meet and 2 us to join are fixed costs); 4 rows
// over 4.1K slots 9.2-9.4 us; 64 sequences of 4.1K 169 us (0.97).
//
// span_simt_kernel (fp32): eight warps, each with 16 slots of a 128-slot tile, on its own: it copies
// its rows of K and V to shared memory (cp.async), a lane takes one slot and half of the 128 dimensions for the
// logits and four dimensions of every row for P.V, and keeps its own running maximum, sum and output
// (fp32, online softmax).  The warps meet once per unit.  Bound by the fp32 units and shared memory when a unit
// has many rows (each shared-memory vector feeds 4 multiply-adds per row), else by memory.  Measured on B200: 16 sequences of 8195
// visible slots, 32 / 8 heads, 170 us (0.97 of a copy's bandwidth); 13 rows over 3.5K slots, 4 heads, 15.5 us; 256 rows
// over 8K slots, 8 KV heads, 377 us (0.31 of the fp32 rate).
#include <algorithm>
#include <map>
#include <mutex>

#include "hata_ptx.cuh"
#include "hata_span.cuh"

namespace hata {

namespace {

using namespace span;

constexpr int kSpThreads = 256;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kSpKeys = 16;  // slots of a warp in a tile
// Registers of a thread: 256 x 224 of the SM's 65536 leave room for a CTA of the joining kernel (128 x 64), which is
// then there, its prologue done, when the main kernel ends (measured at 240 registers, where it is not: 5 us later).
constexpr int kSpRegs = 224;
constexpr float kSpSlack = 8.f;  // log2 units
static_assert(kSpWarps * kSpKeys == kSpanTile, "the warps share a tile");

// 16-byte copy, or 16 zero bytes where !valid
__device__ __forceinline__ void cp_async16_zfill(uint32_t smem, const void* gmem, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async16_at(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// First cache row of 16 consecutive slots from s0 (a multiple of 16, below L): in one page, since pages
// hold a multiple of 16 slots.
template <bool PAGED>
__device__ __forceinline__ size_t rows_of16(const Params& p, int b, int g, int s0) {
  if constexpr (PAGED) {
    int blk = p.block_table[(size_t)b * p.max_blocks + (s0 >> p.block_shift)];
    if (blk < 0 || blk >= p.n_blocks) {
      set_status(p.status, HATA_ERR_INVALID_ARG);
      blk = 0;
    }
    return (((size_t)blk * p.Hkv + g) << p.block_shift) + (size_t)(s0 & ((1 << p.block_shift) - 1));
  } else {
    return ((size_t)b * p.Hkv + g) * p.max_seq + s0;
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* out, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float* out, float4 v) { *reinterpret_cast<float4*>(out) = v; }
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* out, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), c = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(out) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
}

// The weights that bring the warps' outputs of each row to one maximum: sm_m, sm_l [n][ROWS] (maximum, sum) become
// sm_m = 2^(m - M) and, for row r < rows, (M, sum of l 2^(m - M)) in row_m, row_l.  A warp per row; all threads.
template <int ROWS>
__device__ __forceinline__ void join_weights(float* sm_m, const float* sm_l, int n, int rows, float* row_m, float* row_l) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = warp; r < rows; r += kSpWarps) {
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, sm_m[i * ROWS + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float m = sm_m[i * ROWS + r];
      const float f = m == -INFINITY ? 0.f : exp2f(m - M);
      sm_m[i * ROWS + r] = f;
      l = fmaf(sm_l[i * ROWS + r], f, l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      row_m[r] = M;
      row_l[r] = l;
    }
  }
  __syncthreads();
}

constexpr int kOutRow = kHeadDim + 8;  // floats of a row of a warp's output in shared memory: rows on distinct banks

// A partial: m [ROWS], l [ROWS], O [ROWS][128].
template <int ROWS>
__device__ __forceinline__ float* part_of(const Params& p, int slot) {
  return p.part + (size_t)slot * ROWS * (kHeadDim + 2);
}

// The end of a unit's run in this CTA.  In shared memory: m, l [kSpWarps][ROWS] and o [kSpWarps][ROWS][kOutRow]
// of the warps.  Joins them, then writes the rows of a unit that is all this CTA's, or leaves a partial.
template <typename T, int ROWS>
__device__ __forceinline__ void finish_unit(const Params& p, float* sm_m, float* sm_l, const float* sm_o,
                                            const Piece& pc, int g, int rt) {
  __shared__ float row_m[ROWS], row_l[ROWS];
  const int tid = threadIdx.x, r0 = rt * ROWS, rows = min(ROWS, p.R - r0);
  T* out = static_cast<T*>(p.out) + (((size_t)pc.b * p.Hq + (size_t)g * p.G) * p.T + r0) * kHeadDim;
  float* part = part_of<ROWS>(p, pc.slot);
  join_weights<ROWS>(sm_m, sm_l, kSpWarps, rows, row_m, row_l);
  for (int e = tid; e < rows * (kHeadDim / 4); e += kSpThreads) {
    const int r = e / (kHeadDim / 4), c = e % (kHeadDim / 4);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kSpWarps; ++w) {
      const float f = sm_m[w * ROWS + r];
      const float4 v = *reinterpret_cast<const float4*>(sm_o + (w * ROWS + r) * kOutRow + 4 * c);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    if (pc.whole) {
      const float l = row_l[r], inv = l == 0.f ? 0.f : 1.f / l;
      if ((r0 + r) % p.T < pc.seq.n_b)
        store4<T>(out + 4 * e, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    } else {
      reinterpret_cast<float4*>(part + 2 * ROWS)[e] = o;
    }
  }
  if (!pc.whole && tid < rows) {
    part[tid] = row_m[tid];
    part[ROWS + tid] = row_l[tid];
  }
}

// Joins the partials of a unit in the order of the split: a warp per row, a lane per 4 columns.  The partials were
// just written by other SMs, so a round trip to them costs over a microsecond: eight rows of O are under way
// before the weights are known.  grid = (units + 1, ROWS / 4): what comes next on the stream waits for this grid alone, so
// it must not end before the main one does, and where no unit has anything to join the CTAs past the last unit are what waits.
// (With every CTA waiting, 256 sequences x 8 heads of 100 slots take 56 us instead of 51; with the first one waiting
// on its ways out, a split window of 4096 slots 9.7 instead of 9.2.)
constexpr int kJoinWarps = 4;
constexpr int kJoinBatch = 8;
template <typename T, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32, 8) span_join_kernel(const Params p, int grid_main) {
  const int lane = threadIdx.x & 31, r = (int)blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const int upt = p.Hkv * p.row_tiles, b = (int)blockIdx.x / upt, in_seq = (int)blockIdx.x % upt;
  if (b >= p.B) {
    ptx::pdl_wait();
    return;
  }
  const int g = in_seq % p.Hkv, row = in_seq / p.Hkv * ROWS + r;
  // the lengths are the call's inputs: where the partials lie is found while the main kernel still runs
  const Seq sq = seq_of(p, b);
  if (sq.tiles == 0 || row >= p.R || row % p.T >= sq.n_b) return;
  const Runs runs = runs_of(p, lane, grid_main, b, in_seq, sq);
  const int n = runs.n;
  if (n == 1) return;  // written by the one CTA that had it
  ptx::pdl_wait();
  float4 v[kJoinBatch];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k)
      v[k] = i0 + k < n ? __ldcg(reinterpret_cast<const float4*>(part_of<ROWS>(p, runs.slot(i0 + k)) + 2 * ROWS) +
                                 r * (kHeadDim / 4) + lane)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  fetch(0);
  for (int i0 = 0; i0 < n; i0 += 32) {  // 32 runs: a lane per run for the weights, then a lane per column for O
    float m = -INFINITY, li = 0.f;
    if (i0 + lane < n) {
      const float* pp = part_of<ROWS>(p, runs.slot(i0 + lane));
      m = __ldcg(pp + r);
      li = __ldcg(pp + ROWS + r);
    }
    float mx = m;
#pragma unroll
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float m_new = fmaxf(M, mx);
    const float back = m_new == -INFINITY ? 1.f : exp2f(M - m_new);
    const float f = m == -INFINITY ? 0.f : exp2f(m - m_new);
    float ls = li * f;
#pragma unroll
    for (int k = 16; k; k >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, k);
    l = fmaf(l, back, ls);
    o.x *= back;
    o.y *= back;
    o.z *= back;
    o.w *= back;
    M = m_new;
    for (int k0 = 0; k0 < 32 && i0 + k0 < n; k0 += kJoinBatch) {
      if (i0 + k0 > 0) fetch(i0 + k0);
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k0 + k);  // 0 past the last run
        o.x = fmaf(v[k].x, fk, o.x);
        o.y = fmaf(v[k].y, fk, o.y);
        o.z = fmaf(v[k].z, fk, o.z);
        o.w = fmaf(v[k].w, fk, o.w);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(p.out) + (((size_t)b * p.Hq + (size_t)g * p.G) * p.T + row) * kHeadDim + 4 * lane;
  store4<T>(out, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

__device__ __forceinline__ float4 load4(const unsigned char* row, int d) {
  return *reinterpret_cast<const float4*>(row + 4 * d);
}

template <int ROWS>
struct SimtSmem {
  static constexpr int kRowB = kHeadDim * 4 + 16;  // padded: 16 rows on distinct banks
  static constexpr int kWarpB = 2 * kSpKeys * kRowB;            // K then V of a warp's slots
  static constexpr int kStage = kSpWarps * kWarpB;              // later o [warps][ROWS][kOutRow] fp32
  static_assert(ROWS * kOutRow * 4 <= kWarpB, "the warps' outputs lie over their staged rows");
  static constexpr int kQ = kStage;                               // [ROWS][128] fp32
  static constexpr int kP = kQ + ROWS * kHeadDim * 4;             // [warps][ROWS][16] fp32
  static constexpr int kML = kP + kSpWarps * ROWS * kSpKeys * 4;  // m, l [warps][ROWS]
  static constexpr int kBytes = kML + 2 * kSpWarps * ROWS * 4;
};

template <int ROWS, bool PAGED>
__global__ void __maxnreg__(kSpRegs) span_simt_kernel(const Params p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = SimtSmem<ROWS>;
  using T = float;
  float* sm_q = reinterpret_cast<float*>(smem + S::kQ);
  float* sm_m = reinterpret_cast<float*>(smem + S::kML);
  float* sm_l = sm_m + kSpWarps * ROWS;
  float* sm_o = reinterpret_cast<float*>(smem);  // after a unit's run: over the staged rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* kt = smem + warp * S::kWarpB;
  unsigned char* vt = kt + kSpKeys * S::kRowB;
  float* sm_p = reinterpret_cast<float*>(smem + S::kP) + warp * ROWS * kSpKeys;

  ptx::pdl_wait();
  ptx::pdl_launch_dependents();  // the joining kernel may be set up; it waits for this one to end
  Walker walk;
  walk.begin(p, lane, blockIdx.x == 0 && warp == 0);
  const int key = lane & 15, half = lane >> 4;
  Piece pc;
  while (walk.next(p, pc)) {
    const int rt = p.row_tiles == 1 ? 0 : pc.in_seq / p.Hkv, b = pc.b, g = pc.in_seq - rt * p.Hkv, j0 = pc.j0, j1 = pc.j1;
    const Seq& sq = pc.seq;
    const int r0 = rt * ROWS;
    auto first_slot = [&](int j) {
      return (j < sq.sink_tiles ? j : sq.win_tile + j - sq.sink_tiles) * kSpanTile + warp * kSpKeys;
    };
    // the warp's rows of tile j to shared memory (zeros where nobody sees the slot)
    auto load = [&](int j) {
      const int s0 = first_slot(j);
      const unsigned vis = seen_by_any16(p, sq, b, s0, lane);
      if (!vis) return;
      const size_t row = rows_of16<PAGED>(p, b, g, s0);
      const unsigned char* Kg = static_cast<const unsigned char*>(p.K) + row * kHeadDim * 4 + lane * 16;
      const unsigned char* Vg = static_cast<const unsigned char*>(p.V) + row * kHeadDim * 4 + lane * 16;
      const uint32_t ks = ptx::smem_u32(kt) + lane * 16, vs = ptx::smem_u32(vt) + lane * 16;
#pragma unroll
      for (int k = 0; k < kSpKeys; ++k) {  // a row is 32 pieces of 16 bytes
        const bool ok = (vis >> k) & 1u;
        cp_async16_zfill(ks + k * S::kRowB, Kg + (ok ? k * kHeadDim * 4 : 0), ok);
        cp_async16_zfill(vs + k * S::kRowB, Vg + (ok ? k * kHeadDim * 4 : 0), ok);
      }
    };
    load(j0);
    // queries of this unit's rows (zeros past the last), while the first rows are under way
    const T* q = static_cast<const T*>(p.q) + (((size_t)b * p.Hq + (size_t)g * p.G) * p.T + r0) * kHeadDim;
    for (int e = tid; e < ROWS * kHeadDim; e += kSpThreads) sm_q[e] = r0 + e / kHeadDim < p.R ? q[e] : 0.f;
    __syncthreads();
    float m[ROWS], l[ROWS], o[ROWS][4];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[r][k] = 0.f;
    }
    for (int j = j0; j < j1; ++j) {
      if (j > j0) {
        __syncwarp();  // the last tile's rows and probabilities have been read
        load(j);
      }
      const int s0 = first_slot(j);
      const unsigned vis = seen_by_any16(p, sq, b, s0, lane);
      if (!vis) continue;  // nobody sees the warp's slots
      const bool all_see = vis == 0xffffu && s0 + kSpKeys <= sq.ctx;
      // lane r: what row r sees of the 16 slots
      uint32_t bits = vis;
      if (s0 + kSpKeys > sq.ctx && lane < ROWS) bits &= row_bits(p, sq, b, (r0 + lane) % p.T, s0);
      ptx::cp_async_wait_all();
      __syncwarp();
      // logits of this lane's slot: dimensions 8 c + 4 half .. + 3
      float acc[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) acc[r] = 0.f;
#pragma unroll 4
      for (int c = 0; c < kHeadDim / 8; ++c) {
        const int d = 8 * c + 4 * half;
        const float4 kv = load4(kt + key * S::kRowB, d);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const float4 qv = *reinterpret_cast<const float4*>(sm_q + r * kHeadDim + d);
          acc[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, acc[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float x = (acc[r] + __shfl_xor_sync(0xffffffffu, acc[r], 16)) * p.scale_log2;
        const uint32_t row = __shfl_sync(0xffffffffu, bits, r);
        if (!all_see && !((row >> key) & 1u)) x = -INFINITY;
        float mx = x;
#pragma unroll
        for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float m_new = fmaxf(m[r], mx);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float pr = exp2f(x - base), alpha = exp2f(m[r] - base);
        m[r] = m_new;
        float sum = pr;
#pragma unroll
        for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        l[r] = fmaf(l[r], alpha, sum);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[r][k] *= alpha;
        if (half == 0) sm_p[r * kSpKeys + key] = pr;
      }
      __syncwarp();
      // P.V: this lane's four dimensions of every row
#pragma unroll
      for (int k4 = 0; k4 < kSpKeys / 4; ++k4) {
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = load4(vt + (4 * k4 + k) * S::kRowB, 4 * lane);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const float4 pv = *reinterpret_cast<const float4*>(sm_p + r * kSpKeys + 4 * k4);
          o[r][0] = fmaf(pv.x, v[0].x, fmaf(pv.y, v[1].x, fmaf(pv.z, v[2].x, fmaf(pv.w, v[3].x, o[r][0]))));
          o[r][1] = fmaf(pv.x, v[0].y, fmaf(pv.y, v[1].y, fmaf(pv.z, v[2].y, fmaf(pv.w, v[3].y, o[r][1]))));
          o[r][2] = fmaf(pv.x, v[0].z, fmaf(pv.y, v[1].z, fmaf(pv.z, v[2].z, fmaf(pv.w, v[3].z, o[r][2]))));
          o[r][3] = fmaf(pv.x, v[0].w, fmaf(pv.y, v[1].w, fmaf(pv.z, v[2].w, fmaf(pv.w, v[3].w, o[r][3]))));
        }
      }
    }
    __syncthreads();  // every warp is done with its staged rows
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (lane == 0) {
        sm_m[warp * ROWS + r] = m[r];
        sm_l[warp * ROWS + r] = l[r];
      }
      *reinterpret_cast<float4*>(sm_o + (warp * ROWS + r) * kOutRow + 4 * lane) =
          make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
    }
    __syncthreads();
    finish_unit<T, ROWS>(p, sm_m, sm_l, sm_o, pc, g, rt);
    __syncthreads();
  }
}

// ---- bf16, up to 32 rows: mma.sync tiles -------------------------------------------------------

constexpr int kMmStages = 3;
constexpr int kMmRowB = kHeadDim * 2;              // 16 pieces of 16 bytes, piece c of row k at c ^ (k & 7)
constexpr int kMmStageB = 2 * kSpKeys * kMmRowB;   // K then V of a warp's slots: 8 KB
constexpr int kMmWarpB = kMmStages * kMmStageB;

template <int MT>
struct MmaSmem {
  static constexpr int kRows = 16 * MT;
  static constexpr int kStage = kSpWarps * kMmWarpB;  // later o [warps][rows][kOutRow] fp32
  static constexpr int kQ = kStage;                   // query rows, pieces placed as those of K
  static constexpr int kML = kQ + kRows * kMmRowB;    // m, l [warps][rows]
  static constexpr int kBytes = kML + 2 * kSpWarps * kRows * 4;
  static_assert(kRows * kOutRow * 4 <= kMmWarpB, "the warps' outputs lie over their stages");
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D += A B, A 16 x 16 (row), B 16 x 8 (col), bf16 in, fp32 accumulate.  With g = lane / 4, c = lane % 4:
// a0 = A[g][2c..], a1 = A[g + 8][2c..], a2 = A[g][2c + 8..], a3 = A[g + 8][2c + 8..]; b0 = B[2c..][g],
// b1 = B[2c + 8..][g]; d0, d1 = D[g][2c, 2c + 1], d2, d3 = D[g + 8][..]
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int MT, bool PAGED>
__global__ void __maxnreg__(kSpRegs) span_mma_kernel(const Params p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using S = MmaSmem<MT>;
  constexpr int ROWS = S::kRows;
  float* sm_m = reinterpret_cast<float*>(smem + S::kML);
  float* sm_l = sm_m + kSpWarps * ROWS;
  float* sm_o = reinterpret_cast<float*>(smem);
  const uint32_t sm_q = ptx::smem_u32(smem) + S::kQ;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, cq = lane & 3;
  const uint32_t stages_u = ptx::smem_u32(smem) + (uint32_t)(warp * kMmWarpB);
  uint32_t to[4];  // where copy e goes, less 512 e
#pragma unroll
  for (int i = 0; i < 4; ++i)
    to[i] = (uint32_t)((lane >> 4) * kMmRowB + (((lane & 15) ^ ((2 * i + (lane >> 4)) & 7)) << 4));
  // this lane's row of the fragments: piece 0 of K (slots 0-7 and 8-15, low and high 8 dimensions) and of V
  const int kkey = ((lane >> 4) << 3) + (lane & 7), vkey = (((lane >> 3) & 1) << 3) + (lane & 7);
  const uint32_t kfrag = (uint32_t)(kkey * kMmRowB + ((((lane >> 3) & 1) ^ (kkey & 7)) << 4));
  const uint32_t vfrag = (uint32_t)(vkey * kMmRowB + (((lane >> 4) ^ (vkey & 7)) << 4)) + kSpKeys * kMmRowB;

  ptx::pdl_wait();
  ptx::pdl_launch_dependents();  // the joining kernel may be set up; it waits for this one to end
  Walker walk;
  walk.begin(p, lane, blockIdx.x == 0 && warp == 0);
  Piece pc;
  while (walk.next(p, pc)) {
    const int rt = p.row_tiles == 1 ? 0 : pc.in_seq / p.Hkv, b = pc.b, g = pc.in_seq - rt * p.Hkv, j0 = pc.j0, j1 = pc.j1;
    const Seq& sq = pc.seq;
    const int r0 = rt * ROWS;
    auto first_slot = [&](int j) {
      return (j < sq.sink_tiles ? j : sq.win_tile + j - sq.sink_tiles) * kSpanTile + warp * kSpKeys;
    };
    // tile j's rows of this warp -> stage j % 3 (zeros where nobody sees the slot); one group of copies per call
    auto load = [&](int j) {
      if (j < j1) {
        const int s0 = first_slot(j);
        const unsigned vis = seen_by_any16(p, sq, b, s0, lane);
        if (vis) {
          const size_t row = rows_of16<PAGED>(p, b, g, s0);
          const unsigned char* Kg = static_cast<const unsigned char*>(p.K) + row * kMmRowB;
          const unsigned char* Vg = static_cast<const unsigned char*>(p.V) + row * kMmRowB;
          const uint32_t st = stages_u + (uint32_t)((j % kMmStages) * kMmStageB);
          // copy e: row 2 e + lane / 16, piece lane % 16
          if (vis == 0xffffu) {
            const unsigned char *Kl = Kg + lane * 16, *Vl = Vg + lane * 16;
#pragma unroll
            for (int e = 0; e < kSpKeys / 2; ++e) {
              cp_async16_at(st + to[e & 3] + 512 * e, Kl + 512 * e);
              cp_async16_at(st + to[e & 3] + 512 * e + kSpKeys * kMmRowB, Vl + 512 * e);
            }
          } else {
#pragma unroll
            for (int e = 0; e < kSpKeys / 2; ++e) {
              const bool ok = (vis >> (2 * e + (lane >> 4))) & 1u;
              const int off = ok ? lane * 16 + 512 * e : 0;
              cp_async16_zfill(st + to[e & 3] + 512 * e, Kg + off, ok);
              cp_async16_zfill(st + to[e & 3] + 512 * e + kSpKeys * kMmRowB, Vg + off, ok);
            }
          }
        }
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    // query rows of the unit (zeros past the last), the first group of copies
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                               (((size_t)b * p.Hq + (size_t)g * p.G) * p.T + r0) * kHeadDim;
      for (int e = tid; e < ROWS * 16; e += kSpThreads) {
        const int r = e >> 4, c = e & 15;
        const bool ok = r0 + r < p.R;
        cp_async16_zfill(sm_q + (uint32_t)(r * kMmRowB + ((c ^ (r & 7)) << 4)), q + (ok ? e * 8 : 0), ok);
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
#pragma unroll
    for (int k = 0; k < kMmStages - 1; ++k) load(j0 + k);
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kMmStages - 1) : "memory");
    __syncthreads();
    // query fragments: 32 registers for 16 rows; with 32 rows, whose outputs take 128, they are read again each step
    const uint32_t q_frag = sm_q + (uint32_t)((lane & 15) * kMmRowB + (((lane >> 4) ^ (lane & 7)) << 4));
    uint32_t qa[kHeadDim / 16][4];
    if constexpr (MT == 1) {
#pragma unroll
      for (int ks = 0; ks < kHeadDim / 16; ++ks) ldsm_x4(qa[ks], q_frag ^ (uint32_t)(ks << 5));
    }
    float o[MT][kHeadDim / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < kHeadDim / 8; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[mt][n][k] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
    for (int j = j0; j < j1; ++j) {
      __syncwarp();  // every lane is done with the stage that this load fills
      load(j + kMmStages - 1);
      const int s0 = first_slot(j);
      const unsigned vis = seen_by_any16(p, sq, b, s0, lane);
      const bool all_see = vis == 0xffffu && s0 + kSpKeys <= sq.ctx;
      uint32_t bits[MT][2];  // what this lane's rows see of the 16 slots
      if (!all_see && vis)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            bits[mt][h] = vis;
            if (s0 + kSpKeys > sq.ctx) bits[mt][h] &= row_bits(p, sq, b, (r0 + 16 * mt + gq + 8 * h) % p.T, s0);
          }
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kMmStages - 1) : "memory");
      __syncwarp();
      if (!vis) continue;  // nobody sees the warp's slots
      const uint32_t st = stages_u + (uint32_t)((j % kMmStages) * kMmStageB), kt = st + kfrag, vt = st + vfrag;
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[mt][n][k] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kHeadDim / 16; ++ks) {
        uint32_t kb[4];  // slots 0-7: low and high 8 dimensions; slots 8-15: low and high
        ldsm_x4(kb, kt ^ (uint32_t)(ks << 5));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if constexpr (MT > 1) ldsm_x4(qa[0], (q_frag ^ (uint32_t)(ks << 5)) + (uint32_t)(16 * mt * kMmRowB));
          mma16816(s[mt][0], qa[MT > 1 ? 0 : ks], kb[0], kb[1]);
          mma16816(s[mt][1], qa[MT > 1 ? 0 : ks], kb[2], kb[3]);
        }
      }
      bool moves = false;
      float x_max[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float x = s[mt][n][2 * h + k];
              if (!all_see && !((bits[mt][h] >> (8 * n + 2 * cq + k)) & 1u)) x = -INFINITY;
              s[mt][n][2 * h + k] = x;
              mx = fmaxf(mx, x);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.scale_log2;  // the scale is positive
          x_max[mt][h] = mx;
          moves |= mx > m[mt][h] + kSpSlack;
        }
      // the running maximum moves only when a row passes it by more than 2^8 (p <= 2^8 until then)
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float m_new = fmaxf(m[mt][h], x_max[mt][h]);
            const float alpha = m_new == -INFINITY ? 1.f : ex2(m[mt][h] - m_new);
            m[mt][h] = m_new;
            l[mt][h] *= alpha;
#pragma unroll
            for (int n = 0; n < kHeadDim / 8; ++n) {
              o[mt][n][2 * h] *= alpha;
              o[mt][n][2 * h + 1] *= alpha;
            }
          }
      }
      uint32_t pa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float base = m[mt][h] == -INFINITY ? 0.f : m[mt][h];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const __nv_bfloat162 pr = __floats2bfloat162_rn(ex2(fmaf(s[mt][n][2 * h], p.scale_log2, -base)),
                                                            ex2(fmaf(s[mt][n][2 * h + 1], p.scale_log2, -base)));
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&pr);
            pa[mt][2 * n + h] = u;
            // the row sum takes p as P.V does, rounded: a row that one slot dominates comes out exact
            l[mt][h] += __uint_as_float(u << 16) + __uint_as_float(u & 0xffff0000u);
          }
        }
#pragma unroll
      for (int n = 0; n < kHeadDim / 16; ++n) {
        uint32_t vb[4];  // dimensions 16 n .. + 7: slots 0-7, 8-15; then the next 8 dimensions
        ldsm_x4_trans(vb, vt ^ (uint32_t)(n << 5));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816(o[mt][2 * n], pa[mt], vb[0], vb[1]);
          mma16816(o[mt][2 * n + 1], pa[mt], vb[2], vb[3]);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();  // every warp is done with its stages
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * mt + gq + 8 * h;
        float sum = l[mt][h];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (r0 + r >= p.R) continue;
        if (cq == 0) {
          sm_m[warp * ROWS + r] = m[mt][h];
          sm_l[warp * ROWS + r] = sum;
        }
#pragma unroll
        for (int n = 0; n < kHeadDim / 8; ++n)
          *reinterpret_cast<float2*>(sm_o + (warp * ROWS + r) * kOutRow + 8 * n + 2 * cq) =
              make_float2(o[mt][n][2 * h], o[mt][n][2 * h + 1]);
      }
    __syncthreads();
    finish_unit<__nv_bfloat16, ROWS>(p, sm_m, sm_l, sm_o, pc, g, rt);
    __syncthreads();
  }
}

// Shared-memory attribute of a kernel, set once per device under a mutex; a failed call is returned on
// every later launch on that device.
template <typename Kernel>
cudaError_t configure(Kernel k, int smem) {
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, cudaError_t> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  const std::pair<int, const void*> id(dev, reinterpret_cast<const void*>(k));
  auto it = done.find(id);
  if (it != done.end()) return it->second;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) (void)cudaGetLastError();
  done[id] = e;
  return e;
}

template <typename T, int ROWS, typename Kernel>
cudaError_t launch_rows(Kernel k, int smem, Params p, cudaStream_t st) {
  cudaError_t e = configure(k, smem);
  if (e != cudaSuccess) return e;
  p.row_tiles = (p.R + ROWS - 1) / ROWS;
  const long long units = (long long)p.B * p.Hkv * p.row_tiles;
  if (!span_fits(p, units)) return cudaErrorNotSupported;
  const int grid = span_sms();
  if ((e = launch_early(k, dim3((unsigned)grid), kSpThreads, (size_t)smem, st, p)) != cudaSuccess) return e;
  return launch_early(span_join_kernel<T, ROWS>, dim3((unsigned)units + 1, ROWS / kJoinWarps), kJoinWarps * 32, 0, st, p, grid);
}

template <int ROWS>
cudaError_t launch_simt(const Params& p, bool paged, cudaStream_t st) {
  if (paged) return launch_rows<float, ROWS>(span_simt_kernel<ROWS, true>, SimtSmem<ROWS>::kBytes, p, st);
  return launch_rows<float, ROWS>(span_simt_kernel<ROWS, false>, SimtSmem<ROWS>::kBytes, p, st);
}

template <int MT>
cudaError_t launch_mma(const Params& p, bool paged, cudaStream_t st) {
  if (paged) return launch_rows<__nv_bfloat16, 16 * MT>(span_mma_kernel<MT, true>, MmaSmem<MT>::kBytes, p, st);
  return launch_rows<__nv_bfloat16, 16 * MT>(span_mma_kernel<MT, false>, MmaSmem<MT>::kBytes, p, st);
}

// rows of the largest row tile of the kernels here
constexpr int kSpanMaxRows = 32;

// bf16 with more rows per KV head than a tile of span_mma_kernel holds runs on span_tc_kernel.  Up to two such tiles, both
// of which read all keys, are faster while the keys are few and the fixed costs count: 64 rows, 8 KV heads (tiles of 128
// slots in all: us of span_mma_kernel, of span_tc_kernel): 256: 15, 20; 2048: 45, 50; 8192: 181, 111.  The tiles are counted
// from max_seq, since the lengths are on the device: a cache that is longer than that and holds little takes the 20.
constexpr int kSpanTcRows = 32, kSpanTcTiles = 2048;
bool use_tc(const hata_dims_t& d, int n_tok) {
  const long long rows = (long long)(d.n_q_heads / d.n_kv_heads) * n_tok;
  if (d.dtype != HATA_BF16 || rows <= kSpanTcRows) return false;
  const long long tiles = (long long)d.batch * d.n_kv_heads * ((d.max_seq + kSpanTile - 1LL) / kSpanTile);
  return rows > 2 * kSpanTcRows || tiles > kSpanTcTiles;
}

}  // namespace

int span_sms() {
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 148;
  }
  std::lock_guard<std::mutex> lk(mu);
  auto it = cache.find(dev);
  if (it == cache.end()) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
      (void)cudaGetLastError();
      sms = 148;
    }
    it = cache.emplace(dev, sms).first;
  }
  return it->second;
}

size_t span_ws_bytes(const hata_dims_t& d, int n_tok) {
  const size_t few = (size_t)span_sms() * 2 * kSpanMaxRows * (kHeadDim + 2) * 4;
  return kAlign + (use_tc(d, n_tok) ? span_tc_part_bytes(d, n_tok) : few);
}

cudaError_t launch_span(const hata_dims_t& d, const SpanArgs& a, const PagedCache* pg, char* ws, cudaStream_t st) {
  Params p{};
  p.q = a.q;
  p.K = a.K;
  p.V = a.V;
  p.out = a.out;
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.part = reinterpret_cast<float*>(ws + kAlign);
  p.seq_lens = a.seq_lens;
  p.n_new = a.n_new;
  p.mask = a.mask;
  p.B = d.batch;
  p.Hq = d.n_q_heads;
  p.Hkv = d.n_kv_heads;
  p.G = d.n_q_heads / d.n_kv_heads;
  p.T = a.n_tok;
  p.R = p.G * p.T;
  p.max_seq = d.max_seq;
  p.mask_words = (a.n_tok + 31) / 32;
  p.window = a.window;
  p.sink = a.sink;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (pg) {
    p.block_table = pg->block_table;
    p.block_shift = pg->block_shift;
    p.n_blocks = pg->n_blocks;
    p.max_blocks = pg->max_blocks;
  }
  if (a.window == 0 && use_tc(d, a.n_tok)) return launch_span_tc(d, p, pg, st);
  const bool paged = pg != nullptr;
  if (d.dtype == HATA_BF16) return p.R <= 16 ? launch_mma<1>(p, paged, st) : launch_mma<2>(p, paged, st);
  return p.R <= 4 ? launch_simt<4>(p, paged, st) : launch_simt<16>(p, paged, st);
}

}  // namespace hata
