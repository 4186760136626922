// Window decode and tree attention: softmax(scale * q . K) V of the new tokens' rows over the visible slots
// of a contiguous or paged cache (hata_span.cuh has the split of the work).
//
// span_mma_kernel (bf16, up to 32 rows per KV head): eight warps, each with 16 slots of a 128-slot tile, on its own: it
// streams its rows of K and V through three shared-memory stages (cp.async, 16-byte pieces swizzled so that the eight
// rows of a fragment lie in distinct banks), computes S on m16n8k16 tiles with the query rows as M, turns S
// into P in place (the accumulator of S has the layout of the A operand of P.V), and adds P.V to its own running
// output.  No barrier inside a run of tiles.  The warps meet once per unit.  Bound by memory: at 6.5 TB/s an SM
// receives a warp's 8 KB step every 364 cycles, and 128 KB are in flight.
//
// span_simt_kernel (fp32): eight warps, each with 16 slots of a 128-slot tile, on its own: it copies
// its rows of K and V to shared memory (cp.async), a lane takes one slot and half of the 128 dimensions for the
// logits and four dimensions of every row for P.V, and keeps its own running maximum, sum and output
// (fp32, online softmax).  The warps meet once per unit.  Bound by the fp32 units when a unit
// has many rows (each shared-memory vector feeds 4 multiply-adds per row), else by memory.
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
constexpr float kSpSlack = 8.f;  // log2 units
static_assert(kSpWarps * kSpKeys == kSpanTile, "the warps share a tile");

// 16-byte copy, or 16 zero bytes where !valid
__device__ __forceinline__ void cp_async16_zfill(void* smem, const void* gmem, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(ptx::smem_u32(smem)), "l"(gmem),
               "r"(valid ? 16 : 0)
               : "memory");
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

// The weights that bring n partials of each row to one maximum: sm_m, sm_l [n][ROWS] (maximum, sum) become
// sm_m = 2^(m - M) and, for row r, (M, sum of l 2^(m - M)) in row_m, row_l.  A warp per row; all threads.
template <int ROWS>
__device__ __forceinline__ void join_weights(float* sm_m, const float* sm_l, int n, float* row_m, float* row_l) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = warp; r < ROWS; r += kSpWarps) {
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

// The end of a unit's run in this CTA.  In shared memory: m, l [kSpWarps][ROWS] and o [kSpWarps][ROWS][128]
// of the warps.  Joins them, then writes the rows, or leaves a partial and, as the last to arrive, joins
// the partials.  `scratch`: 2 * gridDim.x * ROWS floats for the latter (over o).  All threads of the CTA.
template <typename T, int ROWS>
__device__ __forceinline__ void finish_unit(const Params& p, float* sm_m, float* sm_l, const float* sm_o, float* scratch,
                                            int b, int n_b, int g, int rt, long long unit, long long u0, long long u1,
                                            long long per, int cta) {
  __shared__ int s_last;
  __shared__ float row_m[ROWS], row_l[ROWS];
  constexpr int kQuads = ROWS * kHeadDim / 4;
  const int tid = threadIdx.x;
  const long long c0 = u0 / per, c1 = (u1 - 1) / per;
  const int r0 = rt * ROWS;
  T* out = static_cast<T*>(p.out) + (((size_t)b * p.Hq + (size_t)g * p.G) * p.T + r0) * kHeadDim;
  auto live = [&](int r) { return r0 + r < p.R && (r0 + r) % p.T < n_b; };
  const int slot = (long long)cta * per > u0 ? 0 : 1;  // a CTA continues one unit at most, and leaves one at most
  float* part = p.part + ((size_t)cta * 2 + slot) * ROWS * (kHeadDim + 2);
  join_weights<ROWS>(sm_m, sm_l, kSpWarps, row_m, row_l);
  for (int e = tid; e < kQuads; e += kSpThreads) {
    const int r = e / (kHeadDim / 4);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kSpWarps; ++w) {
      const float f = sm_m[w * ROWS + r];
      const float4 v = reinterpret_cast<const float4*>(sm_o)[w * kQuads + e];
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    if (c0 == c1) {
      const float l = row_l[r], inv = l == 0.f ? 0.f : 1.f / l;
      if (live(r)) store4<T>(out + 4 * e, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    } else {
      reinterpret_cast<float4*>(part + 2 * ROWS)[e] = o;
    }
  }
  if (c0 == c1) return;
  if (tid < ROWS) {
    part[tid] = row_m[tid];
    part[ROWS + tid] = row_l[tid];
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&p.count[unit], 1u) == (unsigned)(c1 - c0);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const int n = (int)(c1 - c0) + 1;  // at most gridDim.x
  auto part_of = [&](int i) {
    const long long c = c0 + i;
    return p.part + ((size_t)c * 2 + (c * per > u0 ? 0 : 1)) * ROWS * (kHeadDim + 2);
  };
  float *wm = scratch, *wl = scratch + n * ROWS;
  for (int e = tid; e < n * ROWS; e += kSpThreads) {
    const float* pp = part_of(e / ROWS) + e % ROWS;
    wm[e] = __ldcg(pp);
    wl[e] = __ldcg(pp + ROWS);
  }
  __syncthreads();
  join_weights<ROWS>(wm, wl, n, row_m, row_l);
  for (int e = tid; e < kQuads; e += kSpThreads) {
    const int r = e / (kHeadDim / 4);
    if (!live(r)) continue;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float f = wm[i * ROWS + r];
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part_of(i) + 2 * ROWS) + e);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    const float l = row_l[r], inv = l == 0.f ? 0.f : 1.f / l;
    store4<T>(out + 4 * e, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  }
  if (tid == 0) p.count[unit] = 0u;
}

__device__ __forceinline__ float4 load4(const unsigned char* row, int d) {
  return *reinterpret_cast<const float4*>(row + 4 * d);
}

template <int ROWS>
struct SimtSmem {
  static constexpr int kRowB = kHeadDim * 4 + 16;  // padded: 16 rows on distinct banks
  static constexpr int kWarpB = 2 * kSpKeys * kRowB;            // K then V of a warp's slots
  static constexpr int kStage = kSpWarps * kWarpB > kSpWarps * ROWS * kHeadDim * 4 ? kSpWarps * kWarpB
                                                                                   : kSpWarps * ROWS * kHeadDim * 4;
  static constexpr int kQ = kStage;                               // [ROWS][128] fp32
  static constexpr int kP = kQ + ROWS * kHeadDim * 4;             // [warps][ROWS][16] fp32
  static constexpr int kML = kP + kSpWarps * ROWS * kSpKeys * 4;  // m, l [warps][ROWS]
  static constexpr int kBytes = kML + 2 * kSpWarps * ROWS * 4;
};

template <int ROWS, bool PAGED>
__global__ void __launch_bounds__(kSpThreads, 1) span_simt_kernel(const Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
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

  const long long total = total_tiles(p, lane, blockIdx.x == 0 && warp == 0);
  const long long per = max(1LL, (total + gridDim.x - 1) / gridDim.x);
  long long at = (long long)blockIdx.x * per;
  const long long end = min(total, at + per);
  if (at >= end) return;
  Cursor cur = find(p, at, lane);
  const int key = lane & 15, half = lane >> 4;
  while (at < end) {
    while (at >= cur.seq_start + (long long)cur.seq.tiles * p.Hkv * p.row_tiles) {
      cur.seq_start += (long long)cur.seq.tiles * p.Hkv * p.row_tiles;
      cur.seq = seq_of(p, ++cur.b);
    }
    const int b = cur.b;
    const Seq& sq = cur.seq;
    const long long in_seq = (at - cur.seq_start) / sq.tiles;  // unit within the sequence
    const int g = (int)(in_seq % p.Hkv), rt = (int)(in_seq / p.Hkv);
    const long long u0 = cur.seq_start + in_seq * sq.tiles, u1 = u0 + sq.tiles;
    const int j0 = (int)(at - u0), j1 = (int)(min(end, u1) - u0);
    const int r0 = rt * ROWS;
    // queries of this unit's rows (zeros past the last)
    const T* q = static_cast<const T*>(p.q) + (((size_t)b * p.Hq + (size_t)g * p.G) * p.T + r0) * kHeadDim;
    for (int e = tid; e < ROWS * kHeadDim; e += kSpThreads)
      sm_q[e] = r0 + e / kHeadDim < p.R ? q[e] : 0.f;
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
      const int tile = j < sq.sink_tiles ? j : sq.win_tile + j - sq.sink_tiles;
      const int s0 = tile * kSpanTile + warp * kSpKeys;
      const unsigned vis = seen_by_any16(p, sq, b, s0, lane);
      if (!vis) continue;  // the warp's slots are seen by nobody
      const size_t row = rows_of16<PAGED>(p, b, g, s0);
      constexpr int VPR = kHeadDim * (int)sizeof(T) / 16;  // vectors of a row
      const unsigned char* Kg = static_cast<const unsigned char*>(p.K) + row * kHeadDim * sizeof(T);
      const unsigned char* Vg = static_cast<const unsigned char*>(p.V) + row * kHeadDim * sizeof(T);
      __syncwarp();  // the last tile's rows and probabilities have been read
      for (int e = lane; e < kSpKeys * VPR; e += 32) {
        const int k = e / VPR, c = e % VPR;
        const bool ok = (vis >> k) & 1u;
        const size_t off = ok ? (size_t)k * kHeadDim * sizeof(T) + c * 16 : 0;
        cp_async16_zfill(kt + k * S::kRowB + c * 16, Kg + off, ok);
        cp_async16_zfill(vt + k * S::kRowB + c * 16, Vg + off, ok);
      }
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
      const int s = s0 + key;
      const bool live = (vis >> key) & 1u;
      const bool all_see = s0 + kSpKeys <= sq.ctx;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float x = (acc[r] + __shfl_xor_sync(0xffffffffu, acc[r], 16)) * p.scale_log2;
        if (!live || (!all_see && !sees(p, sq, b, (r0 + r) % p.T, s))) x = -INFINITY;
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
      *reinterpret_cast<float4*>(sm_o + ((size_t)warp * ROWS + r) * kHeadDim + 4 * lane) =
          make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
    }
    __syncthreads();
    long long unit = (long long)b * p.Hkv * p.row_tiles + in_seq;
    finish_unit<T, ROWS>(p, sm_m, sm_l, sm_o, sm_o, b, sq.n_b, g, rt, unit, u0, u1, per, (int)blockIdx.x);
    __syncthreads();
    at = u0 + j1;
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
  static constexpr int kStage = kSpWarps * kMmWarpB;  // later o [warps][rows][128] fp32: 64 KB per 16 rows
  static constexpr int kML = kStage;                  // m, l [warps][rows]
  static constexpr int kBytes = kML + 2 * kSpWarps * kRows * 4;
  static_assert(kSpWarps * kRows * kHeadDim * 4 <= kStage, "the warps' outputs lie over their stages");
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
__global__ void __launch_bounds__(kSpThreads, 1) span_mma_kernel(const Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  using S = MmaSmem<MT>;
  constexpr int ROWS = S::kRows;
  float* sm_m = reinterpret_cast<float*>(smem + S::kML);
  float* sm_l = sm_m + kSpWarps * ROWS;
  float* sm_o = reinterpret_cast<float*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, cq = lane & 3;
  unsigned char* stages = smem + warp * kMmWarpB;
  const uint32_t stages_u = ptx::smem_u32(stages);

  const long long total = total_tiles(p, lane, blockIdx.x == 0 && warp == 0);
  const long long per = max(1LL, (total + gridDim.x - 1) / gridDim.x);
  long long at = (long long)blockIdx.x * per;
  const long long end = min(total, at + per);
  if (at >= end) return;
  Cursor cur = find(p, at, lane);
  while (at < end) {
    while (at >= cur.seq_start + (long long)cur.seq.tiles * p.Hkv * p.row_tiles) {
      cur.seq_start += (long long)cur.seq.tiles * p.Hkv * p.row_tiles;
      cur.seq = seq_of(p, ++cur.b);
    }
    const int b = cur.b;
    const Seq& sq = cur.seq;
    const long long in_seq = (at - cur.seq_start) / sq.tiles;  // unit within the sequence
    const int g = (int)(in_seq % p.Hkv), rt = (int)(in_seq / p.Hkv);
    const long long u0 = cur.seq_start + in_seq * sq.tiles, u1 = u0 + sq.tiles;
    const int j0 = (int)(at - u0), j1 = (int)(min(end, u1) - u0);
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
          unsigned char* st = stages + (j % kMmStages) * kMmStageB;
#pragma unroll
          for (int e = 0; e < kSpKeys * 16 / 32; ++e) {
            const int k = 2 * e + (lane >> 4), c = lane & 15;
            const bool ok = (vis >> k) & 1u;
            const int off = ok ? k * kMmRowB + c * 16 : 0;
            const int to = k * kMmRowB + ((c ^ (k & 7)) << 4);
            cp_async16_zfill(st + to, Kg + off, ok);
            cp_async16_zfill(st + kSpKeys * kMmRowB + to, Vg + off, ok);
          }
        }
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < kMmStages - 1; ++k) load(j0 + k);
    // query fragments of the unit's rows (zeros past the last)
    uint32_t qa[MT][kHeadDim / 16][4];
    {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) +
                               (((size_t)b * p.Hq + (size_t)g * p.G) * p.T + r0) * kHeadDim + 2 * cq;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int ks = 0; ks < kHeadDim / 16; ++ks)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = 16 * mt + gq + 8 * (k & 1);
            qa[mt][ks][k] = r0 + r < p.R
                                ? __ldg(reinterpret_cast<const uint32_t*>(q + (size_t)r * kHeadDim + 16 * ks + 8 * (k >> 1)))
                                : 0u;
          }
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
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kMmStages - 1) : "memory");
      __syncwarp();
      const int s0 = first_slot(j);
      const unsigned vis = seen_by_any16(p, sq, b, s0, lane);
      if (!vis) continue;  // nobody sees the warp's slots
      const uint32_t kt = stages_u + (uint32_t)((j % kMmStages) * kMmStageB), vt = kt + kSpKeys * kMmRowB;
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[mt][n][k] = 0.f;
      {
        const int key = ((lane >> 4) << 3) + (lane & 7), hi = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < kHeadDim / 16; ++ks) {
          uint32_t kb[4];  // slots 0-7: low and high 8 dimensions; slots 8-15: low and high
          ldsm_x4(kb, kt + (uint32_t)(key * kMmRowB + (((2 * ks + hi) ^ (key & 7)) << 4)));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(s[mt][0], qa[mt][ks], kb[0], kb[1]);
            mma16816(s[mt][1], qa[mt][ks], kb[2], kb[3]);
          }
        }
      }
      const bool all_see = vis == 0xffffu && s0 + kSpKeys <= sq.ctx;
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
              float x = s[mt][n][2 * h + k] * p.scale_log2;
              if (!all_see) {
                const int e = 8 * n + 2 * cq + k;
                if (!((vis >> e) & 1u) || (s0 + e >= sq.ctx && !sees(p, sq, b, (r0 + 16 * mt + gq + 8 * h) % p.T, s0 + e)))
                  x = -INFINITY;
              }
              s[mt][n][2 * h + k] = x;
              mx = fmaxf(mx, x);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
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
            const float alpha = m_new == -INFINITY ? 1.f : exp2f(m[mt][h] - m_new);
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
            const __nv_bfloat162 pr = __floats2bfloat162_rn(exp2f(s[mt][n][2 * h] - base), exp2f(s[mt][n][2 * h + 1] - base));
            const uint32_t u = *reinterpret_cast<const uint32_t*>(&pr);
            pa[mt][2 * n + h] = u;
            // the row sum takes p as P.V does, rounded: a row that one slot dominates comes out exact
            l[mt][h] += __uint_as_float(u << 16) + __uint_as_float(u & 0xffff0000u);
          }
        }
      {
        const int key = (((lane >> 3) & 1) << 3) + (lane & 7), hi = lane >> 4;
#pragma unroll
        for (int n = 0; n < kHeadDim / 16; ++n) {
          uint32_t vb[4];  // dimensions 16 n .. + 7: slots 0-7, 8-15; then the next 8 dimensions
          ldsm_x4_trans(vb, vt + (uint32_t)(key * kMmRowB + (((2 * n + hi) ^ (key & 7)) << 4)));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(o[mt][2 * n], pa[mt], vb[0], vb[1]);
            mma16816(o[mt][2 * n + 1], pa[mt], vb[2], vb[3]);
          }
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
        if (cq == 0) {
          sm_m[warp * ROWS + r] = m[mt][h];
          sm_l[warp * ROWS + r] = sum;
        }
#pragma unroll
        for (int n = 0; n < kHeadDim / 8; ++n)
          *reinterpret_cast<float2*>(sm_o + ((size_t)warp * ROWS + r) * kHeadDim + 8 * n + 2 * cq) =
              make_float2(o[mt][n][2 * h], o[mt][n][2 * h + 1]);
      }
    __syncthreads();
    finish_unit<__nv_bfloat16, ROWS>(p, sm_m, sm_l, sm_o, sm_o, b, sq.n_b, g, rt,
                                     (long long)b * p.Hkv * p.row_tiles + in_seq, u0, u1, per, (int)blockIdx.x);
    __syncthreads();
    at = u0 + j1;
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

template <int ROWS, bool PAGED>
cudaError_t launch_simt(Params p, cudaStream_t st) {
  constexpr int smem = SimtSmem<ROWS>::kBytes;
  cudaError_t e = configure(span_simt_kernel<ROWS, PAGED>, smem);
  if (e != cudaSuccess) return e;
  p.row_tiles = (p.R + ROWS - 1) / ROWS;
  span_simt_kernel<ROWS, PAGED><<<span_sms(), kSpThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <int MT, bool PAGED>
cudaError_t launch_mma(Params p, cudaStream_t st) {
  constexpr int smem = MmaSmem<MT>::kBytes;
  cudaError_t e = configure(span_mma_kernel<MT, PAGED>, smem);
  if (e != cudaSuccess) return e;
  p.row_tiles = (p.R + 16 * MT - 1) / (16 * MT);
  span_mma_kernel<MT, PAGED><<<span_sms(), kSpThreads, smem, st>>>(p);
  return cudaGetLastError();
}

// rows of the largest row tile, and of the smallest (most units)
constexpr int kSpanMaxRows = 32, kSpanMinRows = 4;

size_t count_bytes(const hata_dims_t& d, int n_tok) {
  const size_t R = (size_t)(d.n_q_heads / d.n_kv_heads) * n_tok;
  return align_up((size_t)d.batch * d.n_kv_heads * ((R + kSpanMinRows - 1) / kSpanMinRows) * 4, kAlign);
}

// bf16 with more rows per KV head than this runs on the tensor cores.
constexpr int kSpanTcRows = 32;
bool use_tc(const hata_dims_t& d, int n_tok) {
  return d.dtype == HATA_BF16 && (d.n_q_heads / d.n_kv_heads) * n_tok > kSpanTcRows;
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
  const size_t simt = (size_t)span_sms() * 2 * kSpanMaxRows * (kHeadDim + 2) * 4;
  return kAlign + count_bytes(d, n_tok) + (use_tc(d, n_tok) ? std::max(simt, span_tc_part_bytes(d, n_tok)) : simt);
}

cudaError_t launch_span(const hata_dims_t& d, const SpanArgs& a, const PagedCache* pg, char* ws, cudaStream_t st) {
  Params p{};
  p.q = a.q;
  p.K = a.K;
  p.V = a.V;
  p.out = a.out;
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.count = reinterpret_cast<uint32_t*>(ws + kAlign);
  p.part = reinterpret_cast<float*>(ws + kAlign + count_bytes(d, a.n_tok));
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
  if (d.dtype == HATA_BF16) {
    if (p.R <= 16) return paged ? launch_mma<1, true>(p, st) : launch_mma<1, false>(p, st);
    return paged ? launch_mma<2, true>(p, st) : launch_mma<2, false>(p, st);
  }
  if (p.R <= 4) return paged ? launch_simt<4, true>(p, st) : launch_simt<4, false>(p, st);
  return paged ? launch_simt<16, true>(p, st) : launch_simt<16, false>(p, st);
}

}  // namespace hata
