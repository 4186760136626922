// Window decode and tree attention: softmax(scale * q . K) V of the new tokens' rows over the visible slots
// of a contiguous or paged cache (hata_span.cuh has the split of the work).
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

// The end of a unit's run in this CTA.  In shared memory: m, l [kSpWarps][ROWS] and o [kSpWarps][ROWS][128]
// of the warps.  Merges them, then writes the rows, or leaves a partial and, as the last to arrive, merges
// the partials.  All threads of the CTA.
template <typename T, int ROWS>
__device__ __forceinline__ void finish_unit(const Params& p, const float* sm_m, const float* sm_l, const float* sm_o,
                                            int b, int n_b, int g, int rt, long long unit, long long u0, long long u1,
                                            long long per, int cta) {
  __shared__ int s_last;
  const int tid = threadIdx.x;
  const long long c0 = u0 / per, c1 = (u1 - 1) / per;
  const int r0 = rt * ROWS;
  T* out = static_cast<T*>(p.out) + (((size_t)b * p.Hq + (size_t)g * p.G) * p.T) * kHeadDim;
  const int slot = (long long)cta * per > u0 ? 0 : 1;  // a CTA continues one unit at most, and leaves one at most
  float* part = p.part + ((size_t)cta * 2 + slot) * ROWS * (kHeadDim + 2);
  for (int e = tid; e < ROWS * kHeadDim; e += kSpThreads) {
    const int r = e / kHeadDim, d = e % kHeadDim;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSpWarps; ++w) M = fmaxf(M, sm_m[w * ROWS + r]);
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kSpWarps; ++w) {
      const float mw = sm_m[w * ROWS + r];
      const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
      l = fmaf(sm_l[w * ROWS + r], f, l);
      o = fmaf(sm_o[((size_t)w * ROWS + r) * kHeadDim + d], f, o);
    }
    if (c0 == c1) {
      if (r0 + r < p.R && (r0 + r) % p.T < n_b)
        store_out<T>(out + (size_t)(r0 + r) * kHeadDim + d, l == 0.f ? 0.f : o / l);
    } else {
      part[2 * ROWS + e] = o;
      if (d == 0) {
        part[r] = M;
        part[ROWS + r] = l;
      }
    }
  }
  if (c0 == c1) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(&p.count[unit], 1u) == (unsigned)(c1 - c0);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int e = tid; e < ROWS * kHeadDim; e += kSpThreads) {
    const int r = e / kHeadDim, d = e % kHeadDim;
    if (r0 + r >= p.R || (r0 + r) % p.T >= n_b) continue;
    float M = -INFINITY;
    for (long long c = c0; c <= c1; ++c) {
      const int sl = c * per > u0 ? 0 : 1;
      M = fmaxf(M, __ldcg(p.part + ((size_t)c * 2 + sl) * ROWS * (kHeadDim + 2) + r));
    }
    float l = 0.f, o = 0.f;
    for (long long c = c0; c <= c1; ++c) {
      const int sl = c * per > u0 ? 0 : 1;
      const float* pp = p.part + ((size_t)c * 2 + sl) * ROWS * (kHeadDim + 2);
      const float mc = __ldcg(pp + r);
      const float f = mc == -INFINITY ? 0.f : exp2f(mc - M);
      l = fmaf(__ldcg(pp + ROWS + r), f, l);
      o = fmaf(__ldcg(pp + 2 * ROWS + e), f, o);
    }
    store_out<T>(out + (size_t)(r0 + r) * kHeadDim + d, l == 0.f ? 0.f : o / l);
  }
  if (tid == 0) p.count[unit] = 0u;
}

template <typename T>
__device__ __forceinline__ float4 load4(const unsigned char* row, int d);
template <>
__device__ __forceinline__ float4 load4<float>(const unsigned char* row, int d) {
  return *reinterpret_cast<const float4*>(row + 4 * d);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const unsigned char* row, int d) {
  const uint2 u = *reinterpret_cast<const uint2*>(row + 2 * d);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

template <typename T, int ROWS>
struct SimtSmem {
  static constexpr int kRowB = kHeadDim * (int)sizeof(T) + 16;  // padded: 16 rows on distinct banks
  static constexpr int kWarpB = 2 * kSpKeys * kRowB;            // K then V of a warp's slots
  static constexpr int kStage = kSpWarps * kWarpB > kSpWarps * ROWS * kHeadDim * 4 ? kSpWarps * kWarpB
                                                                                   : kSpWarps * ROWS * kHeadDim * 4;
  static constexpr int kQ = kStage;                               // [ROWS][128] fp32
  static constexpr int kP = kQ + ROWS * kHeadDim * 4;             // [warps][ROWS][16] fp32
  static constexpr int kML = kP + kSpWarps * ROWS * kSpKeys * 4;  // m, l [warps][ROWS]
  static constexpr int kBytes = kML + 2 * kSpWarps * ROWS * 4;
};

template <typename T, int ROWS, bool PAGED>
__global__ void __launch_bounds__(kSpThreads, 1) span_simt_kernel(const Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  using S = SimtSmem<T, ROWS>;
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
      sm_q[e] = r0 + e / kHeadDim < p.R ? to_f32<T>(q[e]) : 0.f;
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
        const float4 kv = load4<T>(kt + key * S::kRowB, d);
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
        for (int k = 0; k < 4; ++k) v[k] = load4<T>(vt + (4 * k4 + k) * S::kRowB, 4 * lane);
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
    finish_unit<T, ROWS>(p, sm_m, sm_l, sm_o, b, sq.n_b, g, rt, unit, u0, u1, per, (int)blockIdx.x);
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

template <typename T, int ROWS, bool PAGED>
cudaError_t launch_simt(Params p, cudaStream_t st) {
  constexpr int smem = SimtSmem<T, ROWS>::kBytes;
  cudaError_t e = configure(span_simt_kernel<T, ROWS, PAGED>, smem);
  if (e != cudaSuccess) return e;
  p.row_tiles = (p.R + ROWS - 1) / ROWS;
  span_simt_kernel<T, ROWS, PAGED><<<span_sms(), kSpThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt_t(const Params& p, cudaStream_t st) {
  if (p.R <= 4) return p.block_table ? launch_simt<T, 4, true>(p, st) : launch_simt<T, 4, false>(p, st);
  return p.block_table ? launch_simt<T, 16, true>(p, st) : launch_simt<T, 16, false>(p, st);
}

// rows of the largest row tile, and of the smallest (most units)
constexpr int kSpanMaxRows = 16, kSpanMinRows = 16;

size_t count_bytes(const hata_dims_t& d, int n_tok) {
  const size_t R = (size_t)(d.n_q_heads / d.n_kv_heads) * n_tok;
  return align_up((size_t)d.batch * d.n_kv_heads * ((R + kSpanMinRows - 1) / kSpanMinRows) * 4, kAlign);
}

// bf16 with more rows per KV head than this runs on the tensor cores.
constexpr int kSpanTcRows = 16;
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
  if (d.dtype == HATA_BF16) return launch_simt_t<__nv_bfloat16>(p, st);
  return launch_simt_t<float>(p, st);
}

}  // namespace hata
