// Norms of queries and keys for each head, the position rotation and the cache append in one
// pass over a projection's output: the step between the projection and hata_decode_step (which
// encodes and scores the new key from its cache slot).
//
// For token i of sequence b, with slot s = L_b - n_b + i and position t = positions[b][i] (or s):
//   y = x * rsqrt(mean(x^2) + eps) * w          (fp32; w NULL: y = x)
//   (y_a, y_b) -> (y_a c - y_b s', y_b c + y_a s')   with (c, s') = table[t][.][pair]
// for the rot / 2 pairs of the first rot elements: (e, e + rot / 2) or, interleaved, (2 e, 2 e + 1).
// Queries go to q_out[b][h][i], keys to K[.][g][s], values are copied to V[.][g][s].  Everything
// is fp32 between the load and the one rounding of the store.
//
// Bound by memory: each row is read once and written once.  A row is 16 (bf16) or 32 (fp32) lanes
// of 16 bytes, so the mean square is a shuffle tree and the partner of a half-split pair lies rot / 2
// elements, a whole number of lanes, away.  The 8 warps of a CTA take 8 consecutive tokens and the same rows of
// each, so that the scattered stores of neighbouring tokens meet in L2 as 2 KB runs per head.
// Measured on B200: 4 prompts of up to 8192 tokens (32 / 8 heads, bf16, 617 MB in and out on average) 108-125 us from one run
// to another, 0.75-0.87 of a copy's bandwidth; 4 of up to 4096 in fp32 106 us, 0.89; one token of 16 sequences into a paged
// cache 2.9 us.  A warp per four rows of a token, each fetching
// positions, table and weights for itself, took 240 us; a warp per token with norm weights, cosines and sines
// in registers 144 us (two CTAs per SM; with three it spilled, 232 us).
#include <algorithm>

#include "hata_kernels.cuh"

namespace hata {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeBatch = 2;  // row steps whose loads go out together, while those of the batch before are turned
constexpr int kRopeCtas = 3;   // per SM: 80 registers a thread

struct RopeParams {
  const void *q_in, *k_in, *v_in;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const float *q_weight, *k_weight;
  const float* table;
  const int32_t *n_new, *positions, *seq_lens;
  void *q_out, *K, *V;
  const int32_t* block_table;
  uint32_t* status;
  float eps;
  int n_tok, Hq, Hkv, max_seq, n_pos, rot;
  int block_shift, n_blocks, max_blocks;
  int tok_blocks;      // ceil(n_tok / kRopeWarps)
  int steps_per_warp;  // row steps of one warp
  int n_split;         // warps that share a token's rows
};

template <typename T>
struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[N]);
  static __device__ __forceinline__ uint4 pack(const float (&x)[N]);
};
template <>
__device__ __forceinline__ void Vec16<float>::unpack(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
template <>
__device__ __forceinline__ uint4 Vec16<float>::pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
template <>
__device__ __forceinline__ void Vec16<__nv_bfloat16>::unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the high half of the fp32 of the same value
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ uint4 Vec16<__nv_bfloat16>::pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, bool INTER, bool PAGED>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeCtas) norm_rope_kernel(const RopeParams p) {
  constexpr int N = Vec16<T>::N;           // elements of a lane's vector
  constexpr int LANES = kHeadDim / N;      // lanes of a row
  constexpr int RPS = 32 / LANES;          // rows of one warp step
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int li = lane % LANES, sub = lane / LANES;
  const int b = (int)(blockIdx.y), tb = (int)(blockIdx.x) / p.n_split, sp = (int)(blockIdx.x) % p.n_split;
  const int i = tb * kRopeWarps + warp;
  const int n_b = p.n_new ? p.n_new[b] : p.n_tok;
  const int L = p.seq_lens[b];
  if (n_b < 0 || n_b > p.n_tok || L < n_b || L > p.max_seq) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, HATA_ERR_INVALID_ARG);
    return;
  }
  if (i >= n_b) return;
  const int slot = L - n_b + i;
  const size_t tok = (size_t)b * p.n_tok + i;
  const int pos = p.positions ? p.positions[tok] : slot;
  if (p.rot > 0 && (pos < 0 || pos >= p.n_pos)) {
    if (lane == 0) set_status(p.status, HATA_ERR_INVALID_ARG);
    return;
  }
  // the cache row of KV head 0; head g is `head_rows` * g rows on
  size_t row0, head_rows;
  bool stored = true;
  if constexpr (PAGED) {
    const int blk = p.block_table[(size_t)b * p.max_blocks + (slot >> p.block_shift)];
    stored = blk >= 0 && blk < p.n_blocks;
    if (!stored && lane == 0) set_status(p.status, HATA_ERR_INVALID_ARG);
    head_rows = (size_t)1 << p.block_shift;
    row0 = (((size_t)(stored ? blk : 0) * p.Hkv) << p.block_shift) + (size_t)(slot & ((1 << p.block_shift) - 1));
  } else {
    head_rows = (size_t)p.max_seq;
    row0 = (size_t)b * p.Hkv * p.max_seq + slot;
  }
  const int half = p.rot / 2, e0 = li * N;
  // this lane's cosines and sines; the partner of a half-split pair is `partner`, half a rotation away
  const bool turns = e0 < p.rot;
  const int partner = !turns || INTER ? lane : e0 < half ? lane + half / N : lane - half / N;
  const float* trow = p.table + (size_t)pos * p.rot;
  const int f0 = INTER ? e0 / 2 : (e0 < half ? e0 : e0 - half);

  const int first = sp * p.steps_per_warp * RPS;
  const int last = min(p.Hq + 2 * p.Hkv, first + p.steps_per_warp * RPS);
  // rows [lo, hi) of one kind: heads of x, normed with w (or not) and turned, to head h of dst at row stride
  // `dst_stride`.  With y = x r w, r the reciprocal root, a turned element is r (x (w c) + x' (w' s)), x' and w' its
  // partner's: two factors per element, made once per token.
  auto rows_of = [&](const void* x_in, size_t x_off, const float* w, int lo, int hi, void* dst, size_t dst_row,
                     size_t dst_stride, bool write) {
    if (lo >= hi) return;
    const T* x0 = static_cast<const T*>(x_in) + x_off + e0;
    T* d0 = static_cast<T*>(dst) + dst_row * kHeadDim + e0;
    float fa[N], fb[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float wk = w ? __ldg(w + e0 + k) : 1.f;
      fa[k] = wk;
      fb[k] = 0.f;
      if (turns) {
        const int f = INTER ? f0 + k / 2 : f0 + k;
        const float c = __ldg(trow + f), sn = __ldg(trow + half + f);
        const bool lead = INTER ? k % 2 == 0 : e0 < half;  // the first of its pair
        const int pe = INTER ? e0 + (k ^ 1) : (lead ? e0 + k + half : e0 + k - half);
        fa[k] = wk * c;
        fb[k] = (w ? __ldg(w + pe) : 1.f) * (lead ? -sn : sn);
      }
    }
    auto load = [&](int r0, uint4 (&v)[kRopeBatch]) {
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        const int r = r0 + u * RPS + sub;
        v[u] = r < hi ? __ldg(reinterpret_cast<const uint4*>(x0 + (size_t)r * kHeadDim)) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    uint4 in[kRopeBatch], nx[kRopeBatch];
    load(lo, nx);
    for (int r0 = lo; r0 < hi; r0 += kRopeBatch * RPS) {
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) in[u] = nx[u];
      load(r0 + kRopeBatch * RPS, nx);  // the next rows are under way while these are turned
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        float x[N];
        Vec16<T>::unpack(in[u], x);
        float rs = 1.f;
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int k = 0; k < N; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
          for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          rs = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
        }
        float y[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float other = INTER ? x[k ^ 1] : __shfl_sync(0xffffffffu, x[k], partner);
          y[k] = rs * (turns ? fmaf(x[k], fa[k], other * fb[k]) : x[k] * fa[k]);  // not turned: no 0 * infinity
        }
        const int r = r0 + u * RPS + sub;
        if (r < hi && write) *reinterpret_cast<uint4*>(d0 + (size_t)r * dst_stride * kHeadDim) = Vec16<T>::pack(y);
      }
    }
  };
  rows_of(p.q_in, tok * (size_t)p.q_stride, p.q_weight, first, min(last, p.Hq), p.q_out,
          (size_t)b * p.Hq * p.n_tok + i, p.n_tok, true);
  rows_of(p.k_in, tok * (size_t)p.k_stride, p.k_weight, max(first - p.Hq, 0), min(last - p.Hq, p.Hkv), p.K, row0,
          head_rows, stored);
  // values are copied
  const T* v = static_cast<const T*>(p.v_in) + tok * (size_t)p.v_stride + e0;
  const int v_lo = max(first - p.Hq - p.Hkv, 0), v_hi = last - p.Hq - p.Hkv;
  if (stored)
#pragma unroll 4
    for (int r = v_lo + sub; r < v_hi; r += RPS)
      *reinterpret_cast<uint4*>(static_cast<T*>(p.V) + (row0 + (size_t)r * head_rows) * kHeadDim + e0) =
          __ldg(reinterpret_cast<const uint4*>(v + (size_t)r * kHeadDim));
}

template <typename T, bool INTER>
void launch_rope_t(const RopeParams& prm, bool paged, dim3 grid, cudaStream_t st) {
  if (paged)
    norm_rope_kernel<T, INTER, true><<<grid, kRopeWarps * 32, 0, st>>>(prm);
  else
    norm_rope_kernel<T, INTER, false><<<grid, kRopeWarps * 32, 0, st>>>(prm);
}

// table[t][0][i] = cos(t * theta^(-2 i / rot)), table[t][1][i] = sin(..), the angle in fp64: at
// t = 131072 an fp32 angle would be off by up to 2^-8 radians.
__global__ void rope_table_kernel(float* __restrict__ table, int n_pos, int half, double theta) {
  const long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= (long long)n_pos * half) return;
  const int i = (int)(e % half);
  const long long t = e / half;
  const double angle = (double)t * pow(theta, -(double)i / (double)half);
  double s, c;
  sincos(angle, &s, &c);
  table[t * 2 * half + i] = (float)c;
  table[t * 2 * half + half + i] = (float)s;
}

}  // namespace

cudaError_t launch_rope_table(float* table, int n_pos, int rot, double theta, cudaStream_t st) {
  const long long n = (long long)n_pos * (rot / 2), blocks = (n + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  rope_table_kernel<<<(unsigned)blocks, 256, 0, st>>>(table, n_pos, rot / 2, theta);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope(const hata_dims_t& d, const RopeArgs& a, const PagedCache* pg, uint32_t* status,
                             cudaStream_t st) {
  RopeParams p{};
  p.q_in = a.q_in;
  p.k_in = a.k_in;
  p.v_in = a.v_in;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_weight = a.q_weight;
  p.k_weight = a.k_weight;
  p.table = a.table;
  p.n_new = a.n_new;
  p.positions = a.positions;
  p.seq_lens = a.seq_lens;
  p.q_out = a.q_out;
  p.K = a.K;
  p.V = a.V;
  p.status = status;
  p.eps = a.eps;
  p.n_tok = a.n_tok;
  p.Hq = d.n_q_heads;
  p.Hkv = d.n_kv_heads;
  p.max_seq = d.max_seq;
  p.n_pos = a.n_pos;
  p.rot = a.rot;
  if (pg) {
    p.block_table = pg->block_table;
    p.block_shift = pg->block_shift;
    p.n_blocks = pg->n_blocks;
    p.max_blocks = pg->max_blocks;
  }
  const int rps = d.dtype == HATA_BF16 ? 2 : 1;
  const int steps = (p.Hq + 2 * p.Hkv + rps - 1) / rps;
  p.tok_blocks = (p.n_tok + kRopeWarps - 1) / kRopeWarps;
  // A warp takes a whole token, so that positions, table and weights are fetched once for all its rows, unless
  // the tokens are too few to fill the SMs twice; then several warps share one, down to a batch of rows each.
  const long long fill = 2LL * kRopeCtas * kRopeWarps * span_sms(), tokens = (long long)d.batch * p.n_tok;
  const int most = (steps + kRopeBatch - 1) / kRopeBatch;
  p.n_split = (int)std::min<long long>(most, std::max<long long>(1, fill / tokens));
  p.steps_per_warp = (steps + p.n_split - 1) / p.n_split;
  const long long gx = (long long)p.tok_blocks * p.n_split;
  if (gx > 0x7fffffffLL || d.batch > 65535) return cudaErrorNotSupported;
  const dim3 grid((unsigned)gx, (unsigned)d.batch);
  if (d.dtype == HATA_BF16) {
    if (a.interleaved) launch_rope_t<__nv_bfloat16, true>(p, pg != nullptr, grid, st);
    else launch_rope_t<__nv_bfloat16, false>(p, pg != nullptr, grid, st);
  } else {
    if (a.interleaved) launch_rope_t<float, true>(p, pg != nullptr, grid, st);
    else launch_rope_t<float, false>(p, pg != nullptr, grid, st);
  }
  return cudaGetLastError();
}

}  // namespace hata
