// jolt_rope: rotary positions of queries and keys.
#include <algorithm>

#include "common.cuh"
#include "stats.h"
#include "vec.cuh"

namespace jolt {
namespace {

struct RopeTensor {
  const void* x;
  void* y;
  int64_t sx, sy;  // elements per token
  int heads;
};
struct RopeArgs {
  RopeTensor t[2];
  const int32_t* pos;
  const float* inv_freq;
  int64_t n_tokens;
  float scaling;
  int d, rot, tb, inverse;
  int rows_at;      // k_rope_vec: rows a thread takes (of kRows)
  uint32_t magic;   // ceil(2^32 / heads)
};

constexpr int kThreads = 256;

// (cos, sin) of pos * inv_freq[i] for the block's tokens into cs[token][pair]. The angle is taken in
// turns in double precision (a float32 product at position 10^5 is off by up to 4e-3 rad), reduced
// to half a turn either way, and only then rounded.
__device__ __forceinline__ void rope_table(const RopeArgs& a, int64_t t0, int nt, float2* cs) {
  const int half = a.rot >> 1;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    double turns = double(a.pos[t0 + t]) * double(a.inv_freq[p]) * 0.15915494309189533577;
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * float(turns), &s, &c);
    cs[i] = make_float2(c * a.scaling, (a.inverse ? -s : s) * a.scaling);
  }
  __syncthreads();
}

// Bound by HBM: every element is read and written once. Four rows of loads in flight a thread: 8192 tokens of
// 64 + 8 heads of 128 in bf16 take 59.6 us (302 MB, 5.1 TB/s), 5003 tokens of 32 + 8 heads in fp32 34.9 us
// (205 MB, 5.9 TB/s). What bf16 lacks to the copy rate is latency: the table (double precision, once a block) and
// the loads of a block are waited for one after the other at 34% of the warps an SM holds (75 registers).
//
// One pass over q and k, whose heads are taken as one run of (token, head) rows: a thread turns the 16-byte
// pieces of one place in the head for up to kRows rows, with all their loads in flight; half layout, a
// piece of each half; interleaved, one piece of whole pairs. Pieces past rot_dim are copied. The block's
// tokens' table is formed once for all their heads. x and y may be the same memory: every piece is read and
// written by one thread.
constexpr int kRows = 4;
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rope_vec(const RopeArgs a) {
  constexpr int V = 16 / sizeof(T);
  extern __shared__ float2 cs[];
  const int half = a.rot >> 1;
  const int rot_units = HALF ? half / V : a.rot / V;
  const int units = rot_units + (a.d - a.rot) / V;  // pieces of a head, at most 128
  const uint32_t heads = a.t[0].heads + a.t[1].heads;
  const int at_once = kThreads / units, rr = threadIdx.x / units, u = threadIdx.x - rr * units;
  const uint64_t first = uint64_t(blockIdx.x) * (at_once * a.rows_at), total = uint64_t(a.n_tokens) * heads;
  const int rows = int(total - first < uint64_t(at_once * a.rows_at) ? total - first : at_once * a.rows_at);
  const int64_t t0 = first / heads;
  const uint32_t h0 = uint32_t(first - t0 * heads);
  // token of the block's x-th row, counted from t0's first head: at most 1024 rows, so one of two tokens
  // where there are more heads
  auto token = [&](uint32_t x) -> int { return heads == 1 ? x : heads > 1024 ? x >= heads : __umulhi(x, a.magic); };
  const bool turn = u < rot_units;
  const int at = turn ? u * V : a.rot + (u - rot_units) * V;
  uint4 pa[kRows], pb[kRows];
  T* dst[kRows];
  int tok[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = rr + i * at_once;
    tok[i] = -1;
    if (i >= a.rows_at || row >= rows || rr >= at_once) continue;
    const uint32_t x = h0 + row;
    tok[i] = token(x);
    uint32_t h = x - tok[i] * heads;
    const int which = h >= uint32_t(a.t[0].heads);
    const RopeTensor& y = a.t[which];
    if (which) h -= a.t[0].heads;
    const T* src = static_cast<const T*>(y.x) + (t0 + tok[i]) * y.sx + int64_t(h) * a.d + at;
    dst[i] = static_cast<T*>(y.y) + (t0 + tok[i]) * y.sy + int64_t(h) * a.d + at;
    pa[i] = *reinterpret_cast<const uint4*>(src);
    if (HALF && turn) pb[i] = *reinterpret_cast<const uint4*>(src + half);
  }
  rope_table(a, t0, token(h0 + rows - 1) + 1, cs);  // under the loads
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (tok[i] < 0) continue;
    if (!turn) {
      *reinterpret_cast<uint4*>(dst[i]) = pa[i];
      continue;
    }
    const float2* c = cs + tok[i] * half;
    float p[V], y[V];
    unpack16<T>(pa[i], p);
    if (HALF) {
      float q[V], z[V];
      unpack16<T>(pb[i], q);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 f = c[u * V + j];
        y[j] = p[j] * f.x - q[j] * f.y;
        z[j] = q[j] * f.x + p[j] * f.y;
      }
      *reinterpret_cast<uint4*>(dst[i] + half) = pack16<T>(z);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 f = c[u * (V / 2) + j];
        y[2 * j] = p[2 * j] * f.x - p[2 * j + 1] * f.y;
        y[2 * j + 1] = p[2 * j + 1] * f.x + p[2 * j] * f.y;
      }
    }
    *reinterpret_cast<uint4*>(dst[i]) = pack16<T>(y);
  }
}

// The same, one pair (or one copied pair) a thread: head sizes, strides or addresses that 16-byte
// pieces do not divide.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rope_any(const RopeArgs a) {
  extern __shared__ float2 cs[];
  const int64_t t0 = int64_t(blockIdx.x) * a.tb;
  const int nt = int(a.n_tokens - t0 < a.tb ? a.n_tokens - t0 : a.tb);
  rope_table(a, t0, nt, cs);
  const int half = a.rot >> 1, pairs = a.d >> 1;
  const int heads = a.t[0].heads + a.t[1].heads;
  const int total = nt * heads * pairs;
  for (int i = threadIdx.x; i < total; i += kThreads) {
    const int row = i / pairs, u = i - row * pairs;
    const int t = row / heads;
    int h = row - t * heads;
    const int which = h >= a.t[0].heads;
    const RopeTensor& x = a.t[which];
    if (which) h -= a.t[0].heads;
    const T* src = static_cast<const T*>(x.x) + (t0 + t) * x.sx + int64_t(h) * a.d;
    T* dst = static_cast<T*>(x.y) + (t0 + t) * x.sy + int64_t(h) * a.d;
    if (u >= half) {
      const T p = src[2 * u], q = src[2 * u + 1];
      dst[2 * u] = p;
      dst[2 * u + 1] = q;
      continue;
    }
    const int ia = HALF ? u : 2 * u, ib = HALF ? u + half : 2 * u + 1;
    const float p = ld_as_float(src, ia), q = ld_as_float(src, ib);
    const float2 f = cs[t * half + u];
    st_from_float(dst, ia, p * f.x - q * f.y);
    st_from_float(dst, ib, q * f.x + p * f.y);
  }
}

template <typename T>
jolt_status launch_rope(RopeArgs a, bool half, bool vec, cudaStream_t st) {
  const int heads = a.t[0].heads + a.t[1].heads, pairs = a.rot / 2;
  const double bytes = double(a.n_tokens) * (2.0 * heads * a.d * sizeof(T) + 4.0);
  if (vec) {
    constexpr int V = 16 / sizeof(T);
    const int units = (half ? pairs : a.rot) / V + (a.d - a.rot) / V, at_once = kThreads / units;
    // the table of a block's tokens within the shared memory that every launch has
    a.rows_at = kRows;
    while (a.rows_at > 1 && (a.rows_at * at_once / heads + 2) * pairs * int(sizeof(float2)) > 48 * 1024) --a.rows_at;
    a.magic = uint32_t(((uint64_t(1) << 32) + heads - 1) / heads);
    const int rows = a.rows_at * at_once;
    const int64_t total = a.n_tokens * heads, grid = (total + rows - 1) / rows;
    if (grid > 0x7fffffff) return JOLT_ERR_INVALID_ARG;
    const size_t smem = size_t(std::min<int64_t>(rows / heads + 2, a.n_tokens)) * pairs * sizeof(float2);
    StatScope sc(JOLT_K_ROPE, st, 0.0, bytes);
    if (half) k_rope_vec<T, true><<<unsigned(grid), kThreads, smem, st>>>(a);
    else k_rope_vec<T, false><<<unsigned(grid), kThreads, smem, st>>>(a);
  } else {
    const unsigned grid = unsigned((a.n_tokens + a.tb - 1) / a.tb);
    const size_t smem = size_t(a.tb) * pairs * sizeof(float2);
    StatScope sc(JOLT_K_ROPE, st, 0.0, bytes);
    if (half) k_rope_any<T, true><<<grid, kThreads, smem, st>>>(a);
    else k_rope_any<T, false><<<grid, kThreads, smem, st>>>(a);
  }
  JOLT_CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

}  // namespace
}  // namespace jolt

using namespace jolt;

extern "C" jolt_status jolt_rope(const void* q, void* q_out, int32_t n_q, int64_t q_stride, int64_t q_out_stride,
                                 const void* k, void* k_out, int32_t n_kv, int64_t k_stride, int64_t k_out_stride,
                                 int64_t n_tokens, int32_t d_h, int32_t rot_dim, int32_t layout, const int32_t* pos,
                                 const float* inv_freq, float scaling, int32_t inverse, int32_t io_dtype,
                                 void* stream) {
  if (n_q < 0 || n_kv < 0 || n_q > 65536 || n_kv > 65536 || n_q + n_kv < 1 || n_tokens < 0)
    return JOLT_ERR_INVALID_ARG;
  if (d_h < 2 || d_h > 512 || d_h % 2 || rot_dim < 2 || rot_dim > d_h || rot_dim % 2) return JOLT_ERR_INVALID_ARG;
  if (layout != JOLT_ROPE_HALF && layout != JOLT_ROPE_INTERLEAVED) return JOLT_ERR_INVALID_ARG;
  if (io_dtype != JOLT_F32 && io_dtype != JOLT_BF16) return JOLT_ERR_INVALID_ARG;
  if (!(scaling - scaling == 0.f) || (inverse != 0 && inverse != 1)) return JOLT_ERR_INVALID_ARG;
  if (n_tokens == 0) return JOLT_OK;
  if (!pos || !inv_freq || (n_q && (!q || !q_out)) || (n_kv && (!k || !k_out))) return JOLT_ERR_INVALID_ARG;
  if (n_tokens > (int64_t(1) << 31) || reinterpret_cast<uintptr_t>(pos) % 4 || reinterpret_cast<uintptr_t>(inv_freq) % 4)
    return JOLT_ERR_INVALID_ARG;
  RopeArgs a{};
  a.t[0] = RopeTensor{q, q_out, q_stride, q_out_stride, n_q};
  a.t[1] = RopeTensor{k, k_out, k_stride, k_out_stride, n_kv};
  const int e = io_dtype == JOLT_F32 ? 4 : 2, v = 16 / e;
  bool vec = (layout == JOLT_ROPE_HALF ? rot_dim / 2 : rot_dim) % v == 0 && d_h % v == 0;
  for (const RopeTensor& t : a.t) {
    if (!t.heads) continue;
    const uintptr_t x = reinterpret_cast<uintptr_t>(t.x), y = reinterpret_cast<uintptr_t>(t.y);
    if (t.sx < int64_t(t.heads) * d_h || t.sy < int64_t(t.heads) * d_h || x % e || y % e) return JOLT_ERR_INVALID_ARG;
    if (x == y && t.sx != t.sy && n_tokens > 1) return JOLT_ERR_INVALID_ARG;
    vec = vec && x % 16 == 0 && y % 16 == 0 && t.sx % v == 0 && t.sy % v == 0;
  }
  a.pos = pos;
  a.inv_freq = inv_freq;
  a.n_tokens = n_tokens;
  a.scaling = scaling;
  a.d = d_h;
  a.rot = rot_dim;
  a.inverse = inverse;
  // several tokens a block once there are blocks enough for every SM
  a.tb = int(std::min<int64_t>(4, std::max<int64_t>(1, n_tokens / (kSmCount * 8))));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return io_dtype == JOLT_F32 ? launch_rope<float>(a, layout == JOLT_ROPE_HALF, vec, st)
                              : launch_rope<__nv_bfloat16>(a, layout == JOLT_ROPE_HALF, vec, st);
}
