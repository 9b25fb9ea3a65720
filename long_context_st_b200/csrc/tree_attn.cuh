// Shared by the two forms of jolt_tree_attn's main kernel.
#pragma once
#include "common.cuh"
#include "pages.cuh"

namespace jolt {

constexpr int kMaxDraft = 64;  // bits of a mask word

struct TreeArgs {
  PagesDev p;
  const void* q;
  const void* k;
  const void* v;
  int64_t qsb, qst, ksb, kst;
  const int32_t* counts;
  const uint64_t* mask;
  const void* prefix_out;
  const float* prefix_lse;
  void* out;
  float* lse;
  float2* ml;   // [rows][parts] (maximum in log2 units, sum)
  float* acc;   // [rows][parts][D]
  int32_t* err;
  float scale2;  // attn_scale * log2(e): scores are kept in log2 units
  int n_new, n_q, gq, splits, parts, batch, blocks, stages, stage_bytes;
  int cached;  // partial results of the pages (splits, or two a split); the drafted tokens' follows them
};

#if defined(__CUDACC__)
__device__ __forceinline__ int draft_count(const TreeArgs& a, int b) {
  return a.counts ? min(max(a.counts[b], 0), a.n_new) : a.n_new;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }
__device__ __forceinline__ uint32_t trans8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2_pack(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 h2_floats(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// The drafted tokens' own keys and values, in fp32 on the CUDA cores (at most 64 keys).
template <typename T, int D, int RB, int THREADS>
__device__ void draft_block(const TreeArgs& a, int b, int h, int r0, uint8_t* smem) {
  constexpr int E = D / 32, KS = D + 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cnt = draft_count(a, b);
  const int rows = min(RB, cnt * a.gq - r0);
  if (rows <= 0) return;
  float* ks = reinterpret_cast<float*>(smem);           // [cnt][KS]
  float* vs = ks + kMaxDraft * KS;                      // [cnt][D]
  float* qs = vs + kMaxDraft * D;                       // [RB][D]
  float* ps = qs + RB * D;                              // [warp][4][64]
  const T* kb = static_cast<const T*>(a.k) + int64_t(b) * a.ksb + int64_t(h) * D;
  const T* vb = static_cast<const T*>(a.v) + int64_t(b) * a.ksb + int64_t(h) * D;
  for (int i = tid; i < cnt * D; i += THREADS) {
    const int t = i / D, f = i % D;
    ks[t * KS + f] = ld_as_float(kb, t * a.kst + f);
    vs[t * D + f] = ld_as_float(vb, t * a.kst + f);
  }
  const T* qb = static_cast<const T*>(a.q) + int64_t(b) * a.qsb + int64_t(h) * a.gq * D;
  for (int i = tid; i < rows * D; i += THREADS) {
    const int r = r0 + i / D, f = i % D;
    qs[i] = ld_as_float(qb, int64_t(r / a.gq) * a.qst + (r % a.gq) * D + f) * a.scale2;
  }
  __syncthreads();
  for (int q0 = warp * 4; q0 < rows; q0 += (THREADS / 32) * 4) {
    uint64_t bits[4];
    float s[4][2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = (r0 + q0 + r) / a.gq;
      bits[r] = 0;
      if (q0 + r < rows) bits[r] = a.mask ? a.mask[int64_t(b) * a.n_new + i] : ~uint64_t(0) >> (63 - i);
      if (cnt < 64) bits[r] &= (uint64_t(1) << cnt) - 1;
      s[r][0] = s[r][1] = 0.f;
    }
    const int j1 = min(lane, cnt - 1), j2 = min(lane + 32, cnt - 1);
    for (int f = 0; f < D; f += 4) {
      const float4 k1 = *reinterpret_cast<const float4*>(ks + j1 * KS + f);
      const float4 k2 = *reinterpret_cast<const float4*>(ks + j2 * KS + f);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(qs + min(q0 + r, rows - 1) * D + f);
        s[r][0] += x.x * k1.x + x.y * k1.y + x.z * k1.z + x.w * k1.w;
        s[r][1] += x.x * k2.x + x.y * k2.y + x.z * k2.z + x.w * k2.w;
      }
    }
    float o[4][E];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool v1 = (bits[r] >> lane) & 1, v2 = (bits[r] >> (lane + 32)) & 1;
      const float s1 = v1 ? s[r][0] : -INFINITY, s2 = v2 ? s[r][1] : -INFINITY;
      const float mx = warp_max(fmaxf(s1, s2));
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float p1 = v1 ? exp2f(s1 - ref) : 0.f, p2 = v2 ? exp2f(s2 - ref) : 0.f;
      const float l = warp_sum(p1 + p2);
      ps[(warp * 4 + r) * 64 + lane] = p1;
      ps[(warp * 4 + r) * 64 + lane + 32] = p2;
      if (lane == 0 && q0 + r < rows) {
        const int row = r0 + q0 + r;
        const int64_t gr = (int64_t(b) * a.n_new + row / a.gq) * a.n_q + h * a.gq + row % a.gq;
        a.ml[gr * a.parts + a.cached] = make_float2(mx, l);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    __syncwarp();
    for (int j = 0; j < cnt; ++j) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = vs[j * D + lane * E + e];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if ((bits[r] >> j) & 1) {  // a masked row of v is not touched: it may hold anything
          const float p = ps[(warp * 4 + r) * 64 + j];
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] += p * v[e];
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (q0 + r < rows) {
        const int row = r0 + q0 + r;
        const int64_t gr = (int64_t(b) * a.n_new + row / a.gq) * a.n_q + h * a.gq + row % a.gq;
        float* dst = a.acc + (gr * a.parts + a.cached) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[e] = o[r][e];
      }
    __syncwarp();
  }
}

#endif

// The form for bf16 and more than 32 query rows a KV head (tree_tc.cu).
size_t tree_tc_smem(int d_h);
jolt_status launch_tree_tc(const TreeArgs& a, int d_h, bool draft, size_t smem, cudaStream_t st);

}  // namespace jolt
