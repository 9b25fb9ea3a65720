// Shared by the two forms of jolt_tree_attn's main kernel.
#pragma once
#include "common.cuh"
#include "pages.cuh"
#if defined(__CUDACC__)
#include "sm100.cuh"
#endif

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
  int n_new, n_q, gq, parts, batch, blocks, stages, stage_bytes;
  int splits;        // most splits of a sequence; the drafted tokens' part follows them
  int shares;        // blocks a (KV head, row block) has for all sequences' splits
  int least;         // tiles of a split at least
  int balanced;      // splits of equal size over all sequences (else `splits` of every sequence)
  uint32_t gq_magic;  // ceil(2^32 / gq)
  int perm;           // features of acc are in tree_tc.cu's order for this many value bits (0: their own order)
};

// Shared memory of the drafted tokens' part for blocks of `rows` query rows.
inline size_t draft_smem(int d_h, int rows, int threads) {
  const size_t cores = size_t(kMaxDraft) * (2 * d_h + 4) * 4 + size_t(rows) * d_h * 4 + size_t(threads / 32) * 4 * 64 * 4;
  const size_t mma = size_t(2 * kMaxDraft + (rows + 15) / 16 * 16) * (d_h + 8) * 2 + 8;
  return cores > mma ? cores : mma;
}

#if defined(__CUDACC__)
__device__ __forceinline__ int draft_count(const TreeArgs& a, int b) {
  return a.counts ? min(max(a.counts[b], 0), a.n_new) : a.n_new;
}
// Drafted token and head of the group of a query row.
__device__ __forceinline__ int row_token(const TreeArgs& a, int row) {
  return a.gq == 1 ? row : int(__umulhi(uint32_t(row), a.gq_magic));
}
// Element offset of a row from its KV head's first query row.
__device__ __forceinline__ int64_t q_offset(const TreeArgs& a, int row, int d) {
  const int t = row_token(a, row);
  return int64_t(t) * a.qst + (row - t * a.gq) * d;
}
// Row of out, lse, ml and acc.
__device__ __forceinline__ int64_t out_row(const TreeArgs& a, int b, int h, int row) {
  const int t = row_token(a, row);
  return (int64_t(b) * a.n_new + t) * a.n_q + h * a.gq + (row - t * a.gq);
}
// ---- how the pages' tokens are divided ----
// A (KV head, row block) has `shares` blocks for the tiles of all sequences (tree_plan says how many; where they
// only equal the sequences in number, each gets one split). Balanced: a split has c tiles, the
// least c (of a few) for which all sequences' splits number at most `shares`, so a ragged batch keeps every
// block equally long (lengths 64K, 56K, 48K, 40K: 23% over a division of each sequence by the same number).
// The lengths are on the device, so a warp works this out for itself; lane i has sequences 4 i .. + 3.
constexpr int kMaxBalanced = 128;  // sequences
struct Shares {
  int tiles[4], c;
};
// ceil(t / c) for t + c <= 2^21, rc = fl(1 / c): (t + c - 1/2) / c is 1 / (2 c) or more from a whole number, 2^-22 of
// itself, and the two roundings come to 2^-23.
__device__ __forceinline__ int ceil_div(int t, int c, float rc) { return int((float(t + c - 1) + 0.5f) * rc); }
template <int TILE>
__device__ __forceinline__ Shares shares_of(const TreeArgs& a, int lane) {
  Shares s;
  const int cap = a.p.max_pages << a.p.ps_log2;
  int sum = 0, top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = lane * 4 + i;
    const int raw = b < a.batch ? a.p.lens[b] : 0, len = min(max(raw, 0), cap);
    if (len != raw) report_error(a.err, JOLT_ERR_INVALID_ARG);
    s.tiles[i] = (len + TILE - 1) / TILE;
    sum += s.tiles[i];
    top = max(top, s.tiles[i]);
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  top = __reduce_max_sync(0xffffffffu, top);
  const int least = max(a.least, ceil_div(top, a.splits, __frcp_rn(float(a.splits))));
  // c = sum / (shares - k) does for some k <= batch: each sequence rounds up by less than one
  const int step = max(1, a.batch >> 3);
  for (int k = 0;; k += step) {
    const int left = max(a.shares - min(k, a.batch), 1);
    // sums that ceil_div does not take exactly: a little more than sum / left
    const float rl = __frcp_rn(float(left));
    s.c = max(least, sum < (1 << 20) ? ceil_div(sum, left, rl) : int(float(sum) * rl * 1.000001f) + 1);
    int n = 0;
    const float rc = __frcp_rn(float(s.c));
#pragma unroll
    for (int i = 0; i < 4; ++i) n += ceil_div(s.tiles[i], s.c, rc);
    if (k >= a.batch || int(__reduce_add_sync(0xffffffffu, n)) <= a.shares) return s;
  }
}
// What a block works on: a split's tiles, or the drafted tokens (split == splits; these blocks come last:
// they are short and fill the SMs that the splits leave).
struct Work {
  int b, h, block, split, tile0, n_tiles, len;
};
template <int TILE>
__device__ __forceinline__ bool work_of(const TreeArgs& a, Work* w) {
  const int heads = a.p.n_kv * a.blocks, lane = threadIdx.x & 31;
  int id = int(blockIdx.x) / heads;
  const int hb = int(blockIdx.x) - id * heads;
  w->h = hb / a.blocks;
  w->block = hb - w->h * a.blocks;
  w->tile0 = w->n_tiles = w->len = 0;
  if (id >= a.shares) {
    w->b = id - a.shares;
    w->split = a.splits;
    return true;
  }
  int c, tiles;
  if (a.balanced) {
    const Shares s = shares_of<TILE>(a, lane);
    int n[4], mine = 0;
    const float rc = __frcp_rn(float(s.c));
#pragma unroll
    for (int i = 0; i < 4; ++i) mine += n[i] = ceil_div(s.tiles[i], s.c, rc);
    int first = mine;  // splits before this lane's sequences
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, first, x);
      if (lane >= x) first += y;
    }
    first -= mine;
    int found = -1, split = 0, t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (id >= first && id < first + n[i]) found = lane * 4 + i, split = id - first, t = s.tiles[i];
      first += n[i];
    }
    const uint32_t who = __ballot_sync(0xffffffffu, found >= 0);
    if (!who) return false;  // more blocks than splits
    const int src = __ffs(who) - 1;
    w->b = __shfl_sync(0xffffffffu, found, src);
    w->split = __shfl_sync(0xffffffffu, split, src);
    tiles = __shfl_sync(0xffffffffu, t, src);
    c = s.c;
    w->len = pages_len(a.p, w->b, a.err);
  } else {
    w->b = id / a.splits;
    w->split = id - w->b * a.splits;
    w->len = pages_len(a.p, w->b, a.err);
    tiles = (w->len + TILE - 1) / TILE;
    c = (tiles + a.splits - 1) / a.splits;
  }
  w->tile0 = w->split * c;
  w->n_tiles = max(0, min(tiles, w->tile0 + c) - w->tile0);
  return true;
}
// Splits of sequence b (of which a partial result is there).
template <int TILE>
__device__ __forceinline__ int splits_of(const TreeArgs& a, int b, int lane) {
  if (!a.balanced) return a.splits;
  const Shares s = shares_of<TILE>(a, lane);
  const int i = b & 3;
  const int t = __shfl_sync(0xffffffffu, i == 0 ? s.tiles[0] : i == 1 ? s.tiles[1] : i == 2 ? s.tiles[2] : s.tiles[3], b >> 2);
  return (t + s.c - 1) / s.c;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// A warp's bounded wait for an mbarrier phase (false and JOLT_ERR_TIMEOUT after 2 s). A poll asks to be held
// for up to a millisecond, so that waiting warps leave the issue slots to the others, and the timer (whose
// read takes longer than most waits here) is read after a poll that came back empty only.
__device__ __forceinline__ bool wait_all(uint32_t bar, int parity, int32_t* err) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    const uint64_t now = sm100::global_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(0xffffffffu, now - t0 > 2000000000ull)) {
      report_error(err, JOLT_ERR_TIMEOUT);
      return false;
    }
  }
}

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
    qs[i] = ld_as_float(qb, q_offset(a, r, D) + f) * a.scale2;
  }
  __syncthreads();
  for (int q0 = warp * 4; q0 < rows; q0 += (THREADS / 32) * 4) {
    uint64_t bits[4];
    float s[4][2];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = row_token(a, r0 + q0 + r);
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
        const int64_t gr = out_row(a, b, h, row);
        a.ml[gr * a.parts + a.splits] = make_float2(mx, l);
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
        const int64_t gr = out_row(a, b, h, row);
        float* dst = a.acc + (gr * a.parts + a.splits) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[e] = o[r][e];
      }
    __syncwarp();
  }
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))));
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf2_pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The same for bf16 on m16n8k16 MMAs, 16 query rows a warp: q, k and v are bf16 as given, so the scores are
// exact products; p goes in as two bf16 terms (16 bits). A row that masks a token multiplies its values by 0,
// so values that are not finite are taken as 0 in the MMAs and added to the rows that see them.
template <int D, int RB, int THREADS>
__device__ void draft_mma(const TreeArgs& a, int b, int h, int r0, uint8_t* smem) {
  constexpr int LD = D + 8, RT = (RB + 15) / 16, V = D / 8;  // padded row; row tiles; 16-byte pieces of a row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, m = lane & 3;
  const int cnt = draft_count(a, b), keys = (cnt + 15) / 16 * 16;
  const int rows = min(RB, cnt * a.gq - r0);
  __nv_bfloat16* ks = reinterpret_cast<__nv_bfloat16*>(smem);  // [64][LD]
  __nv_bfloat16* vs = ks + kMaxDraft * LD;                     // [64][LD]
  __nv_bfloat16* qs = vs + kMaxDraft * LD;                     // [RT * 16][LD]
  const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(a.k) + int64_t(b) * a.ksb + int64_t(h) * D;
  const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(a.v) + int64_t(b) * a.ksb + int64_t(h) * D;
  const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.q) + int64_t(b) * a.qsb + int64_t(h) * a.gq * D;
  unsigned long long* bad = reinterpret_cast<unsigned long long*>(qs + RT * 16 * LD);  // tokens with such values
  if (tid == 0) *bad = 0;
  __syncthreads();
  for (int i = tid; i < keys * V; i += THREADS) {
    const int t = i / V, f = (i % V) * 8;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (t < cnt) {
      x = *reinterpret_cast<const uint4*>(kb + t * a.kst + f);
      y = *reinterpret_cast<const uint4*>(vb + t * a.kst + f);
    }
    *reinterpret_cast<uint4*>(ks + t * LD + f) = x;
    uint32_t w[4] = {y.x, y.y, y.z, y.w};
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((w[e] & 0x7F80u) == 0x7F80u) odd = true, w[e] &= 0xFFFF0000u;
      if ((w[e] & 0x7F800000u) == 0x7F800000u) odd = true, w[e] &= 0xFFFFu;
    }
    if (odd) atomicOr(bad, 1ull << t);
    *reinterpret_cast<uint4*>(vs + t * LD + f) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const int tiles = (rows + 15) / 16;
  for (int i = tid; i < tiles * 16 * V; i += THREADS) {
    const int r = i / V, f = (i % V) * 8, row = r0 + r;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < rows) x = *reinterpret_cast<const uint4*>(qb + q_offset(a, row, D) + f);
    *reinterpret_cast<uint4*>(qs + r * LD + f) = x;
  }
  __syncthreads();
  const uint64_t not_finite = *bad;
  for (int rt = warp; rt < tiles; rt += THREADS / 32) {
    float s[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[nt][c] = 0.f;
#pragma unroll 2
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t q[4];
      ldsm4(q, qs + (rt * 16 + (lane & 15)) * LD + kk * 16 + (lane >> 4) * 8);
#pragma unroll
      for (int nt = 0; nt < 8; nt += 2)
        if (nt * 8 < keys) {
          uint32_t k[4];
          ldsm4(k, ks + (nt * 8 + (lane & 7) + (lane >> 4) * 8) * LD + kk * 16 + ((lane >> 3) & 1) * 8);
          mma_bf16_16816(s[nt], q, k[0], k[1]);
          mma_bf16_16816(s[nt + 1], q, k[2], k[3]);
        }
    }
    uint32_t ph[4][4], pl[4][4];
    uint64_t extra[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {  // rows g and g + 8
      const int r = rt * 16 + g + 8 * x, i = row_token(a, r0 + r);
      uint64_t bits = 0;
      if (r < rows) bits = a.mask ? a.mask[int64_t(b) * a.n_new + i] : ~uint64_t(0) >> (63 - i);
      if (cnt < 64) bits &= (uint64_t(1) << cnt) - 1;
      extra[x] = bits & not_finite;
      bits >>= 2 * m;
      float mx = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float& v = s[nt][2 * x + c];
          v = (bits >> (8 * nt + c)) & 1 ? v * a.scale2 : -INFINITY;
          mx = fmaxf(mx, v);
        }
#pragma unroll
      for (int y = 1; y <= 2; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
      const float ref = mx == -INFINITY ? 0.f : mx;
      float l = 0.f;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        float p[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          p[c] = (bits >> (8 * nt + c)) & 1 ? exp2f(s[nt][2 * x + c] - ref) : 0.f;
          l += p[c];
        }
        const uint32_t hi = bf2_pack(p[0], p[1]);
        ph[nt >> 1][x + 2 * (nt & 1)] = hi;
        pl[nt >> 1][x + 2 * (nt & 1)] = bf2_pack(p[0] - __uint_as_float(hi << 16), p[1] - __uint_as_float(hi & 0xFFFF0000u));
      }
#pragma unroll
      for (int y = 1; y <= 2; y <<= 1) l += __shfl_xor_sync(0xffffffffu, l, y);
      if (r < rows && m == 0) {
        a.ml[out_row(a, b, h, r0 + r) * a.parts + a.splits] = make_float2(mx, l);
      }
    }
    float* dst[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rt * 16 + g + 8 * x, row = r0 + r;
      dst[x] = r < rows ? a.acc + (out_row(a, b, h, row) * a.parts + a.splits) * D
                        : nullptr;
    }
#pragma unroll 2
    for (int f = 0; f < D; f += 16) {
      float o[2][4] = {};
#pragma unroll
      for (int kg = 0; kg < 4; ++kg)
        if (kg * 16 < keys) {
          uint32_t v[4];  // keys kg*16 .. + 15, features f .. + 15
          ldsm4_trans(v, vs + (kg * 16 + (lane & 15)) * LD + f + (lane >> 4) * 8);
          mma_bf16_16816(o[0], ph[kg], v[0], v[1]);
          mma_bf16_16816(o[0], pl[kg], v[0], v[1]);
          mma_bf16_16816(o[1], ph[kg], v[2], v[3]);
          mma_bf16_16816(o[1], pl[kg], v[2], v[3]);
        }
      if (not_finite) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          for (uint64_t left = extra[x]; left; left &= left - 1) {
            const __nv_bfloat16* v = vb + int64_t(__ffsll(left) - 1) * a.kst + f + 2 * m;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = __bfloat162float(v[(e >> 1) * 8 + (e & 1)]);
              if (!(fabsf(y) < INFINITY)) o[e >> 1][2 * x + (e & 1)] += y;
            }
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (dst[x]) {
          *reinterpret_cast<float2*>(dst[x] + f + 2 * m) = make_float2(o[0][2 * x], o[0][2 * x + 1]);
          *reinterpret_cast<float2*>(dst[x] + f + 8 + 2 * m) = make_float2(o[1][2 * x], o[1][2 * x + 1]);
        }
    }
  }
}

template <typename T, int D, int RB, int THREADS>
__device__ __forceinline__ void draft_part(const TreeArgs& a, int b, int h, int r0, uint8_t* smem) {
  if (draft_count(a, b) * a.gq <= r0) return;
  if constexpr (sizeof(T) == 2) draft_mma<D, RB, THREADS>(a, b, h, r0, smem);
  else draft_block<T, D, RB, THREADS>(a, b, h, r0, smem);
}
#endif

// The form for bf16 and more than 16 query rows a KV head (tree_tc.cu).
size_t tree_tc_smem(int d_h);
// Place of feature f in a row of that form's code tiles (in elements) when its codes have 2^lnc a word:
// quarter row m, piece i of it (pairs 4i .. 4i+3 of code_pair's order), at piece i * 4 + m.
#if defined(__CUDACC__)
__device__ __forceinline__ int place_of(int f, int lnc, int D) {
  const int m = f / (D / 4), fq = f % (D / 4), half = 1 << (lnc - 1);
  const int c = fq & (2 * half - 1), pair = ((fq >> lnc) << (lnc - 1)) + (c & (half - 1));
  return ((pair >> 2) * 4 + m) * 8 + (pair & 3) * 2 + (c >> (lnc - 1));
}
__device__ __forceinline__ int log2_codes(int bits) { return bits == 2 ? 4 : bits == 4 ? 3 : 2; }
#endif
jolt_status launch_tree_tc(const TreeArgs& a, int d_h, bool draft, size_t smem, cudaStream_t st);

}  // namespace jolt
