// jolt_tree_attn: attention of drafted tokens over the tail cache's pages.
//
// With y = R k the stored (rotated) key, q.k = (R q).y, and y_j = scale * c_j + zero with whole
// codes c_j, so a score needs one product of (R q) with the codes themselves:
//   s = scale * ((R q).(c - o)) + (zero + o * scale) * sum(R q),   o = 2^(b-1) (codes centred at 0).
// The same for values: sum_t p_t y_t = sum_t (p_t scale_t) (c_t - o) + sum_t p_t (zero_t + o scale_t),
// whose second term is one number for all features; R^T is applied once, to the sum.
//
// A code's field is a whole number c 2^-24 as the bits of an f16 (a subnormal; its place in the byte a
// further power of two), so codes feed m16n8k16 MMAs after one mask a pair. The places' powers are taken
// from R q (keys) and from the outputs (values); o and the zeros enter through sums: o sum(R q) in the
// scores, and for the values a further MMA row of ones, which adds up p * scale exactly as rounded.
// The MMA aligns a subnormal's product by f16's least exponent, which costs the sum about 10 - b bits of its
// 24: against 64 bits the outputs of fp32 were off by 5e-6 (8 bits) to 3e-4 (2 bits), and the log-sum-exp
// of 2-bit keys by 3e-6. So fp32, and 2-bit keys, take one more operation a pair: c - o as normal numbers.
// What is rounded is the other operand: R q is carried as two f16 terms (22 bits: the log-sum-exp stays
// fp32-accurate), p * scale as one f16 term for bf16 output (11 bits, against the 8 the output keeps) and
// as two for fp32. Both are first scaled by powers of two into f16's normal range: R q by the block's
// largest element, p * scale by the largest value scale met so far.
#include <cuda.h>

#include <algorithm>

#include "pages_codes.cuh"
#include "sm100.cuh"
#include "stats.h"
#include "tree_attn.cuh"
#include "vec.cuh"

namespace jolt {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;        // tokens a warp takes at a time
constexpr int kMaxSplits = 63;   // + the drafted tokens' own partial: two per lane in the merge
constexpr int kMaxStages = 4;
// References (see k_tree): room above a row's maximum when one is set, what a thread's four p of a tile may add
// up to, and the power of two p * scale is carried with (times 2^-ve), so that it stays below 2^15. fp32
// output takes less room: its second f16 term of p * scale must not run out of f16's range below.
template <typename T>
struct Ref {
  static constexpr float room = sizeof(T) == 4 ? 1.f : 4.f, most = sizeof(T) == 4 ? 8.f : 256.f;
  static constexpr int p_exp = sizeof(T) == 4 ? 12 : 7;
};

// Keys of one tile: acc[grp][nt] += fields (tokens grp*16 + {g, g+8}) x R q (columns of tile nt).
template <int D, int B, int NT, int QT, bool NORMAL>
__device__ __forceinline__ void keys_tile(const uint8_t* kc, const uint2* qf, int lane, float (&s)[2][NT][4]) {
  constexpr int W = D * B / 128;  // words of a lane's quarter row
  const int g = lane >> 2, m = lane & 3;
  uint32_t w[4][W];  // rows g, g+8, g+16, g+24
#pragma unroll
  for (int r = 0; r < 4; ++r) load_words<W>(kc + (g + 8 * r) * (D * B / 8) + m * (4 * W), w[r]);
#pragma unroll
  for (int st = 0; st < D / 16; ++st) {
    uint32_t a0[4], a1[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      a0[2 * x] = NORMAL ? code_pair<B, W>(w[0], 2 * st + x) : field_pair<B, W>(w[0], 2 * st + x);
      a0[2 * x + 1] = NORMAL ? code_pair<B, W>(w[1], 2 * st + x) : field_pair<B, W>(w[1], 2 * st + x);
      a1[2 * x] = NORMAL ? code_pair<B, W>(w[2], 2 * st + x) : field_pair<B, W>(w[2], 2 * st + x);
      a1[2 * x + 1] = NORMAL ? code_pair<B, W>(w[3], 2 * st + x) : field_pair<B, W>(w[3], 2 * st + x);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        const uint2 b = qf[((t * NT + nt) * (D / 16) + st) * 32 + lane];
        mma_f16_16816(s[0][nt], a0, b.x, b.y);
        mma_f16_16816(s[1][nt], a1, b.x, b.y);
      }
  }
}

// Values of one tile: o[mt][nt] += fields^T (features) x (p scale) (tokens), PT terms of the latter; o[D / 16]
// the sum of p scale (a row of ones; not with NORMAL, whose codes are centred).
template <int D, int B, int NT, int PT, bool NORMAL>
__device__ __forceinline__ void values_tile(const uint8_t* vc, const uint32_t (&pf)[PT][2][NT][2], int lane,
                                            float (&o)[D / 16 + 1][NT][4]) {
  constexpr int CB = D * B / 64;             // bytes of a lane's eighth row
  constexpr int W = CB >= 4 ? CB / 4 : 1;
  const int g = lane >> 2, m = lane & 3;
  const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
#pragma unroll
  for (int grp = 0; grp < 2; ++grp) {
    uint32_t w[4][W];  // tokens 2m, 2m+1, 2m+8, 2m+9
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* src = vc + (grp * 16 + 2 * m + (r & 1) + (r >> 1) * 8) * (D * B / 8) + g * CB;
      if constexpr (CB == 2) w[r][0] = *reinterpret_cast<const uint16_t*>(src);
      else load_words<W>(src, w[r]);
    }
#pragma unroll
    for (int mt = 0; mt < D / 16 + (NORMAL ? 0 : 1); ++mt) {
      uint32_t a[4];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        a[f] = mt == D / 16 ? ones[f] : NORMAL ? code_across<B, W>(w[0], w[1], 2 * mt + f) : field_across<B, W>(w[0], w[1], 2 * mt + f);
        a[f + 2] = mt == D / 16 ? ones[f] : NORMAL ? code_across<B, W>(w[2], w[3], 2 * mt + f) : field_across<B, W>(w[2], w[3], 2 * mt + f);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int t = 0; t < PT; ++t) mma_f16_16816(o[mt][nt], a, pf[t][grp][nt][0], pf[t][grp][nt][1]);
    }
  }
}

// Scores, online softmax and values of one split of a sequence's pages for one KV head and up to RB
// query rows (drafted token x head of the group). The MMAs have tokens (keys) or features (values)
// as their 16 rows and query rows as their 8 columns, so single-token decoding wastes little; with
// PACK (at most 4 rows) columns 0-3 carry the first term of R q and 4-7 the second, and the values
// the two terms of p likewise. Each warp takes 32-token tiles of its own through a ring of bulk
// copies (one mbarrier a stage); the warps meet at the end, to add up their partial results.
// Bound by latency: some 385 instructions for 16 tokens of both kinds at 4 bits (codes to operands, MMAs that fill 4
// of 8 columns, one softmax over 32 tokens at a time) are one chain a warp, four warps a scheduler; and by some
// 10 us of launch, first loads and merge. One token of four sequences of 64K to 40K, 8 KV heads, takes 65.7 us with the merge (232 MB, 3.5 TB/s; each further token
// costs what 4.4 TB/s would), issue slots 60% busy at two blocks of 126 registers an SM.
template <typename T, int D, int NT, bool PACK>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) k_tree(const TreeArgs a) {
  using namespace sm100;
  constexpr int RB = PACK ? 4 : 8 * NT;
  constexpr int QT = PACK ? 1 : 2;
  constexpr int PT = !PACK && sizeof(T) == 4 ? 2 : 1;
  constexpr int E = D / 32, NS = D / 16, C = 8 * NT;
  constexpr bool kWhole = sizeof(T) == 4;       // codes as normal numbers
  const bool k_whole = kWhole || a.p.bk == 2;  // keys' codes
  extern __shared__ __align__(128) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, m = lane & 3;
  Work wk;
  if (!work_of<kTile>(a, &wk)) return;
  const int h = wk.h, r0 = wk.block * RB, b = wk.b, split = wk.split;
  if (split == a.splits) {
    draft_part<T, D, RB, kThreads>(a, b, h, r0, smem);
    return;
  }
  const int cnt = draft_count(a, b);
  const int rows = min(RB, cnt * a.gq - r0);
  if (rows <= 0) return;

  // this warp's rows of q, on their way while the first tiles are asked for
  constexpr int kPer = (RB + kWarps - 1) / kWarps;
  float v[kPer][E];
  {
    const T* qb = static_cast<const T*>(a.q) + int64_t(b) * a.qsb + int64_t(h) * a.gq * D;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = warp + i * kWarps;
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = 0.f;
      if (r < rows) {
        const T* x = qb + q_offset(a, r0 + r, D) + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = ld_as_float(x, e);
      }
    }
  }

  uint2* qf = reinterpret_cast<uint2*>(smem);                        // [QT][NT][NS][32]
  float* qsum = reinterpret_cast<float*>(qf + QT * NT * NS * 32);    // [C]
  float* xm = qsum + C;                                              // [kWarps][C]
  float* xl = xm + kWarps * C;                                       // [kWarps][C]
  float* xz = xl + kWarps * C;                                       // [kWarps][C]
  uint64_t* bars = reinterpret_cast<uint64_t*>(xz + kWarps * C);     // [kWarps][kMaxStages]
  uint32_t* there = reinterpret_cast<uint32_t*>(bars + kWarps * kMaxStages);  // pieces of a stage that hold tokens
  uint8_t* ring0 = reinterpret_cast<uint8_t*>(there + kWarps * kMaxStages);

  const int len = wk.len, t_first = wk.tile0 + warp, t_end = wk.tile0 + wk.n_tiles;
  const int n_mine = t_first < t_end ? (t_end - t_first + kWarps - 1) / kWarps : 0;
  const int rbk = D * a.p.bk / 8, rbv = D * a.p.bv / 8;
  uint8_t* ring = ring0 + warp * a.stages * a.stage_bytes;
  uint32_t bar0 = smem_u32(bars + warp * kMaxStages);
  if (lane == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();

  // A tile spans one or two pages (pieces); lane 4 piece + kind copies kind's rows of its piece. The table
  // entry is read a fetch early.
  const int ps = 1 << a.p.ps_log2, pt = min(kTile, ps);
  const int piece = lane >> 2, kind = lane & 3;
  const bool copies = piece * pt < kTile;
  const uint32_t rb = kind == 0 ? rbk : kind == 2 ? rbv : 4;
  const uint32_t from = (kind == 0 ? a.p.kc : kind == 1 ? a.p.ks : kind == 2 ? a.p.vc : a.p.vs) + uint32_t(h) * ps * rb;
  const uint32_t into = (kind == 0 ? 0 : kind == 1 ? kTile * rbk : kind == 2 ? kTile * (rbk + 4) : kTile * (rbk + 4 + rbv)) +
                        piece * pt * rb + smem_u32(ring);
  const int32_t* entries = a.p.table + int64_t(b) * a.p.max_pages;
  int ahead = t_first * kTile + piece * pt;  // first token of this lane's piece of the tile that is fetched next
  int id = -1;
  auto entry = [&] { id = copies && ahead < len ? entries[ahead >> a.p.ps_log2] : -1; };
  auto fetch = [&](int st) {
    const bool ok = uint32_t(id) < uint32_t(a.p.n_pages);
    if (copies && !ok && ahead < len) report_error(a.err, JOLT_ERR_INVALID_ARG);
    const uint32_t okm = __ballot_sync(0xffffffffu, ok) & 0x11u;
    const uint32_t bar = bar0 + 8 * st;
    if (lane == 0) {
      there[warp * kMaxStages + st] = okm;
      mbar_expect_tx(bar, __popc(okm) * pt * (rbk + rbv + 8));
    }
    __syncwarp();
    if (ok)
      bulk_load(into + st * a.stage_bytes, a.p.pool + uint64_t(uint32_t(id)) * a.p.page_bytes + from + (ahead & (ps - 1)) * rb,
                pt * rb, bar);
    ahead += kWarps * kTile;
    entry();
  };
  entry();
  for (int n = 0; n < min(a.stages, n_mine); ++n) fetch(n);

  // R q of this block's rows as MMA operands: lane (g, m) of k-step st holds column g, the features
  // that the codes of quarter row m give at that step. One power of two for all rows.
  float unscale;
  {
    const float isd = rsqrtf(float(D));
    __half* qh = reinterpret_cast<__half*>(qf);
    float top = 0.f;
    float sign[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sign[e] = rot_sign(a.p.seed, lane * E + e) * a.scale2;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = warp + i * kWarps;
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] *= sign[e];
      if (lane == 0 && r < RB) {  // the elements of H x add up to D x_0
        qsum[r] = v[i][0] * (float(D) * isd);
        if (PACK) qsum[r + 4] = qsum[r];
      }
      warp_fwht<E>(v[i]);
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[i][e] *= isd;
        most = fmaxf(most, fabsf(v[i][e]));
      }
      if (most < INFINITY) top = fmaxf(top, most);  // a row that is not finite is on its own
    }
    top = warp_max(top);
    if (lane == 0) xm[warp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, xm[i]);
    __syncthreads();
    int k = 0;  // 2^k top in [2^14, 2^15)
    if (top > 0.f) k = min(max(14 - (int(__float_as_uint(top) >> 23) - 127), -100), 100);
    unscale = pow2i((k_whole ? 0 : 24) - k);
    const int lnc = log2_codes(a.p.bk), half = 1 << (lnc - 1);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int f = lane * E + e;
      const int mm = f / (D / 4), fq = f % (D / 4);       // quarter row, feature in it
      const int c = fq & (2 * half - 1);                  // code in its word
      const int pair = ((fq >> lnc) << (lnc - 1)) + (c & (half - 1)), hi = c >> (lnc - 1);
      const float up = pow2i(k - (k_whole ? 0 : (a.p.bk * pair) & 7));  // less the field's place in its byte
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = warp + i * kWarps;
        if (r >= RB) break;
        const float x = v[i][e] * up;
        const __half x1 = __float2half_rn(x);
        const __half x2 = __float2half_rn(x - __half2float(x1));
        // [term][nt][st][lane = 4 * column + mm][reg][hi]
        const int at = (((pair >> 1) * 32 + 4 * (r & 7) + mm) * 2 + (pair & 1)) * 2 + hi;
        if (PACK) {
          qh[at] = x1;
          qh[at + 4 * 4 * 4] = x2;  // column r + 4
        } else {
          const int nt = r >> 3;
          qh[at + nt * NS * 128] = x1;
          qh[at + (NT + nt) * NS * 128] = x2;
        }
      }
    }
  }
  __syncthreads();

  // A column's (query row's) reference is a whole number, some room above its maximum when it was last set; it
  // is set anew only when a thread's four p of a tile add up to too much, so the usual tile takes no maximum.
  float o[NS + 1][NT][4], ref[NT][2], l[NT][2], z[NT][2], cqs[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      ref[nt][c] = -INFINITY;  // before the first every p is too large
      l[nt][c] = z[nt][c] = 0.f;
      cqs[nt][c] = qsum[nt * 8 + 2 * m + c];
    }
#pragma unroll
    for (int mt = 0; mt <= NS; ++mt)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[mt][nt][c] = 0.f;
  }
  int ve = -30;            // value scales met so far are below 2^ve
  float v_lim = pow2i(ve), v_up = pow2i(Ref<T>::p_exp - ve);
  const float ov_off = float(1 << (a.p.bv - 1)), ok_off = k_whole ? float(1 << (a.p.bk - 1)) : 0.f;
  for (int n = 0, st = 0, par = 0; n < n_mine; ++n) {
    if (!wait_all(bar0 + 8 * st, par, a.err)) {
      // gave up (reported): wait, with the same limit, for what is still in flight, then stop
      for (int x = n + 1; x < min(n + a.stages, n_mine); ++x)
        wait_all(bar0 + 8 * (x % a.stages), (x / a.stages) & 1, a.err);
      break;
    }
    const uint8_t* kc = ring + st * a.stage_bytes;
    const __half2* ksz = reinterpret_cast<const __half2*>(kc + kTile * rbk) + g;
    const uint8_t* vc = kc + kTile * (rbk + 4);
    const __half2* vsz = reinterpret_cast<const __half2*>(vc + kTile * rbv) + g;
    const uint32_t okm = there[warp * kMaxStages + st];
    const int left = len - (t_first + n * kWarps) * kTile;  // tokens from this tile's first on
    const bool whole = left >= kTile && okm == (pt == kTile ? 1u : 0x11u);

    int unseen = 0;  // bit i: token g + 8 i
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        unseen |= int(g + 8 * i >= left || !((pt == kTile ? okm : okm >> (4 * (i >> 1))) & 1)) << i;
    }
    // scores to p in place; a tile that calls for new references is done once more, from the keys
    float s[2][NT][4], sum[NT][2], vsc[4], vze[4];
    for (bool anew = false;; anew = true) {
#pragma unroll
      for (int grp = 0; grp < 2; ++grp)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[grp][nt][c] = 0.f;
      if (a.p.bk == 4) keys_tile<D, 4, NT, QT, kWhole>(kc, qf, lane, s);
      else if (a.p.bk == 8) keys_tile<D, 8, NT, QT, kWhole>(kc, qf, lane, s);
      else keys_tile<D, 2, NT, QT, true>(kc, qf, lane, s);
      if (PACK) {  // the two terms of R q
#pragma unroll
        for (int grp = 0; grp < 2; ++grp)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[grp][0][c] += __shfl_xor_sync(0xffffffffu, s[grp][0][c], 2);
      }
      // scales and zeros of this lane's four tokens, rows g + 8 i; scores in log2 units
      float v_top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 kf = __half22float2(ksz[8 * i]), vf = __half22float2(vsz[8 * i]);
        const float ks = kf.x * unscale, kz = kf.y + ok_off * kf.x;
        vsc[i] = vf.x;
        vze[i] = vf.y + ov_off * vf.x;
        if (!whole && (unseen >> i & 1)) vsc[i] = vze[i] = 0.f;
        v_top = fmaxf(v_top, fabsf(vsc[i]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& x = s[i >> 1][nt][2 * (i & 1) + c];
            x = x * ks + kz * cqs[nt][c];
          }
      }
      if (anew) {
        const uint32_t big = __reduce_max_sync(0xffffffffu, __float_as_uint(v_top));
        const int ve_new = max(ve, int(big >> 23) - 126);
        const float drop = pow2i(max(ve - ve_new, -126));
        ve = ve_new;
        v_lim = pow2i(min(ve, 127));
        v_up = pow2i(Ref<T>::p_exp - ve);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float t = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(unseen >> i & 1)) t = fmaxf(t, s[i >> 1][nt][2 * (i & 1) + c]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
            const float now = fmaxf(ref[nt][c], ceilf(t) + Ref<T>::room);
            const float f = now == ref[nt][c] ? 1.f : ex2(ref[nt][c] - now);
            ref[nt][c] = now;
            l[nt][c] *= f;
            z[nt][c] *= f;
#pragma unroll
            for (int mt = 0; mt <= NS; ++mt) {
              o[mt][nt][c] *= f * drop;
              o[mt][nt][c + 2] *= f * drop;
            }
          }
      }
      float most = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& x = s[i >> 1][nt][2 * (i & 1) + c];
            x = ex2(x - ref[nt][c]);
          }
        }
      if (!whole) {  // also while ref is -inf
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (unseen >> i & 1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[i >> 1][nt][2 * (i & 1)] = s[i >> 1][nt][2 * (i & 1) + 1] = 0.f;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sum[nt][c] = (s[0][nt][c] + s[0][nt][c + 2]) + (s[1][nt][c] + s[1][nt][c + 2]);
          most = fmaxf(most, sum[nt][c]);
        }
      if (anew || !__any_sync(0xffffffffu, most > Ref<T>::most || v_top > v_lim)) break;
    }
    uint32_t pf[PT][2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nt][c] += sum[nt][c];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[nt][c] += s[i >> 1][nt][2 * (i & 1) + c] * vze[i];
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) vsc[i] *= v_up;
#pragma unroll
    for (int grp = 0; grp < 2; ++grp)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x0 = s[grp][nt][2 * i] * vsc[2 * grp + i], x1 = s[grp][nt][2 * i + 1] * vsc[2 * grp + i];
          uint32_t hi = h2_pack(x0, x1);
          if (sizeof(T) == 4) {
            const float2 f = h2_floats(hi);
            const uint32_t lo = h2_pack(x0 - f.x, x1 - f.y);
            if (PACK) hi = m < 2 ? hi : lo;
            else pf[PT - 1][grp][nt][i] = trans8x8(lo);
          } else if (PACK) {
            hi = m < 2 ? hi : 0u;
          }
          pf[0][grp][nt][i] = trans8x8(hi);
        }
    if (a.p.bv == 4) values_tile<D, 4, NT, PT, kWhole>(vc, pf, lane, o);
    else if (a.p.bv == 8) values_tile<D, 8, NT, PT, kWhole>(vc, pf, lane, o);
    else values_tile<D, 2, NT, PT, kWhole>(vc, pf, lane, o);
    __syncwarp();  // every lane is done with the stage
    if (n + a.stages < n_mine) fetch(st);
    if (++st == a.stages) {
      st = 0;
      par ^= 1;
    }
  }

  // ---- the warps' partial results into one ----
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
        z[nt][c] += __shfl_xor_sync(0xffffffffu, z[nt][c], x);
      }
      if (g == 0) xm[warp * C + nt * 8 + 2 * m + c] = ref[nt][c];
    }
  __syncthreads();
  // fields' powers of two, and o sum(p scale), out of the outputs
  const float unit = pow2i(ve - Ref<T>::p_exp);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = nt * 8 + 2 * m + c;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, xm[w * C + col]);
      const float f = ref[nt][c] == -INFINITY ? 0.f : ex2(ref[nt][c] - top);
      if (g == 0) {
        xl[warp * C + col] = l[nt][c] * f;
        xz[warp * C + col] = z[nt][c] * f;
      }
      const float off = kWhole ? 0.f : ov_off * o[NS][nt][c];
#pragma unroll
      for (int mt = 0; mt < NS; ++mt) {
        o[mt][nt][c] = (o[mt][nt][c] * (kWhole ? 1.f : pow2i(24 - ((2 * mt * a.p.bv) & 7))) - off) * (f * unit);
        o[mt][nt][c + 2] = (o[mt][nt][c + 2] * (kWhole ? 1.f : pow2i(24 - (((2 * mt + 1) * a.p.bv) & 7))) - off) * (f * unit);
        if (PACK) {
          o[mt][nt][c] += __shfl_xor_sync(0xffffffffu, o[mt][nt][c], 2);
          o[mt][nt][c + 2] += __shfl_xor_sync(0xffffffffu, o[mt][nt][c + 2], 2);
        }
      }
    }
  // every warp leaves its sums, and adds up some of them over the warps: four features of a column a group
  float* red = reinterpret_cast<float*>(ring0);  // [kWarps][NS * NT * 4][32]
  constexpr int NR = NS * NT * 4;
#pragma unroll
  for (int i = 0; i < NR; ++i) red[(warp * NR + i) * 32 + lane] = o[i / (NT * 4)][(i / 4) % NT][i % 4];
  __syncthreads();
#pragma unroll 1
  for (int q = warp; q < NS * NT; q += kWarps) {
    const int mt = 2 * (q % (NS / 2)), nt = q / NS, c = q / (NS / 2) % 2, col = nt * 8 + 2 * m + c;
    if (col >= rows) continue;
    float x[4] = {0.f, 0.f, 0.f, 0.f}, ls = 0.f, zs = 0.f, top = -INFINITY;
    const float* from = red + (mt * NT * 4 + nt * 4 + c) * 32 + lane;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += from[(w * NR + (i >> 1) * NT * 4 + (i & 1) * 2) * 32];
      top = fmaxf(top, xm[w * C + col]);
      ls += xl[w * C + col];
      zs += xz[w * C + col];
    }
    const int64_t part = out_row(a, b, h, r0 + col) * a.parts + split;
    if (g == 0 && mt == 0) a.ml[part] = make_float2(top, ls);
    if (top != -INFINITY)
      *reinterpret_cast<float4*>(a.acc + part * D + g * (D / 8) + 2 * mt) = make_float4(x[0] + zs, x[1] + zs, x[2] + zs, x[3] + zs);
  }
}

// One warp a row: joins the splits, rotates their sum back, then adds the drafted tokens' part and the
// prefix. Launched while k_tree still runs (its blocks start as k_tree's leave room); what k_tree does not
// write is read at once, the rest after k_tree's end, all of it in one go.
template <typename T, int D, int TILE>
__global__ void __launch_bounds__(128) k_tree_merge(const TreeArgs a, bool draft) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t rows = int64_t(a.batch) * a.n_new * a.n_q, bi = (row < rows ? row : 0) / a.n_q;
  const int b = int(bi / a.n_new), i = int(bi % a.n_new);
  const bool mine = row < rows && i < draft_count(a, b);
  const int splits = splits_of<TILE>(a, b, lane);
  float back[E], po[E];
  float pre = -INFINITY;
  if (mine && a.prefix_lse) pre = a.prefix_lse[row] * 1.4426950408889634f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    back[e] = rsqrtf(float(D)) * rot_sign(a.p.seed, lane * E + e);
    po[e] = 0.f;
  }
  if (pre != -INFINITY) {
#pragma unroll
    for (int e = 0; e < E; ++e) po[e] = ld_as_float(static_cast<const T*>(a.prefix_out) + row * D + lane * E, e);
  }
  // every block waits, so that this grid never ends before k_tree
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const float* acc = a.acc + row * a.parts * D + lane * E;
  auto part = [&](int s, float (&x)[E]) {
    if constexpr (E == 4) {
      const float4 y = *reinterpret_cast<const float4*>(acc + int64_t(s) * D);
      x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(acc + int64_t(s) * D);
      x[0] = y.x, x[1] = y.y;
    }
  };
  constexpr int kBatch = 8;  // splits whose loads are in flight together
  float x[kBatch][E], xd[E];
#pragma unroll
  for (int k = 0; k < kBatch; ++k)
    if (k < splits) part(k, x[k]);
  if (draft) part(a.splits, xd);
  float2 p[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = lane + 32 * k;
    const bool there = s < splits || (draft && s == a.splits);
    p[k] = there ? a.ml[row * a.parts + s] : make_float2(-INFINITY, 0.f);
  }
  const float top = fmaxf(warp_max(fmaxf(p[0].x, p[1].x)), pre);
  const float ref = top == -INFINITY ? 0.f : top;
  float w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) w[k] = exp2f(p[k].x - ref);
  const float wp = pre == -INFINITY ? 0.f : exp2f(pre - ref);
  const float sum = warp_sum(w[0] * p[0].y + w[1] * p[1].y) + wp;
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int s0 = 0;;) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int s = s0 + k;
      const float f = __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31);
      if (s < splits && f != 0.f) {  // a split that saw nothing has left nothing
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f * x[k][e];
      }
    }
    s0 += kBatch;
    if (s0 >= splits) break;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (s0 + k < splits) part(s0 + k, x[k]);
  }
  if (a.perm) {
    __shared__ float row_s[4][D];
    float* rs = row_s[threadIdx.x >> 5];
#pragma unroll
    for (int e = 0; e < E; ++e) rs[lane * E + e] = o[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = rs[place_of(lane * E + e, log2_codes(a.perm), D)];
  }
  warp_fwht<E>(o);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] *= back[e];
  if (draft) {
    const float f = __shfl_sync(0xffffffffu, a.splits < 32 ? w[0] : w[1], a.splits & 31);
    if (f != 0.f) {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += f * xd[e];
    }
  }
  if (wp != 0.f) {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += wp * po[e];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* out = static_cast<T*>(a.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) st_from_float(out, e, o[e] * inv);
  if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

// ---- host -------------------------------------------------------------------------------------------

struct TreePlan {
  int nt, blocks, splits, shares, least, parts, stages, stage_bytes;
  bool pack, tc, balanced;
  size_t smem, ws_acc, ws_total;
};

TreePlan tree_plan(const jolt_pages& p, int batch, int n_new, int n_q, int max_pages) {
  TreePlan t{};
  const int rows = n_new * (n_q / p.n_kv);
  // tcgen05 pays for 128 rows whatever their number, mma.sync for each 16. Four ragged sequences of up to 8192
  // tokens, 8 KV heads, tcgen05 against mma.sync: 16 rows 34.1 and 26.8 us, 32 rows 34.6 and 43.2, 64 rows 36.3
  // and 84; one sequence of 131072: 16 rows 103 and 69.2 us, 32 rows 103 and 123.2; 32 rows over 512 tokens
  // 17.0 and 22.2.
  if (rows > 16 && p.io_dtype == JOLT_BF16) {
    t.tc = true;
    t.blocks = (rows + 127) / 128;
    t.least = 2;
    t.smem = tree_tc_smem(p.d_h);
  } else {
    t.pack = rows <= 4;
    t.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    t.blocks = (rows + 8 * t.nt - 1) / (8 * t.nt);
    t.least = kWarps;
    t.stage_bytes = kTile * (p.d_h * (p.b_k + p.b_v) / 8 + 8);
    const int budget = (t.nt == 1 ? 100 : 190) * 1024;
    t.stages = std::max(2, std::min(kMaxStages, budget / (kWarps * t.stage_bytes)));
    const int C = 8 * t.nt, qt = t.pack ? 1 : 2;
    const size_t head = size_t(qt) * t.nt * (p.d_h / 16) * 256 + C * 4 + 3 * kWarps * C * 4 + kWarps * kMaxStages * 12;
    const size_t ring = size_t(kWarps) * t.stages * t.stage_bytes;
    const size_t red = size_t(kWarps) * (p.d_h / 16) * t.nt * 4 * 128;
    const size_t draft = draft_smem(p.d_h, t.pack ? 4 : C, kThreads);
    t.smem = std::max(head + std::max(ring, red), draft);
  }
  // As many shares as are resident at once: one block an SM, or two where the registers allow (at 8 bits of both kinds
  // and d_h 128 the ring leaves room for one, and the shares run in two rounds: four tokens over 64K each take 118
  // us against 78 at 4 bits, on 1.9 times the bytes). A batch with more (sequence, KV head) pairs than that, or as
  // many, leaves a pair one block, and the longest sequence sets the time: 8 KV heads, one token, one sequence of 64K and 15
  // of 2K take 41 us (four equal ones of as many tokens in all: 38), with 36 of 2K 376 (48).
  const int heads = p.n_kv * t.blocks, resident = kSmCount * (!t.tc && t.nt == 1 ? 2 : 1);
  const int64_t tile = t.tc ? 128 : kTile;
  const int64_t tiles = (int64_t(max_pages) * p.page_size + tile - 1) / tile;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, (tiles + t.least - 1) / t.least));
  t.balanced = batch <= kMaxBalanced && resident / heads >= batch;
  t.shares = t.balanced ? int(std::min<int64_t>(resident / heads, most * batch)) : batch;
  t.splits = t.balanced ? int(std::min<int64_t>(most, t.shares)) : 1;
  t.parts = t.splits + 1;
  const size_t nrows = size_t(batch) * n_new * n_q;
  t.ws_acc = align_up(sizeof(WsHeader) + nrows * t.parts * sizeof(float2), 256);
  t.ws_total = align_up(t.ws_acc + nrows * t.parts * p.d_h * sizeof(float), 256);
  return t;
}

bool tree_dims_ok(const jolt_pages* p, int batch, int n_new, int n_q, int max_pages) {
  return pages_ok(p) && batch >= 0 && batch <= 65535 && n_new >= 0 && n_new <= kMaxDraft && n_q >= p->n_kv &&
         n_q % p->n_kv == 0 && n_q / p->n_kv <= 4096 && n_q <= 65536 && max_pages >= 1 && int64_t(max_pages) * p->page_size <= (int64_t(1) << 24);
}

template <typename T, int D, int TILE>
jolt_status launch_merge(const TreeArgs& a, bool draft, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned((int64_t(a.batch) * a.n_new * a.n_q + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  JOLT_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_tree_merge<T, D, TILE>, a, draft));
  return JOLT_OK;
}

template <typename T, int D, int NT, bool PACK>
jolt_status launch_tree(const TreeArgs& a, const TreePlan& t, bool draft, cudaStream_t st) {
  JOLT_CUDA_TRY(cudaFuncSetAttribute(k_tree<T, D, NT, PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(t.smem)));
  const unsigned grid = unsigned(t.shares + (draft ? a.batch : 0)) * a.p.n_kv * t.blocks;
  k_tree<T, D, NT, PACK><<<grid, kThreads, t.smem, st>>>(a);
  JOLT_CUDA_TRY(cudaGetLastError());
  return launch_merge<T, D, kTile>(a, draft, st);
}

template <typename T, int D>
jolt_status launch_tree_d(const TreeArgs& a, const TreePlan& t, bool draft, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (t.tc) {
      const jolt_status r = launch_tree_tc(a, D, draft, t.smem, st);
      return r != JOLT_OK ? r : launch_merge<T, D, 128>(a, draft, st);
    }
  }
  if (t.pack) return launch_tree<T, D, 1, true>(a, t, draft, st);
  if (t.nt == 1) return launch_tree<T, D, 1, false>(a, t, draft, st);
  if (t.nt == 2) return launch_tree<T, D, 2, false>(a, t, draft, st);
  if constexpr (sizeof(T) == 4) return launch_tree<T, D, 4, false>(a, t, draft, st);
  return JOLT_ERR_INVALID_ARG;  // bf16 of more than 16 rows is t.tc
}

}  // namespace
}  // namespace jolt

using namespace jolt;

extern "C" size_t jolt_tree_attn_workspace(const jolt_pages* pages, int32_t batch, int32_t n_new, int32_t n_q,
                                           int32_t max_pages) {
  if (!tree_dims_ok(pages, batch, n_new, n_q, max_pages)) return 0;
  // What any call of at most these sizes takes. A larger batch or tree can take less: blocks of more rows, or of more
  // sequences than there are shares, leave fewer splits. For a tree size the most is at the given batch, or at the
  // largest that is still divided evenly; wider tables only add splits.
  size_t most = 0;
  for (int n = 1; n <= std::max(n_new, 1); ++n) {
    int even = std::min(batch, kMaxBalanced);
    while (even > 1 && !tree_plan(*pages, even, n, n_q, max_pages).balanced) --even;
    for (int b : {std::max(batch, 1), std::max(even, 1)}) most = std::max(most, tree_plan(*pages, b, n, n_q, max_pages).ws_total);
  }
  return most;
}

extern "C" jolt_status jolt_tree_attn(const jolt_pages* pages, const void* pool, const int32_t* table,
                                      int32_t max_pages, const int32_t* lens, int32_t batch, int32_t n_new,
                                      int32_t n_q, const int32_t* counts, const uint64_t* mask, const void* q,
                                      int64_t q_stride_b, int64_t q_stride_t, const void* k, const void* v,
                                      int64_t kv_stride_b, int64_t kv_stride_t, float attn_scale,
                                      const void* prefix_out, const float* prefix_lse, void* out, float* lse,
                                      void* ws, size_t ws_bytes, void* stream) {
  if (!tree_dims_ok(pages, batch, n_new, n_q, max_pages)) return JOLT_ERR_INVALID_ARG;
  if (!(attn_scale > 0.f) || !(attn_scale < INFINITY)) return JOLT_ERR_INVALID_ARG;
  if (batch == 0 || n_new == 0) return JOLT_OK;
  if (!pool || !table || !lens || !q || !out || !ws) return JOLT_ERR_INVALID_ARG;
  if (!aligned(pool, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(counts, 4) || !aligned(mask, 8) ||
      !aligned(prefix_out, pages->io_dtype == JOLT_F32 ? 4 : 2) || !aligned(prefix_lse, 4) || !aligned(lse, 4) ||
      !aligned(out, 16) || !aligned(ws, 256))
    return JOLT_ERR_INVALID_ARG;
  if (!rows_ok(q, q_stride_b, q_stride_t) || (!k != !v) || (!prefix_out != !prefix_lse)) return JOLT_ERR_INVALID_ARG;
  if (k && (!rows_ok(k, kv_stride_b, kv_stride_t) || !rows_ok(v, kv_stride_b, kv_stride_t))) return JOLT_ERR_INVALID_ARG;
  const TreePlan t = tree_plan(*pages, batch, n_new, n_q, max_pages);
  if (int64_t(batch + t.shares) * pages->n_kv * t.blocks > (1 << 30)) return JOLT_ERR_INVALID_ARG;
  if (ws_bytes < t.ws_total) return JOLT_ERR_WORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(ws);
  TreeArgs a{};
  a.p = pages_dev(*pages, pool, table, max_pages, lens);
  a.q = q;
  a.k = k;
  a.v = v;
  a.qsb = q_stride_b;
  a.qst = q_stride_t;
  a.ksb = kv_stride_b;
  a.kst = kv_stride_t;
  a.counts = counts;
  a.mask = mask;
  a.prefix_out = prefix_out;
  a.prefix_lse = prefix_lse;
  a.out = out;
  a.lse = lse;
  a.ml = reinterpret_cast<float2*>(w + sizeof(WsHeader));
  a.acc = reinterpret_cast<float*>(w + t.ws_acc);
  a.err = reinterpret_cast<int32_t*>(w);
  a.scale2 = attn_scale * 1.4426950408889634f;
  a.n_new = n_new;
  a.n_q = n_q;
  a.gq = n_q / pages->n_kv;
  a.gq_magic = uint32_t(((uint64_t(1) << 32) + a.gq - 1) / a.gq);
  a.perm = t.tc ? pages->b_v : 0;
  a.splits = t.splits;
  a.shares = t.shares;
  a.least = t.least;
  a.balanced = t.balanced;
  a.parts = k ? t.parts : t.splits;
  a.batch = batch;
  a.blocks = t.blocks;
  a.stages = t.stages;
  a.stage_bytes = t.stage_bytes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = pages->io_dtype == JOLT_F32;
  StatScope sc(JOLT_K_TREE, st, 0.0, 0.0);
  if (pages->d_h == 128)
    return f32 ? launch_tree_d<float, 128>(a, t, k != nullptr, st) : launch_tree_d<__nv_bfloat16, 128>(a, t, k != nullptr, st);
  return f32 ? launch_tree_d<float, 64>(a, t, k != nullptr, st) : launch_tree_d<__nv_bfloat16, 64>(a, t, k != nullptr, st);
}
