// jolt_tree_attn for bf16 and more than 32 query rows a KV head: the products on tcgen05 (see tree_attn.cu
// for the arithmetic, which is the same).
//
// A block takes 128 query rows (drafted token x head of the group) of one KV head and a range of the
// sequence's pages, 128 tokens a tile. Query rows are the MMA's M, so a row's softmax stays with one
// warp. Even and odd tiles are two streams, each with its own scores and output accumulator in
// tensor memory, so that one stream's softmax runs under the other's MMAs:
//   S = (R q, two f16 terms) x codes^T    A, B from shared memory, K-major
//   O += P x codes                        A = P (f16) in tensor memory over the scores it came from,
//                                         B = codes from shared memory, token rows as they are (MN-major)
// Warps: 0-3 and 4-7 softmax of the two streams, 8-11 widen the keys' codes (global -> registers -> f16
// tiles in shared memory), 12-15 the values', 16 issues the MMAs. Both code tiles have one layout: a
// token's row of 64-feature chunks, 16-byte pieces of 8 features swizzled by token % 8. Features stand in
// the order in which the widening leaves them; R q is laid out to match, and the outputs are put back
// at the end.
#include <cuda.h>

#include <algorithm>

#include "pages_codes.cuh"
#include "sm100.cuh"
#include "tree_attn.cuh"

namespace jolt {
namespace {

using namespace sm100;

constexpr int kThreads = 640;  // five warpgroups
constexpr int kRows = 128;   // query rows of a block
constexpr int kTok = 128;    // tokens of a tile
// registers a thread after the warpgroups' re-split (launch: 96 each)
constexpr int kRegLaunch = 96, kRegSoft = 152, kRegWiden = 64, kRegMma = 48;
static_assert(2 * kRegSoft + 2 * kRegWiden + kRegMma <= 5 * kRegLaunch, "register shares");
constexpr float kSlack = 8.f;  // log2 units a row's scores may pass its reference by: p <= 2^8
constexpr int kPExp = 7;       // p * scale is carried times 2^(7 - ve): below 2^15

template <int D>
struct Smem {
  static constexpr int kChunk = 128 * 128;        // 128 rows x 64 f16
  static constexpr int kTile = kChunk * (D / 64);  // one f16 tile
  static constexpr int q = 0;                      // two terms
  static constexpr int k = q + 2 * kTile;          // two buffers
  static constexpr int v = k + 2 * kTile;          // two buffers
  static constexpr int sc = v + 2 * kTile;         // [2][64 token pairs][8] floats
  static constexpr int rs = sc + 2 * 64 * 32;      // [128] 2^-k
  static constexpr int qs = rs + 512;              // [128] 2^k sum(R q)
  static constexpr int vis = qs + 512;             // [2][4] words: visible tokens
  static constexpr int ve = vis + 32;              // [2] value exponent; [2][4] warps' maxima
  static constexpr int bars = ve + 48;             // 10 mbarriers
  static constexpr int slot = bars + 80;           // tensor memory base
  static constexpr int used = slot + 16;
  static constexpr int total = used + 1024;        // swizzled tiles start at 1024-byte boundaries
};

__device__ __forceinline__ uint32_t idesc_f16(int N, int b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_get(f2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 lanes x 32 columns of tensor memory: register 4a + {0, 1} = (lane g, columns 8a + 2m, +1), + {2, 3} the
// same of lane g + 8.
__device__ __forceinline__ void ld_16x256(uint32_t t, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}
__device__ __forceinline__ void st_16x256(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 16 columns: register 2a = (lane g, column 4a + m), 2a + 1 the same of lane g + 8.
__device__ __forceinline__ void st_16x128(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void ld_16x128(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}

// Place of feature f in a code tile's row (in elements) when its codes have nc = 32 / b a word: quarter
// row m, piece i of it (pairs 4i .. 4i+3 of code_pair's order), at piece i * 4 + m.
__device__ __forceinline__ int place_of(int f, int nc, int D) {
  const int m = f / (D / 4), fq = f % (D / 4);
  const int c = fq % nc, pair = (fq / nc) * (nc / 2) + c % (nc / 2);
  return ((pair >> 2) * 4 + m) * 8 + (pair & 3) * 2 + c / (nc / 2);
}

// Swaps the raw codes of pieces 0 and 1, 2 and 3 of a lane's quarter row (odd token rows: then the eight
// lanes of a store phase, two rows of four quarters, meet all eight 16-byte slots).
template <int D, int B>
__device__ __forceinline__ void swap_pieces(uint32_t (&w)[D * B / 128], bool odd) {
  constexpr int W = D * B / 128;
  if constexpr (B == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __byte_perm(w[i], 0, odd ? 0x2301 : 0x3210);
  } else {
    constexpr int P = B / 4;  // words a piece
#pragma unroll
    for (int i = 0; i < W; i += 2 * P)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const uint32_t x = w[i + j], y = w[i + P + j];
        w[i + j] = odd ? y : x;
        w[i + P + j] = odd ? x : y;
      }
  }
}

// This warp's 32 token rows of raw codes (row it*8 + g, quarter m) to f16 pieces in the tile. off[i]: where
// piece i (after the swap) goes in the row group's 8 rows; row groups are 1024 bytes apart.
template <int D, int B>
__device__ __forceinline__ void widen(uint32_t (&w)[4][D * B / 128], uint8_t* tile, const int (&off)[D / 32], bool odd) {
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    swap_pieces<D, B>(w[it], odd);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t h[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) h[x] = code_pair<B, D * B / 128>(w[it], 4 * i + x);
      *reinterpret_cast<uint4*>(tile + off[i] + it * 1024) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}
template <int D>
__device__ __forceinline__ void piece_offsets(int row0, int g, int m, int (&off)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int piece = (i ^ (g & 1)) * 4 + m;
    off[i] = (piece >> 3) * (128 * 128) + (row0 + g) * 128 + (((piece & 7) ^ g) << 4);
  }
}

// Raw codes of this warp's 32 token rows: rows of page pg[it] (-1: zeros).
template <int D, int B>
__device__ __forceinline__ void load_raw(const PagesDev& p, uint32_t seg, const int (&pg)[4], int h, int tok0, int g, int m,
                                         uint32_t (&w)[4][D * B / 128]) {
  constexpr int W = D * B / 128;
  const int ps = 1 << p.ps_log2;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    if (pg[it] >= 0) {
      const uint8_t* src = p.pool + uint64_t(pg[it]) * p.page_bytes + seg +
                           (uint32_t(h) * ps + ((tok0 + it * 8 + g) & (ps - 1))) * uint32_t(D * B / 8) + m * (4 * W);
      load_words<W>(src, w[it]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[it][i] = 0;
    }
  }
}

template <int D>
struct Ctx {
  uint8_t* smem;
  uint32_t sb, bar0;
  int n_tiles, tile0, len, h, b;
  __device__ __forceinline__ uint32_t k_full(int s) const { return bar0 + 8 * s; }
  __device__ __forceinline__ uint32_t v_full(int s) const { return bar0 + 16 + 8 * s; }
  __device__ __forceinline__ uint32_t s_done(int s) const { return bar0 + 32 + 8 * s; }
  __device__ __forceinline__ uint32_t p_full(int s) const { return bar0 + 48 + 8 * s; }
  __device__ __forceinline__ uint32_t pv_done(int s) const { return bar0 + 64 + 8 * s; }
};

__device__ __forceinline__ bool wait_all(uint32_t bar, int parity, int32_t* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
}

// Pages of the four 8-token row groups that a warp widens (-1: past the end, or no page).
template <int D>
__device__ __forceinline__ void tile_pages(const TreeArgs& a, const Ctx<D>& c, int tok0, int (&pg)[4]) {
#pragma unroll
  for (int half = 0; half < 2; ++half)
    pg[2 * half] = pg[2 * half + 1] = tok0 + half * 16 < c.len ? page_of(a.p, c.b, tok0 + half * 16, a.err) : -1;
}

// Warps 8-11: the keys' codes to f16 tiles, and per token pair (scale, zero) of keys and values as the
// softmax uses them. After a wait that gave up (reported) a warp only keeps step at the named barrier.
template <int D, int BK>
__device__ void keys_role(const TreeArgs& a, const Ctx<D>& c, int wq, int lane) {
  using S = Smem<D>;
  const int g = lane >> 2, m = lane & 3;
  const int ps = 1 << a.p.ps_log2;
  uint32_t w[4][D * BK / 128];
  int off[D / 32];
  piece_offsets<D>(wq * 32, g, m, off);
  const float ko = float(1 << (BK - 1)), vo = float(1 << (a.p.bv - 1));
  __half2 ksz, vsz;
  bool seen;
  auto fetch = [&](int n) {
    int pg[4];
    const int tok0 = (c.tile0 + n) * kTok + wq * 32;
    tile_pages<D>(a, c, tok0, pg);
    load_raw<D, BK>(a.p, a.p.kc, pg, c.h, tok0, g, m, w);
    const int page = lane < 16 ? pg[0] : pg[2];  // the lane's own token
    seen = page >= 0 && tok0 + lane < c.len;
    ksz = vsz = __floats2half2_rn(0.f, 0.f);
    if (seen) {
      const uint8_t* base = a.p.pool + uint64_t(page) * a.p.page_bytes;
      const uint32_t row = uint32_t(c.h) * ps + ((tok0 + lane) & (ps - 1));
      ksz = reinterpret_cast<const __half2*>(base + a.p.ks)[row];
      vsz = reinterpret_cast<const __half2*>(base + a.p.vs)[row];
    }
  };
  fetch(0);
  int ve = -30;
  float* red = reinterpret_cast<float*>(c.smem + S::ve + 8);
  bool ok = true;
  for (int n = 0; n < c.n_tiles; ++n) {
    const int s = n & 1, prev = ((n >> 1) & 1) ^ 1;  // parity of the phase that tile n - 2 completed
    if (n >= 2) ok = ok && wait_all(c.s_done(s), prev, a.err);
    if (ok) widen<D, BK>(w, c.smem + S::k + s * S::kTile, off, g & 1);
    const float2 kf = __half22float2(ksz), vf = __half22float2(vsz);
    const uint32_t word = __ballot_sync(0xffffffffu, seen);
    const uint32_t big = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(vf.x)));
    if (n + 1 < c.n_tiles) fetch(n + 1);
    // the softmax of tile n - 2 is done with this buffer's scales
    if (n >= 2) ok = ok && wait_all(c.p_full(s), prev, a.err);
    if (ok && lane == 0) {
      red[s * 4 + wq] = __uint_as_float(big);
      reinterpret_cast<uint32_t*>(c.smem + S::vis)[s * 4 + wq] = word;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (!ok) continue;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, red[s * 4 + i]);
    ve = max(ve, int(__float_as_uint(top) >> 23) - 126);
    const bool here = (word >> lane) & 1;
    float* dst = reinterpret_cast<float*>(c.smem + S::sc + s * 2048) + (wq * 16 + (lane >> 1)) * 8 + (lane & 1);
    dst[0] = here ? kf.x : 0.f;
    dst[2] = here ? kf.y + ko * kf.x : 0.f;
    dst[4] = here ? vf.x * pow2i(kPExp - ve) : 0.f;
    dst[6] = here ? vf.y + vo * vf.x : 0.f;
    if (wq == 0 && lane == 0) reinterpret_cast<int*>(c.smem + S::ve)[s] = ve;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.k_full(s));
  }
}

// Warps 12-15: the values' codes to f16 tiles.
template <int D, int BV>
__device__ void values_role(const TreeArgs& a, const Ctx<D>& c, int wq, int lane) {
  using S = Smem<D>;
  const int g = lane >> 2, m = lane & 3;
  uint32_t w[4][D * BV / 128];
  int off[D / 32];
  piece_offsets<D>(wq * 32, g, m, off);
  auto fetch = [&](int n) {
    int pg[4];
    const int tok0 = (c.tile0 + n) * kTok + wq * 32;
    tile_pages<D>(a, c, tok0, pg);
    load_raw<D, BV>(a.p, a.p.vc, pg, c.h, tok0, g, m, w);
  };
  fetch(0);
  for (int n = 0; n < c.n_tiles; ++n) {
    const int s = n & 1, prev = ((n >> 1) & 1) ^ 1;
    if (n >= 2 && !wait_all(c.pv_done(s), prev, a.err)) return;
    widen<D, BV>(w, c.smem + S::v + s * S::kTile, off, g & 1);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.v_full(s));
    if (n + 1 < c.n_tiles) fetch(n + 1);
  }
}

// Warp 16: scores of tile n, then outputs of tile n - 1.
template <int D>
__device__ void mma_role(const TreeArgs& a, const Ctx<D>& c, uint32_t tmem, int lane) {
  using S = Smem<D>;
  const uint32_t is = idesc_f16(kTok, 0), io = idesc_f16(D, 1);
  bool ok = true;
  for (int n = 0; n <= c.n_tiles && ok; ++n) {
    if (n < c.n_tiles) {
      const int s = n & 1;
      ok = wait_all(c.k_full(s), (n >> 1) & 1, a.err);
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t q0 = c.sb + S::q, k0 = c.sb + S::k + s * S::kTile;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = (kk >> 2) * S::kChunk + (kk & 3) * 32;
            mma_bf16(tmem + s * 128, smem_desc_sw128(q0 + t * S::kTile + at, 16, 1024),
                     smem_desc_sw128(k0 + at, 16, 1024), is, t + kk > 0);
          }
        mma_commit(c.s_done(s));
      }
      __syncwarp();
    }
    if (n >= 1) {
      const int p = n - 1, s = p & 1;
      ok = wait_all(c.p_full(s), (p >> 1) & 1, a.err) && wait_all(c.v_full(s), (p >> 1) & 1, a.err);
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t v0 = c.sb + S::v + s * S::kTile, pt = tmem + s * 128;
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk) {
          const uint64_t bd = smem_desc_sw128(v0 + kk * 2048, S::kChunk, 1024);
          const uint32_t at = pt + (kk >> 1) * 32 + (kk & 1) * 8;
          mma_bf16_tmem_a(tmem + 256 + s * 128, at, bd, io, p >= 2 || kk > 0);
        }
        mma_commit(c.pv_done(s));
      }
      __syncwarp();
    }
  }
}

// Softmax of one stream. Thread (g, m) of warp wq has rows 32 wq + {g, g+8, g+16, g+24} and the tokens
// 8j + 2m, 8j + 2m + 1: four lanes share a row, and a token pair's scales serve four rows.
// With t = scale_k acc + zero_k qs (scores are rs t): p = 2^(rs t - ref). ref is a whole number, at least
// the row's maximum when it was last set. It is set anew only when a score passes it by 2^8 (p * scale
// then still fits f16), which after a row's first tokens is rare; what was formed under the old one (this
// tile's P, the sums, O) is multiplied by a power of two.
template <int D>
__device__ void softmax_role(const TreeArgs& a, const Ctx<D>& c, uint32_t tmem, int strm, int wq, int lane, int r0,
                             int rows, int split) {
  using S = Smem<D>;
  const int g = lane >> 2, m = lane & 3;
  const uint32_t ts = tmem + strm * 128 + (uint32_t(wq * 32) << 16);
  const uint32_t to = tmem + 256 + strm * 128 + (uint32_t(wq * 32) << 16);
  constexpr uint32_t kLow = 16u << 16;  // the quarter's lanes 16-31
  float rs[4], ref[4], qs[4];
  f2 l2[4], z2[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    rs[r] = reinterpret_cast<const float*>(c.smem + S::rs)[wq * 32 + g + 8 * r];
    qs[r] = reinterpret_cast<const float*>(c.smem + S::qs)[wq * 32 + g + 8 * r];
    ref[r] = -INFINITY;
    l2[r] = z2[r] = f2_make(0.f, 0.f);
  }
  int ve = -30;
  bool ok = true;
  // O of this stream times f, after the last product into it (tile n - 2's)
  auto scale_o = [&](const float (&f)[4], int par) {
    if (!wait_all(c.pv_done(strm), par ^ 1, a.err)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t x[2][16];
      ld_16x256(to + ch * 32, x[0]);
      ld_16x256(to + kLow + ch * 32, x[1]);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[0][i] = __float_as_uint(__uint_as_float(x[0][i]) * f[(i >> 1) & 1]);
        x[1][i] = __float_as_uint(__uint_as_float(x[1][i]) * f[2 + ((i >> 1) & 1)]);
      }
      st_16x256(to + ch * 32, x[0]);
      st_16x256(to + kLow + ch * 32, x[1]);
    }
    tmem_st_wait();
    return true;
  };
  for (int n = strm; n < c.n_tiles; n += 2) {
    const int par = (n >> 1) & 1;
    ok = wait_all(c.k_full(strm), par, a.err) && wait_all(c.s_done(strm), par, a.err);
    if (!ok) break;
    tc_fence_after();
    const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(c.smem + S::sc + strm * 2048);
    const uint32_t* vis = reinterpret_cast<const uint32_t*>(c.smem + S::vis) + strm * 4;
    const int ve_now = reinterpret_cast<const int*>(c.smem + S::ve)[strm];
    if (ve_now != ve) {
      const float drop = pow2i(max(ve - ve_now, -126));
      const float f[4] = {drop, drop, drop, drop};
      ve = ve_now;
      if (n >= 2) ok = scale_o(f, par);
      if (!ok) break;
    }
    const bool whole = (vis[0] & vis[1] & vis[2] & vis[3]) == 0xffffffffu;
#pragma unroll 1
    for (int ch = 0; ch < 4; ++ch) {
      uint32_t x[2][16];
      ld_16x256(ts + ch * 32, x[0]);
      ld_16x256(ts + kLow + ch * 32, x[1]);
      tmem_ld_wait();
      f2 t[4][4];
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int at = 0; at < 4; ++at) {
        const ulonglong2 k = sc[((ch * 4 + at) * 4 + m) * 2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f2 acc = f2_make(__uint_as_float(x[r >> 1][4 * at + 2 * (r & 1)]), __uint_as_float(x[r >> 1][4 * at + 2 * (r & 1) + 1]));
          t[at][r] = f2_fma(acc, k.x, f2_mul(k.y, f2_make(qs[r], qs[r])));
        }
      }
      if (!whole) {
        const uint32_t word = vis[ch] >> (2 * m);
#pragma unroll
        for (int at = 0; at < 4; ++at)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float2 f = f2_get(t[at][r]);
            if (!((word >> (8 * at)) & 1)) f.x = -INFINITY;
            if (!((word >> (8 * at)) & 2)) f.y = -INFINITY;
            t[at][r] = f2_make(f.x, f.y);
          }
      }
      bool past = false;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int at = 0; at < 4; ++at) {
          const float2 f = f2_get(t[at][r]);
          top[r] = fmaxf(top[r], fmaxf(f.x, f.y));
        }
        past = past || top[r] * rs[r] > ref[r] + kSlack;
      }
      if (__any_sync(0xffffffffu, past)) {
        float f[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x1 = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * rs[r];
          const float now = x1 > ref[r] + kSlack ? ceilf(x1) : ref[r];
          f[r] = now == ref[r] ? 1.f : ex2(ref[r] - now);
          ref[r] = now;
          l2[r] = f2_mul(l2[r], f2_make(f[r], f[r]));
          z2[r] = f2_mul(z2[r], f2_make(f[r], f[r]));
        }
        tmem_st_wait();
#pragma unroll 1
        for (int e = 0; e < ch; ++e)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t y[8];
            ld_16x128(ts + hh * kLow + e * 32, y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&y[i]), __float2half2_rn(f[2 * hh + (i & 1)]));
              y[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            st_16x128(ts + hh * kLow + e * 32, y);
          }
        if (n >= 2) ok = scale_o(f, par);
        if (!ok) break;
      }
      uint32_t pk[2][8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float neg = ref[r] == -INFINITY ? 0.f : -ref[r];
        const f2 neg2 = f2_make(neg, neg), rs2 = f2_make(rs[r], rs[r]);
#pragma unroll
        for (int at = 0; at < 4; ++at) {
          const ulonglong2 v = sc[((ch * 4 + at) * 4 + m) * 2 + 1];
          const float2 e = f2_get(f2_fma(t[at][r], rs2, neg2));
          const f2 p = f2_make(ex2(e.x), ex2(e.y));
          l2[r] = f2_add(l2[r], p);
          z2[r] = f2_fma(p, v.y, z2[r]);
          const float2 w = f2_get(f2_mul(p, v.x));
          pk[r >> 1][2 * at + (r & 1)] = h2_pack(w.x, w.y);
        }
      }
      st_16x128(ts + ch * 32, pk[0]);
      st_16x128(ts + kLow + ch * 32, pk[1]);
    }
    if (!ok) break;
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.p_full(strm));
  }
  // ---- this stream's partial result ----
  const int mine = (c.n_tiles - strm + 1) >> 1;  // tiles of the stream
  if (mine > 0 && ok) {
    ok = wait_all(c.pv_done(strm), (mine - 1) & 1, a.err);
    tc_fence_after();
  }
  const float unit = pow2i(ve - kPExp);
  float z[4];
  float* dst[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float2 lf = f2_get(l2[r]), zf = f2_get(z2[r]);
    float l = lf.x + lf.y;
    z[r] = zf.x + zf.y;
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, x);
      z[r] += __shfl_xor_sync(0xffffffffu, z[r], x);
    }
    const int row = wq * 32 + g + 8 * r;
    dst[r] = nullptr;
    if (row < rows) {
      const int q = r0 + row;
      const int64_t gr = (int64_t(c.b) * a.n_new + q / a.gq) * a.n_q + c.h * a.gq + q % a.gq;
      const int64_t part = gr * a.parts + 2 * split + strm;
      if (m == 0) a.ml[part] = make_float2(ref[r], l);
      if (ref[r] != -INFINITY) dst[r] = a.acc + part * D;
    }
  }
  if (mine <= 0 || !ok) return;
  const int nc = 32 / a.p.bv, hn = nc / 2;
#pragma unroll 1
  for (int ch = 0; ch < D / 32; ++ch) {
    uint32_t x[2][16];
    ld_16x256(to + ch * 32, x[0]);
    ld_16x256(to + (16u << 16) + ch * 32, x[1]);
    tmem_ld_wait();
#pragma unroll
    for (int at = 0; at < 4; ++at) {
      const int pair = ch * 4 + m;  // piece ch * 4 + at: quarter row `at`, pairs 4 ch ..
      const int f = at * (D / 4) + (pair / hn) * nc + pair % hn;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (dst[r]) {
          dst[r][f] = __uint_as_float(x[r >> 1][4 * at + 2 * (r & 1)]) * unit + z[r];
          dst[r][f + hn] = __uint_as_float(x[r >> 1][4 * at + 2 * (r & 1) + 1]) * unit + z[r];
        }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_tree_tc(const TreeArgs a, int draft_x) {
  using S = Smem<D>;
  constexpr int E = D / 32;
  extern __shared__ uint8_t raw[];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y / a.blocks, r0 = (blockIdx.y % a.blocks) * kRows, b = blockIdx.z;
  const int split = int(blockIdx.x) - draft_x;  // the drafted tokens' blocks come first: they are short
  uint8_t* smem = align_smem_1024(raw);
  if (split < 0) {
    draft_block<__nv_bfloat16, D, kRows, kThreads>(a, b, h, r0, smem);
    return;
  }
  const int rows = min(kRows, draft_count(a, b) * a.gq - r0);
  if (rows <= 0) return;
  Ctx<D> c;
  c.smem = smem;
  c.sb = smem_u32(smem);
  c.bar0 = c.sb + S::bars;
  c.h = h;
  c.b = b;
  c.len = pages_len(a.p, b, a.err);
  const int tiles = (c.len + kTok - 1) / kTok, per = (tiles + a.splits - 1) / a.splits;
  c.tile0 = split * per;
  c.n_tiles = max(0, min(tiles, c.tile0 + per) - c.tile0);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + S::slot);
  if (warp == 16) {
    tmem_alloc(smem_u32(slot), 512);
    if (lane == 0) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(c.k_full(s), 4);
        mbar_init(c.v_full(s), 4);
        mbar_init(c.s_done(s), 1);
        mbar_init(c.p_full(s), 4);
        mbar_init(c.pv_done(s), 1);
      }
      fence_mbar_init();
    }
    __syncwarp();
  }
  // R q as two f16 terms, scaled by a power of two of the row
  {
    const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.q) + int64_t(b) * a.qsb + int64_t(h) * a.gq * D;
    const float isd = rsqrtf(float(D));
    const int nc = 32 / a.p.bk;
    int at[E];
#pragma unroll
    for (int e = 0; e < E; ++e) at[e] = place_of(lane * E + e, nc, D);
    float sign[E];
#pragma unroll
    for (int e = 0; e < E; ++e) sign[e] = rot_sign(a.p.seed, lane * E + e);
    for (int r = warp; r < kRows; r += kThreads / 32) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
      if (r < rows) {
        const int row = r0 + r;
        const __nv_bfloat16* x = qb + int64_t(row / a.gq) * a.qst + (row % a.gq) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = ld_as_float(x, e) * a.scale2 * sign[e];
      }
      warp_fwht<E>(v);
      float top = 0.f, sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] *= isd;
        top = fmaxf(top, fabsf(v[e]));
        sum += v[e];
      }
      top = warp_max(top);
      sum = warp_sum(sum);
      int k = 0;
      if (top > 0.f && top < INFINITY) k = min(max(14 - (int(__float_as_uint(top) >> 23) - 127), -100), 100);
      const float up = pow2i(k);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = v[e] * up;
        const __half x1 = __float2half_rn(x), x2 = __float2half_rn(x - __half2float(x1));
        const int off = (at[e] >> 6) * S::kChunk + r * 128 + ((((at[e] >> 3) & 7) ^ (r & 7)) << 4) + (at[e] & 7) * 2;
        *reinterpret_cast<__half*>(smem + S::q + off) = x1;
        *reinterpret_cast<__half*>(smem + S::q + S::kTile + off) = x2;
      }
      if (lane == 0) {
        reinterpret_cast<float*>(smem + S::rs)[r] = pow2i(-k);
        reinterpret_cast<float*>(smem + S::qs)[r] = sum * up;
      }
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoft));
    softmax_role<D>(a, c, tmem, warp >> 2, warp & 3, lane, r0, rows, split);
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegWiden));
    if (c.n_tiles > 0) {
      const int bits = warp < 12 ? a.p.bk : a.p.bv;
      if (warp < 12) {
        if (bits == 4) keys_role<D, 4>(a, c, warp & 3, lane);
        else if (bits == 8) keys_role<D, 8>(a, c, warp & 3, lane);
        else keys_role<D, 2>(a, c, warp & 3, lane);
      } else {
        if (bits == 4) values_role<D, 4>(a, c, warp & 3, lane);
        else if (bits == 8) values_role<D, 8>(a, c, warp & 3, lane);
        else values_role<D, 2>(a, c, warp & 3, lane);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegMma));
    if (warp == 16) mma_role<D>(a, c, tmem, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
jolt_status launch(const TreeArgs& a, bool draft, size_t smem, cudaStream_t st) {
  // the warpgroups re-split the block's registers (setmaxnreg): what they take must not pass what the
  // launch gives, which this build's register count decides
  static const cudaError_t fits = [] {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, k_tree_tc<D>);
    return e != cudaSuccess ? e : at.numRegs == kRegLaunch ? cudaSuccess : cudaErrorInvalidConfiguration;
  }();
  JOLT_CUDA_TRY(fits);
  JOLT_CUDA_TRY(cudaFuncSetAttribute(k_tree_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
  const dim3 grid(a.splits + (draft ? 1 : 0), a.p.n_kv * a.blocks, a.batch);
  k_tree_tc<D><<<grid, kThreads, smem, st>>>(a, draft ? 1 : 0);
  JOLT_CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

}  // namespace

size_t tree_tc_smem(int d_h) {
  const size_t draft = size_t(kMaxDraft) * (2 * d_h + 4) * 4 + size_t(kRows) * d_h * 4 + kThreads / 32 * 4 * 64 * 4 + 1024;
  return std::max<size_t>(d_h == 128 ? Smem<128>::total : Smem<64>::total, draft);
}

jolt_status launch_tree_tc(const TreeArgs& a, int d_h, bool draft, size_t smem, cudaStream_t st) {
  return d_h == 128 ? launch<128>(a, draft, smem, st) : launch<64>(a, draft, smem, st);
}

}  // namespace jolt
