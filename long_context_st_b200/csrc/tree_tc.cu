// jolt_tree_attn for bf16 and more than 16 query rows a KV head: the products on tcgen05. Scores as in
// tree_attn.cu; p is one f16 term, and the values are widened to f16 themselves (kVExp below), where tree_attn.cu
// takes their codes whole and their scales into p.
//
// A block takes 128 query rows (drafted token x head of the group) of one KV head and a range of the
// sequence's pages, 128 tokens a tile. Query rows are the MMA's M, so a row's softmax stays with one
// warp at a time: two sets of softmax warps take the even and the odd tiles. Tensor memory holds the
// output (128 columns) and three tiles' scores (128 each), so that the scores of the next two tiles are
// formed under the softmax of this one:
//   S = (R q, two f16 terms) x codes^T    A, B from shared memory, K-major
//   O += P x values                       A = P (f16) in tensor memory over the scores it came from,
//                                         B = values from shared memory, token rows as they are (MN-major)
// Warps: 0-7 and 8-15 softmax of even and odd tiles (16 rows each), 16-19 widen the keys' codes (global ->
// registers -> f16 tiles in shared memory), 20-23 the values', 24 issues the MMAs, 25 prepares the scales. Both code tiles have
// one layout: a token's row of 64-feature chunks, 16-byte pieces of 8 features swizzled by token % 8.
// Features stand in the order in which the widening leaves them; R q is laid out to match, and the merge puts
// the outputs back.
//
// 256 query rows over 131072 tokens, 8 KV heads: 198 us with the merge in a run of graph replays, 208 with L2 flushed
// between them; 0.69 and 0.66 PFLOP/s of the two products (the keys' second term makes it half as much again of MMA
// work; tensor pipe 48% busy). The roles alone take 115 us (MMAs, whose operands share the shared memory with
// the widening's stores), 93 (softmax) and as much (widening); together they wait for one another at a tile's end, with
// two buffers a kind. Each block of 128 rows widens the codes for itself, and a block of fewer rows takes as long.
#include <cuda.h>

#include <algorithm>

#include "pages_codes.cuh"
#include "sm100.cuh"
#include "tree_attn.cuh"
#include "vec.cuh"

namespace jolt {
namespace {

using namespace sm100;

// 26 warps of 72 registers. (A re-split of the registers between the roles, 80 for the softmax and 64 for the
// widening, made the compiler spill in the widening and cost 10%.)
constexpr int kThreads = 832;
constexpr int kRows = 128;   // query rows of a block
constexpr int kTok = 128;    // tokens of a tile
constexpr float kPExp = 7.f;     // p is carried times 2^7
constexpr float kRoom = 4.f;     // how far above a row's maximum its reference is set
constexpr float kMost = 32768.f;  // and a thread's sum of eight of them below 2^15, so that each is within f16
// A value is taken from its code's bits as an f16 number c 2^-24 by one multiply-add, whose factor has to be
// an f16 number too: a token's values are carried times 2^(kVExp - e), 2^e being above all of them, so that a
// scale of at most 2^(e + 1 - b) gives at most 2^15.5. They then reach 2^(b - 10), and besides f16's 2^-11 are off by
// at most 2^-25, 2^-(15 + b) of 2^e. The outputs are kept in one unit for all tokens, 2^(ve - kVExp) with ve the
// largest such exponent met so far. A token within 2^kNear of it takes ve for its e (off by 2^-(11 + b) of its largest at
// most, below the 2^-11); any other its own, and its p goes in times 2^(e - ve). A large value row so takes
// nothing from the others' bits, whatever its weight, until it is some 2^15 times as large (p then leaves f16's
// normal range). One unit for all values put errors of 2^-(15 + b) of the largest row into every one: 2% of the
// output at 2 bits where a row without weight was 2^12 times the others. Without kNear, and with the product on p
// made as p is formed, every tile pays for what few need: 204 us at 256 rows over 131072 tokens, 198 as it is, 193 with
// one unit for all.
constexpr int kNear = 3;
template <int BV>
constexpr int kVExp = BV - 10;
__device__ __forceinline__ int value_exp(float scale, float zero, float levels) {
  const float top = fmaxf(fabsf(zero), fabsf(__fmaf_rn(levels, scale, zero)));
  return min(max(int(__float_as_uint(top) >> 23) - 126, -30), 30);
}

template <int D>
struct Smem {
  static constexpr int kChunk = 128 * 128;        // 128 rows x 64 f16
  static constexpr int kTile = kChunk * (D / 64);  // one f16 tile
  static constexpr int q = 0;                      // two terms
  static constexpr int k = q + 2 * kTile;          // two buffers
  static constexpr int v = k + 2 * kTile;          // two buffers
  static constexpr int sc = v + 2 * kTile;         // [4][64 token pairs][4] floats: key scales, key zeros
  static constexpr int pe = sc + 4 * 64 * 16;      // [4][64 token pairs] f16 pairs: what p is multiplied by, 2^(e - ve)
  static constexpr int own = pe + 4 * 64 * 4;      // [4][128] what values are multiplied by for it, 2^(ve - e)
  static constexpr int rs = own + 4 * 128 * 4;     // [26] warps' largest |R q|
  static constexpr int qs = rs + 128;              // [128] sum(R q)
  static constexpr int ref = qs + 512;             // [128] the rows' references as the last finished tile left them
  static constexpr int l = ref + 512;              // [128] the odd tiles' sums
  static constexpr int vis = l + 512;              // [4][4] words: visible tokens
  static constexpr int ve = vis + 64;              // [4][2] value exponent of this tile and of the one before
  static constexpr int far = ve + 32;              // [4] whether some token's unit is not ve
  static constexpr int bars = far + 16;            // 23 mbarriers
  static constexpr int slot = bars + 192;          // tensor memory base
  static constexpr int work = slot + 16;           // Work, rows
  static constexpr int un = work + 48;             // power of two of the scores' accumulators
  static constexpr int used = un + 16;
  static constexpr int total = used + 1024;        // swizzled tiles start at 1024-byte boundaries
};

__device__ __forceinline__ uint32_t idesc_f16(int N, int b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(128 >> 4) << 24);
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

// Waits for this warp's tensor memory loads; x is not to be read before.
__device__ __forceinline__ void ld_wait(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]), "+r"(x[8]),
                 "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])
               :: "memory");
}

// The widening warps hold a token row in four lanes, lane = 8 m + g: row it*8 + g, quarter m. The eight lanes of
// a 16-byte store phase then have one piece of eight rows, which the swizzle puts into eight slots.
//
// Keys: codes are whole numbers c 2^-24 already as the f16 bits of their fields (f16's subnormals, with a
// field's place in its byte a further power of two that R q is divided by): one mask a pair. 2-bit keys are
// widened to centred normal numbers, two operations a pair: as subnormals their products lose 8 of the sum's
// 24 bits, which the fp32 log-sum-exp shows (3e-6).
template <int D, int B>
__device__ __forceinline__ void widen_keys(const uint32_t (&w)[D * B / 128], uint8_t* tile, const int (&off)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t h[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      h[x] = B == 2 ? code_pair<B, D * B / 128>(w, 4 * i + x) : field_pair<B, D * B / 128>(w, 4 * i + x);
    *reinterpret_cast<uint4*>(tile + off[i]) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}
// Values: dequantised, code * scale + zero in f16 by one fused multiply-add from the field's bits, in the token's
// units of 2^(e - kVExp): scale[F] holds scale * 2^(24 - place) for the F places of a field in its byte.
template <int D, int B>
__device__ __forceinline__ void widen_values(const uint32_t (&w)[D * B / 128], float2 sz, uint8_t* tile,
                                             const int (&off)[D / 32]) {
  constexpr int F = 8 / B;
  uint32_t s[F];
#pragma unroll
  for (int f = 0; f < F; ++f) s[f] = h2_pack(sz.x * pow2i(-B * f), sz.x * pow2i(-B * f));
  const uint32_t z = h2_pack(sz.y, sz.y);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t h[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) h[x] = h2_fma(field_pair<B, D * B / 128>(w, 4 * i + x), s[(4 * i + x) % F], z);
    *reinterpret_cast<uint4*>(tile + off[i]) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}
// Where the lane's pieces of its row group go; row groups are 1024 bytes apart.
template <int D>
__device__ __forceinline__ void piece_offsets(int row0, int g, int m, int (&off)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int piece = i * 4 + m;
    off[i] = (piece >> 3) * (128 * 128) + (row0 + g) * 128 + (((piece & 7) ^ g) << 4);
  }
}

// Raw codes of rows it * 8 + g of this warp's 32 token rows: two 16-token halves at p[0] and p[1]. A group's next
// codes are asked for as soon as it is widened: waiting for a whole tile's at once took half of these warps' time.
template <int D, int B>
__device__ __forceinline__ void load_raw(const uint8_t* const (&p)[2], uint32_t at0, uint32_t at1, int it,
                                         uint32_t (&w)[D * B / 128]) {
  load_words<D * B / 128>((it < 2 ? p[0] + at0 : p[1] + at1) + (it & 1) * 8 * (D * B / 8), w);
}

template <int D>
struct Ctx {
  uint8_t* smem;
  uint32_t sb, bar0;
  int n_tiles, tile0, len, h, b;
  // by tile, four of each (of v_full two): the next use of a barrier can't complete before everyone who waits
  // for this one has seen it
  __device__ __forceinline__ uint32_t k_full(int n) const { return bar0 + 8 * (n & 3); }
  __device__ __forceinline__ uint32_t s_done(int n) const { return bar0 + 32 + 8 * (n & 3); }
  __device__ __forceinline__ uint32_t p_full(int n) const { return bar0 + 64 + 8 * (n & 3); }
  __device__ __forceinline__ uint32_t v_full(int n) const { return bar0 + 96 + 8 * (n & 1); }
  __device__ __forceinline__ uint32_t pv_done(int n) const { return bar0 + 112 + 8 * (n & 3); }
  __device__ __forceinline__ uint32_t sc_full(int n) const { return bar0 + 144 + 8 * (n & 3); }
  __device__ __forceinline__ uint32_t q_done() const { return bar0 + 176; }
};
// Softmax, values, MMA and scales warps: R q is there, and the staging of its product is free.
__device__ __forceinline__ void q_sync() { asm volatile("bar.sync 4, 704;" ::: "memory"); }

// The pages of the two 16-token halves of a warp's 32 tokens. Table entries are read a tile before they are
// needed. A half past the end, or without a page (which is reported), is read from page 0 and not seen.
template <int D>
struct Halves {
  int id[2];
  __device__ __forceinline__ void read(const TreeArgs& a, const Ctx<D>& c, int tok0) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      id[x] = -1;
      if (tok0 + 16 * x < c.len) id[x] = a.p.table[int64_t(c.b) * a.p.max_pages + ((tok0 + 16 * x) >> a.p.ps_log2)];
    }
  }
  // bit x: half x has a page
  __device__ __forceinline__ int pages(const TreeArgs& a, const Ctx<D>& c, int tok0, const uint8_t* (&page)[2]) const {
    int there = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool ok = uint32_t(id[x]) < uint32_t(a.p.n_pages);
      there |= int(ok) << x;
      page[x] = a.p.pool + (ok ? uint64_t(uint32_t(id[x])) * a.p.page_bytes : 0);
      if (!ok && tok0 + 16 * x < c.len) report_error(a.err, JOLT_ERR_INVALID_ARG);
    }
    return there;
  }
};

// Warps 16-19: the keys' codes to f16 tiles.
template <int D, int BK>
__device__ void keys_role(const TreeArgs& a, const Ctx<D>& c, int wq, int lane) {
  using S = Smem<D>;
  const int g = lane & 7, m = lane >> 3;
  const int ps = 1 << a.p.ps_log2;
  uint32_t w[4][D * BK / 128];
  int off[D / 32];
  piece_offsets<D>(wq * 32, g, m, off);
  // a tile starts at a page's start (pages have at most 128 tokens), so places in a page stay the same
  const uint32_t at0 = a.p.kc + (uint32_t(c.h) * ps + ((wq * 32) & (ps - 1)) + g) * uint32_t(D * BK / 8) + m * (D * BK / 32);
  const uint32_t at1 = at0 + (ps == 16 ? 0 : 16 * (D * BK / 8));
  Halves<D> hv;
  const uint8_t* page[2];
  auto pages = [&](int n) {
    const int tok0 = (c.tile0 + n) * kTok + wq * 32;
    hv.pages(a, c, tok0, page);
    hv.read(a, c, tok0 + kTok);
  };
  hv.read(a, c, c.tile0 * kTok + wq * 32);
  pages(0);
#pragma unroll
  for (int it = 0; it < 4; ++it) load_raw<D, BK>(page, at0, at1, it, w[it]);
  for (int n = 0; n < c.n_tiles; ++n) {
    const bool more = n + 1 < c.n_tiles;
    if (more) pages(n + 1);
    if (n >= 2 && !wait_all(c.s_done(n - 2), ((n - 2) >> 2) & 1, a.err)) return;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      widen_keys<D, BK>(w[it], c.smem + S::k + (n & 1) * S::kTile + it * 1024, off);
      if (more) load_raw<D, BK>(page, at0, at1, it, w[it]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.k_full(n));
  }
}

// Warp 25: per token pair the keys' (scale, zero) as the softmax uses them, which tokens are seen, the exponent of
// the values' largest magnitude so far (ve), and the power of two from each token's own exponent to it. Four
// tokens a lane.
template <int D>
__device__ void scales_role(const TreeArgs& a, const Ctx<D>& c, int lane) {
  using S = Smem<D>;
  const int ps = 1 << a.p.ps_log2;
  const float vtop = float((1 << a.p.bv) - 1), ko = a.p.bk == 2 ? 2.f : 0.f;
  const uint32_t at = (uint32_t(c.h) * ps + ((lane * 4) & (ps - 1))) * 4;
  int id = -1, seen = 0;
  uint4 kz, vz;
  auto entry = [&](int n) {
    const int tok = (c.tile0 + n) * kTok + lane * 4;
    id = tok < c.len ? a.p.table[int64_t(c.b) * a.p.max_pages + (tok >> a.p.ps_log2)] : -1;
  };
  auto fetch = [&](int n) {
    const int tok = (c.tile0 + n) * kTok + lane * 4;
    const bool ok = uint32_t(id) < uint32_t(a.p.n_pages);
    if (!ok && tok < c.len) report_error(a.err, JOLT_ERR_INVALID_ARG);
    seen = ok ? (1 << min(max(c.len - tok, 0), 4)) - 1 : 0;
    const uint8_t* base = a.p.pool + (ok ? uint64_t(uint32_t(id)) * a.p.page_bytes : 0) + at;
    entry(n + 1);
    kz = *reinterpret_cast<const uint4*>(base + a.p.ks);
    vz = *reinterpret_cast<const uint4*>(base + a.p.vs);
  };
  entry(0);
  fetch(0);
  q_sync();
  const float unscale = *reinterpret_cast<const float*>(c.smem + S::un);
  int ve = -30;
  for (int n = 0; n < c.n_tiles; ++n) {
    const int q = n & 3;
    // tile n - 4 is done with this place, the widening of its values among it
    if (n >= 4 && !wait_all(c.pv_done(n - 4), ((n - 4) >> 2) & 1, a.err)) return;
    const uint32_t ku[4] = {kz.x, kz.y, kz.z, kz.w}, vu[4] = {vz.x, vz.y, vz.z, vz.w};
    float sc[4], ze[4];
    int e[4], most = -30;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 k = h2_floats(ku[i]), v = h2_floats(vu[i]);
      const bool here = (seen >> i) & 1;
      sc[i] = here ? k.x * unscale : 0.f;
      ze[i] = here ? k.y + ko * k.x : 0.f;
      e[i] = here ? value_exp(v.x, v.y, vtop) : -30;
      most = max(most, e[i]);
    }
    float4* dst = reinterpret_cast<float4*>(c.smem + S::sc + q * 1024) + lane * 2;
    dst[0] = make_float4(sc[0], sc[1], ze[0], ze[1]);
    dst[1] = make_float4(sc[2], sc[3], ze[2], ze[3]);
    // eight lanes' four tokens a word
    uint32_t word = uint32_t(seen) << (4 * (lane & 7));
#pragma unroll
    for (int x = 1; x <= 4; x <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, x);
    if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(c.smem + S::vis)[q * 4 + (lane >> 3)] = word;
    const int before = ve;
    ve = max(ve, __reduce_max_sync(0xffffffffu, most));
    bool far = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!((seen >> i) & 1) || e[i] >= ve - kNear) e[i] = ve;
      far = far || e[i] != ve;
    }
    far = __any_sync(0xffffffffu, far);
    if (far) {  // f16 has powers of two down to 2^-24
      uint2 up;
      up.x = h2_pack(pow2i(e[0] - ve), pow2i(e[1] - ve));
      up.y = h2_pack(pow2i(e[2] - ve), pow2i(e[3] - ve));
      reinterpret_cast<uint2*>(c.smem + S::pe + q * 256)[lane] = up;
      reinterpret_cast<float4*>(c.smem + S::own + q * 512)[lane] =
          make_float4(pow2i(ve - e[0]), pow2i(ve - e[1]), pow2i(ve - e[2]), pow2i(ve - e[3]));
    }
    if (lane == 0) {
      reinterpret_cast<int2*>(c.smem + S::ve)[q] = make_int2(ve, n ? before : ve);
      reinterpret_cast<int*>(c.smem + S::far)[q] = far;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(c.sc_full(n));
    if (n + 1 < c.n_tiles) fetch(n + 1);
  }
}

// Warps 20-23: the values to f16 tiles. A token that is not seen gets zeros (its scale may be anything).
template <int D, int BV>
__device__ void values_role(const TreeArgs& a, const Ctx<D>& c, int wq, int lane) {
  using S = Smem<D>;
  const int g = lane & 7, m = lane >> 3;
  const int ps = 1 << a.p.ps_log2;
  uint32_t w[4][D * BV / 128];
  __half2 raw[4];
  int off[D / 32];
  piece_offsets<D>(wq * 32, g, m, off);
  const uint32_t head = uint32_t(c.h) * ps, in_page = ((wq * 32) & (ps - 1)) + g;
  const uint32_t at0 = a.p.vc + (head + in_page) * uint32_t(D * BV / 8) + m * (D * BV / 32);
  const uint32_t at1 = at0 + (ps == 16 ? 0 : 16 * (D * BV / 8));
  const uint32_t sz0 = a.p.vs + (head + in_page) * 4, sz1 = sz0 + (ps == 16 ? 0 : 64);
  Halves<D> hv;
  int seen;  // bit it: the lane's row of group it
  const uint8_t* page[2];
  auto pages = [&](int n) {
    const int tok0 = (c.tile0 + n) * kTok + wq * 32;
    const int there = hv.pages(a, c, tok0, page);
    hv.read(a, c, tok0 + kTok);
    seen = 0;
#pragma unroll
    for (int it = 0; it < 4; ++it) seen |= int(((there >> (it >> 1)) & 1) && tok0 + it * 8 + g < c.len) << it;
  };
  auto load = [&](int it) {
    raw[it] = *reinterpret_cast<const __half2*>(page[it >> 1] + (it < 2 ? sz0 : sz1) + (it & 1) * 32);
    load_raw<D, BV>(page, at0, at1, it, w[it]);
  };
  hv.read(a, c, c.tile0 * kTok + wq * 32);
  pages(0);
#pragma unroll
  for (int it = 0; it < 4; ++it) load(it);
  q_sync();
  for (int n = 0; n < c.n_tiles; ++n) {
    const int s = n & 1;
    if (!wait_all(c.sc_full(n), (n >> 2) & 1, a.err)) return;  // ve of this tile
    const bool far = reinterpret_cast<const int*>(c.smem + S::far)[n & 3];
    const float unit = pow2i(kVExp<BV> - reinterpret_cast<const int2*>(c.smem + S::ve)[n & 3].x);
    float2 sz[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const float2 f = __half22float2(raw[it]);
      sz[it] = (seen >> it) & 1 ? make_float2(f.x * (unit * 16777216.f), f.y * unit) : make_float2(0.f, 0.f);
    }
    if (far) {
      const float* own = reinterpret_cast<const float*>(c.smem + S::own) + (n & 3) * 128 + wq * 32 + g;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        sz[it].x *= own[it * 8];
        sz[it].y *= own[it * 8];
      }
    }
    const bool more = n + 1 < c.n_tiles;
    if (more) pages(n + 1);
    if (n >= 2 && !wait_all(c.pv_done(n - 2), ((n - 2) >> 2) & 1, a.err)) return;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      widen_values<D, BV>(w[it], sz[it], c.smem + S::v + s * S::kTile + it * 1024, off);
      if (more) load(it);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.v_full(n));
  }
}

// Warp 24: scores of tiles 0 and 1, then of tile n + 2 before the outputs of tile n.
template <int D>
__device__ void mma_role(const TreeArgs& a, const Ctx<D>& c, uint32_t tmem, int lane) {
  using S = Smem<D>;
  const uint32_t is = idesc_f16(kTok, 0), io = idesc_f16(D, 1);
  // tiles and k-steps differ in the descriptors' start address alone (in 16-byte units, below 2^14)
  const uint64_t qd = smem_desc_sw128(c.sb + S::q, 16, 1024), kd = smem_desc_sw128(c.sb + S::k, 16, 1024);
  const uint64_t vd = smem_desc_sw128(c.sb + S::v, S::kChunk, 1024);
  int buf = 0, pbuf = 0;  // tile % 3
  for (int n = -2; n < c.n_tiles; ++n) {
    const int t2 = n + 2;
    if (t2 < c.n_tiles) {
      if (!wait_all(c.k_full(t2), (t2 >> 2) & 1, a.err)) return;
      tc_fence_after();
      if (lane == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = (kk >> 2) * S::kChunk + (kk & 3) * 32;
            mma_bf16(tmem + 128 + buf * 128, qd + ((t * S::kTile + at) >> 4), kd + (((t2 & 1) * S::kTile + at) >> 4), is,
                     t + kk > 0);
          }
        mma_commit(c.s_done(t2));
      }
      __syncwarp();
      buf = buf == 2 ? 0 : buf + 1;
    }
    if (n >= 0) {
      if (!wait_all(c.p_full(n), (n >> 2) & 1, a.err) || !wait_all(c.v_full(n), (n >> 1) & 1, a.err)) return;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t vs = vd + (((n & 1) * S::kTile) >> 4);
        const uint32_t pt = tmem + 128 + pbuf * 128;
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk)
          mma_bf16_tmem_a(tmem, pt + (kk >> 1) * 32 + (kk & 1) * 8, vs + ((kk * 2048) >> 4), io, n > 0 || kk > 0);
        mma_commit(c.pv_done(n));
      }
      __syncwarp();
      pbuf = pbuf == 2 ? 0 : pbuf + 1;
    }
  }
}

// Softmax of 16 rows in every other tile (strm: even or odd). Thread (g, m) has rows row0 + g and row0 + g + 8
// and the tokens 8j + 2m, 8j + 2m + 1: four lanes share a row, and a token pair's scales serve two rows.
// With s = scale_k acc + zero_k qs: p = 2^(s - ref + 7). ref is a whole number, 4 above the row's maximum
// when it was last set. It is set anew only when a thread's eight p of a chunk add up to more than 2^15
// (some score then passed it by 5 or more; until then p fits f16), which after a row's first tokens is
// rare: the usual pass needs no maximum. What was formed under the old reference is then multiplied by a
// power of two: this tile's P and the sum at once, O at the tile's end, when the two sets of warps also
// agree: a tile's reference is at least the one that the tile before it ended with.
template <int D>
__device__ void softmax_role(const TreeArgs& a, const Ctx<D>& c, uint32_t tmem, int strm, int row0, int lane, int r0,
                             int rows, int split) {
  using S = Smem<D>;
  const int g = lane >> 2, m = lane & 3;
  const uint32_t to = tmem + (uint32_t(row0) << 16);
  float* const ref_s = reinterpret_cast<float*>(c.smem + S::ref) + row0 + g;
  float ref[2];
  f2 l2[2], qs2[2], neg2[2];  // neg2: 7 - ref; +inf before the first: every p is then too large
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float qs = reinterpret_cast<const float*>(c.smem + S::qs)[row0 + g + 8 * r];
    qs2[r] = f2_make(qs, qs);
    ref[r] = -INFINITY;
    neg2[r] = f2_make(INFINITY, INFINITY);
    l2[r] = f2_make(0.f, 0.f);
  }
  // raises row r's reference to `now` (at least ref): the factor of what was formed under the old one
  auto raise = [&](int r, float now) {
    const float f = now == ref[r] ? 1.f : ex2(ref[r] - now);
    ref[r] = now;
    neg2[r] = f2_make(kPExp - now, kPExp - now);
    l2[r] = f2_mul(l2[r], f2_make(f, f));
    return f;
  };
  bool ok = true;
  for (int n = strm; n < c.n_tiles; n += 2) {
    const int par = (n >> 2) & 1;
    ok = wait_all(c.sc_full(n), par, a.err) && wait_all(c.s_done(n), par, a.err);
    if (!ok) break;
    tc_fence_after();
    const uint32_t ts = tmem + 128 + (n % 3) * 128 + (uint32_t(row0) << 16);
    const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(c.smem + S::sc + (n & 3) * 1024) + m;
    const uint32_t* vis = reinterpret_cast<const uint32_t*>(c.smem + S::vis) + (n & 3) * 4;
    const int2 ve = reinterpret_cast<const int2*>(c.smem + S::ve)[n & 3];
    const bool whole = (vis[0] & vis[1] & vis[2] & vis[3]) == 0xffffffffu;
    // this tile's P of chunks [0, end) times f, and into the unit of the outputs (far)
    auto scale_p = [&](float f0, float f1, int end, bool far) {
      const __half2* pe = reinterpret_cast<const __half2*>(c.smem + S::pe + (n & 3) * 256) + m;
      tmem_st_wait();
#pragma unroll 1
      for (int e = 0; e < end; ++e) {
        uint32_t y[8];
        ld_16x128(ts + e * 32, y);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&y[i]), __float2half2_rn((i & 1) ? f1 : f0));
          if (far) v = __hmul2(v, pe[(e * 4 + (i >> 1)) * 4]);
          y[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        st_16x128(ts + e * 32, y);
      }
    };
    bool tried = false;
#pragma unroll 1  // one copy of the body: the roles' code together is already long for the instruction cache
    for (int ch = 0; ch < 4;) {
      uint32_t x[16];
      ld_16x256(ts + ch * 32, x);
      ld_wait(x);
      f2 e2[4][2];
#pragma unroll
      for (int at = 0; at < 4; ++at) {
        const ulonglong2 k = sc[(ch * 4 + at) * 4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
          e2[at][r] = f2_fma(f2_make(__uint_as_float(x[4 * at + 2 * r]), __uint_as_float(x[4 * at + 2 * r + 1])), k.x,
                             f2_fma(k.y, qs2[r], neg2[r]));
      }
      if (!whole) {
        const uint32_t word = vis[ch] >> (2 * m);
#pragma unroll
        for (int at = 0; at < 4; ++at)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float2 f = f2_get(e2[at][r]);
            if (!((word >> (8 * at)) & 1)) f.x = -INFINITY;
            if (!((word >> (8 * at)) & 2)) f.y = -INFINITY;
            e2[at][r] = f2_make(f.x, f.y);
          }
      }
      uint32_t pk[8];
      f2 sum[2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int at = 0; at < 4; ++at) {
          const float2 e = f2_get(e2[at][r]);
          const float p0 = ex2(e.x), p1 = ex2(e.y);
          sum[r] = at ? f2_add(sum[r], f2_make(p0, p1)) : f2_make(p0, p1);
          pk[2 * at + r] = h2_pack(p0, p1);
        }
      const float2 s0 = f2_get(sum[0]), s1 = f2_get(sum[1]);
      if (!tried && __any_sync(0xffffffffu, fmaxf(s0.x + s0.y, s1.x + s1.y) > kMost)) {
        // new references, from this chunk's scores read again; then the chunk once more
        tried = true;
        float top[2] = {-INFINITY, -INFINITY};
        ld_16x256(ts + ch * 32, x);
        ld_wait(x);
#pragma unroll
        for (int at = 0; at < 4; ++at) {
          const ulonglong2 k = sc[(ch * 4 + at) * 4];
          const uint32_t word = vis[ch] >> (2 * m + 8 * at);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 t = f2_get(f2_fma(f2_make(__uint_as_float(x[4 * at + 2 * r]), __uint_as_float(x[4 * at + 2 * r + 1])),
                                           k.x, f2_mul(k.y, qs2[r])));
            if (word & 1) top[r] = fmaxf(top[r], t.x);
            if (word & 2) top[r] = fmaxf(top[r], t.y);
          }
        }
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
          f[r] = raise(r, fmaxf(ref[r], ceilf(top[r]) + kRoom));
        }
        scale_p(f[0], f[1], ch, false);
        continue;
      }
      tried = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) l2[r] = f2_add(l2[r], sum[r]);
      st_16x128(ts + ch * 32, pk);
      ++ch;
    }
    // tokens whose values are in units of their own, and the references that tile n - 1 ended with
    const bool far = reinterpret_cast<const int*>(c.smem + S::far)[n & 3];
    float fp[2] = {1.f, 1.f};
    bool p_too = far;
    if (n > 0) {
      // the references that tile n - 1 ended with, and O, which is in their and its values' units
      ok = wait_all(c.p_full(n - 1), ((n - 1) >> 2) & 1, a.err);
      if (!ok) break;
      const float drop = pow2i(max(ve.y - ve.x, -126));
      float fo[2];
      bool o_too = drop != 1.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float was = ref_s[8 * r];
        const float now = fmaxf(was, ref[r]);
        fo[r] = (now == was ? 1.f : ex2(was - now)) * drop;
        p_too = p_too || now != ref[r];
        o_too = o_too || now != was;
        fp[r] = raise(r, now);
      }
      if (__any_sync(0xffffffffu, o_too)) {
        ok = wait_all(c.pv_done(n - 1), ((n - 1) >> 2) & 1, a.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t x[16];
          ld_16x256(to + ch * 32, x);
          ld_wait(x);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * fo[(i >> 1) & 1]);
          st_16x256(to + ch * 32, x);
        }
      }
    }
    if (__any_sync(0xffffffffu, p_too)) scale_p(fp[0], fp[1], 4, far);
    if (m == 0) {
      ref_s[0] = ref[0];
      ref_s[8] = ref[1];
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.p_full(n));
  }
  // ---- the block's partial result: the two sets' sums together, half of O's columns each ----
  const int last = c.n_tiles - 1;
  if (ok && last >= 0) {
    ok = wait_all(c.p_full(last), (last >> 2) & 1, a.err) && wait_all(c.pv_done(last), (last >> 2) & 1, a.err);
    tc_fence_after();
  }
  float l[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (ok && last >= 0) raise(r, fmaxf(ref[r], ref_s[8 * r]));
    const float2 f = f2_get(l2[r]);
    l[r] = f.x + f.y;
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
    if (strm == 1 && m == 0) reinterpret_cast<float*>(c.smem + S::l)[row0 + g + 8 * r] = l[r];
  }
  asm volatile("bar.sync 2, 512;" ::: "memory");
  float* dst[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = row0 + g + 8 * r;
    dst[r] = nullptr;
    if (row < rows) {
      const int64_t part = out_row(a, c.b, c.h, r0 + row) * a.parts + split;
      if (strm == 0 && m == 0)  // p and O were carried times 2^7
        a.ml[part] = make_float2(ref[r] - kPExp, l[r] + reinterpret_cast<const float*>(c.smem + S::l)[row]);
      if (ref[r] != -INFINITY) dst[r] = a.acc + part * D;
    }
  }
  if (last < 0 || !ok) return;
  const float unit = pow2i(reinterpret_cast<const int2*>(c.smem + S::ve)[last & 3].x - (a.p.bv - 10));  // kVExp
  // in the tiles' order of features: the merge puts the sum over the splits into their own
#pragma unroll 1
  for (int ch = strm * (D / 64); ch < (strm + 1) * (D / 64); ++ch) {
    uint32_t x[16];
    ld_16x256(to + ch * 32, x);
    ld_wait(x);
#pragma unroll
    for (int at = 0; at < 4; ++at)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (dst[r])
          *reinterpret_cast<float2*>(dst[r] + ch * 32 + at * 8 + 2 * m) =
              make_float2(__uint_as_float(x[4 * at + 2 * r]) * unit, __uint_as_float(x[4 * at + 2 * r + 1]) * unit);
  }
}

// Feature at place p of a code tile's row (place_of's inverse).
template <int D>
__device__ __forceinline__ int feature_at(int p, int lnc) {
  const int half = 1 << (lnc - 1), pair = (p >> 5) * 4 + ((p & 7) >> 1);
  return ((p >> 3) & 3) * (D / 4) + ((pair >> (lnc - 1)) << lnc) + (pair & (half - 1)) + ((p & 1) << (lnc - 1));
}

// Warps 0-15 with warp 24: R q of the block's rows as two f16 terms in the tiles' order, times one power of two for
// all rows: the largest element then has 2^14, and the second term's last place is 2^-24, 2^-39 of it. The
// transform is itself a product on tcgen05: q, bf16 as given, with the matrix of its signs (row: a place's feature;
// warps 8-23 form it while warp 0 finds the block's work), both staged where the values' tiles will be, so that
// no row waits for shuffles (7400 cycles by a transform in registers, of 28000 for a block of one tile).
template <int D>
__device__ void q_signs(const TreeArgs& a, uint8_t* signs, int tid) {
  using S = Smem<D>;
  constexpr int V = D / 8, kB = D * V / 512;  // 16-byte pieces of a row; of a thread
  const int lane = tid & 31, t = tid % V, row0 = tid / V;
  uint32_t neg = 0;  // this piece's eight signs
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    const uint32_t bits = __ballot_sync(0xffffffffu, rot_sign(a.p.seed, 32 * w + lane) < 0.f);
    if ((t >> 2) == w) neg = (bits >> (8 * (t & 3))) & 0xFFu;
  }
#pragma unroll
  for (int i = 0; i < kB; ++i) {
    const int p = row0 + i * (512 / V), f = feature_at<D>(p, log2_codes(a.p.bk));
    // bit e: element (f, 8 t + e) is negative, the parity of f & (8 t + e) and the column's own sign
    uint32_t bits = neg ^ ((f & 1) ? 0xAAu : 0u) ^ ((f & 2) ? 0xCCu : 0u) ^ ((f & 4) ? 0xF0u : 0u);
    if (__popc(f & (8 * t)) & 1) bits ^= 0xFFu;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = 0x3F803F80u | ((bits << (15 - 2 * e)) & 0x8000u) | ((bits << (30 - 2 * e)) & 0x80000000u);
    *reinterpret_cast<uint4*>(signs + (t >> 3) * S::kChunk + p * 128 + (((t & 7) ^ (p & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <int D>
__device__ void q_stage(const TreeArgs& a, const Ctx<D>& c, int tid, int r0, int rows) {
  using S = Smem<D>;
  constexpr int V = D / 8, kQ = 128 * V / 512;  // 16-byte pieces of a row; of a thread
  const int t = tid % V, row0 = tid / V;
  const float qs = rot_sign(a.p.seed, 0) * a.scale2 * (float(D) * rsqrtf(float(D)));
  const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.q) + int64_t(c.b) * a.qsb + int64_t(c.h) * a.gq * D;
  uint4 x[kQ];
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int r = row0 + i * (512 / V);
    x[i] = make_uint4(0, 0, 0, 0);
    if (r < rows) x[i] = *reinterpret_cast<const uint4*>(qb + q_offset(a, r0 + r, D) + t * 8);
  }
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int r = row0 + i * (512 / V);
    *reinterpret_cast<uint4*>(c.smem + S::v + S::kTile + (t >> 3) * S::kChunk + r * 128 + (((t & 7) ^ (r & 7)) << 4)) = x[i];
    // the elements of H x add up to D x_0
    if (t == 0) reinterpret_cast<float*>(c.smem + S::qs)[r] = __uint_as_float(x[i].x << 16) * qs;
  }
  fence_proxy_async_smem();
  asm volatile("bar.sync 3, 544;" ::: "memory");
}
template <int D>
__device__ void q_finish(const TreeArgs& a, const Ctx<D>& c, uint32_t tmem, int warp, int lane) {
  using S = Smem<D>;
  constexpr int C = D / 4;  // a thread has a row's quarter
  const int quarter = warp & 3, part = warp >> 2, r = quarter * 32 + lane;
  wait_all(c.q_done(), 0, a.err);  // a wait that gave up is reported, and ends the call like any other
  tc_fence_after();
  uint32_t x[C];
  if constexpr (C == 32) tmem_ld32(tmem + (uint32_t(quarter * 32) << 16) + part * C, x);
  else tmem_ld16(tmem + (uint32_t(quarter * 32) << 16) + part * C, x);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < C; ++i) asm volatile("" : "+r"(x[i]));  // not read before the wait
  const float f = a.scale2 * rsqrtf(float(D));
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) top = fmaxf(top, fabsf(__uint_as_float(x[i]) * f));
  if (!(top < INFINITY)) top = 0.f;  // a row that is not finite is on its own
  top = warp_max(top);
  float* rs = reinterpret_cast<float*>(c.smem + S::rs);
  if (lane == 0) rs[warp] = top;
  asm volatile("bar.sync 2, 512;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, rs[i]);
  int k = 0;
  if (top > 0.f) k = min(max(14 - (int(__float_as_uint(top) >> 23) - 127), -100), 100);
  if (warp + lane == 0) *reinterpret_cast<float*>(c.smem + S::un) = pow2i((a.p.bk == 2 ? 0 : 24) - k);
  // less a 4-bit field's place in its byte, that of odd pairs (b times a pair's number is 0 modulo 8 at 8 bits; 2-bit
  // codes are normal numbers)
  const float up = pow2i(k), odd = a.p.bk == 4 ? 0.0625f : 1.f;
  uint8_t* const q = c.smem + S::q + r * 128;
#pragma unroll
  for (int i = 0; i < C / 8; ++i) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y0 = __uint_as_float(x[8 * i + 2 * e]) * f * up * ((e & 1) ? odd : 1.f);
      const float y1 = __uint_as_float(x[8 * i + 2 * e + 1]) * f * up * ((e & 1) ? odd : 1.f);
      h[e] = h2_pack(y0, y1);
      const float2 z = h2_floats(h[e]);
      l[e] = h2_pack(y0 - z.x, y1 - z.y);
    }
    const int piece = part * (C / 8) + i;
    uint8_t* dst = q + (piece >> 3) * S::kChunk + (((piece & 7) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(dst + S::kTile) = make_uint4(l[0], l[1], l[2], l[3]);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  q_sync();
  tc_fence_after();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_tree_tc(const TreeArgs a) {
  using S = Smem<D>;
  extern __shared__ uint8_t raw[];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = align_smem_1024(raw);
  Work wk;
  if (int(blockIdx.x) >= a.shares * a.p.n_kv * a.blocks) {
    work_of<kTok>(a, &wk);
    draft_part<__nv_bfloat16, D, kRows, kThreads>(a, wk.b, wk.h, wk.block * kRows, smem);
    return;
  }
  Ctx<D> c;
  c.smem = smem;
  c.sb = smem_u32(smem);
  c.bar0 = c.sb + S::bars;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + S::slot);
  Work* shared_work = reinterpret_cast<Work*>(smem + S::work);
  int* shared_rows = reinterpret_cast<int*>(shared_work + 1);
  if (warp == 0) {  // one warp: all 26 at once would take 5000 cycles
    const bool any = work_of<kTok>(a, &wk);
    const int rows = any ? min(kRows, draft_count(a, wk.b) * a.gq - wk.block * kRows) : 0;
    if (lane == 0) {
      *shared_work = wk;
      *shared_rows = rows;
    }
  }
  if (warp >= 8 && warp < 24) {
    q_signs<D>(a, smem + S::v, tid - 256);
    fence_proxy_async_smem();
  }
  if (warp == 24) {
    tmem_alloc(smem_u32(slot), 512);
    if (lane == 0) {
      for (int n = 0; n < 4; ++n) {
        mbar_init(c.k_full(n), 4);
        mbar_init(c.s_done(n), 1);
        mbar_init(c.p_full(n), 8);
        if (n < 2) mbar_init(c.v_full(n), 4);
        mbar_init(c.pv_done(n), 1);
        mbar_init(c.sc_full(n), 1);
      }
      mbar_init(c.q_done(), 1);
      fence_mbar_init();
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const int rows = *shared_rows;
  if (rows <= 0) {
    if (warp == 24) tmem_dealloc(tmem, 512);
    return;
  }
  wk = *shared_work;
  const int r0 = wk.block * kRows;
  c.h = wk.h;
  c.b = wk.b;
  c.len = wk.len;
  c.tile0 = wk.tile0;
  c.n_tiles = wk.n_tiles;
  if (warp < 16) {
    q_stage<D>(a, c, tid, r0, rows);
    q_finish<D>(a, c, tmem, warp, lane);
    // a warp reaches the 32 lanes of its quarter, warp % 4
    softmax_role<D>(a, c, tmem, warp >> 3, (warp & 3) * 32 + ((warp >> 2) & 1) * 16, lane, r0, rows, wk.split);
  } else if (warp < 20) {
    if (c.n_tiles > 0) {
      if (a.p.bk == 4) keys_role<D, 4>(a, c, warp & 3, lane);
      else if (a.p.bk == 8) keys_role<D, 8>(a, c, warp & 3, lane);
      else keys_role<D, 2>(a, c, warp & 3, lane);
    }
  } else if (warp == 24) {
    asm volatile("bar.sync 3, 544;" ::: "memory");
    tc_fence_after();
    if (lane == 0) {
      const uint64_t qd = smem_desc_sw128(c.sb + S::v + S::kTile, 16, 1024), sd = smem_desc_sw128(c.sb + S::v, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t at = ((kk >> 2) * S::kChunk + (kk & 3) * 32) >> 4;
        mma_bf16(tmem, qd + at, sd + at, idesc_bf16_f32(kRows, D, 0, 0), kk > 0);
      }
      mma_commit(c.q_done());
    }
    __syncwarp();
    q_sync();
    tc_fence_after();
    mma_role<D>(a, c, tmem, lane);
  } else if (c.n_tiles == 0) {
    q_sync();
  } else if (warp == 25) {
    scales_role<D>(a, c, lane);
  } else {
    if (a.p.bv == 4) values_role<D, 4>(a, c, warp & 3, lane);
    else if (a.p.bv == 8) values_role<D, 8>(a, c, warp & 3, lane);
    else values_role<D, 2>(a, c, warp & 3, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 24) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
jolt_status launch(const TreeArgs& a, bool draft, size_t smem, cudaStream_t st) {
  JOLT_CUDA_TRY(cudaFuncSetAttribute(k_tree_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
  const unsigned grid = unsigned(a.shares + (draft ? a.batch : 0)) * a.p.n_kv * a.blocks;
  k_tree_tc<D><<<grid, kThreads, smem, st>>>(a);
  JOLT_CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

}  // namespace

size_t tree_tc_smem(int d_h) {
  const size_t draft = draft_smem(d_h, kRows, kThreads) + 1024;
  return std::max<size_t>(d_h == 128 ? Smem<128>::total : Smem<64>::total, draft);
}

jolt_status launch_tree_tc(const TreeArgs& a, int d_h, bool draft, size_t smem, cudaStream_t st) {
  return d_h == 128 ? launch<128>(a, draft, smem, st) : launch<64>(a, draft, smem, st);
}

}  // namespace jolt
