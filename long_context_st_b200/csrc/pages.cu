// jolt_pages_append / jolt_pages_read: the tail cache's rows coded as they are written, and read back.
#include <algorithm>

#include "common.cuh"
#include "pages_codes.cuh"
#include "pages.cuh"
#include "stats.h"
#include "vec.cuh"

namespace jolt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Both kernels hold a row of D elements in four lanes, eight rows a warp (or sixteen as MMA rows): lane
// m = lane % 4 has the 8-element pieces j*4 + m, j < D/32, so a load or store of one piece a lane covers
// 64 contiguous bytes (bf16) of each row.
__device__ __forceinline__ int piece_at(int j, int m) { return (j * 4 + m) * 8; }

// Signs of this lane's elements: bit 8*j + e set when element piece_at(j, m) + e is negated.
template <int D>
__device__ __forceinline__ uint32_t lane_signs(uint64_t seed, int lane) {
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const uint32_t w = __ballot_sync(0xffffffffu, rot_sign(seed, 32 * j + lane) < 0.f);
    mine |= ((w >> (8 * (lane & 3))) & 0xFFu) << (8 * j);
  }
  return mine;
}

struct AppendArgs {
  PagesDev p;
  const void* x[2];
  const int32_t* counts;
  const int32_t* src;
  int64_t stride_b, stride_t;
  int32_t* err;
  int n_new, n_src;
  uint32_t rows;  // of K, and of V
};

// Eight elements as loaded, and as floats.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float* f) const {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) unpack16<T>(v[i], f + 16 / int(sizeof(T)) * i);
  }
};

// Packs this lane's codes and stores them: piece j is B bytes at (j*4 + m)*B of the row. c: floats
// 1.5 * 2^23 + code; as bits kBits + code, so that sums of them times 2^(B e) are the codes' fields plus a
// constant.
template <int B, int J>
__device__ __forceinline__ void store_codes(const float (&c)[8 * J], uint8_t* row, int m) {
  constexpr uint32_t kBits = 0x4B400000u;
  constexpr int P = B == 8 ? 4 : 8;  // codes of a word (or half word)
  uint32_t base = 0;
#pragma unroll
  for (int e = 0; e < P; ++e) base += kBits << (e * B);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    uint32_t w[8 / P];
#pragma unroll
    for (int i = 0; i < 8 / P; ++i) {
      w[i] = 0;
#pragma unroll
      for (int e = P - 1; e >= 0; --e) w[i] = (w[i] << B) + __float_as_uint(c[8 * j + P * i + e]);
      w[i] -= base;
    }
    uint8_t* dst = row + (j * 4 + m) * B;
    if constexpr (B == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else if constexpr (B == 4) *reinterpret_cast<uint32_t*>(dst) = w[0];
    else *reinterpret_cast<uint16_t*>(dst) = uint16_t(w[0]);
  }
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Rotate, quantise and pack rows as they are written. The arithmetic is jolt_rotate_rows then
// jolt_quantize_pack, operation by operation (butterflies over strides 1, 2, .. D/2 in that order, the
// same roundings), so the codes are theirs bit for bit. The quotient a / scale is taken as
// a * fl(1 / scale): with both roundings it is within 1.5 * 2^-23 |q| of the exact quotient and the
// rounded one within 2^-24 |q|, so for |q| < levels + 1/2 both round to the same whole number unless
// the product lies within levels * 2^-21 of a half-integer (2^-22 |q| would do). A warp where some element does, or where some
// product leaves (-1/2, levels + 1/2) and has to be clipped (the extremes' products tell), takes the
// division for all of its rows; on Gaussian rows that is one warp in 70 at 4 bits, one in 5 at 8.
// Four lanes a row keep two of the seven butterfly stages between lanes; the others are packed adds in registers,
// and the next rows' loads are in flight meanwhile. Bound by latency, 108 instructions a row in chains that 16 warps an SM
// do not cover, and by a grid whose last round is part empty (K and V rows in blocks of their own): 8191 tokens of 8
// heads at 8 and 4 bits take 27.5 us (46 MB; 1.7 TB/s, issue slots 54% busy at 128 registers, two blocks an SM).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) k_append(const AppendArgs a) {
  constexpr int J = D / 32, N = 8 * J;  // pieces and elements of a lane
  const int lane = threadIdx.x & 31, g = lane >> 2, m = lane & 3;
  const int kv = blockIdx.y;
  const float isd = rsqrtf(float(D));
  const uint32_t neg = lane_signs<D>(a.p.seed, lane);
  const int bits = kv ? a.p.bv : a.p.bk;
  const float levels = float((1 << bits) - 1);
  const uint32_t step = gridDim.x * kWarps * 8;
  // where row r comes from (loaded) and goes to; a row that is not written runs along on zeros
  Raw8<T> raw[J];
  uint8_t* page_base;
  int row;
  auto fetch = [&](uint32_t r) {
    const T* x = nullptr;
    page_base = nullptr;
    row = 0;
    if (r < a.rows) {
      const uint32_t bi = r / uint32_t(a.p.n_kv), b = bi / uint32_t(a.n_new);
      const int h = int(r - bi * a.p.n_kv), i = int(bi - b * a.n_new);
      if (!a.counts || i < a.counts[b]) {
        const int from = a.src ? a.src[int64_t(b) * a.n_new + i] : i;
        const int len = a.p.lens[b], at = len + i;
        if (from < 0 || from >= a.n_src || len < 0 || len > (a.p.max_pages << a.p.ps_log2) - 1 - i) {
          report_error(a.err, JOLT_ERR_INVALID_ARG);
        } else {
          const int page = page_of(a.p, b, at, a.err);
          if (page >= 0) {
            page_base = a.p.pool + uint64_t(page) * a.p.page_bytes;
            row = (h << a.p.ps_log2) + (at & ((1 << a.p.ps_log2) - 1));
            x = static_cast<const T*>(a.x[kv]) + int64_t(b) * a.stride_b + int64_t(from) * a.stride_t + int64_t(h) * D;
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (x) raw[j].load(x + piece_at(j, m));
      else raw[j].zero();
    }
  };
  uint32_t base = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * 8;
  if (base < a.rows) fetch(base + g);
  for (; base < a.rows; base += step) {
    float v[N];
#pragma unroll
    for (int j = 0; j < J; ++j) raw[j].floats(v + 8 * j);
    uint8_t* const to_page = page_base;
    const int to_row = row;
    // the next rows arrive while these are worked on
    if (base + step < a.rows) fetch(base + step + g);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(__float_as_uint(v[i]) ^ ((neg << (31 - i)) & 0x80000000u));
    // stride 1 inside the packed pairs, then 2 and 4 on pairs
    f2 y[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) y[i] = f2_make(v[2 * i] + v[2 * i + 1], v[2 * i] - v[2 * i + 1]);
    const f2 minus = f2_make(-1.f, -1.f);
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1)
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (!(i & s)) {
          const f2 p = y[i], q = y[i + s];
          y[i] = f2_add(p, q);
          y[i + s] = f2_fma(q, minus, p);
        }
    // strides 8 and 16 between lanes: p + q in the lower, p - q in the upper
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1) {
      const float f = (m & s) ? -1.f : 1.f;
      const f2 ff = f2_make(f, f);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 o = f2_get(y[i]);
        const f2 other = f2_make(__shfl_xor_sync(0xffffffffu, o.x, s), __shfl_xor_sync(0xffffffffu, o.y, s));
        y[i] = f2_fma(y[i], ff, other);
      }
    }
    // strides 32 and 64 between pieces
#pragma unroll
    for (int s = 4; s < N / 2; s <<= 1)
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (!(i & s)) {
          const f2 p = y[i], q = y[i + s];
          y[i] = f2_add(p, q);
          y[i + s] = f2_fma(q, minus, p);
        }
    const f2 isd2 = f2_make(isd, isd);
    float lo = INFINITY, hi = -INFINITY;  // NaN when some element is
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      y[i] = f2_mul(y[i], isd2);
      const float2 t = f2_get(y[i]);
      lo = min_nan(lo, min_nan(t.x, t.y));
      hi = max_nan(hi, max_nan(t.x, t.y));
    }
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, s));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, s));
    }
    const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), levels)), hz = __float2half_rn(lo);
    const float sc = __half2float(hs), zero = __half2float(hz);
    const bool numeric = !(fabsf(sc) < INFINITY) || !(fabsf(zero) < INFINITY);
    const float rs = sc != 0.f ? __frcp_rn(sc) : 0.f;
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, ties to even
    float c[N], off = 0.f;
    {
      const f2 mz = f2_make(-zero, -zero), rs2 = f2_make(rs, rs), up = f2_make(kMagic, kMagic), down = f2_make(-kMagic, -kMagic);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const f2 q = f2_mul(f2_add(y[i], mz), rs2);
        const f2 r = f2_add(q, up);
        const float2 d = f2_get(f2_fma(f2_add(r, down), minus, q)), t = f2_get(r);
        c[2 * i] = t.x;
        c[2 * i + 1] = t.y;
        off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
      }
    }
    const float q_lo = (lo - zero) * rs, q_hi = (hi - zero) * rs;
    const bool plain = off < 0.5f - levels * 4.76837158203125e-7f && q_lo > -0.4375f && q_hi < levels + 0.4375f;
    if (!__all_sync(0xffffffffu, plain)) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 t = f2_get(y[i >> 1]);
        float q = 0.f;
        if (sc != 0.f) q = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn((i & 1) ? t.y : t.x, zero), sc)), 0.f), levels);
        c[i] = q + kMagic;
      }
    }
    if (to_page) {
      uint8_t* dst = to_page + (kv ? a.p.vc : a.p.kc) + int64_t(to_row) * (D * bits / 8);
      if (bits == 4) store_codes<4, J>(c, dst, m);
      else if (bits == 8) store_codes<8, J>(c, dst, m);
      else store_codes<2, J>(c, dst, m);
      if (m == 0) reinterpret_cast<__half2*>(to_page + (kv ? a.p.vs : a.p.ks))[to_row] = __halves2half2(hs, hz);
      if (numeric) report_error(a.err, JOLT_ERR_NUMERIC);
    }
  }
}

struct ReadArgs {
  PagesDev p;
  void* out[2];
  const int32_t* start;
  int64_t stride_b, stride_h;
  int32_t* err;
  int n_out;
};

// Words of this lane's pieces of a row, as code_pair takes them. Two bits: pieces 2i and 2i+1 share word i.
template <int B, int J>
__device__ __forceinline__ void load_codes(const uint8_t* row, int m, uint32_t (&w)[J * B / 4]) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const uint8_t* src = row + (j * 4 + m) * B;
    if constexpr (B == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(src);
      w[2 * j] = v.x;
      w[2 * j + 1] = v.y;
    } else if constexpr (B == 4) {
      w[j] = *reinterpret_cast<const uint32_t*>(src);
    } else {
      const uint32_t v = *reinterpret_cast<const uint16_t*>(src);
      w[j / 2] = (j & 1) ? (w[j / 2] | (v << 16)) : v;
    }
  }
}

// Sixteen rows (16 aligned tokens of one head, so of one page) a warp. With the codes centred,
//   H (scale c + zero) = scale (H c') + (D (zero + o scale)) e_0,   o = 2^(b-1),
// so the Hadamard transform runs on whole numbers, exactly: four of the feature index's bits (those of
// a pair's place among the k-slots of one m16n8k16 step) by MMAs with a matrix of signs, the others (the
// step's) by butterflies of the accumulators. One rounding for scale / sqrt(D), one product, one
// rounding to the output's type. Bound by latency at 16 warps an SM (32 instructions a row; a store covers 64 bytes of
// one), at 72% of the copy rate:
// 65536 tokens of 8 heads at 4 bits into bf16 take 71.9 us (340 MB, 4.7 TB/s, issue slots 48% busy).
template <typename T, int D, int B>
__device__ __forceinline__ void read_tile(const uint32_t (&w)[2][D * B / 128], const __half2 (&szs)[2], int g, int m, float isd,
                                          uint32_t neg, T* out, int64_t first, int lo, int hi) {
  constexpr int J = D / 32, NS = D / 16, W = J * B / 4;
  // sign matrix: rows k = (lane m, register x, half hi), columns n = nt*8 + (m' * 2 + c): the output
  // bit of m is m', that of x is c, that of hi is nt
  const int mm = (g >> 1) & 3, c = g & 1;
  const uint32_t s0 = (__popc(m & mm) & 1) ? 0xBC00BC00u : 0x3C003C00u;  // (-1, -1) or (1, 1)
  const uint32_t s1 = c ? s0 ^ 0x80008000u : s0;
  f2 acc[NS][2][2];
#pragma unroll
  for (int st = 0; st < NS; ++st) {
    uint32_t a[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      a[2 * x] = code_pair<B, W>(w[0], 2 * st + x);
      a[2 * x + 1] = code_pair<B, W>(w[1], 2 * st + x);
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t flip = nt ? 0x80000000u : 0u;
      mma_f16_16816(d, a, s0 ^ flip, s1 ^ flip);
      acc[st][nt][0] = f2_make(d[0], d[1]);
      acc[st][nt][1] = f2_make(d[2], d[3]);
    }
  }
  const f2 minus = f2_make(-1.f, -1.f);
#pragma unroll
  for (int s = 1; s < NS; s <<= 1)
#pragma unroll
    for (int st = 0; st < NS; ++st)
      if (!(st & s)) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const f2 p = acc[st][nt][r], q = acc[st + s][nt][r];
            acc[st][nt][r] = f2_add(p, q);
            acc[st + s][nt][r] = f2_fma(q, minus, p);
          }
      }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int t = g + 8 * r;
    if (t < lo || t >= hi) continue;
    const float2 sz = __half22float2(szs[r]);
    const float f = sz.x * isd;
    const f2 ff = f2_make(f, f);
    const float z0 = m == 0 ? (sz.y + float(1 << (B - 1)) * sz.x) * (isd * float(D)) : 0.f;
    T* dst = out + (first + t) * D;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        // where the transform left element (j, e): see code_pair's order of a word's codes
        const int st = B == 2 ? (j >> 1) * 4 + (e >> 1) : B == 4 ? 2 * j + ((e >> 1) & 1) : 2 * j + (e >> 2);
        const int nt = B == 2 ? j & 1 : B == 4 ? e >> 2 : (e >> 1) & 1;
        float2 x = f2_get(f2_mul(acc[st][nt][r], ff));
        if (j == 0 && e == 0) x.x += z0;
        v[e] = __uint_as_float(__float_as_uint(x.x) ^ ((neg << (31 - 8 * j - e)) & 0x80000000u));
        v[e + 1] = __uint_as_float(__float_as_uint(x.y) ^ ((neg << (30 - 8 * j - e)) & 0x80000000u));
      }
#pragma unroll
      for (int i = 0; i < int(sizeof(T)) / 2; ++i)
        reinterpret_cast<uint4*>(dst + piece_at(j, m))[i] = pack16<T>(v + 16 / int(sizeof(T)) * i);
    }
  }
}

// The tiles of a warp, each one's codes loaded while the one before is worked on, and its table entry
// before that. A tile without a page (reported) is read from page 0 and not written.
template <typename T, int D, int B>
__device__ __forceinline__ void read_tiles(const ReadArgs& a, int kv, int h, int b, int g, int m, int from, int end, T* out,
                                           uint32_t neg) {
  constexpr int W = D * B / 128;
  const float isd = rsqrtf(float(D));
  const int ps = 1 << a.p.ps_log2;
  const int32_t* entries = a.p.table + int64_t(b) * a.p.max_pages;
  const int step = gridDim.x * kWarps, last = (end - 1) >> 4;
  int t = (from >> 4) + blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t > last) return;
  uint32_t w[2][W];
  __half2 sz[2];
  auto load = [&](int tile, int id) {
    const bool ok = uint32_t(id) < uint32_t(a.p.n_pages);
    if (!ok) report_error(a.err, JOLT_ERR_INVALID_ARG);
    const uint8_t* base = a.p.pool + (ok ? uint64_t(uint32_t(id)) * a.p.page_bytes : 0);
    const uint32_t row = uint32_t(h) * ps + ((tile * 16) & (ps - 1)) + g;
    const uint8_t* codes = base + (kv ? a.p.vc : a.p.kc) + uint64_t(row) * (D * B / 8);
    const __half2* s = reinterpret_cast<const __half2*>(base + (kv ? a.p.vs : a.p.ks)) + row;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      load_codes<B, D / 32>(codes + 8 * r * (D * B / 8), m, w[r]);
      sz[r] = s[8 * r];
    }
    return ok;
  };
  bool ok = load(t, entries[(t * 16) >> a.p.ps_log2]);
  int id = t + step <= last ? entries[((t + step) * 16) >> a.p.ps_log2] : 0;
  while (true) {
    uint32_t now[2][W];
    __half2 now_sz[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int i = 0; i < W; ++i) now[r][i] = w[r][i];
      now_sz[r] = sz[r];
    }
    const bool now_ok = ok;
    const int next = t + step;
    if (next <= last) {
      ok = load(next, id);
      if (next + step <= last) id = entries[((next + step) * 16) >> a.p.ps_log2];
    }
    if (now_ok) read_tile<T, D, B>(now, now_sz, g, m, isd, neg, out, int64_t(t) * 16 - from, from - t * 16, end - t * 16);
    if (next > last) return;
    t = next;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) k_read(const ReadArgs a) {
  const int lane = threadIdx.x & 31, g = lane >> 2, m = lane & 3;
  const int kv = blockIdx.y >= a.p.n_kv, h = blockIdx.y - kv * a.p.n_kv, b = blockIdx.z;
  T* out = static_cast<T*>(a.out[kv]);
  if (!out) return;
  const int from = a.start ? a.start[b] : 0;
  if (from < 0) {
    report_error(a.err, JOLT_ERR_INVALID_ARG);
    return;
  }
  const int len = pages_len(a.p, b, a.err);
  if (from >= len) return;
  const int end = from + min(a.n_out, len - from);
  out += int64_t(b) * a.stride_b + int64_t(h) * a.stride_h;
  const uint32_t neg = lane_signs<D>(a.p.seed, lane);
  const int bits = kv ? a.p.bv : a.p.bk;
  if (bits == 4) read_tiles<T, D, 4>(a, kv, h, b, g, m, from, end, out, neg);
  else if (bits == 8) read_tiles<T, D, 8>(a, kv, h, b, g, m, from, end, out, neg);
  else read_tiles<T, D, 2>(a, kv, h, b, g, m, from, end, out, neg);
}

// Checks shared by the calls over a pool.
bool pool_args_ok(const jolt_pages* p, const void* pool, const int32_t* table, int32_t max_pages,
                  const int32_t* lens, int32_t batch) {
  if (!pages_ok(p) || max_pages < 1 || batch < 0 || batch > 65535) return false;
  if (int64_t(max_pages) * p->page_size > (int64_t(1) << 24)) return false;
  if (batch == 0) return true;
  return pool && table && lens && aligned(pool, 16) && aligned(table, 4) && aligned(lens, 4);
}
// Bytes of a K row, of a V row, or of both: coded, and as given.
double row_bytes(const jolt_pages& p, bool k, bool v) {
  const double plain = double(p.d_h) * dtype_bytes(p.io_dtype) + 4;
  return (k ? p.d_h * p.b_k / 8 + plain : 0.0) + (v ? p.d_h * p.b_v / 8 + plain : 0.0);
}
}  // namespace
}  // namespace jolt

using namespace jolt;

extern "C" jolt_status jolt_pages_append(const jolt_pages* pages, void* pool, const int32_t* table,
                                         int32_t max_pages, const int32_t* lens, int32_t batch, int32_t n_new,
                                         const int32_t* counts, const int32_t* src, int32_t n_src, const void* k,
                                         const void* v, int64_t stride_b, int64_t stride_t, int32_t* err,
                                         void* stream) {
  if (!pool_args_ok(pages, pool, table, max_pages, lens, batch) || n_new < 0 || n_src < 0) return JOLT_ERR_INVALID_ARG;
  if (batch == 0 || n_new == 0) return JOLT_OK;
  if (!k || !v || (!src && n_new > n_src) || !rows_ok(k, stride_b, stride_t) || !rows_ok(v, stride_b, stride_t))
    return JOLT_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(src, 4) || !aligned(err, 4)) return JOLT_ERR_INVALID_ARG;
  const int64_t rows = int64_t(batch) * n_new * pages->n_kv;
  if (rows >= int64_t(1) << 31) return JOLT_ERR_INVALID_ARG;
  AppendArgs a{};
  a.p = pages_dev(*pages, pool, table, max_pages, lens);
  a.x[0] = k;
  a.x[1] = v;
  a.counts = counts;
  a.src = src;
  a.stride_b = stride_b;
  a.stride_t = stride_t;
  a.rows = uint32_t(rows);
  a.err = err;
  a.n_new = n_new;
  a.n_src = n_src;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(unsigned(std::min<int64_t>((rows + kWarps * 8 - 1) / (kWarps * 8), kSmCount * 2)), 2);
  const bool f32 = pages->io_dtype == JOLT_F32;
  StatScope sc(JOLT_K_PAGES, st, 0.0, double(rows) * row_bytes(*pages, true, true));
  if (pages->d_h == 128) {
    if (f32) k_append<float, 128><<<grid, kThreads, 0, st>>>(a);
    else k_append<__nv_bfloat16, 128><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (f32) k_append<float, 64><<<grid, kThreads, 0, st>>>(a);
    else k_append<__nv_bfloat16, 64><<<grid, kThreads, 0, st>>>(a);
  }
  JOLT_CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}

extern "C" jolt_status jolt_pages_read(const jolt_pages* pages, const void* pool, const int32_t* table,
                                       int32_t max_pages, const int32_t* lens, int32_t batch, const int32_t* start,
                                       int32_t n_out, void* k_out, void* v_out, int64_t stride_b, int64_t stride_h,
                                       int32_t* err, void* stream) {
  if (!pool_args_ok(pages, pool, table, max_pages, lens, batch) || n_out < 0) return JOLT_ERR_INVALID_ARG;
  if (batch == 0 || n_out == 0) return JOLT_OK;
  if ((!k_out && !v_out) || !rows_ok(k_out, stride_b, stride_h) || !rows_ok(v_out, stride_b, stride_h))
    return JOLT_ERR_INVALID_ARG;
  if (!aligned(start, 4) || !aligned(err, 4)) return JOLT_ERR_INVALID_ARG;
  // rows of different heads or sequences must not fall on one another: the heads' lie between the sequences', or
  // the other way round
  const int64_t row = int64_t(n_out) * pages->d_h, nh = pages->n_kv;
  auto nested = [row](int64_t inner, int64_t n_inner, int64_t outer, int64_t n_outer) {
    return (n_inner == 1 || inner >= row) &&
           (n_outer == 1 || (outer >= row && (n_inner == 1 || (outer - row) / (n_inner - 1) >= inner)));
  };
  if (!nested(stride_h, nh, stride_b, batch) && !nested(stride_b, batch, stride_h, nh)) return JOLT_ERR_INVALID_ARG;
  ReadArgs a{};
  a.p = pages_dev(*pages, pool, table, max_pages, lens);
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.start = start;
  a.stride_b = stride_b;
  a.stride_h = stride_h;
  a.err = err;
  a.n_out = n_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // tiles of 16 aligned tokens that n_out rows can touch, and warps for them until the GPU is full
  const int64_t tiles = (int64_t(n_out) + 30) / 16, lines = int64_t(batch) * pages->n_kv * 2;
  const int64_t most = std::max<int64_t>(1, (kSmCount * 8 + lines - 1) / lines);
  const dim3 grid(unsigned(std::min((tiles + kWarps - 1) / kWarps, most)), 2 * pages->n_kv, batch);
  const bool f32 = pages->io_dtype == JOLT_F32;
  StatScope sc(JOLT_K_PAGES, st, 0.0, double(batch) * n_out * pages->n_kv * row_bytes(*pages, k_out, v_out));
  if (pages->d_h == 128) {
    if (f32) k_read<float, 128><<<grid, kThreads, 0, st>>>(a);
    else k_read<__nv_bfloat16, 128><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (f32) k_read<float, 64><<<grid, kThreads, 0, st>>>(a);
    else k_read<__nv_bfloat16, 64><<<grid, kThreads, 0, st>>>(a);
  }
  JOLT_CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}
