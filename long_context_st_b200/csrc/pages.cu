// jolt_pages_append / jolt_pages_read: the tail cache's rows coded as they are written, and read back.
#include "common.cuh"
#include "pages.cuh"

namespace jolt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// E elements of a row at lane*E, as floats.
template <int E>
__device__ __forceinline__ void load_row(const float* p, float (&v)[E]) {
  if constexpr (E == 4) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x; v[1] = f.y;
  }
}
template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&v)[E]) {
  uint32_t w[E / 2];
  if constexpr (E == 4) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    w[0] = r.x; w[1] = r.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <int E>
__device__ __forceinline__ void store_row(float* p, const float (&v)[E]) {
  if constexpr (E == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
}
template <int E>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&v)[E]) {
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if constexpr (E == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(p) = w[0];
}

struct AppendArgs {
  PagesDev p;
  const void* k;
  const void* v;
  const int32_t* counts;
  const int32_t* src;
  int64_t stride_b, stride_t, rows;
  int32_t* err;
  int n_new, n_src;
};

// One warp a row: rotate, quantise, pack. The arithmetic is jolt_rotate_rows then
// jolt_quantize_pack, operation by operation, so the codes are theirs bit for bit.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads) k_append(const AppendArgs a) {
  constexpr int D = 32 * E;
  const int lane = threadIdx.x & 31;
  const float isd = rsqrtf(float(D));
  float sign[E];
#pragma unroll
  for (int i = 0; i < E; ++i) sign[i] = rot_sign(a.p.seed, lane * E + i);
  const int64_t warps = int64_t(gridDim.x) * kWarps;
  for (int64_t r = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < a.rows; r += warps) {
    const int kv = int(r & 1);
    const int64_t r2 = r >> 1;
    const int h = int(r2 % a.p.n_kv);
    const int64_t bi = r2 / a.p.n_kv;
    const int i = int(bi % a.n_new), b = int(bi / a.n_new);
    if (a.counts && i >= a.counts[b]) continue;
    const int from = a.src ? a.src[int64_t(b) * a.n_new + i] : i;
    const int at = pages_len(a.p, b, a.err) + i;
    if (from < 0 || from >= a.n_src || at >= (a.p.max_pages << a.p.ps_log2)) {
      report_error(a.err, JOLT_ERR_INVALID_ARG);
      continue;
    }
    const int page = page_of(a.p, b, at, a.err);
    if (page < 0) continue;
    const T* x = static_cast<const T*>(kv ? a.v : a.k) + int64_t(b) * a.stride_b + int64_t(from) * a.stride_t +
                 int64_t(h) * D + lane * E;
    float v[E];
    load_row<E>(x, v);
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] *= sign[j];
    warp_fwht<E>(v);
    float bad = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      v[j] *= isd;
      bad += v[j] * 0.f;
    }
    const int bits = kv ? a.p.bv : a.p.bk;
    uint8_t c[E];
    __half hs, hz;
    const bool ok = warp_quantize<E>(v, bits, c, &hs, &hz) && bad == 0.f;
    if (!ok) report_error(a.err, JOLT_ERR_NUMERIC);
    uint32_t packed = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) packed |= uint32_t(c[j]) << (j * bits);
    uint8_t* base = a.p.pool + uint64_t(page) * a.p.page_bytes;
    const int row = (h << a.p.ps_log2) + (at & ((1 << a.p.ps_log2) - 1));
    uint8_t* dst = base + (kv ? a.p.vc : a.p.kc) + int64_t(row) * (D * bits / 8);
    const int mine = E * bits;  // bits of this lane
    if (mine == 32) {
      reinterpret_cast<uint32_t*>(dst)[lane] = packed;
    } else if (mine == 16) {
      reinterpret_cast<uint16_t*>(dst)[lane] = uint16_t(packed);
    } else if (mine == 8) {
      dst[lane] = uint8_t(packed);
    } else {
      const uint32_t next = __shfl_down_sync(0xffffffffu, packed, 1);
      if (!(lane & 1)) dst[lane >> 1] = uint8_t(packed | (next << 4));
    }
    if (lane == 0)
      reinterpret_cast<__half2*>(base + (kv ? a.p.vs : a.p.ks))[row] = __halves2half2(hs, hz);
  }
}

struct ReadArgs {
  PagesDev p;
  void* out[2];
  const int32_t* start;
  int64_t stride_b, stride_h, rows;
  int32_t* err;
  int n_out;
};

// One warp a row: unpack, dequantise, rotate back.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads) k_read(const ReadArgs a) {
  constexpr int D = 32 * E;
  const int lane = threadIdx.x & 31;
  const float isd = rsqrtf(float(D));
  float back[E];
#pragma unroll
  for (int i = 0; i < E; ++i) back[i] = isd * rot_sign(a.p.seed, lane * E + i);
  const int64_t warps = int64_t(gridDim.x) * kWarps;
  for (int64_t r = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < a.rows; r += warps) {
    const int i = int(r % a.n_out);
    const int64_t r2 = r / a.n_out;
    const int kv = int(r2 & 1);
    const int h = int((r2 >> 1) % a.p.n_kv), b = int((r2 >> 1) / a.p.n_kv);
    T* out = static_cast<T*>(a.out[kv]);
    if (!out) continue;
    const int from = a.start ? a.start[b] : 0;
    if (from < 0) {
      report_error(a.err, JOLT_ERR_INVALID_ARG);
      continue;
    }
    const int len = pages_len(a.p, b, a.err);
    if (from >= len || i >= len - from) continue;
    const int at = from + i;
    const int page = page_of(a.p, b, at, a.err);
    if (page < 0) continue;
    const int bits = kv ? a.p.bv : a.p.bk;
    const uint8_t* base = a.p.pool + uint64_t(page) * a.p.page_bytes;
    const int row = (h << a.p.ps_log2) + (at & ((1 << a.p.ps_log2) - 1));
    const uint8_t* codes = base + (kv ? a.p.vc : a.p.kc) + int64_t(row) * (D * bits / 8);
    const int mine = E * bits;
    uint32_t packed;
    if (mine == 32) packed = reinterpret_cast<const uint32_t*>(codes)[lane];
    else if (mine == 16) packed = reinterpret_cast<const uint16_t*>(codes)[lane];
    else if (mine == 8) packed = codes[lane];
    else packed = codes[lane >> 1] >> ((lane & 1) * 4);
    const __half2 sz = reinterpret_cast<const __half2*>(base + (kv ? a.p.vs : a.p.ks))[row];
    const float s = __low2float(sz), z = __high2float(sz);
    float v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = dequant((packed >> (j * bits)) & ((1u << bits) - 1u), s, z);
    warp_fwht<E>(v);
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] *= back[j];
    store_row<E>(out + int64_t(b) * a.stride_b + int64_t(h) * a.stride_h + int64_t(i) * D + lane * E, v);
  }
}

unsigned grid_for(int64_t rows) {
  const int64_t g = (rows + kWarps - 1) / kWarps;
  return unsigned(g < 148 * 8 ? g : 148 * 8);
}

// Checks shared by the calls over a pool.
bool pool_args_ok(const jolt_pages* p, const void* pool, const int32_t* table, int32_t max_pages,
                  const int32_t* lens, int32_t batch) {
  if (!pages_ok(p) || max_pages < 1 || batch < 0) return false;
  if (int64_t(max_pages) * p->page_size > (int64_t(1) << 24)) return false;
  if (batch == 0) return true;
  return pool && table && lens && reinterpret_cast<uintptr_t>(pool) % 16 == 0;
}
bool rows_ok(const void* x, int64_t s0, int64_t s1) {
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && s0 >= 0 && s1 >= 0 && s0 % 8 == 0 && s1 % 8 == 0;
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
  AppendArgs a{};
  a.p = pages_dev(*pages, pool, table, max_pages, lens);
  a.k = k;
  a.v = v;
  a.counts = counts;
  a.src = src;
  a.stride_b = stride_b;
  a.stride_t = stride_t;
  a.rows = int64_t(batch) * n_new * pages->n_kv * 2;
  a.err = err;
  a.n_new = n_new;
  a.n_src = n_src;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = grid_for(a.rows);
  const bool f32 = pages->io_dtype == JOLT_F32;
  if (pages->d_h == 128) {
    if (f32) k_append<float, 4><<<grid, kThreads, 0, st>>>(a);
    else k_append<__nv_bfloat16, 4><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (f32) k_append<float, 2><<<grid, kThreads, 0, st>>>(a);
    else k_append<__nv_bfloat16, 2><<<grid, kThreads, 0, st>>>(a);
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
  ReadArgs a{};
  a.p = pages_dev(*pages, pool, table, max_pages, lens);
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.start = start;
  a.stride_b = stride_b;
  a.stride_h = stride_h;
  a.rows = int64_t(batch) * pages->n_kv * 2 * n_out;
  a.err = err;
  a.n_out = n_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = grid_for(a.rows);
  const bool f32 = pages->io_dtype == JOLT_F32;
  if (pages->d_h == 128) {
    if (f32) k_read<float, 4><<<grid, kThreads, 0, st>>>(a);
    else k_read<__nv_bfloat16, 4><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (f32) k_read<float, 2><<<grid, kThreads, 0, st>>>(a);
    else k_read<__nv_bfloat16, 2><<<grid, kThreads, 0, st>>>(a);
  }
  JOLT_CUDA_TRY(cudaGetLastError());
  return JOLT_OK;
}
