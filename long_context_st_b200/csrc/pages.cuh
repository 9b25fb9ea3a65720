// Layout of the tail cache's pages and the device-side checks every kernel over them makes.
#pragma once
#include <cstdint>

#include "jolt_internal.h"

namespace jolt {

bool pages_ok(const jolt_pages* p);
inline bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }  // NULL is

// Rows of K, V or q with these element strides can be loaded 16 bytes at a time.
inline bool rows_ok(const void* x, int64_t s0, int64_t s1) {
  return aligned(x, 16) && s0 >= 0 && s1 >= 0 && s0 % 8 == 0 && s1 % 8 == 0;
}

// Byte offsets of a page's segments and its size.
struct PageLayout {
  uint32_t kc, ks, vc, vs;
  uint64_t bytes;
};
inline PageLayout page_layout(const jolt_pages& p) {
  const uint64_t rows = uint64_t(p.n_kv) * p.page_size;
  PageLayout l;
  uint64_t at = 0;
  l.kc = uint32_t(at); at += rows * (p.d_h * p.b_k / 8);
  l.ks = uint32_t(at); at += rows * 4;
  l.vc = uint32_t(at); at += rows * (p.d_h * p.b_v / 8);
  l.vs = uint32_t(at); at += rows * 4;
  l.bytes = align_up(at, kSegAlign);
  return l;
}

// What every kernel over pages needs of them.
struct PagesDev {
  uint8_t* pool;
  const int32_t* table;
  const int32_t* lens;
  uint64_t page_bytes, seed;
  uint32_t kc, ks, vc, vs;  // segment offsets in a page
  int32_t n_pages, max_pages, ps_log2, n_kv, bk, bv;
};
inline PagesDev pages_dev(const jolt_pages& p, const void* pool, const int32_t* table, int32_t max_pages,
                          const int32_t* lens) {
  const PageLayout l = page_layout(p);
  PagesDev d{};
  d.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  d.table = table;
  d.lens = lens;
  d.page_bytes = l.bytes;
  d.seed = p.rot_seed;
  d.kc = l.kc; d.ks = l.ks; d.vc = l.vc; d.vs = l.vs;
  d.n_pages = p.n_pages;
  d.max_pages = max_pages;
  d.ps_log2 = p.page_size == 16 ? 4 : p.page_size == 32 ? 5 : p.page_size == 64 ? 6 : 7;
  d.n_kv = p.n_kv;
  d.bk = p.b_k;
  d.bv = p.b_v;
  return d;
}

#if defined(__CUDACC__)
// Tokens sequence b holds, clamped to what its table row can name.
__device__ __forceinline__ int pages_len(const PagesDev& p, int b, int32_t* err) {
  const int len = p.lens[b], most = p.max_pages << p.ps_log2;
  if (len < 0 || len > most) {
    report_error(err, JOLT_ERR_INVALID_ARG);
    return len < 0 ? 0 : most;
  }
  return len;
}
// Page that holds token t of sequence b, or -1 (reported) when the table names none.
__device__ __forceinline__ int page_of(const PagesDev& p, int b, int t, int32_t* err) {
  const int id = p.table[int64_t(b) * p.max_pages + (t >> p.ps_log2)];
  if (id < 0 || id >= p.n_pages) {
    report_error(err, JOLT_ERR_INVALID_ARG);
    return -1;
  }
  return id;
}
#endif

}  // namespace jolt
