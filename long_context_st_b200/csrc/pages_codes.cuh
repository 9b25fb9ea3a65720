// Packed codes of the tail cache as f16 MMA operands, centred: c - 2^(b-1), a whole number in
// [-2^(b-1), 2^(b-1)), exact in f16. As in mma_codes.cuh the field is set into the mantissa of 1024
// and one f16x2 add or fused multiply-add with constants takes the offset (here with the centre)
// and the field's shift away; every intermediate is exact.
#pragma once
#include "mma_codes.cuh"

namespace jolt {

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[W]) {
  static_assert(W == 1 || W == 2 || W == 4 || W == 8, "");
  if constexpr (W == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
}

// Fields at bit `sub * B` of each 16-bit half of x.
template <int B>
__device__ __forceinline__ uint32_t centred(uint32_t x, int sub) {
  if constexpr (B == 8) {
    return h2_add(field_or(x, 0x00FF00FFu), 0xE480E480u);  // - 1024 - 128
  } else if constexpr (B == 4) {
    return sub ? h2_fma(field_or(x, 0x00F000F0u), 0x2C002C00u, 0xD480D480u)  // / 16 - 64 - 8
               : h2_add(field_or(x, 0x000F000Fu), 0xE408E408u);              // - 1024 - 8
  } else {
    switch (sub) {
      case 0: return h2_add(field_or(x, 0x00030003u), 0xE402E402u);                // - 1024 - 2
      case 1: return h2_fma(field_or(x, 0x000C000Cu), 0x34003400u, 0xDC08DC08u);   // / 4 - 256 - 2
      case 2: return h2_fma(field_or(x, 0x00300030u), 0x2C002C00u, 0xD420D420u);   // / 16 - 64 - 2
      default: return h2_fma(field_or(x, 0x00C000C0u), 0x24002400u, 0xCC80CC80u);  // / 64 - 16 - 2
    }
  }
}

// Pair `i` of a run of words: with n = 32 / B codes a word, word i / (n/2), its codes p and p + n/2,
// p = i % (n/2) (what one mask over both halves of the word gives).
template <int B, int W>
__device__ __forceinline__ uint32_t code_pair(const uint32_t (&w)[W], int i) {
  constexpr int H = 16 / B;
  const int p = i % H;
  const uint32_t x = w[i / H];
  constexpr int S = 8 / B;  // fields a byte
  return centred<B>(p >= S ? x >> 8 : x, p % S);
}

// Code `j` of the rows held in x and y, as the pair (x_j, y_j).
template <int B, int W>
__device__ __forceinline__ uint32_t code_across(const uint32_t (&x)[W], const uint32_t (&y)[W], int j) {
  const int bit = j * B;
  return centred<B>(bytes_xy(x[bit / 32], y[bit / 32], (bit % 32) / 8), (bit % 8) / B);
}

// The fields themselves: whole numbers c 2^-24 as f16 bits (subnormals), times 2^(a field's place in its byte).
template <int B, int W>
__device__ __forceinline__ uint32_t field_pair(const uint32_t (&w)[W], int i) {
  constexpr int H = 16 / B, F = 8 / B;  // pairs a word, fields a byte
  const int p = i % H;
  const uint32_t x = p >= F ? w[i / H] >> 8 : w[i / H];
  return x & (0x00010001u * (((1u << B) - 1) << (B * (p % F))));
}
// Field `j` of the rows held in x and y, as the pair (x_j, y_j).
template <int B, int W>
__device__ __forceinline__ uint32_t field_across(const uint32_t (&x)[W], const uint32_t (&y)[W], int j) {
  const int bit = j * B;
  return bytes_xy(x[bit / 32], y[bit / 32], (bit % 32) / 8) & (0x00010001u * (((1u << B) - 1) << (bit % 8)));
}

}  // namespace jolt
