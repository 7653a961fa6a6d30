// Microscaled 4-bit rows: blocks of 32 elements along a row share a scale 2^e.
//
//   e = the smallest whole number with max |z| <= 7 * 2^e, kept in -126 ... 126
//   code = nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to |z| / 2^e (ties to the even
//          code; above 6: 6), sign in bit 3
//
// The largest element of a block lies in (3.5, 7] times 2^e, so it is at most
// 1 * 2^e off: half the step between 4 and 6, as everywhere else on the grid.  (A
// scale of the largest element's own exponent less 2 would leave up to 8 * 2^e,
// and 2 * 2^e of error.)  Everything here is a matter of the bits of z, so codes and
// scales are the same however the work is split.
//
// A block with an infinite or NaN element gets the scale byte 255 (NaN) and
// codes 0; the matrix cores take that byte as NaN too.
#pragma once

#include "common.hpp"

namespace twell {

constexpr int MX4_BLOCK = 32;
constexpr int MX4_GROUP = 512;  // elements whose 16 scale bytes lie together

// The place of block b's scale byte in its row.  The 16 bytes of a group of 16
// blocks are kept transposed (4 x 4): the matrix instruction takes blocks 4 s ... 4 s
// + 3 in step s, one per quarter of the wave, and so finds the bytes of four
// steps in one dword per lane, without a shift.
__host__ __device__ __forceinline__ int mx4_place(int b) { return (b & ~15) | ((b & 3) << 2) | ((b >> 2) & 3); }

// Scale byte of a block whose largest |z| has these bits; 255 for inf and NaN.
// Adding 2^21 - 1 carries into the exponent where the mantissa is over 1.75.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t top) {
  const int e = (int)((top + 0x1FFFFFu) >> 23) - 2;
  return top >= 0x7F800000u ? 255u : (uint32_t)max(e, 1);
}

// The largest of v over the lanes of a block: 4 lanes of 8 elements, or 8 of 4.
template <int E>
__device__ __forceinline__ uint32_t mx4_block_top(uint32_t v) {
  static_assert(E == 8 || E == 4, "a 16-byte chunk per lane");
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
  if constexpr (E == 4)
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
  return v;
}

// E elements of a lane to codes, the first one in the lowest bits.  The lanes of a
// block (consecutive, the first a multiple of their number) are active
// together; `byte`: the block's scale.
template <int E>
__device__ __forceinline__ uint32_t mx4_codes(const float (&z)[E], uint32_t &byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(z[i]) & 0x7FFFFFFFu);
  byte = mx4_scale(mx4_block_top<E>(top));
  const float scale = __uint_as_float(byte << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[0], z[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[2], z[3], scale, 1);
  if constexpr (E == 8) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[4], z[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[6], z[7], scale, 3);
  }
  return byte == 255u ? 0u : w;
}

// Stores a lane's codes at element e0 of a row of d elements, and the block's
// scale byte by its first lane.  Nothing past the row's last byte and last block
// is written.
template <int E>
__device__ __forceinline__ void mx4_store(uint8_t *q, uint8_t *scale, int e0, int d, uint32_t w, uint32_t byte) {
  uint8_t *p = q + (e0 >> 1);
  if (e0 + E <= d) {
    if constexpr (E == 8)
      *reinterpret_cast<uint32_t *>(p) = w;
    else
      *reinterpret_cast<uint16_t *>(p) = (uint16_t)w;
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 2)
      if (e0 + i < d) p[i / 2] = (uint8_t)(w >> (4 * i));
  }
  if (e0 % MX4_BLOCK == 0 && e0 < d) scale[mx4_place(e0 / MX4_BLOCK)] = (uint8_t)byte;
}

}  // namespace twell
