// Rows of storage elements in chunks of 16 bytes per lane (the norms, the
// quantisers).
#pragma once

#include "common.hpp"

namespace twell {

// How a kernel reads and writes its rows, in chunks of 16 bytes.
enum class Rows {
  WHOLE,  // all 16-byte aligned and a whole number of chunks
  ANY,    // aligned to the element only, at least one chunk long
  TINY,   // shorter than one chunk
};

// A row of d elements; `p` is the same for a whole wave.
//
// WHOLE rows go through a buffer descriptor of exactly their bytes, so that
// chunks past the end load zeros and store nothing, with no branch.
//
// ANY rows go through 16-byte accesses at the element's alignment.  The chunk
// that crosses the end, and those past it, load the row's last 16 bytes
// instead; trim() then moves the row's elements into place and zeroes the
// others.  It is apart from load() because it needs the loaded value: a row's
// loads are all under way before the first is waited for.  The crossing chunk
// is stored by elements.  8192 x 2047 bf16 with residual: 30 us (25 at 2048),
// element by element 84, as each load is waited for by itself.
//
// Stores of whole rows (h, y, dx) carry the non-temporal bit: written this way
// they leave L2 to the inputs (bf16, 8192 x 2048 with residual and 8 bits:
// 29.6 -> 23.4 us, and no slower with the product that reads them behind it).
// Stores of q do not: its reader then misses (the quantiser of 8192 x 8192
// and the 8-bit product together 151 against 160 us).  Loads carry the bit
// (NT) where no other kernel's copy in cache is worth keeping: in the
// quantiser (36.3 -> 32.8 us) and the gradient (16384 x 4096: 96 -> 89 us);
// in the norm it costs 4 us, as x and residual come from the kernel before.
// ANY rows share lines between waves, and the bit drops them in between: the
// quantiser loads those without it (8192 x 2047 fp32: 16.3 -> 14.1 us; the
// gradient does not gain, 51.8 -> 55.7), and the gradient stores them without
// it (16384 x 4095 fp32: 195 -> 168 us; the norm does not gain).
constexpr int NON_TEMPORAL = 2;

// The offset stays 32-bit and apart from the row's address, which is in scalar
// registers: the compiler otherwise adds the two first and keeps a 64-bit address
// per access (up to 19 more vector registers, and spills).
__device__ __forceinline__ void keep_offset(uint32_t &at) { asm volatile("" : "+v"(at)); }

typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

// A chunk without its first n bytes (a multiple of the element's size S), zeros
// behind the others.
template <int S>
__device__ __forceinline__ u32x4_t drop_bytes(u32x4_t w, int n) {
  u32x4_t v = w;
  if constexpr (S == 2) {
    const bool half = (n & 2) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = half ? (v[i] >> 16) | (i < 3 ? w[i < 3 ? i + 1 : 3] << 16 : 0u) : v[i];
  }
  const bool one = (n & 4) != 0, two = (n & 8) != 0, all = n >= 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = one ? (i < 3 ? v[i < 3 ? i + 1 : 3] : 0u) : v[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = two ? (i < 2 ? w[i < 2 ? i + 2 : 3] : 0u) : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = all ? 0u : w[i];
  return w;
}

template <Dt D, Rows R, bool NT = false>
struct Row {
  using T = typename DtT<D>::T;
  static constexpr int E = 16 / DtT<D>::size;  // elements per chunk
  __amdgpu_buffer_rsrc_t rsrc;
  T *p;
  int d;

  __device__ __forceinline__ Row(const void *base, int64_t t, int64_t ld, int d_)
      : p(const_cast<T *>(static_cast<const T *>(base)) + t * ld), d(d_) {
    if constexpr (R == Rows::WHOLE) rsrc = __builtin_amdgcn_make_buffer_rsrc(p, 0, d * (int)sizeof(T), 0x00020000);
  }
  // elements e0 .. e0 + E - 1, +0 past the end; of ANY rows after trim()
  __device__ __forceinline__ u32x4_t load(int e0) const {
    if constexpr (R == Rows::WHOLE) {
      return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rsrc, e0 * (int)sizeof(T), 0, NT ? NON_TEMPORAL : 0));
    } else if constexpr (R == Rows::ANY) {
      if (__builtin_amdgcn_readfirstlane(e0) >= d) return u32x4_t{0u, 0u, 0u, 0u};  // nothing for this wave
      uint32_t at = min((uint32_t)e0, (uint32_t)(d - E)) * (uint32_t)sizeof(T);
      keep_offset(at);
      const u32x4_any_t *q = reinterpret_cast<const u32x4_any_t *>(reinterpret_cast<const char *>(p) + at);
      if constexpr (NT)
        return __builtin_nontemporal_load(q);
      else
        return *q;
    } else {
      u32x4_t w = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (e0 + i < d) {
          if constexpr (D == Dt::BF16)
            w[i / 2] |= (uint32_t)p[e0 + i] << (16 * (i % 2));
          else
            w[i] = __float_as_uint(p[e0 + i]);
        }
      }
      return w;
    }
  }
  __device__ __forceinline__ u32x4_t trim(u32x4_t w, int e0) const {
    if constexpr (R == Rows::ANY) {
      if (__builtin_amdgcn_readfirstlane(e0) + 64 * E > d) {  // the wave's chunks reach the end
        w = drop_bytes<(int)sizeof(T)>(w, max(e0 - (d - E), 0) * (int)sizeof(T));
      }
    }
    return w;
  }
  template <bool NTS = true>
  __device__ __forceinline__ void store(int e0, u32x4_t w) const {
    if constexpr (R == Rows::WHOLE) {
      __builtin_amdgcn_raw_buffer_store_b128(w, rsrc, e0 * (int)sizeof(T), 0, NON_TEMPORAL);
    } else if (R == Rows::ANY && e0 + E <= d) {
      uint32_t at = (uint32_t)e0 * (uint32_t)sizeof(T);
      keep_offset(at);
      u32x4_any_t *q = reinterpret_cast<u32x4_any_t *>(reinterpret_cast<char *>(p) + at);
      if constexpr (NTS)
        __builtin_nontemporal_store(w, q);
      else
        *q = w;
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (e0 + i < d) {
          if constexpr (D == Dt::BF16)
            p[e0 + i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
          else
            p[e0 + i] = __uint_as_float(w[i]);
        }
      }
    }
  }
};

template <Dt D>
__device__ __forceinline__ void unpack(u32x4_t w, float (&v)[16 / DtT<D>::size]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (D == Dt::BF16) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}

// Rounds to the storage type.
template <Dt D>
__device__ __forceinline__ u32x4_t pack_chunk(const float (&v)[16 / DtT<D>::size]) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (D == Dt::BF16)
      w[i] = (uint32_t)bf16_rne(v[2 * i]) | ((uint32_t)bf16_rne(v[2 * i + 1]) << 16);
    else
      w[i] = __float_as_uint(v[i]);
  }
  return w;
}

}  // namespace twell
