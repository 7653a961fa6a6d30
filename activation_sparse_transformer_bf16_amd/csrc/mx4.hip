// Rows of microscaled 4-bit floats (mx4.hpp): the quantiser and the reader.
//
// A lane takes one 16-byte chunk of x or y (8 bf16 or 4 fp32 elements), a block's lanes
// lie together, and a wave takes a piece of a row (512 or 256 elements) or, of rows
// shorter than half of that, several rows.  A workgroup takes the same piece of
// EACH * 4 (groups of) rows, each wave EACH of them at a time, whose loads are all
// under way before the first is waited for.  9 instructions an element each way, which
// hide behind the memory.
//
// Memory bound: 8192 x 8192 bf16, operands in memory, 31 us to quantise (170 MB, 5.5
// TB/s) and 28.5 to read (6.0 TB/s; a plain copy of the card moves 6.1 to 6.3); fp32 51
// and 50 (304 MB, 6.0); one row of 8192 2.5 us each.  Loads of x and stores of y
// carry the non-temporal bit: neither is read again here, and y is far longer than the
// codes.  Rows of no alignment share lines between waves: 8192 x 8191 bf16 38 us each
// way.  Their loads go without the bit, which drops the shared lines (8192 x 2047
// 11.2 us, with it 13.0; 8192 x 8191 the same), their stores with it (8192 x 8191 39 us,
// without 50; 8192 x 2047, where the Infinity Cache holds the results, 11.5 against 10.0).
#include "launch.hpp"
#include "mx4.hpp"
#include "rows.hpp"

namespace twell {

constexpr int MX4_WAVES = 4, MX4_EACH = 4;

struct Mx4Units {
  int shift;   // log2 of the lanes per row: a power of two that covers whole blocks, at most a wave
  int pieces;  // of a row
};
template <int E>
static Mx4Units mx4_units(int cols) {
  const int64_t lanes = ((int64_t)cols + MX4_BLOCK - 1) / MX4_BLOCK * (MX4_BLOCK / E);
  int shift = E == 8 ? 2 : 3;
  while (shift < 6 && (1 << shift) < lanes) ++shift;
  return {shift, (int)(((int64_t)cols + 64 * E - 1) / (64 * E))};
}

// Rows (or groups of rows) u0 + 4 i of the workgroup's piece for wave w, i < EACH.
struct Mx4Place {
  int64_t t;   // the lane's row
  int e0;      // and first element
};
template <int E>
__device__ __forceinline__ Mx4Place mx4_lane(int shift, int piece, int64_t u, int lane) {
  return {shift == 6 ? u : (u << (6 - shift)) + (lane >> shift), (piece * 64 + (lane & ((1 << shift) - 1))) * E};
}

template <Dt D, Rows R>
__global__ __launch_bounds__(64 * MX4_WAVES) void k_mx4_quantize(Mx4Args a, int shift, int pieces, int64_t units) {
  constexpr int E = 16 / DtT<D>::size, S = DtT<D>::size;
  using T = typename DtT<D>::T;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int piece = blockIdx.x % pieces;
  const int64_t step = (int64_t)(gridDim.x / pieces) * (MX4_WAVES * MX4_EACH);
  for (int64_t u0 = (int64_t)(blockIdx.x / pieces) * (MX4_WAVES * MX4_EACH) + wave; u0 < units; u0 += step) {
    u32x4_t w[MX4_EACH];
#pragma unroll
    for (int i = 0; i < MX4_EACH; ++i) {
      const Mx4Place p = mx4_lane<E>(shift, piece, u0 + MX4_WAVES * i, lane);
      w[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (p.t < a.rows && p.e0 < a.cols) {
        const T *x = static_cast<const T *>(a.x) + p.t * a.ld_x;
        if constexpr (R == Rows::WHOLE) {
          w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(x + p.e0));
        } else if constexpr (R == Rows::ANY) {
          w[i] = *reinterpret_cast<const u32x4_any_t *>(x + min(p.e0, a.cols - E));
        } else {
          w[i] = Row<D, Rows::TINY>(x, 0, 0, a.cols).load(p.e0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MX4_EACH; ++i) {
      const Mx4Place p = mx4_lane<E>(shift, piece, u0 + MX4_WAVES * i, lane);
      if (R == Rows::ANY && __builtin_expect(p.e0 + E > a.cols, 0)) w[i] = drop_bytes<S>(w[i], min(p.e0 + E - a.cols, E) * S);
      float z[E];
      unpack<D>(w[i], z);
      uint32_t byte;
      const uint32_t codes = mx4_codes<E>(z, byte);
      if (p.t < a.rows) mx4_store<E>(a.q + p.t * a.ld_q, a.scale + p.t * a.ld_scale, p.e0, a.cols, codes, byte);
    }
  }
}

// Element times 2^e, exact in fp32, times the row's factor, rounded once.
template <Dt D, Rows R>
__global__ __launch_bounds__(64 * MX4_WAVES) void k_mx4_dequantize(Mx4Args a, int shift, int pieces, int64_t units) {
  constexpr int E = 16 / DtT<D>::size;
  using T = typename DtT<D>::T;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int piece = blockIdx.x % pieces;
  const int64_t step = (int64_t)(gridDim.x / pieces) * (MX4_WAVES * MX4_EACH);
  for (int64_t u0 = (int64_t)(blockIdx.x / pieces) * (MX4_WAVES * MX4_EACH) + wave; u0 < units; u0 += step) {
    uint32_t w[MX4_EACH], byte[MX4_EACH];
    float factor[MX4_EACH];
#pragma unroll
    for (int i = 0; i < MX4_EACH; ++i) {
      const Mx4Place p = mx4_lane<E>(shift, piece, u0 + MX4_WAVES * i, lane);
      w[i] = byte[i] = 0;
      factor[i] = 1.0f;
      if (p.t < a.rows && p.e0 < a.cols) {
        // rows of q are whole 16-byte chunks
        const uint8_t *q = a.q + p.t * a.ld_q + (p.e0 >> 1);
        if constexpr (E == 8)
          w[i] = *reinterpret_cast<const uint32_t *>(q);
        else
          w[i] = *reinterpret_cast<const uint16_t *>(q);
        byte[i] = a.scale[p.t * a.ld_scale + mx4_place(p.e0 / MX4_BLOCK)];
        if (a.factor != nullptr) factor[i] = a.factor[p.t];
      }
    }
#pragma unroll
    for (int i = 0; i < MX4_EACH; ++i) {
      const Mx4Place p = mx4_lane<E>(shift, piece, u0 + MX4_WAVES * i, lane);
      if (p.t >= a.rows || p.e0 >= a.cols) continue;
      const float scale = byte[i] == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(max(byte[i] << 23, 0x400000u));
      f32x2_t v[E / 2];
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1);
      if constexpr (E == 8) {
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3);
      }
      float z[E];
#pragma unroll
      for (int k = 0; k < E; ++k) z[k] = v[k / 2][k % 2] * scale * factor[i];
      const u32x4_t out = pack_chunk<D>(z);
      T *y = static_cast<T *>(a.y) + p.t * a.ld_y + p.e0;
      if (R == Rows::WHOLE) {
        __builtin_nontemporal_store(out, reinterpret_cast<u32x4_t *>(y));
      } else if (p.e0 + E <= a.cols) {
        __builtin_nontemporal_store(out, reinterpret_cast<u32x4_any_t *>(y));
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (p.e0 + k < a.cols) y[k] = from_f32<D>(z[k]);
      }
    }
  }
}

template <Dt D>
static hipError_t launch_mx4(const Mx4Args &a, bool read, hipStream_t s) {
  constexpr int S = DtT<D>::size, E = 16 / S;
  const Mx4Units un = mx4_units<E>(a.cols);
  const int64_t units = ((int64_t)a.rows + (64 >> un.shift) - 1) >> (6 - un.shift);
  const int64_t sets = (units + MX4_WAVES * MX4_EACH - 1) / (MX4_WAVES * MX4_EACH);
  // at most about 2^22 workgroups, which take more rows in turn
  const int64_t grid = std::min(sets, std::max<int64_t>(1, (1 << 22) / un.pieces)) * un.pieces;
  if (grid > (int64_t)UINT32_MAX / (64 * MX4_WAVES)) return hipErrorInvalidValue;
  const dim3 g((unsigned)grid), b(64 * MX4_WAVES);
  const void *p = read ? a.y : a.x;
  const int64_t ld = read ? a.ld_y : a.ld_x;
  const bool whole = a.cols % E == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * S) % 16 == 0;
  if (read) {
    if (whole)
      hipLaunchKernelGGL((k_mx4_dequantize<D, Rows::WHOLE>), g, b, 0, s, a, un.shift, un.pieces, units);
    else
      hipLaunchKernelGGL((k_mx4_dequantize<D, Rows::ANY>), g, b, 0, s, a, un.shift, un.pieces, units);
  } else if (whole) {
    hipLaunchKernelGGL((k_mx4_quantize<D, Rows::WHOLE>), g, b, 0, s, a, un.shift, un.pieces, units);
  } else if (a.cols >= E) {
    hipLaunchKernelGGL((k_mx4_quantize<D, Rows::ANY>), g, b, 0, s, a, un.shift, un.pieces, units);
  } else {
    hipLaunchKernelGGL((k_mx4_quantize<D, Rows::TINY>), g, b, 0, s, a, un.shift, un.pieces, units);
  }
  return hipGetLastError();
}

hipError_t mx4_rows(const Mx4Args &a, bool read, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  return a.dtype == Dt::BF16 ? launch_mx4<Dt::BF16>(a, read, s) : launch_mx4<Dt::F32>(a, read, s);
}

}  // namespace twell
