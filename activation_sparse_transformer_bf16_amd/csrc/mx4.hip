// Rows of microscaled 4-bit floats (mx4.hpp): the quantiser and the reader.
#include "launch.hpp"
#include "mx4.hpp"
#include "rows.hpp"

namespace twell {

// Lanes per row: a power of two that covers the row's whole blocks, at most a
// wave; longer rows are cut into pieces of one wave's 16-byte chunks.
struct Mx4Units {
  int shift;   // log2 of the lanes per row
  int pieces;  // of a row
};
template <int E>
static Mx4Units mx4_units(int cols) {
  const int lanes = (cols + MX4_BLOCK - 1) / MX4_BLOCK * (MX4_BLOCK / E);
  int shift = E == 8 ? 2 : 3;
  while (shift < 6 && (1 << shift) < lanes) ++shift;
  return {shift, (int)(((int64_t)cols + 64 * E - 1) / (64 * E))};
}

// A lane takes one 16-byte chunk of x.
template <Dt D, Rows R>
__global__ __launch_bounds__(256) void k_mx4_quantize(Mx4Args a, int shift, int pieces, int64_t waves) {
  constexpr int E = 16 / DtT<D>::size;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < waves; u += (int64_t)gridDim.x * 4) {
    const int64_t t = shift == 6 ? u / pieces : (u << (6 - shift)) + (lane >> shift);
    const int e0 = (shift == 6 ? (int)(u % pieces) * 64 * E : 0) + (lane & ((1 << shift) - 1)) * E;
    float z[E];
#pragma unroll
    for (int i = 0; i < E; ++i) z[i] = 0.0f;
    if (t < a.rows && e0 < a.cols) {
      const typename DtT<D>::T *p = static_cast<const typename DtT<D>::T *>(a.x) + t * a.ld_x + e0;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e0 + i < a.cols) z[i] = to_f32(p[i]);
    }
    uint32_t byte;
    const uint32_t w = mx4_codes<E>(z, byte);
    if (t < a.rows) mx4_store<E>(a.q + t * a.ld_q, a.scale + t * a.ld_scale, e0, a.cols, w, byte);
  }
}

// A lane writes one 16-byte chunk of y: element times 2^e, exact in fp32, times the
// row's factor, rounded once.
template <Dt D>
__global__ __launch_bounds__(256) void k_mx4_dequantize(Mx4Args a, int shift, int pieces, int64_t waves) {
  constexpr int E = 16 / DtT<D>::size;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < waves; u += (int64_t)gridDim.x * 4) {
    const int64_t t = shift == 6 ? u / pieces : (u << (6 - shift)) + (lane >> shift);
    const int e0 = (shift == 6 ? (int)(u % pieces) * 64 * E : 0) + (lane & ((1 << shift) - 1)) * E;
    if (t >= a.rows || e0 >= a.cols) continue;
    const uint8_t *p = a.q + t * a.ld_q + (e0 >> 1);
    const uint32_t byte = a.scale[t * a.ld_scale + mx4_place(e0 / MX4_BLOCK)];
    const float scale = byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(max(byte << 23, 0x400000u));
    const float factor = a.factor != nullptr ? a.factor[t] : 1.0f;
    typename DtT<D>::T *y = static_cast<typename DtT<D>::T *>(a.y) + t * a.ld_y + e0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (e0 + i >= a.cols) break;
      const int code = (p[i / 2] >> (4 * (i % 2))) & 15;
      const int c = code & 7;
      const float level = c < 4 ? 0.5f * c : c < 6 ? c - 2.0f : 2.0f * c - 8.0f;
      y[i] = from_f32<D>((code & 8 ? -level : level) * scale * factor);
    }
  }
}

template <Dt D>
static hipError_t launch_mx4(const Mx4Args &a, bool read, hipStream_t s) {
  const Mx4Units un = mx4_units<16 / DtT<D>::size>(a.cols);
  const int64_t waves = un.shift == 6 ? (int64_t)a.rows * un.pieces : ((int64_t)a.rows + (64 >> un.shift) - 1) >> (6 - un.shift);
  const dim3 grid((unsigned)std::min<int64_t>((waves + 3) / 4, 1 << 20));
  if (read)
    hipLaunchKernelGGL((k_mx4_dequantize<D>), grid, dim3(256), 0, s, a, un.shift, un.pieces, waves);
  else
    hipLaunchKernelGGL((k_mx4_quantize<D, Rows::ANY>), grid, dim3(256), 0, s, a, un.shift, un.pieces, waves);
  return hipGetLastError();
}

hipError_t mx4_rows(const Mx4Args &a, bool read, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  return a.dtype == Dt::BF16 ? launch_mx4<Dt::BF16>(a, read, s) : launch_mx4<Dt::F32>(a, read, s);
}

}  // namespace twell
