// Product of microscaled 4-bit rows (mx4.hpp) on the matrix cores:
//
//   y_mn = round((sum_k a_mk b_nk) fa_m fb_n + bias_m)
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows of 128 elements of both
// sides and applies the scales: lane 16 h + r holds elements 32 h ... 32 h + 31 of
// row r (16 bytes) and that block's scale byte.
#include "launch.hpp"
#include "mx4.hpp"

namespace twell {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// acc += a b^T over 128 elements; S: the byte of the two scale dwords.
template <int S>
__device__ __forceinline__ f32x4_t mx4_mfma(u32x4_t a, u32x4_t b, f32x4_t acc, uint32_t sa, uint32_t sb) {
  const i32x8_t x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, S, (int)sa, S, (int)sb);
}

// Keeps the first `left` elements of a 32-element chunk.
__device__ __forceinline__ u32x4_t mx4_keep(u32x4_t v, int left) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(max(left - 8 * j, 0), 8);
    v[j] &= n == 8 ? 0xFFFFFFFFu : (1u << (4 * n)) - 1u;
  }
  return v;
}

// One wave per 16 x 16 results.
template <Dt D>
__global__ __launch_bounds__(64) void k_mx4_simple(Mx4MatmulArgs a) {
  const int lane = threadIdx.x, rho = lane & 15, h = lane >> 4;
  const int tiles_n = (a.N + 15) / 16;
  const int m0 = blockIdx.x / tiles_n * 16, n0 = blockIdx.x % tiles_n * 16;
  const int m = min(m0 + rho, a.M - 1), n = min(n0 + rho, a.N - 1);
  const uint8_t *pa = a.a + (int64_t)m * a.ld_a, *pb = a.b + (int64_t)n * a.ld_b;
  const uint8_t *sa = a.a_scale + (int64_t)m * a.ld_sa, *sb = a.b_scale + (int64_t)n * a.ld_sb;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  for (int k = 0; k < a.K; k += 128) {
    const int e = k + 32 * h;
    u32x4_t x = zero, y = zero;
    uint32_t s = 0, t = 0;
    if (e < a.K) {
      x = mx4_keep(*reinterpret_cast<const u32x4_t *>(pa + e / 2), a.K - e);
      y = *reinterpret_cast<const u32x4_t *>(pb + e / 2);
      s = sa[mx4_place(e / 32)];
      t = sb[mx4_place(e / 32)];
    }
    acc = mx4_mfma<0>(y, x, acc, t, s);
  }
  using T = typename DtT<D>::T;
  const int row = m0 + rho;
  if (row >= a.M) return;
  const float fa = a.a_factor ? a.a_factor[row] : 1.0f, bias = a.bias ? a.bias[row] : 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int col = n0 + 4 * h + q;
    if (col < a.N)
      static_cast<T *>(a.y)[(int64_t)row * a.ld_y + col] =
          from_f32<D>(acc[q] * fa * (a.b_factor ? a.b_factor[col] : 1.0f) + bias);
  }
}

size_t mx4_matmul_workspace(int M, int N, int K) { return 0; }

hipError_t mx4_matmul(const Mx4MatmulArgs &a, void *workspace, hipStream_t s) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  const int64_t tiles = (int64_t)((a.M - 1) / 16 + 1) * ((a.N - 1) / 16 + 1);
  if (tiles > (int64_t)UINT32_MAX / 64) return hipErrorInvalidValue;
  if (a.dtype == Dt::BF16)
    hipLaunchKernelGGL(k_mx4_simple<Dt::BF16>, dim3((unsigned)tiles), dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL(k_mx4_simple<Dt::F32>, dim3((unsigned)tiles), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace twell
