// Product of 8-bit integer rows with a scale for each row of both sides:
//
//   y_mn = round((sum_k a_mk b_nk) sa_m sb_n + bias_m)
//
// The sums are 32-bit integers: exact, and the same in any order (K is at most
// INT8_MAX_K = 65536, so |sum| <= 2^14 * 2^16 stays below 2^31).
#include "launch.hpp"

namespace twell {

// The scaled value of one sum.
__device__ __forceinline__ float scaled(int acc, float sa, float sb, float bias) {
  return (float)acc * sa * sb + bias;
}

// 64 x 64 outputs per workgroup of 16 x 16 threads, 4 x 4 each; K in slabs of
// 64 bytes through LDS.  Bytes at and past K are zeroed on the a side.
constexpr int TM = 64, TK = 64;
template <Dt D>
__global__ __launch_bounds__(256) void k_int8_simple(Int8Args a) {
  using T = typename DtT<D>::T;
  __shared__ __attribute__((aligned(16))) uint32_t As[TM][TK / 4 + 4], Bs[TM][TK / 4 + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TM;
  const int row = tid >> 2, ch = tid & 3;  // 64 rows x 4 chunks of 16 bytes
  const int8_t *pa = a.a + (int64_t)min(m0 + row, a.M - 1) * a.ld_a;
  const int8_t *pb = a.b + (int64_t)min(n0 + row, a.N - 1) * a.ld_b;
  const int last = (a.K - 1) / 16 * 16;  // a row's last readable chunk
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += TK) {
    const int k = k0 + ch * 16;
    u32x4_t va = *reinterpret_cast<const u32x4_t *>(pa + min(k, last));
    const u32x4_t vb = *reinterpret_cast<const u32x4_t *>(pb + min(k, last));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int left = min(max(a.K - k - 4 * j, 0), 4);
      va[j] &= left == 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u;
    }
    __syncthreads();
    *reinterpret_cast<u32x4_t *>(&As[row][ch * 4]) = va;
    *reinterpret_cast<u32x4_t *>(&Bs[row][ch * 4]) = vb;
    __syncthreads();
#pragma unroll 4
    for (int kk = 0; kk < TK / 4; ++kk) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_sdot4((int)As[ty + 16 * i][kk], (int)Bs[tx + 16 * j][kk], acc[i][j], false);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty + 16 * i;
    if (m >= a.M) continue;
    const float sa = a.a_scale[m], bias = a.bias ? a.bias[m] : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n < a.N) static_cast<T *>(a.y)[m * a.ld_y + n] = from_f32<D>(scaled(acc[i][j], sa, a.b_scale[n], bias));
    }
  }
}

hipError_t int8_matmul(const Int8Args &a, hipStream_t s) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  const dim3 grid((a.N + TM - 1) / TM, (a.M + TM - 1) / TM);
  if (a.dtype == Dt::BF16)
    hipLaunchKernelGGL(k_int8_simple<Dt::BF16>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_int8_simple<Dt::F32>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace twell
