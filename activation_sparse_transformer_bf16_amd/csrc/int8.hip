// Product of 8-bit integer rows with a scale for each row of both sides:
//
//   y_mn = round((sum_k a_mk b_nk) sa_m sb_n + bias_m)
//
// The sums are 32-bit integers on the matrix cores: exact, and the same in any
// order (K is at most INT8_MAX_K = 65536, so |sum| <= 2^14 * 2^16 stays below
// 2^31).  Both operands are rows along K, so a wave's operand fragments are 16
// contiguous bytes per lane, and any assignment of K to lanes is right as long
// as a and b share it.
//
// K need not fill the last slab: chunks past a row's last readable chunk are
// loaded from that chunk again, and the a side is zeroed past K, so what the b
// rows hold there does not count.  Rows past M and N repeat the last row and
// are not stored.
//
// Two kernels:
//  * k_int8_tile: tiles of BM x BN outputs, operands through a ring of LDS
//    stages (the direct-to-LDS loads and fragment layout of gemm.hpp).
//  * k_int8_rows: at most 64 rows of a (decoding): 16 columns per workgroup,
//    the waves split K, operands straight into registers.
#include "gemm.hpp"
#include "launch.hpp"

namespace twell {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// The scaled value of one sum.
__device__ __forceinline__ float scaled(int acc, float sa, float sb, float bias) {
  return (float)acc * sa * sb + bias;
}

// Zeroes the bytes of a 16-byte chunk from its byte `left` on.
__device__ __forceinline__ u32x4_t keep_bytes(u32x4_t v, int left) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(max(left - 4 * j, 0), 4);
    v[j] &= n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
  }
  return v;
}

// E consecutive results of one row (E * sizeof(T) == 16) from 16 staged bytes.
template <Dt D>
__device__ __forceinline__ void put_results(void *row, int n, int N, u32x4_t v, bool wide) {
  using T = typename DtT<D>::T;
  constexpr int E = 16 / DtT<D>::size;
  T *p = static_cast<T *>(row) + n;
  if (wide && n + E <= N) {
    *reinterpret_cast<u32x4_t *>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (n + i >= N) break;
      if constexpr (D == Dt::BF16)
        p[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
      else
        p[i] = __uint_as_float(v[i]);
    }
  }
}

// ---- tiles ----------------------------------------------------------------------

// Rows of one operand tile: as DmaRows, with chunks past `last` (the byte
// offset of a row's last readable chunk) read from there.
template <int NR, int WAVES>
struct I8Rows {
  static constexpr int PER_WAVE = NR / 16 / WAVES;
  static_assert(PER_WAVE >= 1 && NR % (16 * WAVES) == 0, "whole 1 KB blocks per wave");
  const int8_t *ptr[PER_WAVE];
  uint32_t off[PER_WAVE];  // the lane's byte offset in the slab
  uint32_t lds[PER_WAVE];  // the wave's 1 KB block in the stage

  __device__ __forceinline__ void init(int wave_u, int lane, int region, const int8_t *base, int64_t ld, int r0,
                                       int rows) {
#pragma unroll
    for (int j = 0; j < PER_WAVE; ++j) {
      const int blk = wave_u * PER_WAVE + j;
      const int row = blk * 16 + (lane >> 2);
      off[j] = ((lane & 3) ^ ((row >> 2) & 3)) * 16;
      ptr[j] = base + (int64_t)min(r0 + row, rows - 1) * ld;
      lds[j] = region + blk * 1024;
    }
  }
  __device__ __forceinline__ void issue(int kt, uint32_t last, uint32_t stage) {
#pragma unroll
    for (int j = 0; j < PER_WAVE; ++j) dma16(ptr[j] + min(off[j] + (uint32_t)kt * SLAB, last), stage + lds[j]);
  }
};

// The second operand's rows become the lanes of the result and the first's its
// registers: with b first, a lane holds one row m and runs of 4 columns n.
template <int NWM, int NWN>
__device__ __forceinline__ void mfma_i8(i32x16_t (&acc)[NWM][NWN], const Frag<NWM, NWN> &f) {
#pragma unroll
  for (int i = 0; i < NWM; ++i)
#pragma unroll
    for (int j = 0; j < NWN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, f.b[j]),
                                                       __builtin_bit_cast(i32x4_t, f.a[i]), acc[i][j], 0, 0, 0);
}

template <class Cfg, int BN>
struct I8Tile {
  static constexpr int RING = gemm_dma_ring_bytes<Cfg>(BN);
  static constexpr int VALS = 2 * Cfg::BM + BN;  // sa, bias, sb
  static constexpr int PITCH = 64 * 4 + 16;      // bytes of a staged row of 64 fp32 results
  static constexpr int STAGED = Cfg::WAVES * 32 * PITCH;
  static constexpr int LDS = (RING > STAGED ? RING : STAGED) + VALS * 4;
};

template <Dt D, class Cfg, int BN>
__global__ __launch_bounds__(Cfg::THREADS, Cfg::WAVES_PER_SIMD) void k_int8_tile(Int8Args a, bool wide) {
  using T = typename DtT<D>::T;
  using WT = WaveTile<BN, Cfg>;
  using L = I8Tile<Cfg, BN>;
  constexpr int BM = Cfg::BM, WAVES = Cfg::WAVES, STAGES = Cfg::STAGES;
  constexpr int NWM = WT::NWM, NWN = WT::NWN;
  constexpr int STAGE = (BM + BN) * SLAB;
  constexpr int OPS = I8Rows<BM, WAVES>::PER_WAVE + I8Rows<BN, WAVES>::PER_WAVE;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = WT::row0(wave), col0 = WT::col0(wave);
  int tm, tn;
  tile_coords(blockIdx.x, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const uint32_t base = lds_address(smem);
  float *vals = reinterpret_cast<float *>(smem + L::LDS - L::VALS * 4);
  const uint32_t vbase = base + L::LDS - L::VALS * 4;

  // scales and biases, 64 at a time; issued before the stages, so that the
  // stage waits below cover them (loads complete in order)
#pragma unroll
  for (int g = 0; g < L::VALS / 64; ++g) {
    if (g % WAVES != wave) continue;
    const float *src = g < BM / 64       ? a.a_scale + min(m0 + 64 * g + lane, a.M - 1)
                       : g < 2 * BM / 64 ? (a.bias ? a.bias + min(m0 + 64 * (g - BM / 64) + lane, a.M - 1) : nullptr)
                                         : a.b_scale + min(n0 + 64 * (g - 2 * BM / 64) + lane, a.N - 1);
    if (g < BM / 64 || g >= 2 * BM / 64 || a.bias != nullptr) dma4(src, vbase + 256 * g);
  }
  I8Rows<BM, WAVES> da;
  I8Rows<BN, WAVES> db;
  da.init(wave, lane, 0, a.a, a.ld_a, m0, a.M);
  db.init(wave, lane, BM * SLAB, a.b, a.ld_b, n0, a.N);
  const int nk = (a.K + SLAB - 1) / SLAB;
  const uint32_t last = (uint32_t)(a.K - 1) / 16 * 16;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    if (s < nk) {
      da.issue(s, last, base + s * STAGE);
      db.issue(s, last, base + s * STAGE);
    }
  }
  i32x16_t acc[NWM][NWN];
#pragma unroll
  for (int i = 0; i < NWM; ++i)
#pragma unroll
    for (int j = 0; j < NWN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  wait_stages<OPS>(min(nk - 1, STAGES - 1));
  __syncthreads();
  Frag<NWM, NWN> f0, f1;
  read_frag<BM>(f0, smem, row0, col0, 0, lane);
  auto slab = [&](auto wait_c, auto issue_c, int kt) {
    constexpr int WAIT = decltype(wait_c)::value;
    constexpr bool ISSUE = decltype(issue_c)::value;
    const int slot = kt % STAGES;
    read_frag<BM>(f1, smem + slot * STAGE, row0, col0, 1, lane);
    mfma_i8(acc, f0);
#pragma unroll
    for (int q = 0; q < NWM + NWN; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
    }
    wait_vmcnt<WAIT * OPS>();
    __syncthreads();
    if constexpr (ISSUE) {
      const uint32_t sb = base + slot * STAGE;
      da.issue(kt + STAGES, last, sb);
      db.issue(kt + STAGES, last, sb);
    }
    read_frag<BM>(f0, smem + ((kt + 1) % STAGES) * STAGE, row0, col0, 0, lane);
    mfma_i8(acc, f1);
#pragma unroll
    for (int q = 0; q < NWM + NWN; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using IW = std::integral_constant<int, STAGES - 2>;
  using BT = std::integral_constant<bool, true>;
  using BF = std::integral_constant<bool, false>;
  int kt = 0;
  for (; kt + STAGES < nk; ++kt) slab(IW(), BT(), kt);
  if constexpr (STAGES == 4) {
    if (kt == nk - 4) slab(I2(), BF(), kt++);
  }
  if (kt == nk - 3) slab(I1(), BF(), kt++);
  if (kt == nk - 2) slab(I0(), BF(), kt++);
  // the last slab: the a side counts up to K only
  read_frag<BM>(f1, smem + (kt % STAGES) * STAGE, row0, col0, 1, lane);
  if (a.K % SLAB != 0) {
    const int left = a.K - kt * SLAB - 16 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < NWM; ++i) {
      f0.a[i] = keep_bytes(f0.a[i], left);
      f1.a[i] = keep_bytes(f1.a[i], left - 32);
    }
  }
  mfma_i8(acc, f0);
  mfma_i8(acc, f1);
  __syncthreads();  // the ring is free: every wave has read its last fragments

  // Results: 32 rows x 64 columns at a time through the wave's own LDS rows,
  // so that global stores are whole runs of a row.
  constexpr int S = DtT<D>::size;
  constexpr int PITCH = 64 * S + 16;
  char *mine = smem + wave * 32 * L::PITCH;
  const float *va = vals, *vbias = vals + BM, *vb = vals + 2 * BM;
  const int h = lane >> 5, r = lane & 31;
#pragma unroll
  for (int i = 0; i < NWM; ++i) {
    const float sa = va[row0 + 32 * i + r];
    const float bias = a.bias ? vbias[row0 + 32 * i + r] : 0.0f;
#pragma unroll
    for (int j = 0; j < NWN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t sb = *reinterpret_cast<const f32x4_t *>(vb + col0 + 32 * j + 8 * g + 4 * h);
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = scaled(acc[i][j][4 * g + q], sa, sb[q], bias);
        char *dst = mine + r * PITCH + (32 * j + 8 * g + 4 * h) * S;
        if constexpr (D == Dt::BF16)
          *reinterpret_cast<u32x2_t *>(dst) = u32x2_t{(uint32_t)bf16_rne(v[0]) | ((uint32_t)bf16_rne(v[1]) << 16),
                                                     (uint32_t)bf16_rne(v[2]) | ((uint32_t)bf16_rne(v[3]) << 16)};
        else
          *reinterpret_cast<f32x4_t *>(dst) = f32x4_t{v[0], v[1], v[2], v[3]};
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    constexpr int PER_ROW = 64 * S / 16;  // lanes per row
#pragma unroll
    for (int p = 0; p < 32 * PER_ROW / 64; ++p) {
      const int rr = p * (64 / PER_ROW) + lane / PER_ROW, c = lane % PER_ROW;
      const int m = m0 + row0 + 32 * i + rr, n = n0 + col0 + c * (16 / S);
      const u32x4_t v = *reinterpret_cast<const u32x4_t *>(mine + rr * PITCH + c * 16);
      if (m < a.M && n < a.N) put_results<D>(static_cast<T *>(a.y) + (int64_t)m * a.ld_y, n, a.N, v, wide);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// ---- few rows -------------------------------------------------------------------

// MT blocks of 16 rows of a, NT blocks of 16 columns, WAVES waves that split K
// in runs of 64 * U bytes.
template <Dt D, int MT, int NT, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void k_int8_rows(Int8Args a, bool wide) {
  using T = typename DtT<D>::T;
  __shared__ i32x4_t red[WAVES][MT * NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16 * NT;
  const int r = lane & 15, kl = (lane >> 4) * 16;
  const int8_t *pa[MT], *pb[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) pa[i] = a.a + (int64_t)min(16 * i + r, a.M - 1) * a.ld_a;
#pragma unroll
  for (int j = 0; j < NT; ++j) pb[j] = a.b + (int64_t)min(n0 + 16 * j + r, a.N - 1) * a.ld_b;
  i32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  const int last = (a.K - 1) / 16 * 16;
  for (int k0 = wave * 64 * U; k0 < a.K; k0 += WAVES * 64 * U) {
    u32x4_t fa[U][MT], fb[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(k0 + 64 * u + kl, last);
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[u][j] = *reinterpret_cast<const u32x4_t *>(pb[j] + k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(k0 + 64 * u + kl, last);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[u][i] = *reinterpret_cast<const u32x4_t *>(pa[i] + k);
    }
    if (k0 + 64 * U > a.K) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i) fa[u][i] = keep_bytes(fa[u][i], a.K - (k0 + 64 * u + kl));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, fb[u][j]),
                                                           __builtin_bit_cast(i32x4_t, fa[u][i]), acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // wave w adds the waves' sums of blocks w, w + WAVES, ...: integers, so the
  // order does not matter; a lane holds row lane % 16 and 4 columns
  for (int blk = wave; blk < MT * NT; blk += WAVES) {
    i32x4_t s = red[0][blk][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += red[w][blk][lane];
    const int m = 16 * (blk / NT) + r, n = n0 + 16 * (blk % NT) + 4 * (lane >> 4);
    if (m >= a.M || n >= a.N) continue;
    const float sa = a.a_scale[m], bias = a.bias ? a.bias[m] : 0.0f;
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = scaled(s[q], sa, a.b_scale[min(n + q, a.N - 1)], bias);
    T *p = static_cast<T *>(a.y) + (int64_t)m * a.ld_y + n;
    if (wide && n + 4 <= a.N) {
      if constexpr (D == Dt::BF16)
        *reinterpret_cast<u32x2_t *>(p) = u32x2_t{(uint32_t)bf16_rne(v[0]) | ((uint32_t)bf16_rne(v[1]) << 16),
                                                 (uint32_t)bf16_rne(v[2]) | ((uint32_t)bf16_rne(v[3]) << 16)};
      else
        *reinterpret_cast<f32x4_t *>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < a.N) p[q] = from_f32<D>(v[q]);
    }
  }
}

// ---- launch -----------------------------------------------------------------------

using I8Big = DmaCfg<256, 8, 4>;
using I8Mid = DmaCfg<128, 4, 4>;
using I8Small = DmaCfg<64, 4, 4>;

template <Dt D, class Cfg, int BN>
static hipError_t launch_tile(const Int8Args &a, bool wide, hipStream_t s) {
  auto kern = k_int8_tile<D, Cfg, BN>;
  constexpr int lds = I8Tile<Cfg, BN>::LDS;
  hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  const int64_t tiles = (int64_t)((a.M - 1) / Cfg::BM + 1) * ((a.N - 1) / BN + 1);
  if (tiles > (1 << 22)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(Cfg::THREADS), lds, s, a, wide);
  return hipGetLastError();
}

template <Dt D, int MT, int NT, int WAVES, int U>
static hipError_t launch_few(const Int8Args &a, bool wide, hipStream_t s) {
  hipLaunchKernelGGL((k_int8_rows<D, MT, NT, WAVES, U>), dim3((a.N - 1) / (16 * NT) + 1), dim3(64 * WAVES), 0, s, a,
                     wide);
  return hipGetLastError();
}

template <Dt D>
static hipError_t matmul_dt(const Int8Args &a, hipStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && (a.ld_y * DtT<D>::size) % 16 == 0;
  if (a.M <= 16) return launch_few<D, 1, 1, 8, 4>(a, wide, s);
  if (a.M <= 32) return launch_few<D, 2, 1, 8, 4>(a, wide, s);
  if (a.M <= 64) return launch_few<D, 4, 1, 8, 4>(a, wide, s);
  const int64_t big = (int64_t)((a.M - 1) / 256 + 1) * ((a.N - 1) / 256 + 1);
  const int64_t mid = (int64_t)((a.M - 1) / 128 + 1) * ((a.N - 1) / 128 + 1);
  if (big >= 192) return launch_tile<D, I8Big, 256>(a, wide, s);
  if (mid >= 256) return launch_tile<D, I8Mid, 128>(a, wide, s);
  return launch_tile<D, I8Small, 128>(a, wide, s);
}

hipError_t int8_matmul(const Int8Args &a, hipStream_t s) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  return a.dtype == Dt::BF16 ? matmul_dt<Dt::BF16>(a, s) : matmul_dt<Dt::F32>(a, s);
}

}  // namespace twell
