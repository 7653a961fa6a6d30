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
// K need not fill the last slab: nothing behind a row's last readable chunk
// counts, as the a side is zeroed past K.  Nothing outside the operands is
// read, and results past M and N are not stored.
//
// Three kernels:
//  * k_int8_tile: tiles of BM x BN outputs, operands through a ring of LDS
//    stages (the direct-to-LDS loads of gemm.hpp); where the tiles are too few
//    for the chip, K is cut into ranges whose integer sums go to the workspace,
//  * k_int8_join, which adds them and writes the results.
//  * k_int8_small: products too small to fill the chip with such tiles: 16 to
//    64 rows and columns per workgroup, whose waves split K.
#include "launch.hpp"
#include "narrow.hpp"

namespace twell {

// The scaled value of one sum.
__device__ __forceinline__ float scaled(int acc, float sa, float sb, float bias) {
  return (float)acc * sa * sb + bias;
}

// Four results of one row from column n on.
template <Dt D>
__device__ __forceinline__ void store4(typename DtT<D>::T *row, int n, int N, i32x4_t s, float sa,
                                       const float (&sb)[4], float bias) {
  float v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = scaled(s[q], sa, sb[q], bias);
  typename DtT<D>::T *p = row + n;
  if (n + 4 <= N) {
    if constexpr (D == Dt::BF16)
      *reinterpret_cast<u32x2_any_t *>(p) = u32x2_any_t{(uint32_t)bf16_rne(v[0]) | ((uint32_t)bf16_rne(v[1]) << 16),
                                                       (uint32_t)bf16_rne(v[2]) | ((uint32_t)bf16_rne(v[3]) << 16)};
    else
      *reinterpret_cast<u32x4_any_t *>(p) = u32x4_any_t{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                       __float_as_uint(v[2]), __float_as_uint(v[3])};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < N) p[q] = from_f32<D>(v[q]);
  }
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

// ---- tiles ----------------------------------------------------------------------
//
// The products are v_mfma_i32_16x16x64_i8, not the 32x32x32 form of the same
// rate: per operation it reads and writes half as many accumulators.  On
// random operands the chip lowers its clock to hold its power, and from
// registers alone this form then sustains 3.95 POP/s against 3.37.

// LDS: the ring, then sa, bias and sb of the tile (fp32).
template <class Cfg, int BN>
struct I8Tile {
  static constexpr int RING = gemm_dma_ring_bytes<Cfg>(BN);
  static constexpr int VALS = 2 * Cfg::BM + BN;
  static_assert(Cfg::BM % 64 == 0 && BN % 64 == 0, "copied 64 at a time");
  static constexpr int LDS = RING + VALS * 4;
};

// Tiles of BM x BN outputs through a ring of LDS stages (gemm.hpp): a wave owns
// 64 columns (4 b fragments) and 2 H 16-row blocks of a, taken in two halves
// of H.  Registers hold the b fragments, and both halves of a: while the lower
// half is multiplied the upper one is read, and while the upper half is
// multiplied the next slab's lower half, each b fragment after its last use;
// the copies for the slab STAGES ahead go out between the products.
//
// Measured (256 x 256 tiles, Gaussian operands, back to back over the same
// buffers): 8192 x 8192 x 2048 127-131 us, 2.1 POP/s (132-140 over buffers in turn
// or all in memory; fp32 results, all in memory, 171); 8192^3 413 us, 2.66 POP/s;
// 16384 x 14336 x 4096 762-783 us, 2.5 POP/s (fp32 results 828), against 2.0 POP/s
// of the library's 8-bit product at 8192^3, 3.95 from registers alone and 5 of the
// specification.  Two things bound it.  The power of the chip: operands of zeros
// take 103, 315 and 597 us; by parts, at 8192^3 with random operands and 32 x 32 x 32
// products, registers only 3.4 POP/s, with the fragment reads 3.0, with the copies
// into LDS 2.4; the 16 x 16 x 64 form then gained 10%.  And what each tile spends
// before its first and after its last product, which a short K does not hide: with
// zeros 2.67 POP/s at K = 2048, 3.49 at 8192; the results' stores alone are 20 us of
// 8192 x 8192 x 2048 (110 us without them).  A persistent workgroup that starts the
// next tile's copies before them gains nothing, nor do 128 x 128 wave tiles on four
// waves (accumulators in AGPRs, 583 us at 8192^3).
// STREAM: the results are stored non-temporally (a template, as the compiler
// joins the two kinds of store into the ordinary one under a run-time choice).
template <Dt D, class Cfg, int BN, bool STREAM>
__global__ __launch_bounds__(Cfg::THREADS, Cfg::WAVES_PER_SIMD) void k_int8_tile(Int8Args a, int tiles) {
  using T = typename DtT<D>::T;
  using WT = WaveTile<BN, Cfg>;
  using L = I8Tile<Cfg, BN>;
  constexpr int BM = Cfg::BM, WAVES = Cfg::WAVES, STAGES = Cfg::STAGES;
  constexpr int H = WT::NWM, NB = 4;
  constexpr int STAGE = (BM + BN) * SLAB;
  constexpr int SB = D == Dt::BF16 ? 3 : 2;  // b's swizzle: the rows of a fragment are 8 (4) apart in groups of 4
  using RowsA = I8Rows<BM, WAVES, 2>;
  using RowsB = I8Rows<BN, WAVES, SB>;
  constexpr int OPS = RowsA::PER_WAVE + RowsB::PER_WAVE;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = WT::row0(wave), col0 = WT::col0(wave);
  int tm, tn;
  tile_coords(blockIdx.x % tiles, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  // this workgroup's range of K: from here on the operands begin and end with it
  const int part = blockIdx.x / tiles;
  const int k0 = part * a.k_part;
  a.a += k0;
  a.b += k0;
  a.K = min(a.K - k0, a.k_part);
  const uint32_t base = lds_address(smem);

  // scales and biases, 64 at a time; issued before the stages, so that the
  // stage waits below cover them (loads complete in order)
#pragma unroll
  for (int g = 0; g < L::VALS / 64; ++g) {
    if (g % WAVES != wave) continue;
    const float *src = g < BM / 64       ? a.a_scale + min(m0 + 64 * g + lane, a.M - 1)
                       : g < 2 * BM / 64 ? (a.bias ? a.bias + min(m0 + 64 * (g - BM / 64) + lane, a.M - 1) : nullptr)
                                            : a.b_scale + min(n0 + 64 * (g - 2 * BM / 64) + lane, a.N - 1);
    if (g < BM / 64 || g >= 2 * BM / 64 || a.bias != nullptr)
      copy4(src, __builtin_amdgcn_readfirstlane((int)(base + L::RING + 256 * g)));
  }
  RowsA da;
  RowsB db;
  da.init(wave, lane, 0, a.a, a.ld_a, m0, a.M, a.K);
  db.init(wave, lane, BM * SLAB, a.b, a.ld_b, n0, a.N, a.K);
  const int nk = (a.K + SLAB - 1) / SLAB;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    if (s < nk) {
      da.issue_all(base + s * STAGE);
      db.issue_all(base + s * STAGE);
    }
  }
  i32x4_t acc[2 * H][NB];
#pragma unroll
  for (int i = 0; i < 2 * H; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  const int rho = lane & 15;
  i32x4_t alo[H], ahi[H], b[NB];
  auto read_a = [&](i32x4_t(&f)[H], int slot, int half) {
#pragma unroll
    for (int i = 0; i < H; ++i) f[i] = read_i8<2>(smem + slot * STAGE, row0 + 16 * (half * H + i) + rho, lane);
  };
  auto read_b = [&](int j, int slot) {
    b[j] = read_i8<SB>(smem + slot * STAGE + BM * SLAB, col0 + i8_col<D>(j, rho), lane);
  };
  auto multiply = [&](const i32x4_t(&f)[H], int half, int j) {
#pragma unroll
    for (int i = 0; i < H; ++i)
      acc[half * H + i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j], f[i], acc[half * H + i][j], 0, 0, 0);
  };
  wait_stages<OPS>(min(nk - 1, STAGES - 1));
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NB; ++j) read_b(j, 0);
  read_a(alo, 0, 0);
  auto slab = [&](auto wait_c, auto issue_c, int kt) {
    constexpr int WAIT = decltype(wait_c)::value;
    constexpr bool ISSUE = decltype(issue_c)::value;
    const int slot = kt % STAGES, next = (kt + 1) % STAGES;
    read_a(ahi, slot, 1);
#pragma unroll
    for (int j = 0; j < NB; ++j) multiply(alo, 0, j);
    __builtin_amdgcn_sched_barrier(0);
    // every wave has read all of slab kt (the barrier waits for its LDS
    // reads) and slab kt + 1 has landed for every wave
    wait_vmcnt<WAIT * OPS>();
    __syncthreads();
    read_a(alo, next, 0);
    // the loads of slab kt + STAGES among the products, not in one block
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      multiply(ahi, 1, j);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (ISSUE) {
#pragma unroll
        for (int q = j; q < OPS; q += NB) {
          if (q < RowsA::PER_WAVE)
            da.issue(q, base + slot * STAGE);
          else
            db.issue(q - RowsA::PER_WAVE, base + slot * STAGE);
        }
      }
      read_b(j, next);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (ISSUE) {
      da.advance();
      db.advance();
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
  read_a(ahi, kt % STAGES, 1);
  if (a.K % SLAB != 0) {
    const int left = a.K - kt * SLAB - 16 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      alo[i] = __builtin_bit_cast(i32x4_t, keep_bytes(__builtin_bit_cast(u32x4_t, alo[i]), left));
      ahi[i] = __builtin_bit_cast(i32x4_t, keep_bytes(__builtin_bit_cast(u32x4_t, ahi[i]), left));
    }
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    multiply(alo, 0, j);
    multiply(ahi, 1, j);
  }

  if (a.partial != nullptr) {
    // the range's sums, 4 columns per lane; rows of n_pad (a multiple of 4)
    const int n_pad = (a.N + 3) / 4 * 4;
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) {
      const int m = m0 + row0 + 16 * i + rho;
      if (m >= a.M) continue;
      int *row = a.partial + ((int64_t)part * a.M + m) * n_pad;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int n = n0 + col0 + i8_col<D>(j, 4 * (lane >> 4));
        if (n < a.N) *reinterpret_cast<i32x4_t *>(row + n) = acc[i][j];
      }
    }
    return;
  }
  __syncthreads();  // every wave has read its last fragments: the ring is free

  // Results, 16 rows of 64 columns at a time through the wave's own LDS rows,
  // so that a store covers whole 128-byte lines.
  constexpr int S = DtT<D>::size;
  constexpr int PITCH = 64 * S + 16, PER_ROW = 64 * S / 16;  // bytes of a staged row, lanes that store it
  static_assert(WAVES * 16 * PITCH <= L::RING, "the staged rows fit the ring");
  char *mine = smem + wave * 16 * PITCH;
  const float *va = reinterpret_cast<const float *>(smem + L::RING), *vbias = va + BM, *vb = va + 2 * BM;
  const int h = lane >> 4;
  f32x4_t sb[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) sb[j] = *reinterpret_cast<const f32x4_t *>(vb + col0 + i8_col<D>(j, 4 * h));
#pragma unroll
  for (int i = 0; i < 2 * H; ++i) {
    const int row = row0 + 16 * i;
    const float sa = va[row + rho];
    const float bias = a.bias ? vbias[row + rho] : 0.0f;
    float v[NB][4];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j][q] = scaled(acc[i][j][q], sa, sb[j][q], bias);
#pragma unroll
    for (int j = 0; j < NB; j += D == Dt::BF16 ? 2 : 1) {
      u32x4_t w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (D == Dt::BF16)
          w[k] = (uint32_t)bf16_rne(v[j + k / 2][2 * (k % 2)]) | ((uint32_t)bf16_rne(v[j + k / 2][2 * (k % 2) + 1]) << 16);
        else
          w[k] = __float_as_uint(v[j][k]);
      }
      *reinterpret_cast<u32x4_t *>(mine + rho * PITCH + i8_col<D>(j, 4 * h) * S) = w;
    }
    wave_sync();
#pragma unroll
    for (int p = 0; p < PER_ROW / 4; ++p) {
      const int r = p * (64 / PER_ROW) + lane / PER_ROW, c = lane % PER_ROW;
      const int m = m0 + row + r, n = n0 + col0 + c * (16 / S);
      const u32x4_t w = *reinterpret_cast<const u32x4_t *>(mine + r * PITCH + c * 16);
      if (m < a.M && n < a.N) store_run<D, STREAM>(static_cast<T *>(a.y) + (int64_t)m * a.ld_y, n, a.N, w);
    }
    wave_sync();
  }
}

// The ranges' sums added, scaled and written: 4 columns per thread, a row per
// blockIdx.y; four ranges' loads in flight at a time.
template <Dt D>
__global__ __launch_bounds__(256) void k_int8_join(Int8Args a, int parts) {
  using T = typename DtT<D>::T;
  const int n_pad = (a.N + 3) / 4 * 4;
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= a.N) return;
  float sb[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) sb[q] = a.b_scale[min(n + q, a.N - 1)];
  for (int m = blockIdx.y; m < a.M; m += gridDim.y) {
    const float sa = a.a_scale[m], bias = a.bias ? a.bias[m] : 0.0f;
    const int *src = a.partial + (int64_t)m * n_pad + n;
    i32x4_t s = {0, 0, 0, 0};
    for (int p = 0; p < parts; p += 4) {
      i32x4_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = *reinterpret_cast<const i32x4_t *>(src + (int64_t)min(p + k, parts - 1) * a.M * n_pad);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (p + k < parts) s += v[k];
    }
    store4<D>(static_cast<T *>(a.y) + (int64_t)m * a.ld_y, n, a.N, s, sa, sb, bias);
  }
}

// ---- small products ----------------------------------------------------------------

// Tiles of 16 MF x 16 NF results, too small to share an operand's loads between
// waves: the WAVES waves take slabs of 128 bytes of K in turn, each through a
// ring of its own in LDS (so the loop has no barrier), and add their sums
// through LDS at the end.
//
// Fragments loaded straight into registers cost four times the copies' time:
// lanes next to each other hold different rows, so a load touches a line per
// lane.  The copies take 8 lanes, 128 bytes, to a row, and the transposition
// is the LDS read's.  Chunk c of row r is kept at c ^ (r / 2 % 8) of its 128
// bytes: the 16 lanes of a read group (see i8_swizzle) then meet 16 different
// bank quads.
//
// Bound by what a CU can have loaded, 105 GB/s each, after about 2 us for the
// launch, the first loads and the sums, or by the memory's rate.  Measured (us,
// in the shape chosen, against k_int8_tile with its ranges of K): 1 x 8192 x
// 2048 4.9 (7.8), 1 x 14336 x 14336 36 (66; 205 MB), 16 x 2048 x 8192 5.4 (9.0),
// 64 x 2048 x 2048 3.3 (7.4), 64 x 2048 x 8192 6.9 (11.3), 64 x 8192 x 2048 6.3
// (9.2), 512 x 2048 x 4096 10.7 (14.8).  Fragments straight into registers take
// 5.5, 41, 9.3, 4.8, 13 and 12 us for the first six.  Twice the waves with half the
// ring, or longer rings, change 3% either way.
template <int MF_, int NF_, int WAVES_, int STAGES_>
struct I8Small {
  static constexpr int MF = MF_, NF = NF_, WAVES = WAVES_, STAGES = STAGES_;
  static constexpr int BM = 16 * MF, BN = 16 * NF, THREADS = 64 * WAVES;
  static constexpr int ROW = 128, STAGE = (BM + BN) * ROW, OPS = STAGE / 1024;
  static constexpr int FRAGS = MF * NF, PER = (FRAGS + WAVES - 1) / WAVES;  // fragments of the results, and of one wave
  static constexpr int LDS = WAVES * STAGES * STAGE;
  static_assert(WAVES * FRAGS * 1024 <= LDS && LDS <= 160 * 1024, "the sums take the rings' place");
};
template <Dt D, class C>
__global__ __launch_bounds__(C::THREADS) void k_int8_small(Int8Args a, int tiles) {
  using T = typename DtT<D>::T;
  constexpr int MF = C::MF, NF = C::NF, WAVES = C::WAVES, STAGES = C::STAGES, OPS = C::OPS;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rho = lane & 15, h = lane >> 4;
  // an eighth of the tiles, column of tiles after column, for each XCD
  // (workgroups go to the 8 in turn), whose L2 then keeps their rows of b
  const int tiles_m = (a.M - 1) / C::BM + 1, each = gridDim.x / 8;
  const int tile = blockIdx.x % 8 * each + blockIdx.x / 8;
  const int n0 = tile / tiles_m * C::BN, m0 = tile % tiles_m * C::BM;
  if (tile >= tiles) return;

  // the scales of the results that this wave writes, loaded before the sums
  float sa[C::PER], bias[C::PER], sb[C::PER][4];
#pragma unroll
  for (int p = 0; p < C::PER; ++p) {
    const int f = min(wave + p * WAVES, C::FRAGS - 1);
    const int m = min(m0 + 16 * (f / NF) + rho, a.M - 1), n = n0 + 16 * (f % NF) + 4 * h;
    sa[p] = a.a_scale[m];
    bias[p] = a.bias ? a.bias[m] : 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) sb[p][q] = a.b_scale[min(n + q, a.N - 1)];
  }

  // copy j: rows 8 j .. 8 j + 7 of the stage, a's first, 128 bytes each
  const int8_t *row[OPS];
#pragma unroll
  for (int j = 0; j < OPS; ++j) {
    const int r = 8 * j + (lane >> 3);
    row[j] = 8 * j < C::BM ? a.a + (int64_t)min(m0 + r, a.M - 1) * a.ld_a
                           : a.b + (int64_t)min(n0 + r - C::BM, a.N - 1) * a.ld_b;
  }
  int chunk[2];  // the lane's, by the parity of j
#pragma unroll
  for (int p = 0; p < 2; ++p) chunk[p] = ((lane & 7) ^ (4 * p + (lane >> 4))) * 16;
  const int last = (a.K - 1) / 16 * 16;
  const int slabs = (a.K + C::ROW - 1) / C::ROW;
  const int mine = slabs > wave ? (slabs - wave - 1) / WAVES + 1 : 0;
  char *ring = smem + wave * (STAGES * C::STAGE);
  const uint32_t base = lds_address(ring);
  auto issue = [&](int i) {
    const int k0 = (wave + i * WAVES) * C::ROW;
    const uint32_t stage = base + (uint32_t)(i % STAGES * C::STAGE);
#pragma unroll
    for (int j = 0; j < OPS; ++j)
      copy16(row[j] + min(k0 + chunk[j & 1], last), __builtin_amdgcn_readfirstlane((int)(stage + 1024 * j)));
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i)
    if (i < mine) issue(i);
  i32x4_t acc[MF][NF];
#pragma unroll
  for (int x = 0; x < MF; ++x)
#pragma unroll
    for (int y = 0; y < NF; ++y) acc[x][y] = i32x4_t{0, 0, 0, 0};
  for (int i = 0; i < mine; ++i) {
    wait_stages<OPS>(min(mine - 1 - i, STAGES - 1));
    const char *stage = ring + i % STAGES * C::STAGE + rho * C::ROW;
    u32x4_t fa[2][MF], fb[2][NF];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int at = ((4 * s + h) ^ (rho >> 1)) * 16;
#pragma unroll
      for (int x = 0; x < MF; ++x) fa[s][x] = *reinterpret_cast<const u32x4_t *>(stage + x * 16 * C::ROW + at);
#pragma unroll
      for (int y = 0; y < NF; ++y) fb[s][y] = *reinterpret_cast<const u32x4_t *>(stage + (MF + y) * 16 * C::ROW + at);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage is read, and may be written again
    if (i + STAGES < mine) issue(i + STAGES);
    const int left = a.K - (wave + i * WAVES) * C::ROW;
    if (left < C::ROW) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int x = 0; x < MF; ++x) fa[s][x] = keep_bytes(fa[s][x], left - 16 * (4 * s + h));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int x = 0; x < MF; ++x)
#pragma unroll
        for (int y = 0; y < NF; ++y)
          acc[x][y] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, fb[s][y]),
                                                           __builtin_bit_cast(i32x4_t, fa[s][x]), acc[x][y], 0, 0, 0);
  }
  __syncthreads();  // every wave has read its stages
  i32x4_t *sums = reinterpret_cast<i32x4_t *>(smem);
#pragma unroll
  for (int x = 0; x < MF; ++x)
#pragma unroll
    for (int y = 0; y < NF; ++y) sums[(wave * C::FRAGS + x * NF + y) * 64 + lane] = acc[x][y];
  __syncthreads();
#pragma unroll
  for (int p = 0; p < C::PER; ++p) {
    const int f = wave + p * WAVES;
    const int m = m0 + 16 * (f / NF) + rho, n = n0 + 16 * (f % NF) + 4 * h;
    if (f >= C::FRAGS || m >= a.M || n >= a.N) continue;
    i32x4_t s = sums[f * 64 + lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += sums[(w * C::FRAGS + f) * 64 + lane];
    store4<D>(static_cast<T *>(a.y) + (int64_t)m * a.ld_y, n, a.N, s, sa[p], sb[p], bias[p]);
  }
}

// ---- launch -----------------------------------------------------------------------

// The tile shapes of k_int8_tile: rows, columns, and the time of one 64-byte
// slab of K per tile on a CU, in units of 10 ns (measured over K = 2048 and
// 8192 with the chip full; the smaller ones are bound by the loads a CU can have
// in flight, the largest by the power of the matrix cores).  1024 x 8192 x 2048:
// 28 us in 256 x 256 tiles, 21.6 in 256 x 128; 2048 x 2048 x 8192: 52 us in 256
// x 128, 40 in 128 x 128.
enum I8Shape { I8_256x256, I8_256x128, I8_128x128, I8_64x128, I8_SHAPES };
struct I8ShapeCost {
  int bm, bn, slab;
};
constexpr I8ShapeCost I8_COST[I8_SHAPES] = {{256, 256, 80}, {256, 128, 53}, {128, 128, 30}, {64, 128, 19}};
constexpr int I8_TILE_COST = 250;   // of a tile besides its slabs: start, ring fill, results
constexpr int I8_JOIN_COST = 250;   // of the second launch
constexpr int I8_MAX_PARTS = 16;
constexpr size_t I8_MAX_PARTIAL = (size_t)64 << 20;

// Those of k_int8_small: rows, columns, workgroups that a CU holds, and the
// time besides the loads, once and for each round of workgroups (fitted to 31
// sizes of 1 to 2048 rows: 10% in the mean; over 50 sizes the shape chosen is
// the fastest one, or within 7% of it but for 128 x 4096 x 16384, 14%).
enum I8SmallShape { I8_16x16, I8_16x32, I8_32x32, I8_32x64, I8_64x64, I8_SMALL_SHAPES };
struct I8SmallCost {
  int bm, bn, held, start, round;
};
constexpr I8SmallCost I8_SMALL[I8_SMALL_SHAPES] = {
    {16, 16, 2, 155, 85}, {16, 32, 3, 200, 40}, {32, 32, 2, 140, 115}, {32, 64, 1, 40, 235}, {64, 64, 1, 0, 380}};
constexpr int I8_SMALL_RATE = 1050;  // bytes a CU loads in 10 ns

struct I8Plan {
  bool small;         // `shape` is an I8SmallShape
  int shape;
  int parts, k_part;  // k_int8_tile: the ranges of K
  size_t bytes;       // of the workspace: 0 with one range
};

static int64_t i8_tiles(int bm, int bn, int M, int N) { return (int64_t)((M - 1) / bm + 1) * ((N - 1) / bn + 1); }

// The kernel, shape and number of K ranges with the least estimated time: 256
// CUs take the tiles in rounds; the ranges' sums are written and read once (4
// bytes each way at about 4 TB/s), the operands read at 5 TB/s at most.
static I8Plan i8_plan(int M, int N, int K) {
  const int nk = (K + SLAB - 1) / SLAB;
  I8Plan best{false, I8_256x256, 1, nk * SLAB, 0};
  int64_t least = INT64_MAX;
  const int64_t bytes = ((int64_t)M + N) * K;
  for (int shape = 0; shape < I8_SMALL_SHAPES; ++shape) {
    const I8SmallCost &c = I8_SMALL[shape];
    const int64_t tiles = i8_tiles(c.bm, c.bn, M, N);
    const int64_t per_cu = (tiles + 255) / 256, rounds = (tiles + 256 * c.held - 1) / (256 * c.held);
    const int64_t cost =
        c.start + rounds * c.round + per_cu * ((int64_t)(c.bm + c.bn) * K / I8_SMALL_RATE) + bytes / 140000;
    if (cost < least) {
      least = cost;
      best = I8Plan{true, shape, 1, nk * SLAB, 0};
    }
  }
  for (int shape = 0; shape < I8_SHAPES; ++shape) {
    const int64_t tiles = i8_tiles(I8_COST[shape].bm, I8_COST[shape].bn, M, N);
    for (int want = 1; want <= I8_MAX_PARTS; want *= 2) {
      const int per = (nk + want - 1) / want, parts = (nk + per - 1) / per;
      const size_t sums = (size_t)parts * M * ((N + 3) / 4 * 4);
      if (want > 1 && (parts < want || per < 4 || sums * 4 > I8_MAX_PARTIAL)) break;
      const int64_t rounds = (tiles * parts + 255) / 256;
      const int64_t cost = std::max(rounds * (per * I8_COST[shape].slab + I8_TILE_COST), bytes / 50000 + I8_TILE_COST) +
                           (parts > 1 ? I8_JOIN_COST + (int64_t)(sums / 5000) : 0);
      if (cost < least) {
        least = cost;
        best = I8Plan{false, shape, parts, per * SLAB, parts > 1 ? sums * 4 : 0};
      }
    }
  }
  return best;
}

// Rows too far apart for 32-bit offsets within a tile: k_int8_small, which has
// 64-bit addresses, takes those.
static bool i8_far(const Int8Args &a) {
  return std::max(a.ld_a, a.ld_b) > ((int64_t)1 << 31) / 256 - INT8_MAX_K;
}

size_t int8_matmul_workspace(int M, int N, int K) {
  return M <= 0 || N <= 0 ? 0 : i8_plan(M, N, K).bytes;
}

template <Dt D, class Cfg, int BN, bool STREAM = false>
static hipError_t launch_tile(const Int8Args &a, int parts, hipStream_t s) {
  auto kern = k_int8_tile<D, Cfg, BN, STREAM>;
  constexpr int lds = I8Tile<Cfg, BN>::LDS;
  hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  const int64_t tiles = i8_tiles(Cfg::BM, BN, a.M, a.N);
  if (tiles * parts > (int64_t)UINT32_MAX / Cfg::THREADS) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * parts)), dim3(Cfg::THREADS), lds, s, a, (int)tiles);
  return hipGetLastError();
}

template <Dt D, int MF, int NF, int WAVES, int STAGES>
static hipError_t launch_small(const Int8Args &a, hipStream_t s) {
  using C = I8Small<MF, NF, WAVES, STAGES>;
  auto kern = k_int8_small<D, C>;
  if constexpr (C::LDS > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
  }
  const int64_t tiles = i8_tiles(C::BM, C::BN, a.M, a.N), wgs = (tiles + 7) / 8 * 8;
  if (wgs > (int64_t)UINT32_MAX / C::THREADS) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(C::THREADS), C::LDS, s, a, (int)tiles);
  return hipGetLastError();
}

// Results beyond the Infinity Cache (256 MB) are stored non-temporally, so that
// they do not take cache lines from the operands of the tiles still to come
// (470 MB, 16384 x 14336 x 4096: 762 against 792 us); smaller ones, where it
// makes no difference (134 to 235 MB, within 1%), stay there for their reader.
template <Dt D>
static bool i8_stream(const Int8Args &a) {
  return (size_t)a.M * a.N * DtT<D>::size > ((size_t)256 << 20);
}

template <Dt D>
static hipError_t matmul_dt(const Int8Args &args, void *workspace, hipStream_t s) {
  Int8Args a = args;
  I8Plan p = i8_plan(a.M, a.N, a.K);
  if (i8_far(a) && !p.small) p = I8Plan{true, I8_64x64, 1, 0, 0};
  if (p.small) {
    switch (p.shape) {
      case I8_16x16: return launch_small<D, 1, 1, 8, 2>(a, s);
      case I8_16x32: return launch_small<D, 1, 2, 4, 2>(a, s);
      case I8_32x32: return launch_small<D, 2, 2, 4, 2>(a, s);
      case I8_32x64: return launch_small<D, 2, 4, 8, 1>(a, s);
      case I8_64x64: return launch_small<D, 4, 4, 8, 1>(a, s);
    }
    return hipErrorInvalidValue;
  }
  a.k_part = p.k_part;
  a.partial = p.parts > 1 ? static_cast<int *>(workspace) : nullptr;
  hipError_t e = hipErrorInvalidValue;
  switch (p.shape) {
    case I8_256x256:
      e = i8_stream<D>(a) ? launch_tile<D, DmaCfg<256, 8, 4>, 256, true>(a, p.parts, s)
                          : launch_tile<D, DmaCfg<256, 8, 4>, 256>(a, p.parts, s);
      break;
    case I8_256x128: e = launch_tile<D, DmaCfg<256, 8, 4>, 128>(a, p.parts, s); break;
    case I8_128x128: e = launch_tile<D, DmaCfg<128, 4, 4>, 128>(a, p.parts, s); break;
    case I8_64x128: e = launch_tile<D, DmaCfg<64, 4, 4>, 128>(a, p.parts, s); break;
  }
  if (e != hipSuccess || p.parts == 1) return e;
  const dim3 grid((unsigned)((a.N - 1) / 1024 + 1), (unsigned)std::min(a.M, 1 << 15));
  hipLaunchKernelGGL(k_int8_join<D>, grid, dim3(256), 0, s, a, p.parts);
  return hipGetLastError();
}

hipError_t int8_matmul(const Int8Args &a, void *workspace, hipStream_t s) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  return a.dtype == Dt::BF16 ? matmul_dt<Dt::BF16>(a, workspace, s) : matmul_dt<Dt::F32>(a, workspace, s);
}

}  // namespace twell
