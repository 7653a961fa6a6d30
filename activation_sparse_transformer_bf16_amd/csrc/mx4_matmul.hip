// Product of microscaled 4-bit rows (mx4.hpp) on the matrix cores:
//
//   y_mn = round((sum_k a_mk b_nk) fa_m fb_n + bias_m)
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows of 128 elements of both
// sides and applies the blocks' scales: lane 16 h + r holds elements 32 h ... 32 h + 31
// of row r (16 bytes) and, in one byte of a dword, that block's scale.  The byte is
// chosen by the instruction, so a dword serves four steps of 128 elements: a group
// of 512, whose 16 scale bytes lie in a row as mx4_place says.
//
// K need not fill the last group: codes of a past K are zeroed and scales past the
// last block set to 2^-127 on both sides (what lies there may be NaN).  Nothing
// outside the operands is read, and results past M and N are not stored.
//
// Three kernels, as for 8-bit rows (int8.hip), whose tiles have the same bytes:
//  * k_mx4_tile: tiles of BM x BN outputs, operands through a ring of LDS stages;
//    where the tiles are too few for the chip, K is cut into ranges whose sums go
//    to the workspace,
//  * k_mx4_join, which adds them in order and writes the results.
//  * k_mx4_small: products too small to fill the chip with such tiles: 16 to 64
//    rows and columns per workgroup, whose waves split K.
//
// The instruction at full rate, from registers alone, does 7.0 PFLOP/s on random
// codes and 9.7 on zeros (32 x 32 x 64: 6.3 and 9.65): the chip's power bounds it.
#include "launch.hpp"
#include "mx4.hpp"
#include "narrow.hpp"

namespace twell {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// acc += b a^T over 128 elements; S: the byte of the scale dwords.
template <int S>
__device__ __forceinline__ f32x4_t mx4_mfma(u32x4_t b, u32x4_t a, f32x4_t acc, uint32_t sb, uint32_t sa) {
  const i32x8_t x = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8_t y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, S, (int)sb, S, (int)sa);
}

// The first `left` elements of a 32-element chunk, zeros for the others.
__device__ __forceinline__ u32x4_t mx4_keep(u32x4_t v, int left) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(max(left - 8 * j, 0), 8);
    v[j] &= n == 8 ? 0xFFFFFFFFu : (1u << (4 * n)) - 1u;
  }
  return v;
}

// Which bytes of a lane's scale dword are blocks of the row: byte s is block 4 s + h
// of a group with `left` elements.
__device__ __forceinline__ uint32_t mx4_scale_mask(int left, int h) {
  const int n = min(max((left - MX4_BLOCK * h + 127) / 128, 0), 4);
  return n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
}

__device__ __forceinline__ float mx4_result(float acc, float fa, float fb, float bias) { return acc * fa * fb + bias; }

// Four results of one row from column n on.
template <Dt D>
__device__ __forceinline__ void mx4_store4(typename DtT<D>::T *row, int n, int N, f32x4_t s, float fa,
                                           const float (&fb)[4], float bias) {
  float v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = mx4_result(s[q], fa, fb[q], bias);
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

// ---- tiles ----------------------------------------------------------------------

// LDS: the ring and four groups' scales (64 bytes per row): all of it for the largest
// tile.  fa, bias and fb of the tile (fp32) come last, to the end of the ring's first half.
template <class Cfg, int BN>
struct Mx4Tile {
  static constexpr int RING = gemm_dma_ring_bytes<Cfg>(BN);
  static constexpr int ROWS = Cfg::BM + BN;
  static constexpr bool RANGES = BN < 256;  // of K: the largest tile takes all of it (mx4_plan)
  static constexpr int SCALES = ROWS * 64;
  static constexpr int VALS = 2 * Cfg::BM + BN;
  static_assert(Cfg::BM % 64 == 0 && BN % 64 == 0, "copied 64 at a time");
  static_assert(Cfg::STAGES == 4, "two pairs of slabs");
  static constexpr int VALS_AT = RING / 2 - VALS * 4;
  static constexpr int LDS = RING + SCALES;
};

// Tiles as k_int8_tile's (int8.hip): a wave owns 64 columns (4 b fragments) and 2 H
// 16-row blocks of a, taken in two halves; fragments and scales are read from LDS
// half a slab ahead.  A slab is 64 bytes of each row, 128 elements.  The loop goes by
// groups of four slabs, one for each byte of the scale dwords; the scales of four groups
// are copied at a time, once the last of those before are in registers everywhere.
//
// Slabs are copied in pairs because a line is 128 bytes: copied one by one, every line
// is fetched twice (8192^3: 41 million L2 requests, in pairs 25).
//
// 8192 x 8192 x 2048 bf16 96 to 100 us (2.8 PFLOP/s), 8192^3 275 to 287 (3.9), 16384 x
// 14336 x 4096 468 to 485 (4.0), by card; MFMA busy 0.31 to 0.43.  What bounds the loop
// is the copies: of the 233 us that another K = 8192 of 8192 x 8192 takes, 73 go without
// them, 8 without the LDS reads, and the products alone take 140.  Two pairs of slabs fill
// the LDS, so a pair has the time of one other to arrive, and a miss in L2 takes longer;
// but with all tiles reading the same rows 8192 x 8192 x 2048 takes 92 us, 8192^3 260, so
// misses are at most 17 of the 73, and the rest (issue and waits, LDS writes beside reads,
// a barrier per pair) is not told apart.  At K = 2048 the loop is 58 of 98 us, the
// tiles' starts and results 40.  Power is a fifth (operands of zeros: 78, 233 and 444
// us).  Slower or no faster: one workgroup per CU that starts the next tile's copies
// before its results' stores (K = 2048 115 us, K = 512 66 against 54: copies behind
// stores wait for them), two workgroups of 128 x 256 per CU (K = 2048 107, 8192^3
// 335), results straight from registers (100, 495 at 16384 x 14336 x 4096), raised
// wave priority, panels of 1, 4 and 8 tiles of rows where a panel has 1024 rows now (K
// = 2048 91 to 98, but 16384 x 14336 x 4096 476 to 522), non-temporal stores of 134 MB
// (83 us, but the kernel that reads the result next takes 41 more).
template <Dt D, class Cfg, int BN, bool STREAM>
__global__ __launch_bounds__(Cfg::THREADS, Cfg::WAVES_PER_SIMD) void k_mx4_tile(Mx4MatmulArgs a, int tiles) {
  using T = typename DtT<D>::T;
  using WT = WaveTile<BN, Cfg>;
  using L = Mx4Tile<Cfg, BN>;
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
  tile_coords<1024 / BM>(blockIdx.x % tiles, (a.M + BM - 1) / BM, (a.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  // this workgroup's range of K (whole groups): from here on the operands begin and end with it
  const int part = blockIdx.x / tiles;
  const int k0 = part * a.k_part;
  a.a += k0 / 2;
  a.b += k0 / 2;
  a.a_scale += k0 / 32;
  a.b_scale += k0 / 32;
  a.K = min(a.K - k0, a.k_part);
  const int groups = (a.K + MX4_GROUP - 1) / MX4_GROUP;
  const uint32_t base = lds_address(smem);

  // 16 rows of scales at a time, 64 bytes of each for four groups (of fewer, the last
  // one's again, as nothing behind a row is read); group g of row r is kept at (g ^ r / 4) % 4
  // of its 64 bytes (b: r / 2^SB), so that the 16 rows of a fragment lie in all banks
  constexpr int SCALE_COPIES = L::ROWS / 16;
  auto copy_scales = [&](int g) {
    int l = lane;
    asm volatile("" : "+v"(l));  // (else the rows' addresses stay in registers)
    for (int c = wave; c < SCALE_COPIES; c += WAVES) {
      const int r = 16 * c + (l >> 2);
      const uint8_t *p;
      int f = r >> 2;
      if (16 * c < BM) {
        p = a.a_scale + (int64_t)min(m0 + r, a.M - 1) * a.ld_sa;
      } else {
        p = a.b_scale + (int64_t)min(n0 + r - BM, a.N - 1) * a.ld_sb;
        f = r >> SB;
      }
      copy16(p + min(g + ((l ^ f) & 3), groups - 1) * 16, __builtin_amdgcn_readfirstlane((int)(base + L::RING + 1024 * c)));
    }
  };
  static_assert(BM / 64 <= WAVES && BN / 64 <= WAVES, "64 factors for a wave");
  auto copy_vals = [&]() {
    auto copy = [&](const float *src, int first, int end, int count, int at) {
      if (src != nullptr && wave < count / 64)
        copy4(src + min(first + 64 * wave + lane, end - 1),
              __builtin_amdgcn_readfirstlane((int)(base + L::VALS_AT + 4 * at + 256 * wave)));
    };
    copy(a.a_factor, m0, a.M, BM, 0);
    copy(a.bias, m0, a.M, BM, BM);
    copy(a.b_factor, n0, a.N, BN, 2 * BM);
  };
  // scales are issued before the stages, so that the stage waits below cover them (loads
  // complete in order)
  copy_scales(0);
  RowsA da;
  RowsB db;
  const int bytes = (a.K + 1) / 2;
  da.init(wave, lane, 0, reinterpret_cast<const int8_t *>(a.a), a.ld_a, m0, a.M, bytes);
  db.init(wave, lane, BM * SLAB, reinterpret_cast<const int8_t *>(a.b), a.ld_b, n0, a.N, bytes);
  auto issue_pair = [&](int q, int p) {  // copies q of both slabs of a pair into the ring's half p
    if (q < RowsA::PER_WAVE)
      da.issue_pair(q, base + 2 * p * STAGE, base + (2 * p + 1) * STAGE);
    else
      db.issue_pair(q - RowsA::PER_WAVE, base + 2 * p * STAGE, base + (2 * p + 1) * STAGE);
  };
  auto next_pair = [&]() {
    da.advance();
    da.advance();
    db.advance();
    db.advance();
  };
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int q = 0; q < OPS; ++q) issue_pair(q, p);
    next_pair();
  }
  f32x4_t acc[2 * H][NB];
#pragma unroll
  for (int i = 0; i < 2 * H; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int rho = lane & 15, h = lane >> 4;
  u32x4_t alo[H], ahi[H], b[NB];
  uint32_t salo[H], sahi[H], sb[NB];
  // Where the lane reads: fragments of a and their scales lie 16 rows apart, those of b
  // as i8_col says, and the swizzle of a lane's rows is the same for all of them, so one
  // offset each for the ring's two halves does, and constants for the rest.
  const int col = i8_col<D>(0, rho);
  uint32_t at_a[2], at_b[2];
  const uint32_t at_sa = L::RING + (row0 + rho) * 64 + ((rho >> 2) << 4) + 4 * h;
  const uint32_t at_sb = L::RING + (BM + col0 + col) * 64 + ((rho >> 2) << 4) + 4 * h;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    at_a[p] = 2 * p * STAGE + (row0 + rho) * SLAB + ((h ^ i8_swizzle<2>(rho)) << 4);
    at_b[p] = 2 * p * STAGE + BM * SLAB + (col0 + col) * SLAB + ((h ^ i8_swizzle<SB>(col)) << 4);
    asm volatile("" : "+v"(at_a[p]), "+v"(at_b[p]));  // (else an address per read, and spills)
  }
  constexpr auto b_row = [](int j) { return i8_col<D>(j, 0); };
  auto read_a = [&](u32x4_t(&f)[H], int s, int half) {
#pragma unroll
    for (int i = 0; i < H; ++i)
      f[i] = *reinterpret_cast<const u32x4_t *>(smem + at_a[s / 2] + s % 2 * STAGE + 16 * (half * H + i) * SLAB);
  };
  auto read_b = [&](int j, int s) {
    b[j] = *reinterpret_cast<const u32x4_t *>(smem + at_b[s / 2] + s % 2 * STAGE + b_row(j) * SLAB);
  };
  auto read_sa = [&](uint32_t(&f)[H], int half, int g) {
    const char *p = smem + (at_sa ^ (g & 3) << 4);
#pragma unroll
    for (int i = 0; i < H; ++i) f[i] = *reinterpret_cast<const uint32_t *>(p + 16 * (half * H + i) * 64);
  };
  auto read_sb = [&](int j, int g) { sb[j] = *reinterpret_cast<const uint32_t *>(smem + (at_sb ^ (g & 3) << 4) + b_row(j) * 64); };
  auto multiply = [&](auto step, const u32x4_t(&f)[H], const uint32_t(&sf)[H], int half, int j) {
#pragma unroll
    for (int i = 0; i < H; ++i)
      acc[half * H + i][j] = mx4_mfma<decltype(step)::value>(b[j], f[i], acc[half * H + i][j], sb[j], sf[i]);
  };
  wait_vmcnt<2 * OPS>();  // the second pair
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    read_b(j, 0);
    read_sb(j, 0);
  }
  read_a(alo, 0, 0);
  read_sa(salo, 0, 0);
  const int left = a.K - (groups - 1) * MX4_GROUP;  // elements of the last group
  // Slab S of a group.  LAST: of the last group, whose codes of a count up to K only.
  auto slab = [&](auto step, auto last_c, int g) {
    constexpr int S = decltype(step)::value;
    constexpr bool LAST = decltype(last_c)::value, ODD = S % 2 == 1;
    constexpr bool ISSUE = !LAST && ODD, NEXT = !LAST || S < 3;
    constexpr int next = (S + 1) % 4;
    read_a(ahi, S, 1);
    if constexpr (S == 0) {
      read_sa(sahi, 1, g);
      if constexpr (LAST) {
        const uint32_t mask = mx4_scale_mask(left, h);
#pragma unroll
        for (int i = 0; i < H; ++i) sahi[i] &= mask;
      }
    }
    if (LAST && left < (S + 1) * 128) {
      const int n = left - S * 128 - 32 * h;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        alo[i] = mx4_keep(alo[i], n);
        ahi[i] = mx4_keep(ahi[i], n);
      }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) multiply(step, alo, salo, 0, j);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (NEXT && ODD) {
      // every wave has read all of this pair (the barrier waits for its LDS reads) and
      // the next pair has landed for every wave, and the scales before it
      wait_vmcnt<0>();
      __syncthreads();
      if (!LAST && S == 1 && g % 4 == 3) copy_scales(g + 1);
      if (LAST && S == 1) copy_vals();  // this half of the ring is done with
    }
    if constexpr (NEXT) {
      read_a(alo, next, 0);
      if constexpr (S == 3) read_sa(salo, 0, g + 1);
    }
    // the copies of the pair that takes this one's place among the products, not in one block
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      multiply(step, ahi, sahi, 1, j);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (ISSUE) {
#pragma unroll
        for (int q = j; q < OPS; q += NB) issue_pair(q, S / 2);
      }
      if constexpr (NEXT) {
        read_b(j, next);
        if constexpr (S == 3) read_sb(j, g + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (ISSUE) next_pair();
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  using BT = std::integral_constant<bool, true>;
  using BF = std::integral_constant<bool, false>;
  for (int g = 0; g < groups - 1; ++g) {
    slab(I0(), BF(), g);
    slab(I1(), BF(), g);
    slab(I2(), BF(), g);
    slab(I3(), BF(), g);
  }
  // the last group: scales count up to K only
  const uint32_t mask = mx4_scale_mask(left, h);
#pragma unroll
  for (int i = 0; i < H; ++i) salo[i] &= mask;
#pragma unroll
  for (int j = 0; j < NB; ++j) sb[j] &= mask;
  slab(I0(), BT(), groups - 1);
  if (left > 128) slab(I1(), BT(), groups - 1);
  if (left > 256) slab(I2(), BT(), groups - 1);
  if (left > 384) slab(I3(), BT(), groups - 1);
  wait_vmcnt<0>();  // copies of slabs past K, into LDS that the results (or the next workgroup) take
  if (L::RANGES && a.partial != nullptr) {
    // the range's sums, 4 columns per lane; rows of n_pad (a multiple of 4)
    const int n_pad = (a.N + 3) / 4 * 4;
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) {
      const int m = m0 + row0 + 16 * i + rho;
      if (m >= a.M) continue;
      float *row = a.partial + ((int64_t)part * a.M + m) * n_pad;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int n = n0 + col0 + i8_col<D>(j, 4 * h);
        if (n < a.N) *reinterpret_cast<f32x4_t *>(row + n) = acc[i][j];
      }
    }
    return;
  }
  __syncthreads();  // every wave has read its last fragments: the ring is free
  if (left <= 128) {
    copy_vals();
    wait_vmcnt<0>();
    __syncthreads();
  }

  // Results, 16 rows of 64 columns at a time through the wave's own LDS rows,
  // so that a store covers whole 128-byte lines.
  constexpr int S = DtT<D>::size;
  constexpr int PITCH = 64 * S + 16, PER_ROW = 64 * S / 16;  // bytes of a staged row, lanes that store it
  static_assert(WAVES * 16 * PITCH <= L::VALS_AT, "the staged rows fit the ring, before the factors");
  char *mine = smem + wave * 16 * PITCH;
  const float *va = reinterpret_cast<const float *>(smem + L::VALS_AT), *vbias = va + BM, *vb = va + 2 * BM;
  f32x4_t fb[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
    fb[j] = a.b_factor ? *reinterpret_cast<const f32x4_t *>(vb + col0 + i8_col<D>(j, 4 * h)) : f32x4_t{1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
  for (int i = 0; i < 2 * H; ++i) {
    const int row = row0 + 16 * i;
    const float fa = a.a_factor ? va[row + rho] : 1.0f;
    const float bias = a.bias ? vbias[row + rho] : 0.0f;
    float v[NB][4];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j][q] = mx4_result(acc[i][j][q], fa, fb[j][q], bias);
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

// The ranges' sums added in order, scaled and written: 4 columns per thread, a row
// per blockIdx.y; four ranges' loads in flight at a time.  A second launch costs 2.3 us
// and the sums' bytes each way; 16 x 16 x 65536 in 16 ranges takes 11.5 us in all.
template <Dt D>
__global__ __launch_bounds__(256) void k_mx4_join(Mx4MatmulArgs a, int parts) {
  using T = typename DtT<D>::T;
  const int n_pad = (a.N + 3) / 4 * 4;
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= a.N) return;
  float fb[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) fb[q] = a.b_factor ? a.b_factor[min(n + q, a.N - 1)] : 1.0f;
  for (int m = blockIdx.y; m < a.M; m += gridDim.y) {
    const float fa = a.a_factor ? a.a_factor[m] : 1.0f, bias = a.bias ? a.bias[m] : 0.0f;
    const float *src = a.partial + (int64_t)m * n_pad + n;
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < parts; p += 4) {
      f32x4_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = *reinterpret_cast<const f32x4_t *>(src + (int64_t)min(p + k, parts - 1) * a.M * n_pad);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (p + k < parts) s += v[k];
    }
    mx4_store4<D>(static_cast<T *>(a.y) + (int64_t)m * a.ld_y, n, a.N, s, fa, fb, bias);
  }
}

// ---- small products ----------------------------------------------------------------

// Tiles of 16 MF x 16 NF results as k_int8_small's: the WAVES waves take slabs of 128
// bytes of K (256 elements, two steps) in turn, each through a ring of its own in LDS,
// and add their sums through LDS at the end.  A slab's copies are 8 rows of 128 bytes
// each, chunk c of row r kept at c ^ (r / 2 % 8), then a dword of scales for each lane
// of each fragment, of which the slab uses two bytes.
//
// Bound by latency: 1 x 8192 x 2048 3.7 us (8.9 MB, 2.4 TB/s; an empty launch 2.0), 16
// and 64 x 8192 x 2048 3.9 and 6.0, 64 x 2048 x 8192 7.4, 333 x 1000 x 777 4.5.  As tiles
// of 64 x 128 with 8 ranges of K 64 x 2048 x 8192 takes 11.1 us, 1 x 2048 x 8192 6.8
// (here 4.5).  K is not cut across workgroups: 16 x 300 x 60000, in 19 of them, 27 us.
template <int MF_, int NF_, int WAVES_, int STAGES_>
struct Mx4Small {
  static constexpr int MF = MF_, NF = NF_, WAVES = WAVES_, STAGES = STAGES_;
  static constexpr int BM = 16 * MF, BN = 16 * NF, THREADS = 64 * WAVES;
  static constexpr int ROW = 128, CODES = (BM + BN) * ROW, STAGE = CODES + (MF + NF) * 256;
  static constexpr int COPIES = CODES / 1024, OPS = COPIES + MF + NF;
  static constexpr int FRAGS = MF * NF, PER = (FRAGS + WAVES - 1) / WAVES;  // fragments of the results, and of one wave
  static constexpr int LDS = WAVES * STAGES * STAGE;
  static_assert(WAVES * FRAGS * 1024 <= LDS && LDS <= 160 * 1024, "the sums take the rings' place");
};
template <Dt D, class C>
__global__ __launch_bounds__(C::THREADS) void k_mx4_small(Mx4MatmulArgs a, int tiles) {
  using T = typename DtT<D>::T;
  constexpr int MF = C::MF, NF = C::NF, WAVES = C::WAVES, STAGES = C::STAGES, COPIES = C::COPIES;
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

  // the factors of the results that this wave writes, loaded before the sums
  float fa[C::PER], bias[C::PER], fb[C::PER][4];
#pragma unroll
  for (int p = 0; p < C::PER; ++p) {
    const int f = min(wave + p * WAVES, C::FRAGS - 1);
    const int m = min(m0 + 16 * (f / NF) + rho, a.M - 1), n = n0 + 16 * (f % NF) + 4 * h;
    fa[p] = a.a_factor ? a.a_factor[m] : 1.0f;
    bias[p] = a.bias ? a.bias[m] : 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) fb[p][q] = a.b_factor ? a.b_factor[min(n + q, a.N - 1)] : 1.0f;
  }

  // copy j: rows 8 j .. 8 j + 7 of the stage, a's first, 128 bytes each
  const uint8_t *row[COPIES], *scales[MF + NF];
#pragma unroll
  for (int j = 0; j < COPIES; ++j) {
    const int r = 8 * j + (lane >> 3);
    row[j] = 8 * j < C::BM ? a.a + (int64_t)min(m0 + r, a.M - 1) * a.ld_a
                           : a.b + (int64_t)min(n0 + r - C::BM, a.N - 1) * a.ld_b;
  }
#pragma unroll
  for (int f = 0; f < MF + NF; ++f)
    scales[f] = 4 * h + (f < MF ? a.a_scale + (int64_t)min(m0 + 16 * f + rho, a.M - 1) * a.ld_sa
                                : a.b_scale + (int64_t)min(n0 + 16 * (f - MF) + rho, a.N - 1) * a.ld_sb);
  int chunk[2];  // the lane's, by the parity of j
#pragma unroll
  for (int p = 0; p < 2; ++p) chunk[p] = ((lane & 7) ^ (4 * p + (lane >> 4))) * 16;
  const int bytes = (a.K + 1) / 2, last = (bytes - 1) / 16 * 16;
  const int slabs = (bytes + C::ROW - 1) / C::ROW;
  const int mine = slabs > wave ? (slabs - wave - 1) / WAVES + 1 : 0;
  char *ring = smem + wave * (STAGES * C::STAGE);
  const uint32_t base = lds_address(ring);
  auto issue = [&](int i) {
    const int slab = wave + i * WAVES;
    const uint32_t stage = base + (uint32_t)(i % STAGES * C::STAGE);
#pragma unroll
    for (int j = 0; j < COPIES; ++j)
      copy16(row[j] + min(slab * C::ROW + chunk[j & 1], last), __builtin_amdgcn_readfirstlane((int)(stage + 1024 * j)));
#pragma unroll
    for (int f = 0; f < MF + NF; ++f)
      copy4(scales[f] + slab / 2 * 16, __builtin_amdgcn_readfirstlane((int)(stage + C::CODES + 256 * f)));
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i)
    if (i < mine) issue(i);
  f32x4_t acc[MF][NF];
#pragma unroll
  for (int x = 0; x < MF; ++x)
#pragma unroll
    for (int y = 0; y < NF; ++y) acc[x][y] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < mine; ++i) {
    wait_stages<C::OPS>(min(mine - 1 - i, STAGES - 1));
    const char *stage = ring + i % STAGES * C::STAGE;
    u32x4_t xa[2][MF], xb[2][NF];
    uint32_t sa[MF], sb[NF];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int at = rho * C::ROW + ((4 * s + h) ^ (rho >> 1)) * 16;
#pragma unroll
      for (int x = 0; x < MF; ++x) xa[s][x] = *reinterpret_cast<const u32x4_t *>(stage + x * 16 * C::ROW + at);
#pragma unroll
      for (int y = 0; y < NF; ++y) xb[s][y] = *reinterpret_cast<const u32x4_t *>(stage + (MF + y) * 16 * C::ROW + at);
    }
    const int slab = wave + i * WAVES;
    const int down = slab % 2 * 16;  // an odd slab's two bytes are the upper ones
#pragma unroll
    for (int x = 0; x < MF; ++x) sa[x] = *reinterpret_cast<const uint32_t *>(stage + C::CODES + 256 * x + 4 * lane) >> down;
#pragma unroll
    for (int y = 0; y < NF; ++y) sb[y] = *reinterpret_cast<const uint32_t *>(stage + C::CODES + 256 * (MF + y) + 4 * lane) >> down;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage is read, and may be written again
    if (i + STAGES < mine) issue(i + STAGES);
    const int left = a.K - slab * 2 * C::ROW;
    if (left < 2 * C::ROW) {
      const uint32_t mask = mx4_scale_mask(left, h);
#pragma unroll
      for (int x = 0; x < MF; ++x) {
        sa[x] &= mask;
        xa[0][x] = mx4_keep(xa[0][x], left - 32 * h);
        xa[1][x] = mx4_keep(xa[1][x], left - 128 - 32 * h);
      }
#pragma unroll
      for (int y = 0; y < NF; ++y) sb[y] &= mask;
    }
#pragma unroll
    for (int x = 0; x < MF; ++x)
#pragma unroll
      for (int y = 0; y < NF; ++y) acc[x][y] = mx4_mfma<0>(xb[0][y], xa[0][x], acc[x][y], sb[y], sa[x]);
#pragma unroll
    for (int x = 0; x < MF; ++x)
#pragma unroll
      for (int y = 0; y < NF; ++y) acc[x][y] = mx4_mfma<1>(xb[1][y], xa[1][x], acc[x][y], sb[y], sa[x]);
  }
  __syncthreads();  // every wave has read its stages
  f32x4_t *sums = reinterpret_cast<f32x4_t *>(smem);
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
    f32x4_t s = sums[f * 64 + lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += sums[(w * C::FRAGS + f) * 64 + lane];
    mx4_store4<D>(static_cast<T *>(a.y) + (int64_t)m * a.ld_y, n, a.N, s, fa[p], fb[p], bias[p]);
  }
}

// ---- launch -----------------------------------------------------------------------

// The tile shapes of k_mx4_tile: rows, columns, workgroups that a CU holds, the time
// of one slab (128 elements of K) per tile, and of a tile besides its slabs (start, ring
// fill, results), in units of 10 ns.  Fitted, with those of k_mx4_small, to 159 sizes of
// 1 to 8192 rows, each timed in every shape that could pay and with 1 to 8 ranges: the
// shape chosen takes 0.8% longer than the fastest in the mean, 15% at most (328 x 9749 x
// 2689); by the 8-bit product's figures 2% in the mean and 42% at most.
enum Mx4Shape { MX4_256x256, MX4_256x128, MX4_128x128, MX4_64x128, MX4_SHAPES };
struct Mx4ShapeCost {
  int bm, bn, held, slab, tile;
};
constexpr Mx4ShapeCost MX4_COST[MX4_SHAPES] = {
    {256, 256, 1, 96, 436}, {256, 128, 1, 46, 366}, {128, 128, 2, 27, 182}, {64, 128, 2, 23, 186}};
constexpr int MX4_JOIN_COST = 228;   // of the second launch
constexpr int MX4_MAX_PARTS = 16;
constexpr size_t MX4_MAX_PARTIAL = (size_t)64 << 20;

// Those of k_mx4_small: rows, columns, workgroups that a CU holds, and the time
// besides the loads, once and for each round of workgroups.
enum Mx4SmallShape { MX4_16x16, MX4_16x32, MX4_32x32, MX4_32x64, MX4_64x64, MX4_SMALL_SHAPES };
struct Mx4SmallCost {
  int bm, bn, held, start, round;
};
constexpr Mx4SmallCost MX4_SMALL[MX4_SMALL_SHAPES] = {
    {16, 16, 2, 34, 185}, {16, 32, 2, 107, 113}, {32, 32, 2, 49, 222}, {32, 64, 1, 182, 164}, {64, 64, 1, 99, 224}};
constexpr int MX4_SMALL_RATE = 437;  // bytes a CU loads in 10 ns

struct Mx4Plan {
  bool small;         // `shape` is an Mx4SmallShape
  int shape;
  int parts, k_part;  // k_mx4_tile: the ranges of K
  size_t bytes;       // of the workspace: 0 with one range
};

static int64_t mx4_tiles(int bm, int bn, int M, int N) { return (int64_t)((M - 1) / bm + 1) * ((N - 1) / bn + 1); }

// The kernel, shape and number of K ranges with the least estimated time: 256
// CUs take the tiles in rounds; the ranges' sums are written and read once (4
// bytes each way at about 4 TB/s), the operands read at 5 TB/s at most.  Numbers of
// ranges are powers of two up to the first that K's groups do not fill (118 groups:
// 15 ranges and not 16), which leaves some out whose estimates are 10 to 40% lower.
static Mx4Plan mx4_plan(int M, int N, int K) {
  const int ng = (K + MX4_GROUP - 1) / MX4_GROUP, row = (K + 1) / 2;
  Mx4Plan best{false, MX4_256x256, 1, ng * MX4_GROUP, 0};
  int64_t least = INT64_MAX;
  const int64_t bytes = ((int64_t)M + N) * row;
  for (int shape = 0; shape < MX4_SMALL_SHAPES; ++shape) {
    const Mx4SmallCost &c = MX4_SMALL[shape];
    const int64_t tiles = mx4_tiles(c.bm, c.bn, M, N);
    const int64_t per_cu = (tiles + 255) / 256, rounds = (tiles + 256 * c.held - 1) / (256 * c.held);
    const int64_t cost =
        c.start + rounds * c.round + per_cu * ((int64_t)(c.bm + c.bn) * row / MX4_SMALL_RATE);
    if (cost < least) {
      least = cost;
      best = Mx4Plan{true, shape, 1, ng * MX4_GROUP, 0};
    }
  }
  for (int shape = 0; shape < MX4_SHAPES; ++shape) {
    const Mx4ShapeCost &c = MX4_COST[shape];
    const int64_t tiles = mx4_tiles(c.bm, c.bn, M, N);
    for (int want = 1; want <= MX4_MAX_PARTS; want *= 2) {
      const int per = (ng + want - 1) / want, parts = (ng + per - 1) / per;
      const size_t sums = (size_t)parts * M * ((N + 3) / 4 * 4);
      // (P ranges of 256 x 256 tiles: as many workgroups as P / 2 of 256 x 128, of which two
      // slabs take 92, one of theirs 96)
      if (want > 1 && (shape == MX4_256x256 || parts < want || sums * 4 > MX4_MAX_PARTIAL)) break;
      const int64_t rounds = (tiles * parts + 256 * c.held - 1) / (256 * c.held);
      const int slabs = std::min((K + 127) / 128, 4 * per);
      const int64_t cost = std::max(rounds * (slabs * c.held * c.slab + c.tile), bytes / 50000 + c.tile) +
                           (parts > 1 ? MX4_JOIN_COST + (int64_t)(sums / 5000) : 0);
      if (cost < least) {
        least = cost;
        best = Mx4Plan{false, shape, parts, per * MX4_GROUP, parts > 1 ? (sums * 4 + 255) / 256 * 256 : 0};
      }
    }
  }
  return best;
}

// Rows too far apart for 32-bit offsets within a tile: k_mx4_small, which has
// 64-bit addresses, takes those.
static bool mx4_far(const Mx4MatmulArgs &a) {
  return std::max(a.ld_a, a.ld_b) > ((int64_t)1 << 31) / 256 - MX4_MAX_K / 2;
}

size_t mx4_matmul_workspace(int M, int N, int K) { return M <= 0 || N <= 0 ? 0 : mx4_plan(M, N, K).bytes; }

template <Dt D, class Cfg, int BN, bool STREAM = false>
static hipError_t launch_tile(const Mx4MatmulArgs &a, int parts, hipStream_t s) {
  auto kern = k_mx4_tile<D, Cfg, BN, STREAM>;
  constexpr int lds = Mx4Tile<Cfg, BN>::LDS;
  hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  const int64_t tiles = mx4_tiles(Cfg::BM, BN, a.M, a.N);
  if (tiles * parts > (int64_t)UINT32_MAX / Cfg::THREADS) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * parts)), dim3(Cfg::THREADS), lds, s, a, (int)tiles);
  return hipGetLastError();
}

template <Dt D, int MF, int NF, int WAVES, int STAGES>
static hipError_t launch_small(const Mx4MatmulArgs &a, hipStream_t s) {
  using C = Mx4Small<MF, NF, WAVES, STAGES>;
  auto kern = k_mx4_small<D, C>;
  if constexpr (C::LDS > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
  }
  const int64_t tiles = mx4_tiles(C::BM, C::BN, a.M, a.N), wgs = (tiles + 7) / 8 * 8;
  if (wgs > (int64_t)UINT32_MAX / C::THREADS) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(C::THREADS), C::LDS, s, a, (int)tiles);
  return hipGetLastError();
}

// Results beyond the Infinity Cache (256 MB) are stored non-temporally, as those of
// the 8-bit product.
template <Dt D>
static bool mx4_stream(const Mx4MatmulArgs &a) {
  return (size_t)a.M * a.N * DtT<D>::size > ((size_t)256 << 20);
}

template <Dt D>
static hipError_t matmul_dt(const Mx4MatmulArgs &args, void *workspace, hipStream_t s) {
  Mx4MatmulArgs a = args;
  Mx4Plan p = mx4_plan(a.M, a.N, a.K);
  if (mx4_far(a) && !p.small) p = Mx4Plan{true, MX4_64x64, 1, 0, 0};
  if (p.small) {
    switch (p.shape) {
      case MX4_16x16: return launch_small<D, 1, 1, 8, 2>(a, s);
      case MX4_16x32: return launch_small<D, 1, 2, 4, 2>(a, s);
      case MX4_32x32: return launch_small<D, 2, 2, 4, 2>(a, s);
      case MX4_32x64: return launch_small<D, 2, 4, 8, 1>(a, s);
      case MX4_64x64: return launch_small<D, 4, 4, 8, 1>(a, s);
    }
    return hipErrorInvalidValue;
  }
  a.k_part = p.k_part;
  a.partial = p.parts > 1 ? static_cast<float *>(workspace) : nullptr;
  hipError_t e = hipErrorInvalidValue;
  switch (p.shape) {
    case MX4_256x256:
      e = mx4_stream<D>(a) ? launch_tile<D, DmaCfg<256, 8, 4>, 256, true>(a, p.parts, s)
                           : launch_tile<D, DmaCfg<256, 8, 4>, 256>(a, p.parts, s);
      break;
    case MX4_256x128: e = launch_tile<D, DmaCfg<256, 8, 4>, 128>(a, p.parts, s); break;
    case MX4_128x128: e = launch_tile<D, DmaCfg<128, 4, 4>, 128>(a, p.parts, s); break;
    case MX4_64x128: e = launch_tile<D, DmaCfg<64, 4, 4>, 128>(a, p.parts, s); break;
  }
  if (e != hipSuccess || p.parts == 1) return e;
  const dim3 grid((unsigned)((a.N - 1) / 1024 + 1), (unsigned)std::min(a.M, 1 << 15));
  hipLaunchKernelGGL(k_mx4_join<D>, grid, dim3(256), 0, s, a, p.parts);
  return hipGetLastError();
}

hipError_t mx4_matmul(const Mx4MatmulArgs &a, void *workspace, hipStream_t s) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  return a.dtype == Dt::BF16 ? matmul_dt<Dt::BF16>(a, workspace, s) : matmul_dt<Dt::F32>(a, workspace, s);
}

}  // namespace twell
