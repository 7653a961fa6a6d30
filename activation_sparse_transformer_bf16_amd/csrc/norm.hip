// Residual RMS norm, its gradient, and rows of 8-bit integers with scales.
//
//   h = round(x + residual),  r_t = 1 / sqrt(mean_j h_tj^2 + eps)
//   y_tj = round(h_tj r_t w_j)
//   8 bits: z = h w,  m_t = max(max_j |z_tj|, 2^-100),
//           q_tj = rint(z_tj (127 / m_t)),  scale_t = r_t (m_t / 127)
//   gradient: g = dy w,  dx = round(dh + r (g - h r^2 mean(g h))),
//             dw_j = sum_t dy_tj h_tj r_t
//
// The row's factor r cancels between a value and the row's largest one, so q
// is formed from z alone: it holds no sum, and is the same to the bit however
// the row is split over lanes.  Only scale carries r.  m_t is kept above
// 2^-100 so that 127 / m_t stays finite: an all-zero row gives q = 0.  A row
// in which some z is infinite or NaN gives q = 0 and scale = NaN, so that the
// values it stands for are NaN and not silently zero.
//
// A row stays in the registers of its W waves between its loads and its
// stores (NC chunks of 16 bytes per lane, in storage bits), so every input is
// read and every output written once; an output may be the same buffer as an
// input of the same row, since all of a row's loads come before its stores.
// Above 32 KB a row the registers do not hold everything in each variant, and some
// of it goes through scratch; which variants, and their times, is said at each
// kernel.
#include "launch.hpp"

namespace twell {

constexpr float Q_MAX = 127.0f;
constexpr float Q_TINY = 0x1p-100f;
constexpr uint32_t INF_BITS = 0x7F800000u;

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
        const int n = max(e0 - (d - E), 0) * (int)sizeof(T);  // bytes to move by
        u32x4_t v = w;
        if constexpr (sizeof(T) == 2) {
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

// The chunk's bits only from here on: without this the compiler keeps the
// unpacked values of the first pass over a row alive for the second, twice the
// registers, which costs waves or spills.
__device__ __forceinline__ void keep_packed(u32x4_t &w) { asm volatile("" : "+v"(w)); }

// E (8 or 4) 8-bit values of a row from element e0; rows of q are 16-byte
// aligned.  Nothing past d is written.  Adding 1.5 * 2^23 to the product
// rounds it to a whole number (ties to even) whose low byte is the 8-bit
// value; the product is rounded by itself first (no fused multiply-add), as
// the definition says.
template <int E, Rows R>
__device__ __forceinline__ void store_q(int8_t *row, int e0, int d, const float (&z)[E], float inv, bool bad) {
#pragma clang fp contract(off)
  uint32_t w[E / 4];
#pragma unroll
  for (int k = 0; k < E / 4; ++k) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = z[4 * k + i] * inv;
      b[i] = __float_as_uint(p + 12582912.0f);
    }
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);  // bytes b0, b1, 0, 0
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);  // bytes 0, 0, b2, b3
    w[k] = bad ? 0u : (lo | hi);
  }
  if constexpr (R == Rows::WHOLE) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(row, 0, d, 0x00020000);
    if constexpr (E == 8)
      __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{w[0], w[1]}, rsrc, e0, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(w[0], rsrc, e0, 0, 0);
  } else if (e0 + E <= d) {
    if constexpr (E == 8)
      *reinterpret_cast<u32x2_t *>(row + e0) = u32x2_t{w[0], w[1]};
    else
      *reinterpret_cast<uint32_t *>(row + e0) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (e0 + i < d) row[e0 + i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// Sum and maximum over the 64 lanes of a wave with DPP moves; every lane gets
// the result (from lane 63).
__device__ __forceinline__ float wave_total(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_to_lane63(v)), 63));
}
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
#define TWELL_DPP_MAX(CTRL, ROWS) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false))
  TWELL_DPP_MAX(0xB1, 0xF);   // quad_perm 1,0,3,2
  TWELL_DPP_MAX(0x4E, 0xF);   // quad_perm 2,3,0,1
  TWELL_DPP_MAX(0x124, 0xF);  // row_ror 4
  TWELL_DPP_MAX(0x128, 0xF);  // row_ror 8
  TWELL_DPP_MAX(0x142, 0xA);  // row_bcast15 into rows 1, 3
  TWELL_DPP_MAX(0x143, 0xC);  // row_bcast31 into rows 2, 3
#undef TWELL_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Three values of every wave, in LDS.
struct RowSums {
  float a, b;
  uint32_t top;
};

// Sums and maximum over the W waves that hold one row (`wave` is uniform);
// the same order for every lane.  `buf`: a slot per wave, not written again
// before the next barrier.
template <int W>
__device__ __forceinline__ RowSums row_reduce(float a, float b, uint32_t top, RowSums *buf, int wave) {
  RowSums s{wave_total(a), wave_total(b), wave_top(top)};
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) buf[wave] = s;
    __syncthreads();
    const RowSums *row = buf + wave / W * W;
    s = row[0];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      s.a += row[w].a;
      s.b += row[w].b;
      s.top = max(s.top, row[w].top);
    }
  }
  return s;
}

// Waves of a workgroup of the forward and the quantiser.
constexpr int row_waves(int W) { return W > 4 ? W : 4; }

// x, residual, weight -> h, y, q + scale (each output optional).  NORM false:
// the plain quantiser (h = x, no weight, r = 1).  With eight chunks per lane
// the weight is loaded again where it is used instead of being held.
//
// Memory bound: bf16 8192 x 2048 with residual and 8 bits 23.7 us over three sets
// of operands in turn (151 MB, 6.4 TB/s; a plain copy of the card moves 6.1-6.3),
// 28.2 with all of them in memory, the quantiser of 8192 x 8192 32.8 us (201 MB, 6.1
// TB/s); one row 2.1 us, launch and one round trip.
//
// Long rows with residual, all in memory (us): 2000 x 12288 fp32 70, 2000 x 24576
// bf16 73, 1000 x 24576 fp32 73 (393 MB, 5.4 TB/s each), 1000 x 40000 bf16 63 (320 MB,
// 5.1).  Rows of no alignment need registers for their ends, and beyond 64 KB (16
// waves, 8 chunks) 97 to 139 of them are spilled, in the quantiser 20 to 61: 1000 x
// 39999 bf16 212, 1000 x 24575 fp32 185 (quantiser 85 and 38, whole rows 23 and 22).
// Of 32 to 64 KB only bf16 spills (24): 2000 x 24575 138 us, 2000 x 12287 fp32 79.
template <Dt D, int W, int NC, Rows R, bool NORM>
__global__ __launch_bounds__(64 * row_waves(W)) void k_norm_rows(NormArgs a) {
  constexpr int E = 16 / DtT<D>::size;
  constexpr int RB = row_waves(W) / W;
  constexpr bool HOLD = NORM && NC <= 4;
  __shared__ RowSums sums[2][row_waves(W)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int d = a.d;
  const int first = ((wave % W) * 64 + lane) * E;  // the lane's element of chunk 0
  constexpr int STEP = W * 64 * E;
  const Row<D, R> weight(a.weight, 0, 0, d);
  const float count = (float)d * a.unit;
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * RB; t0 < a.rows; t0 += (int64_t)gridDim.x * RB) {
    const int64_t t = t0 + wave / W;
    const bool live = t < a.rows;  // the same for all waves of a row
    u32x4_t hv[NC], wv[HOLD ? NC : 1];
    float ss = 0.0f;
    uint32_t top = 0;
    if (live) {
      const Row<D, R, !NORM && R == Rows::WHOLE> x(a.x, t, a.ld_x, d);
#pragma unroll
      for (int c = 0; c < NC; ++c) hv[c] = x.load(first + c * STEP);
      if constexpr (HOLD) {
#pragma unroll
        for (int c = 0; c < NC; ++c) wv[c] = weight.load(first + c * STEP);
      }
      if (NORM && a.residual != nullptr) {
        const Row<D, R> residual(a.residual, t, a.ld_res, d);
        u32x4_t rv[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) rv[c] = residual.load(first + c * STEP);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float u[E], v[E];
          unpack<D>(x.trim(hv[c], first + c * STEP), u);
          unpack<D>(residual.trim(rv[c], first + c * STEP), v);
#pragma unroll
          for (int i = 0; i < E; ++i) u[i] += v[i];
          hv[c] = pack_chunk<D>(u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) hv[c] = x.trim(hv[c], first + c * STEP);
      }
      if constexpr (HOLD) {
#pragma unroll
        for (int c = 0; c < NC; ++c) wv[c] = weight.trim(wv[c], first + c * STEP);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float u[E], z[E];
        unpack<D>(hv[c], u);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (NORM) ss += u[i] * a.unit * u[i];
          z[i] = u[i];
        }
        if (a.q != nullptr) {
          if constexpr (NORM) {
            float w[E];
            unpack<D>(HOLD ? wv[c] : weight.trim(weight.load(first + c * STEP), first + c * STEP), w);
#pragma unroll
            for (int i = 0; i < E; ++i) z[i] = u[i] * w[i];
          }
#pragma unroll
          for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(z[i]) & 0x7FFFFFFFu);
        }
      }
    }
    const RowSums s = row_reduce<W>(ss, 0.0f, top, sums[turn], wave);
    turn ^= 1;  // the next row's sums go to the other half: no barrier before they are written
    if (!live) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      keep_packed(hv[c]);
      if constexpr (HOLD) keep_packed(wv[c]);
    }
    const float r = NORM ? rsqrtf(s.a / count + a.eps) : 1.0f;
    const bool bad = s.top >= INF_BITS;
    const float m = fmaxf(__uint_as_float(s.top), Q_TINY);
    const float inv = Q_MAX / m;
    const Row<D, R> h(a.h, t, a.ld_h, d), y(a.y, t, a.ld_y, d);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e0 = first + c * STEP;
      float u[E];
      unpack<D>(hv[c], u);
      if constexpr (NORM) {
        float w[E];
        unpack<D>(HOLD ? wv[c] : weight.trim(weight.load(e0), e0), w);
        if (a.h != nullptr) h.store(e0, hv[c]);
        if (a.y != nullptr) {
          float v[E];
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] = u[i] * r * w[i];
          y.store(e0, pack_chunk<D>(v));
        }
#pragma unroll
        for (int i = 0; i < E; ++i) u[i] *= w[i];
      }
      if (a.q != nullptr) store_q<E, R>(a.q + t * a.ld_q, e0, d, u, inv, bad);
    }
    if (a.q != nullptr && lane == 0 && wave % W == 0)
      a.scale[t] = bad ? __uint_as_float(0x7FC00000u) : r * (m / Q_MAX);
  }
}

// Gradient: a workgroup of 16 waves walks groups of RB = 16 / W rows, its
// own, + grid, ...; each wave keeps its columns' dw sums in registers over all
// its rows, the workgroup adds its row groups in order and writes one row of
// partial sums.  The weight is held in registers where it fits (with four chunks
// per lane beside whole rows only, whose ends take no registers: 2000 x 12287 fp32
// 154 us, held 200), and loaded for each row where it does not; with eight chunks
// per lane the registers hold no sums either: the workgroup, which then takes one
// row at a time, adds each row to its partial row in memory (every element by the
// one lane that owns it).
//
// bf16 8192 x 2048 with dh: 26.0 us (134 MB, 5.2 TB/s) and 4 us for the sums, both
// together back to back 27.8; 16384 x 4096 89 us (6.0 TB/s).  Two waves a row and
// two chunks a lane leave room to load the next row ahead (1 us); one wave with
// four chunks spills (40 us), 512 workgroups write twice the partial rows (28 us),
// 192 or 128 leave CUs idle (from memory 32.6 and 34.9 against 28.8 us, both kernels).
//
// Away from that shape, bf16 with dh, both kernels, all in memory (us, and the bytes'
// time at 6.2 TB/s): 64 x 2048 8.3 (0.2) and 300 x 2048 8.9 (0.8): two launches, and
// groups of rows for 8 and 38 of the 256 CUs; 1024 x 4096 13.1 (5.4); 4096 x 5120 39
// (27), 2000 x 8192 31 (21), 1000 x 14336 38 (18), 500 x 16000 31 (10): the 256 partial
// rows, 16 to 33 MB written and read again, beside 64 to 168 MB of rows.
//
// Above 32 KB a row registers are spilled in every variant: 18 to 84 with four
// chunks per lane, 117 to 376 with eight, more for rows of no alignment.  2000 x
// 12288 fp32 93 (63), 12287 154; 2000 x 24576 bf16 114 (63), 24575 261; 1000 x 24576
// fp32 265 (63), 24575 459; 1000 x 40000 bf16 409 (52), 39999 690: there the sums in
// memory are read and written for each row as well.
constexpr int BACK_WAVES = 16;
template <Dt D, int W, int NC, Rows R>
__global__ __launch_bounds__(64 * BACK_WAVES) void k_norm_backward(NormBackwardArgs a) {
  constexpr int E = 16 / DtT<D>::size;
  constexpr int RB = BACK_WAVES / W;
  constexpr bool HOLD = NC <= 4;         // the sums
  constexpr bool HOLD_W = NC * E <= 16 && (NC <= 2 || R == Rows::WHOLE);  // the weight
  static_assert(HOLD || RB == 1, "sums in memory: one row per workgroup at a time");
  __shared__ RowSums sums[2][BACK_WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int d = a.d;
  const int first = ((wave % W) * 64 + lane) * E;
  constexpr int STEP = W * 64 * E;
  float *out = a.partial + (size_t)blockIdx.x * d;
  const Row<D, R> weight(a.weight, 0, 0, d);
  const float count = (float)d * a.unit;
  u32x4_t wv[HOLD_W ? NC : 1];
  float dw[HOLD ? NC : 1][E];
  if constexpr (HOLD_W) {
#pragma unroll
    for (int c = 0; c < NC; ++c) wv[c] = weight.trim(weight.load(first + c * STEP), first + c * STEP);
  }
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < E; ++i) dw[c][i] = 0.0f;
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      for (int i = 0; i < E; ++i)
        if (first + c * STEP + i < d) out[first + c * STEP + i] = 0.0f;
  }
  // A wave's rows are t, t + step, ...: with at most two chunks per lane the
  // next row is loaded before the present one is worked on.
  const int64_t step = (int64_t)gridDim.x * RB;
  constexpr bool AHEAD = NC <= 2;
  u32x4_t hv[NC], gv[NC], sv[NC];
  auto load_row = [&](int64_t t) {
    if (t >= a.rows) return;
    const Row<D, R, true> h(a.h, t, a.ld_h, d), dy(a.dy, t, a.ld_dy, d);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      hv[c] = h.load(first + c * STEP);
      gv[c] = dy.load(first + c * STEP);
    }
    if (AHEAD && a.dh != nullptr) {
      const Row<D, R, true> dh(a.dh, t, a.ld_dh, d);
#pragma unroll
      for (int c = 0; c < NC; ++c) sv[c] = dh.load(first + c * STEP);
    }
  };
#pragma unroll
  for (int c = 0; c < NC; ++c) sv[c] = u32x4_t{0u, 0u, 0u, 0u};
  int turn = 0;
  if (AHEAD) load_row((int64_t)blockIdx.x * RB + wave / W);
  for (int64_t t0 = (int64_t)blockIdx.x * RB; t0 < a.rows; t0 += step) {
    const int64_t t = t0 + wave / W;
    const bool live = t < a.rows;
    if (!AHEAD) load_row(t);
    u32x4_t hc[NC], gc[NC], sc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      hc[c] = weight.trim(hv[c], first + c * STEP);
      gc[c] = weight.trim(gv[c], first + c * STEP);
      sc[c] = weight.trim(sv[c], first + c * STEP);
    }
    if (AHEAD) load_row(t + step);
    float ss = 0.0f, dot = 0.0f;
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float h[E], g[E], w[E];
        unpack<D>(hc[c], h);
        unpack<D>(gc[c], g);
        unpack<D>(HOLD_W ? wv[c] : weight.trim(weight.load(first + c * STEP), first + c * STEP), w);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          ss += h[i] * a.unit * h[i];
          dot += g[i] * w[i] * a.unit * h[i];
        }
      }
    }
    const RowSums s = row_reduce<W>(ss, dot, 0u, sums[turn], wave);
    turn ^= 1;
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        keep_packed(hc[c]);
        keep_packed(gc[c]);
        if constexpr (HOLD_W) keep_packed(wv[c]);
      }
      const float r = rsqrtf(s.a / count + a.eps);
      const float k = r * (r * (s.b / count));  // r^2 alone can leave the range of fp32
      const Row<D, R, true> dh(a.dh, t, a.ld_dh, d), dx(a.dx, t, a.ld_dx, d);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e0 = first + c * STEP;
        float h[E], g[E], w[E], o[E];
        unpack<D>(hc[c], h);
        unpack<D>(gc[c], g);
        unpack<D>(HOLD_W ? wv[c] : weight.trim(weight.load(e0), e0), w);
        if (!AHEAD && a.dh != nullptr) sc[c] = dh.trim(dh.load(e0), e0);
        unpack<D>(sc[c], o);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float p = g[i] * h[i] * r;
          if constexpr (HOLD)
            dw[c][i] += p;
          else if (e0 + i < d)
            out[e0 + i] += p;
          o[i] += r * (g[i] * w[i] - h[i] * k);
        }
        dx.template store<R == Rows::WHOLE>(e0, pack_chunk<D>(o));
        // one chunk after the other: interleaved, their values do not fit the registers
        if constexpr (NC > 2) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if constexpr (HOLD) {
    // the workgroup's partial row: its RB row groups added in order
    if constexpr (RB == 1) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (first + c * STEP + i < d) out[first + c * STEP + i] = dw[c][i];
    } else {
      __shared__ float sum[RB][STEP];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) sum[wave / W][first + i] = dw[c][i];
        __syncthreads();
        for (int e = threadIdx.x; e < STEP; e += 64 * BACK_WAVES) {
          float v = 0.0f;
#pragma unroll
          for (int g = 0; g < RB; ++g) v += sum[g][e];
          if (c * STEP + e < d) out[c * STEP + e] = v;
        }
      }
    }
  }
}

// dw_j = the partial rows added in a fixed order: a workgroup takes 32 columns,
// a whole 128-byte line of each row; a thread adds every 32nd row, 32 threads
// the 32 sums of their columns.  256 rows of 2048: 3.0 us in a graph, of 8192
// 5.2; half lines (16 columns) take 3.2 and 8.0, quarter lines 4.7 and 12.6, 64
// columns 3.3 and 5.3.
constexpr int DW_COLS = 32, DW_ROWS = 32;
static_assert(NORM_BACKWARD_WGS % DW_ROWS == 0, "whole rows per thread");
__global__ __launch_bounds__(DW_COLS * DW_ROWS) void k_norm_dweight(const float *__restrict__ partial, int n, int d,
                                                                    float *__restrict__ dweight) {
  constexpr int PER = NORM_BACKWARD_WGS / DW_ROWS;
  __shared__ float sum[DW_ROWS][DW_COLS + 1];
  const int col = threadIdx.x % DW_COLS, grp = threadIdx.x / DW_COLS;
  const int j = blockIdx.x * DW_COLS + col;
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = i * DW_ROWS + grp;
    v[i] = j < d && row < n ? partial[(size_t)row * d + j] : 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) s += v[i];
  sum[grp][col] = s;
  __syncthreads();
  if (grp != 0 || j >= d) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < DW_ROWS; ++i) s += sum[i][col];
  dweight[j] = s;
}

// ---- launchers ----------------------------------------------------------------

static bool rows16(const void *p, int64_t ld, int s) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld * s) % 16 == 0);
}

template <Dt D, int W, int NC, bool NORM>
static hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
  constexpr int S = DtT<D>::size, RB = row_waves(W) / W;
  const bool whole = (a.d * S) % 16 == 0 && rows16(a.x, a.ld_x, S) && rows16(a.residual, a.ld_res, S) &&
                     rows16(a.weight, 0, S) && rows16(a.h, a.ld_h, S) && rows16(a.y, a.ld_y, S);
  // at most 2^20 workgroups, which take more rows in turn
  const dim3 grid(std::min((a.rows - 1) / RB + 1, 1 << 20)), block(64 * row_waves(W));
  if (whole) {
    hipLaunchKernelGGL((k_norm_rows<D, W, NC, Rows::WHOLE, NORM>), grid, block, 0, s, a);
  } else if (a.d * S >= 16) {
    hipLaunchKernelGGL((k_norm_rows<D, W, NC, Rows::ANY, NORM>), grid, block, 0, s, a);
  } else if constexpr (W * NC == 1) {
    hipLaunchKernelGGL((k_norm_rows<D, W, NC, Rows::TINY, NORM>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

// Chunks of 64 lanes x 16 bytes in a row: a wave each up to 4 of them, then 4
// waves, 16 from 17 chunks on (measured at 4, 8 and 16 chunks, W = 1 ... 16:
// fewer waves with more chunks each hold fewer rows in flight, 24.1 against
// 23.0 us at 8192 x 2048 bf16; more waves pay for the barrier, 27.9 us).  16 waves
// take two chunks each where that is enough (2000 x 8192 fp32 with residual
// 43.9 -> 40.9 us against four).
template <Dt D, bool NORM>
static hipError_t norm_rows_dt(const NormArgs &a, hipStream_t s) {
  const int chunks = norm_chunks(a.d, D);
  if (chunks <= 1) return launch_rows<D, 1, 1, NORM>(a, s);
  if (chunks <= 2) return launch_rows<D, 2, 1, NORM>(a, s);
  if (chunks <= 4) return launch_rows<D, 4, 1, NORM>(a, s);
  if (chunks <= 8) return launch_rows<D, 4, 2, NORM>(a, s);
  if (chunks <= 16) return launch_rows<D, 4, 4, NORM>(a, s);
  if (chunks <= 32) return launch_rows<D, 16, 2, NORM>(a, s);
  if (chunks <= 64) return launch_rows<D, 16, 4, NORM>(a, s);
  if (chunks <= NORM_MAX_CHUNKS) return launch_rows<D, 16, 8, NORM>(a, s);
  return hipErrorInvalidValue;
}

// The factor on the terms of a row's sums (the squares, and g h), so that a sum
// stays below 2^128 where its mean does: the power of two at or below 1 / d, which
// rounds nothing.  But a term below 2^-126 d loses digits to it, and one below
// 2^-149 d is lost, which counts only beside an eps as small as that: there the
// terms stay as they are.
static float norm_unit(int d, float eps) {
  float unit = 1.0f;
  if (eps >= 0x1p-100f)
    while (unit * (float)d > 1.0f) unit *= 0.5f;
  return unit;
}

hipError_t norm_rows(const NormArgs &args, hipStream_t s) {
  if (args.rows <= 0) return hipSuccess;
  NormArgs a = args;
  a.unit = norm_unit(a.d, a.eps);
  if (a.weight != nullptr)
    return a.dtype == Dt::BF16 ? norm_rows_dt<Dt::BF16, true>(a, s) : norm_rows_dt<Dt::F32, true>(a, s);
  return a.dtype == Dt::BF16 ? norm_rows_dt<Dt::BF16, false>(a, s) : norm_rows_dt<Dt::F32, false>(a, s);
}

template <Dt D, int W, int NC>
static hipError_t launch_backward(const NormBackwardArgs &a, hipStream_t s) {
  constexpr int S = DtT<D>::size;
  const bool whole = (a.d * S) % 16 == 0 && rows16(a.dy, a.ld_dy, S) && rows16(a.h, a.ld_h, S) &&
                     rows16(a.weight, 0, S) && rows16(a.dh, a.ld_dh, S) && rows16(a.dx, a.ld_dx, S);
  const dim3 grid(a.n_partial), block(64 * BACK_WAVES);
  if (whole) {
    hipLaunchKernelGGL((k_norm_backward<D, W, NC, Rows::WHOLE>), grid, block, 0, s, a);
  } else if (a.d * S >= 16) {
    hipLaunchKernelGGL((k_norm_backward<D, W, NC, Rows::ANY>), grid, block, 0, s, a);
  } else if constexpr (W * NC == 1) {
    hipLaunchKernelGGL((k_norm_backward<D, W, NC, Rows::TINY>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

template <Dt D>
static hipError_t backward_dt(const NormBackwardArgs &a, hipStream_t s) {
  const int chunks = norm_chunks(a.d, D);
  if (chunks <= 1) return launch_backward<D, 1, 1>(a, s);
  if (chunks <= 2) return launch_backward<D, 1, 2>(a, s);
  if (chunks <= 4) return launch_backward<D, 2, 2>(a, s);
  if (chunks <= 8) return launch_backward<D, 4, 2>(a, s);
  if (chunks <= 16) return launch_backward<D, 8, 2>(a, s);
  if (chunks <= 32) return launch_backward<D, 16, 2>(a, s);
  if (chunks <= 64) return launch_backward<D, 16, 4>(a, s);
  if (chunks <= NORM_MAX_CHUNKS) return launch_backward<D, 16, 8>(a, s);
  return hipErrorInvalidValue;
}

// Workgroups of the row kernel: a row group each, at most NORM_BACKWARD_WGS.
int norm_backward_partials(int rows, int d, Dt dt) {
  const int chunks = norm_chunks(d, dt);
  const int rb = BACK_WAVES / (chunks <= 2 ? 1 : chunks <= 4 ? 2 : chunks <= 8 ? 4 : chunks <= 16 ? 8 : 16);
  return std::max(1, std::min((int)(((int64_t)rows + rb - 1) / rb), NORM_BACKWARD_WGS));
}

hipError_t norm_backward(const NormBackwardArgs &args, hipStream_t s) {
  // one workgroup writes dweight itself (zeros with no rows)
  NormBackwardArgs a = args;
  a.unit = norm_unit(a.d, a.eps);
  if (a.n_partial == 1) a.partial = a.dweight;
  hipError_t e = a.dtype == Dt::BF16 ? backward_dt<Dt::BF16>(a, s) : backward_dt<Dt::F32>(a, s);
  if (e != hipSuccess || a.n_partial == 1) return e;
  hipLaunchKernelGGL(k_norm_dweight, dim3((a.d + DW_COLS - 1) / DW_COLS), dim3(DW_COLS * DW_ROWS), 0, s, a.partial,
                     a.n_partial, a.d, a.dweight);
  return hipGetLastError();
}

}  // namespace twell
