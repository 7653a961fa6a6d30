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
// stores (NC chunks of 16 bytes per lane), so every input is read and every
// output written once; an output may be the same buffer as an input of the
// same row, since all of a row's loads come before its stores.
#include "launch.hpp"

namespace twell {

constexpr float Q_MAX = 127.0f;
constexpr float Q_TINY = 0x1p-100f;
constexpr uint32_t INF_BITS = 0x7F800000u;

// One 16-byte chunk of a row as fp32: elements e0 .. e0 + E - 1, 0 past d.
// AL: rows are 16-byte aligned, so a whole chunk is one load.
template <Dt D, bool AL>
__device__ __forceinline__ void load_chunk(const void *row, int e0, int d, float (&v)[16 / DtT<D>::size]) {
  using T = typename DtT<D>::T;
  constexpr int E = 16 / DtT<D>::size;
  const T *p = static_cast<const T *>(row) + e0;
  if (AL && e0 + E <= d) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t *>(p);
    if constexpr (D == Dt::BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = e0 + i < d ? to_f32(p[i]) : 0.0f;
  }
}

// Rounds v to the storage type, in place, and stores the chunk.
template <Dt D, bool AL>
__device__ __forceinline__ void store_chunk(void *row, int e0, int d, const float (&v)[16 / DtT<D>::size]) {
  using T = typename DtT<D>::T;
  constexpr int E = 16 / DtT<D>::size;
  T *p = static_cast<T *>(row) + e0;
  if (AL && e0 + E <= d) {
    u32x4_t w;
    if constexpr (D == Dt::BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)bf16_rne(v[2 * i]) | ((uint32_t)bf16_rne(v[2 * i + 1]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    }
    *reinterpret_cast<u32x4_t *>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (e0 + i < d) p[i] = from_f32<D>(v[i]);
  }
}

// E (8 or 4) 8-bit values of a row from element e0; rows of q are 16-byte
// aligned.  Nothing past d is written.
template <int E>
__device__ __forceinline__ void store_q(int8_t *row, int e0, int d, const float (&z)[E], float inv, bool bad) {
  uint32_t w[E / 4];
#pragma unroll
  for (int k = 0; k < E / 4; ++k) {
    w[k] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = bad ? 0 : (int)rintf(z[4 * k + i] * inv);
      w[k] |= (uint32_t)(v & 255) << (8 * i);
    }
  }
  if (e0 + E <= d) {
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

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m, 64));
  return v;
}

// Sum (a, b) and maximum (of bits) over the W waves that hold one row; every
// lane gets the result, in the same order whatever the lane.
template <int W>
__device__ __forceinline__ void row_reduce(float &a, float &b, uint32_t &top, float (*lds)[3], int wave) {
  a = wave_sum(a);
  b = wave_sum(b);
  top = wave_max_bits(top);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) {
      lds[wave][0] = a;
      lds[wave][1] = b;
      lds[wave][2] = __uint_as_float(top);
    }
    __syncthreads();
    const int w0 = wave / W * W;
    a = b = 0.0f;
    top = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a += lds[w0 + w][0];
      b += lds[w0 + w][1];
      top = max(top, __float_as_uint(lds[w0 + w][2]));
    }
  }
}

// Waves of a workgroup and rows it takes at a time.
constexpr int row_waves(int W) { return W > 4 ? W : 4; }

// x, residual, weight -> h, y, q + scale (each output optional).  NORM false:
// the plain quantiser (h = x, no weight, r = 1).
template <Dt D, int W, int NC, bool AL, bool NORM>
__global__ __launch_bounds__(64 * row_waves(W)) void k_norm_rows(NormArgs a) {
  constexpr int E = 16 / DtT<D>::size;
  constexpr int S = DtT<D>::size;
  constexpr int RB = row_waves(W) / W;
  __shared__ float lds[2][row_waves(W)][3];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int d = a.d;
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * RB; t0 < a.rows; t0 += (int64_t)gridDim.x * RB) {
    const int64_t t = t0 + wave / W;
    const bool live = t < a.rows;  // the same for all waves of a row
    const char *xr = static_cast<const char *>(a.x) + t * a.ld_x * S;
    const char *rr = NORM && a.residual ? static_cast<const char *>(a.residual) + t * a.ld_res * S : nullptr;
    float v[NC][E], z[NC][E];
    float ss = 0.0f, none = 0.0f;
    uint32_t top = 0;
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c) load_chunk<D, AL>(xr, ((c * W + wave % W) * 64 + lane) * E, d, v[c]);
      if (rr != nullptr) {
#pragma unroll
        for (int c = 0; c < NC; ++c) load_chunk<D, AL>(rr, ((c * W + wave % W) * 64 + lane) * E, d, z[c]);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < E; ++i) v[c][i] = to_f32(from_f32<D>(v[c][i] + z[c][i]));
      }
      if constexpr (NORM) {
#pragma unroll
        for (int c = 0; c < NC; ++c) load_chunk<D, AL>(a.weight, ((c * W + wave % W) * 64 + lane) * E, d, z[c]);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          ss += v[c][i] * v[c][i];
          if (a.q != nullptr) {
            const float p = NORM ? v[c][i] * z[c][i] : v[c][i];
            top = max(top, __float_as_uint(p) & 0x7FFFFFFFu);
          }
        }
    }
    row_reduce<W>(ss, none, top, lds[turn], wave);
    turn ^= 1;  // the next row's sums go to the other half: no barrier before they are written
    if (!live) continue;
    const float r = NORM ? rsqrtf(ss / (float)d + a.eps) : 1.0f;
    const bool bad = top >= INF_BITS;
    const float m = fmaxf(__uint_as_float(top), Q_TINY);
    const float inv = Q_MAX / m;
    char *hr = a.h ? static_cast<char *>(a.h) + t * a.ld_h * S : nullptr;
    char *yr = a.y ? static_cast<char *>(a.y) + t * a.ld_y * S : nullptr;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e0 = ((c * W + wave % W) * 64 + lane) * E;
      if (NORM && hr != nullptr) store_chunk<D, AL>(hr, e0, d, v[c]);
      if (NORM && yr != nullptr) {
        float y[E];
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = v[c][i] * r * z[c][i];
        store_chunk<D, AL>(yr, e0, d, y);
      }
      if (a.q != nullptr) {
        float p[E];
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = NORM ? v[c][i] * z[c][i] : v[c][i];
        store_q<E>(a.q + t * a.ld_q, e0, d, p, inv, bad);
      }
    }
    if (a.q != nullptr && lane == 0 && wave % W == 0)
      a.scale[t] = bad ? __uint_as_float(0x7FC00000u) : r * (m / Q_MAX);
  }
}

// Gradient: a workgroup walks rows t = its own, + grid, ...; each wave keeps
// its columns' dw sums in registers over all its rows, the workgroup adds its
// row groups in order and writes one row of partial sums.
template <Dt D, int W, int NC, bool AL>
__global__ __launch_bounds__(64 * row_waves(W)) void k_norm_backward(NormBackwardArgs a) {
  constexpr int E = 16 / DtT<D>::size;
  constexpr int S = DtT<D>::size;
  constexpr int RW = row_waves(W), RB = RW / W;
  __shared__ float lds[2][RW][3];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int d = a.d;
  float w[NC][E], dw[NC][E];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    load_chunk<D, AL>(a.weight, ((c * W + wave % W) * 64 + lane) * E, d, w[c]);
#pragma unroll
    for (int i = 0; i < E; ++i) dw[c][i] = 0.0f;
  }
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * RB; t0 < a.rows; t0 += (int64_t)gridDim.x * RB) {
    const int64_t t = t0 + wave / W;
    const bool live = t < a.rows;
    float h[NC][E], g[NC][E];
    float ss = 0.0f, dot = 0.0f;
    if (live) {
      const char *hr = static_cast<const char *>(a.h) + t * a.ld_h * S;
      const char *gr = static_cast<const char *>(a.dy) + t * a.ld_dy * S;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        load_chunk<D, AL>(hr, ((c * W + wave % W) * 64 + lane) * E, d, h[c]);
        load_chunk<D, AL>(gr, ((c * W + wave % W) * 64 + lane) * E, d, g[c]);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          ss += h[c][i] * h[c][i];
          dot += g[c][i] * w[c][i] * h[c][i];
        }
    }
    uint32_t top = 0;
    row_reduce<W>(ss, dot, top, lds[turn], wave);
    turn ^= 1;  // the next row's sums go to the other half: no barrier before they are written
    if (live) {
      const float r = rsqrtf(ss / (float)d + a.eps);
      const float k = r * r * (dot / (float)d);
      const char *sr = a.dh ? static_cast<const char *>(a.dh) + t * a.ld_dh * S : nullptr;
      char *xr = static_cast<char *>(a.dx) + t * a.ld_dx * S;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e0 = ((c * W + wave % W) * 64 + lane) * E;
        float o[E];
        if (sr != nullptr)
          load_chunk<D, AL>(sr, e0, d, o);
        else
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          dw[c][i] += g[c][i] * h[c][i] * r;
          o[i] += r * (g[c][i] * w[c][i] - h[c][i] * k);
        }
        store_chunk<D, AL>(xr, e0, d, o);
      }
    }
  }
  // the workgroup's partial row: its RB row groups added in order
  float *out = a.partial + (size_t)blockIdx.x * d;
  if constexpr (RB == 1) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int e = ((c * W + wave % W) * 64 + lane) * E + i;
        if (e < d) out[e] = dw[c][i];
      }
  } else {
    __shared__ float sum[RB][W * 64 * E];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) sum[wave / W][((wave % W) * 64 + lane) * E + i] = dw[c][i];
      __syncthreads();
      for (int e = threadIdx.x; e < W * 64 * E; e += 64 * RW) {
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < RB; ++g) s += sum[g][e];
        const int j = c * W * 64 * E + e;
        if (j < d) out[j] = s;
      }
    }
  }
}

// dw_j = the partial rows added in order: 64 columns per workgroup, 16 groups
// of rows, their sums added in order.
constexpr int DW_GROUPS = 16;
__global__ __launch_bounds__(64 * DW_GROUPS) void k_norm_dweight(const float *__restrict__ partial, int n, int d,
                                                                 float *__restrict__ dweight) {
  __shared__ float sum[DW_GROUPS][64];
  const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const int j = blockIdx.x * 64 + lane;
  const int per = (n + DW_GROUPS - 1) / DW_GROUPS;
  float s = 0.0f;
  if (j < d)
    for (int i = grp * per; i < min(n, (grp + 1) * per); ++i) s += partial[(size_t)i * d + j];
  sum[grp][lane] = s;
  __syncthreads();
  if (grp == 0 && j < d) {
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < DW_GROUPS; ++g) v += sum[g][lane];
    dweight[j] = v;
  }
}

// ---- launchers ----------------------------------------------------------------

static bool rows16(const void *p, int64_t ld, int s) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld * s) % 16 == 0);
}

template <Dt D, int W, int NC, bool NORM>
static hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
  constexpr int S = DtT<D>::size;
  constexpr int RB = row_waves(W) / W;
  const bool al = rows16(a.x, a.ld_x, S) && rows16(a.residual, a.ld_res, S) && rows16(a.weight, 0, S) &&
                  rows16(a.h, a.ld_h, S) && rows16(a.y, a.ld_y, S);
  // at most 2^20 workgroups, which take more rows in turn
  const dim3 grid(std::min((a.rows - 1) / RB + 1, 1 << 20)), block(64 * row_waves(W));
  if (al)
    hipLaunchKernelGGL((k_norm_rows<D, W, NC, true, NORM>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_norm_rows<D, W, NC, false, NORM>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Chunks of 64 lanes x 16 bytes in a row: one wave up to 4 of them, 4 waves
// up to 16, 16 waves up to NORM_MAX_CHUNKS.
template <Dt D, bool NORM>
static hipError_t norm_rows_dt(const NormArgs &a, hipStream_t s) {
  const int chunks = norm_chunks(a.d, D);
  if (chunks <= 1) return launch_rows<D, 1, 1, NORM>(a, s);
  if (chunks <= 2) return launch_rows<D, 1, 2, NORM>(a, s);
  if (chunks <= 4) return launch_rows<D, 1, 4, NORM>(a, s);
  if (chunks <= 8) return launch_rows<D, 4, 2, NORM>(a, s);
  if (chunks <= 16) return launch_rows<D, 4, 4, NORM>(a, s);
  if (chunks <= 64) return launch_rows<D, 16, 4, NORM>(a, s);
  if (chunks <= NORM_MAX_CHUNKS) return launch_rows<D, 16, 8, NORM>(a, s);
  return hipErrorInvalidValue;
}

hipError_t norm_rows(const NormArgs &a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  if (a.weight != nullptr)
    return a.dtype == Dt::BF16 ? norm_rows_dt<Dt::BF16, true>(a, s) : norm_rows_dt<Dt::F32, true>(a, s);
  return a.dtype == Dt::BF16 ? norm_rows_dt<Dt::BF16, false>(a, s) : norm_rows_dt<Dt::F32, false>(a, s);
}

template <Dt D, int W, int NC>
static hipError_t launch_backward(const NormBackwardArgs &a, hipStream_t s) {
  constexpr int S = DtT<D>::size;
  const bool al = rows16(a.dy, a.ld_dy, S) && rows16(a.h, a.ld_h, S) && rows16(a.weight, 0, S) &&
                  rows16(a.dh, a.ld_dh, S) && rows16(a.dx, a.ld_dx, S);
  const dim3 grid(a.n_partial), block(64 * row_waves(W));
  if (al)
    hipLaunchKernelGGL((k_norm_backward<D, W, NC, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_norm_backward<D, W, NC, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <Dt D>
static hipError_t backward_dt(const NormBackwardArgs &a, hipStream_t s) {
  const int chunks = norm_chunks(a.d, D);
  if (chunks <= 1) return launch_backward<D, 1, 1>(a, s);
  if (chunks <= 2) return launch_backward<D, 1, 2>(a, s);
  if (chunks <= 4) return launch_backward<D, 1, 4>(a, s);
  if (chunks <= 8) return launch_backward<D, 4, 2>(a, s);
  if (chunks <= 16) return launch_backward<D, 4, 4>(a, s);
  if (chunks <= 64) return launch_backward<D, 16, 4>(a, s);
  if (chunks <= NORM_MAX_CHUNKS) return launch_backward<D, 16, 8>(a, s);
  return hipErrorInvalidValue;
}

int norm_backward_partials(int rows, int d, Dt dt) {
  const int rb = norm_chunks(d, dt) <= 4 ? 4 : 1;  // rows per workgroup step
  return std::max(1, std::min((int)(((int64_t)rows + rb - 1) / rb), NORM_BACKWARD_WGS));
}

hipError_t norm_backward(const NormBackwardArgs &a, hipStream_t s) {
  // with no rows the one workgroup writes a partial row of zeros
  hipError_t e = a.dtype == Dt::BF16 ? backward_dt<Dt::BF16>(a, s) : backward_dt<Dt::F32>(a, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_norm_dweight, dim3((a.d + 63) / 64), dim3(64 * DW_GROUPS), 0, s, a.partial, a.n_partial, a.d,
                     a.dweight);
  return hipGetLastError();
}

}  // namespace twell
