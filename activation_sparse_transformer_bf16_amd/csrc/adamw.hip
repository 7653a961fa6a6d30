// The optimiser: AdamW over many tensors at once, and the norm of their gradients.
//
//   g = grad * factor
//   m = b1 m + (1 - b1) g,   v = b2 v + ((1 - b2) g) g
//   w = (1 - lr decay) w - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in fp32, one rounding per operation in m and v, which are what 8-bit states are
// rounded from.
//
// States in 8 bits: blocks of 32 elements of a tensor share a scale 2^E, E the
// smallest whole number with max <= 1.875 * 2^E.  m is a sign, 4 exponent and 3
// mantissa bits; v, which has no sign, 5 and 3.  The topmost exponent stands for 2^E
// and the lowest for subnormal numbers, so m reaches down to 2^(E-17) and v to
// 2^(E-33), half as far in sqrt(v).
//
// A step changes v by (1 - b2) of it, 0.1 to 5%, far less than the step between
// two codes (6 to 12%): rounded to nearest, v would never move.  So states are rounded
// to one of their two neighbours by 16 random bits, up as often as the value lies
// near the upper one, and the mean is right.  v > 0 is not rounded to 0, which
// would leave m / eps.  bf16 weights with no fp32 copy are rounded in the same way,
// for the same reason.
//
// The random bits are a hash of the step (and the caller's seed), the tensor's
// place in the list and the element: the same call gives the same results.
#include "launch.hpp"

#include <math.h>

namespace twell {

constexpr int STATE_BLOCK = 32;
constexpr int M_TOP = 15, V_TOP = 31;  // the topmost exponent fields
constexpr int E_MIN = 40, E_MAX = 240; // scale bytes: 2^-87 ... 2^113; a larger block is NaN (255)

__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0x85EBCA6Bu;
  return x ^ (x >> 16);
}

// 2^e for the exponents of normal numbers.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Codes are the top bits of an fp32 number whose exponent field is the code's own,
// subnormal where the code is.  Such numbers are below 2^-90, so the scale comes
// in two factors: 2^100, which is exact, and the rest.
__device__ __forceinline__ float state_unit(uint32_t byte, int top) {
  return byte > (uint32_t)E_MAX ? __uint_as_float(0x7FC00000u) : pow2(max((int)byte, E_MIN) - top - 100);
}
__device__ __forceinline__ float state_value(uint32_t code, float unit) {
  return __uint_as_float(code << 20) * 0x1p100f * unit;
}
// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t state_scale(uint32_t top_bits) {
  const uint32_t e = (top_bits + 0xFFFFFu) >> 23;
  return e > (uint32_t)E_MAX ? 255u : max(e, (uint32_t)E_MIN);
}
// A magnitude to its code; `down` = 2^(top + 100 - E).  The dropped 20 bits plus
// 16 random ones (and half of the last one's step) carry into the code.
__device__ __forceinline__ uint32_t state_code(float x, float down, uint32_t random16) {
  const float y = x * down * 0x1p-100f;
  return (__float_as_uint(y) + (random16 << 4 | 8u)) >> 20;
}

// The largest of v over the 4 lanes (8 elements each) of a block.
__device__ __forceinline__ uint32_t quad_top(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));     // quad_perm 1,0,3,2
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
}

// ---- lists of tensors -----------------------------------------------------------

constexpr int STEP_WAVES = 4, STEP_EACH = 8;                 // elements per lane
constexpr int STEP_CHUNK = 64 * STEP_WAVES * STEP_EACH;      // elements per workgroup

// Tensors of one launch and the number of their first chunk; by value, so that
// nothing has to be copied to the GPU before it.
template <class T, int MAX>
struct List {
  int count;
  int64_t chunks;  // in all
  int64_t first[MAX];
  T t[MAX];
};

// The tensor that holds chunk c.
template <class T, int MAX>
__device__ __forceinline__ int list_find(const List<T, MAX> &l, int64_t c) {
  int i = 0;
  while (i + 1 < l.count && l.first[i + 1] <= c) ++i;
  return i;
}

// E elements from p on, of which `left` are the tensor's; aligned to the element only.
template <Dt D, int E>
__device__ __forceinline__ void load_elements(const void *p, int64_t at, int64_t left, float (&v)[E]) {
  using T = typename DtT<D>::T;
  const T *q = static_cast<const T *>(p) + at;
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = i < left ? to_f32(q[i]) : 0.0f;
}

// ---- the step ----------------------------------------------------------------------

struct StepScalars {
  float beta1, rest1, beta2, rest2, eps;  // rest: 1 - beta
  double lr, log1, log2;                  // logarithms of the betas
  int64_t step;
  uint64_t seed;
  const float *lr_device;
  const int64_t *step_device;
  const float *clip;
};

using StepList = List<AdamWTensor, ADAMW_LIST>;

template <Dt W, Dt G, bool BITS8, bool MASTER>
__global__ __launch_bounds__(64 * STEP_WAVES) void k_adamw(StepList list, StepScalars c) {
#pragma clang fp contract(off)
  constexpr int E = STEP_EACH;
  using T = typename DtT<W>::T;
  const float factor = c.clip != nullptr ? c.clip[1] : 1.0f;
  if (!(fabsf(factor) <= 3.0e38f)) return;  // gradients with inf or NaN: the step is left out
  const int64_t step = c.step_device != nullptr ? *c.step_device : c.step;
  if (step < 1) return;
  const double lr = c.lr_device != nullptr ? (double)*c.lr_device : c.lr;
  const float rate = (float)(lr / -expm1((double)step * c.log1));
  const float root = (float)(1.0 / sqrt(-expm1((double)step * c.log2)));
  const uint64_t seed = c.seed + (uint64_t)step;
  const uint32_t key0 = mix32((uint32_t)seed ^ mix32((uint32_t)(seed >> 32)));
  for (int64_t chunk = blockIdx.x; chunk < list.chunks; chunk += gridDim.x) {
    const int at = list_find(list, chunk);
    const AdamWTensor &t = list.t[at];
    const int64_t e0 = (chunk - list.first[at]) * STEP_CHUNK + threadIdx.x * E;
    const int64_t left = t.n - e0;
    const uint64_t group = (uint64_t)e0 / 8;
    const uint32_t key = mix32(key0 + (uint32_t)t.place) + (uint32_t)(group >> 32) * 0x9E3779B1u;
    const uint32_t base = mix32((uint32_t)group + key);
    float g[E], m[E], v[E], w[E];
    uint32_t random[E];
    load_elements<G>(t.grad, e0, left, g);
    if (MASTER)
      load_elements<Dt::F32>(t.master, e0, left, w);
    else
      load_elements<W>(t.weight, e0, left, w);
    if constexpr (BITS8) {
      const uint8_t *mc = static_cast<const uint8_t *>(t.m) + e0, *vc = static_cast<const uint8_t *>(t.v) + e0;
      const float mu = left > 0 ? state_unit(t.m_scale[e0 / STATE_BLOCK], M_TOP) : 0.0f;
      const float vu = left > 0 ? state_unit(t.v_scale[e0 / STATE_BLOCK], V_TOP) : 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint32_t a = i < left ? mc[i] : 0u, b = i < left ? vc[i] : 0u;
        const float x = state_value(a & 127u, mu);
        m[i] = a & 128u ? -x : x;
        v[i] = state_value(b, vu);
      }
    } else {
      load_elements<Dt::F32>(t.m, e0, left, m);
      load_elements<Dt::F32>(t.v, e0, left, v);
    }
    const float keep = (float)(1.0 - lr * (double)t.decay);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float x = g[i] * factor;
      m[i] = m[i] * c.beta1 + x * c.rest1;
      v[i] = v[i] * c.beta2 + (x * c.rest2) * x;
      const float denom = sqrtf(v[i]) * root + c.eps;
      w[i] = w[i] * keep - rate * (m[i] / denom);
      random[i] = (base + (uint32_t)i * 0x9E3779B9u) * 0x85EBCA6Bu;
      random[i] ^= random[i] >> 16;
    }
    if constexpr (BITS8) {
      uint32_t mt = 0, vt = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (i >= left) continue;
        mt = max(mt, __float_as_uint(m[i]) & 0x7FFFFFFFu);
        vt = max(vt, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      }
      const uint32_t ms = state_scale(quad_top(mt)), vs = state_scale(quad_top(vt));
      const float md = pow2(M_TOP + 100 - min((int)ms, E_MAX)), vd = pow2(V_TOP + 100 - min((int)vs, E_MAX));
      uint8_t *mc = static_cast<uint8_t *>(t.m) + e0, *vc = static_cast<uint8_t *>(t.v) + e0;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (i >= left) break;
        const uint32_t a = state_code(fabsf(m[i]), md, random[i] & 0xFFFFu);
        const uint32_t b = max(state_code(v[i], vd, random[i] >> 16), v[i] > 0.0f ? 1u : 0u);
        mc[i] = ms == 255u ? 0 : (uint8_t)(a | (__float_as_uint(m[i]) >> 31) << 7);
        vc[i] = vs == 255u ? 0 : (uint8_t)b;
      }
      if (threadIdx.x % 4 == 0 && left > 0) {
        t.m_scale[e0 / STATE_BLOCK] = (uint8_t)ms;
        t.v_scale[e0 / STATE_BLOCK] = (uint8_t)vs;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (i >= left) break;
        static_cast<float *>(t.m)[e0 + i] = m[i];
        static_cast<float *>(t.v)[e0 + i] = v[i];
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (i >= left) break;
      if (MASTER) t.master[e0 + i] = w[i];
      if constexpr (W == Dt::BF16 && !MASTER) {
        const uint32_t bits = __float_as_uint(w[i]);
        const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
        static_cast<T *>(t.weight)[e0 + i] =
            finite ? (uint16_t)((bits + ((random[i] >> 8) & 0xFFFFu)) >> 16) : from_f32<W>(w[i]);
      } else {
        static_cast<T *>(t.weight)[e0 + i] = from_f32<W>(w[i]);
      }
    }
  }
}

template <class T, int MAX, class Size>
static int64_t list_fill(List<T, MAX> &l, const T *t, int count, int chunk, Size size) {
  l.count = count;
  l.chunks = 0;
  for (int i = 0; i < count; ++i) {
    l.t[i] = t[i];
    l.first[i] = l.chunks;
    l.chunks += (size(t[i]) + chunk - 1) / chunk;
  }
  return l.chunks;
}

template <Dt W, Dt G, bool BITS8, bool MASTER>
static hipError_t launch_step(const AdamWTensor *t, int count, const StepScalars &c, hipStream_t s) {
  StepList l{};
  if (list_fill(l, t, count, STEP_CHUNK, [](const AdamWTensor &x) { return x.n; }) == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(l.chunks, 1 << 20));
  hipLaunchKernelGGL((k_adamw<W, G, BITS8, MASTER>), grid, dim3(64 * STEP_WAVES), 0, s, l, c);
  return hipGetLastError();
}

template <Dt W, Dt G>
static hipError_t step_kinds(const AdamWTensor *t, int count, bool bits8, bool master, const StepScalars &c, hipStream_t s) {
  if constexpr (W == Dt::BF16) {
    if (master) return bits8 ? launch_step<W, G, true, true>(t, count, c, s) : launch_step<W, G, false, true>(t, count, c, s);
  }
  return bits8 ? launch_step<W, G, true, false>(t, count, c, s) : launch_step<W, G, false, false>(t, count, c, s);
}

hipError_t adamw_step(const AdamWTensor *t, int count, Dt weight, Dt grad, bool bits8, const AdamWArgs &a,
                      hipStream_t s) {
  if (count <= 0) return hipSuccess;
  if (count > ADAMW_LIST) return hipErrorInvalidValue;
  const bool master = t[0].master != nullptr;
  const StepScalars c{(float)a.beta1, (float)(1.0 - a.beta1), (float)a.beta2, (float)(1.0 - a.beta2), (float)a.eps,
                      a.lr, log(a.beta1), log(a.beta2), a.step, a.seed, a.lr_device, a.step_device, a.clip};
  if (weight == Dt::BF16)
    return grad == Dt::BF16 ? step_kinds<Dt::BF16, Dt::BF16>(t, count, bits8, master, c, s)
                            : step_kinds<Dt::BF16, Dt::F32>(t, count, bits8, master, c, s);
  return grad == Dt::BF16 ? step_kinds<Dt::F32, Dt::BF16>(t, count, bits8, master, c, s)
                          : step_kinds<Dt::F32, Dt::F32>(t, count, bits8, master, c, s);
}

// ---- reading 8-bit states ------------------------------------------------------------

using ReadList = List<StateRead, STATE_LIST>;

template <Dt D>
__global__ __launch_bounds__(64 * STEP_WAVES) void k_state_read(ReadList list) {
  for (int64_t chunk = blockIdx.x; chunk < list.chunks; chunk += gridDim.x) {
    const int at = list_find(list, chunk);
    const StateRead &t = list.t[at];
    const int64_t e0 = (chunk - list.first[at]) * STEP_CHUNK + threadIdx.x * STEP_EACH;
    const int64_t left = t.n - e0;
    if (left <= 0) continue;
    const float unit = state_unit(t.scale[e0 / STATE_BLOCK], t.is_signed ? M_TOP : V_TOP);
#pragma unroll
    for (int i = 0; i < STEP_EACH; ++i) {
      if (i >= left) break;
      const uint32_t c = t.code[e0 + i];
      const float x = state_value(t.is_signed ? c & 127u : c, unit);
      static_cast<typename DtT<D>::T *>(t.out)[e0 + i] = from_f32<D>(t.is_signed && (c & 128u) ? -x : x);
    }
  }
}

hipError_t state_read(const StateRead *r, int count, Dt dtype, hipStream_t s) {
  if (count > STATE_LIST) return hipErrorInvalidValue;
  ReadList l{};
  const int64_t chunks = list_fill(l, r, count, STEP_CHUNK, [](const StateRead &x) { return x.n; });
  if (chunks == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(chunks, 1 << 20)), block(64 * STEP_WAVES);
  if (dtype == Dt::BF16)
    hipLaunchKernelGGL(k_state_read<Dt::BF16>, grid, block, 0, s, l);
  else
    hipLaunchKernelGGL(k_state_read<Dt::F32>, grid, block, 0, s, l);
  return hipGetLastError();
}

// ---- the gradients' norm ---------------------------------------------------------------
//
// Squares and sums in 64 bits: no gradient overflows, and the order of the sum does
// not show in 32 bits.  Each workgroup leaves one partial sum, a second launch
// adds them in order.

constexpr int GRAD_CHUNK = 64 * STEP_WAVES * 16;  // elements
constexpr int GRAD_WGS = 2048;                    // partial sums of a launch, at most
using GradList = List<GradRef, GRAD_LIST>;

__device__ __forceinline__ double block_sum(double v, double *buf) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < (int)blockDim.x / 64; ++i) v += buf[i];
  return v;
}

__global__ __launch_bounds__(64 * STEP_WAVES) void k_grad_squares(GradList list, double *partial) {
  __shared__ double buf[STEP_WAVES];
  double sum = 0.0;
  for (int64_t chunk = blockIdx.x; chunk < list.chunks; chunk += gridDim.x) {
    const int at = list_find(list, chunk);
    const GradRef &t = list.t[at];
    const int64_t e0 = (chunk - list.first[at]) * GRAD_CHUNK + threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (e0 + i >= t.n) break;
      const double x = t.dtype == Dt::BF16 ? (double)to_f32(static_cast<const uint16_t *>(t.p)[e0 + i])
                                           : (double)static_cast<const float *>(t.p)[e0 + i];
      sum += x * x;
    }
  }
  sum = block_sum(sum, buf);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void k_grad_norm(const double *partial, int n, float max_norm, float *out) {
  __shared__ double buf[16];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) sum += partial[i];
  sum = block_sum(sum, buf);
  if (threadIdx.x != 0) return;
  const float norm = (float)sqrt(sum);
  out[0] = norm;
  // an infinite or NaN norm gives a NaN factor, which the step takes as "leave it out"
  out[1] = norm <= 3.0e38f ? fminf(1.0f, max_norm / norm) : __uint_as_float(0x7FC00000u);
}

static int64_t grad_fill(GradList &l, const GradRef *g, int count) {
  return list_fill(l, g, count, GRAD_CHUNK, [](const GradRef &x) { return x.n; });
}

int grad_wgs(const GradRef *g, int count) {
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) chunks += (g[i].n + GRAD_CHUNK - 1) / GRAD_CHUNK;
  return (int)std::min<int64_t>(chunks, GRAD_WGS);
}

hipError_t grad_squares(const GradRef *g, int count, double *partial, hipStream_t s) {
  if (count > GRAD_LIST) return hipErrorInvalidValue;
  GradList l{};
  if (grad_fill(l, g, count) == 0) return hipSuccess;
  hipLaunchKernelGGL(k_grad_squares, dim3(grad_wgs(g, count)), dim3(64 * STEP_WAVES), 0, s, l, partial);
  return hipGetLastError();
}

hipError_t grad_norm(const double *partial, int n, float max_norm, float *out, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(1024), 0, s, partial, n, max_norm, out);
  return hipGetLastError();
}

}  // namespace twell
