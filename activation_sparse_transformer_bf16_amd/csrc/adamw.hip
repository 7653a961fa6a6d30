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

#include <float.h>
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

// Codes are the top bits of an fp32 number whose exponent field is the code's own,
// subnormal where the code is, so that v_ldexp_f32 (one rounding, subnormal numbers
// kept) takes a code to its value and back.  The exponent to add to a code:
__device__ __forceinline__ int state_exponent(uint32_t byte, int top) { return max((int)byte, E_MIN) - top; }
__device__ __forceinline__ bool state_is_nan(uint32_t byte) { return byte > (uint32_t)E_MAX; }
// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t state_scale(uint32_t top_bits) {
  const uint32_t e = (top_bits + 0xFFFFFu) >> 23;
  return e > (uint32_t)E_MAX ? 255u : max(e, (uint32_t)E_MIN);
}
// The bits of x scaled down to its code, which the dropped 20 bits plus 16 random ones
// (and half of the last one's step) carry into; the code is bits 20 to 27, the sign
// stays in bit 31.
__device__ __forceinline__ uint32_t state_bits(float x, int exponent, uint32_t random16) {
  return __float_as_uint(__builtin_amdgcn_ldexpf(x, -exponent)) + (random16 << 4 | 8u);
}

// The largest of v over the 4 lanes (8 elements each) of a block.
__device__ __forceinline__ uint32_t quad_top(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));     // quad_perm 1,0,3,2
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
}

// ---- lists of tensors -----------------------------------------------------------

constexpr int STEP_WAVES = 4, STEP_EACH = 8;             // waves of a workgroup, elements of a lane
constexpr int STEP_CHUNK = 64 * STEP_WAVES * STEP_EACH;  // elements of a workgroup
constexpr int STEP_WGS = 1 << 20;                        // workgroups, which take more chunks in turn

// Tensors of one launch and the number of their first chunk; by value, so that
// nothing has to be copied to the GPU before it.
template <class T, int MAX>
struct List {
  int count;
  int64_t chunks;  // in all
  int64_t first[MAX];
  T t[MAX];
};

// The list's first chunks, one per lane: which tensor a chunk belongs to is then one
// comparison for all of them, with no walk through memory.
template <class T, int MAX>
struct Finder {
  static constexpr int N = (MAX + 63) / 64;
  int64_t first[N];
  __device__ __forceinline__ explicit Finder(const List<T, MAX> &l) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < N; ++k) first[k] = lane + 64 * k < l.count ? l.first[min(lane + 64 * k, MAX - 1)] : INT64_MAX;
  }
  // The last tensor that starts at or before chunk c: of several without an element,
  // all of which start there, the one that has some.
  __device__ __forceinline__ int operator()(int64_t c) const {
    int n = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) n += popc64(ballot(first[k] <= c));
    return __builtin_amdgcn_readfirstlane(n - 1);
  }
};

// 16 bytes at any alignment.
typedef uint32_t u32x4_free_t __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_free_t __attribute__((ext_vector_type(2), aligned(1)));

// Loads and stores carry the non-temporal bit but for the norm's loads of the
// gradients, which the step reads next: what a step writes is not read again before
// memory has it, and without the bit the writes of one kernel are still under way to
// memory, and in the way, while the next one reads (norm and step of 50M weights with
// fp32 states 327 -> 302 us, with 8-bit states and their reading 216 -> 183; the norm
// alone 44 to 66 -> 36 us; with the bit in the norm 327 and 192).
template <bool NT, class V>
__device__ __forceinline__ V load_free(const void *p) {
  if constexpr (NT)
    return __builtin_nontemporal_load(static_cast<const V *>(p));
  else
    return *static_cast<const V *>(p);
}

// 8 elements from p + at on.  WHOLE: all there are the tensor's; otherwise `left` of
// them, and zeros.  LANES: a lane that has all 8 loads them at once (the step itself
// loads the last chunk of a tensor by elements: 104 us for 50M weights with 8-bit
// states, with both kinds of load in its code 112).
template <Dt D, bool WHOLE, bool NT = true, bool LANES = false>
__device__ __forceinline__ void load8(const void *p, int64_t at, int64_t left, float (&v)[8]) {
  using T = typename DtT<D>::T;
  const T *q = static_cast<const T *>(p) + at;
  if constexpr (!WHOLE) {
    if (LANES && left >= 8) return load8<D, true, NT>(p, at, left, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(q[i]) : 0.0f;
  } else if constexpr (D == Dt::BF16) {
    const u32x4_t w = load_free<NT, u32x4_free_t>(q);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i % 2 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
  } else {
    const u32x4_t a = load_free<NT, u32x4_free_t>(q), b = load_free<NT, u32x4_free_t>(q + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i < 4 ? a[i] : b[i - 4]);
  }
}
template <bool WHOLE, bool LANES = false>
__device__ __forceinline__ u32x2_t load8_codes(const uint8_t *p, int64_t left) {
  if (WHOLE || (LANES && left >= 8)) return load_free<true, u32x2_free_t>(p);
  u32x2_t c = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) c[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  return c;
}
// 8 elements' bits: fp32, or bf16 in the low halves.
template <class V>
__device__ __forceinline__ void store_free(void *p, V v) {
  __builtin_nontemporal_store(v, static_cast<V *>(p));
}
template <Dt D, bool WHOLE, bool LANES = false>
__device__ __forceinline__ void store8(void *p, int64_t at, int64_t left, const uint32_t (&v)[8]) {
  using T = typename DtT<D>::T;
  T *q = static_cast<T *>(p) + at;
  if constexpr (!WHOLE) {
    if (LANES && left >= 8) return store8<D, true>(p, at, left, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= left) break;
      if constexpr (D == Dt::BF16)
        q[i] = (uint16_t)v[i];
      else
        q[i] = __uint_as_float(v[i]);
    }
  } else if constexpr (D == Dt::BF16) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x05040100u);
    store_free<u32x4_free_t>(q, w);
  } else {
    store_free<u32x4_free_t>(q, u32x4_t{v[0], v[1], v[2], v[3]});
    store_free<u32x4_free_t>(q + 4, u32x4_t{v[4], v[5], v[6], v[7]});
  }
}
template <Dt D, bool WHOLE, bool LANES = false>
__device__ __forceinline__ void store8_f32(void *p, int64_t at, int64_t left, const float (&v)[8]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = D == Dt::BF16 ? (uint32_t)bf16_rne(v[i]) : __float_as_uint(v[i]);
  store8<D, WHOLE, LANES>(p, at, left, w);
}
template <bool WHOLE>
__device__ __forceinline__ void store8_codes(uint8_t *p, int64_t left, u32x2_t c) {
  if constexpr (WHOLE) {
    store_free<u32x2_free_t>(p, c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint8_t)(c[i / 4] >> (8 * (i % 4)));
  }
}

// The bits of byte i's code as state_exponent() takes them.
template <bool SIGNED>
__device__ __forceinline__ uint32_t code_at(uint32_t c, int i) {
  const uint32_t at20 = i < 3 ? c << (20 - 8 * i) : c >> 4;
  return SIGNED ? (at20 & 0x07F00000u) | (c << (24 - 8 * i) & 0x80000000u) : at20 & 0x0FF00000u;
}
// The topmost bytes of four numbers, the first one lowest.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0703u), hi = __builtin_amdgcn_perm(d, c, 0x07030C0Cu);
  return lo | hi;
}

// ---- the step ----------------------------------------------------------------------
//
// A lane takes 8 elements, a workgroup a chunk of 2048: every buffer in accesses of 16
// bytes, and a block's scale from four neighbours by two DPP moves.  A chunk each rather
// than several in turn, which would wait for one another, and the step's numbers from
// the host where they are known there (both together: 50M weights with fp32 states and
// the norm 352 -> 326 us).
//
// Memory bound (50.3 million weights, clip on; times in a row of graphs): bf16 weights
// with fp32 copy and states 264 to 285 us (1.51 GB, 5.3 to 5.7 TB/s), bf16 gradients 265
// (1.41 GB), fp32 weights 263 (1.41 GB); 8-bit states, bf16 weights alone 95 to 107 us
// (610 MB, 5.7 to 6.4), bf16 gradients too 95 (510 MB, 5.4: the codes' and the hash's 55
// instructions an element show), with fp32 copy 164, fp32 weights 148.  13 tensors of
// 333 to 43290 elements 6.0 us.  A launch takes 40 tensors (kernel arguments hold 4 KB):
// 1000 tensors of 4096 take 25 launches, 93 us.

struct StepScalars {
  float beta1, rest1, beta2, rest2, eps;  // rest: 1 - beta
  float rate, root;                       // with lr and step from the host
  double lr, log1, log2;                  // logarithms of the betas
  int64_t step;
  uint64_t seed;
  const float *lr_device;
  const int64_t *step_device;
  const float *clip;
};

using StepList = List<AdamWTensor, ADAMW_LIST>;

// lr / (1 - beta1^t) and 1 / sqrt(1 - beta2^t); log = log(beta)
__host__ __device__ inline float step_rate(double lr, int64_t t, double log1) { return (float)(lr / -expm1((double)t * log1)); }
__host__ __device__ inline float step_root(int64_t t, double log2) { return (float)(1.0 / sqrt(-expm1((double)t * log2))); }

// A step's numbers, the same for all tensors.
struct StepNow {
  float factor, rate, root;
  double lr;
  uint32_t key;
};

// One lane's 8 elements.
template <Dt W, Dt G, bool BITS8, bool MASTER, bool WHOLE>
__device__ __forceinline__ void step8(const AdamWTensor &t, int64_t e0, const StepScalars &c, const StepNow &now) {
#pragma clang fp contract(off)
  const int64_t left = t.n - e0;
  float g[8], m[8], v[8], w[8];
  load8<G, WHOLE>(t.grad, e0, left, g);
  if constexpr (MASTER)
    load8<Dt::F32, WHOLE>(t.master, e0, left, w);
  else
    load8<W, WHOLE>(t.weight, e0, left, w);
  uint8_t *mc = static_cast<uint8_t *>(t.m) + e0, *vc = static_cast<uint8_t *>(t.v) + e0;
  const int64_t block = e0 / STATE_BLOCK;
  if constexpr (BITS8) {
    const u32x2_t a = load8_codes<WHOLE>(mc, left), b = load8_codes<WHOLE>(vc, left);
    const bool some = WHOLE || left > 0;
    const uint32_t mb = some ? t.m_scale[block] : 0u, vb = some ? t.v_scale[block] : 0u;
    const int me = state_exponent(mb, M_TOP), ve = state_exponent(vb, V_TOP);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = __builtin_amdgcn_ldexpf(__uint_as_float(code_at<true>(a[i / 4], i % 4)), me);
      v[i] = __builtin_amdgcn_ldexpf(__uint_as_float(code_at<false>(b[i / 4], i % 4)), ve);
    }
    if (__builtin_expect(state_is_nan(mb) || state_is_nan(vb), 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (state_is_nan(mb)) m[i] = __uint_as_float(0x7FC00000u);
        if (state_is_nan(vb)) v[i] = __uint_as_float(0x7FC00000u);
      }
    }
  } else {
    load8<Dt::F32, WHOLE>(t.m, e0, left, m);
    load8<Dt::F32, WHOLE>(t.v, e0, left, v);
  }
  const float keep = (float)(1.0 - now.lr * (double)t.decay);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = g[i] * now.factor;
    m[i] = m[i] * c.beta1 + x * c.rest1;
    v[i] = v[i] * c.beta2 + (x * c.rest2) * x;
    // the root and the reciprocal to 1 ulp each, as the instructions give them
    const float denom = fmaf(__builtin_amdgcn_sqrtf(v[i]), now.root, c.eps);
    w[i] = fmaf(-now.rate, m[i] * __builtin_amdgcn_rcpf(denom), w[i] * keep);
  }
  uint32_t random[8];
  if constexpr (BITS8 || (W == Dt::BF16 && !MASTER)) {
    const uint64_t group = (uint64_t)e0 / 8;
    const uint32_t key = mix32(now.key + (uint32_t)t.place) + (uint32_t)(group >> 32) * 0x9E3779B1u;
    // (base + i * 0x9E3779B9) * 0x85EBCA6B, the group's part multiplied once
    const uint32_t base = mix32((uint32_t)group + key) * 0x85EBCA6Bu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      random[i] = base + (uint32_t)i * (0x9E3779B9u * 0x85EBCA6Bu);
      random[i] ^= random[i] >> 16;
    }
  }
  if constexpr (BITS8) {
    // the largest magnitudes; NaN wins
    float mt = 0.0f, vt = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mt = __builtin_elementwise_maximum(mt, fabsf(m[i]));
      vt = __builtin_elementwise_maximum(vt, v[i]);
    }
    const uint32_t ms = state_scale(quad_top(__float_as_uint(mt) & 0x7FFFFFFFu));
    const uint32_t vs = state_scale(quad_top(__float_as_uint(vt) & 0x7FFFFFFFu));
    const int md = state_exponent(min(ms, (uint32_t)E_MAX), M_TOP), vd = state_exponent(min(vs, (uint32_t)E_MAX), V_TOP);
    uint32_t x[8], y[8], low = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = state_bits(m[i], md, random[i] & 0xFFFFu);
      x[i] = (x[i] & 0x80000000u) | (x[i] << 4 & 0x7FFFFFFFu);  // sign and code in the topmost byte
      y[i] = state_bits(v[i], vd, random[i] >> 16);
      low = min(low, y[i]);
      y[i] <<= 4;
    }
    u32x2_t a = {top_bytes(x[0], x[1], x[2], x[3]), top_bytes(x[4], x[5], x[6], x[7])};
    u32x2_t b = {top_bytes(y[0], y[1], y[2], y[3]), top_bytes(y[4], y[5], y[6], y[7])};
    if (__builtin_expect(low < 1u << 20, 0)) {  // some v has the code 0: those above 0 get 1
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (y[i] < 1u << 24 && v[i] > 0.0f) b[i / 4] |= 1u << (8 * (i % 4));
    }
    if (__builtin_expect(ms == 255u || vs == 255u, 0)) {
      if (ms == 255u) a = u32x2_t{0u, 0u};
      if (vs == 255u) b = u32x2_t{0u, 0u};
    }
    store8_codes<WHOLE>(mc, left, a);
    store8_codes<WHOLE>(vc, left, b);
    if (threadIdx.x % 4 == 0 && (WHOLE || left > 0)) {
      t.m_scale[block] = (uint8_t)ms;
      t.v_scale[block] = (uint8_t)vs;
    }
  } else {
    store8_f32<Dt::F32, WHOLE>(t.m, e0, left, m);
    store8_f32<Dt::F32, WHOLE>(t.v, e0, left, v);
  }
  if constexpr (MASTER) store8_f32<Dt::F32, WHOLE>(t.master, e0, left, w);
  if constexpr (W == Dt::BF16 && !MASTER) {
    uint32_t bits[8];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bits[i] = (__float_as_uint(w[i]) + (random[i] >> 8 & 0xFFFFu)) >> 16;
      top = __builtin_elementwise_maximum(top, fabsf(w[i]));
    }
    if (__builtin_expect(!(top <= 3.4e38f), 0)) {
      // infinities and NaN as they are: the addition would carry through them
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(fabsf(w[i]) <= 3.4e38f)) bits[i] = bf16_rne(w[i]);
    }
    store8<W, WHOLE>(t.weight, e0, left, bits);
  } else {
    store8_f32<W, WHOLE>(t.weight, e0, left, w);
  }
}

template <Dt W, Dt G, bool BITS8, bool MASTER>
__global__ __launch_bounds__(64 * STEP_WAVES) void k_adamw(StepList list, StepScalars c) {
  StepNow now;
  now.factor = c.clip != nullptr ? c.clip[1] : 1.0f;
  if (!(fabsf(now.factor) <= FLT_MAX)) return;  // gradients with inf or NaN: the step is left out
  int64_t step = c.step;
  now.lr = c.lr;
  now.rate = c.rate;
  now.root = c.root;
  if (c.step_device != nullptr || c.lr_device != nullptr) {  // about 1 us of fp64 arithmetic, once per wave
    if (c.step_device != nullptr) step = *c.step_device;
    if (step < 1) return;
    if (c.lr_device != nullptr) now.lr = (double)*c.lr_device;
    now.rate = step_rate(now.lr, step, c.log1);
    now.root = step_root(step, c.log2);
  }
  const uint64_t seed = c.seed + (uint64_t)step;
  now.key = mix32((uint32_t)seed ^ mix32((uint32_t)(seed >> 32)));
  const Finder<AdamWTensor, ADAMW_LIST> find(list);
  for (int64_t chunk = blockIdx.x; chunk < list.chunks; chunk += gridDim.x) {
    const int at = find(chunk);
    const AdamWTensor &t = list.t[at];
    const int64_t start = (chunk - list.first[at]) * STEP_CHUNK;
    const int64_t e0 = start + threadIdx.x * STEP_EACH;
    if (start + STEP_CHUNK <= t.n)
      step8<W, G, BITS8, MASTER, true>(t, e0, c, now);
    else
      step8<W, G, BITS8, MASTER, false>(t, e0, c, now);
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
  const dim3 grid((unsigned)std::min<int64_t>(l.chunks, STEP_WGS));
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
  const double log1 = log(a.beta1), log2 = log(a.beta2);
  const StepScalars c{(float)a.beta1, (float)(1.0 - a.beta1), (float)a.beta2, (float)(1.0 - a.beta2), (float)a.eps,
                      step_rate(a.lr, a.step, log1), step_root(a.step, log2), a.lr, log1, log2, a.step, a.seed,
                      a.lr_device, a.step_device, a.clip};
  if (weight == Dt::BF16)
    return grad == Dt::BF16 ? step_kinds<Dt::BF16, Dt::BF16>(t, count, bits8, master, c, s)
                            : step_kinds<Dt::BF16, Dt::F32>(t, count, bits8, master, c, s);
  return grad == Dt::BF16 ? step_kinds<Dt::F32, Dt::BF16>(t, count, bits8, master, c, s)
                          : step_kinds<Dt::F32, Dt::F32>(t, count, bits8, master, c, s);
}

// ---- reading 8-bit states ------------------------------------------------------------

using ReadList = List<StateRead, STATE_LIST>;

// A workgroup takes READ_EACH pieces of a chunk at a time, whose codes are all on
// their way before the first is waited for.  Memory bound: m and v of 50.3 million
// weights to bf16 51 us (305 MB, 6.0 TB/s).
constexpr int READ_EACH = 4, READ_CHUNK = READ_EACH * STEP_CHUNK;

template <Dt D, bool WHOLE>
__device__ __forceinline__ void read_chunk(const StateRead &t, int64_t start) {
  u32x2_t c[READ_EACH];
  uint32_t byte[READ_EACH];
#pragma unroll
  for (int k = 0; k < READ_EACH; ++k) {
    const int64_t e0 = start + k * STEP_CHUNK + threadIdx.x * STEP_EACH, left = t.n - e0;
    c[k] = load8_codes<WHOLE, true>(t.code + e0, left);
    byte[k] = WHOLE || left > 0 ? t.scale[e0 / STATE_BLOCK] : 0u;
  }
#pragma unroll
  for (int k = 0; k < READ_EACH; ++k) {
    const int64_t e0 = start + k * STEP_CHUNK + threadIdx.x * STEP_EACH, left = t.n - e0;
    const int e = state_exponent(byte[k], t.is_signed ? M_TOP : V_TOP);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = t.is_signed ? code_at<true>(c[k][i / 4], i % 4) : code_at<false>(c[k][i / 4], i % 4);
      x[i] = state_is_nan(byte[k]) ? __uint_as_float(0x7FC00000u) : __builtin_amdgcn_ldexpf(__uint_as_float(b), e);
    }
    store8_f32<D, WHOLE, true>(t.out, e0, left, x);
  }
}

template <Dt D>
__global__ __launch_bounds__(64 * STEP_WAVES) void k_state_read(ReadList list) {
  const Finder<StateRead, STATE_LIST> find(list);
  for (int64_t chunk = blockIdx.x; chunk < list.chunks; chunk += gridDim.x) {
    const int at = find(chunk);
    const StateRead &t = list.t[at];
    const int64_t start = (chunk - list.first[at]) * READ_CHUNK;
    if (start + READ_CHUNK <= t.n)
      read_chunk<D, true>(t, start);
    else
      read_chunk<D, false>(t, start);
  }
}

hipError_t state_read(const StateRead *r, int count, Dt dtype, hipStream_t s) {
  if (count > STATE_LIST) return hipErrorInvalidValue;
  ReadList l{};
  const int64_t chunks = list_fill(l, r, count, READ_CHUNK, [](const StateRead &x) { return x.n; });
  if (chunks == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(chunks, STEP_WGS)), block(64 * STEP_WAVES);
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
// adds them in order.  50.3 million fp32 gradients 36 us (201 MB, 5.6 TB/s) and 4 for
// the second launch, bf16 21 in all.

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

template <Dt D, bool WHOLE>
__device__ __forceinline__ double squares8(const void *p, int64_t at, int64_t left) {
  float x[8];
  load8<D, WHOLE, false, true>(p, at, left, x);
  double s[2] = {0.0, 0.0};
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i % 2] = fma((double)x[i], (double)x[i], s[i % 2]);
  return s[0] + s[1];
}

__global__ __launch_bounds__(64 * STEP_WAVES) void k_grad_squares(GradList list, double *partial) {
  __shared__ double buf[STEP_WAVES];
  const Finder<GradRef, GRAD_LIST> find(list);
  double sum = 0.0;
  for (int64_t chunk = blockIdx.x; chunk < list.chunks; chunk += gridDim.x) {
    const int at = find(chunk);
    const GradRef &t = list.t[at];
    const int64_t start = (chunk - list.first[at]) * GRAD_CHUNK;
    const int64_t e0 = start + threadIdx.x * 8;
    double s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t e = e0 + k * (64 * STEP_WAVES * 8);
      if (start + GRAD_CHUNK <= t.n)
        s[k] = t.dtype == Dt::BF16 ? squares8<Dt::BF16, true>(t.p, e, 8) : squares8<Dt::F32, true>(t.p, e, 8);
      else
        s[k] = t.dtype == Dt::BF16 ? squares8<Dt::BF16, false>(t.p, e, t.n - e) : squares8<Dt::F32, false>(t.p, e, t.n - e);
    }
    sum += s[0] + s[1];
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
  out[1] = norm <= FLT_MAX ? fminf(1.0f, max_norm / norm) : __uint_as_float(0x7FC00000u);
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
