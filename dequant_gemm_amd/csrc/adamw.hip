// adamw.hip -- one AdamW step over many tensors, with fp32 or 8-bit states.
//
//   g' = g s (s an optional device scalar), m = b1 m + (1 - b1) g',
//   v = b2 v + (1 - b2) g'^2,
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32; the parameter is rounded once to its type.
//
// 8-bit states: blocks of 256 consecutive elements of a tensor, an fp32 scale
// each; m as e4m3, v as its square root in e4m3 (half the exponent range, and
// the root is what the step divides by).  Three mantissa bits cannot follow a
// moving average with b2 = 0.999 if they are rounded to nearest: a step's
// change is far below half a code step, and the state would never move.  The
// codes are therefore rounded up with the probability of the remainder, by 16
// random bits per value hashed from the element's index in its tensor, the
// tensor's number and the caller's seed: unbiased, and the same on every run.
// One exception: a root that is not zero takes at least the smallest code.  A
// root rounded to zero beside a moment rounded up would make the next step as
// long as the two are wrong (gradients 10^-6 of their block's largest: up to 410
// times the learning rate in 400 steps; held at the smallest code 1.4, and 2.6 at
// other ratios).
// Non-finite moments take no part in a block's scale and become NaN codes.
//
// One pass over the tensors, HBM bound (45 million bf16 parameters: fp32 states
// 192 us, 5.2 TB/s; 8-bit states 88 us, 5.1 TB/s).  Tensor descriptors travel as
// kernel arguments, as many as 4 KiB hold per launch: whole ones (Batch), or for a
// state in flat buffers the parameters' and gradients' addresses (Flat).
#include "nf4.h"
#include "ops_common.h"

namespace nf4 {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kRun = kAdamRun;   // elements per workgroup, 8 a thread
static_assert(kRun == kThreads * 8, "8 elements a thread");

// A workgroup's tensor and its place there.
struct Place {
  uint64_t p, g, m, v, ms, vs;   // addresses
  int64_t n, base;               // elements of the tensor, first one of the workgroup
  uint32_t number;               // of the tensor in the caller's list
  // (through a global pointer, or the compiler takes the address for any kind of memory's)
  template <typename T>
  static __device__ __forceinline__ T *at(uint64_t a) {
    typedef __attribute__((address_space(1))) T global_t;
    return (T *)(global_t *)a;
  }
};

// A launch's tensors, in under 4 KiB of kernel arguments: each address is an
// offset from the launch's base for it, in 16-byte units (scales: 4-byte units).
// 448 adapters take 4 launches (7 with whole addresses; each costs its ramp and
// its tail, about 5 us: seven took 99 us, four 92).
template <bool BITS8>
struct Batch {
  static constexpr int kAddresses = BITS8 ? 6 : 4;       // p, g, m, v (ms, vs)
  static constexpr int kMost = BITS8 ? 120 : 156;
  uint64_t base[kAddresses];
  int32_t off[kAddresses][kMost];
  uint32_t n_low[kMost];
  uint32_t end[kMost];           // workgroups of tensors 0 .. i
  uint8_t n_high[kMost];
  int32_t count;
  uint32_t first;                // the number of tensor 0 in the caller's list

  static constexpr int unit(int a) { return a < 4 ? 16 : 4; }
  __device__ __forceinline__ uint64_t at(int a, int i) const { return base[a] + (int64_t)off[a][i] * unit(a); }
  __device__ __forceinline__ Place place(uint32_t group) const {
    // the tensors that end at or before this workgroup, counted by a wave at once
    int t = 0;
#pragma unroll
    for (int k = 0; k < kMost; k += 64) {
      const int l = k + (int)(threadIdx.x & 63);
      t += __popcll(__ballot(l < count - 1 && end[l < kMost ? l : 0] <= group));
    }
    t = __builtin_amdgcn_readfirstlane(t);
    Place w;
    w.p = at(0, t);
    w.g = at(1, t);
    w.m = at(2, t);
    w.v = at(3, t);
    w.ms = BITS8 ? at(kAddresses - 2, t) : 0;
    w.vs = BITS8 ? at(kAddresses - 1, t) : 0;
    w.n = (int64_t)n_low[t] | ((int64_t)n_high[t] << 32);
    w.base = (int64_t)(group - (t ? end[t - 1] : 0u)) * kRun;
    w.number = first + (uint32_t)t;
    return w;
  }

  // Takes `t` as the next tensor; false if an address is too far from the first one's.
  bool add(const AdamTensor &t, uint32_t ends) {
    const uint64_t all[6] = {(uint64_t)t.p, (uint64_t)t.g, (uint64_t)t.m, (uint64_t)t.v, (uint64_t)t.ms, (uint64_t)t.vs};
    for (int a = 0; a < kAddresses; ++a) {
      if (count == 0) base[a] = t.n ? all[a] : 0;
      const int64_t d = t.n ? (int64_t)(all[a] - base[a]) / unit(a) : 0;   // (addresses are multiples: checked)
      if (d != (int32_t)d) return false;
      off[a][count] = (int32_t)d;
    }
    n_low[count] = (uint32_t)t.n;
    n_high[count] = (uint8_t)((uint64_t)t.n >> 32);
    end[count++] = ends;
    return true;
  }
};

// The same for a state in flat buffers: where its tensors lie is in its owner's
// layout, and a launch carries two offsets a tensor.  One launch then takes 448
// adapters, and a workgroup finds its tensor by two scalar loads where a Batch is
// searched (bf16 parameters, 8-bit states, a Batch and a Flat in turn: 40 million
// in 448 tensors 102 and 80 us a step, 20 million in 448 60 and 40, 45 million in 7
// 89 and 88; 65 norms 7 either way, the host's time).
template <bool BITS8>
struct Flat {
  static constexpr int kMost = 480;
  uint64_t base[2];              // of p, of g
  int32_t off[2][kMost];         // 16-byte units
  uint64_t m, v, ms, vs;
  const uint32_t *tensor_of;     // by workgroup of the whole list
  const AdamEntry *entries;
  int32_t count;
  uint32_t first, first_group;   // the launch's first tensor and workgroup

  __device__ __forceinline__ Place place(uint32_t group) const {
    // constant memory: scalar loads
    typedef const __attribute__((address_space(4))) uint32_t *numbers_t;
    typedef const __attribute__((address_space(4))) AdamEntry *entries_t;
    group += first_group;
    const uint32_t i = ((numbers_t)(uint64_t)tensor_of)[group];
    const entries_t e = (entries_t)(uint64_t)entries + i;
    const int t = (int)(i - first);
    Place w;
    w.p = base[0] + (int64_t)off[0][t] * 16;
    w.g = base[1] + (int64_t)off[1][t] * 16;
    const int64_t start = e->start;
    w.m = m + (uint64_t)start * (BITS8 ? 1 : 4);
    w.v = v + (uint64_t)start * (BITS8 ? 1 : 4);
    w.ms = BITS8 ? ms + (uint64_t)start / kAdamBlock * 4 : 0;
    w.vs = BITS8 ? vs + (uint64_t)start / kAdamBlock * 4 : 0;
    w.n = e->n;
    w.base = (int64_t)(group - e->first_group) * kRun;
    w.number = i;
    return w;
  }

  bool add(const AdamTensor &t) {
    const uint64_t all[2] = {(uint64_t)t.p, (uint64_t)t.g};
    for (int a = 0; a < 2; ++a) {
      if (count == 0) base[a] = t.n ? all[a] : 0;
      const int64_t d = t.n ? (int64_t)(all[a] - base[a]) / 16 : 0;
      if (d != (int32_t)d) return false;
      off[a][count] = (int32_t)d;
    }
    ++count;
    return true;
  }
};
static_assert(sizeof(Flat<true>) + sizeof(AdamConfig) <= 4096, "kernel arguments");
static_assert(sizeof(Batch<true>) + sizeof(AdamConfig) <= 4096 && sizeof(Batch<false>) + sizeof(AdamConfig) <= 4096,
              "kernel arguments");

__host__ __device__ constexpr uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x983B6369u;
  x = (x ^ (x >> 15)) * 0xC1F49415u;
  return x ^ (x >> 16);
}

// e4m3 code of |n| <= 448 in the top byte, rounded up when the remainder's 20
// bits plus u20 (16 random bits at the top of them) carry.  Times 2^-120 an
// fp32 value has the code's exponent bias: its exponent field and top three
// mantissa bits are the code, and fp32's subnormals fall on e4m3's.  (A value
// that rounding left a few steps above 448 still takes 448's code.)
// SIGNED: a first moment; else a root, whose code is zero only where it is zero.
template <bool SIGNED>
__device__ __forceinline__ uint32_t code_random(float n, uint32_t u20) {
  const uint32_t c = (__float_as_uint(fabsf(n) * 0x1p-120f) + u20) << 4;
  return SIGNED ? (c & 0x7fffffffu) | (__float_as_uint(n) & 0x80000000u) : n > 0.f ? max(c, 0x01000000u) : c;
}

__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x00000703u), hi = __builtin_amdgcn_perm(d, c, 0x00000703u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
// Maximum over 32 lanes.
__device__ __forceinline__ uint32_t umax32(uint32_t v) {
  v = max(v, dpp_u<kXor1>(v));
  v = max(v, dpp_u<kXor2>(v));
  v = max(v, dpp_u<kHalfMirror>(v));
  v = max(v, dpp_u<kMirror>(v));
  return max(v, (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401F));
}

// Eight states of a block of 256 held by 32 lanes: codes and the block's scale.
// u[k]: 16 random bits in bits 4 .. 19.
template <bool SIGNED>
__device__ __forceinline__ uint2 encode_state(const float x[8], const uint32_t u[8], float &scale) {
  // magnitudes compared as integers: infinities and NaNs come out on top
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
  top = umax32(top);
  float factor;
  uint32_t c[8];
  if (top < 0x7f800000u) {
    block_scale(__uint_as_float(top), kE4M3Max, scale, factor);
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = code_random<SIGNED>(x[k] * factor, u[k]);
  } else {   // the finite values' scale; the others become NaN codes
    top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t a = __float_as_uint(x[k]) & 0x7fffffffu;
      top = max(top, a < 0x7f800000u ? a : 0u);
    }
    top = umax32(top);
    block_scale(__uint_as_float(top), kE4M3Max, scale, factor);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool finite = (__float_as_uint(x[k]) & 0x7fffffffu) < 0x7f800000u;
      c[k] = finite ? code_random<SIGNED>(x[k] * factor, u[k]) : 0x7f000000u;
    }
  }
  return make_uint2(top_bytes(c[0], c[1], c[2], c[3]), top_bytes(c[4], c[5], c[6], c[7]));
}

// Square roots, off by half a step but for a few values in 2^23: one Newton step
// on the remainder, s + (v - s s) q / 2 with s = v q and q the hardware's
// reciprocal root, rounds wrongly only where q itself is off (by one step: 1 to 3
// of the 2^23 significands, then by one step of the root).  Where the root's
// square or its remainder could leave fp32 the library's function takes over.
__device__ __forceinline__ void roots8(const float v[8], float r[8]) {
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    lo = fminf(lo, v[k]);
    hi = fmaxf(hi, v[k]);
  }
  if (lo >= 0x1p-96f && hi <= 0x1p+126f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float q = __builtin_amdgcn_rsqf(v[k]);
      const float s = v[k] * q;
      r[k] = __builtin_fmaf(__builtin_fmaf(-s, s, v[k]), 0.5f * q, s);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = sqrtf(v[k]);
  }
}

template <int SEL>
__device__ __forceinline__ float decode1(uint32_t w) { return __builtin_amdgcn_cvt_f32_fp8((int)w, SEL); }

__device__ __forceinline__ void decode8(uint2 c, float scale, float v[8]) {
  v[0] = decode1<0>(c.x) * scale;
  v[1] = decode1<1>(c.x) * scale;
  v[2] = decode1<2>(c.x) * scale;
  v[3] = decode1<3>(c.x) * scale;
  v[4] = decode1<0>(c.y) * scale;
  v[5] = decode1<1>(c.y) * scale;
  v[6] = decode1<2>(c.y) * scale;
  v[7] = decode1<3>(c.y) * scale;
}

// Writes elements i .. i+7 of a tensor of n.
template <typename T>
__device__ __forceinline__ void give8(T *t, int64_t i, int64_t n, const float v[8]) {
  if (i + 8 <= n) {
    store8(t + i, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) store1(t + i + k, v[k]);
  }
}

// The two moments of eight elements.
template <bool BITS8>
struct State;
template <>
struct State<true> {
  uint2 mc, vc;
  float ms, vs;
  template <bool WHOLE>
  __device__ __forceinline__ void load(const Place &w, int64_t i) {
    mc = *reinterpret_cast<const uint2 *>(Place::at<const uint8_t>(w.m) + i);
    vc = *reinterpret_cast<const uint2 *>(Place::at<const uint8_t>(w.v) + i);
    ms = Place::at<const float>(w.ms)[i / kAdamBlock];
    vs = Place::at<const float>(w.vs)[i / kAdamBlock];
  }
  __device__ __forceinline__ void values(float m[8], float v[8]) const {
    decode8(mc, ms, m);
    decode8(vc, vs, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= v[k];
  }
  static __device__ __forceinline__ void store(const Place &w, int64_t i, const float m[8], const float[8],
                                               const float root[8], uint32_t key) {
    uint32_t um[8], uv[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t h = mix((uint32_t)i + k + key);
      um[k] = (h << 4) & 0xffff0u;
      uv[k] = (h >> 12) & 0xffff0u;
    }
    float sm, sv;
    *reinterpret_cast<uint2 *>(Place::at<uint8_t>(w.m) + i) = encode_state<true>(m, um, sm);
    *reinterpret_cast<uint2 *>(Place::at<uint8_t>(w.v) + i) = encode_state<false>(root, uv, sv);
    if ((threadIdx.x & 31) == 0) {
      Place::at<float>(w.ms)[i / kAdamBlock] = sm;
      Place::at<float>(w.vs)[i / kAdamBlock] = sv;
    }
  }
};
template <>
struct State<false> {
  Part<float> mp, vp;
  template <bool WHOLE>
  __device__ __forceinline__ void load(const Place &w, int64_t i) {
    const float *const ma = Place::at<const float>(w.m), *const va = Place::at<const float>(w.v);
    if (WHOLE) {
      mp.template whole<true>(ma + i);
      vp.template whole<true>(va + i);
    } else {
      mp.some(ma, i, w.n);
      vp.some(va, i, w.n);
    }
  }
  __device__ __forceinline__ void values(float m[8], float v[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m[k] = mp.get(k);
      v[k] = vp.get(k);
    }
  }
  static __device__ __forceinline__ void store(const Place &w, int64_t i, const float m[8], const float v[8],
                                               const float[8], uint32_t) {
    give8(Place::at<float>(w.m), i, w.n, m);
    give8(Place::at<float>(w.v), i, w.n, v);
  }
};

// A workgroup takes 2048 elements of one tensor, thread t elements 8t .. 8t+7, all
// loads first.  States of an 8-bit tensor are padded to whole blocks by their
// owner, so their 8-byte accesses need no tail; p, g and fp32 states end at n.
// (Two or more such parts a thread were slower: 448 adapters in 7 launches 99,
// 117, 133 us with 1, 2, 4.)
template <typename P, typename G, bool BITS8, typename B>
__global__ __launch_bounds__(kThreads) void adamw_kernel(B b, AdamConfig cfg) {
  const Place w = b.place(blockIdx.x);
  const int64_t i = w.base + threadIdx.x * 8, n = w.n;
  // a block of 256 is 32 lanes: they leave together
  if ((i & ~(int64_t)(kAdamBlock - 1)) >= n) return;
  Part<P> pp;
  Part<G> gp;
  State<BITS8> state;
  P *const pa = Place::at<P>(w.p);
  const G *const ga = Place::at<const G>(w.g);
  if (i + 8 <= n) {
    pp.template whole<true>(pa + i);
    gp.template whole<true>(ga + i);
    state.template load<true>(w, i);
  } else {
    pp.some(pa, i, n);
    gp.some(ga, i, n);
    state.template load<false>(w, i);
  }
  const float gs = cfg.grad_scale ? *cfg.grad_scale : 1.f;
  uint32_t key = 0;
  if (BITS8) {
    // a workgroup's elements share the high half of their index
    key = mix(w.number + cfg.seed);
    const uint32_t high = (uint32_t)((uint64_t)w.base >> 32);
    if (high) key = mix(key + high * 0x11D5D725u);
  }
  float p[8], m[8], v[8], root[8];
  state.values(m, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float g = gp.get(k) * gs;
    m[k] = cfg.beta1 * m[k] + cfg.c1 * g;
    v[k] = cfg.beta2 * v[k] + cfg.c2 * (g * g);
  }
  roots8(v, root);
  // the quotient by the hardware's reciprocal: a step of 2^-23 beside the
  // parameter's own rounding
#pragma unroll
  for (int k = 0; k < 8; ++k)
    p[k] = pp.get(k) * cfg.decay - cfg.step * (m[k] * __builtin_amdgcn_rcpf(root[k] * cfg.rbc2 + cfg.eps));
  give8(pa, i, n, p);
  State<BITS8>::store(w, i, m, v, root, key);
}

constexpr int64_t kMostGroups = ((int64_t)1 << 24) - 1;   // of a launch: fewer than 2^32 threads
static_assert(NF4_ADAM_MAX_NUMEL / kRun <= kMostGroups, "a single tensor fits");

template <bool BITS8, typename B>
hipError_t launch_one(const B &b, int64_t groups, bool p_bf16, bool g_bf16, const AdamConfig &cfg, hipStream_t stream) {
  const dim3 grid((unsigned)groups), blk(kThreads);
  if (p_bf16 && g_bf16) hipLaunchKernelGGL((adamw_kernel<uint16_t, uint16_t, BITS8, B>), grid, blk, 0, stream, b, cfg);
  else if (p_bf16) hipLaunchKernelGGL((adamw_kernel<uint16_t, float, BITS8, B>), grid, blk, 0, stream, b, cfg);
  else if (g_bf16) hipLaunchKernelGGL((adamw_kernel<float, uint16_t, BITS8, B>), grid, blk, 0, stream, b, cfg);
  else hipLaunchKernelGGL((adamw_kernel<float, float, BITS8, B>), grid, blk, 0, stream, b, cfg);
  return hipGetLastError();
}

template <bool BITS8>
hipError_t run_flat(const AdamTensor *tensors, int64_t count, bool p_bf16, bool g_bf16, const AdamConfig &cfg,
                    const void *layout, int64_t all_groups, hipStream_t stream) {
  int64_t at = 0, done = 0;
  while (at < count && tensors[at].n == 0) ++at;
  if (at == count) return hipSuccess;
  const AdamTensor &start = tensors[at];
  while (at < count) {
    Flat<BITS8> b;
    b.count = 0;
    b.first = (uint32_t)at;
    b.first_group = (uint32_t)done;
    b.m = (uint64_t)start.m;
    b.v = (uint64_t)start.v;
    b.ms = (uint64_t)start.ms;
    b.vs = (uint64_t)start.vs;
    b.tensor_of = static_cast<const uint32_t *>(layout);
    b.entries = reinterpret_cast<const AdamEntry *>(b.tensor_of + round_up(all_groups, 2));
    int64_t groups = 0;
    for (; at < count && b.count < Flat<BITS8>::kMost; ++at) {
      if (tensors[at].n == 0 && b.count == 0) {   // as in run_batches
        b.first = (uint32_t)(at + 1);
        continue;
      }
      const int64_t c = (tensors[at].n + kRun - 1) / kRun;
      if (groups + c > kMostGroups || !b.add(tensors[at])) break;
      groups += c;
    }
    if (!groups) continue;
    done += groups;
    const hipError_t e = launch_one<BITS8>(b, groups, p_bf16, g_bf16, cfg, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool BITS8>
hipError_t run_batches(const AdamTensor *tensors, int64_t count, bool p_bf16, bool g_bf16, const AdamConfig &cfg,
                       hipStream_t stream) {
  int64_t at = 0;
  while (at < count) {
    Batch<BITS8> b;
    b.count = 0;
    b.first = (uint32_t)at;
    int64_t groups = 0;
    for (; at < count && b.count < Batch<BITS8>::kMost; ++at) {
      // an empty tensor opens no batch (it has no addresses to measure from) but keeps its number in one
      if (tensors[at].n == 0 && b.count == 0) {
        b.first = (uint32_t)(at + 1);
        continue;
      }
      const int64_t c = (tensors[at].n + kRun - 1) / kRun;
      if (groups + c > kMostGroups || !b.add(tensors[at], (uint32_t)(groups + c))) break;
      groups += c;
    }
    if (!groups) continue;   // the rest was empty
    const hipError_t e = launch_one<BITS8>(b, groups, p_bf16, g_bf16, cfg, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_adamw(const AdamTensor *tensors, int64_t count, bool p_bf16, bool g_bf16, bool bits8,
                        const AdamConfig &cfg, const void *layout, int64_t groups, hipStream_t stream) {
  if (layout)
    return bits8 ? run_flat<true>(tensors, count, p_bf16, g_bf16, cfg, layout, groups, stream)
                 : run_flat<false>(tensors, count, p_bf16, g_bf16, cfg, layout, groups, stream);
  return bits8 ? run_batches<true>(tensors, count, p_bf16, g_bf16, cfg, stream)
               : run_batches<false>(tensors, count, p_bf16, g_bf16, cfg, stream);
}

}  // namespace nf4
