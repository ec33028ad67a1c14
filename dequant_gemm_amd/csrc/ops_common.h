// ops_common.h -- device helpers and host launchers of the operators around the
// quantized linear layers: the RMS norm, the 8-bit block-scaled product and the
// AdamW step.  All arguments are validated by the caller (nf4_api.hip);
// launchers only configure grids and enqueue on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4 {

constexpr int kFp8Block = 128;            // values per scale along a row of an 8-bit tensor
constexpr float kE4M3Max = 448.f;
constexpr float kE5M2Max = 57344.f;
// A block whose largest magnitude is below this is held as zeros: the quotient
// max / magnitude would leave fp32.
constexpr float kSmallestAmax = 7.888609052210118e-31f;   // 2^-100
constexpr int kAdamBlock = 256;           // values per scale of an 8-bit optimizer state

__host__ __device__ constexpr int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// ------------------------------------------------------------------ values of either dtype

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = to_bf16(v); }

// The value as it will be read back from memory of type T.
template <typename T>
__device__ __forceinline__ float rounded(float v) {
  if (sizeof(T) == 2) return __uint_as_float((uint32_t)to_bf16(v) << 16);
  return v;
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  return (uint32_t)to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16);
}

// Eight consecutive values from a 16-byte aligned address.
__device__ __forceinline__ void load8(const float *p, float v[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t *p, float v[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float *p, const float v[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t *p, const float v[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]),
                                             pack2_bf16(v[6], v[7]));
}

// The same from any address of the type (the hardware takes 16-byte accesses at
// any alignment; the type tells the compiler not to count on 16).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void load8_any(const float *p, float v[8]) {
  const f32x4_any a = reinterpret_cast<const f32x4_any *>(p)[0], b = reinterpret_cast<const f32x4_any *>(p)[1];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = a[k];
    v[4 + k] = b[k];
  }
}
__device__ __forceinline__ void load8_any(const uint16_t *p, float v[8]) {
  const u32x4_any a = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(a[k] << 16);
    v[2 * k + 1] = __uint_as_float(a[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8_any(float *p, const float v[8]) {
  reinterpret_cast<f32x4_any *>(p)[0] = f32x4_any{v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4_any *>(p)[1] = f32x4_any{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8_any(uint16_t *p, const float v[8]) {
  *reinterpret_cast<u32x4_any *>(p) = u32x4_any{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]),
                                                pack2_bf16(v[6], v[7])};
}

// Values i .. i+7 of a row of n (zeros past n); VEC: the row starts 16-byte
// aligned and n is a multiple of 8.
template <bool VEC, typename T>
__device__ __forceinline__ void load_part(const T *row, int64_t i, int64_t n, float v[8]) {
  if (VEC) {
    if (i < n) {
      load8(row + i, v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.f;
    }
  } else if (i + 8 <= n) {
    load8_any(row + i, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + k < n ? load1(row + i + k) : 0.f;
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_part(T *row, int64_t i, int64_t n, const float v[8]) {
  if (VEC) {
    if (i < n) store8(row + i, v);
  } else if (i + 8 <= n) {
    store8_any(row + i, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) store1(row + i + k, v[k]);
  }
}
template <bool VEC>
__device__ __forceinline__ void load_part(const void *row, bool is_bf16, int64_t i, int64_t n, float v[8]) {
  if (is_bf16)
    load_part<VEC>(reinterpret_cast<const uint16_t *>(row), i, n, v);
  else
    load_part<VEC>(reinterpret_cast<const float *>(row), i, n, v);
}

// Eight consecutive values as they lie in memory, widened when used: a bf16 part
// waits in half the registers.
template <typename T>
struct Part;
template <>
struct Part<uint16_t> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int k) const {
    return __uint_as_float((k & 1) ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  // all eight from p; VEC: 16-byte aligned
  template <bool VEC>
  __device__ __forceinline__ void whole(const uint16_t *p) {
    const u32x4_any a = VEC ? __builtin_bit_cast(u32x4_any, *reinterpret_cast<const uint4 *>(p))
                            : *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = a[k];
  }
  // values i .. i+7 of a row of n, zeros past n; loaded without branches (the last value in their place)
  __device__ __forceinline__ void some(const uint16_t *row, int64_t i, int64_t n) {
    uint16_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = row[i + k < n ? i + k : n - 1];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (i + 2 * k < n ? (uint32_t)e[2 * k] : 0u) | (i + 2 * k + 1 < n ? (uint32_t)e[2 * k + 1] << 16 : 0u);
  }
  // values i .. i+7 of a row of n (zeros past n), as load_part
  template <bool VEC>
  __device__ __forceinline__ void load(const uint16_t *row, int64_t i, int64_t n) {
    if (VEC ? i < n : i + 8 <= n) {
      whole<VEC>(row + i);
    } else {
      zero();
      if (!VEC) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i + k < n) w[k >> 1] |= (uint32_t)row[i + k] << (16 * (k & 1));
      }
    }
  }
};
template <>
struct Part<float> {
  float v[8];
  __device__ __forceinline__ float get(int k) const { return v[k]; }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
  }
  template <bool VEC>
  __device__ __forceinline__ void whole(const float *p) {
    if (VEC) load8(p, v);
    else load8_any(p, v);
  }
  __device__ __forceinline__ void some(const float *row, int64_t i, int64_t n) {
    float e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = row[i + k < n ? i + k : n - 1];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + k < n ? e[k] : 0.f;
  }
  template <bool VEC>
  __device__ __forceinline__ void load(const float *row, int64_t i, int64_t n) { load_part<VEC>(row, i, n, v); }
};

// ------------------------------------------------------------------ reductions

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// lane ^ 1, lane ^ 2, then mirrors of 8 and of 16: every lane of 16 has the result
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// The maximum of finite or infinite magnitudes (fmaxf drops a NaN).
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, dpp<kXor1>(v));
  v = fmaxf(v, dpp<kXor2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  return fmaxf(v, dpp<kMirror>(v));
}
__device__ __forceinline__ float swap16(float v) {   // lane ^ 16
  return __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F));
}
__device__ __forceinline__ float max32(float v) {
  v = max16(v);
  return fmaxf(v, swap16(v));
}
__device__ __forceinline__ float max64(float v) {
  v = max32(v);
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum64(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  v += swap16(v);
  return v + __shfl_xor(v, 32);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true),
                 hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum64(double v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// ------------------------------------------------------------------ 8-bit codes

// Eight values to e4m3 (E5M2 false) or e5m2 codes, each rounded to nearest-even
// by the conversion instruction; |v| must not exceed the format's largest value
// by more than its last rounding (a NaN gives the NaN code).
template <bool E5M2>
__device__ __forceinline__ uint2 codes8(const float v[8]) {
  int a = 0, b = 0;
  if (E5M2) {
    a = __builtin_amdgcn_cvt_pk_bf8_f32(v[0], v[1], a, false);
    a = __builtin_amdgcn_cvt_pk_bf8_f32(v[2], v[3], a, true);
    b = __builtin_amdgcn_cvt_pk_bf8_f32(v[4], v[5], b, false);
    b = __builtin_amdgcn_cvt_pk_bf8_f32(v[6], v[7], b, true);
  } else {
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], a, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
  }
  return make_uint2((uint32_t)a, (uint32_t)b);
}

// Scale and its inverse factor for a block of largest magnitude `amax`:
// fp32(amax fp32(1 / top)) and fp32(fp32(1 / amax) top).  An infinite amax gives
// scale inf and factor 0: the infinity codes NaN (0 * inf) and every value of
// the block reads back as NaN.
__device__ __forceinline__ void block_scale(float amax, float top, float &scale, float &factor) {
  const bool keep = amax >= kSmallestAmax;
  scale = keep ? amax * (1.f / top) : 0.f;
  factor = keep ? (1.f / amax) * top : 0.f;
}

__device__ __forceinline__ float amax8(const float v[8]) {
  float a = fmaxf(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int k = 2; k < 8; ++k) a = fmaxf(a, fabsf(v[k]));
  return a;
}

// ------------------------------------------------------------------ launchers

// A grid for `n` workgroups of up to 1024 threads numbered by group_number(): a
// launch holds fewer than 2^32 threads along x, which many short rows or small
// tiles would pass.  Workgroups past n leave at once.
inline dim3 grid_of(int64_t n) {
  constexpr int64_t kX = (int64_t)1 << 21;
  return n <= kX ? dim3((unsigned)n) : dim3((unsigned)kX, (unsigned)((n + kX - 1) / kX));
}
__device__ __forceinline__ int64_t group_number() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

struct RowsIn {          // a matrix whose rows are contiguous
  const void *p;
  int64_t ld;            // elements between rows
};

struct Fp8Out {
  uint8_t *data;         // rows x pitch
  float *scale;          // scale rows x spitch
  int64_t pitch;
  int64_t spitch;
};

// y (y_bf16) or, with q.data set, 8-bit codes; h is written when res.p is set.
hipError_t launch_rmsnorm_fwd(RowsIn x, bool x_bf16, RowsIn res, const void *w, bool w_bf16, int64_t rows,
                              int64_t cols, float eps, void *h, void *y, bool y_bf16, Fp8Out q, float *rstd,
                              hipStream_t stream);

int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols);   // rows of the fp32 workspace (one partial dw each)
hipError_t launch_rmsnorm_bwd(RowsIn dy, bool dy_bf16, RowsIn h, bool h_bf16, const void *w, bool w_bf16,
                              const float *rstd, RowsIn dh, int64_t rows, int64_t cols, void *dx, void *dw,
                              float *partial, hipStream_t stream);

hipError_t launch_fp8_quantize(RowsIn x, bool x_bf16, int64_t rows, int64_t cols, int block_rows, bool e5m2,
                               Fp8Out q, hipStream_t stream);

struct Fp8In {
  const uint8_t *data;
  const float *scale;
  int64_t rows;
  int64_t pitch;
  int64_t spitch;
};
bool fp8_matmul_fits(int64_t M, int64_t N);   // whether the grid's sizes hold M x N
hipError_t launch_fp8_matmul(const Fp8In &x, bool x_e5m2, const Fp8In &w, void *y, bool y_bf16, hipStream_t stream);

// One tensor of an AdamW step; scales are set for 8-bit states.
struct AdamTensor {
  void *p;
  const void *g;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
};
struct AdamConfig {
  float beta1, beta2, c1, c2;      // c = 1 - beta
  float eps, decay, step, rbc2;    // 1 - lr wd, lr / bias correction 1, 1 / sqrt(bias correction 2)
  const float *grad_scale;         // device scalar, may be null
  uint32_t seed;
};
constexpr int64_t kAdamRun = 2048;   // elements a workgroup takes
// One tensor's entry of a flat state's layout; the tensor's number for every workgroup
// (uint32, padded to 8 bytes) comes before the entries.
struct AdamEntry {
  int64_t n;
  int64_t start;         // of its state, in elements
  uint32_t first_group;
  uint32_t pad;
};
// `tensors` (host) has `count` entries; layout (device) may be null, else it has
// `groups` workgroup numbers.
hipError_t launch_adamw(const AdamTensor *tensors, int64_t count, bool p_bf16, bool g_bf16, bool bits8,
                        const AdamConfig &cfg, const void *layout, int64_t groups, hipStream_t stream);

}  // namespace nf4
