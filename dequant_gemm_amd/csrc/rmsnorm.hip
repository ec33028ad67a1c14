// rmsnorm.hip -- the root-mean-square norm with the residual's addition, and its gradient.
//
//   h = x + r (fp32, rounded once to the stream's type, so that the backward
//       pass reads the very values the norm saw); h = x without a residual
//   rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
// y leaves in bf16 or fp32, or in e4m3 with one fp32 scale per 128 columns,
// quantized from the fp32 y.  Gradient, with g = dy w:
//   dx = rstd (g - h rstd^2 mean(g h)) + dh,   dw = sum over rows of dy h rstd
// where dh is the gradient that reaches h along the residual stream.
//
// One workgroup holds a row in registers between the sum and the outputs (one
// read of every input); rows wider than the registers re-read the row from
// cache.  HBM bound: 4096 x 4096 with the residual and e4m3 out 20.8 us (5.7
// TB/s), the gradient of 8192 x 8192 with dh 104 us (5.1 TB/s, of the 5.0 that
// a large copy reaches).  Row sums run over the lanes and then the waves in a fixed
// order; dw is summed over the rows a workgroup takes, then over workgroups in
// a fixed order, without atomics.
#include "ops_common.h"

namespace nf4 {
namespace {

// Sum over the workgroup's TPB threads, in every thread; S is float or double.
template <int TPB, typename S>
__device__ __forceinline__ S block_sum(S v, S *lds) {
  v = sum64(v);
  if (TPB == 64) return v;
  const int wave = threadIdx.x >> 6;
  __syncthreads();   // the previous use of lds is over
  if ((threadIdx.x & 63) == 0) lds[wave] = v;
  __syncthreads();
  S s = lds[0];
#pragma unroll
  for (int i = 1; i < TPB / 64; ++i) s += lds[i];
  return s;
}

enum { kOutF32 = 0, kOutBf16 = 1, kOutFp8 = 2 };

// Writes values c .. c+7 of one output row (and their scale).
template <int OUT, bool VEC>
__device__ __forceinline__ void put_y(const float y[8], int64_t row, int64_t c, int64_t cols, void *yout,
                                      const Fp8Out &q) {
  if (OUT == kOutF32) store_part<VEC>(reinterpret_cast<float *>(yout) + row * cols, c, cols, y);
  if (OUT == kOutBf16) store_part<VEC>(reinterpret_cast<uint16_t *>(yout) + row * cols, c, cols, y);
  if (OUT == kOutFp8) {
    // 16 lanes hold the 128 columns of a scale
    const float amax = max16(amax8(y));
    float scale, factor, n[8];
    block_scale(amax, kE4M3Max, scale, factor);
#pragma unroll
    for (int k = 0; k < 8; ++k) n[k] = y[k] * factor;
    if (c < q.pitch) *reinterpret_cast<uint2 *>(q.data + row * q.pitch + c) = codes8<false>(n);
    if ((threadIdx.x & 15) == 0 && c / kFp8Block < q.spitch) q.scale[row * q.spitch + c / kFp8Block] = scale;
  }
}

// One row per workgroup; thread t holds columns 8(t + TPB j) .. +7, j < VPT.
// VPT == 0: any width, the row read twice.
template <int TPB, int VPT, typename T, int OUT, bool VEC>
__global__ __launch_bounds__(TPB) void rmsnorm_fwd_kernel(RowsIn x, RowsIn res, const void *w, bool w_bf16,
                                                          int64_t rows, int64_t cols, double inv_cols, float eps,
                                                          T *__restrict__ h, void *__restrict__ y, Fp8Out q,
                                                          float *__restrict__ rstd) {
  __shared__ double lds[TPB / 64];
  const int64_t row = group_number();
  if (row >= rows) return;
  const T *xr = reinterpret_cast<const T *>(x.p) + row * x.ld;
  const T *rr = res.p ? reinterpret_cast<const T *>(res.p) + row * res.ld : nullptr;
  T *hr = h + row * cols;
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  constexpr int64_t STEP = (int64_t)TPB * 8;
  float v[VPT ? VPT : 1][8];
  float sum = 0.f;

  auto take = [&](int64_t c, float e[8]) {
    load_part<VEC>(xr, c, cols, e);
    if (rr) {
      float r[8];
      load_part<VEC>(rr, c, cols, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = rounded<T>(e[k] + r[k]);
      store_part<VEC>(hr, c, cols, e);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += e[k] * e[k];
  };
  if (VPT) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) take(c0 + j * STEP, v[j]);
  } else {
    for (int64_t c = c0; c < cols; c += STEP) take(c, v[0]);
  }
  // A row's scalar: one rounding, where the sum over lanes, the mean, the root and the quotient in fp32 would
  // be ten (the root mean square of its error 0.30 of a step, and 0.5 to 0.6; e4m3 codes near a tie fall by it).
  const float rs = (float)rsqrt(block_sum<TPB>((double)sum, lds) * inv_cols + (double)eps);
  if (threadIdx.x == 0) rstd[row] = rs;

  auto give = [&](int64_t c, const float e[8]) {
    float g[8], o[8];
    load_part<VEC>(w, w_bf16, c, cols, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = e[k] * rs * g[k];
    if (OUT == kOutFp8 && c + 8 > cols) {   // the padding is zeros, also of a row whose rs is not finite
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = c + k < cols ? o[k] : 0.f;
    }
    put_y<OUT, VEC>(o, row, c, cols, y, q);
  };
  if (VPT) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) give(c0 + j * STEP, v[j]);
  } else {
    // columns past the row's end matter for the padded codes and scales; a
    // workgroup's threads leave together, so that the 16-lane maxima are whole
    const int64_t end = OUT == kOutFp8 ? q.spitch * kFp8Block : cols;
    for (int64_t c = c0; c - c0 < end; c += STEP) {
      float e[8];
      load_part<VEC>(rr ? (const T *)hr : xr, c, cols, e);   // this thread's own stores
      give(c, e);
    }
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; partial [gridDim.x][cols] gets
// each workgroup's share of dw.  Thread t holds columns 8(t + TPB j) .. +7, j < VPT.
template <int TPB, int VPT, typename D, typename T, typename W, bool VEC>
__global__ __launch_bounds__(TPB) void rmsnorm_bwd_kernel(RowsIn dy, RowsIn h, const W *__restrict__ w,
                                                          const float *__restrict__ rstd, RowsIn dh, int64_t rows,
                                                          int64_t cols, T *__restrict__ dx,
                                                          float *__restrict__ partial) {
  __shared__ float lds[TPB / 64];
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  constexpr int64_t STEP = (int64_t)TPB * 8;
  Part<W> wv[VPT];
  float acc[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    wv[j].template load<VEC>(w, c0 + j * STEP, cols);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[j][k] = 0.f;
  }
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const D *dr = reinterpret_cast<const D *>(dy.p) + row * dy.ld;
    const T *hr = reinterpret_cast<const T *>(h.p) + row * h.ld;
    const T *er = dh.p ? reinterpret_cast<const T *>(dh.p) + row * dh.ld : nullptr;
    const float rs = rstd[row];
    Part<D> a[VPT];
    Part<T> b[VPT], e[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t c = c0 + j * STEP;
      a[j].template load<VEC>(dr, c, cols);
      b[j].template load<VEC>(hr, c, cols);
      if (er) e[j].template load<VEC>(er, c, cols);
      else e[j].zero();
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += a[j].get(k) * wv[j].get(k) * b[j].get(k);
    sum = block_sum<TPB>(sum, lds);
    const float mean = rs * rs * (sum / (float)cols);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = a[j].get(k), x = b[j].get(k);
        o[k] = rs * (d * wv[j].get(k) - x * mean) + e[j].get(k);
        acc[j][k] += d * x * rs;
      }
      store_part<VEC>(dx + row * cols, c0 + j * STEP, cols, o);
    }
  }
  float *prow = partial + (int64_t)blockIdx.x * cols;
#pragma unroll
  for (int j = 0; j < VPT; ++j) store_part<VEC>(prow, c0 + j * STEP, cols, acc[j]);
}

// The same for rows wider than the registers: each row read twice, dw summed in
// `partial` (a thread's own columns).
template <int TPB, typename D, typename T, typename W, bool VEC>
__global__ __launch_bounds__(TPB) void rmsnorm_bwd_wide_kernel(RowsIn dy, RowsIn h, const W *__restrict__ w,
                                                               const float *__restrict__ rstd, RowsIn dh, int64_t rows,
                                                               int64_t cols, T *__restrict__ dx,
                                                               float *__restrict__ partial) {
  __shared__ float lds[TPB / 64];
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  constexpr int64_t STEP = (int64_t)TPB * 8;
  float *prow = partial + (int64_t)blockIdx.x * cols;
  bool first = true;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const D *dr = reinterpret_cast<const D *>(dy.p) + row * dy.ld;
    const T *hr = reinterpret_cast<const T *>(h.p) + row * h.ld;
    const T *er = dh.p ? reinterpret_cast<const T *>(dh.p) + row * dh.ld : nullptr;
    const float rs = rstd[row];
    float sum = 0.f;
    for (int64_t c = c0; c < cols; c += STEP) {
      float a[8], b[8], g[8];
      load_part<VEC>(dr, c, cols, a);
      load_part<VEC>(hr, c, cols, b);
      load_part<VEC>(w, c, cols, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += a[k] * g[k] * b[k];
    }
    sum = block_sum<TPB>(sum, lds);
    const float mean = rs * rs * (sum / (float)cols);
    for (int64_t c = c0; c < cols; c += STEP) {
      float a[8], b[8], g[8], o[8], dw[8];
      load_part<VEC>(dr, c, cols, a);
      load_part<VEC>(hr, c, cols, b);
      load_part<VEC>(w, c, cols, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        o[k] = rs * (a[k] * g[k] - b[k] * mean);
        dw[k] = a[k] * b[k] * rs;
      }
      if (er) {
        load_part<VEC>(er, c, cols, a);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] += a[k];
      }
      store_part<VEC>(dx + row * cols, c, cols, o);
      if (!first) {
        load_part<VEC>(prow, c, cols, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[k] += b[k];
      }
      store_part<VEC>(prow, c, cols, dw);
    }
    first = false;
  }
}

// dw[c] = sum over `groups` rows of partial, in a fixed order: row lane q of 64
// takes rows q, q + 64, ..., then the lanes' sums are added in order.  16
// columns a workgroup: a 64-byte piece of each row, and workgroups enough.  Four
// rows' loads are in flight (with a whole gradient of 30000 x 256, one at a time
// 30.5 us, four 25.0; of 5787 x 1123 29.8 and 27.3; of 1111 x 5001 17.2 and 17.5).
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float *__restrict__ partial, int64_t groups,
                                                          int64_t cols, void *__restrict__ dw, bool w_bf16) {
  __shared__ float lds[64][17];
  const int col = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + col;
  float s = 0.f;
  if (c < cols) {
    int64_t r = q;
    for (; r + 64 * 3 < groups; r += 64 * 4) {   // four loads in flight
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = partial[(r + 64 * i) * cols + c];
#pragma unroll
      for (int i = 0; i < 4; ++i) s += p[i];
    }
    // the last three at most, together as well
    float p[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) p[i] = r + 64 * i < groups ? partial[(r + 64 * i) * cols + c] : 0.f;
#pragma unroll
    for (int i = 0; i < 3; ++i) s += p[i];
  }
  lds[q][col] = s;
  __syncthreads();
  if (q >= 4) return;
  // four lanes of 16 rows each, then their sums (the first wave)
  s = lds[16 * q][col];
#pragma unroll
  for (int i = 1; i < 16; ++i) s += lds[16 * q + i][col];
  s += swap16(s);
  s += __shfl_xor(s, 32);
  if (q || c >= cols) return;
  if (w_bf16)
    reinterpret_cast<uint16_t *>(dw)[c] = to_bf16(s);
  else
    reinterpret_cast<float *>(dw)[c] = s;
}

template <int TPB, int VPT, typename T, int OUT>
void fwd_vec(bool vec, RowsIn x, RowsIn res, const void *w, bool w_bf16, int64_t rows, int64_t cols, float eps,
             void *h, void *y, const Fp8Out &q, float *rstd, hipStream_t s) {
  const dim3 g = grid_of(rows), b(TPB);
  if (vec)
    hipLaunchKernelGGL((rmsnorm_fwd_kernel<TPB, VPT, T, OUT, true>), g, b, 0, s, x, res, w, w_bf16, rows, cols,
                       1.0 / (double)cols, eps, reinterpret_cast<T *>(h), y, q, rstd);
  else
    hipLaunchKernelGGL((rmsnorm_fwd_kernel<TPB, VPT, T, OUT, false>), g, b, 0, s, x, res, w, w_bf16, rows, cols,
                       1.0 / (double)cols, eps, reinterpret_cast<T *>(h), y, q, rstd);
}

template <typename T, int OUT>
void fwd_width(bool vec, RowsIn x, RowsIn res, const void *w, bool w_bf16, int64_t rows, int64_t cols, float eps,
               void *h, void *y, const Fp8Out &q, float *rstd, hipStream_t s) {
  // columns a workgroup has to cover: the row, or the padded codes and scales
  const int64_t n = OUT == kOutFp8 ? q.spitch * kFp8Block : cols;
#define NF4_FWD(TPB, VPT) fwd_vec<TPB, VPT, T, OUT>(vec, x, res, w, w_bf16, rows, cols, eps, h, y, q, rstd, s)
  if (n <= 512) NF4_FWD(64, 1);
  else if (n <= 2048) NF4_FWD(256, 1);
  else if (n <= 4096) NF4_FWD(256, 2);
  else if (n <= 8192) NF4_FWD(512, 2);
  else if (n <= 16384) NF4_FWD(1024, 2);
  else NF4_FWD(1024, 0);
#undef NF4_FWD
}

struct BwdArgs {
  RowsIn dy, h;
  const void *w;
  const float *rstd;
  RowsIn dh;
  int64_t rows, cols;
  void *dx;
  float *partial;
  int64_t groups;
  bool vec;
  hipStream_t stream;
};

// VPT 0: the wide kernel.
template <int TPB, int VPT, typename D, typename T, typename W>
void bwd_launch(const BwdArgs &a) {
  const dim3 g((unsigned)a.groups), b(TPB);
  const W *w = reinterpret_cast<const W *>(a.w);
  T *dx = reinterpret_cast<T *>(a.dx);
#define NF4_BWD(...) \
  hipLaunchKernelGGL((__VA_ARGS__), g, b, 0, a.stream, a.dy, a.h, w, a.rstd, a.dh, a.rows, a.cols, dx, a.partial)
  if constexpr (VPT == 0) {
    if (a.vec) NF4_BWD(rmsnorm_bwd_wide_kernel<TPB, D, T, W, true>);
    else NF4_BWD(rmsnorm_bwd_wide_kernel<TPB, D, T, W, false>);
  } else {
    if (a.vec) NF4_BWD(rmsnorm_bwd_kernel<TPB, VPT, D, T, W, true>);
    else NF4_BWD(rmsnorm_bwd_kernel<TPB, VPT, D, T, W, false>);
  }
#undef NF4_BWD
}

template <typename D, typename T, typename W>
void bwd_width(const BwdArgs &a) {
  if (a.cols <= 512) bwd_launch<64, 1, D, T, W>(a);
  else if (a.cols <= 1024) bwd_launch<128, 1, D, T, W>(a);
  else if (a.cols <= 2048) bwd_launch<256, 1, D, T, W>(a);
  else if (a.cols <= 4096) bwd_launch<512, 1, D, T, W>(a);
  else if (a.cols <= 6144) bwd_launch<768, 1, D, T, W>(a);
  else if (a.cols <= 8192) bwd_launch<1024, 1, D, T, W>(a);
  else if (a.cols <= 16384) bwd_launch<1024, 2, D, T, W>(a);
  else bwd_launch<1024, 0, D, T, W>(a);
}

template <typename D, typename T>
void bwd_w(const BwdArgs &a, bool w_bf16) {
  if (w_bf16) bwd_width<D, T, uint16_t>(a);
  else bwd_width<D, T, float>(a);
}

bool row_vec(const RowsIn &r, bool bf16) { return !r.p || r.ld * (bf16 ? 2 : 4) % 16 == 0; }

}  // namespace

hipError_t launch_rmsnorm_fwd(RowsIn x, bool x_bf16, RowsIn res, const void *w, bool w_bf16, int64_t rows,
                              int64_t cols, float eps, void *h, void *y, bool y_bf16, Fp8Out q, float *rstd,
                              hipStream_t stream) {
  const bool vec = cols % 8 == 0 && row_vec(x, x_bf16) && row_vec(res, x_bf16);
#define NF4_OUT(T, OUT) fwd_width<T, OUT>(vec, x, res, w, w_bf16, rows, cols, eps, h, y, q, rstd, stream)
  if (x_bf16) {
    if (q.data) NF4_OUT(uint16_t, kOutFp8);
    else if (y_bf16) NF4_OUT(uint16_t, kOutBf16);
    else NF4_OUT(uint16_t, kOutF32);
  } else {
    if (q.data) NF4_OUT(float, kOutFp8);
    else if (y_bf16) NF4_OUT(float, kOutBf16);
    else NF4_OUT(float, kOutF32);
  }
#undef NF4_OUT
  return hipGetLastError();
}

// Workgroups, and rows of the workspace: as many as the chip holds at once and
// no more, since each writes a partial dw that is read again, and rows shared
// evenly.  Measured (bf16, with dh): 8192 x 8192 104 us with 256, 107 with 512;
// 4096 x 4096 35.1 with 256, 29.8 with 512, 33.2 with 768; 16384 x 1024 43.1
// with 512, 31.0 with 1024; 30000 x 256 36.7 with 1024, 25.2 with 2048.  Rows
// that are not whole 16-byte parts wait longer for their loads, and many of them
// take twice the workgroups (5787 x 1123 37.9 -> 27.4 us, 8000 x 3001 67.4 ->
// 55.1; 1111 x 5001 and 2000 x 1123 lose by it).
int64_t rmsnorm_bwd_groups(int64_t rows, int64_t cols) {
  int64_t most = cols <= 512 ? 2048 : cols <= 1024 ? 1024 : cols <= 6144 ? 512 : 256;
  if (cols % 8 && cols <= 4096 && rows > 4 * most) most *= 2;
  const int64_t each = (rows + most - 1) / most;
  return each ? (rows + each - 1) / each : 0;
}

hipError_t launch_rmsnorm_bwd(RowsIn dy, bool dy_bf16, RowsIn h, bool h_bf16, const void *w, bool w_bf16,
                              const float *rstd, RowsIn dh, int64_t rows, int64_t cols, void *dx, void *dw,
                              float *partial, hipStream_t stream) {
  const int64_t groups = rmsnorm_bwd_groups(rows, cols);
  const bool vec = cols % 8 == 0 && row_vec(dy, dy_bf16) && row_vec(h, h_bf16) && row_vec(dh, h_bf16);
  if (groups) {
    const BwdArgs a = {dy, h, w, rstd, dh, rows, cols, dx, partial, groups, vec, stream};
    if (dy_bf16 && h_bf16) bwd_w<uint16_t, uint16_t>(a, w_bf16);
    else if (dy_bf16) bwd_w<uint16_t, float>(a, w_bf16);
    else if (h_bf16) bwd_w<float, uint16_t>(a, w_bf16);
    else bwd_w<float, float>(a, w_bf16);
  }
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((unsigned)((cols + 15) / 16)), dim3(1024), 0, stream, partial, groups,
                     cols, dw, w_bf16);
  return hipGetLastError();
}

}  // namespace nf4
