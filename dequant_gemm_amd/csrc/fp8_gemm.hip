// fp8_gemm.hip -- the product of two 8-bit block-scaled matrices:
//
//   Y[m, n] = sum_kb sx[m, kb] sw[n / 128, kb] sum_{k in block kb} X[m, k] W[n, k]
//
// X [M, K] holds activations (e4m3 or e5m2, a scale per row and 128 columns),
// W [N, K] weights (e4m3, a scale per 128 x 128).  One 16x16x128 MFMA forms a
// whole block's sum in fp32 from a zero accumulator; a fused multiply-add with
// the product of the two scales adds it to the fp32 result.  The weight's rows
// are the MFMA's rows and the activations' rows its columns, so that a lane's
// results share one row of X: one scale per lane and block, and four
// consecutive columns of Y.  Both operands take the same order of the 128
// reduction indexes over lanes, so the sum does not depend on which it is.
// (For an fp32 Y four bf16 MFMAs take the block's place, see Frag.)
#include "ops_common.h"

namespace nf4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A lane's part of one block of 16 rows: 32 of its row's 128 codes (two 16-byte
// chunks).  The fp8 matrix cores take the codes as they are, but keep only 13
// bits below the largest of the products they add at once: measured 1.4e-5
// relative error of a block's sum for normal values (each product truncated),
// far below a bf16 output's rounding (2^-9 and more) and far above an fp32
// output's.  An fp32 output therefore takes the codes as bf16 (the conversion is
// exact) and the bf16 matrix cores, which add in full (1e-8 measured).
template <bool E5M2, bool F32OUT>
struct Frag;

template <bool E5M2>
struct Frag<E5M2, false> {
  i32x8 v;
  __device__ __forceinline__ void set(uint4 a, uint4 b) {
    v = i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
  }
};

template <bool E5M2>
struct Frag<E5M2, true> {
  bf16x8 v[4];
  __device__ __forceinline__ bf16x8 eight(uint32_t a, uint32_t b) {
    bf16x2 p[4];
    if (E5M2) {
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, 1.f, false);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, 1.f, true);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, 1.f, false);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, 1.f, true);
    } else {
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
    }
    return __builtin_shufflevector(__builtin_shufflevector(p[0], p[1], 0, 1, 2, 3),
                                   __builtin_shufflevector(p[2], p[3], 0, 1, 2, 3), 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ __forceinline__ void set(uint4 a, uint4 b) {
    v[0] = eight(a.x, a.y);
    v[1] = eight(a.z, a.w);
    v[2] = eight(b.x, b.y);
    v[3] = eight(b.z, b.w);
  }
};

// The block's sums of 16 rows of W by 16 rows of X: lane l has row 4 (l / 16) + k
// of W by row l % 16 of X.
template <bool E5M2>
__device__ __forceinline__ f32x4 block_dot(const Frag<false, false> &w, const Frag<E5M2, false> &x) {
  const f32x4 z = {0.f, 0.f, 0.f, 0.f};
  // operand formats: 0 e4m3, 1 e5m2; no hardware scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, z, 0, E5M2 ? 1 : 0, 0, 0, 0, 0);
}
template <bool E5M2>
__device__ __forceinline__ f32x4 block_dot(const Frag<false, true> &w, const Frag<E5M2, true> &x) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], d, 0, 0, 0);
  return d;
}

// 16 bytes per lane, lane l's to dst + 16 l (zeros past the descriptor's end).
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rs, uint8_t *dst, uint32_t voffset, int soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)dst, 16, voffset, soffset, 0, 0);
}

// 4 bytes per lane, lane l's to dst + 4 l.
__device__ __forceinline__ void load_to_lds4(__amdgpu_buffer_rsrc_t rs, uint8_t *dst, uint32_t voffset, int soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)dst, 4, voffset, soffset, 0, 0);
}

// Columns n .. n+3 of row m; VEC: N is a multiple of 4.
template <bool F32OUT, bool VEC>
__device__ __forceinline__ void put4(void *y, int64_t M, int64_t N, int64_t m, int64_t n, f32x4 v) {
  if (m >= M) return;
  const float e[4] = {v[0], v[1], v[2], v[3]};
  const int64_t at = m * N + n;
  if (VEC) {
    if (n >= N) return;
    if (F32OUT)
      *reinterpret_cast<float4 *>(reinterpret_cast<float *>(y) + at) = make_float4(e[0], e[1], e[2], e[3]);
    else
      *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(y) + at) =
          make_uint2(pack2_bf16(e[0], e[1]), pack2_bf16(e[2], e[3]));
  } else if (n + 4 <= N) {   // at any alignment
    if (F32OUT)
      *reinterpret_cast<f32x4_any *>(reinterpret_cast<float *>(y) + at) = f32x4_any{e[0], e[1], e[2], e[3]};
    else
      *reinterpret_cast<u32x2_any *>(reinterpret_cast<uint16_t *>(y) + at) =
          u32x2_any{pack2_bf16(e[0], e[1]), pack2_bf16(e[2], e[3])};
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < N) {
        if (F32OUT) reinterpret_cast<float *>(y)[at + k] = e[k];
        else reinterpret_cast<uint16_t *>(y)[at + k] = to_bf16(e[k]);
      }
  }
}

// ------------------------------------------------------------------ few rows of X
//
// A workgroup takes NR groups of 16 rows of W and MT groups of 16 rows of X;
// each wave takes a run of K blocks, U at a time with every load of the U blocks
// issued first, and the waves' sums are joined in LDS in a fixed order.  W is
// read once, straight into the MFMA's registers.  Runs, not blocks in turn: the
// waves of a workgroup then start at addresses spread over a row, where 8
// neighbouring blocks share a few memory channels (4096 x 4096, one row of X:
// 5.9 -> 5.0 us).
template <int MT, int NR, int U, int WAVES, bool E5M2, bool F32OUT, bool VEC>
__global__ __launch_bounds__(64 * WAVES) void fp8_small_kernel(Fp8In x, Fp8In w, void *__restrict__ y) {
  __shared__ f32x4 part[WAVES][NR][MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * (16 * NR), m0 = (int64_t)blockIdx.y * (16 * MT);
  if (n0 >= w.rows) return;   // past the last of a grid of several layers
  const int KB = (int)(w.pitch / kFp8Block);
  const uint8_t *wp[NR], *xp[MT];
  const float *sw[NR], *sx[MT];
  // rows past the end repeat the last, never stored
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int64_t n = n0 + 16 * i, nr = n + r < w.rows ? n + r : w.rows - 1;
    wp[i] = w.data + nr * w.pitch + 16 * g;
    sw[i] = w.scale + (n < w.rows ? n : w.rows - 1) / 128 * w.spitch;
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = m0 + 16 * j + r, mr = m < x.rows ? m : x.rows - 1;
    xp[j] = x.data + mr * x.pitch + 16 * g;
    sx[j] = x.scale + mr * x.spitch;
  }
  f32x4 acc[NR][MT];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // blocks of this wave's run; past its end the loads repeat the last and the sums are dropped
  const int run = (KB + WAVES - 1) / WAVES, end = (wave + 1) * run < KB ? (wave + 1) * run : KB;
  for (int kb0 = wave * run; kb0 < end; kb0 += U) {
    uint4 wv[U][NR][2], xv[U][MT][2];
    float s[U][NR], t[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + u < end ? kb0 + u : end - 1;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        wv[u][i][0] = *reinterpret_cast<const uint4 *>(wp[i] + kb * kFp8Block);
        wv[u][i][1] = *reinterpret_cast<const uint4 *>(wp[i] + kb * kFp8Block + 64);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + u < end ? kb0 + u : end - 1;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        xv[u][j][0] = *reinterpret_cast<const uint4 *>(xp[j] + kb * kFp8Block);
        xv[u][j][1] = *reinterpret_cast<const uint4 *>(xp[j] + kb * kFp8Block + 64);
        t[u][j] = sx[j][kb];
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) s[u][i] = sw[i][kb];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u && kb0 + u >= end) break;
      Frag<false, F32OUT> wf[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) wf[i].set(wv[u][i][0], wv[u][i][1]);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        Frag<E5M2, F32OUT> xf;
        xf.set(xv[u][j][0], xv[u][j][1]);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const f32x4 d = block_dot(wf[i], xf);
          const float sc = t[u][j] * s[u][i];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][k] = __builtin_fmaf(d[k], sc, acc[i][j][k]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  static_assert(NR * MT <= WAVES, "a wave per joined tile");
  if (wave >= NR * MT) return;
  const int i = wave / MT, j = wave % MT;
  f32x4 s = part[0][i][j][lane];
#pragma unroll
  for (int q = 1; q < WAVES; ++q) {
    const f32x4 p = part[q][i][j][lane];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] += p[k];
  }
  put4<F32OUT, VEC>(y, x.rows, w.rows, m0 + 16 * j + r, n0 + 16 * i + 4 * g, s);
}

// ------------------------------------------------------------------ tiles
//
// WN x WM waves, each 16 TN rows of W by 16 TM rows of X; K steps of one block.
// With KS > 1 as many such groups of waves share the workgroup's tile: group q
// takes blocks q, q + KS, ... in stages of its own, and the groups' sums are
// added in LDS in their order at the end (few tiles would leave CUs idle).
// Both operands and X's scales reach LDS by buffer-to-LDS loads, in two stages
// of one block.  16-byte chunk c of row r sits at chunk c ^ ((r / 2) & 7) of
// its 128-byte row: the 16 rows that a fragment read takes at once then cover
// all 64 LDS banks.  Rows past the tensors load zeros (the buffer descriptor
// ends at the last row).
//
// A wave goes through its TN rows of tiles; row i's MFMAs run while row i + 1's
// W fragment is read and row i - 1's sums are scaled and added.  Before the
// last row every fragment of the stage is in registers: there the waves meet,
// the refill of the stage with the block after the next begins (a few loads
// beside each row of tiles: all at once they hold up the MFMAs, 1.08x), and the
// next block's first fragments are read behind the last row's MFMAs, each X fragment in the
// registers of the one just used.  So one barrier a step, and no wave waits for
// LDS after it.  There are no branches in a step (a refill past the last block
// repeats it, never read): with one, the compiler sinks the additions past it
// and keeps every block sum of the step in registers.  28672 x 8192 x 8192:
// 2950 -> 1650 us (2.33 PFLOP/s) against the plain two-stage loop on 128 x 128
// tiles, bitwise the same sums; the matrix cores are busy 62% of the cycles at
// a clock that the load holds to 1.55 GHz.  32 x 32 x 64 MFMAs took the same
// time.
template <int WN, int WM, int KS, int TN, int TM, bool E5M2, bool F32OUT, bool VEC>
__global__ __launch_bounds__(64 * WN * WM * KS) __attribute__((amdgpu_waves_per_eu(2)))
void fp8_tile_kernel(Fp8In x, Fp8In w, void *__restrict__ y, int tiles_n, int tiles_m) {
  constexpr int BN = 16 * TN * WN, BM = 16 * TM * WM, NW = WN * WM;
  constexpr int PW = BN / 8 / NW, PX = BM / 8 / NW;   // a wave's 1 KiB pieces (8 rows) of W and of X
  static_assert(BN % (8 * NW) == 0 && BM % (8 * NW) == 0, "whole pieces");
  static_assert(BM % 64 == 0 && BM / 64 < NW, "a wave loads 64 scales of X, another those of W");
  static_assert(TN % 2 == 0, "fragment slots alternate over the rows of tiles");
  constexpr int STAGE = (BN + BM) * 128 + NW * 256;
  __shared__ __attribute__((aligned(1024))) uint8_t stages0[KS * STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t stages1[KS * STAGE];
  const int lane = threadIdx.x & 63, all_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = all_wave % NW, kg = all_wave / NW;   // wave of the K group, K group
  uint8_t *const stage0 = stages0 + kg * STAGE, *const stage1 = stages1 + kg * STAGE;
  const int r = lane & 15, g = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int KB = (int)(w.pitch / kFp8Block), steps = (KB + KS - 1) / KS;

  // workgroups are dealt round-robin to 8 XCDs: each XCD takes a contiguous run
  // of tiles, in columns of 4 tiles of X (28672 x 8192 x 8192: 1630 us; of 2
  // 1694, of 8 1690, of 32 1931)
  const int total = tiles_n * tiles_m;
  int t;
  {
    const int group = (int)group_number();      // (a row of the grid is a multiple of 8 workgroups)
    if (group >= total) return;
    const int q = total / 8, rem = total % 8, xcd = group % 8, idx = group / 8;
    t = xcd * q + (xcd < rem ? xcd : rem) + idx;
  }
  int tn, tm;
  {
    const int band = 4 * tiles_n, b = t / band, in = t - b * band;
    const int h = tiles_m - 4 * b < 4 ? tiles_m - 4 * b : 4;
    tn = in / h;
    tm = 4 * b + in - tn * h;
  }
  const int64_t n0 = (int64_t)tn * BN, m0 = (int64_t)tm * BM;

  // this wave's pieces: tile rows 8 (PW wave + i) + lane / 8 of W, 8 (PX wave + i) + lane / 8 of X
  const int64_t wrow0 = n0 + 8 * PW * wave, xrow0 = m0 + 8 * PX * wave;
  const int64_t wleft = w.rows - wrow0, xleft = x.rows - xrow0;
  uint8_t *const wfrom = const_cast<uint8_t *>(w.data + (wleft > 0 ? wrow0 : 0) * w.pitch);
  uint8_t *const xfrom = const_cast<uint8_t *>(x.data + (xleft > 0 ? xrow0 : 0) * x.pitch);
  // bytes to the last row (a wave's rows span less than 2^31)
  const int wspan = wleft < 0 ? 0 : (int)((wleft < 8 * PW ? wleft : 8 * PW) * w.pitch);
  const int xspan = xleft < 0 ? 0 : (int)((xleft < 8 * PX ? xleft : 8 * PX) * x.pitch);
  uint32_t woff[PW], xoff[PX];
#pragma unroll
  for (int i = 0; i < PW; ++i) {
    const int lr = 8 * i + (lane >> 3), tr = 8 * PW * wave + lr;
    woff[i] = (uint32_t)(lr * (int)w.pitch) + (uint32_t)(((lane & 7) ^ ((tr >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int i = 0; i < PX; ++i) {
    const int lr = 8 * i + (lane >> 3), tr = 8 * PX * wave + lr;
    xoff[i] = (uint32_t)(lr * (int)x.pitch) + (uint32_t)(((lane & 7) ^ ((tr >> 1) & 7)) << 4);
  }
  // wave v < BM / 64 loads the scales of X's rows 64 v + lane, the next one those of W's
  // 128-row blocks (the others zeros, never read)
  const bool sw_wave = wave == BM / 64;
  const int64_t srow0 = sw_wave ? n0 / 128 : m0 + 64 * wave;
  const int64_t srows = sw_wave ? (w.rows + 127) / 128 : (wave < BM / 64 ? x.rows : 0);
  const int64_t sleft = srows > srow0 ? srows - srow0 : 0;
  const int64_t spitch = w.spitch;    // x's too: both have w.pitch / 128 blocks a row
  float *const sfrom = const_cast<float *>((sw_wave ? w.scale : x.scale) + (sleft > 0 ? srow0 : 0) * spitch);
  const int sspan = (int)((sleft < 64 ? sleft : 64) * spitch * 4);
  const uint32_t soff = (uint32_t)(lane * (int)spitch * 4);
  constexpr int LOADS = PW + PX + 1;
  constexpr int PPR = (LOADS + TN - 1) / TN;   // loads issued beside a row of tiles
  // load p (below LOADS) of this K group's step t: block KS t + kg; past the last block zeros
  auto issue1 = [&](uint8_t *st, int t, int p) {
    const int kb = t * KS + kg;
    const bool in = kb < KB;
    if (p < PW) {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(wfrom, (short)0, in ? wspan : 0, 0x00020000);
      load_to_lds(rs, st + (PW * wave + p) * 1024, woff[p < PW ? p : 0], in ? kb * kFp8Block : 0);
    } else if (p < PW + PX) {
      const int i = p - PW;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(xfrom, (short)0, in ? xspan : 0, 0x00020000);
      load_to_lds(rs, st + BN * 128 + (PX * wave + i) * 1024, xoff[i < 0 ? 0 : i], in ? kb * kFp8Block : 0);
    } else {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(sfrom, (short)0, in ? sspan : 0, 0x00020000);
      load_to_lds4(rs, st + (BN + BM) * 128 + wave * 256, soff, in ? kb * 4 : 0);
    }
  };
  auto issue = [&](uint8_t *st, int t, int from, int to) {
#pragma unroll
    for (int p = 0; p < LOADS; ++p)
      if (p >= from && p < to) issue1(st, t, p);
  };

  const int chunk = (g ^ (r >> 1)) << 4;
  const int wbase = (wn * 16 * TN + r) * 128 + chunk;
  const int xbase = (BN + wm * 16 * TM + r) * 128 + chunk;
  const int sbase = (BN + BM) * 128 + (wm * 16 * TM + r) * 4;
  const int swbase = (BN + BM) * 128 + BM * 4 + (wn * 16 * TN / 128) * 4;

  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4 d[2][TM];                     // block sums of a row of tiles, by the row's parity
  Frag<E5M2, F32OUT> xf[TM];
  Frag<false, F32OUT> wf[2];          // by the row's parity
  float s[TM];                        // scale products: of the previous block until its last row is added

  auto read_w = [&](const uint8_t *st, int i) {
    wf[i & 1].set(*reinterpret_cast<const uint4 *>(st + wbase + i * 2048),
                  *reinterpret_cast<const uint4 *>(st + (wbase ^ 64) + i * 2048));
  };
  auto read_x = [&](const uint8_t *st, int j) {
    xf[j].set(*reinterpret_cast<const uint4 *>(st + xbase + j * 2048),
              *reinterpret_cast<const uint4 *>(st + (xbase ^ 64) + j * 2048));
  };
  auto add = [&](int i, int j) {
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[i][j][k] = __builtin_fmaf(d[i & 1][j][k], s[j], acc[i][j][k]);
  };
  auto meet = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // step t from stage rd; nx holds step t + 1 once its loads have landed
  auto step = [&](uint8_t *rd, uint8_t *nx, int t) {
    const float swv = *reinterpret_cast<const float *>(rd + swbase);
    float sx[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) sx[j] = *reinterpret_cast<const float *>(rd + sbase + j * 64);
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      if (i < TN - 1) {
        read_w(rd, i + 1);
        issue(nx, t + 1, (i + 1) * PPR, (i + 2) * PPR);
      } else {
        meet();
        issue(rd, t + 2, 0, PPR);
        read_w(nx, 0);
      }
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        if (i == 0) add(TN - 1, j);          // the previous block's last row (zeros before the first)
        d[i & 1][j] = block_dot(wf[i & 1], xf[j]);
        if (i > 0) add(i - 1, j);
        if (i == TN - 1) read_x(nx, j);
      }
      if (i == 0) {
#pragma unroll
        for (int j = 0; j < TM; ++j) s[j] = sx[j] * swv;
      }
      // one MFMA, then the additions that fit behind it
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x8, F32OUT ? 4 : 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    d[(TN - 1) & 1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    s[j] = 0.f;
  }
  issue(stage0, 0, 0, LOADS);
  meet();
  issue(stage1, 1, 0, PPR);
  read_w(stage0, 0);
#pragma unroll
  for (int j = 0; j < TM; ++j) read_x(stage0, j);
  for (int k = 0; k + 1 < steps; k += 2) {
    step(stage0, stage1, k);
    step(stage1, stage0, k + 1);
  }
  if (steps & 1) step(stage0, stage1, steps - 1);
  __builtin_amdgcn_s_waitcnt(0);      // no load into this workgroup's LDS outlives it
#pragma unroll
  for (int j = 0; j < TM; ++j) add(TN - 1, j);
  if constexpr (KS > 1) {
    // the K groups' sums, added in their order by the first
    static_assert((KS - 1) * NW * TN * TM * 1024 <= KS * STAGE, "the sums fit a stage");
    f32x4 *const sums = reinterpret_cast<f32x4 *>(stages0);
    __syncthreads();                  // every wave is done with the stages
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) sums[((((kg - 1) * NW + wave) * TN + i) * TM + j) * 64 + lane] = acc[i][j];
    }
    __syncthreads();
    if (kg > 0) return;
    for (int q = 0; q < KS - 1; ++q)
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          const f32x4 v = sums[(((q * NW + wave) * TN + i) * TM + j) * 64 + lane];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][k] += v[k];
        }
  }
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
      put4<F32OUT, VEC>(y, x.rows, w.rows, m0 + wm * 16 * TM + 16 * j + r, n0 + wn * 16 * TN + 16 * i + 4 * g,
                        acc[i][j]);
}

template <int WN, int WM, int KS, int TN, int TM, bool E5M2, bool F32OUT, bool VEC>
void launch_tile(const Fp8In &x, const Fp8In &w, void *y, hipStream_t s) {
  constexpr int BN = 16 * TN * WN, BM = 16 * TM * WM;
  const int tn = (int)((w.rows + BN - 1) / BN), tm = (int)((x.rows + BM - 1) / BM);
  hipLaunchKernelGGL((fp8_tile_kernel<WN, WM, KS, TN, TM, E5M2, F32OUT, VEC>), grid_of((int64_t)tn * tm),
                     dim3(64 * WN * WM * KS), 0, s, x, w, y, tn, tm);
}

template <int MT, int NR, int U, int WAVES, bool E5M2, bool F32OUT, bool VEC>
void launch_small(const Fp8In &x, const Fp8In &w, void *y, hipStream_t s) {
  const dim3 n = grid_of((w.rows + 16 * NR - 1) / (16 * NR));
  const dim3 g(n.x, (unsigned)((x.rows + 16 * MT - 1) / (16 * MT)), n.y);
  hipLaunchKernelGGL((fp8_small_kernel<MT, NR, U, WAVES, E5M2, F32OUT, VEC>), g, dim3(64 * WAVES), 0, s, x, w, y);
}

// Estimated time (us, less a constant) of the tile kernel with KS groups of
// waves: (steps + 1) steps of KS blocks, each at a measured us[r - 1] a block
// while a CU holds r workgroups (at most per_cu).  Tiles beyond that come in
// rounds, whole ones where a CU holds one workgroup, else running into each other.
double tile_time(int64_t M, int64_t N, int64_t KB, int bn, int bm, int ks, int per_cu, const double *us) {
  const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn), held = (tiles + 255) / 256;
  const double steps = (double)((KB + ks - 1) / ks + 1) * ks;
  if (held <= per_cu) return steps * us[held - 1];
  const double some = (double)tiles / (256.0 * per_cu), whole = (double)((held + per_cu - 1) / per_cu);
  return (per_cu == 1 || whole < some + 0.35 ? whole : some + 0.35) * steps * us[per_cu - 1];
}

// The kernel for M x N x K by those estimates; the constants fit K = 4096 at
// M = 24 ... 4096 and N = 4096 ... 11008, where the choice was the fastest or
// within 8% of it (bf16 output, 256 x 4096: 25.0 us on 128 x 128 tiles, 13.1 on
// 64 x 64 with four K groups; 1024 x 4096: 28.4 and 25.3 with two groups of
// 128 x 128; fp32, 64 x 11008: 44.7 and 19.7, 777 x 5004 x 2600: 38.2 on
// 128 x 128 and 33.9 on 128 x 64).
template <bool E5M2, bool F32OUT, bool VEC>
void launch_any(const Fp8In &x, const Fp8In &w, void *y, hipStream_t s) {
  const int64_t M = x.rows, N = w.rows, KB = w.pitch / kFp8Block;
  if (M <= 16) {
    // One or two rows of X: the weight's stream is all, and one row group a
    // workgroup carries it best, in 16 waves where the rows are long (28672 x
    // 8192: 39.2 us, 42.0 with 8 waves; 8192 x 4096: 7.8 and 7.3).
    if (M <= 2) {
      if (KB > 32) launch_small<1, 1, 2, 16, E5M2, F32OUT, VEC>(x, w, y, s);
      else launch_small<1, 1, 4, 8, E5M2, F32OUT, VEC>(x, w, y, s);
      return;
    }
    // More rows: every workgroup reads all of X, so about as many workgroups as
    // CUs (16 rows of X, us with 1, 2, 4, 8 row groups a workgroup: 4096 x 4096
    // 6.7, 8.3, 10.7; 8192 x 4096 11.8, 8.9, 12.4, 20.0; 28672 x 8192 67.7, 57.8,
    // 47.2, 45.4; with 3 and 4: 11008 x 4096 11.8 and 12.9; with 5, 6, 8: 20480 x
    // 4096 17.1, 19.0, 21.9, 24576 x 4096 28.6, 18.6, 21.8; with 7 and 8: 28672 x
    // 8192 43.0 and 45.6).  The waves and the blocks in flight beside them, here
    // and for up to 64 rows, were taken from runs at one or two of those widths
    // each.  Among 1, 2, 4 blocks and 4, 8, 12, 16 waves at K = 2048, 4096, 8192
    // they are the fastest or within 9% of it for bf16 outputs (16 x 20416 x 4096
    // 19.1 us, 17.5 with 1 and 12; 16 x 32704 x 4096 27.1, the fastest), and within
    // 19% for fp32 ones, where 12 or 16 waves lead from five row groups on and with
    // two groups of X (16 x 20416 x 4096 22.7 and 19.5).
    switch ((N + 16 * 256 - 1) / (16 * 256)) {
      case 1: launch_small<1, 1, 4, 8, E5M2, F32OUT, VEC>(x, w, y, s); break;
      case 2: launch_small<1, 2, 4, 8, E5M2, F32OUT, VEC>(x, w, y, s); break;
      case 3: launch_small<1, 3, 1, 12, E5M2, F32OUT, VEC>(x, w, y, s); break;
      case 4:
        // (an fp32 output's fragments take more registers: fewer waves, 13.7 us for 15.7)
        if constexpr (F32OUT) launch_small<1, 4, 4, 4, E5M2, F32OUT, VEC>(x, w, y, s);
        else launch_small<1, 4, 1, 16, E5M2, F32OUT, VEC>(x, w, y, s);
        break;
      case 5: launch_small<1, 5, 2, 8, E5M2, F32OUT, VEC>(x, w, y, s); break;
      case 6: launch_small<1, 6, 1, 8, E5M2, F32OUT, VEC>(x, w, y, s); break;
      case 7: launch_small<1, 7, 2, 8, E5M2, F32OUT, VEC>(x, w, y, s); break;
      default: launch_small<1, 8, 2, 8, E5M2, F32OUT, VEC>(x, w, y, s);
    }
    return;
  }
  if (M <= 64) {
    // Likewise with two groups of 16 rows of X a workgroup, and one or two of
    // those (weights from HBM, us with the small and the tile kernel: 24 x 8192 x
    // 4096 10.8 and 11.4, 32 x 11008 x 4096 15.4 and 18.3, 32 x 20480 x 4096 22.4
    // and 30.4, 64 x 6000 x 4096 15.1 and 20.0, 64 x 8192 x 4096 16.6 and 20.7;
    // beyond: 32 x 28672 x 8192 79.8 and 60.3, 64 x 16384 x 4096 31.7 and 23.1).
    const int64_t rows = (M + 31) / 32;
    switch ((rows * N + 16 * 256 - 1) / (16 * 256)) {
      case 1: launch_small<2, 1, 2, 8, E5M2, F32OUT, VEC>(x, w, y, s); return;
      case 2:   // (fp32: 11.3 us with 8 waves, 12.7 with 16)
        if constexpr (F32OUT) launch_small<2, 2, 2, 8, E5M2, F32OUT, VEC>(x, w, y, s);
        else launch_small<2, 2, 1, 16, E5M2, F32OUT, VEC>(x, w, y, s);
        return;
      case 3: launch_small<2, 3, 1, 12, E5M2, F32OUT, VEC>(x, w, y, s); return;
      case 4: launch_small<2, 4, 1, 12, E5M2, F32OUT, VEC>(x, w, y, s); return;
      case 5:
      case 6:
        // (an fp32 output's fragments leave no registers for these; four groups
        // of X and three of W take 18.5 us for 48 x 11008 x 4096, two and six 20.1)
        if constexpr (!F32OUT) {
          if (rows == 1) launch_small<2, 6, 1, 12, E5M2, F32OUT, VEC>(x, w, y, s);
          else launch_small<4, 3, 1, 12, E5M2, F32OUT, VEC>(x, w, y, s);
          return;
        }
    }
  }
  enum { k64x4, k64x2, k64, k128x64, k128x2, k128, k256, kCount };
  double t[kCount];
  for (double &v : t) v = 1e300;
  static const double u64x4[2][1] = {{0.31}, {0.36}}, u64x2[2][2] = {{0.37, 0.52}, {0.40, 0.64}},
                      u64[4] = {0.5, 0.76, 1.0, 1.27}, u128x64[3] = {0.92, 1.21, 1.6},
                      u128x2[2][1] = {{0.70}, {1.05}}, u128[2][2] = {{0.82, 1.2}, {1.2, 2.05}}, u256[1] = {1.85};
  constexpr int F = F32OUT ? 1 : 0;
  t[k64x4] = tile_time(M, N, KB, 64, 64, 4, 1, u64x4[F]);
  t[k64x2] = tile_time(M, N, KB, 64, 64, 2, 2, u64x2[F]);
  t[k128x2] = tile_time(M, N, KB, 128, 128, 2, 1, u128x2[F]);
  t[k128] = tile_time(M, N, KB, 128, 128, 1, 2, u128[F]);
  // fp32 outputs only; 256 x 256 for bf16 ones only, since an fp32 output's
  // fragments take twice the registers
  if (F32OUT) {
    t[k64] = tile_time(M, N, KB, 64, 64, 1, 4, u64);
    t[k128x64] = tile_time(M, N, KB, 128, 64, 1, 3, u128x64);
  } else {
    t[k256] = tile_time(M, N, KB, 256, 256, 1, 1, u256);
  }
  int best = 0;
  for (int i = 1; i < kCount; ++i)
    if (t[i] < t[best]) best = i;
  switch (best) {
    case k64x4: launch_tile<2, 2, 4, 2, 2, E5M2, F32OUT, VEC>(x, w, y, s); break;
    case k64x2: launch_tile<2, 2, 2, 2, 2, E5M2, F32OUT, VEC>(x, w, y, s); break;
    case k128x2: launch_tile<2, 2, 2, 4, 4, E5M2, F32OUT, VEC>(x, w, y, s); break;
    case k128: launch_tile<2, 2, 1, 4, 4, E5M2, F32OUT, VEC>(x, w, y, s); break;
    case k64:
      if constexpr (F32OUT) launch_tile<2, 2, 1, 2, 2, E5M2, F32OUT, VEC>(x, w, y, s);
      break;
    case k128x64:
      if constexpr (F32OUT) launch_tile<2, 2, 1, 4, 2, E5M2, F32OUT, VEC>(x, w, y, s);
      break;
    default:
      if constexpr (!F32OUT) launch_tile<2, 4, 1, 8, 4, E5M2, F32OUT, VEC>(x, w, y, s);
  }
}

template <bool E5M2>
void launch_out(const Fp8In &x, const Fp8In &w, void *y, bool y_bf16, hipStream_t s) {
  const bool vec = w.rows % 4 == 0;
  if (y_bf16) {
    if (vec) launch_any<E5M2, false, true>(x, w, y, s);
    else launch_any<E5M2, false, false>(x, w, y, s);
  } else {
    if (vec) launch_any<E5M2, true, true>(x, w, y, s);
    else launch_any<E5M2, true, false>(x, w, y, s);
  }
}

}  // namespace

bool fp8_matmul_fits(int64_t M, int64_t N) {
  // a tile's number, and eight rows of tiles, stay below 2^31 at 64 x 64
  return N < ((int64_t)1 << 26) && (M + 63) / 64 <= ((int64_t)1 << 31) / 8 / ((N + 63) / 64);
}

hipError_t launch_fp8_matmul(const Fp8In &x, bool x_e5m2, const Fp8In &w, void *y, bool y_bf16, hipStream_t stream) {
  if (x_e5m2) launch_out<true>(x, w, y, y_bf16, stream);
  else launch_out<false>(x, w, y, y_bf16, stream);
  return hipGetLastError();
}

}  // namespace nf4
