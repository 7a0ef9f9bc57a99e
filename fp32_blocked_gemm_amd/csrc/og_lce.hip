// og_lce.hip -- og_linear_cross_entropy and its gradient: the softmax cross
// entropy of the logits z = X W^T (X n x d, W v x d, a row per vocabulary
// entry), the logits never kept.
//
//   lse_i = log sum_j exp z_ij,  loss_i = lse_i - z_i,t(i)
//   g_ij = dloss_i (exp(z_ij - lse_i) - [j = t(i)]),  dX = g W,  dW = g^T X
//
// Rows that do not count (the ignored index) are left out before anything is
// computed: the others are packed to the front, so that ignored rows cost
// nothing and whatever they hold (NaN in a padded batch) reaches nothing.
// The number of rows left stays on the device; the products read it there.
//
// Forward: one tile product whose epilogue keeps a running maximum and sum of
// each row over the tile's columns; a second kernel joins the tiles.  The
// gradient recomputes the logits in pieces of the vocabulary, stores g of a
// piece and runs both products on it.  All of it is bound by the matrix cores:
// 2 n v d operations forward, 6 n v d backward.
//
// (The gradient comes with lse and dloss after the forward call, so the logits are
// computed twice; nothing is kept between the calls.)
//
// bf16 tensors run as they are, g in bf16 and divided by the largest |dloss|,
// by which the sums are multiplied in fp32: where all rows weigh the same (a
// mean), the target's entry p - 1 then rounds by its p alone, and not every row's
// by the same error of the weight (4096 x 32768 x 4096: errors of dX and dW
// 0.0019 for 0.0023 to 0.0032, 0.0017 of them their own rounding).
//
// fp32 ones run as two fp16 planes (og_tile.hpp).  For the logits each row of X (and,
// forward, of W) has a power of two of its own that brings its largest value to
// [2^13, 2^14); the epilogue undoes both.  The gradients' sums run over rows of W and
// of X, whose powers cannot differ inside a sum, so they get planes of one common
// power each: W's of its largest value, and a second set of X's, row i times the power
// of two of dloss_i, of the largest |dloss_i| max |X_i| (scan_kernel finds both).  g is
// stored as (p - [j = t]) times dloss_i's mantissa and 2^14: it serves both products,
// keeps 22 bits down to probabilities of 2^-16 and some down to 2^-38 whatever the
// sizes of the rows of X, W and dloss, and stays below 2^14 for rows of zeros too.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "og.h"
#include "og_host.hpp"
#include "og_tile.hpp"

namespace og::lce {

using namespace og::tile;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBias = 4096;

// The compact list of the rows that count.
struct Rows {
  int *count;     // how many
  int *pos;       // original row -> place in the list, -1 if it does not count
  int *row;       // place -> original row
  int *target;    // by place, as the next two
  float *lse;
  float *dloss;
  float *zt;      // the target's logit (forward)
  int *xexp;      // fp32: the exponent of a row of X, by place
  // fp32 gradient: the largest exponent of |dloss| x row maximum of X, and of W's
  // maximum, each + kBias (0: none)
  int *most;
  float *scale;   // bf16: the largest finite |dloss| of the rows that count, or 1
};

// The largest of the wave's (non-negative) values, in every lane.
__device__ __forceinline__ float wave_max(float v) {
#define OG_ROR(N)                                                                                  \
  v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v),      \
                                                                  0x120 + N, 0xf, 0xf, true)))
  OG_ROR(8);
  OG_ROR(4);
  OG_ROR(2);
  OG_ROR(1);
#undef OG_ROR
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// One block: the rows' places by a running count, in order (a launch's time up
// to some thousand rows: 1000 in 3.5 us, 4096 in 8).  Rows that do not
// count get their loss here (forward): 0 for the ignored index, NaN for a
// target outside the vocabulary.
__global__ __launch_bounds__(1024) void rows_kernel(int n, int64_t v, const int64_t *target,
                                                    int64_t ignore, Rows r, const float *lse_in,
                                                    const float *dloss, float *loss, float *lse) {
  __shared__ int waves[16];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int done = 0;
  float largest = 0;
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    const int64_t t = i < n ? target[i] : ignore;
    const bool counts = i < n && t != ignore && t >= 0 && t < v;
    const uint64_t vote = __ballot(counts);
    if (lane == 0) waves[w] = __popcll(vote);
    __syncthreads();
    int at = done, all = 0;
    for (int k = 0; k < 16; ++k) {
      if (k < w) at += waves[k];
      all += waves[k];
    }
    at += __popcll(vote & ((1ull << lane) - 1));
    if (counts) {
      r.pos[i] = at;
      r.row[at] = i;
      r.target[at] = (int)t;
      if (lse_in) {
        const float d = dloss[i];
        r.lse[at] = lse_in[i];
        r.dloss[at] = d;
        if (__builtin_isfinite(d)) largest = fmaxf(largest, fabsf(d));
      }
    } else if (i < n) {
      r.pos[i] = -1;
      if (loss) {
        loss[i] = t == ignore ? 0.0f : __builtin_nanf("");
        lse[i] = 0.0f;
      }
    }
    done += all;
    __syncthreads();
  }
  __shared__ float tops[16];
  largest = wave_max(largest);
  if (lane == 0) tops[w] = largest;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 16; ++k) largest = fmaxf(largest, tops[k]);
    *r.scale = largest > 0 ? largest : 1.0f;
    *r.count = done;
    r.most[0] = r.most[1] = 0;
  }
}

template <class T, bool VEC>
__device__ __forceinline__ f32x4 load4(const T *p, int left) {
  f32x4 v = {0, 0, 0, 0};
  if constexpr (VEC) {
    if (left >= 4) {
      if constexpr (sizeof(T) == 4) {
        v = *reinterpret_cast<const f32x4 *>(p);
      } else {
        const bf16x4 h = *reinterpret_cast<const bf16x4 *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)h[e];
      }
      return v;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) v[e] = (float)p[e];
  return v;
}

// `rows` rows of `cols` bf16 values, padded with zeros to ld columns.  With
// pos, row i goes to place pos[i], and a row without a place clears its row of
// `clear` instead (the gradient of an ignored row).  Bound by the bytes: 4096
// rows of 4096 in 19 us.
template <bool VEC>
__global__ __launch_bounds__(256) void copy_kernel(int rows, int cols, const __bf16 *x, int64_t ldx,
                                                   const int *pos, uint16_t *out, int64_t ld,
                                                   __bf16 *clear, int64_t ldc) {
  const int per = (int)(ld / 4);
  const int64_t total = (int64_t)rows * per, step = (int64_t)gridDim.x * 256;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += step) {
    const int i = (int)(q / per), c = (int)(q - (int64_t)i * per) * 4;
    const int to = pos ? pos[i] : i;
    if (to < 0) {
      if (clear)
        for (int e = 0; e < 4; ++e)
          if (c + e < cols) clear[i * ldc + c + e] = (__bf16)0.0f;
      continue;
    }
    const f32x4 v = load4<__bf16, VEC>(x + i * ldx + c, cols - c);
    bf16x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = (__bf16)v[e];
    *reinterpret_cast<bf16x4 *>(out + to * ld + c) = h;
  }
}

// fp32 rows: a wave takes one, of which the first 768 columns stay in registers
// between its maximum and its planes.
constexpr int kHeld = 3;

// The first columns of a row and the largest finite magnitude of all of it, in every lane.
template <bool VEC>
__device__ __forceinline__ float row_top(const float *row, int cols, int lane, f32x4 (&held)[kHeld]) {
  float top = 0;
  auto larger = [&](const f32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, __builtin_isfinite(v[e]) ? fabsf(v[e]) : 0.0f);
  };
#pragma unroll
  for (int q = 0; q < kHeld; ++q) held[q] = load4<float, VEC>(row + 4 * lane + 256 * q, cols - 4 * lane - 256 * q);
#pragma unroll
  for (int q = 0; q < kHeld; ++q) larger(held[q]);
  for (int c = 4 * lane + 256 * kHeld; c < cols; c += 256) larger(load4<float, VEC>(row + c, cols - c));
  return wave_max(top);
}

// Four columns' planes, times 2^e, zero beyond the row.
__device__ __forceinline__ void store_planes(uint16_t *out, int c, f32x4 v, int e) {
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = __builtin_ldexpf(v[q], e);
  f16x4 h, l;
  split4(v, h, l);
  *reinterpret_cast<f16x4 *>(out + column<2>(c, 0)) = h;
  *reinterpret_cast<f16x4 *>(out + column<2>(c, 1)) = l;
}

// A row's planes, padded with zeros to `width` columns, times the power of two that brings its
// largest value to [2^13, 2^14), whose exponent goes to *exp.  Returns that value.
template <bool VEC>
__device__ __forceinline__ float own_planes(const float *row, int cols, uint16_t *out, int width,
                                            int *exp, int lane) {
  f32x4 held[kHeld];
  const float top = row_top<VEC>(row, cols, lane, held);
  const int e2 = top > 0 ? 14 - (int)__builtin_amdgcn_frexp_expf(top) : 0;
  if (lane == 0) *exp = e2;
#pragma unroll
  for (int q = 0; q < kHeld; ++q)
    if (4 * lane + 256 * q < width) store_planes(out, 4 * lane + 256 * q, held[q], e2);
  for (int c = 4 * lane + 256 * kHeld; c < width; c += 256)
    store_planes(out, c, load4<float, VEC>(row + c, cols - c), e2);
  return top;
}

// copy_kernel for fp32: the planes of each row by its own power (forward).  Bound by the bytes:
// 50021 rows of 768 in 54 us.
template <bool VEC>
__global__ __launch_bounds__(256) void planes_kernel(int rows, int cols, const float *x, int64_t ldx,
                                                     const int *pos, uint16_t *out, int64_t ld, int *exp) {
  const int lane = threadIdx.x & 63;
  for (int i = blockIdx.x * 4 + (threadIdx.x >> 6); i < rows; i += gridDim.x * 4) {
    const int to = pos ? pos[i] : i;
    if (to >= 0) own_planes<VEC>(x + i * ldx, cols, out + to * ld, (int)(ld / 2), exp + to, lane);
  }
}

// The fp32 gradient's operands, in two launches.
struct Sides {
  int n, d;
  int64_t v;
  const float *x, *w;  // (common_kernel: w and v are a piece's)
  int64_t ldx, ldw, ld;  // ld: elements of a row of planes
  Rows r;
  uint16_t *x_own, *x_common, *w_common;
  float *clear;  // the gradient of rows of X that do not count is zero
  int64_t ldc;
  int x_blocks;  // of the launch; the others are W's
};

// X's planes by row, and the exponents of both common powers: by an atomic maximum of each
// block's, which does not depend on their order.  W is only read.  Blocks of 16 waves: what
// the launch takes beyond the bytes' time is its atomics on one address (8191 x 384 and 1000
// rows of X: 2300 blocks of 4 waves 29 us, 319 of 16 8).
constexpr int kScanWaves = 16;
template <bool VEC>
__global__ __launch_bounds__(64 * kScanWaves) void scan_kernel(Sides a) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const bool first = (int)blockIdx.x < a.x_blocks;
  int seen = 0;
  if (first) {
    for (int i = blockIdx.x * kScanWaves + w; i < a.n; i += a.x_blocks * kScanWaves) {
      const int to = a.r.pos[i];
      if (to < 0) {
        if (a.clear)
          for (int c = lane; c < a.d; c += 64) a.clear[i * a.ldc + c] = 0.0f;
        continue;
      }
      const float by = a.r.dloss[to];
      const float top = own_planes<VEC>(a.x + i * a.ldx, a.d, a.x_own + to * a.ld, (int)(a.ld / 2),
                                        a.r.xexp + to, lane);
      if (top > 0 && by != 0 && __builtin_isfinite(by))
        seen = max(seen, kBias + (int)__builtin_amdgcn_frexp_expf(top) + (int)__builtin_amdgcn_frexp_expf(by));
    }
  } else {
    const int block = blockIdx.x - a.x_blocks, blocks = gridDim.x - a.x_blocks;
    float top = 0;
    for (int64_t j = block * kScanWaves + w; j < a.v; j += blocks * kScanWaves) {
      f32x4 held[kHeld];
      top = fmaxf(top, row_top<VEC>(a.w + j * a.ldw, a.d, lane, held));
    }
    if (top > 0) seen = kBias + (int)__builtin_amdgcn_frexp_expf(top);
  }
  __shared__ int waves[kScanWaves];
  if (lane == 0) waves[w] = seen;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kScanWaves; ++k) seen = max(seen, waves[k]);
    if (seen) atomicMax(a.r.most + (first ? 0 : 1), seen);
  }
}

// The exponent of a common power, which brings the largest value to [2^13, 2^14) (of dloss
// times X: to [2^12, 2^14)).
__device__ __forceinline__ int common_exponent(int most) { return most ? 14 - (most - kBias) : 0; }

// Planes by the common powers: of a piece of W, and (x_blocks not 0) of X times the powers of
// two of dloss; a row of dloss zero, whose g is zero, is zero (the same sizes: 6 us).
template <bool VEC>
__global__ __launch_bounds__(256) void common_kernel(Sides a) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, width = (int)(a.ld / 2);
  auto planes = [&](const float *row, uint16_t *out, int e) {
    for (int c = 4 * lane; c < width; c += 256) store_planes(out, c, load4<float, VEC>(row + c, a.d - c), e);
  };
  if ((int)blockIdx.x < a.x_blocks) {
    const int e = common_exponent(a.r.most[0]);
    for (int i = blockIdx.x * 4 + w; i < a.n; i += a.x_blocks * 4) {
      const int to = a.r.pos[i];
      if (to < 0) continue;
      const float by = a.r.dloss[to];
      uint16_t *out = a.x_common + to * a.ld;
      if (by != 0) {
        planes(a.x + i * a.ldx, out, e + (int)__builtin_amdgcn_frexp_expf(by));
      } else {
        for (int c = 4 * lane; c < width; c += 256) store_planes(out, c, f32x4{0, 0, 0, 0}, 0);
      }
    }
  } else {
    const int e = common_exponent(a.r.most[1]);
    for (int64_t j = (int64_t)(blockIdx.x - a.x_blocks) * 4 + w; j < a.v; j += (gridDim.x - a.x_blocks) * 4)
      planes(a.w + j * a.ldw, a.w_common + j * a.ld, e);
  }
}

// Four logits: fp32 sums as they are, or less their rows' powers of two.
template <int P>
__device__ __forceinline__ f32x4 logits(f32x4 v, int xexp, const int *wexp, int n, int N) {
  if constexpr (P == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = __builtin_ldexpf(v[q], -(xexp + wexp[min(n + q, N - 1)]));
  }
  return v;
}

// Epilogue of the forward product: each row's maximum over the tile's columns
// and the sum of exp against it, and the target's logit where it lies here.  Two
// numbers a row and tile go to memory where the logits would be BN.  One bf16 row
// against 32768 x 4096 is bound by W's bytes (55 us, 4.9 TB/s), 3891 rows by the
// matrix cores (874 us, 1195 TFLOP/s), 700 fp32 rows against 50021 x 768 too (160
// to 186 us, 290 to 335 TFLOP/s of fp32 operations, 3 of the matrix cores' each).
struct LseArgs {
  float2 *part;  // [tile column][n]
  const int *target;
  float *zt;
  const int *xexp, *wexp;  // exponents of the planes' rows
  int n, v0, part0;  // rows of part, first column, first tile column
};
template <int P>
struct Lse {
  using Args = LseArgs;
  static constexpr bool kSymmetric = false;
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t,
                                               const Args &e) {
    float2 *sh = reinterpret_cast<float2 *>(t.lds);  // [WN][BM]
    const int nc = t.n0 + 4 * (t.lane >> 4);
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = t.m0 + 16 * i + (t.lane & 15);
      const int want = m < t.M ? e.target[m] - e.v0 - nc : -1;
      const int xexp = P == 2 && m < t.M ? e.xexp[m] : 0;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        acc[i][j] = logits<P>(acc[i][j], xexp, e.wexp, nc + 16 * j, t.N);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (want == 16 * j + q) e.zt[m] = acc[i][j][q];
          if (nc + 16 * j + q >= t.N) acc[i][j][q] = -INFINITY;
          top = fmaxf(top, acc[i][j][q]);
        }
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float from = top == -INFINITY ? 0.0f : top;
      float sum = 0;
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          sum += __builtin_amdgcn_exp2f((acc[i][j][q] - from) * kLog2e);
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (t.lane < 16) sh[t.wn * S::BM + t.wm * S::FM * 16 + 16 * i + t.lane] = {top, sum};
    }
    __syncthreads();
    const int m0 = t.tile_m * S::BM;
    for (int r = threadIdx.x; r < S::BM; r += S::NW * 64) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < S::WN; ++w) top = fmaxf(top, sh[w * S::BM + r].x);
      const float from = top == -INFINITY ? 0.0f : top;
      float sum = 0;
#pragma unroll
      for (int w = 0; w < S::WN; ++w)
        sum += sh[w * S::BM + r].y * __builtin_amdgcn_exp2f((sh[w * S::BM + r].x - from) * kLog2e);
      if (m0 + r < t.M) e.part[(int64_t)(e.part0 + t.tile_n) * e.n + m0 + r] = {top, sum};
    }
  }
};

// Joins the tiles of 8 rows per block: 32 threads a row.  (4 to 10 us: a launch
// and a few dependent loads.)
__global__ __launch_bounds__(256) void finish_kernel(Rows r, const float2 *part, int n, int tiles,
                                                     float *loss, float *lse) {
  __shared__ float2 sh[32][8];
  const int m = blockIdx.x * 8 + (threadIdx.x & 7), w = threadIdx.x >> 3;
  const int count = *r.count;
  float top = -INFINITY, sum = 0;
  if (m < count)
    for (int t0 = w; t0 < tiles; t0 += 32 * 4) {
      float2 p[4];  // four loads in flight
      float to = top;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = t0 + 32 * q;
        p[q] = t < tiles ? part[(int64_t)t * n + m] : float2{-INFINITY, 0};
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) to = fmaxf(to, p[q].x);
      const float from = to == -INFINITY ? 0.0f : to;
      sum *= __builtin_amdgcn_exp2f((top - from) * kLog2e);
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += p[q].y * __builtin_amdgcn_exp2f((p[q].x - from) * kLog2e);
      top = to;
    }
  sh[w][threadIdx.x & 7] = {top, sum};
  __syncthreads();
  if (threadIdx.x >= 8 || m >= count) return;
  top = -INFINITY;
  for (int k = 0; k < 32; ++k) top = fmaxf(top, sh[k][threadIdx.x].x);
  const float from = top == -INFINITY ? 0.0f : top;
  sum = 0;
  for (int k = 0; k < 32; ++k)
    sum += sh[k][threadIdx.x].y * __builtin_amdgcn_exp2f((sh[k][threadIdx.x].x - from) * kLog2e);
  const float l = top + logf(sum);
  const int i = r.row[m];
  lse[i] = l;
  loss[i] = l - r.zt[m];
}

// Epilogue of the recomputed logits: g in planes, zero beyond the vocabulary.
// Bound by the matrix cores (3891 x 16384 x 4096 bf16 463 us, 1128 TFLOP/s).
struct GradArgs {
  uint16_t *g;
  int64_t ld;
  const int *target;
  const float *lse, *dloss, *scale;
  const int *xexp;
  const int *most;  // of W
  int v0;
};
template <int P>
struct Grad {
  using Args = GradArgs;
  static constexpr bool kSymmetric = false;
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t,
                                               const Args &e) {
    const int nc = t.n0 + 4 * (t.lane >> 4);
    const int wexp = P == 2 ? common_exponent(*e.most) : 0;
    const float by = *e.scale;
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = t.m0 + 16 * i + (t.lane & 15);
      if (m >= t.M) continue;
      const float l = e.lse[m], dl = e.dloss[m];
      const float d = P == 2 ? __builtin_ldexpf(dl, 14 - (int)__builtin_amdgcn_frexp_expf(dl)) : dl / by;
      const int want = e.target[m] - e.v0 - nc;
      const int up = P == 2 ? -(e.xexp[m] + wexp) : 0;
      uint16_t *to = e.g + m * e.ld;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int n = nc + 16 * j;
        if (n >= e.ld / P) continue;
        f32x4 v = acc[i][j];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (P == 2) v[q] = __builtin_ldexpf(v[q], up);
          const float p = __builtin_amdgcn_exp2f((v[q] - l) * kLog2e);
          v[q] = n + q < t.N ? (want == 16 * j + q ? p - 1.0f : p) * d : 0.0f;
        }
        if constexpr (P == 1) {
          bf16x4 h;
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = (__bf16)v[q];
          *reinterpret_cast<bf16x4 *>(to + n) = h;
        } else {
          store_planes(to, n, v, 0);
        }
      }
    }
  }
};

// Up to four values of a row.
template <class T>
__device__ __forceinline__ void store4(T *to, const f32x4 v, int left, bool whole) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  T4 h;
#pragma unroll
  for (int q = 0; q < 4; ++q) h[q] = (T)v[q];
  if (whole && left >= 4) {
    *reinterpret_cast<T4 *>(to) = h;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) to[q] = h[q];
  }
}

// Epilogue of dX and dW.  The sum so far (dX, over the pieces) is kept in fp32
// and rounded once, with the last piece; a product whose k is split stores its
// parts for join_kernel.  Bound by the matrix cores where there are tiles enough
// (3891 x 16384 x 4096 bf16: dX 422 us, 1239 TFLOP/s, dW 443 us), else by the few
// tiles (700 x 8191 x 384 fp32: dX 29 us and 5 of joining, dW 23).
struct OutArgs {
  float *sum;    // the sum over pieces, or the parts; not used by a single piece
  int64_t lds;
  int64_t part;  // from one part to the next; 0: not split
  int first, last;
  void *out;
  int64_t ldo;
  int whole;       // four values of a row of out are one aligned store
  const int *row;  // null: row m is row m of out
  const int *most;      // fp32: of the other operand, whose common power is undone
  const float *weight;  // fp32, dX: dloss, of whose power of two g was relieved; else null
  const float *scale;   // bf16: what g was divided by
};
template <class T>
struct Out {
  using Args = OutArgs;
  static constexpr bool kSymmetric = false;
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t,
                                               const Args &e) {
    const int nc = t.n0 + 4 * (t.lane >> 4);
    const int common = S::P == 2 ? 14 + common_exponent(*e.most) : 0;
    const float by = *e.scale;
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = t.m0 + 16 * i + (t.lane & 15);
      if (m >= t.M) continue;
      const int up = S::P == 2 && e.weight ? (int)__builtin_amdgcn_frexp_expf(e.weight[m]) - common : -common;
      T *to = static_cast<T *>(e.out) + (e.row ? e.row[m] : m) * e.ldo;
      float *sum = e.sum + t.batch * e.part + m * e.lds;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int n = nc + 16 * j;
        if (n >= t.N) continue;
        f32x4 v = acc[i][j];
        if constexpr (S::P == 2) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = __builtin_ldexpf(v[q], up);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] *= by;
        }
        if (!e.first) {
          const f32x4 was = *reinterpret_cast<const f32x4 *>(sum + n);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += was[q];
        }
        if (!e.last) *reinterpret_cast<f32x4 *>(sum + n) = v;
        else store4(to + n, v, t.N - n, e.whole);
      }
    }
  }
};

// Adds the parts of a split product in order, the sum of the pieces before it
// first; the result goes where Out would store it.
template <class T>
__global__ __launch_bounds__(256) void join_kernel(int rows, int cols, const int *count, int parts,
                                                   const float *from, int64_t part, float *sum,
                                                   int64_t lds, int first, int last, T *out,
                                                   int64_t ldo, int whole, const int *row) {
  const int per = (cols + 3) / 4;
  if (count) rows = *count;
  const int64_t total = (int64_t)rows * per, step = (int64_t)gridDim.x * 256;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += step) {
    const int m = (int)(at / per), n = (int)(at - (int64_t)m * per) * 4;
    f32x4 v = {0, 0, 0, 0};
    if (!first) v = *reinterpret_cast<const f32x4 *>(sum + m * lds + n);
    for (int p = 0; p < parts; ++p) {
      const f32x4 w = *reinterpret_cast<const f32x4 *>(from + p * part + m * lds + n);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += w[q];
    }
    if (!last) *reinterpret_cast<f32x4 *>(sum + m * lds + n) = v;
    else store4(out + (row ? row[m] : m) * ldo + n, v, cols - n, whole);
  }
}

// Few rows of fp32 in the forward call (up to kFew): no planes, whose making
// alone would read and write as many bytes as W has.  Plain fp32 multiply-adds,
// each weight read once; bound by the latency of a wave's loads of W (25543 x 2048:
// 1 row 70 us, 8 rows 108, 1.9 TB/s; with X read from one place all along 108, with a
// quarter of the multiply-adds 103; 9 rows by planes 147).
constexpr int kFew = 8, kFewWaves = 1024;

__device__ __forceinline__ float wave_sum(float v) {
#define OG_ROR(N)                                                                                  \
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + N,   \
                                                          0xf, 0xf, true))
  OG_ROR(8);
  OG_ROR(4);
  OG_ROR(2);
  OG_ROR(1);
#undef OG_ROR
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// The logits of N rows, four vocabulary rows a wave at a time.  Each wave's
// running maximum and sum go to part as a tile's would.
template <int N, bool VEC>
__global__ __launch_bounds__(256) void few_logits_kernel(Rows r, int n, int64_t v, int d, const float *x,
                                                         int64_t ldx, const float *w, int64_t ldw,
                                                         float2 *part) {
  constexpr int R = 4;
  int count = *r.count;
  if (count == 0) return;
  // kept in a vector register, and with it what the rows' places give: they are
  // more than the scalar registers hold
  asm volatile("" : "+v"(count));
  const int lane = threadIdx.x & 63, wave = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float *xp[N];  // from the lane's first column on
  float top[N], sum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    xp[i] = x + r.row[min(i, count - 1)] * ldx + 4 * lane;
    top[i] = -INFINITY;
    sum[i] = 0;
  }
  for (int64_t j0 = (int64_t)wave * R; j0 < v; j0 += (int64_t)gridDim.x * 4 * R) {
    float acc[N][R];
    const float *wp[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      wp[q] = w + min(j0 + q, v - 1) * ldw + 4 * lane;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i][q] = 0;
    }
    for (int c = 0; c < d; c += 256) {
      const int left = d - c - 4 * lane;
      f32x4 b[R];
#pragma unroll
      for (int q = 0; q < R; ++q) b[q] = load4<float, VEC>(wp[q] + c, left);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const f32x4 a = load4<float, VEC>(xp[i] + c, left);
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][q] = fmaf(a[e], b[q][e], acc[i][q]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int place = min(i, count - 1), want = r.target[place] - (int)j0;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const float z = wave_sum(acc[i][q]);
        if (j0 + q >= v) continue;
        if (want == q && lane == 0 && i < count) r.zt[i] = z;
        const float to = fmaxf(top[i], z), from = to == -INFINITY ? 0.0f : to;
        sum[i] = sum[i] * __builtin_amdgcn_exp2f((top[i] - from) * kLog2e) +
                 __builtin_amdgcn_exp2f((z - from) * kLog2e);
        top[i] = to;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 0 && i < count) part[(int64_t)wave * n + i] = {top[i], sum[i]};
}

struct Plan {
  int planes;
  bool few;             // forward, fp32 of up to kFew rows
  int64_t dp;           // d padded
  int64_t piece;        // vocabulary rows of a piece
  int dx_parts, dw_parts;  // parts of k of a piece's gradient products
  int64_t rows_at, wexp_at, x_at, x2_at, w_at, part_at, g_at, sum_at, parts_at, total;
};

// Parts of k of an m x n product: as many as make up two tiles of 64 x 64 for
// each compute unit, of at least 512 k each (one part costs its own fp32 copy
// of the result and a pass that adds the copies: 1000 x 384 over 8191 took 107
// us whole, 48 in five parts, 34 since with smaller tiles).
int parts_of(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = std::max<int64_t>(1, (m + 63) / 64 * ((n + 63) / 64));
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / tiles, k / 512, 16}));
}

// A piece keeps g (and the planes of its weights) at up to 2^26 values a
// plane (128 MB): large enough to fill the card with tiles (16384 columns of 4096
// rows are 1024 of them), small enough to stay in the 256 MB last-level cache.
Plan plan(int64_t n, int64_t v, int64_t d, int type, bool grad) {
  Plan p;
  p.planes = type == OG_F32 ? 2 : 1;
  p.dp = round_up(d, 64);
  p.few = !grad && p.planes == 2 && n > 0 && n <= kFew;
  const int64_t most = (int64_t(1) << 26) / std::max(n, p.dp) / 256 * 256;
  p.piece = std::min(round_up(v, 256), std::max<int64_t>(2048, most));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  p.rows_at = take(256 + 7 * round_up(n, 64) * 4);
  if (p.few) {
    p.part_at = take(kFewWaves * n * 8);
    p.wexp_at = p.x_at = p.x2_at = p.w_at = p.g_at = p.sum_at = p.parts_at = p.total = at;
    p.dx_parts = p.dw_parts = 1;
    return p;
  }
  p.wexp_at = take(p.planes == 2 && !grad ? p.piece * 4 : 0);
  p.x_at = take(p.planes * n * p.dp * 2);
  p.x2_at = grad && p.planes == 2 ? take(p.planes * n * p.dp * 2) : at;  // by the common power
  // (of bf16 W only where its rows cannot be read in place, which its stride and alignment
  // decide: the size function knows neither)
  p.w_at = take(p.planes * p.piece * p.dp * 2);
  p.part_at = grad ? at : take((round_up(v, p.piece) / (p.planes == 2 ? 32 : 64)) * n * 8);
  p.g_at = grad ? take(p.planes * n * p.piece * 2) : at;
  p.sum_at = grad ? take(n * p.dp * 4) : at;
  const int64_t piece = std::min(p.piece, v);
  p.dx_parts = parts_of(n, d, piece);
  p.dw_parts = parts_of(piece, d, n);
  p.parts_at = grad ? take(std::max(p.dx_parts > 1 ? p.dx_parts * n : 0,
                                    p.dw_parts > 1 ? p.dw_parts * piece : 0) * p.dp * 4)
                    : at;
  p.total = at;
  return p;
}

Rows rows_of(char *at, int64_t n) {
  const int64_t s = round_up(n, 64);
  int *p = reinterpret_cast<int *>(at + 256);
  return Rows{reinterpret_cast<int *>(at), p, p + s, p + 2 * s, reinterpret_cast<float *>(p + 3 * s),
              reinterpret_cast<float *>(p + 4 * s), reinterpret_cast<float *>(p + 5 * s), p + 6 * s,
              reinterpret_cast<int *>(at) + 1, reinterpret_cast<float *>(at) + 3};
}

void operand_rows(int64_t rows, int64_t cols, const __bf16 *x, int64_t ldx, const int *pos,
                  uint16_t *out, int64_t dp, int *, hipStream_t s, __bf16 *clear = nullptr,
                  int64_t ldc = 0) {
  const dim3 grid((unsigned)std::min<int64_t>((rows * (dp / 4) + 255) / 256, 8192));
  const bool vec = ldx % 4 == 0 && reinterpret_cast<uintptr_t>(x) % 8 == 0;
  const auto kernel = vec ? copy_kernel<true> : copy_kernel<false>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, (int)rows, (int)cols, x, ldx, pos, out, dp,
                     clear, ldc);
}
void operand_rows(int64_t rows, int64_t cols, const float *x, int64_t ldx, const int *pos,
                  uint16_t *out, int64_t dp, int *exp, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>((rows + 3) / 4, 4096));
  const bool vec = ldx % 4 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  const auto kernel = vec ? planes_kernel<true> : planes_kernel<false>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, (int)rows, (int)cols, x, ldx, pos, out, 2 * dp, exp);
}

struct Call {
  int64_t n, v, d;
  const void *x, *w;
  int64_t ldx, ldw;
  const int64_t *target;
  int64_t ignore;
  char *ws;
};

// Rows [v0, v0 + c) of W as an operand: in place where the kernels can read
// it (bf16, whole aligned granules of 8), else its copy or planes in the workspace.
template <class T, int P>
Operand weights(const Plan &p, const Call &c, int64_t v0, int64_t rows, bool in_place, hipStream_t s) {
  const T *w = static_cast<const T *>(c.w) + v0 * c.ldw;
  if (in_place) return Operand{reinterpret_cast<const uint16_t *>(w), c.ldw, 0};
  uint16_t *to = reinterpret_cast<uint16_t *>(c.ws + p.w_at);
  operand_rows(rows, c.d, w, c.ldw, nullptr, to, p.dp, reinterpret_cast<int *>(c.ws + p.wexp_at), s);
  return Operand{to, P * p.dp, 0};
}
template <class T>
bool readable(const Call &c) {
  return sizeof(T) == 2 && c.d % 8 == 0 && c.ldw % 8 == 0 &&
         reinterpret_cast<uintptr_t>(c.w) % 16 == 0;
}

// The matrix cores' elements: bf16 as given, fp32 as fp16 planes.
template <class T>
using Element = std::conditional_t<std::is_same_v<T, float>, _Float16, __bf16>;

template <class T>
int whole(const T *p, int64_t ld) {
  return ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0;
}

template <int N, bool VEC>
void few_forward(const Call &c, const Rows &r, float2 *part, int waves, hipStream_t s) {
  hipLaunchKernelGGL((few_logits_kernel<N, VEC>), dim3(waves / 4), dim3(256), 0, s, r, (int)c.n, c.v,
                     (int)c.d, static_cast<const float *>(c.x), c.ldx, static_cast<const float *>(c.w),
                     c.ldw, part);
}
// Whether four fp32 values of a row of X or W are one aligned load.
bool whole_loads(const Call &c) {
  return c.ldx % 4 == 0 && c.ldw % 4 == 0 && reinterpret_cast<uintptr_t>(c.x) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(c.w) % 16 == 0;
}
// f(N, VEC) for a call of few rows.
template <class F>
void few(const Call &c, F f) {
  const bool vec = whole_loads(c);
  auto by = [&](auto n) {
    if (vec) f(n, std::true_type());
    else f(n, std::false_type());
  };
  if (c.n <= 2) by(std::integral_constant<int, 2>());
  else if (c.n <= 4) by(std::integral_constant<int, 4>());
  else by(std::integral_constant<int, kFew>());
}
int few_waves(int64_t v) { return (int)std::min<int64_t>(kFewWaves, (v + 15) / 16 * 4); }

template <class T, int P>
void forward(const Plan &p, const Call &c, float *loss, float *lse, hipStream_t s) {
  const Rows r = rows_of(c.ws + p.rows_at, c.n);
  uint16_t *x = reinterpret_cast<uint16_t *>(c.ws + p.x_at);
  const int *wexp = reinterpret_cast<const int *>(c.ws + p.wexp_at);
  hipLaunchKernelGGL(rows_kernel, dim3(1), dim3(1024), 0, s, (int)c.n, c.v, c.target, c.ignore, r,
                     (const float *)nullptr, (const float *)nullptr, loss, lse);
  if (p.few) {
    float2 *part = reinterpret_cast<float2 *>(c.ws + p.part_at);
    const int waves = few_waves(c.v);
    few(c, [&](auto n, auto vec) { few_forward<n(), vec()>(c, r, part, waves, s); });
    hipLaunchKernelGGL(finish_kernel, dim3((unsigned)((c.n + 7) / 8)), dim3(256), 0, s, r, part,
                       (int)c.n, waves, loss, lse);
    return;
  }
  operand_rows(c.n, c.d, static_cast<const T *>(c.x), c.ldx, r.pos, x, p.dp, r.xexp, s);
  float2 *part = reinterpret_cast<float2 *>(c.ws + p.part_at);
  const bool in_place = readable<T>(c);
  // (a launch's tiles stay far below 2^32 threads)
  const int64_t piece = in_place ? std::max<int64_t>(256, (int64_t(1) << 36) / c.n / 256 * 256) : p.piece;
  int tiles = 0;
  for (int64_t v0 = 0; v0 < c.v; v0 += piece) {
    const int rows = (int)std::min(piece, c.v - v0);
    const Operand X{x, P * p.dp, 0}, W = weights<T, P>(p, c, v0, rows, in_place, s);
    tiles += product<Element<T>, P, false, false, Lse<P>>(
        Args{X, W, (int)c.n, rows, (int)c.d, r.count, 0, 0, 0, 0},
        LseArgs{part, r.target, r.zt, r.xexp, wexp, (int)c.n, (int)v0, tiles}, 1, s);
  }
  hipLaunchKernelGGL(finish_kernel, dim3((unsigned)((c.n + 7) / 8)), dim3(256), 0, s, r, part,
                     (int)c.n, tiles, loss, lse);
}

// A product with Out's epilogue, its k in `parts` parts (each a multiple of
// the stages' depth; `room` rows of a part have their place in the workspace).
template <class T, int P, bool TA>
void summed(Args g, int parts, OutArgs o, int64_t room, char *ws, hipStream_t s) {
  if (parts < 2) {
    product<Element<T>, P, TA, true, Out<T>>(g, o, 1, s);
    return;
  }
  float *from = reinterpret_cast<float *>(ws);
  g.k_split = (int)round_up((g.K + parts - 1) / parts, 64);
  const OutArgs part{from, o.lds, room * o.lds, 1, 0, nullptr, 0, 0, nullptr, o.most, o.weight,
                     o.scale};
  product<Element<T>, P, TA, true, Out<T>>(g, part, parts, s);
  const int64_t quads = (int64_t)g.M * ((g.N + 3) / 4);
  hipLaunchKernelGGL(join_kernel<T>, dim3((unsigned)std::min<int64_t>((quads + 255) / 256, 4096)),
                     dim3(256), 0, s, g.M, g.N, g.count_is_k ? nullptr : g.count, parts, from,
                     part.part, o.sum, o.lds, o.first, o.last, static_cast<T *>(o.out), o.ldo, o.whole,
                     o.row);
}

// The launches of the fp32 gradient's operands (see Sides).
void scan(const Plan &p, const Call &c, const Rows &r, float *dx, int64_t lddx, hipStream_t s) {
  auto blocks = [](int64_t rows) { return (int)std::min<int64_t>((rows + kScanWaves - 1) / kScanWaves, 256); };
  const Sides a{(int)c.n, (int)c.d, c.v, static_cast<const float *>(c.x), static_cast<const float *>(c.w), c.ldx,
                c.ldw, 2 * p.dp, r, reinterpret_cast<uint16_t *>(c.ws + p.x_at), nullptr, nullptr, dx, lddx,
                blocks(c.n)};
  const auto kernel = whole_loads(c) ? scan_kernel<true> : scan_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3(a.x_blocks + blocks(c.v)), dim3(64 * kScanWaves), 0, s, a);
}
Operand common(const Plan &p, const Call &c, const Rows &r, int64_t v0, int64_t rows, bool x, hipStream_t s) {
  auto blocks = [](int64_t rows) { return (int)std::min<int64_t>((rows + 3) / 4, 4096); };
  uint16_t *w = reinterpret_cast<uint16_t *>(c.ws + p.w_at);
  const Sides a{(int)c.n, (int)c.d, rows, static_cast<const float *>(c.x),
                static_cast<const float *>(c.w) + v0 * c.ldw, c.ldx, c.ldw, 2 * p.dp, r, nullptr,
                reinterpret_cast<uint16_t *>(c.ws + p.x2_at), w, nullptr, 0, x ? blocks(c.n) : 0};
  const auto kernel = whole_loads(c) ? common_kernel<true> : common_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3(a.x_blocks + blocks(rows)), dim3(256), 0, s, a);
  return Operand{w, a.ld, 0};
}

template <class T, int P>
void gradient(const Plan &p, const Call &c, const float *lse, const float *dloss, T *dx,
              int64_t lddx, T *dw, int64_t lddw, hipStream_t s) {
  const Rows r = rows_of(c.ws + p.rows_at, c.n);
  uint16_t *x = reinterpret_cast<uint16_t *>(c.ws + p.x_at);
  uint16_t *g = reinterpret_cast<uint16_t *>(c.ws + p.g_at);
  const int n = (int)c.n, d = (int)c.d;
  // X for the logits and for dW
  const Operand X{x, P * p.dp, 0}, G{g, P * p.piece, 0},
      X2{P == 2 ? reinterpret_cast<uint16_t *>(c.ws + p.x2_at) : x, P * p.dp, 0};
  // (n = 0 runs this too: it clears what the epilogues read)
  hipLaunchKernelGGL(rows_kernel, dim3(1), dim3(1024), 0, s, n, c.v, c.target, c.ignore, r, lse,
                     dloss, (float *)nullptr, (float *)nullptr);
  if (n > 0) {
    if constexpr (P == 2) scan(p, c, r, dx, lddx, s);
    else operand_rows(n, d, static_cast<const T *>(c.x), c.ldx, r.pos, x, p.dp, nullptr, s, dx, lddx);
  }
  const bool in_place = readable<T>(c);
  for (int64_t v0 = 0; v0 < c.v; v0 += p.piece) {
    const int rows = (int)std::min(p.piece, c.v - v0);
    if (n > 0) {
      Operand W;
      if constexpr (P == 2) W = common(p, c, r, v0, rows, v0 == 0 && dw, s);
      else W = weights<T, P>(p, c, v0, rows, in_place, s);
      product<Element<T>, P, false, false, Grad<P>>(
          Args{X, W, n, rows, d, r.count, 0, 0, 0, 0},
          GradArgs{g, P * p.piece, r.target, r.lse, r.dloss, r.scale, r.xexp, r.most + 1, (int)v0}, 1, s);
      if (dx)
        summed<T, P, false>(Args{G, W, n, d, rows, r.count, 0, 0, 0, 0}, p.dx_parts,
                            OutArgs{reinterpret_cast<float *>(c.ws + p.sum_at), p.dp, 0, v0 == 0,
                                    v0 + p.piece >= c.v, dx, lddx, whole(dx, lddx), r.row, r.most + 1, r.dloss,
                                    r.scale},
                            n, c.ws + p.parts_at, s);
    }
    if (dw)
      summed<T, P, true>(Args{G, X2, rows, d, n, r.count, 1, 0, 0, 0}, p.dw_parts,
                         OutArgs{nullptr, p.dp, 0, 1, 1, dw + v0 * lddw, lddw, whole(dw, lddw), nullptr,
                                 r.most, nullptr, r.scale},
                         std::min(p.piece, c.v), c.ws + p.parts_at, s);
  }
}

og_status check_sizes(int64_t n, int64_t v, int64_t d, int type) {
  using og::host::fail;
  if (type != OG_F32 && type != OG_BF16)
    return fail(OG_ERR_INVALID_ARG, "type %d: linear_cross_entropy takes OG_F32 or OG_BF16", type);
  if (n < 0 || v < 1 || d < 1)
    return fail(OG_ERR_INVALID_ARG, "n %lld must be >= 0, v %lld and d %lld >= 1", (long long)n,
                (long long)v, (long long)d);
  if (n > (1 << 24) || v > (1 << 28) || d > (1 << 18))
    return fail(OG_ERR_TOO_LARGE, "n %lld, v %lld, d %lld: at most 2^24, 2^28 and 2^18",
                (long long)n, (long long)v, (long long)d);
  return OG_OK;
}

og_status check(const Call &c, int type, int64_t workspace_bytes, bool grad, Plan &p) {
  using og::host::fail;
  if (c.ldx < c.d || c.ldw < c.d)
    return fail(OG_ERR_INVALID_ARG, "ldx %lld or ldw %lld below d %lld", (long long)c.ldx,
                (long long)c.ldw, (long long)c.d);
  if (c.ldw > (1 << 22))
    return fail(OG_ERR_TOO_LARGE, "ldw %lld: at most 2^22", (long long)c.ldw);
  if (c.n > 0 && (!c.x || !c.w || !c.target))
    return fail(OG_ERR_INVALID_ARG, "X, W or target is null");
  p = plan(c.n, c.v, c.d, type, grad);
  if (!c.ws || workspace_bytes < p.total)
    return fail(OG_ERR_INVALID_ARG, "workspace of %lld bytes: %lld needed",
                (long long)(c.ws ? workspace_bytes : 0), (long long)p.total);
  if (reinterpret_cast<uintptr_t>(c.ws) % 256)
    return fail(OG_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return OG_OK;
}

}  // namespace og::lce

extern "C" {

int64_t og_linear_cross_entropy_workspace(int64_t n, int64_t v, int64_t d, int type, int grad) {
  const og_status st = og::lce::check_sizes(n, v, d, type);
  if (st != OG_OK) return st;
  og::host::ok();
  return og::lce::plan(n, v, d, type, grad != 0).total;
}

og_status og_linear_cross_entropy(int64_t n, int64_t v, int64_t d, const void *X, int64_t ldx,
                                  const void *W, int64_t ldw, int type, const int64_t *target,
                                  int64_t ignore_index, float *loss, float *lse, void *workspace,
                                  int64_t workspace_bytes) {
  using namespace og::host;
  og_status st = og::lce::check_sizes(n, v, d, type);
  if (st != OG_OK) return st;
  const og::lce::Call c{n, v, d, X, W, ldx, ldw, target, ignore_index, static_cast<char *>(workspace)};
  og::lce::Plan p;
  if ((st = og::lce::check(c, type, workspace_bytes, false, p)) != OG_OK) return st;
  if (n == 0) return ok();
  if (!loss || !lse) return fail(OG_ERR_INVALID_ARG, "loss or lse is null");
  if ((st = check_device()) != OG_OK) return st;
  if (type == OG_F32)
    og::lce::forward<float, 2>(p, c, loss, lse, current_stream());
  else
    og::lce::forward<__bf16, 1>(p, c, loss, lse, current_stream());
  return check_launch("linear_cross_entropy");
}

og_status og_linear_cross_entropy_grad(int64_t n, int64_t v, int64_t d, const void *X, int64_t ldx,
                                       const void *W, int64_t ldw, int type, const int64_t *target,
                                       int64_t ignore_index, const float *lse, const float *dloss,
                                       void *dX, int64_t lddx, void *dW, int64_t lddw,
                                       void *workspace, int64_t workspace_bytes) {
  using namespace og::host;
  og_status st = og::lce::check_sizes(n, v, d, type);
  if (st != OG_OK) return st;
  const og::lce::Call c{n, v, d, X, W, ldx, ldw, target, ignore_index, static_cast<char *>(workspace)};
  og::lce::Plan p;
  if ((st = og::lce::check(c, type, workspace_bytes, true, p)) != OG_OK) return st;
  if ((dX && lddx < d) || (dW && lddw < d))
    return fail(OG_ERR_INVALID_ARG, "lddx %lld or lddw %lld below d %lld", (long long)lddx,
                (long long)lddw, (long long)d);
  if (n > 0 && (!lse || !dloss)) return fail(OG_ERR_INVALID_ARG, "lse or dloss is null");
  if ((n == 0 && !dW) || (!dX && !dW)) return ok();
  if ((st = check_device()) != OG_OK) return st;
  if (type == OG_F32)
    og::lce::gradient<float, 2>(p, c, lse, dloss, static_cast<float *>(dX), lddx,
                                static_cast<float *>(dW), lddw, current_stream());
  else
    og::lce::gradient<__bf16, 1>(p, c, lse, dloss, static_cast<__bf16 *>(dX), lddx,
                                 static_cast<__bf16 *>(dW), lddw, current_stream());
  return check_launch("linear_cross_entropy_grad");
}

}  // extern "C"
