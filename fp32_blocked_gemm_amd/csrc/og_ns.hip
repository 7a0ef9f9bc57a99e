// og_ns.hip -- og_newton_schulz: the orthogonalised update of a matrix by
// Newton-Schulz products.
//
//   X = G / (|G| + eps)   (the Frobenius norm; the shorter side as rows, r <= k)
//   each step:  A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// Every product runs on the fp16 matrix cores (og_tile.hpp).  X is kept as two
// fp16 planes (22 bits).  For fp32 input all products take both planes, and A
// and B have two.  For bf16 input (of more than kNarrow rows) they take the
// first plane, and A and B have one (11 bits): an error of A or B enters X through B X, whose entries the
// polynomial's own slope lifts little, and stays a third of the result's own
// rounding to bf16, while X itself in 11 bits would not do: the slope of up to
// a per step lifts its rounding by a^steps, 484 at the usual coefficients, in
// the directions it stretches most (hence X's second plane, which enters
// through a X).
//
// Each matrix is stored times a power of two that its largest possible value
// sets: the singular values of X stay below s (at first the power of two from
// |G| / (|G| + eps) on, 1 where eps is small, then the largest |p| over [0, s]),
// those of A below s^2 and those of B below the largest |b x^2 + c x^4|.  The
// first s is known on the device only, and with it the others (pack_kernel).
//
// A and A A are symmetric: only the tiles on and below the diagonal are
// computed and each is stored to both places, a quarter of the step's work at
// r = k.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "og.h"
#include "og_host.hpp"
#include "og_tile.hpp"

namespace og::ns {

using namespace og::tile;

// Up to this many rows bf16 input runs like fp32: the error of one plane shows
// against a result whose norm is sqrt(r) (measured over the plain chain's:
// 1.5 times at 33 rows, 1.2 at 777, 1.02 at 4096), and costs no time there.
constexpr int kNarrow = 256;
constexpr int kNormBlocks = 1024;  // partial sums of squares per matrix

// X: two planes, interleaved where the products take both (P = 2), one after
// the other where they take the first (P = 1).
template <int P>
struct Wide {
  uint16_t *p;
  int64_t ld, batch, plane;
  int width;  // columns of a row, padding included
  __device__ __forceinline__ uint16_t *at(int m, int r, int c, int q) const {
    return p + m * batch + r * ld + (P == 2 ? column<2>(c, q) : c + q * plane);
  }
  __device__ __forceinline__ f32x4 load(int m, int r, int c) const {
    const f16x4 h = *reinterpret_cast<const f16x4 *>(at(m, r, c, 0));
    const f16x4 l = *reinterpret_cast<const f16x4 *>(at(m, r, c, 1));
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)h[e] + (float)l[e];
    return v;
  }
  __device__ __forceinline__ void store(int m, int r, int c, const f32x4 v) const {
    f16x4 h, l;
    split4(v, h, l);
    *reinterpret_cast<f16x4 *>(at(m, r, c, 0)) = h;
    *reinterpret_cast<f16x4 *>(at(m, r, c, 1)) = l;
  }
};

struct Input {
  const void *g;
  int64_t ld, batch;
  int m, n;  // of G
};

// Partial sums of squares of G, in 64 bits (no square of an fp32 value
// overflows there): a block takes every gridDim.x-th row, eight sums a lane in
// flight.  One pass over G: bound by its bytes (4096 x 11008 bf16 in 27 us).
template <class T>
__global__ __launch_bounds__(256) void norm_kernel(Input in, double *part) {
  const int batch = blockIdx.y;
  double s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const T *g = static_cast<const T *>(in.g) + batch * in.batch;
  for (int row = blockIdx.x; row < in.m; row += gridDim.x) {
    const T *r = g + row * in.ld;
    int c = threadIdx.x;
    for (; c + 7 * 256 < in.n; c += 8 * 256) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = (float)r[c + q * 256];
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += (double)v[q] * v[q];
    }
    for (; c < in.n; c += 256) {
      const double v = (float)r[c];
      s[0] += v * v;
    }
  }
  __shared__ double sum[256];
  sum[threadIdx.x] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if (threadIdx.x < h) sum[threadIdx.x] += sum[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) part[batch * kNormBlocks + blockIdx.x] = sum[0];
}

// The polynomial a x + b x^3 + c x^5 of a step, and b x^2 + c x^4 of B, with their extreme values
// besides those at the ends: the squares of their places and the values there (place 0: none).
struct Poly {
  double a, b, c;
  double next_at[2], next_top[2], factor_at, factor_top;
  __host__ __device__ double p(double x) const { return fabs((a + (b + c * x * x) * x * x) * x); }
  __host__ __device__ double f(double square) const { return fabs((b + c * square) * square); }
  // The largest over [0, s]; a hundredth more is for the roundings.
  __host__ __device__ double largest_next(double s) const {
    double top = p(s);
    for (int i = 0; i < 2; ++i)
      if (next_at[i] > 0 && next_at[i] < s * s && next_top[i] > top) top = next_top[i];
    return top * 1.01;
  }
  __host__ __device__ double largest_factor(double s) const {
    const double top = f(s * s);
    return (factor_at > 0 && factor_at < s * s && factor_top > top ? factor_top : top) * 1.01;
  }
};
Poly poly(double a, double b, double c) {
  Poly p{a, b, c, {0, 0}, {0, 0}, 0, 0};
  // where the derivative, a quadratic in x^2, is zero
  const double d = 9 * b * b - 20 * a * c;
  if (c == 0) {
    if (b != 0) p.next_at[0] = -a / (3 * b);
  } else if (d >= 0) {
    p.next_at[0] = (-3 * b + std::sqrt(d)) / (10 * c);
    p.next_at[1] = (-3 * b - std::sqrt(d)) / (10 * c);
  }
  for (int i = 0; i < 2; ++i)
    if (p.next_at[i] > 0) p.next_top[i] = p.p(std::sqrt(p.next_at[i]));
  if (c != 0) p.factor_at = -b / (2 * c);
  p.factor_top = p.f(p.factor_at);
  return p;
}

// The exponent that brings values up to `bound` to 2^14 (a quarter of fp16's
// range: the bound is exact arithmetic's).
__device__ __forceinline__ int exponent(double bound, int most) {
  int e = 0;
  if (bound > 0 && bound < HUGE_VAL) frexp(bound, &e);
  return min(most, max(-60, 14 - e));
}
// Of X: values below 2^-144 vanish, as they do in fp32.
constexpr int kMostX = 120;

constexpr int kMaxSteps = 64;
// What the epilogues of a step multiply by, (a, c) of each of its three products.
struct Factors {
  float2 of[kMaxSteps][3];
};
// X's singular values are at most 2^q at first, its planes times 2^ex.
__device__ void factors(const Poly &p, int q, int ex, int steps, Factors &to) {
  double top = ldexp(1.0, q);
  for (int i = 0; i < steps; ++i) {
    const int ea = exponent(top * top, 400), eb = exponent(p.largest_factor(top), 800);
    const double next = p.largest_next(top);
    const int en = i + 1 == steps ? 0 : exponent(next, kMostX);
    to.of[i][0] = {0.0f, (float)ldexp(1.0, ea - 2 * ex)};
    to.of[i][1] = {(float)ldexp(p.b, eb - ea), (float)ldexp(p.c, eb - 2 * ea)};
    to.of[i][2] = {(float)ldexp(p.a, en - ex), (float)ldexp(1.0, en - eb - ex)};
    top = next;
    ex = en;
  }
}

// X's planes from G: 64 x 64 tiles through LDS (G is read along its rows
// whichever way X lies), padded with zeros to a multiple of 64 columns.  One thread
// of a matrix's first block writes the factors of all steps.  Bound by the bytes of
// both planes: 4096 x 11008 bf16 (270 MB) in 88 us.
template <class T, int P, bool TALL>
__global__ __launch_bounds__(256) void pack_kernel(Input in, const double *part, int blocks,
                                                   float eps, Poly poly, int steps, Factors *out,
                                                   Wide<P> x) {
  __shared__ float tile[64][65];
  __shared__ double factor;
  const int batch = blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int R = TALL ? in.n : in.m;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const T *g = static_cast<const T *>(in.g) + batch * in.batch;
  float v[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    // row i of G's part of the tile
    const int i = w + 4 * q, row = (TALL ? c0 : r0) + i, col = (TALL ? r0 : c0) + lane;
    v[q] = row < in.m && col < in.n ? (float)g[row * in.ld + col] : 0.0f;
  }
  if (threadIdx.x < 64) {
    double s = 0;
    for (int i = threadIdx.x; i < blocks; i += 64) s += part[batch * kNormBlocks + i];
    for (int h = 32; h > 0; h >>= 1) s += __shfl_xor(s, h);
    if (threadIdx.x == 0) {
      const double norm = sqrt(s), size = norm / (norm + (double)eps);
      int q = 0;  // (a matrix of zeros or one that is not finite is so with any power)
      if (size > 0 && size < 1 && frexp(size, &q) == 0.5) --q;
      const int ex = min(13 - q, kMostX);
      factor = ldexp(1.0, ex) / (norm + (double)eps);
      if (blockIdx.x == 0 && blockIdx.y == 0) factors(poly, q, ex, steps, out[batch]);
    }
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    if (TALL) tile[lane][w + 4 * q] = v[q];
    else tile[w + 4 * q][lane] = v[q];
  }
  __syncthreads();
  const double f = factor;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int at = threadIdx.x + 256 * q, i = at >> 4, j = (at & 15) * 4;
    if (r0 + i >= R) continue;
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (float)(tile[i][j + e] * f);
    x.store(batch, r0 + i, c0 + j, y);
  }
}

// A or B: P planes of an r x r matrix.
template <int P>
struct Square {
  uint16_t *p;
  int64_t ld, batch;
  __device__ __forceinline__ f32x4 load(int m, int r, int c) const {
    const uint16_t *row = p + m * batch + r * ld;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int q = P - 1; q >= 0; --q) {
      const f16x4 h = *reinterpret_cast<const f16x4 *>(row + column<P>(c, q));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += (float)h[e];
    }
    return v;
  }
  // four columns of a row; their mirror, four rows of a column (each where flagged)
  __device__ __forceinline__ void store(int m, int r, int c, const f32x4 v, bool row, bool mirror,
                                        int n) const {
    f16x4 h[2];
    split4(v, h[0], h[1]);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      if (row) *reinterpret_cast<f16x4 *>(p + m * batch + r * ld + column<P>(c, q)) = h[q];
      if (mirror)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < n)
            reinterpret_cast<_Float16 *>(p)[m * batch + (c + e) * ld + column<P>(r, q)] = h[q][e];
    }
  }
};

// Epilogue of the symmetric products: out = was a + acc c; each tile below
// the diagonal is stored to its mirror too (straight from the registers:
// through LDS, as whole rows, it took 36 us where this takes 33; without the mirror
// an update of 4096 x 11008 takes 3320 us for 3476, of 12 x 768 x 768 fp32 534 for
// 571).  Bound by the matrix cores for large matrices (4096 x 11008: A 184 GFLOP and
// A A 69 in 255 us together, 994 TFLOP/s), by the number of tiles for small ones
// (777 x 1531 8 us each, 128 x 512 6), in between by both and the epilogue, which
// nothing overlaps with one block a compute unit (12 of 768 x 768 fp32: 31 us, of which
// the 24 stages of its 252 tiles are 16).
template <int P>
struct SymArgs {
  Square<P> out, was;  // was.p null: acc c alone
  const Factors *by;   // by matrix
  int step, product;   // by->of[step][product]: a and c
};
template <int P>
struct Sym {
  using Args = SymArgs<P>;
  static constexpr bool kSymmetric = true;
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t,
                                               const Args &e) {
    const int mr = t.m0 + (t.lane & 15), nc = t.n0 + 4 * (t.lane >> 4);
    const int width = (int)(e.out.ld / P);
    const float2 by = e.by[t.batch].of[e.step][e.product];
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = mr + 16 * i;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int n = nc + 16 * j;
        const bool in = m < t.M && n < width;
        f32x4 v = {0, 0, 0, 0};
        if (e.was.p && in) v = e.was.load(t.batch, m, n);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[q] = m < t.M && n + q < t.N ? fmaf(by.y, acc[i][j][q], by.x * v[q]) : 0.0f;
        e.out.store(t.batch, m, n, v, in, t.tile_m != t.tile_n && m < width, t.N);
      }
    }
  }
};

// Epilogue of X <- a X + B X: out = x a + acc c, the next step's X, or the
// result in its own type and orientation.  4096 x 11008: 430 us, 859 TFLOP/s, of
// which X's planes, read and written (360 MB), are 80 us at the rate of a copy;
// 12 of 768 x 768 fp32 52 us.
template <int P>
struct NextArgs {
  Wide<P> x, out;
  const Factors *by;  // by->of[step][2]: a and c
  int step;
  void *o;  // the result, after the last step; else null
  int64_t ldo, batch_o;
  int tall;   // the result is X's transpose
  int whole;  // it is not, and four of its values are one aligned store
};
template <int P, class T>
struct Next {
  using Args = NextArgs<P>;
  static constexpr bool kSymmetric = false;
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t,
                                               const Args &e) {
    const int mr = t.m0 + (t.lane & 15), nc = t.n0 + 4 * (t.lane >> 4);
    const float2 by = e.by[t.batch].of[e.step][2];
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = mr + 16 * i;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int n = nc + 16 * j;
        if (m >= t.M || n >= e.x.width) continue;
        f32x4 v = e.x.load(t.batch, m, n);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = n + q < t.N ? fmaf(by.y, acc[i][j][q], by.x * v[q]) : 0.0f;
        if (!e.o) {
          e.out.store(t.batch, m, n, v);
        } else {
          typedef T T4 __attribute__((ext_vector_type(4)));
          T *o = static_cast<T *>(e.o) + t.batch * e.batch_o;
          T4 y;
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = (T)v[q];
          if (e.whole && n + 3 < t.N) {
            *reinterpret_cast<T4 *>(o + (int64_t)m * e.ldo + n) = y;
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + q < t.N) o[e.tall ? (int64_t)(n + q) * e.ldo + m : (int64_t)m * e.ldo + n + q] = y[q];
          }
        }
      }
    }
  }
};

struct Plan {
  int r, k, planes;                      // planes of A, B and of the products' operands
  int64_t rp, kp;                        // r and k padded to blocks of 64
  int64_t x_bytes, a_bytes, norm_bytes, factor_bytes;  // of one buffer, over the batch
  int64_t total() const { return norm_bytes + factor_bytes + 2 * x_bytes + 2 * a_bytes; }
};

Plan plan(int64_t batch, int64_t m, int64_t n, int type) {
  Plan p;
  p.r = (int)std::min(m, n);
  p.k = (int)std::max(m, n);
  p.planes = type == OG_F32 || p.r <= kNarrow ? 2 : 1;
  p.rp = round_up(p.r, 64);
  p.kp = round_up(p.k, 64);
  p.x_bytes = round_up(batch * 2 * p.r * p.kp * 2, 256);
  p.a_bytes = round_up(batch * p.planes * p.r * p.rp * 2, 256);
  p.norm_bytes = round_up(batch * kNormBlocks * 8, 256);
  p.factor_bytes = round_up(batch * (int64_t)sizeof(Factors), 256);
  return p;
}

// Whether every matrix has its power of two: the bounds of X before each step
// within [2^-23, 2^37] (or zero) where it starts at 1, so that A's stay within the
// exponents above, and those of B below 2^74.
bool in_range(int steps, const Poly &p) {
  double top = 1;
  for (int i = 0; i < steps; ++i) {
    if (top != 0 && !(top >= std::ldexp(1.0, -23) && top <= std::ldexp(1.0, 37))) return false;
    if (!(p.largest_factor(top) <= std::ldexp(1.0, 74))) return false;
    top = p.largest_next(top);
  }
  return true;
}

template <class T, int P>
void run(const Plan &p, const Input &in, int batch, int steps, const Poly &poly, float eps, void *o,
         int64_t ldo, int64_t stride_o, char *ws, hipStream_t s) {
  double *norm = reinterpret_cast<double *>(ws);
  Factors *by = reinterpret_cast<Factors *>(ws + p.norm_bytes);
  char *planes = ws + p.norm_bytes + p.factor_bytes;
  const bool tall = in.m > in.n;
  const bool whole = !tall && ldo % 4 == 0 && stride_o % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(o) % (4 * sizeof(T)) == 0;
  const int64_t lda = P * p.rp, ab = p.r * lda;
  Wide<P> x[2];
  for (int i = 0; i < 2; ++i) {
    x[i].p = reinterpret_cast<uint16_t *>(planes + i * p.x_bytes);
    x[i].ld = P * p.kp;
    x[i].batch = p.r * x[i].ld;
    x[i].plane = batch * x[i].batch;
    x[i].width = (int)p.kp;
  }
  Square<P> A{reinterpret_cast<uint16_t *>(planes + 2 * p.x_bytes), lda, ab};
  Square<P> B{reinterpret_cast<uint16_t *>(planes + 2 * p.x_bytes + p.a_bytes), lda, ab};
  const int blocks = std::min(kNormBlocks, in.m);
  hipLaunchKernelGGL(norm_kernel<T>, dim3(blocks, batch), dim3(256), 0, s, in, norm);
  const dim3 grid((unsigned)(p.kp / 64), (unsigned)(p.rp / 64), batch);
  const auto pack = tall ? pack_kernel<T, P, true> : pack_kernel<T, P, false>;
  hipLaunchKernelGGL(pack, grid, dim3(256), 0, s, in, norm, blocks, eps, poly, steps, by, x[0]);
  for (int i = 0; i < steps; ++i) {
    const Wide<P> &from = x[i & 1], &to = x[(i + 1) & 1];
    const Operand X{from.p, from.ld, from.batch}, OA{A.p, lda, ab}, OB{B.p, lda, ab};
    product<_Float16, P, false, false, Sym<P>>(Args{X, X, p.r, p.r, p.k, nullptr, 0, 0, 0, 0},
                                               SymArgs<P>{A, Square<P>{nullptr, 0, 0}, by, i, 0}, batch, s);
    product<_Float16, P, false, false, Sym<P>>(Args{OA, OA, p.r, p.r, p.r, nullptr, 0, 0, 0, 0},
                                               SymArgs<P>{B, A, by, i, 1}, batch, s);
    product<_Float16, P, false, true, Next<P, T>>(
        Args{OB, X, p.r, p.k, p.r, nullptr, 0, 0, 0, 0},
        NextArgs<P>{from, to, by, i, i + 1 == steps ? o : nullptr, ldo, stride_o, tall, whole}, batch, s);
  }
}

og_status check_sizes(int64_t batch, int64_t m, int64_t n, int type) {
  using og::host::fail;
  if (type != OG_F32 && type != OG_BF16)
    return fail(OG_ERR_INVALID_ARG, "type %d: newton_schulz takes OG_F32 or OG_BF16", type);
  if (batch < 0 || m < 0 || n < 0)
    return fail(OG_ERR_INVALID_ARG, "negative size: batch %lld, %lld x %lld", (long long)batch,
                (long long)m, (long long)n);
  if (m > (1 << 18) || n > (1 << 18) || batch > 65535)
    return fail(OG_ERR_TOO_LARGE, "batch %lld of %lld x %lld: at most 65535 of 2^18 x 2^18",
                (long long)batch, (long long)m, (long long)n);
  return OG_OK;
}

}  // namespace og::ns

extern "C" {

int64_t og_newton_schulz_workspace(int64_t batch, int64_t m, int64_t n, int type) {
  const og_status st = og::ns::check_sizes(batch, m, n, type);
  if (st != OG_OK) return st;
  og::host::ok();
  if (batch == 0 || m == 0 || n == 0) return 0;
  return og::ns::plan(batch, m, n, type).total();
}

og_status og_newton_schulz(int64_t batch, int64_t m, int64_t n, const void *G, int64_t ldg,
                           int64_t strideg, int type, int steps, float a, float b, float c,
                           float eps, void *O, int64_t ldo, int64_t strideo, void *workspace,
                           int64_t workspace_bytes) {
  using namespace og::host;
  og_status st = og::ns::check_sizes(batch, m, n, type);
  if (st != OG_OK) return st;
  if (steps < 1 || steps > og::ns::kMaxSteps) return fail(OG_ERR_INVALID_ARG, "steps %d: 1 to 64", steps);
  if (!(eps >= 0) || !std::isfinite(eps) || !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
    return fail(OG_ERR_INVALID_ARG, "eps must be finite and not negative, a, b and c finite");
  const og::ns::Poly poly = og::ns::poly(a, b, c);
  if (!og::ns::in_range(steps, poly))
    return fail(OG_ERR_INVALID_ARG, "coefficients that may bring X's singular values out of "
                "[2^-23, 2^37] before the last step, or b A + c A A past 2^74");
  if (ldg < std::max<int64_t>(1, n) || ldo < std::max<int64_t>(1, n))
    return fail(OG_ERR_INVALID_ARG, "ldg %lld or ldo %lld below n %lld", (long long)ldg,
                (long long)ldo, (long long)n);
  if (batch > 1 && m > 0 && (strideg < 0 || strideo < (m - 1) * ldo + n))
    return fail(OG_ERR_INVALID_ARG, "strides %lld and %lld: inputs may repeat, outputs not overlap",
                (long long)strideg, (long long)strideo);
  if (batch == 0 || m == 0 || n == 0) return ok();
  if (!G || !O) return fail(OG_ERR_INVALID_ARG, "null matrix");
  const og::ns::Plan p = og::ns::plan(batch, m, n, type);
  if (!workspace || workspace_bytes < p.total())
    return fail(OG_ERR_INVALID_ARG, "workspace of %lld bytes: %lld needed",
                (long long)(workspace ? workspace_bytes : 0), (long long)p.total());
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(OG_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if ((st = check_device()) != OG_OK) return st;
  const og::ns::Input in{G, ldg, strideg, (int)m, (int)n};
  if (type == OG_F32)
    og::ns::run<float, 2>(p, in, (int)batch, steps, poly, eps, O, ldo, strideo,
                          static_cast<char *>(workspace), current_stream());
  else if (p.planes == 2)
    og::ns::run<__bf16, 2>(p, in, (int)batch, steps, poly, eps, O, ldo, strideo,
                           static_cast<char *>(workspace), current_stream());
  else
    og::ns::run<__bf16, 1>(p, in, (int)batch, steps, poly, eps, O, ldo, strideo,
                           static_cast<char *>(workspace), current_stream());
  return check_launch("newton_schulz");
}

}  // extern "C"
