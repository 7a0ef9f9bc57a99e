// og_ns.hip -- og_newton_schulz_f32 / _bf16: the orthogonalised update of a
// matrix by Newton-Schulz products.
//
//   X = G / (|G| + eps)   (the Frobenius norm; the shorter side as rows, r <= k)
//   each step:  A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// Every product runs on the bf16 matrix cores with its operands in planes
// (og_tile.hpp): three planes for fp32 input (fp32 accuracy), two for bf16
// input (16 bits: the polynomial's slope of up to a per step lifts a rounding
// of X by a^steps, 484 at the usual coefficients, in the directions it
// stretches most, so that X held in 8 bits, as one plane, would lose the
// result's last bits; 16 bits keep the error two hundred times below the
// rounding of the output).  A and A A are symmetric: only the tiles on and
// below the diagonal are computed and each is stored to both places, a
// quarter of the step's work at r = k.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "og.h"
#include "og_host.hpp"
#include "og_tile.hpp"

namespace og::ns {

using namespace og::tile;

constexpr int kNormBlocks = 1024;  // partial sums of squares per matrix

struct Input {
  const void *g;
  int64_t ld, batch;
  int m, n;  // of G
};

// Partial sums of squares of G, in 64 bits (no square of an fp32 value
// overflows there): a block takes every gridDim.x-th row, eight sums a lane in
// flight.  One pass over G: bound by its bytes.
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

// X's planes from G: 64 x 64 tiles through LDS (G is read along its rows
// whichever way X lies), padded with zeros to a multiple of 64 columns.
template <class T, int P, bool TALL>
__global__ __launch_bounds__(256) void pack_kernel(Input in, const double *part, int blocks,
                                                   float eps, uint16_t *x, int64_t ld) {
  __shared__ float tile[64][65];
  __shared__ float factor;
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
    if (threadIdx.x == 0) factor = (float)(1.0 / ((double)(float)sqrt(s) + (double)eps));
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    if (TALL) tile[lane][w + 4 * q] = v[q];
    else tile[w + 4 * q][lane] = v[q];
  }
  __syncthreads();
  const float f = factor;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int at = threadIdx.x + 256 * q, i = at >> 4, j = (at & 15) * 4;
    if (r0 + i >= R) continue;
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = tile[i][j + e] * f;
    bf16x4 out[P];
    split4<P>(y, out);
    uint16_t *to = x + (batch * (int64_t)R + r0 + i) * ld;
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x4 *>(to + column<P>(c0 + j, p)) = out[p];
  }
}

template <int P>
__device__ __forceinline__ f32x4 load_planes(const uint16_t *row, int c) {
  f32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int q = P - 1; q >= 0; --q) {
    const bf16x4 h = *reinterpret_cast<const bf16x4 *>(row + column<P>(c, q));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += (float)h[e];
  }
  return v;
}

// Epilogue of the symmetric products: A = acc, or B = b A + c acc; each
// tile below the diagonal is stored to its mirror too.
struct SymArgs {
  uint16_t *out;
  const uint16_t *a;  // null: store acc itself
  int64_t ld, batch;
  float b, c;
};
template <int P>
struct Sym {
  using Args = SymArgs;
  static constexpr bool kSymmetric = true;
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t,
                                               const Args &e) {
    uint16_t *out = e.out + t.batch * e.batch;
    const uint16_t *a = e.a ? e.a + t.batch * e.batch : nullptr;
    const int mr = t.m0 + (t.lane & 15), nc = t.n0 + 4 * (t.lane >> 4);
    const int width = (int)(e.ld / P);
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = mr + 16 * i;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int n = nc + 16 * j;
        f32x4 v = acc[i][j];
        if (a && m < t.M && n < width) {
          const f32x4 was = load_planes<P>(a + (int64_t)m * e.ld, n);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = fmaf(e.c, v[q], e.b * was[q]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (m >= t.M || n + q >= t.N) v[q] = 0;
        bf16x4 h[P];
        split4<P>(v, h);
        if (m < t.M && n < width) {
#pragma unroll
          for (int p = 0; p < P; ++p)
            *reinterpret_cast<bf16x4 *>(out + (int64_t)m * e.ld + column<P>(n, p)) = h[p];
        }
        if (t.tile_m != t.tile_n && m < width) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < t.N) {
#pragma unroll
              for (int p = 0; p < P; ++p)
                reinterpret_cast<__bf16 *>(out)[(int64_t)(n + q) * e.ld + column<P>(m, p)] = h[p][q];
            }
        }
      }
    }
  }
};

// Epilogue of X <- a X + B X: planes of the next step's X, or the result in
// its own type and orientation.
struct NextArgs {
  const uint16_t *x;
  uint16_t *out;  // null after the last step
  int64_t ld, batch;
  float a;
  void *o;
  int64_t ldo, batch_o;
  int tall;
};
template <int P, class T>
struct Next {
  using Args = NextArgs;
  static constexpr bool kSymmetric = false;
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t,
                                               const Args &e) {
    const uint16_t *x = e.x + t.batch * e.batch;
    const int mr = t.m0 + (t.lane & 15), nc = t.n0 + 4 * (t.lane >> 4);
    const int width = (int)(e.ld / P);
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = mr + 16 * i;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int n = nc + 16 * j;
        if (m >= t.M || n >= width) continue;
        f32x4 v = load_planes<P>(x + (int64_t)m * e.ld, n);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = n + q < t.N ? fmaf(e.a, v[q], acc[i][j][q]) : 0.0f;
        if (e.out) {
          bf16x4 h[P];
          split4<P>(v, h);
          uint16_t *to = e.out + t.batch * e.batch + (int64_t)m * e.ld;
#pragma unroll
          for (int p = 0; p < P; ++p) *reinterpret_cast<bf16x4 *>(to + column<P>(n, p)) = h[p];
        } else {
          T *o = static_cast<T *>(e.o) + t.batch * e.batch_o;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < t.N) o[e.tall ? (int64_t)(n + q) * e.ldo + m : (int64_t)m * e.ldo + n + q] = (T)v[q];
        }
      }
    }
  }
};

struct Plan {
  int r, k, planes;
  int64_t rp, kp;                         // r and k padded to blocks of 64
  int64_t x_bytes, a_bytes, norm_bytes;   // of one buffer, over the batch
  int64_t total() const { return norm_bytes + 2 * x_bytes + 2 * a_bytes; }
};

Plan plan(int64_t batch, int64_t m, int64_t n, int type) {
  Plan p;
  p.r = (int)std::min(m, n);
  p.k = (int)std::max(m, n);
  p.planes = type == OG_F32 ? 3 : 2;
  p.rp = round_up(p.r, 64);
  p.kp = round_up(p.k, 64);
  p.x_bytes = round_up(batch * p.planes * p.r * p.kp * 2, 256);
  p.a_bytes = round_up(batch * p.planes * p.r * p.rp * 2, 256);
  p.norm_bytes = round_up(batch * kNormBlocks * 8, 256);
  return p;
}

template <class T, int P>
void run(const Plan &p, const Input &in, int batch, int steps, float a, float b, float c, float eps,
         void *o, int64_t ldo, int64_t stride_o, char *ws, hipStream_t s) {
  double *norm = reinterpret_cast<double *>(ws);
  uint16_t *x[2] = {reinterpret_cast<uint16_t *>(ws + p.norm_bytes),
                    reinterpret_cast<uint16_t *>(ws + p.norm_bytes + p.x_bytes)};
  uint16_t *A = reinterpret_cast<uint16_t *>(ws + p.norm_bytes + 2 * p.x_bytes);
  uint16_t *B = reinterpret_cast<uint16_t *>(ws + p.norm_bytes + 2 * p.x_bytes + p.a_bytes);
  const bool tall = in.m > in.n;
  const int blocks = std::min(kNormBlocks, in.m);
  hipLaunchKernelGGL(norm_kernel<T>, dim3(blocks, batch), dim3(256), 0, s, in, norm);
  const dim3 grid((unsigned)(p.kp / 64), (unsigned)(p.rp / 64), batch);
  if (tall)
    hipLaunchKernelGGL((pack_kernel<T, P, true>), grid, dim3(256), 0, s, in, norm, blocks, eps,
                       x[0], P * p.kp);
  else
    hipLaunchKernelGGL((pack_kernel<T, P, false>), grid, dim3(256), 0, s, in, norm, blocks, eps,
                       x[0], P * p.kp);
  const int64_t ldx = P * p.kp, lda = P * p.rp, xb = p.r * ldx, ab = p.r * lda;
  for (int i = 0; i < steps; ++i) {
    uint16_t *from = x[i & 1], *to = i + 1 < steps ? x[(i + 1) & 1] : nullptr;
    const Operand X{from, ldx, xb}, OA{A, lda, ab}, OB{B, lda, ab};
    product<P, false, false, Sym<P>>(Args{X, X, p.r, p.r, p.k, nullptr, 0, 0, 0, 0},
                                     SymArgs{A, nullptr, lda, ab, 0, 0}, batch, s);
    product<P, false, false, Sym<P>>(Args{OA, OA, p.r, p.r, p.r, nullptr, 0, 0, 0, 0},
                                     SymArgs{B, A, lda, ab, b, c}, batch, s);
    product<P, false, true, Next<P, T>>(Args{OB, X, p.r, p.k, p.r, nullptr, 0, 0, 0, 0},
                                        NextArgs{from, to, ldx, xb, a, o, ldo, stride_o, tall},
                                        batch, s);
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
  if (steps < 1 || steps > 64) return fail(OG_ERR_INVALID_ARG, "steps %d: 1 to 64", steps);
  if (!(eps >= 0) || !std::isfinite(eps) || !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
    return fail(OG_ERR_INVALID_ARG, "eps must be finite and not negative, a, b and c finite");
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
    og::ns::run<float, 3>(p, in, (int)batch, steps, a, b, c, eps, O, ldo, strideo,
                          static_cast<char *>(workspace), current_stream());
  else
    og::ns::run<__bf16, 2>(p, in, (int)batch, steps, a, b, c, eps, O, ldo, strideo,
                           static_cast<char *>(workspace), current_stream());
  return check_launch("newton_schulz");
}

}  // extern "C"
