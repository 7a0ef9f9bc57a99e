// og_epi.hpp -- what og_gemm_nt_epi and its gradient share: the activations
// with their derivatives, the operands of the tile product (og_tile.hpp) and
// its epilogue, and products whose k is split.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <limits>
#include <type_traits>

#include "og.h"
#include "og_host.hpp"
#include "og_tile.hpp"

namespace og::epi {

using namespace og::tile;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The logistic function of x: 1 / (1 + e), e = exp(-x).
struct Logistic {
  float e, s;
  __device__ __forceinline__ explicit Logistic(float x) {
    e = exp2_of(-kLog2e * x);
    s = __builtin_amdgcn_rcpf(1.0f + e);
  }
};

// The normal distribution Phi and e = exp(-x^2 / 2).  The tail beyond |x| is e times a polynomial
// of degree 9 in s = 1 / (1 + p |x|), fitted to exp(x^2 / 2) Phi(-|x|) for |x| up to 20 by least
// squares of the relative error, reweighted until its largest values are even: with the coefficients
// rounded to fp32, as here, at most 7.4e-8 (at 12.5), so that the tail keeps its relative accuracy.
struct Normal {
  float e, phi;
  __device__ __forceinline__ explicit Normal(float x) {
    e = exp2_of(-0.5f * kLog2e * (x * x));
    const float s = __builtin_amdgcn_rcpf(fmaf(0.26870057f, fabsf(x), 1.0f));
    float q = 0.029144833f;
    q = fmaf(q, s, -0.12963144f);
    q = fmaf(q, s, 0.17909917f);
    q = fmaf(q, s, -0.077821545f);
    q = fmaf(q, s, 0.113234f);
    q = fmaf(q, s, 0.06998415f);
    q = fmaf(q, s, 0.101809844f);
    q = fmaf(q, s, 0.10697627f);
    q = fmaf(q, s, 0.10720471f);
    const float tail = e * (q * s);
    phi = x < 0 ? tail : 1.0f - tail;
  }
};

constexpr float kTanh = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

// act(x).  Far to the left, where the value is 0 in fp32, x times 0 would make an infinity NaN.
template <int ACT>
__device__ __forceinline__ float act_of(float x) {
  if constexpr (ACT == OG_ACT_RELU) return x > 0 ? x : x == x ? 0.0f : x;
  if constexpr (ACT == OG_ACT_GELU) return x < -20 ? -0.0f : x * Normal(x).phi;
  if constexpr (ACT == OG_ACT_GELU_TANH)
    return x < -20 ? -0.0f : x * Logistic(kTanh * x * fmaf(kCube, x * x, 1.0f)).s;
  if constexpr (ACT == OG_ACT_SILU) return x < -120 ? -0.0f : x * Logistic(x).s;
  return x;
}

// act'(x); far to the left and the right 0 and 1, where it is that to 2^-200 (GELU), 2^-116 (by tanh) and
// 2^-108 (SiLU) and its terms would meet 0 times infinity.
template <int ACT>
__device__ __forceinline__ float slope_of(float x) {
  const float side = x > 0 ? 1.0f : 0.0f;
  if constexpr (ACT == OG_ACT_RELU) return x == x ? side : x;
  if constexpr (ACT == OG_ACT_GELU) {
    const Normal n(x);
    return fabsf(x) > 20 ? side : fmaf(x * 0.3989422804014327f, n.e, n.phi);
  }
  if constexpr (ACT == OG_ACT_GELU_TANH) {
    const Logistic l(kTanh * x * fmaf(kCube, x * x, 1.0f));
    // (e s is 1 - s without the difference)
    return fabsf(x) > 10 ? side : l.s + x * l.s * (l.e * l.s) * fmaf(3.0f * kCube * kTanh, x * x, kTanh);
  }
  if constexpr (ACT == OG_ACT_SILU) {
    const Logistic l(x);
    return fabsf(x) > 80 ? side : fmaf(l.s * x, l.e * l.s, l.s);
  }
  return 1.0f;
}

// f(ACT) for act, outside the loops over values.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case OG_ACT_RELU: f(std::integral_constant<int, OG_ACT_RELU>()); break;
    case OG_ACT_GELU: f(std::integral_constant<int, OG_ACT_GELU>()); break;
    case OG_ACT_GELU_TANH: f(std::integral_constant<int, OG_ACT_GELU_TANH>()); break;
    case OG_ACT_SILU: f(std::integral_constant<int, OG_ACT_SILU>()); break;
    default: f(std::integral_constant<int, OG_ACT_NONE>());
  }
}

inline bool valid_act(int act) { return act >= OG_ACT_NONE && act <= OG_ACT_SILU; }

// Elements of the matrix cores: 16-bit types as given, fp32 as two fp16 planes.
template <class T>
using Element = std::conditional_t<std::is_same_v<T, float>, _Float16, T>;
template <class T>
constexpr int kPlanes = sizeof(T) == 4 ? 2 : 1;

// Whether four values of a row are one aligned access.
template <class T>
int whole(const T *p, int64_t ld) {
  return ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0;
}

template <class T>
__device__ __forceinline__ f32x4 load4(const T *p, int left, bool vec) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  f32x4 v = {0, 0, 0, 0};
  if (vec && left >= 4) {
    const T4 h = *reinterpret_cast<const T4 *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)h[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) v[e] = (float)p[e];
  }
  return v;
}
template <class T>
__device__ __forceinline__ void store4(T *to, const f32x4 v, int left, bool vec) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  T4 h;
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = (T)v[e];
  if (vec && left >= 4) {
    *reinterpret_cast<T4 *>(to) = h;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) to[e] = h[e];
  }
}

// The power of two, as an exponent, by which a row or column of fp32 is held in planes: it
// brings its largest finite magnitude `top` to [2^13, 2^14).
__device__ __forceinline__ int power_of(float top) {
  return top > 0 ? 14 - (int)__builtin_amdgcn_frexp_expf(top) : 0;
}

// Four columns' planes, times 2^e.
__device__ __forceinline__ void store_planes(uint16_t *out, int c, f32x4 v, const int (&e)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = __builtin_ldexpf(v[q], e[q]);
  f16x4 h, l;
  split4(v, h, l);
  *reinterpret_cast<f16x4 *>(out + column<2>(c, 0)) = h;
  *reinterpret_cast<f16x4 *>(out + column<2>(c, 1)) = l;
}

// What becomes of a finished sum at (m, n):
//   v = sum 2^-(the powers of its row and column) + bias[n];  P = v;  C = act(v) + residual
// (out is C of a forward product, dA or dW of the gradient's).
struct Finish {
  const float *mtop, *ntop;  // operands held by powers of two: the magnitudes that give them; else null
  const void *bias;
  int act;
  const void *residual;
  int64_t ldr;
  void *pre;
  int64_t ldp;
  void *out;
  int64_t ldo;
  int vec_b, vec_r, vec_p, vec_o;  // four values are one access
  int whole;                       // all of them are, and 256 rows apart is within 32 bits
};
template <class T>
Finish set_accesses(Finish f) {
  f.vec_b = whole(static_cast<const T *>(f.bias), 0);
  f.vec_r = whole(static_cast<const T *>(f.residual), f.ldr);
  f.vec_p = whole(static_cast<const T *>(f.pre), f.ldp);
  f.vec_o = whole(static_cast<const T *>(f.out), f.ldo);
  const int64_t far = std::max({f.residual ? f.ldr : 0, f.pre ? f.ldp : 0, f.ldo});
  f.whole = (f.vec_r || !f.residual) && (f.vec_p || !f.pre) && f.vec_o && far <= (1 << 21);
  return f;
}

// Whether the operands of a product may be held by powers of two: fp32 ones, and the gradient's (PLAIN).
template <class T, bool PLAIN>
constexpr bool kPowers = kPlanes<T> == 2 || PLAIN;

template <class T, bool PLAIN>
__device__ __forceinline__ void scale(const Finish &f, f32x4 &v, int mpower, const int (&npower)[4]) {
  if constexpr (kPowers<T, PLAIN>) {
    if (kPlanes<T> == 2 || f.mtop) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_ldexpf(v[e], -mpower - npower[e]);
    }
  }
}

// What belongs to four columns from n on, `left` of them inside, and to a row.
template <class T, bool PLAIN>
__device__ __forceinline__ void of_columns(const Finish &f, int n, int left, int (&npower)[4], f32x4 &bias) {
#pragma unroll
  for (int e = 0; e < 4; ++e) npower[e] = 0;
  if constexpr (kPowers<T, PLAIN>) {
    if (f.ntop) {
      const f32x4 top = load4(f.ntop + n, left, true);
#pragma unroll
      for (int e = 0; e < 4; ++e) npower[e] = power_of(top[e]);
    }
  }
  if (!PLAIN && f.bias) bias = load4(static_cast<const T *>(f.bias) + n, left, f.vec_b);
}
template <class T, bool PLAIN>
__device__ __forceinline__ int of_row(const Finish &f, int m) {
  if constexpr (kPowers<T, PLAIN>) return f.mtop ? power_of(f.mtop[m]) : 0;
  return 0;
}

// All steps of four neighbouring sums of row m.
template <class T, bool PLAIN>
__device__ __forceinline__ void finish(const Finish &f, int64_t m, int n, int left, f32x4 v) {
  int npower[4];
  f32x4 bias = {0, 0, 0, 0};
  of_columns<T, PLAIN>(f, n, left, npower, bias);
  scale<T, PLAIN>(f, v, of_row<T, PLAIN>(f, (int)m), npower);
  if constexpr (!PLAIN) {
    v += bias;
    if (f.pre) store4(static_cast<T *>(f.pre) + m * f.ldp + n, v, left, f.vec_p);
    with_act(f.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_of<act()>(v[e]);
    });
    if (f.residual) v += load4(static_cast<const T *>(f.residual) + m * f.ldr + n, left, f.vec_r);
  }
  store4(static_cast<T *>(f.out) + m * f.ldo + n, v, left, f.vec_o);
}

// The tile product's epilogue: finished, or (a product whose k is split) the part's sums.  PLAIN:
// a gradient's, only scaled and stored.
struct StoreArgs {
  Finish f;
  float *part;     // null: not split
  int64_t ld, step;  // of a row of a part, and from one part to the next
};
template <class T, bool PLAIN>
struct Store {
  using Args = StoreArgs;
  static constexpr bool kSymmetric = false;
  // A block whose rows and columns are all the product's, all accesses whole: places as 32-bit
  // offsets from the wave's first element, which is uniform.  Each four values go all the way
  // before the next (fences): together their activations would need more registers than there
  // are.  (4096 x 11008 x 4096 bf16, calls back to back: 298 us without activation and P, 298 with
  // SiLU, 342 with SiLU and P, whose 90 MB more leave the compute units all at once at the end of a
  // round of tiles.  With places of 64 bits, the activation chosen for each value and IEEE
  // divisions the last took 110 us more.)
  template <class S, int ACT>
  static __device__ __forceinline__ void inside(f32x4 (&acc)[S::FM][S::FN], const Place &t, const Finish &f) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    const uint32_t row = t.lane & 15, col = 4 * (t.lane >> 4);
    const int64_t m = t.m0, n = t.n0;
    char *out = reinterpret_cast<char *>(static_cast<T *>(f.out) + m * f.ldo + n);
    char *pre = PLAIN || !f.pre ? nullptr : reinterpret_cast<char *>(static_cast<T *>(f.pre) + m * f.ldp + n);
    const char *residual =
        PLAIN || !f.residual ? nullptr : reinterpret_cast<const char *>(static_cast<const T *>(f.residual) + m * f.ldr + n);
    const uint32_t ldo = (uint32_t)f.ldo * sizeof(T), ldp = (uint32_t)f.ldp * sizeof(T), ldr = (uint32_t)f.ldr * sizeof(T);
    f32x4 bias[S::FN];
    int npower[S::FN][4];
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
      bias[j] = f32x4{0, 0, 0, 0};
      of_columns<T, PLAIN>(f, t.n0 + 16 * j + col, 4, npower[j], bias[j]);
    }
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const uint32_t r = row + 16 * i;
      const int mpower = of_row<T, PLAIN>(f, t.m0 + r);
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const uint32_t c = (col + 16 * j) * sizeof(T);
        f32x4 v = acc[i][j];
        T4 h;
        scale<T, PLAIN>(f, v, mpower, npower[j]);
        if constexpr (!PLAIN) {
          v += bias[j];
          if (pre) {
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = (T)v[e];
            *reinterpret_cast<T4 *>(pre + r * ldp + c) = h;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = act_of<ACT>(v[e]);
          if (residual) {
            h = *reinterpret_cast<const T4 *>(residual + r * ldr + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += (float)h[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (T)v[e];
        *reinterpret_cast<T4 *>(out + r * ldo + c) = h;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  template <class S>
  static __device__ __forceinline__ void store(f32x4 (&acc)[S::FM][S::FN], const Place &t, const Args &e) {
    const int nc = t.n0 + 4 * (t.lane >> 4);
    if (!e.part && e.f.whole && (t.tile_m + 1) * S::BM <= t.M && (t.tile_n + 1) * S::BN <= t.N) {
      if constexpr (PLAIN) inside<S, OG_ACT_NONE>(acc, t, e.f);
      else with_act(e.f.act, [&](auto act) __attribute__((always_inline)) { inside<S, act()>(acc, t, e.f); });
      return;
    }
#pragma unroll
    for (int i = 0; i < S::FM; ++i) {
      const int m = t.m0 + 16 * i + (t.lane & 15);
      if (m >= t.M) continue;
      float *to = e.part + t.batch * e.step + m * e.ld;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int n = nc + 16 * j;
        if (n >= t.N) continue;
        if (e.part) *reinterpret_cast<f32x4 *>(to + n) = acc[i][j];
        else finish<T, PLAIN>(e.f, m, n, t.N - n, acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
};

// Adds the parts of a split product in order and finishes.  FOLD 2: every part is followed by that of
// the remainder, which counts where the matrix's own sum is finite (an infinity of the other operand
// times a remainder of 0, or of the other sign, would make it NaN).
template <class T, bool PLAIN, int FOLD>
static __global__ __launch_bounds__(256) void join_kernel(int M, int N, int parts, const float *part, int64_t ld,
                                                   int64_t step, Finish f) {
  const int per = (N + 3) / 4;
  const int64_t total = (int64_t)M * per;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += (int64_t)gridDim.x * 256) {
    const int m = (int)(at / per), n = (int)(at - (int64_t)m * per) * 4;
    f32x4 v = {0, 0, 0, 0}, own = {0, 0, 0, 0};
    for (int p = 0; p < parts; ++p) {
      const float *at = part + p * (FOLD * step) + m * ld + n;
      const f32x4 w = *reinterpret_cast<const f32x4 *>(at);
      v += w;
      if constexpr (FOLD == 2) {
        own += w;
        v += *reinterpret_cast<const f32x4 *>(at + step);
      }
    }
    if constexpr (FOLD == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_isfinite(own[e]) ? v[e] : own[e];
    }
    finish<T, PLAIN>(f, m, n, N - n, v);
  }
}

// A tile and what it costs (as og_tile.hpp's Choice): nanoseconds of a stage alone, as one of 256
// blocks and as a share, and of a round of blocks besides its stages (start and epilogue).
template <class S_, int ALONE, int ONE, int SHARE, int ROUND>
struct Cost {
  using S = S_;
  static double time(bool, int64_t M, int64_t N, int64_t K, int64_t batch) {
    const int64_t n = (M + S::BM - 1) / S::BM * ((N + S::BN - 1) / S::BN) * batch;
    const double stages = (double)((K + depth(S::P) - 1) / depth(S::P));
    if (n <= 256) return stages * (ALONE + (ONE - ALONE) * (n / 256.0)) + ROUND;
    return (double)((n + 255) / 256) * stages * SHARE + (double)((n + 256 * S::BLOCKS - 1) / (256 * S::BLOCKS)) * ROUND;
  }
};

// The tiles by planes and by whether both operands are transposed (dW).  Beside og_tile.hpp's squares
// are oblong ones, which fill the compute units where squares leave a part of a round (512 x 11008
// x 4096 fp32: 174 tiles of 192 x 192 168 us, 232 of 128 x 192 122).  Times measured on stages of k from 1024
// on.  (144 seeded products of 65 to 11008 rows and columns, 24 of each kind: the chosen tile and
// parts take 1.01 to 1.05 times the fastest listed ones' time in the mean, at most 1.20.)
template <class E, int P, bool TT>
struct EpiTiles {
  using type = Choices<Cost<Shape<E, 1, 256, 256, 2, 4, 2, 1>, 1010, 1505, 1462, 15000>,
                       Cost<Shape<E, 1, 192, 256, 2, 4, 2, 1>, 753, 1140, 1160, 11000>,
                       Cost<Shape<E, 1, 192, 192, 2, 4, 3, 1>, 620, 898, 887, 9500>,
                       Cost<Shape<E, 1, 128, 192, 2, 4, 3, 1>, 455, 650, 720, 7500>,
                       Cost<Shape<E, 1, 128, 128, 2, 2, 2, 2>, 386, 780, 442, 7000>,
                       Cost<Shape<E, 1, 128, 64, 4, 2, 4, 1>, 253, 348, 337, 6000>,
                       Cost<Shape<E, 1, 64, 64, 2, 2, 4, 2>, 187, 252, 193, 5000>>;
};
template <class E>
struct EpiTiles<E, 1, true> {
  using type = Choices<Cost<Shape<E, 1, 256, 256, 2, 4, 2, 1>, 999, 1569, 1540, 13000>,
                       Cost<Shape<E, 1, 192, 256, 2, 4, 2, 1>, 845, 1196, 1202, 11000>,
                       Cost<Shape<E, 1, 192, 192, 2, 4, 3, 1>, 702, 982, 1072, 9000>,
                       Cost<Shape<E, 1, 128, 192, 2, 4, 3, 1>, 549, 693, 831, 7000>,
                       Cost<Shape<E, 1, 128, 128, 2, 2, 2, 2>, 471, 879, 466, 8000>,
                       Cost<Shape<E, 1, 128, 64, 4, 2, 4, 1>, 290, 372, 343, 6000>,
                       Cost<Shape<E, 1, 64, 64, 2, 2, 4, 2>, 262, 276, 180, 5000>>;
};
template <class E>
struct EpiTiles<E, 2, false> {
  using type = Choices<Cost<Shape<E, 2, 256, 256, 2, 4, 2, 1>, 1412, 2400, 2050, 16000>,
                       Cost<Shape<E, 2, 192, 256, 2, 4, 2, 1>, 1090, 1600, 1600, 11500>,
                       Cost<Shape<E, 2, 192, 192, 2, 4, 3, 1>, 861, 1223, 1213, 11000>,
                       Cost<Shape<E, 2, 128, 192, 2, 4, 3, 1>, 610, 861, 856, 9500>,
                       Cost<Shape<E, 2, 128, 128, 2, 4, 2, 2>, 410, 727, 598, 8000>,
                       Cost<Shape<E, 2, 128, 64, 4, 2, 4, 1>, 343, 404, 402, 5500>,
                       Cost<Shape<E, 2, 64, 64, 2, 2, 4, 2>, 214, 273, 206, 6000>>;
};
template <class E>
struct EpiTiles<E, 2, true> {
  // (256 x 256 needs a register more than there are)
  using type = Choices<Cost<Shape<E, 2, 192, 256, 2, 4, 2, 1>, 1171, 1604, 1625, 12000>,
                       Cost<Shape<E, 2, 192, 192, 2, 4, 3, 1>, 980, 1327, 1294, 11000>,
                       Cost<Shape<E, 2, 128, 192, 2, 4, 3, 1>, 721, 954, 990, 9000>,
                       Cost<Shape<E, 2, 128, 128, 2, 4, 2, 2>, 474, 728, 613, 8000>,
                       Cost<Shape<E, 2, 128, 64, 4, 2, 4, 1>, 375, 477, 461, 6000>,
                       Cost<Shape<E, 2, 64, 64, 2, 2, 4, 2>, 271, 327, 220, 6000>>;
};

// Parts of k: as many as take the least time, where the parts' sums cost a launch and their
// bytes, written and read (at 6.5 TB/s: mostly in the caches).
constexpr int kMostParts = 16;
template <class T, bool TT>
int parts_of(int64_t M, int64_t N, int64_t K) {
  using C = typename EpiTiles<Element<T>, kPlanes<T>, TT>::type;
  double best = std::numeric_limits<double>::infinity();
  int parts = 1;
  for (int p = 1; p <= kMostParts && (p == 1 || K / p >= 256); p += p < 4 ? 1 : p) {
    Args g{};
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.k_split = p > 1 ? (int)round_up((K + p - 1) / p, 64) : 0;
    const double t = least(C(), false, g, p) + (p > 1 ? 3500 + 8.0 * p * M * N / 6500 : 0);
    if (t < best) best = t, parts = p;
  }
  return parts;
}

// Bytes of a product's parts.  (fold: see run_product)
template <class T, bool TT>
int64_t parts_bytes(int64_t M, int64_t N, int64_t K, int fold = 1) {
  const int p = parts_of<T, TT>(fold * M, N, K);
  return p * fold > 1 ? p * fold * M * round_up(N, 4) * 4 : 0;
}

// The most matrices below one another that a product's operand has: 16-bit gradients' may be two.
template <class T, bool PLAIN>
constexpr int kFold = PLAIN && kPlanes<T> == 1 ? 2 : 1;

// The product, its k in parts where that is faster.  fold 2: the rows of A come twice, as a matrix
// and its remainder below it (g.M rows in all), whose sums are added like parts.
// E: the operands' elements.
template <class T, bool TA, bool TB, bool PLAIN, class E = Element<T>>
void run_product(Args g, const Finish &f, char *ws, hipStream_t s, int fold = 1) {
  using C = typename EpiTiles<E, kPlanes<T>, TA && TB>::type;
  const int parts = parts_of<T, TA && TB>(g.M, g.N, g.K);
  StoreArgs e{f, nullptr, 0, 0};
  if (parts * fold > 1) {
    e.part = reinterpret_cast<float *>(ws);
    e.ld = round_up(g.N, 4);
    e.step = g.M * e.ld;
  }
  if (parts > 1) g.k_split = (int)round_up((g.K + parts - 1) / parts, 64);
  product_of<TA, TB, Store<T, PLAIN>>(C(), least(C(), false, g, parts), g, e, parts, s);
  if (!e.part) return;
  const int rows = g.M / fold;
  const int64_t quads = (int64_t)rows * ((g.N + 3) / 4);
  const auto join = fold == 1 ? join_kernel<T, PLAIN, 1> : join_kernel<T, PLAIN, kFold<T, PLAIN>>;
  hipLaunchKernelGGL(join, dim3((unsigned)std::min<int64_t>((quads + 255) / 256, 4096)), dim3(256), 0, s, rows, g.N, parts,
                     e.part, e.ld, rows * e.ld, f);
}

// Whether the tile product can read a 16-bit matrix where it lies; else each call copies it first (64, 512 and
// 4096 rows of bf16 on 11008 x 4096 27, 56 and 317 us, on 11008 x 4095 67, 96 and 361).
inline bool readable(const void *p, int64_t cols, int64_t ld) {
  return cols % 8 == 0 && ld % 8 == 0 && ld <= (1 << 22) && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// Places in a workspace.
struct Room {
  int64_t at = 0;
  int64_t take(int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  }
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

template <class T>
struct Eight {
  T v[8];
};
// Eight values of a row from k on, zero past its end.  FULL: it does not end here.
template <class T, bool FULL>
__device__ __forceinline__ Eight<T> load8(const T *row, int k, int K) {
  Eight<T> t;
  if (FULL || k + 8 <= K) {
    __builtin_memcpy(&t, row + k, sizeof t);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) t.v[e] = k + e < K ? row[k + e] : (T)0.0f;
  }
  return t;
}

// Fragments and their product: 16-bit values as they are; fp32 as three bf16 planes, cut, 24 bits
// (h + m + l = the value; the products left out are 2^-24 of the whole and below), which need no
// power of two.
template <class T>
struct Fragment {
  s16x8 v;
  Fragment() = default;
  __device__ __forceinline__ explicit Fragment(const Eight<T> &x) { __builtin_memcpy(&v, &x, sizeof v); }
  static __device__ __forceinline__ f32x4 product(const Fragment &x, const Fragment &w, f32x4 c) {
    return mfma<T>(x.v, w.v, c);
  }
};
template <>
struct Fragment<float> {
  s16x8 p[3];
  Fragment() = default;
  __device__ __forceinline__ explicit Fragment(const Eight<float> &x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // (a NaN is made quiet first: its highest mantissa bit then stays)
      float r = __builtin_canonicalizef(x.v[e]);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const uint32_t top = __builtin_bit_cast(uint32_t, r) & 0xFFFF0000u;
        const float h = __builtin_bit_cast(float, top);
        p[q][e] = (short)(top >> 16);
        r = __builtin_isfinite(h) ? r - h : 0.0f;
      }
    }
  }
  static __device__ __forceinline__ f32x4 product(const Fragment &x, const Fragment &w, f32x4 c) {
    constexpr int kX[6] = {2, 0, 1, 1, 0, 0}, kW[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
    for (int i = 0; i < 6; ++i) c = mfma<__bf16>(x.p[kX[i]], w.p[kW[i]], c);
    return c;
  }
};

// Rows of 16-bit values, zero from cols to ld (a multiple of 8); times 2: below them once more, with 0
// for what is not finite (bits of the exponent all set) -- a remainder's product has no more to say there.
static __global__ __launch_bounds__(256) void copy_kernel(const uint16_t *x, int64_t ldx, int rows, int cols,
                                                          uint16_t *out, int ld, int times, int exponent) {
  const int per = ld / 8;
  const int64_t total = (int64_t)rows * per;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += (int64_t)gridDim.x * 256) {
    const int64_t i = at / per;
    const int c = (int)(at - i * per) * 8;
    s16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? (short)x[i * ldx + c + e] : (short)0;
    *reinterpret_cast<s16x8 *>(out + i * ld + c) = v;
    if (times == 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (v[e] & exponent) == exponent ? (short)0 : v[e];
      *reinterpret_cast<s16x8 *>(out + (i + rows) * ld + c) = v;
    }
  }
}

// A 16-bit matrix as an operand, its rows `times` over (see copy_kernel).
template <class T>
Operand operand16(const void *x, int64_t ld, int64_t rows, int64_t cols, int64_t padded, char *ws, hipStream_t s,
                         int times = 1) {
  if (rows == 0 || cols == 0 || (times == 1 && readable(x, cols, ld))) return Operand{static_cast<const uint16_t *>(x), ld, 0};
  uint16_t *to = reinterpret_cast<uint16_t *>(ws);
  const int64_t granules = rows * (padded / 8);
  hipLaunchKernelGGL(copy_kernel, dim3((unsigned)std::min<int64_t>((granules + 255) / 256, 8192)), dim3(256), 0, s,
                     static_cast<const uint16_t *>(x), ld, (int)rows, (int)cols, to, (int)padded, times,
                     std::is_same_v<T, __bf16> ? 0x7F80 : 0x7C00);
  return Operand{to, padded, 0};
}

inline og_status check_sizes(int64_t m, int64_t n, int64_t k, int type) {
  using og::host::fail;
  if (type < OG_F32 || type > OG_F16)
    return fail(OG_ERR_INVALID_ARG, "type %d: OG_F32, OG_BF16 or OG_F16", type);
  if (m < 0 || n < 0 || k < 0)
    return fail(OG_ERR_INVALID_ARG, "negative size: m %lld, n %lld, k %lld", (long long)m, (long long)n, (long long)k);
  if (m > (1 << 24) || n > (1 << 20) || k > (1 << 20))
    return fail(OG_ERR_TOO_LARGE, "m %lld, n %lld or k %lld: at most 2^24, 2^20 and 2^20", (long long)m, (long long)n,
                (long long)k);
  if (m * n > (int64_t(1) << 36) || m * k > (int64_t(1) << 36) || n * k > (int64_t(1) << 36))
    return fail(OG_ERR_TOO_LARGE, "m %lld, n %lld, k %lld: at most 2^36 elements a matrix", (long long)m, (long long)n,
                (long long)k);
  return OG_OK;
}

}  // namespace og::epi
