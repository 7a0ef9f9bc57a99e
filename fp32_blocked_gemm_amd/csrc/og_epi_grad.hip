// og_epi_grad.hip -- the gradient of og_gemm_nt_epi:
//
//   dP = dC act'(P);  dA = dP W;  dW = dP^T A;  dbias = sum over the rows of dP
//
// One sweep over dC and P forms dP and its column sums; two tile products
// (og_tile.hpp) do the rest, with W and A as operands whose rows run along k
// (the transposing reads).
//
// 16-bit types: dP of no activation or ReLU is of the type, as dC is.  That of a smooth one has more bits; rounded
// to bf16 it would give dA and dW 1.41 times the error of their own rounding (0.0023 and 0.0017).  So
//   - bf16 up to 384 rows: what dP leaves to its rounding is a second matrix below the first (A comes twice for
//     it); where W or A is not finite it is left out, so that infinities follow the formula;
//   - bf16 of more rows: dP, W and A in fp16, whose 11 bits hold bf16's 8, by powers of two, as below: 1.01
//     times (4096 x 11008 x 4096 833 us, rounded to bf16 657; 4096 x 1536 x 384 64 and 46);
//   - fp16: dP by powers of two, so that neither small values become subnormal nor large ones, times a slope
//     above 1, infinite (256 x 512 x 256 with dC of 1e-5: errors of dW 5.6e-3 with dP as it is, 3.1e-4 so, 2.4e-4 of
//     the result's rounding); W and A are as they lie.  Up to 128 rows, where the bytes of W bound the time, with
//     its remainder.  The largest magnitudes cost a sweep: 4096 x 11008 x 4096 663 and 804 us, 200 x 4096 x
//     4096 50 and 68.
// dbias sums dP before any of that.  (P's own rounding to the type leaves errors of 1.06 times a plain form's, which
// keeps P in fp32.)
//
// fp32: two fp16 planes.  A product's powers of two belong to the indices that
// it does not sum over, so that every row and column of a gradient keeps the bits
// of its own size: dA takes dP by rows and W by columns, dW takes dP and A by
// columns.  A first sweep finds all largest magnitudes (by atomic maxima, whose
// order does not matter), a second lays out the planes.
#include "og_epi.hpp"

namespace og::epi::grad {

// A block of a sweep: 16 bytes of a row a lane, the rows by the waves in turn, one after another
// (more of a wave's rows in flight at once cost the registers that more waves hide latency with:
// dC and P of 4096 x 11008 in bf16, 42 us for their column sums; two rows 53, four 86).  Maxima take
// more rows a block where there are many, for fewer atomics on a column's (all of the gradient by 32 and
// 64 rows a block, fp32: 16384 x 1536 x 384 293 and 280 us, 4096 of them 102 and 103, 300 x 1001 x 3001 65 and
// 74; fp16: 153 and 140, 62 and 68, 71 and 94).
constexpr int kWaves = 8, kRows = 32;
template <class T>
int rows_per(int64_t rows, bool tops) {
  return tops && rows >= (kPlanes<T> == 2 ? 2048 : 8192) ? 2 * kRows : kRows;
}
template <class T>
constexpr int kPer = 16 / (int)sizeof(T);  // columns of a lane
template <class T>
constexpr int kCols = 64 * kPer<T>;  // of a block

struct Matrix {
  const void *x;
  int64_t ldx;
  const void *pre;   // null: x itself
  int64_t ldp;
  int act;
  int rows, cols, width;  // width: padded columns of the outputs
  int vec_x, vec_p;
  uint16_t *out;          // null: not wanted; else the values or (LAYOUT) what the row's power makes of them in fp16
  uint16_t *out_c;        // LAYOUT: by the column's power (null: not wanted)
  int twice;              // 16-bit types: below each output the same size again, what its rounding leaves
  float *rtop, *ctop;     // largest magnitudes (null: not wanted)
  float *sums;            // column sums of the block's rows, [row block][width] (null: not wanted)
  int rows_per;           // rows of a block
  float *plain;           // fp32 of few rows: the values (null: not wanted)
  void *bias;             // where the column sums go in the end; without sums, of a single row block, at once
  int blocks;             // of a launch
};

// A lane's columns as fp32.
template <class T>
struct Lane {
  f32x4 v[kPer<T> / 4];
};
template <class T>
__device__ __forceinline__ void load_lane(const T *p, int left, bool vec, Lane<T> &lane) {
  if (vec && left >= kPer<T>) {
    typedef T V __attribute__((ext_vector_type(kPer<T>)));
    const V w = *reinterpret_cast<const V *>(p);
#pragma unroll
    for (int e = 0; e < kPer<T>; ++e) lane.v[e / 4][e % 4] = (float)w[e];
  } else {
#pragma unroll
    for (int e = 0; e < kPer<T>; ++e) lane.v[e / 4][e % 4] = e < left ? (float)p[e] : 0.0f;
  }
}

// A lane's values of row i, zero past the matrix.
template <class T>
__device__ __forceinline__ void values(const Matrix &a, int64_t i, int c, Lane<T> &v) {
  const int left = a.cols - c;
  load_lane<T>(static_cast<const T *>(a.x) + i * a.ldx + c, left, a.vec_x, v);
  if (!a.pre) return;
  Lane<T> p;
  load_lane<T>(static_cast<const T *>(a.pre) + i * a.ldp + c, left, a.vec_p, p);
  with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < kPer<T>; ++e)
      v.v[e / 4][e % 4] = e < left ? v.v[e / 4][e % 4] * slope_of<act()>(p.v[e / 4][e % 4]) : 0.0f;
  });
}

// A lane's values rounded to a 16-bit type, and (rest not null) what that leaves of the finite ones, rounded too.
template <class T>
__device__ __forceinline__ void store_rounded(T *to, T *rest, const float (&v)[8]) {
  typedef T V __attribute__((ext_vector_type(8)));
  V w;
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = (T)v[e];
  *reinterpret_cast<V *>(to) = w;
  if (rest) {
    V r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (T)(__builtin_isfinite((float)w[e]) ? v[e] - (float)w[e] : 0.0f);
    *reinterpret_cast<V *>(rest) = r;
  }
}

// Row i's columns from c on times 2^e: fp32 as two fp16 planes, fp16 as it is.
template <class T>
__device__ __forceinline__ void store_scaled(const Matrix &a, uint16_t *out, int64_t i, int c, const Lane<T> &v,
                                             const int (&e)[kPer<T>]) {
  if constexpr (kPlanes<T> == 2) {
    store_planes(out + i * a.width * 2, c, v.v[0], e);
  } else {
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = __builtin_ldexpf(v.v[q / 4][q % 4], e[q]);
    _Float16 *to = reinterpret_cast<_Float16 *>(out) + i * a.width + c;
    store_rounded(to, a.twice ? to + (int64_t)a.rows * a.width : nullptr, x);
  }
}

// dbias from the row blocks' sums: 64 columns a block, the row blocks by its waves in turn, in a
// fixed order in 64 bits.
template <class T, int WAVES>
__device__ __forceinline__ void bias_columns(const Matrix &a, int block, double (&of)[WAVES][64]) {
  const int c = block * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  const int blocks = (a.rows + a.rows_per - 1) / a.rows_per;
  double sum = 0;
  if (c < a.cols)
    for (int b = w; b < blocks; b += WAVES) sum += (double)a.sums[(int64_t)b * a.width + c];
  of[w][threadIdx.x & 63] = sum;
  __syncthreads();
  if (w || c >= a.cols) return;
  for (int k = 1; k < WAVES; ++k) sum += of[k][threadIdx.x];
  static_cast<T *>(a.bias)[c] = (T)(float)sum;
}

// One sweep over up to three matrices.  LAYOUT: the operands by powers of two, and in blocks behind all
// others dbias from m0's sums; else the values and their sums, or (TOPS) their largest magnitudes and sums.
template <class T, bool LAYOUT, bool TOPS>
__global__ __launch_bounds__(64 * kWaves) void sweep_kernel(Matrix m0, Matrix m1, Matrix m2) {
  constexpr int H = kPer<T> / 4;
  __shared__ f32x4 of_waves[LAYOUT ? 1 : TOPS ? 2 * H : H][kWaves][64];
  int block = blockIdx.x;
  if constexpr (LAYOUT) {
    const int all = m0.blocks + m1.blocks + m2.blocks;
    if (block >= all)
      return bias_columns<T, kWaves>(m0, block - all, *reinterpret_cast<double(*)[kWaves][64]>(of_waves));
  }
  const Matrix &a = block < m0.blocks ? m0 : block < m0.blocks + m1.blocks ? m1 : m2;
  block -= block < m0.blocks ? 0 : block < m0.blocks + m1.blocks ? m0.blocks : m0.blocks + m1.blocks;
  const int across = (a.width + kCols<T> - 1) / kCols<T>, rb = block / across;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (block - rb * across) * kCols<T> + kPer<T> * lane;
  const int64_t i0 = (int64_t)rb * a.rows_per + wave, end = min((int64_t)(rb + 1) * a.rows_per, (int64_t)a.rows);
  if constexpr (LAYOUT) {
    if (c >= a.width) return;
    int cpower[kPer<T>] = {};
    if (a.out_c) {
#pragma unroll
      for (int e = 0; e < kPer<T>; ++e) cpower[e] = c + e < a.cols ? power_of(a.ctop[c + e]) : 0;
    }
    for (int64_t i = i0; i < end; i += kWaves) {
      Lane<T> v;
      values<T>(a, i, c, v);
      if (a.out) {
        const int p = power_of(a.rtop[i]);
        int powers[kPer<T>];
#pragma unroll
        for (int e = 0; e < kPer<T>; ++e) powers[e] = p;
        store_scaled<T>(a, a.out, i, c, v, powers);
      }
      if (a.out_c) store_scaled<T>(a, a.out_c, i, c, v, cpower);
    }
  } else {
    f32x4 sum[H], top[H];
#pragma unroll
    for (int h = 0; h < H; ++h) sum[h] = top[h] = f32x4{0, 0, 0, 0};
    for (int64_t i = i0; i < end; i += kWaves) {
      Lane<T> v;
      values<T>(a, i, c, v);
#pragma unroll
      for (int h = 0; h < H; ++h) sum[h] += v.v[h];
      if constexpr (kPlanes<T> == 2) {
        if (a.plain && c < a.width) *reinterpret_cast<f32x4 *>(a.plain + i * a.width + c) = v.v[0];
      }
      if constexpr (TOPS) {
        float most = 0;
#pragma unroll
        for (int e = 0; e < kPer<T>; ++e) {
          const float x = v.v[e / 4][e % 4], size = __builtin_isfinite(x) ? fabsf(x) : 0.0f;
          top[e / 4][e % 4] = fmaxf(top[e / 4][e % 4], size);
          most = fmaxf(most, size);
        }
        if (a.rtop) {
          most = wave_max(most);
          if (lane == 0 && most > 0)
            atomicMax(reinterpret_cast<uint32_t *>(a.rtop + i), __builtin_bit_cast(uint32_t, most));
        }
      } else if (a.out && c < a.width) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v.v[e / 4][e % 4];
        T *to = reinterpret_cast<T *>(a.out) + i * a.width + c;
        store_rounded(to, a.twice ? to + (int64_t)a.rows * a.width : nullptr, x);
      }
    }
    if (!a.sums && !a.ctop && !a.bias) return;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      of_waves[h][wave][lane] = sum[h];
      if (TOPS) of_waves[H + h][wave][lane] = top[h];
    }
    __syncthreads();
    // a column a thread, the waves in turn
    const int q = threadIdx.x, column = (block - rb * across) * kCols<T> + q;
    if (q >= kCols<T> || column >= a.width) return;
    auto held = [&](int w, int what) __attribute__((always_inline)) {
      return of_waves[what * H + q % kPer<T> / 4][w][q / kPer<T>][q % 4];
    };
    float total = held(0, 0);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) total += held(w, 0);
    if (a.sums) a.sums[(int64_t)rb * a.width + column] = total;
    if (column >= a.cols) return;
    if (a.bias && !a.sums) static_cast<T *>(a.bias)[column] = (T)total;
    if constexpr (TOPS) {
      if (!a.ctop) return;
      float most = held(0, 1);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) most = fmaxf(most, held(w, 1));
      if (most > 0) atomicMax(reinterpret_cast<uint32_t *>(a.ctop + column), __builtin_bit_cast(uint32_t, most));
    }
  }
}

__global__ __launch_bounds__(256) void clear_kernel(float *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

template <class T>
__global__ __launch_bounds__(1024) void bias_kernel(Matrix a) {
  __shared__ double of[16][64];
  bias_columns<T, 16>(a, blockIdx.x, of);
}

// Few fp32 rows of dC and A (up to kFew): bound by the bytes of W, read, and of dW, written.  Both
// products run from memory through registers as three bf16 planes, 24 bits, so that nothing of W is
// scanned and laid out first (forward and gradient of one row on 4096 x 4096 61 us, 103 with the tile
// products; 16-bit types, whose W lies ready for those, gain nothing).  dP lies in fp32: the
// sweep's, or dC.
constexpr int kFew = 32;
template <class T>
constexpr bool few_rows(int64_t m) {
  return kPlanes<T> == 2 && m <= kFew;
}

struct FewRows {
  int m, n, k;
  const float *dp, *a, *w;
  int64_t lddp, lda, ldw;
  int vec;         // four columns of a row of W are one access
  int steps;       // of 32 rows of W: of a part
  Finish f;
  float *part;     // dA in parts; null: whole
  int64_t ld, step;
};

// dA: a block takes 64 columns of W and 16 MT rows of dP, its four waves share the part's rows of W.
// A lane reads four columns of eight rows, 256 neighbouring bytes a row and instruction; its
// column 4 i + e is the fragment e's column i, so that four fragments' sums are four neighbours.
// (4096 x 4096: 20 us, 3.3 TB/s.)
template <int MT>
__global__ __launch_bounds__(256) void few_da_kernel(FewRows p) {
  __shared__ __align__(16) float sums[4][16 * MT][68];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int c = blockIdx.x * 64 + 4 * i;
  const int s0 = blockIdx.y * p.steps, s1 = min(s0 + p.steps, (p.n + 31) / 32);
  f32x4 acc[4][MT];
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[e][t] = f32x4{0, 0, 0, 0};
  f32x4 next[8];
  auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int j = 32 * s + 8 * g + r;
      next[r] = load4(p.w + (int64_t)j * p.ldw + c, j < p.n ? p.k - c : 0, p.vec);
    }
  };
  if (s0 + wave < s1) load(s0 + wave);
  for (int s = s0 + wave; s < s1; s += 4) {
    f32x4 now[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) now[r] = next[r];
    Eight<float> x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int m = 16 * t + i;
      x[t] = load8<float, false>(p.dp + (int64_t)min(m, p.m - 1) * p.lddp, 32 * s + 8 * g, m < p.m ? p.n : 0);
    }
    if (s + 4 < s1) load(s + 4);
    Fragment<float> d[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) d[t] = Fragment<float>(x[t]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      Eight<float> column;
#pragma unroll
      for (int r = 0; r < 8; ++r) column.v[r] = now[r][e];
      const Fragment<float> w(column);
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[e][t] = Fragment<float>::product(w, d[t], acc[e][t]);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<f32x4 *>(&sums[wave][16 * t + i][16 * g + 4 * r]) =
          f32x4{acc[0][t][r], acc[1][t][r], acc[2][t][r], acc[3][t][r]};
  __syncthreads();
  for (int o = threadIdx.x; o < MT * 256; o += 256) {
    const int m = o / 16, col = o % 16 * 4, n = blockIdx.x * 64 + col;
    if (m >= p.m || n >= p.k) continue;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) v += *reinterpret_cast<const f32x4 *>(&sums[w][m][col]);
    if (p.part) *reinterpret_cast<f32x4 *>(p.part + blockIdx.y * p.step + m * p.ld + n) = v;
    else finish<float, true>(p.f, m, n, p.k - n, v);
  }
}

// dW: a wave takes 64 columns, whose fragments of A stay in registers, and kTall rows, 16 at a time;
// one instruction sums over all rows of dP and A.  A lane's four sums are neighbours in a row.
constexpr int kTall = 64;
__global__ __launch_bounds__(256) void few_dw_kernel(FewRows p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, m = 8 * (lane >> 4);
  const int c0 = (blockIdx.x * 4 + wave) * 64;
  if (c0 >= p.k) return;
  auto eight = [&](const float *x, int64_t ld, int at, int cols) __attribute__((always_inline)) {
    Eight<float> v;
#pragma unroll
    for (int r = 0; r < 8; ++r) v.v[r] = m + r < p.m && at < cols ? x[(int64_t)(m + r) * ld + at] : 0.0f;
    return v;
  };
  const int first = blockIdx.y * kTall, last = min(first + kTall, p.n);
  Eight<float> next = eight(p.dp, p.lddp, first + i, p.n);
  Fragment<float> a[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) a[e] = Fragment<float>(eight(p.a, p.lda, c0 + 16 * e + i, p.k));
  for (int j0 = first; j0 < last; j0 += 16) {
    const Fragment<float> d(next);
    if (j0 + 16 < last) next = eight(p.dp, p.lddp, j0 + 16 + i, p.n);
    f32x4 acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = Fragment<float>::product(a[e], d, f32x4{0, 0, 0, 0});
    if (j0 + i >= p.n) continue;
    float *to = static_cast<float *>(p.f.out) + (int64_t)(j0 + i) * p.f.ldo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = c0 + 16 * e + 4 * (lane >> 4);
      if (c < p.k) store4(to + c, acc[e], p.k - c, p.f.vec_o);
    }
  }
}

// Parts of dA's sums: blocks for two a compute unit, each wave of a part with at least four steps.
struct FewParts {
  int parts, steps;
};
FewParts few_parts(int64_t n, int64_t k) {
  const int64_t blocks = std::max<int64_t>(1, (k + 63) / 64), steps = (n + 31) / 32;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>({512 / blocks, steps / 16, kMostParts}));
  const int64_t per = std::max<int64_t>(1, (steps + want - 1) / want);
  return FewParts{(int)std::max<int64_t>(1, (steps + per - 1) / per), (int)per};
}

// 16-bit types: rows up to which dP is held with its remainder.  bf16: as long as that is faster than fp16 by
// powers of two (gradient by 256 rows of 4096 x 4096 81 and 79 us, by 384 105 and 90, of 11008 x 4096 191 and
// 198, by 512 254 and 222, by 4096 1329 and 833; 512 x 1536 x 384 38 and 42, 2048 of it 52 and 50).
template <class T>
constexpr int kTwice = std::is_same_v<T, __bf16> ? 384 : 128;
// Whether W and A are laid out by powers of two, too.
template <class T>
constexpr bool kAll = !std::is_same_v<T, _Float16>;

struct Call {
  int64_t m, n, k;
  const void *dc, *a, *w, *pre;
  int64_t lddc, lda, ldw, ldp;
  int act;
  void *da, *dw, *dbias;
  int64_t ldda, lddw;
  char *ws;
};

struct Plan {
  int64_t np, kp;
  int64_t tops_at, p_at, pc_at, a_at, w_at, sums_at, parts_at, total;
};

template <class T>
Plan plan(int64_t m, int64_t n, int64_t k) {
  Plan p{};
  Room r;
  constexpr int P = kPlanes<T>;
  p.np = round_up(n, P == 2 ? 32 : 8);
  p.kp = round_up(k, P == 2 ? 32 : 8);
  if (few_rows<T>(m)) {
    p.p_at = r.take(m * p.np * 4);
    const int parts = few_parts(n, k).parts;
    p.parts_at = r.take(parts > 1 ? parts * m * round_up(k, 4) * 4 : 0);
    p.total = r.at;
    return p;
  }
  // (whatever the activation)
  const int fold = P == 1 && m <= kTwice<T> ? 2 : 1;
  const bool held = fold == 1 || std::is_same_v<T, _Float16>;
  p.tops_at = r.take(held ? (round_up(m, 64) + round_up(n, 64) + 2 * round_up(k, 64)) * 4 : 0);
  p.p_at = r.take(fold * P * m * p.np * 2);
  p.pc_at = r.take(held ? fold * P * m * p.np * 2 : 0);
  p.a_at = r.take(fold * P * m * p.kp * 2);
  p.w_at = r.take(P * n * p.kp * 2);
  p.sums_at = r.take((m + kRows - 1) / kRows * p.np * 4);
  p.parts_at = r.take(std::max({parts_bytes<T, false>(m, k, n), parts_bytes<T, false>(m, k, n, fold),
                                parts_bytes<T, true>(n, k, m), parts_bytes<T, true>(n, k, fold * m)}));
  p.total = r.at;
  return p;
}
Plan plan_of(int64_t m, int64_t n, int64_t k, int type) {
  return type == OG_F32 ? plan<float>(m, n, k) : type == OG_BF16 ? plan<__bf16>(m, n, k) : plan<_Float16>(m, n, k);
}

template <class T>
int sweep_blocks(const Matrix &a) {
  return (int)((int64_t)((a.rows + a.rows_per - 1) / a.rows_per) * ((a.width + kCols<T> - 1) / kCols<T>));
}
// Whether a lane's columns are one aligned load.
template <class T>
int lanes_whole(const void *p, int64_t ld) {
  return ld % kPer<T> == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

template <class T>
Finish output(void *out, int64_t ld, const float *mtop, const float *ntop) {
  Finish f{};
  f.mtop = mtop;
  f.ntop = ntop;
  f.out = out;
  f.ldo = ld;
  return set_accesses<T>(f);
}

void few_gradient(const Call &c, const Plan &p, hipStream_t s) {
  const int m = (int)c.m, n = (int)c.n, k = (int)c.k;
  const bool place = c.act == OG_ACT_NONE;  // dC is dP
  Matrix a{};
  a.x = c.dc;
  a.ldx = c.lddc;
  a.pre = place ? nullptr : c.pre;
  a.ldp = c.ldp;
  a.act = c.act;
  a.rows = m;
  a.cols = n;
  a.width = (int)p.np;
  a.rows_per = kFew;
  a.vec_x = lanes_whole<float>(c.dc, c.lddc);
  a.vec_p = lanes_whole<float>(c.pre, c.ldp);
  a.bias = c.dbias;
  if (!place && (c.da || c.dw)) a.plain = reinterpret_cast<float *>(c.ws + p.p_at);
  a.blocks = (a.width + kCols<float> - 1) / kCols<float>;  // (m 0 clears dbias)
  if (a.blocks > 0 && (a.bias || a.plain)) {
    hipLaunchKernelGGL((sweep_kernel<float, false, true>), dim3(a.blocks), dim3(64 * kWaves), 0, s, a, Matrix{}, Matrix{});
  }
  FewRows q{};
  q.m = m, q.n = n, q.k = k;
  q.dp = place ? static_cast<const float *>(c.dc) : a.plain;
  q.lddp = place ? c.lddc : p.np;
  q.a = static_cast<const float *>(c.a), q.w = static_cast<const float *>(c.w);
  q.lda = c.lda, q.ldw = c.ldw;
  if (c.da) {
    const FewParts parts = few_parts(n, k);
    q.f = output<float>(c.da, c.ldda, nullptr, nullptr);
    q.vec = whole(q.w, q.ldw);
    q.steps = parts.steps;
    if (parts.parts > 1) {
      q.part = reinterpret_cast<float *>(c.ws + p.parts_at);
      q.ld = round_up(k, 4);
      q.step = m * q.ld;
    }
    const dim3 grid((k + 63) / 64, parts.parts);
    if (m <= 16) hipLaunchKernelGGL(few_da_kernel<1>, grid, dim3(256), 0, s, q);
    else hipLaunchKernelGGL(few_da_kernel<2>, grid, dim3(256), 0, s, q);
    if (q.part) {
      const int64_t quads = (int64_t)m * ((k + 3) / 4);
      hipLaunchKernelGGL((join_kernel<float, true, 1>), dim3((unsigned)std::min<int64_t>((quads + 255) / 256, 4096)),
                         dim3(256), 0, s, m, k, parts.parts, q.part, q.ld, q.step, q.f);
    }
  }
  if (c.dw) {
    q.f = output<float>(c.dw, c.lddw, nullptr, nullptr);
    hipLaunchKernelGGL(few_dw_kernel, dim3((k + 255) / 256, (n + kTall - 1) / kTall), dim3(256), 0, s, q);
  }
}

template <class T>
void gradient(const Call &c, const Plan &p, hipStream_t s) {
  if (few_rows<T>(c.m)) return few_gradient(c, p, s);
  constexpr int P = kPlanes<T>;
  const int m = (int)c.m, n = (int)c.n, k = (int)c.k;
  auto at = [&](int64_t place) { return reinterpret_cast<uint16_t *>(c.ws + place); };
  const bool same = c.act == OG_ACT_NONE;
  // a dP of more bits than the type, wanted as an operand
  const bool rounds = P == 1 && m > 0 && c.act > OG_ACT_RELU && (c.da || c.dw);
  const int fold = rounds && m <= kTwice<T> ? 2 : 1;
  // dP by powers of two
  const bool held = P == 2 || (rounds && (fold == 1 || std::is_same_v<T, _Float16>));
  Matrix dp{};
  dp.rows_per = rows_per<T>(m, P == 2 || c.act > OG_ACT_RELU);  // (dbias is the same whatever else is wanted)
  dp.x = c.dc;
  dp.ldx = c.lddc;
  dp.pre = same ? nullptr : c.pre;
  dp.ldp = c.ldp;
  dp.act = c.act;
  dp.rows = m;
  dp.cols = n;
  dp.width = (int)p.np;
  dp.vec_x = lanes_whole<T>(c.dc, c.lddc);
  dp.vec_p = lanes_whole<T>(c.pre, c.ldp);
  dp.bias = c.dbias;
  dp.sums = c.dbias ? reinterpret_cast<float *>(c.ws + p.sums_at) : nullptr;
  Operand rows, cols, A, W;  // dP by rows and by columns, A, W
  const float *rtop = nullptr, *ctop = nullptr, *atop = nullptr, *wtop = nullptr;
  dp.twice = fold == 2;
  if (P == 1 && m <= kRows) dp.sums = nullptr;  // one row block has all of a column's sum
  if constexpr (kPowers<T, true>) {
    if (held) {
      float *tops = reinterpret_cast<float *>(c.ws + p.tops_at);
      float *r = tops, *t = r + round_up(m, 64), *ta = t + round_up(n, 64), *tw = ta + round_up(k, 64);
      const int64_t total = tw + round_up(k, 64) - tops;
      auto of = [&](const void *x, int64_t ld, int64_t count, float *top, uint16_t *out) {
        Matrix a{};
        a.rows_per = rows_per<T>(count, true);
        a.x = x;
        a.ldx = ld;
        a.rows = (int)count;
        a.cols = k;
        a.width = (int)p.kp;
        a.vec_x = lanes_whole<T>(x, ld);
        a.ctop = top;
        a.out_c = out;
        return a;
      };
      Matrix ma{}, mw{};
      ma.rows_per = mw.rows_per = kRows;
      if (c.da) {
        dp.rtop = r;
        dp.out = at(p.p_at);
        if (kAll<T>) mw = of(c.w, c.ldw, n, tw, at(p.w_at));
      }
      if (c.dw) {
        dp.ctop = t;
        dp.out_c = at(p.pc_at);
        if (kAll<T>) ma = of(c.a, c.lda, m, ta, at(p.a_at));
      }
      for (Matrix *x : {&dp, &ma, &mw}) x->blocks = sweep_blocks<T>(*x);
      const int blocks = dp.blocks + ma.blocks + mw.blocks;
      hipLaunchKernelGGL(clear_kernel, dim3((unsigned)std::min<int64_t>((total + 255) / 256, 1024)), dim3(256), 0, s,
                         tops, total);
      if (blocks > 0)
        hipLaunchKernelGGL((sweep_kernel<T, false, true>), dim3(blocks), dim3(64 * kWaves), 0, s, dp, ma, mw);
      if (blocks > 0 && (c.da || c.dw)) {
        const int behind = dp.sums ? (n + 63) / 64 : 0;
        hipLaunchKernelGGL((sweep_kernel<T, true, true>), dim3(blocks + behind), dim3(64 * kWaves), 0, s, dp, ma, mw);
        dp.sums = nullptr;  // (done)
      }
      rows = Operand{at(p.p_at), P * p.np, 0};
      cols = Operand{at(p.pc_at), P * p.np, 0};
      rtop = r, ctop = t;
      if (kAll<T>) {
        A = Operand{at(p.a_at), P * p.kp, 0};
        W = Operand{at(p.w_at), P * p.kp, 0};
        atop = ta, wtop = tw;
      }
    }
  }
  if constexpr (P == 1) {
    if (!held) {
      const bool place = same && readable(c.dc, n, c.lddc);
      dp.out = place || !(c.da || c.dw) ? nullptr : at(p.p_at);
      if (dp.out || dp.bias) {
        // (m 0 clears dbias)
        dp.blocks = std::max(sweep_blocks<T>(dp), dp.bias && !dp.sums ? (dp.width + kCols<T> - 1) / kCols<T> : 0);
        if (dp.blocks > 0)
          hipLaunchKernelGGL((sweep_kernel<T, false, false>), dim3(dp.blocks), dim3(64 * kWaves), 0, s, dp, Matrix{},
                             Matrix{});
      }
      rows = cols = place ? Operand{static_cast<const uint16_t *>(c.dc), c.lddc, 0} : Operand{at(p.p_at), p.np, 0};
    }
    if (!held || !kAll<T>) {
      if (c.dw) A = operand16<T>(c.a, c.lda, m, k, p.kp, c.ws + p.a_at, s, fold);
      if (c.da) W = operand16<T>(c.w, c.ldw, n, k, p.kp, c.ws + p.w_at, s);
    }
  }
  if (dp.sums) hipLaunchKernelGGL(bias_kernel<T>, dim3((n + 63) / 64), dim3(1024), 0, s, dp);
  auto products = [&](auto element) {
    using E = decltype(element);
    Args g{};
    if (c.da && m > 0 && k > 0) {
      g.a = rows, g.b = W, g.M = fold * m, g.N = k, g.K = n;
      run_product<T, false, true, true, E>(g, output<T>(c.da, c.ldda, rtop, wtop), c.ws + p.parts_at, s, fold);
    }
    if (c.dw && n > 0 && k > 0) {
      g.a = cols, g.b = A, g.M = n, g.N = k, g.K = fold * m;
      run_product<T, true, true, true, E>(g, output<T>(c.dw, c.lddw, ctop, atop), c.ws + p.parts_at, s);
    }
  };
  if (held) products(_Float16());
  else products(Element<T>());
}

}  // namespace og::epi::grad

extern "C" {

int64_t og_gemm_nt_epi_grad_workspace(int64_t m, int64_t n, int64_t k, int type) {
  const og_status st = og::epi::check_sizes(m, n, k, type);
  if (st != OG_OK) return st;
  og::host::ok();
  return og::epi::grad::plan_of(m, n, k, type).total;
}

og_status og_gemm_nt_epi_grad(int64_t m, int64_t n, int64_t k, const void *dC, int64_t lddc, const void *A,
                              int64_t lda, const void *W, int64_t ldw, int type, const void *P, int64_t ldp, int act,
                              void *dA, int64_t ldda, void *dW, int64_t lddw, void *dbias, void *workspace,
                              int64_t workspace_bytes) {
  using namespace og::host;
  using namespace og::epi;
  using namespace og::epi::grad;
  og_status st = check_sizes(m, n, k, type);
  if (st != OG_OK) return st;
  if (!valid_act(act)) return fail(OG_ERR_INVALID_ARG, "act %d: OG_ACT_NONE to OG_ACT_SILU", act);
  const int64_t least_k = std::max<int64_t>(1, k), least_n = std::max<int64_t>(1, n);
  if (lddc < least_n || (act != OG_ACT_NONE && ldp < least_n) || (dW && lda < least_k) || (dA && ldw < least_k) ||
      (dA && ldda < least_k) || (dW && lddw < least_k))
    return fail(OG_ERR_INVALID_ARG, "a row stride is below its row: lddc %lld, ldp %lld, lda %lld, ldw %lld, ldda "
                "%lld, lddw %lld", (long long)lddc, (long long)ldp, (long long)lda, (long long)ldw, (long long)ldda,
                (long long)lddw);
  // what there is to write
  const bool da = dA && m > 0 && k > 0, dw = dW && n > 0 && k > 0, db = dbias && n > 0;
  if (!da && !dw && !db) return ok();
  if (m > 0 && n > 0 && (!dC || (act != OG_ACT_NONE && !P) || (dw && !A) || (da && !W)))
    return fail(OG_ERR_INVALID_ARG, "dC, P, A or W is null");
  const Plan p = plan_of(m, n, k, type);
  if (p.total > 0 && (!workspace || workspace_bytes < p.total))
    return fail(OG_ERR_INVALID_ARG, "workspace of %lld bytes: %lld needed",
                (long long)(workspace ? workspace_bytes : 0), (long long)p.total);
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(OG_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if ((st = check_device()) != OG_OK) return st;
  const Call c{m, n, k, dC, A, W, P, lddc, lda, ldw, ldp, act, da ? dA : nullptr, dw ? dW : nullptr,
               db ? dbias : nullptr, ldda, lddw, static_cast<char *>(workspace)};
  if (type == OG_F32) gradient<float>(c, p, current_stream());
  else if (type == OG_BF16) gradient<__bf16>(c, p, current_stream());
  else gradient<_Float16>(c, p, current_stream());
  return check_launch("gemm_nt_epi_grad");
}

}  // extern "C"
