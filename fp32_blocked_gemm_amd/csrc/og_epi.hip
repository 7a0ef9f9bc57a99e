// og_epi.hip -- og_gemm_nt_epi: C = act(A W^T + bias) + residual.
//
// The epilogue runs on the finished fp32 sums, so the sum is rounded to the
// type once, after the residual (and once for P, where it is wanted).
//
// fp32 matrices run as two fp16 planes (og_tile.hpp), each row of A and of W
// times a power of two of its own; 16-bit ones run where they lie, or from a
// copy where their rows are not whole aligned granules.
#include "og_epi.hpp"

namespace og::epi::fwd {

struct Call {
  int64_t m, n, k;
  const void *a, *w;
  int64_t lda, ldw;
  Finish f;
  char *ws;
};

// One or two matrices that a launch lays out, rows of `cols` values.
struct Side {
  const void *x;
  int64_t ld;
  int rows;
  uint16_t *out;
  float *top;
};

// fp32 rows as planes of `width` columns, zero past the row, by the power of the row's largest
// magnitude, which goes to top.  WR waves take a row, whose first columns stay in registers
// between its maximum and its planes: one wave up to 1024 columns, four of more (512 and 11008 rows
// of 4096 in 58 us, 6.5 TB/s of reads and writes with the caches' part, by one wave 88; 2000 and 2000
// of 2000 12 and 14; 4096 and 1536 of 384 14 and 10).
constexpr int kHeld = 4;
template <int WR>
__global__ __launch_bounds__(256) void planes_kernel(Side a, Side b, int cols, int width, int vec_a, int vec_b) {
  __shared__ float tops[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = WR == 1 ? 4 * lane : 4 * threadIdx.x;
  constexpr int kStep = 256 * WR, kRows = 4 / WR;
  const int64_t i = (int64_t)blockIdx.x * kRows + (WR == 1 ? wave : 0);
  const bool of_a = i < a.rows;
  const int64_t r = of_a ? i : i - a.rows;
  const bool in = r < (of_a ? a.rows : b.rows);  // (WR 4: one for the block)
  const int left = in ? cols : 0;
  const bool vec = of_a ? vec_a : vec_b;
  const float *row = static_cast<const float *>(of_a ? a.x : b.x) + r * (of_a ? a.ld : b.ld);
  f32x4 held[kHeld];
  float top = 0;
  auto larger = [&](const f32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, __builtin_isfinite(v[e]) ? fabsf(v[e]) : 0.0f);
  };
#pragma unroll
  for (int q = 0; q < kHeld; ++q) held[q] = load4(row + first + kStep * q, left - first - kStep * q, vec);
#pragma unroll
  for (int q = 0; q < kHeld; ++q) larger(held[q]);
  for (int c = first + kStep * kHeld; c < left; c += kStep) larger(load4(row + c, left - c, vec));
  top = wave_max(top);
  if constexpr (WR == 4) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  }
  if (!in) return;
  if (first == 0) (of_a ? a.top : b.top)[r] = top;
  uint16_t *out = (of_a ? a.out : b.out) + r * width * 2;
  const int p = power_of(top), powers[4] = {p, p, p, p};
#pragma unroll
  for (int q = 0; q < kHeld; ++q)
    if (first + kStep * q < width) store_planes(out, first + kStep * q, held[q], powers);
  for (int c = first + kStep * kHeld; c < width; c += kStep)
    store_planes(out, c, load4(row + c, cols - c, vec), powers);
}

// Few rows of A: bound by the bytes of W, which goes from memory to the matrix cores through
// registers alone.  A block takes 16 NT rows of W and 16 MT rows of A; its W waves share k (their
// sums meet in LDS, in wave order).  A lane's 16 bytes of a load are the 8 values its fragment
// needs, so that one instruction reads 64 neighbouring bytes of 16 rows.  The loads of the next
// chunk are in flight while one is multiplied.
struct Rows {
  int m, n, k;
  const void *a, *w;
  int64_t lda, ldw;
  Finish f;
};

template <class T, int MT, int NT>
struct Chunk {
  static constexpr int kSteps = sizeof(T) == 4 ? 2 : 4, kDepth = 32 * kSteps;
  Eight<T> w[NT][kSteps], x[MT][kSteps];
  template <bool FULL>
  __device__ __forceinline__ void load(const T *const (&a)[MT], const bool (&in)[MT], const T *const (&b)[NT], int k,
                                       int K) {
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int j = 0; j < kSteps; ++j) w[u][j] = load8<T, FULL>(b[u], k + 32 * j, K);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
        if (in[t]) x[t][j] = load8<T, FULL>(a[t], k + 32 * j, K);
  }
};

template <class T, int W, int MT, int NT>
__global__ __launch_bounds__(W * 64) void rows_kernel(Rows p) {
  using C = Chunk<T, MT, NT>;
  __shared__ __align__(16) float sums[W][16 * MT][16 * NT + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int across = (p.n + 16 * NT - 1) / (16 * NT), below = blockIdx.x / across;
  const int n0 = (blockIdx.x - below * across) * 16 * NT, m0 = below * 16 * MT;
  const int chunks = (p.k + C::kDepth - 1) / C::kDepth;
  const int c0 = (int)((int64_t)chunks * wave / W), c1 = (int)((int64_t)chunks * (wave + 1) / W);
  const T *a[MT], *b[NT];
  bool in[MT];
  C next;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + i;
    in[t] = m < p.m;
    a[t] = static_cast<const T *>(p.a) + (int64_t)min(m, p.m - 1) * p.lda;
#pragma unroll
    for (int j = 0; j < C::kSteps; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) next.x[t][j].v[e] = (T)0.0f;  // what rows past m hold
  }
#pragma unroll
  for (int u = 0; u < NT; ++u) b[u] = static_cast<const T *>(p.w) + (int64_t)min(n0 + 16 * u + i, p.n - 1) * p.ldw;
  auto load = [&](int c) __attribute__((always_inline)) {
    const int k = c * C::kDepth + 8 * g;
    if ((c + 1) * C::kDepth <= p.k) next.template load<true>(a, in, b, k, p.k);
    else next.template load<false>(a, in, b, k, p.k);
  };
  // acc[u][t][r]: row 16 u + i of W, row 16 t + 4 g + r of A
  f32x4 acc[NT][MT];
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[u][t] = f32x4{0, 0, 0, 0};
  if (c0 < c1) load(c0);
  for (int c = c0; c < c1; ++c) {
    const C now = next;
    if (c + 1 < c1) load(c + 1);
#pragma unroll
    for (int j = 0; j < C::kSteps; ++j) {
      Fragment<T> w[NT];
#pragma unroll
      for (int u = 0; u < NT; ++u) w[u] = Fragment<T>(now.w[u][j]);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const Fragment<T> x(now.x[t][j]);
#pragma unroll
        for (int u = 0; u < NT; ++u) acc[u][t] = Fragment<T>::product(x, w[u], acc[u][t]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave][16 * t + 4 * g + r][16 * u + i] = acc[u][t][r];
  __syncthreads();
  for (int o = threadIdx.x; o < MT * NT * 64; o += W * 64) {
    const int row = o / (4 * NT), col = o % (4 * NT) * 4, m = m0 + row, n = n0 + col;
    if (m >= p.m || n >= p.n) continue;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const f32x4 part = *reinterpret_cast<const f32x4 *>(&sums[w][row][col]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += part[e];
    }
    finish<T, false>(p.f, m, n, p.n - n, v);
  }
}

template <class T, int W, int MT, int NT>
void launch_rows(const Rows &p, hipStream_t s) {
  // (one axis: a second would end at 65535 blocks)
  const unsigned across = (p.n + 16 * NT - 1) / (16 * NT), below = (p.m + 16 * MT - 1) / (16 * MT);
  hipLaunchKernelGGL((rows_kernel<T, W, MT, NT>), dim3(across * below), dim3(W * 64), 0, s, p);
}

// Whether a product runs on the rows kernel: up to 16 rows (fp32: 64, whose tile product needs
// the planes of W made first), or where W read once for each 16 (32) rows is little.  us, rows
// kernel and tile product, W rotating through memory: 16 rows of bf16 on 11008 x 4096 27.4 and 26.9,
// on 4096 x 4096 10.7 and 12.3; 32 there 17.7 and 12.9; 64 on 1531 x 1000 5.1 and 8.6, 128 6.4 and 8.5.
// fp32: 64 rows on 11008 x 4096 101 and 148, 128 186 and 153; 128 on 1531 x 1000 12.9 and 15.8.
//
// A block takes its time however little of k there is, so that more of them than run at once (four a
// compute unit) are for tiles, whose blocks are larger: 4096 x 4096 x 16 in bf16 359 and 17 us (fp32 166 and 27),
// 2048 x 2048 x 32 81 and 10 (37 and 14), 65536 x 64 x 64 74 and 11, 14 x 58422 x 136 26 and 10; but not where
// 16 rows have much of k each (a block's bytes then take longer), nor narrow fp32 products, for which tiles are
// half empty and all of A is laid out first (65536 x 64 x 64 28 and 39).  (110 seeded products for each type of 1
// to 65536 rows, 4 to 65536 columns and k of 4 to 16384: the chosen kernel takes 1.05 times the faster
// one's time in the mean in bf16, 1.04 in fp32, 110 others 1.02 and 1.03; odd k of some thousands up to 2.9.)
template <class T>
bool few_rows(int64_t m, int64_t n, int64_t k) {
  constexpr bool wide = sizeof(T) == 4;
  constexpr int64_t tile = wide ? 32 : 16, most = wide ? 1 << 23 : 1 << 24;
  const int64_t down = (m + tile - 1) / tile, blocks = down * ((n + tile - 1) / tile);
  const bool little = down * n * std::max<int64_t>(k, 1) <= most;
  if constexpr (wide) return m <= 64 || (little && (n <= 64 || blocks <= 1024));
  return blocks <= 1024 ? m <= 16 || little : m <= 16 && k >= 512;
}

// Tiles of a block: one of each up to 16 rows and for 16-bit types (11008 x 4096 bf16 by one row
// 21.3 us, two tiles of W 24.5); two of A for more of fp32, and two of W where that leaves every
// compute unit a block (4096 x 11008 by 64 rows 89 us with two, 124 with one; by 32, 128 blocks, 89
// and 72).  Bound by the bytes of W: 90 MB of bf16 by one row at 4.2 TB/s, 180 MB of fp32 in 41 us at 4.4.
template <class T>
void run_rows(const Rows &p, hipStream_t s) {
  if constexpr (sizeof(T) == 4) {
    if (p.m > 16) {
      const bool many = (int64_t)((p.n + 31) / 32) * ((p.m + 31) / 32) >= 256;
      return many ? launch_rows<T, 4, 2, 2>(p, s) : launch_rows<T, 4, 2, 1>(p, s);
    }
  }
  launch_rows<T, 8, 1, 1>(p, s);
}

struct Plan {
  int64_t kp;  // k padded
  int64_t tops_at, a_at, w_at, parts_at, total;
};

template <class T>
Plan plan(int64_t m, int64_t n, int64_t k) {
  Plan p{};
  Room r;
  constexpr int P = kPlanes<T>;
  p.kp = round_up(k, P == 2 ? 32 : 8);
  if (few_rows<T>(m, n, k)) return Plan{};
  p.tops_at = r.take(P == 2 ? (round_up(m, 64) + round_up(n, 64)) * 4 : 0);
  p.a_at = r.take(P * m * p.kp * 2);
  p.w_at = r.take(P * n * p.kp * 2);
  p.parts_at = r.take(parts_bytes<T, false>(m, n, k));
  p.total = r.at;
  return p;
}
Plan plan_of(int64_t m, int64_t n, int64_t k, int type) {
  return type == OG_F32 ? plan<float>(m, n, k) : type == OG_BF16 ? plan<__bf16>(m, n, k) : plan<_Float16>(m, n, k);
}

template <class T>
void forward(const Call &c, const Plan &p, hipStream_t s) {
  Finish f = set_accesses<T>(c.f);
  if (few_rows<T>(c.m, c.n, c.k)) {
    run_rows<T>(Rows{(int)c.m, (int)c.n, (int)c.k, c.a, c.w, c.lda, c.ldw, f}, s);
    return;
  }
  Args g{};
  g.M = (int)c.m;
  g.N = (int)c.n;
  g.K = (int)c.k;
  if constexpr (kPlanes<T> == 2) {
    float *mtop = reinterpret_cast<float *>(c.ws + p.tops_at), *ntop = mtop + round_up(c.m, 64);
    uint16_t *a = reinterpret_cast<uint16_t *>(c.ws + p.a_at), *w = reinterpret_cast<uint16_t *>(c.ws + p.w_at);
    const int64_t rows = c.m + c.n;
    const Side sa{c.a, c.lda, (int)c.m, a, mtop}, sw{c.w, c.ldw, (int)c.n, w, ntop};
    const bool wide = c.k > 256 * kHeld && rows <= (1 << 22);  // (a launch has fewer than 2^32 threads)
    hipLaunchKernelGGL(wide ? planes_kernel<4> : planes_kernel<1>, dim3((unsigned)(wide ? rows : (rows + 3) / 4)),
                       dim3(256), 0, s, sa, sw, (int)c.k, (int)p.kp, whole(static_cast<const float *>(c.a), c.lda),
                       whole(static_cast<const float *>(c.w), c.ldw));
    f.mtop = mtop;
    f.ntop = ntop;
    g.a = Operand{a, 2 * p.kp, 0};
    g.b = Operand{w, 2 * p.kp, 0};
  } else {
    g.a = operand16<T>(c.a, c.lda, c.m, c.k, p.kp, c.ws + p.a_at, s);
    g.b = operand16<T>(c.w, c.ldw, c.n, c.k, p.kp, c.ws + p.w_at, s);
  }
  run_product<T, false, false, false>(g, f, c.ws + p.parts_at, s);
}

}  // namespace og::epi::fwd

extern "C" {

int64_t og_gemm_nt_epi_workspace(int64_t m, int64_t n, int64_t k, int type) {
  const og_status st = og::epi::check_sizes(m, n, k, type);
  if (st != OG_OK) return st;
  og::host::ok();
  if (m == 0 || n == 0) return 0;
  return og::epi::fwd::plan_of(m, n, k, type).total;
}

og_status og_gemm_nt_epi(int64_t m, int64_t n, int64_t k, const void *A, int64_t lda, const void *W, int64_t ldw,
                         int type, const void *bias, int act, const void *residual, int64_t ldr, void *P, int64_t ldp,
                         void *C, int64_t ldc, void *workspace, int64_t workspace_bytes) {
  using namespace og::host;
  using namespace og::epi;
  using namespace og::epi::fwd;
  og_status st = check_sizes(m, n, k, type);
  if (st != OG_OK) return st;
  if (!valid_act(act)) return fail(OG_ERR_INVALID_ARG, "act %d: OG_ACT_NONE to OG_ACT_SILU", act);
  if (lda < std::max<int64_t>(1, k) || ldw < std::max<int64_t>(1, k) || ldc < std::max<int64_t>(1, n) ||
      (residual && ldr < std::max<int64_t>(1, n)) || (P && ldp < std::max<int64_t>(1, n)))
    return fail(OG_ERR_INVALID_ARG, "a row stride is below its row: lda %lld, ldw %lld, ldr %lld, ldp %lld, ldc %lld",
                (long long)lda, (long long)ldw, (long long)ldr, (long long)ldp, (long long)ldc);
  if (m == 0 || n == 0) return ok();
  if (!C || (k > 0 && (!A || !W))) return fail(OG_ERR_INVALID_ARG, "A, W or C is null");
  if (residual == C && ldr != ldc && m > 1)
    return fail(OG_ERR_INVALID_ARG, "a residual in the output needs its stride: ldr %lld, ldc %lld", (long long)ldr,
                (long long)ldc);
  if (P == C) return fail(OG_ERR_INVALID_ARG, "P and C are one buffer");
  const Plan p = plan_of(m, n, k, type);
  if (p.total > 0 && (!workspace || workspace_bytes < p.total))
    return fail(OG_ERR_INVALID_ARG, "workspace of %lld bytes: %lld needed",
                (long long)(workspace ? workspace_bytes : 0), (long long)p.total);
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(OG_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if ((st = check_device()) != OG_OK) return st;
  const Call c{m, n, k, A, W, lda, ldw,
               Finish{nullptr, nullptr, bias, act, residual, ldr, P, ldp, C, ldc, 0, 0, 0, 0, 0},
               static_cast<char *>(workspace)};
  if (type == OG_F32) forward<float>(c, p, current_stream());
  else if (type == OG_BF16) forward<__bf16>(c, p, current_stream());
  else forward<_Float16>(c, p, current_stream());
  return check_launch("gemm_nt_epi");
}

}  // extern "C"
