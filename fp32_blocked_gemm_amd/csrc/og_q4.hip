// og_q4.hip -- og_gemm_nt_q4: C = A W^T with W in 4 bits.
//
//   C[i][j] = sum over groups t of s[j][t] * sum over p in t of A[i][p] (q[j][p] - z[j][t])
//
// For one to some tens of rows of A the product is bound by the bytes of the
// codes, so both kernels are built around asking for all of them at once, in
// long rows (no branch lies between the loads of a piece of k: the pieces that
// reach the end of a row have code of their own), and around few operations
// per code.  A code becomes fp16 in one operation for two of them: OR-ed into
// the mantissa of 1024 it is 1024 + q, and subtracting 1024 + z is exact, so A
// is multiplied by the whole numbers q - z, and the group's scale multiplies
// the fp32 sum of its terms (at least 32 of them).
//
//  - Up to 3 rows of A (fp32: 4): row_kernel, fp32 multiply-adds that take the fp16
//    code as an operand.  A lane holds 32 consecutive k of A in registers and
//    runs them against the same 32 of several weight rows.
//  - More: block_kernel on the matrix cores, 16 weight rows x 16 rows of A.
//    fp16 activations run against the fp16 codes; bf16 ones against the codes
//    made bf16 (whole numbers up to 255 are); fp32 ones as three bf16 planes,
//    24 bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "og.h"
#include "og_host.hpp"

namespace og::q4 {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct Problem {
  int m, n, k;
  int group;            // a multiple of 32
  int shift;            // log2 of group, or -1
  const void *a;
  int64_t lda;
  const uint8_t *q;
  int64_t ldq;          // bytes
  const void *s;
  int s_type;
  int64_t lds;
  const uint8_t *z;     // null: 8
  int64_t ldz;
  void *c;
  int64_t ldc;
};

__device__ __forceinline__ int group_of(const Problem &p, int k) {
  return p.shift >= 0 ? k >> p.shift : k / p.group;
}

// A group's scale and zero point as they lie in memory, so that nothing waits
// for them where they are loaded, and as values.
struct Group {
  uint32_t s, z;
  __device__ __forceinline__ void load(const Problem &p, int64_t n, int64_t t) {
    const int64_t i = n * p.lds + t;
    if (p.s_type == OG_F32) s = static_cast<const uint32_t *>(p.s)[i];
    else s = static_cast<const uint16_t *>(p.s)[i];
    z = p.z ? p.z[n * p.ldz + t] : 8;
  }
  __device__ __forceinline__ float scale(int type) const {
    const float h = (float)__builtin_bit_cast(_Float16, (uint16_t)s);
    const float b = __builtin_bit_cast(float, s << 16);
    return type == OG_F32 ? __builtin_bit_cast(float, s) : type == OG_BF16 ? b : h;
  }
  // -(1024 + z) twice
  __device__ __forceinline__ f16x2 minus_zero() const {
    const _Float16 h = (_Float16)(float)(-1024 - (int)z);
    return f16x2{h, h};
  }
};

// Two of a dword's codes (nibbles J and J + 4) as fp16, less the zero point.
template <int J>
__device__ __forceinline__ f16x2 codes(uint32_t w, f16x2 minus_zero) {
  const uint32_t b = ((w >> (4 * J)) & 0x000F000Fu) | 0x64006400u;
  return __builtin_bit_cast(f16x2, b) + minus_zero;
}

// 16 bytes of a row of `size` (at least 16) from byte `at` on; FULL false: zero
// past its end, by loading its last 16 bytes and shifting.  (No branch holds
// the loads of a piece apart.)
template <bool FULL>
__device__ __forceinline__ u32x4 load16(const uint8_t *row, int at, int size) {
  u32x4 w;
  if constexpr (FULL) {
    __builtin_memcpy(&w, row + at, 16);
  } else {
    const int from = min(at, size - 16), past = 8 * (at - from);
    unsigned __int128 v;
    __builtin_memcpy(&v, row + from, 16);
    v = past < 128 ? v >> past : 0;
    __builtin_memcpy(&w, &v, 16);
  }
  return w;
}

// 32 codes of a row from k on (k a multiple of 32).
template <bool FULL>
__device__ __forceinline__ u32x4 load_codes(const uint8_t *row, int k, int K) {
  return load16<FULL>(row, k >> 1, (K + 1) >> 1);
}

template <class T>
struct Eight {
  T v[8];
};
// Eight activations of a row from k on.
template <class T, bool FULL>
__device__ __forceinline__ Eight<T> load8(const T *row, int k, int K) {
  Eight<T> t;
  u32x4 w[sizeof t / 16];
#pragma unroll
  for (int i = 0; i < (int)sizeof t / 16; ++i)
    w[i] = load16<FULL>(reinterpret_cast<const uint8_t *>(row), k * (int)sizeof(T) + 16 * i,
                        K * (int)sizeof(T));
  __builtin_memcpy(&t, w, sizeof t);
  return t;
}

// Sum over the wave, in every lane.  The swaps exchange rows of 16 (then
// halves) of two registers; given one register twice the compiler takes both
// results for equal, so the second is a copy it cannot see through.
__device__ __forceinline__ float wave_sum(float v) {
  auto bits = [](float x) { return __builtin_bit_cast(uint32_t, x); };
  auto value = [](uint32_t x) { return __builtin_bit_cast(float, x); };
#define OG_ROR(N) v += value(__builtin_amdgcn_mov_dpp(bits(v), 0x120 + N, 0xf, 0xf, true))
  OG_ROR(8);
  OG_ROR(4);
  OG_ROR(2);
  OG_ROR(1);
#undef OG_ROR
  uint32_t u = bits(v), copy = u;
  asm volatile("" : "+v"(copy));
  const u32x2 a = __builtin_amdgcn_permlane16_swap(u, copy, false, false);
  u = copy = bits(value(a[0]) + value(a[1]));
  asm volatile("" : "+v"(copy));
  const u32x2 b = __builtin_amdgcn_permlane32_swap(u, copy, false, false);
  return value(b[0]) + value(b[1]);
}

// 32 k of R weight rows against M rows of A.
template <class T, int M, int R, bool FULL>
__device__ __forceinline__ void row_piece(const Problem &p, const int64_t (&row)[R], int k,
                                          float (&acc)[M][R]) {
  u32x4 w[R];
  Group gr[R];
  Eight<T> x[M][4];
  const int t = group_of(p, k);
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = load_codes<FULL>(p.q + row[r] * p.ldq, k, p.k);
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int d = 0; d < 4; ++d)
      x[m][d] = load8<T, FULL>(static_cast<const T *>(p.a) + m * p.lda, k + 8 * d, p.k);
#pragma unroll
  for (int r = 0; r < R; ++r) gr[r].load(p, row[r], t);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const f16x2 mz = gr[r].minus_zero();
    float sum[M][2];
#pragma unroll
    for (int m = 0; m < M; ++m) sum[m][0] = sum[m][1] = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const f16x2 q[4] = {codes<0>(w[r][d], mz), codes<1>(w[r][d], mz), codes<2>(w[r][d], mz),
                          codes<3>(w[r][d], mz)};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < M; ++m) {
          sum[m][0] = fmaf((float)q[j][0], (float)x[m][d].v[j], sum[m][0]);
          sum[m][1] = fmaf((float)q[j][1], (float)x[m][d].v[j + 4], sum[m][1]);
        }
    }
    const float s = gr[r].scale(p.s_type);
#pragma unroll
    for (int m = 0; m < M; ++m) acc[m][r] = fmaf(s, sum[m][0] + sum[m][1], acc[m][r]);
  }
}

// Up to 4 rows of A.  Block: 4 waves; KS of them share R weight rows, each
// taking every KS-th piece of 2048 k (64 lanes x 32).  Bound by the bytes of the
// codes and, for small layers, by the time of one load after another (calls in a
// graph, weights in turn): 4096 x 4096 by one bf16 row 5.2 us (8.7 MB), 11008 x 4096
// 8.7, by a fp32 row 10.2.
template <class T, int M, int R, int KS>
__global__ __launch_bounds__(256) void row_kernel(Problem p) {
  __shared__ float part[4][M * R];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = wave % KS, n0 = (blockIdx.x * (4 / KS) + wave / KS) * R;
  float acc[M][R];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[m][r] = 0;
  if (n0 < p.n) {
    int64_t row[R];
#pragma unroll
    for (int r = 0; r < R; ++r) row[r] = min(n0 + r, p.n - 1);
    for (int k0 = ks * 2048; k0 < p.k; k0 += KS * 2048) {
      const int k = k0 + lane * 32;
      if (k + 32 <= p.k) row_piece<T, M, R, true>(p, row, k, acc);
      else if (k < p.k) row_piece<T, M, R, false>(p, row, k, acc);
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float v = wave_sum(acc[m][r]);
      if (lane == 0) part[wave][m * R + r] = v;
    }
  __syncthreads();
  // (wave group, m, r) of the block's sums, the pieces of k in order
  for (int o = threadIdx.x; o < 4 / KS * M * R; o += 256) {
    const int group = o / (M * R), m = o % (M * R) / R, r = o % R;
    float v = 0;
#pragma unroll
    for (int q = 0; q < KS; ++q) v += part[group * KS + q][m * R + r];
    const int n = (blockIdx.x * (4 / KS) + group) * R + r;
    if (n < p.n) static_cast<T *>(p.c)[m * p.ldc + n] = (T)v;
  }
}

// The element type and planes of a block's fragments.
template <class T>
struct Planes {
  using V = bf16x8;
  static constexpr int P = sizeof(T) == 4 ? 3 : 1;
  // the planes of eight activations in the order of the codes' extraction:
  // 0 4 1 5 2 6 3 7 (nibbles j and j + 4 of a dword come out together)
  static __device__ __forceinline__ void split(const Eight<T> &x, V (&out)[P]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int from = (e >> 1) + 4 * (e & 1);
      if constexpr (P == 1) {
        out[0][e] = x.v[from];
      } else {
        // by cutting, not rounding: each plane takes the next 8 bits, 24 in all, and the largest
        // values have no bf16 above them to become infinite (a NaN is made quiet first: its
        // highest mantissa bit then stays)
        float r = __builtin_canonicalizef(x.v[from]);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          const uint32_t top = __builtin_bit_cast(uint32_t, r) & 0xFFFF0000u;
          const float h = __builtin_bit_cast(float, top);
          out[q][e] = __builtin_bit_cast(__bf16, (uint16_t)(top >> 16));
          r = __builtin_isfinite(h) ? r - h : 0.0f;
        }
      }
    }
  }
  static __device__ __forceinline__ V weights(const f16x2 (&q)[4]) {
    V w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = (__bf16)(float)q[e >> 1][e & 1];
    return w;
  }
  static __device__ __forceinline__ f32x4 mfma(V x, V w, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
  }
};
template <>
struct Planes<_Float16> {
  using V = f16x8;
  static constexpr int P = 1;
  static __device__ __forceinline__ void split(const Eight<_Float16> &x, V (&out)[1]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[0][e] = x.v[(e >> 1) + 4 * (e & 1)];
  }
  static __device__ __forceinline__ V weights(const f16x2 (&q)[4]) {
    return V{q[0][0], q[0][1], q[1][0], q[1][1], q[2][0], q[2][1], q[3][0], q[3][1]};
  }
  static __device__ __forceinline__ f32x4 mfma(V x, V w, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w, c, 0, 0, 0);
  }
};

// 128 k of a wave's operands, as loaded.
template <class T, int MT, int NT>
struct Chunk {
  u32x4 w[NT];
  Group gr[NT];  // of the lane's row and its lane group's 32 k
  Eight<T> x[MT][4];
  template <bool FULL>
  __device__ __forceinline__ void load(const Problem &p, const T *const (&a)[MT], const bool (&in)[MT],
                                       const int64_t (&n)[NT], int c, int g) {
    const int k = c * 128, u = group_of(p, k + 32 * g);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w[t] = load_codes<FULL>(p.q + n[t] * p.ldq, k + 32 * g, p.k);
      // (a lane group past the row has a zero sum, which an infinite scale would make NaN)
      if (FULL || k + 32 * g < p.k) gr[t].load(p, n[t], u);
      else gr[t] = Group{0, 0};
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (in[t]) x[t][j] = load8<T, FULL>(a[t], k + 32 * j + 8 * g, p.k);
  }
};

// MT x 16 rows of A and NT x 16 weight rows per block; k split among W waves
// (their sums meet in LDS, in wave order), so that even a 4096-row layer has
// sixteen waves on every compute unit asking for its bytes at once.  Each lane
// takes 16 bytes (32 codes) of a weight row, 128 k in all; four lane-swap
// instructions transpose the dwords among the four lane groups so that each of
// the next four matrix-core instructions (16 x 16 x 32) covers 32 consecutive
// k, that is, one group of scales, which one lane group has loaded.  The
// operands of the next 128 k are read ahead.  Bound by the latency of those
// reads: 16 bf16 rows take 10.0 us on 4096 x 4096 (0.9 TB/s of codes), 20.4 on 4096 x
// 11008 and 22.3 on 11008 x 4096; with the codes not converted 8.8, 18.6 and 19.1, with
// A read from one place all along (it comes from L2 once per block, four times the
// codes' bytes) 10.1, 18.9 and 24.0.  64 rows on 11008 x 4096 take 44.
template <class T, int W, int MT, int NT>
__global__ __launch_bounds__(W * 64) void block_kernel(Problem p) {
  using Pl = Planes<T>;
  constexpr int P = Pl::P;
  __shared__ float sums[W][16 * MT][16 * NT + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
  const int chunks = (p.k + 127) / 128;
  const int c0 = (int)((int64_t)chunks * wave / W), c1 = (int)((int64_t)chunks * (wave + 1) / W);

  // lane i's rows of A (fragment rows) and of W (fragment columns)
  const T *a[MT];
  bool in[MT];
  Chunk<T, MT, NT> next;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = m0 + 16 * t + i;
    in[t] = m < p.m;
    a[t] = static_cast<const T *>(p.a) + (int64_t)min(m, p.m - 1) * p.lda;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) next.x[t][j].v[e] = (T)0.0f;  // what rows past m hold
  }
  int64_t n[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) n[t] = min(n0 + 16 * t + i, p.n - 1);
  auto load = [&](int c) __attribute__((always_inline)) {
    if (c * 128 + 128 <= p.k) next.template load<true>(p, a, in, n, c, g);
    else next.template load<false>(p, a, in, n, c, g);
  };
  // acc[u][t][r]: weight row 16 u + i, A row m0 + 16 t + 4 g + r
  f32x4 acc[NT][MT];
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[u][t] = f32x4{0, 0, 0, 0};

  if (c0 < c1) load(c0);
  for (int c = c0; c < c1; ++c) {
    const Chunk<T, MT, NT> now = next;
    if (c + 1 < c1) load(c + 1);
    typename Pl::V x[MT][4][P];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) Pl::split(now.x[t][j], x[t][j]);
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      // dword d of lane group g (k 32 g + 8 d) to dword g of lane group d
      const u32x2 s0 = __builtin_amdgcn_permlane32_swap(now.w[u][0], now.w[u][2], false, false);
      const u32x2 s1 = __builtin_amdgcn_permlane32_swap(now.w[u][1], now.w[u][3], false, false);
      const u32x2 lo = __builtin_amdgcn_permlane16_swap(s0[0], s1[0], false, false);
      const u32x2 hi = __builtin_amdgcn_permlane16_swap(s0[1], s1[1], false, false);
      const uint32_t d[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // the group that lane group j loaded
        const Group gr{(uint32_t)__shfl((int)now.gr[u].s, i + 16 * j),
                       (uint32_t)__shfl((int)now.gr[u].z, i + 16 * j)};
        const f16x2 mz = gr.minus_zero();
        const f16x2 q[4] = {codes<0>(d[j], mz), codes<1>(d[j], mz), codes<2>(d[j], mz), codes<3>(d[j], mz)};
        const typename Pl::V w = Pl::weights(q);
        const float s = gr.scale(p.s_type);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          f32x4 sum = {0, 0, 0, 0};
#pragma unroll
          for (int h = P - 1; h >= 0; --h) sum = Pl::mfma(x[t][j][h], w, sum);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[u][t][r] = fmaf(s, sum[r], acc[u][t][r]);
        }
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
  for (int o = threadIdx.x; o < MT * NT * 256; o += W * 64) {
    const int row = o / (16 * NT), col = o % (16 * NT);
    float v = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) v += sums[w][row][col];
    if (m0 + row < p.m && n0 + col < p.n)
      static_cast<T *>(p.c)[(int64_t)(m0 + row) * p.ldc + n0 + col] = (T)v;
  }
}

// Rows of fewer than 31 codes (16 bytes, what the others load at once): a thread an output.
template <class T>
__device__ __forceinline__ void short_one(const Problem &p, int64_t at) {
  const int m = (int)(at / p.n), n = (int)(at - (int64_t)m * p.n);
  const T *a = static_cast<const T *>(p.a) + m * p.lda;
  const uint8_t *q = p.q + n * p.ldq;
  float sum = 0, s = 0;  // (a single group: p.group >= 32 > k)
  if (p.k > 0) {
    Group g;
    g.load(p, n, 0);
    s = g.scale(p.s_type);
    for (int k = 0; k < p.k; ++k)
      sum = fmaf((float)((int)(q[k >> 1] >> (4 * (k & 1)) & 15) - (int)g.z), (float)a[k], sum);
  }
  static_cast<T *>(p.c)[m * p.ldc + n] = (T)(s * sum);
}
template <class T>
__global__ __launch_bounds__(256) void short_kernel(Problem p) {
  const int64_t total = (int64_t)p.m * p.n, step = (int64_t)gridDim.x * 256;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += step) short_one<T>(p, at);
}

template <class T, int M, int R>
void run_rows(const Problem &p, hipStream_t s) {
  const int groups = (p.n + R - 1) / R;
  // As many waves share a row as its pieces keep busy (one row of bf16: 1024 x
  // 8192 by one wave 8.3 us, by four 3.5; 11008 x 2048 6.2 and 8.4).
  const int pieces = (p.k + 2047) / 2048;
  const int ks = pieces >= 4 ? 4 : pieces >= 2 ? 2 : 1;
  const dim3 block(256);
  if (ks == 4)
    hipLaunchKernelGGL((row_kernel<T, M, R, 4>), dim3(groups), block, 0, s, p);
  else if (ks == 2)
    hipLaunchKernelGGL((row_kernel<T, M, R, 2>), dim3((groups + 1) / 2), block, 0, s, p);
  else
    hipLaunchKernelGGL((row_kernel<T, M, R, 1>), dim3((groups + 3) / 4), block, 0, s, p);
}

template <class T, int W, int MT, int NT>
void run_blocks(const Problem &p, hipStream_t s) {
  hipLaunchKernelGGL((block_kernel<T, W, MT, NT>),
                     dim3((p.n + 16 * NT - 1) / (16 * NT), (p.m + 16 * MT - 1) / (16 * MT)),
                     dim3(W * 64), 0, s, p);
}

template <class T>
void run(const Problem &p, hipStream_t s) {
  if (p.k < 31) {
    const int64_t blocks = std::min<int64_t>(((int64_t)p.m * p.n + 255) / 256, 1 << 20);
    hipLaunchKernelGGL(short_kernel<T>, dim3((unsigned)blocks), dim3(256), 0, s, p);
    return;
  }
  // Row kernel and matrix cores, 4096 x 4096, by rows of A: bf16 1 5.2 and 7.8
  // us, 3 7.4 and 8.2, 4 8.7 and 8.3; fp32 (three products) 1 6.1 and 12.3, 4
  // 12.4 and 12.9, 5 12.9 there.
  constexpr bool wide = sizeof(T) == 4;
  if (p.m == 1) return run_rows<T, 1, 4>(p, s);
  if (p.m == 2) return run_rows<T, 2, 4>(p, s);
  if (p.m == 3) return run_rows<T, 3, 4>(p, s);
  if constexpr (wide)
    if (p.m == 4) return run_rows<T, 4, 4>(p, s);
  // Two tiles of weight rows a block read A half as often, where that leaves
  // every compute unit a block (one tile and two: 64 bf16 rows of A on 4096 x
  // 4096 21.8 and 15.6 us, on 11008 x 4096 56.4 and 44.1; 16 on 8192 x 4096 17.1
  // and 12.9, fp32 27.2 and 19.6; but 16 on 4096 x 4096, 128 blocks, 9.6 and
  // 12.5); sixteen waves where fp32's planes do not need the registers of eight.
  const int tall = p.m <= 16 ? 16 : 32;
  const bool many = (int64_t)((p.n + 31) / 32) * ((p.m + tall - 1) / tall) >= 256;
  if (p.m <= 16) return many ? run_blocks<T, 8, 1, 2>(p, s) : run_blocks<T, wide ? 8 : 16, 1, 1>(p, s);
  if constexpr (!wide)
    if (many) return run_blocks<T, 8, 2, 2>(p, s);
  return run_blocks<T, 8, 2, 1>(p, s);
}

}  // namespace og::q4

extern "C" og_status og_gemm_nt_q4(int64_t m, int64_t n, int64_t k, const void *A, int type,
                                   int64_t lda, const uint8_t *Q, int64_t ldq, const void *S,
                                   int scale_type, int64_t lds, const uint8_t *Z, int64_t ldz,
                                   int64_t group, void *C, int64_t ldc) {
  using namespace og::host;
  if (type < OG_F32 || type > OG_F16 || scale_type < OG_F32 || scale_type > OG_F16)
    return fail(OG_ERR_INVALID_ARG, "type %d or scale type %d: OG_F32, OG_BF16 or OG_F16", type,
                scale_type);
  if (m < 0 || n < 0 || k < 0)
    return fail(OG_ERR_INVALID_ARG, "negative size: m %lld, n %lld, k %lld", (long long)m,
                (long long)n, (long long)k);
  if (group < 32 || group % 32)
    return fail(OG_ERR_INVALID_ARG, "group %lld must be a positive multiple of 32", (long long)group);
  const int64_t groups = (k + group - 1) / group;
  if (lda < std::max<int64_t>(1, k) || ldq < std::max<int64_t>(1, (k + 1) / 2) ||
      ldc < std::max<int64_t>(1, n) || lds < std::max<int64_t>(1, groups) ||
      (Z && ldz < std::max<int64_t>(1, groups)))
    return fail(OG_ERR_INVALID_ARG, "a row stride is below its row: lda %lld, ldq %lld, lds %lld, "
                "ldz %lld, ldc %lld", (long long)lda, (long long)ldq, (long long)lds, (long long)ldz,
                (long long)ldc);
  // (n: a row kernel's launch has up to 64 n threads, of fewer than 2^32)
  if (m > (1 << 19) || n > (1 << 25) || k > (1 << 28) || group > (1 << 30))
    return fail(OG_ERR_TOO_LARGE, "m %lld, n %lld, k %lld or group %lld: at most 2^19, 2^25, 2^28, 2^30",
                (long long)m, (long long)n, (long long)k, (long long)group);
  if (m * n > (int64_t(1) << 38))
    return fail(OG_ERR_TOO_LARGE, "%lld x %lld outputs: at most 2^38", (long long)m, (long long)n);
  if (m == 0 || n == 0) return ok();
  if (!C || (k > 0 && (!A || !Q || !S))) return fail(OG_ERR_INVALID_ARG, "a null pointer");
  og_status st = check_device();
  if (st != OG_OK) return st;
  const bool whole = (group & (group - 1)) == 0;
  const og::q4::Problem p{(int)m, (int)n, (int)k, (int)group,
                          whole ? __builtin_ctzll((unsigned long long)group) : -1, A, lda, Q, ldq, S, scale_type, lds,
                          Z, ldz, C, ldc};
  if (type == OG_F32) og::q4::run<float>(p, current_stream());
  else if (type == OG_BF16) og::q4::run<__bf16>(p, current_stream());
  else og::q4::run<_Float16>(p, current_stream());
  return check_launch("gemm_nt_q4");
}
