// og_q4.hip -- og_gemm_nt_q4: C = A W^T with W in 4 bits.
//
//   C[i][j] = sum over groups t of s[j][t] * sum over p in t of A[i][p] (q[j][p] - z[j][t])
//
// For one to some tens of rows of A the product is bound by the bytes of the
// codes, so the kernel is built around reading them once, in long rows, with
// everything else on the side: a wave takes 16 weight rows, each lane 16
// bytes (32 codes) of one of them, 128 k in all; four lane-swap instructions
// transpose the dwords among the four lane groups so that each of the next
// four matrix-core instructions (16 x 16 x 32, fp16) covers 32 consecutive k,
// that is, one group of scales.  A code becomes fp16 in one operation for two
// of them: OR-ed into the mantissa of 1024 it is 1024 + q, and subtracting
// 1024 + z is exact, so the matrix cores multiply A by the whole numbers
// q - z, and the group's scale multiplies the fp32 sum of its 32 k.  The
// activations are fp16 fragments: fp16 ones as they are; bf16 ones are whole
// in fp16 after a power of two that each wave takes from the largest of its
// row slice (2^15 at most, so 2^-39 of it is the last bit kept); fp32 ones
// are two such planes (22 bits and the rounding of the second, 2^-24 in all).
//
// k is split among the waves of a block (their sums meet in LDS, in wave
// order) so that even one 4096 x 4096 layer has sixteen waves on every
// compute unit asking for its bytes at once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "og.h"
#include "og_host.hpp"

namespace og::q4 {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct Problem {
  int m, n, k, group;   // group: a multiple of 32
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

__device__ __forceinline__ float scale_at(const void *s, int type, int64_t i) {
  if (type == OG_F32) return static_cast<const float *>(s)[i];
  if (type == OG_BF16) return (float)static_cast<const __bf16 *>(s)[i];
  return (float)static_cast<const _Float16 *>(s)[i];
}

// Eight activations of a row from k on, zero past its end.
template <class T>
__device__ __forceinline__ void load8(const T *row, int k, int K, float (&v)[8]) {
  if (k + 8 <= K) {
    T t[8];
    __builtin_memcpy(t, row + k, sizeof t);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k + e < K ? (float)row[k + e] : 0.0f;
  }
}

// The planes of eight activations in the order of the codes' extraction:
// 0 4 1 5 2 6 3 7 (nibbles j and j + 4 of a dword come out together).
template <int P>
__device__ __forceinline__ void fragment(const float (&v)[8], float up, f16x8 (&out)[P]) {
  constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = v[order[e]] * up;
    const _Float16 h = (_Float16)x;
    out[0][e] = h;
    if constexpr (P == 2) {
      const float d = x - (float)h;
      out[1][e] = (_Float16)(__builtin_isfinite(x) ? d : 0.0f);
    }
  }
}

// Two of a dword's codes (nibbles j and j + 4) as fp16, less the zero point:
// minus_zero is -(1024 + z) twice.
template <int J>
__device__ __forceinline__ f16x2 codes(uint32_t w, f16x2 minus_zero) {
  const uint32_t b = ((w >> (4 * J)) & 0x000F000Fu) | 0x64006400u;
  return __builtin_bit_cast(f16x2, b) + minus_zero;
}

// 32 codes of a row from k on (k a multiple of 32): whole 16-byte loads
// inside the row, single bytes at its end, zero past it.
__device__ __forceinline__ u32x4 load_codes(const uint8_t *row, int k, int K) {
  u32x4 w = {0, 0, 0, 0};
  const int at = k >> 1, bytes = (K + 1) >> 1;
  if (at + 16 <= bytes) {
    __builtin_memcpy(&w, row + at, 16);
  } else if (at < bytes) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (at + 4 * d + b < bytes) w[d] |= (uint32_t)row[at + 4 * d + b] << (8 * b);
  }
  return w;
}

// Block: W waves, each a slice of k; NT tiles of 16 weight rows, 16 rows of A.
template <class T, int W, int NT>
__global__ __launch_bounds__(W * 64) void q4_kernel(Problem p) {
  constexpr int P = sizeof(T) == 4 ? 2 : 1;
  __shared__ float sums[W][NT * 16][17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * NT * 16, m0 = blockIdx.y * 16;
  const int chunks = (p.k + 127) / 128;
  const int c0 = (int)((int64_t)chunks * wave / W), c1 = (int)((int64_t)chunks * (wave + 1) / W);

  // lane i's row of A (fragment column) and row of W (fragment row)
  const int m = m0 + i;
  const bool in = m < p.m;
  const T *arow = static_cast<const T *>(p.a) + (int64_t)min(m, p.m - 1) * p.lda;
  int64_t nrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) nrow[t] = min(n0 + 16 * t + i, p.n - 1);

  // the slice's power of two for each row of A
  float up = 1, down = 1;
  if constexpr (!__is_same(T, _Float16)) {
    float top = 0;
    if (in)
      for (int k = c0 * 128 + g * 8; k < c1 * 128 && k < p.k; k += 32) {
        float v[8];
        load8(arow, k, p.k, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, __builtin_isfinite(v[e]) ? fabsf(v[e]) : 0.0f);
      }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    // 2^e with top 2^e in [2^14, 2^15), e kept where 2^e and 2^-e are normal
    const int e = top > 0 ? min(126, max(-126, 14 - (int)__builtin_amdgcn_frexp_expf(top) + 1)) : 0;
    up = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
    down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
  }

  // acc[t][r]: weight row 16 t + i, A row m0 + 4 g + r
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};

  u32x4 next[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    next[t] = c0 < c1 ? load_codes(p.q + nrow[t] * p.ldq, c0 * 128 + 32 * g, p.k) : u32x4{0, 0, 0, 0};
  for (int c = c0; c < c1; ++c) {
    u32x4 w[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w[t] = next[t];
      if (c + 1 < c1) next[t] = load_codes(p.q + nrow[t] * p.ldq, (c + 1) * 128 + 32 * g, p.k);
    }
    f16x8 x[4][P];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (in) load8(arow, c * 128 + 32 * j + 8 * g, p.k, v);
      fragment<P>(v, up, x[j]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // dword d of lane group g (k 32 g + 8 d) to dword g of lane group d
      const u32x2 a = __builtin_amdgcn_permlane32_swap(w[t][0], w[t][2], false, false);
      const u32x2 b = __builtin_amdgcn_permlane32_swap(w[t][1], w[t][3], false, false);
      const u32x2 lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
      const u32x2 hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
      const uint32_t d[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = c * 128 + 32 * j;
        const int64_t at = min(k, p.k - 1) / p.group;
        const float s = scale_at(p.s, p.s_type, nrow[t] * p.lds + at);
        const int z = p.z ? p.z[nrow[t] * p.ldz + at] : 8;
        const _Float16 mz = (_Float16)(float)(-1024 - z);
        const f16x2 zz = {mz, mz};
        const f16x2 q0 = codes<0>(d[j], zz), q1 = codes<1>(d[j], zz), q2 = codes<2>(d[j], zz),
                    q3 = codes<3>(d[j], zz);
        const f16x8 q = {q0[0], q0[1], q1[0], q1[1], q2[0], q2[1], q3[0], q3[1]};
        f32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int h = P - 1; h >= 0; --h)
          sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[j][h], q, sum, 0, 0, 0);
        // sum[r]: A row 4 g + r, weight row i
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(s, sum[r], acc[t][r]);
      }
    }
  }
  // the rows' powers of two are held by lanes 0..15: row 4 g + r's by lane 4 g + r
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float d = __shfl(down, 4 * g + r);
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[wave][16 * t + i][4 * g + r] = acc[t][r] * d;
  }
  __syncthreads();
  for (int o = threadIdx.x; o < NT * 256; o += W * 64) {
    const int row = o / (NT * 16), col = o % (NT * 16);
    float v = 0;
    for (int w = 0; w < W; ++w) v += sums[w][col][row];
    if (m0 + row < p.m && n0 + col < p.n)
      static_cast<T *>(p.c)[(int64_t)(m0 + row) * p.ldc + n0 + col] = (T)v;
  }
}

template <class T>
void run(const Problem &p, hipStream_t s) {
  const unsigned my = (unsigned)((p.m + 15) / 16);
  const int tiles = (p.n + 15) / 16;
  hipLaunchKernelGGL((q4_kernel<T, 16, 1>), dim3(tiles, my), dim3(1024), 0, s, p);
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
  if (m > (1 << 19) || n > (1 << 30) || k > (1 << 30) || group > (1 << 30))
    return fail(OG_ERR_TOO_LARGE, "m %lld, n %lld, k %lld or group %lld: at most 2^19, 2^30, 2^30, 2^30",
                (long long)m, (long long)n, (long long)k, (long long)group);
  if (m == 0 || n == 0) return ok();
  if (!C || (k > 0 && (!A || !Q || !S))) return fail(OG_ERR_INVALID_ARG, "a null pointer");
  og_status st = check_device();
  if (st != OG_OK) return st;
  const og::q4::Problem p{(int)m, (int)n, (int)k, (int)group, A, lda, Q, ldq, S, scale_type, lds,
                          Z, ldz, C, ldc};
  if (type == OG_F32) og::q4::run<float>(p, current_stream());
  else if (type == OG_BF16) og::q4::run<__bf16>(p, current_stream());
  else og::q4::run<_Float16>(p, current_stream());
  return check_launch("gemm_nt_q4");
}
