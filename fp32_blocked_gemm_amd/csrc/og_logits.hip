// og_logits.hip -- og_logit_penalties: penalties for the tokens that a
// sequence holds, a bias and a mask of allowed tokens on the logits of a row.
//
//   z = seen_j ? (z > 0 ? z / r : z r) : z            seen among all tokens
//   z = z - f c_j - p [c_j > 0]                       c_j times among those generated
//   z = z + bias_j;   z = allowed_j ? z : -inf
//
// A block takes a segment of one row's vocabulary: it counts the row's tokens
// that fall into the segment in LDS (whole numbers: the order of the atomic
// additions does not matter), then passes over the segment's logits once.
// Every segment reads all of the row's tokens, so segments are as long as
// leaves the card full.  Logits are read and written once, in fp32 between.
// 64 rows of 131072 bf16 logits under a bias and masks with 2000 tokens each take 12.9 us
// (36 MB, 2.8 TB/s; the bias is read once for each row, from L2), 9 rows of 50021 fp32 with 16384
// tokens 9.2 (the way to memory three times one after another: length, tokens, logits; and 49 segments a
// row that each read the row's tokens, some 43 MB from L2 beside 3.6 MB of logits), one row of 32768 with
// 200 tokens 4.4 (a launch).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "og.h"
#include "og_host.hpp"

namespace og::logits {

// Wide blocks: their waves' loads hide the way to memory that a row's tokens go first (9 rows of
// 50021 with 16384 tokens: 1024 threads 9.7 us, 512 13.9, 256 23.5).
constexpr int kThreads = 1024, kAtOnce = 8;  // values of a thread whose loads are in flight together
constexpr int kSingles = 4;  // logits, where they are not whole vectors
constexpr int kLeast = 1024, kMost = 16384;  // entries of a segment (4 bytes each in LDS)
// The counter of an entry: how often it was generated, or kPrompt where it is in the prompt.
constexpr uint32_t kPrompt = 0x80000000u;

struct Problem {
  int v, segment;
  int64_t t;
  const void *z;
  int64_t ldz;
  const int64_t *tokens;  // null: nothing is counted
  int64_t ldt;
  const int64_t *lengths, *prompts;
  const float *repetition, *frequency, *presence;
  const float *bias;
  int64_t ldb;
  const uint32_t *mask;
  int64_t ldm;
  void *o;
  int64_t ldo;
  int in_place;
};

// What a block counts: how often each token of its segment is among the row's.
__device__ __forceinline__ void count(const Problem &p, int64_t row, int v0, int size, uint32_t *counts) {
  const int tid = threadIdx.x;
  for (int i = 4 * tid; i < p.segment; i += 4 * kThreads) *reinterpret_cast<uint4 *>(counts + i) = uint4{0, 0, 0, 0};
  const int length = (int)(p.lengths ? min(max(p.lengths[row], (int64_t)0), p.t) : p.t);
  const int64_t prompt = p.prompts ? p.prompts[row] : 0;
  const int64_t *tokens = p.tokens + row * p.ldt;
  __syncthreads();
  for (int64_t i0 = tid; i0 < length; i0 += kAtOnce * kThreads) {
    uint64_t at[kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q)  // (of a foreign token, a negative one too: beyond any size)
      at[q] = i0 + q * kThreads < length ? (uint64_t)tokens[i0 + q * kThreads] - v0 : ~0ull;
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      if (at[q] >= (uint64_t)size) continue;
      if (i0 + q * kThreads >= prompt) atomicAdd(&counts[at[q]], 1u);
      else atomicOr(&counts[at[q]], kPrompt);
    }
  }
  __syncthreads();
}

// A row's steps.
struct Steps {
  float r, f, p;
  bool repetition, frequency, presence, bias;
  // Whether a penalty changes a logit of count c.
  __device__ __forceinline__ bool penalise(uint32_t c) const {
    return (c && repetition) || ((c & ~kPrompt) && (frequency || presence));
  }
  __device__ __forceinline__ float operator()(float x, uint32_t c, float b, uint32_t allowed) const {
    if (c) {
      if (repetition) x = x > 0 ? x / r : x * r;
      const uint32_t made = c & ~kPrompt;
      if (made) {
        if (frequency) x -= f * (float)made;
        if (presence) x -= p;
      }
    }
    if (bias) x += b;
    return allowed ? x : -INFINITY;
  }
};

// VEC: eight neighbouring logits a thread (rows of z, o and bias are aligned to vectors of eight); else single ones, a block's width apart.
template <class T, bool VEC>
__global__ __launch_bounds__(kThreads, 8) void penalties_kernel(Problem p) {
  extern __shared__ __align__(32) uint32_t counts[];
  const int64_t row = blockIdx.y;
  const int v0 = blockIdx.x * p.segment, size = min(p.segment, p.v - v0);
  const int tid = threadIdx.x;
  const Steps steps{p.repetition ? p.repetition[row] : 1.0f, p.frequency ? p.frequency[row] : 0.0f,
                    p.presence ? p.presence[row] : 0.0f, p.repetition != nullptr, p.frequency != nullptr,
                    p.presence != nullptr, p.bias != nullptr};
  const T *z = static_cast<const T *>(p.z) + row * p.ldz + v0;
  T *o = static_cast<T *>(p.o) + row * p.ldo + v0;
  const float *bias = p.bias ? p.bias + row * p.ldb + v0 : nullptr;
  const uint32_t *mask = p.mask ? p.mask + row * p.ldm + v0 / 32 : nullptr;
  const bool all = !p.in_place || bias || mask;
  // The first logits are on their way while the tokens are counted.
  if constexpr (VEC) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    T8 in;
    f32x8 b;
    uint32_t bits = 0xFF;
    if (!all) {
      // only what a penalty changes; others of a vector keep their bits, of a NaN too (stored one by one: up to
      // 2 us more)
      if (!p.tokens) return;
      count(p, row, v0, size, counts);
      for (int i = 8 * tid; i < size; i += 8 * kThreads) {
        if (i + 8 <= size) {
          const u32x8 c = *reinterpret_cast<const u32x8 *>(counts + i);
          if (!(c[0] | c[1] | c[2] | c[3] | c[4] | c[5] | c[6] | c[7])) continue;
          T8 now = *reinterpret_cast<const T8 *>(z + i);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (steps.penalise(c[e])) now[e] = (T)steps((float)now[e], c[e], 0.0f, 1);
          *reinterpret_cast<T8 *>(o + i) = now;
        } else {
          for (int k = i; k < size; ++k)
            if (steps.penalise(counts[k])) o[k] = (T)steps((float)z[k], counts[k], 0.0f, 1);
        }
      }
      return;
    }
    auto load = [&](int i) __attribute__((always_inline)) {
      if (i + 8 > size) return;
      in = *reinterpret_cast<const T8 *>(z + i);
      if (bias) b = *reinterpret_cast<const f32x8 *>(bias + i);
      if (mask) bits = reinterpret_cast<const uint8_t *>(mask)[i >> 3];
    };
    load(8 * tid);
    if (p.tokens) count(p, row, v0, size, counts);
    for (int i = 8 * tid; i < size; i += 8 * kThreads) {
      if (i + 8 <= size) {
        T8 now = in;
        const f32x8 add = b;
        const uint32_t allowed = bits;
        load(i + 8 * kThreads);
        u32x8 c = {0, 0, 0, 0, 0, 0, 0, 0};
        if (p.tokens) c = *reinterpret_cast<const u32x8 *>(counts + i);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          now[e] = (T)steps((float)now[e], c[e], bias ? add[e] : 0.0f, allowed & (1u << e));
        *reinterpret_cast<T8 *>(o + i) = now;
      } else {
        for (int k = i; k < size; ++k) {
          const uint32_t c = p.tokens ? counts[k] : 0;
          o[k] = (T)steps((float)z[k], c, bias ? bias[k] : 0.0f, mask ? mask[k >> 5] >> (k & 31) & 1 : 1);
        }
      }
    }
  } else {
    T in[kSingles];
    float b[kSingles];
    uint32_t bits[kSingles];
    auto load = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < kSingles; ++q) {
        const int i = i0 + q * kThreads;
        if (i >= size) continue;
        if (all) in[q] = z[i];
        b[q] = bias ? bias[i] : 0.0f;
        bits[q] = mask ? mask[i >> 5] >> (i & 31) & 1 : 1;
      }
    };
    load(tid);
    if (p.tokens) count(p, row, v0, size, counts);
    for (int i0 = tid; i0 < size; i0 += kSingles * kThreads) {
      if (i0 != tid) load(i0);
#pragma unroll
      for (int q = 0; q < kSingles; ++q) {
        const int i = i0 + q * kThreads;
        if (i >= size) continue;
        const uint32_t c = p.tokens ? counts[i] : 0;
        if (!all && !steps.penalise(c)) continue;
        o[i] = (T)steps((float)(all ? in[q] : z[i]), c, b[q], bits[q]);
      }
    }
  }
}

template <class T>
void run(int64_t n, Problem p, hipStream_t s) {
  // Segments as long as leaves two blocks for each compute unit (64 rows of 131072 bf16 with 2000
  // tokens: 512 blocks 13.1 us, 1024 16.3, 2048 22.0).
  const int64_t want = (n * p.v / 512 + kLeast - 1) / kLeast * kLeast;
  p.segment = (int)std::min<int64_t>(std::max<int64_t>(want, kLeast), kMost);
  const int64_t eight = 8 * sizeof(T);
  const bool vec = p.ldz % 8 == 0 && p.ldo % 8 == 0 && p.ldb % 8 == 0 &&
                   reinterpret_cast<uintptr_t>(p.z) % eight == 0 &&
                   reinterpret_cast<uintptr_t>(p.o) % eight == 0 && reinterpret_cast<uintptr_t>(p.bias) % 32 == 0;
  const auto kernel = vec ? penalties_kernel<T, true> : penalties_kernel<T, false>;
  const unsigned segments = (unsigned)((p.v + p.segment - 1) / p.segment);
  // (a launch's y is at most 65535)
  for (int64_t i = 0; i < n; i += 65535) {
    Problem q = p;
    q.z = static_cast<const T *>(p.z) + i * p.ldz;
    q.o = static_cast<T *>(p.o) + i * p.ldo;
    if (p.tokens) q.tokens += i * p.ldt;
    if (p.lengths) q.lengths += i;
    if (p.prompts) q.prompts += i;
    if (p.repetition) q.repetition += i;
    if (p.frequency) q.frequency += i;
    if (p.presence) q.presence += i;
    if (p.bias) q.bias += i * p.ldb;
    if (p.mask) q.mask += i * p.ldm;
    hipLaunchKernelGGL(kernel, dim3(segments, (unsigned)std::min<int64_t>(n - i, 65535)), dim3(kThreads),
                       p.tokens ? p.segment * 4 : 0, s, q);
  }
}

}  // namespace og::logits

extern "C" og_status og_logit_penalties(int64_t n, int64_t v, const void *Z, int64_t ldz, int type,
                                        int64_t t, const int64_t *tokens, int64_t ldt,
                                        const int64_t *lengths, const int64_t *prompt_lengths,
                                        const float *repetition, const float *frequency,
                                        const float *presence, const float *bias, int64_t ldb,
                                        const uint32_t *mask, int64_t ldm, void *O, int64_t ldo) {
  using namespace og::host;
  if (type < OG_F32 || type > OG_F16)
    return fail(OG_ERR_INVALID_ARG, "type %d: OG_F32, OG_BF16 or OG_F16", type);
  if (n < 0 || v < 0 || t < 0)
    return fail(OG_ERR_INVALID_ARG, "negative size: n %lld, v %lld, t %lld", (long long)n, (long long)v,
                (long long)t);
  const int64_t words = (v + 31) / 32;
  if (ldz < std::max<int64_t>(1, v) || ldo < std::max<int64_t>(1, v) ||
      (tokens && ldt < std::max<int64_t>(1, t)) || (bias && ldb != 0 && ldb < v) ||
      (mask && ldm != 0 && ldm < words))
    return fail(OG_ERR_INVALID_ARG, "a row stride is below its row: ldz %lld, ldt %lld, ldb %lld, ldm %lld, "
                "ldo %lld", (long long)ldz, (long long)ldt, (long long)ldb, (long long)ldm, (long long)ldo);
  if (n > (1 << 24) || v > (1 << 28) || t >= (int64_t(1) << 31))
    return fail(OG_ERR_TOO_LARGE, "n %lld, v %lld or t %lld: at most 2^24, 2^28 and 2^31 - 1", (long long)n,
                (long long)v, (long long)t);
  if (n == 0 || v == 0) return ok();
  if (!Z || !O) return fail(OG_ERR_INVALID_ARG, "the logits or the output are null");
  const bool counted = t > 0 && (repetition || frequency || presence);
  if (counted && !tokens) return fail(OG_ERR_INVALID_ARG, "a penalty without tokens");
  if (Z == O && ldz != ldo && n > 1)
    return fail(OG_ERR_INVALID_ARG, "in place the strides must be the same: ldz %lld, ldo %lld", (long long)ldz,
                (long long)ldo);
  const og_status st = check_device();
  if (st != OG_OK) return st;
  const og::logits::Problem p{(int)v, 0, t, Z, ldz, counted ? tokens : nullptr, ldt, lengths, prompt_lengths,
                              repetition, frequency, presence, bias, bias ? ldb : 0, mask, ldm, O, ldo, Z == O};
  if (type == OG_F32) og::logits::run<float>(n, p, current_stream());
  else if (type == OG_BF16) og::logits::run<__bf16>(n, p, current_stream());
  else og::logits::run<_Float16>(n, p, current_stream());
  return check_launch("logit_penalties");
}
