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
#include <hip/hip_runtime.h>

#include <algorithm>

#include "og.h"
#include "og_host.hpp"

namespace og::logits {

constexpr int kThreads = 512;
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

typedef float f32x4 __attribute__((ext_vector_type(4)));

// VEC: four neighbouring logits a thread (rows of z and o, and of bias, are whole
// aligned vectors of four); else single ones a block's width apart.
template <class T, bool VEC>
__global__ __launch_bounds__(kThreads) void penalties_kernel(Problem p) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  extern __shared__ uint32_t counts[];
  const int64_t row = blockIdx.y;
  const int v0 = blockIdx.x * p.segment, size = min(p.segment, p.v - v0);
  const int tid = threadIdx.x;
  if (p.tokens) {
    for (int i = tid; i < p.segment; i += kThreads) counts[i] = 0;
    const int64_t length = p.lengths ? min(max(p.lengths[row], (int64_t)0), p.t) : p.t;
    const int64_t prompt = p.prompts ? p.prompts[row] : 0;
    const int64_t *tokens = p.tokens + row * p.ldt;
    __syncthreads();
    for (int64_t i = tid; i < length; i += kThreads) {
      const uint64_t at = (uint64_t)tokens[i] - v0;  // (of a negative token: beyond any size)
      if (at >= (uint64_t)size) continue;
      if (i >= prompt) atomicAdd(&counts[at], 1u);
      else atomicOr(&counts[at], kPrompt);
    }
    __syncthreads();
  }
  const float r = p.repetition ? p.repetition[row] : 1.0f;
  const float f = p.frequency ? p.frequency[row] : 0.0f, pr = p.presence ? p.presence[row] : 0.0f;
  const T *z = static_cast<const T *>(p.z) + row * p.ldz + v0;
  T *o = static_cast<T *>(p.o) + row * p.ldo + v0;
  const float *bias = p.bias ? p.bias + row * p.ldb + v0 : nullptr;
  const uint32_t *mask = p.mask ? p.mask + row * p.ldm + v0 / 32 : nullptr;
  const bool all = !p.in_place || bias || mask;

  auto changed = [&](float x, uint32_t c, float b, uint32_t allowed) __attribute__((always_inline)) {
    if (c) {
      if (p.repetition) x = x > 0 ? x / r : x * r;
      const uint32_t made = c & ~kPrompt;
      if (made) {
        if (p.frequency) x -= f * (float)made;
        if (p.presence) x -= pr;
      }
    }
    if (bias) x += b;
    return allowed ? x : -INFINITY;
  };
  if constexpr (VEC) {
    for (int i = 4 * tid; i < size; i += 4 * kThreads) {
      uint4 c = {0, 0, 0, 0};
      if (p.tokens) c = *reinterpret_cast<const uint4 *>(counts + i);
      if (!all && !(c.x | c.y | c.z | c.w)) continue;
      if (i + 4 <= size) {
        const T4 in = *reinterpret_cast<const T4 *>(z + i);
        const uint32_t bits = mask ? mask[i >> 5] >> (i & 31) : ~0u;
        const f32x4 b = bias ? *reinterpret_cast<const f32x4 *>(bias + i) : f32x4{0, 0, 0, 0};
        T4 out;
        out[0] = (T)changed((float)in[0], c.x, b[0], bits & 1);
        out[1] = (T)changed((float)in[1], c.y, b[1], bits & 2);
        out[2] = (T)changed((float)in[2], c.z, b[2], bits & 4);
        out[3] = (T)changed((float)in[3], c.w, b[3], bits & 8);
        *reinterpret_cast<T4 *>(o + i) = out;
      } else {
        const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
        for (int e = 0; i + e < size; ++e)
          o[i + e] = (T)changed((float)z[i + e], cs[e], bias ? bias[i + e] : 0.0f,
                                mask ? mask[(i + e) >> 5] >> ((i + e) & 31) & 1 : 1);
      }
    }
  } else {
    for (int i = tid; i < size; i += kThreads) {
      const uint32_t c = p.tokens ? counts[i] : 0;
      if (!all && !c) continue;
      o[i] = (T)changed((float)z[i], c, bias ? bias[i] : 0.0f, mask ? mask[i >> 5] >> (i & 31) & 1 : 1);
    }
  }
}

template <class T>
void run(int64_t n, Problem p, hipStream_t s) {
  // Segments as long as leaves two blocks for each compute unit.
  const int64_t want = (n * p.v / 512 + kLeast - 1) / kLeast * kLeast;
  p.segment = (int)std::min<int64_t>(std::max<int64_t>(want, kLeast), kMost);
  const int64_t four = 4 * sizeof(T);
  const bool vec = p.ldz % 4 == 0 && p.ldo % 4 == 0 && p.ldb % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(p.z) % four == 0 &&
                   reinterpret_cast<uintptr_t>(p.o) % four == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
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
