// og_clip.hip -- og_grad_norm and og_clip_grad_norm: the Euclidean norm over
// all elements of many tensors, and the tensors times min(1, max / (norm + eps)).
//
// Two passes over the data, both bound by its bytes.  The tensors of a launch
// are a table in the kernel's arguments (no copy of it goes through memory, so
// a call can be captured); together they are a row of chunks of 16 KB, of which
// every block takes one run.  Squares are added in 64 bits (those of 32-bit
// values are exact there), by lane, wave, block and launch in a fixed order.
//
// Norm and scaling, kernels traced one by one: 1.08 GB of bf16 217 and 398 us (5.0 TB/s, 5.4 of reads and
// writes; back to back 620 together), 102 MB of fp32 in 55 tensors 32 and 34, 1 MB in nine 4 and 4.  512 to
// 4096 blocks, 128 to 1024 threads and 1 to 8 loads a thread at once are within 4 % of each other on the
// large ones.
// Tensors that do not begin on 16 bytes, and rows apart, go an element at a time: 500 MB of bf16 91 and 193 us
// aligned, 460 and 504 from an odd element on; 16384 rows of fp32 42 and 104 dense (4096 columns), 148 and 206
// apart (4095), of bf16 24 and 37, 117 and 139.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <functional>
#include <memory>
#include <new>

#include "og.h"
#include "og_host.hpp"

namespace og::clip {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kLoads = 4;       // of a thread, in flight together
constexpr int kBlocks = 1024;   // and partial sums
constexpr int kTensors = 64;    // of a launch: the arguments are at most 4 KB
constexpr int kChunk = 16 * kThreads * kLoads;   // bytes

struct Tensor {
  const void *x;
  void *y;
  int64_t size;       // elements
  int64_t ldx, ldy;   // row strides; both 0: the elements follow one another
  int32_t cols;
  int32_t type;       // + kWhole: x and y are aligned to 16 bytes and dense
};
constexpr int kWhole = 16;

struct Table {
  Tensor t[kTensors];
  int32_t first[kTensors + 1];  // chunk of a tensor's beginning
  int32_t count;
  int32_t add;  // the partial sums of earlier launches stay
};
static_assert(sizeof(Table) <= 3840, "room for the other arguments");

template <class T>
struct Values {
  static constexpr int kOne = 16 / sizeof(T), kPer = kChunk / sizeof(T);
  static __device__ __forceinline__ void load(u32x4 w, float (&v)[kOne]) {
    typedef T V __attribute__((ext_vector_type(kOne)));
    const V h = __builtin_bit_cast(V, w);
#pragma unroll
    for (int e = 0; e < kOne; ++e) v[e] = (float)h[e];
  }
  static __device__ __forceinline__ u32x4 store(const float (&v)[kOne]) {
    typedef T V __attribute__((ext_vector_type(kOne)));
    V h;
#pragma unroll
    for (int e = 0; e < kOne; ++e) h[e] = (T)v[e];
    return __builtin_bit_cast(u32x4, h);
  }
};

// Where element i of a tensor lies.
__device__ __forceinline__ int64_t place(int64_t i, int cols, int64_t ld) {
  if (!ld) return i;
  const int64_t r = i / cols;
  return r * ld + (i - r * cols);
}

// Sum of the squares of the lane's part of chunk c of t.
template <class T>
__device__ __forceinline__ double squares(const Tensor &t, int c) {
  using V = Values<T>;
  const int64_t from = (int64_t)c * V::kPer, end = min(from + V::kPer, t.size);
  const T *x = static_cast<const T *>(t.x);
  double sum[4] = {0, 0, 0, 0};
  if ((t.type & kWhole) && end - from == V::kPer) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(x + from) + threadIdx.x;
    u32x4 w[kLoads];
#pragma unroll
    for (int q = 0; q < kLoads; ++q) w[q] = p[q * kThreads];
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      float v[V::kOne];
      V::load(w[q], v);
#pragma unroll
      for (int e = 0; e < V::kOne; ++e) sum[e % 4] = fma((double)v[e], (double)v[e], sum[e % 4]);
    }
  } else {
    for (int64_t i = from + threadIdx.x; i < end; i += kThreads) {
      const double v = (float)x[place(i, t.cols, t.ldx)];
      sum[0] = fma(v, v, sum[0]);
    }
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// The factor, m 2^e with 24 bits of m in [1/2, 1], e at most 0: it may be far below fp32's range,
// a product with m cannot leave it, and 1 (m 1) leaves subnormal values as they are.
struct Factor {
  float m;
  int e;
  __device__ __forceinline__ explicit Factor(double f)
      : m(f == 1.0 ? 1.0f : (float)__builtin_amdgcn_frexp_mant(f)), e(f == 1.0 ? 0 : __builtin_amdgcn_frexp_exp(f)) {}
  __device__ __forceinline__ float operator()(float x) const { return __builtin_ldexpf(x * m, e); }
};

template <class T>
__device__ __forceinline__ void scaled(const Tensor &t, int c, Factor by) {
  using V = Values<T>;
  const int64_t from = (int64_t)c * V::kPer, end = min(from + V::kPer, t.size);
  const T *x = static_cast<const T *>(t.x);
  T *y = static_cast<T *>(t.y);
  if ((t.type & kWhole) && end - from == V::kPer) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(x + from) + threadIdx.x;
    u32x4 *to = reinterpret_cast<u32x4 *>(y + from) + threadIdx.x;
    u32x4 w[kLoads];
#pragma unroll
    for (int q = 0; q < kLoads; ++q) w[q] = p[q * kThreads];
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      float v[V::kOne];
      V::load(w[q], v);
#pragma unroll
      for (int e = 0; e < V::kOne; ++e) v[e] = by(v[e]);
      to[q * kThreads] = V::store(v);
    }
  } else {
    for (int64_t i = from + threadIdx.x; i < end; i += kThreads)
      y[place(i, t.cols, t.ldy)] = (T)by((float)x[place(i, t.cols, t.ldx)]);
  }
}

// The tensor that chunk c lies in.
__device__ __forceinline__ int tensor_of(const Table &a, int c) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The sum over the block, in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double waves[kThreads / 64];
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = waves[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) sum += waves[w];
  return sum;
}

__global__ __launch_bounds__(kThreads) void squares_kernel(Table a, double *part) {
  const int chunks = a.first[a.count];
  const int c0 = (int)((int64_t)chunks * blockIdx.x / kBlocks), c1 = (int)((int64_t)chunks * (blockIdx.x + 1) / kBlocks);
  double sum = 0;
  if (c0 < c1) {
    int t = tensor_of(a, c0);
    for (int c = c0; c < c1; ++c) {
      while (c >= a.first[t + 1]) ++t;
      const Tensor &x = a.t[t];
      const int at = c - a.first[t];
      switch (x.type & 3) {
        case OG_F32: sum += squares<float>(x, at); break;
        case OG_BF16: sum += squares<__bf16>(x, at); break;
        default: sum += squares<_Float16>(x, at);
      }
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = a.add ? part[blockIdx.x] + sum : sum;
}

// The norm from the partial sums, in every thread.
__device__ __forceinline__ double norm_of(const double *part) {
  double sum = 0;
#pragma unroll
  for (int i = 0; i < kBlocks; i += kThreads) sum += part[i + threadIdx.x];
  return sqrt(block_sum(sum));
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const double *part, float *norm) {
  const double n = norm_of(part);
  if (threadIdx.x == 0) *norm = (float)n;
}

__global__ __launch_bounds__(kThreads) void scale_kernel(Table a, const double *part, float most, float eps,
                                                         float *norm) {
  const double n = norm_of(part), with = n + (double)eps;
  if (blockIdx.x == 0 && threadIdx.x == 0 && !a.add) *norm = (float)n;
  // (a norm that is NaN gives NaN)
  const double factor = with <= (double)most ? 1.0 : (double)most / with;
  const Factor by(factor);
  const int chunks = a.first[a.count];
  const int c0 = (int)((int64_t)chunks * blockIdx.x / kBlocks), c1 = (int)((int64_t)chunks * (blockIdx.x + 1) / kBlocks);
  if (c0 >= c1) return;
  int t = tensor_of(a, c1 - 1);
  // Last chunks first: the caches hold what the first pass read last.
  for (int c = c1 - 1; c >= c0; --c) {
    while (c < a.first[t]) --t;
    const Tensor &x = a.t[t];
    if (factor == 1.0 && x.x == x.y) continue;
    const int at = c - a.first[t];
    switch (x.type & 3) {
      case OG_F32: scaled<float>(x, at, by); break;
      case OG_BF16: scaled<__bf16>(x, at, by); break;
      default: scaled<_Float16>(x, at, by);
    }
  }
}

// Whether two tensors begin at one place (each would be scaled twice).
bool shared_output(int64_t count, const og_grad *grads) {
  std::unique_ptr<const void *[]> outs(new (std::nothrow) const void *[count]);
  int64_t n = 0;
  for (int64_t i = 0; outs && i < count; ++i)
    if (grads[i].rows && grads[i].cols) outs[n++] = grads[i].y;
  std::sort(outs.get(), outs.get() + n, std::less<const void *>());
  return std::adjacent_find(outs.get(), outs.get() + n) != outs.get() + n;
}

og_status check(int64_t count, const og_grad *grads, bool clip, const float *norm, const void *workspace,
                int64_t bytes) {
  using og::host::fail;
  if (count < 0) return fail(OG_ERR_INVALID_ARG, "negative count %lld", (long long)count);
  if (count > (1 << 20)) return fail(OG_ERR_TOO_LARGE, "%lld tensors: at most 2^20", (long long)count);
  if (count > 0 && !grads) return fail(OG_ERR_INVALID_ARG, "the tensors are null");
  for (int64_t i = 0; i < count; ++i) {
    const og_grad &g = grads[i];
    if (g.type < OG_F32 || g.type > OG_F16)
      return fail(OG_ERR_INVALID_ARG, "tensor %lld: type %lld: OG_F32, OG_BF16 or OG_F16", (long long)i,
                  (long long)g.type);
    if (g.rows < 0 || g.cols < 0)
      return fail(OG_ERR_INVALID_ARG, "tensor %lld: negative size: %lld x %lld", (long long)i, (long long)g.rows,
                  (long long)g.cols);
    if (g.rows == 0 || g.cols == 0) continue;
    const bool rows = g.rows > 1;
    if (rows && (g.ldx < g.cols || (clip && g.ldy < g.cols)))
      return fail(OG_ERR_INVALID_ARG, "tensor %lld: ldx %lld or ldy %lld below %lld columns", (long long)i,
                  (long long)g.ldx, (long long)g.ldy, (long long)g.cols);
    if (g.cols > (int64_t(1) << 40) || g.rows > (int64_t(1) << 40) || g.rows > (int64_t(1) << 40) / g.cols ||
        (rows && (g.ldx > (int64_t(1) << 40) || g.ldy > (int64_t(1) << 40))))
      return fail(OG_ERR_TOO_LARGE, "tensor %lld: %lld x %lld: at most 2^40 elements, strides 2^40", (long long)i,
                  (long long)g.rows, (long long)g.cols);
    const bool dense = !rows || (g.ldx == g.cols && (!clip || g.ldy == g.cols));
    if (!dense && g.cols > 0x7FFFFFFF)
      return fail(OG_ERR_TOO_LARGE, "tensor %lld: rows of %lld columns apart: at most 2^31 - 1", (long long)i,
                  (long long)g.cols);
    if (!g.x || (clip && !g.y)) return fail(OG_ERR_INVALID_ARG, "tensor %lld is null", (long long)i);
    if (clip && g.x == g.y && rows && g.ldx != g.ldy)
      return fail(OG_ERR_INVALID_ARG, "tensor %lld: in place the strides must be the same", (long long)i);
  }
  if (clip && shared_output(count, grads)) return fail(OG_ERR_INVALID_ARG, "two tensors have one output");
  if (!norm) return fail(OG_ERR_INVALID_ARG, "norm is null");
  if (!workspace || bytes < kBlocks * 8)
    return fail(OG_ERR_INVALID_ARG, "workspace of %lld bytes: %d needed", (long long)(workspace ? bytes : 0),
                kBlocks * 8);
  if (reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(OG_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return OG_OK;
}

// f(table) for the tensors, as many at a time as a table holds; once at least.
template <class F>
void tables(int64_t count, const og_grad *grads, bool clip, F f) {
  Table a;
  bool add = false;
  auto begin = [&] {
    a.count = 0;
    a.first[0] = 0;
    a.add = add;
  };
  auto end = [&] {
    f(a);
    add = true;
  };
  begin();
  for (int64_t i = 0; i < count; ++i) {
    const og_grad &g = grads[i];
    if (g.rows == 0 || g.cols == 0) continue;
    const int size = g.type == OG_F32 ? 4 : 2;
    const bool dense = g.rows == 1 || (g.ldx == g.cols && (!clip || g.ldy == g.cols));
    const bool whole = dense && reinterpret_cast<uintptr_t>(g.x) % 16 == 0 &&
                       (!clip || reinterpret_cast<uintptr_t>(g.y) % 16 == 0);
    const int64_t n = g.rows * g.cols, chunks = (n * size + kChunk - 1) / kChunk;
    // (2^40 elements are 2^28 chunks at most: four tensors of that size at least fit a table)
    if (a.count == kTensors || a.first[a.count] + chunks > 0x40000000) {
      end();
      begin();
    }
    a.t[a.count] = Tensor{g.x, clip ? g.y : nullptr, n, dense ? 0 : g.ldx, dense ? 0 : g.ldy,
                          dense ? 1 : (int32_t)g.cols, (int32_t)g.type | (whole ? kWhole : 0)};
    a.first[a.count + 1] = a.first[a.count] + (int32_t)chunks;
    ++a.count;
  }
  end();
}

}  // namespace og::clip

extern "C" {

int64_t og_grad_norm_workspace(void) {
  og::host::ok();
  return og::clip::kBlocks * 8;
}

og_status og_grad_norm(int64_t count, const og_grad *grads, float *norm, void *workspace,
                       int64_t workspace_bytes) {
  using namespace og::host;
  using namespace og::clip;
  og_status st = check(count, grads, false, norm, workspace, workspace_bytes);
  if (st != OG_OK || (st = check_device()) != OG_OK) return st;
  double *part = static_cast<double *>(workspace);
  hipStream_t s = current_stream();
  tables(count, grads, false,
         [&](const Table &a) { hipLaunchKernelGGL(squares_kernel, dim3(kBlocks), dim3(kThreads), 0, s, a, part); });
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kThreads), 0, s, part, norm);
  return check_launch("grad_norm");
}

og_status og_clip_grad_norm(int64_t count, const og_grad *grads, float max_norm, float eps, float *norm,
                            void *workspace, int64_t workspace_bytes) {
  using namespace og::host;
  using namespace og::clip;
  if (!(max_norm >= 0) || !std::isfinite(max_norm) || !(eps >= 0) || !std::isfinite(eps))
    return fail(OG_ERR_INVALID_ARG, "max_norm %g and eps %g must be finite and >= 0", max_norm, eps);
  og_status st = check(count, grads, true, norm, workspace, workspace_bytes);
  if (st != OG_OK || (st = check_device()) != OG_OK) return st;
  double *part = static_cast<double *>(workspace);
  hipStream_t s = current_stream();
  tables(count, grads, true,
         [&](const Table &a) { hipLaunchKernelGGL(squares_kernel, dim3(kBlocks), dim3(kThreads), 0, s, a, part); });
  tables(count, grads, true, [&](const Table &a) {
    hipLaunchKernelGGL(scale_kernel, dim3(kBlocks), dim3(kThreads), 0, s, a, part, max_norm, eps, norm);
  });
  return check_launch("clip_grad_norm");
}

}  // extern "C"
