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
// magnitude, which goes to top.  A wave takes a row, whose first columns stay in registers
// between its maximum and its planes.
constexpr int kHeld = 4;
__device__ __forceinline__ void row_planes(const Side &s, int i, int cols, int width, bool vec, int lane) {
  const float *row = static_cast<const float *>(s.x) + i * s.ld;
  uint16_t *out = s.out + (int64_t)i * width * 2;
  f32x4 held[kHeld];
  float top = 0;
  auto larger = [&](const f32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, __builtin_isfinite(v[e]) ? fabsf(v[e]) : 0.0f);
  };
#pragma unroll
  for (int q = 0; q < kHeld; ++q) held[q] = load4(row + 4 * lane + 256 * q, cols - 4 * lane - 256 * q, vec);
#pragma unroll
  for (int q = 0; q < kHeld; ++q) larger(held[q]);
  for (int c = 4 * lane + 256 * kHeld; c < cols; c += 256) larger(load4(row + c, cols - c, vec));
  top = wave_max(top);
  if (lane == 0) s.top[i] = top;
  const int p = power_of(top), powers[4] = {p, p, p, p};
#pragma unroll
  for (int q = 0; q < kHeld; ++q)
    if (4 * lane + 256 * q < width) store_planes(out, 4 * lane + 256 * q, held[q], powers);
  for (int c = 4 * lane + 256 * kHeld; c < width; c += 256)
    store_planes(out, c, load4(row + c, cols - c, vec), powers);
}
__global__ __launch_bounds__(256) void planes_kernel(Side a, Side b, int cols, int width, int vec_a, int vec_b) {
  const int lane = threadIdx.x & 63, wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  for (int64_t i = wave; i < (int64_t)a.rows + b.rows; i += gridDim.x * 4) {
    if (i < a.rows) row_planes(a, (int)i, cols, width, vec_a, lane);
    else row_planes(b, (int)(i - a.rows), cols, width, vec_b, lane);
  }
}

struct Plan {
  int64_t kp;  // k padded
  int64_t tops_at, a_at, w_at, parts_at, total;
};

template <class T>
Plan plan(int64_t m, int64_t n, int64_t k) {
  Plan p;
  Room r;
  constexpr int P = kPlanes<T>;
  p.kp = round_up(k, P == 2 ? 32 : 8);
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
  Finish f = c.f;
  f.vec_b = whole(static_cast<const T *>(f.bias), 0);
  f.vec_r = whole(static_cast<const T *>(f.residual), f.ldr);
  f.vec_p = whole(static_cast<const T *>(f.pre), f.ldp);
  f.vec_o = whole(static_cast<const T *>(f.out), f.ldo);
  Args g{};
  g.M = (int)c.m;
  g.N = (int)c.n;
  g.K = (int)c.k;
  if constexpr (kPlanes<T> == 2) {
    float *mtop = reinterpret_cast<float *>(c.ws + p.tops_at), *ntop = mtop + round_up(c.m, 64);
    uint16_t *a = reinterpret_cast<uint16_t *>(c.ws + p.a_at), *w = reinterpret_cast<uint16_t *>(c.ws + p.w_at);
    const int64_t rows = c.m + c.n;
    hipLaunchKernelGGL(planes_kernel, dim3((unsigned)std::min<int64_t>((rows + 3) / 4, 4096)), dim3(256), 0, s,
                       Side{c.a, c.lda, (int)c.m, a, mtop}, Side{c.w, c.ldw, (int)c.n, w, ntop}, (int)c.k, (int)p.kp,
                       whole(static_cast<const float *>(c.a), c.lda), whole(static_cast<const float *>(c.w), c.ldw));
    f.mtop = mtop;
    f.ntop = ntop;
    g.a = Operand{a, 2 * p.kp, 0};
    g.b = Operand{w, 2 * p.kp, 0};
  } else {
    g.a = operand16(c.a, c.lda, c.m, c.k, p.kp, c.ws + p.a_at, s);
    g.b = operand16(c.w, c.ldw, c.n, c.k, p.kp, c.ws + p.w_at, s);
  }
  run_product<T, false, false>(g, f, c.ws + p.parts_at, s);
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
               Finish{nullptr, nullptr, 0, bias, act, residual, ldr, P, ldp, C, ldc, 0, 0, 0, 0},
               static_cast<char *>(workspace)};
  if (type == OG_F32) forward<float>(c, p, current_stream());
  else if (type == OG_BF16) forward<__bf16>(c, p, current_stream());
  else forward<_Float16>(c, p, current_stream());
  return check_launch("gemm_nt_epi");
}

}  // extern "C"
