// og_tile.hpp -- the 16-bit matrix-core tile product the language-model
// operators share: acc[m][n] = sum over k of A(m, k) * B(n, k), fp32 sums,
// with the operator's own epilogue on the finished tile.
//
// Operands are bf16, or fp16 times a power of two.  An fp32 matrix is held as
// two fp16 planes h + l, l the rounding of what h leaves (22 bits in all, the
// last of them 2^-38 of the matrix's or row's largest at the least), and a
// product of two such matrices is the sum of the plane products hh, hl and lh
// in the same accumulators: it leaves out terms of 2^-22 and below, each a
// rounding of its own, which is less than what the fp32 additions lose from a
// few dozen terms on (errors measured: those of fp32 products or below), at a
// third of the 16-bit matrix-core rate (830 TFLOP/s of the nominal peak) where
// the fp32 matrix cores have 157.  bf16 planes would need no scale but three
// planes and six products for the same bits (measured 1.5 to 2 times the
// time).  Planes are interleaved by blocks of 32 columns: element (r, c) of
// plane p of two lies at r ld + 32 (2 (c / 32) + p) + c % 32, so that a stage's
// k of one row is one run in memory.
//
// An operand is stored with k contiguous (rows of m, "plain") or with m
// contiguous (rows of k, "transposed"); both are loaded straight into LDS
// (buffer_load ... lds, 16 bytes a lane) in stages of 64 k (one plane) or 32 k
// (all planes) and read back as matrix-core fragments: ds_read_b128 for plain
// ones, ds_read_b64_tr_b16 (which transposes 16 x 4 blocks on the way) for
// transposed ones.  The LDS image is what the loads write, lane after lane, so
// the bank swizzle sits in the global address each lane loads: 16-byte granule
// g of a plain row is kept in slot g ^ f(row), the 32-byte units of a
// transposed row k are permuted by a hash of k; f and the hash put what one
// instruction reads in one cycle (16 rows, half of them one granule further
// on) in different banks.
//
// The main loop is a pipeline of three, a row of matrix instructions at a
// time: while a row runs, the fragments of a row ahead are read from LDS and
// loads of a later stage are issued.  Each stage has one barrier, placed where
// its last fragments have been read: before it every wave waits for those and
// for its own loads of the next stage (a counted wait: later stages stay in
// flight), after it the next stage may be read and this one's buffer loaded
// again.
//
// What bounds it: the matrix cores and, beside them, the loads into LDS, which
// take turns with the fragments' reads (4096 x 32768 x 4096 bf16, 256 x 256 tiles:
// 885 us, 1240 TFLOP/s; with the loads left out 1707, with nothing but the
// matrix instructions 1870, with the loads alone 1404).  Stages of 32 k in four
// or five buffers, four waves of 128 x 128, the 32 x 32 x 16 instruction, wave
// priorities and loads of the next tiles into L2 were measured too and were no faster.
//
// k beyond the operand (the tail of the last stage) is loaded from an
// offset past the buffer's range, which the hardware returns as +0; rows
// beyond m repeat the last one and are masked by the epilogue.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

namespace og::tile {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr uint32_t kRange = 0xFFFFFF00u;  // range of a staging buffer, in bytes
constexpr uint32_t kOutside = kRange;     // an offset at or past the range: the load returns +0

// k of one stage.
constexpr int depth(int planes) { return planes == 1 ? 64 : 32; }

// One operand: 16-bit elements, ld and batch in elements.  ld is a multiple of 8
// and p 16-byte aligned; the elements between a row's length and the next
// multiple of 8 are zero (plain) or readable (transposed).  Planes: rows of
// whole blocks of 32.
struct Operand {
  const uint16_t *p;
  int64_t ld;
  int64_t batch;  // from one matrix of a batch to the next
};

struct Args {
  Operand a, b;
  int M, N, K;
  const int *count;  // when not null, *count (on the device, at most M or K) stands for M or K
  int count_is_k;
  int tiles_m, tiles_n;
  int k_split;  // when not 0, batch y takes k from y k_split to the next split
};

// Where column c of plane p lies in a row of P planes.
template <int P>
__device__ __forceinline__ int64_t column(int c, int p) {
  return P == 1 ? c : (int64_t)(c >> 5) * (32 * P) + p * 32 + (c & 31);
}

// The plane products: product i is of plane kPlaneA[i] of A and kPlaneB[i] of B.
constexpr int plane_products(int planes) { return planes == 1 ? 1 : 3; }
constexpr int kPlaneA[3] = {0, 0, 1}, kPlaneB[3] = {0, 1, 0};

template <class E>
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (__is_same(E, __bf16))
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 buffer_of(const uint16_t *base) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, kRange, 0x00020000u};
}
// 16 bytes a lane from the buffer into LDS, lane after lane from `lds` on (a
// uniform LDS address).  Written as asm because the compiler waits for every
// such load in flight before any LDS read it cannot tell apart; here the
// stages are told apart by the counted waits of the main loop.  No register
// is written (the LDS address goes through m0, set in the same block, which
// needs one wait state; nothing else in these kernels uses m0).
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t off, u32x4 rs) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(off), "s"(rs)
               : "memory");
}

// The swizzles (see the top): the slot permutation of a plain row, and the
// unit permutation of row k of BX transposed columns.
__device__ __forceinline__ int slots(int row) {
  return ((row >> 1) & 1) << 2 | ((row >> 3) & 1) << 1;
}
template <int BX, int P>
__device__ __forceinline__ int hash(int k) {
  static_assert(BX * P * 2 % 128 == 0, "whole groups of four units");
  // rows that are not a multiple of 256 bytes alternate between the bank halves by themselves
  return BX * P * 2 % 256 ? ((k >> 1) & 1) | ((k >> 3) & 1) << 1 : (k & 3) | ((k >> 3) & 1) << 2;
}

// Loads one operand's stages: BX rows of m by depth(P) of k, P planes.
template <int BX, int NW, bool T, int P>
struct Stager {
  static constexpr int kBytes = BX * depth(P) * P * 2;
  static constexpr int kLoads = kBytes / (NW * 1024);  // 1 KiB per wave and load
  static_assert(kLoads * NW * 1024 == kBytes, "whole loads");
  // 16-byte granules of a row of LDS
  static constexpr int kRow = T ? BX * P / 8 : 8;
  // The k of the stage that a load's lane brings: for plain rows that of the
  // first load (the swizzle repeats), for transposed ones kStep further a load
  // where the waves' loads are whole rows.
  static constexpr bool kVary = T && NW * 64 % kRow != 0;
  static constexpr int kStep = T ? NW * 64 / kRow : 0;
  static_assert(NW % 2 == 0, "a plain load's rows of 8 have one parity");
  // Offsets kept: each load's; of whole rows one, or two where bit 3 of the row
  // (in the hash) alternates from load to load.
  static constexpr bool kEach = !T || kVary;
  static constexpr int kOffs = kEach ? kLoads : kStep % 16 == 0 ? 1 : 2;
  static_assert(kEach || kStep % 8 == 0, "the hash repeats every second load at the latest");
  uint32_t off[kOffs];
  int kpos[kVary ? kLoads : 1];
  int wave;
  uint32_t step;  // bytes from one load's rows to the next's

  __device__ __forceinline__ void init(const Operand &o, int x0, int X, int w, int lane) {
    wave = w;
    step = (uint32_t)(kStep * (int)o.ld) * 2u;
#pragma unroll
    for (int j = 0; j < kOffs; ++j) {
      const int at = (j * NW + w) * 64 + lane, row = at / kRow, s = at % kRow;
      if constexpr (!T) {
        const int g = s ^ slots(row);
        if (j == 0) kpos[0] = (P == 1 ? g : g & 3) * 8;
        off[j] = (uint32_t)(min(row, X - 1 - x0) * (int)o.ld) * 2u + g * 16;
      } else {
        const int u = (s >> 1) ^ hash<BX, P>(row);  // 16 columns of one plane
        const int c = P == 1 ? u * 16 + (s & 1) * 8 : u / (2 * P) * 32;
        if (kVary || j == 0) kpos[kVary ? j : 0] = row;
        off[j] = (uint32_t)(row * (int)o.ld) * 2u + u * 32 + (s & 1) * 16;
        if (x0 + c >= X) off[j] = kOutside;
      }
    }
  }
  // load j of a stage; rs: the tile's first row (plain) or column (transposed) at its first k,
  // of which `left` remain
  __device__ __forceinline__ void issue(int j, uint32_t lds, u32x4 rs, int left) const {
    uint32_t o;
    if constexpr (kEach) o = kpos[kVary ? j : 0] < left ? off[j] : kOutside;
    else o = off[j % kOffs] != kOutside && kpos[0] < left - j * kStep ? off[j % kOffs] + (j / kOffs * kOffs) * step : kOutside;
    load_to_lds(lds + (j * NW + wave) * 1024, o, rs);
  }
};

// Reads one operand's matrix-core fragments (16 rows of m by 32 of k): lane l
// holds row l % 16, k = 8 (l / 16) .. + 7.
template <int BX, bool T, int P>
struct Reader {
  int base, swz, unit;
  // x: the wave's first row within the tile (a multiple of the wave's rows)
  __device__ __forceinline__ void init(int x, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (!T) {
      base = (x + i) * 128 + ((g ^ slots(i)) * 16);
    } else {
      const int k = 8 * g + (i >> 2);
      base = k * BX * P * 2 + (i & 3) * 8;
      swz = hash<BX, P>(k) << 5;
      unit = x >> 4;
    }
  }
  // fragment `f` of the wave's rows; b: the k half of the stage (one plane) or the plane
  __device__ __forceinline__ s16x8 read(const char *lds, int f, int b) const {
    if constexpr (!T) {
      return *reinterpret_cast<const s16x8 *>(lds + (base ^ (b << 6)) + f * 2048);
    } else {
      const int c = unit + f, u = P == 1 ? c : (c >> 1) * 2 * P + b * 2 + (c & 1);
      const int at = base + ((u << 5) ^ swz) + (P == 1 ? b * 32 * BX * 2 : 0);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds + at));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds + at + 8 * BX * P));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Where a wave's accumulators lie: acc[i][j][e] of lane l is row
// m0 + 16 i + l % 16 and column n0 + 16 j + 4 (l / 16) + e.
struct Place {
  int m0, n0;    // the wave's first row and column
  int M, N;      // rows and columns of the product (M after Args::count)
  int lane, wm, wn, batch;
  int tile_m, tile_n;
  char *lds;     // the block's stages, free once every wave has passed a barrier
};

// A tile of BM x BN by WM x WN waves, elements E, NST stages of P planes in LDS; BLOCKS: blocks a
// compute unit is to hold (the register budget).
template <class E_, int P_, int BM_, int BN_, int WM_, int WN_, int NST_, int BLOCKS_>
struct Shape {
  using E = E_;
  static constexpr int P = P_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_, BLOCKS = BLOCKS_;
  static constexpr int NW = WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int kWavesPerSimd = BLOCKS * NW > 4 ? BLOCKS * NW / 4 : 1;
  static constexpr int kStage = (BM + BN) * depth(P) * P * 2;
};

// The block's tile: blocks go to the eight XCDs in turn, so each XCD gets a
// run of neighbouring tiles (its L2 holds their rows), walked in bands of 8
// tile rows; symmetric products run the tiles on and below the diagonal.
template <bool SYM>
__device__ __forceinline__ void tile_of(int id, int tm, int tn, int &m, int &n) {
  const int total = SYM ? tm * (tm + 1) / 2 : tm * tn;
  const int x = id & 7, per = total >> 3, rem = total & 7;
  const int t = x * per + min(x, rem) + (id >> 3);
  if constexpr (SYM) {
    int r = (int)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > t) --r;
    while ((r + 1) * (r + 2) / 2 <= t) ++r;
    m = r;
    n = t - r * (r + 1) / 2;
  } else {
    constexpr int kBand = 8;
    const int band = t / (kBand * tn), in = t - band * kBand * tn;
    const int rows = min(kBand, tm - band * kBand);
    m = band * kBand + in % rows;
    n = in / rows;
  }
}

template <class S, bool TA, bool TB, class Epi>
__global__ __launch_bounds__(S::NW * 64, S::kWavesPerSimd) void tile_kernel(Args g, typename Epi::Args e) {
  constexpr int P = S::P, FM = S::FM, FN = S::FN, kDepth = depth(P);
  __shared__ __align__(1024) char lds[S::kStage * S::NST];
  using SA = Stager<S::BM, S::NW, TA, P>;
  using SB = Stager<S::BN, S::NW, TB, P>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tm, tn;
  tile_of<Epi::kSymmetric>(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
  int M = g.M, K = g.K;
  if (g.count) {
    const int c = *g.count;
    if (g.count_is_k) K = c; else M = c;
  }
  const int x0 = tm * S::BM, y0 = tn * S::BN;
  if (x0 >= M) return;
  const int batch = blockIdx.y;
  int k_next = 0;
  if (g.k_split) {
    k_next = batch * g.k_split;
    K = min(K, k_next + g.k_split);
  }
  const uint16_t *ap = g.a.p + batch * g.a.batch + (TA ? (int64_t)x0 * P : x0 * g.a.ld);
  const uint16_t *bp = g.b.p + batch * g.b.batch + (TB ? (int64_t)y0 * P : y0 * g.b.ld);

  SA sa;
  SB sb;
  sa.init(g.a, x0, M, wave, lane);
  sb.init(g.b, y0, g.N, wave, lane);
  const int wm = wave / S::WN, wn = wave % S::WN;
  Reader<S::BM, TA, P> ra;
  Reader<S::BN, TB, P> rb;
  ra.init(wm * FM * 16, lane);
  rb.init(wn * FN * 16, lane);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  // stages past the last load zeros
  const int total = (K - k_next + kDepth - 1) / kDepth;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void *)lds;
  int buf_next = 0;
  u32x4 rsa, rsb;
  uint32_t to;
  int left;
  auto next_stage = [&]() __attribute__((always_inline)) {
    to = lds0 + buf_next * S::kStage;
    rsa = buffer_of(ap + (TA ? k_next * g.a.ld : (int64_t)k_next * P));
    rsb = buffer_of(bp + (TB ? k_next * g.b.ld : (int64_t)k_next * P));
    left = K - k_next;
    if (++buf_next == S::NST) buf_next = 0;
    k_next += kDepth;
  };
  // A row's reads run kAhead rows before its products.  The loads of the stage
  // NST ahead: kRate a row, from right after the barrier on.
  constexpr int kAhead = P == 1 ? 2 : 1;
  constexpr int kPer = SA::kLoads + SB::kLoads;
  constexpr int kRate = P == 1 ? kPer / 4 : (kPer + FM / 2 - 1) / (FM / 2);
  constexpr int kEarly = kPer < kRate * kAhead ? kPer : kRate * kAhead;
  auto issue = [&](int j) __attribute__((always_inline)) {
    if (j < SA::kLoads) sa.issue(j, to, rsa, left);
    else sb.issue(j - SA::kLoads, to + SA::kBytes, rsb, left);
  };
  if (total > 0) {
    for (int p = 0; p < S::NST; ++p) {
      next_stage();
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (p + 1 < S::NST || j < kEarly) issue(j);
    }
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"i"(kPer * (S::NST - 2) + kEarly) : "memory");
    const char *la = lds, *lb = lds + SA::kBytes;
    int buf = 0;
    auto meet = [&]() __attribute__((always_inline)) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(kPer * (S::NST - 2)) : "memory");
      if (++buf == S::NST) buf = 0;
      la = lds + buf * S::kStage;
      lb = la + SA::kBytes;
      next_stage();
    };
    if constexpr (P == 1) {
      s16x8 fa[4], fb[2][FN];  // rows of A: a ring; columns of B: two halves
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[0][j] = rb.read(lb, j, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i] = ra.read(la, i, 0);
      for (int t = 0; t < total; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            // each row's reads, loads and products keep together (fences)
            __builtin_amdgcn_sched_barrier(0);
            const int ahead = i + kAhead, slot = (h * FM + ahead) % 4;
            if (h == 1 && ahead == FM) meet();
            // columns of the next half: over its predecessor's rows, or after the barrier
            if (h == 0) {
#pragma unroll
              for (int j = i * FN / FM; j < (i + 1) * FN / FM; ++j) fb[1][j] = rb.read(lb, j, 1);
            } else if (ahead >= FM) {
#pragma unroll
              for (int j = (ahead - FM) * FN / 2; j < (ahead - FM + 1) * FN / 2; ++j)
                fb[0][j] = rb.read(lb, j, 0);
            }
            if (ahead < FM) fa[slot] = ra.read(la, ahead, h);
            else fa[slot] = ra.read(la, ahead - FM, h ^ 1);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              if (h == 0 && j >= kEarly + i * kRate && j < kEarly + (i + 1) * kRate) issue(j);
              if (h == 1 && ahead >= FM && j >= (ahead - FM) * kRate && j < (ahead - FM + 1) * kRate) issue(j);
            }
#pragma unroll
            for (int j = 0; j < FN; ++j)
              acc[i][j] = mfma<typename S::E>(fb[h][j], fa[(h * FM + i) % 4], acc[i][j]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      s16x8 fa[2][P], fb[2][FN][P];  // rows of A in turn; columns of B by stage
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[0][j][p] = rb.read(lb, j, p);
        fa[0][p] = ra.read(la, 0, p);
      }
      for (int t = 0; t < total; t += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (i + 1 == FM) meet();
#pragma unroll
            for (int p = 0; p < P; ++p) {
              if (i + 1 < FM) fa[(i + 1) & 1][p] = ra.read(la, i + 1, p);
              else fa[(i + 1) & 1][p] = ra.read(la, 0, p);
            }
            if (i + 1 == FM) {
#pragma unroll
              for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int p = 0; p < P; ++p) fb[h ^ 1][j][p] = rb.read(lb, j, p);
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              if (i + 1 < FM && j >= kEarly + i * kRate && j < kEarly + (i + 1) * kRate) issue(j);
              if (i + 1 == FM && j < kEarly) issue(j);
            }
#pragma unroll
            for (int q = 0; q < plane_products(P); ++q)
#pragma unroll
              for (int j = 0; j < FN; ++j)
                acc[i][j] = mfma<typename S::E>(fb[h][j][kPlaneB[q]], fa[i & 1][kPlaneA[q]], acc[i][j]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // loads past the last stage still write LDS: none may be in flight when the
  // epilogue uses it or the block ends
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  Place at{x0 + wm * FM * 16, y0 + wn * FN * 16, M, g.N, lane, wm, wn, batch, tm, tn, lds};
  Epi::template store<S>(acc, at, e);
}

template <class S, bool TA, bool TB, class Epi>
int launch(Args g, const typename Epi::Args &e, int batches, hipStream_t s) {
  g.tiles_m = (g.M + S::BM - 1) / S::BM;
  g.tiles_n = (g.N + S::BN - 1) / S::BN;
  const int64_t n = Epi::kSymmetric ? (int64_t)g.tiles_m * (g.tiles_m + 1) / 2
                                    : (int64_t)g.tiles_m * g.tiles_n;
  hipLaunchKernelGGL((tile_kernel<S, TA, TB, Epi>), dim3((unsigned)n, batches), dim3(S::NW * 64), 0,
                     s, g, e);
  return g.tiles_n;
}

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// A tile and what it costs: nanoseconds a block spends on a stage, alone on an
// idle card, as one of 256 (one a compute unit) and as its share of a compute
// unit that has more.  (192 seeded products of 128 to 14336 columns, 24 of each
// kind: the chosen tile takes 1.01 to 1.02 times the fastest listed one's time in
// the mean, at most 1.17.)
template <class S_, int ALONE, int ONE, int SHARE>
struct Choice {
  using S = S_;
  static double time(bool sym, int64_t M, int64_t N, int64_t K, int64_t batch) {
    const int64_t tm = (M + S::BM - 1) / S::BM, tn = (N + S::BN - 1) / S::BN;
    const int64_t n = (sym ? tm * (tm + 1) / 2 : tm * tn) * batch;
    const double per = n <= 256 ? ALONE + (ONE - ALONE) * (n / 256.0) : (n + 255) / 256 * SHARE;
    return (double)((K + depth(S::P) - 1) / depth(S::P)) * per;
  }
};
template <class... C>
struct Choices {};

// The tiles by number of planes.  Large ones reuse each loaded value more
// often (a compute unit loads about 30 bytes a cycle at most), small ones
// spread a small product over more compute units; 128 x 128 comes with two
// blocks a compute unit for many tiles and with four stages in flight for few.
// Symmetric products need square tiles; with both operands transposed two
// planes of 256 x 256 need more registers than there are.
template <class E, int P, bool TT>
struct Tiles {
  using type = Choices<Choice<Shape<E, 1, 256, 256, 2, 4, 2, 1>, 1250, 1600, 1700>,
                       Choice<Shape<E, 1, 192, 192, 2, 4, 3, 1>, 720, 1050, 1100>,
                       Choice<Shape<E, 1, 128, 128, 2, 2, 2, 2>, 630, 640, 510>,
                       Choice<Shape<E, 1, 128, 128, 2, 4, 4, 1>, 450, 600, 640>,
                       Choice<Shape<E, 1, 64, 64, 2, 2, 4, 2>, 200, 210, 190>>;
};
template <class E>
struct Tiles<E, 2, true> {
  using type = Choices<Choice<Shape<E, 2, 192, 192, 2, 4, 3, 1>, 900, 1250, 1420>,
                       Choice<Shape<E, 2, 128, 128, 2, 4, 2, 2>, 640, 700, 640>,
                       Choice<Shape<E, 2, 128, 128, 2, 4, 4, 1>, 560, 680, 760>,
                       Choice<Shape<E, 2, 64, 64, 2, 2, 4, 2>, 220, 230, 230>,
                       Choice<Shape<E, 2, 32, 32, 1, 2, 4, 4>, 150, 160, 129>>;
};
template <class E>
struct Tiles<E, 2, false> {
  using type = Choices<Choice<Shape<E, 2, 256, 256, 2, 4, 2, 1>, 1500, 2100, 2250>,
                       Choice<Shape<E, 2, 192, 192, 2, 4, 3, 1>, 900, 1250, 1420>,
                       Choice<Shape<E, 2, 128, 128, 2, 4, 2, 2>, 640, 700, 640>,
                       Choice<Shape<E, 2, 128, 128, 2, 4, 4, 1>, 560, 680, 760>,
                       Choice<Shape<E, 2, 64, 64, 2, 2, 4, 2>, 220, 230, 230>,
                       Choice<Shape<E, 2, 32, 32, 1, 2, 4, 4>, 150, 160, 129>>;
};

// Runs a product on the tile with the least time; returns the number of tile
// columns.
template <bool TA, bool TB, class Epi, class First, class... Rest>
int product_of(Choices<First, Rest...>, double best, const Args &g, const typename Epi::Args &e,
               int batch, hipStream_t s) {
  constexpr bool sym = Epi::kSymmetric;
  const int64_t k = g.k_split ? g.k_split : g.K;
  if constexpr (sizeof...(Rest) > 0) {
    if (First::time(sym, g.M, g.N, k, batch) > best)
      return product_of<TA, TB, Epi>(Choices<Rest...>(), best, g, e, batch, s);
  }
  return launch<typename First::S, TA, TB, Epi>(g, e, batch, s);
}
template <class... C>
double least(Choices<C...>, bool sym, const Args &g, int batch) {
  const int64_t k = g.k_split ? g.k_split : g.K;
  return std::min({C::time(sym, g.M, g.N, k, batch)...});
}
template <class E, int P, bool TA, bool TB, class Epi>
int product(const Args &g, const typename Epi::Args &e, int batch, hipStream_t s) {
  using T = typename Tiles<E, P, TA && TB>::type;
  return product_of<TA, TB, Epi>(T(), least(T(), Epi::kSymmetric, g, batch), g, e, batch, s);
}

// The fp16 planes of four values (scaled by the caller): the second rounds
// what the first leaves; a value that is not finite stays in the first.
__device__ __forceinline__ void split4(const f32x4 v, f16x4 &h, f16x4 &l) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h[e] = (_Float16)v[e];
    const float d = v[e] - (float)h[e];
    l[e] = (_Float16)(__builtin_isfinite((float)h[e]) ? d : 0.0f);
  }
}

}  // namespace og::tile
