// Gated feed-forward of a transformer block, forward and backward, with its C
// entry points.
//
//     G = x Wg^T, U = x Wu^T, h = act(G) * U         x [M, D], W [F, D]
//     dU = dh * act(G), dG = dh * U * act'(G)
//     dx = dG Wg + dU Wu,  dWg = dG^T x,  dWu = dU^T x
//
// Four products of one shape of loop, all on the matrix cores (bf16 operands,
// float32 sums): a workgroup computes a tile of rows x columns, walking the
// summed dimension in steps of 64.  Each step's two operand tiles go from
// memory straight to LDS (16 bytes per lane, no registers), double-buffered:
// the loads of step s + 1 are in flight while step s is multiplied.
//
// An operand is stored with the summed dimension contiguous (x and W in the
// forward) or across it (W in dx; both in dW).  Its LDS tile keeps the
// memory's order, 128-byte rows of 64 summed elements or rows of 128 or 256
// columns, and the fragment reads do the rest: 16 bytes of a row as they are,
// or 4 x 16 blocks transposed by the LDS read itself.  The 16-byte pieces of
// a row are permuted by an exclusive or with bits of the row's number, so
// that the lanes of a read meet distinct banks; the loads apply the same
// permutation to the addresses they read from, since they can only fill LDS
// in order.
#include <algorithm>

#include "adaln.h"
#include "common.hpp"
#include "launch.hpp"

#define ADALN_API extern "C" __attribute__((visibility("default")))

#define ADALN_TRY(expr)          \
  do {                           \
    const int rc_ = (expr);      \
    if (rc_ != ADALN_OK) return rc_; \
  } while (0)

namespace adaln {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kStep = 64;  // summed elements per step

// What lanes past an operand's end load instead: 16 zero bytes.
__device__ const uint4 kZeros = {0, 0, 0, 0};

// 16 bytes per lane from memory to LDS at `lds` + 16 * lane.  Two forms: a
// wave-uniform base with a 32-bit offset per lane, or an address per lane.
// The count of outstanding loads is waited for by arrive() below, by hand:
// the compiler does not see these loads.  (m0 takes the LDS address; nothing
// else in these kernels uses it.  The s_nop is the wait state that the ISA
// asks for between writing m0 and a load to LDS.)
__device__ __forceinline__ void dma(uint32_t lds, const void *base,
                                    uint32_t offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(offset), "s"(base)
      : "memory");
}

__device__ __forceinline__ void dma_at(uint32_t lds, const void *p) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(p)
      : "memory");
}

// Every load of this wavefront has landed, then every wavefront's.
__device__ __forceinline__ void arrive() {
  asm volatile(
      "s_waitcnt vmcnt(0) lgkmcnt(0)\n\t"
      "s_barrier" ::
          : "memory");
}

// An operand whose summed dimension is contiguous: ROWS rows of kStep
// elements, 128 bytes each, 8 pieces of 16.  Row r keeps its piece c at
// c ^ ((r >> 1) & 7): 16 consecutive rows then cover all banks.  Rows past
// the operand's last repeat it (their products are not stored); elements past
// the end of the sum are loaded as zeros.
template <int ROWS, int WAVES>
struct Along {
  static constexpr int kBytes = ROWS * kStep * 2;
  static constexpr int kLoads = ROWS / (8 * WAVES);
  uint32_t off[kLoads];  // byte offsets of the lane's loads from the base

  static __device__ __forceinline__ int lane_row() {
    return wave_id() * 8 + lane_id() / 8;
  }
  static __device__ __forceinline__ int lane_piece() {
    return (lane_id() % 8) ^ ((lane_row() >> 1) & 7);
  }
  // Rows from row0 of an operand of `rows` rows.
  __device__ __forceinline__ void start(int row0, int rows, int pitch) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      off[i] = (uint32_t)min(i * 8 * WAVES + lane_row(), rows - 1 - row0) *
                   (uint32_t)pitch * 2 +
               lane_piece() * 16;
  }
  // Load i of a whole step; base: the operand at row row0, element k0.
  __device__ __forceinline__ void load(int i, uint32_t lds, const char *base,
                                       int64_t pitch2) const {
    dma(lds + (wave_id() + i * WAVES) * 1024, base, off[i]);
  }
  // The same where only `left` < kStep elements are left of the sum.
  __device__ __forceinline__ void load_tail(int i, uint32_t lds,
                                            const char *base, int64_t pitch2,
                                            int left) const {
    dma_at(lds + (wave_id() + i * WAVES) * 1024,
           lane_piece() * 8 < left ? base + off[i] : (const char *)&kZeros);
  }
  // Fragment of 32 rows from `row`, elements 16 * kk ...: lane l holds row
  // l % 32, elements 8 * (l / 32) + [0, 8).
  static __device__ __forceinline__ bf16x8 frag(const char *tile, int row,
                                                int kk) {
    const int l = lane_id();
    const int r = l % 32;
    const int piece = (kk * 2 + l / 32) ^ ((r >> 1) & 7);
    return *reinterpret_cast<const bf16x8 *>(tile + row * 128 + r * 128 +
                                             piece * 16);
  }
};

// An operand stored across the summed dimension: kStep rows of COLS columns,
// COLS / 8 pieces of 16 bytes; row k keeps its piece c at c ^ ((k & 3) << 2),
// so that the four rows that a transposing read takes lie in distinct banks.
// Columns past the last repeat the last eight.
template <int COLS, int WAVES>
struct Across {
  static constexpr int kBytes = COLS * kStep * 2;
  static constexpr int kPieces = COLS / 8;
  static constexpr int kRows = 64 / kPieces * WAVES;  // rows per load
  static constexpr int kLoads = kStep / kRows;
  uint32_t off;

  static __device__ __forceinline__ int lane_row() {
    return (wave_id() * 64 + lane_id()) / kPieces;
  }
  static __device__ __forceinline__ int lane_piece() {
    return (lane_id() % kPieces) ^ ((lane_row() & 3) << 2);
  }
  __device__ __forceinline__ void start(int col0, int cols, int pitch) {
    off = (uint32_t)lane_row() * (uint32_t)pitch * 2 +
          min(lane_piece() * 8, cols - 8 - col0) * 2;
  }
  // base: the operand at row k0, column col0; pitch2: bytes per row.
  __device__ __forceinline__ void load(int i, uint32_t lds, const char *base,
                                       int64_t pitch2) const {
    dma(lds + (wave_id() + i * WAVES) * 1024, base + i * kRows * pitch2, off);
  }
  __device__ __forceinline__ void load_tail(int i, uint32_t lds,
                                            const char *base, int64_t pitch2,
                                            int left) const {
    dma_at(lds + (wave_id() + i * WAVES) * 1024,
           i * kRows + lane_row() < left ? base + i * kRows * pitch2 + off
                                         : (const char *)&kZeros);
  }
  static __device__ __forceinline__ bf16x8 frag(const char *tile, int col,
                                                int kk) {
    const int l = lane_id();
    const int k = kk * 16 + (l / 32) * 8 + (l % 16) / 4;
    const int piece =
        (col / 8 + ((l >> 4) & 1) * 2 + ((l & 3) >> 1)) ^ ((k & 3) << 2);
    const char *p = tile + k * COLS * 2 + piece * 16 + (l & 1) * 8;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4 *)(p + 4 * COLS * 2));
    const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
};

// ------------------------------------------------------------- activations

enum { kSilu = 0, kGeluTanh = 1 };

// act(g) and act'(g).  Both are g times a logistic function s, of g or of
// twice the tanh form's polynomial v: (1 + tanh(v)) / 2 = 1 / (1 + exp(-2v))
// keeps its digits where 1 + tanh(v) cancels, and both ends saturate.
template <int ACT>
__device__ __forceinline__ void activate(float g, float &a, float &da) {
  if constexpr (ACT == kSilu) {
    const float s = 1.f / (1.f + __expf(-g));
    a = g * s;
    da = s * (1.f + g * (1.f - s));
  } else {
    constexpr float c = 0.7978845608028654f, e = 0.044715f;
    const float g2 = g * g;
    const float s = 1.f / (1.f + __expf(-2.f * c * g * (1.f + e * g2)));
    a = g * s;
    da = s + 2.f * g * s * (1.f - s) * c * (1.f + 3.f * e * g2);
  }
}

__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
  uint2 u;
  const f32x2 a = {f[0], f[1]}, b = {f[2], f[3]};
  u.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
  u.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2));
  return u;
}

// ------------------------------------------------------------- the products

enum {
  kHidden = 0,  // h (and G, U): rows tokens, columns hidden features
  kGrads = 1,   // dG, dU with G, U computed again
  kDx = 2,      // dx: rows tokens, columns features, sum over 2 F
  kDw = 3       // dWg, dWu: rows hidden features, columns features, sum over M
};

struct Product {
  const bf16 *x;          // [M, D]
  const bf16 *w[2];       // Wg, Wu [F, D]
  bf16 *h;                // [M, F]
  float *gu;              // saved G, U [2, M, F] (or NULL)
  const bf16 *dh;         // [M, F]
  bf16 *dgu;              // dG, dU [2, M, F]
  bf16 *out[2];           // dx, or dWg and dWu
  float *part;            // partial sums [slices, 2 or 1, rows, cols], or NULL
  int32_t M, D, F;
  int32_t tiles_r, tiles_c;
  int32_t slices, steps_per_slice, steps;
  int32_t block0;         // first block of this launch
};

// Tile of the calling workgroup.  Workgroups go to the eight XCDs in turn;
// this gives each XCD a contiguous run of tiles, and orders the run in bands
// of 8 tile rows, so that the tiles that run together share operands in the
// XCD's L2.
__device__ __forceinline__ void tile_of(int id, int total, int tiles_r,
                                        int tiles_c, int &tr, int &tc) {
  const int per = total / 8;
  const int n = id < per * 8 ? (id % 8) * per + id / 8 : id;
  constexpr int kBand = 8;
  const int band = n / (kBand * tiles_c);
  const int in = n - band * kBand * tiles_c;
  const int rows = min(kBand, tiles_r - band * kBand);
  tr = band * kBand + in % rows;
  tc = in / rows;
}

// BIG: 256 x 256 tiles by 8 wavefronts (2 x 4, each 128 x 64); else 128 x 128
// by 4 (2 x 2, each 64 x 64).  Columns of kHidden and kGrads: half of them of
// G, half the same ones of U, so that a lane holds both of an element.
template <int FORM, bool BIG, int ACT>
__global__ __launch_bounds__(BIG ? 512 : 256, BIG ? 2 : 2) void product_kernel(
    Product p) {
  constexpr int kWaves = BIG ? 8 : 4;
  constexpr int kTile = BIG ? 256 : 128;
  constexpr int kWn = BIG ? 4 : 2;          // wavefronts across the columns
  constexpr int MI = kTile / 2 / 32;        // 32-row blocks of a wavefront
  constexpr int NI = kTile / kWn / 32;      // 32-column blocks
  constexpr bool kPair = FORM == kHidden || FORM == kGrads;
  constexpr int kCols = kPair ? kTile / 2 : kTile;
  static_assert(!kPair || NI == 2, "a block of G and one of U");
  using Row = std::conditional_t<FORM == kDw, Across<kTile, kWaves>,
                                 Along<kTile, kWaves>>;
  // (of a pair, the rows of one weight)
  using Col = std::conditional_t<kPair, Along<kTile / 2, kWaves>,
                                 Across<kTile, kWaves>>;
  constexpr uint32_t kColBytes = kPair ? 2 * Col::kBytes : Col::kBytes;
  constexpr uint32_t kBuf = Row::kBytes + kColBytes;
  __shared__ __align__(1024) char lds[2][kBuf];

  int id = blockIdx.x + p.block0;
  const int tiles = p.tiles_r * p.tiles_c;
  const int slice = id / tiles;  // slices, then planes, outermost
  id -= slice * tiles;
  int tr, tc;
  tile_of(id, tiles, p.tiles_r, p.tiles_c, tr, tc);
  int plane = 0, split = slice;
  if constexpr (FORM == kDw) {
    plane = slice & 1;
    split = slice >> 1;
  }
  const int row0 = tr * kTile, col0 = tc * kCols;
  const int M = p.M, D = p.D, F = p.F;
  const int s0 = split * p.steps_per_slice;
  const int s1 = min(s0 + p.steps_per_slice, p.steps);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char *)&lds[0][0];

  Row row;
  Col col;
  row.start(row0, FORM == kDw ? F : M, FORM == kDx || FORM == kDw ? F : D);
  col.start(col0, kPair ? F : D, D);
  // The operands of the step to be loaded next (of a pair: x, Wg, Wu), and
  // how far apart two steps are.
  const char *pr, *pc, *pu = nullptr;
  const int64_t pitch_r = 2 * (int64_t)(kPair ? D : F), pitch_c = 2 * (int64_t)D;
  const int64_t next_r = FORM == kDw ? kStep * pitch_r : 2 * kStep;
  const int64_t next_c = kPair ? 2 * kStep : kStep * pitch_c;
  const int K = kPair ? D : FORM == kDx ? F : M;
  const int per = FORM == kDx ? p.steps / 2 : p.steps;  // steps per plane
  auto seek = [&](int s) {
    const int pl = FORM == kDx ? s >= per : 0;
    const int64_t k = s - pl * per;
    if constexpr (kPair) {
      pr = (const char *)(p.x + (int64_t)row0 * D) + k * next_r;
      pc = (const char *)(p.w[0] + (int64_t)col0 * D) + k * next_c;
      pu = (const char *)(p.w[1] + (int64_t)col0 * D) + k * next_c;
    } else if constexpr (FORM == kDx) {
      pr = (const char *)(p.dgu + ((int64_t)pl * M + row0) * F) + k * next_r;
      pc = (const char *)(p.w[pl] + col0) + k * next_c;
    } else {
      pr = (const char *)(p.dgu + (int64_t)plane * M * F + row0) + k * next_r;
      pc = (const char *)(p.x + col0) + k * next_c;
    }
  };
  // Load n of the 8 (4 of each operand) of that step, into a buffer.
  constexpr int kLoads = Row::kLoads + (kPair ? 2 : 1) * Col::kLoads;
  auto load = [&](int n, int buf) {
    const uint32_t at = lds0 + buf * kBuf;
    if (n < Row::kLoads)
      row.load(n, at, pr, pitch_r);
    else if (n < Row::kLoads + Col::kLoads)
      col.load(n - Row::kLoads, at + Row::kBytes, pc, pitch_c);
    else
      col.load(n - Row::kLoads - Col::kLoads,
               at + Row::kBytes + Col::kBytes, pu, pitch_c);
  };
  auto load_tail = [&](int left, int buf) {
    const uint32_t at = lds0 + buf * kBuf;
#pragma unroll
    for (int i = 0; i < Row::kLoads; ++i)
      row.load_tail(i, at, pr, pitch_r, left);
#pragma unroll
    for (int i = 0; i < Col::kLoads; ++i) {
      col.load_tail(i, at + Row::kBytes, pc, pitch_c, left);
      if constexpr (kPair)
        col.load_tail(i, at + Row::kBytes + Col::kBytes, pu, pitch_c, left);
    }
  };
  // Elements of the sum that step s has left, of its plane.
  auto left = [&](int s) {
    return K - (FORM == kDx && s >= per ? s - per : s) * kStep;
  };
  auto advance = [&](int s) {  // from step s to the one after it
    pr += next_r;
    pc += next_c;
    if constexpr (kPair) pu += next_c;
    if constexpr (FORM == kDx)
      if (s + 1 == per) seek(per);
  };

  const int wave = wave_id();
  const int wm = wave / kWn, wn = wave % kWn;
  const int wrow = wm * MI * 32;
  f32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Fragments of the next 16 summed elements are read while the present
  // ones are multiplied.  The one barrier of a step stands before its last
  // multiplications: by then its own tile has been read (so the loads of the
  // step after next may overwrite it) and the next step's has landed, so the
  // first fragments of that are read under the last multiplications too.
  constexpr int KK = kStep / 16;
  bf16x8 a[2][MI], b[2][NI];
  auto read = [&](int buf, int kk) {
    const char *rt = lds[buf];
    const char *ct = lds[buf] + Row::kBytes;
#pragma unroll
    for (int j = 0; j < NI; ++j)
      b[kk & 1][j] = Col::frag(ct, kPair ? j * (kTile / 2) + wn * 32
                                         : wn * NI * 32 + j * 32, kk);
#pragma unroll
    for (int i = 0; i < MI; ++i)
      a[kk & 1][i] = Row::frag(rt, wrow + i * 32, kk);
  };
  auto multiply = [&](int kk, int i0, int i1) {
#pragma unroll
    for (int i = i0; i < i1; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            b[kk & 1][j], a[kk & 1][i], acc[i][j], 0, 0, 0);
  };
  if (s0 < s1) {
    seek(s0);
    for (int s = s0; s < min(s0 + 2, s1); ++s) {
      if (left(s) >= kStep) {
#pragma unroll
        for (int n = 0; n < kLoads; ++n) load(n, s - s0);
      } else {
        load_tail(left(s), s - s0);
      }
      advance(s);
      if (s == s0) arrive();
    }
    read(0, 0);
  }
  for (int s = s0; s < s1; ++s) {
    const int buf = (s - s0) & 1;
#pragma unroll
    for (int kk = 0; kk < KK - 1; ++kk) {
      read(buf, kk + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(kk, 0, MI);
      __builtin_amdgcn_sched_barrier(0);
    }
    arrive();
    read(buf ^ 1, 0);  // past the last step: what lies there, not used
    __builtin_amdgcn_sched_barrier(0);
    const bool more = s + 2 < s1;
    const bool whole = more && left(s + 2) >= kStep;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      multiply(KK - 1, i, i + 1);
      __builtin_amdgcn_sched_barrier(0);
      if (whole) {
#pragma unroll
        for (int n = i * kLoads / MI; n < (i + 1) * kLoads / MI; ++n)
          load(n, buf);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (more) {
      if (!whole) load_tail(left(s + 2), buf);
      advance(s + 2);
    }
  }

  // acc[i][j][4 q + e] of lane l is row l % 32 of block i, column
  // 8 q + 4 (l / 32) + e of block j: four neighbouring columns per store.
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = row0 + wrow + i * 32 + lane % 32;
    const int rows = FORM == kDw ? F : M;
    if (r >= rows) continue;
    if constexpr (kPair) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = col0 + wn * 32 + 8 * q + 4 * (lane / 32);
        if (c >= F) continue;
        const int64_t at = (int64_t)r * F + c;
        const int64_t plane_size = (int64_t)M * F;
        float v0[4], v1[4];
        if constexpr (FORM == kHidden) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a, da;
            activate<ACT>(acc[i][0][4 * q + e], a, da);
            v0[e] = a * acc[i][1][4 * q + e];
          }
          *reinterpret_cast<uint2 *>(p.h + at) = pack4(v0);
          if (p.gu != nullptr) {
            f32x4 g, u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              g[e] = acc[i][0][4 * q + e];
              u[e] = acc[i][1][4 * q + e];
            }
            *reinterpret_cast<f32x4 *>(p.gu + at) = g;
            *reinterpret_cast<f32x4 *>(p.gu + plane_size + at) = u;
          }
        } else {
          const uint2 d = *reinterpret_cast<const uint2 *>(p.dh + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t w = e < 2 ? d.x : d.y;
            const float dh = __builtin_bit_cast(
                float, (e & 1) ? (w & 0xffff0000u) : (w << 16));
            float a, da;
            activate<ACT>(acc[i][0][4 * q + e], a, da);
            v0[e] = dh * acc[i][1][4 * q + e] * da;
            v1[e] = dh * a;
          }
          *reinterpret_cast<uint2 *>(p.dgu + at) = pack4(v0);
          *reinterpret_cast<uint2 *>(p.dgu + plane_size + at) = pack4(v1);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c =
              col0 + wn * NI * 32 + j * 32 + 8 * q + 4 * (lane / 32);
          if (c >= D) continue;
          const int64_t at = (int64_t)r * D + c;
          if (p.part != nullptr) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
            *reinterpret_cast<f32x4 *>(p.part + (int64_t)slice * rows * D +
                                       at) = v;
          } else {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
            *reinterpret_cast<uint2 *>(p.out[plane] + at) = pack4(v);
          }
        }
    }
  }
}

// dG, dU from the saved G, U: one pass, 8 elements per thread.
template <int ACT>
__global__ __launch_bounds__(kBlock) void gate_grads_kernel(
    const float *__restrict__ gu, const bf16 *__restrict__ dh,
    bf16 *__restrict__ dgu, int64_t n) {
  const int64_t stride = (int64_t)gridDim.x * kBlock * 8;
  for (int64_t at = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 8; at < n;
       at += stride) {
    const Vec d = load_stream(dh + at);
    const Vec g0 = load_stream(gu + at), g1 = load_stream(gu + at + 4);
    const Vec u0 = load_stream(gu + n + at), u1 = load_stream(gu + n + at + 4);
    float dg[8], du[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = elem<float>(e < 4 ? g0 : g1, e % 4);
      const float u = elem<float>(e < 4 ? u0 : u1, e % 4);
      const float t = elem<bf16>(d, e);
      float a, da;
      activate<ACT>(g, a, da);
      dg[e] = t * u * da;
      du[e] = t * a;
    }
    store_vec(dgu + at, pack<bf16>(dg));
    store_vec(dgu + n + at, pack<bf16>(du));
  }
}

// Sum of the slices' partial products, in slice order; plane q of a slice
// goes to out[q].
__global__ __launch_bounds__(kBlock) void slices_kernel(
    const float *__restrict__ part, bf16 *__restrict__ out0,
    bf16 *__restrict__ out1, int64_t n, int32_t planes, int32_t slices) {
  const int64_t stride = (int64_t)gridDim.x * kBlock * 8;
  const int64_t total = n * planes;
  for (int64_t at = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 8;
       at < total; at += stride) {
    float v[8] = {};
    for (int s = 0; s < slices; ++s) {
      const Vec a = load_stream(part + s * total + at);
      const Vec b = load_stream(part + s * total + at + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += elem<float>(e < 4 ? a : b, e % 4);
    }
    store_vec(at < n ? out0 + at : out1 + (at - n), pack<bf16>(v));
  }
}

// ----------------------------------------------------------------- planning

struct GluPlan {
  bool big = false;
  int32_t tiles_r = 0, tiles_c = 0;
  int32_t steps = 0, slices = 1, per_slice = 0;
  int64_t blocks = 0;
};

GluPlan glu_plan(int form, int64_t M, int64_t D, int64_t F) {
  const bool pair = form == kHidden || form == kGrads;
  const int64_t rows = form == kDw ? F : M, cols = pair ? F : D;
  const int64_t planes = form == kDw ? 2 : 1;
  const int64_t steps = pair ? (D + kStep - 1) / kStep
                        : form == kDx ? 2 * ((F + kStep - 1) / kStep)
                                      : (M + kStep - 1) / kStep;
  auto tiles = [&](int64_t t, int64_t *r, int64_t *c) {
    *r = (rows + t - 1) / t;
    *c = (cols + (pair ? t / 2 : t) - 1) / (pair ? t / 2 : t);
    return *r * *c * planes;
  };
  GluPlan g;
  int64_t r, c;
  int64_t n = tiles(256, &r, &c);
  g.big = n >= 192;
  if (!g.big) n = tiles(128, &r, &c);
  g.tiles_r = (int32_t)r;
  g.tiles_c = (int32_t)c;
  g.steps = (int32_t)steps;
  int64_t slices = 1;
  if (!pair && !g.big && n < kCUs)
    slices = std::max<int64_t>(
        1, std::min<int64_t>(2 * kCUs / n, steps / 4));
  g.per_slice = (int32_t)((steps + slices - 1) / slices);
  g.slices = (int32_t)((steps + g.per_slice - 1) / std::max(g.per_slice, 1));
  if (g.slices < 1) g.slices = 1;
  g.blocks = n * g.slices;
  return g;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of the backward: dG and dU, then the partial products of dx or
// of the weights (whichever needs more; they run one after the other).
size_t glu_bwd_bytes(int64_t M, int64_t D, int64_t F, size_t *part_at) {
  const size_t dgu = align256((size_t)2 * M * F * sizeof(bf16));
  size_t part = 0;
  const GluPlan x = glu_plan(kDx, M, D, F), w = glu_plan(kDw, M, D, F);
  if (x.slices > 1) part = (size_t)x.slices * M * D * sizeof(float);
  if (w.slices > 1)
    part = std::max(part, (size_t)w.slices * 2 * F * D * sizeof(float));
  if (part_at != nullptr) *part_at = dgu;
  return dgu + part;
}

template <int FORM, int ACT>
hipError_t launch_product(const GluPlan &g, Product p, hipStream_t s) {
  p.tiles_r = g.tiles_r;
  p.tiles_c = g.tiles_c;
  p.slices = g.slices;
  p.steps = g.steps;
  p.steps_per_slice = g.per_slice;
  hipError_t e = hipSuccess;
  for (int64_t at = 0; at < g.blocks && e == hipSuccess; at += kMaxGrid) {
    p.block0 = (int32_t)at;
    const int64_t n = std::min(kMaxGrid, g.blocks - at);
    e = g.big ? launch_kernel_threads(product_kernel<FORM, true, ACT>, n, 512,
                                      s, p)
              : launch_kernel_threads(product_kernel<FORM, false, ACT>, n, 256,
                                      s, p);
  }
  return e;
}

int hip_fail(hipError_t e, const char *what) {
  return fail(ADALN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

int check_glu(int64_t M, int64_t D, int64_t F, int act, int dtype) {
  if (dtype != ADALN_BF16)
    return fail(ADALN_ERR_DTYPE, "the gated feed-forward takes bf16 only, got "
                "dtype code %d", dtype);
  if (act != ADALN_ACT_SILU && act != ADALN_ACT_GELU)
    return fail(ADALN_ERR_INVALID, "unknown activation %d", act);
  if (M < 0 || D <= 0 || F <= 0)
    return fail(ADALN_ERR_INVALID, "bad size: M=%lld D=%lld F=%lld",
                (long long)M, (long long)D, (long long)F);
  if (D % 8 != 0 || F % 8 != 0)
    return fail(ADALN_ERR_ALIGN, "D=%lld and F=%lld must be multiples of 8",
                (long long)D, (long long)F);
  if (D > 65536 || F > 262144)
    return fail(ADALN_ERR_UNSUPPORTED, "D exceeds 65536 or F 262144");
  if (M > (int64_t(1) << 24))
    return fail(ADALN_ERR_UNSUPPORTED, "M=%lld exceeds 2^24 tokens",
                (long long)M);
  return ADALN_OK;
}

int check_ptr(const void *p, bool needed, const char *name) {
  if (!needed) return ADALN_OK;
  if (p == nullptr) return fail(ADALN_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
    return fail(ADALN_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return ADALN_OK;
}

template <int ACT>
hipError_t run_fwd(const Product &p, hipStream_t s) {
  return launch_product<kHidden, ACT>(glu_plan(kHidden, p.M, p.D, p.F), p, s);
}

template <int ACT>
hipError_t run_bwd(Product p, bf16 *dx, bf16 *dwg, bf16 *dwu, float *part,
                   hipStream_t s) {
  const int64_t n = (int64_t)p.M * p.F;
  hipError_t e =
      p.gu != nullptr
          ? launch_kernel(gate_grads_kernel<ACT>, (n / 8 + kBlock - 1) / kBlock,
                          s, (const float *)p.gu, p.dh, p.dgu, n)
          : launch_product<kGrads, ACT>(glu_plan(kGrads, p.M, p.D, p.F), p, s);
  if (e != hipSuccess) return e;
  const GluPlan gx = glu_plan(kDx, p.M, p.D, p.F);
  p.part = gx.slices > 1 ? part : nullptr;
  p.out[0] = dx;
  e = launch_product<kDx, 0>(gx, p, s);
  const int64_t nx = (int64_t)p.M * p.D, nw = (int64_t)p.F * p.D;
  if (e == hipSuccess && gx.slices > 1)
    e = launch_kernel(slices_kernel, (nx / 8 + kBlock - 1) / kBlock, s,
                      (const float *)part, dx, dx, nx, (int32_t)1,
                      (int32_t)gx.slices);
  if (e != hipSuccess) return e;
  const GluPlan gw = glu_plan(kDw, p.M, p.D, p.F);
  p.part = gw.slices > 1 ? part : nullptr;
  p.out[0] = dwg;
  p.out[1] = dwu;
  e = launch_product<kDw, 0>(gw, p, s);
  if (e == hipSuccess && gw.slices > 1)
    e = launch_kernel(slices_kernel, (2 * nw / 8 + kBlock - 1) / kBlock, s,
                      (const float *)part, dwg, dwu, nw, (int32_t)2,
                      (int32_t)gw.slices);
  return e;
}

}  // namespace
}  // namespace adaln

using namespace adaln;

ADALN_API int adaln_glu_fwd(const void *x, const void *wg, const void *wu,
                            void *h, float *saved, int64_t M, int64_t D,
                            int64_t F, int act, int dtype, void *stream) {
  ADALN_TRY(check_glu(M, D, F, act, dtype));
  const bool rows = M > 0;
  ADALN_TRY(check_ptr(x, rows, "x"));
  ADALN_TRY(check_ptr(wg, rows, "wg"));
  ADALN_TRY(check_ptr(wu, rows, "wu"));
  ADALN_TRY(check_ptr(h, rows, "h"));
  ADALN_TRY(check_ptr(saved, rows && saved != nullptr, "saved"));
  if (!rows) return ok();
  Product p = {};
  p.x = (const bf16 *)x;
  p.w[0] = (const bf16 *)wg;
  p.w[1] = (const bf16 *)wu;
  p.h = (bf16 *)h;
  p.gu = saved;
  p.M = (int32_t)M;
  p.D = (int32_t)D;
  p.F = (int32_t)F;
  const hipError_t e = act == ADALN_ACT_SILU
                           ? run_fwd<kSilu>(p, (hipStream_t)stream)
                           : run_fwd<kGeluTanh>(p, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "adaln_glu_fwd launch");
  return ok();
}

ADALN_API size_t adaln_glu_bwd_workspace_bytes(int64_t M, int64_t D, int64_t F,
                                               int dtype) {
  if (check_glu(M, D, F, ADALN_ACT_SILU, dtype) != ADALN_OK || M == 0) return 0;
  return glu_bwd_bytes(M, D, F, nullptr);
}

ADALN_API int adaln_glu_bwd(const void *dh, const void *x, const void *wg,
                            const void *wu, const float *saved, void *dx,
                            void *dwg, void *dwu, void *workspace,
                            size_t workspace_bytes, int64_t M, int64_t D,
                            int64_t F, int act, int dtype, void *stream) {
  ADALN_TRY(check_glu(M, D, F, act, dtype));
  const bool rows = M > 0;
  ADALN_TRY(check_ptr(dh, rows, "dh"));
  ADALN_TRY(check_ptr(x, rows, "x"));
  ADALN_TRY(check_ptr(wg, rows, "wg"));
  ADALN_TRY(check_ptr(wu, rows, "wu"));
  ADALN_TRY(check_ptr(saved, rows && saved != nullptr, "saved"));
  ADALN_TRY(check_ptr(dx, rows, "dx"));
  ADALN_TRY(check_ptr(dwg, true, "dwg"));
  ADALN_TRY(check_ptr(dwu, true, "dwu"));
  hipStream_t s = (hipStream_t)stream;
  if (!rows) {
    // no tokens: the weights' gradients are empty sums (no slices to add)
    const int64_t nw = F * D;
    const hipError_t e = launch_kernel(
        slices_kernel, (2 * nw / 8 + kBlock - 1) / kBlock, s,
        (const float *)nullptr, (bf16 *)dwg, (bf16 *)dwu, nw, (int32_t)2,
        (int32_t)0);
    if (e != hipSuccess) return hip_fail(e, "adaln_glu_bwd launch");
    return ok();
  }
  size_t part_at = 0;
  const size_t need = glu_bwd_bytes(M, D, F, &part_at);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ADALN_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu%s",
                need, workspace_bytes, workspace == nullptr ? " (NULL)" : "");
  ADALN_TRY(check_ptr(workspace, true, "workspace"));
  Product p = {};
  p.x = (const bf16 *)x;
  p.w[0] = (const bf16 *)wg;
  p.w[1] = (const bf16 *)wu;
  p.gu = const_cast<float *>(saved);
  p.dh = (const bf16 *)dh;
  p.dgu = (bf16 *)workspace;
  p.M = (int32_t)M;
  p.D = (int32_t)D;
  p.F = (int32_t)F;
  float *part = (float *)((char *)workspace + part_at);
  const hipError_t e =
      act == ADALN_ACT_SILU
          ? run_bwd<kSilu>(p, (bf16 *)dx, (bf16 *)dwg, (bf16 *)dwu, part, s)
          : run_bwd<kGeluTanh>(p, (bf16 *)dx, (bf16 *)dwg, (bf16 *)dwu, part,
                               s);
  if (e != hipSuccess) return hip_fail(e, "adaln_glu_bwd launch");
  return ok();
}
