// Gated feed-forward of a transformer block, forward and backward, with its C
// entry points.
//
//     G = x Wg^T, U = x Wu^T, h = act(G) * U         x [M, D], W [F, D]
//     dU = dh * act(G), dG = dh * U * act'(G)
//     dx = dG Wg + dU Wu,  dWg = dG^T x,  dWu = dU^T x
//
// Four products of one shape of loop, all on the matrix cores (bf16 or f32
// operands, float32 sums): a workgroup computes a tile of rows x columns,
// walking the summed dimension in steps of 128 bytes.  Each step's two operand
// tiles go from memory straight to LDS (16 bytes per lane, no registers),
// double-buffered: the loads of step s + 1 are in flight while step s is
// multiplied.
//
// An operand is stored with the summed dimension contiguous (x and W in the
// forward) or across it (W in dx; both in dW).  Its LDS tile keeps the
// memory's order, 128-byte rows of summed elements or rows of 128 or 256
// columns, and the fragment reads do the rest: 16 bytes of a row as they are,
// or, across, 4 x 16 blocks of bf16 transposed by the LDS read itself, or f32
// elements one by one.  The 16-byte pieces of
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
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) char lds_char;

// Summed elements per step: 128 bytes of them.
template <typename T>
constexpr int kStep = 128 / sizeof(T);

// 16 bytes per lane from memory to LDS at `lds` + 16 * lane: a wave-uniform
// base and a 32-bit offset per lane.  Outstanding loads are waited for by
// arrive() below, by hand: the compiler does not see these loads.  (m0 takes
// the LDS address.  The s_nop is the wait state that the ISA asks for between
// writing m0 and a load to LDS.)
__device__ __forceinline__ void dma(uint32_t lds, const void *base,
                                    uint32_t offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(offset), "s"(base)
      : "memory", "m0");
}

// All loads of this wavefront but the last LATER have landed, then those of
// every wavefront.  (Loads return in order; a store among them, which may
// not, only makes the wait longer.)
template <int LATER>
__device__ __forceinline__ void arrive() {
  asm volatile(
      "s_waitcnt vmcnt(%0) lgkmcnt(0)\n\t"
      "s_barrier" ::"n"(LATER)
      : "memory");
}

// A lane's part of a fragment of 32 rows or columns: 16 bytes, the elements
// 8 (l / 32) + [0, 8) of 16 (bf16) or 4 (l / 32) + [0, 4) of 8 (f32) of row
// l % 32.
template <typename T>
struct Frag;
template <>
struct Frag<bf16> {
  bf16x8 v;
};
template <>
struct Frag<float> {
  f32x4 v;
};

// acc += a b^T over the fragments' summed elements.  (f32: the cores take two
// elements at a time, one of each half of the lanes; any pairing of elements
// does as long as both operands have the same.)
__device__ __forceinline__ void multiply_add(f32x16 &acc, const Frag<bf16> &a,
                                             const Frag<bf16> &b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void multiply_add(f32x16 &acc,
                                             const Frag<float> &a,
                                             const Frag<float> &b) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[c], b.v[c], acc, 0, 0, 0);
}

// An operand whose summed dimension is contiguous: ROWS rows of a step's 128
// bytes, 8 pieces of 16.  Row r keeps its piece c at c ^ ((r >> 1) & 7): 16
// consecutive rows then cover all banks.  Rows past the operand's last repeat
// it (their products are not stored); past the end of the sum, `left`
// elements into the step, a lane loads the last piece again, and clear() puts
// zeros in its place.
template <typename T, int ROWS, int WAVES>
struct Along {
  static constexpr int E = Elems<T>::value;
  static constexpr int kBytes = ROWS * 128;
  static constexpr int kLoads = ROWS / (8 * WAVES);
  uint32_t off[kLoads];  // byte offset of each load's row

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
               (uint32_t)pitch * (uint32_t)sizeof(T);
  }
  // Load i of a step; base: the operand at row row0, element k0.
  __device__ __forceinline__ void load(int i, uint32_t lds, const char *base,
                                       uint32_t, int left) const {
    dma(lds + (wave_id() + i * WAVES) * 1024, base,
        off[i] + min(lane_piece() * 16, (left - E) * (int)sizeof(T)));
  }
  static __device__ __forceinline__ void clear(char *tile, int left) {
    if (lane_piece() * E >= left) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        store_vec(tile + (wave_id() + i * WAVES) * 1024 + lane_id() * 16,
                  vzero());
    }
  }
  // Fragment of 32 rows from `row`, sub-step kk of 4.
  static __device__ __forceinline__ Frag<T> frag(const char *tile, int row,
                                                 int kk) {
    const int l = lane_id();
    const int r = l % 32;
    const int piece = (kk * 2 + l / 32) ^ ((r >> 1) & 7);
    return *reinterpret_cast<const Frag<T> *>(tile + row * 128 + r * 128 +
                                              piece * 16);
  }
};

// An operand stored across the summed dimension: a step's rows of COLS
// columns, in pieces of 16 bytes; row k keeps its piece c at c ^ turn(k), so
// that what a read takes of several rows lies in distinct banks: of bf16 the
// four rows of a transposing read, of f32 the rows of the two lane halves.
// Columns past the last repeat the last piece; rows past the end of the sum
// repeat the last, and are cleared.
template <typename T, int COLS, int WAVES>
struct Across {
  static constexpr int E = Elems<T>::value;
  static constexpr int kPitch = COLS * sizeof(T);
  static constexpr int kBytes = kPitch * kStep<T>;
  static constexpr int kPieces = COLS / E;
  static constexpr int kRows = 64 / kPieces * WAVES;  // rows per load
  static constexpr int kLoads = kStep<T> / kRows;
  uint32_t off;  // byte offset of the lane's columns

  static __device__ __forceinline__ int turn(int k) {
    return sizeof(T) == 2 ? (k & 3) << 2 : (k >> 2 & 1) << 3;
  }
  static __device__ __forceinline__ int lane_row() {
    return (wave_id() * 64 + lane_id()) / kPieces;
  }
  static __device__ __forceinline__ int lane_piece() {
    return (lane_id() % kPieces) ^ turn(lane_row());
  }
  __device__ __forceinline__ void start(int col0, int cols, int) {
    off = (uint32_t)min(lane_piece() * E, cols - E - col0) *
          (uint32_t)sizeof(T);
  }
  // base: the operand at row k0, column col0; pitch: its bytes per row.
  __device__ __forceinline__ void load(int i, uint32_t lds, const char *base,
                                       uint32_t pitch, int left) const {
    dma(lds + (wave_id() + i * WAVES) * 1024, base,
        off + (uint32_t)min(i * kRows + lane_row(), left - 1) * pitch);
  }
  static __device__ __forceinline__ void clear(char *tile, int left) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i * kRows + lane_row() >= left)
        store_vec(tile + (wave_id() + i * WAVES) * 1024 + lane_id() * 16,
                  vzero());
  }
  // Fragment of 32 columns from `col`, sub-step kk of 4.
  static __device__ __forceinline__ Frag<T> frag(const char *tile, int col,
                                                 int kk) {
    const int l = lane_id();
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
      const int k = kk * 16 + (l / 32) * 8 + (l % 16) / 4;
      const int piece =
          (col / 8 + ((l >> 4) & 1) * 2 + ((l & 3) >> 1)) ^ turn(k);
      const char *p = tile + k * kPitch + piece * 16 + (l & 1) * 8;
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4 *)(p + 4 * kPitch));
      const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      f.v = __builtin_bit_cast(bf16x8, v);
    } else {
      const int k = kk * 8 + (l / 32) * 4, c = col + l % 32;
      const char *p =
          tile + k * kPitch + ((c / 4) ^ turn(k)) * 16 + c % 4 * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f.v[i] = *reinterpret_cast<const float *>(p + i * kPitch);
    }
    return f;
  }
};

// ------------------------------------------------------------- activations

enum { kSilu = 0, kGeluTanh = 1 };

// exp(-v).  float32 results keep its digits; for those rounded to bfloat16 (or
// to two of them, 2^-16) the hardware's exp2 of a rounded product will do,
// |v| * 2^-24 of itself.  (MI355X, f32 forward, the full exponential against
// the other: 24960 x 1536 -> 4096 4465 us against 4434, 16380 x 64 -> 8192,
// where little else is computed, 380 against 344.)
template <typename T>
__device__ __forceinline__ float exp_minus(float v) {
  return sizeof(T) == 2 ? __expf(-v) : expf(-v);
}

// act(g) and act'(g).  Both are g times a logistic function s = 1 / (1 + e),
// e = exp(-v), of v = g or twice the tanh form's polynomial: (1 + tanh(w)) / 2
// = 1 / (1 + exp(-2w)) keeps its digits where 1 + tanh(w) cancels.  act' needs
// 1 - s too, which is e s: a difference would leave few digits of it where s is
// near 1, and g times as much of the error.  So float32 derivatives are within
// a few 2^-24 of themselves for positive g (a difference: up to 24 of them for
// SiLU, 800 for GELU).  Both ends saturate: where e is infinite, s is 0 and 1 -
// s is 1; g^2, which passes float32 at |g| = 1.8e19, stops at 1e30, where s or
// 1 - s is 0 long since and must not meet an infinity.
// The hardware's reciprocal (one unit in the last place; a correctly rounded
// quotient takes ten instructions more per element) gives zero for quotients
// below 2^-126: a quarter of 1 + e has none.
template <typename T, int ACT>
__device__ __forceinline__ void activate(float g, float &a, float &da) {
  constexpr float c = 0.7978845608028654f, p = 0.044715f;
  const float g2 = fminf(g * g, 1e30f);
  const float e =
      exp_minus<T>(ACT == kSilu ? g : 2.f * c * g * (1.f + p * g2));
  const float s4 = __builtin_amdgcn_rcpf(fmaf(e, 0.25f, 0.25f));
  const float s = 0.25f * s4;
  const float rest = e < INFINITY ? 0.25f * e * s4 : 1.f;
  a = 0.25f * g * s4;
  if constexpr (ACT == kSilu)
    da = s * (1.f + g * rest);
  else
    da = s + s * rest * g * (2.f * c * (1.f + 3.f * p * g2));
}

__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
  uint2 u;
  const f32x2 a = {f[0], f[1]}, b = {f[2], f[3]};
  u.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
  u.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2));
  return u;
}

__device__ __forceinline__ void store_one(bf16 *p, float f) {
  const f32x2 v = {f, f};
  const uint32_t w =
      __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  *p = bf16{(uint16_t)w};
}
__device__ __forceinline__ void store_one(float *p, float f) { *p = f; }

__device__ __forceinline__ float load_one(const bf16 *p) {
  return __builtin_bit_cast(float, (uint32_t)p->bits << 16);
}
__device__ __forceinline__ float load_one(const float *p) { return *p; }

// Four neighbouring elements.
__device__ __forceinline__ void load4(const bf16 *p, float (&f)[4]) {
  const uint2 d = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = e < 2 ? d.x : d.y;
    f[e] = __builtin_bit_cast(float, (e & 1) ? (w & 0xffff0000u) : (w << 16));
  }
}
__device__ __forceinline__ void load4(const float *p, float (&f)[4]) {
  const Vec v = load_vec(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = elem<float>(v, e);
}

__device__ __forceinline__ void store4(bf16 *p, const float (&f)[4]) {
  *reinterpret_cast<uint2 *>(p) = pack4(f);
}
__device__ __forceinline__ void store4(float *p, const float (&f)[4]) {
  store_vec(p, pack<float>(f));
}

// Eight neighbouring elements, 16-byte aligned.
__device__ __forceinline__ void store8(bf16 *p, const float (&f)[8]) {
  store_vec(p, pack<bf16>(f));
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
  store_vec(p, pack<float>(a));
  store_vec(p + 4, pack<float>(b));
}

// ------------------------------------------------------- storing a block

// What lanes of a wavefront wrote to LDS before it, the others read after it.
// The hardware keeps a wavefront's accesses to LDS in order; this keeps the
// compiler from moving them.
__device__ __forceinline__ void lanes_agree() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A 32 x 32 block as the matrix cores leave it (lane l: row l % 32, columns
// 8 q + 4 (l / 32) + e in register 4 q + e) to memory, in row order: through
// LDS of the wavefront's own, so that 8 lanes write a whole 128-byte line
// (float32) or 4 lanes half of one (bf16) at a time instead of 32 lanes 32
// pieces of lines.  The rows' pitch keeps both sides free of bank conflicts.
// n_r, n_c: rows and columns of the block that exist.  Forward of 24960 x
// 1536 -> 4096 with G and U saved, on MI355X: 952 -> 673 us (with later steps
// 605-650).
constexpr int kStageBytes = 32 * (32 * 4 + 16);

__device__ __forceinline__ void store_block(char *stage, const f32x16 &v,
                                            float *out, int64_t pitch, int n_r,
                                            int n_c) {
  const int lane = lane_id();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f32x4 f = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    *reinterpret_cast<f32x4 *>(stage + (lane % 32) * 144 +
                               (8 * q + 4 * (lane / 32)) * 4) = f;
  }
  lanes_agree();
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int r = t * 8 + lane / 8, c = lane % 8 * 4;
    const Vec f = load_vec(stage + r * 144 + c * 4);
    if (r < n_r && c < n_c) store_stream(out + r * pitch + c, f);
  }
  lanes_agree();
}

__device__ __forceinline__ void store_block(char *stage, const f32x16 &v,
                                            bf16 *out, int64_t pitch, int n_r,
                                            int n_c) {
  const int lane = lane_id();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float f[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    *reinterpret_cast<uint2 *>(stage + (lane % 32) * 80 +
                               (8 * q + 4 * (lane / 32)) * 2) = pack4(f);
  }
  lanes_agree();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r = t * 16 + lane / 4, c = lane % 4 * 8;
    const Vec f = load_vec(stage + r * 80 + c * 2);
    if (r < n_r && c < n_c) store_vec(out + r * pitch + c, f);
  }
  lanes_agree();
}

// ------------------------------------------------------------- the products

enum {
  kHidden = 0,  // h (and G, U): rows tokens, columns hidden features
  kGrads = 1,   // dG, dU with G, U computed again
  kDx = 2,      // dx: rows tokens, columns features, sum over 2 F
  kDw = 3       // dWg, dWu: rows hidden features, columns features, sum over M
};

template <typename T>
struct Product {
  const T *x;             // [M, D]
  const T *w[2];          // Wg, Wu [F, D]
  T *h;                   // [M, F]
  float *gu;              // saved G, U [2, M, F] (or NULL)
  const T *dh;            // [M, F]
  T *dgu;                 // dG, dU [2, M, F]
  T *dx;                  // [M, D]
  T *dw[2];               // dWg, dWu [F, D]
  int32_t M, D, F;
  int32_t fold;           // not 0: dx's row m is the sum of rows m, m + fold
};

// How a product is cut: tiles of a plane (dW has two), `full` of them
// computed whole, `rem` that follow in `slices` of `per_slice` steps each.
struct Tiles {
  float *part = nullptr;  // partial tiles [slices, rem, tile, tile]
  int32_t tiling = 0;
  int32_t tiles_r = 0, tiles_c = 0;
  int32_t steps = 0;
  int32_t full = 0, rem = 0;
  int32_t slices = 1, per_slice = 0;
  int32_t block0 = 0;     // first block of this launch
  __host__ __device__ int tile() const;
};

// Workgroups go to the eight XCDs in turn: item `id` of `total` in an order
// that gives each XCD a contiguous run of items.
__device__ __forceinline__ int xcd_run(int id, int total) {
  const int per = total / 8;
  return id < per * 8 ? (id % 8) * per + id / 8 : id;
}

// Tile n of the plan: its plane, row and column.  In bands of 8 tile rows, so
// that tiles that run together share operands in an XCD's L2.
__device__ __forceinline__ void tile_of(int n, int tiles_r, int tiles_c,
                                        int &plane, int &tr, int &tc) {
  plane = n / (tiles_r * tiles_c);
  n -= plane * tiles_r * tiles_c;
  constexpr int kBand = 8;
  const int band = n / (kBand * tiles_c);
  const int in = n - band * kBand * tiles_c;
  const int rows = min(kBand, tiles_r - band * kBand);
  tr = band * kBand + in % rows;
  tc = in / rows;
}

// Four tilings.  kBig: 256 x 256 tiles by 8 wavefronts (2 x 4, each 128 x
// 64), two steps in LDS (128 KiB); kSmall: 128 x 128 by 4 (2 x 2, each 64 x
// 64), two steps (64 KiB, so two workgroups to a CU); kDeep: the same with
// four steps (128 KiB), for calls of so few tiles that a CU has one at most
// and a step's arithmetic is far shorter than its loads take to arrive; kFine:
// 64 x 64 by 2, four steps (64 KiB), of pairs whose deep tiles would leave CUs
// idle.
// Columns of kHidden and kGrads: half of them of G, half the same ones of U,
// so that a lane holds both of an element.
enum { kSmall = 0, kBig = 1, kDeep = 2, kFine = 3 };

__host__ __device__ inline int Tiles::tile() const {
  return tiling == kBig ? 256 : tiling == kFine ? 64 : 128;
}

constexpr int tiling_threads(int tiling) {
  return tiling == kBig ? 512 : tiling == kFine ? 128 : 256;
}
constexpr int tiling_waves(int tiling) {
  return tiling == kDeep || tiling == kFine ? 1 : 2;
}
// LDS: two steps' operand tiles, or four.
constexpr int tiling_lds(int tiling) {
  return (tiling == kDeep || tiling == kFine ? 4 : 2) * 2 *
         (tiling == kBig ? 256 : tiling == kFine ? 64 : 128) * 128;
}

// Block `id` of a product.
template <typename T, int FORM, int TILING, int ACT>
__device__ __forceinline__ void product(const Product<T> &p, const Tiles &q,
                                        int id, char *lds) {
  constexpr bool BIG = TILING == kBig;
  constexpr bool FINE = TILING == kFine;
  constexpr int kWaves = BIG ? 8 : FINE ? 2 : 4;
  constexpr int kTile = BIG ? 256 : FINE ? 64 : 128;
  constexpr int kBufs = TILING == kDeep || FINE ? 4 : 2;
  constexpr int kWn = kWaves / 2;          // wavefronts across the columns
  constexpr int MI = kTile / 2 / 32;        // 32-row blocks of a wavefront
  constexpr int NI = kTile / kWn / 32;      // 32-column blocks
  constexpr bool kPair = FORM == kHidden || FORM == kGrads;
  constexpr int kCols = kPair ? kTile / 2 : kTile;
  constexpr int NP = NI / 2;  // of a pair: blocks of G, then as many of U
  using Row = std::conditional_t<FORM == kDw, Across<T, kTile, kWaves>,
                                 Along<T, kTile, kWaves>>;
  // (of a pair, the rows of one weight)
  using Col = std::conditional_t<kPair, Along<T, kTile / 2, kWaves>,
                                 Across<T, kTile, kWaves>>;
  constexpr uint32_t kColBytes = kPair ? 2 * Col::kBytes : Col::kBytes;
  constexpr uint32_t kBuf = Row::kBytes + kColBytes;
  static_assert(kBufs * kBuf == tiling_lds(TILING), "");

  // The first `full` blocks compute a tile each; the rest, slices of the
  // sums of the last `rem` tiles.
  int n, split = 0;
  if (id < q.full) {
    n = xcd_run(id, q.full);
  } else {
    split = (id - q.full) / q.rem;
    n = q.full + xcd_run(id - q.full - split * q.rem, q.rem);
  }
  const bool partial = id >= q.full;
  int plane, tr, tc;
  tile_of(n, q.tiles_r, q.tiles_c, plane, tr, tc);
  const int row0 = tr * kTile, col0 = tc * kCols;
  const int M = p.M, D = p.D, F = p.F;
  const int s0 = partial ? split * q.per_slice : 0;
  const int s1 = partial ? min(s0 + q.per_slice, q.steps) : q.steps;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char *)lds;

  Row row;
  Col col;
  row.start(row0, FORM == kDw ? F : M, FORM == kDx || FORM == kDw ? F : D);
  col.start(col0, kPair ? F : D, D);
  // The operands of the step to be loaded next (of a pair: x, Wg, Wu), and
  // how far apart two steps are.
  const char *pr, *pc, *pu = nullptr;
  constexpr int S = kStep<T>;
  const uint32_t pitch_r = sizeof(T) * (uint32_t)(kPair ? D : F);
  const uint32_t pitch_c = sizeof(T) * (uint32_t)D;
  const int64_t next_r = FORM == kDw ? S * (int64_t)pitch_r : 128;
  const int64_t next_c = kPair ? 128 : S * (int64_t)pitch_c;
  const int K = kPair ? D : FORM == kDx ? F : M;
  const int per = FORM == kDx ? q.steps / 2 : q.steps;  // steps per plane
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
  // Elements of the sum that step s has left, of its plane.
  auto left = [&](int s) {
    return K - (FORM == kDx && s >= per ? s - per : s) * S;
  };
  // On to step s, the one after the last loaded; past the end, the last step
  // is loaded again, into a buffer that nobody reads any more.
  int pl_left = 0;
  auto advance = [&](int s) {
    if (s < s1) {
      pr += next_r;
      pc += next_c;
      if constexpr (kPair) pu += next_c;
      if constexpr (FORM == kDx)
        if (s == per) seek(per);
      pl_left = left(s);
    }
  };
  // Load n of that step, into a buffer.
  constexpr int kLoads = Row::kLoads + (kPair ? 2 : 1) * Col::kLoads;
  auto load = [&](int n, int buf) {
    const uint32_t at = lds0 + buf * kBuf;
    if (n < Row::kLoads)
      row.load(n, at, pr, pitch_r, pl_left);
    else if (n < Row::kLoads + Col::kLoads)
      col.load(n - Row::kLoads, at + Row::kBytes, pc, pitch_c, pl_left);
    else
      col.load(n - Row::kLoads - Col::kLoads,
               at + Row::kBytes + Col::kBytes, pu, pitch_c, pl_left);
  };
  // Zeros past the end of the sum in the tile of step s, which has landed.
  auto clear = [&](int s, int buf) {
    if (s < s1 && left(s) < S) {
      char *tile = lds + buf * kBuf;
      Row::clear(tile, left(s));
      Col::clear(tile + Row::kBytes, left(s));
      if constexpr (kPair)
        Col::clear(tile + Row::kBytes + Col::kBytes, left(s));
      __syncthreads();
    }
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
  constexpr int KK = 4;
  Frag<T> a[2][MI], b[2][NI];
  // Fragment n of the NI + MI of sub-step kk.
  auto read = [&](int n, int buf, int kk) {
    const char *rt = lds + buf * kBuf;
    const char *ct = rt + Row::kBytes;
    if (n < NI)
      b[kk & 1][n] = Col::frag(
          ct,
          kPair ? n / NP * (kTile / 2) + wn * NP * 32 + n % NP * 32
                : wn * NI * 32 + n * 32,
          kk);
    else
      a[kk & 1][n - NI] = Row::frag(rt, wrow + (n - NI) * 32, kk);
  };
  constexpr int kMul = MI * NI;
  constexpr int kFirst = kLoads / 2;
  auto multiply = [&](int n, int kk) {
    const int i = n / NI, j = n % NI;
    multiply_add(acc[i][j], b[kk & 1][j], a[kk & 1][i]);
  };
  if (s0 < s1) {
    seek(s0);
    pl_left = left(s0);
#pragma unroll
    for (int s = 0; s < kBufs - 1; ++s) {
#pragma unroll
      for (int n = 0; n < kLoads; ++n) load(n, s);
      advance(s0 + s + 1);
    }
    arrive<(kBufs - 2) * kLoads>();
#pragma unroll
    for (int n = 0; n < kFirst; ++n) load(n, kBufs - 1);
    clear(s0, 0);
#pragma unroll
    for (int n = 0; n < NI + MI; ++n) read(n, 0, 0);
  }
  int buf = 0;
  for (int s = s0; s < s1; ++s) {
    const int before = buf == 0 ? kBufs - 1 : buf - 1;
    const int after = buf == kBufs - 1 ? 0 : buf + 1;
#pragma unroll
    for (int kk = 0; kk < KK - 1; ++kk) {
#pragma unroll
      for (int n = 0; n < kMul; ++n) {
        multiply(n, kk);
        if (n < NI + MI) read(n, buf, kk + 1);
        if (kk == 0) {
#pragma unroll
          for (int l = kFirst + n * (kLoads - kFirst) / kMul;
               l < kFirst + (n + 1) * (kLoads - kFirst) / kMul; ++l)
            load(l, before);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = kMul; n < NI + MI; ++n) read(n, buf, kk + 1);
    }
    arrive<(kBufs - 2) * kLoads>();
    clear(s + 1, after);
    advance(s + kBufs);
#pragma unroll
    for (int n = 0; n < kMul; ++n) {
      multiply(n, KK - 1);
      // (past the last step: what lies there, not used)
      if (n < NI + MI) read(n, after, 0);
#pragma unroll
      for (int l = n * kFirst / kMul; l < (n + 1) * kFirst / kMul; ++l)
        load(l, buf);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = kMul; n < NI + MI; ++n) read(n, after, 0);
    buf = after;
  }
  arrive<0>();  // LDS is free: nothing on its way in, nobody reading

  // acc[i][j][4 q + e] of lane l is row l % 32 of block i, column
  // 8 q + 4 (l / 32) + e of block j.
  char *stage = lds + wave * kStageBytes;
  static_assert(kWaves * kStageBytes <= kBufs * kBuf, "");
  const int lane = lane_id();
  const int rows = FORM == kDw ? F : M, cols = kPair ? F : D;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int r = row0 + wrow + i * 32;
    if (r >= rows) break;
    const int n_r = rows - r;
#pragma unroll
    for (int j = 0; j < (kPair ? NP : NI); ++j) {
      const int c = col0 + (wn * (kPair ? NP : NI) + j) * 32;
      if (c >= cols) break;
      const int n_c = cols - c;
      const int64_t at = (int64_t)r * cols + c;
      const int64_t plane_size = (int64_t)M * F;
      if constexpr (kPair) {
        const f32x16 g = acc[i][j], u = acc[i][NP + j];
        f32x16 v0, v1;
        if constexpr (FORM == kHidden) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, da;
            activate<T, ACT>(g[e], a, da);
            v0[e] = a * u[e];
          }
          store_block(stage, v0, p.h + at, cols, n_r, n_c);
          if (p.gu != nullptr) {
            store_block(stage, g, p.gu + at, cols, n_r, n_c);
            store_block(stage, u, p.gu + plane_size + at, cols, n_r, n_c);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int mine = 8 * q + 4 * (lane / 32);
            float dh[4] = {};
            if (lane % 32 < n_r && mine < n_c)
              load4(p.dh + at + (int64_t)(lane % 32) * cols + mine, dh);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a, da;
              activate<T, ACT>(g[4 * q + e], a, da);
              v0[4 * q + e] = dh[e] * u[4 * q + e] * da;
              v1[4 * q + e] = dh[e] * a;
            }
          }
          store_block(stage, v0, p.dgu + at, cols, n_r, n_c);
          store_block(stage, v1, p.dgu + plane_size + at, cols, n_r, n_c);
        }
      } else if (partial) {
        store_block(stage, acc[i][j],
                    q.part + (((int64_t)split * q.rem + n - q.full) * kTile +
                              (r - row0)) * kTile + (c - col0),
                    kTile, n_r, n_c);
      } else {
        store_block(stage, acc[i][j],
                    (FORM == kDx ? p.dx : p.dw[plane]) + at, cols, n_r, n_c);
      }
    }
  }
}

template <typename T, int FORM, int TILING, int ACT>
__global__ __launch_bounds__(tiling_threads(TILING),
                             tiling_waves(TILING)) void
product_kernel(Product<T> p, Tiles q) {
  __shared__ __align__(1024) char lds[tiling_lds(TILING)];
  product<T, FORM, TILING, ACT>(p, q, blockIdx.x + q.block0, lds);
}

// dx and dW in one launch, where the tiles of either alone would leave CUs
// idle; the product with the longer blocks comes first.
template <typename T, int TILING>
__global__ __launch_bounds__(tiling_threads(TILING),
                             tiling_waves(TILING)) void
grads_kernel(Product<T> p, Tiles x, Tiles w, int32_t first, int32_t w_first) {
  __shared__ __align__(1024) char lds[tiling_lds(TILING)];
  const bool second = (int)blockIdx.x >= first;
  const int id = blockIdx.x - (second ? first : 0);
  if (second == (w_first != 0))
    product<T, kDx, TILING, 0>(p, x, id, lds);
  else
    product<T, kDw, TILING, 0>(p, w, id, lds);
}

// dG, dU of 8 elements from G, U [2, n].
template <typename T, int ACT>
__device__ __forceinline__ void gate_grads(const float *gu, const T *dh,
                                           int64_t n, int64_t at,
                                           float (&dg)[8], float (&du)[8]) {
  Vec d[8 / Elems<T>::value];
#pragma unroll
  for (int i = 0; i < 8 / Elems<T>::value; ++i)
    d[i] = load_stream(dh + at + i * Elems<T>::value);
  const Vec g0 = load_stream(gu + at), g1 = load_stream(gu + at + 4);
  const Vec u0 = load_stream(gu + n + at), u1 = load_stream(gu + n + at + 4);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float g = elem<float>(e < 4 ? g0 : g1, e % 4);
    const float u = elem<float>(e < 4 ? u0 : u1, e % 4);
    const float t = elem<T>(d[e / Elems<T>::value], e % Elems<T>::value);
    float a, da;
    activate<T, ACT>(g, a, da);
    dg[e] = t * u * da;
    du[e] = t * a;
  }
}

// dG, dU from the saved G, U: one pass, 8 elements per thread.  In bf16 they
// are rounded to it, as kGrads rounds them: the matrix cores' operands of dx
// and dW.  Kept in two parts, as for few tokens (GluBackward::split), they
// would double those products, for 1.41 times less error of dx and dW.
template <typename T, int ACT>
__global__ __launch_bounds__(kBlock) void gate_grads_kernel(
    const float *__restrict__ gu, const T *__restrict__ dh,
    T *__restrict__ dgu, int64_t n) {
  const int64_t stride = (int64_t)gridDim.x * kBlock * 8;
  for (int64_t at = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 8; at < n;
       at += stride) {
    float dg[8], du[8];
    gate_grads<T, ACT>(gu, dh, n, at, dg, du);
    store8(dgu + at, dg);
    store8(dgu + n + at, du);
  }
}

// The same for few tokens, without the rounding to bf16: each of dG, dU is the
// sum of two bf16 (exact to 2^-16), the second in the rows of as many tokens
// more, and x stands there twice.  The products of 2 M tokens then give dW,
// and dx in the sums of rows m and M + m.
template <int ACT>
__global__ __launch_bounds__(kBlock) void split_grads_kernel(
    const float *__restrict__ gu, const bf16 *__restrict__ dh,
    const bf16 *__restrict__ x, bf16 *__restrict__ dgu, bf16 *__restrict__ x2,
    int64_t n, int64_t n_x) {
  const int64_t stride = (int64_t)gridDim.x * kBlock * 8;
  for (int64_t i = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 8;
       i < n + n_x; i += stride) {
    if (i >= n) {
      const Vec v = load_vec(x + i - n);
      store_vec(x2 + i - n, v);
      store_vec(x2 + n_x + i - n, v);
      continue;
    }
    float d[2][8];
    gate_grads<bf16, ACT>(gu, dh, n, i, d[0], d[1]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const Vec hi = pack<bf16>(d[q]);
      float lo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = elem<bf16>(hi, e);
        lo[e] = fabsf(f) < INFINITY ? d[q][e] - f : 0.f;
      }
      store_vec(dgu + 2 * q * n + i, hi);
      store8(dgu + (2 * q + 1) * n + i, lo);
    }
  }
}

// --------------------------------------------------------------- few tokens

// kHidden and kGrads of up to 16 * TB tokens: bound by the weights' bytes, so
// they go from memory to registers as matrix fragments, each read once, and
// the tokens' fragments come from the caches.  A workgroup owns 16 hidden
// features; its 8 wavefronts take the steps of 64 bytes of the sum in turn (so
// that together they read 512 contiguous bytes of every row), four steps'
// loads in flight each, and their sums meet in LDS, added in order.  (Plain
// loads: with the streaming hint one token took 8.4 us, not 7.4, D = 1536, F =
// 4096; 32 features per workgroup, 11.6.)
template <typename T>
__device__ __forceinline__ void multiply_few(f32x4 &acc, const Vec &a,
                                             const Vec &b) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0,
        0, 0);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(elem<float>(a, c),
                                                 elem<float>(b, c), acc, 0, 0,
                                                 0);
  }
}

constexpr int kFewWaves = 8;
constexpr int kFewUnroll = 4;

template <typename T, int FORM, int TB, int ACT>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(Product<T> p) {
  constexpr int E = Elems<T>::value;
  constexpr int S = 4 * E;  // summed elements per step
  __shared__ f32x4 sums[kFewWaves][2][TB][64];
  const int lane = lane_id(), wave = wave_id();
  const int M = p.M, D = p.D, F = p.F;
  const int f0 = blockIdx.x * 16;
  const int64_t f = min(f0 + lane % 16, F - 1);
  const T *wg = p.w[0] + f * D, *wu = p.w[1] + f * D;
  const T *x[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t)
    x[t] = p.x + (int64_t)min(t * 16 + lane % 16, M - 1) * D;
  f32x4 acc[2][TB] = {};
  const int steps = (D + S - 1) / S;
  const int whole = D / S;  // steps that need no bounds
  for (int s = wave; s < steps; s += kFewWaves * kFewUnroll) {
    Vec g[kFewUnroll], u[kFewUnroll], v[kFewUnroll][TB];
#pragma unroll
    for (int i = 0; i < kFewUnroll; ++i) {
      const int k0 = (s + i * kFewWaves) * S + lane / 16 * E;
      const int k = min(k0, D - E);
      g[i] = load_vec(wg + k);
      u[i] = load_vec(wu + k);
#pragma unroll
      for (int t = 0; t < TB; ++t) v[i][t] = load_vec(x[t] + k);
      if (s + i * kFewWaves >= whole && k0 >= D) {
        g[i] = u[i] = vzero();
#pragma unroll
        for (int t = 0; t < TB; ++t) v[i][t] = vzero();
      }
    }
#pragma unroll
    for (int i = 0; i < kFewUnroll; ++i)
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        multiply_few<T>(acc[0][t], g[i], v[i][t]);
        multiply_few<T>(acc[1][t], u[i], v[i][t]);
      }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < TB; ++t) sums[wave][q][t][lane] = acc[q][t];
  __syncthreads();
  // lane l, register e: feature 4 (l / 16) + e, token l % 16
  for (int n = threadIdx.x; n < 256 * TB; n += 64 * kFewWaves) {
    const int ff = n % 16, m = n / 16;
    if (m >= M || f0 + ff >= F) continue;
    float gu[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      gu[q] = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w)
        gu[q] += sums[w][q][m / 16][ff / 4 * 16 + m % 16][ff % 4];
    }
    const int64_t at = (int64_t)m * F + f0 + ff;
    const int64_t plane_size = (int64_t)M * F;
    float a, da;
    activate<T, ACT>(gu[0], a, da);
    if constexpr (FORM == kHidden) {
      store_one(p.h + at, a * gu[1]);
      if (p.gu != nullptr) {
        p.gu[at] = gu[0];
        p.gu[plane_size + at] = gu[1];
      }
    } else {
      const float dh = load_one(p.dh + at);
      store_one(p.dgu + at, dh * gu[1] * da);
      store_one(p.dgu + plane_size + at, dh * a);
    }
  }
}

// The tiles of dx (`blocks_x` workgroups) and of dW that were computed in
// slices: the sum of these, in slice order (of folded rows, both in turn).
// Four elements per thread, in a tile of the workgroup's own, so that the
// tile's place is scalar arithmetic, and several loads in flight: over few
// tokens it is a chain of instructions with nothing beside it (MI355X, 12
// slices of 1 x 1536: 6.9 -> 4.0 us, of 64 x 1536 8.0 -> 4.9, against 8
// elements per thread of any tile).
constexpr int kSumElems = 4 * kBlock;  // of a workgroup

template <typename T>
__global__ __launch_bounds__(kBlock) void slices_kernel(Product<T> p, Tiles x,
                                                        Tiles w,
                                                        int32_t blocks_x) {
  constexpr int kBatch = 8;
  const bool is_w = (int)blockIdx.x >= blocks_x;
  const Tiles q = is_w ? w : x;
  const int id = blockIdx.x - (is_w ? blocks_x : 0);
  const int bits = q.tiling == kBig ? 8 : 7;  // of a tile's side
  const int tile = 1 << bits, size = tile << bits;
  const int t = id / (size / kSumElems);
  const int in = (id * kBlock + (int)threadIdx.x) * 4 - t * size;
  int plane, tr, tc;
  tile_of(q.full + t, q.tiles_r, q.tiles_c, plane, tr, tc);
  const int fold = is_w ? 0 : p.fold;
  const int rows = is_w ? p.F : fold > 0 ? fold : p.M;
  const int r = tr * tile + (in >> bits), c = tc * tile + (in & (tile - 1));
  if (r >= rows || c >= p.D) return;
  const float *src = q.part + (int64_t)t * size + in;
  const int64_t next = (int64_t)q.rem * size;
  float v[4] = {};
  auto add = [&](auto two) {
    const int terms = q.slices << two;
    for (int s = 0; s < terms; s += kBatch) {
      Vec a[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int n = min(s + i, terms - 1);
        a[i] = load_stream(src + (n >> two) * next + (n & two) * fold * tile);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] += s + i < terms ? elem<float>(a[i], e) : 0.f;
    }
  };
  if (fold > 0)
    add(std::integral_constant<int, 1>());
  else
    add(std::integral_constant<int, 0>());
  T *out = is_w ? p.dw[plane] : p.dx;
  store4(out + (int64_t)r * p.D + c, v);
}

__global__ __launch_bounds__(kBlock) void zero_kernel(char *a, char *b,
                                                      int64_t n) {
  for (int64_t at = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 16; at < n;
       at += (int64_t)gridDim.x * kBlock * 16) {
    store_vec(a + at, vzero());
    store_vec(b + at, vzero());
  }
}

// ----------------------------------------------------------------- planning

struct GluPlan : Tiles {
  int64_t blocks = 0;
  double us = 0;  // what the model below says
  size_t part_bytes() const {
    return (size_t)slices * rem * tile() * tile() * sizeof(float);
  }
};

// The sizes of one product.
struct Shape {
  int64_t rows, cols, planes, steps;
  int col_share;  // columns of a tile, of its side: 1, or 2 for half of it
  bool fold;      // all tiles go through the slices' sums, which add its rows
  Shape(int form, int dtype, int64_t M, int64_t D, int64_t F,
        bool fold = false)
      : fold(fold) {
    const int S = dtype == ADALN_F32 ? kStep<float> : kStep<bf16>;
    const bool pair = form == kHidden || form == kGrads;
    rows = form == kDw ? F : M;
    cols = pair ? F : D;
    planes = form == kDw ? 2 : 1;
    steps = pair ? (D + S - 1) / S
            : form == kDx ? 2 * ((F + S - 1) / S) : (M + S - 1) / S;
    col_share = pair ? 2 : 1;
  }
  int64_t tiles(int64_t tile) const {
    const int64_t side = tile / col_share;
    return (rows + tile - 1) / tile * ((cols + side - 1) / side) * planes;
  }
};

// A plan's time, in microseconds, is modelled from what a tile takes (bf16;
// of f32 a step has half the elements at a sixteenth of the rate): the big
// ones run one to a CU, 1.65 per step and 5 for filling the pipeline and
// storing; the small ones two to a CU, 1.0 and 4; the deep ones one to a CU,
// 0.55 and 4; the fine ones two to a CU, 0.5 and 3 (MI355X, D = 1536, F =
// 4096, forward, by fine, deep and small tiles: 128 tokens 12.3 us, 18.7, -;
// 256 tokens 15.8, 18.1, 20.5; 1024 tokens -, 31.6, 27.7; f32, 128 tokens 61.2
// and 99.9).  Adding slices up takes 4 and, per partial sum, 2 x 4 bytes at 5
// TB/s.
struct Costs {
  int64_t tile, slots;
  double step, fill;
  Costs(int tiling, int dtype) {
    tile = tiling == kBig ? 256 : tiling == kFine ? 64 : 128;
    slots = tiling == kSmall || tiling == kFine ? 2 * kCUs : kCUs;
    fill = tiling == kBig ? 5 : tiling == kFine ? 3 : 4;
    constexpr double kF32[] = {4.5, 9, 2.3, 1.2};
    constexpr double kBf16[] = {1.0, 1.65, 0.55, 0.5};
    step = dtype == ADALN_F32 ? kF32[tiling] : kBf16[tiling];
  }
  double adding(int64_t blocks) const {
    return 4 + 8e-6 / 5 * blocks * tile * tile;
  }
};

// Tiles of a shape, the last `rem` of them in s slices of `per` steps.
GluPlan cut(const Shape &h, int tiling, int64_t tile, int64_t rem, int64_t s,
            int64_t per) {
  GluPlan g;
  const int64_t r = (h.rows + tile - 1) / tile;
  const int64_t side = tile / h.col_share;
  const int64_t c = (h.cols + side - 1) / side;
  g.tiling = tiling;
  g.tiles_r = (int32_t)r;
  g.tiles_c = (int32_t)c;
  g.steps = (int32_t)h.steps;
  g.rem = (int32_t)(s > 1 || h.fold ? rem : 0);
  g.full = (int32_t)(h.tiles(tile) - g.rem);
  g.slices = (int32_t)s;
  g.per_slice = (int32_t)per;
  g.blocks = g.full + g.rem * s;
  return g;
}

// One product in a launch of its own.  Whole rounds of tiles (as many as run
// at a time) are computed unsplit; the tiles left over, less than a round,
// are split into slices of the sum where that pays: s slices take
// ceil(rem * s / slots) / s of a round.  Measured on MI355X for the weights'
// gradients of 24960 x 1536 x 4096 (192 big tiles, 4 slices) 654 -> 570 us,
// dx (588, the last 76 in 3 slices) 717 -> 589 us.
GluPlan glu_plan(int form, int dtype, int64_t M, int64_t D, int64_t F,
                 bool fold = false) {
  const Shape h(form, dtype, M, D, F, fold);
  const bool pair = form == kHidden || form == kGrads;
  GluPlan best;
  for (int tiling = 0; tiling <= (pair ? kFine : kDeep); ++tiling) {
    const Costs k(tiling, dtype);
    const int64_t n = h.tiles(k.tile);
    if (n > INT32_MAX) continue;  // (the finest only)
    const int64_t full = fold ? 0 : n / k.slots * k.slots, rem = n - full;
    for (int64_t s = 1; s <= 16; ++s) {
      if (s > 1 && (pair || rem == 0 || h.steps < 4 * s)) break;
      const int64_t per = (h.steps + s - 1) / s;
      if ((h.steps + per - 1) / per != s) continue;  // an empty slice
      double us = full / k.slots * (h.steps * k.step + k.fill);
      if (rem > 0)
        us += (rem * s + k.slots - 1) / k.slots * (per * k.step + k.fill);
      if (s > 1 || fold) us += k.adding(rem * s);
      if (best.blocks > 0 && us >= best.us) continue;
      best = cut(h, tiling, k.tile, rem, s, per);
      best.us = us;
    }
  }
  return best;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The backward's two products and its workspace: dG and dU, what a split call
// has besides, then the partial sums.
struct GluBackward {
  GluPlan x, w;
  bool joint = false;
  // dG, dU in two parts (split_grads_kernel).  Rounded to bf16 they add as
  // much to the error of dx and dW as these' own rounding does, 1.41 times it
  // together, and over few tokens, where it does not average out, up to 1.7.
  // Up to 64 tokens both parts' rows fit into one row of tiles and the
  // weights' bytes bound the products, so the parts cost little (MI355X, D =
  // 1536, F = 4096: 1 token 22.1 -> 23.1 us, 16 22.6 -> 24.2, 64 23.4 -> 28.5;
  // D = 5120, F = 13824: 1 token 161 -> 162, 64 165 -> 182; at most 2.5 us
  // where dx alone was one slice).  Past that they would double the work.
  bool split = false;
  size_t bytes = 0;
  size_t x2 = 0, gu = 0, h = 0;   // offsets: x twice; G, U computed again; h
  size_t x_part = 0, w_part = 0;
};
constexpr int64_t kSplitTokens = 64;

// When the last of n1 blocks of t1 and then n2 of t2 <= t1 ends, on `slots`
// that each take the next block when they are free.
double makespan(int64_t slots, int64_t n1, double t1, int64_t n2, double t2) {
  if (n1 + n2 <= slots) return n1 > 0 ? t1 : t2;
  const int64_t rounds = n1 / slots, late = n1 - rounds * slots;
  // `late` slots start on the second kind at s1, the others at s0
  const double s0 = rounds * t1, s1 = late > 0 ? s0 + t1 : s0;
  if (n2 == 0) return s1;
  auto done = [&](double t) {
    auto of = [&](double s) {
      return t >= s ? (int64_t)((t - s) / t2 + 1e-9) : 0;
    };
    return late * of(s1) + (slots - late) * of(s0) >= n2;
  };
  // it ends a whole number of blocks after s0 or s1, no sooner than the
  // average load
  const double average = (n1 * t1 + n2 * t2) / slots;
  double best = 0;
  for (double s : {s0, s1}) {
    double t = s + std::max<double>(1, (int64_t)((average - s) / t2)) * t2;
    while (!done(t)) t += t2;
    if (best == 0 || t < best) best = t;
  }
  return std::max(best, s1);
}

// In one launch where the model finds that shorter: all tiles of both
// products, in slices or not, taken by free CUs in turn, the longer ones
// first.  Two launches cost 3 more.  Measured on MI355X, whole backward, two
// launches against one: 777 x 1000 x 1480 40.5 -> 33.6 us, 4096 x 256 x 1024
// 47.5 -> 37.4, 64 x 512 x 1024 24.4 -> 21.5; big tiles, which fill the
// rounds that the other product leaves open: 8190 x 1536 x 4096 536 -> 424,
// 12000 x 1000 x 3000 444 -> 351, 24960 x 1536 x 4096 1341 -> 1313.  (Where
// it is wrong it costs less: 3000 x 640 x 5000 142 -> 157.)
GluBackward glu_backward(int dtype, int64_t M, int64_t D, int64_t F) {
  GluBackward b;
  b.split = dtype == ADALN_BF16 && M <= kSplitTokens;
  const int64_t rows = b.split ? 2 * M : M;
  b.x = glu_plan(kDx, dtype, rows, D, F, b.split);
  b.w = glu_plan(kDw, dtype, rows, D, F);
  const Shape hx(kDx, dtype, rows, D, F, b.split);
  const Shape hw(kDw, dtype, rows, D, F);
  double best = b.x.us + b.w.us + 3;
  for (int tiling : {(int)kSmall, (int)kBig, (int)kDeep}) {
    // (f32's small tiles are as fast as its big ones and end more evenly)
    if (tiling == kBig && dtype == ADALN_F32) continue;
    const Costs k(tiling, dtype);
    const int64_t nx = hx.tiles(k.tile), nw = hw.tiles(k.tile);
    // (many tiles: the slices' sums would cost more than they even out)
    const int64_t most = nx + nw > 4 * k.slots ? 1 : 16;
    for (int64_t sx : {1, 2, 3, 4, 6, 8, 12, 16}) {
      const int64_t px = (hx.steps + sx - 1) / sx;
      if (sx > most) break;
      if (sx > 1 && (hx.steps < 4 * sx || (hx.steps + px - 1) / px != sx))
        continue;
      for (int64_t sw : {1, 2, 3, 4, 6, 8, 12, 16}) {
        const int64_t pw = (hw.steps + sw - 1) / sw;
        if (sw > most) break;
        if (sw > 1 && (hw.steps < 4 * sw || (hw.steps + pw - 1) / pw != sw))
          continue;
        const double tx = px * k.step + k.fill, tw = pw * k.step + k.fill;
        if (nx * sx + nw * sw > kMaxGrid ||
            (nx * sx * tx + nw * sw * tw) / k.slots >= best)
          continue;
        double us = tw > tx ? makespan(k.slots, nw * sw, tw, nx * sx, tx)
                            : makespan(k.slots, nx * sx, tx, nw * sw, tw);
        const bool add_x = sx > 1 || b.split;
        if (add_x || sw > 1)
          us += k.adding((add_x ? nx * sx : 0) + (sw > 1 ? nw * sw : 0));
        if (us >= best) continue;
        best = us;
        b.joint = true;
        b.x = cut(hx, tiling, k.tile, nx, sx, px);
        b.w = cut(hw, tiling, k.tile, nw, sw, pw);
      }
    }
  }
  b.x2 = align256((size_t)2 * rows * F * (dtype == ADALN_F32 ? 4 : 2));
  b.gu = b.x2 + (b.split ? align256((size_t)rows * D * 2) : 0);
  b.h = b.gu + (b.split ? align256((size_t)2 * M * F * 4) : 0);
  b.x_part = b.w_part = b.h + (b.split ? align256((size_t)M * F * 2) : 0);
  if (b.joint) b.w_part += align256(b.x.part_bytes());
  b.bytes = std::max(b.x_part + b.x.part_bytes(), b.w_part + b.w.part_bytes());
  return b;
}

// Few tokens: few_kernel.  Past 4 tokens only where deep tiles, of 64 hidden
// features, leave half the CUs idle.  Elsewhere the tiles stream the weights
// as fast and its repeated reads of the tokens cost more (MI355X, D = 5120, F =
// 13824: 1 token 61 us, 16 tokens 80, 64 tokens 137, against 43-52).  Past 48
// tokens of bf16 the fine tiles are faster once they fill half the CUs (D =
// 1536, F = 4096: 1 token 7.4 us, 32 tokens 10.6, 48 13.5, 64 15.3, against
// 12.3 for 17-64; D = F = 2048: 64 tokens 13.7 against 14.8; f32, D = 1536, F =
// 4096: 64 tokens 35 against 61).
bool few_tokens(int dtype, int64_t M, int64_t F) {
  const int64_t tiles = (F + 63) / 64;
  if (M <= 4) return true;
  return tiles < kCUs / 2 &&
         M <= (dtype == ADALN_F32 || tiles < kCUs / 4 ? 64 : 48);
}

template <typename T>
constexpr int kDtype = sizeof(T) == 2 ? ADALN_BF16 : ADALN_F32;

template <typename T, int FORM, int ACT>
hipError_t launch_few(Product<T> p, hipStream_t s) {
  const int64_t blocks = (p.F + 15) / 16;  // at most 16384
  const int threads = 64 * kFewWaves;
  return p.M <= 16 ? launch_kernel_threads(few_kernel<T, FORM, 1, ACT>, blocks,
                                           threads, s, p)
         : p.M <= 32 ? launch_kernel_threads(few_kernel<T, FORM, 2, ACT>,
                                             blocks, threads, s, p)
                     : launch_kernel_threads(few_kernel<T, FORM, 4, ACT>,
                                             blocks, threads, s, p);
}

template <typename T, int FORM, int ACT>
hipError_t launch_tiles(const Product<T> &p, const GluPlan &g,
                        hipStream_t s) {
  Tiles q = g;
  hipError_t e = hipSuccess;
  for (int64_t at = 0; at < g.blocks && e == hipSuccess; at += kMaxGrid) {
    q.block0 = (int32_t)at;
    const int64_t n = std::min<int64_t>(kMaxGrid, g.blocks - at);
    auto go = [&](auto kernel) {
      return launch_kernel_threads(kernel, n, tiling_threads(g.tiling), s, p,
                                   q);
    };
    if constexpr (FORM == kHidden || FORM == kGrads) {
      if (g.tiling == kFine) e = go(product_kernel<T, FORM, kFine, ACT>);
    }
    if (g.tiling == kSmall) e = go(product_kernel<T, FORM, kSmall, ACT>);
    if (g.tiling == kBig) e = go(product_kernel<T, FORM, kBig, ACT>);
    if (g.tiling == kDeep) e = go(product_kernel<T, FORM, kDeep, ACT>);
  }
  return e;
}

// kHidden or kGrads.
template <typename T, int FORM, int ACT>
hipError_t launch_pair(const Product<T> &p, hipStream_t s) {
  // (few tokens' gradients in bf16 come from split_grads_kernel)
  if constexpr (FORM == kHidden || kDtype<T> == ADALN_F32)
    if (few_tokens(kDtype<T>, p.M, p.F)) return launch_few<T, FORM, ACT>(p, s);
  return launch_tiles<T, FORM, ACT>(
      p, glu_plan(FORM, kDtype<T>, p.M, p.D, p.F), s);
}

template <typename T>
hipError_t launch_slices(const Product<T> &p, const Tiles &x, const Tiles &w,
                         hipStream_t s) {
  // (at most 4 * 512 tiles are cut in slices: below 2^17 workgroups)
  auto blocks = [](const Tiles &q) {
    return q.rem * (q.tile() * q.tile() / kSumElems);
  };
  return launch_kernel(slices_kernel<T>, (int64_t)blocks(x) + blocks(w), s, p,
                       x, w, (int32_t)blocks(x));
}

template <typename T>
hipError_t launch_grads(const Product<T> &p, const GluBackward &b, char *ws,
                        hipStream_t s) {
  GluPlan x = b.x, w = b.w;
  x.part = (float *)(ws + b.x_part);
  w.part = (float *)(ws + b.w_part);
  hipError_t e = hipSuccess;
  if (b.joint) {
    const bool w_first = w.per_slice > x.per_slice;
    const int32_t first = (int32_t)(w_first ? w.blocks : x.blocks);
    const int64_t n = x.blocks + w.blocks;
    auto go = [&](auto kernel) {
      return launch_kernel_threads(kernel, n, tiling_threads(x.tiling), s, p,
                                   (Tiles)x, (Tiles)w, first,
                                   (int32_t)w_first);
    };
    if constexpr (kDtype<T> == ADALN_BF16) {
      if (x.tiling == kBig) e = go(grads_kernel<T, kBig>);
    }
    if (x.tiling == kSmall) e = go(grads_kernel<T, kSmall>);
    if (x.tiling == kDeep) e = go(grads_kernel<T, kDeep>);
    if (e != hipSuccess) return e;
    return launch_slices<T>(p, x, w, s);
  }
  Tiles none;
  e = launch_tiles<T, kDx, 0>(p, x, s);
  if (e == hipSuccess) e = launch_slices<T>(p, x, none, s);
  if (e == hipSuccess) e = launch_tiles<T, kDw, 0>(p, w, s);
  if (e == hipSuccess) e = launch_slices<T>(p, none, w, s);
  return e;
}

int hip_fail(hipError_t e, const char *what) {
  return fail(ADALN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

int check_glu(int64_t M, int64_t D, int64_t F, int act, int dtype) {
  if (dtype != ADALN_F32 && dtype != ADALN_BF16)
    return fail(ADALN_ERR_DTYPE, "unknown dtype code %d", dtype);
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

template <typename T>
Product<T> product_of(const void *x, const void *wg, const void *wu, int64_t M,
                      int64_t D, int64_t F) {
  Product<T> p = {};
  p.x = (const T *)x;
  p.w[0] = (const T *)wg;
  p.w[1] = (const T *)wu;
  p.M = (int32_t)M;
  p.D = (int32_t)D;
  p.F = (int32_t)F;
  return p;
}

template <typename T>
hipError_t run_fwd(const void *x, const void *wg, const void *wu, void *h,
                   float *saved, int64_t M, int64_t D, int64_t F, int act,
                   hipStream_t s) {
  Product<T> p = product_of<T>(x, wg, wu, M, D, F);
  p.h = (T *)h;
  p.gu = saved;
  return act == ADALN_ACT_SILU ? launch_pair<T, kHidden, kSilu>(p, s)
                               : launch_pair<T, kHidden, kGeluTanh>(p, s);
}

template <typename T, int ACT>
hipError_t launch_gate_grads(const Product<T> &p, hipStream_t s) {
  if (p.gu == nullptr) return launch_pair<T, kGrads, ACT>(p, s);
  const int64_t n = (int64_t)p.M * p.F;
  return launch_kernel(gate_grads_kernel<T, ACT>,
                       (n / 8 + kBlock - 1) / kBlock, s, (const float *)p.gu,
                       p.dh, p.dgu, n);
}

// Of a split call: G, U computed again if they were not saved (the h that
// comes with them is not used), then the parts.  The products are then those
// of 2 M tokens.
template <int ACT>
hipError_t launch_split_grads(Product<bf16> &p, const GluBackward &b, char *ws,
                              hipStream_t s) {
  if (p.gu == nullptr) {
    p.gu = (float *)(ws + b.gu);
    p.h = (bf16 *)(ws + b.h);
    const hipError_t e = launch_pair<bf16, kHidden, ACT>(p, s);
    if (e != hipSuccess) return e;
  }
  bf16 *x2 = (bf16 *)(ws + b.x2);
  const int64_t n = (int64_t)p.M * p.F, n_x = (int64_t)p.M * p.D;
  const hipError_t e = launch_kernel(
      split_grads_kernel<ACT>, ((n + n_x) / 8 + kBlock - 1) / kBlock, s,
      (const float *)p.gu, p.dh, p.x, p.dgu, x2, n, n_x);
  p.x = x2;
  p.fold = p.M;
  p.M *= 2;
  return e;
}

template <typename T>
hipError_t run_bwd(const void *dh, const void *x, const void *wg,
                   const void *wu, const float *saved, void *dx, void *dwg,
                   void *dwu, void *workspace, const GluBackward &b,
                   int64_t M, int64_t D, int64_t F, int act, hipStream_t s) {
  Product<T> p = product_of<T>(x, wg, wu, M, D, F);
  p.gu = const_cast<float *>(saved);
  p.dh = (const T *)dh;
  p.dgu = (T *)workspace;
  p.dx = (T *)dx;
  p.dw[0] = (T *)dwg;
  p.dw[1] = (T *)dwu;
  const bool silu = act == ADALN_ACT_SILU;
  hipError_t e = hipSuccess;
  if constexpr (kDtype<T> == ADALN_BF16) {
    if (b.split)
      e = silu ? launch_split_grads<kSilu>(p, b, (char *)workspace, s)
               : launch_split_grads<kGeluTanh>(p, b, (char *)workspace, s);
  }
  if (!b.split)
    e = silu ? launch_gate_grads<T, kSilu>(p, s)
             : launch_gate_grads<T, kGeluTanh>(p, s);
  if (e != hipSuccess) return e;
  return launch_grads<T>(p, b, (char *)workspace, s);
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
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      dtype == ADALN_BF16
          ? run_fwd<bf16>(x, wg, wu, h, saved, M, D, F, act, s)
          : run_fwd<float>(x, wg, wu, h, saved, M, D, F, act, s);
  if (e != hipSuccess) return hip_fail(e, "adaln_glu_fwd launch");
  return ok();
}

ADALN_API size_t adaln_glu_bwd_workspace_bytes(int64_t M, int64_t D, int64_t F,
                                               int dtype) {
  if (check_glu(M, D, F, ADALN_ACT_SILU, dtype) != ADALN_OK || M == 0) return 0;
  return glu_backward(dtype, M, D, F).bytes;
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
    // no tokens: the weights' gradients are empty sums
    const int64_t bytes = F * D * (dtype == ADALN_BF16 ? 2 : 4);
    const hipError_t e =
        launch_kernel(zero_kernel, (bytes / 16 + kBlock - 1) / kBlock, s,
                      (char *)dwg, (char *)dwu, bytes);
    if (e != hipSuccess) return hip_fail(e, "adaln_glu_bwd launch");
    return ok();
  }
  const GluBackward b = glu_backward(dtype, M, D, F);
  const size_t need = b.bytes;
  if (workspace == nullptr || workspace_bytes < need)
    return fail(ADALN_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu%s",
                need, workspace_bytes, workspace == nullptr ? " (NULL)" : "");
  ADALN_TRY(check_ptr(workspace, true, "workspace"));
  const hipError_t e =
      dtype == ADALN_BF16
          ? run_bwd<bf16>(dh, x, wg, wu, saved, dx, dwg, dwu, workspace, b, M,
                          D, F, act, s)
          : run_bwd<float>(dh, x, wg, wu, saved, dx, dwg, dwu, workspace, b,
                           M, D, F, act, s);
  if (e != hipSuccess) return hip_fail(e, "adaln_glu_bwd launch");
  return ok();
}
