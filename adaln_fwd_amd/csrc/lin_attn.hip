// Linear attention with a decay for each head, forward, backward and one token
// at a time, with their C entry points.
//
//     S_t = l S_{t-1} + k_t v_t^T      o_t = c S_t^T q_t      l = exp(log_decay)
//
// In chunks of 32 tokens, t and s counted from the chunk's first, S the state
// before it and n its tokens:
//
//     o_t = c l^(t+1) S^T q_t + sum_{s <= t} c l^(t-s) (q_t . k_s) v_s
//     S'  = l^n S + sum_s k_s (l^(n-1-s) v_s)^T
//
// The powers of l are never negative ones, so no decay, however strong,
// overflows.  The gradients are the same operator with its parts exchanged,
// dq = lin(do, v, k) with S^T, and, from the last token to the first, with G
// the gradient of the state:
//
//     dv = lin(k, q, do) with G        dk = lin(v, do, q) with G^T
//     G_{t-1} = l (G_t + c q_t do_t^T)
//
// A workgroup walks a stretch of tokens of one head, d / 32 wavefronts with 32
// columns of the state each, which stay in the accumulators of the matrix
// cores.  Their layout is the point of the design: a lane of an accumulator
// holds, of one column, the rows (r / 4) * 8 + 4 * (lane / 32) + r % 4, and if
// the summed dimension of a product is numbered in this order in both
// operands, an accumulator's registers are an operand as they stand.  So
// the scores q k^T, computed with k as the rows, and the state go into the
// next product without crossing lanes.  Sequences are split into stretches to
// fill the GPU: one pass computes what each adds to the state, a second one
// adds these up along the sequence, the third walks the stretches from there.
#include <algorithm>
#include <math.h>

#include "adaln.h"
#include "checks.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace adaln {
namespace {

constexpr int kMaxHead = 128;
constexpr int kChunk = 32;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Eight elements of a row or column: those numbered slot(i) of 16 summed ones.
template <typename T>
struct Frag;
template <>
struct Frag<bf16> {
  bf16x8 v;
};
template <>
struct Frag<float> {
  f32x8 v;
};

__device__ __forceinline__ int half_of() { return lane_id() / 32; }
__device__ __forceinline__ int slot(int i) {
  return (i / 4) * 8 + 4 * half_of() + i % 4;
}

// acc[row of a][row of b] += a b^T over 16 summed elements.
__device__ __forceinline__ void mma(f32x16 &acc, const Frag<bf16> &a,
                                    const Frag<bf16> &b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16 &acc, const Frag<float> &a,
                                    const Frag<float> &b) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[i], b.v[i], acc, 0, 0, 0);
}

// Eight float32 as a fragment.
__device__ __forceinline__ void to_frag(Frag<bf16> &f, const float (&x)[8]) {
  const Vec v = pack<bf16>(x);
  f.v = __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ void to_frag(Frag<float> &f, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f.v[i] = x[i];
}
__device__ __forceinline__ void from_frag(float (&x)[8], const Frag<bf16> &f) {
  const Vec v = __builtin_bit_cast(Vec, f.v);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = elem<bf16>(v, i);
}
__device__ __forceinline__ void from_frag(float (&x)[8],
                                          const Frag<float> &f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = f.v[i];
}

// Float32 numbers as fragments: of bf16 the sum of PARTS, each the rounded rest
// of those before it, so that what the matrix cores are given is within
// 2^(-8 PARTS) of the number (three: as good as itself).  The rest of a pair is
// x - 1 * hi - 0 * other, a dot product of the two packed numbers with (1, 0),
// exact, in one instruction where unpacking and subtracting takes two.  (Its
// constants stay in registers: as an inline constant of the instruction, (-1,
// 0) was read as something else.)
template <typename T, int PARTS>
struct Parts {
  static constexpr int kParts = sizeof(T) == 2 ? PARTS : 1;
  Frag<T> f[kParts];

  __device__ __forceinline__ void set(float (&x)[8]) {
#pragma unroll
    for (int a = 0; a < kParts; ++a) {
      to_frag(f[a], x);
      if constexpr (sizeof(T) == 2) {
        if (a + 1 == kParts) break;
        uint32_t first = 0x0000bf80u, second = 0xbf800000u;
        asm("" : "+s"(first), "+s"(second));
        const Vec v = __builtin_bit_cast(Vec, f[a].v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x2 hi = __builtin_bit_cast(bf16x2, v.w[i]);
          x[2 * i] = __builtin_amdgcn_fdot2_f32_bf16(
              hi, __builtin_bit_cast(bf16x2, first), x[2 * i], false);
          x[2 * i + 1] = __builtin_amdgcn_fdot2_f32_bf16(
              hi, __builtin_bit_cast(bf16x2, second), x[2 * i + 1], false);
        }
      }
    }
  }
};

template <typename T, int PARTS>
__device__ __forceinline__ void mma(f32x16 &acc, const Parts<T, PARTS> &a,
                                    const Frag<T> &b) {
#pragma unroll
  for (int i = 0; i < Parts<T, PARTS>::kParts; ++i) mma(acc, a.f[i], b);
}
template <typename T, int PARTS>
__device__ __forceinline__ void mma(f32x16 &acc, const Frag<T> &a,
                                    const Parts<T, PARTS> &b) {
#pragma unroll
  for (int i = 0; i < Parts<T, PARTS>::kParts; ++i) mma(acc, a, b.f[i]);
}

// ----------------------------------------------------------- tiles in LDS

typedef __attribute__((address_space(3))) char lds_char;

// LDS by its 32-bit addresses.
template <typename V>
__device__ __forceinline__ V lds_read(uint32_t at) {
  return *(__attribute__((address_space(3))) const V *)(lds_char *)at;
}
template <typename V>
__device__ __forceinline__ void lds_write(uint32_t at, const V &v) {
  *(__attribute__((address_space(3))) V *)(lds_char *)at = v;
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(lds_char *)p;
}

// 16 bytes per lane from memory to LDS at `lds` + 16 * lane: a wave-uniform
// base and a 32-bit offset per lane.  The compiler does not see these loads:
// arrive() waits for them.  (m0 takes the LDS address; the s_nop is the wait
// state that the ISA asks for between writing m0 and a load to LDS.)
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

// All of this wavefront's accesses to memory but the last LATER have landed, then
// those of every wavefront.  LATER is the least number of loads that any wavefront
// has begun behind those awaited, and counts no stores: loads return in order, so
// with at most LATER accesses of any kind left, none of the awaited ones is among
// them.  (Stores begun meanwhile only make it wait for more.)
template <int LATER>
__device__ __forceinline__ void arrive() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATER)
               : "memory");
}

// The 32 tokens of a chunk of one tensor, a row of kPieces pieces of 16 bytes
// each.  Piece c of token r stands at c ^ turn(r), which spreads the rows that a
// read takes together over the banks: 16 rows of 8 bytes, four rows of 32 (a
// transposing read), or of f32 8 rows of 16 bytes, two of 128.  (Not all the way:
// 8-byte accesses take 32 rows, and in tiles of four pieces, those of scores, of
// a wavefront's own columns and of outputs, rows 16 apart share their banks.  36%
// of the LDS's active cycles are conflicts in out_kernel, none in state_kernel,
// which has no such tile.)  The loads apply the turn to the addresses that they
// read from.  A turn's bits are the pieces' own, so a lane's place for block b or
// columns 32 m is that for the first by an exclusive or.
template <typename T, int DP>
struct Tile {
  static constexpr bool kHalf = sizeof(T) == 2;
  static constexpr int E = Elems<T>::value;
  static constexpr int kRowVecs = DP / E;
  static constexpr int kPieces = kHalf ? (DP <= 32   ? 4
                                          : DP <= 64 ? 8
                                                     : 16)
                                       : (DP <= 64 ? 16 : 32);
  static constexpr int kPitch = kPieces * 16;
  static constexpr int kBytes = kChunk * kPitch;
  static constexpr int kCols = kHalf ? 2 : 4;  // places of a column read

  static __device__ __forceinline__ int turn(int r) {
    if (!kHalf) return ((r >> 2 & 1) << 3) | (r & 3);
    if (kPieces == 16) return ((r & 3) << 2) | (r >> 2 & 3);
    if (kPieces == 8) return ((r >> 1 & 1) << 2) | (r >> 2 & 3);
    return r >> 2 & 3;
  }
  // The lane's place in rows(), relative to the tile.
  static __device__ __forceinline__ uint32_t row_place() {
    const int r = lane_id() % 32, h = half_of();
    return kHalf ? r * kPitch + turn(r) * 16 + h * 8
                 : r * kPitch + (turn(r) ^ h) * 16;
  }
  // Token lane % 32, features 16 b + slot(i); at: the tile's address in LDS
  // plus the lane's place.
  static __device__ __forceinline__ Frag<T> rows(uint32_t at, int b) {
    Frag<T> f;
    if constexpr (kHalf) {
      const s16x4 x = lds_read<s16x4>(at ^ (32 * b));
      const s16x4 y = lds_read<s16x4>(at ^ (32 * b) ^ 16);
      const s16x8 v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
      f.v = __builtin_bit_cast(bf16x8, v);
    } else {
      const f32x4 x = lds_read<f32x4>(at ^ (64 * b));
      const f32x4 y = lds_read<f32x4>(at ^ (64 * b) ^ 32);
      f.v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return f;
  }
  // The same in the order of a state's rows: bf16, eight features
  // side by side, one read.
  static __device__ __forceinline__ uint32_t pair_place() {
    const int r = lane_id() % 32, h = half_of();
    return kHalf ? r * kPitch + (turn(r) ^ h) * 16 : row_place();
  }
  static __device__ __forceinline__ Frag<T> pairs(uint32_t at, int b) {
    if constexpr (kHalf) {
      Frag<T> f;
      f.v = __builtin_bit_cast(bf16x8, lds_read<u32x4>(at ^ (32 * b)));
      return f;
    } else {
      return rows(at, b);
    }
  }
  // The lane's places in cols(); STATE: of features in the order of a state's
  // rows.
  template <bool STATE>
  static __device__ __forceinline__ void col_places(uint32_t (&place)[kCols]) {
    const int l = lane_id(), h = half_of();
#pragma unroll
    for (int x = 0; x < kCols; ++x) {
      if (kHalf) {
        // 16 lanes read four tokens of 16 features, and get a feature's four
        // tokens each
        const int r = 8 * x + 4 * h + (l % 16) / 4;
        // (the lanes' units of four features: 0, 1, 2, 3, or 0, 2, 1, 3)
        const int c = (l >> 4 & 1) * 2 + (STATE ? l & 1 : l >> 1 & 1);
        place[x] = r * kPitch + (c ^ turn(r)) * 16 +
                   (STATE ? l >> 1 & 1 : l & 1) * 8;
      } else {
        const int r = 4 * h + x;
        place[x] = r * kPitch + ((l % 32 / 4) ^ turn(r)) * 16 + l % 4 * 4;
      }
    }
  }
  // Feature 32 m + lane % 32, tokens 16 j + slot(i).
  static __device__ __forceinline__ Frag<T> cols(const uint32_t (&at)[kCols],
                                                 int j, int m) {
    Frag<T> f;
    if constexpr (kHalf) {
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4 *)(lds_char *)((at[0] ^ (64 * m)) + 16 * j * kPitch));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4 *)(lds_char *)((at[1] ^ (64 * m)) + 16 * j * kPitch));
      const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      f.v = __builtin_bit_cast(bf16x8, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f.v[i] = lds_read<float>((at[i % 4] ^ (128 * m)) +
                                 (16 * j + 8 * (i / 4)) * kPitch);
    }
    return f;
  }
  // 16 rows of a score block: lane l has row l % 16, pieces 4 b + l / 16.
  static __device__ __forceinline__ uint32_t score_place(int r0) {
    const int r = r0 + lane_id() % 16;
    return r * kPitch + ((lane_id() / 16) ^ turn(r)) * 16;
  }
};

// ------------------------------------------------------------------ the work

// One tensor of heads, distances in vectors of 16 bytes.
struct Part {
  const char *data;
  int64_t batch, token;
  int32_t head;
};

// Stretches of up to `len` tokens: B sequences of N tokens, `splits` each, or
// the segments of a table (a segment without tokens has one stretch too, which
// hands its state on).
struct Stretches {
  int32_t nseg;    // 0: sequences of N tokens
  int32_t splits;
  int64_t N, len;
  int32_t first[kMaxSegments + 1];  // stretches before a segment
  int64_t row[kMaxSegments + 1];    // tokens before it
};

struct Stretch {
  int seq;        // which state
  int64_t batch;  // which sample of the tensors
  int64_t start;  // first token
  int n;          // tokens
  bool head, tail;  // the sequence's first, last stretch
};

__device__ __forceinline__ Stretch find_stretch(const Stretches &m, int id) {
  Stretch s;
  if (m.nseg == 0) {
    s.seq = id / m.splits;
    const int j = id - s.seq * m.splits;
    s.batch = s.seq;
    s.start = j * m.len;
    s.n = (int)min(m.len, m.N - s.start);
    s.head = j == 0;
    s.tail = j == m.splits - 1;
    return s;
  }
  int lo = 0, hi = m.nseg - 1;  // last segment with first[] <= id
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (m.first[mid] <= id)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int j = id - m.first[lo];
  s.seq = lo;
  s.batch = 0;
  s.start = m.row[lo] + j * m.len;
  s.n = (int)min(m.len, m.row[lo + 1] - s.start);
  s.head = j == 0;
  s.tail = id == m.first[lo + 1] - 1;
  return s;
}

struct Lin {
  Part in[4];
  Part out[2];
  const float *log_decay;
  const float *init;     // [sequences, H, d, d]: the state before, or NULL
  float *states;         // [stretches, H, d, d], or NULL: one to a sequence
  float *final;          // [sequences, H, d, d]: the state behind, or NULL
  float scale;
  int32_t H, d;
  int32_t nvec;          // vectors of a head
  int64_t first;         // workgroups in the launches before
  int64_t jobs;          // stretches * H
};

// log2 of the decay; so strong that 0 tokens leave 1 and one leaves 0.
__device__ __forceinline__ float decay_of(const Lin &p, int h) {
  const float g = p.log_decay[h] * 1.44269504088896341f;
  return g < -1e30f ? -1e30f : g;
}

// The same number, but new to the compiler: what a loop computes from it is
// computed where it is used, an instruction or two, and not kept in registers
// throughout, where it would push others out (its scratch loads would then wait
// behind the loads in flight).
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Pieces that no load fills hold zeros: features past the head's, and tokens
// past the end.
__device__ __forceinline__ void clear(uint32_t lds, int from, int to, int id,
                                      int threads) {
  for (int x = from + id; x < to; x += threads)
    lds_write(lds + x * 16, u32x4{0, 0, 0, 0});
}

// A tile's chunks on their way to LDS, a set of tiles for each that is there or
// under way: the loads of TEAM threads (`id` of them), pieces x = id, id +
// TEAM, ... of each chunk.
template <typename Tl, int TEAM>
struct Loader {
  static constexpr int kAll = kChunk * Tl::kPieces;
  static constexpr int kPer = (kAll + TEAM - 1) / TEAM;
  // loads that every wavefront has of a whole chunk, at least
  static constexpr int kLoads = kAll / TEAM;
  const char *next;  // the next chunk's first token
  int64_t step;      // from chunk to chunk, bytes
  uint32_t off[kPer];
  bool ok[kPer];

  // j0: the tile's first vector of nvec; tokens from `start`, chunk by chunk,
  // forwards or backwards
  __device__ __forceinline__ void init(const Part &in, int64_t start, int dir,
                                       int j0, int nvec, int id) {
    next = in.data + start * in.token * 16;
    step = dir * in.token * (kChunk * 16);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int x = id + i * TEAM;
      const int r = x / Tl::kPieces;
      const int c = (x % Tl::kPieces) ^ Tl::turn(r);
      off[i] = ((uint32_t)r * (uint32_t)in.token + j0 + c) * 16;
      ok[i] = x < kAll && c < Tl::kRowVecs && j0 + c < nvec;
    }
  }
  // A chunk into the tile at `lds`, which nobody reads any more; wave: the
  // wavefront's first id.  all(): every token and every piece.
  __device__ __forceinline__ void all(uint32_t lds, uint32_t wave) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (kAll % TEAM == 0 || (int)wave + i * TEAM < kAll)
        dma(lds + (wave + i * TEAM) * 16, next, off[i]);
    next += step;
  }
  __device__ __forceinline__ void some(uint32_t lds, uint32_t wave, int n,
                                       int id) {
    if (n < kChunk) clear(lds, n * Tl::kPieces, kAll, id, TEAM);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (ok[i] && (id + i * TEAM) / Tl::kPieces < n)
        dma(lds + (wave + i * TEAM) * 16, next, off[i]);
    next += step;
  }
};

// A state's rows stand in the order in which they are summed, in bf16: of 16
// rows, 0 to 3, 8 to 11, 4 to 7 and 12 to 15, which gives a lane's eight summed
// elements, slot(i), eight features side by side.

// A wavefront's 32 columns of a state, rows by blocks of 32.
template <typename T, int DP>
struct State {
  f32x16 s[DP / 32];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < DP / 32; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[m][r] = 0.f;
  }
  // [d, d] in memory; `across`: its transpose.  Register 4 y + i of
  // 8 in the lanes of half h is row kY y + kH h + i of 16.
  static constexpr int kH = sizeof(T) == 2 ? 8 : 4;
  static constexpr int kY = 12 - kH;

  // The lane's first element, column c's in the half's first row.  It stands in
  // for what is outside the state, so it is inside also where that row is not
  // (d = kH).
  static __host__ __device__ __forceinline__ int first_at(int d, int c,
                                                          int half,
                                                          bool across) {
    const int col = c < d ? c : d - 1;
    const int row = kH * half < d ? kH * half : 0;
    return across ? col * d + row : row * d + col;
  }
  static __host__ __device__ __forceinline__ bool inside(int d, int c,
                                                         int half, int row) {
    return row + kH * half < d && c < d;  // d is a multiple of four
  }

  __device__ __forceinline__ void load(const float *src, int d, int c0,
                                       bool across) {
    const int c = c0 + lane_id() % 32, h = half_of();
    const float *lane = src + first_at(d, c, h, across);
#pragma unroll
    for (int m = 0; m < DP / 32; ++m)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int row = 32 * m + 16 * (r / 8) + kY * (r / 4 % 2);
        const bool in = inside(d, c, h, row);
        float x[4];
        if (across) {
          const float4 v =
              *reinterpret_cast<const float4 *>(lane + (in ? row : 0));
          x[0] = v.x;
          x[1] = v.y;
          x[2] = v.z;
          x[3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = lane[in ? (row + i) * d : 0];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[m][r + i] = in ? x[i] : 0.f;
      }
  }
  __device__ __forceinline__ void store(float *dst, int d, int c0) const {
    const int c = c0 + lane_id() % 32, r0 = kH * half_of();
    float *lane = dst + (int64_t)r0 * d + c;
#pragma unroll
    for (int m = 0; m < DP / 32; ++m)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int row = 32 * m + 16 * (r / 8) + kY * (r / 4 % 2);
        if (row + r0 < d && c < d)
#pragma unroll
          for (int i = 0; i < 4; ++i) lane[(row + i) * d] = s[m][r + i];
      }
  }
};

// The powers of the decay on the way of a chunk's tokens into the state:
// token 16 j + slot(i), of n.  (REV, from the last token to the first: the
// state is a gradient's, with c in it.)
template <bool REV>
struct Powers {
  float add[16];
  float own;   // of the state, for the lane's token
  float over;  // of the state over the chunk
  int n = 0;

  // (only a sequence's last chunk has less than 32: one of the two ends)
  __device__ __forceinline__ void set(float g, float c, int tokens) {
    if (n == tokens) return;
    n = tokens;
    const int t = lane_id() % 32;
    own = REV ? exp2f(g * max(n - 1 - t, 0)) : c * exp2f(g * (t + 1));
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const int s = 16 * (x / 8) + slot(x % 8);
      add[x] = REV ? c * exp2f(g * (s + 1)) : exp2f(g * max(n - 1 - s, 0));
    }
    over = exp2f(g * n);
  }
};

// v on its way into the state, add w v: as three bf16, which a state in float32
// is worth.  (Two, for a state that only outputs in bf16 are made from, are off
// by up to 2^-17, which shows where later products cancel earlier ones; 32760
// tokens of 24 heads of 128 take 293 us then, with three 311, backward 657 and
// 709.)
template <typename T, bool REV>
__device__ __forceinline__ void decayed(Parts<T, 3> (&x)[2],
                                        const Frag<T> (&v)[2],
                                        const Powers<REV> &pw, float w) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float y[8];
    from_frag(y, v[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= pw.add[8 * j + i] * w;
    x[j].set(y);
  }
}

// The chunk's k by columns, as both uses of a state's update want it.
template <typename T, int DP>
struct KeyCols {
  Frag<T> f[DP / 32][2];
  __device__ __forceinline__ void read(
      const uint32_t (&k_at)[Tile<T, DP>::kCols], int m) {
#pragma unroll
    for (int j = 0; j < 2; ++j) f[m][j] = Tile<T, DP>::cols(k_at, j, m);
  }
};

// S = over S + sum over the chunk's tokens of k x^T.
template <typename T, int DP>
__device__ __forceinline__ void gather(State<T, DP> &S,
                                       const KeyCols<T, DP> &k, int m,
                                       const Parts<T, 3> (&x)[2], float over) {
#pragma unroll
  for (int r = 0; r < 16; ++r) S.s[m][r] *= over;
#pragma unroll
  for (int j = 0; j < 2; ++j) mma(S.s[m], k.f[m][j], x[j]);
}

// What each stretch adds to the state (from zero): S of its own tokens, at the
// place of the state that the next one starts from.  It walks the stretch the
// other way round than the pass behind it does, so that this one finds what
// was read last in the caches.  Bound by HBM: 32760 tokens of 24 bf16 heads of
// 128 take 81-98 us (4.4-5.4 TB/s), the matrix cores busy for half of it.
template <typename T, int DP, bool REV>
__global__ __launch_bounds__(2 * DP, 2) void state_kernel(Lin p, Stretches map) {
  typedef Tile<T, DP> Tl;
  // bf16: three sets of chunks.  Little is computed here, and two chunks' loads
  // in flight hide the memory's latency where one's do not.
  constexpr int kSets = Tl::kHalf ? 3 : 2;
  constexpr int kSet = 2 * Tl::kBytes;
  typedef Loader<Tl, 2 * DP> Ld;
  __shared__ __align__(1024) char tiles[kSets * kSet];
  const uint32_t lds = lds_address(tiles);
  const int64_t job = p.first + blockIdx.x;
  const int id = (int)(job / p.H), h = (int)(job - (int64_t)id * p.H);
  const Stretch st = find_stretch(map, id);
  // nobody starts from the last one's end
  if ((REV ? st.head : st.tail) && p.final == nullptr) return;
  const int chunks = (st.n + kChunk - 1) / kChunk;
  auto from = [&](int i) { return (REV ? i : chunks - 1 - i) * kChunk; };
  const int tid = threadIdx.x;
  const uint32_t wave0 = wave_id() * kWave;
  Ld ld[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    Part in = p.in[a];
    in.data += (st.batch * in.batch + (int64_t)h * in.head) * 16;
    ld[a].init(in, st.start + from(0), REV ? 1 : -1, 0, p.nvec, tid);
  }
  const bool whole = Tl::kPieces == Tl::kRowVecs && p.nvec == Tl::kRowVecs;
  auto load = [&](int i) {
    const int n = min(kChunk, st.n - from(i));
    const uint32_t set = lds + i % kSets * kSet;
    if (whole && n == kChunk) {
#pragma unroll
      for (int a = 0; a < 2; ++a) ld[a].all(set + a * Tl::kBytes, wave0);
    } else {
#pragma unroll
      for (int a = 0; a < 2; ++a) ld[a].some(set + a * Tl::kBytes, wave0, n, tid);
    }
  };
  if (p.nvec < Tl::kRowVecs) {
    clear(lds, 0, kSets * kSet / 16, tid, 2 * DP);
    __syncthreads();
  }
  for (int i = 0; i < min(chunks, kSets - 1); ++i) load(i);
  const float g = decay_of(p, h);
  uint32_t k_place[Tl::kCols], v_place[Tl::kCols];
  Tl::template col_places<true>(k_place);
  Tl::template col_places<false>(v_place);
#pragma unroll
  for (int x = 0; x < Tl::kCols; ++x)
    v_place[x] ^= wave_id() * (Tl::kHalf ? 64 : 128);
  State<T, DP> S;
  S.clear();
  Powers<REV> pw;
  for (int i = 0; i < chunks; ++i) {
    const int n = min(kChunk, st.n - from(i));
    // (a chunk that is not whole may have fewer loads)
    if (kSets > 2 && i + 1 < chunks && from(i + 1) + kChunk <= st.n)
      arrive<(kSets - 2) * 2 * Ld::kLoads>();
    else
      arrive<0>();
    if (i + kSets - 1 < chunks) load(i + kSets - 1);
    pw.set(g, p.scale, n);
    const float w = exp2f(g * (REV ? from(i) : st.n - from(i) - n));
    uint32_t k_at[Tl::kCols], v_at[Tl::kCols];
#pragma unroll
    for (int x = 0; x < Tl::kCols; ++x) {
      k_at[x] = fresh(k_place[x] + lds + i % kSets * kSet);
      v_at[x] = v_place[x] + lds + i % kSets * kSet + Tl::kBytes;
    }
    Frag<T> v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = Tl::cols(v_at, j, 0);
    Parts<T, 3> x[2];
    decayed<T, REV>(x, v, pw, w);
    KeyCols<T, DP> keys;
#pragma unroll
    for (int m = 0; m < DP / 32; ++m) {
      keys.read(k_at, m);
      gather(S, keys, m, x, 1.f);
    }
  }
  S.store(p.states + job * p.d * p.d, p.d, 32 * wave_id());
}

// Along each sequence: states[j] = the state before stretch j, and the state
// behind the last.  A thread's next reads are under way together, else each
// would wait for memory in turn: 504 stretches of 128 x 128 take 15 us (4.5
// TB/s), with one read at a time 18.
constexpr int kScanAtOnce = 8;

template <bool REV>
__global__ __launch_bounds__(kBlock) void scan_kernel(Lin p, Stretches map,
                                                      int32_t blocks) {
  const int64_t row = blockIdx.x / blocks;  // sequence, head
  const int seq = (int)(row / p.H), h = (int)(row - (int64_t)seq * p.H);
  const int dd = p.d * p.d;
  const int at = ((int)(blockIdx.x - row * blocks) * kBlock + threadIdx.x) * 4;
  if (at >= dd) return;
  const int first = map.nseg == 0 ? seq * map.splits : map.first[seq];
  const int count = map.nseg == 0 ? map.splits : map.first[seq + 1] - first;
  const float g = decay_of(p, h);
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.init != nullptr)
    run = *reinterpret_cast<const float4 *>(p.init + row * dd + at);
  const int64_t tokens =
      map.nseg == 0 ? map.N : map.row[seq + 1] - map.row[seq];
  const auto turn = [&](int i) { return REV ? count - 1 - i : i; };
  const auto place = [&](int i) {
    return reinterpret_cast<float4 *>(
        p.states + ((int64_t)(first + turn(i)) * p.H + h) * dd + at);
  };
  const int used = p.final != nullptr ? count : count - 1;
  for (int i0 = 0; i0 < count; i0 += kScanAtOnce) {
    float4 own[kScanAtOnce];
#pragma unroll
    for (int u = 0; u < kScanAtOnce; ++u)
      if (i0 + u < used) own[u] = *place(i0 + u);
#pragma unroll
    for (int u = 0; u < kScanAtOnce; ++u) {
      const int i = i0 + u;
      if (i >= count) break;
      *place(i) = run;
      if (i >= used) break;
      const float over =
          exp2f(g * (float)min(map.len, tokens - turn(i) * map.len));
      run.x = fmaf(run.x, over, own[u].x);
      run.y = fmaf(run.y, over, own[u].y);
      run.z = fmaf(run.z, over, own[u].z);
      run.w = fmaf(run.w, over, own[u].w);
    }
  }
  if (p.final != nullptr)
    *reinterpret_cast<float4 *>(p.final + row * dd + at) = run;
}

// a[s][t] = k_s . q_t for 16 tokens each.  As long as both take the features
// in the same order, any will do: piece 4 b + l / 16 of block b.
template <typename T, int DP>
__device__ __forceinline__ void score(f32x4 &a, uint32_t k_at, uint32_t q_at) {
#pragma unroll
  for (int b = 0; b < Tile<T, DP>::kRowVecs / 4; ++b) {
    const u32x4 k = lds_read<u32x4>(k_at ^ (64 * b));
    const u32x4 q = lds_read<u32x4>(q_at ^ (64 * b));
    if constexpr (sizeof(T) == 2) {
      a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q), a, 0,
          0, 0);
    } else {
      const f32x4 kf = __builtin_bit_cast(f32x4, k),
                  qf = __builtin_bit_cast(f32x4, q);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[i], qf[i], a, 0, 0, 0);
    }
  }
}

// Four scores of token t, s = 4 u + [0, 4), into the tiles of their parts.
template <typename T>
__device__ __forceinline__ uint32_t put_place(int t, int u) {
  typedef Tile<T, 32> Sc;
  return Sc::kHalf
             ? t * Sc::kPitch + ((u / 2) ^ Sc::turn(t)) * 16 + u % 2 * 8
             : t * Sc::kPitch + (u ^ Sc::turn(t)) * 16;
}
template <typename T>
__device__ __forceinline__ void put_scores(uint32_t at, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    Parts<T, 2> y;
    y.set(x);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const s16x8 v = __builtin_bit_cast(s16x8, y.f[part].v);
      const s16x4 four = __builtin_shufflevector(v, v, 0, 1, 2, 3);
      lds_write(at + part * Tile<T, 32>::kBytes, four);
    }
  } else {
    lds_write(at, f32x4{x[0], x[1], x[2], x[3]});
  }
}

// In the product with the scores every token meets every v, with zeros where it
// does not count; one that is not finite spoils them all.  clean() puts zeros in
// the place of such, and gives the chunk's first token (REV: the last) that has
// one.  v: feature lane % 32 of 32, tokens 16 j + slot(i).
template <bool REV, typename T>
__device__ __forceinline__ int clean(Frag<T> (&v)[2]) {
  int at = REV ? -1 : kChunk;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float y[8];
    from_frag(y, v[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!isfinite(y[i])) {
        y[i] = 0.f;
        const int token = 16 * j + slot(i);
        at = REV ? max(at, token) : min(at, token);
      }
    to_frag(v[j], y);
  }
  const int other = __shfl_xor(at, 32);
  return REV ? max(at, other) : min(at, other);
}
// That token's output, and those of tokens that it counts for, become NaN.
template <bool REV>
__device__ __forceinline__ void spoil(f32x16 &o, int at) {
  const int t = lane_id() % 32;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int from = __shfl(at, r / 4 * 8 + 4 * half_of() + r % 4);
    if (REV ? t <= from : t >= from) o[r] = __builtin_nanf("");
  }
}

// What this wavefront has written to LDS is there, then that of every one.
__device__ __forceinline__ void arrive_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The outputs of a stretch, from the state before it.  ROLES 1: in = q, k, v.
// ROLES 2, the two gradients that run backwards: in = q, k, v, do, out = dv
// (of k, q, do) and dk (of v, do, q), a set of wavefronts for each.  ONE: each
// sequence is one stretch, which starts from its initial state and also makes
// the state behind it.  `across` (bit by role): the states in memory are the
// transpose of this role's.
// Bound by HBM and the matrix cores together, on a card at its power limit:
// 32760 tokens of 24 bf16 heads of 128 take 193-225 us (3.9-4.5 TB/s, matrix
// cores 49%); 16 x 1560 of 12, a sequence to a workgroup, 106-124 us, their dv
// and dk 171-199 (matrix cores 50%, on three of four CUs).  f32, 2 x 1777 of
// 10 heads of 72: 36 and 56 us, five chunks in a row on each CU.  (A wavefront
// stores 64 bytes of a token, half a line, with the streaming hint: up to a fifth
// more than the outputs' bytes is written, 240 MB for 201 in the first case.
// Plain stores write 201, but take 3% longer.)
template <typename T, int DP, bool REV, int ROLES, bool ONE>
__global__ __launch_bounds__(2 * DP * ROLES,
                             ROLES == 1 ? 2 : 1) void out_kernel(
    Lin p, Stretches map, int32_t across) {
  typedef Tile<T, DP> Tl;
  typedef Tile<T, 32> Sc;
  constexpr int kThreads = 2 * DP * ROLES, NT = ROLES + 2;
  constexpr int kWaves = kThreads / kWave;
  constexpr int E = Elems<T>::value;
  // bf16: three sets of chunks, two of them under way; f32 has room for two
  constexpr int kSets = Tl::kHalf ? 3 : 2;
  // V, of which a wavefront reads its own 32 columns alone, has tiles by
  // wavefront where no role has it for something else; they take its outputs
  // once V has been read
  constexpr bool kOwn = Tl::kHalf && ROLES == 1;
  constexpr int kShared = kOwn ? 2 : NT;  // tensors with a tile for all
  constexpr int kSet =
      kShared * Tl::kBytes + (kOwn ? kWaves * Sc::kBytes : 0);
  typedef Loader<Tl, kThreads> Ld;
  typedef Loader<Sc, kWave> OwnLd;
  __shared__ __align__(1024) char tiles[kSets * kSet];
  // outputs on their way out (f32: 16 bytes a lane as they stand, for which
  // LDS has no room beside two sets of tiles anyway)
  __shared__ __align__(1024) char outs[Tl::kHalf && !kOwn ? kWaves : 1]
                                    [kOwn || !Tl::kHalf ? 16 : kChunk * 64];
  // the scores, decayed, in two parts: rows are the tokens t, 32 scores each
  constexpr int kScParts = Parts<T, 2>::kParts;
  __shared__ __align__(1024) char scores[ROLES * kScParts * Sc::kBytes];
  const uint32_t lds = lds_address(tiles), P = lds_address(scores);
  const int64_t job = p.first + blockIdx.x;
  const int id = (int)(job / p.H), h = (int)(job - (int64_t)id * p.H);
  const Stretch st = find_stretch(map, id);
  const int wave = wave_id(), tid = threadIdx.x;
  const int role = ROLES == 1 ? 0 : wave / (DP / 32);
  const int m0 = ROLES == 1 ? wave : wave % (DP / 32);
  const int c0 = 32 * m0;
  const int chunks = (st.n + kChunk - 1) / kChunk;
  auto from = [&](int i) { return (REV ? chunks - 1 - i : i) * kChunk; };
  Ld ld[kShared];
  OwnLd own;
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    Part in = p.in[a];
    in.data += (st.batch * in.batch + (int64_t)h * in.head) * 16;
    if (a < kShared)
      ld[a].init(in, st.start + from(0), REV ? -1 : 1, 0, p.nvec, tid);
    else
      own.init(in, st.start + from(0), REV ? -1 : 1, c0 / E, p.nvec, lane_id());
  }
  const bool whole = Tl::kPieces == Tl::kRowVecs && p.nvec == Tl::kRowVecs;
  auto tokens = [&](int i) { return min(kChunk, st.n - from(i)); };
  auto set_at = [&](int i) { return lds + i % kSets * kSet; };
  auto own_at = [&](int i) {
    return set_at(i) + kShared * Tl::kBytes + wave * Sc::kBytes;
  };
  auto load_all = [&](int i) {
#pragma unroll
    for (int a = 0; a < kShared; ++a)
      ld[a].all(set_at(i) + a * Tl::kBytes, wave * kWave);
  };
  auto load_some = [&](int i) {
#pragma unroll
    for (int a = 0; a < kShared; ++a)
      ld[a].some(set_at(i) + a * Tl::kBytes, wave * kWave, tokens(i), tid);
    if constexpr (kOwn) own.some(own_at(i), 0, tokens(i), lane_id());
  };
  if (p.nvec < Tl::kRowVecs) {
    clear(lds, 0, kSets * kSet / 16, tid, kThreads);
    __syncthreads();
  }
  for (int i = 0; i < min(chunks, kSets - 1); ++i) load_some(i);
  // the block of scores that does not count is never written
  clear(P, 0, sizeof scores / 16, tid, kThreads);
  const Part out = p.out[role];
  char *dst = const_cast<char *>(out.data) +
              (st.batch * out.batch + (int64_t)h * out.head) * 16;
  const float g = decay_of(p, h);
  const int64_t dd = (int64_t)p.d * p.d;
  State<T, DP> S;
  const float *src = !ONE ? p.states + job * dd
                     : p.init != nullptr
                         ? p.init + ((int64_t)st.seq * p.H + h) * dd
                         : nullptr;
  if (src != nullptr)
    S.load(src, p.d, c0, across >> role & 1);
  else
    S.clear();
  // Of the 32 x 32 scores of a chunk only those of t >= s (REV: s >= t) count:
  // of their four blocks of 16 x 16 three, a wavefront of the role each (one
  // wavefront, or two, take them in turn; a fourth computes one again, which
  // costs nothing that a branch would not).
  constexpr int kTeam = DP / 32;
  constexpr int kTurns = (2 + kTeam) / kTeam;
  auto block_s = [](int i) { return REV ? (i > 0) : (i == 2); };
  auto block_t = [](int i) { return REV ? (i == 2) : (i > 0); };
  // powers of the lane's scores: s = 4 (lane / 16) + r, t = lane % 16; those
  // of the block off the diagonal are 16 tokens further apart
  float near[kTurns][4];
#pragma unroll
  for (int turn = 0; turn < kTurns; ++turn)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int s = 4 * (lane_id() / 16) + r, t = lane_id() % 16;
      const int e = (REV ? s - t : t - s) +
                    (min(m0 + turn * kTeam, 2) == 1 ? 16 : 0);
      near[turn][r] = e >= 0 ? p.scale * exp2f(g * e) : 0.f;
    }
  // minus one where a row of 32 is summed element 16 x + slot(i)
  Frag<T> minus[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = lane_id() % 32 == 16 * x + slot(i) ? -1.f : 0.f;
    to_frag(minus[x], y);
  }
  Powers<REV> pw;
  // the lane's places in the tiles
  const int lane = lane_id();
  const uint32_t q_tile = (ROLES == 1 ? 0 : role == 0 ? 1 : 2) * Tl::kBytes;
  const uint32_t k_tile = (ROLES == 1 ? 1 : role == 0 ? 0 : 3) * Tl::kBytes;
  const uint32_t v_tile = kOwn ? kShared * Tl::kBytes + wave * Sc::kBytes
                          : (ROLES == 1 ? 2 : role == 0 ? 3 : 0) * Tl::kBytes;
  const uint32_t q_place = Tl::pair_place() + q_tile;
  uint32_t k_place[Tl::kCols], v_place[Tl::kCols];
  Tl::template col_places<true>(k_place);
  if constexpr (kOwn) {
    Sc::template col_places<false>(v_place);
  } else {
    Tl::template col_places<false>(v_place);
  }
#pragma unroll
  for (int x = 0; x < Tl::kCols; ++x) {
    k_place[x] += k_tile;
    if (!kOwn) v_place[x] ^= m0 * (Tl::kHalf ? 64 : 128);
    v_place[x] += v_tile;
  }
  const uint32_t scores_at = P + role * kScParts * Sc::kBytes;
  const uint32_t score_row = scores_at + Sc::row_place();
  uint32_t score_k[kTurns], score_q[kTurns], score_put[kTurns];
#pragma unroll
  for (int turn = 0; turn < kTurns; ++turn) {
    const int i3 = min(m0 + turn * kTeam, 2);
    const int s0 = 16 * block_s(i3), t0 = 16 * block_t(i3);
    score_k[turn] = Tl::score_place(s0) + k_tile;
    score_q[turn] = Tl::score_place(t0) + q_tile;
    // s along the token's row: four of them side by side
    score_put[turn] =
        scores_at + put_place<T>(t0 + lane % 16, s0 / 4 + lane / 16);
  }
  // The wavefront's outputs of a chunk are kept (in LDS, or f32 in registers)
  // until the next one's loads are awaited, so that a store has a chunk's time
  // to complete.  Unit u, 4 bf16 of token t, stands at u ^ (t / 4) % 4 of the
  // token's eight, for the banks' sake.
  auto out_at = [&](int i) {
    return kOwn ? own_at(i) : lds_address(outs[kOwn ? 0 : wave]);
  };
  const uint32_t put_out =
      lane % 32 * 64 + (half_of() ^ (lane % 32 >> 2 & 3)) * 8;
  const uint32_t take_out =
      lane / 4 * 64 + ((2 * (lane % 4)) ^ (lane / 4 >> 2 & 3)) * 8;
  constexpr int kRow = 32 / E;                    // vectors of 32 features
  constexpr int kKept = Tl::kHalf ? kChunk * kRow / kWave : 4;
  float kept[Tl::kHalf ? 1 : 16];
  uint32_t out_off[kKept];
  bool out_ok[kKept];
  int out_t[kKept];
#pragma unroll
  for (int x = 0; x < kKept; ++x) {
    const int t = Tl::kHalf ? (lane + x * kWave) / kRow : lane % 32;
    const int j = Tl::kHalf ? (lane + x * kWave) % kRow
                            : (16 * (x / 2) + slot(x % 2 * 4)) / 4;
    out_t[x] = t;
    out_off[x] = ((uint32_t)t * (uint32_t)out.token + c0 / E + j) * 16;
    out_ok[x] = c0 / E + j < p.nvec;
  }
  auto take = [&](int i, Vec (&y)[kKept]) {
#pragma unroll
    for (int x = 0; x < kKept; ++x) {
      if constexpr (Tl::kHalf) {
        const uint32_t at = out_at(i) + take_out;
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 lo = lds_read<u32x2>(at + x * 1024),
                    hi = lds_read<u32x2>((at ^ 8) + x * 1024);
        y[x].w[0] = lo[0];
        y[x].w[1] = lo[1];
        y[x].w[2] = hi[0];
        y[x].w[3] = hi[1];
      } else {
        const float f[4] = {kept[4 * x], kept[4 * x + 1], kept[4 * x + 2],
                            kept[4 * x + 3]};
        y[x] = pack<float>(f);
      }
    }
  };
  // every token and feature, or some
  auto store_all = [&](int i, const Vec (&y)[kKept]) {
    char *base = dst + (st.start + from(i)) * out.token * 16;
#pragma unroll
    for (int x = 0; x < kKept; ++x) store_stream(base + out_off[x], y[x]);
  };
  auto store_some = [&](int i, const Vec (&y)[kKept]) {
    char *base = dst + (st.start + from(i)) * out.token * 16;
#pragma unroll
    for (int x = 0; x < kKept; ++x)
      if (out_ok[x] && out_t[x] < tokens(i))
        store_stream(base + out_off[x], y[x]);
  };
  for (int i = 0; i < chunks; ++i) {
    // (a chunk that is not whole may have fewer loads)
    if (kSets > 2 && i + 1 < chunks && from(i + 1) + kChunk <= st.n)
      arrive<(kSets - 2) * (kShared * Ld::kLoads + (kOwn ? OwnLd::kLoads : 0))>();
    else
      arrive<0>();
    {
      const int more = i + kSets - 1;
      Vec y[kKept];
      // (V goes into the tile that the outputs have just been taken from)
      if (whole && i > 0 && more < chunks && tokens(i - 1) == kChunk &&
          tokens(more) == kChunk) {
        take(i - 1, y);
        load_all(more);
        store_all(i - 1, y);
        if constexpr (kOwn) own.all(own_at(more), 0);
      } else {
        if (i > 0) {
          take(i - 1, y);
          store_some(i - 1, y);
        }
        if (more < chunks) load_some(more);
      }
    }
    pw.set(g, p.scale, min(kChunk, st.n - from(i)));
    const uint32_t set = set_at(i);
#pragma unroll
    for (int turn = 0; turn < kTurns; ++turn) {
      f32x4 a = {};
      score<T, DP>(a, fresh(score_k[turn] + set), fresh(score_q[turn] + set));
      float x[8] = {};
#pragma unroll
      for (int r = 0; r < 4; ++r)
        // (selected: a k or q that is not finite does not reach the tokens
        // that it does not count for)
        x[r] = near[turn][r] != 0.f ? a[r] * near[turn][r] : 0.f;
      put_scores<T>(score_put[turn], x);
    }
    uint32_t q_at = fresh(q_place + set), k_at[Tl::kCols], v_at[Tl::kCols];
#pragma unroll
    for (int x = 0; x < Tl::kCols; ++x) {
      k_at[x] = fresh(k_place[x] + set);
      v_at[x] = fresh(v_place[x] + set);
    }
    // the state's part; what its rounding to bf16 leaves, the matrix cores
    // subtract (exactly): S - 1 * hi.  They take some time for it, so the rest
    // of one block of rows follows behind the next one's rounding.
    f32x16 o = {};
    f32x16 rest[2];
    Frag<T> q[2][2];
    auto low = [&](int m) {
      if constexpr (Tl::kHalf) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = rest[m & 1][8 * x + e];
          Frag<T> lo;
          to_frag(lo, y);
          mma(o, lo, q[m & 1][x]);
        }
      }
    };
#pragma unroll
    for (int m = 0; m < DP / 32; ++m) {
      Frag<T> hi[2];
      rest[m & 1] = S.s[m];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        q[m & 1][x] = Tl::pairs(q_at, 2 * m + x);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = S.s[m][8 * x + e];
        to_frag(hi[x], y);
        if constexpr (Tl::kHalf) mma(rest[m & 1], minus[x], hi[x]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) mma(o, hi[x], q[m & 1][x]);
      if (m > 0) low(m - 1);
    }
    low(DP / 32 - 1);
    Frag<T> v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kOwn)
        v[j] = Sc::cols(v_at, j, 0);
      else
        v[j] = Tl::cols(v_at, j, 0);
    }
    Parts<T, 3> vs[2];
    decayed<T, REV>(vs, v, pw, 1.f);
    // (bf16: k is read before the wavefronts wait for each other, f32 has no
    // registers for that)
    constexpr bool kEarly = Tl::kHalf;
    KeyCols<T, DP> keys;
    if constexpr (kEarly)
#pragma unroll
      for (int m = 0; m < DP / 32; ++m) keys.read(k_at, m);
    if (kTeam > 1) {
      arrive_lds();
    } else {
      __builtin_amdgcn_wave_barrier();
    }
    f32x16 near_o = {};
    auto scored = [&] {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int part = 0; part < kScParts; ++part)
          mma(near_o, v[j], Sc::rows(score_row + part * Sc::kBytes, j));
    };
    scored();
#pragma unroll
    for (int m = 0; m < DP / 32; ++m) {
      if (!kEarly) keys.read(k_at, m);
      gather(S, keys, m, vs, pw.over);
    }
    // (a v that is not finite has left its column of the state so, each row: one
    // of them tells, and stays so, which costs these sequences some time)
    if (__builtin_expect(__any(!isfinite(S.s[0][0])), 0)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (kOwn)
          v[j] = Sc::cols(v_at, j, 0);
        else
          v[j] = Tl::cols(v_at, j, 0);
      }
      const int at = clean<REV>(v);
      near_o = f32x16{};
      scored();
      spoil<REV>(near_o, at);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) o[r] = fmaf(o[r], pw.own, near_o[r]);
    // o: rows are features, the lane's column its token
    if constexpr (Tl::kHalf) {
      const uint32_t at = fresh(out_at(i) + put_out);
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const float x[8] = {o[r], o[r + 1], o[r + 2], o[r + 3], 0, 0, 0, 0};
        const Vec y = pack<bf16>(x);
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        lds_write(at ^ (4 * r), u32x2{y.w[0], y.w[1]});
      }
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) kept[r] = o[r];
    }
  }
  if (chunks > 0) {
    __builtin_amdgcn_wave_barrier();
    Vec y[kKept];
    take(chunks - 1, y);
    store_some(chunks - 1, y);
  }
  if (ONE && p.final != nullptr && role == 0)
    S.store(p.final + ((int64_t)st.seq * p.H + h) * dd, p.d, c0);
}

// One token of each sample: S' = l S + k v^T, o = c S'^T q.  A thread holds
// four columns of every R-th row, the next kStepRows of them under way while
// it works on these.  Bound by the state, read and written once.  It is not
// read again before the other layers' states have been, so it goes past the
// caches: 128 samples of 12 heads of 128 take 38 us (5.3 TB/s), 43 without
// the streaming hint; 512 of 24 296 and 312.  Eight rows under way at once
// take 268 us there, but 22 us, not 17, for 200 samples of 10 f32 heads of 72,
// whose threads have six.
struct Step {
  Part q, k, v, o;
  const float *log_decay, *state;
  float *state_out;
  float scale;
  int32_t H, d;
  int32_t cols;    // threads across a workgroup's columns
  int32_t groups;  // workgroups across the state's
  int64_t jobs;
};

template <typename T>
__device__ __forceinline__ float scalar(const Part &p, int64_t b, int h,
                                        int i) {
  const char *at = p.data + (b * p.batch + (int64_t)h * p.head) * 16;
  if constexpr (sizeof(T) == 2)
    return __builtin_bit_cast(
        float, (uint32_t)reinterpret_cast<const uint16_t *>(at)[i] << 16);
  else
    return reinterpret_cast<const float *>(at)[i];
}

constexpr int kStepRows = 4;

template <typename T>
__global__ __launch_bounds__(kBlock) void step_kernel(Step p) {
  __shared__ float sums[kBlock][4];
  __shared__ float qk[2][kMaxHead];
  const int t = threadIdx.x;
  const int c = t % p.cols, r0 = t / p.cols, R = kBlock / p.cols;
  for (int64_t job = blockIdx.x; job < p.jobs; job += gridDim.x) {
    const int64_t bh = job / p.groups;
    const int64_t b = bh / p.H;
    const int h = (int)(bh - b * p.H);
    const int col = ((int)(job - bh * p.groups) * p.cols + c) * 4;
    const bool active = r0 < R && col < p.d;
    const float *src = p.state + bh * p.d * p.d + col;
    float *dst = p.state_out + bh * p.d * p.d + col;
    f32x4 rows[kStepRows], next[kStepRows];
    const auto read = [&](f32x4 (&x)[kStepRows], int r) {
#pragma unroll
      for (int u = 0; u < kStepRows; ++u)
        if (active && r + u * R < p.d)
          x[u] = __builtin_nontemporal_load(
              reinterpret_cast<const f32x4 *>(src + (r + u * R) * p.d));
    };
    // (every load is under way before the first is awaited)
    float mine = 0.f, v[4] = {}, sum[4] = {};
    const int own = t % kMaxHead;
    if (own < p.d) mine = scalar<T>(t < kMaxHead ? p.q : p.k, b, h, own);
    if (active)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = scalar<T>(p.v, b, h, col + i);
    read(rows, r0);
    // l near 1 as its distance from there: rounded to 24 bits itself, it would
    // be off by the same amount in every step, 1.2e-4 after 4096 of them.  (A
    // small l would lose its digits as a distance.)
    const float g = p.log_decay[h];
    const bool near = g > -0.5f;
    const float l = near ? expm1f(g) : expf(g);
    __syncthreads();
    if (own < p.d) qk[t / kMaxHead][own] = mine;
    __syncthreads();
    for (int r = r0; r < p.d; r += kStepRows * R) {
      read(next, r + kStepRows * R);
#pragma unroll
      for (int u = 0; u < kStepRows; ++u) {
        const int row = r + u * R;
        if (active && row < p.d) {
          const float k = qk[1][row], q = qk[0][row];
          f32x4 n;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            n[i] = fmaf(k, v[i],
                        fmaf(l, rows[u][i], near ? rows[u][i] : 0.f));
            sum[i] = fmaf(q, n[i], sum[i]);
          }
          __builtin_nontemporal_store(
              n, reinterpret_cast<f32x4 *>(dst + row * p.d));
        }
        rows[u] = next[u];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[t][i] = sum[i];
    __syncthreads();
    if (active && r0 == 0) {
      for (int r = 1; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += sums[t + r * p.cols][i];
      char *at = const_cast<char *>(p.o.data) +
                 (b * p.o.batch + (int64_t)h * p.o.head) * 16;
      const float x[8] = {p.scale * sum[0], p.scale * sum[1],
                          p.scale * sum[2], p.scale * sum[3], 0, 0, 0, 0};
      if constexpr (sizeof(T) == 2) {
        const Vec y = pack<bf16>(x);
        *reinterpret_cast<uint2 *>(at + col * 2) = make_uint2(y.w[0], y.w[1]);
      } else {
        *reinterpret_cast<float4 *>(at + col * 4) =
            make_float4(x[0], x[1], x[2], x[3]);
      }
    }
  }
}

// ----------------------------------------------------------------- planning

int elems_per_vec(int dtype) { return dtype == ADALN_BF16 ? 8 : 4; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

// How long the stretches are.  A stretch more is more work at once, but its
// state is written, read and written, and read: the traffic of some 200
// tokens, a fourth of the chunk that it starts with, and a share of the scan.
// Measured, forward and backward in us:
// - Sequences none of which is longer than 3/2 of a CU's share stay whole,
//   without states, a workgroup each: equal ones from 171 of them (times heads)
//   on.  Fewer, two workgroups to a CU have room for three stretches of each,
//   more only for two.  Tokens 1560, bf16, whole and cut (stretches):
//     160 (480) heads of 128 94 and 244, 104 and 240; of 96 86 and 215, 82 and
//               182; of 64 74 and 168, 64 and 118
//     176 (352) heads of 128 95 and 246, 123 and 290; of 96 87 and 216, 102 and
//               236; of 64 74 and 169, 84 and 154
//     192 (384) heads of 128 98 and 263, 132 and 311; of 96 87 and 215, 104 and
//               239; of 64 74 and 167, 85 and 158
//   A workgroup of heads of up to 32 is one wavefront, so that whole sequences
//   leave most of a CU idle.  Theirs are cut up to 4/3 of the share: 176 (352)
//   take 55 and 105, whole 58 and 132.  (So would 256 gain, 55 and 107.)
// - Else one workgroup per CU, for less than a whole second one would run
//   alone: 4096 tokens of 16 such heads take 45 and 79 cut in 16, 51 and 102
//   in 22.  f32's tiles leave room for one (8190 tokens of 12 heads: 147 and
//   316 in 20, 169 and 346 in 37).
// - bf16's leave room for two, which pays if stretches stay long: 32760 tokens
//   of 24 heads take 295 and 684 in 21, 327 and 718 in 10, and 8 x 1560 of 12
//   74 and 158 in 5, 85 and 171 in 2, but 4 x 1560 47 and 85 in 5, 52 and 98
//   in 10.
//   (Those are heads of 128.  Narrower ones leave room for more, f32's of up to 64
//   for two, which these rules do not use: 8190 f32 tokens of 12 heads of 64 take
//   84 and 150 in 20, 68 and 144 in 37; 4 x 1560 bf16 of 12 of 64 35 and 58 in 5,
//   33 and 53 in 10; 32760 of 24 of 64 161 and 315 in 21, 157 and 316 in 41.)
// - What is done in four chunks is not worth two more launches.
constexpr int64_t kLong = 256;
constexpr int64_t kWhole = 4 * kChunk;

// Whether sequences stay whole: in exact arithmetic, so that of equal ones
// their number alone decides, not their length too.
bool stay_whole(int64_t longest, int64_t tokens, int64_t H, int64_t d) {
  if (longest <= kWhole) return true;
  return d <= 32 ? longest * kCUs * 3 <= tokens * H * 4
                 : longest * kCUs * 2 <= tokens * H * 3;
}

int64_t stretches_of(int64_t tokens, int64_t len) {
  return std::max<int64_t>(1, (tokens + len - 1) / len);
}

// false: more stretches than can be numbered.
bool make_stretches(Stretches &m, const int64_t *off, int64_t nseg, int64_t B,
                    int64_t N, int64_t H, int64_t d, int dtype,
                    int64_t *count) {
  m = Stretches{};
  const auto sum = [&](int64_t len) {
    if (off == nullptr) return B * stretches_of(N, len);
    int64_t n = 0;
    for (int64_t s = 0; s < nseg; ++s)
      n += stretches_of(off[s + 1] - off[s], len);
    return n;
  };
  int64_t longest = off == nullptr ? N : 0;
  if (off != nullptr)
    for (int64_t s = 0; s < nseg; ++s)
      longest = std::max(longest, off[s + 1] - off[s]);
  const int64_t tokens = off == nullptr ? B * N : off[nseg];
  const int64_t share = tokens * H / kCUs;
  const auto chunks = [](int64_t n) {
    return std::max<int64_t>(1, (n + kChunk - 1) / kChunk) * kChunk;
  };
  int64_t len = chunks(longest);
  if (!stay_whole(longest, tokens, H, d)) {
    const int64_t each = dtype == ADALN_BF16 && share / 2 >= kLong ? 2 : 1;
    const int64_t even = chunks(share / each), step = chunks(even / 16);
    // the ends of sequences are stretches too: up to twice as long, if that
    // leaves no workgroup over
    len = even;
    while (len < 2 * even && sum(len) * H > each * kCUs) len += step;
    if (sum(len) * H > each * kCUs) len = even;
  }
  m.N = N;
  m.len = len;
  *count = sum(len);
  m.splits = (int32_t)(off == nullptr ? stretches_of(N, len)
                                      : 1 + (longest > len));
  if (off != nullptr) {
    m.nseg = (int32_t)nseg;
    int64_t n = 0;
    for (int64_t s = 0; s < nseg; ++s) {
      m.first[s] = (int32_t)n;
      m.row[s] = off[s];
      n += stretches_of(off[s + 1] - off[s], len);
    }
    m.first[nseg] = (int32_t)n;
    m.row[nseg] = off[nseg];
  }
  return *count * H <= kMaxRows;
}

size_t states_bytes(const Stretches &m, int64_t count, int64_t H, int64_t d) {
  return m.splits > 1 ? (size_t)count * H * d * d * sizeof(float) : 0;
}

int hip_fail(hipError_t e, const char *what) {
  return fail(ADALN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kLaunch = 1 << 20;  // workgroups of a launch

template <typename K, typename... A>
hipError_t launch_jobs(K k, int threads, Lin p, hipStream_t s, A... args) {
  for (p.first = 0; p.first < p.jobs; p.first += kLaunch) {
    void *argv[] = {(void *)&p, (void *)&args...};
    const hipError_t e = hipLaunchKernel(
        (const void *)k, dim3((unsigned)std::min(kLaunch, p.jobs - p.first)),
        dim3(threads), argv, 0, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, bool REV>
hipError_t run_states(const Lin &p, const Stretches &m, hipStream_t s) {
  if (p.d <= 32)
    return launch_jobs(state_kernel<T, 32, REV>, 64, p, s, m);
  if (p.d <= 64)
    return launch_jobs(state_kernel<T, 64, REV>, 128, p, s, m);
  if (p.d <= 96)
    return launch_jobs(state_kernel<T, 96, REV>, 192, p, s, m);
  return launch_jobs(state_kernel<T, 128, REV>, 256, p, s, m);
}

template <typename T, bool REV, int ROLES, bool ONE>
hipError_t run_out(const Lin &p, const Stretches &m, int32_t across,
                   hipStream_t s) {
  if (p.d <= 32)
    return launch_jobs(out_kernel<T, 32, REV, ROLES, ONE>, 64 * ROLES, p, s, m,
                       across);
  if (p.d <= 64)
    return launch_jobs(out_kernel<T, 64, REV, ROLES, ONE>, 128 * ROLES, p, s,
                       m, across);
  if (p.d <= 96)
    return launch_jobs(out_kernel<T, 96, REV, ROLES, ONE>, 192 * ROLES, p, s,
                       m, across);
  return launch_jobs(out_kernel<T, 128, REV, ROLES, ONE>, 256 * ROLES, p, s, m,
                     across);
}

template <bool REV, int ROLES>
hipError_t outputs(const Lin &p, const Stretches &m, int32_t across, int dtype,
                   hipStream_t s) {
  if (p.states == nullptr)
    return dtype == ADALN_BF16
               ? run_out<bf16, REV, ROLES, true>(p, m, across, s)
               : run_out<float, REV, ROLES, true>(p, m, across, s);
  return dtype == ADALN_BF16
             ? run_out<bf16, REV, ROLES, false>(p, m, across, s)
             : run_out<float, REV, ROLES, false>(p, m, across, s);
}

// The states that the stretches start from: p.in are the two parts that make
// up the state.
template <bool REV>
hipError_t make_states(const Lin &p, const Stretches &m, int64_t sequences,
                       int dtype, hipStream_t s) {
  hipError_t e = dtype == ADALN_BF16 ? run_states<bf16, REV>(p, m, s)
                                     : run_states<float, REV>(p, m, s);
  if (e != hipSuccess) return e;
  const int32_t blocks = (p.d * p.d / 4 + kBlock - 1) / kBlock;
  void *argv[] = {(void *)&p, (void *)&m, (void *)&blocks};
  return hipLaunchKernel((const void *)scan_kernel<REV>,
                         dim3((unsigned)(sequences * p.H * blocks)),
                         dim3(kBlock), argv, 0, s);
}

// Offsets within a chunk are 32 bits.
int check_part(const adaln_heads_t *t, int64_t B, int64_t N, int64_t H,
               int64_t d, int dtype, bool output, const char *name) {
  ADALN_TRY(check_heads(t, B, N, H, d, dtype, output, name));
  if (t != nullptr && B * N * H > 0 && N > 1 &&
      t->token_stride / elems_per_vec(dtype) > (int64_t(1) << 22))
    return fail(ADALN_ERR_UNSUPPORTED, "%s: tokens more than 64 MiB apart",
                name);
  return ADALN_OK;
}

Part part_of(const adaln_heads_t *t, int64_t B, int64_t N, int64_t H,
             int dtype) {
  Part h = {};
  if (t == nullptr) return h;
  const int E = elems_per_vec(dtype);
  h.data = static_cast<const char *>(t->data);
  h.batch = B > 1 ? t->batch_stride / E : 0;
  h.token = N > 1 ? t->token_stride / E : 0;
  h.head = H > 1 ? (int32_t)(t->head_stride / E) : 0;
  return h;
}

int check_lin(const float *log_decay, float scale, const int64_t *off,
              int64_t nseg, int64_t B, int64_t N, int64_t H, int64_t d,
              int dtype) {
  if (dtype != ADALN_F32 && dtype != ADALN_BF16)
    return fail(ADALN_ERR_DTYPE, "unknown dtype code %d", dtype);
  if (B < 0 || N < 0 || H < 0)
    return fail(ADALN_ERR_INVALID, "negative size: B=%lld N=%lld H=%lld",
                (long long)B, (long long)N, (long long)H);
  if (d <= 0)
    return fail(ADALN_ERR_INVALID, "d must be positive, got %lld",
                (long long)d);
  const int E = elems_per_vec(dtype);
  if (d % E != 0)
    return fail(ADALN_ERR_ALIGN, "d=%lld is not a multiple of %d",
                (long long)d, E);
  if (d > kMaxHead)
    return fail(ADALN_ERR_UNSUPPORTED, "d=%lld exceeds the widest head (%d)",
                (long long)d, kMaxHead);
  if (H > 4096) return fail(ADALN_ERR_INVALID, "more than 4096 heads");
  if (B > (int64_t(1) << 20))
    return fail(ADALN_ERR_INVALID, "B=%lld exceeds 2^20", (long long)B);
  if (N > kMaxRows || (N > 0 && B > kMaxRows / N))
    return fail(ADALN_ERR_INVALID, "B*N exceeds 2^31-1 tokens");
  if (off != nullptr) {
    if (B != 1)
      return fail(ADALN_ERR_INVALID, "packed sequences need B=1, got %lld",
                  (long long)B);
    if (nseg < 1)
      return fail(ADALN_ERR_INVALID, "nseg=%lld outside [1, %d]",
                  (long long)nseg, kMaxSegments);
    ADALN_TRY(check_segments(off, nullptr, nseg, nseg, 8, ADALN_BF16));
    if (off[nseg] != N)
      return fail(ADALN_ERR_INVALID, "seg_offsets end at %lld, N is %lld",
                  (long long)off[nseg], (long long)N);
  }
  if (!isfinite(scale))
    return fail(ADALN_ERR_INVALID, "scale is not finite");
  const bool work = H > 0 && B > 0;
  if (work && log_decay == nullptr)
    return fail(ADALN_ERR_INVALID, "log_decay is NULL");
  if (work && reinterpret_cast<uintptr_t>(log_decay) % 4 != 0)
    return fail(ADALN_ERR_ALIGN, "log_decay is not 4-byte aligned");
  return ADALN_OK;
}

int check_workspace(const void *ws, size_t have, size_t need,
                    const char *name) {
  if (need == 0) return ADALN_OK;
  if (ws == nullptr || have < need)
    return fail(ADALN_ERR_WORKSPACE, "%s needs %zu bytes, got %zu%s", name,
                need, have, ws == nullptr ? " (NULL)" : "");
  return check_ptr(ws, true, name);
}

Lin lin_of(const float *log_decay, float scale, int64_t H, int64_t d,
           int64_t count, int dtype) {
  Lin p = {};
  p.log_decay = log_decay;
  p.scale = scale;
  p.H = (int32_t)H;
  p.d = (int32_t)d;
  p.nvec = (int32_t)(d / elems_per_vec(dtype));
  p.jobs = count * H;
  return p;
}

const int kTooMany = ADALN_ERR_UNSUPPORTED;

}  // namespace
}  // namespace adaln

using namespace adaln;

ADALN_API size_t adaln_lin_attn_states_bytes(const int64_t *seg_offsets,
                                             int64_t nseg, int64_t B,
                                             int64_t N, int64_t H, int64_t d,
                                             int dtype) {
  static const float any = 0.f;
  if (check_lin(&any, 1.f, seg_offsets, nseg, B, N, H, d, dtype) != ADALN_OK)
    return 0;
  Stretches m;
  int64_t count;
  if (!make_stretches(m, seg_offsets, nseg, B, N, H, d, dtype, &count)) return 0;
  return states_bytes(m, count, H, d);
}

ADALN_API int adaln_lin_attn_fwd(
    const adaln_heads_t *q, const adaln_heads_t *k, const adaln_heads_t *v,
    const float *log_decay, float scale, const float *state,
    const adaln_heads_t *o, float *state_out, float *states,
    size_t states_size, const int64_t *seg_offsets, int64_t nseg, int64_t B,
    int64_t N, int64_t H, int64_t d, int dtype, void *stream) {
  ADALN_TRY(check_lin(log_decay, scale, seg_offsets, nseg, B, N, H, d, dtype));
  ADALN_TRY(check_part(q, B, N, H, d, dtype, false, "q"));
  ADALN_TRY(check_part(k, B, N, H, d, dtype, false, "k"));
  ADALN_TRY(check_part(v, B, N, H, d, dtype, false, "v"));
  ADALN_TRY(check_part(o, B, N, H, d, dtype, true, "o"));
  ADALN_TRY(check_ptr(state, state != nullptr, "state"));
  ADALN_TRY(check_ptr(state_out, state_out != nullptr, "state_out"));
  if (B == 0 || H == 0) return ok();
  Stretches m;
  int64_t count;
  if (!make_stretches(m, seg_offsets, nseg, B, N, H, d, dtype, &count))
    return fail(kTooMany, "too many sequences and heads");
  const size_t need = states_bytes(m, count, H, d);
  ADALN_TRY(check_workspace(states, states_size, need, "states"));
  const hipStream_t s = (hipStream_t)stream;
  const int64_t sequences = seg_offsets != nullptr ? nseg : B;
  Lin p = lin_of(log_decay, scale, H, d, count, dtype);
  p.init = state;
  p.states = need > 0 ? states : nullptr;
  p.final = state_out;
  hipError_t e = hipSuccess;
  if (need > 0) {
    p.in[0] = part_of(k, B, N, H, dtype);
    p.in[1] = part_of(v, B, N, H, dtype);
    e = make_states<false>(p, m, sequences, dtype, s);
    if (e != hipSuccess) return hip_fail(e, "adaln_lin_attn_fwd states");
  }
  p.in[0] = part_of(q, B, N, H, dtype);
  p.in[1] = part_of(k, B, N, H, dtype);
  p.in[2] = part_of(v, B, N, H, dtype);
  p.out[0] = part_of(o, B, N, H, dtype);
  e = outputs<false, 1>(p, m, 0, dtype, s);
  if (e != hipSuccess) return hip_fail(e, "adaln_lin_attn_fwd launch");
  return ok();
}

ADALN_API size_t adaln_lin_attn_bwd_workspace_bytes(
    int saved, const int64_t *seg_offsets, int64_t nseg, int64_t B, int64_t N,
    int64_t H, int64_t d, int dtype) {
  return (saved ? 1 : 2) * adaln_lin_attn_states_bytes(seg_offsets, nseg, B, N,
                                                       H, d, dtype);
}

ADALN_API int adaln_lin_attn_bwd(
    const adaln_heads_t *d_o, const adaln_heads_t *q, const adaln_heads_t *k,
    const adaln_heads_t *v, const float *log_decay, float scale,
    const float *state, const float *states, const float *dstate_out,
    const adaln_heads_t *dq, const adaln_heads_t *dk, const adaln_heads_t *dv,
    float *dstate, void *workspace, size_t workspace_bytes,
    const int64_t *seg_offsets, int64_t nseg, int64_t B, int64_t N, int64_t H,
    int64_t d, int dtype, void *stream) {
  ADALN_TRY(check_lin(log_decay, scale, seg_offsets, nseg, B, N, H, d, dtype));
  ADALN_TRY(check_part(d_o, B, N, H, d, dtype, false, "do"));
  ADALN_TRY(check_part(q, B, N, H, d, dtype, false, "q"));
  ADALN_TRY(check_part(k, B, N, H, d, dtype, false, "k"));
  ADALN_TRY(check_part(v, B, N, H, d, dtype, false, "v"));
  ADALN_TRY(check_part(dq, B, N, H, d, dtype, true, "dq"));
  ADALN_TRY(check_part(dk, B, N, H, d, dtype, true, "dk"));
  ADALN_TRY(check_part(dv, B, N, H, d, dtype, true, "dv"));
  ADALN_TRY(check_ptr(state, state != nullptr, "state"));
  ADALN_TRY(check_ptr(states, states != nullptr, "states"));
  ADALN_TRY(check_ptr(dstate_out, dstate_out != nullptr, "dstate_out"));
  ADALN_TRY(check_ptr(dstate, dstate != nullptr, "dstate"));
  if (B == 0 || H == 0) return ok();
  Stretches m;
  int64_t count;
  if (!make_stretches(m, seg_offsets, nseg, B, N, H, d, dtype, &count))
    return fail(kTooMany, "too many sequences and heads");
  const size_t one = states_bytes(m, count, H, d);
  ADALN_TRY(check_workspace(workspace, workspace_bytes,
                            one * (states != nullptr ? 1 : 2), "workspace"));
  const hipStream_t s = (hipStream_t)stream;
  const int64_t sequences = seg_offsets != nullptr ? nseg : B;
  float *ws = static_cast<float *>(workspace);
  const Part pq = part_of(q, B, N, H, dtype), pk = part_of(k, B, N, H, dtype),
             pv = part_of(v, B, N, H, dtype),
             pdo = part_of(d_o, B, N, H, dtype);
  Lin p = lin_of(log_decay, scale, H, d, count, dtype);
  hipError_t e;
  // dq, from the forward's states
  p.init = state;
  if (one > 0) {
    if (states != nullptr) {
      p.states = const_cast<float *>(states);
    } else {
      p.states = ws + one / sizeof(float);
      p.in[0] = pk;
      p.in[1] = pv;
      e = make_states<false>(p, m, sequences, dtype, s);
      if (e != hipSuccess) return hip_fail(e, "adaln_lin_attn_bwd states");
    }
  }
  p.in[0] = pdo;
  p.in[1] = pv;
  p.in[2] = pk;
  p.out[0] = part_of(dq, B, N, H, dtype);
  e = outputs<false, 1>(p, m, 1, dtype, s);
  if (e != hipSuccess) return hip_fail(e, "adaln_lin_attn_bwd dq");
  // dk and dv, from the states' gradients
  p.init = dstate_out;
  p.final = dstate;
  if (one > 0) {
    p.states = ws;
    p.in[0] = pq;
    p.in[1] = pdo;
    e = make_states<true>(p, m, sequences, dtype, s);
    if (e != hipSuccess) return hip_fail(e, "adaln_lin_attn_bwd gradients");
  }
  p.in[0] = pq;
  p.in[1] = pk;
  p.in[2] = pv;
  p.in[3] = pdo;
  p.out[0] = part_of(dv, B, N, H, dtype);
  p.out[1] = part_of(dk, B, N, H, dtype);
  e = outputs<true, 2>(p, m, 2, dtype, s);
  if (e != hipSuccess) return hip_fail(e, "adaln_lin_attn_bwd dk, dv");
  return ok();
}

ADALN_API int adaln_lin_attn_step(const adaln_heads_t *q,
                                  const adaln_heads_t *k,
                                  const adaln_heads_t *v,
                                  const float *log_decay, float scale,
                                  const float *state, const adaln_heads_t *o,
                                  float *state_out, int64_t B, int64_t H,
                                  int64_t d, int dtype, void *stream) {
  ADALN_TRY(check_lin(log_decay, scale, nullptr, 0, B, 1, H, d, dtype));
  ADALN_TRY(check_part(q, B, 1, H, d, dtype, false, "q"));
  ADALN_TRY(check_part(k, B, 1, H, d, dtype, false, "k"));
  ADALN_TRY(check_part(v, B, 1, H, d, dtype, false, "v"));
  ADALN_TRY(check_part(o, B, 1, H, d, dtype, true, "o"));
  const bool work = B > 0 && H > 0;
  ADALN_TRY(check_ptr(state, work, "state"));
  ADALN_TRY(check_ptr(state_out, work, "state_out"));
  if (!work) return ok();
  Step p = {};
  p.q = part_of(q, B, 1, H, dtype);
  p.k = part_of(k, B, 1, H, dtype);
  p.v = part_of(v, B, 1, H, dtype);
  p.o = part_of(o, B, 1, H, dtype);
  p.log_decay = log_decay;
  p.scale = scale;
  p.state = state;
  p.state_out = state_out;
  p.H = (int32_t)H;
  p.d = (int32_t)d;
  // whole rows to a workgroup, or pieces of 32 columns where that would leave
  // most CUs idle
  const int quads = (int)(d / 4);
  p.cols = B * H < kCUs ? std::min(quads, 8) : quads;
  p.groups = (quads + p.cols - 1) / p.cols;
  p.jobs = B * H * p.groups;
  const hipError_t e =
      dtype == ADALN_BF16
          ? launch_kernel(step_kernel<bf16>, p.jobs, (hipStream_t)stream, p)
          : launch_kernel(step_kernel<float>, p.jobs, (hipStream_t)stream, p);
  if (e != hipSuccess) return hip_fail(e, "adaln_lin_attn_step launch");
  return ok();
}
