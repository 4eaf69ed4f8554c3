// Rotary positions with several axes, alone and behind the RMS norm of each
// query and key head, forward and backward, with their C entry points.
//
//     angle[n, j] = sum_a pos[n, a] * freqs[a, j]          j < R / 2
//     (u, v)     -> (u cos - v sin, u sin + v cos)         for pair j
//     y = rot(x * r * w),  r = 1 / sqrt(mean_d x^2 + eps)
//     t = rot^-1(dy), g = t * w, xh = x * r
//     dx = r * (g - xh * mean_d(g * xh)),  dw = sum_{n, h} t * xh
//
// Every pass reads each head once and writes it once, so HBM bounds all of
// them; the arithmetic that could get in the way is the sines, one pair per
// (token, j), which all heads of a token share.  A workgroup therefore takes
// a block of tokens with all their heads, computes the block's sines once
// into LDS (64 pairs per token at d = 128, against 64 per head), and streams
// the heads past them.  L lanes share a head, each with two 16-byte vectors:
// in the half layout the two ends of its own pairs, so no value crosses
// lanes but the sums of the norm.
#include <algorithm>
#include <math.h>

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

constexpr int kMaxFreqs = 384;  // entries of the [axes, pairs] table
constexpr int kMaxAxes = 4;
constexpr int kMaxHead = 512;   // features per head
constexpr int kMaxTokens = 16;  // tokens per block
constexpr int kBlockRows = 4;   // rows of a block per lane group, about
constexpr int kFillBlocks = 4;  // blocks per CU before blocks get longer
constexpr int kBwdPerCu = 6;    // workgroups per CU of the norm's backward
constexpr int kSingleRows = 4;  // rows per lane group of a lone workgroup

// Frequencies in turns per unit position, as 64-bit fractions of a turn:
// pos * turns, wrapping modulo 2^64, is the phase modulo one turn with no
// loss for any position.  They travel as kernel arguments, whose size a
// launch pays for (MI355X: 11 us per call with 3.5 KiB of them, 3.8 with
// the small form), so the usual case, up to 64 pairs turned by one axis
// each, has a form of its own.
struct OneAxis {
  static constexpr int kPairs = 64;
  uint64_t turns[kPairs];
  uint8_t axis[kPairs];
  __device__ __forceinline__ uint64_t phase(const int32_t *pos, int j, int,
                                            int) const {
    return (uint64_t)(int64_t)pos[axis[j]] * turns[j];
  }
};

struct AllAxes {
  uint64_t turns[kMaxFreqs];  // [axes, pairs]
  __device__ __forceinline__ uint64_t phase(const int32_t *pos, int j,
                                            int axes, int pairs) const {
    uint64_t p = 0;
    for (int a = 0; a < axes; ++a)
      p += (uint64_t)(int64_t)pos[a] * turns[a * pairs + j];
    return p;
  }
};

// One tensor's heads: strides in 16-byte vectors.
struct Heads {
  const char *data;
  int64_t batch;
  int64_t token;
  int32_t head;
};

struct Job {
  Heads in[2];            // x (rope: the tensor to rotate), of q and of k
  Heads dy[2];            // backward of the norm only
  Heads out[2];
  const void *w[2];       // norm weights
  float *part[2];         // backward: partial rows of dw, [workgroups, d]
  const int32_t *pos;
  int64_t pos_batch;      // elements
  int32_t H[2];
  uint32_t magic[2];      // ceil(2^32 / H)
  int32_t grid_q;         // workgroups of q; the rest are k's
  int32_t N;
  int32_t d;
  int32_t nvec;           // vectors per head
  int32_t rot_vecs;       // half layout: vectors of the first half's pairs
  int32_t tb;             // tokens per block
  int32_t blocks_n;       // blocks per sample
  int64_t blocks;
  int32_t cached;         // plain loads (else the streaming hint)
  float eps;
  float inv_d;
  float dir;              // +1: by the angle, -1: by the negative angle
  int32_t axes;
  int32_t pairs;
};

// cos and sin of a phase given as a 64-bit fraction of a turn, which is taken
// to the nearest quarter turn.  What remains, at most pi/4, is converted as a
// signed whole number, so that small angles keep all their digits, and goes
// through the Taylor polynomials of degree 9 and 10 (truncation below 2e-9 and
// 2e-10): both results are within 4 * 2^-24 of themselves.  (Of the phase
// itself the frequencies' last place is uncertain, half of 2^-64 turns per
// unit position.  Once per pair and token of a block: the conversion from 64
// bits costs nothing that can be measured.)
__device__ __forceinline__ void cos_sin(uint64_t phase, float &c, float &s) {
  const uint32_t quarter = (uint32_t)((phase + (uint64_t(1) << 61)) >> 62);
  const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));
  // 2 pi / 2^64, and what float32 leaves of it
  constexpr double kTurn = 6.283185307179586 / 18446744073709551616.0;
  constexpr float kHi = (float)kTurn, kLo = (float)(kTurn - (double)kHi);
  const float f = (float)rest;
  const float x = fmaf(f, kHi, f * kLo);
  const float x2 = x * x;
  float a = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  a = fmaf(x2, a, 8.3333333e-3f);
  a = fmaf(x2, a, -1.6666667e-1f);
  const float sn = fmaf(x * x2, a, x);
  float b = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  b = fmaf(x2, b, -1.3888889e-3f);
  b = fmaf(x2, b, 4.1666667e-2f);
  b = fmaf(x2, b, -0.5f);
  const float cs = fmaf(x2, b, 1.0f);
  const float u = (quarter & 1) ? sn : cs;
  const float v = (quarter & 1) ? cs : sn;
  c = ((quarter + 1) & 2) ? -u : u;
  s = (quarter & 2) ? -v : v;
}

// Sum over the L lanes that share a head (L a power of two, the lanes
// aligned to it), in a fixed order; every lane gets it.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L >= 2) v = dpp_add<0xB1>(v);
  if constexpr (L >= 4) v = dpp_add<0x4E>(v);
  if constexpr (L >= 8) v = dpp_add<0x141>(v);
  if constexpr (L >= 16) v = dpp_add<0x140>(v);
  if constexpr (L >= 32) v += __shfl_xor(v, 16);
  if constexpr (L >= 64) v += __shfl_xor(v, 32);
  return v;
}

// The two vectors of a head that a lane holds.  Interleaved: vectors slot and
// slot + ceil(nvec / 2).  Half: the rot_vecs slots of rotated pairs hold
// vectors slot and slot + rot_vecs, the rest of the head follows.
template <bool HALF>
__device__ __forceinline__ void slot_vectors(const Job &job, int slot, int &a,
                                             int &b) {
  if constexpr (HALF) {
    const int rv = job.rot_vecs;
    if (slot < rv) {
      a = slot;
      b = slot + rv;
    } else {
      a = rv + slot;
      b = a + (job.nvec - 2 * rv + 1) / 2;
    }
  } else {
    a = slot;
    b = slot + (job.nvec + 1) / 2;
  }
}

// Rotates the lane's 2 * E values; cs: its E (cos, sin) entries.
template <int E, bool HALF>
__device__ __forceinline__ void rotate_all(float (&xa)[E], float (&xb)[E],
                                           const float2 (&cs)[E]) {
  if constexpr (HALF) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float u = xa[i], v = xb[i];
      xa[i] = u * cs[i].x - v * cs[i].y;
      xb[i] = u * cs[i].y + v * cs[i].x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      float u = xa[2 * i], v = xa[2 * i + 1];
      xa[2 * i] = u * cs[i].x - v * cs[i].y;
      xa[2 * i + 1] = u * cs[i].y + v * cs[i].x;
      u = xb[2 * i], v = xb[2 * i + 1];
      xb[2 * i] = u * cs[E / 2 + i].x - v * cs[E / 2 + i].y;
      xb[2 * i + 1] = u * cs[E / 2 + i].y + v * cs[E / 2 + i].x;
    }
  }
}

// How many pairs of the lane's vectors are rotated (half layout: those of
// both vectors together), and whether any feature of the head is not.
struct Part {
  bool some;
  int a, b;
  template <int E, bool HALF>
  __device__ __forceinline__ bool rotated(bool second, int i) const {
    return HALF ? a > 0 : i / 2 < (second ? b : a);
  }
};

// Rotates those of the values that are.  The others keep theirs: a rotation
// by no angle is u * 1 - v * 0, which takes an infinite or undefined v, and
// the sign of a zero, to u.  BRANCH: whole heads rotated go past the selection;
// it pays in the norm's backward, which issues more than it loads (MI355X,
// 75600 x 80 heads of 128 bf16, 801 us against 820), and not in its forward
// (3554 x 15 heads of 72 f32, 64 of them rotated, 9.9 us against 9.1).
template <int E, bool HALF, bool BRANCH>
__device__ __forceinline__ void rotate(float (&xa)[E], float (&xb)[E],
                                       const float2 (&cs)[E],
                                       const Part &part) {
  if (BRANCH && !part.some) {
    rotate_all<E, HALF>(xa, xb, cs);
    return;
  }
  float ra[E], rb[E];
#pragma unroll
  for (int i = 0; i < E; ++i) ra[i] = xa[i], rb[i] = xb[i];
  rotate_all<E, HALF>(ra, rb, cs);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (part.rotated<E, HALF>(false, i)) xa[i] = ra[i];
    if (part.rotated<E, HALF>(true, i)) xb[i] = rb[i];
  }
}

// The vector y of a rotation of x with the bits of x where it is not rotated
// (a conversion to float and back would make a signalling NaN a quiet one).
template <int E, bool HALF>
__device__ __forceinline__ void keep_bits(Vec &y, const Vec &x,
                                          const Part &part, bool second) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!part.rotated<E, HALF>(second, i * (E / 4))) y.w[i] = x.w[i];
}

enum { kRope = 0, kNormFwd = 1, kNormBwd = 2 };

// A lane's part of one row (a head of a token of the block): its vectors of
// x, and of dy in the backward of the norm.
struct Row {
  Vec xa, xb, ya, yb;
  int tok, head;
  bool live;
};

// A block of tokens: tb of them (fewer at a sample's end) from n0 of sample b.
struct Block {
  int b, n0, tb;
  __device__ __forceinline__ Block(const Job &job, int64_t blk) {
    // (fewer than 2^31 blocks: as many tokens)
    b = (int)((uint32_t)blk / (uint32_t)job.blocks_n);
    n0 = ((int)blk - b * job.blocks_n) * job.tb;
    tb = min(job.tb, job.N - n0);
  }
  __device__ __forceinline__ int64_t at(const Heads &h, int tok,
                                        int head) const {
    return (b * h.batch + (int64_t)(n0 + tok) * h.token +
            (int64_t)head * h.head) * 16;
  }
};

template <typename T, int L, bool HALF, int OP, typename ROT>
__global__ __launch_bounds__(kBlock) void heads_kernel(Job job, ROT rot) {
  constexpr int E = Elems<T>::value;
  constexpr int kRows = kBlock / L;   // heads a workgroup takes at a time
  constexpr int kPitch = L * E;       // table entries per token
  extern __shared__ float2 tables[];  // 2 x [tb][kPitch]
  const int tid = threadIdx.x;
  const int slot = tid % L;
  const int group = tid / L;
  int va, vb;
  slot_vectors<HALF>(job, slot, va, vb);
  const bool ok_a = va < job.nvec && slot < (job.nvec + 1) / 2;
  const bool ok_b = ok_a && vb < job.nvec;
  if (!ok_a) va = 0;
  if (!ok_b) vb = va;
  // entries of the lane's pairs in the table's row of a token
  const int ta = HALF ? slot * E : (ok_a ? va : 0) * (E / 2);
  const int tbl = HALF ? slot * E + E / 2 : (ok_b ? vb : 0) * (E / 2);

  // half layout: slots of rotated pairs, and the others
  const Part part = {2 * job.pairs < job.d,
                     HALF ? slot < job.rot_vecs : job.pairs - ta,
                     HALF ? 0 : job.pairs - tbl};

  // the workgroups of q, then those of k
  const int t = blockIdx.x >= job.grid_q;
  const int wg = blockIdx.x - (t ? job.grid_q : 0);
  const int wgs = t ? gridDim.x - job.grid_q : job.grid_q;
  const int H = job.H[t];
  const uint32_t magic = job.magic[t];
  const Heads in = job.in[t], out = job.out[t];

  float w[OP == kRope ? 1 : 2 * E];
  if constexpr (OP != kRope) {
    const Vec wa = load_vec((const char *)job.w[t] + va * 16);
    const Vec wb = load_vec((const char *)job.w[t] + vb * 16);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      w[i] = elem<T>(wa, i);
      w[E + i] = elem<T>(wb, i);
    }
  }
  float acc[OP == kNormBwd ? 2 * E : 1] = {};

  auto load = [&](const Block &k, int row0) {
    Row r;
    r.live = row0 + group < k.tb * H;
    const int row = r.live ? row0 + group : 0;
    r.tok = H == 1 ? row : (int)__umulhi((uint32_t)row, magic);
    r.head = row - r.tok * H;
    const char *src = in.data + k.at(in, r.tok, r.head);
    const char *dy = nullptr;
    if constexpr (OP == kNormBwd)
      dy = job.dy[t].data + k.at(job.dy[t], r.tok, r.head);
    if (job.cached) {
      r.xa = load_vec(src + va * 16);
      r.xb = load_vec(src + vb * 16);
      if constexpr (OP == kNormBwd) {
        r.ya = load_vec(dy + va * 16);
        r.yb = load_vec(dy + vb * 16);
      }
    } else {
      r.xa = load_stream(src + va * 16);
      r.xb = load_stream(src + vb * 16);
      if constexpr (OP == kNormBwd) {
        r.ya = load_stream(dy + va * 16);
        r.yb = load_stream(dy + vb * 16);
      }
    }
    return r;
  };
  // the sines of a block's tokens; the entries past the rotated pairs' are
  // read, but not used
  auto sines = [&](const Block &k, float2 *table) {
    const int32_t *pos =
        job.pos + k.b * job.pos_batch + (int64_t)k.n0 * job.axes;
    for (int i = tid; i < k.tb * kPitch; i += kBlock) {
      const int tok = i / kPitch;
      const int j = i % kPitch;
      float2 cs = {1.f, 0.f};
      if (j < job.pairs) {
        cos_sin(rot.phase(pos + tok * job.axes, j, job.axes, job.pairs), cs.x,
                cs.y);
        cs.y *= job.dir;
      }
      table[i] = cs;
    }
  };

  // One barrier per block: the sines of the next one go to the other half of
  // the table, and its first rows are on their way, before the present one is
  // done.
  Block k(job, wg);
  Row next = load(k, 0);
  sines(k, tables);
  int half = 0;
  for (int64_t blk = wg; blk < job.blocks; blk += wgs) {
    const float2 *table = tables + half * job.tb * kPitch;
    half ^= 1;
    __syncthreads();
    const bool more = blk + wgs < job.blocks;
    const Block after(job, more ? blk + wgs : blk);
    if (more) sines(after, tables + half * job.tb * kPitch);
    const int rows = k.tb * H;
    for (int row0 = 0; row0 < rows; row0 += kRows) {
      Row r = next;
      if (row0 + kRows < rows)
        next = load(k, row0 + kRows);
      else if (more)
        next = load(after, 0);
      float2 cs[E];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        cs[i] = table[r.tok * kPitch + ta + i];
        cs[E / 2 + i] = table[r.tok * kPitch + tbl + i];
      }
      if (!ok_a) r.xa = vzero(), r.ya = vzero();
      if (!ok_b) r.xb = vzero(), r.yb = vzero();
      float fa[E], fb[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        fa[i] = elem<T>(r.xa, i);
        fb[i] = elem<T>(r.xb, i);
      }
      if constexpr (OP != kRope) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(fa[i], fa[i], ss);
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(fb[i], fb[i], ss);
        if constexpr (OP == kNormFwd) {
          ss = lanes_sum<L>(ss);
          const float s = rsqrtf(fmaf(ss, job.inv_d, job.eps));
#pragma unroll
          for (int i = 0; i < E; ++i) {
            fa[i] = fa[i] * s * w[i];
            fb[i] = fb[i] * s * w[E + i];
          }
          rotate<E, HALF, false>(fa, fb, cs, part);
        } else {
          float ga[E], gb[E];
#pragma unroll
          for (int i = 0; i < E; ++i) {
            ga[i] = elem<T>(r.ya, i);
            gb[i] = elem<T>(r.yb, i);
          }
          rotate<E, HALF, true>(ga, gb, cs, part);
          // t * x is what both sums need
          float pa[E], pb[E], sg = 0.f;
#pragma unroll
          for (int i = 0; i < E; ++i) {
            pa[i] = ga[i] * fa[i];
            pb[i] = gb[i] * fb[i];
            sg = fmaf(pa[i], w[i], sg);
            sg = fmaf(pb[i], w[E + i], sg);
          }
          ss = lanes_sum<L>(ss);
          sg = lanes_sum<L>(sg);
          const float s = rsqrtf(fmaf(ss, job.inv_d, job.eps));
          const float m = sg * s * s * job.inv_d;  // r * mean(g * xh)
          if (r.live) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
              acc[i] = fmaf(pa[i], s, acc[i]);
              acc[E + i] = fmaf(pb[i], s, acc[E + i]);
            }
          }
#pragma unroll
          for (int i = 0; i < E; ++i) {
            fa[i] = s * (ga[i] * w[i] - fa[i] * m);
            fb[i] = s * (gb[i] * w[E + i] - fb[i] * m);
          }
        }
      } else {
        rotate_all<E, HALF>(fa, fb, cs);
      }
      char *dst = const_cast<char *>(out.data) + k.at(out, r.tok, r.head);
      Vec oa = pack<T>(fa), ob = pack<T>(fb);
      if constexpr (OP == kRope) {
        if (part.some) {
          keep_bits<E, HALF>(oa, r.xa, part, false);
          keep_bits<E, HALF>(ob, r.xb, part, true);
        }
      }
      if (r.live && ok_a) store_stream(dst + va * 16, oa);
      if (r.live && ok_b) store_stream(dst + vb * 16, ob);
    }
    k = after;
  }

  // One partial row of dw per workgroup: the lane groups of a wavefront are
  // added by a butterfly, the four wavefronts in order through LDS.
  if constexpr (OP == kNormBwd) {
    __shared__ float stage[4][2 * L * E];
    const int wave = wave_id();
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) {
      float v = acc[i];
#pragma unroll
      for (int o = L; o < kWave; o *= 2) v += __shfl_xor(v, o);
      const bool ok = i < E ? ok_a : ok_b;
      if (ok && lane_id() < L) stage[wave][(i < E ? va : vb) * E + i % E] = v;
    }
    __syncthreads();
    float *part = job.part[t] + (int64_t)wg * job.d;
    for (int c = tid; c < job.d; c += kBlock)
      part[c] = ((stage[0][c] + stage[1][c]) + stage[2][c]) + stage[3][c];
  }
}

// dw = the sum of a tensor's partial rows, in a fixed order: slice s of 64
// adds rows s, s + 64, ..., then the slices are added in order.  A workgroup
// per tensor and 16 features; zero where there are no rows.
constexpr int kSumSlices = 64;
constexpr int kSumCols = 16;

struct Sums {
  const float *part[2];
  float *dw[2];
  int32_t rows[2];
  int32_t d;
};

__global__ __launch_bounds__(kSumSlices * kSumCols) void sum_kernel(Sums p) {
  __shared__ float stage[kSumSlices][kSumCols];
  const int per = (p.d + kSumCols - 1) / kSumCols;
  const int t = blockIdx.x / per;
  if (p.dw[t] == nullptr) return;
  const int c = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const int f = (blockIdx.x - t * per) * kSumCols + c;
  float v = 0.f;
  if (f < p.d) {
    const float *src = p.part[t] + f;
    int r = slice;
    for (; r + 3 * kSumSlices < p.rows[t]; r += 4 * kSumSlices) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = src[(int64_t)(r + i * kSumSlices) * p.d];
#pragma unroll
      for (int i = 0; i < 4; ++i) v += x[i];
    }
    for (; r < p.rows[t]; r += kSumSlices) v += src[(int64_t)r * p.d];
  }
  stage[slice][c] = v;
  __syncthreads();
  if (slice == 0 && f < p.d) {
    for (int s = 1; s < kSumSlices; ++s) v += stage[s][c];
    p.dw[t][f] = v;
  }
}

// ------------------------------------------------------------------- checks

int elems_per_vec(int dtype) { return dtype == ADALN_BF16 ? 8 : 4; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

int check_sizes(int64_t B, int64_t N, int64_t Hq, int64_t Hk, int64_t d,
                int dtype) {
  if (dtype != ADALN_F32 && dtype != ADALN_BF16)
    return fail(ADALN_ERR_DTYPE, "unknown dtype code %d", dtype);
  if (B < 0 || N < 0 || Hq < 0 || Hk < 0)
    return fail(ADALN_ERR_INVALID, "negative size: B=%lld N=%lld Hq=%lld Hk=%lld",
                (long long)B, (long long)N, (long long)Hq, (long long)Hk);
  if (d <= 0)
    return fail(ADALN_ERR_INVALID, "d must be positive, got %lld", (long long)d);
  const int E = elems_per_vec(dtype);
  if (d % E != 0)
    return fail(ADALN_ERR_ALIGN, "d=%lld is not a multiple of %d", (long long)d, E);
  if (d > kMaxHead)
    return fail(ADALN_ERR_UNSUPPORTED, "d=%lld exceeds the widest head (%d)",
                (long long)d, kMaxHead);
  if (Hq > 4096 || Hk > 4096)
    return fail(ADALN_ERR_INVALID, "more than 4096 heads");
  if (B > kMaxRows || N > kMaxRows || (N > 0 && B > kMaxRows / N))
    return fail(ADALN_ERR_INVALID, "B*N exceeds 2^31-1 tokens");
  return ADALN_OK;
}

int check_rotation(const adaln_rotation_t *rot, int64_t d, int dtype,
                   bool rows) {
  if (rot == nullptr) return fail(ADALN_ERR_INVALID, "rot is NULL");
  if (rot->axes < 1 || rot->axes > kMaxAxes)
    return fail(ADALN_ERR_INVALID, "axes must be 1 to %d, got %d", kMaxAxes,
                rot->axes);
  if (rot->pairs < 1 || 2 * (int64_t)rot->pairs > d)
    return fail(ADALN_ERR_INVALID, "pairs must be 1 to d/2, got %d", rot->pairs);
  if ((int64_t)rot->axes * rot->pairs > kMaxFreqs)
    return fail(ADALN_ERR_UNSUPPORTED, "axes*pairs exceeds %d", kMaxFreqs);
  if (rot->layout != ADALN_ROPE_INTERLEAVED && rot->layout != ADALN_ROPE_HALF)
    return fail(ADALN_ERR_INVALID, "unknown layout %d", rot->layout);
  if (rot->layout == ADALN_ROPE_HALF && rot->pairs % elems_per_vec(dtype) != 0)
    return fail(ADALN_ERR_ALIGN,
                "half layout: pairs=%d is not a multiple of %d", rot->pairs,
                elems_per_vec(dtype));
  if (rot->pos_batch_stride < 0 || rot->pos_batch_stride % rot->axes != 0)
    return fail(ADALN_ERR_INVALID, "bad pos_batch_stride %lld",
                (long long)rot->pos_batch_stride);
  if (rot->freqs == nullptr) return fail(ADALN_ERR_INVALID, "freqs is NULL");
  for (int i = 0; i < rot->axes * rot->pairs; ++i)
    if (!(fabs(rot->freqs[i]) <= 1e6))
      return fail(ADALN_ERR_INVALID, "freqs[%d] is not within 1e6", i);
  if (rows && rot->pos == nullptr)
    return fail(ADALN_ERR_INVALID, "pos is NULL");
  if (rows && reinterpret_cast<uintptr_t>(rot->pos) % 4 != 0)
    return fail(ADALN_ERR_ALIGN, "pos is not 4-byte aligned");
  return ADALN_OK;
}

// One tensor: pointer, alignment, strides; an output's rows must not overlap.
int check_heads(const adaln_heads_t *t, int64_t B, int64_t N, int64_t H,
                int64_t d, int dtype, bool output, const char *name) {
  if (B * N == 0 || H == 0) return ADALN_OK;
  if (t == nullptr || t->data == nullptr)
    return fail(ADALN_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0)
    return fail(ADALN_ERR_ALIGN, "%s is not 16-byte aligned", name);
  const int E = elems_per_vec(dtype);
  struct Dim {
    int64_t stride, size;
  } dim[3] = {{t->head_stride, H}, {t->token_stride, N}, {t->batch_stride, B}};
  for (Dim &s : dim) {
    if (s.size == 1) s.stride = 0;
    if (s.stride < 0 || s.stride > (int64_t(1) << 40))
      return fail(ADALN_ERR_INVALID, "%s has a stride of %lld", name,
                  (long long)s.stride);
    if (s.stride % E != 0)
      return fail(ADALN_ERR_ALIGN,
                  "%s has a stride that is not a multiple of %d", name, E);
  }
  if (dim[0].stride / E >= (int64_t(1) << 31))
    return fail(ADALN_ERR_UNSUPPORTED, "%s: heads too far apart", name);
  if (output) {
    std::sort(dim, dim + 3,
              [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    int64_t extent = d;
    for (const Dim &s : dim) {
      if (s.size == 1) continue;
      if (s.stride < extent)
        return fail(ADALN_ERR_INVALID, "%s: heads overlap", name);
      extent += s.stride * (s.size - 1);
    }
  }
  return ADALN_OK;
}

// ---------------------------------------------------------------- launching

Heads heads_of(const adaln_heads_t *t, int64_t B, int64_t N, int64_t H,
               int dtype) {
  Heads h = {};
  if (t == nullptr || H == 0) return h;
  const int E = elems_per_vec(dtype);
  h.data = static_cast<const char *>(t->data);
  h.batch = B > 1 ? t->batch_stride / E : 0;
  h.token = N > 1 ? t->token_stride / E : 0;
  h.head = H > 1 ? (int32_t)(t->head_stride / E) : 0;
  return h;
}

int lanes_per_head(int nvec) {
  int L = 1;
  while (2 * L < nvec) L *= 2;
  return L;
}

struct HeadsPlan {
  int tb;            // tokens per block
  int64_t blocks_n;  // blocks per sample
  int64_t blocks;
  int64_t grid[2];   // workgroups of q and of k
  // backward of so few rows that a workgroup per tensor takes them all, whose
  // partial row is dw itself: no workspace and no second launch (MI355X, 24
  // heads of 128, in a graph: 1 token 5.0 us, 8 tokens 7.1, 16 tokens 10.2;
  // with the second launch 7.3 from 22 tokens on)
  bool single;
};

// A block has up to kBlockRows rows for each lane group of a workgroup, and
// fewer where the GPU would not be filled: short blocks keep the window of
// memory that is read and written at a time small.  Measured on MI355X (bf16,
// 128 features): 32760 tokens x 24 heads rotated, 16 tokens per block 78.4
// us, 8 (96 rows of 32 lane groups) 72.2; norm and rotation of 75600 x 80
// heads, 16 tokens 590 us, 4 (160 rows) 546, 2 (80 rows) 508.
// The backward of the norm runs a persistent grid, so that each workgroup
// adds up dw over many blocks before it writes its partial row: 6 per CU,
// twice what its registers admit at a time in bf16, evens out the end (75600 x
// 80 heads: 3 per CU 815 us, 6 per CU 800; f32, 24960 x 24 heads, where a CU
// holds 4: 160 and 170).  q and k share it by their numbers of heads.
HeadsPlan heads_plan(int64_t B, int64_t N, int64_t Hq, int64_t Hk, int64_t d,
                     int dtype, bool bwd) {
  HeadsPlan p = {};
  const int lanes = lanes_per_head((int)(d / elems_per_vec(dtype)));
  const int rows = kBlock / lanes;
  // both halves of the table of sines within 32 KiB of LDS
  const int fits = 32768 / (2 * lanes * elems_per_vec(dtype) * 8);
  const int tensors = (Hq > 0) + (Hk > 0);
  p.tb = kMaxTokens;
  while (p.tb > 1 && (p.tb > fits ||
                      p.tb * std::max(Hq, Hk) > kBlockRows * rows ||
                      tensors * B * ((N + p.tb - 1) / p.tb) <
                          kFillBlocks * kCUs))
    p.tb /= 2;
  p.single = bwd && B * N * std::max(Hq, Hk) <= kSingleRows * rows;
  if (p.single) p.tb = std::min(kMaxTokens, fits);
  p.blocks_n = (N + p.tb - 1) / p.tb;
  p.blocks = B * p.blocks_n;
  if (p.single) {
    p.grid[0] = Hq > 0;
    p.grid[1] = Hk > 0;
    return p;
  }
  const int64_t most = bwd ? kBwdPerCu * kCUs : kMaxGrid;
  const int64_t all = std::min(most, tensors * p.blocks);
  p.grid[0] = Hq == 0 ? 0 : Hk == 0 ? all : all * Hq / (Hq + Hk);
  if (Hq > 0) p.grid[0] = std::max<int64_t>(1, std::min(p.grid[0], p.blocks));
  p.grid[1] = Hk == 0 ? 0
                      : std::max<int64_t>(
                            1, std::min(all - p.grid[0], p.blocks));
  return p;
}

// Inputs that another kernel has just written or read may still lie in the
// 256 MB Infinity Cache; the streaming hint reads past it.  Up to twice its
// size of bytes read and written a call takes plain loads, past it the hint.
// MI355X, bf16, heads of 128, three sets of inputs and outputs in turn, plain
// loads against the hint: rotation of 10000 x 24 (122 MB) 20.7 against 25.2 us,
// 24960 x 24 (307 MB) 56.4 and 55.2, 32760 x 24 (402 MB) 72.2 and 71.1, 90000 x
// 24 (1.1 GB) 192 and 184.  Alone the hint would win from 300 MB on, by 2%; but
// the backward of the norm of 24960 x 24 heads (460 MB) comes right behind its
// forward, and the two take 139 us with plain loads, 143 with the hint (by
// itself 92 and 89; 75600 x 80 heads, 4.6 GB, 856 and 812).  One bound for all
// of them costs the rotations those 2%.  (Plain stores of the outputs were
// slower from 100 MB on, but for outputs written over again while the cache
// still held them.)
constexpr int64_t kCachedBytes = int64_t(512) << 20;

void fill_job(Job &job, const HeadsPlan &p, const adaln_rotation_t *rot,
              bool inverse, int tensors, int64_t B, int64_t N, int64_t Hq,
              int64_t Hk, int64_t d, int dtype) {
  const int E = elems_per_vec(dtype);
  const int64_t H[2] = {Hq, Hk};
  for (int t = 0; t < 2; ++t) {
    job.H[t] = (int32_t)H[t];
    // exact quotients for rows < 16 * 4096 = 2^16: the error of the quotient,
    // row * H / 2^32, stays below 1 / H
    job.magic[t] =
        H[t] > 1 ? (uint32_t)(((uint64_t(1) << 32) + H[t] - 1) / H[t]) : 0;
  }
  job.pos = rot->pos;
  job.pos_batch = rot->pos_batch_stride;
  job.N = (int32_t)N;
  job.d = (int32_t)d;
  job.nvec = (int32_t)(d / E);
  job.rot_vecs = rot->layout == ADALN_ROPE_HALF ? rot->pairs / E : 0;
  job.tb = p.tb;
  job.grid_q = (int32_t)p.grid[0];
  job.blocks_n = (int32_t)p.blocks_n;
  job.blocks = p.blocks;
  job.cached = B * N * (Hq + Hk) * d * (16 / E) * tensors <= kCachedBytes;
  job.dir = inverse ? -1.f : 1.f;
  job.axes = rot->axes;
  job.pairs = rot->pairs;
}

// Radians per unit position -> turns, modulo 1, in 64 bits.  The double's 53
// bits times 1 / (2 pi) to 128 bits, in integers: the fraction of a turn is
// within a unit of its last place (and a call turns up to 384 of these).
uint64_t turns_of(double radians) {
  // floor(2^128 / (2 pi))
  constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;
  const uint64_t bits = __builtin_bit_cast(uint64_t, radians);
  const int e = (int)(bits >> 52 & 0x7ff) - 1022;
  if (e < -70) return 0;  // (subnormal ones among them)
  // |radians| = m 2^(e - 53)
  const uint64_t m = (bits & ((uint64_t(1) << 52) - 1)) | uint64_t(1) << 52;
  // turns * 2^64 = m (kHi:kLo) 2^(e - 53 - 64), so the upper 128 bits of the
  // product, to the right by 53 - e: at least 33, as |radians| <= 1e6
  typedef unsigned __int128 u128;
  const u128 t = (u128)m * kHi + (uint64_t)(((u128)m * kLo) >> 64);
  const int shift = 53 - e;
  const uint64_t f = (uint64_t)((t >> shift) + ((t >> (shift - 1)) & 1));
  return radians < 0 ? ~f + 1 : f;
}

// The small form, where it holds the rotation.
bool fill(OneAxis &r, const adaln_rotation_t *rot) {
  if (rot->pairs > OneAxis::kPairs) return false;
  for (int j = 0; j < rot->pairs; ++j) {
    int axis = -1;
    for (int a = 0; a < rot->axes; ++a)
      if (rot->freqs[a * rot->pairs + j] != 0) {
        if (axis >= 0) return false;
        axis = a;
      }
    r.axis[j] = (uint8_t)std::max(axis, 0);
    r.turns[j] =
        axis < 0 ? 0 : turns_of(rot->freqs[axis * rot->pairs + j]);
  }
  return true;
}

void fill(AllAxes &r, const adaln_rotation_t *rot) {
  for (int i = 0; i < rot->axes * rot->pairs; ++i)
    r.turns[i] = turns_of(rot->freqs[i]);
}

template <typename T, int OP, int L, typename ROT>
hipError_t go(const Job &job, const ROT &rot, bool half, int64_t grid,
              hipStream_t stream) {
  const size_t lds =
      (size_t)2 * job.tb * L * Elems<T>::value * sizeof(float2);
  return half ? launch_kernel_lds(heads_kernel<T, L, true, OP, ROT>, grid,
                                  kBlock, lds, stream, job, rot)
              : launch_kernel_lds(heads_kernel<T, L, false, OP, ROT>, grid,
                                  kBlock, lds, stream, job, rot);
}

template <typename T, int OP, typename ROT>
hipError_t launch_heads(const Job &job, const ROT &rot, bool half,
                        int64_t grid, hipStream_t stream) {
  switch (lanes_per_head(job.nvec)) {
    case 1: return go<T, OP, 1>(job, rot, half, grid, stream);
    case 2: return go<T, OP, 2>(job, rot, half, grid, stream);
    case 4: return go<T, OP, 4>(job, rot, half, grid, stream);
    case 8: return go<T, OP, 8>(job, rot, half, grid, stream);
    case 16: return go<T, OP, 16>(job, rot, half, grid, stream);
    case 32: return go<T, OP, 32>(job, rot, half, grid, stream);
    default:
      if constexpr (Elems<T>::value == 4)
        return go<T, OP, 64>(job, rot, half, grid, stream);
      return hipErrorInvalidValue;
  }
}

int hip_fail(hipError_t e, const char *what) {
  return fail(ADALN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

template <int OP>
int enqueue(const Job &job, const adaln_rotation_t *rot, int64_t grid,
            int dtype, hipStream_t stream, const char *what) {
  const bool half = rot->layout == ADALN_ROPE_HALF;
  auto run = [&](const auto &r) {
    return dtype == ADALN_BF16 ? launch_heads<bf16, OP>(job, r, half, grid,
                                                        stream)
                               : launch_heads<float, OP>(job, r, half, grid,
                                                         stream);
  };
  OneAxis one;
  hipError_t e;
  if (fill(one, rot)) {
    e = run(one);
  } else {
    AllAxes all;
    fill(all, rot);
    e = run(all);
  }
  return e == hipSuccess ? ADALN_OK : hip_fail(e, what);
}

int check_weight(const void *w, bool needed, const char *name) {
  if (!needed) return ADALN_OK;
  if (w == nullptr) return fail(ADALN_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(w) % 16 != 0)
    return fail(ADALN_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return ADALN_OK;
}

int rope(const adaln_heads_t *q, const adaln_heads_t *k,
         const adaln_rotation_t *rot, const adaln_heads_t *q_out,
         const adaln_heads_t *k_out, bool inverse, int64_t B, int64_t N,
         int64_t Hq, int64_t Hk, int64_t d, int dtype, void *stream,
         const char *what) {
  ADALN_TRY(check_sizes(B, N, Hq, Hk, d, dtype));
  const bool rows = B * N > 0 && Hq + Hk > 0;
  ADALN_TRY(check_rotation(rot, d, dtype, rows));
  ADALN_TRY(check_heads(q, B, N, Hq, d, dtype, false, "q"));
  ADALN_TRY(check_heads(k, B, N, Hk, d, dtype, false, "k"));
  ADALN_TRY(check_heads(q_out, B, N, Hq, d, dtype, true, "q_out"));
  ADALN_TRY(check_heads(k_out, B, N, Hk, d, dtype, true, "k_out"));
  if (!rows) return ok();
  const HeadsPlan p = heads_plan(B, N, Hq, Hk, d, dtype, false);
  Job job = {};
  fill_job(job, p, rot, inverse, 2, B, N, Hq, Hk, d, dtype);
  job.in[0] = heads_of(q, B, N, Hq, dtype);
  job.in[1] = heads_of(k, B, N, Hk, dtype);
  job.out[0] = heads_of(q_out, B, N, Hq, dtype);
  job.out[1] = heads_of(k_out, B, N, Hk, dtype);
  ADALN_TRY(enqueue<kRope>(job, rot, p.grid[0] + p.grid[1], dtype,
                           (hipStream_t)stream, what));
  return ok();
}

}  // namespace
}  // namespace adaln

using namespace adaln;

ADALN_API int adaln_rope_fwd(const adaln_heads_t *q, const adaln_heads_t *k,
                             const adaln_rotation_t *rot,
                             const adaln_heads_t *q_out,
                             const adaln_heads_t *k_out, int64_t B, int64_t N,
                             int64_t Hq, int64_t Hk, int64_t d, int dtype,
                             void *stream) {
  return rope(q, k, rot, q_out, k_out, false, B, N, Hq, Hk, d, dtype, stream,
              "adaln_rope_fwd launch");
}

ADALN_API int adaln_rope_bwd(const adaln_heads_t *dq_out,
                             const adaln_heads_t *dk_out,
                             const adaln_rotation_t *rot,
                             const adaln_heads_t *dq, const adaln_heads_t *dk,
                             int64_t B, int64_t N, int64_t Hq, int64_t Hk,
                             int64_t d, int dtype, void *stream) {
  return rope(dq_out, dk_out, rot, dq, dk, true, B, N, Hq, Hk, d, dtype,
              stream, "adaln_rope_bwd launch");
}

ADALN_API int adaln_qk_norm_rope_fwd(
    const adaln_heads_t *q, const adaln_heads_t *k, const void *wq,
    const void *wk, float eps, const adaln_rotation_t *rot,
    const adaln_heads_t *q_out, const adaln_heads_t *k_out, int64_t B,
    int64_t N, int64_t Hq, int64_t Hk, int64_t d, int dtype, void *stream) {
  ADALN_TRY(check_sizes(B, N, Hq, Hk, d, dtype));
  const bool rows = B * N > 0 && Hq + Hk > 0;
  if (!(eps >= 0.f) || isinf(eps))
    return fail(ADALN_ERR_INVALID, "eps must be finite and not negative");
  ADALN_TRY(check_rotation(rot, d, dtype, rows));
  ADALN_TRY(check_heads(q, B, N, Hq, d, dtype, false, "q"));
  ADALN_TRY(check_heads(k, B, N, Hk, d, dtype, false, "k"));
  ADALN_TRY(check_heads(q_out, B, N, Hq, d, dtype, true, "q_out"));
  ADALN_TRY(check_heads(k_out, B, N, Hk, d, dtype, true, "k_out"));
  ADALN_TRY(check_weight(wq, rows && Hq > 0, "wq"));
  ADALN_TRY(check_weight(wk, rows && Hk > 0, "wk"));
  if (!rows) return ok();
  const HeadsPlan p = heads_plan(B, N, Hq, Hk, d, dtype, false);
  Job job = {};
  fill_job(job, p, rot, false, 2, B, N, Hq, Hk, d, dtype);
  job.in[0] = heads_of(q, B, N, Hq, dtype);
  job.in[1] = heads_of(k, B, N, Hk, dtype);
  job.out[0] = heads_of(q_out, B, N, Hq, dtype);
  job.out[1] = heads_of(k_out, B, N, Hk, dtype);
  job.w[0] = wq;
  job.w[1] = wk;
  job.eps = eps;
  job.inv_d = 1.f / (float)d;
  ADALN_TRY(enqueue<kNormFwd>(job, rot, p.grid[0] + p.grid[1], dtype,
                              (hipStream_t)stream,
                              "adaln_qk_norm_rope_fwd launch"));
  return ok();
}

ADALN_API size_t adaln_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t N,
                                                        int64_t Hq, int64_t Hk,
                                                        int64_t d, int dtype) {
  if (check_sizes(B, N, Hq, Hk, d, dtype) != ADALN_OK) return 0;
  if (B * N == 0 || Hq + Hk == 0) return 0;
  const HeadsPlan p = heads_plan(B, N, Hq, Hk, d, dtype, true);
  if (p.single) return 0;
  return (size_t)(p.grid[0] + p.grid[1]) * (size_t)d * sizeof(float);
}

ADALN_API int adaln_qk_norm_rope_bwd(
    const adaln_heads_t *dq_out, const adaln_heads_t *dk_out,
    const adaln_heads_t *q, const adaln_heads_t *k, const void *wq,
    const void *wk, float eps, const adaln_rotation_t *rot,
    const adaln_heads_t *dq, const adaln_heads_t *dk, float *dwq, float *dwk,
    void *workspace, size_t workspace_bytes, int64_t B, int64_t N, int64_t Hq,
    int64_t Hk, int64_t d, int dtype, void *stream) {
  ADALN_TRY(check_sizes(B, N, Hq, Hk, d, dtype));
  const bool rows = B * N > 0 && Hq + Hk > 0;
  if (!(eps >= 0.f) || isinf(eps))
    return fail(ADALN_ERR_INVALID, "eps must be finite and not negative");
  ADALN_TRY(check_rotation(rot, d, dtype, rows));
  ADALN_TRY(check_heads(dq_out, B, N, Hq, d, dtype, false, "dq_out"));
  ADALN_TRY(check_heads(dk_out, B, N, Hk, d, dtype, false, "dk_out"));
  ADALN_TRY(check_heads(q, B, N, Hq, d, dtype, false, "q"));
  ADALN_TRY(check_heads(k, B, N, Hk, d, dtype, false, "k"));
  ADALN_TRY(check_heads(dq, B, N, Hq, d, dtype, true, "dq"));
  ADALN_TRY(check_heads(dk, B, N, Hk, d, dtype, true, "dk"));
  ADALN_TRY(check_weight(wq, rows && Hq > 0, "wq"));
  ADALN_TRY(check_weight(wk, rows && Hk > 0, "wk"));
  ADALN_TRY(check_weight(dwq, Hq > 0 || dwq != nullptr, "dwq"));
  ADALN_TRY(check_weight(dwk, Hk > 0 || dwk != nullptr, "dwk"));
  if (dwq == nullptr && dwk == nullptr) return ok();  // no heads at all
  HeadsPlan p = {};
  if (rows) p = heads_plan(B, N, Hq, Hk, d, dtype, true);
  const size_t need =
      p.single ? 0
               : (size_t)(p.grid[0] + p.grid[1]) * (size_t)d * sizeof(float);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(ADALN_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu%s",
                  need, workspace_bytes,
                  workspace == nullptr ? " (NULL)" : "");
    ADALN_TRY(check_weight(workspace, true, "workspace"));
  }
  float *part[2] = {dwq, dwk};
  if (!p.single) {
    part[0] = static_cast<float *>(workspace);
    part[1] = part[0] + p.grid[0] * d;
  }
  if (rows) {
    Job job = {};
    fill_job(job, p, rot, true, 3, B, N, Hq, Hk, d, dtype);
    job.in[0] = heads_of(q, B, N, Hq, dtype);
    job.in[1] = heads_of(k, B, N, Hk, dtype);
    job.dy[0] = heads_of(dq_out, B, N, Hq, dtype);
    job.dy[1] = heads_of(dk_out, B, N, Hk, dtype);
    job.out[0] = heads_of(dq, B, N, Hq, dtype);
    job.out[1] = heads_of(dk, B, N, Hk, dtype);
    job.w[0] = wq;
    job.w[1] = wk;
    job.part[0] = part[0];
    job.part[1] = part[1];
    job.eps = eps;
    job.inv_d = 1.f / (float)d;
    ADALN_TRY(enqueue<kNormBwd>(job, rot, p.grid[0] + p.grid[1], dtype,
                                (hipStream_t)stream,
                                "adaln_qk_norm_rope_bwd launch"));
  }
  if (p.single && p.grid[0] + p.grid[1] == (dwq != nullptr) + (dwk != nullptr))
    return ok();
  const Sums sums = {{part[0], part[1]},
                     {dwq, dwk},
                     {(int32_t)p.grid[0], (int32_t)p.grid[1]},
                     (int32_t)d};
  const hipError_t e = launch_kernel_threads(
      sum_kernel, 2 * ((d + kSumCols - 1) / kSumCols), kSumSlices * kSumCols,
      (hipStream_t)stream, sums);
  if (e != hipSuccess) return hip_fail(e, "adaln_qk_norm_rope_bwd finish");
  return ok();
}
