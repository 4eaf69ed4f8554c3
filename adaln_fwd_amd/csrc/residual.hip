// The join of a branch with the residual stream: the gate that AdaLN's
// conditioning gives beside scale and shift, and dropout whose mask is never
// stored, forward and backward, with their C entry points.
//
//     y  = x + gate[b] * drop(h)       drop(h) = h * s where kept, else 0
//     dh = dy * gate[b] * s where kept, else 0       (dx = dy)
//     dgate[b] = sum_n dy * drop(h)                  (f32)
//
// Every pass reads its inputs once and writes its output once, so HBM bounds
// it, if the random numbers do not get in the way: the generator runs again in
// the backward instead of a mask being kept.  One Philox block (128 bits, ten
// rounds of two 32 x 32 bit products) serves 8 features of a token row, 16 bits
// each.  A lane is pinned to its features, as in the D-tile reduction of the
// modulation's gradients, so dgate is added up in registers, with nothing
// crossing lanes; a workgroup holds r rows of a tile of w vectors at a time,
// its workgroups' windows lying side by side in memory.  75600 x 5120 bf16, a
// tenth dropped: forward 383 us (6.1 TB/s), backward 434 (5.4), with nothing
// dropped 402 and 431: the generator is hidden.
#include <algorithm>
#include <math.h>

#include "adaln.h"
#include "checks.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace adaln {
namespace {

constexpr int kThreads = 512;     // most threads of a workgroup
// Rows a lane takes at a time; the next ones' loads are in flight meanwhile.
constexpr int unroll_of(bool bwd) { return bwd ? 1 : 2; }
constexpr int kSumCols = 64;      // of the sum over the partial rows
constexpr int kSumSlices = 16;

struct Residual {
  const char *a;       // x (may be NULL), or dy
  const char *h;
  const char *gate;    // [nmod, D], or NULL
  char *out;           // y, or dh
  float *part;         // backward with a gate: partial rows of dgate
  const uint64_t *rng; // seed, number of the call
  uint32_t limit;      // kept: 16 random bits < limit
  float scale;         // 65536 / limit
  int32_t nvec;        // vectors of a row
  int32_t w;           // vectors of a column tile
  int32_t r;           // rows a workgroup holds at a time
};

// Philox 4x32 in ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011).
__device__ __forceinline__ void philox(uint64_t counter, uint64_t call,
                                       uint64_t seed, uint32_t (&x)[4]) {
  x[0] = (uint32_t)counter;
  x[1] = (uint32_t)(counter >> 32);
  x[2] = (uint32_t)call;
  x[3] = (uint32_t)(call >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)x[0] * 0xD2511F53u;
    const uint64_t b = (uint64_t)x[2] * 0xCD9E8D57u;
    const uint32_t y1 = x[1], y3 = x[3];
    x[0] = (uint32_t)(b >> 32) ^ y1 ^ k0;
    x[1] = (uint32_t)b;
    x[2] = (uint32_t)(a >> 32) ^ y3 ^ k1;
    x[3] = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// 16 bits for each element of vector j of a row: element e of 8 takes the low
// (even e) or high half of word e / 2.  The numbers go by row and feature
// alone, not by type: two f32 vectors share a block.
template <int E>
__device__ __forceinline__ void kept(const Residual &p, uint64_t row, int j,
                                     uint64_t seed, uint64_t call,
                                     bool (&keep)[E]) {
  constexpr int P = 8 / E;  // vectors of a block
  uint32_t x[4];
  philox(row * (uint32_t)((p.nvec + P - 1) / P) + (uint32_t)(j / P), call,
         seed, x);
  if (P == 2 && (j & 1)) {
    x[0] = x[2];
    x[1] = x[3];
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    keep[e] = ((e & 1) ? x[e / 2] >> 16 : x[e / 2] & 0xffffu) < p.limit;
}

template <bool STREAM>
__device__ __forceinline__ Vec load_as(const void *p) {
  return STREAM ? load_stream(p) : load_vec(p);
}
template <bool STREAM>
__device__ __forceinline__ void store_as(void *p, const Vec &v) {
  if (STREAM)
    store_stream(p, v);
  else
    store_vec(p, v);
}

template <typename T, bool DROP, bool BWD, bool STREAM, typename Map>
__global__ __launch_bounds__(kThreads) void residual_kernel(Residual p,
                                                            Map map) {
  constexpr int E = Elems<T>::value;
  constexpr int kUnroll = unroll_of(BWD);
  __shared__ float stage[BWD ? kThreads : 1][BWD ? E : 1];
  const int t = threadIdx.x;
  const int slot = t / p.w;
  const int j = blockIdx.y * p.w + (t - slot * p.w);
  const bool active = slot < p.r && j < p.nvec;
  uint64_t seed = 0, call = 0;
  if (DROP) {
    seed = p.rng[0];
    call = p.rng[1];
  }
  for_each_segment(map, [&](int64_t row0, int64_t rows, int mod, int k_in,
                            int bps, int64_t part_row, int) {
    float g[E], sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      g[e] = 1.f;
      sum[e] = 0.f;
    }
    if (active) {
      if (p.gate != nullptr) {
        const Vec v = load_vec(p.gate + ((int64_t)mod * p.nvec + j) * 16);
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = elem<T>(v, e);
      }
      // rows n, n + step, ..., kUnroll of them at a time, the next ones' loads
      // in flight meanwhile
      const int64_t step = (int64_t)bps * p.r;
      int64_t n = (int64_t)k_in * p.r + slot;
      Vec a[kUnroll], h[kUnroll];
      auto load = [&](int64_t from) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (from + u * step >= rows) break;
          const int64_t at = ((row0 + from + u * step) * p.nvec + j) * 16;
          a[u] = p.a != nullptr ? load_as<STREAM>(p.a + at) : vzero();
          h[u] = p.h != nullptr ? load_as<STREAM>(p.h + at) : vzero();
        }
      };
      load(n);
      for (; n < rows; n += kUnroll * step) {
        Vec av[kUnroll], hv[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          av[u] = a[u];
          hv[u] = h[u];
        }
        load(n + kUnroll * step);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (n + u * step >= rows) break;
          const int64_t row = row0 + n + u * step;
          bool keep[E];
          if (DROP) kept<E>(p, (uint64_t)row, j, seed, call, keep);
          float out[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float x = elem<T>(av[u], e);
            const float hs = DROP ? elem<T>(hv[u], e) * p.scale
                                  : elem<T>(hv[u], e);
            // selected, not multiplied by zero: what is dropped leaves
            // nothing behind, be it infinite or no number
            if (BWD) {
              const float d = DROP ? x * p.scale * g[e] : x * g[e];
              out[e] = !DROP || keep[e] ? d : 0.f;
              sum[e] += !DROP || keep[e] ? x * hs : 0.f;
            } else {
              out[e] = !DROP || keep[e] ? fmaf(g[e], hs, x) : x;
            }
          }
          store_as<STREAM>(p.out + (row * p.nvec + j) * 16, pack<T>(out));
        }
      }
    }
    if constexpr (BWD) {
      if (p.part != nullptr) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) stage[t][e] = sum[e];
        __syncthreads();
        // the r rows' sums, in order
        if (active && slot == 0) {
          for (int i = 1; i < p.r; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] += stage[t + i * p.w][e];
          float *dst = p.part + (part_row * p.nvec + j) * E;
#pragma unroll
          for (int e = 0; e < E; ++e) dst[e] = sum[e];
        }
      }
    }
  });
}

// dgate[m] = the sum of its workgroups' partial rows, in a fixed order: of
// each slice of them, then of the slices.
struct Rows {
  int64_t first, count;
};
__device__ __forceinline__ int row_runs(const UniformMap &) { return 1; }
__device__ __forceinline__ int row_runs(const SegMap &m) { return m.nseg; }
__device__ __forceinline__ Rows row_run(const UniformMap &m, int, int mod) {
  return {(int64_t)mod * m.bps, m.N > 0 ? m.bps : 0};
}
__device__ __forceinline__ Rows row_run(const SegMap &m, int s, int mod) {
  return {m.wg_start[s],
          m.mod[s] == mod ? m.wg_start[s + 1] - m.wg_start[s] : 0};
}

template <typename Map>
__global__ __launch_bounds__(kSumSlices * kSumCols) void gate_sum_kernel(
    const float *part, float *dgate, int32_t D, int32_t col_blocks,
    int64_t blocks, Map map) {
  __shared__ float stage[kSumSlices][kSumCols];
  const int c = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  for (int64_t id = blockIdx.x; id < blocks; id += gridDim.x) {
    const int mod = (int)(id / col_blocks);
    const int f = (int)(id - (int64_t)mod * col_blocks) * kSumCols + c;
    float v = 0.f;
    if (f < D) {
      for (int s = 0; s < row_runs(map); ++s) {
        const Rows run = row_run(map, s, mod);
        const float *src = part + run.first * D + f;
        int64_t i = slice;
        for (; i + 3 * kSumSlices < run.count; i += 4 * kSumSlices) {
          float x[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) x[u] = src[(i + u * kSumSlices) * D];
#pragma unroll
          for (int u = 0; u < 4; ++u) v += x[u];
        }
        for (; i < run.count; i += kSumSlices) v += src[i * D];
      }
    }
    __syncthreads();
    stage[slice][c] = v;
    __syncthreads();
    if (slice == 0 && f < D) {
      for (int s = 1; s < kSumSlices; ++s) v += stage[s][c];
      dgate[(int64_t)mod * D + f] = v;
    }
  }
}

// ----------------------------------------------------------------- planning

int elems_per_vec(int dtype) { return dtype == ADALN_BF16 ? 8 : 4; }

// Columns: a row of up to 512 vectors is one tile, a wider one tiles of equal
// width; a workgroup takes as many rows at a time as 512 threads hold.
struct Shape {
  int32_t nvec, w, r, tiles, threads;
};

Shape shape_of(int64_t D, int dtype) {
  Shape s;
  s.nvec = (int32_t)(D / elems_per_vec(dtype));
  s.tiles = (s.nvec + kThreads - 1) / kThreads;
  s.w = (s.nvec + s.tiles - 1) / s.tiles;
  s.r = kThreads / s.w;
  s.threads = (s.w * s.r + kWave - 1) / kWave * kWave;
  return s;
}

// Workgroups of rows.  The forward covers the rows with its grid, four steps
// of its rows each.  The backward runs a fixed number of workgroups on every
// CU, so that few partial rows of dgate are left to add up: a whole number,
// since the CUs with one more end last (MI355X, 75600 x 5120 bf16: 818
// workgroups of 320 threads 476-518 us, 1024, four to a CU, 457).
constexpr int64_t kFwdSteps = 4;
constexpr int64_t kBwdThreads = 1280;  // of a CU, at most

int64_t most_groups(const Shape &s, bool bwd) {
  if (!bwd) return kMaxGrid;
  return std::max<int64_t>(1, kCUs * (kBwdThreads / s.threads) / s.tiles);
}

UniformMap uniform_map(int64_t B, int64_t N, const Shape &s, bool bwd) {
  UniformMap m = {};
  m.B = (int32_t)B;
  m.N = (int32_t)N;
  const int64_t most = most_groups(s, bwd);
  const int64_t steps = std::max<int64_t>(1, (N + s.r - 1) / s.r);
  const int64_t want = bwd ? steps : (steps + kFwdSteps - 1) / kFwdSteps;
  m.bps = (int32_t)std::min(want, std::max<int64_t>(1, most / std::max<int64_t>(B, 1)));
  // (without rows there is nothing to visit; dgate is then zero)
  m.groups = N == 0 ? 0 : (int32_t)std::min<int64_t>(
                              B, std::max<int64_t>(1, most / m.bps));
  return m;
}

SegMap seg_map(const int64_t *off, const int32_t *mod, int64_t nseg,
               const Shape &s, bool bwd) {
  SegMap m = {};
  m.nseg = (int32_t)nseg;
  const int64_t rows = nseg > 0 ? off[nseg] : 0;
  // rows of a workgroup: whole steps
  int64_t per = (rows + most_groups(s, bwd) - 1) / most_groups(s, bwd);
  if (!bwd) per = std::max(per, kFwdSteps * s.r);
  per = std::max<int64_t>(1, (per + s.r - 1) / s.r) * s.r;
  for (int64_t i = 0; i < nseg; ++i) {
    m.row_start[i] = off[i];
    m.mod[i] = mod ? mod[i] : (int32_t)i;
    m.wg_start[i + 1] =
        m.wg_start[i] + (int32_t)((off[i + 1] - off[i] + per - 1) / per);
  }
  m.row_start[nseg] = rows;
  return m;
}

int64_t grid_of(const UniformMap &m) { return (int64_t)m.bps * m.groups; }
int64_t grid_of(const SegMap &m) { return m.wg_start[m.nseg]; }
int64_t rows_of(const UniformMap &m) { return (int64_t)m.B * m.N; }
int64_t rows_of(const SegMap &m) { return m.row_start[m.nseg]; }
int64_t part_rows(const UniformMap &m) {
  return m.N > 0 ? (int64_t)m.B * m.bps : 0;
}
int64_t part_rows(const SegMap &m) { return m.wg_start[m.nseg]; }

int hip_fail(hipError_t e, const char *what) {
  return fail(ADALN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Inputs that another kernel has just written may still lie in the 256 MB
// Infinity Cache, and the next one finds the output there: up to kCachedBytes
// read and written a call takes plain accesses, past it the streaming hint.
// (With it and plainly, forward: 75600 x 5120 bf16 383 and 436 us, 24960 x 1536
// 39.3 and 43.5, but 3333 x 1156 f32 10.9 and 9.9, 16384 x 1152 21.0 and 20.4.)
constexpr int64_t kCachedBytes = int64_t(192) << 20;

template <typename T, bool BWD, typename Map>
hipError_t launch_residual(const Residual &p, const Map &map, const Shape &s,
                           int64_t rows, hipStream_t stream) {
  const int64_t grid = grid_of(map);
  if (grid <= 0) return hipSuccess;
  void *argv[] = {(void *)&p, (void *)&map};
  const bool stream_hint = rows * s.nvec * 16 * 3 > kCachedBytes;
  void (*k)(Residual, Map) =
      p.rng != nullptr
          ? (stream_hint ? residual_kernel<T, true, BWD, true, Map>
                         : residual_kernel<T, true, BWD, false, Map>)
          : (stream_hint ? residual_kernel<T, false, BWD, true, Map>
                         : residual_kernel<T, false, BWD, false, Map>);
  return hipLaunchKernel((const void *)k, dim3((unsigned)grid, s.tiles),
                         dim3(s.threads), argv, 0, stream);
}

// --------------------------------------------------------------- the calls

// The dropout's numbers; rng stays NULL where nothing is dropped.
int set_drop(Residual &job, double p, const int64_t *rng) {
  if (!(p >= 0.) || p > 1. - 1. / 65536)
    return fail(ADALN_ERR_INVALID, "p must be from 0 to 1 - 2^-16, got %g", p);
  job.limit = (uint32_t)floor((1. - p) * 65536 + 0.5);
  job.scale = (float)(65536. / job.limit);
  if (job.limit == 65536) return ADALN_OK;
  if (rng == nullptr) return fail(ADALN_ERR_INVALID, "rng is NULL");
  if (reinterpret_cast<uintptr_t>(rng) % 8 != 0)
    return fail(ADALN_ERR_ALIGN, "rng is not 8-byte aligned");
  job.rng = reinterpret_cast<const uint64_t *>(rng);
  return ADALN_OK;
}

template <typename Map>
int residual_fwd(Residual job, const Map &map, const Shape &s, int dtype,
                 void *stream) {
  job.nvec = s.nvec;
  job.w = s.w;
  job.r = s.r;
  const hipStream_t st = (hipStream_t)stream;
  const hipError_t e = dtype == ADALN_BF16
                           ? launch_residual<bf16, false>(job, map, s, rows_of(map), st)
                           : launch_residual<float, false>(job, map, s, rows_of(map), st);
  if (e != hipSuccess) return hip_fail(e, "adaln_residual_fwd launch");
  return ok();
}

// Workspace of the partial rows; none where the one workgroup of each vector
// writes dgate itself, and none without rows.
bool direct(const UniformMap &m) { return m.bps == 1 && m.N > 0; }
bool direct(const SegMap &) { return false; }

template <typename Map>
size_t part_bytes(const Map &m, const Shape &s, int dtype) {
  return direct(m) ? 0
                   : (size_t)part_rows(m) * s.nvec * elems_per_vec(dtype) *
                         sizeof(float);
}

template <typename Map>
int residual_bwd(Residual job, const Map &map, const Shape &s, float *dgate,
                 int64_t nmod, void *workspace, size_t workspace_bytes,
                 int dtype, void *stream) {
  job.nvec = s.nvec;
  job.w = s.w;
  job.r = s.r;
  const hipStream_t st = (hipStream_t)stream;
  if (dgate != nullptr) {
    const size_t need = part_bytes(map, s, dtype);
    if (need > 0) {
      if (workspace == nullptr || workspace_bytes < need)
        return fail(ADALN_ERR_WORKSPACE,
                    "workspace needs %zu bytes, got %zu%s", need,
                    workspace_bytes, workspace == nullptr ? " (NULL)" : "");
      ADALN_TRY(check_ptr(workspace, true, "workspace"));
    }
    job.part = direct(map) ? dgate : static_cast<float *>(workspace);
  }
  hipError_t e = dtype == ADALN_BF16
                     ? launch_residual<bf16, true>(job, map, s, rows_of(map), st)
                     : launch_residual<float, true>(job, map, s, rows_of(map), st);
  if (e != hipSuccess) return hip_fail(e, "adaln_residual_bwd launch");
  if (dgate != nullptr && !direct(map)) {
    const int32_t D = s.nvec * elems_per_vec(dtype);
    const int32_t cols = (D + kSumCols - 1) / kSumCols;
    const int64_t blocks = nmod * cols;
    e = launch_kernel_threads(gate_sum_kernel<Map>, blocks,
                              kSumSlices * kSumCols, st,
                              (const float *)job.part, dgate, D, cols, blocks,
                              map);
    if (e != hipSuccess) return hip_fail(e, "adaln_residual_bwd finish");
  }
  return ok();
}

Residual job_of(const void *a, const void *h, const void *gate, void *out) {
  Residual p = {};
  p.a = static_cast<const char *>(a);
  p.h = static_cast<const char *>(h);
  p.gate = static_cast<const char *>(gate);
  p.out = static_cast<char *>(out);
  return p;
}

}  // namespace
}  // namespace adaln

using namespace adaln;

ADALN_API int adaln_residual_fwd(const void *x, const void *h,
                                 const void *gate, double p,
                                 const int64_t *rng, void *y, int64_t B,
                                 int64_t N, int64_t D, int dtype,
                                 void *stream) {
  ADALN_TRY(check_shape(B, N, D, dtype));
  const bool rows = B * N > 0;
  ADALN_TRY(check_ptr(x, rows && x != nullptr, "x"));
  ADALN_TRY(check_ptr(h, rows, "h"));
  ADALN_TRY(check_ptr(gate, rows && gate != nullptr, "gate"));
  ADALN_TRY(check_ptr(y, rows, "y"));
  Residual job = job_of(x, h, gate, y);
  ADALN_TRY(set_drop(job, p, rows ? rng : (const int64_t *)8));
  if (!rows) return ok();
  const Shape s = shape_of(D, dtype);
  return residual_fwd(job, uniform_map(B, N, s, false), s, dtype, stream);
}

ADALN_API size_t adaln_residual_bwd_workspace_bytes(int64_t B, int64_t N,
                                                    int64_t D, int dtype) {
  if (check_shape(B, N, D, dtype) != ADALN_OK || B * N == 0) return 0;
  const Shape s = shape_of(D, dtype);
  return part_bytes(uniform_map(B, N, s, true), s, dtype);
}

ADALN_API int adaln_residual_bwd(const void *dy, const void *h,
                                 const void *gate, double p,
                                 const int64_t *rng, void *dh, float *dgate,
                                 void *workspace, size_t workspace_bytes,
                                 int64_t B, int64_t N, int64_t D, int dtype,
                                 void *stream) {
  ADALN_TRY(check_shape(B, N, D, dtype));
  const bool rows = B * N > 0, gated = B > 0 && (gate != nullptr || dgate != nullptr);
  ADALN_TRY(check_ptr(dy, rows, "dy"));
  ADALN_TRY(check_ptr(h, rows && gated, "h"));
  ADALN_TRY(check_ptr(gate, rows && gated, "gate"));
  ADALN_TRY(check_ptr(dh, rows, "dh"));
  ADALN_TRY(check_ptr(dgate, gated, "dgate"));
  Residual job = job_of(dy, gated ? h : nullptr, gate, dh);
  ADALN_TRY(set_drop(job, p, rows ? rng : (const int64_t *)8));
  if (!rows && !gated) return ok();
  const Shape s = shape_of(D, dtype);
  return residual_bwd(job, uniform_map(B, N, s, true), s,
                      gated ? dgate : nullptr, B, workspace, workspace_bytes,
                      dtype, stream);
}

ADALN_API int adaln_residual_fwd_segments(
    const void *x, const void *h, const void *gate, double p,
    const int64_t *rng, void *y, const int64_t *seg_offsets,
    const int32_t *seg_mod, int64_t nseg, int64_t nmod, int64_t D, int dtype,
    void *stream) {
  ADALN_TRY(check_segments(seg_offsets, seg_mod, nseg, nmod, D, dtype));
  const bool rows = nseg > 0 && seg_offsets[nseg] > 0;
  ADALN_TRY(check_ptr(x, rows && x != nullptr, "x"));
  ADALN_TRY(check_ptr(h, rows, "h"));
  ADALN_TRY(check_ptr(gate, rows, "gate"));
  ADALN_TRY(check_ptr(y, rows, "y"));
  Residual job = job_of(x, h, gate, y);
  ADALN_TRY(set_drop(job, p, rows ? rng : (const int64_t *)8));
  if (!rows) return ok();
  const Shape s = shape_of(D, dtype);
  return residual_fwd(job, seg_map(seg_offsets, seg_mod, nseg, s, false), s,
                      dtype, stream);
}

ADALN_API size_t adaln_residual_bwd_segments_workspace_bytes(
    const int64_t *seg_offsets, int64_t nseg, int64_t D, int dtype) {
  if (check_segments(seg_offsets, nullptr, nseg, nseg > 0 ? nseg : 1, D,
                     dtype) != ADALN_OK ||
      nseg == 0)
    return 0;
  const Shape s = shape_of(D, dtype);
  return part_bytes(seg_map(seg_offsets, nullptr, nseg, s, true), s, dtype);
}

ADALN_API int adaln_residual_bwd_segments(
    const void *dy, const void *h, const void *gate, double p,
    const int64_t *rng, void *dh, float *dgate, void *workspace,
    size_t workspace_bytes, const int64_t *seg_offsets, const int32_t *seg_mod,
    int64_t nseg, int64_t nmod, int64_t D, int dtype, void *stream) {
  ADALN_TRY(check_segments(seg_offsets, seg_mod, nseg, nmod, D, dtype));
  const bool rows = nseg > 0 && seg_offsets[nseg] > 0;
  ADALN_TRY(check_ptr(dy, rows, "dy"));
  ADALN_TRY(check_ptr(h, rows, "h"));
  ADALN_TRY(check_ptr(gate, rows, "gate"));
  ADALN_TRY(check_ptr(dh, rows, "dh"));
  ADALN_TRY(check_ptr(dgate, nmod > 0, "dgate"));
  Residual job = job_of(dy, h, gate, dh);
  ADALN_TRY(set_drop(job, p, rows ? rng : (const int64_t *)8));
  if (nmod == 0) return ok();
  const Shape s = shape_of(D, dtype);
  return residual_bwd(job, seg_map(seg_offsets, seg_mod, nseg, s, true), s,
                      dgate, nmod, workspace, workspace_bytes, dtype, stream);
}
