// The way of token rows to the experts of a mixture and back, with their C
// entry points.  Of T tokens each has k choices of an expert:
//
//     slot[t, j] = where choice (t, j) stands when all choices are sorted by
//                  expert, those of one expert by token, then by j; -1 for
//                  an expert outside [0, E)
//     sort:  xs[slot[t, j]] = x[t]             dx[t] = sum_j dxs[slot[t, j]]
//     join:  y[t] = sum_j w[t, j] ys[slot[t, j]]
//            dys[slot[t, j]] = w[t, j] dy[t]    dw[t, j] = dy[t] . ys[slot[t, j]]
//
// The sort is a counting sort: each workgroup counts its run of choices by
// expert, then places them behind those of the runs before it.  The ranks are
// counted, not drawn from atomics, so every call gives the same order.  The
// rows are moved by token: a wavefront reads a token's row once for all its k
// places, or gathers its k rows into one, so each byte of HBM moves once and
// HBM bounds it.
#include <algorithm>

#include "adaln.h"
#include "checks.hpp"
#include "common.hpp"
#include "launch.hpp"

namespace adaln {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kMaxChoices = 64;  // of a token: a lane each
constexpr int kSortWaves = 16;
constexpr int kSortThreads = kSortWaves * kWave;
// Choices that one workgroup sorts by itself; of more, each takes kRun, and
// more than that where there would be over kMostRuns: every workgroup reads
// the counts of all the others.  (Of 64 experts, 4096 choices take 5.4 us so,
// 8192 9.4 and 16384 16; in two launches 8192 to 32768 take 8.5 to 8.7.  131040
// choices take 10 us, by 1024 a workgroup the same.)
constexpr int64_t kSingle = 6144;
constexpr int64_t kRun = 4096;
constexpr int64_t kMostRuns = 256;

// ---------------------------------------------------------------- the sort

template <typename I>
__device__ __forceinline__ int expert_of(const I *expert, int64_t i,
                                         int64_t end, int E) {
  if (i >= end) return -1;
  const I e = expert[i];
  return e >= 0 && e < E ? (int)e : -1;
}

// counts[run][e]: the choices of expert e in each run.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void count_kernel(
    const I *expert, int32_t *counts, int64_t n, int64_t run, int32_t E) {
  __shared__ int32_t hist[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * run, end = min(n, first + run);
  for (int64_t i = first + threadIdx.x; i < end; i += kSortThreads) {
    const int e = expert_of(expert, i, end, E);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads)
    counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

// Lanes of the wavefront with the same expert (bits: those of the largest).
__device__ __forceinline__ uint64_t same_lanes(int e, int bits) {
  uint64_t same = __ballot(e >= 0);
  for (int b = 0; b < bits; ++b) {
    const uint64_t one = __ballot((e >> b) & 1);
    same &= ((e >> b) & 1) ? one : ~one;
  }
  return same;
}

// slot of a run's choices: the experts before, the runs before, the
// wavefronts before, the rounds before and the lanes before.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void place_kernel(
    const I *expert, const int32_t *counts, int32_t *slot, int32_t *offsets,
    int64_t n, int64_t run, int32_t E, int32_t bits) {
  __shared__ int32_t at[kSortWaves][kMaxExperts];
  __shared__ int32_t start[kMaxExperts], total[kMaxExperts];
  __shared__ int32_t wave_total[kSortWaves];
  const int t = threadIdx.x, lane = lane_id(), wave = wave_id();
  const int64_t first = blockIdx.x * run, end = min(n, first + run);
  // each wavefront's stretch of the run, whole rounds of 64
  const int64_t per =
      ((end - first + kSortThreads - 1) / kSortThreads) * kWave;
  const int64_t from = first + wave * per, to = min(end, from + per);
  for (int e = lane; e < E; e += kWave) at[wave][e] = 0;
  for (int e = t; e < E; e += kSortThreads) start[e] = total[e] = 0;
  __syncthreads();
  for (int64_t i = from + lane; i < to; i += kWave) {
    const int e = expert_of(expert, i, to, E);
    if (e >= 0) atomicAdd(&at[wave][e], 1);
  }
  // what stands before this run, and the whole: `split` threads an expert
  if (counts != nullptr) {
    const int split = max(1, kSortThreads / E);
    const int e = t % E, part = t / E;
    if (part < split) {
      int32_t before = 0, all = 0;
      for (int r = part; r < (int)gridDim.x; r += split) {
        const int32_t c = counts[(int64_t)r * E + e];
        all += c;
        if (r < (int)blockIdx.x) before += c;
      }
      atomicAdd(&start[e], before);
      atomicAdd(&total[e], all);
    }
  }
  __syncthreads();
  // wavefronts before, in place; without counts the run is the whole
  if (t < E) {
    int32_t sum = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t c = at[w][t];
      at[w][t] = sum;
      sum += c;
    }
    if (counts == nullptr) total[t] = sum;
  }
  __syncthreads();
  // experts before: a sum along the experts, one a thread
  int32_t mine = t < E ? total[t] : 0, sum = mine;
  for (int d = 1; d < kWave; d *= 2) {
    const int32_t other = __shfl_up(sum, d);
    if (lane >= d) sum += other;
  }
  if (lane == kWave - 1) wave_total[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += wave_total[w];
  if (t < E) {
    start[t] += sum - mine;
    if (blockIdx.x == 0) {
      offsets[t] = sum - mine;
      if (t == E - 1) offsets[E] = sum;
    }
  }
  __syncthreads();
  for (int64_t i = from; i < to; i += kWave) {
    const int e = expert_of(expert, i + lane, to, E);
    const uint64_t same = same_lanes(e, bits);
    int32_t place = -1;
    if (e >= 0) {
      const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      const int32_t base = at[wave][e];
      place = start[e] + base + rank;
      // every lane has read the count before the last of its kind moves it on
      __builtin_amdgcn_wave_barrier();
      if ((same >> lane) == 1) at[wave][e] = base + rank + 1;
    }
    __builtin_amdgcn_wave_barrier();
    if (i + lane < to) slot[i + lane] = place;
  }
}

// --------------------------------------------------------------- the rows

struct Move {
  const char *one;      // a row for each token: x, dy
  const char *many;     // sorted rows: ys, dxs
  char *one_out;        // y, dx
  char *many_out;       // xs, dys
  const float *w;       // [T, k], or NULL: ones
  float *dw;
  const int32_t *slot;  // [T, k]
  int64_t T;
  int64_t rows;         // sorted rows, T * k
  int32_t k;
  int32_t nvec;         // vectors of a row
  int32_t tiles;        // wavefronts a row is shared between
};

constexpr int kTileVecs = 2;  // vectors a lane holds of a row at a time
constexpr int kTile = kTileVecs * kWave;
constexpr int kAtOnce = 4;    // sorted rows whose loads are in flight together
// The same for the join's backward.  (MI355X, bf16: 32760 tokens, 4 choices of
// 64 experts, 5120 features: 588 us, 586 by tiles of two vectors and four rows;
// 4096 tokens, 8 choices, 4096 features: 110 and 120.)
constexpr int kBwdVecs = 4;
constexpr int kBwdAtOnce = 2;

enum { kScatter, kGather };

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

// The sorted row of a token's choice, lane j's of choice j; -1 for none.
__device__ __forceinline__ int slot_of(const Move &p, int64_t t, int lane) {
  if (lane >= p.k) return -1;
  const int s = p.slot[t * p.k + lane];
  return s < p.rows ? s : -1;
}

// A wavefront takes a tile of 128 vectors of a token's row.  kScatter: the
// token's row to its places.  kGather: the sum of the rows at its places, times
// w if there is one, in float32, in the order of the choices.
// Bound by HBM: 32760 tokens of 5120 bf16 features, 4 choices, take 326 us
// scattered (5.1 TB/s) and 281 gathered (6.0).
template <typename T, int OP, bool STREAM>
__device__ __forceinline__ void move_tile(const Move &p, int64_t id) {
  constexpr int E = Elems<T>::value;
  const int lane = lane_id();
  const int64_t t = id / p.tiles;
  const int v0 = (int)(id - t * p.tiles) * kTile + lane;
  const int my_slot = slot_of(p, t, lane);
  if constexpr (OP == kScatter) {
    Vec x[kTileVecs];
#pragma unroll
    for (int i = 0; i < kTileVecs; ++i)
      if (v0 + i * kWave < p.nvec)
        x[i] = load_as<STREAM>(p.one + (t * p.nvec + v0 + i * kWave) * 16);
    for (int j = 0; j < p.k; ++j) {
      const int s = __builtin_amdgcn_readlane(my_slot, j);
      if (s < 0) continue;
#pragma unroll
      for (int i = 0; i < kTileVecs; ++i)
        if (v0 + i * kWave < p.nvec)
          store_as<STREAM>(
              p.many_out + ((int64_t)s * p.nvec + v0 + i * kWave) * 16, x[i]);
    }
  } else {
    float my_w = 1.f;
    if (p.w != nullptr && lane < p.k) my_w = p.w[t * p.k + lane];
    float sum[kTileVecs][E] = {};
    for (int j0 = 0; j0 < p.k; j0 += kAtOnce) {
      Vec v[kAtOnce][kTileVecs];
      int s[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        s[j] = j0 + j < p.k ? __builtin_amdgcn_readlane(my_slot, j0 + j) : -1;
        if (s[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < kTileVecs; ++i)
          if (v0 + i * kWave < p.nvec)
            v[j][i] = load_as<STREAM>(
                p.many + ((int64_t)s[j] * p.nvec + v0 + i * kWave) * 16);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (s[j] < 0) continue;
        const float w = lane_read(my_w, j0 + j);
#pragma unroll
        for (int i = 0; i < kTileVecs; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e)
            sum[i][e] = fmaf(w, elem<T>(v[j][i], e), sum[i][e]);
      }
    }
#pragma unroll
    for (int i = 0; i < kTileVecs; ++i)
      if (v0 + i * kWave < p.nvec)
        store_as<STREAM>(p.one_out + (t * p.nvec + v0 + i * kWave) * 16,
                         pack<T>(sum[i]));
  }
}

template <typename T, int OP, bool STREAM>
__global__ __launch_bounds__(kBlock) void move_kernel(Move p) {
  const int64_t ids = p.T * p.tiles;
  for (int64_t id = (int64_t)blockIdx.x * (kBlock / kWave) + wave_id();
       id < ids; id += (int64_t)gridDim.x * (kBlock / kWave))
    move_tile<T, OP, STREAM>(p, id);
}

// The join's gradients in one pass: a wavefront takes a token and two of its
// choices at a time, reads its dy and their rows of ys, writes their rows of
// dys (which may stand in ys' place: a lane reads what it writes before) and
// adds up dw.  The same tokens take 577-589 us (5.2 TB/s): dy is read once for
// two choices, from the caches at best.
template <typename T, bool STREAM>
__device__ __forceinline__ void join_bwd_row(const Move &p, int64_t t) {
  constexpr int E = Elems<T>::value;
  const int lane = lane_id();
  const int my_slot = slot_of(p, t, lane);
  float my_w = 0.f, my_dw = 0.f;
  if (lane < p.k) my_w = p.w[t * p.k + lane];
  for (int j0 = 0; j0 < p.k; j0 += kBwdAtOnce) {
    int s[kBwdAtOnce];
    float w[kBwdAtOnce], dot[kBwdAtOnce];
#pragma unroll
    for (int j = 0; j < kBwdAtOnce; ++j) {
      s[j] = j0 + j < p.k ? __builtin_amdgcn_readlane(my_slot, j0 + j) : -1;
      w[j] = lane_read(my_w, min(j0 + j, kWave - 1));
      dot[j] = 0.f;
    }
    for (int v0 = lane; v0 < p.nvec; v0 += kBwdVecs * kWave) {
      Vec dy[kBwdVecs], ys[kBwdAtOnce][kBwdVecs];
#pragma unroll
      for (int i = 0; i < kBwdVecs; ++i)
        if (v0 + i * kWave < p.nvec)
          dy[i] = load_vec(p.one + (t * p.nvec + v0 + i * kWave) * 16);
#pragma unroll
      for (int j = 0; j < kBwdAtOnce; ++j)
        if (s[j] >= 0)
#pragma unroll
          for (int i = 0; i < kBwdVecs; ++i)
            if (v0 + i * kWave < p.nvec)
              ys[j][i] = load_as<STREAM>(
                  p.many + ((int64_t)s[j] * p.nvec + v0 + i * kWave) * 16);
#pragma unroll
      for (int j = 0; j < kBwdAtOnce; ++j) {
        if (s[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < kBwdVecs; ++i) {
          if (v0 + i * kWave >= p.nvec) break;
          float f[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float g = elem<T>(dy[i], e);
            dot[j] = fmaf(g, elem<T>(ys[j][i], e), dot[j]);
            f[e] = w[j] * g;
          }
          store_as<STREAM>(
              p.many_out + ((int64_t)s[j] * p.nvec + v0 + i * kWave) * 16,
              pack<T>(f));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBwdAtOnce; ++j) {
      if (s[j] < 0) continue;
      const float all = wave_sum(dot[j]);
      if (lane == j0 + j) my_dw = all;
    }
  }
  if (lane < p.k) p.dw[t * p.k + lane] = my_dw;
}

template <typename T, bool STREAM>
__global__ __launch_bounds__(kBlock) void join_bwd_kernel(Move p) {
  for (int64_t t = (int64_t)blockIdx.x * (kBlock / kWave) + wave_id();
       t < p.T; t += (int64_t)gridDim.x * (kBlock / kWave))
    join_bwd_row<T, STREAM>(p, t);
}

// ------------------------------------------------------------------- checks

int hip_fail(hipError_t e, const char *what) {
  return fail(ADALN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

int check_choices(int64_t T, int64_t k) {
  if (T < 0) return fail(ADALN_ERR_INVALID, "negative size: T=%lld", (long long)T);
  if (k < 1 || k > kMaxChoices)
    return fail(ADALN_ERR_INVALID, "k must be 1 to %d, got %lld", kMaxChoices,
                (long long)k);
  if (T > ((int64_t(1) << 31) - 1) / k)
    return fail(ADALN_ERR_INVALID, "T*k exceeds 2^31-1 rows");
  return ADALN_OK;
}

// Small arrays: NULL only without tokens; aligned to their elements.
int check_array(const void *p, bool needed, size_t align, const char *name) {
  if (!needed) return ADALN_OK;
  if (p == nullptr) return fail(ADALN_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return fail(ADALN_ERR_ALIGN, "%s is not %zu-byte aligned", name, align);
  return ADALN_OK;
}

int check_rows(const void *one, const void *many, const int32_t *slot,
               int64_t T, int64_t k, int64_t D, int dtype,
               const char *one_name, const char *many_name) {
  ADALN_TRY(check_choices(T, k));
  ADALN_TRY(check_shape(1, T, D, dtype));
  ADALN_TRY(check_ptr(one, T > 0, one_name));
  ADALN_TRY(check_ptr(many, T > 0, many_name));
  return check_array(slot, T > 0, 4, "slot");
}

Move move_of(const int32_t *slot, int64_t T, int64_t k, int64_t D, int dtype) {
  Move p = {};
  p.slot = slot;
  p.T = T;
  p.rows = T * k;
  p.k = (int32_t)k;
  p.nvec = (int32_t)(D / (dtype == ADALN_BF16 ? 8 : 4));
  p.tiles = (p.nvec + kTile - 1) / kTile;
  return p;
}

template <typename K>
hipError_t launch_waves(K k, int64_t waves, hipStream_t s, const Move &p) {
  return launch_kernel(k, (waves + kBlock / kWave - 1) / (kBlock / kWave), s,
                       p);
}

// Rows that another kernel has just written may still lie in the 256 MB
// Infinity Cache, and the next one finds them there: up to kCachedBytes read
// and written a call takes plain accesses, past it the streaming hint (those
// 32760 tokens: gathered 281 us, plainly 319, the join's backward 589 and 614,
// scattered 326 and 313, but the kernels behind it then take longer, all four
// together 1472 and 1496; 100000 of 1024 features, one choice: 66 and 73 each
// way; 777 of 1000 f32 features: within 0.3 us).
constexpr int64_t kCachedBytes = int64_t(192) << 20;

bool past_caches(const Move &p, int rows) {
  return p.T * rows * p.nvec * 16 > kCachedBytes;
}

template <int OP>
int move(const Move &p, int dtype, void *stream, const char *what) {
  if (p.T == 0) return ok();
  const hipStream_t s = (hipStream_t)stream;
  const int64_t n = p.T * p.tiles;
  const bool hint = past_caches(p, 1 + p.k);
  const hipError_t e =
      dtype == ADALN_BF16
          ? launch_waves(hint ? move_kernel<bf16, OP, true>
                              : move_kernel<bf16, OP, false>, n, s, p)
          : launch_waves(hint ? move_kernel<float, OP, true>
                              : move_kernel<float, OP, false>, n, s, p);
  if (e != hipSuccess) return hip_fail(e, what);
  return ok();
}

// Choices each workgroup sorts.
int64_t sort_run(int64_t n) {
  if (n <= kSingle) return kSingle;
  return std::max(kRun, (n + kMostRuns - 1) / kMostRuns);
}

template <typename I>
int plan(const void *expert, int32_t *offsets, int32_t *slot, int32_t *counts,
         int64_t n, int64_t E, hipStream_t s) {
  const I *from = static_cast<const I *>(expert);
  const int64_t run = sort_run(n);
  const int64_t runs = std::max<int64_t>(1, (n + run - 1) / run);
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  if (runs > 1) {
    const hipError_t e =
        launch_kernel_threads(count_kernel<I>, runs, kSortThreads, s, from,
                              counts, n, run, (int32_t)E);
    if (e != hipSuccess) return hip_fail(e, "adaln_experts_plan count");
  }
  const hipError_t e = launch_kernel_threads(
      place_kernel<I>, runs, kSortThreads, s, from,
      runs > 1 ? (const int32_t *)counts : (const int32_t *)nullptr, slot,
      offsets, n, run, (int32_t)E, (int32_t)bits);
  if (e != hipSuccess) return hip_fail(e, "adaln_experts_plan launch");
  return ok();
}

}  // namespace
}  // namespace adaln

using namespace adaln;

ADALN_API size_t adaln_experts_plan_workspace_bytes(int64_t T, int64_t k,
                                                    int64_t E) {
  if (check_choices(T, k) != ADALN_OK || E < 1 || E > kMaxExperts) return 0;
  const int64_t run = sort_run(T * k), runs = (T * k + run - 1) / run;
  return runs > 1 ? (size_t)runs * (size_t)E * sizeof(int32_t) : 0;
}

ADALN_API int adaln_experts_plan(const void *expert, int wide,
                                 int32_t *offsets, int32_t *slot,
                                 void *workspace, size_t workspace_bytes,
                                 int64_t T, int64_t k, int64_t E,
                                 void *stream) {
  ADALN_TRY(check_choices(T, k));
  if (E < 1 || E > kMaxExperts)
    return fail(ADALN_ERR_INVALID, "E must be 1 to %d, got %lld", kMaxExperts,
                (long long)E);
  ADALN_TRY(check_array(expert, T > 0, wide ? 8 : 4, "expert"));
  ADALN_TRY(check_array(slot, T > 0, 4, "slot"));
  ADALN_TRY(check_array(offsets, true, 4, "offsets"));
  const size_t need = adaln_experts_plan_workspace_bytes(T, k, E);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(ADALN_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu%s",
                  need, workspace_bytes,
                  workspace == nullptr ? " (NULL)" : "");
    ADALN_TRY(check_array(workspace, true, 4, "workspace"));
  }
  int32_t *counts = static_cast<int32_t *>(workspace);
  return wide ? plan<int64_t>(expert, offsets, slot, counts, T * k, E,
                              (hipStream_t)stream)
              : plan<int32_t>(expert, offsets, slot, counts, T * k, E,
                              (hipStream_t)stream);
}

ADALN_API int adaln_experts_sort_fwd(const void *x, const int32_t *slot,
                                     void *xs, int64_t T, int64_t k, int64_t D,
                                     int dtype, void *stream) {
  ADALN_TRY(check_rows(x, xs, slot, T, k, D, dtype, "x", "xs"));
  Move p = move_of(slot, T, k, D, dtype);
  p.one = static_cast<const char *>(x);
  p.many_out = static_cast<char *>(xs);
  return move<kScatter>(p, dtype, stream, "adaln_experts_sort_fwd launch");
}

ADALN_API int adaln_experts_sort_bwd(const void *dxs, const int32_t *slot,
                                     void *dx, int64_t T, int64_t k, int64_t D,
                                     int dtype, void *stream) {
  ADALN_TRY(check_rows(dx, dxs, slot, T, k, D, dtype, "dx", "dxs"));
  Move p = move_of(slot, T, k, D, dtype);
  p.many = static_cast<const char *>(dxs);
  p.one_out = static_cast<char *>(dx);
  return move<kGather>(p, dtype, stream, "adaln_experts_sort_bwd launch");
}

ADALN_API int adaln_experts_join_fwd(const void *ys, const int32_t *slot,
                                     const float *w, void *y, int64_t T,
                                     int64_t k, int64_t D, int dtype,
                                     void *stream) {
  ADALN_TRY(check_rows(y, ys, slot, T, k, D, dtype, "y", "ys"));
  ADALN_TRY(check_array(w, T > 0, 4, "w"));
  Move p = move_of(slot, T, k, D, dtype);
  p.many = static_cast<const char *>(ys);
  p.one_out = static_cast<char *>(y);
  p.w = w;
  return move<kGather>(p, dtype, stream, "adaln_experts_join_fwd launch");
}

ADALN_API int adaln_experts_join_bwd(const void *dy, const void *ys,
                                     const int32_t *slot, const float *w,
                                     void *dys, float *dw, int64_t T,
                                     int64_t k, int64_t D, int dtype,
                                     void *stream) {
  ADALN_TRY(check_rows(dy, ys, slot, T, k, D, dtype, "dy", "ys"));
  ADALN_TRY(check_array(w, T > 0, 4, "w"));
  ADALN_TRY(check_ptr(dys, T > 0, "dys"));
  ADALN_TRY(check_array(dw, T > 0, 4, "dw"));
  if (T == 0) return ok();
  Move p = move_of(slot, T, k, D, dtype);
  p.one = static_cast<const char *>(dy);
  p.many = static_cast<const char *>(ys);
  p.many_out = static_cast<char *>(dys);
  p.w = w;
  p.dw = dw;
  const hipStream_t s = (hipStream_t)stream;
  const bool hint = past_caches(p, 1 + 2 * p.k);
  const hipError_t e =
      dtype == ADALN_BF16
          ? launch_waves(hint ? join_bwd_kernel<bf16, true>
                              : join_bwd_kernel<bf16, false>, T, s, p)
          : launch_waves(hint ? join_bwd_kernel<float, true>
                              : join_bwd_kernel<float, false>, T, s, p);
  if (e != hipSuccess) return hip_fail(e, "adaln_experts_join_bwd launch");
  return ok();
}
