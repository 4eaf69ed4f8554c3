// Which elements of a d x d state the linear attention's lanes read: for every
// line "dtype d across" of the input, the least and the largest that any lane
// of any wavefront reads, and how many of the state's elements are loaded into
// the accumulators.
#include "../../adaln_fwd_amd/csrc/lin_attn.hip"

#include <stdio.h>

#include <set>

// Built for the host alone and linked without a HIP runtime: nothing is
// launched, and the kernels that the library registers are not there.
extern "C" {
void **__hipRegisterFatBinary(const void *) { return nullptr; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *, char *, const char *, int,
                           void *, void *, void *, void *, int *) {}
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *,
                                     hipStream_t *) {
  return hipErrorNotSupported;
}
hipError_t hipLaunchKernel(const void *, dim3, dim3, void **, size_t,
                           hipStream_t) {
  return hipErrorNotSupported;
}
const char *hipGetErrorString(hipError_t) { return ""; }
}

namespace adaln {
int fail(int code, const char *, ...) { return code; }
int ok() { return ADALN_OK; }
int check_ptr(const void *, bool, const char *) { return ADALN_OK; }
int check_segments(const int64_t *, const int32_t *, int64_t, int64_t, int64_t,
                   int) {
  return ADALN_OK;
}
int check_heads(const adaln_heads_t *, int64_t, int64_t, int64_t, int64_t, int,
                bool, const char *) {
  return ADALN_OK;
}

// As State::load() goes through a state, lane by lane.
template <typename T, int DP>
void walk(int d, bool across) {
  typedef State<T, DP> S;
  int least = 0, largest = 0;
  std::set<int> loaded;
  for (int c = 0; c < DP; ++c)
    for (int half = 0; half < 2; ++half)
      for (int m = 0; m < DP / 32; ++m)
        for (int r = 0; r < 16; r += 4) {
          const int row = 32 * m + 16 * (r / 8) + S::kY * (r / 4 % 2);
          const bool in = S::inside(d, c, half, row);
          const int first = S::first_at(d, c, half, across);
          for (int i = 0; i < 4; ++i) {
            const int at = first + (across ? (in ? row : 0) + i
                                           : in ? (row + i) * d : 0);
            least = std::min(least, at);
            largest = std::max(largest, at);
            if (in) loaded.insert(at);
          }
        }
  printf("%d %d %d\n", least, largest, (int)loaded.size());
}
template <typename T>
void walk(int d, bool across) {
  d <= 32   ? walk<T, 32>(d, across)
  : d <= 64 ? walk<T, 64>(d, across)
  : d <= 96 ? walk<T, 96>(d, across)
            : walk<T, 128>(d, across);
}
}  // namespace adaln

int main() {
  int dtype, d, across;
  while (scanf("%d %d %d", &dtype, &d, &across) == 3)
    dtype == ADALN_BF16 ? adaln::walk<adaln::bf16>(d, across)
                        : adaln::walk<float>(d, across);
  return 0;
}
