// The gated feed-forward's launch plans, on the host: for every line "dtype M
// D F" of the input, the tiling and the whole and sliced tiles of each product
// that the library would launch.
#include "../../adaln_fwd_amd/csrc/glu.hip"

#include <stdio.h>

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
}  // namespace adaln

int main() {
  using namespace adaln;
  int dtype;
  long long M, D, F;
  while (scanf("%d %lld %lld %lld", &dtype, &M, &D, &F) == 4) {
    const GluPlan f = glu_plan(kHidden, dtype, M, D, F);
    const GluBackward b = glu_backward(dtype, M, D, F);
    printf("%d %d  %d %d %d %d  %d %d %d %d  %d %d %d %d\n",
           (int)few_tokens(dtype, M, F), (int)b.joint, f.tiling, f.full, f.rem,
           f.slices, b.x.tiling, b.x.full, b.x.rem, b.x.slices, b.w.tiling,
           b.w.full, b.w.rem, b.w.slices);
  }
  return 0;
}
