// Argument checks of the C ABI that several sources share.  Each returns
// ADALN_OK or records a message and returns an error code.
#pragma once

#include <stdint.h>

#include "adaln.h"
#include "launch.hpp"

#define ADALN_API extern "C" __attribute__((visibility("default")))

#define ADALN_TRY(expr)          \
  do {                           \
    const int rc_ = (expr);      \
    if (rc_ != ADALN_OK) return rc_; \
  } while (0)

namespace adaln {

// abi.hip: a [B, N, D] call, a pointer that is needed when its tensor has
// elements, and a segment table (host arrays).
int check_shape(int64_t B, int64_t N, int64_t D, int dtype);
int check_ptr(const void *p, bool needed, const char *name);
int check_segments(const int64_t *off, const int32_t *mod, int64_t nseg,
                   int64_t nmod, int64_t D, int dtype);

// heads.hip: one tensor of heads, its pointer, alignment and strides; an
// output's heads must not overlap.
int check_heads(const adaln_heads_t *t, int64_t B, int64_t N, int64_t H,
                int64_t d, int dtype, bool output, const char *name);

}  // namespace adaln
