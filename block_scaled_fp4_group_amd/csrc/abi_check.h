// Argument checks shared by the C entry points: a failed check sets the
// calling thread's error message and returns MOE_ERR_INVALID.
#pragma once
#include "common.h"

namespace moe {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

#define MOE_CHECK(cond, ...)      \
  do {                            \
    if (!(cond)) {                \
      moe::set_error(__VA_ARGS__); \
      return MOE_ERR_INVALID;     \
    }                             \
  } while (0)

}  // namespace moe
