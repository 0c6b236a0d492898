// Integer helpers of the host code.
#pragma once

#include <stdint.h>

namespace mx {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t hmin(int64_t a, int64_t b) { return a < b ? a : b; }

}  // namespace mx
