// sizes.h -- arithmetic on sizes that host code shares, with no HIP in it.  Not part
// of the public ABI.
#pragma once

#include <cstdint>

#include "rar.h"

namespace rar {

constexpr int64_t kMaxLanes = (int64_t(1) << 32) - 1;  // of a grid, along x

inline int esize(rar_dtype d) { return d == RAR_BF16 ? 2 : 4; }
inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
inline int64_t div_up(int64_t v, int64_t by) { return (v + by - 1) / by; }

}  // namespace rar
