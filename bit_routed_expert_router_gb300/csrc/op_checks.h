// Argument checks that the operators' C entry points share.
#pragma once

#include <cstdint>

#include "moe.h"

namespace moe {

constexpr int kMaxExperts = 1024, kMaxSide = 65536, kMaxRows = 1 << 24;

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// m rows of values of which `unit` are 16 bytes, that the TMA engine or 16-byte accesses can take (no rows need no memory)
inline bool rows_ok(const void* p, int m, int64_t ld, int64_t cols, int unit = 8) {
  return (p || m == 0) && aligned(p, 16) && ld >= cols && ld % unit == 0 && ld < (int64_t{1} << 36);
}

inline bool gelu_ok(int v) { return v == MOE_GELU_ERF || v == MOE_GELU_TANH; }

inline moe_status status(bool ok) { return ok ? MOE_OK : MOE_ECUDA; }

}  // namespace moe
