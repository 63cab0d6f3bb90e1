// checks.h -- argument checks and workspace layout shared by the C entry points.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace invmoe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The first of two arrays of n bytes is the second, or they have no byte in common (or one is absent).
inline bool same_or_apart(const void* a, const void* b, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a == nullptr || b == nullptr || (x > y ? x - y : y - x) >= n || x == y;
}

inline size_t route_ws(int T, int E) {
  const size_t NC = (static_cast<size_t>(T) + kDispatchChunk - 1) / kDispatchChunk;
  return align_up(NC * static_cast<size_t>(E) * sizeof(int32_t), 256);
}

inline unsigned int* status_word(void* ws) { return static_cast<unsigned int*>(ws); }
inline uint8_t* scratch(void* ws) { return static_cast<uint8_t*>(ws) + kStatusBytes; }

}  // namespace invmoe

#define REQUIRE(cond, code, ...)             \
  do {                                       \
    if (!(cond)) return set_error(code, __VA_ARGS__); \
  } while (0)

#define REQUIRE_PTR(p) REQUIRE((p) != nullptr, INVMOE_ERR_INVALID_ARG, "%s is NULL", #p)
#define REQUIRE_ALIGNED(p) REQUIRE(aligned16(p), INVMOE_ERR_MISALIGNED, "%s is not 16-byte aligned", #p)
