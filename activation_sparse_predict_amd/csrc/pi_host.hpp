// Host helpers shared by the translation units of libpi.so.
#pragma once
#include "pi.h"

#include <cstddef>
#include <cstdint>

namespace pih {

constexpr size_t kWsAlign = 256;   // alignment of every workspace and of its parts

inline size_t ws_align(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }
inline bool on(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t up_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// PI_OK, or PI_EHIP with the error kept for pi_last_hip_error (defined in pi_ffn.hip).
pi_status launched();

// Shape limits of a cache (pointers, sizes, alignment); see pi_cache in pi.h.
pi_status check_cache(const pi_cache* c);
// Alignment of a [tokens][heads][dim] tensor; see pi_heads in pi.h.
pi_status check_heads(const pi_heads* h, int32_t tokens);

}  // namespace pih
