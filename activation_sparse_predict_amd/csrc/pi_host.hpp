// Host helpers shared by the translation units of libpi.so.
#pragma once
#include "pi.h"

#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <utility>

namespace pih {

constexpr size_t kWsAlign = 256;   // alignment of every workspace and of its parts

inline size_t ws_align(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }
inline bool on(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t up_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// PI_OK, or PI_EHIP with the error kept for pi_last_hip_error (defined in pi_ffn.hip).
pi_status launched();

// Whether a launch in one dimension holds so many blocks: its threads are counted in 32 bits, and what is more is cut off
// without an error.
inline bool launches(int64_t blocks, int threads) { return blocks <= UINT32_MAX / threads; }

// Shape limits of a cache (pointers, sizes, alignment); see pi_cache in pi.h.
pi_status check_cache(const pi_cache* c);
// Alignment of a [tokens][heads][dim] tensor; see pi_heads in pi.h.
pi_status check_heads(const pi_heads* h, int32_t tokens);

// Whether rows of `dim` elements of an output lie over each other.
inline bool folded(const pi_heads* h, int64_t tokens, int64_t heads, int64_t dim) {
  int64_t s = std::abs(h->token_stride), ns = tokens, l = std::abs(h->head_stride), nl = heads;
  if (ns > 1 && s < dim) return true;
  if (nl > 1 && l < dim) return true;
  if (ns == 1 || nl == 1) return false;
  if (s > l) std::swap(s, l), std::swap(ns, nl);
  if (l >= s * (ns - 1) + dim) return false;       // one after the other, as tensors are laid out
  for (int64_t i = 1; i < heads; ++i) {
    const int64_t at = i * std::abs(h->head_stride), step = std::abs(h->token_stride), t = at / step;
    if ((t < tokens && at - t * step < dim) || (t + 1 < tokens && (t + 1) * step - at < dim)) return true;
  }
  return false;
}

}  // namespace pih
