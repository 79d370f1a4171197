// Host helpers shared by the translation units of the attention operators.
#pragma once
#include "pi_attn.hpp"

#include <cmath>

#include "pi_host.hpp"

namespace pih {

inline pi_status check_shape(int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || dim < 8 || dim % 8 != 0) return PI_EINVAL;
  if (dtype != PI_F16 && dtype != PI_BF16) return dtype == PI_F32 ? PI_EUNSUPPORTED : PI_EINVAL;
  if (dim > 256 || heads > 4096) return PI_EUNSUPPORTED;
  return PI_OK;
}

// 2^x instead of e^x: c = scale log2(e); false if the scale is not finite and positive
inline bool scale_of(float scale, int dim, float* c) {
  const double s = scale == 0.f ? 1.0 / std::sqrt((double)dim) : (double)scale;
  *c = (float)(s * 1.4426950408889634);
  return std::isfinite(*c) && *c > 0.f;
}

inline pia::Rows rows_of(const pi_heads* h) {
  return pia::Rows{static_cast<const uint16_t*>(h->p), h->token_stride, h->head_stride};
}

// f(a value of the element type, a constant of the padded dim)
template <class F>
void with_type(int dtype, int dim, F f) {
  auto by_dim = [&](auto t) {
    if (dim <= 64) f(t, std::integral_constant<int, 64>());
    else if (dim <= 96) f(t, std::integral_constant<int, 96>());
    else if (dim <= 128) f(t, std::integral_constant<int, 128>());
    else f(t, std::integral_constant<int, 256>());
  };
  if (dtype == PI_F16) by_dim(pit::H16());
  else by_dim(pit::B16());
}

// What the kernels see of a cache's layer.
inline pia::Pages pages_of(const pi_cache* c, int32_t layer) {
  const int64_t at = (int64_t)layer * c->pages * c->kv_heads * c->page * c->dim;
  int32_t* lens = c->meta + (int64_t)c->slots * c->max_pages;
  return pia::Pages{static_cast<const uint16_t*>(c->k) + at,
                    static_cast<const uint16_t*>(c->v) + at,
                    c->meta,
                    lens,
                    lens + c->slots + 2 * (int64_t)c->pages + 1,
                    c->pages,
                    c->page,
                    c->max_pages,
                    c->slots};
}

}  // namespace pih
