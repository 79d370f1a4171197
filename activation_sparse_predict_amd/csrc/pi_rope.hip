// Host side of rotary positions and norms of heads (pi.h): frequencies, checks, launches.
#include "pi_rope.hpp"

#include <algorithm>
#include <cmath>

#include "pi_host.hpp"

using namespace pih;

namespace {

constexpr double TURN = 6.283185307179586476925;

// A head's tensors that a call reads or writes: none at all, or all of them.
pi_status check_part(const pi_heads* x, const pi_heads* out, int32_t heads, int32_t tokens, int32_t dim) {
  if (heads == 0 && !x && !out) return PI_OK;
  if (heads < 1) return PI_EINVAL;
  if (heads > 4096) return PI_EUNSUPPORTED;
  pi_status s;
  if ((s = check_heads(x, tokens)) != PI_OK || (s = check_heads(out, tokens)) != PI_OK) return s;
  return folded(out, tokens, heads, dim) ? PI_EINVAL : PI_OK;
}

pi_status check_rope(const pi_rope* r, int32_t dim) {
  if (!r) return PI_OK;
  if (!r->steps || !on(r->steps, 16) || r->rotary < 2 || r->rotary % 2 != 0 || r->rotary > dim) return PI_EINVAL;
  if (r->layout != PI_ROPE_HALF && r->layout != PI_ROPE_PAIRS) return PI_EINVAL;
  return std::isfinite(r->magnitude) && r->magnitude >= 0.f ? PI_OK : PI_EINVAL;
}

pi_status check_norms(const float* q_norm, const float* k_norm, float eps) {
  if (!on(q_norm, 16) || !on(k_norm, 16)) return PI_EINVAL;
  return (q_norm || k_norm) && !(std::isfinite(eps) && eps > 0.f) ? PI_EINVAL : PI_OK;
}

pir::Part part_of(const pi_heads* x, const pi_heads* out, int32_t heads, const float* weight) {
  pir::Part p{};
  if (heads == 0) return p;
  p.src = static_cast<const uint16_t*>(x->p), p.src_token = x->token_stride, p.src_head = x->head_stride;
  if (out) p.dst = static_cast<uint16_t*>(out->p), p.dst_token = out->token_stride, p.dst_head = out->head_stride;
  p.weight = weight, p.heads = heads;
  return p;
}

pi_status launch(bool paged, int dtype, const pi_rope* r, const pir::Part& q, const pir::Part& k, const pir::Part& v,
                 const int32_t* pos, const pic::Meta& m, const int32_t* cu, const int32_t* seqs, int n,
                 int tokens, int dim, float eps, void* stream) {
  const int rotary = r ? r->rotary : 0;
  const int mode = !r ? pir::NONE : r->layout == PI_ROPE_PAIRS ? pir::PAIRS : rotary % 16 == 0 ? pir::HALF : pir::ODD;
  const int lanes = mode == pir::ODD ? (int)(up_div(rotary / 2, 8) + up_div(dim - rotary, 16)) : (int)up_div(dim, 16);
  int shift = 0;
  while (1 << shift < lanes) ++shift;
  const int per = 64 >> shift;                                  // heads of a wave's turn, all of one kind
  const int turns = (int)(up_div(q.heads, per) + up_div(k.heads, per) + up_div(v.heads, per));
  // waves that the card does not hold at once anyway make the angles for several turns
  const int64_t all = (int64_t)tokens * turns;
  const int its = all >= 16384 && turns > 2 ? 4 : all >= 8192 && turns > 1 ? 2 : 1;
  const int waves = (int)up_div(turns, its);                    // of a token
  if ((int64_t)tokens * waves > INT32_MAX) return PI_EUNSUPPORTED;
  const pir::Turn turn{r ? r->steps : nullptr, rotary, !r || r->magnitude == 0.f ? 1.f : r->magnitude};
  // a launch counts the threads of a dimension in 32 bits, and what is more is cut off without an error
  const int64_t blocks = up_div((int64_t)tokens * waves, 4);
  const unsigned across = (unsigned)std::min<int64_t>(blocks, 1 << 23);
  (void)hipGetLastError();
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(across, (unsigned)up_div(blocks, across)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), turn, q, k, v, pos, m, cu, seqs, n, tokens, dim, eps, shift, (uint32_t)waves);
  };
  auto with_its = [&](auto t, auto m, auto p) {
    using T = decltype(t);
    constexpr int M = decltype(m)::value;
    constexpr bool P = decltype(p)::value;
    if (its == 1) go(pir::k_rope<T, M, P, 1>);
    else if (its == 2) go(pir::k_rope<T, M, P, 2>);
    else go(pir::k_rope<T, M, P, 4>);
  };
  auto with_mode = [&](auto t, auto p) {
    if (mode == pir::NONE) with_its(t, std::integral_constant<int, pir::NONE>(), p);
    else if (mode == pir::HALF) with_its(t, std::integral_constant<int, pir::HALF>(), p);
    else if (mode == pir::PAIRS) with_its(t, std::integral_constant<int, pir::PAIRS>(), p);
    else with_its(t, std::integral_constant<int, pir::ODD>(), p);
  };
  auto with_pages = [&](auto t) {
    if (paged) with_mode(t, std::true_type());
    else with_mode(t, std::false_type());
  };
  if (dtype == PI_F16) with_pages(pit::H16());
  else with_pages(pit::B16());
  return launched();
}

}  // namespace

extern "C" {

pi_status pi_rope_freqs(const pi_rope_scaling* sc, int32_t rotary, double* freqs, float* magnitude) {
  if (!sc || !freqs || rotary < 2 || rotary % 2 != 0 || rotary > 256) return PI_EINVAL;
  if (!(std::isfinite(sc->base) && sc->base > 1.0) || sc->rule < PI_ROPE_PLAIN || sc->rule > PI_ROPE_RAMP) return PI_EINVAL;
  const bool scaled = sc->rule != PI_ROPE_PLAIN, bands = sc->rule == PI_ROPE_BANDS, ramp = sc->rule == PI_ROPE_RAMP;
  if (scaled && !(std::isfinite(sc->factor) && sc->factor >= 1.0)) return PI_EINVAL;
  if ((bands || ramp) && !(std::isfinite(sc->trained) && sc->trained > 0.0 && sc->low > 0.0 && sc->high > sc->low &&
                           std::isfinite(sc->high)))
    return PI_EINVAL;
  if (sc->rule == PI_ROPE_BASE && rotary == 2) return PI_EINVAL;
  const double r = rotary, factor = scaled ? sc->factor : 1.0;
  const double base = sc->rule == PI_ROPE_BASE ? sc->base * std::pow(factor, r / (r - 2.0)) : sc->base;
  double from = 0.0, to = 0.0;
  if (ramp) {
    auto pair_of = [&](double turns) { return r * std::log(sc->trained / (TURN * turns)) / (2.0 * std::log(base)); };
    from = std::max(std::floor(pair_of(sc->high)), 0.0);
    to = std::min(std::ceil(pair_of(sc->low)), r - 1.0);
    if (to == from) to += 0.001;
  }
  for (int32_t i = 0; i < rotary / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    double own = 1.0;                                           // how much of the pair's own frequency stays
    if (sc->rule == PI_ROPE_LINEAR) own = 0.0;
    else if (bands) own = (sc->trained * f / TURN - sc->low) / (sc->high - sc->low);
    else if (ramp) own = 1.0 - (i - from) / (to - from);
    own = std::min(1.0, std::max(0.0, own));
    freqs[i] = f * own + f / factor * (1.0 - own);
  }
  if (magnitude) *magnitude = ramp ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return PI_OK;
}

pi_status pi_rope_steps(const double* freqs, int32_t n, uint64_t* steps) {
  if (!freqs || !steps || n < 1) return PI_EINVAL;
  for (int32_t i = 0; i < n; ++i)
    if (!std::isfinite(freqs[i])) return PI_EINVAL;
  for (int32_t i = 0; i < n; ++i) {
    // a long double has 64 bits: those of the part of a turn are all kept
    const long double turns = (long double)freqs[i] / 6.283185307179586476925286766559L;
    const long double part = turns - floorl(turns);
    const long double step = roundl(part * 18446744073709551616.0L);
    steps[i] = step >= 18446744073709551616.0L ? 0 : (uint64_t)step;
  }
  return PI_OK;
}

pi_status pi_rope_heads(const pi_rope* rope, const int32_t* pos, const pi_heads* q, const pi_heads* q_out, int32_t heads,
                        const float* q_norm, const pi_heads* k, const pi_heads* k_out, int32_t kv_heads,
                        const float* k_norm, float eps, int32_t tokens, int32_t dim, int32_t dtype, void* stream) {
  if (dim < 8 || dim % 8 != 0 || tokens < 0 || heads < 1) return PI_EINVAL;
  if (dtype != PI_F16 && dtype != PI_BF16) return dtype == PI_F32 ? PI_EUNSUPPORTED : PI_EINVAL;
  if (dim > 256) return PI_EUNSUPPORTED;
  pi_status s;
  if ((s = check_rope(rope, dim)) != PI_OK || (s = check_norms(q_norm, k_norm, eps)) != PI_OK) return s;
  if (rope && (!on(pos, 4) || (!pos && tokens > 0))) return PI_EINVAL;
  if ((s = check_part(q, q_out, heads, tokens, dim)) != PI_OK) return s;
  if ((s = check_part(k, k_out, kv_heads, tokens, dim)) != PI_OK) return s;
  if (tokens == 0) return PI_OK;
  return launch(false, dtype, rope, part_of(q, q_out, heads, q_norm), part_of(k, k_out, kv_heads, k_norm), pir::Part{},
                pos, pic::Meta{}, nullptr, nullptr, 0, tokens, dim, eps, stream);
}

pi_status pi_cache_append_rope(const pi_cache* c, int32_t layer, const pi_rope* rope, const pi_heads* q,
                               const pi_heads* q_out, int32_t heads, const float* q_norm, const pi_heads* k,
                               const pi_heads* v, const float* k_norm, float eps, int32_t tokens, const int32_t* cu,
                               const int32_t* seqs, int32_t n, void* stream) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if (layer < 0 || layer >= c->layers || tokens < 0 || n < 1 || !cu || !on(cu, 4) || !seqs || !on(seqs, 4))
    return PI_EINVAL;
  if ((s = check_rope(rope, c->dim)) != PI_OK || (s = check_norms(q_norm, k_norm, eps)) != PI_OK) return s;
  if ((s = check_part(q, q_out, heads, tokens, c->dim)) != PI_OK) return s;
  if ((s = check_heads(k, tokens)) != PI_OK || (s = check_heads(v, tokens)) != PI_OK) return s;
  if (tokens == 0) return PI_OK;
  const int64_t at = (int64_t)layer * c->pages * c->kv_heads * c->page * c->dim;
  pir::Part kp = part_of(k, nullptr, c->kv_heads, k_norm), vp = part_of(v, nullptr, c->kv_heads, nullptr);
  kp.dst = static_cast<uint16_t*>(c->k) + at;
  vp.dst = static_cast<uint16_t*>(c->v) + at;
  return launch(true, c->dtype, rope, part_of(q, q_out, heads, q_norm), kp, vp, nullptr,
                pic::meta_of(c), cu, seqs, n, tokens, c->dim, eps, stream);
}

}  // extern "C"
