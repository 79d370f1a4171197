// Host side of attention of chunks over a paged cache (pi.h): checks, workspace, launches.
#include "pi_chunk.hpp"

#include <algorithm>

#include "pi_attn_host.hpp"

using namespace pih;

namespace {

constexpr int BLOCKS = 512;              // blocks that shares are dealt to: two for each compute unit

// How a call is cut up.
struct Cut {
  int64_t tiles;  // of rows, at most
  int free;       // shares beside one a tile
  int slots;      // for sums: tiles with several shares have fewer than twice as many of these as were dealt
  int rows;       // of a slot
};
Cut cut_of(const pi_cache* c, int tokens, int heads, int n) {
  Cut u{};
  const int64_t group = heads / c->kv_heads;
  u.tiles = up_div(tokens * group, pia::CH_ROWS) + std::min(n, tokens);
  u.free = (int)up_div(BLOCKS, c->kv_heads);
  u.slots = 2 * u.free;
  u.rows = (int)std::min<int64_t>(pia::CH_ROWS, up_div(tokens * group, 32) * 32);
  return u;
}

struct Ws {
  size_t joints, part, stat, total;
};
Ws ws_of(const pi_cache* c, const Cut& u) {
  const size_t rows = (size_t)u.slots * c->kv_heads * u.rows;
  Ws w{};
  w.joints = kWsAlign;
  w.part = w.joints + ws_align(sizeof(pia::Joint) * u.slots);
  w.stat = w.part + ws_align(sizeof(float) * rows * c->dim);
  w.total = w.stat + ws_align(sizeof(float) * 2 * rows);
  return w;
}

pi_status check_sizes(const pi_cache* c, int32_t tokens, int32_t heads, int32_t n) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if (tokens < 0 || n < 1) return PI_EINVAL;
  if ((s = check_shape(heads, c->kv_heads, c->dim, c->dtype)) != PI_OK) return s;
  // rows and blocks are 32-bit numbers
  if (n > 4096 || (int64_t)tokens * heads > INT32_MAX - 127) return PI_EUNSUPPORTED;
  const Cut u = cut_of(c, tokens, heads, n);
  return (u.tiles + u.free) * c->kv_heads > INT32_MAX ? PI_EUNSUPPORTED : PI_OK;
}

}  // namespace

extern "C" {

size_t pi_attn_chunk_workspace_bytes(const pi_cache* c, int32_t tokens, int32_t heads, int32_t n) {
  return check_sizes(c, tokens, heads, n) == PI_OK ? ws_of(c, cut_of(c, tokens, heads, n)).total : 0;
}

pi_status pi_attn_chunk(const pi_cache* cache, int32_t layer, const pi_heads* q, const pi_heads* out, int32_t tokens,
                        int32_t heads, const int32_t* cu, const int32_t* seqs, int32_t n, float scale, float cap,
                        const float* slopes, int32_t window, void* ws, size_t ws_bytes, void* stream) {
  pi_status s;
  if ((s = check_sizes(cache, tokens, heads, n)) != PI_OK) return s;
  if (layer < 0 || layer >= cache->layers || !cu || !on(cu, 4) || !on(seqs, 4) || !on(slopes, 4) || window < 0)
    return PI_EINVAL;
  if (!seqs && n > cache->slots) return PI_EINVAL;
  if ((s = check_heads(q, tokens)) != PI_OK || (s = check_heads(out, tokens)) != PI_OK) return s;
  pia::ChunkScore sc{};
  if (!scale_of(scale, cache->dim, &sc.c) || !(cap >= 0.f)) return PI_EINVAL;
  if (cap > 1024.f) return PI_EUNSUPPORTED;
  if (cap > 0.f) {
    sc.pre = (float)(2.0 * sc.c / cap), sc.cap = (float)(cap * 1.4426950408889634);
    if (!std::isfinite(sc.pre) || sc.cap < 1e-30f) return PI_EINVAL;
  }
  sc.slopes = slopes, sc.window = window;
  if (tokens == 0) return PI_OK;
  const Cut u = cut_of(cache, tokens, heads, n);
  const Ws W = ws_of(cache, u);
  if (!ws || ws_bytes < W.total || !on(ws, kWsAlign)) return PI_EWORKSPACE;
  if (folded(out, tokens, heads, cache->dim)) return PI_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* base = static_cast<char*>(ws);
  int32_t* count = reinterpret_cast<int32_t*>(base);
  auto* joints = reinterpret_cast<pia::Joint*>(base + W.joints);
  auto floats = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  // the page of a place of 16 keys by a multiplication: ceil(2^(31 + shift) / per) is off by less than 1, and with
  // 2^shift <= per < 2^(shift + 1) that changes no quotient of a place below 2^30
  const uint32_t per = cache->page / 16;
  uint32_t shift = 0;
  while (per >> (shift + 1)) ++shift;
  const uint32_t mul = (uint32_t)(((uint64_t(1) << (31 + shift)) + per - 1) / per);
  const pia::Chunks ch{cu, seqs, n, tokens, heads, cache->kv_heads, cache->dim, u.free, 1, u.slots, u.rows, mul, shift};
  const pia::Pages pg = pages_of(cache, layer);
  uint16_t* dst = static_cast<uint16_t*>(out->p);
  (void)hipGetLastError();
  with_type(cache->dtype, cache->dim, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)((u.tiles + u.free) * cache->kv_heads)), dim3(256), 0, st, pg, rows_of(q),
                         dst, out->token_stride, out->head_stride, ch, sc, joints, count, floats(W.part), floats(W.stat));
    };
    if (cap > 0.f && slopes) go(pia::k_attn_chunk<T, D, pia::CH_CAP | pia::CH_SLOPES>);
    else if (cap > 0.f) go(pia::k_attn_chunk<T, D, pia::CH_CAP>);
    else if (slopes) go(pia::k_attn_chunk<T, D, pia::CH_SLOPES>);
    else go(pia::k_attn_chunk<T, D, 0>);
    hipLaunchKernelGGL(pia::k_chunk_join<T>,
                       dim3((unsigned)(std::min<int64_t>(u.free, u.tiles) * cache->kv_heads), (unsigned)(u.rows / 4)),
                       dim3(256), 0, st, joints, count, floats(W.part), floats(W.stat), dst, out->token_stride,
                       out->head_stride, ch);
  });
  return launched();
}

}  // extern "C"
