// Host side of the attention operators (pi.h): checks, workspace, launches.
#include "pi_attn.hpp"

#include <algorithm>

#include "pi_attn_host.hpp"

using namespace pih;

namespace {

// How a decode call is cut up.
struct Cut {
  int tiles;      // 16-query tiles of a key head's group, over all key heads
  int free;       // shares of the rows' keys to deal, beside one for each row
  int least;      // units of a share at least, where a row has several
  int blocks;     // for each such tile
  int qtiles;     // 128-query tiles of a key head over the whole batch, for the common keys
  int shares;     // of the common keys at most
};
Cut cut_of(const pi_cache* c, int batch, int heads) {
  Cut u{};
  const int group = heads / c->kv_heads;
  u.tiles = c->kv_heads * (int)up_div(group, 16);
  // two blocks for each compute unit, beside a row's first.  Where the first ones fill the card, only what is longer than 8
  // units and than twice the average is dealt.  (32 rows of 32 heads on 32, 128 wide, 500 tokens and one row of 32768:
  // 1642 us with one share a row, 178 so, 180 with all dealt; 100 tokens each 12.9, 13.5, 16.8 us; 1500 each 146, 150, 151;
  // 1024 rows of one key head, 300 tokens each, 17.0, 16.9, 32.)
  u.least = (int64_t)batch * u.tiles >= pia::DC_ROWS ? 8 : 1;
  u.free = pish::units_of(c->max_pages * c->page) > u.least ? (int)up_div(512, u.tiles) : 0;
  u.blocks = batch + u.free;
  // of the common keys as many shares as make two blocks for each compute unit: three would fit for heads up to 64 wide, but
  // there are more sums then.  (512 and 768 blocks: 32 rows behind 4096 tokens, 128 wide, 36.6 and 37.9 us; 24 behind 32768,
  // 64 wide, 73 and 76 us.)
  u.qtiles = (int)up_div((int64_t)batch * group, 128);
  u.shares = (int)std::max<int64_t>(1, std::min<int64_t>(64, 512 / ((int64_t)u.qtiles * c->kv_heads)));
  return u;
}

struct Ws {
  size_t cpart, cstat, part, stat, total;
};
Ws ws_of(const pi_cache* c, int batch, int heads) {
  const Cut u = cut_of(c, batch, heads);
  const size_t crows = (size_t)batch * heads * u.shares, rows = (size_t)u.blocks * u.tiles * 16;
  Ws w{};
  w.cpart = ws_align(sizeof(int4) * batch);
  w.cstat = w.cpart + ws_align(sizeof(float) * crows * c->dim);
  w.part = w.cstat + ws_align(sizeof(float) * 2 * crows);
  w.stat = w.part + ws_align(sizeof(float) * rows * c->dim);
  w.total = w.stat + ws_align(sizeof(float) * 2 * rows);
  return w;
}

pi_status check_batch(const pi_cache* c, int32_t batch, int32_t heads) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if (batch < 1) return PI_EINVAL;
  if ((s = check_shape(heads, c->kv_heads, c->dim, c->dtype)) != PI_OK) return s;
  return batch > 4096 ? PI_EUNSUPPORTED : PI_OK;
}

}  // namespace

pi_status pih::check_heads(const pi_heads* h, int32_t tokens) {
  if (!h || (!h->p && tokens > 0) || !on(h->p, 16)) return PI_EINVAL;
  return h->token_stride % 8 != 0 || h->head_stride % 8 != 0 ? PI_EINVAL : PI_OK;
}

extern "C" {

pi_status pi_attn_prompt(const pi_heads* q, const pi_heads* k, const pi_heads* v, const pi_heads* out, int32_t tokens,
                         int32_t heads, int32_t kv_heads, int32_t dim, int32_t dtype, const int32_t* cu, int32_t n,
                         float scale, void* stream) {
  pi_status s;
  if ((s = check_shape(heads, kv_heads, dim, dtype)) != PI_OK) return s;
  if (tokens < 0 || n < 1 || !cu || !on(cu, 4)) return PI_EINVAL;
  for (const pi_heads* h : {q, k, v, out})
    if ((s = check_heads(h, tokens)) != PI_OK) return s;
  float c;
  if (!scale_of(scale, dim, &c)) return PI_EINVAL;
  for (const pi_heads* h : {k, v})                 // byte offsets inside a tile are 32-bit
    if (h->token_stride < 0 || h->token_stride > (1 << 24)) return PI_EUNSUPPORTED;
  if (tokens == 0) return PI_OK;
  // heads of a block: as many of those that share their keys as 4 waves take
  const int group = heads / kv_heads;
  const int hg = group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1, rows = 128 / hg;
  // a tile of each sequence may be short
  const int64_t blocks = (up_div(tokens, rows) + std::min(n, tokens)) * (heads / hg);
  if (!launches(blocks, 256)) return PI_EUNSUPPORTED;
  if (folded(out, tokens, heads, dim)) return PI_EINVAL;
  (void)hipGetLastError();
  with_type(dtype, dim, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), rows_of(q),
                         rows_of(k), rows_of(v), static_cast<uint16_t*>(out->p), out->token_stride, out->head_stride,
                         cu, n, tokens, heads, group, dim, c);
    };
    if (hg == 4) go(pia::k_attn_prompt<T, D, 4>);
    else if (hg == 2) go(pia::k_attn_prompt<T, D, 2>);
    else go(pia::k_attn_prompt<T, D, 1>);
  });
  return launched();
}

size_t pi_attn_workspace_bytes(const pi_cache* c, int32_t batch, int32_t heads) {
  return check_batch(c, batch, heads) == PI_OK ? ws_of(c, batch, heads).total : 0;
}

pi_status pi_attn_decode(const pi_cache* cache, int32_t layer, const pi_heads* q, const pi_heads* out, int32_t batch,
                         int32_t heads, const int32_t* seqs, const int32_t* prefix, float scale, void* ws,
                         size_t ws_bytes, void* stream) {
  pi_status s;
  if ((s = check_batch(cache, batch, heads)) != PI_OK) return s;
  if (layer < 0 || layer >= cache->layers || !on(seqs, 4) || !on(prefix, 4)) return PI_EINVAL;
  if (!seqs && batch > cache->slots) return PI_EINVAL;
  if ((s = check_heads(q, batch)) != PI_OK || (s = check_heads(out, batch)) != PI_OK) return s;
  float c;
  if (!scale_of(scale, cache->dim, &c)) return PI_EINVAL;
  const Ws W = ws_of(cache, batch, heads);
  if (!ws || ws_bytes < W.total || !on(ws, kWsAlign)) return PI_EWORKSPACE;
  if (folded(out, batch, heads, cache->dim)) return PI_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Cut u = cut_of(cache, batch, heads);
  const int dim = cache->dim;
  char* base = static_cast<char*>(ws);
  auto floats = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  const pia::Pages pg = pages_of(cache, layer);
  (void)hipGetLastError();
  with_type(cache->dtype, dim, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    if (prefix)
      hipLaunchKernelGGL((pia::k_attn_common<T, D>),
                         dim3((unsigned)(8 * up_div((int64_t)cache->kv_heads * u.shares, 8) * u.qtiles)), dim3(256), 0,
                         st, pg, rows_of(q), seqs, prefix, batch, heads, cache->kv_heads, dim, u.shares, u.qtiles, c,
                         floats(W.cpart), floats(W.cstat));
    hipLaunchKernelGGL((pia::k_attn_decode<T, D>), dim3((unsigned)u.blocks, (unsigned)u.tiles + (prefix ? 1 : 0)),
                       dim3(pia::DC_WAVES * pia::WAVE), 0, st, pg, rows_of(q), static_cast<uint16_t*>(out->p),
                       out->token_stride, out->head_stride, seqs, prefix, batch, heads, cache->kv_heads, dim, u.free,
                       u.least, u.shares, c, reinterpret_cast<int4*>(base), floats(W.part), floats(W.stat));
    if (prefix || u.free)
      hipLaunchKernelGGL((pia::k_attn_join<T, D <= 64 ? 16 : D <= 128 ? 32 : 64>), dim3((unsigned)up_div((int64_t)batch * heads, 4)),
                         dim3(256), 0, st, reinterpret_cast<const int4*>(base), floats(W.cpart), floats(W.cstat),
                         floats(W.part), floats(W.stat), static_cast<uint16_t*>(out->p), out->token_stride,
                         out->head_stride, batch, heads, cache->kv_heads, dim, u.shares);
  });
  return launched();
}

}  // extern "C"
