// Host side of attention of chunks over a paged cache (pi.h): checks, workspace, launches.
#include "pi_chunk.hpp"

#include <algorithm>

#include "pi_attn_host.hpp"
#include "pi_chunk_host.hpp"

using namespace pih;

namespace {

// How a call is cut up.
struct Cut {
  int few;        // 16-row tiles of a block of k_chunk_few, or 0: k_attn_chunk
  int tile;       // rows of a block
  int64_t tiles;  // of rows, at most
  int free;       // shares beside one a tile
  int slots;      // for sums: tiles with several shares have fewer than twice as many of these as were dealt
  int rows;       // of a slot
};
Cut cut_of(const pi_cache* c, int tokens, int heads, int few) {
  const int64_t group = heads / c->kv_heads;
  Cut u{};
  u.few = few;
  u.tile = few ? 16 * few : pia::CH_ROWS;
  // Blocks that run at once: two, three or (wide heads) one for each compute unit.  (256, 512, 768 and 1024 blocks: one token
  // behind 1500, 32 heads, 14.2, 14.4, 14.3, 15.7 us; 8 single tokens with a bias behind up to 2900 57, 50, 52, 50; 32 single
  // tokens of 64 heads on 8 behind up to 4000 67, 58, 58, 65; 16 sequences of 5 drafts 55, 49, 58, 57; 512 tokens behind 32768
  // 346, 288, 298, 291; capped, heads of 256, 114, 139, 144, 157.)
  const int blocks = c->dim > 128 ? 256 : few == 1 || c->dim <= 64 ? 768 : 512;
  u.free = (int)up_div(blocks, c->kv_heads);
  u.slots = 2 * u.free;
  u.rows = (int)std::min<int64_t>(u.tile, up_div(tokens * group, 16) * 16);
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
// Of all ways a call with so many rows may go, so that room for more rows is room for fewer.
size_t ws_bytes_of(const pi_cache* c, int tokens, int heads) {
  size_t most = 0;
  for (int few = 0; few <= 2; ++few) most = std::max(most, ws_of(c, cut_of(c, tokens, heads, few)).total);
  return most;
}

pi_status check_sizes(const pi_cache* c, int32_t tokens, int32_t heads, int32_t n) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if (tokens < 0 || n < 1) return PI_EINVAL;
  if ((s = check_shape(heads, c->kv_heads, c->dim, c->dtype)) != PI_OK) return s;
  // rows and blocks are 32-bit numbers: a tile for every 16 rows, for each chunk and for each of 768 shares at most
  if (n > 4096 || (int64_t)tokens * heads > INT32_MAX / 2) return PI_EUNSUPPORTED;
  return PI_OK;
}

}  // namespace

extern "C" {

size_t pi_attn_chunk_workspace_bytes(const pi_cache* c, int32_t tokens, int32_t heads, int32_t n) {
  return check_sizes(c, tokens, heads, n) == PI_OK ? ws_bytes_of(c, tokens, heads) : 0;
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
  if (!ws || ws_bytes < ws_bytes_of(cache, tokens, heads) || !on(ws, kWsAlign)) return PI_EWORKSPACE;
  if (folded(out, tokens, heads, cache->dim)) return PI_EINVAL;
  const Cut u = cut_of(cache, tokens, heads, pish::few_tiles(tokens, n, heads / cache->kv_heads));
  const Ws W = ws_of(cache, u);
  const int64_t most = std::min(n, tokens);        // a tile of each chunk may be short
  const int64_t tiles = up_div((int64_t)tokens * (heads / cache->kv_heads), u.tile) + most;
  const int64_t blocks = (tiles + u.free) * cache->kv_heads;
  if (!launches(blocks, 64 * (u.few || cache->dim <= 128 ? 4 : 8))) return PI_EUNSUPPORTED;
  char* base = static_cast<char*>(ws);
  auto floats = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
  pia::ChunkCall call{};
  call.pg = pages_of(cache, layer);
  call.q = rows_of(q);
  call.out = static_cast<uint16_t*>(out->p), call.out_token = out->token_stride, call.out_head = out->head_stride;
  call.ch = pia::Chunks{cu, seqs, n, tokens, heads, cache->kv_heads, cache->dim, u.tile, u.free, u.slots, u.rows,
                       pish::divide_by(cache->page / 16)};
  call.sc = sc;
  call.count = reinterpret_cast<int32_t*>(base), call.joints = reinterpret_cast<pia::Joint*>(base + W.joints);
  call.part = floats(W.part), call.stat = floats(W.stat);
  call.mod = (cap > 0.f ? pia::CH_CAP : 0) | (slopes ? pia::CH_SLOPES : 0);
  call.few = u.few;
  call.blocks = (unsigned)blocks;
  call.stream = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (u.few) {
    pia::launch_few(cache->dtype, call);
  } else {
    with_type(cache->dtype, cache->dim, [&](auto t, auto d) {
      using T = decltype(t);
      constexpr int D = decltype(d)::value;
      pia::with_mod(call.mod, [&](auto m) { pia::launch(pia::k_attn_chunk<T, D, decltype(m)::value>, call, pia::ch_waves<D>()); });
    });
  }
  // rows of a block of the join: four a wave where there may be many blocks with nothing to do, else one.  (24 chunks of 1201
  // tokens, heads 64 wide, nothing to join: 78 us, 81 with one; wide heads, most tiles joined: 117 us, 110 with one.)
  const int each = u.rows >= 64 && cache->dim <= 128 ? 16 : 4;
  with_type(cache->dtype, cache->dim, [&](auto t, auto d) {
    constexpr int D = decltype(d)::value;
    hipLaunchKernelGGL((pia::k_chunk_join<decltype(t), D <= 64 ? 16 : D <= 128 ? 32 : 64>),
                       dim3((unsigned)(std::min<int64_t>(u.free, tiles) * cache->kv_heads), (unsigned)up_div(u.rows, each)),
                       dim3(256), 0, call.stream, call.joints, call.count, call.part, call.stat, call.out, call.out_token,
                       call.out_head, call.ch);
  });
  return launched();
}

}  // extern "C"
