// Host side of the paged key/value cache (pi.h): checks, workspace, launches.
#include "pi_cache.hpp"

#include <algorithm>

#include "pi_host.hpp"

using namespace pih;

namespace {

pic::Meta meta_of(const pi_cache* c) {
  int32_t* table = c->meta;
  int32_t* lens = table + (int64_t)c->slots * c->max_pages;
  int32_t* ref = lens + c->slots;
  return pic::Meta{table, lens, ref, ref + c->pages, ref + 2 * (int64_t)c->pages, c->slots, c->max_pages, c->pages,
                   c->page};
}

// plan: count, sources, targets; then the map of a compaction
struct Ws {
  size_t src, dst, to, total;
};
Ws ws_of(const pi_cache* c) {
  Ws w{};
  w.src = kWsAlign;
  // a fork copies at most a page per child, a compaction at most half the pool
  w.dst = w.src + ws_align(sizeof(int32_t) * (size_t)c->pages);
  w.to = w.dst + ws_align(sizeof(int32_t) * (size_t)c->pages);
  w.total = w.to + ws_align(sizeof(int32_t) * (size_t)c->pages);
  return w;
}
pic::Plan plan_of(const pi_cache* c, void* ws) {
  char* b = static_cast<char*>(ws);
  const Ws w = ws_of(c);
  return pic::Plan{reinterpret_cast<int32_t*>(b), reinterpret_cast<int32_t*>(b + w.src),
                   reinterpret_cast<int32_t*>(b + w.dst)};
}

pi_status check_ws(const pi_cache* c, const void* ws, size_t bytes) {
  return !ws || bytes < ws_of(c).total || !on(ws, kWsAlign) ? PI_EWORKSPACE : PI_OK;
}

pi_status check_list(const int32_t* list, int32_t n) {
  if (!list || !on(list, 4) || n < 1) return PI_EINVAL;
  return n > pic::MAX_N ? PI_EUNSUPPORTED : PI_OK;
}

// Enough blocks to fill the chip several times over; each block takes whole pages.  to: the map that the tables follow
// (a compaction's), or NULL.
void copy_pages(const pi_cache* c, int most, const pic::Plan& plan, const int32_t* to, int32_t* moved, hipStream_t st) {
  const int64_t chunks = (int64_t)c->kv_heads * c->page * c->dim / 8;
  int x = std::max(1, std::min(most, (int)up_div(4096, 2 * c->layers)));
  if (to) x = std::max(x, 64);                     // the tables' blocks
  hipLaunchKernelGGL(pic::k_cache_copy, dim3(x, 2 * c->layers + (to ? 1 : 0)), dim3(256), 0, st,
                     static_cast<pit::u4*>(c->k), static_cast<pit::u4*>(c->v), chunks * c->pages, (int)chunks,
                     c->layers, plan, meta_of(c), to, moved);
}

}  // namespace

pi_status pih::check_cache(const pi_cache* c) {
  if (!c || !c->k || !c->v || !c->meta) return PI_EINVAL;
  if (!on(c->k, 16) || !on(c->v, 16) || !on(c->meta, 4)) return PI_EINVAL;
  if (c->layers < 1 || c->pages < 1 || c->kv_heads < 1 || c->page < 1 || c->dim < 1 || c->slots < 1 ||
      c->max_pages < 1)
    return PI_EINVAL;
  if (c->dtype != PI_F16 && c->dtype != PI_BF16) return c->dtype == PI_F32 ? PI_EUNSUPPORTED : PI_EINVAL;
  if (c->dim % 8 != 0 || c->page % 16 != 0) return PI_EINVAL;
  if (c->dim > 256 || c->page > 4096 || c->kv_heads > 1024 || c->pages > (1 << 20) || c->layers > 16384)
    return PI_EUNSUPPORTED;
  // lengths, with a tile of keys behind them, and table entries are 32-bit
  if ((int64_t)c->max_pages * c->page > INT32_MAX - 127 || (int64_t)c->slots * c->max_pages > (int64_t(1) << 30))
    return PI_EUNSUPPORTED;
  return PI_OK;
}

extern "C" {

size_t pi_cache_meta_words(int32_t slots, int32_t max_pages, int32_t pages) {
  if (slots < 1 || max_pages < 1 || pages < 1) return 0;
  return (size_t)slots * max_pages + slots + 2 * (size_t)pages + 4;
}

size_t pi_cache_workspace_bytes(const pi_cache* c) { return check_cache(c) == PI_OK ? ws_of(c).total : 0; }

pi_status pi_cache_extend(const pi_cache* c, const int32_t* seqs, const int32_t* counts, int32_t n, void* stream) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if ((s = check_list(seqs, n)) != PI_OK || (s = check_list(counts, n)) != PI_OK) return s;
  (void)hipGetLastError();
  hipLaunchKernelGGL(pic::k_cache_extend, dim3(1), dim3(pic::PL_T), 0, static_cast<hipStream_t>(stream), meta_of(c),
                     seqs, counts, n);
  return launched();
}

pi_status pi_cache_append(const pi_cache* c, int32_t layer, const pi_heads* k, const pi_heads* v, int32_t tokens,
                          const int32_t* cu, const int32_t* seqs, int32_t n, void* stream) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if (layer < 0 || layer >= c->layers || tokens < 0 || n < 1 || !cu || !on(cu, 4) || !seqs || !on(seqs, 4))
    return PI_EINVAL;
  if ((s = check_heads(k, tokens)) != PI_OK || (s = check_heads(v, tokens)) != PI_OK) return s;
  if (tokens == 0) return PI_OK;
  const int64_t threads = (int64_t)tokens * c->kv_heads * (c->dim / 8);
  if (up_div(threads, 256) > INT32_MAX) return PI_EUNSUPPORTED;
  const int64_t at = (int64_t)layer * c->pages * c->kv_heads * c->page * c->dim;
  (void)hipGetLastError();
  hipLaunchKernelGGL(pic::k_cache_append, dim3((unsigned)up_div(threads, 256)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), meta_of(c), static_cast<uint16_t*>(c->k) + at,
                     static_cast<uint16_t*>(c->v) + at, c->kv_heads, c->dim, static_cast<const uint16_t*>(k->p),
                     k->token_stride, k->head_stride, static_cast<const uint16_t*>(v->p), v->token_stride,
                     v->head_stride, cu, seqs, n, tokens);
  return launched();
}

pi_status pi_cache_fork(const pi_cache* c, const int32_t* parents, const int32_t* children, int32_t n, void* ws,
                        size_t ws_bytes, void* stream) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if ((s = check_list(parents, n)) != PI_OK || (s = check_list(children, n)) != PI_OK) return s;
  if ((s = check_ws(c, ws, ws_bytes)) != PI_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const pic::Plan plan = plan_of(c, ws);
  (void)hipGetLastError();
  hipLaunchKernelGGL(pic::k_cache_fork, dim3(1), dim3(pic::PL_T), 0, st, meta_of(c), parents, children, n, plan);
  copy_pages(c, n, plan, nullptr, nullptr, st);
  return launched();
}

pi_status pi_cache_release(const pi_cache* c, const int32_t* seqs, int32_t n, void* stream) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if ((s = check_list(seqs, n)) != PI_OK) return s;
  (void)hipGetLastError();
  hipLaunchKernelGGL(pic::k_cache_release, dim3(1), dim3(pic::PL_T), 0, static_cast<hipStream_t>(stream), meta_of(c),
                     seqs, n);
  return launched();
}

pi_status pi_cache_compact(const pi_cache* c, int32_t* moved, void* ws, size_t ws_bytes, void* stream) {
  pi_status s;
  if ((s = check_cache(c)) != PI_OK) return s;
  if (!on(moved, 4)) return PI_EINVAL;
  if ((s = check_ws(c, ws, ws_bytes)) != PI_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const pic::Plan plan = plan_of(c, ws);
  int32_t* to = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + ws_of(c).to);
  const pic::Meta m = meta_of(c);
  (void)hipGetLastError();
  hipLaunchKernelGGL(pic::k_cache_compact, dim3(1), dim3(pic::PL_T), 0, st, m, plan, to);
  copy_pages(c, std::max(1, c->pages / 2), plan, to, moved, st);
  return launched();
}

}  // extern "C"
