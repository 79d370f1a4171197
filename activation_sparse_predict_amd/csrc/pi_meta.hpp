// Where a cache's tables and counts lie in pi_cache.meta.
#pragma once
#include "pi.h"

#include <stdint.h>

namespace pic {

// The parts of pi_cache.meta.
struct Meta {
  int32_t *table, *lens, *ref, *free, *words;
  int slots, max_pages, pages, page;
};

inline Meta meta_of(const pi_cache* c) {
  int32_t* table = c->meta;
  int32_t* lens = table + (int64_t)c->slots * c->max_pages;
  int32_t* ref = lens + c->slots;
  return Meta{table, lens, ref, ref + c->pages, ref + 2 * (int64_t)c->pages, c->slots, c->max_pages, c->pages,
              c->page};
}

}  // namespace pic
