// How attention over a cache is cut into shares, and how page numbers are
// followed: plain integer functions, which the tests also run on the host.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pish {

#define PI_BOTH __host__ __device__ __forceinline__

constexpr int UNIT = 128;                // keys of a unit of work of the rows' own keys
constexpr int MOST = 128;                // shares of a row's own keys at most
constexpr int TILE = 64;                 // keys of a tile of the common keys
constexpr int TILES = 4;                 // of those, a share has at least

// Tokens of a slot as they can be used: 0 where the length cannot be.
PI_BOTH int usable_len(int len, int max_pages, int page) {
  return len < 0 || len > (int64_t)max_pages * page ? 0 : len;
}

// Common tokens for a prefix of n pages; a prefix that no table row can hold is none.
PI_BOTH int common_tokens(int n, int max_pages, int page) { return n > 0 && n <= max_pages ? n * page : 0; }

// Page number `id` as it can be followed, or -1.
PI_BOTH int usable_page(int id, int pages) { return (unsigned)id < (unsigned)pages ? id : -1; }

// Table place of a key; keys behind a row's last place stay on it.
PI_BOTH int place_of(int key, int page, int max_pages) {
  const int p = key / page;
  return p < max_pages ? p : max_pages - 1;
}

// Pieces of `size` keys; near the largest length the sum would not fit an int.
PI_BOTH int pieces(int keys, int size) { return (int)(((uint32_t)keys + size - 1) / size); }

// Shares of the common keys: whole tiles, TILES of them at least, and `most` shares at most.  (4096 common keys, 32
// rows of 64 heads on 8, 128 wide: 37 us a call; with 2 tiles 49 us, with 8 42 us: more shares, more sums to write and
// join, or fewer blocks.)
PI_BOTH int common_shares(int total, int most) {
  const int n = pieces(total, TILE) / TILES;
  return n < 1 ? 1 : n < most ? n : most;
}

// Units of a row's own keys.
PI_BOTH int units_of(int keys) { return pieces(keys, UNIT); }

// `free` shares are dealt to the rows, of `share_size` units each (the last of a row may be smaller): all rows together
// take no more than `free` and one each.  32-bit division: what is lost of `all` by it is made up for.
PI_BOTH uint32_t share_size(uint64_t all, int free) {
  int s = 0;
  while (all >> s >> 31) ++s;
  const uint32_t n = ((uint32_t)(all >> s) + free - 1) / free << s;
  return (n > 1 ? n : 1) + (s ? 1u << s : 0u);
}
PI_BOTH int deal(int units, uint32_t size) {
  const uint32_t n = ((uint32_t)units + size - 1) / size;
  return n < 1 ? 1 : n < (uint32_t)MOST ? (int)n : MOST;
}

// The first of share i of n of `steps`; the share ends where the next begins.
PI_BOTH int share_begin(int steps, int i, int n) { return (int)((int64_t)steps * i / n); }

}  // namespace pish
