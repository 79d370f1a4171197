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

// The page of a place of 16 keys by a multiplication, `per` places a page (1 .. 256): ceil(2^(31 + shift) / per) is off by
// less than 1, and with 2^shift <= per < 2^(shift + 1) that changes no quotient of a place below 2^30.
struct Divide {
  uint32_t mul, shift;
};
PI_BOTH Divide divide_by(uint32_t per) {
  Divide d{0, 0};
  while (per >> (d.shift + 1)) ++d.shift;
  d.mul = (uint32_t)(((uint64_t(1) << (31 + d.shift)) + per - 1) / per);
  return d;
}
PI_BOTH int divided(uint32_t place, Divide d) { return (int)((uint32_t)((uint64_t)(2 * place) * d.mul >> 32) >> d.shift); }

// Which kernel takes a call with chunks of `tokens` tokens in all, `group` rows (heads of a key head) a token: that for few
// rows, 16 or 32 a block (1, 2), or that of 128 rows a block (0).  A chunk comes out the same on either; only its time hangs on
// this.  The host knows no chunk's own length, so the first takes calls with up to 32 rows a chunk on the average, whose longest
// chunk has 256 at most: all tokens but one for each other chunk, or all of them where some chunks must be empty.  It reads a
// longer one's keys for every 32 rows.  Few rows first, in us:
//   one token behind 1500, 32 heads 14.5 and 16.7, 16 heads on 8, 256 wide, 14.6 and 22.1; 8 tokens of 40 heads on 8, 80 wide,
//   behind up to 1500 13.1 and 17.5; 8 times 4 tokens of 16 heads on 8, 256 wide, behind up to 4000 47 and 58
//   31 single tokens behind up to 4000 and 512 behind 32768, 32 heads, 796 and 466; 63 and 512 1547 and 606; 31 and 64 of 32
//   heads on 8 205 and 112
// What the limit costs where chunks are alike: 32 times 8 tokens of 16 heads on 8, 256 wide, behind up to 4000 160 and 181.
PI_BOTH int few_tiles(int tokens, int n, int group) {
  const int chunks = n < 1 ? 1 : n < tokens ? n : tokens < 1 ? 1 : tokens;
  const int64_t mean = (int64_t)((tokens + chunks - 1) / chunks) * group;
  const int64_t most = (int64_t)(n > tokens ? tokens : tokens - chunks + 1) * group;
  return mean > 32 || most > 256 ? 0 : mean > 16 ? 2 : 1;
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
