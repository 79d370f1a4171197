// Device code of attention of chunks of new tokens over a paged cache, for gfx950.
//
// The mathematics and the steps of a tile are those of pi_attn.hpp; here the queries
// of a key head are the rows (token, head of its group) of a sequence's chunk, packed
// 128 to a block, whatever the group, and keys are found through the slot's pages.
// Scores may be changed on the way, in units of log2(e):
//   cap:     cap tanh(x / cap) = cap (1 - 2 / (1 + e^(2 x / cap)))
//   slopes:  + slope (j - p)
#pragma once
#include "pi_attn.hpp"

namespace pia {

constexpr int CH_ROWS = 128;             // rows of a block of k_attn_chunk
constexpr int CH_MOST = 64;              // shares of a tile's keys at most
template <int D> constexpr int ch_waves() { return D > 128 ? 8 : 4; }   // of a block of k_attn_chunk

enum { CH_CAP = 1, CH_SLOPES = 2 };

struct ChunkScore {
  float c;                               // scale log2(e)
  float pre, cap;                        // 2 scale log2(e) / cap, cap log2(e)
  const float* slopes;                   // [heads] or NULL
  int window;                            // 0: none
};

// The batch of a call and how it is cut up.
struct Chunks {
  const int32_t *cu, *seqs;
  int n, tokens, heads, kv_heads, dim;
  int tile;                              // rows of a block
  int free;                              // shares to deal beside one a tile
  int slots, rows;                       // places for sums in the workspace, rows of each
  Divide page;                           // a place's page from its number
};

// A tile of rows whose keys are shared out, for k_chunk_join.
struct Joint {
  int slot, shares;                      // the first share's sums for key head 0; shares 1: nothing to join
  int first, row0, rows;                 // the chunk's first token, the tile's first row, its rows
  int step;                              // slots from one share to the next
};

// A sequence of the batch.
struct Seq {
  int first, count, slot, len, raw;      // its tokens in q, what its slot holds, as it is written there
  int tiles, keys;                       // tiles of rows, key tiles that any of them sees at most
};
__device__ __forceinline__ Seq seq_of(const Pages& pg, const Chunks& ch, int window, int i) {
  Seq s{0, 0, -1, 0, 0, 0, 0};
  if (i >= ch.n) return s;
  s.first = min(max(ch.cu[i], 0), ch.tokens);
  s.count = min(max(ch.cu[i + 1], s.first), ch.tokens) - s.first;
  s.slot = slot_of(ch.seqs, i, pg.slots);
  s.raw = s.slot >= 0 ? pg.lens[s.slot] : 0;
  s.len = usable_len(s.raw, pg.max_pages, pg.page);
  const int group = ch.heads / ch.kv_heads;
  s.tiles = (int)(((int64_t)s.count * group + ch.tile - 1) / ch.tile);
  s.keys = pieces(s.len, PT_K);
  // a tile's rows lie at 127 / group + 2 places at most
  if (window > 0) s.keys = (int)min((uint32_t)s.keys, ((uint32_t)min(window, s.len) + 127 / group + 1) / PT_K + 2);
  return s;
}

// What a block does.
struct Piece {
  Seq s;                                 // count 0: nothing
  int tile, share, shares;               // shares of the longest tile
  uint32_t size;                         // key tiles of a share
  int slot, joint;                       // of the tile, where shares > 1
  int joints;                            // tiles with several shares, where it was asked for
};

__device__ __forceinline__ float add64(float v) {        // over the wave, the same sum in every lane
#pragma unroll
  for (int x = 32; x; x >>= 1) v += __shfl_xor(v, x);
  return v;
}

__device__ __forceinline__ int shares_of(const Seq& s, uint32_t size) {
  return max(1, min(CH_MOST, (int)(((uint32_t)s.keys + size - 1) / size)));
}

// Every tile of rows has one share, and up to `free` more are dealt.  Where there are fewer tiles than that, a share is made
// as small as it can be with no more than `free` of them in all, so that all blocks run at once: a few steps towards that
// size, for up to 64 sequences.  Where there are more, those sequences come first whose blocks have most to do.  (24 chunks
// of 1201 tokens behind up to 2050, 1280 blocks of uneven length on 1024 places: 86 us in the batch's order, 83 so.)  Sums are
// float32: what they may be off by is made up for in the size of a share, so that the blocks there are suffice.  `count`:
// count the tiles that are shared out too.
__device__ __forceinline__ Piece find_piece(const Pages& pg, const Chunks& ch, int window, int idx, bool count) {
  const int lane = threadIdx.x & (WAVE - 1);
  Seq s = seq_of(pg, ch, window, lane);
  float work = (float)s.tiles * (float)s.keys, tiles = (float)s.tiles;
  for (int base = WAVE; base < ch.n; base += WAVE) {
    const Seq x = seq_of(pg, ch, window, base + lane);
    work += (float)x.tiles * (float)x.keys;
    tiles += (float)x.tiles;
  }
  const float all = add64(work), free = (float)ch.free;
  float want = all / free * 1.0001f;
  const bool roomy = add64(tiles) < free;
  if (ch.n <= WAVE && roomy) {
    for (int i = 0; i < 4; ++i) {
      const float got = add64((float)s.tiles * (float)shares_of(s, (uint32_t)min(want, 2e9f) + 1));
      if (got <= free) break;
      want = max(want * (got / free), want + 1.f);
    }
  }
  const uint32_t size = __builtin_amdgcn_readfirstlane((uint32_t)min(want, 2e9f) + 1);
  if (ch.n > 1 && ch.n <= WAVE && !roomy) {
    const int load = s.tiles ? min(s.keys, (int)min(size, (uint32_t)INT32_MAX)) : -1;
    int rank = 0;
    for (int j = 0; j < ch.n; ++j) {
      const int other = __builtin_amdgcn_readlane(load, j);
      rank += other > load || (other == load && j < lane);
    }
    if (lane >= ch.n) rank = lane;
    auto to = [&](int v) { return __builtin_amdgcn_ds_permute(4 * rank, v); };
    s = Seq{to(s.first), to(s.count), to(s.slot), to(s.len), to(s.raw), to(s.tiles), to(s.keys)};
  }
  Piece p{};
  p.size = size;
  int slot = 0, joint = 0;
  bool found = false;
  for (int base = 0; base < ch.n; base += WAVE) {
    if (base) s = seq_of(pg, ch, window, base + lane);
    const int n = shares_of(s, size);
    const int blocks = s.tiles * n, upto = scan64(blocks);
    const int js = n > 1 ? s.tiles : 0, jupto = scan64(js), supto = scan64(n > 1 ? blocks : 0);
    const uint64_t hit = __ballot(upto > idx);
    if (hit && !found) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      p.s = Seq{of(s.first), of(s.count), of(s.slot), of(s.len), of(s.raw), of(s.tiles), of(s.keys)};
      p.shares = of(n);
      const int in = idx - (of(upto) - of(blocks));
      p.share = in / p.s.tiles;
      const int nth = in % p.s.tiles;              // the last tile, which sees most, first
      p.tile = p.s.tiles - 1 - nth;
      p.slot = slot + of(supto) - of(n > 1 ? blocks : 0) + nth;
      p.joint = joint + of(jupto) - of(js) + nth;
      if (in < 0 || in >= of(blocks) || p.slot < 0) p.s.count = 0;   // offsets that do not ascend: the sums may not fit
      found = true;
      if (!count) return p;
    }
    idx -= __builtin_amdgcn_readlane(upto, WAVE - 1);
    joint += __builtin_amdgcn_readlane(jupto, WAVE - 1);
    slot += __builtin_amdgcn_readlane(supto, WAVE - 1);
    if (found) idx = INT32_MAX;
  }
  p.joints = joint;
  return p;
}

// A value that is the same in all lanes, where the compiler cannot see that.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t a = __builtin_amdgcn_readfirstlane((uint32_t)v), b = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (int64_t)((uint64_t)b << 32 | a);
}

// A tile's scores as the softmax takes them, in units of log2(e).  `back` is the tile's first key minus the row's place.
template <int MOD, int H>
__device__ __forceinline__ void change(f16v* s, const ChunkScore& sc, float slope, int back) {
  const float at = slope * (float)(back + 4 * (int)((threadIdx.x & 63) >> 5));
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x;
      if constexpr (MOD & CH_CAP) {
        const float e = exp2_fast(s[h][i] * sc.pre);
        x = fmaf(-2.f * sc.cap, __builtin_amdgcn_rcpf(e + 1.f), sc.cap);
      } else {
        x = s[h][i] * sc.c;
      }
      if constexpr (MOD & CH_SLOPES) x += fmaf(slope, (float)(32 * h + 8 * (i / 4) + i % 4), at);
      s[h][i] = x;
    }
}

// The same for the scores of a step of 32 keys of k_chunk_few.
template <int MOD>
__device__ __forceinline__ void change16(f4* s, const ChunkScore& sc, float slope, int back) {
  const float at = slope * (float)(back + 4 * (int)((threadIdx.x & 63) >> 4));
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x;
      if constexpr (MOD & CH_CAP) {
        const float e = exp2_fast(s[h][i] * sc.pre);
        x = fmaf(-2.f * sc.cap, __builtin_amdgcn_rcpf(e + 1.f), sc.cap);
      } else {
        x = s[h][i] * sc.c;
      }
      if constexpr (MOD & CH_SLOPES) x += fmaf(slope, (float)(16 * h + i), at);
      s[h][i] = x;
    }
}

// Scores of keys that a row does not see: it sees those from `lo` on and before `hi` in the places of 16 that `bits` names.
template <int H>
__device__ __forceinline__ void hide(f16v* s, int lo, int hi, uint32_t bits) {
  const int half = 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = 32 * h + 8 * (i / 4) + i % 4;
      if (key >= hi - half || key < lo - half || !(bits >> (2 * h + i / 8) & 1)) s[h][i] = NEG_INF;
    }
}

// Whether a tile in LDS holds a value that is not finite, by all threads of a block.
template <class T, int D> __device__ __forceinline__ bool wild(const char* tile) {
  typedef unsigned short h2 __attribute__((ext_vector_type(2)));
  constexpr int N = PT_K * Tile<D>::NC / (ch_waves<D>() * WAVE);
  h2 top = {0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const u4 x = *reinterpret_cast<const u4*>(tile + 16 * (ch_waves<D>() * WAVE * i + threadIdx.x));
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(h2, x[e] & 0x7fff7fffu));
  }
  return __syncthreads_or(top[0] >= T::INF || top[1] >= T::INF) != 0;
}

// 0 times an infinity or NaN is NaN, for a value that a row does not see as for one whose key has no weight.  So where a tile
// that not all of a block's rows see whole holds such values, they count as zeros there (`tame`); and where there were any, or
// a sum came out not finite, the elements that see such values get at the end what these make of them, whatever the keys'
// weights are (`add_wild`): that hangs on no tile, share or order.  Infinities of one sign give that infinity, else NaN.
enum { WILD_UP = 1, WILD_DOWN = 2, WILD_NAN = 4 };
template <class T> __device__ __forceinline__ int kind_of(uint32_t x) {          // of a value's 16 bits
  return (x & 0x7fffu) < T::INF ? 0 : (x & 0x7fffu) > T::INF ? WILD_NAN : x & 0x8000u ? WILD_DOWN : WILD_UP;
}
__device__ __forceinline__ float value_of(int kinds) {
  return kinds == WILD_UP ? -NEG_INF : kinds == WILD_DOWN ? NEG_INF : __builtin_nanf("");
}
template <class T> __device__ __forceinline__ uint32_t finite(uint32_t x) {      // a mask of the halves that are
  return ((x & 0x7fffu) >= T::INF ? 0u : 0xffffu) | ((x >> 16 & 0x7fffu) >= T::INF ? 0u : 0xffff0000u);
}
template <class T, int D> __device__ __forceinline__ void tame(char* sv) {
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < PT_K * Tile<D>::NC; i += blockDim.x) {
    u4 x = *reinterpret_cast<const u4*>(sv + 16 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] &= finite<T>(x[e]);
    *reinterpret_cast<u4*>(sv + 16 * i) = x;
  }
  __syncthreads();
}

// What a block has to do, beside the tensors.
struct Task {
  int g, first, last;                    // key head; key tiles of the share
  int from, to;                          // keys that any row sees
  int window;                            // 0 where it is no smaller than what the slot holds, so that differences with it fit
  int before, t0, t1;                    // place of the chunk's first token; first and last token of the rows
  int row0, rows, token;                 // first row, rows (0: nothing to do); the chunk's first token in q
  int64_t table;                         // the slot's row of the table
  int slot, shares;                      // place for the sums; shares of the tile's keys (1: the result is written)
};

// That of this block, with what the join and the error word have to know.  Key heads of a piece run side by side, those of
// one head on one die where they can (block b runs on die b % 8).
__device__ __forceinline__ Task find_task(const Pages& pg, const Chunks& ch, int window, Joint* joints, int32_t* count) {
  const int idx = blockIdx.x / ch.kv_heads;
  const Piece pc = find_piece(pg, ch, window, idx, blockIdx.x == 0);
  if (blockIdx.x == 0 && threadIdx.x == 0) *count = pc.joints;
  Task k{};
  if (pc.s.count == 0) return k;
  const int group = ch.heads / ch.kv_heads;
  k.g = blockIdx.x % ch.kv_heads;
  k.before = pc.s.len - pc.s.count;
  k.row0 = ch.tile * pc.tile;
  const int rows = min(ch.tile, pc.s.count * group - k.row0);
  k.t0 = k.row0 / group, k.t1 = (k.row0 + rows - 1) / group;
  k.window = window < pc.s.len ? window : 0;
  k.to = max(0, k.before + k.t1 + 1), k.from = k.window > 0 ? max(0, k.before + k.t0 + 1 - k.window) : 0;
  const int tiles = k.to > k.from ? (k.to - 1) / PT_K - k.from / PT_K + 1 : 0;
  // shares of this tile: no more than its keys need
  k.shares = max(1, min(pc.shares, (int)(((uint32_t)tiles + pc.size - 1) / pc.size)));
  if (k.g == 0 && pc.share == 0 && threadIdx.x == 0) {
    if (pc.s.slot < 0 || pc.s.len != pc.s.raw || k.before < 0)
      atomicOr(pg.flags, pc.s.slot < 0 ? PI_CACHE_ESLOT : PI_CACHE_ELENGTH);
    if (pc.shares > 1 && (unsigned)pc.joint < (unsigned)ch.slots / 2)
      joints[pc.joint] = Joint{pc.slot, k.shares, pc.s.first, k.row0, rows, pc.s.tiles};
  }
  k.slot = pc.slot + pc.share * pc.s.tiles;
  if (pc.share >= k.shares || (k.shares > 1 && k.slot >= ch.slots)) return k;
  k.first = k.from / PT_K + share_begin(tiles, pc.share, k.shares);
  k.last = k.from / PT_K + share_begin(tiles, pc.share + 1, k.shares) - 1;
  k.token = pc.s.first;
  k.table = (int64_t)max(pc.s.slot, 0) * pg.max_pages;
  k.rows = rows;
  return k;
}

__device__ __forceinline__ int page_of(const Chunks& ch, uint32_t place) { return divided(place, ch.page); }

// Whether some of the rows do not see all keys of a tile.
__device__ __forceinline__ bool at_edge(const Task& k, int tile) {
  return PT_K * tile + PT_K - 1 > k.before + k.t0 || (k.window > 0 && PT_K * tile <= k.before + k.t1 - k.window);
}

// Elements that see values which are not finite, for all threads of a block after the sums were written.  A row's total
// weight is in `total`: where it is NaN, a score was, and so is the row.  `kinds`: room for `dim` numbers.
template <class T>
__device__ __forceinline__ void add_wild(const Pages& pg, const Chunks& ch, const Task& k, uint16_t* out,
                                         int64_t out_token, int64_t out_head, float* part, const float* total, int* kinds) {
  const int group = ch.heads / ch.kv_heads, dim = ch.dim, nchunk = dim / 8;
  const int64_t sums = ((int64_t)k.slot * ch.kv_heads + k.g) * ch.rows;
  auto value_at = [&](int key) -> const uint16_t* {        // NULL in a broken page
    const int id = usable_page(pg.table[k.table + page_of(ch, key / 16)], pg.pages);
    return id < 0 ? nullptr : pg.v + (((int64_t)id * ch.kv_heads + k.g) * pg.page + key % pg.page) * dim;
  };
  for (int d = threadIdx.x; d < dim; d += blockDim.x) kinds[d] = 0;
  __syncthreads();
  // of tiles that all rows see
  const int at_once = blockDim.x / nchunk, c = threadIdx.x % nchunk, mine = threadIdx.x / nchunk;
  if (mine < at_once) {
#pragma unroll 1
    for (int j = k.first; j <= k.last; ++j) {
      if (at_edge(k, j)) continue;
#pragma unroll 1
      for (int key = PT_K * j + mine; key < PT_K * j + PT_K; key += at_once) {
        const uint16_t* v = value_at(key);
        if (!v) continue;
        const u4 x = *reinterpret_cast<const u4*>(v + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int kind = kind_of<T>(x[e / 2] >> 16 * (e % 2));
          if (kind) atomicOr(&kinds[8 * c + e], kind);
        }
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int e = threadIdx.x; e < k.rows * dim; e += blockDim.x) {
    const int x = e / dim, row = k.row0 + x, d = e % dim, place = k.before + row / group;
    const int lo = k.window > 0 ? max(k.from, place + 1 - k.window) : k.from;
    int all = kinds[d];
#pragma unroll 1
    for (int j = k.first; j <= k.last; ++j) {
      if (!at_edge(k, j)) continue;
#pragma unroll 1
      for (int key = max(PT_K * j, lo); key < min(PT_K * j + PT_K, place + 1); ++key) {
        const uint16_t* v = value_at(key);
        if (v) all |= kind_of<T>(v[d]);
      }
    }
    if (all == 0) continue;
    const float value = total[x] == total[x] ? value_of(all) : total[x];
    if (k.shares > 1) part[(sums + x) * dim + d] = value;
    else out[(k.token + row / group) * out_token + (k.g * group + row % group) * out_head + d] = (uint16_t)T::pack(value, 0.f);
  }
}

// ---- chunks of few rows: 16 MT of them for a block, with the products and the layout of k_attn_decode.  The four waves take
// steps of 32 keys in turn, whose keys and values go straight to registers: what a compute unit has on its way from memory
// bounds these, and its registers hold more than its LDS (192 KB with three blocks of MT 1, 64 KB in two blocks' tiles).
// 8 sequences of one token behind up to 2900, 32 heads of 128: 40 us, 5.5 TB/s of keys and values; one token behind 1500:
// 10.4 us, latency: slots and lengths, page numbers, pages, the join of the waves.
template <class T, int D, int MOD, int MT>
__global__ void __launch_bounds__(4 * WAVE, D > 128 ? 1 : D <= 64 || MT == 1 ? 3 : 2)
k_chunk_few(Pages pg, Rows q, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head, Chunks ch, ChunkScore sc,
            Joint* __restrict__ joints, int32_t* __restrict__ count, float* __restrict__ part, float* __restrict__ stat) {
  using V = Vec<D>;
  constexpr int NF = V::W * V::G, ROW = 16 * NF + 4;
  __shared__ __attribute__((aligned(16))) float so[4 * 16 * ROW], sm[4 * 16 * 2], total[16 * MT];
  __shared__ int odds[4];
  const Task k = find_task(pg, ch, sc.window, joints, count);
  if (k.rows == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kg = lane >> 4, group = ch.heads / ch.kv_heads, nchunk = ch.dim / 8, dim = ch.dim;

  int place[MT];
  float slope[MT];
  u4 qf[MT][V::KS];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = k.row0 + min(16 * m + r, k.rows - 1), t = row / group, head = k.g * group + row % group;
    place[m] = k.before + t;
    slope[m] = (MOD & CH_SLOPES) && sc.slopes ? sc.slopes[head] * 1.44269504f : 0.f;
    const uint16_t* src = q.at(k.token + t, head);
#pragma unroll
    for (int s = 0; s < V::KS; ++s) {
      const int c = 4 * s + kg;
      qf[m][s] = c < nchunk ? *reinterpret_cast<const u4*>(src + 8 * c) : u4{0, 0, 0, 0};
    }
  }
  f4 o[MT][NF];
  float mc[MT], l[MT];                             // mc: HIGH under c times the largest score so far
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mc[m] = NEG_INF, l[m] = 0.f;
#pragma unroll
    for (int f = 0; f < NF; ++f) o[m][f] = (f4)(0.f);
  }
  const int32_t* table = pg.table + k.table;
  const int64_t head_at = (int64_t)pg.page * dim, page_at = head_at * ch.kv_heads;
  bool odd = false;                                // whether there were values that are not finite

  for (int st = 2 * k.first + w; st < 2 * (k.last + 1); st += 4) {
    const int k0 = 32 * st;
    const uint16_t *kp[2], *vp[2];
    int from[2], to[2];                            // of the half's keys, those that some row sees
    bool gone = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = k0 + 16 * h, x = key / 16;
      from[h] = max(0, k.from - key), to[h] = min(16, k.to - key);
      int id = 0;
      if (to[h] > from[h]) {
        const int number = fixed(table, page_of(ch, x));
        id = usable_page(number, pg.pages);
        if (id < 0) {                              // a broken table: its keys are not seen
          if (lane == 0) atomicOr(pg.flags, PI_CACHE_EPAGE);
          to[h] = 0, id = 0, gone = true;
        }
      }
      const int64_t at = id * page_at + k.g * head_at + (int64_t)((x - page_of(ch, x) * (pg.page / 16)) * 16 * dim);
      kp[h] = pg.k + at;
      vp[h] = pg.v + at;
    }
    // all of the step's loads are on their way before the first product; keys that do not exist lie in a page all the same
    u4 kf[2][V::KS];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ks = 0; ks < V::KS; ++ks) {
        const int c = 4 * ks + kg;
        kf[h][ks] = *reinterpret_cast<const u4*>(kp[h] + r * dim + 8 * min(c, nchunk - 1));
        if (c >= nchunk) kf[h][ks] = u4{0, 0, 0, 0};
      }
    uint32_t x[V::G][8][V::W / 2];                 // V: keys 4 kg + 0..3 of both halves
#pragma unroll
    for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d0 = (16 * gr + r) * V::W;
        const uint16_t* src = vp[i / 4] + (4 * kg + i % 4) * dim + (d0 < dim ? d0 : 0);
        if constexpr (V::W == 8) {
          const u4 y = *reinterpret_cast<const u4*>(src);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[gr][i][e] = y[e];
        } else {
          const u2 y = *reinterpret_cast<const u2*>(src);
#pragma unroll
          for (int e = 0; e < 2; ++e) x[gr][i][e] = y[e];
        }
      }
    // whether some row does not see one of the keys
    const bool some = gone || k0 + 31 > k.before + k.t0 || k0 < k.from || (k.window > 0 && k0 <= k.before + k.t1 - k.window);
    u4 pf[MT];
    float alpha[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      f4 s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[h] = (f4)(0.f);
#pragma unroll
        for (int ks = 0; ks < V::KS; ++ks) s[h] = T::mma16(kf[h][ks], qf[m][ks], s[h]);
      }
      if constexpr (MOD != 0) change16<MOD>(s, sc, slope[m], k0 - place[m]);
      if (some) {
        const int hi = place[m] + 1 - k0, lo = k.window > 0 ? hi - k.window : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 4 * kg + i;            // in its half
            if (16 * h + key >= hi || 16 * h + key < lo || key >= to[h]) s[h][i] = NEG_INF;
          }
      }
      const float c = MOD ? 1.f : sc.c;
      float mt = NEG_INF;
#pragma unroll
      for (int i = 0; i < 4; ++i) mt = fmaxf(mt, fmaxf(s[0][i], s[1][i]));
      const float top = fmaxf(mc[m], max16(mt) * c - T::HIGH);
      const float base = top == NEG_INF ? 0.f : top;   // rows whose scores so far are all -inf
      alpha[m] = exp2_fast(mc[m] - base);
      mc[m] = top;
      float p[8], ls = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_fast(fmaf(s[i / 4][i % 4], c, -base));
        ls += p[i];
      }
      l[m] = fmaf(l[m], alpha[m], ls);
      pf[m] = u4{T::pack(p[0], p[1]), T::pack(p[2], p[3]), T::pack(p[4], p[5]), T::pack(p[6], p[7])};
    }
    if (some) {
      // what no row sees counts as zeros, whatever is stored there
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (4 * kg + i % 4 >= to[i / 4] || 4 * kg + i % 4 < from[i / 4])
#pragma unroll
          for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
            for (int e = 0; e < V::W / 2; ++e) x[gr][i][e] = 0;
    }
    if (k.t0 != k.t1 && at_edge(k, st / 2)) {
#pragma unroll
      for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < V::W / 2; ++e) {
            const uint32_t keep = finite<T>(x[gr][i][e]);
            odd |= keep != ~0u;
            x[gr][i][e] &= keep;
          }
    }
#pragma unroll
    for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
      for (int e = 0; e < V::W / 2; ++e) {
        auto& y = x[gr];
        const u4 a = {lows(y[0][e], y[1][e]), lows(y[2][e], y[3][e]), lows(y[4][e], y[5][e]), lows(y[6][e], y[7][e])};
        const u4 z = {highs(y[0][e], y[1][e]), highs(y[2][e], y[3][e]), highs(y[4][e], y[5][e]),
                      highs(y[6][e], y[7][e])};
        const int f = gr * V::W + 2 * e;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[m][f][i] *= alpha[m];
            o[m][f + 1][i] *= alpha[m];
          }
          o[m][f] = T::mma16(a, pf[m], o[m][f]);
          o[m][f + 1] = T::mma16(z, pf[m], o[m][f + 1]);
        }
      }
  }

  // join the waves, 16 rows at a time: o[m][f][i] belongs to dim (16 gr + 4 kg + i) W + f % W of row 16 m + r
  // of wave w's in so [4][16][ROW], (reference point, l) in sm [4][16][2]
  const int64_t sums = ((int64_t)k.slot * ch.kv_heads + k.g) * ch.rows;
  float bad = 0.f;                                 // NaN where a sum is not finite
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) bad = fmaf(o[m][f][i], 0.f, bad);
  const bool any = __ballot(odd || bad != bad) != 0;
  if (lane == 0) odds[w] = any;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (16 * m >= k.rows) break;
    if (m > 0) __syncthreads();
    const float ll = sum16(l[m]);
    if (lane < 16) *reinterpret_cast<float2*>(sm + (16 * w + r) * 2) = float2{mc[m], ll};
#pragma unroll
    for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int f = 0; f < V::W; ++f) so[(16 * w + r) * ROW + (16 * gr + 4 * kg + i) * V::W + f] = o[m][gr * V::W + f][i];
    __syncthreads();
    const int left = min(16, k.rows - 16 * m);
    for (int e = 2 * tid; e < left * dim; e += 2 * 4 * WAVE) {
      const int x = e / dim, d = e % dim;
      float mm = NEG_INF;
#pragma unroll
      for (int i = 0; i < 4; ++i) mm = fmaxf(mm, sm[(16 * i + x) * 2]);
      const float base = mm == NEG_INF ? 0.f : mm;
      float tl = 0.f, oo = 0.f, od = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = exp2_fast(sm[(16 * i + x) * 2] - base);
        tl = fmaf(sm[(16 * i + x) * 2 + 1], a, tl);
        oo = fmaf(so[(16 * i + x) * ROW + d], a, oo);
        od = fmaf(so[(16 * i + x) * ROW + d + 1], a, od);
      }
      if (d == 0) total[16 * m + x] = tl;
      if (k.shares == 1) {
        const float inv = tl == 0.f ? 0.f : 1.f / tl;   // a row that sees no key is zero
        const int row = k.row0 + 16 * m + x;
        *reinterpret_cast<uint32_t*>(out + (k.token + row / group) * out_token + (k.g * group + row % group) * out_head + d) =
            T::pack(oo * inv, od * inv);
      } else {
        *reinterpret_cast<float2*>(part + (sums + 16 * m + x) * dim + d) = float2{oo, od};
        if (d == 0) *reinterpret_cast<float2*>(stat + 2 * (sums + 16 * m + x)) = float2{mm, tl};
      }
    }
  }
  if (!(odds[0] | odds[1] | odds[2] | odds[3])) return;
  __syncthreads();
  add_wild<T>(pg, ch, k, out, out_token, out_head, part, total, reinterpret_cast<int*>(so));
}

// One block: 128 rows of a key head, 32 for each wave, over one share of the keys that any of them sees, in tiles of 64 from
// the last one down, which go to LDS past the registers one tile ahead of the products.  Four waves; for heads wider than 128,
// whose sums and tiles leave room for no second block, eight, of which two take half of a tile's keys each for the same rows.
//
// 512 tokens of 32 heads on 8, 128 wide, behind 32768: 280 us, 990 TFLOP/s, the matrix cores busy for about half of the
// cycles, as in k_attn_prompt (see there).  The inner loop is that of whole tiles that all rows see, 350 instructions a wave and tile;
// with page numbers, edges and masks looked at in each tile it was 820 (430 us).  24 chunks, 128 heads on 8, 64 wide: 78 us,
// vector instructions (the exponentials) and the uneven lengths of blocks: waves wait for 37 % of their time.  Heads 256 wide:
// 730 TFLOP/s (4096 tokens, 16 heads), products, LDS reads and exponentials of eight waves that keep step follow one another
// more than they overlap; four waves with 32 more registers of scores took 166 us where eight take 131.  These spill 22 to 25
// registers a lane, the offsets `off` among them, and a reload waits for all loads before it: tiles at the edge wait so, and
// heads of 136 to 248 in every tile (512 tokens behind 8192, 16 heads on 8: 152 us 192 wide, 98 us 256 wide).  Wave priorities for
// half of them change nothing; a first round without looking for values that are not finite, and a second one where any came
// out, costs registers (capped 118 -> 128 us).
template <class T, int D, int MOD>
__global__ void __launch_bounds__(ch_waves<D>() * WAVE, D <= 64 ? 4 : D <= 128 ? 2 : 1)
k_attn_chunk(Pages pg, Rows q, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head, Chunks ch, ChunkScore sc,
             Joint* __restrict__ joints, int32_t* __restrict__ count, float* __restrict__ part, float* __restrict__ stat) {
  using L = Tile<D>;
  constexpr int NT = ch_waves<D>() * WAVE, S = 2, KW = ch_waves<D>() / 4, H = 2 / KW;
  using R = Ring<D, S, NT>;
  constexpr int SUMS = D <= 64 ? 4 * 32 * 68 * 4 : 0;   // sums on their way out, which take more than small tiles do
  __shared__ float2 stats[KW > 1 ? NT / 2 : 1];
  __shared__ int odds[4];
  // K tiles, then V tiles
  __shared__ __attribute__((aligned(1024))) char ring[2 * S * R::BYTES > SUMS ? 2 * S * R::BYTES : SUMS];

  const Task task = find_task(pg, ch, sc.window, joints, count);
  if (task.rows == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), hi = lane >> 5;
  const int group = ch.heads / ch.kv_heads, nchunk = ch.dim / 8;
  const int first = task.first, last = task.last, from = task.from, to = task.to;
  const int before = task.before, t0 = task.t0, t1 = task.t1;

  const int half = w / 4, row0 = task.row0 + 32 * (w % 4), row = row0 + (lane & 31), end = task.row0 + task.rows;
  const bool live = row0 < end;
  const int mine = min(row, end - 1), t = mine / group, head = task.g * group + mine % group;
  const int place = before + t;                    // the row sees keys up to here
  const int least = before + row0 / group, most = before + (min(row0 + 32, end) - 1) / group;   // of the wave's rows
  if (nchunk < L::NC) {
    for (int e = tid; e < 2 * S * R::BYTES / 16; e += NT) reinterpret_cast<u4*>(ring)[e] = u4{0, 0, 0, 0};
    __syncthreads();
  }
  u4 qf[L::KS];
  {
    const uint16_t* src = q.at(task.token + t, head);
#pragma unroll
    for (int s = 0; s < L::KS; ++s) {
      const int at = 2 * s + hi;
      qf[s] = at < nchunk ? *reinterpret_cast<const u4*>(src + 8 * at) : u4{0, 0, 0, 0};
    }
  }
  const float slope = (MOD & CH_SLOPES) && sc.slopes ? sc.slopes[head] * 1.44269504f : 0.f;

  const int32_t* table = pg.table + task.table;
  const uint32_t head_bytes = 2 * pg.page * ch.dim, page_bytes = head_bytes * ch.kv_heads;     // at most 2^31
  const char *kg = reinterpret_cast<const char*>(pg.k) + (int64_t)task.g * head_bytes;
  const char *vg = reinterpret_cast<const char*>(pg.v) + (int64_t)task.g * head_bytes;
  // byte of a place of 16 keys, from its page's number
  auto place_at = [&](int x, int id) {
    const uint32_t in = (uint32_t)(x - page_of(ch, x) * (pg.page / 16)) * (uint32_t)(32 * ch.dim);
    return uniform((int64_t)((uint64_t)(uint32_t)id * page_bytes + in));
  };
  // A wave loads one place of a tile, LW times 1024 bytes (of eight waves four the keys and four the values).  What a lane takes
  // of it is the chunk that its place in LDS asks for.
  constexpr int LW = L::NC / 4, RL = 64 / L::NC;
  const bool keys = KW == 1 || half == 0, values = KW == 1 || half == 1;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)ring + 1024 * LW * (w % 4);
  uint32_t off[LW];
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int r = i * RL + lane / L::NC, c = (lane % L::NC) ^ L::swz(r);
    off[i] = c < nchunk ? 2 * (uint32_t)(r * ch.dim + 8 * c) : ~0u;
  }
  auto look_up = [&](int j) { return fixed(table, page_of(ch, 4 * j + w % 4)); };
  // a tile that is whole: every place is there, and some row sees every key
  auto fetch = [&](int j, int id) {
    const int64_t at = place_at(4 * j + w % 4, id);
    const char *ka = kg + at, *va = vg + at;
    const uint32_t dst = lds0 + j % S * R::BYTES;
    if (nchunk == L::NC) {
      if (keys)
#pragma unroll
        for (int i = 0; i < LW; ++i) to_lds(ka, off[i], dst + 1024 * i);
      if (values)
#pragma unroll
        for (int i = 0; i < LW; ++i) to_lds(va, off[i], dst + S * R::BYTES + 1024 * i);
    } else {
#pragma unroll
      for (int i = 0; i < LW; ++i)
        if (off[i] != ~0u) {
          if (keys) to_lds(ka, off[i], dst + 1024 * i);
          if (values) to_lds(va, off[i], dst + S * R::BYTES + 1024 * i);
        }
    }
  };
  // Any tile; keys that no row sees are zeros: with anything else there, 0 times an infinity would be NaN.  Which places
  // there are.
  auto fetch_part = [&](int j) {
    const int x = 4 * j + w % 4;
    const bool inside = 16 * x < to && 16 * x + 16 > from;
    const int id = inside ? usable_page(fixed(table, page_of(ch, x)), pg.pages) : -1;
    const int64_t at = place_at(x, max(id, 0));
    const uint32_t dst = lds0 + j % S * R::BYTES;
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int key = 16 * x + i * RL + lane / L::NC;
      if (id >= 0 && key < to && key >= from) {
        if (off[i] != ~0u) {
          if (keys) to_lds(kg + at, off[i], dst + 1024 * i);
          if (values) to_lds(vg + at, off[i], dst + S * R::BYTES + 1024 * i);
        }
      } else {
        char* own = ring + j % S * R::BYTES + 1024 * (LW * (w % 4) + i) + 16 * lane;
        if (keys) *reinterpret_cast<u4*>(own) = u4{0, 0, 0, 0};
        if (values) *reinterpret_cast<u4*>(own + S * R::BYTES) = u4{0, 0, 0, 0};
      }
    }
    uint32_t bits = 0;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int y = 4 * j + i;
      if (16 * y >= to || 16 * y + 16 <= from) continue;
      if (usable_page(fixed(table, page_of(ch, y)), pg.pages) >= 0) bits |= 1u << i;
      else if (tid == 0) atomicOr(pg.flags, PI_CACHE_EPAGE);
    }
    return bits;
  };
  const Reads<D> rd(lane);
  Sums<T, D, H> sum;
  sum.clear();
  f16v s[H];
  uint32_t pw[8 * H];
  bool odd = false;                                // whether there were values that are not finite
  uint32_t bits = 0;
  if (first <= last) bits = fetch_part(last);
  // tiles below the last one that lie whole in what some row sees, and of these such as every row of the block sees whole;
  // none where a page is broken
  int whole = max(first, (from + PT_K - 1) / PT_K), upper = min(last - 1, (before + t0 + 1) / PT_K - 1), lower = whole;
  if (task.window > 0) lower = max(lower, (before + t1 - task.window) / PT_K + 1);
  if (whole < last) {
    bool broken = false;
    for (int e = page_of(ch, 4 * whole) + tid, end = page_of(ch, 4 * last); e <= end; e += NT)
      broken |= usable_page(table[e], pg.pages) < 0;
    if (__syncthreads_or(broken)) whole = last, upper = lower - 1;
  }
  const int mine_at = KW > 1 ? 32 * 16 * L::NC * half : 0;        // the wave's part of a tile in LDS
  // one tile of any kind, which lies in LDS; `there`: its places
  auto take = [&](int j, uint32_t there) {
    const int k0 = PT_K * j;
    char *sk = ring + j % S * R::BYTES, *sv = sk + S * R::BYTES;
    const int below = place + 1 - k0, above = task.window > 0 ? below - task.window : 0;
    if (t0 != t1 && at_edge(task, j) && __builtin_expect(wild<T, D>(sv), 0)) {
      tame<T, D>(sv);
      odd = true;
    }
    if (!live || k0 > most || (task.window > 0 && k0 + PT_K - 1 <= least - task.window)) return;
    sum.scores(sk + mine_at, qf, rd, s);
    if constexpr (MOD != 0) change<MOD, H>(s, sc, slope, k0 + 32 * H * half - place);
    if (there != 15 || k0 + PT_K - 1 > least || (task.window > 0 && k0 <= most - task.window))
      hide<H>(s, above - 32 * H * half, below - 32 * H * half, there >> 2 * H * half);
    sum.weigh(s, MOD ? 1.f : sc.c, pw);
    sum.add(sv + mine_at, pw, rd);
  };
  for (int j = last; j >= first;) {
    arrive<0>();
    const uint32_t there = bits;
    if (j > first) {
      bits = 15;
      if (j > whole) fetch(j - 1, look_up(j - 1));
      else bits = fetch_part(j - 1);
    }
    take(j, there);
    if (--j != upper || upper < lower) continue;
    int id = look_up(max(j - 1, lower));
    for (; j > lower; --j) {
      arrive<0>();
      fetch(j - 1, id);
      id = look_up(max(j - 2, lower));
      if (live) {
        sum.scores(ring + j % S * R::BYTES + mine_at, qf, rd, s);
        if constexpr (MOD != 0) change<MOD, H>(s, sc, slope, PT_K * j + 32 * H * half - place);
        sum.weigh(s, MOD ? 1.f : sc.c, pw);
        sum.add(ring + (S + j % S) * R::BYTES + mine_at, pw, rd);
      }
    }
    bits = 15;
  }
  auto mark = [&] {                                // whether the wave's sums hold what is not finite
    float bad = 0.f;
#pragma unroll
    for (int d = 0; d < L::DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) bad = fmaf(sum.o[d][i], 0.f, bad);
    const bool any = __ballot(bad != bad) != 0;
    if (lane == 0) odds[w % 4] = any;
  };
  if constexpr (KW == 1) mark();
  arrive<0>();
  if constexpr (KW > 1) {                          // the second half's sums go through LDS, lane by lane
    f4* theirs = reinterpret_cast<f4*>(ring) + (w % 4) * 64 * 4 * L::DT + lane;
    if (half == 1) {
#pragma unroll
      for (int d = 0; d < L::DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          theirs[64 * (4 * d + i)] = f4{sum.o[d][4 * i], sum.o[d][4 * i + 1], sum.o[d][4 * i + 2], sum.o[d][4 * i + 3]};
      stats[tid % (NT / 2)] = float2{sum.mc, sum.l};
    }
    __syncthreads();
    if (half == 0) {
      const float2 st = stats[tid];
      const float top = fmaxf(sum.mc, st.x), base = top == NEG_INF ? 0.f : top;
      const float a = exp2_fast(sum.mc - base), b = exp2_fast(st.x - base);
      sum.mc = top, sum.l = fmaf(st.y, b, sum.l * a);
#pragma unroll
      for (int d = 0; d < L::DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f4 y = theirs[64 * (4 * d + i)];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum.o[d][4 * i + e] = fmaf(y[e], b, sum.o[d][4 * i + e] * a);
        }
      mark();
      stats[tid].y = sum32(sum.l);
    }
    __syncthreads();
  }
  const bool writes = live && half == 0;
  if (task.shares == 1) {
    if (writes) sum.store(out + (task.token + t) * out_token + head * out_head, row < end, nchunk);
  } else if (writes) {
    // 64 dims at a time through LDS, so that rows are written whole
    float* own = reinterpret_cast<float*>(ring) + w * 32 * 68;
    const int64_t sums = ((int64_t)task.slot * ch.kv_heads + task.g) * ch.rows + 32 * w;
    const int left = end - row0;
#pragma unroll
    for (int d0 = 0; d0 < L::DT; d0 += 2) {
#pragma unroll
      for (int d = d0; d < min(d0 + 2, L::DT); ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f4*>(own + (lane & 31) * 68 + 32 * (d - d0) + 8 * (i / 4) + 4 * hi) =
              f4{sum.o[d][i], sum.o[d][i + 1], sum.o[d][i + 2], sum.o[d][i + 3]};
      __builtin_amdgcn_wave_barrier();
      const int d = 32 * d0 + 4 * (lane & 15);
      const bool there = d < ch.dim && 4 * (lane & 15) < 32 * (L::DT - d0);
#pragma unroll 2
      for (int x = lane / 16; x < min(left, 32); x += 4) {
        const f4 y = *reinterpret_cast<const f4*>(own + x * 68 + 4 * (lane & 15));
        if (there) *reinterpret_cast<f4*>(part + (sums + x) * ch.dim + d) = y;
      }
      __builtin_amdgcn_wave_barrier();
    }
    const float l = sum32(sum.l);
    if (hi == 0 && lane < left) *reinterpret_cast<float2*>(stat + 2 * (sums + lane)) = float2{sum.mc, l};
  }
  if (__builtin_expect(!(odd || (odds[0] | odds[1] | odds[2] | odds[3])), 1)) return;
  __syncthreads();
  float* total = reinterpret_cast<float*>(ring);
  if constexpr (KW > 1) {                          // (from there, not from a register: fewer are spilled in the loop)
    if (tid < CH_ROWS) total[tid] = stats[64 * (tid / 32) + tid % 32].y;
  } else {
    const float l = sum32(sum.l);
    if (hi == 0) total[32 * w + lane] = l;
  }
  add_wild<T>(pg, ch, task, out, out_token, out_head, part, total, reinterpret_cast<int*>(total + CH_ROWS));
}

// Join the shares of a row: a wave each, N lanes (of 4 dims each) for a share, 64 / N shares at once, eight loads on their way.
// A wave takes several rows of a tile where that has many: most calls with such tiles have nothing to join, and the blocks that
// find this out take their time too.
template <class T, int N>
__global__ void __launch_bounds__(256)
k_chunk_join(const Joint* __restrict__ joints, const int32_t* __restrict__ count, const float* __restrict__ part,
             const float* __restrict__ stat, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head, Chunks ch) {
  constexpr int AT_ONCE = 64 / N, AHEAD = 8;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g = blockIdx.x % ch.kv_heads, x = blockIdx.x / ch.kv_heads;
  const Joint jt = joints[x];                      // where there is none, what lies there is not used
  if (x >= min(*count, ch.slots / 2)) return;
  const int group = ch.heads / ch.kv_heads;
  // with offsets that do not ascend a tile may have no block, and its place here holds anything
  if (jt.shares <= 1 || jt.shares > CH_MOST || jt.slot < 0 || jt.step < 0 ||
      jt.slot + (int64_t)(jt.shares - 1) * jt.step >= ch.slots || jt.first < 0 || jt.row0 < 0)
    return;
  for (int r = 4 * blockIdx.y + w; r < min(jt.rows, ch.rows); r += 4 * gridDim.y) {
    const int64_t row = (int64_t)jt.row0 + r, token = jt.first + row / group;
    if (token >= ch.tokens) return;
    auto sums = [&](int i) { return ((int64_t)(jt.slot + i * jt.step) * ch.kv_heads + g) * ch.rows + r; };
    const int d = min(4 * (lane % N), ch.dim - 4), mine = lane / N;
    auto load = [&](int i) { return *reinterpret_cast<const f4*>(part + sums(min(i, jt.shares - 1)) * ch.dim + d); };
    const float2 raw = *reinterpret_cast<const float2*>(stat + 2 * sums(min(lane, jt.shares - 1)));
    f4 y[AHEAD];                                   // the first sums are on their way while the weights are made
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) y[i] = load(AT_ONCE * i + mine);
    const float2 st = lane < jt.shares ? raw : float2{NEG_INF, 0.f};
    float mm = st.x;
#pragma unroll
    for (int z = 32; z; z >>= 1) mm = fmaxf(mm, __shfl_xor(mm, z));
    const float base = mm == NEG_INF ? 0.f : mm;
    const float weight = exp2_fast(st.x - base), total = add64(st.y * weight);
    const float inv = total == 0.f ? 1.f : 1.f / total;  // sums of a row that sees no key are zero
    f4 sum = (f4)(0.f);
    for (int i0 = 0; i0 < jt.shares; i0 += AT_ONCE * AHEAD) {
      if (i0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) y[i] = load(i0 + AT_ONCE * i + mine);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int k = i0 + AT_ONCE * i + mine;
        const float a = __shfl(weight, min(k, 63));
        if (k < jt.shares) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = fmaf(y[i][e], fabsf(y[i][e]) < -NEG_INF ? a : 1.f, sum[e]);
        }
      }
    }
#pragma unroll
    for (int z = N; z < 64; z *= 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], z);
    if (lane < N && 4 * lane < ch.dim)
      *reinterpret_cast<u2*>(out + token * out_token + (g * group + row % group) * out_head + d) =
          u2{T::pack(sum[0] * inv, sum[1] * inv), T::pack(sum[2] * inv, sum[3] * inv)};
  }
}

}  // namespace pia
