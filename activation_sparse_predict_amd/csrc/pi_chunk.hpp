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

constexpr int CH_ROWS = 128;             // rows of a block
constexpr int CH_MOST = 64;              // shares of a tile's keys at most

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
  int free, least;                       // shares to deal beside one a tile; key tiles of a share at least
  int slots, rows;                       // places for sums in the workspace, rows of each
  uint32_t mul, shift;                   // a place's page: mulhi(2 place, mul) >> shift
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
  s.tiles = (int)(((int64_t)s.count * group + CH_ROWS - 1) / CH_ROWS);
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

// Every tile of rows has one share; `free` more go to those with most keys.  Sums are float32: what they may be off by is
// made up for in the size of a share, so that the blocks there are suffice.  `count`: count the tiles that are shared out too.
__device__ __forceinline__ Piece find_piece(const Pages& pg, const Chunks& ch, int window, int idx, bool count) {
  const int lane = threadIdx.x & (WAVE - 1);
  Seq s = seq_of(pg, ch, window, lane);
  float work = (float)s.tiles * (float)s.keys;
  for (int base = WAVE; base < ch.n; base += WAVE) {
    const Seq x = seq_of(pg, ch, window, base + lane);
    work += (float)x.tiles * (float)x.keys;
  }
  const float all = add64(work);
  const uint32_t size = __builtin_amdgcn_readfirstlane(
      max((uint32_t)ch.least, (uint32_t)min(all / (float)ch.free * 1.0001f, 2e9f) + 1));
  Piece p{};
  p.size = size;
  int slot = 0, joint = 0;
  bool found = false;
  for (int base = 0; base < ch.n; base += WAVE) {
    if (base) s = seq_of(pg, ch, window, base + lane);
    const int n = max(1, min(CH_MOST, (int)(((uint32_t)s.keys + size - 1) / size)));
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

// A table's entry by a scalar load: the tables do not change while the kernel runs.
__device__ __forceinline__ int entry(const int32_t* table, int at) {
  typedef const __attribute__((address_space(4))) int32_t* fixed;
  return reinterpret_cast<fixed>(reinterpret_cast<uintptr_t>(table))[at];
}

// A tile's scores as the softmax takes them, in units of log2(e).  `back` is the tile's first key minus the row's place.
template <int MOD>
__device__ __forceinline__ void change(f16v* s, const ChunkScore& sc, float slope, int back) {
  const float at = slope * (float)(back + 4 * (int)((threadIdx.x & 63) >> 5));
#pragma unroll
  for (int h = 0; h < 2; ++h)
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

// Scores of keys that a row does not see: it sees those from `lo` on and before `hi` in the places of 16 that `bits` names.
__device__ __forceinline__ void hide(f16v* s, int lo, int hi, uint32_t bits) {
  const int half = 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = 32 * h + 8 * (i / 4) + i % 4;
      if (key >= hi - half || key < lo - half || !(bits >> (2 * h + i / 8) & 1)) s[h][i] = NEG_INF;
    }
}

// Whether a tile in LDS holds a value that is not finite.
template <class T, int D> __device__ __forceinline__ bool wild(const char* tile) {
  typedef unsigned short h2 __attribute__((ext_vector_type(2)));
  h2 top = {0, 0};
#pragma unroll
  for (int i = 0; i < Tile<D>::NC; ++i) {
    const u4 x = *reinterpret_cast<const u4*>(tile + 16 * (64 * i + (threadIdx.x & 63)));
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(h2, x[e] & 0x7fff7fffu));
  }
  return __ballot(top[0] >= T::INF || top[1] >= T::INF) != 0;
}

// 0 times an infinity or NaN of a value that a row does not see is NaN.  So where a tile that is not seen by all of a block's
// rows holds such values, they are added as they are, by the rows that see them (a weight times an infinity is that
// infinity, times NaN is NaN), and count as zeros after that: `add_wild` by every wave, then `tame` by all threads.
template <class T, int D>
__device__ __forceinline__ void add_wild(Sums<T, D>& sum, const char* sv, int lo, int hi) {
  using L = Tile<D>;
  const int half = (threadIdx.x & 63) >> 5;
#pragma unroll 1
  for (int key = 0; key < PT_K; ++key) {
    const bool seen = key < hi && key >= lo;
#pragma unroll
    for (int c = 0; c < 4 * L::DT; ++c) {          // dims 8 c + 4 half ..
      const u2 x = *reinterpret_cast<const u2*>(sv + 16 * L::chunk(key, c) + 8 * half);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (seen && (x[e] & 0x7fffu) >= T::INF) sum.o[c / 4][4 * (c % 4) + 2 * e] += T::low(x[e]);
        if (seen && (x[e] >> 16 & 0x7fffu) >= T::INF) sum.o[c / 4][4 * (c % 4) + 2 * e + 1] += T::high(x[e]);
      }
    }
  }
}
template <class T, int D> __device__ __forceinline__ void tame(char* sv) {
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < PT_K * Tile<D>::NC; i += blockDim.x) {
    u4 x = *reinterpret_cast<const u4*>(sv + 16 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] &= ((x[e] & 0x7fffu) >= T::INF ? 0u : 0xffffu) | ((x[e] >> 16 & 0x7fffu) >= T::INF ? 0u : 0xffff0000u);
    *reinterpret_cast<u4*>(sv + 16 * i) = x;
  }
  __syncthreads();
}

// One block of 4 waves: 128 rows of a key head, 32 for each wave, over one share of the keys that any of them sees, in
// tiles of 64 from the last one down, which go to LDS past the registers one tile ahead of the products.
template <class T, int D, int MOD>
__global__ void __launch_bounds__(4 * WAVE, D <= 64 ? 4 : D <= 128 ? 2 : 1)
k_attn_chunk(Pages pg, Rows q, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head, Chunks ch, ChunkScore sc,
             Joint* __restrict__ joints, int32_t* __restrict__ count, float* __restrict__ part, float* __restrict__ stat) {
  using L = Tile<D>;
  constexpr int NT = 4 * WAVE, S = 2;
  using R = Ring<D, S, NT>;
  constexpr int SUMS = 4 * 32 * 68 * 4;            // sums on their way out
  __shared__ __attribute__((aligned(1024))) char ring[2 * S * R::BYTES > SUMS ? 2 * S * R::BYTES : SUMS];   // K tiles, then V tiles

  // key heads of a piece run side by side, those of one head on one die where they can (block b runs on die b % 8)
  const int g = blockIdx.x % ch.kv_heads, idx = blockIdx.x / ch.kv_heads;
  const Piece pc = find_piece(pg, ch, sc.window, idx, blockIdx.x == 0);
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), hi = lane >> 5;
  if (blockIdx.x == 0 && tid == 0) *count = pc.joints;
  if (pc.s.count == 0) return;
  const int group = ch.heads / ch.kv_heads, nchunk = ch.dim / 8;
  const int before = pc.s.len - pc.s.count;        // place of the chunk's first token
  const int rows = min(CH_ROWS, pc.s.count * group - CH_ROWS * pc.tile);
  const int row_first = CH_ROWS * pc.tile;
  const int t0 = row_first / group, t1 = (row_first + rows - 1) / group;     // its tokens
  const int to = max(0, before + t1 + 1), from = sc.window > 0 ? max(0, before + t0 + 1 - sc.window) : 0;
  const int tiles = to > from ? (to - 1) / PT_K - from / PT_K + 1 : 0;
  // shares of this tile: no more than its keys need
  const int n = max(1, min(pc.shares, (int)(((uint32_t)tiles + pc.size - 1) / pc.size)));
  if (blockIdx.x % ch.kv_heads == 0 && pc.share == 0 && tid == 0) {
    if (pc.s.slot < 0 || pc.s.len != pc.s.raw || before < 0)
      atomicOr(pg.flags, pc.s.slot < 0 ? PI_CACHE_ESLOT : PI_CACHE_ELENGTH);
    if (pc.shares > 1 && pc.joint < ch.slots / 2)
      joints[pc.joint] = Joint{pc.slot, n, pc.s.first, row_first, rows, pc.s.tiles};
  }
  if (pc.share >= n) return;
  const int first = from / PT_K + share_begin(tiles, pc.share, n), last = from / PT_K + share_begin(tiles, pc.share + 1, n) - 1;

  const int row0 = row_first + 32 * w, row = row0 + (lane & 31), end = row_first + rows;
  const bool live = row0 < end;
  const int mine = min(row, end - 1), t = mine / group, head = g * group + mine % group;
  const int place = before + t;                    // the row sees keys up to here
  const int least = before + row0 / group, most = before + (min(row0 + 32, end) - 1) / group;   // of the wave's rows
  if (nchunk < L::NC) {
    for (int e = tid; e < 2 * S * R::BYTES / 16; e += NT) reinterpret_cast<u4*>(ring)[e] = u4{0, 0, 0, 0};
    __syncthreads();
  }
  u4 qf[L::KS];
  {
    const uint16_t* src = q.at(pc.s.first + t, head);
#pragma unroll
    for (int s = 0; s < L::KS; ++s) {
      const int at = 2 * s + hi;
      qf[s] = at < nchunk ? *reinterpret_cast<const u4*>(src + 8 * at) : u4{0, 0, 0, 0};
    }
  }
  const float slope = (MOD & CH_SLOPES) && sc.slopes ? sc.slopes[head] * 1.44269504f : 0.f;

  const int32_t* table = pg.table + (int64_t)max(pc.s.slot, 0) * pg.max_pages;
  const uint32_t head_bytes = 2 * pg.page * ch.dim, page_bytes = head_bytes * ch.kv_heads;     // at most 2^31
  const char *kg = reinterpret_cast<const char*>(pg.k) + (int64_t)g * head_bytes;
  const char *vg = reinterpret_cast<const char*>(pg.v) + (int64_t)g * head_bytes;
  auto page_of = [&](uint32_t x) { return (int)(__umulhi(2 * x, ch.mul) >> ch.shift); };
  // byte of a place of 16 keys, from its page's number
  auto place_at = [&](int x, int id) {
    return uniform((int64_t)((uint64_t)(uint32_t)id * page_bytes + (uint32_t)(x - page_of(x) * (pg.page / 16)) * (uint32_t)(32 * ch.dim)));
  };
  // A wave loads one place of a tile, LW times 1024 bytes.  What a lane takes of it is the chunk that its place in LDS asks for.
  constexpr int LW = L::NC / 4, RL = 64 / L::NC;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)ring + 1024 * LW * w;
  uint32_t off[LW];
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int r = i * RL + lane / L::NC, c = (lane % L::NC) ^ L::swz(r);
    off[i] = c < nchunk ? 2 * (uint32_t)(r * ch.dim + 8 * c) : ~0u;
  }
  auto look_up = [&](int j) { return entry(table, page_of(4 * j + w)); };
  // a tile that is whole: every place is there, and some row sees every key
  auto fetch = [&](int j, int id) {
    const int64_t at = place_at(4 * j + w, id);
    const char *ka = kg + at, *va = vg + at;
    const uint32_t dst = lds0 + j % S * R::BYTES;
    if (nchunk == L::NC) {
#pragma unroll
      for (int i = 0; i < LW; ++i) to_lds(ka, off[i], dst + 1024 * i);
#pragma unroll
      for (int i = 0; i < LW; ++i) to_lds(va, off[i], dst + S * R::BYTES + 1024 * i);
    } else {
#pragma unroll
      for (int i = 0; i < LW; ++i)
        if (off[i] != ~0u) {
          to_lds(ka, off[i], dst + 1024 * i);
          to_lds(va, off[i], dst + S * R::BYTES + 1024 * i);
        }
    }
  };
  // Any tile; keys that no row sees are zeros: with anything else there, 0 times an infinity would be NaN.  Which places
  // there are.
  auto fetch_part = [&](int j) {
    const int x = 4 * j + w;
    const bool inside = 16 * x < to && 16 * x + 16 > from;
    const int id = inside ? usable_page(entry(table, page_of(x)), pg.pages) : -1;
    const int64_t at = place_at(x, max(id, 0));
    const uint32_t dst = lds0 + j % S * R::BYTES;
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int key = 16 * x + i * RL + lane / L::NC;
      if (id >= 0 && key < to && key >= from) {
        if (off[i] != ~0u) {
          to_lds(kg + at, off[i], dst + 1024 * i);
          to_lds(vg + at, off[i], dst + S * R::BYTES + 1024 * i);
        }
      } else {
        char* own = ring + j % S * R::BYTES + 1024 * (LW * w + i) + 16 * lane;
        *reinterpret_cast<u4*>(own) = *reinterpret_cast<u4*>(own + S * R::BYTES) = u4{0, 0, 0, 0};
      }
    }
    uint32_t bits = 0;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int y = 4 * j + i;
      if (16 * y >= to || 16 * y + 16 <= from) continue;
      if (usable_page(entry(table, page_of(y)), pg.pages) >= 0) bits |= 1u << i;
      else if (tid == 0) atomicOr(pg.flags, PI_CACHE_EPAGE);
    }
    return bits;
  };
  const Reads<D> rd(lane);
  Sums<T, D> sum;
  sum.clear();
  f16v s[2];
  uint32_t pw[16];
  uint32_t bits = 0;
  if (first <= last) bits = fetch_part(last);
  // tiles below the last one that every row of the block sees whole; none where a page is broken
  int upper = min(last - 1, (before + t0 + 1) / PT_K - 1), lower = max(first, (from + PT_K - 1) / PT_K);
  if (sc.window > 0) lower = max(lower, (before + t1 - sc.window) / PT_K + 1);
  if (upper >= lower) {
    bool broken = false;
    for (int e = page_of(4 * lower) + tid, end = page_of(4 * last); e <= end; e += NT) broken |= usable_page(table[e], pg.pages) < 0;
    if (__syncthreads_or(broken)) upper = lower - 1;
  }
  // one tile of any kind, which lies in LDS; `there`: its places
  auto take = [&](int j, uint32_t there) {
    const int k0 = PT_K * j;
    char *sk = ring + j % S * R::BYTES, *sv = sk + S * R::BYTES;
    const int below = place + 1 - k0, above = sc.window > 0 ? below - sc.window : 0;
    if (t0 != t1 && (k0 + PT_K - 1 > before + t0 || (sc.window > 0 && k0 <= before + t1 - sc.window)) && wild<T, D>(sv)) {
      add_wild(sum, sv, above, below);
      tame<T, D>(sv);
    }
    if (!live || k0 > most || (sc.window > 0 && k0 + PT_K - 1 <= least - sc.window)) return;
    sum.scores(sk, qf, rd, s);
    if constexpr (MOD != 0) change<MOD>(s, sc, slope, k0 - place);
    if (there != 15 || k0 + PT_K - 1 > least || (sc.window > 0 && k0 <= most - sc.window)) hide(s, above, below, there);
    sum.weigh(s, MOD ? 1.f : sc.c, pw);
    sum.add(sv, pw, rd);
  };
  for (int j = last; j >= first;) {
    arrive<0>();
    const uint32_t there = bits;
    if (j > first) bits = fetch_part(j - 1);
    take(j, there);
    if (--j != upper || upper < lower) continue;
    int id = look_up(max(j - 1, lower));
    for (; j > lower; --j) {
      arrive<0>();
      fetch(j - 1, id);
      id = look_up(max(j - 2, lower));
      if (live) {
        sum.scores(ring + j % S * R::BYTES, qf, rd, s);
        if constexpr (MOD != 0) change<MOD>(s, sc, slope, PT_K * j - place);
        sum.weigh(s, MOD ? 1.f : sc.c, pw);
        sum.add(ring + (S + j % S) * R::BYTES, pw, rd);
      }
    }
    bits = 15;
  }
  if (n == 1) {
    if (live) sum.store(out + (pc.s.first + t) * out_token + head * out_head, row < end, nchunk);
    return;
  }
  // 64 dims at a time through LDS, so that rows are written whole
  arrive<0>();
  const int slot = (pc.slot + pc.share * pc.s.tiles) ;
  if (!live || slot >= ch.slots) return;
  float* own = reinterpret_cast<float*>(ring) + w * 32 * 68;
  const int64_t sums = ((int64_t)slot * ch.kv_heads + g) * ch.rows + 32 * w;
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = 4 * i + lane / 16;
      const f4 y = *reinterpret_cast<const f4*>(own + x * 68 + 4 * (lane & 15));
      if (x < left && d < ch.dim && 4 * (lane & 15) < 32 * (L::DT - d0)) *reinterpret_cast<f4*>(part + (sums + x) * ch.dim + d) = y;
    }
    __builtin_amdgcn_wave_barrier();
  }
  const float l = sum32(sum.l);
  if (hi == 0 && lane < left) *reinterpret_cast<float2*>(stat + 2 * (sums + lane)) = float2{sum.mc, l};
}

// Join the shares of a row: a wave each, all lanes on a share's dims.
template <class T>
__global__ void __launch_bounds__(256)
k_chunk_join(const Joint* __restrict__ joints, const int32_t* __restrict__ count, const float* __restrict__ part,
             const float* __restrict__ stat, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head, Chunks ch) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g = blockIdx.x % ch.kv_heads, x = blockIdx.x / ch.kv_heads, r = 4 * blockIdx.y + w;
  if (x >= min(*count, ch.slots / 2)) return;
  const Joint jt = joints[x];
  if (jt.shares <= 1 || r >= jt.rows || jt.slot + (jt.shares - 1) * jt.step >= ch.slots) return;
  const int group = ch.heads / ch.kv_heads, row = jt.row0 + r;
  auto sums = [&](int i) { return ((int64_t)(jt.slot + i * jt.step) * ch.kv_heads + g) * ch.rows + r; };
  float2 st = float2{NEG_INF, 0.f};
  if (lane < jt.shares) st = *reinterpret_cast<const float2*>(stat + 2 * sums(lane));
  float mm = st.x;
#pragma unroll
  for (int y = 32; y; y >>= 1) mm = fmaxf(mm, __shfl_xor(mm, y));
  const float base = mm == NEG_INF ? 0.f : mm;
  const float weight = exp2_fast(st.x - base), total = add64(lane < jt.shares ? st.y * weight : 0.f);
  const float inv = total == 0.f ? 0.f : 1.f / total;    // a row that sees no key is zero
  f4 sum = (f4)(0.f);
  const int d = min(4 * lane, ch.dim - 4);
  for (int i = 0; i < jt.shares; ++i) {
    const f4 y = *reinterpret_cast<const f4*>(part + sums(i) * ch.dim + d);
    const float a = __shfl(weight, i);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = fmaf(y[e], a, sum[e]);
  }
  if (4 * lane < ch.dim)
    *reinterpret_cast<u2*>(out + (jt.first + row / group) * out_token + (g * group + row % group) * out_head + d) =
        u2{T::pack(sum[0] * inv, sum[1] * inv), T::pack(sum[2] * inv, sum[3] * inv)};
}

}  // namespace pia
