// Device code of rotary positions and norms of heads for gfx950.
//
// The angle of pair i at position p is p f_i.  f_i comes as a part of a turn in units
// of 2^-64, so the product modulo 2^64 is the angle modulo a turn without any rounding,
// for every position.  Its upper 32 bits give the nearest quarter turn and, as a float32,
// the rest of at most an eighth of a turn, of which sine and cosine are their series:
// |a| <= pi / 4, what is left out is below 2^-29 (sine, after a^9) and 2^-25 (cosine,
// after a^8).
#pragma once
#include "pi.h"
#include "pi_meta.hpp"
#include "pi_tile.hpp"

namespace pir {

using namespace pit;

// Which dimensions a lane holds as A[0..7] and B[0..7] of a head:
//  NONE, PAIRS  chunks of 8 dims 2 l and 2 l + 1; pairs lie inside a chunk
//  HALF         rotary % 16 == 0: chunk l and the one rotary / 2 dims on; the lanes
//               behind these take what does not turn, two chunks each
//  ODD          other rotary: dims 8 l .. of the first half and of the second, which
//               starts on no chunk; rows come and go in chunks l and l + P and are
//               taken apart in LDS (3018 tokens of 64 heads on 8, 128 wide, 62 of them
//               turned, with norms: 93 us with values loaded and stored one by one, 49 so; 22
//               the bytes take, but lanes that turn and others are counted apart, so of 16
//               lanes a head half have work)
enum { NONE = 0, HALF = 1, PAIRS = 2, ODD = 3 };

struct Turn {
  const uint64_t* steps;
  int rotary;
  float magnitude;
};

// Some heads of a tensor [tokens][heads][dim] and what they become.
struct Part {
  const uint16_t* src;
  int64_t src_token, src_head;
  uint16_t* dst;
  int64_t dst_token, dst_head;
  const float* weight;                   // of their norm, or NULL
  int heads;
};

// cos and sin of 2 pi u 2^-32, times m
__device__ __forceinline__ void sincos_turns(uint32_t u, float m, float* c, float* s) {
  const uint32_t q = (u + 0x20000000u) >> 30;                  // the nearest quarter, modulo 4
  const int32_t rest = (int32_t)(u - (q << 30));               // of it, within an eighth of a turn
  const float a = (float)rest * (6.28318530717958648f / 4294967296.f), b = a * a;
  float sn = fmaf(b, 2.7557319223985893e-6f, -1.9841269841269841e-4f);
  sn = fmaf(b, sn, 8.3333333333333333e-3f);
  sn = fmaf(b, sn, -1.6666666666666667e-1f);
  sn = fmaf(b * a, sn, a);
  float cs = fmaf(b, 2.4801587301587302e-5f, -1.3888888888888889e-3f);
  cs = fmaf(b, cs, 4.1666666666666667e-2f);
  cs = fmaf(b, cs, -0.5f);
  cs = fmaf(b, cs, 1.f);
  const float x = q & 1 ? sn : cs, y = q & 1 ? cs : sn;
  *c = (q == 1 || q == 2 ? -x : x) * m;
  *s = (q & 2 ? -y : y) * m;
}

// The sequence that holds token t, and its first and last offset: the first i whose end cu[i + 1] lies behind t, by a wave, 64
// places at once; -1 if there is none.  `ends`: of up to 64 sequences the lane's end, asked for before.
struct Found {
  int i, from, to;
};
__device__ __forceinline__ Found find_seq(const int32_t* cu, int n, int t, int ends) {
  const int lane = threadIdx.x & (WAVE - 1);
  int lo = 0, len = n;
  while (len > WAVE) {
    const int step = (len + WAVE - 1) / WAVE;
    const uint64_t hit = __ballot(cu[lo + min((lane + 1) * step, len)] > t);
    if (!hit) return Found{-1, 0, 0};
    const int before = (__ffsll((unsigned long long)hit) - 1) * step;
    lo += before;
    len = min(step, len - before);
  }
  if (n > WAVE) ends = cu[lo + min(lane + 1, len)];
  const uint64_t hit = __ballot(ends > t);
  if (!hit) return Found{-1, 0, 0};                // behind the last sequence
  const int l = __ffsll((unsigned long long)hit) - 1;
  const int from = l > 0 ? __builtin_amdgcn_readlane(ends, l - 1) : fixed(cu, lo);
  return Found{from <= t ? lo + l : -1, from, __builtin_amdgcn_readlane(ends, l)};
}

// Dims of a lane: of A from a on (na of them), of B from b on; whether they turn.
struct Dims {
  int a, b, na, nb;
  bool turns;
};
template <int MODE> __device__ __forceinline__ Dims dims_of(int l, int dim, int rotary) {
  auto upto = [&](int at) { return max(0, min(8, dim - at)); };
  if constexpr (MODE == HALF) {
    const int r = rotary / 16;
    if (l < r) return Dims{8 * l, rotary / 2 + 8 * l, 8, 8, true};
    const int at = rotary + 16 * (l - r);
    return Dims{at, at + 8, upto(at), upto(at + 8), false};
  } else if constexpr (MODE == ODD) {
    const int half = rotary / 2, r = (half + 7) / 8;
    if (l < r) return Dims{8 * l, half + 8 * l, min(8, half - 8 * l), min(8, half - 8 * l), true};
    const int at = rotary + 16 * (l - r);
    return Dims{at, at + 8, upto(at), upto(at + 8), false};
  } else {
    return Dims{16 * l, 16 * l + 8, upto(16 * l), upto(16 * l + 8), MODE == PAIRS && 16 * l < rotary};
  }
}

// What a wave's lanes wrote to LDS is there for its other lanes, as they read it in order.
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave takes one token and up to ITS turns, each of 64 / P heads of one kind, P = 2^shift lanes a head: those of q, then of
// k, then of v, which is copied.  All it loads is asked for before anything else, without conditions, and no load follows a
// store: the counter that a wave waits on counts both, in order (with the next turn's loads behind a turn's stores: 133 us,
// not 50, for 6151 tokens of 64 heads on 8, 128 wide, with norms).  The angles are made once for all turns.  That case: 45 us
// in the kernel, 5.0 TB/s read and written, the rate of a large copy.
template <class T, int MODE, bool PAGED, int ITS>
__global__ void __launch_bounds__(256)
k_rope(Turn turn, Part q, Part k, Part v, const int32_t* __restrict__ pos, pic::Meta m,
       const int32_t* __restrict__ cu, const int32_t* __restrict__ seqs, int n, int tokens, int dim, float eps, int shift,
       uint32_t waves) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t job = (blockIdx.y * gridDim.x + blockIdx.x) * 4 + w;   // neighbouring waves take neighbouring heads
  const int t = (int)(job / waves), part = (int)(job % waves);
  if (job / waves >= (uint32_t)tokens) return;
  const int l = lane & ((1 << shift) - 1), mine = lane >> shift, per = 64 >> shift;
  const Dims d = dims_of<MODE>(l, dim, turn.rotary);
  const int q_turns = (q.heads + per - 1) / per, k_turns = (k.heads + per - 1) / per;
  const int begin = part * ITS, end = min(begin + ITS, q_turns + (PAGED ? 2 : 1) * k_turns);

  // a turn's heads: kind 0 q, 1 k, 2 v, from the first one on
  struct Heads {
    int kind, first;
  };
  auto heads_of = [&](int it) {
    if (it < q_turns) return Heads{0, it * per};
    it -= q_turns;
    return it < k_turns ? Heads{1, it * per} : Heads{2, (it - k_turns) * per};
  };
  // What a position in the cache hangs on comes first, as loads come in order.  (Steps behind the rows, before them: 6151
  // tokens of 64 heads on 8, turned, 50.0 and 54.0 us; appended, 32 heads on 8, 36.0 and 34.7.)
  int ends = 0;
  uint64_t steps[8];
  auto load_steps = [&] {
    if constexpr (MODE != NONE) {
      const int first = d.turns ? 8 * l : 0, pairs = turn.rotary / 2;
#pragma unroll
      for (int e = 0; e < 8; ++e) steps[e] = turn.steps[min(first + e, pairs - 1)];
    }
  };
  if constexpr (PAGED) {
    ends = cu[min(lane + 1, n)];
    load_steps();
  }
  const int ca = MODE == ODD ? 8 * l : d.a, cb = MODE == ODD ? 8 * (l + (1 << shift)) : d.b;   // the chunks that a lane moves
  const bool has_a = MODE == ODD ? ca < dim : d.na > 0, has_b = MODE == ODD ? cb < dim : d.nb > 0;
  __shared__ u4 apart[MODE == ODD ? 4 * 128 : 1];
  uint16_t* own = reinterpret_cast<uint16_t*>(apart + (MODE == ODD ? 128 * w : 0)) + mine * dim;   // the lane's head
  u4 ra[ITS], rb[ITS];
#pragma unroll
  for (int i = 0; i < ITS; ++i) {                  // those that are not there are others again
    const Heads h = heads_of(min(begin + i, end - 1));
    const Part& x = h.kind == 0 ? q : h.kind == 1 ? k : v;
    const uint16_t* src = x.src + t * x.src_token + min(h.first + mine, x.heads - 1) * x.src_head;
    ra[i] = *reinterpret_cast<const u4*>(src + min(ca, dim - 8));
    rb[i] = *reinterpret_cast<const u4*>(src + min(cb, dim - 8));
  }
  float qn[16], kn[16];
  auto weights = [&](const float* from, float* n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = from[min(d.a + e, dim - 1)], n[8 + e] = from[min(d.b + e, dim - 1)];
  };
  if (q.weight && begin < q_turns) weights(q.weight, qn);
  if (k.weight && end > q_turns) weights(k.weight, kn);

  if (!PAGED) load_steps();
  int at = 0;                                      // the token's position
  bool paged = true;
  int64_t page_at = 0;                             // of the cache's page and token, in elements
  if constexpr (PAGED) {
    const Found f = find_seq(cu, n, t, ends);
    if (f.i < 0) return;
    const int slot = fixed(seqs, f.i);
    int bad = 0;
    if ((unsigned)slot >= (unsigned)m.slots) {
      bad = PI_CACHE_ESLOT;
    } else {
      const int64_t p = (int64_t)fixed(m.lens, slot) - f.to + t;
      if (p < 0 || p >= (int64_t)m.max_pages * m.page) {
        bad = PI_CACHE_ELENGTH;
      } else {
        at = (int)p;
        const int id = fixed(m.table, (int64_t)slot * m.max_pages + at / m.page);
        if ((unsigned)id >= (unsigned)m.pages) bad = PI_CACHE_EPAGE, paged = false;
        else page_at = ((int64_t)id * k.heads * m.page + at % m.page) * dim;
      }
    }
    if (bad && lane == 0) atomicOr(&m.words[1], bad);
    if (bad & ~PI_CACHE_EPAGE) return;
  } else if (MODE != NONE) {
    at = fixed(pos, t);
  }
  float cs[8], sn[8];
  if constexpr (MODE != NONE) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      sincos_turns((uint32_t)(((uint64_t)(int64_t)at * steps[e]) >> 32), turn.magnitude, &cs[e], &sn[e]);
  }
  const float over = 1.f / (float)dim;
#pragma unroll
  for (int i = 0; i < ITS; ++i) {
    if (begin + i >= end) break;
    const Heads h = heads_of(begin + i);
    const float* weight = h.kind == 0 ? q.weight : h.kind == 1 ? k.weight : nullptr;
    u4 ya = ra[i], yb = rb[i];
    if constexpr (MODE != ODD) {
      if (d.na == 0) ya = u4{0, 0, 0, 0};
      if (d.nb == 0) yb = u4{0, 0, 0, 0};
    }
    if (MODE == ODD && h.kind < 2) {
      if (has_a) *reinterpret_cast<u4*>(own + ca) = ya;
      if (has_b) *reinterpret_cast<u4*>(own + cb) = yb;
      settle();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a0 = own[min(d.a + 2 * e, dim - 1)], a1 = own[min(d.a + 2 * e + 1, dim - 1)];
        const uint32_t b0 = own[min(d.b + 2 * e, dim - 1)], b1 = own[min(d.b + 2 * e + 1, dim - 1)];
        ya[e] = (2 * e < d.na ? a0 : 0) | (2 * e + 1 < d.na ? a1 << 16 : 0);
        yb[e] = (2 * e < d.nb ? b0 : 0) | (2 * e + 1 < d.nb ? b1 << 16 : 0);
      }
      settle();
    }
    if (h.kind < 2 && (MODE != NONE || weight)) {
      float x[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = T::low(ya[e]), x[2 * e + 1] = T::high(ya[e]);
        x[8 + 2 * e] = T::low(yb[e]), x[8 + 2 * e + 1] = T::high(yb[e]);
      }
      if (weight) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        for (int o = 1; o < 1 << shift; o *= 2) ss += __shfl_xor(ss, o);
        const float inv = rsqrtf(fmaf(ss, over, eps));
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= inv * (h.kind == 0 ? qn[e] : kn[e]);
      }
      if constexpr (MODE == HALF || MODE == ODD) {
        if (d.turns) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = x[8 + e];
            x[e] = fmaf(a, cs[e], -(b * sn[e]));
            x[8 + e] = fmaf(b, cs[e], a * sn[e]);
          }
        }
      } else if constexpr (MODE == PAIRS) {
        const int some = turn.rotary / 2 - 8 * l;  // of the lane's pairs, those that turn
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = x[2 * e], b = x[2 * e + 1];
          x[2 * e] = e < some ? fmaf(a, cs[e], -(b * sn[e])) : a;
          x[2 * e + 1] = e < some ? fmaf(b, cs[e], a * sn[e]) : b;
        }
      }
      if (d.turns || weight) {                     // all else is moved bit by bit
        // (a lane may hold pairs of both kinds, and a NaN that is widened and packed again need not keep its bits)
        const int packed = MODE == PAIRS && !weight ? turn.rotary / 2 - 8 * l : 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (MODE != PAIRS || e < packed) ya[e] = T::pack(x[2 * e], x[2 * e + 1]);
          if (MODE != PAIRS || 4 + e < packed) yb[e] = T::pack(x[8 + 2 * e], x[8 + 2 * e + 1]);
        }
      }
    }
    if (MODE == ODD && h.kind < 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e < d.na) own[d.a + e] = (uint16_t)(ya[e / 2] >> 16 * (e % 2));
        if (e < d.nb) own[d.b + e] = (uint16_t)(yb[e / 2] >> 16 * (e % 2));
      }
      settle();
      ya = *reinterpret_cast<const u4*>(own + min(ca, dim - 8));
      yb = *reinterpret_cast<const u4*>(own + min(cb, dim - 8));
      settle();
    }
    const Part& y = h.kind == 0 ? q : h.kind == 1 ? k : v;
    if (h.first + mine >= y.heads || (PAGED && h.kind > 0 && !paged)) continue;
    const int64_t token = PAGED && h.kind > 0 ? page_at : t * y.dst_token;
    const int64_t head = PAGED && h.kind > 0 ? (int64_t)m.page * dim : y.dst_head;
    uint16_t* dst = y.dst + token + h.first * head + mine * head;
    if (has_a) *reinterpret_cast<u4*>(dst + ca) = ya;
    if (has_b) *reinterpret_cast<u4*>(dst + cb) = yb;
  }
}

}  // namespace pir
