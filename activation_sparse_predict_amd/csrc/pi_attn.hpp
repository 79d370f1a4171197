// Device code of the attention operators for gfx950.
//
// For a query row q and the keys j it sees, with c = scale log2(e):
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c (s_j - m)),  s_j = q . k_j
// with m the largest s_j so far; when m grows, what was summed is multiplied by
// 2^(c (m_old - m)).  Scores, m, the sums and o are float32.  The unnormalised
// p_j are rounded to the inputs' type for the second product (as the type's
// matrix instruction takes them): at most half a step each, relative to values
// in (0, 1], and independent between keys, so the output is off by less than
// its own rounding to that type.  sum_j p_j adds the unrounded values.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T, so that a lane holds all
// its scores for one query: softmax statistics need one or two cross-lane
// steps, and the D registers of the first product, rounded, are the B operand
// of the second (the order of the keys inside a matrix instruction is free).
#pragma once
#include "pi.h"
#include "pi_tile.hpp"

#include <type_traits>

namespace pia {

using namespace pit;

// A [tokens][heads][dim] tensor with its strides in elements (dim is contiguous).
struct Rows {
  const uint16_t* p;
  int64_t token, head;
  __device__ __forceinline__ const uint16_t* at(int64_t t, int h) const { return p + t * token + h * head; }
};

constexpr float NEG_INF = -__builtin_inff();

// ------------------------------------------------------- attention over prompts
constexpr int PT_K = 64;                 // keys of a tile
constexpr float RISE = 8.f;              // powers of two that a p_j may grow to before the sums are multiplied

// LDS rows of a tile: a power of two of 16-byte chunks, so that a row starts on
// a fixed bank, and chunk c of row r lies at position c ^ swz(r).  The 32 rows
// one operand read touches, and the 4 rows x 64 bytes that half a wave reads
// transposed, then cover every bank equally.
template <int D> struct Tile {
  static constexpr int NC = D <= 64 ? 8 : D <= 128 ? 16 : 32;   // chunks of a row in LDS
  static constexpr int KS = D / 16;                             // k steps of Q K^T
  static constexpr int DT = D / 32;                             // 32-wide tiles of the output
  static __device__ __forceinline__ int swz(int r) {
    if constexpr (NC == 8) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    else return ((r & 3) << 2) | ((r >> 2) & 3);
  }
  static __device__ __forceinline__ int chunk(int r, int c) { return r * NC + (c ^ swz(r)); }
};

// The block's sequence and its query tile: tiles are numbered sequence by
// sequence, the last (longest) tile of a sequence first.
struct Place {
  int start, len, tile;                  // first token, tokens, tile; len = 0: nothing to do
};
template <int ROWS>
__device__ __forceinline__ Place find_tile(const int32_t* cu, int n, int tokens, int idx) {
  const int lane = threadIdx.x & (WAVE - 1);
  for (int base = 0; base < n; base += WAVE) {
    const int i = base + lane;
    int a = 0, b = 0;
    if (i < n) {
      a = min(max(cu[i], 0), tokens);
      b = min(max(cu[i + 1], a), tokens);
    }
    const int t = (b - a + ROWS - 1) / ROWS;
    const int upto = scan64(t);
    const uint64_t hit = __ballot(upto > idx);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int st = __builtin_amdgcn_readlane(a, l), en = __builtin_amdgcn_readlane(b, l);
      const int last = __builtin_amdgcn_readlane(upto, l) - 1;
      return Place{st, en - st, last - idx};
    }
    idx -= __builtin_amdgcn_readlane(upto, WAVE - 1);
  }
  return Place{0, 0, 0};
}

// 16 bytes per lane from memory (base plus the lane's byte offset) into LDS, past the registers: lane i's go to
// byte lds + 16 i.  Written out because the compiler, which cannot tell buffers of one array apart, would wait for
// every such load before any read of LDS; `Ring` counts and waits for them.
__device__ __forceinline__ void to_lds(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}

// All but the wave's last N loads have come, its LDS reads are done, and so for every wave of the block.
template <int N> __device__ __forceinline__ void arrive() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Byte offsets of a lane's operand reads inside a tile in LDS.  The swizzle takes its bits from the lane alone, so
// the remaining row numbers are multiples of 16 rows that go into the instructions' offsets.
template <int D> struct Reads {
  using L = Tile<D>;
  uint32_t k[L::KS], v[2][L::DT];

  __device__ __forceinline__ explicit Reads(int lane) {
    const int hi = lane >> 5, col = lane & 31;
#pragma unroll
    for (int s = 0; s < L::KS; ++s) k[s] = 16 * L::chunk(col, 2 * s + hi);
    const int j = lane & 15, cc = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int t = 0; t < L::DT; ++t) v[e][t] = 16 * L::chunk(8 * e + 4 * hi + (j >> 2), 4 * t + cc) + 8 * (j & 1);
  }
  // K as A operand: keys 32 h .., dims 16 s ..
  __device__ __forceinline__ u4 kfrag(const char* sk, int h, int s) const {
    return *reinterpret_cast<const u4*>(sk + k[s] + 32 * 16 * L::NC * h);
  }
  // V^T as A operand, keys 16 step .., dims 32 t ..: transposing reads, each giving a lane 4 keys of one dimension
  __device__ __forceinline__ u4 vfrag(const char* sv, int step, int t) const {
    u4 f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const char* at = sv + v[e][t] + 16 * 16 * L::NC * step;
      const u2 x =
          __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)at));
      f[2 * e] = x[0];
      f[2 * e + 1] = x[1];
    }
    return f;
  }
};

// Tiles of K and V in LDS, S of each; tile j lies in place j % S.  NT threads fill them.
template <int D, int S, int NT> struct Ring {
  using L = Tile<D>;
  static constexpr int BYTES = PT_K * L::NC * 16;               // of a tile
  static constexpr int LD = PT_K * L::NC / NT;                  // loads of a thread for a tile
  static constexpr int RN = NT / L::NC;                         // rows that the block loads at once
  static constexpr int NV = RN < 16 ? 16 / RN : 1;              // such loads until the swizzle repeats
};

// A wave's sums for 32 queries: o, l, and the reference point mc of the exponents (c times a score, or -inf).
template <class T, int D> struct Sums {
  using L = Tile<D>;
  f16v o[L::DT];
  float mc, l;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < L::DT; ++t) o[t] = (f16v)(0.f);
    mc = NEG_INF, l = 0.f;
  }

  // Scores of one tile of 64 keys in LDS: register i of s[h] is key 32 h + 8 (i / 4) + 4 (lane / 32) + i % 4.
  static __device__ __forceinline__ void scores(const char* sk, const u4* qf, const Reads<D>& rd, f16v* s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = (f16v)(0.f);
#pragma unroll
      for (int ks = 0; ks < L::KS; ++ks) s[h] = T::mma32(rd.kfrag(sk, h, ks), qf[ks], s[h]);
    }
  }

  // Of a tile's scores, those of keys that a row does not see: it sees the first `seen`.
  static __device__ __forceinline__ void mask(f16v* s, int seen) {
    const int hi = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (32 * h + 8 * (i / 4) + 4 * hi + i % 4 >= seen) s[h][i] = NEG_INF;
  }

  // The weights of a tile's scores, rounded, and their part of l.
  __device__ __forceinline__ void weigh(const f16v* s, float c, uint32_t* pw) {
    // rows whose scores so far are all -inf keep mc = -inf; 0 stands in for it in the differences
    const float base = mc == NEG_INF ? 0.f : mc;
    float x[32], top = NEG_INF;
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = fmaf(s[i / 16][i % 16], c, -base);
#pragma unroll
    for (int i = 0; i < 32; i += 2) top = fmaxf(fmaxf(top, x[i]), x[i + 1]);
    top = max32(top);
    // mc may lag behind the largest score: p stays below 2^RISE, and o is seldom multiplied
    if (__ballot(top > RISE || mc == NEG_INF)) {
      const bool none = mc == NEG_INF;
      const float up = none ? (top == NEG_INF ? 0.f : top) : fmaxf(top, 0.f);
      // where there was no score yet o and l are zero, whatever they are multiplied by
      const float alpha = none ? 1.f : exp2_fast(-up);
      mc = none ? top : mc + up;
      l *= alpha;
#pragma unroll
      for (int t = 0; t < L::DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] *= alpha;
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] -= up;
    }
    float ls = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float a = exp2_fast(x[i]), b = exp2_fast(x[i + 1]);
      ls += a;
      ls += b;
      pw[i / 2] = T::pack(a, b);
    }
    l += ls;
  }

  __device__ __forceinline__ void add(const char* sv, const uint32_t* pw, const Reads<D>& rd) {
#pragma unroll
    for (int st = 0; st < 4; ++st)
#pragma unroll
      for (int t = 0; t < L::DT; ++t)
        o[t] = T::mma32(rd.vfrag(sv, st, t), u4{pw[4 * st], pw[4 * st + 1], pw[4 * st + 2], pw[4 * st + 3]}, o[t]);
  }

  // After the wave's first tile was added, of which a row saw the first `seen` keys: 0 times an infinity or NaN of a
  // key that is not seen is NaN.  Where any value came out non-finite the tile's sum is taken again key by key, adding
  // only to the rows that see the key (o held nothing before).
  __device__ __forceinline__ void mend(const char* sv, const uint32_t* pw, int seen, const Reads<D>& rd) {
    const int hi = (threadIdx.x & 63) >> 5;
    float bad = 0.f;
#pragma unroll
    for (int t = 0; t < L::DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) bad = fmaf(o[t][i], 0.f, bad);
    if (!__ballot(bad != bad)) return;
#pragma unroll
    for (int t = 0; t < L::DT; ++t) {
      o[t] = (f16v)(0.f);
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        const u4 vf = rd.vfrag(sv, st, t);
#pragma unroll 1
        for (int y = 0; y < 16; ++y) {             // key 16 st + y: element e of the lanes of half y / 4 % 2
          const int e = (y & 3) + 4 * (y >> 3);
          const bool mine = ((y >> 2) & 1) == hi;
          u4 va, pa;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t keep = mine && i == e / 2 ? (e & 1 ? 0xffff0000u : 0xffffu) : 0u;
            va[i] = vf[i] & keep;
            pa[i] = pw[4 * st + i] & keep;
          }
          const f16v one = T::mma32(va, pa, (f16v)(0.f));
          if (16 * st + y < seen)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][i] += one[i];
        }
      }
    }
  }

  // The rows' results: rows of `out` from `dst` on for the lane's query, where `live`.
  __device__ __forceinline__ void store(uint16_t* dst, bool live, int nchunk) const {
    const int hi = (threadIdx.x & 63) >> 5;
    const float total = sum32(l);
    const float inv = total == 0.f ? 0.f : 1.f / total;   // no weight at all (every score -inf): zero
#pragma unroll
    for (int t = 0; t < L::DT; ++t)
#pragma unroll
      for (int g = 0; g < 2; ++g) {                // 16 dims: the lane halves trade so that each stores 8
        const int i = 8 * g;
        const uint32_t a0 = T::pack(o[t][i] * inv, o[t][i + 1] * inv);
        const uint32_t a1 = T::pack(o[t][i + 2] * inv, o[t][i + 3] * inv);
        const uint32_t b0 = T::pack(o[t][i + 4] * inv, o[t][i + 5] * inv);
        const uint32_t b1 = T::pack(o[t][i + 6] * inv, o[t][i + 7] * inv);
        const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
        const int at = 4 * t + 2 * g + hi;
        if (live && at < nchunk) *reinterpret_cast<u4*>(dst + 8 * at) = u4{s0[0], s1[0], s0[1], s1[1]};
      }
  }
};

// One block of 4 waves: 32 query rows for each, of HG heads that share their
// keys and 128 / HG tokens of one sequence, over the keys up to the last row in
// tiles of 64 from the last one down.  A wave's rows lie in one 64-aligned span,
// so exactly the first tile it computes is partly masked.  K and V tiles go to
// LDS past the registers, one tile ahead of the products.
//
// At 8192 tokens and 56 heads of 128 the matrix cores are busy for half of the
// cycles and the card lowers its clock from 2.3 to 1.9 GHz (zeros in place of
// random data take 803 us, not 985): tiles three ahead, 8 waves a block, the
// products of one tile interleaved with the exponentials of another or in
// phases of their own, and other wave priorities all took as long or longer.
// Packing the heads of a key head into a block: 188 -> 169 us for 13 prompts of
// 6151 tokens, 128 heads on 8, 64 wide; four blocks a CU there: 164 us.
template <class T, int D, int HG>
__global__ void __launch_bounds__(4 * WAVE, D <= 64 ? 4 : D <= 128 ? 2 : 1)
k_attn_prompt(Rows q, Rows k, Rows v, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head,
              const int32_t* __restrict__ cu, int n, int tokens, int heads, int group, int dim, float c) {
  using L = Tile<D>;
  constexpr int NT = 4 * WAVE, ROWS = 128 / HG, S = 2;
  using R = Ring<D, S, NT>;
  __shared__ __attribute__((aligned(1024))) char ring[2 * S * R::BYTES];   // K tiles, then V tiles

  const int sets = heads / HG;
  int set = blockIdx.x % sets;
  // neighbouring sets of heads, which may share keys too, run on the same die (block b runs on die b % 8)
  if (sets % 8 == 0) set = (set % 8) * (sets / 8) + set / 8;
  const Place pl = find_tile<ROWS>(cu, n, tokens, blockIdx.x / sets);
  if (pl.len == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = set * HG + w % HG;
  const int row0 = ROWS * pl.tile + 32 * (w / HG);  // the wave's first row in the sequence
  const int row = row0 + (lane & 31), hi = lane >> 5;
  const int nchunk = dim / 8;
  if (nchunk < L::NC) {
    for (int e = tid; e < 2 * S * R::BYTES / 16; e += NT) reinterpret_cast<u4*>(ring)[e] = u4{0, 0, 0, 0};
    __syncthreads();
  }
  // A tile's rows into LDS, RN of them at once.  A chunk's place there follows from its thread; what it holds, from the
  // swizzle, which repeats after 16 rows.  Only a sequence's last tile can be short: its missing rows repeat the last.
  const int kv = head / group, r0 = tid / L::NC;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)ring + 1024 * w;
  int ch[R::NV];
#pragma unroll
  for (int i = 0; i < R::NV; ++i) ch[i] = (tid % L::NC) ^ L::swz(r0 + i * R::RN);
  auto load = [&](const Rows& x, int tile, uint32_t lds) {
    const uint16_t* base = x.at(pl.start + (int64_t)tile * PT_K, kv);
    const int left = pl.len - tile * PT_K;
    const uint32_t stride = 2 * (uint32_t)x.token;
#pragma unroll
    for (int i = 0; i < R::LD; ++i) {
      if (ch[i % R::NV] >= nchunk) continue;
      if (left >= PT_K)
        to_lds(reinterpret_cast<const char*>(base) + (int64_t)i * R::RN * stride, r0 * stride + 16 * ch[i % R::NV],
               lds + i * 16 * NT);
      else
        to_lds(base, min(i * R::RN + r0, left - 1) * stride + 16 * ch[i % R::NV], lds + i * 16 * NT);
    }
  };
  auto fetch = [&](int j) {
    load(k, j, lds0 + j % S * R::BYTES);
    load(v, j, lds0 + (S + j % S) * R::BYTES);
  };
  const int last = (min(pl.len, (pl.tile + 1) * ROWS) - 1) / PT_K;
  fetch(last);
  u4 qf[L::KS];
  {
    const uint16_t* src = q.at(pl.start + min(row, pl.len - 1), head);
#pragma unroll
    for (int s = 0; s < L::KS; ++s) {
      const int at = 2 * s + hi;
      qf[s] = at < nchunk ? *reinterpret_cast<const u4*>(src + 8 * at) : u4{0, 0, 0, 0};
    }
  }
  const Reads<D> rd(lane);
  Sums<T, D> sum;
  sum.clear();
  f16v s[2];
  uint32_t pw[16];
  const int mine = row0 / PT_K, seen = row - mine * PT_K + 1;
  int j = last;
  auto turn = [&] {
    arrive<0>();
    if (j > 0) fetch(j - 1);
  };
  for (; j > mine; --j) turn();
  if (j == mine) {
    turn();
    sum.scores(ring + j % S * R::BYTES, qf, rd, s);
    sum.mask(s, seen);
    sum.weigh(s, c, pw);
    sum.add(ring + (S + j % S) * R::BYTES, pw, rd);
    sum.mend(ring + (S + j % S) * R::BYTES, pw, seen, rd);
    --j;
  }
  for (; j >= 0; --j) {
    turn();
    sum.scores(ring + j % S * R::BYTES, qf, rd, s);
    sum.weigh(s, c, pw);
    sum.add(ring + (S + j % S) * R::BYTES, pw, rd);
  }
  if (row0 < pl.len) sum.store(out + (pl.start + row) * out_token + head * out_head, row < pl.len, nchunk);
}

// ------------------------------------------------ attention of single new tokens
// What a decode kernel sees of a cache's layer.
struct Pages {
  const uint16_t *k, *v;                 // the layer's pages [pages][kv_heads][page][dim]
  const int32_t *table, *lens;           // [slots][max_pages], [slots]
  int32_t* flags;                        // the cache's error word
  int pages, page, max_pages, slots;
};

constexpr int DC_WAVES = 4;
constexpr int DC_K = 32;                 // keys of a wave's step

// O^T of the 16x16x32 product: a lane's A operand row l % 16 stands for VW
// consecutive output dims (VW operands), so V is loaded with VW elements per
// lane, whole rows of the page by 16 lanes, and transposed in registers.
template <int D> struct Vec {
  static constexpr int W = D <= 64 ? 4 : 8;        // dims per lane and load
  static constexpr int G = D <= 128 ? 1 : D / 128; // such groups of 16 W dims
  static constexpr int KS = (D + 31) / 32;         // k steps of Q K^T
};

// The slot of batch row b, or -1.
__device__ __forceinline__ int slot_of(const int32_t* seqs, int b, int slots) {
  const int s = seqs ? seqs[b] : b;
  return (unsigned)s < (unsigned)slots ? s : -1;
}

// One block: the query heads [16 rt, 16 rt + 16) of a key head's group, one
// batch row, and one of `splits` shares of its keys; the waves take steps of 32
// keys in turn and join their sums through LDS.  Partial results (or, with one
// share, the output) are written per query head.
template <class T, int D>
__global__ void __launch_bounds__(DC_WAVES * WAVE)
k_attn_decode(Pages pg, Rows q, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head,
              const int32_t* __restrict__ seqs, int heads, int kv_heads, int dim, int splits, float c,
              float* __restrict__ part, float* __restrict__ stat) {
  using V = Vec<D>;
  constexpr int NF = V::W * V::G;                  // operands of the second product
  __shared__ float sm[DC_WAVES][2][16];
  __shared__ float so[DC_WAVES][16][16 * NF + 4];

  const int b = blockIdx.z, split = blockIdx.x, group = heads / kv_heads;
  const int rts = (group + 15) / 16, g = blockIdx.y / rts, rt = blockIdx.y % rts;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kg = lane >> 4;
  const int slot = slot_of(seqs, b, pg.slots);
  int len = slot >= 0 ? pg.lens[slot] : 0;
  if (slot < 0 || len < 0 || len > (int64_t)pg.max_pages * pg.page) {
    if (tid == 0) atomicOr(pg.flags, slot < 0 ? PI_CACHE_ESLOT : PI_CACHE_ELENGTH);
    len = 0;
  }
  const int steps = (len + DC_K - 1) / DC_K;
  const int first = (int)((int64_t)steps * split / splits), last = (int)((int64_t)steps * (split + 1) / splits);
  const int nchunk = dim / 8;

  const int head = g * group + 16 * rt + min(r, group - 16 * rt - 1);
  u4 qf[V::KS];
#pragma unroll
  for (int s = 0; s < V::KS; ++s) {
    const int ch = 4 * s + kg;
    qf[s] = ch < nchunk ? *reinterpret_cast<const u4*>(q.at(b, head) + 8 * ch) : u4{0, 0, 0, 0};
  }
  f4 o[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) o[f] = (f4)(0.f);
  float m = NEG_INF, l = 0.f;
  const int32_t* row = pg.table + (int64_t)max(slot, 0) * pg.max_pages;
  const int64_t head_stride = (int64_t)pg.page * dim, page_stride = head_stride * kv_heads;

  for (int st = first + w; st < last; st += DC_WAVES) {
    // the two halves of 16 keys lie in one page each (pages hold multiples of 16 tokens)
    const uint16_t *kp[2], *vp[2];
    int seen[2];                                   // keys of the half that exist
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = st * DC_K + 16 * h;
      seen[h] = max(0, min(16, len - key));
      const int place = min(key / pg.page, pg.max_pages - 1);
      int id = row[place];
      if ((unsigned)id >= (unsigned)pg.pages) {    // a broken table: its keys are not seen
        if (seen[h] && lane == 0) atomicOr(pg.flags, PI_CACHE_EPAGE);
        seen[h] = 0;
        id = 0;
      }
      const int64_t at = id * page_stride + g * head_stride + (int64_t)(key % pg.page) * dim;
      kp[h] = pg.k + at;
      vp[h] = pg.v + at;
    }
    f4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = (f4)(0.f);
#pragma unroll
      for (int ks = 0; ks < V::KS; ++ks) {
        const int ch = 4 * ks + kg;
        u4 a = {0, 0, 0, 0};
        if (ch < nchunk) a = *reinterpret_cast<const u4*>(kp[h] + r * dim + 8 * ch);
        s[h] = T::mma16(a, qf[ks], s[h]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * kg + i >= seen[h]) s[h][i] = NEG_INF;
    }
    float mt = NEG_INF;
#pragma unroll
    for (int i = 0; i < 4; ++i) mt = fmaxf(mt, fmaxf(s[0][i], s[1][i]));
    const float mn = fmaxf(m, max16(mt));
    const float mc = mn == NEG_INF ? 0.f : mn * c;   // see k_attn_prompt
    const float alpha = exp2_fast(fmaf(m, c, -mc));
    m = mn;
    float p[8], ls = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp2_fast(fmaf(s[i / 4][i % 4], c, -mc));
      ls += p[i];
    }
    l = fmaf(l, alpha, ls);
    const u4 pf = {T::pack(p[0], p[1]), T::pack(p[2], p[3]), T::pack(p[4], p[5]), T::pack(p[6], p[7])};
    // V: keys 4 kg + 0..3 of both halves; rows that do not exist count as zeros, whatever is stored there
#pragma unroll
    for (int gr = 0; gr < V::G; ++gr) {
      uint32_t x[8][V::W / 2];
      const int d0 = (16 * gr + r) * V::W;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = 4 * kg + i % 4;
#pragma unroll
        for (int e = 0; e < V::W / 2; ++e) x[i][e] = 0;
        if (key < seen[i / 4] && d0 < dim) {
          const uint16_t* src = vp[i / 4] + key * dim + d0;
          if constexpr (V::W == 8) {
            const u4 y = *reinterpret_cast<const u4*>(src);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = y[e];
          } else {
            const u2 y = *reinterpret_cast<const u2*>(src);
#pragma unroll
            for (int e = 0; e < 2; ++e) x[i][e] = y[e];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < V::W / 2; ++e) {
        const u4 a = {lows(x[0][e], x[1][e]), lows(x[2][e], x[3][e]), lows(x[4][e], x[5][e]), lows(x[6][e], x[7][e])};
        const u4 z = {highs(x[0][e], x[1][e]), highs(x[2][e], x[3][e]), highs(x[4][e], x[5][e]),
                      highs(x[6][e], x[7][e])};
        const int f = gr * V::W + 2 * e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[f][i] *= alpha;
          o[f + 1][i] *= alpha;
        }
        o[f] = T::mma16(a, pf, o[f]);
        o[f + 1] = T::mma16(z, pf, o[f + 1]);
      }
    }
  }
  l = sum16(l);

  // join the waves: o[f][i] belongs to dim (16 gr + 4 kg + i) W + f % W of query r
  if (lane < 16) {
    sm[w][0][r] = m;
    sm[w][1][r] = l;
  }
#pragma unroll
  for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int f = 0; f < V::W; ++f) so[w][r][(16 * gr + 4 * kg + i) * V::W + f] = o[gr * V::W + f][i];
  __syncthreads();
  for (int e = tid; e < 16 * dim; e += DC_WAVES * WAVE) {
    const int qr = e / dim, d = e % dim;
    if (16 * rt + qr >= group) break;
    float mm = NEG_INF;
#pragma unroll
    for (int i = 0; i < DC_WAVES; ++i) mm = fmaxf(mm, sm[i][0][qr]);
    const float mc = mm == NEG_INF ? 0.f : mm * c;
    float ll = 0.f, oo = 0.f;
#pragma unroll
    for (int i = 0; i < DC_WAVES; ++i) {
      const float a = exp2_fast(fmaf(sm[i][0][qr], c, -mc));
      ll = fmaf(sm[i][1][qr], a, ll);
      oo = fmaf(so[i][qr][d], a, oo);
    }
    const int h = g * group + 16 * rt + qr;
    if (splits == 1) {
      const float y = ll == 0.f ? 0.f : oo / ll;   // a row that sees no key is zero
      out[b * out_token + h * out_head + d] = (uint16_t)T::pack(y, 0.f);
    } else {
      const int64_t at = ((int64_t)b * heads + h) * splits + split;
      part[at * dim + d] = oo;
      if (d == 0) {
        stat[2 * at] = mm;
        stat[2 * at + 1] = ll;
      }
    }
  }
}

// Join a row's shares: one block per (batch row, query head).
template <class T>
__global__ void __launch_bounds__(256)
k_attn_join(const float* __restrict__ part, const float* __restrict__ stat, uint16_t* __restrict__ out,
            int64_t out_token, int64_t out_head, int heads, int dim, int splits, float c) {
  const int b = blockIdx.x / heads, h = blockIdx.x % heads;
  const float* st = stat + 2 * (int64_t)blockIdx.x * splits;
  float mm = NEG_INF;
  for (int i = 0; i < splits; ++i) mm = fmaxf(mm, st[2 * i]);
  const float mc = mm == NEG_INF ? 0.f : mm * c;
  for (int d = threadIdx.x; d < dim; d += blockDim.x) {
    float ll = 0.f, oo = 0.f;
    for (int i = 0; i < splits; ++i) {
      const float a = exp2_fast(fmaf(st[2 * i], c, -mc));
      ll = fmaf(st[2 * i + 1], a, ll);
      oo = fmaf(part[((int64_t)blockIdx.x * splits + i) * dim + d], a, oo);
    }
    out[b * out_token + h * out_head + d] = (uint16_t)T::pack(ll == 0.f ? 0.f : oo / ll, 0.f);
  }
}

}  // namespace pia
