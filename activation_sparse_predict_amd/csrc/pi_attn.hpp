// Device code of the attention operators for gfx950.
//
// For a query row q and the keys j it sees, with c = scale log2(e):
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c (s_j - m)),  s_j = q . k_j
// with c m a reference point near the largest c s_j so far; when it moves, what was
// summed is multiplied by 2^(c (m_old - m)).  Scores, m, the sums and o are float32.
// The p_j are rounded to the inputs' type for the second product, as the type's
// matrix instruction takes them; sum_j p_j adds the unrounded values.  A p_j that is
// normal in the type is off by at most half a step u of its own, so o by at most
// u sum_j p_j |v_j| / sum_j p_j, about as much as by its own rounding.
// binary16 has no normal values below 2^-14: were the largest p_j 1, keys 2^14 times
// below one that outscores all others would lose bits, below 2^25 times vanish, and
// where that one's value is small they are the result.  So c m lies LOW under the
// largest c s_j it was taken from, which makes that p_j 2^LOW, and moves once a p_j
// passes 2^(LOW + LAG), 2^15 in binary16: bits go only 2^25 times below the largest,
// and no more than 2^-36 of it a key.  A kernel that moves c m with every rise puts
// it HIGH under the largest (2^29 times, 2^-40).  bfloat16 has float32's exponents
// and needs neither.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T, so that a lane holds all
// its scores for one query: softmax statistics need one or two cross-lane
// steps, and the D registers of the first product, rounded, are the B operand
// of the second (the order of the keys inside a matrix instruction is free).
#pragma once
#include "pi.h"
#include "pi_share.hpp"
#include "pi_tile.hpp"

#include <type_traits>

namespace pia {

using namespace pit;
using namespace pish;

// A [tokens][heads][dim] tensor with its strides in elements (dim is contiguous).
struct Rows {
  const uint16_t* p;
  int64_t token, head;
  __device__ __forceinline__ const uint16_t* at(int64_t t, int h) const { return p + t * token + h * head; }
};

constexpr float NEG_INF = -__builtin_inff();

// ------------------------------------------------------- attention over prompts
constexpr int PT_K = 64;                 // keys of a tile

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
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(lds), "v"(off), "s"(base) : "memory");
}

// All but the wave's last N loads have come, its LDS reads are done, and so for every wave of the block.
template <int N> __device__ __forceinline__ void arrive() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Byte offsets of a lane's operand reads inside a tile in LDS.  The swizzle takes its bits from the lane alone, so
// the remaining row numbers are multiples of 16 rows that go into the instructions' offsets.
template <int D> struct Reads {
  using L = Tile<D>;
  // The swizzle leaves bit 4 of a chunk's number alone, so in rows of 32 chunks the second 16 lie 256 bytes on.
  static constexpr int KN = L::NC == 32 ? L::KS / 2 : L::KS, VN = L::NC == 32 ? L::DT / 2 : L::DT;
  uint32_t k[KN], v[2][VN];

  __device__ __forceinline__ explicit Reads(int lane) {
    const int hi = lane >> 5, col = lane & 31;
#pragma unroll
    for (int s = 0; s < KN; ++s) k[s] = 16 * L::chunk(col, 2 * s + hi);
    const int j = lane & 15, cc = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int t = 0; t < VN; ++t) v[e][t] = 16 * L::chunk(8 * e + 4 * hi + (j >> 2), 4 * t + cc) + 8 * (j & 1);
  }
  // K as A operand: keys 32 h .., dims 16 s ..
  __device__ __forceinline__ u4 kfrag(const char* sk, int h, int s) const {
    return *reinterpret_cast<const u4*>(sk + k[s % KN] + 256 * (s / KN) + 32 * 16 * L::NC * h);
  }
  // V^T as A operand, keys 16 step .., dims 32 t ..: transposing reads, each giving a lane 4 keys of one dimension
  __device__ __forceinline__ u4 vfrag(const char* sv, int step, int t) const {
    u4 f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const char* at = sv + v[e][t % VN] + 256 * (t / VN) + 16 * 16 * L::NC * step;
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

// A wave's sums for 32 queries: o, l, and the reference point mc of the exponents (c times a score, or -inf).  It takes H
// times 32 keys of a tile.
template <class T, int D, int H = 2> struct Sums {
  using L = Tile<D>;
  f16v o[L::DT];
  float mc, l;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < L::DT; ++t) o[t] = (f16v)(0.f);
    mc = NEG_INF, l = 0.f;
  }

  // Scores of a tile's keys in LDS: register i of s[h] is key 32 h + 8 (i / 4) + 4 (lane / 32) + i % 4.
  static __device__ __forceinline__ void scores(const char* sk, const u4* qf, const Reads<D>& rd, f16v* s) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      s[h] = (f16v)(0.f);
#pragma unroll
      for (int ks = 0; ks < L::KS; ++ks) s[h] = T::mma32(rd.kfrag(sk, h, ks), qf[ks], s[h]);
    }
  }

  // Of a tile's scores, those of keys that a row does not see: it sees the first `seen`.
  static __device__ __forceinline__ void mask(f16v* s, int seen) {
    const int limit = seen - 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (32 * h + 8 * (i / 4) + i % 4 >= limit) s[h][i] = NEG_INF;
  }

  // The weights of a tile's scores, rounded, and their part of l.
  __device__ __forceinline__ void weigh(const f16v* s, float c, uint32_t* pw) {
    // rows whose scores so far are all -inf keep mc = -inf; 0 stands in for it in the differences
    const float base = mc == NEG_INF ? 0.f : mc;
    float x[16 * H], top = NEG_INF;
#pragma unroll
    for (int i = 0; i < 16 * H; ++i) x[i] = fmaf(s[i / 16][i % 16], c, -base);
#pragma unroll
    for (int i = 0; i < 16 * H; i += 2) top = fmaxf(fmaxf(top, x[i]), x[i + 1]);
    top = max32(top);
    // mc may lag behind the largest score by LAG more than LOW, so that o is seldom multiplied.  (binary16, 8192 tokens of
    // 56 heads of 128, scores of deviation 1 and 3: LAG 2 1001 and 1039 us, 4 991 and 1022, 8 991 and 1005.)
    if (__ballot(top > T::LOW + T::LAG || mc == NEG_INF)) {
      const bool none = mc == NEG_INF;
      const float low = top - T::LOW;
      const float up = none ? (top == NEG_INF ? 0.f : low) : fmaxf(low, 0.f);
      // where there was no score yet o and l are zero, whatever they are multiplied by
      const float alpha = none ? 1.f : exp2_fast(-up);
      mc = none ? low : mc + up;
      l *= alpha;
#pragma unroll
      for (int t = 0; t < L::DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] *= alpha;
#pragma unroll
      for (int i = 0; i < 16 * H; ++i) x[i] -= up;
    }
    float ls = 0.f;
#pragma unroll
    for (int i = 0; i < 16 * H; i += 2) {
      const float a = exp2_fast(x[i]), b = exp2_fast(x[i + 1]);
      ls += a;
      ls += b;
      pw[i / 2] = T::pack(a, b);
    }
    l += ls;
  }

  __device__ __forceinline__ void add(const char* sv, const uint32_t* pw, const Reads<D>& rd) {
#pragma unroll
    for (int st = 0; st < 2 * H; ++st)
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

// The slot of batch row b, or -1.
__device__ __forceinline__ int slot_of(const int32_t* seqs, int b, int slots) {
  const int s = seqs ? seqs[b] : b;
  return (unsigned)s < (unsigned)slots ? s : -1;
}

// Tokens of batch row b; none where the slot or its length cannot be.
__device__ __forceinline__ int len_of(const Pages& pg, const int32_t* seqs, int b) {
  const int slot = slot_of(seqs, b, pg.slots);
  return usable_len(slot >= 0 ? pg.lens[slot] : 0, pg.max_pages, pg.page);
}

__device__ __forceinline__ int common_of(const Pages& pg, const int32_t* prefix) {
  return prefix ? common_tokens(*prefix, pg.max_pages, pg.page) : 0;
}

// The batch row whose table names the common pages: the first that holds them, or -1.
__device__ __forceinline__ int holder_of(const Pages& pg, const int32_t* seqs, int batch, int total) {
  const int lane = threadIdx.x & (WAVE - 1);
  for (int base = 0; base < batch; base += WAVE) {
    const int b = base + lane;
    const uint64_t hit = __ballot(b < batch && len_of(pg, seqs, b) >= total);
    if (hit) return base + __ffsll((unsigned long long)hit) - 1;
  }
  return -1;
}

// Whether batch row b has the common pages in common with that row, by all threads of a block; if not, the error word says so.
__device__ __forceinline__ void check_common(const Pages& pg, const int32_t* seqs, int batch, int total, int b) {
  if (total == 0 || b >= batch || len_of(pg, seqs, b) < total) return;
  const int holder = holder_of(pg, seqs, batch, total);
  const int32_t* first = pg.table + (int64_t)slot_of(seqs, holder, pg.slots) * pg.max_pages;
  const int32_t* mine = pg.table + (int64_t)slot_of(seqs, b, pg.slots) * pg.max_pages;
  bool other = false;
#pragma unroll 4
  for (int i = threadIdx.x; i < total / pg.page; i += blockDim.x) other |= first[i] != mine[i];
  if (other) atomicOr(pg.flags, PI_CACHE_EPREFIX);
}

// ---- the common keys, for all queries of a key head at once.
//
// One block of 4 waves: 32 query rows (batch row, head of the group) for each,
// over one share of the common keys, in tiles of 64 through LDS as in
// k_attn_prompt, S - 1 of them ahead.  Tiles are found through the pages; 16
// keys lie in one page.  24 rows of 128 heads on 8, 64 wide, over 32768 common
// keys: 50 us, 520 TFLOP/s, bound by the exponentials and the latency of a tile's
// steps with two waves on a SIMD (17 us without the products and exponentials).
// part, stat: unnormalised sums, and (reference point, l) of each.
constexpr int SH_IDS = 256;              // places of 16 keys that are looked up at once: 64 tiles

template <class T, int D>
__global__ void __launch_bounds__(4 * WAVE, D <= 64 ? 3 : 1)
k_attn_common(Pages pg, Rows q, const int32_t* __restrict__ seqs, const int32_t* __restrict__ prefix, int batch,
              int heads, int kv_heads, int dim, int shares, int qtiles, float c, float* __restrict__ part,
              float* __restrict__ stat) {
  using L = Tile<D>;
  constexpr int NT = 4 * WAVE, S = D <= 128 ? 3 : 2;
  using R = Ring<D, S, NT>;
  __shared__ __attribute__((aligned(1024))) char ring[2 * S * R::BYTES];   // K tiles, then V tiles
  __shared__ int64_t ids[SH_IDS];                  // first element of 16 keys in the layer's pages, or -1: not seen

  // the query tiles of one share run on one die (block b runs on die b % 8)
  const int pair = blockIdx.x % 8 + 8 * (blockIdx.x / (8 * qtiles)), qt = blockIdx.x / 8 % qtiles;
  const int g = pair / shares, share = pair % shares;
  if (g >= kv_heads) return;
  const int total = common_of(pg, prefix);
  if (total == 0) return;
  const int n = common_shares(total, shares);
  if (share >= n) return;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), hi = lane >> 5;
  const int holder = holder_of(pg, seqs, batch, total);
  if (holder < 0) return;
  const int32_t* table = pg.table + (int64_t)slot_of(seqs, holder, pg.slots) * pg.max_pages;

  const int group = heads / kv_heads, nchunk = dim / 8;
  const int row0 = 128 * qt + 32 * w, row = row0 + (lane & 31);
  const bool live = row0 < batch * group;
  const int b = min(row / group, batch - 1), head = g * group + row % group;
  u4 qf[L::KS];
#pragma unroll
  for (int s = 0; s < L::KS; ++s) {
    const int at = 2 * s + hi;
    qf[s] = at < nchunk ? *reinterpret_cast<const u4*>(q.at(b, head) + 8 * at) : u4{0, 0, 0, 0};
  }
  if (nchunk < L::NC) {                            // chunks that no load fills
    for (int e = tid; e < 2 * S * R::BYTES / 16; e += NT) reinterpret_cast<u4*>(ring)[e] = u4{0, 0, 0, 0};
  }
  const int tiles = pieces(total, PT_K);
  const int first = share_begin(tiles, share, n), last = share_begin(tiles, share + 1, n);
  const int r0 = tid / L::NC;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)ring + 1024 * w;
  const int per = pg.page / 16;
  // the places of the tiles from `base` on; whether one of them is broken
  auto look_up = [&](int base) {
    bool bad = false;
    const int at = 4 * base + tid;
    if (at < 4 * last) {
      const bool there = at < total / 16;          // the last tile may be short
      const int x = there ? at : 0, id = usable_page(table[x / per], pg.pages);
      bad = id < 0 && there;
      ids[tid] = bad || !there ? -1 : (((int64_t)id * kv_heads + g) * pg.page + x % per * 16) * dim;
      if (bad) atomicOr(pg.flags, PI_CACHE_EPAGE);
    }
    return __syncthreads_or(bad) != 0;
  };
  auto place = [&](int at) {
    const int64_t v = ids[at];
    const uint32_t a = __builtin_amdgcn_readfirstlane((uint32_t)v), h = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (int64_t)((uint64_t)h << 32 | a);
  };
  // a tile into LDS; keys that are not seen are zeros: with anything else there, 0 times an infinity would be NaN
  auto fetch = [&](int tile, int base) {
#pragma unroll
    for (int i = 0; i < R::LD; ++i) {
      const int r = i * R::RN + r0, ch = (tid % L::NC) ^ L::swz(r);
      const int rw = i * R::RN + 64 * w / L::NC;   // the wave's first row: its rows lie in one page
      const int64_t at = place(4 * (tile - base) + rw / 16);
      const uint32_t to = lds0 + tile % S * R::BYTES + i * 16 * NT;
      if (at >= 0) {
        const uint32_t off = 2 * (uint32_t)(r % 16 * dim + 8 * ch);
        if (ch < nchunk) {
          to_lds(pg.k + at, off, to);
          to_lds(pg.v + at, off, to + S * R::BYTES);
        }
      } else {
        char* own = ring + tile % S * R::BYTES + i * 16 * NT + 16 * tid;
        *reinterpret_cast<u4*>(own) = *reinterpret_cast<u4*>(own + S * R::BYTES) = u4{0, 0, 0, 0};
      }
    }
  };
  // Tiles are fetched S - 1 ahead.  For each on its way, four bits say which of its 16-key places are seen; the next
  // tile's are the lowest.
  int base = first;
  bool broken = look_up(base), any = broken;
  uint32_t seen = 0;
  auto ahead = [&](int t) {                        // the place of tile t - S has been read by every wave
    if (t - base == SH_IDS / 4) {
      __syncthreads();                             // as have the ids
      base = t;
      broken = look_up(base);
      any |= broken;
    }
    uint32_t bits = 15;
    if (broken) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (place(4 * (t - base) + i) < 0) bits &= ~(1u << i);
    }
    if (total - t * PT_K < PT_K) {
      bits &= (1u << (total - t * PT_K) / 16) - 1;
      any = true;
    }
    seen |= bits << 4 * (t % S);
    fetch(t, base);
  };
  for (int t = first; t < min(last, first + S - 1); ++t) ahead(t);
  // what was fetched for the S - 2 tiles behind this one may still be on its way; at the end, and where keys that are not
  // seen were not loaded (`any`), there are fewer
  auto turn = [&](int t) {
    if (t + S - 2 < last && !any) arrive<(S - 2) * 2 * R::LD>();
    else arrive<0>();
    const uint32_t sees = seen >> 4 * (t % S) & 15;
    seen &= ~(15u << 4 * (t % S));
    if (t + S - 1 < last) ahead(t + S - 1);
    return sees;
  };
  if (!live) {                                     // the wave has nothing to do but keep step
    for (int t = first; t < last; ++t) turn(t);
    arrive<0>();
    return;
  }
  const Reads<D> rd(lane);
  Sums<T, D> sum;
  sum.clear();
  for (int t = first; t < last; ++t) {
    const uint32_t sees = turn(t);
    const char *sk = ring + t % S * R::BYTES, *sv = ring + (S + t % S) * R::BYTES;
    f16v s[2];
    uint32_t pw[16];
    if (sees == 15) {
      sum.scores(sk, qf, rd, s);
      sum.weigh(s, c, pw);
      sum.add(sv, pw, rd);
    } else {
      sum.scores(sk, qf, rd, s);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!(sees >> (2 * h + i / 8) & 1)) s[h][i] = NEG_INF;
      sum.weigh(s, c, pw);
      sum.add(sv, pw, rd);
    }
  }
  // 64 dims at a time through LDS, so that rows are written whole
  arrive<0>();
  float* own = reinterpret_cast<float*>(ring) + w * 32 * 68;
  const int rows = min(32, batch * group - row0);
  auto place_of = [&](int x) { return ((int64_t)(x / group) * heads + g * group + x % group) * shares + share; };
#pragma unroll
  for (int t0 = 0; t0 < L::DT; t0 += 2) {
#pragma unroll
    for (int t = t0; t < min(t0 + 2, L::DT); ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f4*>(own + (lane & 31) * 68 + 32 * (t - t0) + 8 * (i / 4) + 4 * hi) =
            f4{sum.o[t][i], sum.o[t][i + 1], sum.o[t][i + 2], sum.o[t][i + 3]};
    __builtin_amdgcn_wave_barrier();
    const int d = 32 * t0 + 4 * (lane & 15);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = 4 * i + lane / 16;
      const f4 y = *reinterpret_cast<const f4*>(own + x * 68 + 4 * (lane & 15));
      if (x < rows && d < dim && 4 * (lane & 15) < 32 * (L::DT - t0)) *reinterpret_cast<f4*>(part + place_of(row0 + x) * dim + d) = y;
    }
    __builtin_amdgcn_wave_barrier();
  }
  const float l = sum32(sum.l);
  if (hi == 0 && lane < rows) *reinterpret_cast<float2*>(stat + 2 * place_of(row)) = float2{sum.mc, l};
}

// ---- the keys of each row's own.
constexpr int DC_WAVES = 4;
constexpr int DC_K = 32;                 // keys of a wave's step
static_assert(DC_WAVES * DC_K == UNIT && PT_K == TILE, "pi_share.hpp");
constexpr int DC_ROWS = 1024;            // tiles of queries that fill the card with one share a row

// O^T of the 16x16x32 product: a lane's A operand row l % 16 stands for VW
// consecutive output dims (VW operands), so V is loaded with VW elements per
// lane, whole rows of the page by 16 lanes, and transposed in registers.
template <int D> struct Vec {
  static constexpr int W = D <= 64 ? 4 : 8;        // dims per lane and load
  static constexpr int G = D <= 128 ? 1 : D / 128; // such groups of 16 W dims
  static constexpr int KS = (D + 31) / 32;         // k steps of Q K^T
};

// A block's batch row, its slot and tokens, and which of how many shares of its own keys the block takes.
struct Share {
  int b, slot, len, i, n;                // n = 0: nothing to do
};

// Block b < batch takes the first share of row b; the others follow the rows, in their order.  A row of no more than
// `least` units has one share, which needs no look at the other rows.
__device__ __forceinline__ Share find_share(const Pages& pg, const int32_t* seqs, int batch, int total, int idx, int free,
                                            int least) {
  const int lane = threadIdx.x & (WAVE - 1);
  int slot = -1, len = 0;                          // of the row that `units` was last asked for
  auto units = [&](int b) {
    slot = b < batch ? slot_of(seqs, b, pg.slots) : -1;
    len = slot >= 0 ? pg.lens[slot] : 0;
    const int n = usable_len(len, pg.max_pages, pg.page);
    return units_of(n - (n >= total ? total : 0));
  };
  int mine, own = 0, own_slot = -1, own_len = 0;
  if (idx < batch && batch > WAVE) {
    own = units(idx), own_slot = slot, own_len = len;
    if (own <= least) return Share{idx, slot, len, 0, 1};
  }
  mine = units(lane);
  if (idx < batch && batch <= WAVE) {
    own = __builtin_amdgcn_readlane(mine, idx);
    own_slot = __builtin_amdgcn_readlane(slot, idx);
    own_len = __builtin_amdgcn_readlane(len, idx);
    if (own <= least) return Share{idx, own_slot, own_len, 0, 1};
  }
  // of one row at most 2^24 units: the sum of 64 rows fits 31 bits
  uint64_t all;
  int most = mine;
  if (batch <= WAVE) {
    all = __builtin_amdgcn_readlane(scan64(mine), WAVE - 1);
  } else {                                         // 64 rows a lane: so do the lanes' sums, and 64 of their halves
    int sum = mine;
#pragma unroll 4
    for (int base = WAVE; base < batch; base += WAVE) {
      const int n = units(base + lane);
      sum += n;
      most = max(most, n);
    }
    all = (uint64_t)__builtin_amdgcn_readlane(scan64(sum & 0xffff), WAVE - 1) +
          ((uint64_t)__builtin_amdgcn_readlane(scan64(sum >> 16), WAVE - 1) << 16);
  }
  const uint32_t size = max(share_size(all, free), (uint32_t)least);
  if (idx < batch) return Share{idx, own_slot, own_len, 0, deal(own, size)};
  if (batch > WAVE && !__ballot(deal(most, size) > 1)) return Share{0, -1, 0, 0, 0};   // nothing to deal
  idx -= batch;
  for (int base = 0; base < batch; base += WAVE) {
    if (batch > WAVE) mine = units(base + lane);
    const int n = base + lane < batch ? deal(mine, size) - 1 : 0;
    const int upto = scan64(n);
    const uint64_t hit = __ballot(upto > idx);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int others = __builtin_amdgcn_readlane(n, l);
      return Share{base + l, __builtin_amdgcn_readlane(slot, l), __builtin_amdgcn_readlane(len, l),
                   1 + idx - (__builtin_amdgcn_readlane(upto, l) - others), 1 + others};
    }
    idx -= __builtin_amdgcn_readlane(upto, WAVE - 1);
  }
  return Share{0, -1, 0, 0, 0};
}

// One block: the query heads [16 rt, 16 rt + 16) of a key head's group, one
// batch row, and one share of the keys behind the common ones; the waves take
// steps of 32 keys in turn and join their sums through LDS.  Where a row has
// one share and no common keys its result is written; else the sums go to
// `part` and `stat` and the row's shares to `plan`, for k_attn_join.  (Joining
// in the row's last block instead costs more: its loads have to pass the die's
// cache.  1500 tokens: 16 us, not 13; with an agent-scope fence 52 us.)
// With a prefix, blocks behind the last query tile compare the rows' tables with
// the one that k_attn_common reads, beside the others.  (32 rows behind 4096
// common tokens: 37.5 us, 37.4 without.)
template <class T, int D>
__global__ void __launch_bounds__(DC_WAVES * WAVE, D <= 128 ? 2 : 1)
k_attn_decode(Pages pg, Rows q, uint16_t* __restrict__ out, int64_t out_token, int64_t out_head,
              const int32_t* __restrict__ seqs, const int32_t* __restrict__ prefix, int batch, int heads, int kv_heads,
              int dim, int free, int least, int shares, float c, int4* __restrict__ plan, float* __restrict__ part,
              float* __restrict__ stat) {
  using V = Vec<D>;
  constexpr int NF = V::W * V::G;                  // operands of the second product
  constexpr int ROW = 16 * NF + 4;
  __shared__ float sm[DC_WAVES][2][16];
  __shared__ float so[DC_WAVES][16][ROW];

  const int group = heads / kv_heads, rts = (group + 15) / 16, g = blockIdx.y / rts, rt = blockIdx.y % rts;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kg = lane >> 4;
  const int total = common_of(pg, prefix), tiles = kv_heads * rts;
  if ((int)blockIdx.y == tiles) return check_common(pg, seqs, batch, total, blockIdx.x);
  const Share me = find_share(pg, seqs, batch, total, blockIdx.x, free, least);
  if (me.n == 0) return;
  const int b = me.b, slot = me.slot;
  const int len = usable_len(me.len, pg.max_pages, pg.page);
  if (tid == 0 && (slot < 0 || len != me.len)) atomicOr(pg.flags, slot < 0 ? PI_CACHE_ESLOT : PI_CACHE_ELENGTH);
  const int from = total > 0 && len >= total ? total : 0;
  const int steps = pieces(len - from, DC_K);
  const int first = share_begin(steps, me.i, me.n), last = share_begin(steps, me.i + 1, me.n);
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
  float mc = NEG_INF, l = 0.f;                     // mc: HIGH under c times the largest score so far
  const int32_t* row = pg.table + (int64_t)max(slot, 0) * pg.max_pages;
  const int64_t head_stride = (int64_t)pg.page * dim, page_stride = head_stride * kv_heads;

  for (int st = first + w; st < last; st += DC_WAVES) {
    // the two halves of 16 keys lie in one page each (pages hold multiples of 16 tokens)
    const uint16_t *kp[2], *vp[2];
    int seen[2];                                   // keys of the half that exist
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = from + st * DC_K + 16 * h;
      seen[h] = max(0, min(16, len - key));
      int id = usable_page(row[place_of(key, pg.page, pg.max_pages)], pg.pages);
      if (id < 0) {                                // a broken table: its keys are not seen
        if (seen[h] && lane == 0) atomicOr(pg.flags, PI_CACHE_EPAGE);
        seen[h] = 0;
        id = 0;
      }
      const int64_t at = id * page_stride + g * head_stride + (int64_t)(key % pg.page) * dim;
      kp[h] = pg.k + at;
      vp[h] = pg.v + at;
    }
    // all of the step's loads are on their way before the first product; keys that do not exist lie in a page all the same
    u4 kf[2][V::KS];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int ks = 0; ks < V::KS; ++ks) {
        const int ch = 4 * ks + kg;
        kf[h][ks] = *reinterpret_cast<const u4*>(kp[h] + r * dim + 8 * min(ch, nchunk - 1));
        if (ch >= nchunk) kf[h][ks] = u4{0, 0, 0, 0};
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
    f4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = (f4)(0.f);
#pragma unroll
      for (int ks = 0; ks < V::KS; ++ks) s[h] = T::mma16(kf[h][ks], qf[ks], s[h]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * kg + i >= seen[h]) s[h][i] = NEG_INF;
    }
    float mt = NEG_INF;
#pragma unroll
    for (int i = 0; i < 4; ++i) mt = fmaxf(mt, fmaxf(s[0][i], s[1][i]));
    const float top = fmaxf(mc, max16(mt) * c - T::HIGH);
    const float base = top == NEG_INF ? 0.f : top;   // rows whose scores so far are all -inf
    const float alpha = exp2_fast(mc - base);
    mc = top;
    float p[8], ls = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp2_fast(fmaf(s[i / 4][i % 4], c, -base));
      ls += p[i];
    }
    l = fmaf(l, alpha, ls);
    const u4 pf = {T::pack(p[0], p[1]), T::pack(p[2], p[3]), T::pack(p[4], p[5]), T::pack(p[6], p[7])};
    // rows that do not exist count as zeros, whatever is stored there
    if (seen[0] < 16 || seen[1] < 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (4 * kg + i % 4 >= seen[i / 4])
#pragma unroll
          for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
            for (int e = 0; e < V::W / 2; ++e) x[gr][i][e] = 0;
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
        for (int i = 0; i < 4; ++i) {
          o[f][i] *= alpha;
          o[f + 1][i] *= alpha;
        }
        o[f] = T::mma16(a, pf, o[f]);
        o[f + 1] = T::mma16(z, pf, o[f + 1]);
      }
  }
  l = sum16(l);

  // join the waves: o[f][i] belongs to dim (16 gr + 4 kg + i) W + f % W of query r
  if (lane < 16) {
    sm[w][0][r] = mc;
    sm[w][1][r] = l;
  }
#pragma unroll
  for (int gr = 0; gr < V::G; ++gr)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int f = 0; f < V::W; ++f) so[w][r][(16 * gr + 4 * kg + i) * V::W + f] = o[gr * V::W + f][i];
  __syncthreads();
  const int queries = min(16, group - 16 * rt), common = from > 0 ? common_shares(total, shares) : 0;
  const bool whole = me.n == 1 && common == 0;
  const int64_t mine = (int64_t)blockIdx.x * tiles + blockIdx.y;       // this block's place among the parts
  uint16_t* dst = out + b * out_token + (g * group + 16 * rt) * out_head;
  for (int e = 2 * tid; e < queries * dim; e += 2 * DC_WAVES * WAVE) {
    const int qr = e / dim, d = e % dim;
    float mm = NEG_INF;
#pragma unroll
    for (int i = 0; i < DC_WAVES; ++i) mm = fmaxf(mm, sm[i][0][qr]);
    const float base = mm == NEG_INF ? 0.f : mm;
    float ll = 0.f, oo = 0.f, od = 0.f;
#pragma unroll
    for (int i = 0; i < DC_WAVES; ++i) {
      const float a = exp2_fast(sm[i][0][qr] - base);
      ll = fmaf(sm[i][1][qr], a, ll);
      oo = fmaf(so[i][qr][d], a, oo);
      od = fmaf(so[i][qr][d + 1], a, od);
    }
    if (whole) {
      const float inv = ll == 0.f ? 0.f : 1.f / ll;   // a row that sees no key is zero
      *reinterpret_cast<uint32_t*>(dst + qr * out_head + d) = T::pack(oo * inv, od * inv);
    } else {
      *reinterpret_cast<float2*>(part + (16 * mine + qr) * dim + d) = float2{oo, od};
      if (d == 0) *reinterpret_cast<float2*>(stat + 2 * (16 * mine + qr)) = float2{mm, ll};
    }
  }
  // the place of the row's second share, how many there are (0: the result is written), and those of the common keys; the
  // second share's block knows, if there is one
  if (blockIdx.y == 0 && tid == 0 && me.i == (me.n > 1 ? 1 : 0)) plan[b] = int4{(int)blockIdx.x, whole ? 0 : me.n, common, 0};
}

// Join the shares of a query: one wave each, N lanes (of 4 dims each) for a share, 64 / N shares at once.
template <class T, int N>
__global__ void __launch_bounds__(256)
k_attn_join(const int4* __restrict__ plan, const float* __restrict__ cpart, const float* __restrict__ cstat,
            const float* __restrict__ part, const float* __restrict__ stat, uint16_t* __restrict__ out,
            int64_t out_token, int64_t out_head, int batch, int heads, int kv_heads, int dim, int shares) {
  constexpr int AT_ONCE = 64 / N, AHEAD = 8;       // shares a load, loads on their way
  __shared__ float weight[4][MOST + 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * 4 + w;
  if (row >= (int64_t)batch * heads) return;
  const int b = (int)(row / heads), h = (int)(row % heads), group = heads / kv_heads, rts = (group + 15) / 16;
  const int4 pl = plan[b];
  if (pl.y == 0) return;
  const int tiles = kv_heads * rts, tile = h / group * rts + h % group / 16;
  const int n = pl.y, all = n + pl.z;
  // the i-th of the row's own shares: block b's, or of those behind the rows
  auto own = [&](int i) { return ((int64_t)(i ? pl.x + i - 1 : b) * tiles + tile) * 16 + h % group % 16; };
  const int d = min(4 * (lane % N), dim - 4), mine = lane / N;
  // the first sums are on their way while the weights are made
  auto at = [&](int i) {
    i = min(i, all - 1);
    return *reinterpret_cast<const f4*>((i < n ? part + own(i) * dim : cpart + (row * shares + i - n) * dim) + d);
  };
  f4 y[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) y[i] = at(AT_ONCE * i + mine);
  constexpr int PER = (MOST + 64) / 64;
  float2 st[PER];
  float mm = NEG_INF, ll = 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = min(64 * j + lane, all - 1);
    st[j] = *reinterpret_cast<const float2*>(i < n ? stat + 2 * own(i) : cstat + 2 * (row * shares + i - n));
    mm = fmaxf(mm, st[j].x);
  }
#pragma unroll
  for (int x = 32; x; x >>= 1) mm = fmaxf(mm, __shfl_xor(mm, x));
  const float base = mm == NEG_INF ? 0.f : mm;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = 64 * j + lane;
    if (i < all) {
      const float a = exp2_fast(st[j].x - base);
      weight[w][i] = a;
      ll = fmaf(st[j].y, a, ll);
    }
  }
#pragma unroll
  for (int x = 32; x; x >>= 1) ll += __shfl_xor(ll, x);
  // a wave reads its own weights only
  __builtin_amdgcn_wave_barrier();
  f4 sum = (f4)(0.f);
  for (int i0 = 0; i0 < all; i0 += AT_ONCE * AHEAD) {
    if (i0) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) y[i] = at(i0 + AT_ONCE * i + mine);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int k = i0 + AT_ONCE * i + mine;
      if (k < all) {
        const float a = weight[w][k];
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = fmaf(y[i][j], a, sum[j]);
      }
    }
  }
#pragma unroll
  for (int x = N; x < 64; x *= 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += __shfl_xor(sum[j], x);
  const float inv = ll == 0.f ? 0.f : 1.f / ll;    // a row that sees no key is zero
  if (lane < N && 4 * lane < dim)
    *reinterpret_cast<u2*>(out + b * out_token + h * out_head + d) =
        u2{T::pack(sum[0] * inv, sum[1] * inv), T::pack(sum[2] * inv, sum[3] * inv)};
}

}  // namespace pia
