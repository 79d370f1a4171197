// Device code of the paged key/value cache for gfx950: page accounting (one
// block each, so that its result does not depend on timing) and page copies.
//
// The accounting kernels check everything they read before they write: a call
// that cannot be carried out whole sets a bit of the cache's error word and
// leaves the tables as they were.
#pragma once
#include "pi.h"
#include "pi_meta.hpp"
#include "pi_tile.hpp"

namespace pic {

using namespace pit;

constexpr int PL_T = 1024;               // threads of an accounting block
constexpr int MAX_N = 4096;              // slots one call may name

__device__ __forceinline__ int pages_of(int64_t tokens, int page) { return (int)((tokens + page - 1) / page); }

// Exclusive prefix sum over the block's threads and the total, by waves.
__device__ __forceinline__ int block_scan(int v, int& total) {
  __shared__ int part[PL_T / WAVE];
  const int w = threadIdx.x / WAVE, lane = threadIdx.x & (WAVE - 1);
  const int up = scan64(v);
  __syncthreads();
  if (lane == WAVE - 1) part[w] = up;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int i = 0; i < (int)(blockDim.x / WAVE); ++i) {
    if (i < w) before += part[i];
    total += part[i];
  }
  return before + up - v;
}

// Whether a thread's `bad` is set anywhere in the block; if so the bits go to the error word.
__device__ __forceinline__ bool refuse(int bad, int32_t* words) {
  if (bad) atomicOr(&words[1], bad);
  return __syncthreads_or(bad) != 0;
}

// slots[i] equal to an earlier one (the list lies in LDS)
__device__ __forceinline__ bool twice(const int* slots, int i) {
  const int mine = slots[i];
  bool any = false;
#pragma unroll 8
  for (int j = 0; j < i; ++j) any |= slots[j] == mine;   // to the end, so that the reads overlap
  return any;
}

// The pages that `total` pops take from the stack: in range, free, each there once, and as many as there are.  Each
// page's count becomes 1, which tells a page that comes twice; `taken` of these are the thread's, for stack_back.
__device__ __forceinline__ int stack_errors(const Meta& m, int total, int& taken) {
  const int top = m.words[0];
  taken = 0;
  if (top < 0 || top > m.pages) return PI_CACHE_EPAGE;
  if (total > top) return PI_CACHE_EFULL;
  for (int i = threadIdx.x; i < total; i += blockDim.x, ++taken) {
    const int p = m.free[top - 1 - i];
    if ((unsigned)p >= (unsigned)m.pages || atomicCAS(&m.ref[p], 0, 1) != 0) return PI_CACHE_EPAGE;
  }
  return 0;
}
__device__ __forceinline__ void stack_back(const Meta& m, int taken) {
  for (int i = 0; i < taken; ++i) m.ref[m.free[m.words[0] - 1 - (int)threadIdx.x - i * (int)blockDim.x]] = 0;
}

// Room for counts[i] more tokens in slot seqs[i]: pages from the stack, in the order of the list.
__global__ void __launch_bounds__(PL_T)
k_cache_extend(Meta m, const int32_t* __restrict__ seqs, const int32_t* __restrict__ counts, int n) {
  __shared__ int slot[MAX_N];
  for (int i = threadIdx.x; i < n; i += blockDim.x) slot[i] = seqs[i];
  __syncthreads();
  int bad = 0, carry = 0;
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int need = 0;
    if (i < n) {
      if ((unsigned)slot[i] >= (unsigned)m.slots || twice(slot, i)) {
        bad |= PI_CACHE_ESLOT;
      } else {
        const int64_t len = m.lens[slot[i]], now = len + counts[i];
        if (len < 0 || counts[i] < 0 || now > (int64_t)m.max_pages * m.page) bad |= PI_CACHE_ELENGTH;
        else need = pages_of(now, m.page) - pages_of(len, m.page);
      }
    }
    int total;
    block_scan(need, total);
    carry = min(carry + total, m.pages + 1);       // more than there are is all the same
  }
  int taken;
  bad |= stack_errors(m, carry, taken);
  if (refuse(bad, m.words)) return stack_back(m, taken);
  const int top = m.words[0];
  int at = 0;
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int need = 0, have = 0, len = 0;
    if (i < n) {
      len = m.lens[slot[i]];
      have = pages_of(len, m.page);
      need = pages_of((int64_t)len + counts[i], m.page) - have;
    }
    int total;
    const int before = at + block_scan(need, total);
    for (int j = 0; j < need; ++j) {
      const int p = m.free[top - 1 - before - j];
      m.table[(int64_t)slot[i] * m.max_pages + have + j] = p;
    }
    if (i < n) m.lens[slot[i]] = len + counts[i];
    at += total;
  }
  __syncthreads();
  if (threadIdx.x == 0) m.words[0] = top - at;
}

// The last counts tokens of each listed slot go to their pages: thread per 16 bytes of a key and a value.
__global__ void __launch_bounds__(256)
k_cache_append(Meta m, uint16_t* __restrict__ kl, uint16_t* __restrict__ vl, int kv_heads, int dim,
               const uint16_t* __restrict__ k, int64_t k_token, int64_t k_head, const uint16_t* __restrict__ v,
               int64_t v_token, int64_t v_head, const int32_t* __restrict__ cu, const int32_t* __restrict__ seqs,
               int n, int tokens) {
  const int per = kv_heads * (dim / 8);
  const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int t = (int)(e / per), head = (int)(e % per) / (dim / 8), ch = (int)(e % per) % (dim / 8);
  if (t >= tokens || t < cu[0] || t >= cu[n]) return;
  int lo = 0, up = n;                              // cu[lo] <= t < cu[up]
  while (up - lo > 1) {
    const int mid = (lo + up) / 2;
    if (cu[mid] <= t) lo = mid;
    else up = mid;
  }
  const int slot = seqs[lo];
  int bad = 0;
  if ((unsigned)slot >= (unsigned)m.slots) {
    bad = PI_CACHE_ESLOT;
  } else {
    const int64_t pos = (int64_t)m.lens[slot] - cu[lo + 1] + t;
    if (pos < 0 || pos >= (int64_t)m.max_pages * m.page) {
      bad = PI_CACHE_ELENGTH;
    } else {
      const int p = m.table[(int64_t)slot * m.max_pages + pos / m.page];
      if ((unsigned)p >= (unsigned)m.pages) {
        bad = PI_CACHE_EPAGE;
      } else {
        const int64_t at = (((int64_t)p * kv_heads + head) * m.page + pos % m.page) * dim + 8 * ch;
        *reinterpret_cast<u4*>(kl + at) = *reinterpret_cast<const u4*>(k + t * k_token + head * k_head + 8 * ch);
        *reinterpret_cast<u4*>(vl + at) = *reinterpret_cast<const u4*>(v + t * v_token + head * v_head + 8 * ch);
      }
    }
  }
  if (bad) atomicOr(&m.words[1], bad);
}

// The pages a call copies: count, then the sources and the targets, each `cap` long.
struct Plan {
  int32_t *count, *src, *dst;
};

// children[i] becomes a copy of parents[i]: it shares the whole pages and gets a page of its own for a
// last page that is not full, whose copy the plan asks for.  Parents are read as they were before the call.
// The pages of all children are dealt to all threads, several a thread at once: what takes time here is one
// read after another.  (24 children of 3001 tokens: 14.6 us with a wave a child and an addition a page and child, 11.6 us so.)
__global__ void __launch_bounds__(PL_T)
k_cache_fork(Meta m, const int32_t* __restrict__ parents, const int32_t* __restrict__ children, int n, Plan plan) {
  __shared__ int kid[MAX_N], dad[MAX_N], len_of[MAX_N], most;
  __shared__ short alike[MAX_N];                   // children of the same parent, at the first of them; else 0
  constexpr int U = 4;                             // table entries of a thread at once
  const int top = m.words[0];
  for (int i = threadIdx.x; i < n; i += blockDim.x) kid[i] = children[i], dad[i] = parents[i];
  if (threadIdx.x == 0) *plan.count = 0, most = 0;
  __syncthreads();
  int bad = 0, all = 0, long_ = 0;
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int part = 0;
    if (i < n) {
      const int p = dad[i], k = kid[i];
      const bool there = (unsigned)k < (unsigned)m.slots && (unsigned)p < (unsigned)m.slots;
      const int len = there ? m.lens[p] : 0, old = there ? m.lens[k] : 0;
      const bool fits = len >= 0 && len <= (int64_t)m.max_pages * m.page;
      if (!there || old != 0 || twice(kid, i)) bad |= PI_CACHE_ESLOT;
      else if (!fits) bad |= PI_CACHE_ELENGTH;
      len_of[i] = there && fits ? len : 0;
      int same = 0;
      bool first = true;
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const bool s = dad[j] == p;
        same += s;
        first &= !s || j >= i;
      }
      alike[i] = first ? same : 0;
      part = len_of[i] % m.page != 0;
      long_ = max(long_, pages_of(len_of[i], m.page));
    }
    int total;
    block_scan(part, total);
    all += total;
  }
  for (int d = 32; d; d >>= 1) long_ = max(long_, __shfl_xor(long_, d));
  if (threadIdx.x % WAVE == 0 && long_) atomicMax(&most, long_);
  __syncthreads();
  // entry e of all: page e % most of child e / most
  const int64_t entries = (int64_t)n * most;
  struct Entry {
    int i, j;
    bool is;
  };
  auto entry = [&](int64_t e) {
    Entry x{0, 0, e < entries};
    if (x.is) {
      x.i = entries <= INT32_MAX ? (int)e / most : (int)(e / most);
      x.j = (int)(e - (int64_t)x.i * most);
      x.is = x.j < pages_of(len_of[x.i], m.page);
    }
    return x;
  };
  for (int64_t base = threadIdx.x; base < entries; base += U * PL_T) {
    int page[U], ref[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Entry x = entry(base + u * PL_T);
      page[u] = x.is && alike[x.i] ? m.table[(int64_t)dad[x.i] * m.max_pages + x.j] : -2;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) ref[u] = (unsigned)page[u] < (unsigned)m.pages ? m.ref[page[u]] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (page[u] != -2 && ref[u] <= 0) bad |= PI_CACHE_EPAGE;
  }
  // a free page in a parent's table has been seen by now; from here on its count may be 1
  __syncthreads();
  int taken;
  bad |= stack_errors(m, all, taken);
  if (refuse(bad, m.words)) return stack_back(m, taken);
  int at = 0;
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + threadIdx.x;
    const int part = i < n && len_of[i] % m.page != 0;
    int total;
    const int before = at + block_scan(part, total);
    if (part) {
      const int whole = len_of[i] / m.page, p = m.free[top - 1 - before];
      plan.src[before] = m.table[(int64_t)dad[i] * m.max_pages + whole];
      plan.dst[before] = p;
      m.table[(int64_t)kid[i] * m.max_pages + whole] = p;
    }
    if (i < n) m.lens[kid[i]] = len_of[i];
    at += total;
  }
  for (int64_t base = threadIdx.x; base < entries; base += U * PL_T) {
    Entry x[U];
    int page[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = entry(base + u * PL_T);
      x[u].is = x[u].is && x[u].j < len_of[x[u].i] / m.page;   // whole pages
      page[u] = x[u].is ? m.table[(int64_t)dad[x[u].i] * m.max_pages + x[u].j] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (x[u].is) {
        m.table[(int64_t)kid[x[u].i] * m.max_pages + x[u].j] = page[u];
        if (alike[x[u].i]) atomicAdd(&m.ref[page[u]], alike[x[u].i]);
      }
  }
  if (threadIdx.x == 0) {
    m.words[0] = top - at;
    *plan.count = at;
  }
}

// After a compaction: the tables, and where each page went.  Entry e of slots max_pages, or page e.
__device__ __forceinline__ void remap(const Meta& m, const int32_t* to, int32_t* moved, int64_t e) {
  if (moved && e < m.pages) moved[e] = to[e];
  if (e >= (int64_t)m.slots * m.max_pages) return;
  const int slot = (int)(e / m.max_pages), place = (int)(e % m.max_pages);
  if ((int64_t)place * m.page >= m.lens[slot]) return;
  const int p = m.table[e];
  const int now = (unsigned)p < (unsigned)m.pages ? to[p] : -1;
  if (now < 0) atomicOr(&m.words[1], PI_CACHE_EPAGE);
  else m.table[e] = now;
}

// Whole pages from src to dst, in every layer of both pools: blockIdx.y is layer * 2 + pool.  Behind the last layer,
// blocks that follow a compaction's map (`to`).
__global__ void __launch_bounds__(256)
k_cache_copy(u4* __restrict__ k, u4* __restrict__ v, int64_t layer_chunks, int page_chunks, int layers, Plan plan, Meta m,
             const int32_t* __restrict__ to, int32_t* __restrict__ moved) {
  if ((int)blockIdx.y == 2 * layers) {
    const int64_t entries = max((int64_t)m.slots * m.max_pages, (int64_t)m.pages);
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < entries; e += (int64_t)gridDim.x * blockDim.x)
      remap(m, to, moved, e);
    return;
  }
  u4* pool = ((blockIdx.y & 1) ? v : k) + (int64_t)(blockIdx.y >> 1) * layer_chunks;
  const int count = *plan.count;
  for (int i = blockIdx.x; i < count; i += gridDim.x) {
    const u4* from = pool + (int64_t)plan.src[i] * page_chunks;
    u4* into = pool + (int64_t)plan.dst[i] * page_chunks;
    for (int e = threadIdx.x; e < page_chunks; e += blockDim.x) into[e] = from[e];
  }
}

// A count of uses, read past the first-level cache (other waves of the block changed it by atomics).
__device__ __forceinline__ int uses(const int32_t* ref) {
  return __hip_atomic_load(ref, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The listed slots become empty; pages that no slot uses any more go to the stack, the lowest on top.
// First every listed use is taken off its page's count; a page that is held more often than counted shows as a count that
// was not positive, and then all of them are put back and the call is refused.  Pages left without a use are marked by a
// count of GONE, which one thread for each sets and counts, so neither the marks nor their number depend on timing, and
// the pool is searched for the marks in the stack's order.  (One slot of 3001 tokens: 11.6 us, 32 of them 25.1 us; without
// the check of the counts 10.8 and 23.2 us.)
__global__ void __launch_bounds__(PL_T) k_cache_release(Meta m, const int32_t* __restrict__ seqs, int n) {
  constexpr int GONE = INT32_MIN;
  __shared__ int slot[MAX_N];
  for (int i = threadIdx.x; i < n; i += blockDim.x) slot[i] = seqs[i];
  __syncthreads();
  int bad = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    if ((unsigned)slot[i] >= (unsigned)m.slots || twice(slot, i)) bad |= PI_CACHE_ESLOT;
    else if (m.lens[slot[i]] < 0 || m.lens[slot[i]] > (int64_t)m.max_pages * m.page) bad |= PI_CACHE_ELENGTH;
  }
  const int top = m.words[0];
  if (top < 0 || top > m.pages) bad |= PI_CACHE_EPAGE;
  if (refuse(bad, m.words)) return;
  const int w = threadIdx.x / WAVE, lane = threadIdx.x & (WAVE - 1), waves = blockDim.x / WAVE;
  // f(page) for every place of every listed slot, in no order; several waves share a slot where there are few
  const int parts = n < waves ? waves / n : 1, part = n < waves ? w / n : 0;
  auto each = [&](auto f) {
    for (int i = n < waves ? w % n : w; i < n && part < parts; i += waves) {
      const int32_t* row = m.table + (int64_t)slot[i] * m.max_pages;
      const int held = pages_of(m.lens[slot[i]], m.page);
      for (int j = part * WAVE + lane; j < held; j += parts * WAVE) f(row[j]);
    }
  };
  each([&](int p) {
    if ((unsigned)p >= (unsigned)m.pages) bad |= PI_CACHE_EPAGE;
  });
  if (refuse(bad, m.words)) return;
  each([&](int p) {
    if (atomicSub(&m.ref[p], 1) <= 0) bad |= PI_CACHE_EPAGE;
  });
  bool back = refuse(bad, m.words);
  int gone = 0, total = 0;
  if (!back) {
    each([&](int p) { gone += atomicCAS(&m.ref[p], 0, GONE) == 0; });
    block_scan(gone, total);
    // more pages than there are places: the stack held one of them already
    back = refuse(total > m.pages - top ? PI_CACHE_EPAGE : 0, m.words);
    if (back) {
      each([&](int p) { atomicCAS(&m.ref[p], GONE, 0); });
      __syncthreads();
    }
  }
  if (back) {
    each([&](int p) { atomicAdd(&m.ref[p], 1); });
    return;
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) m.lens[slot[i]] = 0;
  int at = top;
  for (int base = 0; base < m.pages; base += blockDim.x) {
    const int p = m.pages - 1 - (base + (int)threadIdx.x);
    const int mine = p >= 0 && uses(&m.ref[p]) == GONE;
    int here;
    const int pos = at + block_scan(mine, here);
    if (mine) {
      m.ref[p] = 0;
      if (pos < m.pages) m.free[pos] = p;
    }
    at += here;
  }
  if (threadIdx.x == 0) m.words[0] = top + total;
}

// The pages in use move to the front of the pool: the i-th page in use at or behind place `used` goes to the
// i-th unused place before it.  to[p] is where page p went (itself if it did not move), -1 if it was not in use.
__global__ void __launch_bounds__(PL_T) k_cache_compact(Meta m, Plan plan, int32_t* __restrict__ to) {
  int used = 0;
  for (int base = 0; base < m.pages; base += blockDim.x) {
    const int p = base + threadIdx.x;
    int total;
    block_scan(p < m.pages && m.ref[p] > 0, total);
    used += total;
  }
  int holes = 0, movers = 0;
  for (int base = 0; base < m.pages; base += blockDim.x) {
    const int p = base + threadIdx.x;
    const bool in = p < m.pages, live = in && m.ref[p] > 0;
    int total;
    const int h = in && !live && p < used, mv = live && p >= used;
    // a place is a hole or a mover, not both: one scan holds both counts (pages < 2^20, 1024 a round)
    const int at = block_scan(h + (mv << 16), total);
    if (h) plan.dst[holes + (at & 0xffff)] = p;
    if (mv) plan.src[movers + (at >> 16)] = p;
    if (in) to[p] = live ? p : -1;
    holes += total & 0xffff;
    movers += total >> 16;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += blockDim.x) {
    to[plan.src[i]] = plan.dst[i];
    m.ref[plan.dst[i]] = m.ref[plan.src[i]];
  }
  __syncthreads();
  for (int p = used + threadIdx.x; p < m.pages; p += blockDim.x) {
    m.ref[p] = 0;
    m.free[m.pages - 1 - p] = p;                   // the lowest on top
  }
  if (threadIdx.x == 0) {
    m.words[0] = m.pages - used;
    m.words[2] = used;
    *plan.count = movers;
  }
}

}  // namespace pic
