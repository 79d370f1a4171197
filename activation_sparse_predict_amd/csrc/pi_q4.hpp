// Device code of the products with Q4_0 matrices for gfx950.
//
//   y_b = (W x_b) + bias,  W[n][32 j + e] = scale[n][j] (q - 8),  q in [0, 15]
//
// A 16x16x32 matrix instruction takes one 32-weight block of 16 rows.  Its
// weights are q - 8 in binary16 (exact), and the block's product is multiplied
// by the block's scale in float32, so no weight is rounded.  Rows of x in
// binary16 go in as they are.  Others go in as binary16 after multiplication by
// a power of two that puts the row's largest finite value into [2^14, 2^15):
// one column for bfloat16 rows (their significands fit), two for float32 rows,
// the rounded value and 2^11 times what it leaves, which together are x within
// 2^-23 relative.  Below 2^-14 binary16 rounds to multiples of 2^-24: with L the
// row's largest value, float32 values lose bits from 2^-27 L down and are off by
// at most 2^-50 L, bfloat16 values from 2^-32 L down and by at most 2^-39 L.
// Beside the rounding of a float32 sum with L in it, that shows only where L's
// weight is 0 or far smaller than the others.
//
// The least that the products cost is the read of the matrix, 18 bytes for 32
// weights; unpacking them takes about 13 vector instructions for 288 bytes, a
// quarter of that time.
#pragma once
#include "pi.h"
#include "pi_tile.hpp"

namespace piq {

using namespace pit;

constexpr int MV_ROWS = 16;              // matrix rows of a tile
constexpr int MV_G = 8;                  // 32-blocks of a group: 128 bytes of a row's nibbles, one cache line
constexpr int MV_WAVES = 8;              // waves of a block
constexpr int MV_AHEAD = 2;              // groups of a wave on their way

// Four elements from i on, whatever their alignment.
struct __attribute__((packed, aligned(4))) Four32 {
  float v[4];
};
struct __attribute__((packed, aligned(2))) Four16 {
  uint16_t v[4];
};
template <int X> __device__ __forceinline__ f4 x_four(const void* p, int64_t i) {
  f4 r;
  if constexpr (X == PI_F32) {
    const Four32 a = *reinterpret_cast<const Four32*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = a.v[j];
  } else {
    const Four16 a = *reinterpret_cast<const Four16*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (X == PI_F16) r[j] = (float)__builtin_bit_cast(_Float16, a.v[j]);
      else r[j] = __uint_as_float((uint32_t)a.v[j] << 16);
    }
  }
  return r;
}
template <int Y> __device__ __forceinline__ void y_to(void* p, int64_t i, float v) {
  if constexpr (Y == PI_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (Y == PI_F16) static_cast<_Float16*>(p)[i] = (_Float16)v;
  else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

// Columns an x row takes.
template <int X> constexpr int parts() { return X == PI_F32 ? 2 : 1; }

// Column c of the x operand is row m of its 16: neighbours go to different lane groups of D.
__host__ __device__ constexpr int col_row(int c) { return 4 * (c % 4) + c / 4; }

// The 8 weights of a 4-byte word as binary16 q - 8: 0x6400 | q is 1024 + q, and
// 0x6400 | 16 q is 1024 + 16 q.
__device__ __forceinline__ u4 q4_unpack(uint32_t w) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  const h2 one = {(_Float16)-1032.f, (_Float16)-1032.f};
  const h2 six = {(_Float16)0.0625f, (_Float16)0.0625f}, off = {(_Float16)-72.f, (_Float16)-72.f};
  const uint32_t v = w >> 8;
  u4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, (w & 0x000f000fu) | 0x64006400u) + one);
  r[1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2, (w & 0x00f000f0u) | 0x64006400u), six, off));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, (v & 0x000f000fu) | 0x64006400u) + one);
  r[3] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2, (v & 0x00f000f0u) | 0x64006400u), six, off));
  return r;
}

// The power of two that brings a row with largest finite value `big` into [2^14, 2^15): 1 for zero.
__device__ __forceinline__ float row_scale(float big) {
  const int e = (int)(__float_as_uint(big) >> 23) & 255;
  if (big == 0.f) return 1.f;
  return __uint_as_float((uint32_t)min(max(127 + 14 - (e - 127), 1), 254) << 23);
}

// The largest finite |x| of a row, by all threads of a block (NT of them; part: LDS, NT / 64 floats).
template <int X, int NT>
__device__ __forceinline__ float row_max(const void* x, int64_t at, int cols, float* part) {
  const int tid = threadIdx.x;
  float big = 0.f;
#pragma unroll 8
  for (int k = 4 * tid; k < cols; k += 4 * NT) {
    const f4 v = x_four<X>(x, at + k);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (fabsf(v[j]) < __builtin_inff()) big = fmaxf(big, fabsf(v[j]));   // others are what they are at any scale
  }
  for (int d = 32; d; d >>= 1) big = fmaxf(big, __shfl_xor(big, d));
  __syncthreads();
  if ((tid & 63) == 0) part[tid >> 6] = big;
  __syncthreads();
  big = part[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) big = fmaxf(big, part[i]);
  return big;
}

// The operand's columns of a value: binary16 bits of part p of it.
__device__ __forceinline__ uint32_t x_part(float v, int p) {
  const _Float16 h = (_Float16)v;
  if (p == 0) return __builtin_bit_cast(uint16_t, h);
  // an infinite or NaN value leaves nothing
  const float rest = fabsf(v) <= 65504.f ? (v - (float)h) * 2048.f : 0.f;
  return __builtin_bit_cast(uint16_t, (_Float16)rest);
}

// A block's elements in the operand stand in the order in which q4_unpack gives the weights of word kg: 4 kg + 0, 2,
// 16, 18, 1, 3, 17, 19.  So of elements 4 a .. 4 a + 3, a < 8, the first and third lie in word word_of(a) of the block's
// 16 and the other two in word word_of(a) + 2.
__device__ __forceinline__ int word_of(int a) { return 4 * (a & 3) + (a >> 2); }

// x -> operand [block][column tile][lane][8] and, per row, 1 / scale.  Block (b, i): a share of x row b's blocks.
// Rows from `batch` on are the columns that fill up the last tile.
template <int X>
__global__ void __launch_bounds__(256)
k_mv_operand(const void* __restrict__ x, int64_t ldx, int batch, int cols, int tiles, uint16_t* __restrict__ xo,
             float* __restrict__ inv) {
  __shared__ float part[4];
  const int b = blockIdx.x, tid = threadIdx.x;
  constexpr int P = parts<X>();
  float s = 1.f;
  if (b < batch) {
    if constexpr (X != PI_F16) s = row_scale(row_max<X, 256>(x, b * ldx, cols, part));
    if (tid == 0 && blockIdx.y == 0) inv[b] = 1.f / s;
  }
  for (int e = 4 * (blockIdx.y * 256 + tid); e < cols; e += 4 * 256 * gridDim.y) {
    f4 v = (f4)(0.f);
    if (b < batch) v = x_four<X>(x, b * ldx + e) * s;
    const int kb = e / 32, wd = word_of(e / 4 % 8);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = P * b + p;
      if (c >= 16 * tiles) break;
      uint32_t* to = reinterpret_cast<uint32_t*>(xo) +
                     ((int64_t)(kb * tiles + c / 16) * 64 + 16 * (wd / 4) + col_row(c % 16)) * 4 + wd % 4;
      to[0] = x_part(v[0], p) | x_part(v[2], p) << 16;
      to[2] = x_part(v[1], p) | x_part(v[3], p) << 16;
    }
  }
}

// A lane's share of 8 blocks of one row tile: lane (r, kg) holds blocks 2 kg and 2 kg + 1 of the eight of row r, and
// the scales of all of them.
struct Group {
  u4 q[2], s;
};

// Scales lie on 2 bytes; they are read 16 bytes at once all the same, which global memory allows.
struct __attribute__((packed, aligned(2))) Scales {
  u4 v;
};

// The blocks of group g: 8 g .., but where the row ends inside them the row's last 8, of which the first belong to the
// group before.  So every load is whole and none hangs on a condition, behind which the compiler would wait for all
// loads at once.  TINY: rows of fewer than 8 blocks, read block by block.
__device__ __forceinline__ int group_start(int g, int blocks) { return min(MV_G * g, max(blocks - MV_G, 0)); }

template <bool TINY>
__device__ __forceinline__ Group load_group(const uint8_t* q, const uint16_t* s, int start, int kg, int blocks) {
  Group g;
  if constexpr (!TINY) {
    q += 16 * start + 32 * kg;
    g.q[0] = *reinterpret_cast<const u4*>(q);
    g.q[1] = *reinterpret_cast<const u4*>(q + 16);
    g.s = reinterpret_cast<const Scales*>(s + start)->v;
  } else {
    g.q[0] = *reinterpret_cast<const u4*>(q + 16 * min(2 * kg, blocks - 1));
    g.q[1] = *reinterpret_cast<const u4*>(q + 16 * min(2 * kg + 1, blocks - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) g.s[i] = s[min(2 * i, blocks - 1)] | (uint32_t)s[min(2 * i + 1, blocks - 1)] << 16;
  }
  return g;
}

// f(j) for the blocks of group g, block j of the eight read: all, without branches, so that they overlap, or those that
// are the group's own.
template <class F> __device__ __forceinline__ void each_block(int g, int start, int blocks, F f) {
  if (start == MV_G * g && blocks >= start + MV_G) {
#pragma unroll
    for (int j = 0; j < MV_G; ++j) f(j);
  } else {
#pragma unroll
    for (int j = 0; j < MV_G; ++j)
      if (start + j >= MV_G * g && start + j < blocks) f(j);
  }
}

// Word kg of each of four blocks, from the lanes that hold the blocks whole: block i comes to w[i].
__device__ __forceinline__ void spread(u4 c, uint32_t* w) {
  const auto a = __builtin_amdgcn_permlane16_swap(c[0], c[1], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(c[2], c[3], false, false);
  const auto e = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto o = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  w[0] = e[0], w[1] = o[0], w[2] = e[1], w[3] = o[1];
}

__device__ __forceinline__ float scale_at(u4 s, int i) {
  const uint32_t w = s[i / 2];
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
}

// Products of few columns (parts<X>() * batch = PB <= 16): every block makes the
// operand for itself, in LDS, while its first weights are on their way, and then
// takes row tiles in turn.  The waves take groups of 8 blocks in turn and join
// their sums through LDS.  Columns go to operand rows such that D registers
// 0 .. MA - 1 hold them (col_row).
//
// 36864 x 12288, one float32 row: 59 us, 4.3 TB/s; 74 us with 4 waves a block,
// 61 and 62 us with 3 and 4 groups ahead, 77 us with a branch at each block of
// a whole group.  4096 x 4096: 6.4 us a call.
template <int X, int Y, int MA, bool TINY>
__global__ void __launch_bounds__(MV_WAVES * WAVE)
k_matvec_few(const uint8_t* __restrict__ q, const uint16_t* __restrict__ scale, const float* __restrict__ bias,
             int rows, int cols, const void* __restrict__ x, int64_t ldx, int batch, void* __restrict__ y,
             int64_t ldy) {
  constexpr int P = parts<X>(), W = MV_WAVES, NT = W * WAVE;
  extern __shared__ __attribute__((aligned(16))) char lds[];   // the operand [block][column][32]
  constexpr int RB = MA < 4 ? 2 : 1;               // a second buffer for the sums, while the operand leaves room for it
  __shared__ float red[RB][W][4 * MA][MV_ROWS + 1], part[W], inv[16];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
            kg = lane >> 4;
  const int blocks = cols / 32, groups = (blocks + MV_G - 1) / MV_G, PB = P * batch;
  const int tiles = (rows + MV_ROWS - 1) / MV_ROWS;
  // this block's tiles, and this wave's groups of each: w, w + W, ..
  const int t0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x), t1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  Group buf[MV_AHEAD];                             // groups on their way
  int ta = t0, ga = min(w, groups - 1);            // the next one to load; behind the last one, that one again
  auto ahead = [&](Group& to) {
    const int row = min(min(ta, t1 - 1) * MV_ROWS + r, rows - 1);
    to = load_group<TINY>(q + (int64_t)row * (cols / 2), scale + (int64_t)row * blocks, group_start(ga, blocks), kg, blocks);
    ga += W;
    if (ga >= groups) ga = min(w, groups - 1), ++ta;
  };
#pragma unroll
  for (int i = 0; i < MV_AHEAD; ++i) ahead(buf[i]);

  uint32_t* xo = reinterpret_cast<uint32_t*>(lds);
  for (int b = 0; b < batch; ++b) {
    float s = 1.f;
    if constexpr (X != PI_F16) s = row_scale(row_max<X, NT>(x, b * ldx, cols, part));
    if (tid == 0) inv[b] = 1.f / s;
#pragma unroll 4
    for (int e = 4 * tid; e < cols; e += 4 * NT) {
      const f4 v = x_four<X>(x, b * ldx + e) * s;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        uint32_t* to = xo + (e / 32 * PB + P * b + p) * 16 + word_of(e / 4 % 8);
        to[0] = x_part(v[0], p) | x_part(v[2], p) << 16;
        to[2] = x_part(v[1], p) | x_part(v[3], p) << 16;
      }
    }
  }
  __syncthreads();
  // the operand row's column; rows beyond hold copies
  const char* xl = lds + 64 * (col_row(r) % PB) + 16 * kg;

  f4 acc = (f4)(0.f);
  auto add = [&](const Group& now, int g) {
    uint32_t wd[2][4];
    spread(now.q[0], wd[0]);
    spread(now.q[1], wd[1]);
    const int start = group_start(g, blocks);
    const char* at = xl + 64 * PB * start;
    each_block(g, start, blocks, [&](int j) {
      const u4 xf = *reinterpret_cast<const u4*>(at + 64 * PB * j);
      const f4 d = H16::mma16(xf, q4_unpack(wd[j & 1][j >> 1]), (f4)(0.f));
      const float sf = scale_at(now.s, j);
#pragma unroll
      for (int m = 0; m < MA; ++m) acc[m] = fmaf(sf, d[m], acc[m]);
    });
  };
  auto join = [&](int t) {                         // the waves' sums of tile t
    auto& rd = red[t % RB];
#pragma unroll
    for (int m = 0; m < MA; ++m) rd[w][4 * m + kg][r] = acc[m];   // operand row 4 kg + m is column 4 m + kg
    acc = (f4)(0.f);
    __syncthreads();
    for (int e = tid; e < batch * MV_ROWS; e += NT) {
      const int b = e / MV_ROWS, row = t * MV_ROWS + e % MV_ROWS;
      if (row >= rows) continue;
      float v = 0.f, z = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v += rd[i][P * b][e % MV_ROWS];
        if constexpr (P == 2) z += rd[i][P * b + 1][e % MV_ROWS];
      }
      if constexpr (P == 2) v = fmaf(z, 1.f / 2048.f, v);
      v *= inv[b];
      if (bias) v += bias[row];
      y_to<Y>(y, b * ldy + row, v);
    }
    if (RB == 1) __syncthreads();
  };
  int t = t0, g = w;
  if (w >= groups) {                               // a wave without groups only joins
    for (; t < t1; ++t) join(t);
    return;
  }
  while (t < t1) {
#pragma unroll
    for (int i = 0; i < MV_AHEAD; ++i) {
      if (t >= t1) break;
      const Group now = buf[i];
      ahead(buf[i]);
      add(now, g);
      g += W;
      if (g >= groups) join(t++), g = w;
    }
  }
}

// Products of many columns: one block takes 128 rows, 16 a wave, and one share
// of the groups, whose operand all its waves read from LDS.  Of a group's
// operand each wave brings MT KB, two groups ahead: loaded while one group is
// computed, written to LDS while the next one is.  part: [share][column][row].
//
// What bounds it is the wait for its loads: with 9216 x 8192 and 32 bfloat16 rows
// vector instructions are issued in 30 % of the cycles and matrix instructions
// run in 8 %, while waves wait for 41 % of their time.  Loads come in order, so
// the wait for the next group's operand, which was asked for after the weights of
// the one behind it, is a wait for those too: of two groups of weights one is on
// its way.  25 us a call (in 8 shares 28 us, and with three groups ahead 31 us
// then).  36864 x 12288: 91 us (115 us with 16 rows a block, whose operand came
// from the second-level cache for each).
template <int MT, bool TINY>
__global__ void __launch_bounds__(MV_WAVES * WAVE, 2)
k_matvec(const uint8_t* __restrict__ q, const uint16_t* __restrict__ scale, int rows, int cols,
         const uint16_t* __restrict__ xo, int columns, float* __restrict__ part) {
  __shared__ u4 xs[2][MV_G * MT * WAVE];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
            kg = lane >> 4;
  const int row0 = (blockIdx.x * MV_WAVES + w) * MV_ROWS, row = min(row0 + r, rows - 1);
  const int blocks = cols / 32, groups = (blocks + MV_G - 1) / MV_G;
  const int g0 = (int)((int64_t)groups * blockIdx.y / gridDim.y), g1 = (int)((int64_t)groups * (blockIdx.y + 1) / gridDim.y);
  const uint8_t* qr = q + (int64_t)row * (cols / 2);
  const uint16_t* sr = scale + (int64_t)row * blocks;
  const u4* xl = reinterpret_cast<const u4*>(xo);
  Group buf[MV_AHEAD];
  u4 xr[MT];
  // behind the share's last group, that one again
  auto weights = [&](Group& to, int g) {
    to = load_group<TINY>(qr, sr, group_start(min(g, g1 - 1), blocks), kg, blocks);
  };
  auto operand = [&](int g) {                      // the operand is there for whole groups
    const u4* from = xl + (int64_t)MV_G * MT * WAVE * min(g, g1 - 1) + MT * w * WAVE + lane;
#pragma unroll
    for (int i = 0; i < MT; ++i) xr[i] = from[i * WAVE];
  };
  auto stage = [&](int g) {
#pragma unroll
    for (int i = 0; i < MT; ++i) xs[g & 1][(MT * w + i) * WAVE + lane] = xr[i];
  };
  operand(g0);
#pragma unroll
  for (int i = 0; i < MV_AHEAD; ++i) weights(buf[i], g0 + i);
  stage(g0);
  operand(g0 + 1);
  f4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = (f4)(0.f);
  for (int base = g0; base < g1; base += MV_AHEAD) {
#pragma unroll
    for (int i = 0; i < MV_AHEAD; ++i) {
      const int g = base + i;
      if (g >= g1) break;
      // this group's operand is written, and the one before it has been read; loads stay on their way
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      const Group now = buf[i];
      weights(buf[i], g + MV_AHEAD);
      stage(g + 1);
      operand(g + 2);
      uint32_t wd[2][4];
      spread(now.q[0], wd[0]);
      spread(now.q[1], wd[1]);
      const int start = group_start(g, blocks);
      const u4* at = xs[g & 1] + lane + (start - MV_G * g) * MT * WAVE;
      each_block(g, start, blocks, [&](int j) {
        const u4 wf = q4_unpack(wd[j & 1][j >> 1]);
        const float sf = scale_at(now.s, j);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const f4 d = H16::mma16(at[(j * MT + t) * WAVE], wf, (f4)(0.f));
#pragma unroll
          for (int m = 0; m < 4; ++m) acc[t][m] = fmaf(sf, d[m], acc[t][m]);
        }
      });
    }
  }
  if (row0 + r >= rows) return;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int m = 0; m < 4; ++m) {                  // operand row 4 kg + m is column 4 m + kg
      const int c = 16 * t + 4 * m + kg;
      if (c < columns) part[((int64_t)blockIdx.y * columns + c) * rows + row0 + r] = acc[t][m];
    }
}

// The shares' sums, scaled back: one thread per output.
template <int P, int Y>
__global__ void __launch_bounds__(256)
k_matvec_join(const float* __restrict__ part, const float* __restrict__ inv, const float* __restrict__ bias, int rows,
              int shares, int batch, void* __restrict__ y, int64_t ldy) {
  const int row = blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
  if (row >= rows) return;
  const int64_t step = (int64_t)P * batch * rows;
  const float* at = part + (int64_t)P * b * rows + row;
  float v = 0.f, z = 0.f;
#pragma unroll 8
  for (int i = 0; i < shares; ++i) {
    v += at[i * step];
    if constexpr (P == 2) z += at[i * step + rows];
  }
  if constexpr (P == 2) v = fmaf(z, 1.f / 2048.f, v);
  v *= inv[b];
  if (bias) v += bias[row];
  y_to<Y>(y, b * ldy + row, v);
}

}  // namespace piq
