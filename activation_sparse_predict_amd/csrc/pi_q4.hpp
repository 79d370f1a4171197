// Device code of the products with Q4_0 matrices for gfx950.
//
//   y_b = (W x_b) + bias,  W[n][32 j + e] = scale[n][j] (q - 8),  q in [0, 15]
//
// A 16x16x32 matrix instruction takes one 32-weight block of 16 rows.  Its
// weights are q - 8 in binary16 (exact), and the block's product is multiplied
// by the block's scale in float32, so no weight is rounded.  x goes in as
// binary16 after multiplication by a power of two that puts its row's largest
// value into [2^14, 2^15): one column for binary16 and bfloat16 rows (their
// significands fit), two for float32 rows, the rounded value and 2^11 times
// what it leaves, which together are x within 2^-24 relative, half a step of
// float32.  Values below 2^-39 of their row's largest lose bits to binary16's
// range; they are under 2^-24 of any sum they could show in by then.
#pragma once
#include "pi.h"
#include "pi_tile.hpp"

namespace piq {

using namespace pit;

constexpr int MV_ROWS = 16;              // matrix rows of a block's tile
constexpr int MV_WAVES = 4;

// Load one element of x, stored as dtype X (pi_dtype), as float32.
template <int X> __device__ __forceinline__ float x_at(const void* p, int64_t i) {
  if constexpr (X == PI_F32) return static_cast<const float*>(p)[i];
  else if constexpr (X == PI_F16) return (float)static_cast<const _Float16*>(p)[i];
  else return (float)static_cast<const __bf16*>(p)[i];
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

// Element e of lane group kg inside a 32-block: the order in which the nibbles of
// word kg of the block come out of q4_unpack.
__device__ __forceinline__ int slot_k(int kg, int e) { return 4 * kg + 2 * (e & 1) + (e >> 2) + 16 * ((e >> 1) & 1); }

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

// x -> operand [block][column tile][lane][8] and, per row, 1 / scale.  One block per column pair row.
template <int X>
__global__ void __launch_bounds__(256)
k_mv_operand(const void* __restrict__ x, int64_t ldx, int batch, int cols, int tiles, uint16_t* __restrict__ xo,
             float* __restrict__ inv) {
  __shared__ float part[4];
  const int b = blockIdx.x, tid = threadIdx.x;
  constexpr int P = parts<X>();
  float s = 1.f;
  if (b < batch) {
    float big = 0.f;
    for (int k = tid; k < cols; k += 256) {
      const float v = fabsf(x_at<X>(x, b * ldx + k));
      if (v < __builtin_inff()) big = fmaxf(big, v);   // infinities and NaN are what they are at any scale
    }
    for (int d = 32; d; d >>= 1) big = fmaxf(big, __shfl_xor(big, d));
    if ((tid & 63) == 0) part[tid >> 6] = big;
    __syncthreads();
    s = row_scale(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
    if (tid == 0) inv[b] = 1.f / s;
  }
  for (int e = tid; e < cols; e += 256) {          // operand elements of this row's columns
    const int kb = e / 32, kg = (e / 8) % 4, i = e % 8;
    const float v = b < batch ? x_at<X>(x, b * ldx + 32 * kb + slot_k(kg, i)) * s : 0.f;
    const _Float16 h = (_Float16)v;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = P * b + p;
      if (c >= 16 * tiles) break;
      // an infinite or NaN value leaves nothing
      const float rest = fabsf(v) <= 65504.f ? (v - (float)h) * 2048.f : 0.f;
      const _Float16 y = p ? (_Float16)rest : h;
      const int lane = 16 * kg + col_row(c % 16);
      xo[((int64_t)(kb * tiles + c / 16) * 64 + lane) * 8 + i] = __builtin_bit_cast(uint16_t, y);
    }
  }
}

// One block: 16 matrix rows, the waves taking groups of four 32-blocks in turn.
// Lane (r, kg) loads block 4 j + kg of row r whole; 4 swaps of lane groups
// leave it word kg of each of the four blocks.
template <int X, int Y, int MT>
__global__ void __launch_bounds__(MV_WAVES * WAVE)
k_matvec(const uint8_t* __restrict__ q, const uint16_t* __restrict__ scale, const float* __restrict__ bias, int rows,
         int cols, const uint16_t* __restrict__ xo, const float* __restrict__ inv, int batch, void* __restrict__ y,
         int64_t ldy) {
  constexpr int P = parts<X>();
  __shared__ float red[MV_WAVES][MT * 16][MV_ROWS + 1];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r = lane & 15, kg = lane >> 4;
  const int row0 = blockIdx.x * MV_ROWS, row = min(row0 + r, rows - 1), blocks = cols / 32;
  const uint8_t* qr = q + (int64_t)row * (cols / 2);
  const uint16_t* sr = scale + (int64_t)row * blocks;
  const u4* xl = reinterpret_cast<const u4*>(xo) + lane;
  f4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = (f4)(0.f);
  for (int j = 4 * w; j < blocks; j += 4 * MV_WAVES) {
    const int mine = min(j + kg, blocks - 1);
    const u4 c = *reinterpret_cast<const u4*>(qr + 16 * mine);
    const uint32_t sc = sr[mine];
    const auto a = __builtin_amdgcn_permlane16_swap(c[0], c[1], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(c[2], c[3], false, false);
    const auto e = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto o = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    const auto s0 = __builtin_amdgcn_permlane16_swap(sc, sc, false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(s0[0], s0[0], false, false);
    const auto s2 = __builtin_amdgcn_permlane32_swap(s0[1], s0[1], false, false);
    const uint32_t wd[4] = {e[0], o[0], e[1], o[1]};
    const uint32_t sd[4] = {s1[0], s2[0], s1[1], s2[1]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (j + i >= blocks) break;
      const u4 wf = q4_unpack(wd[i]);
      const float sf = (float)__builtin_bit_cast(_Float16, (uint16_t)sd[i]);
      const int kb = j + i;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const f4 d = H16::mma16(xl[(int64_t)(kb * MT + t) * 64], wf, (f4)(0.f));
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[t][m] = fmaf(sf, d[m], acc[t][m]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int m = 0; m < 4; ++m) red[w][16 * t + 4 * m + kg][r] = acc[t][m];   // operand row 4 kg + m is column 4 m + kg
  __syncthreads();
  for (int e = tid; e < batch * MV_ROWS; e += MV_WAVES * WAVE) {
    const int b = e / MV_ROWS, n = e % MV_ROWS;
    if (row0 + n >= rows) continue;
    float v = 0.f, z = 0.f;
#pragma unroll
    for (int i = 0; i < MV_WAVES; ++i) {
      v += red[i][P * b][n];
      if constexpr (P == 2) z += red[i][P * b + 1][n];
    }
    if constexpr (P == 2) v = fmaf(z, 1.f / 2048.f, v);
    v *= inv[b];
    if (bias) v += bias[row0 + n];
    y_to<Y>(y, b * ldy + row0 + n, v);
  }
}

}  // namespace piq
