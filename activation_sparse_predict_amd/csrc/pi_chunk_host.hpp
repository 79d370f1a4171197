// Launches of attention of chunks, shared by its translation units.
#pragma once
#include "pi_chunk.hpp"

namespace pia {

// A call as the kernels take it.
struct ChunkCall {
  Pages pg;
  Rows q;
  uint16_t* out;
  int64_t out_token, out_head;
  Chunks ch;
  ChunkScore sc;
  Joint* joints;
  int32_t* count;
  float *part, *stat;
  int mod, few;                          // CH_CAP, CH_SLOPES; 16-row tiles of a block of k_chunk_few
  unsigned blocks;
  hipStream_t stream;
};

template <class K> void launch(K kernel, const ChunkCall& c, int waves = 4) {
  hipLaunchKernelGGL(kernel, dim3(c.blocks), dim3(waves * WAVE), 0, c.stream, c.pg, c.q, c.out, c.out_token, c.out_head, c.ch, c.sc,
                     c.joints, c.count, c.part, c.stat);
}

// f(a constant of the score's kind)
template <class F> void with_mod(int mod, F f) {
  if (mod == 0) f(std::integral_constant<int, 0>());
  else if (mod == CH_CAP) f(std::integral_constant<int, CH_CAP>());
  else if (mod == CH_SLOPES) f(std::integral_constant<int, CH_SLOPES>());
  else f(std::integral_constant<int, CH_CAP | CH_SLOPES>());
}

// The calls of few rows (pi_chunk_few.hip).
void launch_few(int dtype, const ChunkCall& c);

}  // namespace pia
