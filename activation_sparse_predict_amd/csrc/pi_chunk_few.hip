// Attention of chunks of few rows over a paged cache: the kernels and their launches.
#include "pi_attn_host.hpp"
#include "pi_chunk_host.hpp"

void pia::launch_few(int dtype, const ChunkCall& c) {
  pih::with_type(dtype, c.ch.dim, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    with_mod(c.mod, [&](auto m) {
      constexpr int MOD = decltype(m)::value;
      if (c.few == 1) launch(k_chunk_few<T, D, MOD, 1>, c);
      else launch(k_chunk_few<T, D, MOD, 2>, c);
    });
  });
}
