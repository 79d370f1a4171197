// Host side of the products with Q4_0 matrices (pi.h): checks, workspace, launches.
#include "pi_q4.hpp"

#include <algorithm>
#include <type_traits>

#include "pi_host.hpp"

using namespace pih;

namespace {

// 12288 float32 values; with the sums of the waves (9 KB) a block keeps to 64 KB
constexpr size_t kOperandLds = 48 << 10;

// the operand made of x, of the largest number of columns a type of x takes, and a row's scale
struct Ws {
  size_t inv, total;
};
Ws ws_of(int32_t cols, int32_t batch) {
  Ws w{};
  w.inv = ws_align((size_t)up_div(2 * batch, 16) * 16 * cols * sizeof(uint16_t));
  w.total = w.inv + ws_align(sizeof(float) * 32);
  return w;
}

int size_of(int32_t dtype) { return dtype == PI_F32 ? 4 : 2; }

pi_status check_sizes(int32_t rows, int32_t cols, int32_t batch) {
  if (rows < 1 || cols < 32 || cols % 32 != 0 || batch < 1 || batch > 32) return PI_EINVAL;
  return rows > (1 << 28) || cols > (1 << 22) ? PI_EUNSUPPORTED : PI_OK;
}

// f(constant of the dtype)
template <class F>
void with_dtype(int32_t dtype, F f) {
  if (dtype == PI_F32) f(std::integral_constant<int, PI_F32>());
  else if (dtype == PI_F16) f(std::integral_constant<int, PI_F16>());
  else f(std::integral_constant<int, PI_BF16>());
}

}  // namespace

extern "C" {

size_t pi_matvec_workspace_bytes(int32_t rows, int32_t cols, int32_t batch) {
  return check_sizes(rows, cols, batch) == PI_OK ? ws_of(cols, batch).total : 0;
}

pi_status pi_matvec(const pi_mat* mat, int32_t rows, int32_t cols, const float* bias, const void* x, int32_t x_dtype,
                    int64_t ldx, void* y, int32_t y_dtype, int64_t ldy, int32_t batch, void* ws, size_t ws_bytes,
                    void* stream) {
  pi_status s;
  if ((s = check_sizes(rows, cols, batch)) != PI_OK) return s;
  if (!mat || !mat->w || !mat->scale || !on(mat->w, 16) || !on(mat->scale, 2) || !on(bias, 4)) return PI_EINVAL;
  for (int32_t t : {x_dtype, y_dtype})
    if (t != PI_F32 && t != PI_F16 && t != PI_BF16) return PI_EINVAL;
  if (!x || !on(x, size_of(x_dtype)) || !y || !on(y, size_of(y_dtype)) || ldx < cols || ldy < rows) return PI_EINVAL;
  const Ws W = ws_of(cols, batch);
  if (!ws || ws_bytes < W.total || !on(ws, kWsAlign)) return PI_EWORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint16_t* xo = static_cast<uint16_t*>(ws);
  float* inv = reinterpret_cast<float*>(static_cast<char*>(ws) + W.inv);
  (void)hipGetLastError();
  with_dtype(x_dtype, [&](auto xt) {
    constexpr int X = decltype(xt)::value, P = piq::parts<X>();
    const int columns = P * batch;
    // few columns whose operand fits beside another block's in LDS: each block makes it for itself
    const size_t lds = (size_t)2 * columns * cols;
    const bool few = columns <= 16 && lds <= kOperandLds;
    const int tiles = (int)up_div(columns, 16);
    if (!few)
      hipLaunchKernelGGL((piq::k_mv_operand<X>), dim3(16 * tiles / P, (unsigned)std::min<int64_t>(16, up_div(cols, 1024))),
                         dim3(256), 0, st, x, ldx, batch, cols, tiles, xo, inv);
    with_dtype(y_dtype, [&](auto yt) {
      constexpr int Y = decltype(yt)::value;
      auto w_of = static_cast<const uint8_t*>(mat->w);
      if (few) {
        auto go = [&](auto ma) {
          // as many blocks as fit at once (up to four a compute unit), each with an even share of the row tiles
          const int64_t fit = std::min<int64_t>(4, (160 << 10) / (int64_t)(lds + (10 << 10)));
          hipLaunchKernelGGL((piq::k_matvec_few<X, Y, decltype(ma)::value>),
                             dim3((unsigned)std::min(up_div(rows, piq::MV_ROWS), 256 * fit)),
                             dim3(piq::MV_WAVES * piq::WAVE), lds, st, w_of, mat->scale, bias, rows, cols, x, ldx,
                             batch, y, ldy);
        };
        if (columns <= 4) go(std::integral_constant<int, 1>());
        else if (columns <= 8) go(std::integral_constant<int, 2>());
        else go(std::integral_constant<int, 4>());
        return;
      }
      auto go = [&](auto mt) {
        hipLaunchKernelGGL((piq::k_matvec<X, Y, decltype(mt)::value>),
                           dim3((unsigned)up_div(rows, piq::MV_ROWS)), dim3(piq::MV_WAVES * piq::WAVE), 0, st, w_of,
                           mat->scale, bias, rows, cols, xo, inv, batch, y, ldy);
      };
      if (tiles == 1) go(std::integral_constant<int, 1>());
      else if (tiles == 2) go(std::integral_constant<int, 2>());
      else if (tiles == 3) go(std::integral_constant<int, 3>());
      else go(std::integral_constant<int, 4>());
    });
  });
  return launched();
}

}  // extern "C"
