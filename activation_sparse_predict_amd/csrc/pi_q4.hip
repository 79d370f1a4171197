// Host side of the products with Q4_0 matrices (pi.h): checks, workspace, launches.
#include "pi_q4.hpp"

#include <algorithm>
#include <type_traits>

#include "pi_host.hpp"

using namespace pih;

namespace {

// The operand of a product of few columns at most: with the sums of the waves (9 KB) a block keeps to 64 KB, what a launch
// may have without asking for more.  (In the few columns' kernel and in the others': one float32 row of 4096 x 4096 7.1 and
// 11.6 us, 4096 x 11008 11.5 and 19.7, 9216 x 8192 23 and 23, 36864 x 12288 61 and 82; but 2 bfloat16 rows of 9216 x 8192
// 27 and 22, 8 of 4096 x 2048 11.3 and 9.6 us.)
constexpr size_t kOperandLds = 48 << 10;

// Shares of the groups of 8 blocks in a product of many columns, 32 at most: those with which the rounds of 512 blocks
// (two for each compute unit), at 2.5 us a group, and the shares' sums, at 1 us for each 9216 rows of 32 columns,
// written and read, take least.  (32 bfloat16 rows, 9216 x 8192: 6, 7, 8, 9, 11 shares 25.9, 25.0, 27.9, 27.1, 29.0 us;
// 18432 x 8192: 3, 4, 5 shares 43, 48, 44 us; 36864 x 12288: 2, 3, 4 shares 98, 91, 91 us.)  The two costs were taken with 32
// columns and serve all numbers of them: with 8 to 64 columns and these and other matrices, down to 4096 x 4096 and
// 12288 x 49152, what they choose takes at most 7 % longer than the best of 1, 2, 3, 4, 6, 8, 12, 16, 24 and 32 shares.
int shares_of(int32_t rows, int32_t cols) {
  const int64_t groups = up_div(cols, 32 * piq::MV_G), blocks = up_div(rows, piq::MV_ROWS * piq::MV_WAVES);
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= std::min<int64_t>(groups, 32); ++s) {
    const int64_t cost = 5 * up_div(blocks * s, 512) * up_div(groups, s) * 9216 + 2 * (int64_t)s * rows;
    if (cost < least) least = cost, best = s;
  }
  return best;
}

// the operand made of x, whole groups of it, of the largest number of columns a type of x takes; a row's scale; the
// shares' sums
struct Ws {
  size_t inv, part, total;
};
Ws ws_of(int32_t rows, int32_t cols, int32_t batch) {
  Ws w{};
  const size_t padded = (size_t)up_div(cols, 32 * piq::MV_G) * 32 * piq::MV_G;
  w.inv = ws_align((size_t)up_div(2 * batch, 16) * 16 * padded * sizeof(uint16_t));
  w.part = w.inv + ws_align(sizeof(float) * 32);
  w.total = w.part + ws_align(sizeof(float) * 2 * batch * (size_t)rows * shares_of(rows, cols));
  return w;
}

int size_of(int32_t dtype) { return dtype == PI_F32 ? 4 : 2; }

pi_status check_sizes(int32_t rows, int32_t cols, int32_t batch) {
  if (rows < 1 || cols < 32 || cols % 32 != 0 || batch < 1 || batch > 32) return PI_EINVAL;
  return rows > (1 << 22) || cols > (1 << 22) ? PI_EUNSUPPORTED : PI_OK;
}

// Whether a row of y lies over a row of x: `n` of each, of xn and yn bytes, every xs and ys bytes.
bool over(const void* x, int64_t xs, int64_t xn, const void* y, int64_t ys, int64_t yn, int n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  if (b >= a + (n - 1) * xs + xn || a >= b + (n - 1) * ys + yn) return false;
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      if (a + i * xs < b + j * ys + yn && b + j * ys < a + i * xs + xn) return true;
  return false;
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
  return check_sizes(rows, cols, batch) == PI_OK ? ws_of(rows, cols, batch).total : 0;
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
  const Ws W = ws_of(rows, cols, batch);
  if (!ws || ws_bytes < W.total || !on(ws, kWsAlign)) return PI_EWORKSPACE;
  // blocks read x while others write y
  const int xb = size_of(x_dtype), yb = size_of(y_dtype);
  if (over(x, ldx * xb, (int64_t)cols * xb, y, ldy * yb, (int64_t)rows * yb, batch)) return PI_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint16_t* xo = static_cast<uint16_t*>(ws);
  float* inv = reinterpret_cast<float*>(static_cast<char*>(ws) + W.inv);
  (void)hipGetLastError();
  with_dtype(x_dtype, [&](auto xt) {
    constexpr int X = decltype(xt)::value, P = piq::parts<X>();
    const int columns = P * batch;
    // few columns whose operand fits beside another block's in LDS: each block makes it for itself
    const size_t lds = (size_t)2 * columns * cols;
    const bool few = columns <= 16 && lds <= kOperandLds, tiny = cols < 32 * piq::MV_G;
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
          auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)std::min(up_div(rows, piq::MV_ROWS), 256 * fit)),
                               dim3(piq::MV_WAVES * piq::WAVE), lds, st, w_of, mat->scale, bias, rows, cols, x, ldx,
                               batch, y, ldy);
          };
          if (tiny) launch(piq::k_matvec_few<X, Y, decltype(ma)::value, true>);
          else launch(piq::k_matvec_few<X, Y, decltype(ma)::value, false>);
        };
        if (columns <= 4) go(std::integral_constant<int, 1>());
        else if (columns <= 8) go(std::integral_constant<int, 2>());
        else go(std::integral_constant<int, 4>());
        return;
      }
      const int shares = shares_of(rows, cols);
      float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + W.part);
      auto go = [&](auto mt) {
        auto launch = [&](auto kernel) {
          hipLaunchKernelGGL(kernel, dim3((unsigned)up_div(rows, piq::MV_ROWS * piq::MV_WAVES), (unsigned)shares),
                             dim3(piq::MV_WAVES * piq::WAVE), 0, st, w_of, mat->scale, rows, cols, xo, columns, part);
        };
        if (tiny) launch(piq::k_matvec<decltype(mt)::value, true>);
        else launch(piq::k_matvec<decltype(mt)::value, false>);
        hipLaunchKernelGGL((piq::k_matvec_join<P, Y>), dim3((unsigned)up_div(rows, 256), (unsigned)batch), dim3(256), 0,
                           st, part, inv, bias, rows, shares, batch, y, ldy);
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
