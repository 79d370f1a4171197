"""The integer functions that cut attention over a cache into shares and follow page numbers (csrc/pi_share.hpp), on the
host: what the kernels do with lengths, prefixes and page numbers that cannot be, and that shares cover every key once."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"

PROGRAM = r"""
#include "pi_share.hpp"
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
using namespace pish;
#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  // numbers that cannot be
  for (int bad : {-1, INT_MIN, 161, INT_MAX}) CHECK(usable_len(bad, 10, 16) == 0);
  for (int n : {0, 1, 160}) CHECK(usable_len(n, 10, 16) == n);
  CHECK(usable_len(INT_MAX - 127, (INT_MAX - 127) / 16, 16) == INT_MAX - 127);
  for (int bad : {-1, INT_MIN, 11, INT_MAX, 0}) CHECK(common_tokens(bad, 10, 16) == 0);
  CHECK(common_tokens(10, 10, 16) == 160 && common_tokens(1, 10, 16) == 16);
  for (int bad : {-1, INT_MIN, 100, INT_MAX}) CHECK(usable_page(bad, 100) == -1);
  for (int id : {0, 99}) CHECK(usable_page(id, 100) == id);
  for (int key : {0, 15, 16, 159, 160, INT_MAX}) {
    const int p = place_of(key, 16, 10);
    CHECK(p >= 0 && p < 10 && (key >= 160 || p == key / 16));
  }
  // shares cover [0, steps) once, in order
  std::mt19937 rng(1);
  auto upto = [&](int64_t n) { return (int)(rng() % (uint64_t)n); };
  for (int t = 0; t < 20000; ++t) {
    const int steps = t < 100 ? t : upto(t % 3 ? 5000 : (1 << 26)), n = 1 + upto(t % 2 ? 64 : MOST);
    CHECK(share_begin(steps, 0, n) == 0 && share_begin(steps, n, n) == steps);
    for (int i = 0; i < n; ++i) CHECK(share_begin(steps, i, n) <= share_begin(steps, i + 1, n));
  }
  // the common keys: no share without a tile
  for (int t = 0; t < 20000; ++t) {
    const int total = 16 * (1 + upto(t % 2 ? 4000 : (1 << 26))), most = 1 + upto(64);
    const int n = common_shares(total, most), tiles = (total + TILE - 1) / TILE;
    CHECK(n >= 1 && n <= most && (n == 1 || tiles / n >= TILES));
    for (int i = 0; i < n; ++i) CHECK(share_begin(tiles, i, n) < share_begin(tiles, i + 1, n));
  }
  // what is dealt to the rows fits `free` and one each, and no row goes without
  for (int t = 0; t < 20000; ++t) {
    const int rows = 1 + upto(t % 5 ? 40 : 1023), free = 1 + upto(512);
    std::vector<int> units(rows);
    uint64_t all = 0;
    for (int& u : units) {
      u = t % 7 == 0 ? 0 : t % 7 == 1 ? units_of(INT_MAX - 127) : t % 7 == 2 ? upto(3) : upto(1 << (1 + upto(23)));
      all += u;
    }
    const uint32_t size = share_size(all, free);
    int64_t n = 0;
    for (int u : units) {
      const int d = deal(u, size);
      CHECK(d >= 1 && d <= MOST && (d == 1 || d <= u));
      n += d;
    }
    CHECK(size >= 1 && n <= rows + free);
  }
  CHECK(units_of(0) == 0 && units_of(1) == 1 && units_of(128) == 1 && units_of(129) == 2 && units_of(INT_MAX - 127) > 0);
  puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_shares_and_page_numbers(tmp_path):
    src, exe = tmp_path / "share.hip", tmp_path / "share"
    src.write_text(PROGRAM)
    subprocess.run([HIPCC, "-O2", "-std=c++17", "-ftrapv", "--cuda-host-only", "-I",
                    os.path.join(ROOT, "activation_sparse_predict_amd", "csrc"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
