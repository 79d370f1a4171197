"""The page of a place of 16 keys by a multiplication (csrc/pi_share.hpp), on the host: for every page size, the same as a
division, at the borders of pages and for the largest places there can be."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"

PROGRAM = r"""
#include "pi_share.hpp"
#include <cstdio>
using namespace pish;
int main() {
  for (uint32_t per = 1; per <= 256; ++per) {
    const Divide d = divide_by(per);
    auto fine = [&](uint32_t x) { return divided(x, d) == (int)(x / per); };
    for (uint32_t x = 0; x < 70000; ++x)
      if (!fine(x)) return printf("%u %u\n", per, x), 1;
    for (uint32_t top : {1u << 20, 1u << 27, 1u << 28, (1u << 30) - 1})
      for (uint32_t page = top / per - 300; page <= top / per; ++page)
        for (uint32_t x : {page * per - 1, page * per, page * per + per / 2})
          if (x < 1u << 30 && !fine(x)) return printf("%u %u\n", per, x), 1;
  }
  puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_pages_of_places(tmp_path):
    src, exe = tmp_path / "pages.hip", tmp_path / "pages"
    src.write_text(PROGRAM)
    subprocess.run([HIPCC, "-O2", "-std=c++17", "--cuda-host-only", "-I",
                    os.path.join(ROOT, "activation_sparse_predict_amd", "csrc"), str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
