"""How the MX products are cut into workgroups, without a GPU: the host
arithmetic of csrc/mx_shape.h compiled by itself and swept over sizes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "communication_tensor_gemm_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")


def run(tmp_path, body):
    """Compiles `body` as main() behind the header; what it prints, which is nothing where all is well."""
    src, exe = tmp_path / "sweep.cc", tmp_path / "sweep"
    src.write_text('#include "mx_shape.h"\n#include <cstdio>\n#include <initializer_list>\nint main() {\n' + body + "\nreturn 0;\n}\n")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-ftrapv", f"-I{CSRC}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_every_column_of_a_workgroup_is_computed(tmp_path):
    """A workgroup computes `most` columns, so its step must not be more: every
    row tile count of up to 8192 rows, every width up to 8192 and some beyond."""
    out = run(tmp_path, """
      const int cus[] = {256, 304, 228, 64, 1};
      const int64_t wide[] = {8193, 9999, 13312, 16383, 65537, 151936, 1000003, 2147483647};
      long bad = 0;
      for (int most = 16; most <= 32; most += 16)
        for (int c : cus)
          for (int64_t tiles = 1; tiles <= 512; ++tiles) {
            auto check = [&](int64_t N) {
              const int step = dg::mx::rows_step(N, tiles, most, c);
              if ((step < 1 || step > most) && ++bad <= 5)
                std::printf("N %ld, %ld row tiles, %d CUs: %d columns of %d\\n", (long)N, (long)tiles, c, step, most);
            };
            for (int64_t N = 1; N <= 8192; ++N) check(N);
            for (int64_t N : wide) check(N);
          }
      if (bad) std::printf("%ld in all\\n", bad);""")
    assert out == ""


def test_tiles_of_sizes_up_to_the_largest(tmp_path):
    """In 32 bits, with the sums trapped where they overflow."""
    out = run(tmp_path, """
      for (int64_t size : {1, 4, 13, 16, 32, 64, 128, 256})
        for (int64_t i = 0; i < 5000; ++i)
          for (int64_t n : {i, i * 429496, int64_t{2147483647} - i})
            if (dg::mx::tile_count((int32_t)n, (int32_t)size) != (n + size - 1) / size) std::printf("%ld / %ld\\n", (long)n, (long)size);""")
    assert out == ""


def test_launches_hold_every_workgroup(tmp_path):
    """Fewer than 2^32 threads of up to 1024 per workgroup along x, fewer than 65536 workgroups along y, no gap."""
    out = run(tmp_path, """
      for (int64_t n : {int64_t{1}, int64_t{2097151}, int64_t{2097152}, int64_t{2097153}, int64_t{134217728}, int64_t{2147483647}}) {
        const int64_t x = dg::mx::grid_x(n), y = dg::mx::grid_y(n);
        if (x < 1 || x * 1024 >= int64_t{1} << 32 || y < 1 || y > 65535 || x * y < n || x * y - n >= x) std::printf("%ld\\n", (long)n);
        if (y > 1 && x != dg::mx::kGridX) std::printf("%ld: x\\n", (long)n);
      }""")
    assert out == ""
