"""CPU check of how F8 products are cut (f8_shape.h, compiled for the host):
every part of K has some of it (a part without any would not end), parts and
tiles fit the CUs, and the workspace holds every part's sums."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <stdio.h>
#include <initializer_list>
#include "f8_shape.h"
int main() {
  const int64_t ms[] = {0, 1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 500, 512, 777,
                        1000, 1024, 2047, 4096, 8192, 16384, 70000, 2147483647};
  const int64_t ns[] = {1, 4, 5, 63, 64, 127, 128, 129, 300, 512, 1000, 1024, 2048, 3584, 8192, 13312, 70000, 2147483647};
  long bad = 0, split = 0, rows = 0, tiles[3] = {0, 0, 0};
  for (int cus : {256, 304, 64, 1})
    for (int64_t M : ms)
      for (int64_t N : ns)
        for (int64_t K = 128; K <= (1 << 22); K = K < 40000 ? K + 128 : K * 3 / 256 * 128 + 128) {
          const dg::F8Choice c = dg::f8_choice(M, N, K, cus);
          const int64_t low = (M + 63) / 64 * ((N + 127) / 128), bytes = dg::f8_gemm_workspace(M, N, K, cus);
          bool ok = c.parts >= 1;
          if (c.rows) {
            ok = ok && c.parts == 1 && (c.rows == 16 || c.rows == 32 || c.rows == 64) && (M <= c.rows || c.rows == 32);
            ++rows;
          } else {
            ok = ok && (c.size == 64 || c.size == 128 || c.size == 256) && (c.parts == 1 || c.size == 64);
            ++tiles[c.size / 128];
          }
          if (c.parts > 1) {
            ++split;
            ok = ok && (c.parts - 1) * dg::f8_part(K, c.parts) < K && low * c.parts <= cus && dg::f8_part(K, c.parts) % 512 == 0 &&
                 c.parts * dg::f8_part(K, c.parts) >= K && bytes >= c.parts * M * N * 4 && bytes % 16 == 0;
          } else {
            ok = ok && bytes == 0;
          }
          if (!ok && ++bad < 10) printf("M %ld N %ld K %ld cus %d: %d %d %d\n", (long)M, (long)N, (long)K, cus, c.rows, c.size, c.parts);
        }
  for (int64_t K = 128; K <= (1 << 22); K += 128 * 37)
    for (int64_t want = 1; want <= 512; want += want < 40 ? 1 : 31) {
      const int p = dg::f8_parts(K, want);
      if (p < 1 || p > want || (p - 1) * dg::f8_part(K, p) >= K) ++bad;
    }
  printf("bad %ld split %ld rows %ld tiles %ld %ld %ld\n", bad, split, rows, tiles[0], tiles[1], tiles[2]);
  return bad || !split || !rows || !tiles[0] || !tiles[1] || !tiles[2];
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_every_choice_over_the_range(tmp_path):
    src, exe = tmp_path / "shape.cpp", tmp_path / "shape"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "communication_tensor_gemm_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


CHOICES = r"""
#include <stdio.h>
#include <initializer_list>
#include "f8_shape.h"
int main() {
  // of the kernels for few rows by their rows, of the tiles by size and whether K is in parts
  long rows[3] = {0, 0, 0}, whole[3] = {0, 0, 0}, parts = 0, few_many = 0, other = 0;
  for (int cus : {256, 304, 64})
    for (int64_t M = 1; M <= 16384; M = M < 130 ? M + 1 : M * 5 / 4)
      for (int64_t N = 1; N <= 70000; N = N < 20 ? N + 3 : N * 6 / 5)
        for (int64_t K = 128; K <= 65536; K = K * 5 / 384 * 128 + 128) {
          const dg::F8Choice c = dg::f8_choice(M, N, K, cus);
          if (c.rows) ++(c.rows == 16 ? rows[0] : c.rows == 32 ? rows[1] : c.rows == 64 ? rows[2] : other);
          else if (c.parts > 1) ++parts;
          else ++(c.size == 64 ? whole[0] : c.size == 128 ? whole[1] : whole[2]);
          // more 64 x 128 tiles than CUs: tiles for every M past 32
          if (M > 32 && (M + 63) / 64 * ((N + 127) / 128) > cus) {
            ++few_many;
            other += c.rows != 0 || (M <= 64 && c.size != 64);
          }
        }
  printf("rows %ld %ld %ld whole %ld %ld %ld parts %ld many %ld other %ld\n", rows[0], rows[1], rows[2], whole[0], whole[1], whole[2],
         parts, few_many, other);
  return !(rows[0] && rows[1] && rows[2] && whole[0] && whole[1] && whole[2] && parts && few_many && !other);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_every_kernel_has_sizes(tmp_path):
    """Each size of the kernel for few rows, each tile and K in parts is taken for some sizes."""
    src, exe = tmp_path / "choices.cpp", tmp_path / "choices"
    src.write_text(CHOICES)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "communication_tensor_gemm_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.skipif(shutil.which("g++") is None or shutil.which("gcov") is None, reason="g++ or gcov not available")
def test_no_part_of_the_choice_is_dead(tmp_path):
    """Every branch of f8_choice goes both ways over the sizes above."""
    (tmp_path / "choices.cpp").write_text(CHOICES)
    header = os.path.join(ROOT, "communication_tensor_gemm_amd", "csrc")
    subprocess.run(["g++", "-O0", "-std=c++17", "--coverage", "-I", header, "choices.cpp", "-o", "choices"], check=True, cwd=tmp_path)
    subprocess.run(["./choices"], check=True, cwd=tmp_path, capture_output=True)
    out = subprocess.run(["gcov", "-b", "-c", "-t", "choices.gcda"], check=True, cwd=tmp_path, capture_output=True, text=True).stdout
    body = out[out.index("inline F8Choice f8_choice"):out.index("inline int64_t f8_gemm_workspace")]
    dead, line = [], ""
    for l in body.splitlines():
        if l.lstrip().startswith("branch"):
            # (a branch of an exception's clean-up is not one of the choice)
            if "(throw)" not in l and ("never" in l or l.split()[3] == "0"):
                dead.append(line)
        elif ":" in l:
            line = l
    assert not dead, dead
