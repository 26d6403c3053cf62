"""CPU tests of how the microscaled attention divides its work over warps: the kernel's own header,
compiled for the host."""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

SOURCE = r"""
#include "mx_walk.cuh"
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
using namespace tq::mx;

struct Kernel {
  struct { int B, Hkv, maxp, pshift; } c;
  const int *lens, *counts;
  int Lq, row_blocks;
};
constexpr int W = 4; // warps of a CTA

#define CHECK(x) if (!(x)) { std::printf("seed %u: %s\n", seed, #x); std::exit(1); }

// Walks every warp's stretch of the space that the lengths span at first. change: lengths are others between any two steps,
// and the cursor is asked on behind its end, as the copies that run ahead do.
void trial(unsigned seed, bool change) {
  std::mt19937 gen(seed);
  auto pick = [&](int lo, int hi) { return static_cast<int>(lo + gen() % (hi - lo + 1)); };
  Kernel k;
  k.c = {pick(1, 9), pick(1, 3), pick(1, 12), pick(4, 6)};
  const int B = k.c.B, cap = k.c.maxp << k.c.pshift, ctas = pick(1, 7);
  k.Lq = pick(1, 16), k.row_blocks = pick(1, 4);
  const int units = k.c.Hkv * k.row_blocks;
  std::vector<int> lens(B), counts(B);
  k.lens = lens.data(), k.counts = counts.data();
  auto roll = [&](int b) { lens[b] = pick(0, 4) ? pick(-3, cap + 40) : 0, counts[b] = pick(-1, k.Lq + 1); };
  for (int b = 0; b < B; ++b) roll(b);
  uint32_t total = 0;
  std::vector<uint32_t> begins(B);
  for (int b = 0; b < B; ++b) {
    begins[b] = total;
    if (tiles_of(k, b)) total += (tiles_of(k, b) + kUnitCost) * units;
  }
  std::vector<int> first_lens = lens, first_counts = counts;
  std::vector<char> met(static_cast<size_t>(B) * units * (cap / 16 + 1), 0);
  const Split split(total, ctas, W);
  CHECK(split.begin(0) == 0 && split.begin(ctas * W) == total);
  for (int w = 0; w < ctas * W; ++w) {
    lens = first_lens, counts = first_counts;
    const uint32_t begin = split.begin(w);
    const int len = static_cast<int>(split.begin(w + 1) - begin);
    if (len == 0) continue;
    for (uint32_t at : {begin, begin + len - 1}) CHECK(split.share_of(at) == static_cast<uint32_t>(w));
    int b0 = 0;
    for (int b = 0; b < B; ++b)
      if (tiles_of(k, b) && begins[b] <= begin) b0 = b;
    Cursor c;
    if (change) for (int b = 0; b < B; ++b) if (pick(0, 1)) roll(b);
    c.start(k, b0, begin - begins[b0]);
    bool more = true;
    for (int behind = 0; behind < 6;) {
      if (more) {
        CHECK(c.b >= 0 && c.b < B && c.h >= 0 && c.h < k.c.Hkv && c.rb >= 0 && c.rb < k.row_blocks);
        const int t0 = c.first(), t1 = c.end(len), e = c.end16(k, len);
        CHECK(e <= cap / 16 && t1 <= cap / 16 + 1);
        for (int t = t0; !change && t < t1; ++t) {
          char &m = met[((static_cast<size_t>(c.b) * k.c.Hkv + c.h) * k.row_blocks + c.rb) * (cap / 16 + 1) + t];
          CHECK(m == 0);
          m = 1;
        }
      } else {
        ++behind;
        if (!change) CHECK(!c.next(k, len));
      }
      if (change) for (int b = 0; b < B; ++b) if (pick(0, 3) == 0) roll(b);
      more = c.next(k, len);
    }
  }
  if (change) return;
  for (int b = 0; b < B; ++b)
    for (int u = 0; u < units; ++u)
      for (int t = 0; t <= cap / 16; ++t) CHECK(met[(static_cast<size_t>(b) * units + u) * (cap / 16 + 1) + t] == (t < tiles_of(k, b)));
}

int main(int, char **argv) {
  for (unsigned seed = 0; seed < 4000; ++seed) trial(seed, std::atoi(argv[1]));
  std::puts("ok");
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("walk")
    (d / "walk.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "quantized_decode_attention_kv_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, "-x", "c++", str(d / "walk.cpp"), "-o", str(d / "walk")], check=True)
    return str(d / "walk")


def test_every_tile_belongs_to_one_warp(program):
    r = subprocess.run([program, "0"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_a_walk_stays_in_range_when_lengths_change(program):
    r = subprocess.run([program, "1"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
