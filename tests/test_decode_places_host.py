"""The kernels' bounds, on the CPU: the functions that say where a token of the
paged cache lies and how a sequence is cut into chunks (decode_launch.hpp, the
kernels' own) are compiled for the host and run over page tables with every
kind of bad entry, and over lengths, windows and new tokens.

Every byte that a token's place allows must be inside the cache, every table
entry inside the table; the chunks must cover the keys that are seen, be whole
blocks, and be no more than the workspace was sized for.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <set>
#include "decode_launch.hpp"
using namespace dsr;
#define NEED(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)
int main() {
  const int32_t bad[] = {INT32_MIN, -2, -1, 0, 1, 6, 7, 8, 1 << 30, INT32_MAX};
  long places = 0;
  for (int shift : {0, 3, 4, 12}) {
    const int page = 1 << shift, hd = 64, heads = 3;
    for (int order = 0; order < 2; ++order) {
      CacheView c{};
      c.n_pages = 7;
      c.page_shift = shift;
      c.heads = heads;
      c.hd = hd;
      c.seqs = 3;
      c.pages_per_seq = 5;
      c.ld_table = 6;
      c.head_bytes = order ? (int64_t)page * hd * 2 : hd * 2;
      c.token_bytes = order ? hd * 2 : heads * hd * 2;
      c.page_bytes = (int64_t)page * heads * hd * 2;
      const int64_t bytes = 7 * c.page_bytes;
      std::set<int64_t> seen;
      for (int64_t seq : {(int64_t)INT32_MIN, (int64_t)-1, (int64_t)0, (int64_t)2, (int64_t)3, (int64_t)INT32_MAX})
        for (int64_t t : {(int64_t)INT32_MIN, (int64_t)-1, (int64_t)0, (int64_t)page - 1, (int64_t)page,
                          (int64_t)5 * page - 1, (int64_t)5 * page, (int64_t)INT32_MAX}) {
          const bool in = token_in_table(c, seq, (int32_t)t);
          NEED(in == (seq >= 0 && seq < 3 && t >= 0 && t < 5 * page));
          if (!in) continue;
          const int64_t e = table_entry(c, seq, (int32_t)t);
          NEED(e >= 0 && e < 2 * 6 + 5 && e % 6 < 5);
          for (int32_t p : bad) {
            const int64_t at = token_bytes_at(c, p, (int32_t)t);
            NEED((at >= 0) == (p >= 0 && p < 7));
            if (at < 0) continue;
            ++places;
            NEED(at + (heads - 1) * c.head_bytes + hd * 2 <= bytes);
          }
        }
      for (int p = 0; p < 7; ++p)            // no two tokens in one place
        for (int t = 0; t < page; ++t) NEED(seen.insert(token_bytes_at(c, p, t)).second);
      c.page_bytes = 1ll << 33;              // offsets past 32 bits
      NEED(token_bytes_at(c, 6, page - 1) == (6ll << 33) + (page - 1) * c.token_bytes);
    }
  }
  for (int cap : {0, 1, 16, 255, 256, 257, 4096, 32768, 32769, 131072, 1 << 30})
    for (int len : {0, 1, 2, 5, 31, 32, 33, 255, 256, 257, 1000, 32768, 32769, 100000, 1 << 30})
      for (int n_new : {1, 2, 16})
        for (int window : {0, 1, 31, 33, 1000, 40000, 1 << 29})
          for (int heads : {1, 4, 12, 96, 1 << 20}) {
            if (len > cap) continue;
            const Span s = span_of(len, n_new, window, heads);
            const int64_t first = window ? (int64_t)len - n_new - window + 1 : 0;
            NEED(s.first == (first > 0 ? first : 0) && s.start % kTile == 0 && s.start <= s.first);
            NEED(s.first - s.start < kTile && s.chunk % kBlock == 0 && s.chunk > 0);
            NEED(s.n >= 1 && s.n <= kMaxChunks && s.n <= most_chunks(cap, n_new, window, heads));
            NEED((int64_t)s.start + (int64_t)s.n * s.chunk >= len);
            NEED(s.n == 1 || (int64_t)s.start + (int64_t)(s.n - 1) * s.chunk < len);   // none empty
            NEED((int64_t)s.start + (int64_t)s.n * s.chunk <= INT32_MAX);
          }
  // every length up to a capacity fits what is sized for it
  for (int heads : {1, 3, 8, 40})
    for (int window : {0, 500, 20000})
      for (int len = 0, most = 0; len < 70000; len += 1 + len / 97) {
        const int n = span_of(len, 3, window, heads).n;
        most = most > n ? most : n;
        NEED(most <= most_chunks(len, 3, window, heads));
      }
  std::printf("places %ld\n", places);
  return 0;
}
"""


def test_places_and_chunks(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("needs hipcc")
    src, exe = tmp_path / "places.hip", tmp_path / "places"
    src.write_text(SOURCE)
    inc = [f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(ROOT, 'scale_invariant_row_amd', 'csrc')}"]
    cc = subprocess.run([hipcc, "--offload-arch=gfx950", "-O1", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                         "-packed-fp32-ops", *inc, str(src), "-o", str(exe)],
                        capture_output=True, text=True, timeout=600)
    assert cc.returncode == 0, cc.stdout + cc.stderr
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and p.stdout.startswith("places "), p.stdout + p.stderr
