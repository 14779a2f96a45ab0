"""How the workspace of the drafting step's scores grows, on the host."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

INCLUDES = r"""
#include <stdio.h>
#include <stdlib.h>
#include "score_room.h"
"""

WIDENING = INCLUDES + r"""
int main() {
  const int64_t most = int64_t{1} << 30, base = 6 << 20, page = 262144;
  {  // a table that widens by a page of 64 requests at a time
    pe::ScoreRoom r;
    int64_t total = 0, calls = 0, short_of = 0;
    auto get = [&](int64_t n) { total += n; ++calls; return (char*)(uintptr_t)(4096 * calls); };
    r.grow(base, base, get);
    for (int64_t w = 1; w <= 20000; ++w) {
      const int64_t want = base + page * w < most ? base + page * w : most;
      r.grow(want, most, get);
      short_of += r.bytes < want;
    }
    const int64_t before = calls;
    for (int64_t w = 20000; w > 0; --w) r.grow(base + page * w, most, get);
    printf("%lld %d %lld %d %d\n", (long long)calls, total < 2 * most, (long long)short_of,
           calls == before, r.bytes == most && r.ptr == (char*)(uintptr_t)(4096 * calls));
  }
  return 0;
}
"""

NO_MEMORY = INCLUDES + r"""
int main() {
  const int64_t most = int64_t{1} << 30, base = 6 << 20, page = 262144;
  {  // no memory: the step goes on with what there is, and does not ask again
     // for as much until it is told that there may be some
    pe::ScoreRoom r;
    int64_t calls = 0, room = base;
    auto get = [&](int64_t n) { ++calls; return n <= room ? (char*)4096 : (char*)nullptr; };
    r.grow(base, base, get);
    for (int64_t w = 1; w <= 1000; ++w) r.grow(base + page * w, most, get);
    printf("%d %lld ", r.bytes == base && r.ptr == (char*)4096, (long long)calls);
    room = most;
    r.refused = INT64_MAX;
    r.grow(base + page * 1000, most, get);
    printf("%d\n", r.bytes == base + page * 1000);
  }
  return 0;
}
"""


def _run(program, tmp_path):
    src, exe = tmp_path / "room.cpp", tmp_path / "room"
    src.write_text(program)
    csrc = os.path.join(ROOT, "speculative_drafting_expand_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    return [int(x) for x in out.split()]


def test_growth_is_bounded(tmp_path):
    calls, bounded, short_of, no_more, last = _run(WIDENING, tmp_path)
    assert calls <= 9 and bounded and short_of == 0 and no_more and last


def test_a_step_goes_on_without_more_room(tmp_path):
    kept, asked, again = _run(NO_MEMORY, tmp_path)
    # the first size and one refused one: every larger one is refused unasked
    assert kept and asked == 2 and again
