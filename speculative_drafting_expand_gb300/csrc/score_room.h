// score_room.h -- how the workspace of the drafting step's scores grows
// (pe_set_kv_scores).  Host code without CUDA.
#pragma once
#include <algorithm>
#include <cstdint>

namespace pe {

// Captured steps may still use earlier buffers,
// which therefore stay with the handle: each is at least twice the one
// before, and one above most / 2 is `most`, the last; so all of them together
// stay below 2 most.
struct ScoreRoom {
  char* ptr = nullptr;
  int64_t bytes = 0;

  // alloc(n): n bytes, or nullptr.  False where there was no memory.
  template <class Alloc>
  bool grow(int64_t want, int64_t most, Alloc alloc) {
    if (std::min(want, most) <= bytes) return true;
    int64_t n = std::max(want, 2 * bytes);
    if (n > most / 2) n = most;
    char* p = alloc(n);
    if (!p) return false;
    ptr = p;
    bytes = n;
    return true;
  }
};

}  // namespace pe
