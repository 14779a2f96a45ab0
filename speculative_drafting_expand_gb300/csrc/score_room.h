// score_room.h -- how the workspace of the drafting step's scores grows
// (pe_set_kv_scores).  Host code without CUDA.
#pragma once
#include <algorithm>
#include <cstdint>

namespace pe {

// The room is for logits that are worked out twice where it ends, so a step
// runs with whatever there is.  Captured steps may still use earlier buffers,
// which therefore stay with the handle: each is at least twice the one
// before, and one above most / 2 is `most`, the last; so all of them together
// stay below 2 most.
struct ScoreRoom {
  char* ptr = nullptr;
  int64_t bytes = 0;
  int64_t refused = INT64_MAX;  // a size that could not be had: not asked for again

  // alloc(n): n bytes, or nullptr.
  template <class Alloc>
  void grow(int64_t want, int64_t most, Alloc alloc) {
    if (std::min(want, most) <= bytes) return;
    int64_t n = std::max(want, 2 * bytes);
    if (n > most / 2) n = most;
    if (n >= refused) return;
    if (char* p = alloc(n)) {
      ptr = p;
      bytes = n;
    } else {
      refused = n;
    }
  }
};

}  // namespace pe
