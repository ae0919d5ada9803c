// How the embedding's lookup is cut into blocks. Plain C++: what holds at the
// limits of muon_embed.h can be checked without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace muon_embed {

constexpr int kThreads = 256;
constexpr int kLookVec = 8;   // consecutive elements per thread of the lookup
constexpr int kLookRuns = 4;  // such vectors per thread, kThreads apart
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;  // a launch holds under 2^32 threads

struct LookGrid {
  int64_t vpr;     // vectors in a row
  int64_t per;     // tokens of a block: about kLookRuns vectors a thread, more where the blocks would be too many
  int64_t blocks;
};
inline LookGrid lookup_grid(int64_t cols, int64_t n) {
  LookGrid g{};
  g.vpr = (cols + kLookVec - 1) / kLookVec;
  g.per = std::max<int64_t>({1, kThreads * kLookRuns / g.vpr, (n + kMaxBlocks - 1) / kMaxBlocks});
  g.blocks = (n + g.per - 1) / g.per;
  return g;
}

}  // namespace muon_embed
