// Which tokens a row of a tree's attention attends (host + device: nothing here needs a GPU).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define VG_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define VG_HOST_DEVICE inline
#endif

namespace vg {

// Which of the tokens first .. first + 63 of sequence `seq`'s range of n prefix tokens and ntok - n nodes query row `row`
// attends (of `rows` = (ntok - n) G; a node's heads are G rows).  Words: const uint64_t*, [sequences][R][words].  A tile has rows
// behind the last one: they attend nothing, and no word is read for them (the last sequence's nodes may end with the array).
template <class Words>
VG_HOST_DEVICE uint64_t tree_bits(Words visible, int R, int words, int G, int seq, int rows, int row, int n, int ntok,
                                  int first) {
  if (row >= rows) return 0;
  const int u = first - n, left = ntok - first;
  const size_t sees = (static_cast<size_t>(seq) * R + row / G) * words;
  uint64_t v;
  if (u <= -64) {
    v = ~uint64_t{0};
  } else if (u < 0) {
    v = (visible[sees] << -u) | ((uint64_t{1} << -u) - 1);
  } else {
    const int i = u >> 6, s = u & 63;
    v = i < words ? visible[sees + i] >> s : 0;
    if (s && i + 1 < words) v |= visible[sees + i + 1] << (64 - s);
  }
  if (left < 64) v &= left <= 0 ? 0 : (uint64_t{1} << left) - 1;
  return v;
}

}  // namespace vg
