// The words that the rows of a tree's attention are masked by, as the kernel asks for them: every thread of a unit's two lanes, in
// every tile that holds nodes.  Built by test_tree_bits_host.py; prints the first wrong access or value, exits 1.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "tree_bits.h"

// A word array that knows its end, and which of its words belong to nodes in use.
struct Words {
  const std::vector<uint64_t>* w;
  size_t from, to;  // the words of the sequence's nodes in use
  uint64_t operator[](size_t i) const {
    if (i < from || i >= to) {
      std::printf("word %zu of [%zu, %zu) read\n", i, from, to);
      std::exit(1);
    }
    return (*w)[i];
  }
};

int main() {
  unsigned x = 1;
  auto rnd = [&] { return (x = x * 1664525u + 1013904223u) >> 8; };
  const int nodes[] = {1, 2, 5, 31, 32, 33, 63, 64, 65, 127, 128, 129, 225, 255, 256};
  const int prefixes[] = {0, 1, 63, 64, 65, 127, 128, 1000};
  long asked = 0;
  for (int G = 1; G <= 16; ++G) {
    const int RT = 128 / G * G;
    for (int N : nodes)
      for (int n : prefixes)
        for (int m : {N, N - 1, N / 2}) {
          if (m < 1) continue;
          const int B = 2, words = (N + 63) / 64, rows = m * G, ntok = n + m;
          std::vector<uint64_t> w(static_cast<size_t>(B) * N * words);
          for (auto& y : w) y = (static_cast<uint64_t>(rnd()) << 40) ^ (static_cast<uint64_t>(rnd()) << 20) ^ rnd();
          const int b = B - 1;
          const size_t at = static_cast<size_t>(b) * N * words;
          const Words seen{&w, at, at + static_cast<size_t>(m) * words};
          for (int r0 = 0; r0 < rows; r0 += RT)
            for (int row = 0; row < 128; ++row)
              for (int first = n / 128 * 128; first < (ntok + 127) / 128 * 128; first += 64) {
                const uint64_t got = vg::tree_bits(seen, N, words, G, b, rows, r0 + row, n, ntok, first);
                ++asked;
                for (int i = 0; i < 64; ++i) {
                  const int u = first + i - n;
                  const bool want = r0 + row < rows && u < m &&
                                    (u < 0 || (w[at + static_cast<size_t>((r0 + row) / G) * words + u / 64] >> (u % 64) & 1));
                  if (static_cast<bool>(got >> i & 1) != want) {
                    std::printf("G %d N %d m %d n %d row %d token %d\n", G, N, m, n, r0 + row, first + i);
                    return 1;
                  }
                }
              }
        }
  }
  std::printf("%ld words asked for\n", asked);
  return 0;
}
