// The operators' launch rules: plain host arithmetic on a call's sizes.
#pragma once

#include <cstdint>

namespace pa {

// Items that a batch of N rows in B sequences is taken to have, at `full` items for a block of
// `rows` rows and `one` for a block of one. Blocks never span sequences, so N / rows blocks are
// too few where sequences are shorter: 64 decode rows called with query_block = 16 are 64
// blocks, not 4. (Sequences without rows count too, as far as there are rows for them: the host
// does not know which they are.)
inline int64_t items_of_batch(int64_t N, int64_t B, int64_t rows, int64_t full, int64_t one) {
  const int64_t long_ones = (N + rows - 1) / rows * full, short_ones = (B < N ? B : N) * one;
  return long_ones > short_ones ? long_ones : short_ones;
}

// Rows of a query block of R rows and G heads that one tile of 128 takes, G at most 128.
inline int rows_of_tile(int R, int G) { return R * G <= 128 ? R : 128 / G; }

// Whether the sparse attention takes the warp-level kernel (sparse.cu has the reason).
inline bool takes_rows_kernel(int R, int G) { return R * G <= 16 || G > 128; }

// CTAs that share an item's pieces (tiles of keys, pages): as many as run at once in `slots`
// places, at most `most`, each with at least `least` pieces.
inline int cluster_size(int64_t items, int64_t slots, int64_t pieces, int least, int most) {
  int c = 1;
  while (2 * c <= most && items * 2 * c <= slots && pieces >= (int64_t)2 * c * least) c *= 2;
  return c;
}

}  // namespace pa
