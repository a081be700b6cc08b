// What ragged_shares.h answers, up to the rows that the products take; compiled so that an overflow or
// a conversion out of range ends the program.
#include <initializer_list>
#include <stdio.h>

#include "ragged_shares.h"

int main() {
  const int tiles[] = {64, 128, 192, 256};
  for (int tile : tiles) {
    for (int shift = 0; shift <= 25; ++shift) {
      for (int off = -1; off <= 1; ++off) {
        const int nk = (1 << shift) + off;          // 64 rows a step: 2^25 for 2^31 rows
        if (nk < 0) continue;
        for (int most : {1, 2, 7, 76, 80}) printf("%d %d %d %d\n", most, nk, tile, moe::shares(most, nk, tile));
      }
    }
  }
  return 0;
}
