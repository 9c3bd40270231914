// Which kernel a product with an 8-bit matrix takes, in plain C++: the tile by
// the matrix's size, the digits of a word by the primes (matmul_kernels.hip).
#pragma once
#include <stdint.h>

#include <algorithm>

namespace ckks {

// The matrix cores' tiles take outputs from kTileRows on (up to 8, a thread's
// own sums read the words once as well) and inputs from a group's 16 on.
constexpr int kTileRows = 9;
inline bool tiled(int n_in, int nj) { return nj >= kTileRows && n_in >= 16; }

// Signed bytes of a word below q: nd of them hold words up to 127 sum_d 2^(8d).
inline int word_digits(uint64_t q) {
  int nd = 4;
  while (nd < 8 && q > 0x7f7f7f7f7f7f7f7full >> (8 * (8 - nd))) ++nd;
  return nd;
}

// The tile of a launch: 32, 64, 128 or 256 outputs.  A word costs its conversion
// for every tile of outputs (some 16 instructions an input) and its sums'
// joining for every output, those past the last included (some 74): 131 outputs
// of 77 inputs (two blocks of 6 limbs at 2^14) take 0.92 ms a call in tiles of 64,
// 1.31 in one of 256; the product of 768 by 768 takes 2.9 ms in tiles of 256, 3.1
// of 128.  Both counts are those of 7 digits without scales on the inputs, and
// stand in for the other forms.
struct Tiles {
  int wm = 1, wn, mt = 1, row_blocks, chunks;
  Tiles(int n_in, int nj) {
    uint64_t least = ~0ull;
    for (int r = 32; r <= 256; r *= 2) {
      const uint64_t blocks = (nj + r - 1) / r, cost = blocks * r * 74 + blocks * n_in * 16;
      if (cost >= least) continue;
      least = cost;
      wm = std::min(r / 32, 4);
      mt = r == 256 ? 2 : 1;
    }
    wn = 4 / wm;
    row_blocks = (nj + rows() - 1) / rows();
    const int nc = 4 / wn;
    chunks = ((n_in + 31) / 32 + nc - 1) / nc * nc;
  }
  int rows() const { return 32 * wm * mt; }
  uint64_t lanes() const { return (uint64_t)row_blocks * wm * mt * chunks * 64; }
};

}  // namespace ckks
