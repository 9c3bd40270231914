// Products of encrypted features with matrices of 8-bit integers: the kernels
// (matmul_kernels.hip) and what their host side (linear.hip) hands them.
#pragma once
#include "consts.h"

namespace ckks {

// sum_i w[j][i] x[b][i] for outputs j0 <= j < j0 + nj of blocks b0 <= b < b0 +
// nb, on every limb i < nl.  The sums times kout (or as they are), times the
// token row (if any), go to limbs below nl - drop of out, the rest to top (item
// (b - b0) * nj + j - j0 of either).
struct MatArgs {
  const uint64_t* x;     // [n_blk][n_in][2][nl][N]
  const int8_t* w;       // element (j, i) at j * w_row + i * w_col
  const uint64_t* kin;   // constants of the inputs (consts.h, n = n_in), or NULL
  const uint64_t* kout;  // of the outputs (n = n_kout: n_out or one for all)
  const uint64_t* bias;  // added to component 0 (n = n_out; drop 0), or NULL
  const uint64_t* tok;   // [n_tok][nl][N], row b % n_tok, or NULL
  uint64_t* out;         // [2][nl - drop][N] an item
  uint64_t* top;         // [2][drop][N] an item
  const PrimeConst* prime;
  uint64_t w_row, w_col;
  int log_n, nl, drop, n_in, n_out, n_kout, n_tok, b0, nb, j0, nj;
};

// Words of the laid-out matrix for a launch of nj outputs.
uint64_t matmul_pack_words(int n_in, int nj);
// Lays the matrix out in `pack` and forms the products.
int launch_matmul(Ctx* c, hipStream_t s, const MatArgs& a, uint64_t* pack);

}  // namespace ckks
