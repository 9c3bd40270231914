// Slotwise kernels of the layer norm calls (norm_kernels.hip), used by their
// host side (layernorm.hip).  Ciphertexts of block b and feature i are at item
// b * n_feat + i.  Parts 0 and 1 of the results are times `kept`, a constant 1
// with `drop` inverses (consts.h): what ks_rescale takes.
#pragma once
#include "consts.h"

namespace ckks {

// sum[b] = S = sum_i x_i and the three parts k (F sum_i x_i (x) x_i - S (x) S)
// for two rescales, with the constant eps on part 0.
struct MomentArgs {
  const uint64_t* x;    // [nb][n_feat][2][nl][N]
  uint64_t* sum;        // [nb][2][nl][N]
  uint64_t* out;        // [nb][3][nl][N]
  const uint64_t* tab;  // consts.h, n = 3: F, k, eps
  const uint64_t* kept;
  const PrimeConst* prime;
  int log_n, nl, n_feat;
};
int launch_moments(Ctx* c, hipStream_t s, const MomentArgs& a, int nb);

// out = k_i (F x_i - S) (x) r, items [first, last) of the call, for two rescales,
// beta_i on part 0.
struct NormArgs {
  const uint64_t *x, *sum, *r;  // [..][2][x_nl][N], same, [..][2][nl][N]
  uint64_t* out;                // [3][nl][N] an item
  const uint64_t *gain, *beta;  // consts.h, n = n_gain and n_feat (beta may be NULL)
  const uint64_t* feat;         // F, n = 1
  const uint64_t* kept;
  const PrimeConst* prime;
  int log_n, nl, x_nl, n_feat, n_gain, first, last;
};
int launch_norm(Ctx* c, hipStream_t s, const NormArgs& a);

// With g_i = k_i dy_i: G[b] = sum_i g_i at limbs below g_nl, and the three parts
// of sum_i g_i (x) xhat_i for two rescales.
struct GradSumArgs {
  const uint64_t *dy, *xhat;  // [nb][n_feat][2][nl][N], [..][2][x_nl][N]
  uint64_t* G;                // [nb][2][g_nl][N]
  uint64_t* out;              // [nb][3][nl][N]
  const uint64_t* gain;       // n = n_gain
  const uint64_t* kept;
  const PrimeConst* prime;
  int log_n, nl, x_nl, g_nl, n_feat, n_gain;
};
int launch_grad_sums(Ctx* c, hipStream_t s, const GradSumArgs& a, int nb);

// out[b] = k (r[b] (x) h[b]) for one rescale.
struct ScaledPairArgs {
  const uint64_t *r, *h;     // [nb][2][r_nl][N], [nb][2][nl][N]
  uint64_t* out;             // [nb][3][nl][N]
  const uint64_t *kept, *k;  // n = 1
  const PrimeConst* prime;
  int log_n, nl, r_nl;
};
int launch_scaled_pair(Ctx* c, hipStream_t s, const ScaledPairArgs& a, int nb);

// out = r (x) (F k_i dy_i - G) - xhat_i (x) R, items [first, last), for two
// rescales.
struct GradArgs {
  const uint64_t *dy, *xhat, *r;  // limbs dy_nl, x_nl, r_nl
  const uint64_t *G, *R;          // [..][2][nl][N]
  uint64_t* out;                  // [3][nl][N] an item
  const uint64_t *gain, *feat;
  const uint64_t* kept;
  const PrimeConst* prime;
  int log_n, nl, dy_nl, x_nl, r_nl, n_feat, n_gain, first, last;
};
int launch_grad(Ctx* c, hipStream_t s, const GradArgs& a);

// Features first ..: the three parts of sum_b dy[b][i] (x) xhat[b][i] for one
// rescale (out), and sum_b dy[b][i] (sum); either may be NULL.
struct WeightArgs {
  const uint64_t *dy, *xhat;
  uint64_t* out;  // [3][nl][N] a feature
  uint64_t* sum;  // [2][nl][N] a feature
  const uint64_t* kept;
  const PrimeConst* prime;
  int log_n, nl, x_nl, n_blk, n_feat, first;
};
int launch_weight_sums(Ctx* c, hipStream_t s, const WeightArgs& a, int n);

}  // namespace ckks
