// The sum over a packed axis (sumrot.hip) and the slotwise kernels of the
// attention calls (attn_kernels.hip), used by their host side (attention.hip).
#pragma once
#include "ops.h"

namespace ckks {

constexpr int kMaxSumRot = CKKS_SUM_MAX_RADIX - 1;  // rotations of one stage

// Words of workspace sum_stages needs for `batch` items at `level`.
size_t sum_ws_words(const Ctx* c, int level, int batch, int n_stage);

// `batch` ciphertexts (item b at in + b*in_stride) through every stage of the
// checked plan into out + b*out_stride.  ws holds sum_ws_words.
int sum_stages(Ctx* c, hipStream_t s, const uint64_t* in, uint64_t in_stride, uint64_t* out, uint64_t out_stride,
               int batch, int level, const ckks_sum_steps& st, uint64_t* ws);

// out[b] = p[(first + b) % n_row] * in[b] on both components, limbs 0..nl-1.
struct PlainMulArgs {
  const uint64_t* in;  // item b at + b*in_bstride, component stride in_comp
  const uint64_t* p;   // [..][nl][N]
  uint64_t* out;       // item b at + b*out_bstride, [2][nl][N]
  uint64_t in_bstride, in_comp, out_bstride;
  const PrimeConst* prime;
  int log_n, nl, n_row, first;
};
int launch_plain_mul(Ctx* c, hipStream_t s, const PlainMulArgs& a, int batch);

// Tensor products of paired ciphertexts: out[b] = a[b] x b[b] at limbs
// 0..nl-1, item b of `a` at a + ia(b)*a_bstride with ia(b) = b / n_k and of
// `b` at (b / n_qk) * n_k + b % n_k (pairs [group][i][j]); with n_qk = 0 both
// are item b.  decay (optional): parts 0 and 1 get decay[row] * state[b] added,
// row = b % n_row (state [2][nl][N] per item, b_bstride apart).
struct PairArgs {
  const uint64_t *a, *b;
  uint64_t* out;  // [3][nl][N] per item
  uint64_t a_bstride, a_comp, b_bstride, b_comp, out_bstride;
  const uint64_t *decay, *state;
  uint64_t state_bstride;
  const PrimeConst* prime;
  int log_n, nl, n_k, n_qk, n_row, first;  // first: index of item 0 in the pair order
};
int launch_pair(Ctx* c, hipStream_t s, const PairArgs& a, int batch);

// Weighted prefix sums over tokens of one block: out[t][g] = init[g] +
// sum_{u <= t} w[u][g % n_row] * (k[u][g] x v[u][g]), three parts; k, v at
// token stride tok_stride; init may be NULL (zero).
struct ScanArgs {
  const uint64_t *k, *v, *w;
  const uint64_t* init;  // [n_grp][3][nl][N]
  uint64_t* out;         // [n_tok][n_grp][3][nl][N]
  uint64_t tok_stride;
  const PrimeConst* prime;
  int log_n, nl, n_tok, n_grp, n_row, g0;  // g0: the block's first group (its row offset)
};
int launch_scan(Ctx* c, hipStream_t s, const ScanArgs& a);

// Masked weighted sums: for row b = (g, i), num[b] = sum_j m[g % n_row][j] *
// (a[b][j] x v[g][j]) (three parts) and, when den is given, den[b] = sum_j
// m[g % n_row][j] * a[b][j]; m NULL: no mask.
struct MixArgs {
  const uint64_t *a, *v, *m;
  uint64_t *num, *den;
  const PrimeConst* prime;
  int log_n, nl, n_q, n_k, n_row, first;  // first: index of row 0
};
int launch_mix(Ctx* c, hipStream_t s, const MixArgs& a, int rows);

}  // namespace ckks
