// The sum over a packed axis (sumrot.hip) and the slotwise kernels of the
// attention calls (attn_kernels.hip), used by their host side (attention.hip).
#pragma once
#include <algorithm>

#include "ops.h"

namespace ckks {

constexpr int kMaxSumRot = CKKS_SUM_MAX_RADIX - 1;  // rotations of one stage

// Words reserved for steps that hold as many of a call's `items` (`per` words
// each) as fit `limit`, one at least.  It never falls when items or per grow,
// as the words of the items that fit would (a buffer of 4 items of 28 limbs is
// smaller than one of 5 items of 23): a call with fewer limbs or items than an
// earlier one finds its buffers large enough, which captures rely on.
inline uint64_t held_words(uint64_t per, uint64_t items, uint64_t limit) {
  return std::min(per * items, std::max(limit, per));
}

// Words of workspace sum_stages needs for `batch` items at `level`, in groups
// that fit `limit` words.
size_t sum_ws_words(const Ctx* c, int level, int batch, int n_stage, uint64_t limit);

// Inner products of n items' raised digits (E: item b at E + b*E_stride,
// [beta][next][N]; own: the NTT-form input [nq][N], own_stride apart) with the
// keys of n_rot rotations, each through tau_g: acc[c] = sum_r sum_j
// tau_{g_r}(D_j) evk_{r,j}.c into A (item b at A + b*A_stride, [2][next][N]).
// c0 (optional, [nq][N], own_stride apart): component 0 of the ciphertext
// limbs gets P sum_r tau_{g_r}(c0) added.  Ciphertext limbs are left congruent
// (below 10 q), special limbs below 4q.
int key_ip(Ctx* c, hipStream_t s, int level, int n, const uint64_t* E, uint64_t E_stride, const uint64_t* own,
           uint64_t own_stride, const uint64_t* c0, uint64_t* A, uint64_t A_stride, int n_rot, const uint32_t* g,
           const uint64_t* const* evk);

// `batch` ciphertexts (item b at in + b*in_stride) through every stage of the
// checked plan into out + b*out_stride.  ws holds sum_ws_words (same limit).
int sum_stages(Ctx* c, hipStream_t s, const uint64_t* in, uint64_t in_stride, uint64_t* out, uint64_t out_stride,
               int batch, int level, const ckks_sum_steps& st, uint64_t* ws, uint64_t limit);

// rescale(p[row] * in[b]) by the top limb `level`; b = t * ng + g (first + the
// launch's item) reads in + (t * n_grp + g)*in_bstride and row t * n_row +
// (g0 + g) % n_row.
struct PlainMul {
  const uint64_t* in;  // component stride in_comp
  const uint64_t* p;   // [..][level+1][N]
  uint64_t* out;       // item b at + b*out_bstride, [2][level][N]
  uint64_t in_bstride, in_comp, out_bstride;
  int level, ng, n_grp, n_row, g0, first;
};
// Limb `level` of the product, [2][N] per item at out + b*out_bstride.
int launch_plain_mul(Ctx* c, hipStream_t s, const PlainMul& m, uint64_t* out, uint64_t out_bstride, int batch);
// The rest (rescale.hip): v = iNTT of that limb, w scratch [2][level][N], per
// words between items of either.
int rescale_mul_fused(Ctx* c, hipStream_t s, const PlainMul& m, const uint64_t* v, uint64_t* w, uint64_t per, int batch);

// Items of a launch of rescale_products at most (fewer where the workspace holds
// fewer).  Each launch's tail leaves the chip part empty: a product of 768 outputs
// at 3 limbs of 2^16, 682 of which a workspace of 2 GiB holds, takes 5.37 ms in
// launches of 682 and 86, 5.46 in launches of 128 and 5.94 of 32.
constexpr int kMaxProducts = 1024;

// Rescales of n products by their top `drop` (1 or 2) limbs, in one transform:
// `top` holds the dropped limbs q_(level+1-drop)..q_level ([2][drop][N] an item, used up), `out` the limbs
// that stay times the inverses of the dropped primes ([2][level+1-drop][N] an
// item, in place; below 4q for primes below 2^61, canonical for larger ones).  add (optional): a constant for component 0 of item b,
// add[(i * n_add + (first + b) % n_add) * 2] in limb i.  ws holds 2 (level+1) N
// words an item of a chunk, one at least.
struct ProductRescale {
  uint64_t *top, *out;
  int n, level, drop;
  const uint64_t* add;
  int n_add, first;
};
int rescale_products(Ctx* c, hipStream_t s, const ProductRescale& p, uint64_t* ws, uint64_t ws_words);

// What the products below do to their output for ks_rescale: parts 0 and 1 of
// the limbs that stay after `drop` rescales are multiplied by the inverses of
// the dropped primes and get `add` added (item's words [2][nl - drop][N], or
// NULL).  rescale: the context's table.
struct DropOut {
  const uint64_t* rescale;
  int L, drop;
};

// Tensor products of paired ciphertexts at limbs 0..nl-1: out[b] = a[ia] x
// b[ib] for p = first + b.  With n_k > 0 the pairs are [group][i][j] (n_qk of
// them a group): ia = p / n_k, ib = (p / n_qk) * n_k + p % n_k.  Otherwise ia
// = p and ib = (p / ng) * n_grp + p % ng.  decay (optional): parts 0 and 1 get
// decay[p % n_row] * state[p] added ([2][nl][N], state_bstride apart).
struct PairArgs {
  const uint64_t *a, *b;
  uint64_t* out;  // [3][nl][N] per item
  uint64_t a_bstride, a_comp, b_bstride, b_comp;
  const uint64_t *decay, *state;
  uint64_t state_bstride;
  DropOut drop;
  const uint64_t* add;  // item p's at + p*add_bstride
  uint64_t add_bstride;
  const PrimeConst* prime;
  int log_n, nl, n_k, n_qk, ng, n_grp, n_row, first;
};
int launch_pair(Ctx* c, hipStream_t s, const PairArgs& a, int batch);

// Weighted prefix sums over tokens of one block: X[t][g] = init[g] +
// sum_{u <= t} w[u][(g0 + g) % n_row] * (k[u][g] x v[u][g]), three parts; k, v
// at token stride tok_stride; init may be NULL (zero).  last (optional)
// receives the last token's sums.
struct ScanArgs {
  const uint64_t *k, *v, *w;
  const uint64_t* init;  // [n_grp][3][nl][N]
  uint64_t* out;         // [n_tok][n_grp][3][nl][N], as DropOut says
  uint64_t* last;        // [n_grp][3][nl][N], may be init
  uint64_t tok_stride;
  DropOut drop;
  const uint64_t* add;   // group g's at + g * 2 * (nl - drop) * N
  const PrimeConst* prime;
  int log_n, nl, n_tok, n_grp, n_row, g0;
};
int launch_scan(Ctx* c, hipStream_t s, const ScanArgs& a);

// Masked weighted sums: for row b = (g, i), num[b] = sum_j m[g % n_row][j] *
// (a[b][j] x v[g][j]) (three parts, as DropOut says) and, when den is given,
// den[b] = sum_j m[g % n_row][j] * a[b][j]; m NULL: no mask.
struct MixArgs {
  const uint64_t *a, *v, *m;
  uint64_t *num, *den;
  DropOut drop;
  const PrimeConst* prime;
  int log_n, nl, n_q, n_k, n_row, first;  // first: index of row 0
};
int launch_mix(Ctx* c, hipStream_t s, const MixArgs& a, int rows);

}  // namespace ckks
