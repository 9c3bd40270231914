/*
 * ckks.h -- C ABI of the MI355X (gfx950) RNS-CKKS rotation hot-path library
 * (libckks_mi355x.so).
 *
 * What it computes.  The AEGIS pages on gist.science ("Problem" section,
 * challenges 2 and 3; "Methodology", communication hiding) state that
 * encrypted Transformer inference runs CKKS over a residue number system and
 * that key switching and rotation, needed by every matrix product and
 * non-linear layer, dominate the work; the FFN layer does local polynomial
 * multiplication and attention computes Q x K^T ("Methodology", items 2 and
 * 3).  The pages give no formula, so every call follows the standard full-RNS
 * CKKS construction with hybrid key switching (Cheon-Kim-Kim-Song 2017;
 * Cheon-Han-Kim-Kim-Song 2018; Han-Ki 2020; fast basis conversion of
 * Bajard-Eynard-Hasan-Zucca 2016; diagonal matvec of Halevi-Shoup 2014).
 *
 * Conventions shared by every call
 *   Words      uint64, one residue per word, fully reduced to [0, m) on entry
 *              and on exit.  Inputs with a word >= its modulus are undefined.
 *   Basis      q_0 .. q_{L-1} (ciphertext primes), then p_0 .. p_{K-1}
 *              (special primes).  A level-l polynomial holds limbs q_0..q_l.
 *   Limb       N consecutive words (one residue polynomial); arrays are
 *              limb-major: [..][limb][N].
 *   NTT form   word j of a limb is the polynomial evaluated at
 *              psi^(2*brv(j)+1) (bit-reversed evaluation order), psi the
 *              limb's 2N-th root of unity (by default the smallest primitive
 *              one).  Ciphertexts, keys and plaintexts are in NTT form.
 *   Ciphertext [2][l+1][N]: component 0 = c0, component 1 = c1; decryption
 *              is c0 + c1*s.
 *   Switch key [dnum][2][L+K][N]: digit j, component 0 = b, 1 = a, with
 *              b_j + a_j*s = e_j + [P]_{m_t} * s' on the limbs t of digit j
 *              (digit j = q_{j*alpha} .. q_{(j+1)*alpha-1}, alpha =
 *              ceil(L/dnum)) and b_j + a_j*s = e_j elsewhere; P = prod p_k.
 *              At level l the same key is used with limbs l+1..L-1 skipped.
 *   Galois     elements are odd integers in [1, 2N); X -> X^g.  The library
 *              has no slot convention: a left rotation by k slots in the
 *              usual encoding is g = 5^k mod 2N.
 *   Memory     d_* arguments are device pointers (HIP), owned by the caller,
 *              not retained after the call's stream work completes, each
 *              16-byte aligned (CKKS_EINVAL otherwise; hipMalloc gives 256)
 *              unless it holds bytes.
 *              Host arrays (galois element lists, key pointer lists) are
 *              read before the call returns.
 *   Streams    every compute call enqueues on `stream` and returns; outputs
 *              are valid after the stream is synchronised.  A context is not
 *              thread-safe: use one context per host thread / stream.
 *   Aliasing   ckks_ntt works in place; every other call requires its
 *              outputs not to overlap its inputs.
 *   Errors     every call returns CKKS_OK (0) or a negative CKKS_E* code; a
 *              detail string is kept per host thread (ckks_last_error).  No
 *              C++ exception crosses this interface.  On error no output is
 *              written unless the code is CKKS_EHIP (a failed launch may
 *              leave outputs partially written).
 */
#ifndef CKKS_MI355X_H
#define CKKS_MI355X_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* ckks_stream_t; /* a hipStream_t; NULL = the null stream */

enum {
  CKKS_OK = 0,
  CKKS_EINVAL = -1,    /* null or misaligned pointer, bad count, even or out-of-range Galois element */
  CKKS_ERANGE = -2,    /* level out of range, rescale at level 0, limb range outside the basis */
  CKKS_ENOMEM = -3,    /* device or host allocation failed */
  CKKS_EHIP = -4,      /* HIP launch or API failure */
  CKKS_EPARAM = -5,    /* invalid parameter set */
  CKKS_EINTERNAL = -6  /* internal error */
};

/* flags */
#define CKKS_ROT_ACCUMULATE 1u /* ckks_rotate: out = in + Rot(in) */
#define CKKS_NO_RESCALE 2u     /* ckks_mul_relin_rescale / ckks_ptmatvec: keep level l */
#define CKKS_W_TRANSPOSED 4u   /* ckks_matmul_i8: d_w is [n_in][n_out] */
#define CKKS_SCALE_IN 8u       /* ckks_matmul_i8: the channel scales are the inputs' */

typedef struct ckks_ctx ckks_ctx;

typedef struct {
  uint32_t log_n;      /* N = 2^log_n, 10 <= log_n <= 16 */
  uint32_t n_q;        /* L: ciphertext primes, 1..64 */
  uint32_t n_p;        /* K: special primes, 0..16; when K > 0, K == ceil(L/dnum) */
  uint32_t dnum;       /* gadget digits, 1..L; when K > 0, ceil(L/dnum) <= 16 */
  const uint64_t* q;   /* host [n_q]: distinct primes, each = 1 mod 2N, < 2^62 */
  const uint64_t* p;   /* host [n_p]: distinct primes, each = 1 mod 2N, < 2^62 */
  const uint64_t* psi; /* host [n_q+n_p] primitive 2N-th roots, or NULL = smallest ones */
} ckks_params;

/* ---- host-only set-up (no GPU needed) ---------------------------------- */

/* The `count` largest primes below 2^bits that are 1 mod 2^(log_n+1), in
 * descending order, written to out[count] (host).  bits in [log_n+2, 62].
 * Parameter set-up for the benchmark parameter reading (largest NTT-friendly
 * primes); CKKS_EPARAM if fewer exist. */
int ckks_find_primes(uint32_t log_n, uint32_t bits, uint32_t count, uint64_t* out);

/* Checks a parameter set: sizes, primality (deterministic Miller-Rabin),
 * q = 1 mod 2N, distinctness, the K == ceil(L/dnum) rule and, when given,
 * that each psi is a primitive 2N-th root.  Returns CKKS_OK or CKKS_EPARAM. */
int ckks_params_validate(const ckks_params* params);

const char* ckks_strerror(int status);
const char* ckks_last_error(void); /* detail of this thread's last failure ("" if none) */

/* ---- context ------------------------------------------------------------- */

/* Validates params, selects HIP device `hip_device`, and uploads the
 * per-prime twiddle tables and basis-conversion constants.  *out owns that
 * device memory plus a workspace grown on demand. */
int ckks_ctx_create(const ckks_params* params, int hip_device, ckks_ctx** out);
int ckks_ctx_destroy(ckks_ctx* ctx);
/* The roots in use (n_q+n_p values, host). */
int ckks_ctx_psi(const ckks_ctx* ctx, uint64_t* out);

/* ---- kernel timing trace (profiling aid) ------------------------------------ */

typedef struct {
  int32_t launches;  /* traced launches since ckks_trace_begin */
  double total_ms;   /* sum of their durations (HIP events on the launch stream) */
  double work_units; /* algorithmic work of those launches, in 64-bit modmul-class
                        operations: one NTT butterfly, one 64x64-bit multiply-
                        accumulate, one modular reduction or one constant
                        multiplication each count 1 */
} ckks_trace_stats;

/* Start tracing the kernel family `kernel`: every later launch of it on any
 * stream is bracketed by a HIP event pair on that stream.  Families:
 * "ntt_pass" (plain NTT / inverse NTT passes), the key switch's fused
 * passes "intt_row_gather" (automorphism gather + inverse row pass),
 * "ip_special" (forward row pass + key inner product on the special limbs +
 * inverse row pass of the accumulators), "comb_ip" (forward row pass + key
 * inner product on the ciphertext limbs + final combination) and
 * "ntt_row_combine" (forward row pass + final combination, hoisted
 * rotations), "automorph", "modup",
 * "moddown_conv", "rescale", "tensor", "ptmac", "ctmac", "add",
 * "const_mul", "term_mac" (polynomial evaluation's constant multiples),
 * "ip_gather", "sum_ip" (inner product of a stage of ckks_rotate_sum),
 * "attn_mac" (slotwise products of the attention calls), "matmul_i8" (products
 * of ckks_matmul_i8; a multiply-accumulate of a word and a byte counts 1),
 * "layernorm" (slotwise products of the layer norm calls).  NULL or "" stops tracing.
 * Tracing adds two event records per traced launch and nothing else. */
int ckks_trace_begin(ckks_ctx* ctx, const char* kernel);
/* Waits for the recorded events, returns the totals and stops tracing. */
int ckks_trace_end(ckks_ctx* ctx, ckks_trace_stats* out);

/* ---- hot path ------------------------------------------------------------ */

/* Source: AEGIS summary (gist.science), "Problem", challenge 2: ciphertexts
 * live as RNS residue polynomials (one per modulus of the chain) and the
 * matrix products and non-linear layers run key switching and rotation on
 * them; the negacyclic NTT per residue polynomial is the transform every one
 * of those operations is built on (the pages name no transform; standard
 * full-RNS CKKS).
 * Negacyclic NTT (inverse = 0) or inverse NTT with the 1/N factor
 * (inverse = 1), in place, on d_data = [npoly][n_limb][N]; limb i of every
 * polynomial uses basis prime limb_begin + i.  Forward maps coefficient form
 * to NTT form (bit-reversed evaluation order), inverse maps back.
 * CKKS_ERANGE if limb_begin + n_limb exceeds L+K. */
int ckks_ntt(ckks_ctx* ctx, uint64_t* d_data, int npoly, int limb_begin, int n_limb, int inverse,
             ckks_stream_t stream);

/* Source: AEGIS summary, "Problem", challenge 2 (rotations are frequent in
 * the matrix products and non-linear layers) and "Methodology", item 4
 * (rotations by several offsets, reordered); the automorphism X -> X^g is the
 * slot permutation of a rotation.
 * Galois automorphism X -> X^g on d_in = [npoly][level+1][N] (limbs
 * q_0..q_level) into d_out (same shape).  domain 0: NTT form (a permutation
 * of words); domain 1: coefficient form (a signed permutation). */
int ckks_automorph(ckks_ctx* ctx, const uint64_t* d_in, uint64_t* d_out, int npoly, int level, uint32_t galois_elt,
                   int domain, ckks_stream_t stream);

/* Source: AEGIS summary, "Problem", challenge 2 (key switching is needed by
 * every matrix product and non-linear layer and couples all RNS components)
 * and "Methodology", item 1 (the components that take part in one key switch
 * are kept together on one device: the whole switch runs in one place, as
 * here).
 * Hybrid key switch of d_poly ([level+1][N], NTT form) with the switch key
 * d_evk ([dnum][2][L+K][N]) into d_out ([2][level+1][N], NTT form):
 * per active digit, ModUp (unsigned fast basis conversion to the other limbs
 * and the special primes), NTT, inner product with the key digit, then
 * ModDown (centered conversion of the special part, multiply by P^-1).
 * Requires K > 0. */
int ckks_keyswitch(ckks_ctx* ctx, const uint64_t* d_poly, const uint64_t* d_evk, uint64_t* d_out, int level,
                   ckks_stream_t stream);

/* Source: AEGIS summary, "Problem", challenge 2 (rotation with key
 * switching in every matrix product and non-linear layer) and
 * "Methodology", item 4 (several rotations with different offsets in flight
 * at once: here a batch, one offset and key per ciphertext).
 * Batched homomorphic rotation: for b < batch, ciphertext b of d_ct_in
 * ([batch][2][level+1][N]) is mapped by Galois element galois_elts[b]
 * (host array) and key-switched back with the switch key d_evks[b] (host
 * array of device pointers, each [dnum][2][L+K][N], the key for
 * tau_g(s) -> s): out = (tau_g(c0) + k0, k1), (k0, k1) = KS(tau_g(c1)).
 * galois element 1 is the identity (copy, no key read; its key pointer may
 * be NULL).  With CKKS_ROT_ACCUMULATE, out = in + Rot(in). */
int ckks_rotate(ckks_ctx* ctx, const uint64_t* d_ct_in, uint64_t* d_ct_out, int batch, int level,
                const uint32_t* galois_elts, const uint64_t* const* d_evks, unsigned flags, ckks_stream_t stream);

/* Allocation-free variant of ckks_rotate, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  Same arguments, checks and output words as
 * ckks_rotate; the difference is where the key-switch workspace comes from
 * and where the work runs:
 *   - the workspace is a library-owned device array of
 *     CKKS_NOALLOC_SCRATCH_BYTES per GPU (held from the first context
 *     created on that GPU until the process ends), not a buffer grown with
 *     hipMalloc; the call makes no allocation of any kind (device, host
 *     pinned, streams or events; kernel tracing is off for it);
 *   - every kernel runs on `stream` in order, in chunks of as many
 *     ciphertexts as the scratch holds (no internal streams).
 * CKKS_ERANGE if one ciphertext's workspace at `level` exceeds the scratch
 * (at N = 2^16 with 24 + 8 primes and dnum = 3 one ciphertext at level 23
 * takes 92 MiB: N x (24 + 3 x 32 + 2 x 8 + 2 x 24) words).  All calls on one GPU share that GPU's scratch: calls that
 * overlap in time on one GPU (other streams, other threads) race and give
 * wrong words.  Nothing in the scratch needs clearing between calls. */
#define CKKS_NOALLOC_SCRATCH_BYTES (128ull << 20)
int ckks_rotate_noalloc(ckks_ctx* ctx, const uint64_t* d_ct_in, uint64_t* d_ct_out, int batch, int level,
                        const uint32_t* galois_elts, const uint64_t* const* d_evks, unsigned flags,
                        ckks_stream_t stream);

/* Hoisted rotations (AEGIS page, "Methodology", item 4: several rotations of
 * one ciphertext): each of the n_in ciphertexts of d_ct_in
 * ([n_in][2][level+1][N]) is rotated by every galois_elts[r] (host array,
 * r < n_rot) with the switch key d_evks[r] (host array of device pointers)
 * into d_ct_out ([n_in][n_rot][2][level+1][N]).  The digits of c1 are raised
 * to the extended basis and transformed once per ciphertext; each rotation
 * then applies tau_g to those extended limbs (an NTT-form permutation) before
 * the inner product, so out = (tau_g(c0) + k0, k1) with (k0, k1) the key
 * switch of tau_g(c1) whose decomposition is tau_g of c1's.  The result
 * decrypts like ckks_rotate's but its words differ: the automorphism's sign
 * changes meet the raised digit rather than the digit.  Galois element 1 is
 * a copy (its key pointer may be NULL).  Requires K > 0. */
int ckks_rotate_hoisted(ckks_ctx* ctx, const uint64_t* d_ct_in, int n_in, int level, int n_rot,
                        const uint32_t* galois_elts, const uint64_t* const* d_evks, uint64_t* d_ct_out,
                        ckks_stream_t stream);

/* Rescale (divide by q_level, rounding to nearest) of d_in
 * ([batch][2][level+1][N]) into d_out ([batch][2][level][N]).
 * CKKS_ERANGE at level 0. */
int ckks_rescale(ckks_ctx* ctx, const uint64_t* d_in, uint64_t* d_out, int batch, int level, ckks_stream_t stream);

/* Source: AEGIS summary, "Methodology", item 3 (self-attention: the product
 * Q x K^T of two encrypted operands, followed by a polynomial softmax, which
 * needs the product relinearised and rescaled).
 * Batched ciphertext product: tensor (d0 = a0 b0, d1 = a0 b1 + a1 b0,
 * d2 = a1 b1), relinearisation with d_rlk (switch key s^2 -> s):
 * (d0, d1) + KS(d2), then rescale.  d_a, d_b: [batch][2][level+1][N];
 * d_out: [batch][2][level][N], or [batch][2][level+1][N] with
 * CKKS_NO_RESCALE.  Requires K > 0; CKKS_ERANGE when rescaling at level 0. */
int ckks_mul_relin_rescale(ckks_ctx* ctx, const uint64_t* d_a, const uint64_t* d_b, const uint64_t* d_rlk,
                           uint64_t* d_out, int batch, int level, unsigned flags, ckks_stream_t stream);

/* Polynomial p(x) = sum_{k<=degree} coeffs[k] x^k (host doubles) on each of
 * the batch ciphertexts d_ct_in ([batch][2][level+1][N], NTT form, scale
 * `scale`), by Horner's rule (the polynomial approximations of the nonlinear
 * layers, AEGIS page "Methodology" and the Nimbus post; no scheme is given):
 *   acc = c_d * x         every limb times K = round(c_d * q_level), rescale
 *                         (the scale stays `scale`)
 *   acc += c_{d-1}        round(c_{d-1} * s_acc) added to c0 in NTT form
 *   for k = d-2 .. 0      acc = rescale(relin(acc * x)) with x restricted to
 *                         acc's limbs, s_acc = s_acc * scale / q_l (l the
 *                         level of acc before the product); acc += c_k
 * Rounding is llround; the constants must stay below 2^62 (CKKS_EINVAL).
 * d_ct_out: [batch][2][level-degree+1][N]; *out_scale receives the output
 * scale.  Needs 1 <= degree <= level and K > 0 (d_rlk: the s^2 -> s key).
 * The scale should be close to the primes so the rescales keep it. */
int ckks_poly_eval(ckks_ctx* ctx, const uint64_t* d_ct_in, int batch, int level, double scale, const double* coeffs,
                   int degree, const uint64_t* d_rlk, uint64_t* d_ct_out, double* out_scale, ckks_stream_t stream);

/* Source: AEGIS summary, "Methodology", items 2-3 (the nonlinear layers,
 * GELU and the softmax exponential, evaluated locally as polynomial
 * approximations) and the Nimbus post on non-linear layers (the exponential's
 * inputs concentrate on [-4, 0]); neither fixes an evaluation scheme.
 * Polynomial p(x) = sum_{k<=degree} coeffs[k] x^k (host doubles, power
 * basis) in E = ceil(log2(degree + 1)) levels (Horner's takes degree), by the
 * baby-step / giant-step split with every scale fixed top-down:
 *   powers y_0 = x, y_j = y_(j-1)^2 (multiply, relinearise with d_rlk,
 *   rescale): level l - j, scale s_j = s_(j-1)^2 / q_(l-j+1);
 *   eval(c[0..n-1], level t, scale T), n counting up to the last nonzero
 *   coefficient:
 *     n <= 1: the trivial ciphertext (llround(c0 T), 0);
 *     n = 2:  x's limbs 0..t+1 times K = llround(c1 T q_(t+1) / s), rescaled
 *             by q_(t+1), plus llround(c0 T);
 *     n > 2:  g = 2^(ceil(log2 n) - 1), p = hi(x) y_j + lo(x) with
 *             y_j = x^g, lo = c[0..g-1], hi = c[g..n-1]; lo is evaluated at
 *             (t, T) (or is the constant llround(c0 T)); a one-coefficient hi
 *             multiplies y_j's limbs 0..t+1 by llround(c T q_(t+1) / s_j) and
 *             rescales; otherwise hi is evaluated at (t+1, T q_(t+1) / s_j),
 *             multiplied by y_j at level t+1, relinearised and rescaled;
 *   output = eval(c, l - E, scale): level l - E, scale `scale`.
 * Doubles combine left to right as written; zero coefficients cost nothing.
 * d_ct_in: [batch][2][level+1][N], NTT form; d_ct_out:
 * [batch][2][level - E + 1][N].  CKKS_ERANGE unless 1 <= degree <= 64 and
 * level >= E; CKKS_EINVAL when a constant reaches 2^62 (checked before any
 * work is enqueued).  Needs K > 0.  The powers and intermediates live in a
 * context-owned buffer grown on demand (growing it synchronises the device);
 * otherwise the call only enqueues work on `stream`. */
int ckks_poly_eval_tree(ckks_ctx* ctx, const uint64_t* d_ct_in, int batch, int level, double scale,
                        const double* coeffs, int degree, const uint64_t* d_rlk, uint64_t* d_ct_out,
                        double* out_scale, ckks_stream_t stream);

/* Source: AEGIS summary, "Methodology", item 2 (FFN: each device multiplies
 * its encrypted activations by the weight slices of one output group, locally,
 * as polynomial products); the diagonal (BSGS) method is the standard way to
 * run that product on packed slots (Halevi-Shoup 2014).
 * Baby-step / giant-step ciphertext x plaintext matrix-vector product.
 *   d_x      [n_in][2][level+1][N] input ciphertexts
 *   d_diags  [n_out][n_in][n2][n1][level+1][N] plaintexts (NTT form); entry
 *            (o, c, g, b) is the diagonal for offset n1*g + b, already
 *            rotated by the inverse of giant step g
 *   baby     n1-1 Galois elements / switch keys for the baby steps 1..n1-1
 *   giant    n2-1 Galois elements / switch keys for the giant steps 1..n2-1
 *   d_y      [n_out][2][level][N] (level+1 with CKKS_NO_RESCALE)
 * y_o = sum_g Rot_g( sum_c sum_b diag(o,c,g,b) * Rot_b(x_c) ), then rescale.
 * The baby-step rotations are computed once and shared by all outputs, as
 * hoisted rotations of each input (ckks_rotate_hoisted).  The intermediate
 * ciphertexts live in a context-owned buffer grown on demand (growing it
 * synchronises the device); otherwise the call only enqueues work. */
int ckks_ptmatvec(ckks_ctx* ctx, const uint64_t* d_x, int n_in, const uint64_t* d_diags, int n_out, int n1, int n2,
                  const uint32_t* baby_galois, const uint64_t* const* d_evk_baby, const uint32_t* giant_galois,
                  const uint64_t* const* d_evk_giant, uint64_t* d_y, int level, unsigned flags,
                  ckks_stream_t stream);

/* Baby-step / giant-step matrix-vector product with encrypted weights: the
 * attention output A x V, where the softmax weights A arrive encrypted
 * (AEGIS page, "Methodology", self-attention: the weights are gathered and
 * multiplied with V; no packing is given, so this is the diagonal method of
 * ckks_ptmatvec with ciphertext diagonals).
 *   d_x      [n_in][2][level+1][N] input ciphertexts (V)
 *   d_diags  [n_out][n_in][n2][n1][2][level+1][N] ciphertexts (A's
 *            diagonals); entry (o, c, g, b) is the diagonal for offset
 *            n1*g + b, already rotated by the inverse of giant step g
 *   d_rlk    [dnum][2][L+K][N] switching key for s^2
 *   baby / giant  Galois elements and keys as in ckks_ptmatvec
 *   d_y      [n_out][2][level][N] (level+1 with CKKS_NO_RESCALE)
 * T_og = sum_c sum_b tensor(diag(o,c,g,b), Rot_b(x_c)) (three parts, summed
 * before one relinearisation per (o, g)); y_o = sum_g Rot_g(relin(T_og)),
 * then rescale.  Buffers and errors as in ckks_ptmatvec; K > 0. */
int ckks_ctmatvec(ckks_ctx* ctx, const uint64_t* d_x, int n_in, const uint64_t* d_diags, int n_out, int n1, int n2,
                  const uint64_t* d_rlk, const uint32_t* baby_galois, const uint64_t* const* d_evk_baby,
                  const uint32_t* giant_galois, const uint64_t* const* d_evk_giant, uint64_t* d_y, int level,
                  unsigned flags, ckks_stream_t stream);

/* ---- attention on packed heads ------------------------------------------------
 *
 * The products of an attention layer whose operands are all ciphertexts.  The
 * calls work slot by slot and on sums over a packed axis; the packing is the
 * caller's.  A layout that serves all of them keeps the summed index
 * outermost: slot = f * (n/F) + r for F features f, r running over (head,
 * token) or (head, value feature); the rotations by multiples of n/F then sum
 * exactly over f, cyclically, and leave the sum in every f.
 *
 * Scales follow from the operations: a product multiplies them, a rescale
 * divides by the dropped prime.  Sums need equal scales; the caller sees to
 * it.  Level l operands hold limbs q_0..q_l.
 *
 * Plaintext rows (masks, weights, decays) are in NTT form, one per head group:
 * item g of n_grp uses row g mod n_rows, so groups that share their heads'
 * constants (the sequences of a batch, in the order [sequence][head group])
 * share the rows.  A row of zeros removes its term: a padded token or key
 * block, or a sequence that is empty altogether, contributes nothing, and
 * sums over nothing decrypt to zero (there is no division).
 *
 * Buffers and streams: intermediates live in the context's buffers, grown on
 * demand; growing synchronises the device.  A call holds 4 GiB of operands and
 * a workspace of 2 GiB (two for ckks_attn_mix and ckks_linattn_chunk) at most,
 * or a single item's if that is more; the environment variable CKKS_BLOCK_MB,
 * read at each call, lowers both limits to that many MiB, or raises the first.
 * ckks_attn_mix with a normaliser
 * and ckks_linattn_chunk with read weights or a carry also use one of the
 * context's internal streams, which their first call creates; the work on it
 * starts and ends with the call's place on the caller's stream.  A call no
 * larger than an earlier one with the same optional operands (no more limbs,
 * groups, items, tokens or stages in any count) allocates and creates nothing
 * and may be captured into a graph; any other returns CKKS_EHIP while its
 * stream is capturing if it would have to.  Buffers a
 * capture has recorded stay allocated until the context is destroyed, so a
 * captured call stays valid while larger calls follow.  Replays use the
 * context like calls do: one at a time. */

#define CKKS_SUM_MAX_RADIX 32
#define CKKS_SUM_MAX_STAGES 16

/* Sum over a packed axis, in stages.  Stage s turns x into
 *   x + sum_{r < radix[s]-1} Rot_{g_r}(x),
 * its radix[s]-1 elements and keys following those of the stages before it.
 * For an axis of length prod(radix) at stride d, stage s holds the rotations
 * by d_s, 2 d_s, .., (radix[s]-1) d_s with d_s = d * radix[0] * .. *
 * radix[s-1].  One decomposition and one ModDown serve a whole stage:
 *   D_j     raised digits of c1, as in ckks_rotate_hoisted
 *   U       = sum_r sum_j tau_{g_r}(D_j) * evk_{r,j}    (extended basis)
 *   out     = (c0 + sum_r tau_{g_r}(c0) + ModDown(U_0), c1 + ModDown(U_1))
 * so a stage of radix 8 takes about half the time of the same sum by three
 * calls of ckks_rotate with CKKS_ROT_ACCUMULATE, for 7 keys instead of 3. */
typedef struct {
  int n_stage;                    /* 0..CKKS_SUM_MAX_STAGES */
  const int* radix;               /* host [n_stage], each 2..CKKS_SUM_MAX_RADIX */
  const uint32_t* galois_elts;    /* host [sum(radix) - n_stage], none of them 1 */
  const uint64_t* const* d_evks;  /* host list of switch keys, one per element */
} ckks_sum_steps;

/* Source: AEGIS summary, "Problem", challenge 2 and "Methodology", items 3-4
 * (rotations aggregate the partial products of Q x K^T; several offsets of one
 * ciphertext are in flight at once).
 * Sum of each of the batch ciphertexts d_ct_in ([batch][2][level+1][N]) by
 * `steps` into d_ct_out (same shape).  Needs n_stage >= 1 and K > 0. */
int ckks_rotate_sum(ckks_ctx* ctx, const uint64_t* d_ct_in, uint64_t* d_ct_out, int batch, int level,
                    const ckks_sum_steps* steps, ckks_stream_t stream);

/* Source: AEGIS summary, "Methodology", item 3 (self-attention: Q x K^T on
 * encrypted operands); cross attention takes K from an encoder's states, of
 * another length.
 * Scores of every query ciphertext against every key ciphertext of its group:
 *   s[g][i][j] = Sum(rescale(relin(q[g][i] x k[g][j])))
 *   d_q  [n_grp][n_q][2][level+1][N]     d_k  [n_grp][n_k][2][level+1][N]
 *   d_s  [n_grp][n_q][n_k][2][level][N]
 * d_rlk is the s^2 -> s key; `steps` with n_stage 0 (or NULL) leaves the
 * slotwise products unsummed.  The polynomial softmax between the scores and
 * ckks_attn_mix is ckks_poly_eval_tree.  CKKS_ERANGE at level 0. */
int ckks_attn_scores(ckks_ctx* ctx, const uint64_t* d_q, int n_q, const uint64_t* d_k, int n_k, int n_grp, int level,
                     const uint64_t* d_rlk, const ckks_sum_steps* steps, uint64_t* d_s, ckks_stream_t stream);

/* Source: AEGIS summary, "Methodology", item 3 (the weights multiplied with V
 * and summed).
 * Masked weighted sum of the value ciphertexts, and the sum of the weights:
 *   num[g][i] = Sum(rescale(rescale(relin(sum_j m_j a[g][i][j] x v[g][j]))))
 *   den[g][i] = Sum(rescale(sum_j m_j a[g][i][j]))
 *   d_a   [n_grp][n_q][n_k][2][level+1][N]   d_v  [n_grp][n_k][2][level+1][N]
 *   d_mask  [n_mask][n_k][level+1][N] plaintexts, 1 <= n_mask <= n_grp, or
 *         NULL with n_mask 0: no mask and one rescale less in each line
 *   d_num  [n_grp][n_q][2][level-1][N]  ([..][level][N] without a mask)
 *   d_den  [n_grp][n_q][2][level][N]    ([..][level+1][N] without a mask),
 *         or NULL
 * One relinearisation per (g, i).  The quotient num / den is the caller's (a
 * polynomial in den, or a division after decryption).  Needs n_k >= 1;
 * CKKS_ERANGE below level 2 with a mask, 1 without. */
int ckks_attn_mix(ckks_ctx* ctx, const uint64_t* d_a, int n_q, const uint64_t* d_v, int n_k, int n_grp,
                  const uint64_t* d_mask, int n_mask, int level, const uint64_t* d_rlk, const ckks_sum_steps* steps,
                  uint64_t* d_num, uint64_t* d_den, ckks_stream_t stream);

/* Linear attention with a decay for each head, chunked form: n_tok tokens of
 * a prompt at once (attention without the softmax, which needs no polynomial
 * approximation; the pages' attention, AEGIS summary, "Methodology", item 3,
 * keeps it).  Per group g and token t, slotwise on a state whose slots hold
 * the outer products of key and value features:
 *   X_t   = sum_{u <= t} w_u (k_u x v_u)          three parts, not relinearised
 *   S_t   = state_in + rescale(rescale(relin(X_t)))               level-2
 *   y_t   = Sum(rescale(relin(rescale(r_t q_t) x S_t)))           level-3
 *   state_out = rescale(carry S_{n_tok-1})  (level-3), or S_{n_tok-1} (level-2)
 * With decay gamma per head, w_u = gamma^-(u+1), r_t = gamma^(t+1) and carry =
 * gamma^n_tok: y_t reads r_t S_t = gamma^(t+1) state_in + sum_{u <= t}
 * gamma^(t-u) k_u v_u, the state that ckks_linattn_step with d_decay = gamma
 * forms token by token from state_in, the state after the token before the
 * chunk; state_out is that state after token n_tok-1, which the next chunk or
 * step takes.  Decays that change from token to token: w_u = 1 / (d_0 .. d_u),
 * r_t = d_0 .. d_t, carry = d_0 .. d_(n_tok-1).  The state takes two levels
 * (carried on: three) however many tokens the chunk has.
 * How long a chunk may be: S_t is held up to gamma^-n_tok times larger than
 * the state it stands for, h = n_tok log2(1 / gamma) bits for the smallest
 * gamma (18.5 for 0.875 and 96 tokens).  They are taken twice: from the
 * modulus (the largest slot of S_t times its scale stays below q_0 .. q_(l-2)
 * / 2, and of state_out's product before its rescale likewise), and from the
 * precision: the errors of r_t q_t (the rescale's, and r_t's and carry's
 * rounding to their scale) are multiplied by S_t, so outputs and carried
 * state keep h bits less than those of single steps.  A longer prompt goes in
 * several chunks, each from the state_out of the one before.
 *   d_q, d_k, d_v  [n_tok][n_grp][2][level+1][N]
 *   d_w, d_r       [n_tok][n_row][level+1][N] plaintexts; d_r may be NULL
 *                  (q_t's limbs 0..level-2 as they are)
 *   d_carry        [n_row][level-1][N] plaintexts, or NULL
 *   d_state_in     [n_grp][2][level-1][N], or NULL (zero)
 *   d_y            [n_tok][n_grp][2][level-2][N]
 *   d_state_out    [n_grp][2][level-1][N], with d_carry [n_grp][2][level-2][N]
 * Needs n_tok >= 1, 1 <= n_row <= n_grp; CKKS_ERANGE below level 3. */
int ckks_linattn_chunk(ckks_ctx* ctx, const uint64_t* d_q, const uint64_t* d_k, const uint64_t* d_v, int n_tok,
                       int n_grp, const uint64_t* d_w, const uint64_t* d_r, const uint64_t* d_carry, int n_row,
                       const uint64_t* d_state_in, int level, const uint64_t* d_rlk, const ckks_sum_steps* steps,
                       uint64_t* d_y, uint64_t* d_state_out, ckks_stream_t stream);

/* Recurrent form of the same, one token per group:
 *   with d_decay:  state_out = rescale(relin(k x v) + decay state_in)
 *   without:       state_out = state_in + rescale(relin(k x v))
 *   y = Sum(rescale(relin(q x state_out))), q at state_out's limbs
 *   d_q, d_k, d_v  [n_grp][2][level+1][N]
 *   d_decay        [n_row][level+1][N] plaintexts, 1 <= n_row <= n_grp, or
 *                  NULL with n_row 0 (the caller weighs k instead, and the
 *                  state keeps its level from token to token)
 *   d_state_in     [n_grp][2][level+1][N] with d_decay, [n_grp][2][level][N]
 *                  without, or NULL (zero: the first token)
 *   d_y            [n_grp][2][level-1][N]
 *   d_state_out    [n_grp][2][level][N]
 * CKKS_ERANGE below level 2. */
int ckks_linattn_step(ckks_ctx* ctx, const uint64_t* d_q, const uint64_t* d_k, const uint64_t* d_v, int n_grp,
                      const uint64_t* d_decay, int n_row, const uint64_t* d_state_in, int level,
                      const uint64_t* d_rlk, const ckks_sum_steps* steps, uint64_t* d_y, uint64_t* d_state_out,
                      ckks_stream_t stream);

/* ---- linear layers and layer norms, a ciphertext a feature ----------------------
 *
 * A block of tokens as one ciphertext for each feature, the tokens along the
 * slots (N/2 of them, of one sequence or several): x[b][i] is feature i of block
 * b.  Sums over features are sums of ciphertexts, so a linear layer and a layer
 * norm need no rotation; the calls of nonlinear layers (ckks_poly_eval_tree)
 * take the features as their batch.  Slots without a token hold anything; a
 * token row of zeros, or gradients of zero, keep them out of the results.  The
 * attention calls take features inside the slots; no call moves between the two.
 *
 * Real constants (scales, weights, biases) are host doubles, rounded to the
 * integer llround(v) next to them; from 2^62 on v is an integer itself.  They
 * enter the words exactly, so results are the operations below word for word.
 * An array may be shorter-lived than the work: it is read before the call
 * returns, and a captured graph replays its constants.
 *
 * Buffers, streams and captures as in the attention calls, whose limits
 * (CKKS_BLOCK_MB) hold here too: a call holds its operands' block, one
 * workspace and, on top, its constants (16 bytes each and limb) and for
 * ckks_matmul_i8 the matrix laid out for its kernel (up to 255 outputs and 127
 * inputs more).  No internal stream is used. */

/* Source: AEGIS summary, "Methodology", item 2 (each device multiplies its
 * encrypted activations by its slices of the weights, locally).
 * Product of encrypted features with a matrix of 8-bit integers:
 *   acc[b][j] = sum_i w[j][i] (k_i x[b][i])        k_i with CKKS_SCALE_IN, else 1
 *   y[b][j]   = rescale^d(tok[b % n_tok] k_j acc[b][j]) + round(bias[j] s_y)
 *   k         = round(scales[.] q_level)
 * d = (scales != NULL) + (d_tok != NULL) rescales, none without either.
 *   d_x     [n_blk][n_in][2][level+1][N]
 *   d_w     [n_out][n_in] bytes, with CKKS_W_TRANSPOSED [n_in][n_out], at any
 *           address (rows of a larger matrix, say)
 *   scales  [n_out], with CKKS_SCALE_IN [n_in], or NULL: none.  Each is rounded
 *           by up to 1 / (2 q_level), as k says; one that rounds to 0 is 0
 *   d_tok   [n_tok][level+1][N] plaintexts (a scale for each token), 1 <= n_tok
 *           <= n_blk, or NULL with n_tok 0.  A zero removes a token.
 *   bias    [n_out] or NULL; added to every slot, also to removed tokens'
 *   d_y     [n_blk][n_out][2][level+1-d][N], at scale s_y = *out_scale:
 *           scale; with d_tok alone scale tok_scale / q_level; with both
 *           scale tok_scale / q_(level-1)
 * The input's gradient of a layer y = diag(scales) w x is the same call on the
 * outputs' gradients with CKKS_W_TRANSPOSED | CKKS_SCALE_IN, and n_in, n_out
 * exchanged.  The noise of y is that of x, up to 128 n_in times as large.
 * 1 <= n_in <= 65536; CKKS_ERANGE below level d; CKKS_EINVAL for a constant of
 * 2^62 or more and for a scale (or a tok_scale of d_tok, or an s_y) that is not
 * positive and finite.  Needs no key and works with K = 0. */
int ckks_matmul_i8(ckks_ctx* ctx, const uint64_t* d_x, int n_blk, int n_in, const int8_t* d_w, int n_out, int level,
                   double scale, const double* scales, const uint64_t* d_tok, int n_tok, double tok_scale,
                   const double* bias, unsigned flags, uint64_t* d_y, double* out_scale, ckks_stream_t stream);

/* Layer norm over the features of each token, in two calls with the caller's
 * polynomial for 1 / sqrt between them (ckks_poly_eval_tree on d_var; the pages
 * replace nonlinear steps by polynomials, AEGIS summary, "Methodology", and fix
 * none).  First half, per block b with F = n_feat, exact in every word:
 *   S      = sum_i x_i
 *   var    = rescale(rescale(relin(k (F sum_i x_i (x) x_i - S (x) S)))) + round(eps scale)
 *   k      = round(q_l q_(l-1) / (F F) / scale)       l = level
 * F sum x^2 - S^2 = F^2 variance, so var holds variance + eps at scale `scale`,
 * two levels down, for one relinearisation a block.  eps may be any number:
 * eps - 1 hands the polynomial u = variance + eps - 1, small around a variance
 * of 1, where (1 + u)^-1/2 has small coefficients.
 *   d_x    [n_blk][n_feat][2][level+1][N] at `scale`
 *   d_sum  [n_blk][2][level+1][N], for ckks_layernorm
 *   d_var  [n_blk][2][level-1][N]
 * The sums need log2(F F) bits above a feature's square: F^2 times the largest
 * variance times scale^2 k stays below q_0 .. q_l / 2.  Rounding k moves var's
 * scale by up to 1 / (2 k) of itself, so k has to be 2^19 or more (2^-20): with
 * primes and a scale of b bits there is room for F^2 <= 2^(b-19), 45 features at
 * 30 bits, 1448 at 40.  1 <= n_feat <= 65536; CKKS_ERANGE below level 2;
 * CKKS_EINVAL when k is below 2^19 or a constant reaches 2^126. */
int ckks_layernorm_var(ckks_ctx* ctx, const uint64_t* d_x, int n_blk, int n_feat, int level, double scale, double eps,
                       const uint64_t* d_rlk, uint64_t* d_sum, uint64_t* d_var, ckks_stream_t stream);

/* Second half: with r = rstd[b], t = rstd_level,
 *   y_i = rescale(rescale(relin(k_i (F x_i - S) (x) r))) + round(beta_i scale)
 *   k_i = round(gamma_i (q_t q_(t-1) / (F rstd_scale)))
 * that is gamma_i (x_i - mean) rstd + beta_i, at scale `scale`.
 *   d_x, d_sum    as in ckks_layernorm_var (read at limbs 0..t)
 *   d_rstd        [n_blk][2][rstd_level+1][N] at rstd_scale, 2 <= rstd_level <= level
 *   gamma, beta   [n_feat], or NULL: 1, 0.  With both NULL y is the normalised
 *                 input that ckks_layernorm_grad takes; gamma and beta may then
 *                 enter the next ckks_matmul_i8 as its inputs' scales and bias.
 *   d_y           [n_blk][n_feat][2][rstd_level-1][N]
 * A weight gamma_i is rounded by up to F rstd_scale / (2 q_t q_(t-1)): that is
 * 2^-20 at most, CKKS_EINVAL otherwise.  One relinearisation a feature.  Errors as
 * above. */
int ckks_layernorm(ckks_ctx* ctx, const uint64_t* d_x, const uint64_t* d_sum, int n_blk, int n_feat, int level,
                   double scale, const uint64_t* d_rstd, int rstd_level, double rstd_scale, const double* gamma,
                   const double* beta, const uint64_t* d_rlk, uint64_t* d_y, ckks_stream_t stream);

/* Backward pass, from the outputs' gradients dy (scale s), the normalised input
 * xhat and r = rstd of the forward pass, l = level:
 *   k_i      = round(gamma_i (q_(l-3) q_(l-4) / (F rstd_scale)))
 *   G        = sum_i k_i dy_i
 *   H        = rescale(rescale(relin(sum_i k_i dy_i (x) xhat_i)))             level l-2
 *   R        = rescale(relin(c r (x) H)),                                     level l-3
 *   c        = round(q_l / xhat_scale * q_(l-1) / xhat_scale * q_(l-2))
 *   dx_i     = rescale(rescale(relin(r (x) (F k_i dy_i - G) - xhat_i (x) R)))   level l-5
 *   dgamma_i = Sum(rescale(relin(sum_b dy_i[b] (x) xhat_i[b])))                 level l-1
 *   dbeta_i  = Sum(sum_b dy_i[b])                                             level l
 * that is dx = rstd (g - mean(g) - xhat mean(g xhat)) with g = gamma dy, at
 * scale s (c makes both products' scales equal); dgamma at s xhat_scale / q_l;
 * dbeta at s.  Sum runs over the tokens of a ciphertext (`steps`, as in the
 * attention calls; NULL or no stages: the tokens' terms as they are).  Slots
 * without a token need dy = 0.
 *   d_dy      [n_blk][n_feat][2][level+1][N]
 *   d_xhat    [n_blk][n_feat][2][xhat_level+1][N], level <= xhat_level
 *   d_rstd    [n_blk][2][rstd_level+1][N], level <= rstd_level
 *   gamma     [n_feat] or NULL: 1
 *   d_dx      [n_blk][n_feat][2][level-4][N]      each may be NULL, but not
 *   d_dgamma  [n_feat][2][level][N]               all of them
 *   d_dbeta   [n_feat][2][level+1][N]
 * xhat and rstd are read at limbs 0..level.  With n_blk 0, dgamma and dbeta are
 * zero.  CKKS_ERANGE below level 5 with d_dx, 1 with d_dgamma; CKKS_EINVAL when c
 * or k (before gamma) is below 2^19, whose rounding would move dx by more than
 * 2^-20 of itself, or a constant reaches 2^126. */
int ckks_layernorm_grad(ckks_ctx* ctx, const uint64_t* d_dy, int n_blk, int n_feat, int level, const uint64_t* d_xhat,
                        int xhat_level, double xhat_scale, const uint64_t* d_rstd, int rstd_level, double rstd_scale,
                        const double* gamma, const uint64_t* d_rlk, const ckks_sum_steps* steps, uint64_t* d_dx,
                        uint64_t* d_dgamma, uint64_t* d_dbeta, ckks_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CKKS_MI355X_H */
