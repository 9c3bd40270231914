// Entry point of the encrypted linear layer: argument checks, constants, and
// the product (matmul_kernels.hip) with its rescales (rescale.hip).
#include "linear.h"

#include "steps.h"

namespace ckks {

namespace {

constexpr int kMaxIn = 1 << 16;       // |digit| |w| n_in <= 2^7 2^7 2^16 stays in 31 bits
constexpr uint64_t kGroup = 1 << 15;  // items of a launch at most

int matmul_i8(Ctx* c, const uint64_t* x, int n_blk, int n_in, const int8_t* w, int n_out, int level, double scale,
              const double* scales, const uint64_t* tok, int n_tok, double tok_scale, const double* bias, unsigned flags,
              uint64_t* y, double* out_scale, hipStream_t s) {
  if (!x || !w || !y || !out_scale || n_blk < 0 || n_out < 0) return set_error(CKKS_EINVAL, "NULL pointer or bad count");
  if (n_in < 1 || n_in > kMaxIn) return set_error(CKKS_EINVAL, "n_in must be 1.." + std::to_string(kMaxIn));
  if (flags & ~(CKKS_W_TRANSPOSED | CKKS_SCALE_IN)) return set_error(CKKS_EINVAL, "unknown flag");
  if (!scales && (flags & CKKS_SCALE_IN)) return set_error(CKKS_EINVAL, "CKKS_SCALE_IN without scales");
  if (tok ? n_tok < 1 || n_tok > std::max(n_blk, 1) : n_tok != 0)
    return set_error(CKKS_EINVAL, "the token scales need 1..n_blk rows (0 without them)");
  int rc = check_level(c, level);
  if (rc) return rc;
  const int l = level, nl = l + 1, drop = (scales != nullptr) + (tok != nullptr), low = nl - drop;
  if (low < 1) return set_error(CKKS_ERANGE, "the level must be at least the number of rescales");
  if ((rc = check_count((uint64_t)n_blk * n_in)) || (rc = check_count((uint64_t)n_blk * n_out)) ||
      (rc = check_count((uint64_t)n_in * n_out >> 8)))
    return rc;
  double s_out = scale;
  if (scales && tok)
    s_out = s_out * tok_scale / (double)c->mod[l - 1];
  else if (tok)
    s_out = s_out * tok_scale / (double)c->mod[l];
  if (!positive(scale) || (tok && !positive(tok_scale)) || !positive(s_out))
    return set_error(CKKS_EINVAL, "the scales must be positive");
  const bool in = flags & CKKS_SCALE_IN;
  // Constants of the outputs and, with CKKS_SCALE_IN, the inputs; the dropped
  // primes' inverses go with either.
  const int n_ki = in ? n_in : 0, n_k = scales && !in ? n_out : 1;
  std::vector<Whole> ki(n_ki), k(n_k, Whole{1, 0}), kb(bias ? n_out : 0);
  for (int j = 0; scales && j < (in ? n_ki : n_k); ++j)
    if (Whole* v = in ? &ki[j] : &k[j]; !whole(scales[j] * (double)c->mod[l], v) || v->e)
      return set_error(CKKS_EINVAL, "a rounded channel scale reaches 2^62");
  for (size_t j = 0; j < kb.size(); ++j)
    if (!whole(bias[j] * s_out, &kb[j]) || kb[j].e) return set_error(CKKS_EINVAL, "a rounded bias reaches 2^62");
  const uint64_t N = c->N, ct = 2ull * nl * N, oct = 2ull * low * N;
  std::vector<Range> ins = {{x, ct * n_blk * n_in}};
  if (tok) ins.push_back({tok, ct / 2 * n_tok});
  if ((rc = check_ranges({{y, oct * n_blk * n_out}}, ins))) return rc;
  // The matrix is read byte by byte and may lie anywhere: the words it touches.
  const uintptr_t w0 = (uintptr_t)w & ~(uintptr_t)7, w1 = ((uintptr_t)w + (uint64_t)n_in * n_out + 7) & ~(uintptr_t)7;
  REJECT_OVERLAP(y, oct * n_blk * n_out, (const void*)w0, (w1 - w0) / 8, "an input");
  *out_scale = s_out;
  if (n_blk == 0 || n_out == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  const Hold hold;
  // Items go in groups of whole blocks, or of a block's outputs where one
  // block's dropped limbs do not fit.
  const uint64_t top = 2ull * drop * N, items = (uint64_t)n_blk * n_out;
  const int fit = (int)std::min<uint64_t>({items, kGroup, std::max<uint64_t>(1, drop ? hold.block / top : items)});
  const int gj = std::min(fit, n_out), gb = std::min(n_blk, std::max(1, fit / n_out));
  const uint64_t w_per = 2ull * nl * N;
  const uint64_t pack_words = matmul_pack_words(n_in, n_out), kw = const_words(n_k, nl), iw = const_words(n_ki, nl);
  const uint64_t bw = const_words((int)kb.size(), nl);
  const uint64_t tops = drop ? held_words(top, std::min(items, kGroup), hold.block) : 0;
  const uint64_t step = drop ? held_words(w_per, std::min<uint64_t>(items, kMaxProducts), hold.step) : 0;
  auto even = [](uint64_t v) { return (v + 1) & ~1ull; };  // 16-byte parts
  if ((rc = ensure_aux(c, tops + even(pack_words) + kw + iw + bw)) || (drop && (rc = ensure_workspace(c, step)))) return rc;
  uint64_t *T = c->aux, *pack = T + tops, *tk = pack + even(pack_words), *ti = tk + kw, *tb = ti + iw;
  const ConstTable tables[] = {{k.data(), n_k, nl, in ? 0 : drop, tk}, {ki.data(), n_ki, nl, drop, ti},
                               {kb.data(), (int)kb.size(), nl, 0, tb}};
  if ((rc = launch_consts(c, s, tables, 3))) return rc;
  MatArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.w = w;
  a.kin = in ? ti : nullptr;
  a.kout = tk;
  a.bias = bias && drop == 0 ? tb : nullptr;
  a.n_kout = n_k;
  a.tok = tok;
  a.top = T;
  a.prime = c->d_prime;
  a.w_row = flags & CKKS_W_TRANSPOSED ? 1 : n_in;
  a.w_col = flags & CKKS_W_TRANSPOSED ? n_out : 1;
  a.log_n = (int)c->log_n;
  a.nl = nl;
  a.drop = drop;
  a.n_in = n_in;
  a.n_out = n_out;
  a.n_tok = n_tok;
  for (a.b0 = 0; a.b0 < n_blk; a.b0 += gb)
    for (a.j0 = 0; a.j0 < n_out; a.j0 += gj) {
      a.nb = std::min(gb, n_blk - a.b0);
      a.nj = std::min(gj, n_out - a.j0);
      a.out = y + ((uint64_t)a.b0 * n_out + a.j0) * oct;
      if ((rc = launch_matmul(c, s, a, pack))) return rc;
      if (!drop) continue;
      const ProductRescale p{T, a.out, a.nb * a.nj, l, drop, bias ? tb : nullptr, n_out, a.j0};
      if ((rc = rescale_products(c, s, p, c->ws, step))) return rc;
    }
  return CKKS_OK;
}

}  // namespace
}  // namespace ckks

using namespace ckks;

extern "C" {

int ckks_matmul_i8(ckks_ctx* ctx, const uint64_t* d_x, int n_blk, int n_in, const int8_t* d_w, int n_out, int level,
                   double scale, const double* scales, const uint64_t* d_tok, int n_tok, double tok_scale,
                   const double* bias, unsigned flags, uint64_t* d_y, double* out_scale, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(matmul_i8(ctx, d_x, n_blk, n_in, d_w, n_out, level, scale, scales, d_tok, n_tok, tok_scale, bias, flags, d_y,
                     out_scale, stream));
}

}  // extern "C"
