// Entry points of the layer norm calls: argument checks, constants, and the
// composition of their slotwise kernels (norm_kernels.hip) with relinearisation,
// rescale and the sum over a packed axis.  Items go in blocks (Hold).
#include "layernorm.h"

#include "steps.h"

namespace ckks {

namespace {

constexpr int kMaxFeat = 1 << 16;
constexpr Whole kOne{1, 0};

int check_norm(const Ctx* c, int n_blk, int n_feat, int level) {
  if (n_blk < 0) return set_error(CKKS_EINVAL, "bad count");
  if (n_feat < 1 || n_feat > kMaxFeat) return set_error(CKKS_EINVAL, "n_feat must be 1.." + std::to_string(kMaxFeat));
  int rc = check_level(c, level);
  if (rc) return rc;
  return check_count((uint64_t)n_blk * n_feat);
}

// Gains gamma_i kappa (kappa alone without gamma); *n receives their number.
int gains(const double* gamma, double kappa, int n_feat, std::vector<Whole>* k) {
  Whole one;
  if (!whole_factor(kappa, &one)) return set_error(CKKS_EINVAL, "the scales leave no room for the weights");
  k->assign(gamma ? n_feat : 1, one);
  for (int i = 0; gamma && i < n_feat; ++i)
    if (!whole(gamma[i] * kappa, &(*k)[i])) return set_error(CKKS_EINVAL, "a rounded weight reaches 2^126");
  return CKKS_OK;
}

int layernorm_var(Ctx* c, const uint64_t* x, int n_blk, int n_feat, int level, double scale, double eps,
                  const uint64_t* rlk, uint64_t* sum, uint64_t* var, hipStream_t s) {
  if (!x || !rlk || !sum || !var) return set_error(CKKS_EINVAL, "NULL pointer");
  int rc = check_norm(c, n_blk, n_feat, level);
  if (rc) return rc;
  const int l = level;
  if (l < 2) return set_error(CKKS_ERANGE, "the level must be at least 2");
  if (c->K == 0) return set_error(CKKS_EPARAM, "relinearisation needs special primes");
  if (!positive(scale)) return set_error(CKKS_EINVAL, "the scale must be positive");
  Whole k[3] = {{n_feat, 0}, {}, {}};
  const double f = n_feat;
  if (!whole_factor((double)c->mod[l] * (double)c->mod[l - 1] / (f * f) / scale, &k[1]))
    return set_error(CKKS_EINVAL, "the scale leaves no room for the variance");
  if (!whole(eps * scale, &k[2])) return set_error(CKKS_EINVAL, "the rounded eps reaches 2^126");
  const uint64_t N = c->N, lim = (uint64_t)(l + 1) * N, ct = 2 * lim, vct = 2ull * (l - 1) * N;
  if ((rc = check_ranges({{sum, ct * n_blk}, {var, vct * n_blk}}, {{x, ct * n_blk * n_feat}, {rlk, key_words(c)}})))
    return rc;
  if (n_blk == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  Tail t{c, s, rlk, {}, {}, nullptr, 0};
  const uint64_t per = 3 * lim, tw = const_words(3, l + 1), ow = const_words(1, l + 1);
  const int block = t.hold.items(per, n_blk);
  if ((rc = ensure_aux(c, tw + ow + t.hold.reserve(per, n_blk))) || (rc = t.reserve(t.relin_words(n_blk, l, 2)))) return rc;
  uint64_t *to = c->aux + tw, *X = to + ow;
  const ConstTable tables[] = {{k, 3, l + 1, 0, c->aux}, {&kOne, 1, l + 1, 2, to}};
  if ((rc = launch_consts(c, s, tables, 2))) return rc;
  for (int b0 = 0; b0 < n_blk; b0 += block) {
    const int n = std::min(block, n_blk - b0);
    const MomentArgs a{x + (uint64_t)b0 * n_feat * ct, sum + b0 * ct, X, c->aux, to, c->d_prime,
                       (int)c->log_n, l + 1, n_feat};
    if ((rc = launch_moments(c, s, a, n)) || (rc = t.relin_rescale(X, var + b0 * vct, n, l, 2))) return rc;
  }
  return CKKS_OK;
}

int layernorm(Ctx* c, const uint64_t* x, const uint64_t* sum, int n_blk, int n_feat, int level, double scale,
              const uint64_t* rstd, int rstd_level, double rstd_scale, const double* gamma, const double* beta,
              const uint64_t* rlk, uint64_t* y, hipStream_t s) {
  if (!x || !sum || !rstd || !rlk || !y) return set_error(CKKS_EINVAL, "NULL pointer");
  int rc = check_norm(c, n_blk, n_feat, level);
  if (rc) return rc;
  const int t_ = rstd_level;
  if (t_ < 2 || t_ > level) return set_error(CKKS_ERANGE, "rstd_level must be 2..level");
  if (c->K == 0) return set_error(CKKS_EPARAM, "relinearisation needs special primes");
  if (!positive(scale) || !positive(rstd_scale)) return set_error(CKKS_EINVAL, "the scales must be positive");
  std::vector<Whole> k, kb(beta ? n_feat : 0);
  if ((rc = gains(gamma, (double)c->mod[t_] * (double)c->mod[t_ - 1] / ((double)n_feat * rstd_scale), n_feat, &k)))
    return rc;
  for (size_t i = 0; i < kb.size(); ++i)
    if (!whole(beta[i] * scale, &kb[i])) return set_error(CKKS_EINVAL, "a rounded bias reaches 2^126");
  const uint64_t N = c->N, ct = 2ull * (level + 1) * N, lim = (uint64_t)(t_ + 1) * N, yct = 2ull * (t_ - 1) * N;
  const uint64_t items = (uint64_t)n_blk * n_feat;
  if ((rc = check_ranges({{y, yct * items}},
                         {{x, ct * items}, {sum, ct * n_blk}, {rstd, 2 * lim * n_blk}, {rlk, key_words(c)}})))
    return rc;
  if (n_blk == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  Tail t{c, s, rlk, {}, {}, nullptr, 0};
  const int nl = t_ + 1, n_k = (int)k.size();
  const uint64_t per = 3 * lim, kw = const_words(n_k, nl), bw = const_words((int)kb.size(), nl), fw = const_words(1, nl);
  const int block = t.hold.items(per, items);
  if ((rc = ensure_aux(c, kw + bw + 2 * fw + t.hold.reserve(per, items))) ||
      (rc = t.reserve(t.relin_words((int)items, t_, 2))))
    return rc;
  uint64_t *tk = c->aux, *tb = tk + kw, *tf = tb + bw, *to = tf + fw, *X = to + fw;
  const Whole feat{n_feat, 0};
  const ConstTable tables[] = {{k.data(), n_k, nl, 0, tk}, {kb.data(), (int)kb.size(), nl, 0, tb}, {&feat, 1, nl, 0, tf},
                               {&kOne, 1, nl, 2, to}};
  if ((rc = launch_consts(c, s, tables, 4))) return rc;
  for (uint64_t b0 = 0; b0 < items; b0 += block) {
    const int n = (int)std::min<uint64_t>(block, items - b0);
    const NormArgs a{x, sum, rstd, X, tk, beta ? tb : nullptr, tf, to, c->d_prime, (int)c->log_n, nl,
                     level + 1, n_feat, n_k, (int)b0, (int)b0 + n};
    if ((rc = launch_norm(c, s, a)) || (rc = t.relin_rescale(X, y + b0 * yct, n, t_, 2))) return rc;
  }
  return CKKS_OK;
}

int layernorm_grad(Ctx* c, const uint64_t* dy, int n_blk, int n_feat, int level, const uint64_t* xhat, int xhat_level,
                   double xhat_scale, const uint64_t* rstd, int rstd_level, double rstd_scale, const double* gamma,
                   const uint64_t* rlk, const ckks_sum_steps* steps, uint64_t* dx, uint64_t* dgamma, uint64_t* dbeta,
                   hipStream_t s) {
  if (!dy || !xhat || !rstd || !rlk || (!dx && !dgamma && !dbeta)) return set_error(CKKS_EINVAL, "NULL pointer");
  int rc = check_norm(c, n_blk, n_feat, level);
  if (rc) return rc;
  if ((rc = check_level(c, xhat_level)) || (rc = check_level(c, rstd_level))) return rc;
  const int l = level;
  if (xhat_level < l || rstd_level < l) return set_error(CKKS_ERANGE, "xhat_level and rstd_level must be at least level");
  if (l < (dx ? 5 : dgamma ? 1 : 0))
    return set_error(CKKS_ERANGE, "the level must be at least 5 with d_dx, 1 with d_dgamma");
  if (c->K == 0) return set_error(CKKS_EPARAM, "relinearisation needs special primes");
  if (dx && (!positive(xhat_scale) || !positive(rstd_scale)))
    return set_error(CKKS_EINVAL, "the scales must be positive");
  std::vector<Whole> k;
  Whole cr{};
  if (dx) {
    auto q = [&](int i) { return (double)c->mod[i]; };
    if ((rc = gains(gamma, q(l - 3) * q(l - 4) / ((double)n_feat * rstd_scale), n_feat, &k))) return rc;
    if (!whole_factor(q(l) / xhat_scale * q(l - 1) / xhat_scale * q(l - 2), &cr))
      return set_error(CKKS_EINVAL, "the scales leave no room for the gradient");
  }
  const uint64_t N = c->N, lim = (uint64_t)(l + 1) * N, ct = 2 * lim, items = (uint64_t)n_blk * n_feat;
  const uint64_t dct = 2ull * (dx ? l - 4 : 0) * N, gct = 2ull * l * N;
  std::vector<Range> ins = {{dy, ct * items}, {xhat, 2ull * (xhat_level + 1) * N * items},
                            {rstd, 2ull * (rstd_level + 1) * N * n_blk}, {rlk, key_words(c)}};
  std::vector<Range> outs;
  if (dx) outs.push_back({dx, dct * items});
  if (dgamma) outs.push_back({dgamma, gct * n_feat});
  if (dbeta) outs.push_back({dbeta, ct * n_feat});
  Tail t{c, s, rlk, {}, {}, nullptr, 0};
  if ((rc = check_steps(c, steps, ins, &t.st)) || (rc = check_ranges(outs, ins))) return rc;
  if (n_blk == 0 && !dgamma && !dbeta) return CKKS_OK;
  CaptureScope cap(c, s);
  // dx: per block G, H and R; then a block of items X.  dgamma, dbeta: X and
  // what is summed, a feature each.
  const int nl = l + 1, n_k = (int)k.size(), low = l - 2;  // low: limbs of the last product
  const uint64_t hct = 2ull * (l - 1) * N, rct = 2ull * low * N;
  const uint64_t kw = dx ? const_words(n_k, nl) : 0, fw = const_words(1, nl);
  const uint64_t per_blk = 3 * lim + rct + hct + rct, per_item = 3ull * std::max(low, 0) * N, per_feat = 3 * lim + ct;
  const int bb = dx ? t.hold.items(per_blk, n_blk) : 0, bi = dx ? t.hold.items(per_item, (uint64_t)bb * n_feat) : 0;
  const int bf = dgamma || dbeta ? t.hold.items(per_feat, n_feat) : 0;
  uint64_t need = 0, work = 0;
  if (dx) {
    need = kw + 5 * fw + t.hold.reserve(per_blk, n_blk) + t.hold.reserve(per_item, items);
    work = std::max({t.relin_words(n_blk, l, 2), t.relin_words(n_blk, l - 2, 1), t.relin_words((int)items, l - 3, 2)});
  }
  if (dgamma || dbeta) need = std::max(need, fw + t.hold.reserve(per_feat, n_feat));
  if (dgamma) work = std::max({work, (uint64_t)t.relin_words(n_feat, l, 1), t.sum_words(n_feat, l - 1)});
  if (dbeta) work = std::max(work, t.sum_words(n_feat, l));
  if ((rc = ensure_aux(c, need)) || (rc = t.reserve(work))) return rc;
  if (dx) {
    uint64_t *tk = c->aux, *tf = tk + kw, *tc = tf + fw, *t2 = tc + fw, *t1 = t2 + fw, *te = t1 + fw,
             *B = te + fw;
    uint64_t *X = B, *G = X + 3 * lim * bb, *H = G + rct * bb, *R = H + hct * bb, *Y = R + rct * bb;
    const Whole feat{n_feat, 0};
    const ConstTable tables[] = {{k.data(), n_k, nl, 0, tk}, {&feat, 1, nl, 0, tf},  {&cr, 1, l - 1, 0, tc},
                                 {&kOne, 1, nl, 2, t2},      {&kOne, 1, l - 1, 1, t1}, {&kOne, 1, low, 2, te}};
    if ((rc = launch_consts(c, s, tables, 6))) return rc;
    for (int b0 = 0; b0 < n_blk; b0 += bb) {
      const int nb = std::min(bb, n_blk - b0);
      const uint64_t *dyb = dy + (uint64_t)b0 * n_feat * ct, *rb = rstd + (uint64_t)b0 * 2 * (rstd_level + 1) * N;
      const uint64_t* xb = xhat + (uint64_t)b0 * n_feat * 2 * (xhat_level + 1) * N;
      const GradSumArgs a{dyb, xb, G, X, tk, t2, c->d_prime, (int)c->log_n, nl, xhat_level + 1, low,
                          n_feat, n_k};
      if ((rc = launch_grad_sums(c, s, a, nb)) || (rc = t.relin_rescale(X, H, nb, l, 2))) return rc;
      const ScaledPairArgs p{rb, H, X, t1, tc, c->d_prime, (int)c->log_n, l - 1, rstd_level + 1};
      if ((rc = launch_scaled_pair(c, s, p, nb)) || (rc = t.relin_rescale(X, R, nb, l - 2, 1))) return rc;
      for (int i0 = 0; i0 < nb * n_feat; i0 += bi) {
        const int n = std::min(bi, nb * n_feat - i0);
        const GradArgs g{dyb, xb, rb, G, R, Y, tk, tf, te, c->d_prime, (int)c->log_n, low, nl,
                         xhat_level + 1, rstd_level + 1, n_feat, n_k, i0, i0 + n};
        if ((rc = launch_grad(c, s, g)) ||
            (rc = t.relin_rescale(Y, dx + ((uint64_t)b0 * n_feat + i0) * dct, n, l - 3, 2)))
          return rc;
      }
    }
  }
  const ConstTable kept{&kOne, 1, nl, 1, c->aux};
  if (dgamma && (rc = launch_consts(c, s, &kept, 1))) return rc;
  for (int f0 = 0; (dgamma || dbeta) && f0 < n_feat; f0 += bf) {
    const int n = std::min(bf, n_feat - f0);
    uint64_t *X = c->aux + fw, *Z = X + 3 * lim * bf;
    uint64_t *tb = dbeta ? t.before_sum(Z, dbeta + f0 * ct) : nullptr;
    const WeightArgs a{dy, xhat, dgamma ? X : nullptr, tb, c->aux, c->d_prime, (int)c->log_n, nl,
                       xhat_level + 1, n_blk, n_feat, f0};
    if ((rc = launch_weight_sums(c, s, a, n)) || (dbeta && (rc = t.sum(tb, dbeta + f0 * ct, n, l)))) return rc;
    if (!dgamma) continue;
    uint64_t* tg = t.before_sum(Z, dgamma + f0 * gct);
    if ((rc = t.relin_rescale(X, tg, n, l, 1)) || (rc = t.sum(tg, dgamma + f0 * gct, n, l - 1))) return rc;
  }
  return CKKS_OK;
}

}  // namespace
}  // namespace ckks

using namespace ckks;

extern "C" {

int ckks_layernorm_var(ckks_ctx* ctx, const uint64_t* d_x, int n_blk, int n_feat, int level, double scale, double eps,
                       const uint64_t* d_rlk, uint64_t* d_sum, uint64_t* d_var, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(layernorm_var(ctx, d_x, n_blk, n_feat, level, scale, eps, d_rlk, d_sum, d_var, stream));
}

int ckks_layernorm(ckks_ctx* ctx, const uint64_t* d_x, const uint64_t* d_sum, int n_blk, int n_feat, int level,
                   double scale, const uint64_t* d_rstd, int rstd_level, double rstd_scale, const double* gamma,
                   const double* beta, const uint64_t* d_rlk, uint64_t* d_y, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(layernorm(ctx, d_x, d_sum, n_blk, n_feat, level, scale, d_rstd, rstd_level, rstd_scale, gamma, beta, d_rlk,
                     d_y, stream));
}

int ckks_layernorm_grad(ckks_ctx* ctx, const uint64_t* d_dy, int n_blk, int n_feat, int level, const uint64_t* d_xhat,
                        int xhat_level, double xhat_scale, const uint64_t* d_rstd, int rstd_level, double rstd_scale,
                        const double* gamma, const uint64_t* d_rlk, const ckks_sum_steps* steps, uint64_t* d_dx,
                        uint64_t* d_dgamma, uint64_t* d_dbeta, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(layernorm_grad(ctx, d_dy, n_blk, n_feat, level, d_xhat, xhat_level, xhat_scale, d_rstd, rstd_level,
                          rstd_scale, gamma, d_rlk, steps, d_dx, d_dgamma, d_dbeta, stream));
}

}  // extern "C"
