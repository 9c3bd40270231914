// Entry points of the attention calls: argument checks, and the composition of
// slotwise products (attn_kernels.hip), relinearisation and rescale (ops.hip)
// and the sum over a packed axis (sumrot.hip).  Items go in blocks (Hold).
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "attention.h"

namespace ckks {

namespace {

constexpr uint64_t kBlockItems = 1024;  // items of a block at most

// What a call may hold at once, read once a call: the words of a block of
// items, CKKS_BLOCK_MB of memory, by default 4 GiB of the card's 288 (some 40
// items at N = 2^16 and 24 limbs, enough to fill the chip many times); and of
// each stream's workspace, 2 GiB but no more than that.  One item is always
// held.
struct Hold {
  uint64_t block, step;
  Hold() {
    const char* e = getenv("CKKS_BLOCK_MB");
    const long mb = e ? atol(e) : 0;
    block = (uint64_t)(mb > 0 ? std::min(mb, 1l << 30) : 4096) << 17;
    step = std::min<uint64_t>(block, 1ull << 28);
  }
  int items(uint64_t per_item, uint64_t n) const {
    return (int)std::max<uint64_t>(1, std::min<uint64_t>({n, block / per_item, kBlockItems}));
  }
  // Words of the operand buffer for such blocks of a call's n items.
  uint64_t reserve(uint64_t per_item, uint64_t n) const {
    return held_words(per_item, std::min(n, kBlockItems), block);
  }
};

// Tells the context's buffers that this call's stream is being captured:
// growing then is an error, and buffers a capture has recorded are kept.
class CaptureScope {
 public:
  CaptureScope(Ctx* c, hipStream_t s) : c_(c) {
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (s && hipStreamIsCapturing(s, &st) == hipSuccess && st == hipStreamCaptureStatusActive)
      c->capturing = c->captured = true;
  }
  ~CaptureScope() { c_->capturing = false; }

 private:
  Ctx* c_;
};

struct Range {
  const void* p;
  uint64_t words;
};

// Every output against every input and against the other outputs.
int check_ranges(const std::vector<Range>& outs, const std::vector<Range>& ins) {
  for (const std::vector<Range>* v : {&outs, &ins})
    for (const Range& r : *v)
      if (misaligned(r.p)) return set_error(CKKS_EINVAL, "device buffers must be 16-byte aligned");
  for (size_t i = 0; i < outs.size(); ++i) {
    for (const Range& r : ins) REJECT_OVERLAP(outs[i].p, outs[i].words, r.p, r.words, "an input");
    for (size_t k = 0; k < i; ++k) REJECT_OVERLAP(outs[i].p, outs[i].words, outs[k].p, outs[k].words, "an output");
  }
  return CKKS_OK;
}

uint64_t key_words(const Ctx* c) { return (uint64_t)c->dnum * 2 * (c->L + c->K) * c->N; }

// Checks a plan and adds its keys to the inputs; *st receives it (no stages
// for NULL).
int check_steps(const Ctx* c, const ckks_sum_steps* steps, std::vector<Range>& ins, ckks_sum_steps* st) {
  memset(st, 0, sizeof(*st));
  if (!steps || steps->n_stage == 0) return CKKS_OK;
  *st = *steps;
  if (st->n_stage < 0 || st->n_stage > CKKS_SUM_MAX_STAGES) return set_error(CKKS_EINVAL, "bad number of sum stages");
  if (!st->radix || !st->galois_elts || !st->d_evks) return set_error(CKKS_EINVAL, "NULL list in the sum stages");
  int n = 0;
  for (int k = 0; k < st->n_stage; ++k) {
    if (st->radix[k] < 2 || st->radix[k] > CKKS_SUM_MAX_RADIX)
      return set_error(CKKS_EINVAL, "a sum stage's radix must be 2.." + std::to_string(CKKS_SUM_MAX_RADIX));
    n += st->radix[k] - 1;
  }
  for (int r = 0; r < n; ++r) {
    int rc = check_galois(c, st->galois_elts[r]);
    if (rc) return rc;
    if (st->galois_elts[r] == 1) return set_error(CKKS_EINVAL, "a sum stage's element is the identity");
    if (!st->d_evks[r]) return set_error(CKKS_EINVAL, "NULL key pointer");
    ins.push_back({st->d_evks[r], key_words(c)});
  }
  return CKKS_OK;
}

int check_count(uint64_t items) {
  return items > (1u << 24) ? set_error(CKKS_EINVAL, "too many ciphertexts in one call") : CKKS_OK;
}

// The steps after a product: relinearisation with its rescales, the sum.
struct Tail {
  Ctx* c;
  hipStream_t s;
  const uint64_t* rlk;
  ckks_sum_steps st;
  Hold hold;

  uint64_t limb(int l) const { return (uint64_t)(l + 1) * c->N; }
  DropOut drop_out(int drop) const { return DropOut{c->d_rescale, (int)c->L, drop}; }

  uint64_t* ws;  // reserved words of the context's workspace
  uint64_t ws_words;

  // Words of workspace that each step reserves for a call of n items;
  // relinearisations go in launches of as many items as fit (the items of a
  // launch share the key).
  int relin_items(int n, int level, int drop) const {
    const uint64_t fit = hold.step / ks_rescale_ws_words(c, level, drop);
    return (int)std::max<uint64_t>(1, std::min<uint64_t>({fit, (uint64_t)kMaxChunk, (uint64_t)n}));
  }
  uint64_t relin_words(int n, int level, int drop) const {
    return held_words(ks_rescale_ws_words(c, level, drop), std::min(n, kMaxChunk), hold.step);
  }
  uint64_t rescale_words(int n, int level) const {
    return held_words((uint64_t)c->N * (2 + 2 * level), std::min(n, kMaxChunk), hold.step);
  }
  uint64_t sum_words(int n, int level) const {
    return st.n_stage ? sum_ws_words(c, level, n, st.n_stage, hold.step) : 0;
  }

  // `main` words for this stream's steps, `side` more for Side's.
  int reserve(uint64_t main, uint64_t side = 0) {
    int rc = ensure_workspace(c, main + side);
    ws = c->ws;
    ws_words = main;
    return rc;
  }

  // n three-part items X ([3][level+1][N] each, written with drop_out(drop))
  // into out ([2][level+1-drop][N] each).
  int relin_rescale(const uint64_t* X, uint64_t* out, int n, int level, int drop) const {
    const int chunk = relin_items(n, level, drop);
    int rc = CKKS_OK;
    for (int b0 = 0; b0 < n && rc == CKKS_OK; b0 += chunk)
      rc = ks_rescale(c, s, level, drop, std::min(chunk, n - b0), X + b0 * 3 * limb(level), 3 * limb(level), rlk,
                      out + b0 * 2 * limb(level - drop), 2 * limb(level - drop), ws);
    return rc;
  }
  uint64_t mul_words(int n, int level) const {
    return held_words((uint64_t)c->N * (4 + 2 * level), std::min(n, kMaxChunk), hold.step);
  }
  // rescale(p in), n items; per item of the workspace the dropped limb's
  // product, its inverse transform, the converted limbs
  int mul_rescale(PlainMul m, int n) const {
    const uint64_t N = c->N, per = N * (4 + 2 * m.level);
    const int chunk = (int)std::max<uint64_t>(1, std::min<uint64_t>(kMaxChunk, ws_words / per));
    NttJobs jobs;
    for (int comp = 0; comp < 2; ++comp) jobs.add(comp, comp, m.level);
    int rc = CKKS_OK;
    for (m.first = 0; m.first < n && rc == CKKS_OK; m.first += chunk) {
      const int k = std::min(chunk, n - m.first);
      if ((rc = launch_plain_mul(c, s, m, ws, per, k)) ||
          (rc = ntt_run(c, s, ws, ws + 2 * N, per, per, k, jobs, true, true)) ||
          (rc = rescale_mul_fused(c, s, m, ws + 2 * N, ws + 4 * N, per, k)))
        break;
    }
    return rc;
  }
  int rescale(const uint64_t* R, uint64_t* Z, int n, int level) const {
    return rescale_batch(c, s, R, 2 * limb(level), Z, 2 * limb(level - 1), n, level, ws, ws_words);
  }
  // Where a step writes the n ciphertexts that sum() takes to out: there
  // already if the plan has no stages.
  uint64_t* before_sum(uint64_t* Z, uint64_t* out) const { return st.n_stage ? Z : out; }
  int sum(const uint64_t* Z, uint64_t* out, int n, int level) const {
    const uint64_t ct = 2 * limb(level);
    if (Z == out) return CKKS_OK;
    if (st.n_stage == 0) {
      CKKS_HIP_CHECK(hipMemcpyAsync(out, Z, ct * n * 8, hipMemcpyDeviceToDevice, s));
      return CKKS_OK;
    }
    return sum_stages(c, s, Z, ct, out, ct, n, level, st, ws, hold.step);
  }
};

// Steps that do not depend on the ones a Tail runs next, on an internal stream
// that starts where the Tail's stream is now; join() (or the end of the scope)
// makes that stream wait for them.  Two chains of launches that each leave the
// chip part empty then overlap: attn_mix with its normaliser, one after the
// other and so, takes 334 and 233 us for one row of 5 limbs at N = 2^13, 1229
// and 899 for one of 13 limbs at N = 2^16, 3640 and 3250 for six of them;
// linattn_chunk's r q beside the states 397 and 385 us for one token of 7 limbs
// at N = 2^14, 2369 and 2288 for 16 of 2^16.  Where the runtime puts both streams
// on one hardware queue nothing overlaps, and the events cost some 18 us a call.
class Side {
 public:
  Side(const Tail& t, uint64_t side_words) : tail(t), c_(t.c), s_(t.s) {
    rc = start();
    if (open_) tail.s = c_->lane[0];
    tail.ws = t.ws + t.ws_words;
    tail.ws_words = side_words;
  }
  ~Side() { (void)join(); }
  int join() {
    if (!open_) return CKKS_OK;
    open_ = false;
    CKKS_HIP_CHECK(hipEventRecord(c_->join_ev[0], tail.s));
    CKKS_HIP_CHECK(hipStreamWaitEvent(s_, c_->join_ev[0], 0));
    return CKKS_OK;
  }
  Tail tail;  // the steps, on the internal stream
  int rc;     // of the constructor

 private:
  int start() {
    if (internal_lanes() < 2) return CKKS_OK;  // on the caller's stream, one after the other
    int r = ensure_lanes(c_);
    if (r) return r;
    CKKS_HIP_CHECK(hipEventRecord(c_->fork_ev, s_));
    CKKS_HIP_CHECK(hipStreamWaitEvent(c_->lane[0], c_->fork_ev, 0));
    open_ = true;
    return CKKS_OK;
  }
  Ctx* c_;
  hipStream_t s_;
  bool open_ = false;
};

int rotate_sum(Ctx* c, const uint64_t* in, uint64_t* out, int batch, int level, const ckks_sum_steps* steps,
               hipStream_t s) {
  if (!in || !out || batch < 0) return set_error(CKKS_EINVAL, "NULL pointer or bad batch");
  int rc = check_level(c, level);
  if (rc) return rc;
  if (c->K == 0) return set_error(CKKS_EPARAM, "rotation needs special primes");
  const uint64_t ct = 2ull * (level + 1) * c->N;
  if ((rc = check_count(batch))) return rc;
  std::vector<Range> ins = {{in, ct * batch}};
  Tail t{c, s, nullptr, {}, {}, nullptr, 0};
  if ((rc = check_steps(c, steps, ins, &t.st)) || (rc = check_ranges({{out, ct * batch}}, ins))) return rc;
  if (t.st.n_stage == 0) return set_error(CKKS_EINVAL, "a sum needs at least one stage");
  if (batch == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  if ((rc = t.reserve(t.sum_words(batch, level)))) return rc;
  return t.sum(in, out, batch, level);
}

int attn_scores(Ctx* c, const uint64_t* q, int n_q, const uint64_t* k, int n_k, int n_grp, int level,
                const uint64_t* rlk, const ckks_sum_steps* steps, uint64_t* out, hipStream_t s) {
  if (!q || !k || !rlk || !out || n_q < 0 || n_k < 0 || n_grp < 0)
    return set_error(CKKS_EINVAL, "NULL pointer or bad count");
  int rc = check_level(c, level);
  if (rc) return rc;
  if (level == 0) return set_error(CKKS_ERANGE, "cannot rescale at level 0");
  if (c->K == 0) return set_error(CKKS_EPARAM, "relinearisation needs special primes");
  if ((rc = check_count((uint64_t)n_grp * n_q)) || (rc = check_count((uint64_t)n_grp * n_k)) ||
      (rc = check_count((uint64_t)n_grp * n_q * n_k)))
    return rc;
  const int items = n_grp * n_q * n_k, l = level;
  const uint64_t N = c->N, lim = (uint64_t)(l + 1) * N, zct = 2ull * l * N;
  std::vector<Range> ins = {{q, 2 * lim * n_grp * n_q}, {k, 2 * lim * n_grp * n_k}, {rlk, key_words(c)}};
  Tail t{c, s, rlk, {}, {}, nullptr, 0};
  if ((rc = check_steps(c, steps, ins, &t.st)) || (rc = check_ranges({{out, zct * items}}, ins))) return rc;
  if (items == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  const uint64_t per = 3 * lim + zct;
  const int block = t.hold.items(per, items);
  if ((rc = ensure_aux(c, t.hold.reserve(per, items)))) return rc;
  if ((rc = t.reserve(std::max(t.relin_words(items, l, 1), t.sum_words(items, l - 1))))) return rc;
  uint64_t *X = c->aux, *Z = X + 3 * lim * block;
  for (int b0 = 0; b0 < items; b0 += block) {
    const int n = std::min(block, items - b0);
    PairArgs a;
    memset(&a, 0, sizeof(a));
    a.a = q;
    a.b = k;
    a.out = X;
    a.a_bstride = a.b_bstride = 2 * lim;
    a.a_comp = a.b_comp = lim;
    a.drop = t.drop_out(1);
    a.prime = c->d_prime;
    a.log_n = (int)c->log_n;
    a.nl = l + 1;
    a.n_k = n_k;
    a.n_qk = n_q * n_k;
    a.n_row = 1;
    a.first = b0;
    uint64_t* dst = out + b0 * zct;
    Z = t.before_sum(Z, dst);
    if ((rc = launch_pair(c, s, a, n)) || (rc = t.relin_rescale(X, Z, n, l, 1)) || (rc = t.sum(Z, dst, n, l - 1))) return rc;
  }
  return CKKS_OK;
}

int attn_mix(Ctx* c, const uint64_t* a, int n_q, const uint64_t* v, int n_k, int n_grp, const uint64_t* mask,
             int n_mask, int level, const uint64_t* rlk, const ckks_sum_steps* steps, uint64_t* num, uint64_t* den,
             hipStream_t s) {
  if (!a || !v || !rlk || !num || n_q < 0 || n_k < 1 || n_grp < 0)
    return set_error(CKKS_EINVAL, "NULL pointer or bad count");
  if (mask ? n_mask < 1 || n_mask > std::max(n_grp, 1) : n_mask != 0)
    return set_error(CKKS_EINVAL, "the mask needs 1..n_grp rows (0 without a mask)");
  int rc = check_level(c, level);
  if (rc) return rc;
  const int l = level, drop = mask ? 2 : 1;  // levels num loses
  if (l < drop) return set_error(CKKS_ERANGE, "the level must be at least 2 with a mask, 1 without");
  if (c->K == 0) return set_error(CKKS_EPARAM, "relinearisation needs special primes");
  if ((rc = check_count((uint64_t)n_grp * n_k)) || (rc = check_count((uint64_t)n_grp * n_q)) ||
      (rc = check_count((uint64_t)n_grp * n_q * n_k)))
    return rc;
  const int rows = n_grp * n_q;
  const uint64_t N = c->N, lim = (uint64_t)(l + 1) * N;
  const uint64_t nct = 2ull * (l + 1 - drop) * N, dct = 2ull * (l + 2 - drop) * N, mid = 2ull * l * N;
  std::vector<Range> ins = {{a, 2 * lim * rows * n_k}, {v, 2 * lim * n_grp * n_k}, {rlk, key_words(c)}};
  if (mask) ins.push_back({mask, lim * n_mask * n_k});
  std::vector<Range> outs = {{num, nct * rows}};
  if (den) outs.push_back({den, dct * rows});
  Tail t{c, s, rlk, {}, {}, nullptr, 0};
  if ((rc = check_steps(c, steps, ins, &t.st)) || (rc = check_ranges(outs, ins))) return rc;
  if (rows == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  const uint64_t per = 3 * lim + 2 * lim + 2 * mid;
  const int block = t.hold.items(per, rows);
  if ((rc = ensure_aux(c, t.hold.reserve(per, rows)))) return rc;
  uint64_t *X = c->aux, *D = X + 3 * lim * block, *Z = D + 2 * lim * block, *Y = Z + mid * block;
  const int ld = mask ? l - 1 : l;  // den's level
  const uint64_t side_words = den ? std::max(mask ? t.rescale_words(rows, l) : 0, t.sum_words(rows, ld)) : 0;
  if ((rc = t.reserve(std::max(t.relin_words(rows, l, drop), t.sum_words(rows, l - drop)), side_words))) return rc;
  for (int b0 = 0; b0 < rows; b0 += block) {
    const int n = std::min(block, rows - b0);
    MixArgs m;
    memset(&m, 0, sizeof(m));
    m.a = a;
    m.v = v;
    m.m = mask;
    m.num = X;
    uint64_t *to = num + b0 * nct, *de = den ? den + b0 * dct : nullptr;
    Z = t.before_sum(Z, to);
    uint64_t* di = t.before_sum(mask ? Y : D, de);  // den before its sum
    m.den = !den ? nullptr : mask ? D : di;
    m.drop = t.drop_out(drop);
    m.prime = c->d_prime;
    m.log_n = (int)c->log_n;
    m.nl = l + 1;
    m.n_q = n_q;
    m.n_k = n_k;
    m.n_row = mask ? n_mask : 1;
    m.first = b0;
    if ((rc = launch_mix(c, s, m, n))) return rc;
    if (den && (mask || t.st.n_stage)) {  // the normaliser's steps beside the sum's
      Side side(t, side_words);
      if ((rc = side.rc) || (mask && (rc = side.tail.rescale(D, di, n, l))) || (rc = side.tail.sum(di, de, n, ld)))
        return rc;
      if ((rc = t.relin_rescale(X, Z, n, l, drop)) || (rc = t.sum(Z, to, n, l - drop)) || (rc = side.join())) return rc;
    } else if ((rc = t.relin_rescale(X, Z, n, l, drop)) || (rc = t.sum(Z, to, n, l - drop))) {
      return rc;
    }
  }
  return CKKS_OK;
}

// X (three parts, one rescale to come) = state x q at `level`, n items in rows
// of ng: q's item (t, g) at q + (t * n_grp + g)*q_bstride, read at its first
// level+1 limbs (components q_comp apart).
int state_times_q(const Tail& t, const uint64_t* state, const uint64_t* q, uint64_t q_bstride, uint64_t q_comp, int ng,
                  int n_grp, uint64_t* X, int n, int level) {
  PairArgs a;
  memset(&a, 0, sizeof(a));
  a.a = state;
  a.b = q;
  a.out = X;
  a.a_bstride = 2 * t.limb(level);
  a.a_comp = t.limb(level);
  a.b_bstride = q_bstride;
  a.b_comp = q_comp;
  a.drop = t.drop_out(1);
  a.prime = t.c->d_prime;
  a.log_n = (int)t.c->log_n;
  a.nl = level + 1;
  a.ng = ng;
  a.n_grp = n_grp;
  a.n_row = 1;
  return launch_pair(t.c, t.s, a, n);
}

// The outputs of a block of nt tokens x ng groups from the states' products X:
// relinearised into Z and summed into y, whose item (token, group) (0, 0) is
// item `at` of n_grp a token.
int outputs(const Tail& t, const uint64_t* X, uint64_t* Z, uint64_t* y, uint64_t at, int nt, int ng, int n_grp, int l) {
  const uint64_t yct = 2 * t.limb(l - 3);
  if (ng == n_grp) Z = t.before_sum(Z, y + at * yct);
  int rc = t.relin_rescale(X, Z, nt * ng, l - 2, 1);
  if (rc) return rc;
  if (ng == n_grp) return t.sum(Z, y + at * yct, nt * ng, l - 3);
  for (int i = 0; i < nt; ++i)  // a token's outputs are contiguous
    if ((rc = t.sum(Z + (uint64_t)i * ng * yct, y + (at + (uint64_t)i * n_grp) * yct, ng, l - 3))) return rc;
  return CKKS_OK;
}

int linattn_chunk(Ctx* c, const uint64_t* q, const uint64_t* k, const uint64_t* v, int n_tok, int n_grp,
                  const uint64_t* w, const uint64_t* r, const uint64_t* carry, int n_row, const uint64_t* state_in,
                  int level, const uint64_t* rlk, const ckks_sum_steps* steps, uint64_t* y, uint64_t* state_out,
                  hipStream_t s) {
  if (!q || !k || !v || !w || !rlk || !y || !state_out || n_tok < 1 || n_grp < 0)
    return set_error(CKKS_EINVAL, "NULL pointer or bad count");
  if (n_row < 1 || n_row > std::max(n_grp, 1)) return set_error(CKKS_EINVAL, "the weights need 1..n_grp rows");
  int rc = check_level(c, level);
  if (rc) return rc;
  const int l = level;
  if (l < 3) return set_error(CKKS_ERANGE, "the level must be at least 3");
  if (c->K == 0) return set_error(CKKS_EPARAM, "relinearisation needs special primes");
  if ((rc = check_count((uint64_t)n_tok * std::max(n_grp, 1)))) return rc;
  const uint64_t N = c->N, lim = (uint64_t)(l + 1) * N, items = (uint64_t)n_tok * n_grp;
  const uint64_t ct = 2 * lim, sct = 2ull * (l - 1) * N, yct = 2ull * (l - 2) * N, oct = carry ? yct : sct;
  std::vector<Range> ins = {{q, ct * items}, {k, ct * items}, {v, ct * items}, {w, lim * n_tok * n_row},
                            {rlk, key_words(c)}};
  if (r) ins.push_back({r, lim * n_tok * n_row});
  if (carry) ins.push_back({carry, sct / 2 * n_row});
  if (state_in) ins.push_back({state_in, sct * n_grp});
  Tail t{c, s, rlk, {}, {}, nullptr, 0};
  if ((rc = check_steps(c, steps, ins, &t.st)) ||
      (rc = check_ranges({{y, yct * items}, {state_out, oct * n_grp}}, ins)))
    return rc;
  if (n_grp == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  // per (token, group): X (then the state's product), C the rescaled r q, S
  // the states, Z the outputs before the sum; per group: the prefix sums carried
  // from one block of tokens to the next
  const uint64_t mid = 2ull * l * N, per = 3 * lim + (r ? mid : 0) + sct + yct;
  const int gb = t.hold.items(per + 3 * lim, n_grp);
  constexpr int kLaunch = 8192;  // items of one launch
  const int tb = std::min(t.hold.items((per + 3 * lim) * gb, n_tok), std::max(1, kLaunch / gb));
  const uint64_t nb = (uint64_t)gb * tb;
  const uint64_t most = per * std::min<uint64_t>(items, kLaunch) + 3 * lim * std::min<uint64_t>(n_grp, kBlockItems);
  if ((rc = ensure_aux(c, std::min(most, std::max(t.hold.block, per + 3 * lim))))) return rc;
  uint64_t *X = c->aux, *S = X + 3 * lim * nb, *Z = S + sct * nb, *C = Z + yct * nb, *P = C + (r ? mid * nb : 0);
  const int all = (int)items;
  const uint64_t side_words = std::max(r ? t.mul_words(all, l) : 0, carry ? t.mul_words(n_grp, l - 2) : 0);
  if ((rc = t.reserve(std::max({t.relin_words(all, l, 2), t.relin_words(all, l - 2, 1), t.sum_words(all, l - 3)}),
                      side_words)))
    return rc;
  for (int g0 = 0; g0 < n_grp; g0 += gb) {
    const int ng = std::min(gb, n_grp - g0);
    for (int t0 = 0; t0 < n_tok; t0 += tb) {
      const int nt = std::min(tb, n_tok - t0), n = nt * ng;
      const uint64_t at = (uint64_t)t0 * n_grp + g0;
      ScanArgs sc;
      memset(&sc, 0, sizeof(sc));
      sc.k = k + at * ct;
      sc.v = v + at * ct;
      sc.w = w + (uint64_t)t0 * n_row * lim;
      sc.init = t0 ? P : nullptr;
      sc.out = X;
      sc.last = t0 + nt < n_tok ? P : nullptr;
      sc.tok_stride = (uint64_t)n_grp * ct;
      sc.drop = t.drop_out(2);
      sc.add = state_in ? state_in + g0 * sct : nullptr;
      sc.prime = c->d_prime;
      sc.log_n = (int)c->log_n;
      sc.nl = l + 1;
      sc.n_tok = nt;
      sc.n_grp = ng;
      sc.n_row = n_row;
      sc.g0 = g0;
      const uint64_t* qt = q + at * ct;
      if (r) {  // rescale(r q) beside the states
        Side side(t, side_words);
        if ((rc = side.rc) ||
            (rc = side.tail.mul_rescale(
                 {qt, r + (uint64_t)t0 * n_row * lim, C, ct, lim, mid, l, ng, n_grp, n_row, g0, 0}, n)))
          return rc;
        if ((rc = launch_scan(c, s, sc)) || (rc = t.relin_rescale(X, S, n, l, 2)) || (rc = side.join())) return rc;
        if ((rc = state_times_q(t, S, C, mid, mid / 2, 1, 1, X, n, l - 2))) return rc;
      } else if ((rc = launch_scan(c, s, sc)) || (rc = t.relin_rescale(X, S, n, l, 2)) ||
                 (rc = state_times_q(t, S, qt, ct, lim, ng, n_grp, X, n, l - 2))) {
        return rc;
      }
      const uint64_t* last = S + (uint64_t)(nt - 1) * ng * sct;
      const bool end = t0 + nt == n_tok;
      if (end && !carry)
        CKKS_HIP_CHECK(hipMemcpyAsync(state_out + g0 * sct, last, sct * ng * 8, hipMemcpyDeviceToDevice, s));
      if (end && carry) {  // rescale(carry S) beside the outputs
        Side side(t, side_words);
        if ((rc = side.rc) ||
            (rc = side.tail.mul_rescale({last, carry, state_out + g0 * yct, sct, sct / 2, yct, l - 2, ng, ng, n_row, g0, 0},
                                        ng)) ||
            (rc = outputs(t, X, Z, y, at, nt, ng, n_grp, l)) ||
            (rc = side.join()))
          return rc;
      } else if ((rc = outputs(t, X, Z, y, at, nt, ng, n_grp, l))) {
        return rc;
      }
    }
  }
  return CKKS_OK;
}

int linattn_step(Ctx* c, const uint64_t* q, const uint64_t* k, const uint64_t* v, int n_grp, const uint64_t* decay,
                 int n_row, const uint64_t* state_in, int level, const uint64_t* rlk, const ckks_sum_steps* steps,
                 uint64_t* y, uint64_t* state_out, hipStream_t s) {
  if (!q || !k || !v || !rlk || !y || !state_out || n_grp < 0)
    return set_error(CKKS_EINVAL, "NULL pointer or bad count");
  if (decay ? n_row < 1 || n_row > std::max(n_grp, 1) : n_row != 0)
    return set_error(CKKS_EINVAL, "the decay needs 1..n_grp rows (0 without a decay)");
  int rc = check_level(c, level);
  if (rc) return rc;
  const int l = level;
  if (l < 2) return set_error(CKKS_ERANGE, "the level must be at least 2");
  if (c->K == 0) return set_error(CKKS_EPARAM, "relinearisation needs special primes");
  if ((rc = check_count(n_grp))) return rc;
  const uint64_t N = c->N, lim = (uint64_t)(l + 1) * N, ct = 2 * lim, sct = 2ull * l * N, yct = 2ull * (l - 1) * N;
  const uint64_t in_ct = decay ? ct : sct;
  std::vector<Range> ins = {{q, ct * n_grp}, {k, ct * n_grp}, {v, ct * n_grp}, {rlk, key_words(c)}};
  if (decay) ins.push_back({decay, lim * n_row});
  if (state_in) ins.push_back({state_in, in_ct * n_grp});
  Tail t{c, s, rlk, {}, {}, nullptr, 0};
  if ((rc = check_steps(c, steps, ins, &t.st)) ||
      (rc = check_ranges({{y, yct * n_grp}, {state_out, sct * n_grp}}, ins)))
    return rc;
  if (n_grp == 0) return CKKS_OK;
  CaptureScope cap(c, s);
  const uint64_t per = 3 * lim + yct;
  const int block = t.hold.items(per, n_grp);
  if ((rc = ensure_aux(c, t.hold.reserve(per, n_grp)))) return rc;
  if ((rc = t.reserve(std::max({t.relin_words(n_grp, l, 1), t.relin_words(n_grp, l - 1, 1), t.sum_words(n_grp, l - 2)}))))
    return rc;
  uint64_t *X = c->aux, *Z = X + 3 * lim * block;
  for (int b0 = 0; b0 < n_grp; b0 += block) {
    const int n = std::min(block, n_grp - b0);
    PairArgs a;
    memset(&a, 0, sizeof(a));
    a.a = k;
    a.b = v;
    a.out = X;
    a.a_bstride = a.b_bstride = ct;
    a.a_comp = a.b_comp = lim;
    if (state_in && decay) {
      a.decay = decay;
      a.state = state_in;
      a.state_bstride = ct;
    } else if (state_in) {
      a.add = state_in;
      a.add_bstride = sct;
    }
    a.drop = t.drop_out(1);
    a.prime = c->d_prime;
    a.log_n = (int)c->log_n;
    a.nl = l + 1;
    a.ng = a.n_grp = 1;
    a.n_row = decay ? n_row : 1;
    a.first = b0;
    uint64_t* S = state_out + b0 * sct;
    if ((rc = launch_pair(c, s, a, n)) || (rc = t.relin_rescale(X, S, n, l, 1))) return rc;
    uint64_t* yb = y + b0 * yct;
    Z = t.before_sum(Z, yb);
    if ((rc = state_times_q(t, S, q + b0 * ct, ct, lim, 1, 1, X, n, l - 1)) || (rc = t.relin_rescale(X, Z, n, l - 1, 1)) ||
        (rc = t.sum(Z, yb, n, l - 2)))
      return rc;
  }
  return CKKS_OK;
}

}  // namespace
}  // namespace ckks

using namespace ckks;

// The composition uses host containers; a failed host allocation is reported
// like a failed device one.
#define NO_THROW(call)                                                          \
  try {                                                                         \
    return call;                                                                \
  } catch (const std::exception&) {                                             \
    return set_error(CKKS_ENOMEM, "out of memory"); /* short: not allocated */  \
  }

extern "C" {

int ckks_rotate_sum(ckks_ctx* ctx, const uint64_t* d_ct_in, uint64_t* d_ct_out, int batch, int level,
                    const ckks_sum_steps* steps, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(rotate_sum(ctx, d_ct_in, d_ct_out, batch, level, steps, stream));
}

int ckks_attn_scores(ckks_ctx* ctx, const uint64_t* d_q, int n_q, const uint64_t* d_k, int n_k, int n_grp, int level,
                     const uint64_t* d_rlk, const ckks_sum_steps* steps, uint64_t* d_s, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(attn_scores(ctx, d_q, n_q, d_k, n_k, n_grp, level, d_rlk, steps, d_s, stream));
}

int ckks_attn_mix(ckks_ctx* ctx, const uint64_t* d_a, int n_q, const uint64_t* d_v, int n_k, int n_grp,
                  const uint64_t* d_mask, int n_mask, int level, const uint64_t* d_rlk, const ckks_sum_steps* steps,
                  uint64_t* d_num, uint64_t* d_den, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(attn_mix(ctx, d_a, n_q, d_v, n_k, n_grp, d_mask, n_mask, level, d_rlk, steps, d_num, d_den, stream));
}

int ckks_linattn_chunk(ckks_ctx* ctx, const uint64_t* d_q, const uint64_t* d_k, const uint64_t* d_v, int n_tok,
                       int n_grp, const uint64_t* d_w, const uint64_t* d_r, const uint64_t* d_carry, int n_row,
                       const uint64_t* d_state_in, int level, const uint64_t* d_rlk, const ckks_sum_steps* steps,
                       uint64_t* d_y, uint64_t* d_state_out, ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(linattn_chunk(ctx, d_q, d_k, d_v, n_tok, n_grp, d_w, d_r, d_carry, n_row, d_state_in, level, d_rlk, steps,
                         d_y, d_state_out, stream));
}

int ckks_linattn_step(ckks_ctx* ctx, const uint64_t* d_q, const uint64_t* d_k, const uint64_t* d_v, int n_grp,
                      const uint64_t* d_decay, int n_row, const uint64_t* d_state_in, int level,
                      const uint64_t* d_rlk, const ckks_sum_steps* steps, uint64_t* d_y, uint64_t* d_state_out,
                      ckks_stream_t stream) {
  CTX_OR_FAIL(ctx);
  NO_THROW(linattn_step(ctx, d_q, d_k, d_v, n_grp, d_decay, n_row, d_state_in, level, d_rlk, steps, d_y, d_state_out,
                        stream));
}

}  // extern "C"
