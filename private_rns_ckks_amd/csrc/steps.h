// Host pieces that the composed calls share (attention.hip, linear.hip,
// layernorm.hip): argument checks, the blocks a call goes in, the buffers it
// holds and the steps after a product.
#pragma once
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <exception>
#include <vector>

#include "attention.h"

namespace ckks {

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
inline int check_ranges(const std::vector<Range>& outs, const std::vector<Range>& ins) {
  for (const std::vector<Range>* v : {&outs, &ins})
    for (const Range& r : *v)
      if (misaligned(r.p)) return set_error(CKKS_EINVAL, "device buffers must be 16-byte aligned");
  for (size_t i = 0; i < outs.size(); ++i) {
    for (const Range& r : ins) REJECT_OVERLAP(outs[i].p, outs[i].words, r.p, r.words, "an input");
    for (size_t k = 0; k < i; ++k) REJECT_OVERLAP(outs[i].p, outs[i].words, outs[k].p, outs[k].words, "an output");
  }
  return CKKS_OK;
}

inline uint64_t key_words(const Ctx* c) { return (uint64_t)c->dnum * 2 * (c->L + c->K) * c->N; }

// Checks a plan and adds its keys to the inputs; *st receives it (no stages
// for NULL).
inline int check_steps(const Ctx* c, const ckks_sum_steps* steps, std::vector<Range>& ins, ckks_sum_steps* st) {
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

inline int check_count(uint64_t items) {
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

}  // namespace ckks

// The composition uses host containers; a failed host allocation is reported
// like a failed device one.
#define NO_THROW(call)                                                          \
  try {                                                                         \
    return call;                                                                \
  } catch (const std::exception&) {                                             \
    return set_error(CKKS_ENOMEM, "out of memory"); /* short: not allocated */  \
  }
