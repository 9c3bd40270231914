// Host pieces shared by the translation units that hold entry points:
// argument checks and the batched steps composed from the kernels.
#pragma once
#include "kernels.h"

namespace ckks {

// Items whose workspace the batched calls of ops.hip hold at once, at most.
constexpr int kBatchItems = 32;

int check_level(const Ctx* c, int level);
int check_galois(const Ctx* c, uint32_t g);

// Rescale of `batch` items: in [2][level+1][N] at in + b*in_stride -> out
// [2][level][N], plus the constants add0 (component 0) and acc (same layout
// as out, may equal it) when given; ws holds at least one item's
// N * (2 + 2 level) words.
int rescale_batch(Ctx* c, hipStream_t s, const uint64_t* in, uint64_t in_stride, uint64_t* out, uint64_t out_stride,
                  int batch, int level, uint64_t* ws, uint64_t ws_words, const uint64_t* add0 = nullptr,
                  const uint64_t* acc = nullptr);

// Internal streams a call may use at once (CKKS_LANES); 1: none, everything runs
// on the caller's.
int internal_lanes();

// device buffers are read and written with 16-byte vector accesses
inline bool misaligned(const void* p) { return ((uintptr_t)p & 15) != 0; }

// True when the word ranges [a, a + a_words) and [b, b + b_words) share a
// byte.  Outputs are written by some workgroups while other workgroups still
// read (and gather) the inputs, so an output that overlaps an input or a key
// would race; such calls are rejected before any launch.
inline bool overlap(const void* a, uint64_t a_words, const void* b, uint64_t b_words) {
  if (!a || !b || !a_words || !b_words) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + b_words * 8 && b0 < a0 + a_words * 8;
}

}  // namespace ckks

#define REJECT_OVERLAP(a, an, b, bn, what) \
  if (overlap((a), (an), (b), (bn))) return set_error(CKKS_EINVAL, "output overlaps " what)

#define CTX_OR_FAIL(ctx)                                             \
  if (!(ctx)) return set_error(CKKS_EINVAL, "ctx is NULL");         \
  if (hipSetDevice((ctx)->device) != hipSuccess) return set_error(CKKS_EHIP, "hipSetDevice failed")
