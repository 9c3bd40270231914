// Sum over a packed axis: stages of x + sum_r Rot_r(x) with one decomposition
// and one ModDown per stage (see ckks_sum_steps in include/ckks.h).
#include <string.h>

#include <algorithm>

#include "arith.h"
#include "attention.h"
#include "automorph.h"
#include "ntt_core.h"

namespace ckks {

namespace {

using nttc::at_u32;

struct SumIPArgs {
  const uint64_t* E;    // item b: E + b*E_bstride, [beta][next][N] raised digits
  const uint64_t* own;  // item b: own + b*own_bstride, [nq][N]: the input (limbs inside their own digit)
  const uint64_t* c0;   // or NULL, own_bstride apart
  uint64_t* acc;        // item b: acc + b*acc_bstride, [2][next][N]
  uint64_t E_bstride, own_bstride, acc_bstride;
  const uint64_t* evk[kMaxSumRot];
  uint32_t g[kMaxSumRot];
  const PrimeConst* prime;
  const uint64_t* pmod;  // [L][2]: {[P]_{q_i}, Shoup}
  int log_n, level, next, beta, alpha, L, K, n_rot, n_items;
};

// Sums of products of two words below 2^(2 SH), split into SH-bit halves, in
// three columns (weights 1, 2^SH, 2^2SH).  SH = 27 takes words below 2^54 and
// 256 products between folds, SH = 30 words below 2^60 and 8: column 1 gets
// two products a term, 2 * 256 * 2^54 = 2^63 and 2 * 8 * (2^30 - 1)^2 + 2^30 <
// 2^64.  A fold carries columns 0 and 1 upwards and reduces column 2 modulo q,
// which leaves it below 2.5 q (reduce_hi; primes that split at 30 bits are
// above 2^54) or below q.
template <int SH>
struct Cols {
  uint64_t a0, a1, a2;
};
template <int SH>
constexpr int kFoldTerms = SH == 27 ? 256 : 8;
template <int SH>
__device__ __forceinline__ uint32_t low_half(uint64_t v) {
  return (uint32_t)v & ((1u << SH) - 1);
}
template <int SH>
__device__ __forceinline__ void cols_mac(Cols<SH>& A, uint32_t xl, uint32_t xh, uint32_t kl, uint32_t kh) {
  A.a0 = mad64(xl, kl, A.a0);
  A.a1 = mad64(xl, kh, A.a1);
  A.a1 = mad64(xh, kl, A.a1);
  A.a2 = mad64(xh, kh, A.a2);
}
template <int SH>
__device__ __forceinline__ void cols_fold(Cols<SH>& A, uint64_t q, uint64_t inv1) {
  constexpr uint64_t M = (1ull << SH) - 1;
  A.a1 += A.a0 >> SH;
  A.a0 &= M;
  const uint64_t v = A.a2 + (A.a1 >> SH);
  A.a2 = SH == 30 ? reduce_hi(v, q, (uint32_t)inv1) : reduce64(v, q, inv1);
  A.a1 &= M;
}
// The sum modulo q, congruent, in [0, 6q).
template <int SH>
__device__ __forceinline__ uint64_t cols_reduce(const Cols<SH>& A, uint64_t q, uint64_t r64, uint64_t r64p,
                                                uint64_t inv1) {
  U128 r;
  uint64_t t = A.a1 << SH;
  const uint64_t lo = A.a0 + t;
  r.hi = (A.a1 >> (64 - SH)) + (lo < t ? 1 : 0);
  t = A.a2 << (2 * SH);
  r.lo = lo + t;
  r.hi += (A.a2 >> (64 - 2 * SH)) + (r.lo < t ? 1 : 0);
  return reduce128_6q(r, q, r64, r64p, inv1);
}

// 16-byte accesses, NT: non-temporal, so that words used once do not push the
// digits out of L2.
typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
template <bool NT>
__device__ __forceinline__ ulonglong2 load_pair(const uint64_t* limb, uint32_t w0) {
  if constexpr (NT) {
    const u64x2 v = __builtin_nontemporal_load(&at_u32(reinterpret_cast<const u64x2*>(limb), w0 >> 1));
    return make_ulonglong2(v.x, v.y);
  } else {
    return at_u32(reinterpret_cast<const ulonglong2*>(limb), w0 >> 1);
  }
}
template <bool NT>
__device__ __forceinline__ void store_pair(uint64_t* limb, uint32_t w0, uint64_t x, uint64_t y) {
  if constexpr (NT) __builtin_nontemporal_store((u64x2){x, y}, &at_u32(reinterpret_cast<u64x2*>(limb), w0 >> 1));
  else at_u32(reinterpret_cast<ulonglong2*>(limb), w0 >> 1) = make_ulonglong2(x, y);
}

// One (digit, rotation) of the inner product: a key word pair per component
// and every item's digit words, in flight while the previous one is computed.
template <int I>
struct SumTerm {
  ulonglong2 kb, ka, x[I];
  bool swap;
};

// acc[t] = sum_j sum_r tau_{g_r}(D_j)[t] evk_{r,j}[t] for two adjacent words of
// I items; on ciphertext limbs component 0 also gets P sum_r tau_{g_r}(c0),
// which ModDown turns into the stage's sum of rotated c0 (P is 0 modulo the
// special primes, so they are not touched).
//
// Each thread holds both words of I items: a key word is loaded once for all
// of them (the keys are the kernel's HBM traffic: 2 beta limbs per target limb
// and rotation).  tau_g maps an aligned pair of words of the bit-reversed
// order onto an aligned pair, perhaps swapped, so a gather is one 16-byte load.
// Digits are the outer loop: the I limbs of one digit (I * 512 KB at N = 2^16)
// stay in an XCD's L2 while the rotations gather from them.
//
// SPLIT > 1: the terms are dealt to SPLIT waves that hold the same words
// (`part` of them in turn), joined through LDS by the first.
template <int I, int SH, bool NT, int SPLIT>
__device__ __forceinline__ void sum_ip_narrow(const SumIPArgs& a, const PrimeConst& pc, int t, int keyl, int item0,
                                              uint32_t w0, int part, uint64_t* lds) {
  const int log_n = a.log_n;
  const uint64_t q = pc.q, inv1 = pc.inv1;
  const uint64_t LKN = (uint64_t)(a.L + a.K) << log_n;
  const uint64_t koff = (uint64_t)keyl << log_n;
  int it[I];
#pragma unroll
  for (int i = 0; i < I; ++i) it[i] = min(item0 + i, a.n_items - 1);
  auto load = [&](int j, int r, SumTerm<I>& s) {
    const uint32_t src = automorph_src(w0, a.g[r], log_n);
    s.swap = src & 1;
    const uint64_t* kb = a.evk[r] + (uint64_t)(2 * j) * LKN + koff;
    s.kb = load_pair<NT>(kb, w0);
    s.ka = load_pair<NT>(kb + LKN, w0);
    const bool own = t >= j * a.alpha && t < (j + 1) * a.alpha && t <= a.level;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const uint64_t* d = own ? a.own + it[i] * a.own_bstride + ((uint64_t)t << log_n)
                              : a.E + it[i] * a.E_bstride + ((uint64_t)(j * a.next + t) << log_n);
      s.x[i] = at_u32(reinterpret_cast<const ulonglong2*>(d), src >> 1);
    }
  };
  Cols<SH> A[I][2][2];  // item, component, word
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) A[i][e >> 1][e & 1] = Cols<SH>{0, 0, 0};
  // DEPTH terms load ahead: with one or two items a term computes for less
  // time than its key words take from HBM (with three or four, a second term's
  // registers would cost a wave)
  constexpr int DEPTH = I <= 2 ? 3 : 1;
  const int terms = a.beta * a.n_rot;
  int since = 0, j = 0, r = part;  // j, r: the next term to load
  auto carry = [&] {
    while (r >= a.n_rot) {
      r -= a.n_rot;
      ++j;
    }
  };
  auto advance = [&] {
    r += SPLIT;
    carry();
  };
  carry();
  SumTerm<I> buf[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (part + d * SPLIT < terms) {
      load(j, r, buf[d]);
      advance();
    }
  for (int n = part; n < terms; n += DEPTH * SPLIT) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (n + d * SPLIT >= terms) break;
      const SumTerm<I> cur = buf[d];
      if (n + (d + DEPTH) * SPLIT < terms) {
        load(j, r, buf[d]);
        advance();
      }
      const uint32_t bl0 = low_half<SH>(cur.kb.x), bh0 = (uint32_t)(cur.kb.x >> SH);
      const uint32_t bl1 = low_half<SH>(cur.kb.y), bh1 = (uint32_t)(cur.kb.y >> SH);
      const uint32_t al0 = low_half<SH>(cur.ka.x), ah0 = (uint32_t)(cur.ka.x >> SH);
      const uint32_t al1 = low_half<SH>(cur.ka.y), ah1 = (uint32_t)(cur.ka.y >> SH);
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const uint64_t x0 = cur.swap ? cur.x[i].y : cur.x[i].x, x1 = cur.swap ? cur.x[i].x : cur.x[i].y;
        const uint32_t l0 = low_half<SH>(x0), h0 = (uint32_t)(x0 >> SH);
        const uint32_t l1 = low_half<SH>(x1), h1 = (uint32_t)(x1 >> SH);
        cols_mac<SH>(A[i][0][0], l0, h0, bl0, bh0);
        cols_mac<SH>(A[i][0][1], l1, h1, bl1, bh1);
        cols_mac<SH>(A[i][1][0], l0, h0, al0, ah0);
        cols_mac<SH>(A[i][1][1], l1, h1, al1, ah1);
      }
      if (++since == kFoldTerms<SH>) {
        since = 0;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) cols_fold<SH>(A[i][e >> 1][e & 1], q, inv1);
      }
    }
  }
  // Ciphertext limbs leave the kernel congruent, below 10 q < 2^64: the last
  // pass multiplies them by P^-1 with a product that takes any 64-bit word.
  // Special limbs go to inverse butterflies, which take words below 4q.
  uint64_t s0[I], s1[I];
#pragma unroll
  for (int i = 0; i < I; ++i) s0[i] = s1[i] = 0;
  const bool low = t <= a.level;
  if (low && a.c0) {
    for (int k = part; k < a.n_rot; k += SPLIT) {
      const uint32_t src = automorph_src(w0, a.g[k], log_n);
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const ulonglong2 v = at_u32(
            reinterpret_cast<const ulonglong2*>(a.c0 + it[i] * a.own_bstride + ((uint64_t)t << log_n)), src >> 1);
        const uint64_t x0 = src & 1 ? v.y : v.x, x1 = src & 1 ? v.x : v.y;
        s0[i] = SH == 27 ? s0[i] + x0 : add_mod(s0[i], x0, q);  // at most 31 words below 2^54
        s1[i] = SH == 27 ? s1[i] + x1 : add_mod(s1[i], x1, q);
      }
    }
  }
  uint64_t v[I][4];
  const uint64_t cut = low && SPLIT == 1 ? ~0ull : 4 * q;
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[i][e] = cols_reduce<SH>(A[i][e >> 1][e & 1], q, pc.r64, pc.r64p, inv1);
      if (v[i][e] >= cut) v[i][e] -= 4 * q;
    }
  if constexpr (SPLIT > 1) {
    constexpr int PER = 6 * I;  // words a lane hands over
    const int lane = threadIdx.x & 63;
    if (part) {
#pragma unroll
      for (int i = 0; i < I; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) lds[((part - 1) * PER + i * 6 + e) * 64 + lane] = v[i][e];
        lds[((part - 1) * PER + i * 6 + 4) * 64 + lane] = s0[i];
        lds[((part - 1) * PER + i * 6 + 5) * 64 + lane] = s1[i];
      }
    }
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int i = 0; i < I; ++i) {
#pragma unroll
      for (int p = 0; p < SPLIT - 1; ++p) {  // 4 x 4q < 2^64, 4 x 31 words below 2^54 or 4 below q
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] += lds[(p * PER + i * 6 + e) * 64 + lane];
        s0[i] += lds[(p * PER + i * 6 + 4) * 64 + lane];
        s1[i] += lds[(p * PER + i * 6 + 5) * 64 + lane];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = reduce64(v[i][e], q, inv1);
    }
  }
  const uint64_t pw = low ? a.pmod[2 * t] : 0, pwp = low ? a.pmod[2 * t + 1] : 0;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    if (item0 + i >= a.n_items) break;
    if (low && a.c0) {  // [0, 4q)
      v[i][0] += mul_shoup_lazy(s0[i], pw, pwp, q);
      v[i][1] += mul_shoup_lazy(s1[i], pw, pwp, q);
    }
    uint64_t* ob = a.acc + (item0 + i) * a.acc_bstride + ((uint64_t)t << log_n);
    uint64_t* oa = ob + ((uint64_t)a.next << log_n);
    store_pair<NT>(ob, w0, v[i][0], v[i][1]);
    store_pair<NT>(oa, w0, v[i][2], v[i][3]);
  }
}

// Primes below 2^60.  The grid is (tiles of 512 words, target limbs, groups of
// I items), groups fastest: the groups of one tile run together on one XCD
// and share its key words in L2.  With one group (ONE) a key word is used once,
// and keys and results bypass L2's replacement: 262 -> 235 us for 4 items,
// radix 8, N = 2^16, level 22, where the keys' 0.68 GB and the digits' and
// results' 0.36 GB move at 4.5 TB/s; with two groups that loses 2 %.  Three or
// four waves a SIMD, one or two words a thread and up to 8 items a thread take
// the same time or more: the kernel is held by memory.
template <int I, bool ONE>
__global__ __launch_bounds__(256) void sum_ip_kernel(SumIPArgs a) {
  const nttc::GridPos gp = nttc::row_grid_pos<true>();
  const int t = gp.job;
  const int keyl = t <= a.level ? t : a.L + (t - a.level - 1);
  const PrimeConst& pc = a.prime[keyl];
  const uint32_t w0 = (gp.tile * 256 + threadIdx.x) * 2;
  if (pc.q < (1ull << 54))
    sum_ip_narrow<I, 27, ONE, 1>(a, pc, t, keyl, gp.item * I, w0, 0, nullptr);
  else
    sum_ip_narrow<I, 30, ONE, 1>(a, pc, t, keyl, gp.item * I, w0, 0, nullptr);
}

// The same for launches of less than a wave a SIMD, whose time is one wave's
// chain of terms: tiles of 128 words, the terms dealt to the workgroup's four
// waves.  1 item, 28 terms, 5 limbs, N = 2^12: 13.7 -> 6.9 us.
constexpr int kSumSplit = 4;
template <int I>
__global__ __launch_bounds__(256) void sum_ip_split_kernel(SumIPArgs a) {
  __shared__ uint64_t lds[(kSumSplit - 1) * 6 * I * 64];
  const int t = blockIdx.y;
  const int keyl = t <= a.level ? t : a.L + (t - a.level - 1);
  const PrimeConst& pc = a.prime[keyl];
  const uint32_t w0 = (blockIdx.x * 64 + (threadIdx.x & 63)) * 2;
  const int part = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (pc.q < (1ull << 54))
    sum_ip_narrow<I, 27, true, kSumSplit>(a, pc, t, keyl, 0, w0, part, lds);
  else
    sum_ip_narrow<I, 30, true, kSumSplit>(a, pc, t, keyl, 0, w0, part, lds);
}

// Primes up to 2^62: lazy Montgomery products as in the key switch, one item.
__global__ __launch_bounds__(256) void sum_ip_wide_kernel(SumIPArgs a) {
  const int t = blockIdx.y, item = blockIdx.z;
  const int keyl = t <= a.level ? t : a.L + (t - a.level - 1);
  const PrimeConst& pc = a.prime[keyl];
  const uint64_t q = pc.q, mp = pc.mprime;
  const int log_n = a.log_n;
  const uint32_t w = blockIdx.x * blockDim.x + threadIdx.x;
  const uint64_t LKN = (uint64_t)(a.L + a.K) << log_n;
  const uint64_t limb = item * a.own_bstride + ((uint64_t)t << log_n);
  const bool add = t <= a.level && a.c0;
  uint64_t b = 0, c = 0, rot = 0;
  const int fold = mont_fold(q);
  int since = 0;
  for (int r = 0; r < a.n_rot; ++r) {
    const uint32_t src = automorph_src(w, a.g[r], log_n);
    const uint64_t* evk = a.evk[r] + ((uint64_t)keyl << log_n) + w;
    for (int j = 0; j < a.beta; ++j) {
      const bool own = t >= j * a.alpha && t < (j + 1) * a.alpha && t <= a.level;
      const uint64_t x = own ? a.own[limb + src]
                             : a.E[item * a.E_bstride + ((uint64_t)(j * a.next + t) << log_n) + src];
      b += mont_mul_lazy(x, evk[(uint64_t)(2 * j) * LKN], q, mp);
      c += mont_mul_lazy(x, evk[(uint64_t)(2 * j + 1) * LKN], q, mp);
      if (++since == fold) {  // mont_fold(m) products since the last reduction
        since = 0;
        b = reduce64(b, q, pc.inv1);
        c = reduce64(c, q, pc.inv1);
      }
    }
    if (add) rot = add_mod(rot, a.c0[limb + src], q);
  }
  b = reduce_4q(mul_shoup_lazy(b, pc.r64, pc.r64p, q), q);
  if (add) b = add_mod(b, reduce_4q(mul_shoup_lazy(rot, a.pmod[2 * t], a.pmod[2 * t + 1], q), q), q);
  uint64_t* o = a.acc + item * a.acc_bstride + ((uint64_t)t << log_n) + w;
  o[0] = b;
  o[(uint64_t)a.next << log_n] = reduce_4q(mul_shoup_lazy(c, pc.r64, pc.r64p, q), q);
}

// Items a thread of the inner product holds: as many as the launch has, up to
// 4 (24 accumulator registers an item).
constexpr int kSumHeld = 4;

int launch_sum_ip(Ctx* c, hipStream_t s, const SumIPArgs& a) {
  TraceScope ts(c, s, "sum_ip", (double)a.n_items * a.next * c->N * (2.0 * a.beta * a.n_rot + 2));
  if (c->wide) {
    hipLaunchKernelGGL(sum_ip_wide_kernel, dim3(c->N / 256, a.next, a.n_items), dim3(256), 0, s, a);
  } else {
    // even groups: past 4 items they hold 3 or 4
    const int groups = (a.n_items + kSumHeld - 1) / kSumHeld, held = (a.n_items + groups - 1) / groups;
    // 1024 SIMDs; a workgroup of the split kernel takes four waves for 128 words
    if (groups == 1 && (uint64_t)(c->N / 128) * a.next <= 1024 && a.beta * a.n_rot >= 2 * kSumSplit) {
      auto fs = held == 1   ? sum_ip_split_kernel<1>
                : held == 2 ? sum_ip_split_kernel<2>
                : held == 3 ? sum_ip_split_kernel<3>
                            : sum_ip_split_kernel<4>;
      hipLaunchKernelGGL(fs, dim3(c->N / 128, a.next), dim3(256), 0, s, a);
      CKKS_HIP_CHECK(hipGetLastError());
      return CKKS_OK;
    }
    auto fn = groups > 1 ? (held == 3 ? sum_ip_kernel<3, false> : sum_ip_kernel<4, false>)
              : held == 1 ? sum_ip_kernel<1, true>
              : held == 2 ? sum_ip_kernel<2, true>
              : held == 3 ? sum_ip_kernel<3, true>
                          : sum_ip_kernel<4, true>;
    hipLaunchKernelGGL(fn, dim3(c->N / 512, a.next, (a.n_items + held - 1) / held), dim3(256), 0, s, a);
  }
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

// Words per item: decomposition, accumulators, ModDown conversion.
size_t stage_words(const Ctx* c, int level) { return ks_dec_words(c, level) + ks_back_words(c, level); }

}  // namespace

int key_ip(Ctx* c, hipStream_t s, int level, int n, const uint64_t* E, uint64_t E_stride, const uint64_t* own,
           uint64_t own_stride, const uint64_t* c0, uint64_t* A, uint64_t A_stride, int n_rot, const uint32_t* g,
           const uint64_t* const* evk) {
  SumIPArgs a;
  memset(&a, 0, sizeof(a));
  a.E = E;
  a.E_bstride = E_stride;
  a.own = own;
  a.own_bstride = own_stride;
  a.c0 = c0;
  a.acc = A;
  a.acc_bstride = A_stride;
  for (int r = 0; r < n_rot; ++r) {
    a.evk[r] = evk[r];
    a.g[r] = g[r];
  }
  a.prime = c->d_prime;
  a.pmod = c->d_moddown + c->md.pmod;
  a.log_n = (int)c->log_n;
  a.level = level;
  a.next = level + 1 + (int)c->K;
  a.beta = c->beta(level);
  a.alpha = (int)c->alpha;
  a.L = (int)c->L;
  a.K = (int)c->K;
  a.n_rot = n_rot;
  a.n_items = n;
  return launch_sum_ip(c, s, a);
}

// One stage on n items (n <= kMaxChunk): decomposition, inner product, and
// the ModDown of a key switch, whose last pass adds the stage's input.
static int sum_stage(Ctx* c, hipStream_t s, const uint64_t* in, uint64_t in_stride, uint64_t* out, uint64_t out_stride,
                     int n, int level, int n_rot, const uint32_t* g, const uint64_t* const* evk, uint64_t* ws) {
  const uint32_t N = c->N;
  const int nq = level + 1, next = nq + (int)c->K;
  const uint64_t dec_per = ks_dec_words(c, level), per = ks_back_words(c, level);
  uint64_t* dec = ws;
  uint64_t* A = ws + dec_per * n;
  const uint64_t* c1 = in + (uint64_t)nq * N;
  int rc = ks_decompose(c, s, level, n, c1, in_stride, dec, dec_per);
  if (rc) return rc;
  if ((rc = key_ip(c, s, level, n, dec + (uint64_t)nq * N, dec_per, c1, in_stride, in, A, per, n_rot, g, evk))) return rc;
  KSItem it[kMaxChunk];
  memset(it, 0, sizeof(KSItem) * n);
  it[0].accum = in;
  it[0].out = out;
  return ks_back(c, s, level, n, it, A, A + 2ull * next * N, per, 0, in_stride, out_stride, nq);
}

// Words of a group of items that goes through the stages together, with the
// two buffers between stages.
static size_t group_words(const Ctx* c, int level, int n, int n_stage) {
  return n * (stage_words(c, level) + (n_stage > 1 ? 4 * (size_t)(level + 1) * c->N : 0));
}

// Items of a group: the launches' limit, or what the words' limit holds (2 GiB
// at N = 2^16 and 24 + 8 limbs: 17 with one stage, 12 with more).  Large groups share each key word among more items; two
// half groups on two streams measured 0-14 % slower (keys are read twice).
static int sum_group(const Ctx* c, int level, int batch, int n_stage, uint64_t limit) {
  const size_t fit = limit / group_words(c, level, 1, n_stage);
  return (int)std::max<size_t>(1, std::min<size_t>({fit, (size_t)kMaxChunk, (size_t)batch}));
}

size_t sum_ws_words(const Ctx* c, int level, int batch, int n_stage, uint64_t limit) {
  return held_words(group_words(c, level, 1, n_stage), std::min(batch, kMaxChunk), limit);
}

int sum_stages(Ctx* c, hipStream_t s, const uint64_t* in, uint64_t in_stride, uint64_t* out, uint64_t out_stride,
               int batch, int level, const ckks_sum_steps& st, uint64_t* ws, uint64_t limit) {
  const uint64_t ct = 2ull * (level + 1) * c->N;
  const int group = sum_group(c, level, batch, st.n_stage, limit);
  for (int b0 = 0; b0 < batch; b0 += group) {
    const int n = std::min(group, batch - b0);
    // the stages between the first and the last alternate between two buffers
    uint64_t* half[2] = {ws + n * stage_words(c, level), ws + n * (stage_words(c, level) + ct)};
    const uint64_t* src = in + b0 * in_stride;
    uint64_t src_stride = in_stride;
    int at = 0;
    for (int k = 0; k < st.n_stage; ++k) {
      const bool last = k == st.n_stage - 1;
      int rc = sum_stage(c, s, src, src_stride, last ? out + b0 * out_stride : half[k & 1], last ? out_stride : ct, n,
                         level, st.radix[k] - 1, st.galois_elts + at, st.d_evks + at, ws);
      if (rc) return rc;
      at += st.radix[k] - 1;
      src = half[k & 1];
      src_stride = ct;
    }
  }
  return CKKS_OK;
}

}  // namespace ckks
