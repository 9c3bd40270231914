// Key-switch steps on small rings (N <= 2^12), where a limb fits one
// workgroup's LDS and a call's time is the latency of its chain of launches: a
// whole transform in one kernel, together with the conversion before it and
// the combination after it.  Per stage of a sum (or relinearisation) five
// launches instead of ten:
//   small_inverse  inverse transform of the input, times the ModUp constant
//   small_raise    ModUp conversion to one target limb, forward transform
//   key_ip         the inner product (sumrot.hip)
//   small_inverse  inverse transform of the special limbs (and of the limbs a
//                  rescale drops)
//   small_combine  ModDown conversion (and the rescale's lift) to one limb,
//                  forward transform, combination with the accumulators
// One workgroup per limb; words and ranges as in the two-pass kernels, so the
// results are the same words.  At N = 2^12 and 4 limbs the kernels take 8.7,
// 11.5, 5 to 7, 8.7 and 12.2 us (17 with a rescale): the latency of the
// transform's six rounds and of the loads before them, with most CUs empty.
#include <stddef.h>
#include <string.h>

#include "arith.h"
#include "automorph.h"
#include "attention.h"
#include "convert.h"
#include "ntt_core.h"

namespace ckks {

namespace {

using namespace nttc;

// A workgroup's T threads hold W words each (4: with 8, and a third fewer
// rounds, a step of 4 limbs takes 226 us instead of 211); a transform runs in rounds of
// LOGW stages in registers with an exchange through LDS between them, the
// round at stride 1 taking the LAST stages that are left.
template <int LOGN>
struct Ring {
  static constexpr int LOGW = 2;
  static constexpr int W = 1 << LOGW, N = 1 << LOGN, T = N >> LOGW;
  static constexpr int LAST = LOGN % LOGW ? LOGN % LOGW : LOGW;
  static constexpr int LDS = N + N / 32;
};

__device__ __forceinline__ int pad(int j) { return j + (j >> 5); }  // strides of 4 to 64 words meet few banks twice

// The round of R stages on blocks of N >> DONE words: words at a stride of
// N >> (DONE + R), group g of the thread's W >> R.
template <int LOGN, int R, int DONE>
__device__ __forceinline__ void round_coords(int g, int& block, int& base) {
  constexpr int LS = LOGN - DONE - R;  // log2 of the stride
  const int u = (int)threadIdx.x + g * Ring<LOGN>::T;
  block = u >> LS;
  base = (block << (LS + R)) + (u & ((1 << LS) - 1));
}

template <int LOGN, int R>
struct RoundTw {
  ulonglong2 w[Ring<LOGN>::W >> R][(1 << R) - 1];
};

template <int LOGN, int R, int DONE>
__device__ __forceinline__ RoundTw<LOGN, R> round_twiddles(const uint64_t* tw) {
  RoundTw<LOGN, R> r;
#pragma unroll
  for (int g = 0; g < (Ring<LOGN>::W >> R); ++g) {
    int block, base;
    round_coords<LOGN, R, DONE>(g, block, base);
#pragma unroll
    for (int s = 0; s < R; ++s)
#pragma unroll
      for (int h = 0; h < (1 << s); ++h)
        r.w[g][(1 << s) - 1 + h] =
            at_u32(reinterpret_cast<const ulonglong2*>(tw), (1u << (DONE + s)) + ((uint32_t)block << s) + h);
  }
  return r;
}

template <int LOGN, int R, int AR>
__device__ __forceinline__ void forward_round(uint64_t (&x)[Ring<LOGN>::W], const RoundTw<LOGN, R>& t, uint64_t q) {
#pragma unroll
  for (int g = 0; g < (Ring<LOGN>::W >> R); ++g)
#pragma unroll
    for (int s = 0; s < R; ++s) {
      const int half = 1 << (R - 1 - s);
#pragma unroll
      for (int h = 0; h < (1 << s); ++h)
#pragma unroll
        for (int p = 0; p < half; ++p) {
          const int a = (g << R) + h * 2 * half + p;
          const ulonglong2 w = t.w[g][(1 << s) - 1 + h];
          ct_butterfly<AR>(x[a], x[a + half], w.x, w.y, q);
        }
    }
}

// HARVEY words stay below 4q (primes below 2^61), STRICT ones below 2q.
template <int LOGN, int R, int AR>
__device__ __forceinline__ void inverse_round(uint64_t (&x)[Ring<LOGN>::W], const RoundTw<LOGN, R>& t, uint64_t q) {
#pragma unroll
  for (int g = 0; g < (Ring<LOGN>::W >> R); ++g)
#pragma unroll
    for (int s = R - 1; s >= 0; --s) {
      const int half = 1 << (R - 1 - s);
#pragma unroll
      for (int h = 0; h < (1 << s); ++h)
#pragma unroll
        for (int p = 0; p < half; ++p) {
          const int a = (g << R) + h * 2 * half + p;
          const ulonglong2 w = t.w[g][(1 << s) - 1 + h];
          gs_butterfly_ar<AR>(x[a], x[a + half], w.x, w.y, q, 0);
        }
    }
}

// Words between the layouts of two rounds.
template <int LOGN, int R, int DONE>
__device__ __forceinline__ void to_lds(const uint64_t (&x)[Ring<LOGN>::W], uint64_t* lds) {
#pragma unroll
  for (int g = 0; g < (Ring<LOGN>::W >> R); ++g) {
    int block, base;
    round_coords<LOGN, R, DONE>(g, block, base);
#pragma unroll
    for (int k = 0; k < (1 << R); ++k) lds[pad(base + (k << (LOGN - DONE - R)))] = x[(g << R) + k];
  }
}
template <int LOGN, int R, int DONE>
__device__ __forceinline__ void from_lds(uint64_t (&x)[Ring<LOGN>::W], const uint64_t* lds) {
#pragma unroll
  for (int g = 0; g < (Ring<LOGN>::W >> R); ++g) {
    int block, base;
    round_coords<LOGN, R, DONE>(g, block, base);
#pragma unroll
    for (int k = 0; k < (1 << R); ++k) x[(g << R) + k] = lds[pad(base + (k << (LOGN - DONE - R)))];
  }
}

// Between the writes of one round's layout and the reads of another's, of which
// the round at DONE has the larger blocks.  Blocks of 64 W words whose rounds
// use one group of W words per thread belong to one wave, which waits for its
// own writes; others for the workgroup's.  The writes after the reads need no
// wait: a thread writes the words it has read.  A stage of radix 8 on 4 limbs at
// N = 2^12 takes 49.1 us with two workgroup barriers an exchange, 46.3 us so.
template <int LOGN, int DONE, int R>
__device__ __forceinline__ void exchange_wait() {
  if constexpr (R == Ring<LOGN>::LOGW && (Ring<LOGN>::N >> DONE) <= 64 * Ring<LOGN>::W) wave_lds_wait();
  else __syncthreads();
}

// Forward transform: x enters in the first round's layout (word k at thread +
// k T) and leaves in the last one's: word ((thread + g T) << LAST) + k.  t: the
// round's twiddles; the next round's load while this one computes.
template <int LOGN, int AR, int DONE, int R>
__device__ __forceinline__ void forward_rounds(uint64_t (&x)[Ring<LOGN>::W], const RoundTw<LOGN, R>& t, uint64_t* lds,
                                               const uint64_t* tw, uint64_t q) {
  constexpr int LOGW = Ring<LOGN>::LOGW, NEXT = DONE + R, RN = LOGN - NEXT < LOGW ? LOGN - NEXT : LOGW;
  if constexpr (NEXT < LOGN) {
    const RoundTw<LOGN, RN> tn = round_twiddles<LOGN, RN, NEXT>(tw);
    forward_round<LOGN, R, AR>(x, t, q);
    to_lds<LOGN, R, DONE>(x, lds);
    exchange_wait<LOGN, DONE, RN>();
    from_lds<LOGN, RN, NEXT>(x, lds);
    forward_rounds<LOGN, AR, NEXT, RN>(x, tn, lds, tw, q);
  } else {
    forward_round<LOGN, R, AR>(x, t, q);
  }
}

// Inverse transform, without its factor: the layouts the other way round.
template <int LOGN, int AR, int DONE, int R>
__device__ __forceinline__ void inverse_rounds(uint64_t (&x)[Ring<LOGN>::W], const RoundTw<LOGN, R>& t, uint64_t* lds,
                                               const uint64_t* tw, uint64_t q) {
  constexpr int LOGW = Ring<LOGN>::LOGW;
  if constexpr (DONE > 0) {
    const RoundTw<LOGN, LOGW> tn = round_twiddles<LOGN, LOGW, DONE - LOGW>(tw);
    inverse_round<LOGN, R, AR>(x, t, q);
    to_lds<LOGN, R, DONE>(x, lds);
    exchange_wait<LOGN, DONE - LOGW, R>();
    from_lds<LOGN, LOGW, DONE - LOGW>(x, lds);
    inverse_rounds<LOGN, AR, DONE - LOGW, LOGW>(x, tn, lds, tw, q);
  } else {
    inverse_round<LOGN, R, AR>(x, t, q);
  }
}

struct InverseArgs {
  const uint64_t* src;  // item b: src + b*src_bstride, limb src_limb[job]
  uint64_t* dst;
  uint64_t src_bstride, dst_bstride;
  const uint64_t* tw;   // inverse twiddles
  const uint64_t* tab;  // {w, w'} at scale_off[job], applied to the result
  const PrimeConst* prime;
  // Jobs with add_limb[job] >= 0 transform src + P add instead (any 64-bit
  // words in src): the limbs a rescale drops.
  const uint64_t* add;
  uint64_t add_bstride;
  const uint64_t* pmod;
  uint32_t scale_off[kMaxJobs];
  uint16_t src_limb[kMaxJobs], dst_limb[kMaxJobs];
  int16_t add_limb[kMaxJobs];
  uint8_t prime_idx[kMaxJobs];
};

template <int LOGN>
__global__ __launch_bounds__((Ring<LOGN>::T)) void small_inverse_kernel(InverseArgs a) {
  typedef Ring<LOGN> G;
  __shared__ uint64_t lds[G::LDS];
  const int job = blockIdx.x, item = blockIdx.y, p = a.prime_idx[job];
  const PrimeConst& pc = a.prime[p];
  const uint64_t q = pc.q;
  const uint64_t* src = a.src + item * a.src_bstride + ((uint64_t)a.src_limb[job] << LOGN);
  const int al = a.add_limb[job];
  const uint64_t* add = al < 0 ? nullptr : a.add + item * a.add_bstride + ((uint64_t)al << LOGN);
  const uint64_t* tw = a.tw + ((uint64_t)p << (LOGN + 1));
  const RoundTw<LOGN, G::LAST> t = round_twiddles<LOGN, G::LAST, LOGN - G::LAST>(tw);
  uint64_t x[G::W];
#pragma unroll
  for (int g = 0; g < (G::W >> G::LAST); ++g)
#pragma unroll
    for (int k = 0; k < (1 << G::LAST); ++k) {
      const uint32_t j = (((uint32_t)threadIdx.x + g * G::T) << G::LAST) + k;
      uint64_t v = at_u32(src, j);
      if (add)
        v = add_mod(reduce64(v, q, pc.inv1),
                    reduce_4q(mul_shoup_lazy(at_u32(add, j), a.pmod[2 * p], a.pmod[2 * p + 1], q), q), q);
      x[(g << G::LAST) + k] = v;
    }
  if (q < (1ull << 61)) inverse_rounds<LOGN, AR_HARVEY, LOGN - G::LAST, G::LAST>(x, t, lds, tw, q);
  else inverse_rounds<LOGN, AR_STRICT, LOGN - G::LAST, G::LAST>(x, t, lds, tw, q);
  const uint64_t w = a.tab[a.scale_off[job]], wp = a.tab[a.scale_off[job] + 1];
  uint64_t* dst = a.dst + item * a.dst_bstride + ((uint64_t)a.dst_limb[job] << LOGN);
#pragma unroll
  for (int k = 0; k < G::W; ++k)
    at_u32(dst, (uint32_t)threadIdx.x + k * G::T) = reduce_2q(mul_shoup(x[k], w, wp, q), q);
}

// Forward transform of words in the ranges the conversions leave (below 6q, or
// q for WIDE), with the butterflies of the prime's size; t: the first round's
// twiddles.
template <int LOGN, bool WIDE>
__device__ __forceinline__ void forward_any(uint64_t (&x)[Ring<LOGN>::W], const RoundTw<LOGN, Ring<LOGN>::LOGW>& t,
                                            uint64_t* lds, const uint64_t* tw, uint64_t q) {
  constexpr int R = Ring<LOGN>::LOGW;
  if constexpr (WIDE) {
    forward_rounds<LOGN, AR_STRICT, 0, R>(x, t, lds, tw, q);
  } else {
    if (q < (1ull << 57)) forward_rounds<LOGN, AR_LAZY, 0, R>(x, t, lds, tw, q);
    else forward_rounds<LOGN, AR_HARVEY, 0, R>(x, t, lds, tw, q);
  }
}

// Conversion sums of a thread's W words to one target: up to 8 sources between
// reductions (conv_dot_c for as many sources as there are).
template <int W, bool WIDE>
struct ConvSum {
  AccT<WIDE> acc[W];
  uint64_t done[W];  // reduced sums of the sources before
  int since, reduced;
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      acc[e] = AccT<WIDE>{};
      done[e] = 0;
    }
    since = reduced = 0;
  }
  __device__ __forceinline__ void add(const Split<WIDE> (&y)[W], uint64_t table, const RedConst& pc) {
    const Split<WIDE> c = split_table<WIDE>(table);
    if (since == 8) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        done[e] = add_mod(done[e], acc_reduce<WIDE>(acc[e], pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
        acc[e] = AccT<WIDE>{};
      }
      since = 0;
      reduced = 1;
    }
#pragma unroll
    for (int e = 0; e < W; ++e) acc_mac<WIDE>(acc[e], y[e], c);
    ++since;
  }
  // below 6q (q for WIDE or past 8 sources)
  __device__ __forceinline__ uint64_t get(int e, const RedConst& pc) const {
    if (!reduced) return acc_reduce_6q<WIDE>(acc[e], pc.q, pc.r64, pc.r64p, pc.inv1);
    return add_mod(done[e], acc_reduce<WIDE>(acc[e], pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
  }
};

// ModUp of digit j to target limb t and its transform, canonical (as
// modup_kernel and the two forward passes).
template <int LOGN, bool WIDE>
__global__ __launch_bounds__((Ring<LOGN>::T)) void small_raise_kernel(ModUpArgs a, const uint64_t* twf) {
  typedef Ring<LOGN> G;
  __shared__ uint64_t lds[G::LDS];
  const int j = blockIdx.x / a.next, t = blockIdx.x % a.next;
  const int lo = a.lo[j], hi = a.hi[j], na = hi - lo;
  if (t >= lo && t < hi) return;
  const int p = t <= a.level ? t : a.L + (t - a.level - 1);
  const RedConst pc = red_const((ConstPrime)a.prime, p);
  const uint64_t* tw = twf + ((uint64_t)p << (LOGN + 1));
  const RoundTw<LOGN, G::LOGW> first = round_twiddles<LOGN, G::LOGW, 0>(tw);
  const ConstU64 conv = (ConstU64)(a.tables + a.offset[j] + 2 * na) + t;
  const uint64_t* src = a.x + blockIdx.y * a.x_bstride + ((uint64_t)lo << LOGN);
  ConvSum<G::W, WIDE> sum;
  sum.init();
#pragma unroll 4
  for (int i = 0; i < na; ++i) {
    Split<WIDE> y[G::W];
#pragma unroll
    for (int k = 0; k < G::W; ++k)
      y[k] = split_word<WIDE>(at_u32(src + ((uint64_t)i << LOGN), (uint32_t)threadIdx.x + k * G::T));
    sum.add(y, conv[i * a.next], pc);
  }
  uint64_t x[G::W];
#pragma unroll
  for (int k = 0; k < G::W; ++k) x[k] = sum.get(k, pc);
  forward_any<LOGN, WIDE>(x, first, lds, tw, pc.q);
  uint64_t* out = a.out + blockIdx.y * a.out_bstride + ((uint64_t)(j * a.next + t) << LOGN);
#pragma unroll
  for (int g = 0; g < (G::W >> G::LAST); ++g)
#pragma unroll
    for (int k = 0; k < (1 << G::LAST); k += 2) {
      const int e = (g << G::LAST) + k;
      const uint32_t w = (((uint32_t)threadIdx.x + g * G::T) << G::LAST) + k;
      at_u32(reinterpret_cast<ulonglong2*>(out), w >> 1) =
          make_ulonglong2(reduce64(x[e], pc.q, pc.inv1), reduce64(x[e + 1], pc.q, pc.inv1));
    }
}

struct CombineArgs {
  // item b at acc + b*acc_bstride, [2][next][N]: accumulators (any 64-bit
  // words) on the limbs that stay; coefficients on the `drop` limbs after them
  // and the special limbs (small_inverse)
  const uint64_t* acc;
  uint64_t acc_bstride;
  const uint64_t* add[2];  // [nq][N] or NULL, read through tau_g where g[item] != 0
  const uint64_t* accum;   // [2][nq][N] or NULL
  uint64_t add_bstride, accum_bstride;
  uint64_t* out;  // [2][out_comp_limbs][N]
  uint64_t out_bstride;
  const uint64_t* conv;     // [NS][L]
  const uint64_t* pinv;     // [L][2]
  const uint64_t* rescale;  // the context's table
  const uint64_t* tw;
  const PrimeConst* prime;
  uint32_t g[kMaxChunk];
  int level, next, L, K, out_comp_limbs;
};

// out_c[i] = (acc_c P^-1 - w) (q_l ..)^-1 - v's share + add + accum, as
// comb_ip_kernel after moddown_conv_kernel, drop_values_kernel and
// drop_col_kernel: limb i of component blockIdx.x / low.  With DROP the
// conversion to the dropped limbs is formed again for every limb.
template <int LOGN, bool WIDE, int DROP>
__global__ __launch_bounds__((Ring<LOGN>::T)) void small_combine_kernel(CombineArgs a) {
  typedef Ring<LOGN> G;
  __shared__ uint64_t lds[G::LDS];
  const int low = a.level + 1 - DROP, l = a.level;
  const int comp = blockIdx.x / low, i = blockIdx.x % low, item = blockIdx.y;
  const ConstPrime prime = (ConstPrime)a.prime;
  const RedConst pc = red_const(prime, i);
  const uint64_t q = pc.q;
  const uint64_t* tw = a.tw + ((uint64_t)i << (LOGN + 1));
  const RoundTw<LOGN, G::LOGW> first = round_twiddles<LOGN, G::LOGW, 0>(tw);
  const uint64_t* acc = a.acc + item * a.acc_bstride + ((uint64_t)(comp * a.next) << LOGN);
  const uint64_t* coef = acc + ((uint64_t)low << LOGN);  // dropped limbs, then special limbs
  uint64_t x[G::W];
  {
    ConvSum<G::W, WIDE> sum[DROP + 1];  // to limbs i, l, l-1
    uint32_t neg[G::W];
    RedConst to[DROP + 1];
    to[0] = pc;
#pragma unroll
    for (int d = 0; d < DROP; ++d) to[d + 1] = red_const(prime, l - d);
#pragma unroll
    for (int d = 0; d <= DROP; ++d) sum[d].init();
#pragma unroll
    for (int e = 0; e < G::W; ++e) neg[e] = 0;
#pragma unroll 2
    for (int k = 0; k < a.K; ++k) {
      const uint64_t half = prime[a.L + k].q >> 1;
      Split<WIDE> y[G::W];
#pragma unroll
      for (int e = 0; e < G::W; ++e) {
        const uint64_t v = at_u32(coef + ((uint64_t)(DROP + k) << LOGN), (uint32_t)threadIdx.x + e * G::T);
        neg[e] += v > half ? 1u : 0u;
        y[e] = split_word<WIDE>(v);
      }
      const ConstU64 conv = (ConstU64)a.conv + (uint64_t)k * a.L;
      sum[0].add(y, conv[i], to[0]);
#pragma unroll
      for (int d = 0; d < DROP; ++d) sum[d + 1].add(y, conv[l - d], to[d + 1]);
    }
#pragma unroll
    for (int e = 0; e < G::W; ++e) {
      const uint32_t c = (uint32_t)threadIdx.x + e * G::T;
      uint64_t w = sub_mod(sum[0].get(e, pc), neg[e], q);
      if constexpr (DROP > 0) {  // v = iNTT(R)_l
        const RedConst& pl = to[1];
        const ConstU64 rs = (ConstU64)(a.rescale + ((uint64_t)l * a.L + i) * 4);
        const uint64_t wl = reduce64(sub_mod(sum[1].get(e, pl), neg[e], pl.q), pl.q, pl.inv1);
        const uint64_t v = sub_mod(at_u32(coef + ((uint64_t)(DROP - 1) << LOGN), c), wl, pl.q);
        const bool up = v > (pl.q >> 1);
        w = mul_shoup(w + v + (up ? q - rs[2] : 0), rs[0], rs[1], q);
        if constexpr (DROP == 2) {  // v' = (iNTT(R)_(l-1) - v) q_l^-1
          const RedConst& p2 = to[2];
          const ConstU64 r1 = (ConstU64)(a.rescale + ((uint64_t)l * a.L + l - 1) * 4);
          const ConstU64 r2 = (ConstU64)(a.rescale + ((uint64_t)(l - 1) * a.L + i) * 4);
          const uint64_t w2 = reduce64(sub_mod(sum[2].get(e, p2), neg[e], p2.q), p2.q, p2.inv1);
          uint64_t u = sub_mod(at_u32(coef, c), w2, p2.q);
          u = sub_mod(u, reduce64(v + (up ? p2.q - r1[2] : 0), p2.q, p2.inv1), p2.q);
          u = reduce_2q(mul_shoup(u, r1[0], r1[1], p2.q), p2.q);
          w = mul_shoup(w + u + (u > (p2.q >> 1) ? q - r2[2] : 0), r2[0], r2[1], q);
        }
      }
      x[e] = w;
    }
  }
  // the words the result takes load during the transform
  acc += (uint64_t)i << LOGN;
  const uint64_t* add = a.add[comp] ? a.add[comp] + item * a.add_bstride + ((uint64_t)i << LOGN) : nullptr;
  const uint64_t* accum =
      a.accum ? a.accum + item * a.accum_bstride + ((uint64_t)(comp * (l + 1) + i) << LOGN) : nullptr;
  const uint32_t g = a.g[item];
  uint64_t va[G::W], vd[G::W], vm[G::W];
#pragma unroll
  for (int e = 0; e < G::W; ++e) {
    const uint32_t j = (((uint32_t)threadIdx.x + (e >> G::LAST) * G::T) << G::LAST) + (e & ((1 << G::LAST) - 1));
    va[e] = at_u32(acc, j);
    vd[e] = add ? at_u32(add, g ? automorph_src(j, g, LOGN) : j) : 0;
    vm[e] = accum ? at_u32(accum, j) : 0;
  }
  forward_any<LOGN, WIDE>(x, first, lds, tw, q);
  uint64_t* out = a.out + item * a.out_bstride + ((uint64_t)(comp * a.out_comp_limbs + i) << LOGN);
#pragma unroll
  for (int e = 0; e < G::W; ++e) {
    const uint32_t j = (((uint32_t)threadIdx.x + (e >> G::LAST) * G::T) << G::LAST) + (e & ((1 << G::LAST) - 1));
    uint64_t v = mul_shoup_lazy(va[e], a.pinv[2 * i], a.pinv[2 * i + 1], q);
#pragma unroll
    for (int d = 0; d < DROP; ++d) {
      const ConstU64 rs = (ConstU64)(a.rescale + ((uint64_t)(l - d) * a.L + i) * 4);
      v = mul_shoup_lazy(v, rs[0], rs[1], q);
    }
    v = sub_mod(reduce_4q(v, q), reduce64(x[e], q, pc.inv1), q);
    at_u32(out, j) = add_mod(add_mod(v, vd[e], q), vm[e], q);
  }
}

#define SMALL_PICK(log_n, f10, f11, f12) ((log_n) == 10 ? (f10) : (log_n) == 11 ? (f11) : (f12))

int launch_inverse(Ctx* c, hipStream_t s, const InverseArgs& a, int n_job, int n_items) {
  auto fn = SMALL_PICK(c->log_n, small_inverse_kernel<10>, small_inverse_kernel<11>, small_inverse_kernel<12>);
  TraceScope ts(c, s, "ntt_pass", (double)n_items * n_job * (c->N / 2) * c->log_n);
  hipLaunchKernelGGL(fn, dim3(n_job, n_items), dim3(c->N / 4), 0, s, a);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

typedef void (*RaiseFn)(ModUpArgs, const uint64_t*);
template <bool WIDE>
RaiseFn pick_raise(int log_n) {
  return SMALL_PICK(log_n, (small_raise_kernel<10, WIDE>), (small_raise_kernel<11, WIDE>),
                    (small_raise_kernel<12, WIDE>));
}
typedef void (*CombineFn)(CombineArgs);
template <bool WIDE, int DROP>
CombineFn pick_combine(int log_n) {
  return SMALL_PICK(log_n, (small_combine_kernel<10, WIDE, DROP>), (small_combine_kernel<11, WIDE, DROP>),
                    (small_combine_kernel<12, WIDE, DROP>));
}

}  // namespace

// The raised digits of n polynomials (NTT form, item b at src + b*src_stride,
// [level+1][N]): coefficients y in Y, digits in E, per apart.
int small_decompose(Ctx* c, hipStream_t s, int level, int n, const uint64_t* src, uint64_t src_stride, uint64_t* Y,
                    uint64_t* E, uint64_t per) {
  const int nq = level + 1, next = nq + (int)c->K, beta = c->beta(level);
  InverseArgs a;
  memset(&a, 0, sizeof(a));
  a.src = src;
  a.src_bstride = src_stride;
  a.dst = Y;
  a.dst_bstride = per;
  a.tw = c->d_tw_inv;
  a.tab = c->d_modup;
  a.prime = c->d_prime;
  ModUpArgs mu;
  memset(&mu, 0, sizeof(mu));
  for (int j = 0; j < beta; ++j) {
    const ModUpEntry& en = c->modup[level][j];
    mu.lo[j] = en.lo;
    mu.hi[j] = en.hi;
    mu.offset[j] = en.offset;
    for (int i = en.lo; i < en.hi; ++i) {
      a.src_limb[i] = a.dst_limb[i] = (uint16_t)i;
      a.prime_idx[i] = (uint8_t)i;
      a.add_limb[i] = -1;
      a.scale_off[i] = (uint32_t)(en.offset + 2 * (i - en.lo));
    }
  }
  int rc = launch_inverse(c, s, a, nq, n);
  if (rc) return rc;
  mu.x = Y;
  mu.out = E;
  mu.x_bstride = mu.out_bstride = per;
  mu.tables = c->d_modup;
  mu.prime = c->d_prime;
  mu.n = c->N;
  mu.level = level;
  mu.next = next;
  mu.L = (int)c->L;
  const int log_n = (int)c->log_n;
  const RaiseFn fn = c->wide ? pick_raise<true>(log_n) : pick_raise<false>(log_n);
  TraceScope ts(c, s, "modup", (double)n * (beta * next - nq) * c->N * (c->alpha + 1 + log_n / 2.0));
  hipLaunchKernelGGL(fn, dim3(beta * next, n), dim3(c->N / 4), 0, s, mu, c->d_tw_fwd);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

// ModDown of n accumulators A (item b at A + b*per, [2][next][N]) with `drop`
// rescales; it[0]'s add, accum and out at the given strides (with drop, add is
// [nq][N] per component as ks_rescale's parts 0 and 1).
int small_back(Ctx* c, hipStream_t s, int level, int drop, int n, const KSItem* it, uint64_t* A, uint64_t per,
               uint64_t add_stride, uint64_t accum_stride, uint64_t out_stride, int out_comp_limbs) {
  const int nq = level + 1, K = (int)c->K, next = nq + K, low = nq - drop;
  InverseArgs a;
  memset(&a, 0, sizeof(a));
  a.src = a.dst = A;
  a.src_bstride = a.dst_bstride = per;
  a.tw = c->d_tw_inv;
  a.tab = c->d_moddown;
  a.prime = c->d_prime;
  a.add = it[0].add[0];
  a.add_bstride = add_stride;
  a.pmod = c->d_moddown + c->md.pmod;
  int jobs = 0;
  for (int comp = 0; comp < 2; ++comp)
    for (int k = 0; k < drop + K; ++k, ++jobs) {
      const bool top = k < drop;
      a.src_limb[jobs] = a.dst_limb[jobs] = (uint16_t)(comp * next + low + k);
      a.prime_idx[jobs] = (uint8_t)(top ? low + k : (int)c->L + k - drop);
      a.add_limb[jobs] = (int16_t)(top ? comp * nq + low + k : -1);
      a.scale_off[jobs] = (uint32_t)(top ? c->md.pinvn + 2 * (low + k) : c->md.phinv + 2 * (k - drop));
    }
  int rc = launch_inverse(c, s, a, jobs, n);
  if (rc) return rc;
  CombineArgs m;
  memset(&m, 0, sizeof(m));
  m.acc = A;
  m.acc_bstride = per;
  m.add[0] = it[0].add[0];
  m.add[1] = it[0].add[1];
  m.add_bstride = add_stride;
  m.accum = it[0].accum;
  m.accum_bstride = accum_stride;
  m.out = it[0].out;
  m.out_bstride = out_stride;
  m.conv = c->d_moddown + c->md.conv;
  m.pinv = c->d_moddown + c->md.pinv;
  m.rescale = c->d_rescale;
  m.tw = c->d_tw_fwd;
  m.prime = c->d_prime;
  for (int b = 0; b < n; ++b) m.g[b] = it[b].add_g;
  m.level = level;
  m.next = next;
  m.L = (int)c->L;
  m.K = K;
  m.out_comp_limbs = out_comp_limbs;
  const int log_n = (int)c->log_n;
  const CombineFn fn = drop == 0   ? (c->wide ? pick_combine<true, 0>(log_n) : pick_combine<false, 0>(log_n))
                       : drop == 1 ? (c->wide ? pick_combine<true, 1>(log_n) : pick_combine<false, 1>(log_n))
                                   : (c->wide ? pick_combine<true, 2>(log_n) : pick_combine<false, 2>(log_n));
  TraceScope ts(c, s, "ntt_row_combine", (double)n * 2 * low * c->N * (K + 2 + log_n / 2.0));
  hipLaunchKernelGGL(fn, dim3(2 * low, n), dim3(c->N / 4), 0, s, m);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

int small_inverse(Ctx* c, hipStream_t s, uint64_t* A, uint64_t per, int n, const NttJobs& jobs) {
  InverseArgs a;
  memset(&a, 0, sizeof(a));
  a.src = a.dst = A;
  a.src_bstride = a.dst_bstride = per;
  a.tw = c->d_tw_inv;
  a.tab = (const uint64_t*)c->d_prime;
  a.prime = c->d_prime;
  for (int j = 0; j < jobs.n; ++j) {
    a.src_limb[j] = jobs.src_limb[j];
    a.dst_limb[j] = jobs.dst_limb[j];
    a.prime_idx[j] = jobs.prime[j];
    a.add_limb[j] = -1;
    a.scale_off[j] = (uint32_t)((jobs.prime[j] * sizeof(PrimeConst) + offsetof(PrimeConst, ninv)) / 8);  // {N^-1, Shoup}
  }
  return launch_inverse(c, s, a, jobs.n, n);
}

// ks_rescale on a small ring.
int small_rescale(Ctx* c, hipStream_t s, int level, int drop, int n, const uint64_t* X, uint64_t x_stride,
                  const uint64_t* rlk, uint64_t* out, uint64_t out_stride, uint64_t* ws, uint64_t per) {
  const uint32_t N = c->N;
  const int nq = level + 1, next = nq + (int)c->K, beta = c->beta(level);
  uint64_t* Y = ws;
  uint64_t* E = Y + (uint64_t)nq * N;
  uint64_t* A = E + (uint64_t)beta * next * N;
  const uint64_t* d2 = X + 2ull * nq * N;
  int rc = small_decompose(c, s, level, n, d2, x_stride, Y, E, per);
  if (rc) return rc;
  const uint32_t one = 1;
  if ((rc = key_ip(c, s, level, n, E, per, d2, x_stride, nullptr, A, per, 1, &one, &rlk))) return rc;
  KSItem it[kMaxChunk];
  memset(it, 0, sizeof(KSItem) * n);
  it[0].add[0] = X;
  it[0].add[1] = X + (uint64_t)nq * N;
  it[0].out = out;
  return small_back(c, s, level, drop, n, it, A, per, x_stride, 0, out_stride, nq - drop);
}

}  // namespace ckks
