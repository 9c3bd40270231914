// Rescale of a batch by its top limb q_l with the basis conversion fused
// into the forward NTT's column pass and the final combination into its row
// pass (the converted limbs make one round trip through memory instead of
// three).  Optionally a per-limb constant (a constant polynomial in NTT form)
// is added to component 0, and another ciphertext to the output, by the same
// final store.  Per item,
// component and limb i < l, with v = iNTT(c_l) canonical and vbar its centred
// lift:
//   w_i   = (vbar mod q_i) * [q_l^-1]_{q_i}
//   out_i = c_i * [q_l^-1]_{q_i} - NTT(w_i)          (mod q_i)
#include <string.h>

#include "attention.h"
#include "kernels.h"
#include "ntt_core.h"

namespace ckks {

namespace {

using namespace nttc;

struct RescalePassArgs {
  const uint64_t* v;   // item b: v + b*v_bstride, [2][N] iNTT of limb l
  uint64_t* w;         // item b: w + b*w_bstride, [2][l][N]
  const uint64_t* ct;  // item b: ct + b*ct_bstride, [2][l+1][N]
  uint64_t* out;       // item b: out + b*out_bstride, [2][l][N]
  const uint64_t* acc; // optional, added to the output: item b at acc + b*acc_bstride, [2][l][N]
  uint64_t v_bstride, w_bstride, ct_bstride, out_bstride, acc_bstride;
  const uint64_t* tab;  // [L][L][4]: for level l, limb i: {q_l^-1, Shoup, q_l mod q_i, 0}
  const PrimeConst* prime;
  const uint64_t* tw;  // forward twiddles
  int log_n, level, L;
  int has_add;
  uint64_t add0[64];  // has_add: added to component 0 of limb i (a constant in NTT form)
};

// Column-pass input: w_i computed from v on load.  A word above half of q_l
// gets neg = -q_l mod q_i added and needs no reduction (below 2^63), since the
// Shoup product takes any 64-bit word; its result, below 2q, is what the first
// butterflies take.
struct PrepIO {
  typedef NoOps Ops;
  const uint64_t* v;
  uint64_t* dst;
  uint64_t q, qinv, qinvp, neg, half;
  __device__ __forceinline__ uint64_t load(uint32_t j) const {
    const uint64_t x = v[j];
    return mul_shoup(x + (x > half ? neg : 0), qinv, qinvp, q);
  }
  __device__ __forceinline__ void after_load(uint32_t, uint64_t) const {}
  __device__ __forceinline__ Ops fetch(uint32_t) const { return Ops(); }
  __device__ __forceinline__ void store(uint32_t j, uint64_t x, const Ops&) const { dst[j] = x; }
};

template <int RA, int RB, int LOGN>
__global__ __launch_bounds__(kThreads) void rescale_col_kernel(RescalePassArgs a) {
  constexpr int ROWS = 1 << (RA + RB);
  __shared__ uint64_t lds[lds_words<true, RB, ROWS>()];
  const int job = blockIdx.y, item = blockIdx.z;  // job = comp * l + i
  const int comp = job / a.level, i = job % a.level;
  const PrimeConst& pc = a.prime[i];
  const uint64_t* rs = a.tab + ((uint64_t)a.level * a.L + i) * 4;
  PrepIO io;
  io.v = a.v + item * a.v_bstride + ((uint64_t)comp << a.log_n);
  io.dst = a.w + item * a.w_bstride + ((uint64_t)job << a.log_n);
  io.q = pc.q;
  io.qinv = rs[0];
  io.qinvp = rs[1];
  io.neg = pc.q - rs[2];
  io.half = (a.prime[a.level].q - 1) / 2;
  Finish fin{0, 0, 0, pc.inv1};
  run_pass<RA, RB, false, true, LOGN>(io, lds, blockIdx.x, a.log_n, a.tw + ((uint64_t)i << (a.log_n + 1)), pc.q,
                                      fin);
}

// Row-pass output: c_i * q_l^-1 - NTT(w_i) (+ constant) (+ acc).  With acc
// equal to out each word is read and written by the same thread.
struct CombOps {
  uint64_t c, a;
};
struct RescaleCombineIO {
  typedef CombOps Ops;
  const uint64_t* w;
  const uint64_t* ct;
  const uint64_t* acc;
  uint64_t* out;
  uint64_t q, qinv, qinvp, add;
  __device__ __forceinline__ uint64_t load(uint32_t j) const { return w[j]; }
  __device__ __forceinline__ void after_load(uint32_t, uint64_t) const {}
  __device__ __forceinline__ Ops fetch(uint32_t j) const { return Ops{ct[j], acc ? acc[j] : 0}; }
  __device__ __forceinline__ void store(uint32_t j, uint64_t x, const Ops& o) const {
    out[j] = add_mod(add_mod(sub_mod(reduce_2q(mul_shoup(o.c, qinv, qinvp, q), q), x, q), add, q), o.a, q);
  }
};

template <int RA, int RB, int LOGN>
__global__ __launch_bounds__(kThreads) void rescale_row_kernel(RescalePassArgs a) {
  constexpr int ROWS = 1 << (RA + RB);
  __shared__ uint64_t lds[lds_words<false, RB, ROWS>()];
  const GridPos gp = row_grid_pos();
  const int job = gp.job, item = gp.item;
  const int comp = job / a.level, i = job % a.level;
  const PrimeConst& pc = a.prime[i];
  const uint64_t* rs = a.tab + ((uint64_t)a.level * a.L + i) * 4;
  RescaleCombineIO io;
  io.w = a.w + item * a.w_bstride + ((uint64_t)job << a.log_n);
  io.ct = a.ct + item * a.ct_bstride + ((uint64_t)(comp * (a.level + 1) + i) << a.log_n);
  io.out = a.out + item * a.out_bstride + ((uint64_t)job << a.log_n);
  io.acc = a.acc ? a.acc + item * a.acc_bstride + ((uint64_t)job << a.log_n) : nullptr;
  io.q = pc.q;
  io.qinv = rs[0];
  io.qinvp = rs[1];
  io.add = (a.has_add && comp == 0) ? a.add0[i] : 0;
  Finish fin{1, 0, 0, pc.inv1};
  run_pass<RA, RB, false, false, LOGN>(io, lds, gp.tile, a.log_n, a.tw + ((uint64_t)i << (a.log_n + 1)), pc.q, fin);
}

// The row pass of a product's rescale (PlainMul): c_i = p_i in_i is formed where
// it is needed, so the product never exists in memory (a ciphertext written
// and read less): linattn_chunk on 3 tokens of 2 groups of 24 limbs at N = 2^16
// 3843 -> 3777 us, on 96 tokens of 7 limbs at N = 2^12 959 -> 942 us.
struct MulRowArgs {
  PlainMul m;
  const uint64_t* w;  // item b at w + b*per, [2][level][N]
  uint64_t per;
  const uint64_t* tab;
  const PrimeConst* prime;
  const uint64_t* tw;
  int log_n, L;
};
struct MulOps {
  uint64_t c, p;
};
struct MulCombineIO {
  typedef MulOps Ops;
  const uint64_t* w;
  const uint64_t* ct;
  const uint64_t* p;
  uint64_t* out;
  uint64_t q, qinv, qinvp, r64, r64p, inv1;
  __device__ __forceinline__ uint64_t load(uint32_t j) const { return w[j]; }
  __device__ __forceinline__ void after_load(uint32_t, uint64_t) const {}
  __device__ __forceinline__ Ops fetch(uint32_t j) const { return Ops{ct[j], p[j]}; }
  __device__ __forceinline__ void store(uint32_t j, uint64_t x, const Ops& o) const {
    const uint64_t c = mul_mod(o.c, o.p, q, r64, r64p, inv1);
    out[j] = sub_mod(reduce_2q(mul_shoup(c, qinv, qinvp, q), q), x, q);
  }
};

template <int RA, int RB, int LOGN>
__global__ __launch_bounds__(kThreads) void rescale_mul_row_kernel(MulRowArgs a) {
  constexpr int ROWS = 1 << (RA + RB);
  __shared__ uint64_t lds[lds_words<false, RB, ROWS>()];
  const GridPos gp = row_grid_pos();
  const int job = gp.job, b = a.m.first + gp.item, t = b / a.m.ng, g = b % a.m.ng;
  const int comp = job / a.m.level, i = job % a.m.level;
  const PrimeConst& pc = a.prime[i];
  const uint64_t* rs = a.tab + ((uint64_t)a.m.level * a.L + i) * 4;
  const uint64_t row = (uint64_t)t * a.m.n_row + (a.m.g0 + g) % a.m.n_row;
  MulCombineIO io;
  io.w = a.w + gp.item * a.per + ((uint64_t)job << a.log_n);
  io.ct = a.m.in + ((uint64_t)t * a.m.n_grp + g) * a.m.in_bstride + comp * a.m.in_comp + ((uint64_t)i << a.log_n);
  io.p = a.m.p + ((row * (a.m.level + 1) + i) << a.log_n);
  io.out = a.m.out + b * a.m.out_bstride + ((uint64_t)job << a.log_n);
  io.q = pc.q;
  io.qinv = rs[0];
  io.qinvp = rs[1];
  io.r64 = pc.r64;
  io.r64p = pc.r64p;
  io.inv1 = pc.inv1;
  Finish fin{1, 0, 0, pc.inv1};
  run_pass<RA, RB, false, false, LOGN>(io, lds, gp.tile, a.log_n, a.tw + ((uint64_t)i << (a.log_n + 1)), pc.q, fin);
}

// ---------------------------------------------------------------------------
// The rescales of a key switch (ks_rescale).
struct DropArgs {
  uint64_t* A;  // item b: A + b*per, [2][comp_limbs][N]: dropped limbs q_(l-drop+1)..q_l first
  uint64_t* W;  // item b: W + b*per, [2][l+1][N]
  uint64_t per;
  const uint64_t* tab;  // as RescalePassArgs
  const PrimeConst* prime;
  const uint64_t* tw;
  int log_n, level, L, drop, comp_limbs;
};

// The centred lift of x mod the dropped prime ql, modulo q.
__device__ __forceinline__ uint64_t lift_mod(uint64_t x, uint64_t half, uint64_t qlmod, uint64_t q, uint64_t inv1) {
  const uint64_t t = x >= q ? reduce64(x, q, inv1) : x;
  return x > half ? sub_mod(t, qlmod, q) : t;
}

// The values dropped, canonical, in place: v = iNTT(R)_l = A_l - w_l and, for
// a second rescale, v' = (A_(l-1) - w_(l-1) - v) q_l^-1 mod q_(l-1).
__global__ __launch_bounds__(256) void drop_values_kernel(DropArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int comp = blockIdx.y, l = a.level;
  uint64_t* v = a.A + blockIdx.z * a.per + ((uint64_t)(comp * a.comp_limbs) << a.log_n) + c;
  const uint64_t* w = a.W + blockIdx.z * a.per + ((uint64_t)(comp * (l + 1)) << a.log_n) + c;
  const uint64_t N = 1ull << a.log_n;
  const PrimeConst& pl = a.prime[l];
  const uint64_t x = sub_mod(v[(a.drop - 1) * N], reduce64(w[l * N], pl.q, pl.inv1), pl.q);
  v[(a.drop - 1) * N] = x;
  if (a.drop == 1) return;
  const PrimeConst& p = a.prime[l - 1];
  const uint64_t* rs = a.tab + ((uint64_t)l * a.L + l - 1) * 4;
  uint64_t u = sub_mod(v[0], reduce64(w[(l - 1) * N], p.q, p.inv1), p.q);
  u = sub_mod(u, lift_mod(x, (pl.q - 1) / 2, rs[2], p.q, p.inv1), p.q);
  v[0] = reduce_2q(mul_shoup(u, rs[0], rs[1], p.q), p.q);
}

// Column-pass input: (w + v) q_l^-1 computed on load, for DROP 2 then
// (that + v') q_(l-1)^-1, v and v' centred: a dropped word above half its prime
// q_l gets -q_l mod q added and needs no reduction, since the Shoup product
// takes any 64-bit word.  w is congruent, below 6q (below q for primes above
// 2^60), a product below 2q, so the sums stay below 8 * 2^60 or 2^64.  The
// result is left below 2q, as the first butterflies take it.
template <int DROP>
struct DropIO {
  typedef NoOps Ops;
  uint64_t* w;
  const uint64_t* v[DROP];
  uint64_t q, qinv[DROP], qinvp[DROP], neg[DROP], half[DROP];
  __device__ __forceinline__ uint64_t load(uint32_t j) const {
    uint64_t x = w[j];
#pragma unroll
    for (int d = 0; d < DROP; ++d) {
      const uint64_t y = v[d][j];
      x = mul_shoup(x + y + (y > half[d] ? neg[d] : 0), qinv[d], qinvp[d], q);
    }
    return x;
  }
  __device__ __forceinline__ void after_load(uint32_t, uint64_t) const {}
  __device__ __forceinline__ Ops fetch(uint32_t) const { return Ops(); }
  __device__ __forceinline__ void store(uint32_t j, uint64_t x, const Ops&) const { w[j] = x; }
};

template <int RA, int RB, int LOGN, int DROP>
__global__ __launch_bounds__(kThreads) void drop_col_kernel(DropArgs a) {
  constexpr int ROWS = 1 << (RA + RB);
  __shared__ uint64_t lds[lds_words<true, RB, ROWS>()];
  const int low = a.level + 1 - DROP;
  const int comp = blockIdx.y / low, i = blockIdx.y % low;
  const PrimeConst& pc = a.prime[i];
  DropIO<DROP> io;
  io.w = a.W + blockIdx.z * a.per + ((uint64_t)(comp * (a.level + 1) + i) << a.log_n);
#pragma unroll
  for (int d = 0; d < DROP; ++d) {  // q_l first
    const uint64_t* rs = a.tab + ((uint64_t)(a.level - d) * a.L + i) * 4;
    io.v[d] = a.A + blockIdx.z * a.per + ((uint64_t)(comp * a.comp_limbs + DROP - 1 - d) << a.log_n);
    io.qinv[d] = rs[0];
    io.qinvp[d] = rs[1];
    io.neg[d] = pc.q - rs[2];
    io.half[d] = (a.prime[a.level - d].q - 1) / 2;
  }
  io.q = pc.q;
  Finish fin{0, 0, 0, pc.inv1};
  run_pass<RA, RB, false, true, LOGN>(io, lds, blockIdx.x, a.log_n, a.tw + ((uint64_t)i << (a.log_n + 1)), pc.q,
                                      fin);
}

}  // namespace

int rescale_mul_fused(Ctx* c, hipStream_t s, const PlainMul& m, const uint64_t* v, uint64_t* w, uint64_t per, int batch) {
  const uint32_t N = c->N;
  const int log_n = (int)c->log_n, lr = logb_row(log_n), lc = logb_col(log_n), level = m.level;
  RescalePassArgs a;
  memset(&a, 0, sizeof(a));
  a.v = v;
  a.w = w;
  a.v_bstride = a.w_bstride = per;
  a.tab = c->d_rescale;
  a.prime = c->d_prime;
  a.tw = c->d_tw_fwd;
  a.log_n = log_n;
  a.level = level;
  a.L = (int)c->L;
  const MulRowArgs r{m, w, per, c->d_rescale, c->d_prime, c->d_tw_fwd, log_n, (int)c->L};
  auto fc = CKKS_PICK_PASS(rescale_col_kernel, log_n, lc);
  auto fr = CKKS_PICK_PASS(rescale_mul_row_kernel, log_n, lr);
  if (!fc || !fr) return set_error(CKKS_EINTERNAL, "unsupported N");
  {
    TraceScope ts(c, s, "rescale", (double)batch * 2 * level * ((double)(N / 2) * lc + N));
    hipLaunchKernelGGL(fc, dim3(pass_tiles(N, lc), 2 * level, batch), dim3(kThreads), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
  }
  {
    TraceScope ts(c, s, "rescale", (double)batch * 2 * level * ((double)(N / 2) * lr + 3.0 * N));
    hipLaunchKernelGGL(fr, dim3(pass_tiles(N, lr), 2 * level, batch), dim3(kThreads), 0, s, r);
    CKKS_HIP_CHECK(hipGetLastError());
  }
  return CKKS_OK;
}

int drop_col_pass(Ctx* c, hipStream_t s, uint64_t* A, uint64_t* W, uint64_t per, int n_items, int level, int drop,
                  int comp_limbs) {
  const uint32_t N = c->N;
  const int log_n = (int)c->log_n, lc = logb_col(log_n), low = level + 1 - drop;
  DropArgs a;
  a.A = A;
  a.W = W;
  a.per = per;
  a.tab = c->d_rescale;
  a.prime = c->d_prime;
  a.tw = c->d_tw_fwd;
  a.log_n = log_n;
  a.level = level;
  a.L = (int)c->L;
  a.drop = drop;
  a.comp_limbs = comp_limbs;
  {
    TraceScope ts(c, s, "rescale", (double)n_items * 2 * drop * N);
    hipLaunchKernelGGL(drop_values_kernel, dim3(N / 256, 2, n_items), dim3(256), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
  }
  auto fn = drop == 1 ? CKKS_PICK_PASS(drop_col_kernel, log_n, lc, 1) : CKKS_PICK_PASS(drop_col_kernel, log_n, lc, 2);
  if (!fn) return set_error(CKKS_EINTERNAL, "unsupported N");
  TraceScope ts(c, s, "rescale", (double)n_items * 2 * low * ((double)(N / 2) * lc + drop * N));
  hipLaunchKernelGGL(fn, dim3(pass_tiles(N, lc), 2 * low, n_items), dim3(kThreads), 0, s, a);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

int rescale_fused(Ctx* c, hipStream_t s, const uint64_t* ct, uint64_t ct_bstride, const uint64_t* v, uint64_t v_bstride,
                  uint64_t* w, uint64_t w_bstride, uint64_t* out, uint64_t out_bstride, int batch, int level,
                  const uint64_t* add0, const uint64_t* acc, uint64_t acc_bstride) {
  const uint32_t N = c->N;
  const int log_n = (int)c->log_n;
  const int lr = logb_row(log_n), lc = logb_col(log_n);
  RescalePassArgs a;
  memset(&a, 0, sizeof(a));
  a.v = v;
  a.w = w;
  a.ct = ct;
  a.out = out;
  a.v_bstride = v_bstride;
  a.w_bstride = w_bstride;
  a.ct_bstride = ct_bstride;
  a.out_bstride = out_bstride;
  a.tab = c->d_rescale;
  a.prime = c->d_prime;
  a.tw = c->d_tw_fwd;
  a.log_n = log_n;
  a.level = level;
  a.L = (int)c->L;
  a.acc = acc;
  a.acc_bstride = acc_bstride;
  if (add0) {
    if (level > 64) return set_error(CKKS_EINTERNAL, "too many limbs for a fused constant");
    a.has_add = 1;
    for (int i = 0; i < level; ++i) a.add0[i] = add0[i];
  }
  auto fc = CKKS_PICK_PASS(rescale_col_kernel, log_n, lc);
  auto fr = CKKS_PICK_PASS(rescale_row_kernel, log_n, lr);
  if (!fc || !fr) return set_error(CKKS_EINTERNAL, "unsupported N");
  {
    TraceScope ts(c, s, "rescale", (double)batch * 2 * level * ((double)(N / 2) * lc + N));
    hipLaunchKernelGGL(fc, dim3(pass_tiles(N, lc), 2 * level, batch), dim3(kThreads), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
  }
  {
    TraceScope ts(c, s, "rescale", (double)batch * 2 * level * ((double)(N / 2) * lr + N));
    hipLaunchKernelGGL(fr, dim3(pass_tiles(N, lr), 2 * level, batch), dim3(kThreads), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
  }
  return CKKS_OK;
}

}  // namespace ckks
