// Slotwise kernels of the layer norm calls (layernorm.h), on ciphertext words in
// NTT form: one thread per word of a limb, blockIdx.y the limb, blockIdx.z the
// item or block.
#include "layernorm.h"

#include "arith.h"
#include "convert.h"

namespace ckks {

namespace {

template <bool WIDE>
__device__ __forceinline__ uint64_t red(const AccT<WIDE>& m, const RedConst& pc) {
  return acc_reduce<WIDE>(m, pc.q, pc.r64, pc.r64p, pc.inv1);
}

// Constant j of a table (consts.h) of n, at limb i; table n = 1: the same for all.
struct Const {
  uint64_t w, p;
};
__device__ __forceinline__ Const constant(const uint64_t* tab, int n, int i, int j) {
  const ConstU64 t = (ConstU64)(tab + ((uint64_t)i * n + (n > 1 ? j : 0)) * 2);
  return Const{t[0], t[1]};
}
__device__ __forceinline__ uint64_t times(uint64_t x, const Const& k, uint64_t q) {
  return reduce_2q(mul_shoup(x, k.w, k.p, q), q);
}

// x (q_(nl-1) .. q_(nl-drop))^-1 at the limbs that stay, canonical.
__device__ __forceinline__ uint64_t keep(uint64_t x, int drop, int nl, int L, int i, const uint64_t* rescale, uint64_t q) {
  if (i >= nl - drop) return x;
  for (int k = 0; k < drop; ++k) {
    const ConstU64 rs = (ConstU64)(rescale + ((uint64_t)(nl - 1 - k) * L + i) * 4);
    x = mul_shoup_lazy(x, rs[0], rs[1], q);
  }
  return reduce_4q(x, q);
}

// Sums of tensor products, reduced once per four pairs (the middle part's
// columns take eight products).
template <bool WIDE>
struct TensorSum {
  AccT<WIDE> m0{}, m1{}, m2{};
  uint64_t r0 = 0, r1 = 0, r2 = 0;
  int since = 0;
  __device__ __forceinline__ void add(uint64_t a0, uint64_t a1, uint64_t b0, uint64_t b1, const RedConst& pc) {
    const Split<WIDE> x0 = split_word<WIDE>(a0), x1 = split_word<WIDE>(a1);
    const Split<WIDE> y0 = split_word<WIDE>(b0), y1 = split_word<WIDE>(b1);
    acc_mac<WIDE>(m0, x0, y0);
    acc_mac<WIDE>(m1, x0, y1);
    acc_mac<WIDE>(m1, x1, y0);
    acc_mac<WIDE>(m2, x1, y1);
    if (++since == 4) fold(pc);
  }
  __device__ __forceinline__ void fold(const RedConst& pc) {
    r0 = add_mod(r0, red<WIDE>(m0, pc), pc.q);
    r1 = add_mod(r1, red<WIDE>(m1, pc), pc.q);
    r2 = add_mod(r2, red<WIDE>(m2, pc), pc.q);
    m0 = m1 = m2 = AccT<WIDE>{};
    since = 0;
  }
};

template <bool WIDE>
__global__ __launch_bounds__(256) void moments_kernel(MomentArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, b = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  const uint64_t* x = a.x + (uint64_t)b * a.n_feat * 2 * lim + off;
  uint64_t s0 = 0, s1 = 0, r0 = 0, r1 = 0, r2 = 0;
  AccT<WIDE> m0{}, m1{}, m2{};
  for (int k = 0, since = 0; k < a.n_feat; ++k, x += 2 * lim) {
    const uint64_t x0 = x[0], x1 = x[lim];
    s0 = add_mod(s0, x0, pc.q);
    s1 = add_mod(s1, x1, pc.q);
    const Split<WIDE> y0 = split_word<WIDE>(x0), y1 = split_word<WIDE>(x1);
    acc_mac<WIDE>(m0, y0, y0);
    acc_mac<WIDE>(m1, y0, y1);
    acc_mac<WIDE>(m2, y1, y1);
    if (++since == 8 || k + 1 == a.n_feat) {
      r0 = add_mod(r0, red<WIDE>(m0, pc), pc.q);
      r1 = add_mod(r1, red<WIDE>(m1, pc), pc.q);
      r2 = add_mod(r2, red<WIDE>(m2, pc), pc.q);
      m0 = m1 = m2 = AccT<WIDE>{};
      since = 0;
    }
  }
  uint64_t* o = a.sum + (uint64_t)b * 2 * lim + off;
  o[0] = s0;
  o[lim] = s1;
  // F r - s s: the product of the sums with a minus sign on one factor
  const Const f = constant(a.tab, 3, i, 0), k = constant(a.tab, 3, i, 1);
  const Split<WIDE> y0 = split_word<WIDE>(s0), y1 = split_word<WIDE>(s1);
  const Split<WIDE> n0 = split_word<WIDE>(sub_mod(0, s0, pc.q)), n1 = split_word<WIDE>(sub_mod(0, s1, pc.q));
  m0 = m1 = m2 = AccT<WIDE>{};
  acc_mac<WIDE>(m0, y0, n0);
  acc_mac<WIDE>(m1, y0, n1);
  acc_mac<WIDE>(m2, y1, n1);
  const uint64_t v0 = add_mod(times(r0, f, pc.q), red<WIDE>(m0, pc), pc.q);
  uint64_t v1 = add_mod(times(r1, f, pc.q), red<WIDE>(m1, pc), pc.q);
  v1 = add_mod(v1, v1, pc.q);
  const uint64_t v2 = add_mod(times(r2, f, pc.q), red<WIDE>(m2, pc), pc.q);
  uint64_t* d = a.out + (uint64_t)b * 3 * lim + off;
  uint64_t e = keep(times(v0, k, pc.q), 2, a.nl, a.L, i, a.rescale, pc.q);
  if (i < a.nl - 2) e = add_mod(e, constant(a.tab, 3, i, 2).w, pc.q);
  d[0] = e;
  d[lim] = keep(times(v1, k, pc.q), 2, a.nl, a.L, i, a.rescale, pc.q);
  d[2 * lim] = times(v2, k, pc.q);
}

template <bool WIDE>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, p = a.first + blockIdx.z, b = p / a.n_feat, feat = p % a.n_feat;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n;
  const uint64_t* x = a.x + (uint64_t)p * 2 * xl + off;
  const uint64_t* s = a.sum + (uint64_t)b * 2 * xl + off;
  const uint64_t* r = a.r + (uint64_t)b * 2 * lim + off;
  const Const f = constant(a.feat, 1, i, 0), k = constant(a.gain, a.n_gain, i, feat);
  const uint64_t u0 = times(sub_mod(times(x[0], f, pc.q), s[0], pc.q), k, pc.q);
  const uint64_t u1 = times(sub_mod(times(x[xl], f, pc.q), s[xl], pc.q), k, pc.q);
  TensorSum<WIDE> t;
  t.add(u0, u1, r[0], r[lim], pc);
  t.fold(pc);
  uint64_t* d = a.out + (uint64_t)blockIdx.z * 3 * lim + off;
  uint64_t e = keep(t.r0, 2, a.nl, a.L, i, a.rescale, pc.q);
  if (a.beta && i < a.nl - 2) e = add_mod(e, constant(a.beta, a.n_feat, i, feat).w, pc.q);
  d[0] = e;
  d[lim] = keep(t.r1, 2, a.nl, a.L, i, a.rescale, pc.q);
  d[2 * lim] = t.r2;
}

template <bool WIDE>
__global__ __launch_bounds__(256) void grad_sums_kernel(GradSumArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, b = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n;
  const uint64_t* dy = a.dy + (uint64_t)b * a.n_feat * 2 * lim + off;
  const uint64_t* xh = a.xhat + (uint64_t)b * a.n_feat * 2 * xl + off;
  uint64_t s0 = 0, s1 = 0;
  TensorSum<WIDE> t;
  for (int f = 0; f < a.n_feat; ++f, dy += 2 * lim, xh += 2 * xl) {
    const Const k = constant(a.gain, a.n_gain, i, f);
    const uint64_t g0 = times(dy[0], k, pc.q), g1 = times(dy[lim], k, pc.q);
    s0 = add_mod(s0, g0, pc.q);
    s1 = add_mod(s1, g1, pc.q);
    t.add(g0, g1, xh[0], xh[xl], pc);
  }
  t.fold(pc);
  if (i < a.g_nl) {
    uint64_t* o = a.G + (((uint64_t)b * 2 * a.g_nl + i) << a.log_n) + c;
    o[0] = s0;
    o[(uint64_t)a.g_nl << a.log_n] = s1;
  }
  uint64_t* d = a.out + (uint64_t)b * 3 * lim + off;
  d[0] = keep(t.r0, 2, a.nl, a.L, i, a.rescale, pc.q);
  d[lim] = keep(t.r1, 2, a.nl, a.L, i, a.rescale, pc.q);
  d[2 * lim] = t.r2;
}

template <bool WIDE>
__global__ __launch_bounds__(256) void scaled_pair_kernel(ScaledPairArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, b = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, rl = (uint64_t)a.r_nl << a.log_n;
  const uint64_t* r = a.r + (uint64_t)b * 2 * rl + off;
  const uint64_t* h = a.h + (uint64_t)b * 2 * lim + off;
  TensorSum<WIDE> t;
  t.add(r[0], r[rl], h[0], h[lim], pc);
  t.fold(pc);
  const Const kept = constant(a.kept, 1, i, 0), k = constant(a.k, 1, i, 0);
  uint64_t* d = a.out + (uint64_t)b * 3 * lim + off;
  d[0] = times(t.r0, kept, pc.q);
  d[lim] = times(t.r1, kept, pc.q);
  d[2 * lim] = times(t.r2, k, pc.q);
}

template <bool WIDE>
__global__ __launch_bounds__(256) void grad_kernel(GradArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, p = a.first + blockIdx.z, b = p / a.n_feat, feat = p % a.n_feat;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  const uint64_t dl = (uint64_t)a.dy_nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n, rl = (uint64_t)a.r_nl << a.log_n;
  const uint64_t* dy = a.dy + (uint64_t)p * 2 * dl + off;
  const uint64_t* xh = a.xhat + (uint64_t)p * 2 * xl + off;
  const uint64_t* r = a.r + (uint64_t)b * 2 * rl + off;
  const uint64_t* G = a.G + (uint64_t)b * 2 * lim + off;
  const uint64_t* R = a.R + (uint64_t)b * 2 * lim + off;
  const Const f = constant(a.feat, 1, i, 0), k = constant(a.gain, a.n_gain, i, feat);
  const uint64_t u0 = sub_mod(times(times(dy[0], k, pc.q), f, pc.q), G[0], pc.q);
  const uint64_t u1 = sub_mod(times(times(dy[dl], k, pc.q), f, pc.q), G[lim], pc.q);
  TensorSum<WIDE> t;
  t.add(u0, u1, r[0], r[rl], pc);
  t.add(sub_mod(0, xh[0], pc.q), sub_mod(0, xh[xl], pc.q), R[0], R[lim], pc);
  t.fold(pc);
  uint64_t* d = a.out + (uint64_t)blockIdx.z * 3 * lim + off;
  d[0] = keep(t.r0, 2, a.nl, a.L, i, a.rescale, pc.q);
  d[lim] = keep(t.r1, 2, a.nl, a.L, i, a.rescale, pc.q);
  d[2 * lim] = t.r2;
}

template <bool WIDE>
__global__ __launch_bounds__(256) void weight_sums_kernel(WeightArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, feat = a.first + blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n;
  uint64_t s0 = 0, s1 = 0;
  TensorSum<WIDE> t;
  for (int b = 0; b < a.n_blk; ++b) {
    const uint64_t p = (uint64_t)b * a.n_feat + feat;
    const uint64_t* dy = a.dy + p * 2 * lim + off;
    const uint64_t d0 = dy[0], d1 = dy[lim];
    s0 = add_mod(s0, d0, pc.q);
    s1 = add_mod(s1, d1, pc.q);
    if (a.out) {
      const uint64_t* xh = a.xhat + p * 2 * xl + off;
      t.add(d0, d1, xh[0], xh[xl], pc);
    }
  }
  if (a.sum) {
    uint64_t* o = a.sum + (uint64_t)blockIdx.z * 2 * lim + off;
    o[0] = s0;
    o[lim] = s1;
  }
  if (!a.out) return;
  t.fold(pc);
  uint64_t* d = a.out + (uint64_t)blockIdx.z * 3 * lim + off;
  d[0] = keep(t.r0, 1, a.nl, a.L, i, a.rescale, pc.q);
  d[lim] = keep(t.r1, 1, a.nl, a.L, i, a.rescale, pc.q);
  d[2 * lim] = t.r2;
}

}  // namespace

#define NORM_LAUNCH(kern, items, units)                                                                      \
  TraceScope ts(c, s, "layernorm", units);                                                                   \
  hipLaunchKernelGGL(c->wide ? kern<true> : kern<false>, dim3(c->N / 256, a.nl, items), dim3(256), 0, s, a); \
  CKKS_HIP_CHECK(hipGetLastError());                                                                         \
  return CKKS_OK

int launch_moments(Ctx* c, hipStream_t s, const MomentArgs& a, int nb) {
  NORM_LAUNCH(moments_kernel, nb, (double)nb * a.n_feat * a.nl * 4 * c->N);
}
int launch_norm(Ctx* c, hipStream_t s, const NormArgs& a, int n) {
  NORM_LAUNCH(norm_kernel, n, (double)n * a.nl * 11 * c->N);
}
int launch_grad_sums(Ctx* c, hipStream_t s, const GradSumArgs& a, int nb) {
  NORM_LAUNCH(grad_sums_kernel, nb, (double)nb * a.n_feat * a.nl * 7 * c->N);
}
int launch_scaled_pair(Ctx* c, hipStream_t s, const ScaledPairArgs& a, int nb) {
  NORM_LAUNCH(scaled_pair_kernel, nb, (double)nb * a.nl * 10 * c->N);
}
int launch_grad(Ctx* c, hipStream_t s, const GradArgs& a, int n) {
  NORM_LAUNCH(grad_kernel, n, (double)n * a.nl * 15 * c->N);
}
int launch_weight_sums(Ctx* c, hipStream_t s, const WeightArgs& a, int n) {
  NORM_LAUNCH(weight_sums_kernel, n, (double)n * a.n_blk * a.nl * 5 * c->N);
}

}  // namespace ckks
