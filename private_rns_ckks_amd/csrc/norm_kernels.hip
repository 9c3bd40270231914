// Slotwise kernels of the layer norm calls (layernorm.h), on ciphertext words in
// NTT form: one thread per word of a limb, blockIdx.y the limb, blockIdx.z the
// block, item or group of items.
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
  return reduce_4q(mul_shoup_lazy(x, k.w, k.p, q), q);
}

// Sums of tensor products, reduced once per four pairs (the middle part's
// columns take eight products).  Operands are below 2^60, wide ones below 2^62.
template <bool WIDE>
struct TensorSum {
  AccT<WIDE> m0{}, m1{}, m2{};
  __device__ __forceinline__ void add(uint64_t a0, uint64_t a1, uint64_t b0, uint64_t b1) {
    const Split<WIDE> x0 = split_word<WIDE>(a0), x1 = split_word<WIDE>(a1);
    const Split<WIDE> y0 = split_word<WIDE>(b0), y1 = split_word<WIDE>(b1);
    acc_mac<WIDE>(m0, x0, y0);
    acc_mac<WIDE>(m1, x0, y1);
    acc_mac<WIDE>(m1, x1, y0);
    acc_mac<WIDE>(m2, x1, y1);
  }
  __device__ __forceinline__ void fold(uint64_t& r0, uint64_t& r1, uint64_t& r2, const RedConst& pc) {
    r0 = add_mod(r0, red<WIDE>(m0, pc), pc.q);
    r1 = add_mod(r1, red<WIDE>(m1, pc), pc.q);
    r2 = add_mod(r2, red<WIDE>(m2, pc), pc.q);
    m0 = m1 = m2 = AccT<WIDE>{};
  }
  // The parts into o (3 of them, lim apart): 0 and 1 times `kept` (the inverses
  // of the primes that the rescales to come drop, or 1), which takes any word.
  __device__ __forceinline__ void store(uint64_t* o, uint64_t lim, const Const& kept, uint64_t add,
                                        const RedConst& pc) const {
    const uint64_t a = acc_reduce_6q<WIDE>(m0, pc.q, pc.r64, pc.r64p, pc.inv1);
    const uint64_t b = acc_reduce_6q<WIDE>(m1, pc.q, pc.r64, pc.r64p, pc.inv1);
    o[0] = add_mod(times(a, kept, pc.q), add, pc.q);
    o[lim] = times(b, kept, pc.q);
    o[2 * lim] = red<WIDE>(m2, pc);
  }
};

// The sums over features run in segments, a thread each, where one thread a
// word would leave the chip empty (below kSegmentWords words, from kSegments
// features on): SEG threads of a word (threadIdx.y) take a range each, and the
// first adds up what they leave in LDS.
constexpr int kSegments = 16;
constexpr uint64_t kSegmentWords = 3u << 15;

// `n` values of a thread, added over its word's segments; valid in segment 0.
template <int SEG, int n>
__device__ __forceinline__ void add_segments(uint64_t (&v)[n], uint64_t q) {
  if (SEG == 1) return;
  __shared__ uint64_t part[SEG][n][64];
  const int x = threadIdx.x, seg = threadIdx.y;
#pragma unroll
  for (int k = 0; k < n; ++k) part[seg][k][x] = v[k];
  __syncthreads();
  if (seg) return;
  for (int s = 1; s < SEG; ++s)
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] = add_mod(v[k], part[s][k][x], q);
}

// The features [k0, k1) of this thread's segment.
template <int SEG>
__device__ __forceinline__ void segment(int n_feat, int& k0, int& k1) {
  const int per = (n_feat + SEG - 1) / SEG, seg = SEG == 1 ? 0 : threadIdx.y;
  k0 = min(n_feat, seg * per);
  k1 = min(n_feat, k0 + per);
}

// Reads every word of the features once: memory.  768 features of 13 limbs at N
// = 2^16 are 10.5 GB, in 1.82-1.88 ms (5.6-5.7 TB/s; 1.95 with a feature's two loads in
// flight).
template <bool WIDE, int SEG>
__global__ __launch_bounds__(SEG == 1 ? 256 : 64 * SEG) void moments_kernel(MomentArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, b = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  int k0, k1;
  segment<SEG>(a.n_feat, k0, k1);
  const uint64_t* x = a.x + ((uint64_t)b * a.n_feat + k0) * 2 * lim + off;
  uint64_t v[5] = {};  // sums of x (two parts) and of x (x) x (three, the middle one halved)
  AccT<WIDE> m0{}, m1{}, m2{};
  auto fold = [&] {
    v[2] = add_mod(v[2], red<WIDE>(m0, pc), pc.q);
    v[3] = add_mod(v[3], red<WIDE>(m1, pc), pc.q);
    v[4] = add_mod(v[4], red<WIDE>(m2, pc), pc.q);
    m0 = m1 = m2 = AccT<WIDE>{};
  };
  auto take = [&](uint64_t x0, uint64_t x1) {
    v[0] = add_mod(v[0], x0, pc.q);
    v[1] = add_mod(v[1], x1, pc.q);
    const Split<WIDE> y0 = split_word<WIDE>(x0), y1 = split_word<WIDE>(x1);
    acc_mac<WIDE>(m0, y0, y0);
    acc_mac<WIDE>(m1, y0, y1);
    acc_mac<WIDE>(m2, y1, y1);
  };
  int k = k0;
  for (; k + 8 <= k1; k += 8, x += 16 * lim) {  // 16 loads in flight, eight products a reduction
    uint64_t y[8][2];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      y[u][0] = x[2 * u * lim];
      y[u][1] = x[(2 * u + 1) * lim];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) take(y[u][0], y[u][1]);
    fold();
  }
  for (; k < k1; ++k, x += 2 * lim) take(x[0], x[lim]);
  fold();
  add_segments<SEG>(v, pc.q);
  if (SEG > 1 && threadIdx.y) return;
  uint64_t* o = a.sum + (uint64_t)b * 2 * lim + off;
  o[0] = v[0];
  o[lim] = v[1];
  // F r - s s: the product of the sums with a minus sign on one factor
  const Const f = constant(a.tab, 3, i, 0), kk = constant(a.tab, 3, i, 1), kept = constant(a.kept, 1, i, 0);
  const Split<WIDE> y0 = split_word<WIDE>(v[0]), y1 = split_word<WIDE>(v[1]);
  const Split<WIDE> n0 = split_word<WIDE>(sub_mod(0, v[0], pc.q)), n1 = split_word<WIDE>(sub_mod(0, v[1], pc.q));
  m0 = m1 = m2 = AccT<WIDE>{};
  acc_mac<WIDE>(m0, y0, n0);
  acc_mac<WIDE>(m1, y0, n1);
  acc_mac<WIDE>(m2, y1, n1);
  const uint64_t v0 = add_mod(times(v[2], f, pc.q), red<WIDE>(m0, pc), pc.q);
  uint64_t v1 = add_mod(times(v[3], f, pc.q), red<WIDE>(m1, pc), pc.q);
  v1 = add_mod(v1, v1, pc.q);
  const uint64_t v2 = add_mod(times(v[4], f, pc.q), red<WIDE>(m2, pc), pc.q);
  uint64_t* d = a.out + (uint64_t)b * 3 * lim + off;
  const uint64_t eps = i < a.nl - 2 ? constant(a.tab, 3, i, 2).w : 0;
  d[0] = add_mod(times(times(v0, kk, pc.q), kept, pc.q), eps, pc.q);
  d[lim] = times(times(v1, kk, pc.q), kept, pc.q);
  d[2 * lim] = times(v2, kk, pc.q);
}

// kFeatures features of a block a thread: r and S are read once for them.  The
// products' arithmetic and memory (an item read, one and a half written) share
// the time: 96 items of 7 limbs at N = 2^16 (1.76 GB) take 454 us, 573 with one
// feature a thread and the dropped primes' inverses one after the other.
constexpr int kFeatures = 4;

template <bool WIDE>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, p0 = a.first + blockIdx.z * kFeatures;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n;
  const Const f = constant(a.feat, 1, i, 0), kept = constant(a.kept, 1, i, 0);
  uint64_t y[kFeatures][2];
#pragma unroll
  for (int u = 0; u < kFeatures; ++u) {
    const uint64_t* x = a.x + (uint64_t)min(p0 + u, a.last - 1) * 2 * xl + off;
    y[u][0] = x[0];
    y[u][1] = x[xl];
  }
  int was = -1;
  uint64_t r0 = 0, r1 = 0, s0 = 0, s1 = 0;
#pragma unroll
  for (int u = 0; u < kFeatures; ++u) {
    const int p = p0 + u, b = p / a.n_feat, feat = p % a.n_feat;
    if (p >= a.last) break;
    if (b != was) {
      const uint64_t* s = a.sum + (uint64_t)b * 2 * xl + off;
      const uint64_t* r = a.r + (uint64_t)b * 2 * lim + off;
      r0 = r[0];
      r1 = r[lim];
      s0 = pc.q - s[0];
      s1 = pc.q - s[xl];
      was = b;
    }
    const Const k = constant(a.gain, a.n_gain, i, feat);
    // F x - S below 2q, then times k
    const uint64_t u0 = times(times(y[u][0], f, pc.q) + s0, k, pc.q);
    const uint64_t u1 = times(times(y[u][1], f, pc.q) + s1, k, pc.q);
    TensorSum<WIDE> t;
    t.add(u0, u1, r0, r1);
    t.store(a.out + (uint64_t)(p - a.first) * 3 * lim + off, lim, kept,
            a.beta && i < a.nl - 2 ? constant(a.beta, a.n_feat, i, feat).w : 0, pc);
  }
}

// 64 features of 8 limbs at N = 2^16, both operands once (1.07 GB): 238 us (4.5
// TB/s), 272 with a feature's four loads in flight.
template <bool WIDE, int SEG>
__global__ __launch_bounds__(SEG == 1 ? 256 : 64 * SEG) void grad_sums_kernel(GradSumArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, b = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n;
  int k0, k1;
  segment<SEG>(a.n_feat, k0, k1);
  const uint64_t* dy = a.dy + ((uint64_t)b * a.n_feat + k0) * 2 * lim + off;
  const uint64_t* xh = a.xhat + ((uint64_t)b * a.n_feat + k0) * 2 * xl + off;
  uint64_t v[5] = {};  // sums of g (two parts) and of g (x) xhat (three)
  TensorSum<WIDE> t;
  auto take = [&](int k, uint64_t d0, uint64_t d1, uint64_t x0, uint64_t x1) {
    const Const w = constant(a.gain, a.n_gain, i, k);
    const uint64_t g0 = times(d0, w, pc.q), g1 = times(d1, w, pc.q);
    v[0] = add_mod(v[0], g0, pc.q);
    v[1] = add_mod(v[1], g1, pc.q);
    t.add(g0, g1, x0, x1);
  };
  int k = k0;
  for (; k + 4 <= k1; k += 4, dy += 8 * lim, xh += 8 * xl) {  // 16 loads in flight
    uint64_t y[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      y[u][0] = dy[2 * u * lim];
      y[u][1] = dy[(2 * u + 1) * lim];
      y[u][2] = xh[2 * u * xl];
      y[u][3] = xh[(2 * u + 1) * xl];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) take(k + u, y[u][0], y[u][1], y[u][2], y[u][3]);
    t.fold(v[2], v[3], v[4], pc);
  }
  for (; k < k1; ++k, dy += 2 * lim, xh += 2 * xl) take(k, dy[0], dy[lim], xh[0], xh[xl]);
  t.fold(v[2], v[3], v[4], pc);
  add_segments<SEG>(v, pc.q);
  if (SEG > 1 && threadIdx.y) return;
  if (i < a.g_nl) {
    uint64_t* o = a.G + (((uint64_t)b * 2 * a.g_nl + i) << a.log_n) + c;
    o[0] = v[0];
    o[(uint64_t)a.g_nl << a.log_n] = v[1];
  }
  const Const kept = constant(a.kept, 1, i, 0);
  uint64_t* d = a.out + (uint64_t)b * 3 * lim + off;
  d[0] = times(v[2], kept, pc.q);
  d[lim] = times(v[3], kept, pc.q);
  d[2 * lim] = v[4];
}

template <bool WIDE>
__global__ __launch_bounds__(256) void scaled_pair_kernel(ScaledPairArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, b = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, rl = (uint64_t)a.r_nl << a.log_n;
  const uint64_t* r = a.r + (uint64_t)b * 2 * rl + off;
  const uint64_t* h = a.h + (uint64_t)b * 2 * lim + off;
  const Const kept = constant(a.kept, 1, i, 0), k = constant(a.k, 1, i, 0);
  TensorSum<WIDE> t;
  t.add(times(r[0], k, pc.q), times(r[rl], k, pc.q), h[0], h[lim]);
  t.store(a.out + (uint64_t)b * 3 * lim + off, lim, kept, 0, pc);
}

// As norm_kernel, with two products: 64 items of 5 limbs at N = 2^16 (1.18 GB) in
// 274 us, 318 with one feature a thread.  Arithmetic: the quotients of four
// constants' products and of the three parts.
template <bool WIDE>
__global__ __launch_bounds__(256) void grad_kernel(GradArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, p0 = a.first + blockIdx.z * kFeatures;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  const uint64_t dl = (uint64_t)a.dy_nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n, rl = (uint64_t)a.r_nl << a.log_n;
  const Const f = constant(a.feat, 1, i, 0), kept = constant(a.kept, 1, i, 0);
  uint64_t y[kFeatures][4];
#pragma unroll
  for (int u = 0; u < kFeatures; ++u) {
    const uint64_t p = min(p0 + u, a.last - 1);
    const uint64_t* dy = a.dy + p * 2 * dl + off;
    const uint64_t* xh = a.xhat + p * 2 * xl + off;
    y[u][0] = dy[0];
    y[u][1] = dy[dl];
    y[u][2] = xh[0];
    y[u][3] = xh[xl];
  }
  int was = -1;
  uint64_t r0 = 0, r1 = 0, g0 = 0, g1 = 0, n0 = 0, n1 = 0;
#pragma unroll
  for (int u = 0; u < kFeatures; ++u) {
    const int p = p0 + u, b = p / a.n_feat, feat = p % a.n_feat;
    if (p >= a.last) break;
    if (b != was) {
      const uint64_t* r = a.r + (uint64_t)b * 2 * rl + off;
      const uint64_t* G = a.G + (uint64_t)b * 2 * lim + off;
      const uint64_t* R = a.R + (uint64_t)b * 2 * lim + off;
      r0 = r[0];
      r1 = r[rl];
      g0 = G[0];
      g1 = G[lim];
      n0 = sub_mod(0, R[0], pc.q);
      n1 = sub_mod(0, R[lim], pc.q);
      was = b;
    }
    const Const k = constant(a.gain, a.n_gain, i, feat);
    TensorSum<WIDE> t;
    t.add(sub_mod(times(mul_shoup_lazy(y[u][0], k.w, k.p, pc.q), f, pc.q), g0, pc.q),
          sub_mod(times(mul_shoup_lazy(y[u][1], k.w, k.p, pc.q), f, pc.q), g1, pc.q), r0, r1);
    t.add(y[u][2], y[u][3], n0, n1);
    t.store(a.out + (uint64_t)(p - a.first) * 3 * lim + off, lim, kept, 0, pc);
  }
}

template <bool WIDE>
__global__ __launch_bounds__(256) void weight_sums_kernel(WeightArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, feat = a.first + blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n, xl = (uint64_t)a.x_nl << a.log_n;
  uint64_t s0 = 0, s1 = 0, v[3] = {};
  TensorSum<WIDE> t;
  for (int b = 0; b < a.n_blk; ++b) {
    const uint64_t p = (uint64_t)b * a.n_feat + feat;
    const uint64_t* dy = a.dy + p * 2 * lim + off;
    const uint64_t d0 = dy[0], d1 = dy[lim];
    s0 = add_mod(s0, d0, pc.q);
    s1 = add_mod(s1, d1, pc.q);
    if (a.out) {
      const uint64_t* xh = a.xhat + p * 2 * xl + off;
      t.add(d0, d1, xh[0], xh[xl]);
      if (b % 4 == 3) t.fold(v[0], v[1], v[2], pc);
    }
  }
  if (a.sum) {
    uint64_t* o = a.sum + (uint64_t)blockIdx.z * 2 * lim + off;
    o[0] = s0;
    o[lim] = s1;
  }
  if (!a.out) return;
  t.fold(v[0], v[1], v[2], pc);
  const Const kept = constant(a.kept, 1, i, 0);
  uint64_t* d = a.out + (uint64_t)blockIdx.z * 3 * lim + off;
  d[0] = times(v[0], kept, pc.q);
  d[lim] = times(v[1], kept, pc.q);
  d[2 * lim] = v[2];
}

}  // namespace

#define NORM_LAUNCH(kern, grid_z, units)                                                                      \
  TraceScope ts(c, s, "layernorm", units);                                                                    \
  hipLaunchKernelGGL(c->wide ? kern<true> : kern<false>, dim3(c->N / 256, a.nl, grid_z), dim3(256), 0, s, a); \
  CKKS_HIP_CHECK(hipGetLastError());                                                                          \
  return CKKS_OK

// Sums over features, in segments or not.
#define SUM_LAUNCH(kern, nb, units)                                                                                  \
  TraceScope ts(c, s, "layernorm", units);                                                                           \
  if ((uint64_t)nb * a.nl * c->N < kSegmentWords && a.n_feat >= kSegments)                                           \
    hipLaunchKernelGGL((c->wide ? kern<true, kSegments> : kern<false, kSegments>), dim3(c->N / 64, a.nl, nb),        \
                       dim3(64, kSegments), 0, s, a);                                                                \
  else                                                                                                               \
    hipLaunchKernelGGL((c->wide ? kern<true, 1> : kern<false, 1>), dim3(c->N / 256, a.nl, nb), dim3(256), 0, s, a);  \
  CKKS_HIP_CHECK(hipGetLastError());                                                                                 \
  return CKKS_OK

int launch_moments(Ctx* c, hipStream_t s, const MomentArgs& a, int nb) {
  SUM_LAUNCH(moments_kernel, nb, (double)nb * a.n_feat * a.nl * 4 * c->N);
}
int launch_norm(Ctx* c, hipStream_t s, const NormArgs& a) {
  const int n = a.last - a.first;
  NORM_LAUNCH(norm_kernel, (n + kFeatures - 1) / kFeatures, (double)n * a.nl * 11 * c->N);
}
int launch_grad_sums(Ctx* c, hipStream_t s, const GradSumArgs& a, int nb) {
  SUM_LAUNCH(grad_sums_kernel, nb, (double)nb * a.n_feat * a.nl * 7 * c->N);
}
int launch_scaled_pair(Ctx* c, hipStream_t s, const ScaledPairArgs& a, int nb) {
  NORM_LAUNCH(scaled_pair_kernel, nb, (double)nb * a.nl * 10 * c->N);
}
int launch_grad(Ctx* c, hipStream_t s, const GradArgs& a) {
  const int n = a.last - a.first;
  NORM_LAUNCH(grad_kernel, (n + kFeatures - 1) / kFeatures, (double)n * a.nl * 15 * c->N);
}
int launch_weight_sums(Ctx* c, hipStream_t s, const WeightArgs& a, int n) {
  NORM_LAUNCH(weight_sums_kernel, n, (double)n * a.n_blk * a.nl * 5 * c->N);
}

}  // namespace ckks
