// Slotwise kernels of the attention calls, on ciphertext words in NTT form:
// products with plaintext rows, tensor products and their weighted sums.  One
// thread per word of a limb, blockIdx.y the limb, blockIdx.z the item.
#include "arith.h"
#include "attention.h"
#include "convert.h"

namespace ckks {

namespace {

constexpr int kSegments = 16;  // token segments of the segmented scan
// The scan runs in segments below this many words (groups x limbs x N) and
// from kSegments tokens on: one thread a word then leaves most of the chip
// empty, while the segments' second pass over the output costs a full chip
// more.  Scan and state product of 96 tokens of 2^14.8 words: 92 us in
// segments, 206 us without; 32 tokens of 2^16.2: 87 and 98; of 2^17.2: 159 and
// 141; 16 tokens of 2^20.6: 910 and 563.
constexpr uint64_t kSegmentWords = 3u << 15;

template <bool WIDE>
__device__ __forceinline__ uint64_t mul_red(const Split<WIDE>& x, const Split<WIDE>& y, const RedConst& pc) {
  AccT<WIDE> m{};
  acc_mac<WIDE>(m, x, y);
  return acc_reduce<WIDE>(m, pc.q, pc.r64, pc.r64p, pc.inv1);
}

// Part 0 or 1 (component comp) of limb i as DropOut says.
__device__ __forceinline__ uint64_t drop_out(uint64_t x, const DropOut& d, int nl, int i, const uint64_t* add,
                                             uint64_t add_off, uint64_t q) {
  if (i >= nl - d.drop) return x;
  for (int k = 0; k < d.drop; ++k) {
    const ConstU64 rs = (ConstU64)(d.rescale + ((uint64_t)(nl - 1 - k) * d.L + i) * 4);
    x = mul_shoup_lazy(x, rs[0], rs[1], q);
  }
  x = reduce_4q(x, q);
  return add ? add_mod(x, add[add_off], q) : x;
}

struct TopMulArgs {
  PlainMul m;
  uint64_t* out;
  uint64_t out_bstride;
  const PrimeConst* prime;
  int log_n;
};

// The limb of a product with a plaintext row that its rescale drops; the other
// limbs' products are formed where the rescale reads them.
template <bool WIDE>
__global__ __launch_bounds__(256) void plain_mul_kernel(TopMulArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int l = a.m.level, b = blockIdx.z, t = (a.m.first + b) / a.m.ng, g = (a.m.first + b) % a.m.ng;
  const RedConst pc = red_const((ConstPrime)a.prime, l);
  const uint64_t off = ((uint64_t)l << a.log_n) + c, lim = (uint64_t)(l + 1) << a.log_n;
  const uint64_t row = (uint64_t)t * a.m.n_row + (a.m.g0 + g) % a.m.n_row;
  const Split<WIDE> p = split_word<WIDE>(a.m.p[row * lim + off]);
  const uint64_t* x = a.m.in + ((uint64_t)t * a.m.n_grp + g) * a.m.in_bstride + off;
  uint64_t* o = a.out + b * a.out_bstride + c;
  o[0] = mul_red<WIDE>(p, split_word<WIDE>(x[0]), pc);
  o[1ull << a.log_n] = mul_red<WIDE>(p, split_word<WIDE>(x[a.m.in_comp]), pc);
}

// (x0, x1) x (y0, y1) = (x0 y0, x0 y1 + x1 y0, x1 y1), plus a row times a
// second ciphertext (the decayed state) in the same column sums; parts 0 and 1
// leave ready for the rescales to come (drop_out).  8 products of 24 limbs at N
// = 2^16 move 503 MB in 125-127 us (4.0 TB/s): memory, with five loads a
// thread in flight; two words a thread take the same time.
template <bool WIDE>
__global__ __launch_bounds__(256) void pair_kernel(PairArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y;
  const int item = blockIdx.z, p = a.first + item;
  const int ia = a.n_k ? p / a.n_k : p;
  const int ib = a.n_k ? (p / a.n_qk) * a.n_k + p % a.n_k : (p / a.ng) * a.n_grp + p % a.ng;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  const uint64_t* x = a.a + ia * a.a_bstride + off;
  const uint64_t* y = a.b + ib * a.b_bstride + off;
  uint64_t* d = a.out + (uint64_t)item * 3 * lim + off;
  const Split<WIDE> x0 = split_word<WIDE>(x[0]), x1 = split_word<WIDE>(x[a.a_comp]);
  const Split<WIDE> y0 = split_word<WIDE>(y[0]), y1 = split_word<WIDE>(y[a.b_comp]);
  AccT<WIDE> m0{}, m1{}, m2{};
  acc_mac<WIDE>(m0, x0, y0);
  acc_mac<WIDE>(m1, x0, y1);
  acc_mac<WIDE>(m1, x1, y0);
  acc_mac<WIDE>(m2, x1, y1);
  if (a.decay) {
    const uint64_t* st = a.state + p * a.state_bstride + off;
    const Split<WIDE> g = split_word<WIDE>(a.decay[(uint64_t)(p % a.n_row) * lim + off]);
    acc_mac<WIDE>(m0, g, split_word<WIDE>(st[0]));
    acc_mac<WIDE>(m1, g, split_word<WIDE>(st[lim]));
  }
  const uint64_t low = (uint64_t)(a.nl - a.drop.drop) << a.log_n;
  const uint64_t* add = a.add ? a.add + p * a.add_bstride : nullptr;
  d[0] = drop_out(acc_reduce<WIDE>(m0, pc.q, pc.r64, pc.r64p, pc.inv1), a.drop, a.nl, i, add, off, pc.q);
  d[lim] = drop_out(acc_reduce<WIDE>(m1, pc.q, pc.r64, pc.r64p, pc.inv1), a.drop, a.nl, i, add, low + off, pc.q);
  d[2 * lim] = acc_reduce<WIDE>(m2, pc.q, pc.r64, pc.r64p, pc.inv1);
}

// r += (a0, a1) x (v0, v1), three parts.
template <bool WIDE>
__device__ __forceinline__ void tensor_add(const Split<WIDE>& a0, const Split<WIDE>& a1, uint64_t v0, uint64_t v1,
                                           const RedConst& pc, uint64_t& r0, uint64_t& r1, uint64_t& r2) {
  const Split<WIDE> b0 = split_word<WIDE>(v0), b1 = split_word<WIDE>(v1);
  AccT<WIDE> m0{}, m1{}, m2{};
  acc_mac<WIDE>(m0, a0, b0);
  acc_mac<WIDE>(m1, a0, b1);
  acc_mac<WIDE>(m1, a1, b0);
  acc_mac<WIDE>(m2, a1, b1);
  r0 = add_mod(r0, acc_reduce<WIDE>(m0, pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
  r1 = add_mod(r1, acc_reduce<WIDE>(m1, pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
  r2 = add_mod(r2, acc_reduce<WIDE>(m2, pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
}

// r += (w k) x v.
template <bool WIDE>
__device__ __forceinline__ void weigh_add(const Split<WIDE>& w, uint64_t k0, uint64_t k1, uint64_t v0, uint64_t v1,
                                          const RedConst& pc, uint64_t& r0, uint64_t& r1, uint64_t& r2) {
  tensor_add<WIDE>(split_word<WIDE>(mul_red<WIDE>(w, split_word<WIDE>(k0), pc)),
                   split_word<WIDE>(mul_red<WIDE>(w, split_word<WIDE>(k1), pc)), v0, v1, pc, r0, r1, r2);
}

// out[t] = sum of (w_j k_j) x v_j over j <= t: the running sums stay in
// registers (canonical words: every prefix is a result), each operand is read
// once and each prefix written once.  3 tokens of 2 groups of 24 limbs at N =
// 2^16 move 650 MB in 144-150 us beside the products r q (4.3-4.5 TB/s).
template <bool WIDE>
__global__ __launch_bounds__(256) void scan_kernel(ScanArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, g = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  const uint64_t row = (uint64_t)((a.g0 + g) % a.n_row);
  uint64_t r0 = 0, r1 = 0, r2 = 0;
  if (a.init) {
    const uint64_t* x = a.init + (uint64_t)g * 3 * lim + off;
    r0 = x[0];
    r1 = x[lim];
    r2 = x[2 * lim];
  }
  const uint64_t low = (uint64_t)(a.nl - a.drop.drop) << a.log_n;
  const uint64_t* add = a.add ? a.add + (uint64_t)g * 2 * low : nullptr;
  for (int t = 0; t < a.n_tok; ++t) {
    const uint64_t* k = a.k + t * a.tok_stride + (uint64_t)g * 2 * lim + off;
    const uint64_t* v = a.v + t * a.tok_stride + (uint64_t)g * 2 * lim + off;
    const Split<WIDE> w = split_word<WIDE>(a.w[((uint64_t)t * a.n_row + row) * lim + off]);
    weigh_add<WIDE>(w, k[0], k[lim], v[0], v[lim], pc, r0, r1, r2);
    uint64_t* o = a.out + ((uint64_t)t * a.n_grp + g) * 3 * lim + off;
    o[0] = drop_out(r0, a.drop, a.nl, i, add, off, pc.q);
    o[lim] = drop_out(r1, a.drop, a.nl, i, add, low + off, pc.q);
    o[2 * lim] = r2;
  }
  if (a.last) {
    uint64_t* o = a.last + (uint64_t)g * 3 * lim + off;
    o[0] = r0;
    o[lim] = r1;
    o[2 * lim] = r2;
  }
}

// The same for few groups on a small ring, where one thread per word leaves
// the chip empty: the workgroup's blockDim.y threads of a word take segments
// of the tokens, form their own prefix sums (left in out), exchange the
// segments' totals, and add what lies before their segment.
template <bool WIDE>
__global__ __launch_bounds__(64 * kSegments) void scan_segments_kernel(ScanArgs a) {
  __shared__ uint64_t total[kSegments][3][64];
  const int x = threadIdx.x, seg = threadIdx.y;
  const uint32_t c = blockIdx.x * 64 + x;
  const int i = blockIdx.y, g = blockIdx.z;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  const uint64_t row = (uint64_t)((a.g0 + g) % a.n_row);
  const int per = (a.n_tok + kSegments - 1) / kSegments;
  const int t0 = min(a.n_tok, seg * per), t1 = min(a.n_tok, t0 + per);
  uint64_t r0 = 0, r1 = 0, r2 = 0;
  for (int t = t0; t < t1; ++t) {
    const uint64_t* k = a.k + t * a.tok_stride + (uint64_t)g * 2 * lim + off;
    const uint64_t* v = a.v + t * a.tok_stride + (uint64_t)g * 2 * lim + off;
    const Split<WIDE> w = split_word<WIDE>(a.w[((uint64_t)t * a.n_row + row) * lim + off]);
    weigh_add<WIDE>(w, k[0], k[lim], v[0], v[lim], pc, r0, r1, r2);
    uint64_t* o = a.out + ((uint64_t)t * a.n_grp + g) * 3 * lim + off;
    o[0] = r0;
    o[lim] = r1;
    o[2 * lim] = r2;
  }
  total[seg][0][x] = r0;
  total[seg][1][x] = r1;
  total[seg][2][x] = r2;
  uint64_t b0 = 0, b1 = 0, b2 = 0;
  if (a.init) {
    const uint64_t* p = a.init + (uint64_t)g * 3 * lim + off;
    b0 = p[0];
    b1 = p[lim];
    b2 = p[2 * lim];
  }
  __syncthreads();  // totals written; init read by every segment before `last` is
  for (int s = 0; s < seg; ++s) {
    b0 = add_mod(b0, total[s][0][x], pc.q);
    b1 = add_mod(b1, total[s][1][x], pc.q);
    b2 = add_mod(b2, total[s][2][x], pc.q);
  }
  const uint64_t low = (uint64_t)(a.nl - a.drop.drop) << a.log_n;
  const uint64_t* add = a.add ? a.add + (uint64_t)g * 2 * low : nullptr;
  for (int t = t0; t < t1; ++t) {
    uint64_t* o = a.out + ((uint64_t)t * a.n_grp + g) * 3 * lim + off;
    const uint64_t x0 = add_mod(o[0], b0, pc.q), x1 = add_mod(o[lim], b1, pc.q), x2 = add_mod(o[2 * lim], b2, pc.q);
    o[0] = drop_out(x0, a.drop, a.nl, i, add, off, pc.q);
    o[lim] = drop_out(x1, a.drop, a.nl, i, add, low + off, pc.q);
    o[2 * lim] = x2;
    if (a.last && t == a.n_tok - 1) {
      uint64_t* p = a.last + (uint64_t)g * 3 * lim + off;
      p[0] = x0;
      p[lim] = x1;
      p[2 * lim] = x2;
    }
  }
}

// num = sum_j (m_j a_j) x v_j and den = sum_j m_j a_j.  The middle part's
// columns take eight products, so the tensor sums are reduced once per four
// terms; the masked words m_j a_j once each.  6 rows of 4 masked terms and 13
// limbs at N = 2^16 (778 MB with each operand once): 181 us, 251 with a
// reduction per term; the reductions and the memory share the time.
template <bool WIDE>
__global__ __launch_bounds__(256) void mix_kernel(MixArgs a) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int i = blockIdx.y, b = blockIdx.z;
  const int row = a.first + b, g = row / a.n_q;
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t off = ((uint64_t)i << a.log_n) + c, lim = (uint64_t)a.nl << a.log_n;
  uint64_t r0 = 0, r1 = 0, r2 = 0, e0 = 0, e1 = 0;
  AccT<WIDE> m0{}, m1{}, m2{};
  int since = 0;
  for (int j = 0; j < a.n_k; ++j) {
    const uint64_t* x = a.a + ((uint64_t)row * a.n_k + j) * 2 * lim + off;
    const uint64_t* v = a.v + ((uint64_t)g * a.n_k + j) * 2 * lim + off;
    uint64_t a0 = x[0], a1 = x[lim];
    if (a.m) {
      const Split<WIDE> m = split_word<WIDE>(a.m[((uint64_t)(g % a.n_row) * a.n_k + j) * lim + off]);
      a0 = mul_red<WIDE>(m, split_word<WIDE>(a0), pc);
      a1 = mul_red<WIDE>(m, split_word<WIDE>(a1), pc);
    }
    e0 = add_mod(e0, a0, pc.q);
    e1 = add_mod(e1, a1, pc.q);
    const Split<WIDE> a0s = split_word<WIDE>(a0), a1s = split_word<WIDE>(a1);
    const Split<WIDE> v0 = split_word<WIDE>(v[0]), v1 = split_word<WIDE>(v[lim]);
    acc_mac<WIDE>(m0, a0s, v0);
    acc_mac<WIDE>(m1, a0s, v1);
    acc_mac<WIDE>(m1, a1s, v0);
    acc_mac<WIDE>(m2, a1s, v1);
    if (++since == 4 || j + 1 == a.n_k) {  // m1 holds the 8 products its columns take
      r0 = add_mod(r0, acc_reduce<WIDE>(m0, pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
      r1 = add_mod(r1, acc_reduce<WIDE>(m1, pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
      r2 = add_mod(r2, acc_reduce<WIDE>(m2, pc.q, pc.r64, pc.r64p, pc.inv1), pc.q);
      m0 = m1 = m2 = AccT<WIDE>{};
      since = 0;
    }
  }
  uint64_t* o = a.num + (uint64_t)b * 3 * lim + off;
  o[0] = drop_out(r0, a.drop, a.nl, i, nullptr, 0, pc.q);
  o[lim] = drop_out(r1, a.drop, a.nl, i, nullptr, 0, pc.q);
  o[2 * lim] = r2;
  if (a.den) {
    uint64_t* e = a.den + (uint64_t)b * 2 * lim + off;
    e[0] = e0;
    e[lim] = e1;
  }
}

}  // namespace

#define ATTN_LAUNCH(kern, batch)                                                                             \
  hipLaunchKernelGGL(c->wide ? kern<true> : kern<false>, dim3(c->N / 256, a.nl, batch), dim3(256), 0, s, a); \
  CKKS_HIP_CHECK(hipGetLastError());                                                                         \
  return CKKS_OK

int launch_plain_mul(Ctx* c, hipStream_t s, const PlainMul& m, uint64_t* out, uint64_t out_bstride, int batch) {
  const TopMulArgs a{m, out, out_bstride, c->d_prime, (int)c->log_n};
  TraceScope ts(c, s, "attn_mac", (double)batch * 4 * c->N);
  hipLaunchKernelGGL(c->wide ? plain_mul_kernel<true> : plain_mul_kernel<false>, dim3(c->N / 256, 1, batch), dim3(256),
                     0, s, a);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

int launch_pair(Ctx* c, hipStream_t s, const PairArgs& a, int batch) {
  TraceScope ts(c, s, "attn_mac", (double)batch * a.nl * (a.decay ? 9 : 7) * c->N);
  ATTN_LAUNCH(pair_kernel, batch);
}

int launch_scan(Ctx* c, hipStream_t s, const ScanArgs& a) {
  TraceScope ts(c, s, "attn_mac", (double)a.n_tok * a.n_grp * a.nl * 11 * c->N);
  if ((uint64_t)a.n_grp * a.nl * c->N < kSegmentWords && a.n_tok >= kSegments) {
    hipLaunchKernelGGL(c->wide ? scan_segments_kernel<true> : scan_segments_kernel<false>, dim3(c->N / 64, a.nl, a.n_grp),
                       dim3(64, kSegments), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
    return CKKS_OK;
  }
  ATTN_LAUNCH(scan_kernel, a.n_grp);
}

int launch_mix(Ctx* c, hipStream_t s, const MixArgs& a, int rows) {
  TraceScope ts(c, s, "attn_mac", (double)rows * a.n_k * a.nl * 11 * c->N);
  ATTN_LAUNCH(mix_kernel, rows);
}

}  // namespace ckks
