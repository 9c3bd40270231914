// Sum over a packed axis: stages of x + sum_r Rot_r(x) with one decomposition
// and one ModDown per stage (see ckks_sum_steps in include/ckks.h).
#include <string.h>

#include "arith.h"
#include "attention.h"
#include "automorph.h"

namespace ckks {

namespace {

struct SumIPArgs {
  const uint64_t* E;  // item b: E + b*E_bstride, [beta][next][N] raised digits
  const uint64_t* T;  // item b: T + b*T_bstride, c1 [nq][N] (limbs inside their own digit)
  uint64_t* acc;      // item b: acc + b*acc_bstride, [2][next][N]
  uint64_t E_bstride, T_bstride, acc_bstride;
  const uint64_t* evk[kMaxSumRot];
  uint32_t g[kMaxSumRot];
  const PrimeConst* prime;
  int log_n, level, next, beta, alpha, L, K, n_rot;
};

// acc_b[t][w] = sum_r sum_j D_j[t][pi_{g_r}(w)] * evk_{r,j}.b[t][w] (and acc_a).
__global__ __launch_bounds__(256) void sum_ip_kernel(SumIPArgs a) {
  constexpr int W = 4;  // consecutive output words per thread
  const int t = blockIdx.y, item = blockIdx.z;
  const int keyl = t <= a.level ? t : a.L + (t - a.level - 1);
  const PrimeConst& pc = a.prime[keyl];
  const uint64_t q = pc.q, mp = pc.mprime;
  const int log_n = a.log_n;
  const uint32_t w0 = (blockIdx.x * blockDim.x + threadIdx.x) * W;
  const uint64_t LKN = (uint64_t)(a.L + a.K) << log_n;
  uint64_t accb[W], acca[W];
#pragma unroll
  for (int i = 0; i < W; ++i) accb[i] = acca[i] = 0;
  const int fold = mont_fold(q);
  int since = 0;
  for (int r = 0; r < a.n_rot; ++r) {
    uint32_t src[W];
#pragma unroll
    for (int i = 0; i < W; ++i) src[i] = automorph_src(w0 + i, a.g[r], log_n);
    const uint64_t* evk = a.evk[r] + ((uint64_t)keyl << log_n) + w0;
    for (int j = 0; j < a.beta; ++j) {
      const bool in_digit = t >= j * a.alpha && t < (j + 1) * a.alpha && t <= a.level;
      const uint64_t* d = in_digit ? a.T + item * a.T_bstride + ((uint64_t)t << log_n)
                                   : a.E + item * a.E_bstride + ((uint64_t)(j * a.next + t) << log_n);
      const uint64_t* kb = evk + (uint64_t)(2 * j) * LKN;
      const uint64_t* ka = evk + (uint64_t)(2 * j + 1) * LKN;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint64_t x = d[src[i]];
        accb[i] += mont_mul_lazy(x, kb[i], q, mp);
        acca[i] += mont_mul_lazy(x, ka[i], q, mp);
      }
      if (++since == fold) {  // mont_fold(m) products since the last reduction
        since = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          accb[i] = reduce64(accb[i], q, pc.inv1);
          acca[i] = reduce64(acca[i], q, pc.inv1);
        }
      }
    }
  }
  uint64_t* ob = a.acc + item * a.acc_bstride + ((uint64_t)t << log_n) + w0;
  uint64_t* oa = ob + ((uint64_t)a.next << log_n);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    ob[i] = reduce_4q(mul_shoup_lazy(accb[i], pc.r64, pc.r64p, q), q);
    oa[i] = reduce_4q(mul_shoup_lazy(acca[i], pc.r64, pc.r64p, q), q);
  }
}

struct SumCombineArgs {
  const uint64_t* acc;  // [2][next][N] per item
  const uint64_t* w;    // [2][nq][N] per item: NTT of the ModDown conversion
  const uint64_t* ct;   // [2][nq][N] per item: the stage's input
  uint64_t acc_bstride, w_bstride, ct_bstride;
  uint64_t* out[kSumItems];  // [2][nq][N]
  const uint64_t* pinv;  // [L][2]
  const PrimeConst* prime;
  uint32_t g[kMaxSumRot];
  int log_n, nq, next, n_rot;
};

// out_c = acc_c P^-1 - w_c + ct_c (+ sum_r tau_{g_r}(ct_0) for c = 0)
__global__ __launch_bounds__(256) void sum_combine_kernel(SumCombineArgs a) {
  const uint32_t j = blockIdx.x * blockDim.x + threadIdx.x;
  const int comp = blockIdx.y / a.nq, i = blockIdx.y % a.nq, item = blockIdx.z;
  const uint64_t q = a.prime[i].q;
  const uint64_t* ct = a.ct + item * a.ct_bstride + ((uint64_t)blockIdx.y << a.log_n);
  const uint64_t v = a.acc[item * a.acc_bstride + ((uint64_t)(comp * a.next + i) << a.log_n) + j];
  const uint64_t w = a.w[item * a.w_bstride + ((uint64_t)blockIdx.y << a.log_n) + j];
  uint64_t r = sub_mod(reduce_4q(mul_shoup_lazy(v, a.pinv[2 * i], a.pinv[2 * i + 1], q), q), w, q);
  r = add_mod(r, ct[j], q);
  if (comp == 0)
    for (int k = 0; k < a.n_rot; ++k) r = add_mod(r, ct[automorph_src(j, a.g[k], a.log_n)], q);
  a.out[item][((uint64_t)blockIdx.y << a.log_n) + j] = r;
}

// Words per item: decomposition, accumulators, ModDown conversion.
size_t stage_words(const Ctx* c, int level) { return ks_dec_words(c, level) + ks_back_words(c, level); }

// One stage on n items (n <= kSumItems).
int sum_stage(Ctx* c, hipStream_t s, const uint64_t* in, uint64_t in_stride, uint64_t* const* out, int n, int level,
              int n_rot, const uint32_t* g, const uint64_t* const* evk, uint64_t* ws) {
  const uint32_t N = c->N;
  const int nq = level + 1, next = nq + (int)c->K, K = (int)c->K;
  const uint64_t dec_per = ks_dec_words(c, level), per = ks_back_words(c, level);
  uint64_t* dec = ws;
  uint64_t* A = ws + dec_per * n;
  uint64_t* W = A + 2ull * next * N;
  const uint64_t* c1 = in + (uint64_t)nq * N;
  int rc = ks_decompose(c, s, level, n, c1, in_stride, dec, dec_per);
  if (rc) return rc;
  {
    SumIPArgs a;
    memset(&a, 0, sizeof(a));
    a.E = dec + (uint64_t)nq * N;
    a.E_bstride = dec_per;
    a.T = c1;
    a.T_bstride = in_stride;
    a.acc = A;
    a.acc_bstride = per;
    for (int r = 0; r < n_rot; ++r) {
      a.evk[r] = evk[r];
      a.g[r] = g[r];
    }
    a.prime = c->d_prime;
    a.log_n = (int)c->log_n;
    a.level = level;
    a.next = next;
    a.beta = c->beta(level);
    a.alpha = (int)c->alpha;
    a.L = (int)c->L;
    a.K = K;
    a.n_rot = n_rot;
    TraceScope ts(c, s, "sum_ip", (double)n * next * N * (2.0 * a.beta * n_rot + 2));
    hipLaunchKernelGGL(sum_ip_kernel, dim3(N / 1024, next, n), dim3(256), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
  }
  {
    NttJobs jobs;
    uint32_t off[kMaxJobs];
    for (int comp = 0; comp < 2; ++comp)
      for (int k = 0; k < K; ++k) {
        off[jobs.n] = (uint32_t)(c->md.phinv + 2 * k);
        jobs.add(comp * next + nq + k, comp * next + nq + k, (int)c->L + k);
      }
    if ((rc = ntt_run_scaled(c, s, A, A, per, per, n, jobs, true, 2, c->d_moddown, off))) return rc;
  }
  {
    ModDownArgs md;
    memset(&md, 0, sizeof(md));
    md.acc = A;
    md.w = W;
    md.acc_bstride = per;
    md.w_bstride = per;
    md.conv = c->d_moddown + c->md.conv;
    md.prime = c->d_prime;
    md.n = N;
    md.level = level;
    md.acc_comp_limbs = next;
    md.acc_k0 = nq;
    md.L = (int)c->L;
    md.K = K;
    if ((rc = launch_moddown_conv(c, s, md, n))) return rc;
    NttJobs jobs;
    for (int i = 0; i < 2 * nq; ++i) jobs.add(i, i, i % nq);
    if ((rc = ntt_pass_only(c, s, W, W, per, per, n, jobs, false, true, 0, nullptr, nullptr))) return rc;
    if ((rc = ntt_pass_only(c, s, W, W, per, per, n, jobs, false, false, 0, nullptr, nullptr))) return rc;
  }
  SumCombineArgs a;
  memset(&a, 0, sizeof(a));
  a.acc = A;
  a.w = W;
  a.ct = in;
  a.acc_bstride = per;
  a.w_bstride = per;
  a.ct_bstride = in_stride;
  for (int b = 0; b < n; ++b) a.out[b] = out[b];
  a.pinv = c->d_moddown + c->md.pinv;
  a.prime = c->d_prime;
  for (int r = 0; r < n_rot; ++r) a.g[r] = g[r];
  a.log_n = (int)c->log_n;
  a.nq = nq;
  a.next = next;
  a.n_rot = n_rot;
  TraceScope ts(c, s, "sum_combine", (double)n * 2 * nq * N);
  hipLaunchKernelGGL(sum_combine_kernel, dim3(N / 256, 2 * nq, n), dim3(256), 0, s, a);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

}  // namespace

size_t sum_ws_words(const Ctx* c, int level, int batch, int n_stage) {
  const size_t n = (size_t)(batch < kSumItems ? batch : kSumItems);
  const size_t ct = 2 * (size_t)(level + 1) * c->N;
  return n * (stage_words(c, level) + (n_stage > 1 ? 2 * ct : 0));
}

int sum_stages(Ctx* c, hipStream_t s, const uint64_t* in, uint64_t in_stride, uint64_t* const* out, int batch,
               int level, const ckks_sum_steps& st, uint64_t* ws) {
  const uint64_t ct = 2ull * (level + 1) * c->N;
  for (int b0 = 0; b0 < batch; b0 += kSumItems) {
    const int n = batch - b0 < kSumItems ? batch - b0 : kSumItems;
    // the stages between the first and the last alternate between two buffers
    uint64_t* half[2] = {ws + n * stage_words(c, level), ws + n * (stage_words(c, level) + ct)};
    const uint64_t* src = in + b0 * in_stride;
    uint64_t src_stride = in_stride;
    int at = 0;
    for (int k = 0; k < st.n_stage; ++k) {
      uint64_t* dst[kSumItems];
      for (int b = 0; b < n; ++b) dst[b] = k == st.n_stage - 1 ? out[b0 + b] : half[k & 1] + b * ct;
      int rc = sum_stage(c, s, src, src_stride, dst, n, level, st.radix[k] - 1, st.galois_elts + at, st.d_evks + at, ws);
      if (rc) return rc;
      at += st.radix[k] - 1;
      src = half[k & 1];
      src_stride = ct;
    }
  }
  return CKKS_OK;
}

}  // namespace ckks
