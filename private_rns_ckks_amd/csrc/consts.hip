// Tables of constants (consts.h).  The host's integers travel in the kernel's
// arguments, 256 a launch, so nothing is copied and a graph keeps its own.
#include "consts.h"

#include "arith.h"

namespace ckks {

namespace {

constexpr int kPerLaunch = 256;

struct ConstArgs {
  int64_t m[kPerLaunch];
  uint8_t e[kPerLaunch];
  uint64_t* table;
  const uint64_t* rescale;
  const PrimeConst* prime;
  int n, first, count, nl, L, drop;
};

__global__ __launch_bounds__(kPerLaunch) void consts_kernel(ConstArgs a) {
  const int k = threadIdx.x, i = blockIdx.x;
  if (k >= a.count) return;
  const PrimeConst& pc = a.prime[i];
  const uint64_t q = pc.q;
  const int64_t m = a.m[k];
  uint64_t v = reduce64(m < 0 ? 0 - (uint64_t)m : (uint64_t)m, q, pc.inv1);
  for (int t = 0; t < a.e[k]; ++t) v = add_mod(v, v, q);
  if (m < 0 && v) v = q - v;
  if (i < a.nl - a.drop)
    for (int d = 0; d < a.drop; ++d) {
      const uint64_t* rs = a.rescale + ((uint64_t)(a.nl - 1 - d) * a.L + i) * 4;
      v = reduce_2q(mul_shoup(v, rs[0], rs[1], q), q);
    }
  uint64_t r = v, w = 0;  // floor(v 2^64 / q), a bit at a time: r < q < 2^62
  for (int t = 0; t < 64; ++t) {
    r <<= 1;
    w = w << 1 | (r >= q);
    r = r >= q ? r - q : r;
  }
  uint64_t* o = a.table + ((uint64_t)i * a.n + a.first + k) * 2;
  o[0] = v;
  o[1] = w;
}

}  // namespace

int launch_consts(Ctx* c, hipStream_t s, const Whole* k, int n, int nl, int drop, uint64_t* table) {
  ConstArgs a;
  a.table = table;
  a.rescale = c->d_rescale;
  a.prime = c->d_prime;
  a.n = n;
  a.nl = nl;
  a.L = (int)c->L;
  a.drop = drop;
  for (a.first = 0; a.first < n; a.first += kPerLaunch) {
    a.count = n - a.first < kPerLaunch ? n - a.first : kPerLaunch;
    for (int j = 0; j < a.count; ++j) {
      a.m[j] = k[a.first + j].m;
      a.e[j] = (uint8_t)k[a.first + j].e;
    }
    hipLaunchKernelGGL(consts_kernel, dim3(nl), dim3(kPerLaunch), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
  }
  return CKKS_OK;
}

}  // namespace ckks
