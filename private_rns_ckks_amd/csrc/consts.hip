// Tables of constants (consts.h).  The host's integers travel in the kernel's
// arguments, 256 a launch, so nothing is copied and a graph keeps its own.
#include "consts.h"

#include <algorithm>

#include "arith.h"

namespace ckks {

namespace {

constexpr int kPerLaunch = 256;

// Constants [start, start + count) of a launch are entries first .. of a table.
struct ConstPart {
  uint64_t* table;
  int n, nl, drop, first, start, count;
};

struct ConstArgs {
  int64_t m[kPerLaunch];
  uint8_t e[kPerLaunch];
  ConstPart part[kMaxConstTables];
  const uint64_t* rescale;
  const PrimeConst* prime;
  int parts, L;
};

__global__ __launch_bounds__(kPerLaunch) void consts_kernel(ConstArgs a) {
  const int k = threadIdx.x, i = blockIdx.x;
  int j = 0;
  while (j < a.parts && k >= a.part[j].start + a.part[j].count) ++j;
  if (j == a.parts || i >= a.part[j].nl) return;
  const ConstPart& p = a.part[j];
  const PrimeConst& pc = a.prime[i];
  const uint64_t q = pc.q;
  const int64_t m = a.m[k];
  uint64_t v = reduce64(m < 0 ? 0 - (uint64_t)m : (uint64_t)m, q, pc.inv1);
  for (int t = 0; t < a.e[k]; ++t) v = add_mod(v, v, q);
  if (m < 0 && v) v = q - v;
  if (i < p.nl - p.drop)
    for (int d = 0; d < p.drop; ++d) {
      const uint64_t* rs = a.rescale + ((uint64_t)(p.nl - 1 - d) * a.L + i) * 4;
      v = reduce_2q(mul_shoup(v, rs[0], rs[1], q), q);
    }
  uint64_t r = v, w = 0;  // floor(v 2^64 / q), a bit at a time: r < q < 2^62
  for (int t = 0; t < 64; ++t) {
    r <<= 1;
    w = w << 1 | (r >= q);
    r = r >= q ? r - q : r;
  }
  uint64_t* o = p.table + ((uint64_t)i * p.n + p.first + k - p.start) * 2;
  o[0] = v;
  o[1] = w;
}

}  // namespace

int launch_consts(Ctx* c, hipStream_t s, const ConstTable* t, int n_tables) {
  ConstArgs a;
  a.rescale = c->d_rescale;
  a.prime = c->d_prime;
  a.L = (int)c->L;
  a.parts = 0;
  int used = 0, limbs = 0;
  auto flush = [&]() -> int {
    if (!used) return CKKS_OK;
    hipLaunchKernelGGL(consts_kernel, dim3(limbs), dim3(kPerLaunch), 0, s, a);
    CKKS_HIP_CHECK(hipGetLastError());
    a.parts = used = limbs = 0;
    return CKKS_OK;
  };
  for (int j = 0; j < n_tables; ++j)
    for (int first = 0; first < t[j].n;) {
      if (used == kPerLaunch || a.parts == kMaxConstTables) {
        int rc = flush();
        if (rc) return rc;
      }
      const int count = std::min(t[j].n - first, kPerLaunch - used);
      a.part[a.parts++] = ConstPart{t[j].table, t[j].n, t[j].nl, t[j].drop, first, used, count};
      limbs = std::max(limbs, t[j].nl);
      for (int k = 0; k < count; ++k) {
        a.m[used + k] = t[j].k[first + k].m;
        a.e[used + k] = (uint8_t)t[j].k[first + k].e;
      }
      used += count;
      first += count;
    }
  return flush();
}

}  // namespace ckks
