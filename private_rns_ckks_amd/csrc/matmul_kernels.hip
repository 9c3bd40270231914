// Kernels of the product with a matrix of 8-bit integers (linear.h).
#include "linear.h"

#include "arith.h"
#include "convert.h"

namespace ckks {

namespace {

constexpr int kRows = 8;  // outputs of a thread

// pack[tile][i][r] = w[j0 + kRows tile + r][i], zero past the last output.
__global__ __launch_bounds__(256) void pack_rows_kernel(MatArgs a, uint64_t* pack) {
  const uint64_t t = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int tiles = (a.nj + kRows - 1) / kRows;
  if (t >= (uint64_t)tiles * a.n_in) return;
  const int tile = (int)(t / a.n_in), i = (int)(t % a.n_in);
  uint64_t v = 0;
  for (int r = 0; r < kRows; ++r) {
    const int j = tile * kRows + r;
    if (j < a.nj) v |= (uint64_t)(uint8_t)a.w[(a.j0 + j) * a.w_row + i * a.w_col] << (8 * r);
  }
  pack[t] = v;
}

// (hi:lo) mod q for a signed 128-bit value below 2^126 in magnitude.
__device__ __forceinline__ uint64_t reduce_signed(__int128 v, const RedConst& pc) {
  const bool neg = v < 0;
  const unsigned __int128 u = neg ? -(unsigned __int128)v : (unsigned __int128)v;
  const uint64_t r = reduce128(U128{(uint64_t)u, (uint64_t)(u >> 64)}, pc.q, pc.r64, pc.r64p, pc.inv1);
  return neg && r ? pc.q - r : r;
}

// What happens to a sum on its way out.
struct Epilogue {
  RedConst pc;
  uint64_t tok;
  const uint64_t *kout, *bias;  // of this limb
  int kstep;  // words between the outputs' constants
  bool has_tok;
  __device__ __forceinline__ uint64_t finish(uint64_t v, int j) const {
    if (kout) v = reduce_2q(mul_shoup(v, kout[j * kstep], kout[j * kstep + 1], pc.q), pc.q);
    if (has_tok) v = mul_mod(v, tok, pc.q, pc.r64, pc.r64p, pc.inv1);
    if (bias) v = add_mod(v, bias[2 * j], pc.q);
    return v;
  }
};

// One word of kRows outputs a thread: the word's 31-bit halves times a byte,
// summed in 64 bits (2^31 2^7 2^16 = 2^54).
__global__ __launch_bounds__(256) void matmul_rows_kernel(MatArgs a, const uint64_t* pack) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  const int comp = blockIdx.y / a.nl, i = blockIdx.y % a.nl;
  const int tiles = (a.nj + kRows - 1) / kRows;
  const int b = blockIdx.z / tiles, tile = blockIdx.z % tiles;
  const uint64_t ct = (uint64_t)(2 * a.nl) << a.log_n;
  const uint64_t* x = a.x + (uint64_t)(a.b0 + b) * a.n_in * ct + ((uint64_t)(comp * a.nl + i) << a.log_n) + c;
  const ConstU64 w = (ConstU64)(pack + (uint64_t)tile * a.n_in);
  Epilogue ep;
  ep.pc = red_const((ConstPrime)a.prime, i);
  const uint64_t q = ep.pc.q;
  const ConstU64 kin = a.kin ? (ConstU64)(a.kin + (uint64_t)i * a.n_in * 2) : nullptr;
  int64_t lo[kRows] = {}, hi[kRows] = {};
  for (int k = 0; k < a.n_in; ++k) {
    uint64_t v = x[k * ct];
    if (kin) v = reduce_2q(mul_shoup(v, kin[2 * k], kin[2 * k + 1], q), q);
    const int32_t l = (int32_t)(v & 0x7fffffff), h = (int32_t)(v >> 31);
    const uint64_t row = w[k];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int32_t m = (int8_t)(row >> (8 * r));
      lo[r] += (int64_t)l * m;
      hi[r] += (int64_t)h * m;
    }
  }
  ep.has_tok = a.tok != nullptr;
  ep.tok = a.tok ? a.tok[((uint64_t)((a.b0 + b) % a.n_tok) * a.nl + i << a.log_n) + c] : 0;
  ep.kout = a.kout ? a.kout + (uint64_t)i * a.n_kout * 2 : nullptr;
  ep.kstep = a.n_kout > 1 ? 2 : 0;
  ep.bias = a.bias && comp == 0 ? a.bias + (uint64_t)i * a.n_out * 2 : nullptr;
  const int low = a.nl - a.drop;
  const uint64_t at = i < low ? ((uint64_t)(comp * low + i) << a.log_n) : ((uint64_t)(comp * a.drop + i - low) << a.log_n);
  uint64_t* o = (i < low ? a.out : a.top) + at + c;
  const uint64_t per = (uint64_t)(i < low ? 2 * low : 2 * a.drop) << a.log_n;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int j = tile * kRows + r;
    if (j >= a.nj) break;
    o[((uint64_t)b * a.nj + j) * per] = ep.finish(reduce_signed((__int128)lo[r] + ((__int128)hi[r] << 31), ep.pc), a.j0 + j);
  }
}

}  // namespace

uint64_t matmul_pack_words(int n_in, int nj) { return (uint64_t)((nj + kRows - 1) / kRows) * n_in; }

int launch_matmul(Ctx* c, hipStream_t s, const MatArgs& a, uint64_t* pack) {
  const int tiles = (a.nj + kRows - 1) / kRows;
  const uint64_t words = matmul_pack_words(a.n_in, a.nj);
  hipLaunchKernelGGL(pack_rows_kernel, dim3((uint32_t)((words + 255) / 256)), dim3(256), 0, s, a, pack);
  CKKS_HIP_CHECK(hipGetLastError());
  TraceScope ts(c, s, "matmul_i8", (double)a.nb * a.nj * a.n_in * 2 * a.nl * c->N);
  hipLaunchKernelGGL(matmul_rows_kernel, dim3(c->N / 256, 2 * a.nl, a.nb * tiles), dim3(256), 0, s, a, pack);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

}  // namespace ckks
