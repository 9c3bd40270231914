// Kernels of the product with a matrix of 8-bit integers (linear.h).
#include "linear.h"

#include <algorithm>

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

// ---------------------------------------------------------------------------
// The product on the matrix cores.  A word x <= 127 sum_d 2^(8d), d < ND, is
// sum_d s_d 2^(8d) with signed bytes s_d: the bytes of x + 128 sum_d 2^(8d), minus
// 128 each.  ND products of bytes with 32-bit sums (|s_d w| n_in <= 2^7 2^7 2^16)
// then give the sum exactly, and the epilogue joins them modulo the prime.
//
// A workgroup of 4 waves takes 32 WM outputs x 32 WN words of one limb; a wave
// 32 outputs x 32 words, all digits, 16 ND accumulators a lane, so that two
// workgroups share a CU: one's epilogue and conversions run beside the other's
// matrix instructions.  The words of a step of 128 / WN inputs (16 a thread, of
// one column) load while the step before is multiplied, are split into digits
// and laid in LDS in the order the instructions take them (16 inputs of a word
// and digit together); the matrix comes from L2 in that order already.

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// Inputs go in groups of 16; the last group starts at n_in - 16, and the inputs
// it shares with the one before have zeros in the matrix.
__device__ __forceinline__ int group_start(int group, int n_in) { return min(group * 16, n_in - 16); }

// pack[row tile of 32][chunk of 32 inputs][lane][16]: the bytes of output row tile
// 32 + lane % 32 at group chunk 2 + lane / 32, zero outside the matrix.
__global__ __launch_bounds__(256) void pack_tiles_kernel(MatArgs a, int chunks, int tiles, uint4* pack) {
  const uint64_t t = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= (uint64_t)tiles * chunks * 64) return;
  const int lane = (int)(t & 63), chunk = (int)((t >> 6) % chunks), tile = (int)((t >> 6) / chunks);
  const int j = tile * 32 + (lane & 31), group = chunk * 2 + (lane >> 5), i0 = group_start(group, a.n_in);
  uint32_t v[4] = {};
  if (j < a.nj)
    for (int k = 0; k < 16; ++k)
      if (i0 + k >= group * 16)
        v[k >> 2] |= (uint32_t)(uint8_t)a.w[(a.j0 + j) * a.w_row + (i0 + k) * a.w_col] << (8 * (k & 3));
  pack[t] = make_uint4(v[0], v[1], v[2], v[3]);
}

// Bytes 0..3 of four words, one dword a byte position.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&o)[4]) {
  const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400), cd0 = __builtin_amdgcn_perm(d, c, 0x05010400);
  const uint32_t ab1 = __builtin_amdgcn_perm(b, a, 0x07030602), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602);
  o[0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100);
  o[1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302);
  o[2] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100);
  o[3] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302);
}

// Digits of four words of a column (a dword of each digit's 16 bytes).
template <int ND>
__device__ __forceinline__ void digits4(const uint64_t* x, uint32_t (&dig)[ND]) {
  constexpr uint64_t kHalf = 0x8080808080808080ull >> (8 * (8 - ND));
  uint64_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = x[k] + kHalf;
  uint32_t o[4];
  transpose4((uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3], o);
#pragma unroll
  for (int d = 0; d < 4; ++d) dig[d] = o[d] ^ 0x80808080u;
  if (ND > 4) {
    transpose4((uint32_t)(v[0] >> 32), (uint32_t)(v[1] >> 32), (uint32_t)(v[2] >> 32), (uint32_t)(v[3] >> 32), o);
#pragma unroll
    for (int d = 4; d < ND; ++d) dig[d] = o[d - 4] ^ 0x80808080u;
  }
}

// a w0 + b w1 mod q, canonical; below 2^56 (ND < 8) the cheaper quotients' 8q fits.
template <int ND>
__device__ __forceinline__ uint64_t join(uint64_t a, const ulonglong2& w0, uint64_t b, const ulonglong2& w1, uint64_t q) {
  if (ND == 8) return reduce_4q(mul_shoup(a, w0.x, w0.y, q) + mul_shoup(b, w1.x, w1.y, q), q);
  uint64_t v = mul_shoup_lazy_split(a, w0.x, w0.y, q);
  if (ND > 4) v += mul_shoup_lazy_split(b, w1.x, w1.y, q);
  v = v >= 4 * q ? v - 4 * q : v;
  return reduce_4q(v, q);
}

template <int ND, int WM, int WN, bool SCALED>
__global__ __launch_bounds__(256, 2) void matmul_tiles_kernel(MatArgs a, const uint4* pack, int chunks, int row_blocks,
                                                              int col_blocks) {
  static_assert(WM * WN == 4, "four waves");
  constexpr int KS = 128 / WN, NC = KS / 32, W = 32 * WN, ROWS = 32 * WM;  // inputs and chunks of a step, a tile
  __shared__ union {
    uint4 dig[2][ND][KS / 16][W];
    ulonglong2 sums[16][256];  // the epilogue's
  } lds;
  __shared__ ulonglong2 kc[ROWS][2];  // {k, Shoup}, {2^32 k, Shoup} of the tile's outputs
  __shared__ ulonglong2 kin[2][SCALED ? KS : 1];
  // Workgroups go round the 8 XCDs: each takes a range of the words, the tiles
  // of the same words next to each other, so that its L2 reads them once.
  const int slot = blockIdx.x >> 3, per_xcd = (col_blocks + 7) / 8;
  const int rb = slot % row_blocks, cb = (blockIdx.x & 7) * per_xcd + slot / row_blocks;
  if (slot / row_blocks >= per_xcd || cb >= col_blocks) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, wm = wave / WN, wn = wave % WN;
  const int per_limb = 1 << (a.log_n - (WN == 1 ? 5 : WN == 2 ? 6 : 7));
  const int poly = cb / per_limb, col0 = (cb % per_limb) * W;  // poly = (b, comp, limb)
  const int i = poly % a.nl, comp = poly / a.nl % 2, b = poly / (2 * a.nl);
  const RedConst pc = red_const((ConstPrime)a.prime, i);
  const uint64_t ct = (uint64_t)(2 * a.nl) << a.log_n;
  const uint64_t* x = a.x + (uint64_t)(a.b0 + b) * a.n_in * ct + ((uint64_t)(comp * a.nl + i) << a.log_n) + col0;
  const int col = tid % W, grp = tid / W;  // this thread's word and group of a step
  const int steps = chunks / NC;
  const ulonglong2* kin_i = SCALED ? (const ulonglong2*)(a.kin + (uint64_t)i * a.n_in * 2) : nullptr;

  for (int r = tid; r < ROWS; r += 256) {  // outputs past the last: those of the last
    const int j = a.n_kout > 1 ? a.j0 + min(rb * ROWS + r, a.nj - 1) : 0;
    const uint64_t at = ((uint64_t)i * a.n_kout + j) * 2;
    kc[r][0] = *(const ulonglong2*)(a.kout + at);
    kc[r][1] = *(const ulonglong2*)(a.kout32 + at);
  }

  uint64_t raw[16];
  v4i frag[NC], fnext[NC];
  const v4i* wp = (const v4i*)pack + (uint64_t)(rb * WM + wm) * chunks * 64 + lane;
  // a step's words and matrix; past the last step those of the last again
  auto load = [&](int t, v4i (&f)[NC]) {
    t = min(t, steps - 1);
#pragma unroll
    for (int c = 0; c < NC; ++c) f[c] = wp[(t * NC + c) * 64];
    const uint64_t* p = x + (uint64_t)group_start(t * (KS / 16) + grp, a.n_in) * ct + col;
#pragma unroll
    for (int k = 0; k < 16; ++k, p += ct) raw[k] = *p;
  };
  // the constants of step t's inputs, by way of one thread each
  auto kin_load = [&](int t) {
    const int g = min(t, steps - 1) * (KS / 16) + tid / 16;
    return SCALED && tid < KS ? kin_i[group_start(g, a.n_in) + tid % 16] : ulonglong2{};
  };
  auto convert = [&](int t, int buf) {
    uint32_t part[ND][4];
    if (SCALED) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const ulonglong2 w = kin[t & 1][grp * 16 + k];
        raw[k] = ND == 8 ? reduce_2q(mul_shoup(raw[k], w.x, w.y, pc.q), pc.q)
                         : reduce_4q(mul_shoup_lazy_split(raw[k], w.x, w.y, pc.q), pc.q);
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t o[ND];
      digits4<ND>(raw + 4 * g, o);
#pragma unroll
      for (int d = 0; d < ND; ++d) part[d][g] = o[d];
    }
#pragma unroll
    for (int d = 0; d < ND; ++d) lds.dig[buf][d][grp][col] = make_uint4(part[d][0], part[d][1], part[d][2], part[d][3]);
  };

  v16i acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[d][r] = 0;
  load(0, frag);
  if (SCALED) {
    const ulonglong2 k0 = kin_load(0), k1 = kin_load(1);
    if (tid < KS) {
      kin[0][tid] = k0;
      kin[1][tid] = k1;
    }
    __syncthreads();
  }
  convert(0, 0);
  __syncthreads();
  for (int t = 0; t < steps; ++t) {
    const int buf = t & 1;
    load(t + 1, fnext);
    const ulonglong2 kn = kin_load(t + 2);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const v4i f = *(const v4i*)&lds.dig[buf][d][c * 2 + (lane >> 5)][wn * 32 + (lane & 31)];
        acc[d] = __builtin_amdgcn_mfma_i32_32x32x32_i8(frag[c], f, acc[d], 0, 0, 0);
      }
    }
    convert(t + 1, buf ^ 1);
    if (SCALED) {
      // step t + 2's constants take the place of step t's, which every thread
      // read before the last barrier
      if (tid < KS) kin[buf][tid] = kn;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c) frag[c] = fnext[c];
  }

  // sum_d acc_d 2^(8d) = lo + 2^32 hi, either below 2^55 in magnitude; a multiple
  // of q from 2^55 on makes them positive
  const int64_t offset = (int64_t)(((1ull << 55) / pc.q + 1) * pc.q);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    int64_t lo = offset, hi = offset;
#pragma unroll
    for (int d = 0; d < 4; ++d) lo += (int64_t)acc[d][r] * (1 << (8 * d));
#pragma unroll
    for (int d = 4; d < ND; ++d) hi += (int64_t)acc[d][r] * (1 << (8 * (d - 4)));
    lds.sums[r][tid] = make_ulonglong2((uint64_t)lo, (uint64_t)hi);
  }
  const int word = col0 + wn * 32 + (lane & 31);
  const uint64_t tok = a.tok ? a.tok[((uint64_t)((a.b0 + b) % a.n_tok) * a.nl + i << a.log_n) + word] : 0;
  const uint64_t* bias = a.bias && comp == 0 ? a.bias + (uint64_t)i * a.n_out * 2 : nullptr;
  const int low = a.nl - a.drop;
  const uint64_t at = i < low ? ((uint64_t)(comp * low + i) << a.log_n) : ((uint64_t)(comp * a.drop + i - low) << a.log_n);
  const uint64_t per = (uint64_t)(i < low ? 2 * low : 2 * a.drop) << a.log_n;
  const int row0 = wm * 32 + (lane >> 5) * 4;
  uint64_t* o = (i < low ? a.out : a.top) + at + word + ((uint64_t)b * a.nj + rb * ROWS) * per;
  // through LDS (a thread's own words): the registers' indexes are constants
  // above, and this loop's code stays small
#pragma unroll 4
  for (int r = 0; r < 16; ++r) {
    const int row = row0 + (r >> 2) * 8 + (r & 3), j = rb * ROWS + row;
    const ulonglong2 v2 = lds.sums[r][tid];
    uint64_t v = join<ND>(v2.x, kc[row][0], v2.y, kc[row][1], pc.q);
    if (a.tok) v = mul_mod(v, tok, pc.q, pc.r64, pc.r64p, pc.inv1);
    if (j < a.nj) {
      if (bias) v = add_mod(v, bias[2 * (a.j0 + j)], pc.q);
      o[row * per] = v;
    }
  }
}

}  // namespace

namespace {

// The matrix cores' tiles take outputs from kTileRows on and inputs from a
// group's 16 on.
constexpr int kTileRows = 9;
bool tiled(int n_in, int nj) { return nj >= kTileRows && n_in >= 16; }

struct Tiles {
  int wm, wn, row_blocks, chunks;
  Tiles(int n_in, int nj) {
    wm = nj > 64 ? 4 : nj > 32 ? 2 : 1;
    if (getenv("XWM")) wm = atoi(getenv("XWM"));
    wn = 4 / wm;
    row_blocks = (nj + 32 * wm - 1) / (32 * wm);
    const int nc = 4 / wn;
    chunks = ((n_in + 31) / 32 + nc - 1) / nc * nc;
  }
  uint64_t words() const { return (uint64_t)row_blocks * wm * chunks * 128; }
};

template <int ND, bool SCALED>
auto pick_rows(int wm) {
  return wm == 4   ? matmul_tiles_kernel<ND, 4, 1, SCALED>
         : wm == 2 ? matmul_tiles_kernel<ND, 2, 2, SCALED>
                   : matmul_tiles_kernel<ND, 1, 4, SCALED>;
}
template <int ND>
auto pick_tiles(int wm, bool scaled) {
  return scaled ? pick_rows<ND, true>(wm) : pick_rows<ND, false>(wm);
}

}  // namespace

uint64_t matmul_pack_words(int n_in, int nj) {
  return std::max(Tiles(n_in, nj).words(), (uint64_t)((nj + kRows - 1) / kRows) * n_in);
}

int launch_matmul(Ctx* c, hipStream_t s, const MatArgs& a, uint64_t* pack) {
  uint64_t q = 0;
  for (int i = 0; i < a.nl; ++i) q = std::max(q, c->mod[i]);
  if (tiled(a.n_in, a.nj)) {
    const Tiles t(a.n_in, a.nj);
    const uint64_t cols = (uint64_t)a.nb * 2 * a.nl * (c->N / (32 * t.wn));
    const uint64_t blocks = (cols + 7) / 8 * 8 * t.row_blocks;
    if (blocks > 0x7fffffff) return set_error(CKKS_EINTERNAL, "too many tiles");
    const uint64_t lanes = (uint64_t)t.row_blocks * t.wm * t.chunks * 64;
    hipLaunchKernelGGL(pack_tiles_kernel, dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, s, a, t.chunks,
                       t.row_blocks * t.wm, (uint4*)pack);
    CKKS_HIP_CHECK(hipGetLastError());
    // nd signed bytes hold words up to 127 sum_d 2^(8d)
    auto fits = [q](int nd) { return q <= 0x7f7f7f7f7f7f7f7full >> (8 * (8 - nd)); };
    auto fn = fits(4)   ? pick_tiles<4>(t.wm, a.kin)
              : fits(5) ? pick_tiles<5>(t.wm, a.kin)
              : fits(6) ? pick_tiles<6>(t.wm, a.kin)
              : fits(7) ? pick_tiles<7>(t.wm, a.kin)
                        : pick_tiles<8>(t.wm, a.kin);
    TraceScope ts(c, s, "matmul_i8", (double)a.nb * a.nj * a.n_in * 2 * a.nl * c->N);
    hipLaunchKernelGGL(fn, dim3((uint32_t)blocks), dim3(256), 0, s, a, (const uint4*)pack, t.chunks, t.row_blocks,
                       (int)cols);
    CKKS_HIP_CHECK(hipGetLastError());
    return CKKS_OK;
  }
  const int tiles = (a.nj + kRows - 1) / kRows;
  const uint64_t words = (uint64_t)tiles * a.n_in;
  hipLaunchKernelGGL(pack_rows_kernel, dim3((uint32_t)((words + 255) / 256)), dim3(256), 0, s, a, pack);
  CKKS_HIP_CHECK(hipGetLastError());
  TraceScope ts(c, s, "matmul_i8", (double)a.nb * a.nj * a.n_in * 2 * a.nl * c->N);
  hipLaunchKernelGGL(matmul_rows_kernel, dim3(c->N / 256, 2 * a.nl, a.nb * tiles), dim3(256), 0, s, a, pack);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

}  // namespace ckks
