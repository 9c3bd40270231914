// Kernels of the product with a matrix of 8-bit integers (linear.h).
#include "linear.h"

#include <algorithm>

#include "arith.h"
#include "convert.h"
#include "matmul_tiles.h"

namespace ckks {

namespace {

constexpr int kRows = 8;  // outputs of a thread at most

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

// One word of R outputs a thread: the word's 31-bit halves times a byte, summed
// in 64 bits (2^31 2^7 2^16 = 2^54).  For few outputs, where the words are all the
// traffic: 768 inputs of 4 limbs at N = 2^16 (3.2 GB) in 630 us, 5.1 TB/s, with 16
// loads in flight; 650 us with eight outputs a thread and a load at a time.
template <int R>
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
  int64_t lo[R] = {}, hi[R] = {};
  auto take = [&](uint64_t v, int k) {
    if (kin) v = reduce_2q(mul_shoup(v, kin[2 * k], kin[2 * k + 1], q), q);
    const int32_t l = (int32_t)(v & 0x7fffffff), h = (int32_t)(v >> 31);
    const uint64_t row = w[k];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int32_t m = (int8_t)(row >> (8 * r));
      lo[r] += (int64_t)l * m;
      hi[r] += (int64_t)h * m;
    }
  };
  constexpr int kAhead = 16;  // loads in flight
  int k = 0;
  for (; k + kAhead <= a.n_in; k += kAhead, x += kAhead * ct) {
    uint64_t v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = x[u * ct];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) take(v[u], k + u);
  }
  for (; k < a.n_in; ++k, x += ct) take(*x, k);
  ep.has_tok = a.tok != nullptr;
  ep.tok = a.tok ? a.tok[(((uint64_t)((a.b0 + b) % a.n_tok) * a.nl + i) << a.log_n) + c] : 0;
  ep.kout = a.kout ? a.kout + (uint64_t)i * a.n_kout * 2 : nullptr;
  ep.kstep = a.n_kout > 1 ? 2 : 0;
  ep.bias = a.bias && comp == 0 ? a.bias + (uint64_t)i * a.n_out * 2 : nullptr;
  const int low = a.nl - a.drop;
  const uint64_t at = i < low ? ((uint64_t)(comp * low + i) << a.log_n) : ((uint64_t)(comp * a.drop + i - low) << a.log_n);
  uint64_t* o = (i < low ? a.out : a.top) + at + c;
  const uint64_t per = (uint64_t)(i < low ? 2 * low : 2 * a.drop) << a.log_n;
#pragma unroll
  for (int r = 0; r < R; ++r) {
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
// A workgroup of 4 waves takes 32 MT WM outputs x 32 WN words of one limb; a wave
// 32 MT outputs x 32 words, all digits: 16 ND MT accumulators a lane.  The words
// of a step of 128 / WN inputs (16 a thread, of one column) are loaded ahead,
// split into digits and laid in LDS in the order the instructions take them (16
// inputs of a word and digit together), which every wave of the word reads; the
// matrix comes from L2 in that order already.
//   MT 2: one wave a SIMD, 256 outputs.  A digit read from LDS serves two
//     instructions (with one it would take LDS's whole rate), and loads, reads,
//     conversions and writes of the steps around stand between a step's matrix
//     instructions: 56 of 32 cycles in 3.0 thousand cycles a step.
//   MT 1: two workgroups a CU, whose phases overlap, for 128, 64 or 32 outputs.
// 768 -> 768 at 3 limbs of 2^16 (300 M words in and out, 7 digits) takes 2.7-3.0
// ms: 1.1-1.2 P byte operations/s, where a large library product of bytes reaches 2.0 on this card;
// 3.1 ms with MT 1.  A tile's 39 thousand cycles are 20 of steps, 12 of joining
// the sums (some 60 vector instructions an output) and 6 before the first words
// are there; tile after tile in one workgroup, the next words loaded early, gained
// nothing (2.9 ms).  With 8 digits (60-bit primes) it takes 2.9 ms where 7 take 2.8;
// with scales on the inputs the 8-digit kernels of 128 and 256 outputs spill 16
// registers (768 -> 128: 910 us against 755; 2048 -> 512 at 4 limbs of 2^15: 3.48 ms
// against 3.24).

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

// a - m if that is not negative, else a, by the borrow.
__device__ __forceinline__ uint64_t below(uint64_t a, uint64_t m) {
  uint64_t t;
  return __builtin_sub_overflow(a, m, &t) ? a : t;
}

// A sum S = lo + 2^32 hi of words below q times bytes, |S| < 2^23 q, modulo q: with
// 2^24 q added (lo0, hi0; 2^56 go from hi to lo, which then is positive) it is U
// 2^32 + its low dword, below 2^25 q.  h, its bits from b - 7 on (b those of q), is
// below 2^32, and h 2^(b-7) / q = h m / 2^32 is less than 1 + 2^-6 below S / q, m =
// floor(2^(b+25) / q) and h being cut off: the whole part leaves a remainder
// below 3q.
struct SumMod {
  int64_t lo0, hi0;
  uint64_t nq;
  uint32_t m;
  int sh;
  bool big;  // b - 7 >= 32: h comes out of U
  __device__ __forceinline__ explicit SumMod(uint64_t q, uint32_t quot) : nq(0 - q), m(quot) {
    lo0 = (int64_t)((q & 0xff) << 24) + (1ll << 56);
    hi0 = (int64_t)(q >> 8) - (1ll << 24);
    const int b = 64 - __builtin_clzll(q);
    big = b >= 39;
    sh = big ? b - 39 : b - 7;
  }
  __device__ __forceinline__ uint64_t rem(int64_t lo, int64_t hi) const {
    const uint64_t u = (uint64_t)hi + ((uint64_t)lo >> 32);
    const uint32_t u1 = (uint32_t)(u >> 32), u0 = (uint32_t)u, l0 = (uint32_t)lo;
    const uint32_t h = big ? __builtin_amdgcn_alignbit(u1, u0, sh) : __builtin_amdgcn_alignbit(u0, l0, sh);
    const uint32_t e = __umulhi(h, m);
    const uint64_t r = mad64(e, (uint32_t)nq, (uint64_t)u0 << 32 | l0);
    return r + ((uint64_t)(e * (uint32_t)(nq >> 32)) << 32);
  }
};

// A scalar base and a lane's byte offset below 2^32, as one address of a load or
// store: the base goes through an empty asm statement, or the compiler moves the
// sum into vector registers, an addition a load.
typedef __attribute__((address_space(1))) char* GlobalBytes;
__device__ __forceinline__ GlobalBytes scalar_base(const void* p) {
  uint64_t u = (uint64_t)p;
  asm("" : "+s"(u));
  return (GlobalBytes)u;
}
template <typename T>
__device__ __forceinline__ T load_at(const void* base, uint32_t bytes) {
  return *(const __attribute__((address_space(1))) T*)(scalar_base(base) + bytes);
}

template <int ND, int WM, int WN, int MT, bool SCALED>
__global__ __launch_bounds__(256, MT == 2 ? 1 : 2) void matmul_tiles_kernel(MatArgs a, const uint4* pack, int chunks, int row_blocks,
                                                              int col_blocks) {
  static_assert(WM * WN == 4, "four waves");
  static_assert(sizeof(uint4) * 2 * ND * 256 >= sizeof(uint64_t) * 16 * 256, "the epilogue's words fit the digits' place");
  constexpr int KS = 128 / WN, NC = KS / 32, W = 32 * WN, ROWS = 32 * WM * MT;  // inputs and chunks of a step, a tile
  constexpr int AHEAD = MT;  // steps that words load ahead: as many as the registers hold
  __shared__ uint4 dig[2][ND][KS / 16][W];
  __shared__ ulonglong2 kc[ROWS];  // {k, Shoup} of the tile's outputs
  __shared__ ulonglong2 kin[2][SCALED ? KS : 1];
  // Workgroups go round the 8 XCDs: each takes a range of the words, the tiles
  // of the same words next to each other, so that its L2 reads them once.
  const int slot = blockIdx.x >> 3, per_xcd = (col_blocks + 7) / 8;
  const int rb = slot % row_blocks, cb = (blockIdx.x & 7) * per_xcd + slot / row_blocks;
  if (slot / row_blocks >= per_xcd || cb >= col_blocks) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
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
    kc[r] = *(const ulonglong2*)(a.kout + at);
  }

  uint64_t raw[2][16];
  v4i frag[2][NC][MT];
  const v4i* wp = (const v4i*)pack + (uint64_t)(rb * WM + wm) * MT * chunks * 64;
  const uint32_t lane16 = lane * 16;
  // a step's matrix and words; past the last step those of the last again
  auto load_matrix = [&](int t, int c, v4i (&f)[NC][MT]) {
    t = min(t, steps - 1);
#pragma unroll
    for (int m = 0; m < MT; ++m) f[c][m] = load_at<v4i>(wp + (m * chunks + t * NC + c) * 64, lane16);
  };
  // Addresses are a scalar and a lane's 32 bits: a wave of a 32-word tile holds
  // two groups, the second at most 16 inputs (below 2^27 words) behind the first.
  const int group0 = __builtin_amdgcn_readfirstlane(tid / W);
  struct Words {
    const uint64_t* p;  // the next input's row
    uint32_t off;
  };
  auto words = [&](int t) {
    t = min(t, steps - 1);
    const int at = group_start(t * (KS / 16) + group0, a.n_in), next = group_start(t * (KS / 16) + group0 + 1, a.n_in);
    return Words{x + (uint64_t)at * ct, ((uint32_t)col + (W == 32 && lane >= 32 ? (uint32_t)(next - at) * (uint32_t)ct : 0)) * 8};
  };
  auto load = [&](Words& w, int k0, int k1, uint64_t (&v)[16]) {
#pragma unroll
    for (int k = k0; k < k1; ++k, w.p += ct) v[k] = load_at<uint64_t>(w.p, w.off);
  };
  // the constants of step t's inputs, by way of one thread each
  auto kin_load = [&](int t) {
    const int g = min(t, steps - 1) * (KS / 16) + tid / 16;
    return SCALED && tid < KS ? kin_i[group_start(g, a.n_in) + tid % 16] : ulonglong2{};
  };
  // the constants of words 4g..4g+3, read a quarter ahead
  ulonglong2 scale[4];
  auto scales = [&](int t, int g) {
#pragma unroll
    for (int k = 0; k < 4; ++k) scale[k] = kin[t & 1][grp * 16 + 4 * g + k];
  };
  // words 4g..4g+3 into their digits; then all 16 into buffer t & 1
  uint32_t part[ND][4];
  auto quarter = [&](int t, uint64_t (&v)[16], int g) {
    if (SCALED) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint64_t& u = v[4 * g + k];
        u = below(below(mul_shoup_lazy_split(u, scale[k].x, scale[k].y, pc.q), 2 * pc.q), pc.q);
      }
      if (g < 3) scales(t, g + 1);
    }
    uint32_t o[ND];
    digits4<ND>(v + 4 * g, o);
#pragma unroll
    for (int d = 0; d < ND; ++d) part[d][g] = o[d];
  };
  // quarters done before chunk c: a scaled one fills its chunk
  auto quarters = [](int c) { return c == 0 ? 0 : NC < 4 ? 4 : SCALED ? c : c == 1 ? 2 : min(c + 1, 4); };
  auto put = [&](int t) {
#pragma unroll
    for (int d = 0; d < ND; ++d) dig[t & 1][d][grp][col] = make_uint4(part[d][0], part[d][1], part[d][2], part[d][3]);
  };

  v16i acc[MT][ND];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][d][r] = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) load_matrix(0, c, frag[0]);
  Words w0 = words(0), w1 = words(1);
  load(w0, 0, 16, raw[0]);
  if (AHEAD == 2) load(w1, 0, 16, raw[1]);
  if (SCALED) {
    const ulonglong2 k0 = kin_load(0), k1 = kin_load(1);
    if (tid < KS) {
      kin[0][tid] = k0;
      kin[1][tid] = k1;
    }
    __syncthreads();
  }
  if (SCALED) scales(0, 0);
#pragma unroll
  for (int g = 0; g < 4; ++g) quarter(0, raw[0], g);
  put(0);
  __syncthreads();
  // step t reads buffer t & 1 (here a constant), and lays step t + 1's digits,
  // whose words are in `next`, in the other
  auto step = [&](int t, int buf, uint64_t (&next)[16], uint64_t (&after)[16]) {
    // a chunk's digits are read while the one before is multiplied
    v4i f[2][ND];
    auto digits = [&](int c) {
#pragma unroll
      for (int d = 0; d < ND; ++d) f[c & 1][d] = *(const v4i*)&dig[buf][d][c * 2 + (lane >> 5)][wn * 32 + (lane & 31)];
    };
    const ulonglong2 kn = kin_load(t + 2);
    Words w = words(t + AHEAD);
    if (AHEAD == 1) {
      // one wave's loads and conversions run beside the other's matrix
      // instructions.  The matrix first: loads return in order
#pragma unroll
      for (int c = 0; c < NC; ++c) load_matrix(t + 1, c, frag[buf ^ 1]);
      load(w, 0, 16, next);
    }
    digits(0);
    if (SCALED) scales(buf ^ 1, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (c + 1 < NC) digits(c + 1);
      if (AHEAD == 2) {
        // one wave a SIMD: loads (of the words two steps on), the conversion of
        // the next step's words and the reads above go between the matrix
        // instructions
        load_matrix(t + 1, c, frag[buf ^ 1]);
        load(w, c * 16 / NC, (c + 1) * 16 / NC, after);
        // (in fewer chunks than there are, to lay the digits out in the last)
#pragma unroll
        for (int g = quarters(c); g < quarters(c + 1); ++g) quarter(buf ^ 1, next, g);
        if (c + 1 == NC) put(buf ^ 1);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][d] = __builtin_amdgcn_mfma_i32_32x32x32_i8(frag[buf][c][m], f[c & 1][d], acc[m][d], 0, 0, 0);
      if (AHEAD == 2) {
#pragma unroll
        for (int d = 0; d < ND * MT; ++d) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction,
          if ((c + 1 < NC && d < ND) || (SCALED && d >= ND * MT - 5)) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read,
          if (d < MT + 16 / NC) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);      // a load,
          if (c + 1 == NC && d < ND) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // a write,
          __builtin_amdgcn_sched_group_barrier(0x002, SCALED ? 13 : 7, 0);               // conversions
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (AHEAD == 1) {
#pragma unroll
      for (int g = 0; g < 4; ++g) quarter(buf ^ 1, next, g);
      put(buf ^ 1);
    }
    // step t + 2's constants take the place of step t's, which every thread
    // read before the last barrier
    if (SCALED && tid < KS) kin[buf][tid] = kn;
    __syncthreads();
  };
  int t = 0;  // no branch in the loop's body: the last steps load and lay out words again
  for (; t + 1 < steps; t += 2) {
    step(t, 0, raw[1], raw[0]);
    step(t + 1, 1, raw[0], raw[1]);
  }
  if (t < steps) step(t, 0, raw[1], raw[0]);

  // 2^(8d) out of the compiler's sight: one multiply-add a digit, not a sign
  // extension, a shift and an addition
  int place[4] = {1, 1 << 8, 1 << 16, 1 << 24};
#pragma unroll
  for (int d = 0; d < 4; ++d) asm("" : "+s"(place[d]));
  const SumMod mod(pc.q, (uint32_t)((ConstPrime)a.prime)[i].top);
  const int word = col0 + wn * 32 + (lane & 31);
  const uint64_t tok = a.tok ? a.tok[(((uint64_t)((a.b0 + b) % a.n_tok) * a.nl + i) << a.log_n) + word] : 0;
  const uint64_t* bias = a.bias && comp == 0 ? a.bias + (uint64_t)i * a.n_out * 2 : nullptr;
  const int low = a.nl - a.drop;
  const uint64_t at = i < low ? ((uint64_t)(comp * low + i) << a.log_n) : ((uint64_t)(comp * a.drop + i - low) << a.log_n);
  const uint64_t per = (uint64_t)(i < low ? 2 * low : 2 * a.drop) << a.log_n;
  const int row0 = wm * MT * 32 + (lane >> 5) * 4;
  uint64_t* o = (i < low ? a.out : a.top) + at + ((uint64_t)b * a.nj + rb * ROWS + wm * MT * 32) * per;
  const uint32_t o_off = ((uint32_t)word + (lane >> 5) * 4 * (uint32_t)per) * 8;  // below 2^29
  // words that the rescale finishes are left below 4q (primes below 2^61)
  const bool lazy = ND < 8 && a.drop && i < low;
  // The rows of a group of four registers lie next to each other; a group's
  // chains do not wait for one another.
  auto sums = [&](int m, int r, uint64_t (&v)[4]) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      int64_t lo = mod.lo0, hi = mod.hi0;
#pragma unroll
      for (int d = 0; d < 4; ++d) lo += (int64_t)acc[m][d][r + n] * place[d];
#pragma unroll
      for (int d = 4; d < ND; ++d) hi += (int64_t)acc[m][d][r + n] * place[d - 4];
      const ulonglong2 k = kc[row0 + m * 32 + r * 2 + n];
      v[n] = mul_shoup_lazy_split(mod.rem(lo, hi), k.x, k.y, pc.q);  // below 4q
    }
    if (lazy) return;
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n] = below(below(v[n], 2 * pc.q), pc.q);
  };
  auto store = [&](int up, uint64_t (&v)[4]) {
    const int j = rb * ROWS + row0 + up;
    if (bias) {
#pragma unroll
      for (int n = 0; n < 4; ++n) v[n] = below(v[n] + bias[2 * (a.j0 + min(j + n, a.nj - 1))], pc.q);
    }
    if (j + 3 < a.nj) {
#pragma unroll
      for (int n = 0; n < 4; ++n) *(__attribute__((address_space(1))) uint64_t*)(scalar_base(o + (up + n) * per) + o_off) = v[n];
    } else {
#pragma unroll
      for (int n = 0; n < 3; ++n)
        if (j + n < a.nj) *(__attribute__((address_space(1))) uint64_t*)(scalar_base(o + (up + n) * per) + o_off) = v[n];
    }
  };
  uint64_t(*done)[256] = (uint64_t(*)[256])dig;  // a thread's own words
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      uint64_t v[4];
      sums(m, r, v);
      if (a.tok) {  // wait in LDS for the loop below, which is not unrolled
#pragma unroll
        for (int n = 0; n < 4; ++n) done[r + n][tid] = v[n];
      } else {
        store(m * 32 + r * 2, v);
      }
    }
    if (!a.tok) continue;
#pragma unroll 1
    for (int r = 0; r < 16; r += 4) {
      uint64_t v[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) v[n] = mul_mod(done[r + n][tid], tok, pc.q, pc.r64, pc.r64p, pc.inv1);
      store(m * 32 + r * 2, v);
    }
  }
}

}  // namespace

namespace {

template <int ND, bool SCALED>
auto pick_rows(const Tiles& t) {
  return t.mt == 2   ? matmul_tiles_kernel<ND, 4, 1, 2, SCALED>
         : t.wm == 4 ? matmul_tiles_kernel<ND, 4, 1, 1, SCALED>
         : t.wm == 2 ? matmul_tiles_kernel<ND, 2, 2, 1, SCALED>
                     : matmul_tiles_kernel<ND, 1, 4, 1, SCALED>;
}
template <int ND>
auto pick_tiles(const Tiles& t, bool scaled) {
  return scaled ? pick_rows<ND, true>(t) : pick_rows<ND, false>(t);
}

}  // namespace

uint64_t matmul_pack_words(int n_in, int nj) {
  // any of the tiles, for this many outputs or fewer: two words a lane
  const uint64_t rows = (uint64_t)(nj + 255) / 256 * 256, inputs = (uint64_t)(n_in + 127) / 128 * 128;
  return std::max(rows * inputs / 8, (uint64_t)((nj + kRows - 1) / kRows) * n_in);
}

int launch_matmul(Ctx* c, hipStream_t s, const MatArgs& a, uint64_t* pack) {
  uint64_t q = 0;
  for (int i = 0; i < a.nl; ++i) q = std::max(q, c->mod[i]);
  if (tiled(a.n_in, a.nj)) {
    const Tiles t(a.n_in, a.nj);
    const uint64_t cols = (uint64_t)a.nb * 2 * a.nl * (c->N / (32 * t.wn));
    const uint64_t blocks = (cols + 7) / 8 * 8 * t.row_blocks;
    if (blocks > 0x7fffffff) return set_error(CKKS_EINTERNAL, "too many tiles");
    const uint64_t lanes = t.lanes();
    hipLaunchKernelGGL(pack_tiles_kernel, dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, s, a, t.chunks,
                       t.row_blocks * t.wm * t.mt, (uint4*)pack);
    CKKS_HIP_CHECK(hipGetLastError());
    const int nd = word_digits(q);
    auto fn = nd == 4   ? pick_tiles<4>(t, a.kin)
              : nd == 5 ? pick_tiles<5>(t, a.kin)
              : nd == 6 ? pick_tiles<6>(t, a.kin)
              : nd == 7 ? pick_tiles<7>(t, a.kin)
                        : pick_tiles<8>(t, a.kin);
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
  auto fn = a.nj <= 2 ? matmul_rows_kernel<2> : a.nj <= 4 ? matmul_rows_kernel<4> : matmul_rows_kernel<kRows>;
  hipLaunchKernelGGL(fn, dim3(c->N / 256, 2 * a.nl, a.nb * tiles), dim3(256), 0, s, a, pack);
  CKKS_HIP_CHECK(hipGetLastError());
  return CKKS_OK;
}

}  // namespace ckks
