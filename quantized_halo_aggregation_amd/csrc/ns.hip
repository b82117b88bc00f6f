// Orthogonalised updates: Newton-Schulz products of many matrices, and the optimiser's step around them.
//
// Mathematics, for a matrix of m x n values with m <= n (a tall one is taken as its transpose):
//   X = U / (|U| + eps),  then `steps` times  A = X X^T,  B = b A + c A^2,  X = a X + B X
// which moves every singular value s of X to a s + b s^3 + c s^5 and keeps the singular vectors.  U is the input, or the step's
// momentum: M = mu M + g, U = g + mu M (Nesterov) or M.  The step ends with p = decay p - step X.
//
// Singular values of X stay below a few units (the host checks the polynomials), so its entries and those of A and B do, too:
// a power of two puts them where half precision has all its bits, and a float32 value is two f16 parts, hi + lo, to 2^-23
// of itself.  A product is rebuilt from hi hi, hi lo and lo hi (the dropped lo lo is below 2^-22 of a term, 2^-25 on the root mean
// square), summed in float32 by the matrix cores: half of what three bf16 parts would cost (six products), at
// float32's error, which the smallest singular values amplify by up to a^steps either way.
// X, A and B are stored as pairs: 8 hi values, then their 8 lo values, so that a step of 32 is one 128-byte line of a row.
//
// A and B are symmetric: tiles on and below the diagonal are formed, and the others stored as their mirror.  The three
// products take the tables of many matrices at once, three launches a step.  Matrices of at most 128 x 128 (the weights of
// node layers) stay in one block's LDS from the gradient to the updated weight: one launch in all.
#include "../../include/qha.h"
#include "qha_internal.hpp"
#include "tile_common.hpp"

namespace qha {
namespace {

// What X, A and B are multiplied by: their entries stay below 16, 16 and 64.
constexpr float kScaleX = 4096.0f, kScaleA = 4096.0f, kScaleB = 1024.0f;

__device__ __forceinline__ f32x4 load4(const void* p, int64_t at, int32_t type) {
  if (type == QHA_F32) return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
  if (type == QHA_BF16) return __builtin_convertvector(*reinterpret_cast<const bf16x4*>(static_cast<const __bf16*>(p) + at), f32x4);
  return __builtin_convertvector(*reinterpret_cast<const f16x4*>(static_cast<const _Float16*>(p) + at), f32x4);
}
__device__ __forceinline__ float load1(const void* p, int64_t at, int32_t type) {
  if (type == QHA_F32) return static_cast<const float*>(p)[at];
  if (type == QHA_BF16) return static_cast<float>(static_cast<const __bf16*>(p)[at]);
  return static_cast<float>(static_cast<const _Float16*>(p)[at]);
}
__device__ __forceinline__ void store4(void* p, int64_t at, int32_t type, f32x4 v) {
  if (type == QHA_F32) *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = v;
  else if (type == QHA_BF16) *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p) + at) = __builtin_convertvector(v, bf16x4);
  else *reinterpret_cast<f16x4*>(static_cast<_Float16*>(p) + at) = __builtin_convertvector(v, f16x4);
}
__device__ __forceinline__ void store1(void* p, int64_t at, int32_t type, float v) {
  if (type == QHA_F32) static_cast<float*>(p)[at] = v;
  else if (type == QHA_BF16) static_cast<__bf16*>(p)[at] = static_cast<__bf16>(v);
  else static_cast<_Float16*>(p)[at] = static_cast<_Float16>(v);
}

// Four neighbours of a matrix's row from column c on, zero past its end; `vec`: rows are aligned to four values.
__device__ __forceinline__ f32x4 read4(const void* p, int64_t ld, int64_t row, int c, int cols, int32_t type, bool vec) {
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (vec && c < cols) return load4(p, row * ld + c, type);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < cols) v[e] = load1(p, row * ld + c + e, type);
  return v;
}
__device__ __forceinline__ void write4(void* p, int64_t ld, int64_t row, int c, int cols, int32_t type, bool vec, f32x4 v) {
  if (vec && c < cols) {
    store4(p, row * ld + c, type, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < cols) store1(p, row * ld + c + e, type, v[e]);
}

// U at four places, from the source and, for the optimiser, the momentum as it is after this step.
__device__ __forceinline__ f32x4 update_of(const NsTable& t, f32x4 g, f32x4 m) {
  if (!t.muon) return g;
  return t.nesterov ? g * t.grad_scale + m * t.mu : m;
}

// The optimiser's new weights and their copy, from four values of X.
__device__ __forceinline__ void apply4(const NsTable& t, const NsMat& a, int64_t row, int c, f32x4 o) {
  if (!t.muon) {
    write4(a.dst, a.ldo, row, c, a.cols, t.out_type, a.vec_out, o);
    return;
  }
  f32x4 p = read4(a.dst, a.ldo, row, c, a.cols, QHA_F32, a.vec_out);
  p = p * t.decay - o * a.step;
  write4(a.dst, a.ldo, row, c, a.cols, QHA_F32, a.vec_out, p);
  if (a.copy) write4(a.copy, a.ldo, row, c, a.cols, t.out_type, a.vec_copy, p);
}

// The matrix that a block works on, by the first blocks of each.
__device__ __forceinline__ int matrix_of(const NsTable& t, const uint32_t* first, uint32_t block) {
  int i = 0;
  while (i + 1 < t.n && first[i + 1] <= block) ++i;
  return i;
}

// Pairs of parts: value (r, c) of a matrix whose rows hold `cols` values.
__device__ __forceinline__ int64_t pair_at(int64_t r, int64_t c, int64_t cols) {
  return r * 2 * cols + (c >> 3) * 16 + (c & 7);
}
__device__ __forceinline__ void split2(f32x4 x, f16x4& hi, f16x4& lo) {
  hi = __builtin_convertvector(x, f16x4);
  lo = __builtin_convertvector(x - __builtin_convertvector(hi, f32x4), f16x4);
}
__device__ __forceinline__ void put_pair(uint16_t* p, int64_t at, f32x4 v) {
  f16x4 hi, lo;
  split2(v, hi, lo);
  *reinterpret_cast<f16x4*>(p + at) = hi;
  *reinterpret_cast<f16x4*>(p + at + 8) = lo;
}
__device__ __forceinline__ f32x4 get_pair(const uint16_t* p, int64_t at) {
  return __builtin_convertvector(*reinterpret_cast<const f16x4*>(p + at), f32x4) +
         __builtin_convertvector(*reinterpret_cast<const f16x4*>(p + at + 8), f32x4);
}

__device__ __forceinline__ double block_sum(double s, double* buf) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
  for (unsigned k = 0; k < blockDim.x / 64; ++k) s += buf[k];
  return s;
}

// What X's entries are U's times: kScaleX / (|U| + eps), 0 for a zero matrix.
__device__ __forceinline__ double scale_of(double squares, double eps) {
  const double size = sqrt(squares) + eps;
  return size == 0.0 ? 0.0 : static_cast<double>(kScaleX) / size;
}

// ---------------------------------------------------------------------------------------------
// from the inputs to X, and from X to the results
// ---------------------------------------------------------------------------------------------

constexpr int kPieceRows = 64, kPieceCols = 256;

// Sum of squares of U by pieces of 64 x 256 values, in float64; the optimiser's momentum is updated here.
__global__ __launch_bounds__(256) void ns_measure_kernel(NsTable t) {
  __shared__ double buf[4];
  const int i = matrix_of(t, t.first_piece, blockIdx.x);
  const NsMat& a = t.m[i];
  const int piece = static_cast<int>(blockIdx.x - t.first_piece[i]);
  const int col_pieces = (a.cols + kPieceCols - 1) / kPieceCols;
  const int c = piece % col_pieces * kPieceCols + (static_cast<int>(threadIdx.x) & 63) * 4;
  const int r0 = piece / col_pieces * kPieceRows, r1 = r0 + kPieceRows < a.rows ? r0 + kPieceRows : a.rows;
  double s = 0.0;
#pragma unroll 4
  for (int r = r0 + static_cast<int>(threadIdx.x >> 6); r < r1; r += 4) {
    const f32x4 g = read4(a.src, a.lds, r, c, a.cols, t.type, a.vec_src);
    f32x4 m = {0.0f, 0.0f, 0.0f, 0.0f};
    if (t.muon) {
      m = read4(a.mom, a.ldo, r, c, a.cols, QHA_F32, a.vec_mom) * t.mu + g * t.grad_scale;
      write4(a.mom, a.ldo, r, c, a.cols, QHA_F32, a.vec_mom, m);
    }
    const f32x4 u = update_of(t, g, m);
#pragma unroll
    for (int e = 0; e < 4; ++e) s += static_cast<double>(u[e]) * static_cast<double>(u[e]);
  }
  s = block_sum(s, buf);
  if (threadIdx.x == 0) a.parts[piece] = s;
}

// X as pairs, by tiles of 64 x 64 of it, zero past the matrix's end.
__global__ __launch_bounds__(256) void ns_split_kernel(NsTable t) {
  __shared__ double buf[4];
  __shared__ float tile[64][68];
  const int i = matrix_of(t, t.first_tile, blockIdx.x);
  const NsMat& a = t.m[i];
  const int at = static_cast<int>(blockIdx.x - t.first_tile[i]), wide = a.n_pad / 64;
  const int x0 = at / wide * 64, y0 = at % wide * 64;            // of X
  const int r0 = a.tall ? y0 : x0, c0 = a.tall ? x0 : y0;        // of the matrix
  const int pieces = ((a.rows + kPieceRows - 1) / kPieceRows) * ((a.cols + kPieceCols - 1) / kPieceCols);
  double s = 0.0;
  for (int k = threadIdx.x; k < pieces; k += 256) s += a.parts[k];
  const double by = scale_of(block_sum(s, buf), t.eps);
  const int cl = (static_cast<int>(threadIdx.x) & 15) * 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int rl = static_cast<int>(threadIdx.x >> 4) + 16 * k;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r0 + rl < a.rows) {
      const f32x4 g = read4(a.src, a.lds, r0 + rl, c0 + cl, a.cols, t.type, a.vec_src);
      const f32x4 m = t.muon ? read4(a.mom, a.ldo, r0 + rl, c0 + cl, a.cols, QHA_F32, a.vec_mom) : g;
      const f32x4 u = update_of(t, g, m);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = c0 + cl + e < a.cols ? static_cast<float>(static_cast<double>(u[e]) * by) : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (a.tall) tile[cl + e][rl] = v[e];
      else tile[rl][cl + e] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int rl = static_cast<int>(threadIdx.x >> 4) + 16 * k;
    put_pair(a.x[0], pair_at(x0 + rl, y0 + cl, a.n_pad), *reinterpret_cast<const f32x4*>(&tile[rl][cl]));
  }
}

// The results from the last X, by the same tiles.
__global__ __launch_bounds__(256) void ns_finish_kernel(NsTable t, int32_t which) {
  __shared__ float tile[64][68];
  const int i = matrix_of(t, t.first_tile, blockIdx.x);
  const NsMat& a = t.m[i];
  const int at = static_cast<int>(blockIdx.x - t.first_tile[i]), wide = a.n_pad / 64;
  const int x0 = at / wide * 64, y0 = at % wide * 64;
  const int r0 = a.tall ? y0 : x0, c0 = a.tall ? x0 : y0;
  const int cl = (static_cast<int>(threadIdx.x) & 15) * 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int rl = static_cast<int>(threadIdx.x >> 4) + 16 * k;
    const f32x4 v = get_pair(a.x[which], pair_at(x0 + rl, y0 + cl, a.n_pad)) * (1.0f / kScaleX);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (a.tall) tile[cl + e][rl] = v[e];
      else tile[rl][cl + e] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int rl = static_cast<int>(threadIdx.x >> 4) + 16 * k;
    if (r0 + rl < a.rows) apply4(t, a, r0 + rl, c0 + cl, *reinterpret_cast<const f32x4*>(&tile[rl][cl]));
  }
}

// ---------------------------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------------------------

enum { NS_GRAM = 0, NS_SQUARE = 1, NS_APPLY = 2 };
constexpr int BK = 32;               // steps of the reduction in LDS at once

// Places of 16-byte chunks in a tile's LDS image.  LDS serves 256 bytes at a time, so reads that go together must fall on
// different sixteenths of 256 bytes.  Along the reduction (rows of 128 bytes), 16 lanes read one chunk of as many rows.
// Across it (rows of 256 bytes or a multiple), a transposing read takes every second chunk of four (hi or lo) of four rows.
__device__ __forceinline__ int place_along(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }
__device__ __forceinline__ int place_cross(int k, int chunk) { return chunk ^ (k & 1) ^ ((k & 2) << 2); }

// A thread's share of an operand's tile: EXTENT rows x 32 steps (along) or 32 steps x EXTENT columns (across), as pairs.
template <bool CROSS, int EXTENT, int NT>
struct PairStager {
  static constexpr int PER = CROSS ? EXTENT / 4 : 2 * BK / 8;     // chunks of a row in LDS
  static constexpr int N = EXTENT * 8 / NT;
  static_assert(EXTENT * 8 % NT == 0, "whole chunks per thread");
  const uint16_t* at[N];
  int64_t next_by;
  // rows x cols values are stored (multiples of 64); the tile begins at row or column `first`.  Those past the
  // end repeat the last ones; their results are not stored.
  __device__ __forceinline__ PairStager(const uint16_t* base, int64_t rows, int64_t cols, int64_t first) {
    next_by = CROSS ? BK * 2 * cols : BK * 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int q = i * NT + static_cast<int>(threadIdx.x), r = q / PER, place = q % PER;
      if constexpr (CROSS) {
        const int64_t chunk = first / 4 + place_cross(r, place), last = cols / 4 - 1;
        at[i] = base + r * 2 * cols + (chunk < last ? chunk : last) * 8;
      } else {
        const int64_t row = first + r < rows ? first + r : rows - 1;
        at[i] = base + row * 2 * cols + place_along(r, place) * 8;
      }
    }
  }
  __device__ __forceinline__ void load(const uint16_t* lds) {
    const uint32_t to = lds_address(lds) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      load_to_lds(at[i], to + i * NT * 16);
      at[i] += next_by;
    }
  }
};

// A matrix operand: one part (0 hi, 1 lo) of 32 rows or columns from `from` on, 16 steps from ks on; lane l holds row
// l % 32, steps 8 (l / 32) .. + 7.
template <bool CROSS, int EXTENT>
__device__ __forceinline__ s16x8 pair_fragment(const uint16_t* lds, int from, int ks, int part, int lane) {
  if constexpr (CROSS) {
    // the transposing read takes 4 steps x 16 columns per 16 lanes: lane j of them addresses step j / 4, columns
    // 4 (j % 4), and receives four steps of column j
    const int j = lane & 15;
    const int col = from + ((lane >> 4) & 1) * 16 + 4 * (j & 3);
    const int k = ks + (lane >> 5) * 8 + (j >> 2);              // k and k + 4 share their places
    const uint16_t* lo = lds + k * 2 * EXTENT + place_cross(k, (col >> 3) * 2 + part) * 8 + (col & 7);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)lo);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(lo + 8 * EXTENT));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const int row = from + (lane & 31);
    const int c = place_along(row, ((ks >> 3) + (lane >> 5)) * 2 + part);
    return *reinterpret_cast<const s16x8*>(lds + row * 2 * BK + c * 8);
  }
}

// C = P Q^T (gram, square) or P Q (apply), with C's other terms: one tile of one matrix.  A wavefront owns MI x NI
// blocks of 32 x 32.  The matrix instruction's operands are swapped (C^T is formed), which leaves a lane four neighbouring
// columns of a row.
template <int KIND, int MI, int NI, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void ns_product_kernel(NsTable t, NsCoef k, int32_t from, uint32_t total) {
  constexpr int BM = MI * 32 * WM, BN = NI * 32 * WN, NT = WM * WN * 64;
  constexpr bool SYM = KIND != NS_APPLY, CROSS = KIND == NS_APPLY;
  static_assert(!SYM || BM == BN, "square tiles of symmetric results");
  constexpr int A_SIZE = BM * BK * 2, BUF = A_SIZE + BN * BK * 2;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * BUF];
  // consecutive blocks go to the eight dies in turn: each takes a run of neighbouring tiles, which share operands
  const uint32_t band = (total + kXcds - 1) / kXcds;
  const uint32_t block = blockIdx.x % kXcds * band + blockIdx.x / kXcds;
  if (block >= total) return;
  const int i = matrix_of(t, t.first_tile, block);
  const NsMat& a = t.m[i];
  const int tile = static_cast<int>(block - t.first_tile[i]);
  int mt, nt;
  if constexpr (SYM) {                         // row mt of the lower triangle begins at mt (mt + 1) / 2
    mt = static_cast<int>((sqrtf(8.0f * static_cast<float>(tile) + 1.0f) - 1.0f) * 0.5f);
    while (mt * (mt + 1) / 2 > tile) --mt;
    while ((mt + 1) * (mt + 2) / 2 <= tile) ++mt;
    nt = tile - mt * (mt + 1) / 2;
  } else {                                     // down groups of eight row tiles before the next column tile
    const int m_tiles = (a.m_pad + BM - 1) / BM, n_tiles = (a.n_pad + BN - 1) / BN;
    const int g = tile / (8 * n_tiles), in = tile % (8 * n_tiles);
    const int rows = m_tiles - 8 * g < 8 ? m_tiles - 8 * g : 8;
    mt = 8 * g + in % rows;
    nt = in / rows;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint16_t* x = a.x[from];
  const uint16_t* P = KIND == NS_GRAM ? x : KIND == NS_SQUARE ? a.a : a.b;
  const uint16_t* Q = KIND == NS_SQUARE ? a.a : x;
  const int64_t depth = KIND == NS_GRAM ? a.n_pad : a.m_pad;

  f32x16 acc[MI][NI];
#pragma unroll
  for (int ii = 0; ii < MI; ++ii)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[ii][j] = 0.0f;
  PairStager<false, BM, NT> sp(P, a.m_pad, depth, static_cast<int64_t>(mt) * BM);
  PairStager<CROSS, BN, NT> sq(Q, a.m_pad, KIND == NS_SQUARE ? a.m_pad : a.n_pad, static_cast<int64_t>(nt) * BN);
  const int steps = static_cast<int>(depth / BK);
  sp.load(lds);
  sq.load(lds + A_SIZE);
  for (int s = 0; s < steps; ++s) {
    const uint16_t* at = lds + (s & 1) * BUF;
    loads_done();
    __syncthreads();                 // step s is there, and everyone has read step s - 1
    if (s + 1 < steps) {
      uint16_t* to = lds + ((s + 1) & 1) * BUF;
      sp.load(to);
      sq.load(to + A_SIZE);
    }
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      s16x8 fp[MI][2], fq[NI][2];
#pragma unroll
      for (int ii = 0; ii < MI; ++ii)
#pragma unroll
        for (int part = 0; part < 2; ++part) fp[ii][part] = pair_fragment<false, BM>(at, (wm * MI + ii) * 32, ks, part, lane);
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int part = 0; part < 2; ++part) fq[j][part] = pair_fragment<CROSS, BN>(at + A_SIZE, (wn * NI + j) * 32, ks, part, lane);
#pragma unroll
      for (int term = 0; term < 3; ++term)            // lo hi, hi lo, hi hi
#pragma unroll
        for (int ii = 0; ii < MI; ++ii)
#pragma unroll
          for (int j = 0; j < NI; ++j)
            acc[ii][j] = mma<_Float16>(fq[j][term == 0], fp[ii][term == 1], acc[ii][j]);
    }
  }

  // Element r of lane l: row l % 32, column 8 (r / 4) + 4 (l / 32) + r % 4 of its block.
  uint16_t* out = KIND == NS_GRAM ? a.a : KIND == NS_SQUARE ? a.b : a.x[from ^ 1];
  const int64_t cols = SYM ? a.m_pad : a.n_pad;
#pragma unroll
  for (int ii = 0; ii < MI; ++ii) {
    const int64_t row = static_cast<int64_t>(mt) * BM + (wm * MI + ii) * 32 + (lane & 31);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t col0 = static_cast<int64_t>(nt) * BN + (wn * NI + j) * 32;
      if (row - (lane & 31) >= a.m_pad || col0 >= cols) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = col0 + 8 * q + 4 * (lane >> 5);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[ii][j][4 * q + e] * k.product;
        if constexpr (KIND == NS_SQUARE) v += get_pair(a.a, pair_at(row, col, cols)) * k.own;
        if constexpr (KIND == NS_APPLY) v += get_pair(x, pair_at(row, col, cols)) * k.own;
        f16x4 hi, lo;
        split2(v, hi, lo);
        uint16_t* o = out + pair_at(row, col, cols);
        *reinterpret_cast<f16x4*>(o) = hi;
        *reinterpret_cast<f16x4*>(o + 8) = lo;
        if (SYM && mt != nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            _Float16* w = reinterpret_cast<_Float16*>(out + pair_at(col + e, row, cols));
            w[0] = hi[e];
            w[8] = lo[e];
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// small matrices
// ---------------------------------------------------------------------------------------------

constexpr int kSmall = 128, kSmallThreads = 512;

// Places of 16-byte chunks in rows of 512 bytes: rows r .. r + 15 fall on different sixteenths, and so do every second
// chunk of four (hi or lo) of the rows 4 i .. 4 i + 3.
__device__ __forceinline__ int place_small(int row, int chunk) {
  return chunk ^ ((row & 1) | ((row & 2) << 2) | ((row & 12) >> 1));
}
__device__ __forceinline__ uint16_t* small_at(uint16_t* lds, int row, int col, int part) {
  return lds + row * 2 * kSmall + place_small(row, (col >> 3) * 2 + part) * 8 + (col & 7);
}
__device__ __forceinline__ s16x8 small_along(const uint16_t* lds, int from, int ks, int part, int lane) {
  const int row = from + (lane & 31);
  return *reinterpret_cast<const s16x8*>(lds + row * 2 * kSmall + place_small(row, ((ks >> 3) + (lane >> 5)) * 2 + part) * 8);
}
__device__ __forceinline__ s16x8 small_cross(const uint16_t* lds, int from, int ks, int part, int lane) {
  const int j = lane & 15;
  const int col = from + ((lane >> 4) & 1) * 16 + 4 * (j & 3), chunk = (col >> 3) * 2 + part;
  const int k = ks + (lane >> 5) * 8 + (j >> 2);
  const uint16_t* p = lds + k * 2 * kSmall + place_small(k, chunk) * 8 + (col & 7);
  const uint16_t* q = lds + (k + 4) * 2 * kSmall + place_small(k + 4, chunk) * 8 + (col & 7);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)q);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One matrix of at most 128 x 128 a block: X and, in turn, A and B as pairs in LDS.  Blocks of 32 x 32 of a result are dealt to
// the eight wavefronts, two to each.
__global__ __launch_bounds__(kSmallThreads) void ns_small_kernel(NsTable t, NsSteps k) {
  __shared__ __attribute__((aligned(16))) uint16_t lds_x[kSmall * kSmall * 2];
  __shared__ __attribute__((aligned(16))) uint16_t lds_a[kSmall * kSmall * 2];
  __shared__ double buf[kSmallThreads / 64];
  const NsMat& a = t.m[blockIdx.x];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mb = (a.m_pad + 31) / 32, nb = (a.n_pad + 31) / 32;      // blocks of 32 (m_pad, n_pad: the sizes themselves here)
  // U in registers, 4 neighbours of a row a turn: 32 lanes a row of up to 128 columns
  constexpr int TURNS = kSmall / (kSmallThreads / 32);
  f32x4 u[TURNS];
  const int c = (static_cast<int>(threadIdx.x) & 31) * 4;
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int r = static_cast<int>(threadIdx.x >> 5) + i * (kSmallThreads / 32);
    u[i] = 0.0f;
    if (r < a.rows && c < a.cols) {
      const f32x4 g = read4(a.src, a.lds, r, c, a.cols, t.type, a.vec_src);
      f32x4 m = {0.0f, 0.0f, 0.0f, 0.0f};
      if (t.muon) {
        m = read4(a.mom, a.ldo, r, c, a.cols, QHA_F32, a.vec_mom) * t.mu + g * t.grad_scale;
        write4(a.mom, a.ldo, r, c, a.cols, QHA_F32, a.vec_mom, m);
      }
      u[i] = update_of(t, g, m);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c + e >= a.cols) u[i][e] = 0.0f;
        s += static_cast<double>(u[i][e]) * static_cast<double>(u[i][e]);
      }
    }
  }
  const double by = scale_of(block_sum(s, buf), t.eps);
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int r = static_cast<int>(threadIdx.x >> 5) + i * (kSmallThreads / 32);
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = r < a.rows && c + e < a.cols ? static_cast<float>(static_cast<double>(u[i][e]) * by) : 0.0f;
    f16x4 hi, lo;
    split2(v, hi, lo);
    if (a.tall) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<_Float16*>(small_at(lds_x, c + e, r, 0)) = hi[e];
        *reinterpret_cast<_Float16*>(small_at(lds_x, c + e, r, 1)) = lo[e];
      }
    } else {
      *reinterpret_cast<f16x4*>(small_at(lds_x, r, c, 0)) = hi;
      *reinterpret_cast<f16x4*>(small_at(lds_x, r, c, 1)) = lo;
    }
  }
  __syncthreads();

  // one product: results in registers, a barrier, results to LDS (where an operand may have been), a barrier
  auto product = [&](uint16_t* p, uint16_t* q, bool cross, int depth, int cols_b, uint16_t* own, uint16_t* out, NsCoef f) {
    f32x16 acc[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      acc[w] = 0.0f;
      const int b = wave + 8 * w, bi = b / cols_b, bj = b % cols_b;
      if (b >= mb * cols_b) continue;
      for (int ks = 0; ks < depth; ks += 16) {
        s16x8 fp[2], fq[2];
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          fp[part] = small_along(p, bi * 32, ks, part, lane);
          fq[part] = cross ? small_cross(q, bj * 32, ks, part, lane) : small_along(q, bj * 32, ks, part, lane);
        }
        acc[w] = mma<_Float16>(fq[1], fp[0], acc[w]);
        acc[w] = mma<_Float16>(fq[0], fp[1], acc[w]);
        acc[w] = mma<_Float16>(fq[0], fp[0], acc[w]);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[w][e] *= f.product;
      if (own) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int row = bi * 32 + (lane & 31), col = bj * 32 + 8 * g + 4 * (lane >> 5);
          const f32x4 v = __builtin_convertvector(*reinterpret_cast<const f16x4*>(small_at(own, row, col, 0)), f32x4) +
                          __builtin_convertvector(*reinterpret_cast<const f16x4*>(small_at(own, row, col, 1)), f32x4);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[w][4 * g + e] += v[e] * f.own;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int b = wave + 8 * w, bi = b / cols_b, bj = b % cols_b;
      if (b >= mb * cols_b) continue;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int row = bi * 32 + (lane & 31), col = bj * 32 + 8 * g + 4 * (lane >> 5);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[w][4 * g + e];
        f16x4 hi, lo;
        split2(v, hi, lo);
        *reinterpret_cast<f16x4*>(small_at(out, row, col, 0)) = hi;
        *reinterpret_cast<f16x4*>(small_at(out, row, col, 1)) = lo;
      }
    }
    __syncthreads();
  };
  for (int step = 0; step < k.steps; ++step) {
    product(lds_x, lds_x, false, 32 * nb, mb, nullptr, lds_a, k.gram);
    product(lds_a, lds_a, false, 32 * mb, mb, lds_a, lds_a, k.square[step]);
    product(lds_a, lds_x, true, 32 * mb, nb, lds_x, lds_x, k.apply[step]);
  }

#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int r = static_cast<int>(threadIdx.x >> 5) + i * (kSmallThreads / 32);
    if (r >= a.rows || c >= a.cols) continue;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int xr = a.tall ? c + e : r, xc = a.tall ? r : c + e;
      v[e] = (static_cast<float>(*reinterpret_cast<const _Float16*>(small_at(lds_x, xr, xc, 0))) +
              static_cast<float>(*reinterpret_cast<const _Float16*>(small_at(lds_x, xr, xc, 1)))) * (1.0f / kScaleX);
    }
    apply4(t, a, r, c, v);
  }
}

// ---------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------

constexpr int64_t kBatchValues = 1LL << 24;      // values of X in flight in a batch of several matrices

int64_t pad64(int64_t x) { return (x + 63) / 64 * 64; }
bool is_small(const NsMatrix& m) { return m.rows <= kSmall && m.cols <= kSmall; }
int64_t piece_count(const NsMatrix& m) {
  return (m.rows + kPieceRows - 1) / kPieceRows * ((m.cols + kPieceCols - 1) / kPieceCols);
}
// X twice, A and B as pairs, and the pieces' sums of squares
size_t bytes_of(const NsMatrix& m) {
  const int64_t s = pad64(m.rows < m.cols ? m.rows : m.cols), l = pad64(m.rows < m.cols ? m.cols : m.rows);
  return static_cast<size_t>(2 * s * l + 2 * s * s) * 4 + static_cast<size_t>((piece_count(m) + 1) / 2 * 16);
}

// The next batch of large (or small) matrices from *at on: their indices, at most kNsBatch.
int next_batch(const NsMatrix* m, int64_t n, bool small, int64_t* at, int64_t* index) {
  int count = 0;
  int64_t values = 0;
  for (; *at < n && count < kNsBatch; ++*at) {
    const NsMatrix& x = m[*at];
    if (x.rows == 0 || x.cols == 0 || is_small(x) != small) continue;
    if (!small && count > 0 && values + x.rows * x.cols > kBatchValues) break;
    values += x.rows * x.cols;
    index[count++] = *at;
  }
  return count;
}

template <int KIND, int MI, int NI, int WM, int WN>
void run_product(NsTable& t, const NsCoef& k, int from, hipStream_t s) {
  constexpr int BM = MI * 32 * WM, BN = NI * 32 * WN;
  uint32_t total = 0;
  for (int i = 0; i < t.n; ++i) {
    t.first_tile[i] = total;
    const uint32_t mt = (t.m[i].m_pad + BM - 1) / BM, nt = (t.m[i].n_pad + BN - 1) / BN;
    total += KIND == NS_APPLY ? mt * nt : mt * (mt + 1) / 2;
  }
  const uint32_t grid = (total + static_cast<uint32_t>(kXcds) - 1) / static_cast<uint32_t>(kXcds) * static_cast<uint32_t>(kXcds);
  ns_product_kernel<KIND, MI, NI, WM, WN><<<grid, WM * WN * 64, 0, s>>>(t, k, from, total);
}

template <int KIND>
int64_t tiles_of(const NsTable& t, int64_t side) {
  int64_t total = 0;
  for (int i = 0; i < t.n; ++i) {
    const int64_t mt = (t.m[i].m_pad + side - 1) / side, nt = (t.m[i].n_pad + side - 1) / side;
    total += KIND == NS_APPLY ? mt * nt : mt * (mt + 1) / 2;
  }
  return total;
}

template <int KIND>
void run_product(NsTable& t, const NsCoef& k, int from, hipStream_t s) {
  if (tiles_of<KIND>(t, 128) >= 256) run_product<KIND, 2, 2, 2, 2>(t, k, from, s);
  else run_product<KIND, 1, 1, 2, 2>(t, k, from, s);
}

}  // namespace

size_t ns_workspace(const NsMatrix* m, int64_t n) {
  size_t most = 0;
  int64_t index[kNsBatch];
  for (int64_t at = 0; at < n;) {
    const int count = next_batch(m, n, false, &at, index);
    size_t need = 0;
    for (int i = 0; i < count; ++i) need += bytes_of(m[index[i]]);
    most = need > most ? need : most;
  }
  return most;
}

hipError_t launch_ns(const NsMatrix* m, int64_t n, const NsArgs& args, void* ws, hipStream_t s) {
  NsTable t = {};
  t.type = args.type;
  t.out_type = args.out_type;
  t.muon = args.muon;
  t.nesterov = args.nesterov;
  t.mu = args.mu;
  t.grad_scale = args.grad_scale;
  t.decay = args.decay;
  t.eps = args.eps;
  NsSteps k = {};
  k.steps = args.steps;
  k.gram = {kScaleA / (kScaleX * kScaleX), 0.0f};
  for (int i = 0; i < args.steps; ++i) {
    const double a = args.coefficients[3 * i], b = args.coefficients[3 * i + 1], c = args.coefficients[3 * i + 2];
    k.square[i] = {static_cast<float>(c * (kScaleB / (kScaleA * kScaleA))), static_cast<float>(b * (kScaleB / kScaleA))};
    k.apply[i] = {1.0f / kScaleB, static_cast<float>(a)};
  }
  int64_t index[kNsBatch];
  bool launched = false;
  const auto fill = [&](int count, bool small) {
    char* at = static_cast<char*>(ws);
    t.n = count;
    launched = true;
    for (int i = 0; i < count; ++i) {
      const NsMatrix& x = m[index[i]];
      NsMat& a = t.m[i];
      a.rows = static_cast<int32_t>(x.rows);
      a.cols = static_cast<int32_t>(x.cols);
      a.tall = x.rows > x.cols;
      const int64_t sh = a.tall ? x.cols : x.rows, lo = a.tall ? x.rows : x.cols;
      a.m_pad = static_cast<int32_t>(small ? sh : pad64(sh));
      a.n_pad = static_cast<int32_t>(small ? lo : pad64(lo));
      a.src = x.src;
      a.lds = x.lds;
      a.dst = x.dst;
      a.ldo = x.ldo;
      a.mom = x.mom;
      a.copy = x.copy;
      a.step = x.step;
      const auto whole = [&](const void* p, int64_t ld, int32_t type) {
        return x.cols % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (type == QHA_F32 ? 15 : 7)) == 0;
      };
      a.vec_src = whole(x.src, x.lds, args.type);
      a.vec_out = whole(x.dst, x.ldo, args.muon ? QHA_F32 : args.out_type);
      a.vec_mom = whole(x.mom, x.ldo, QHA_F32);
      a.vec_copy = whole(x.copy, x.ldo, args.out_type);
      if (small) continue;
      const int64_t mn = static_cast<int64_t>(a.m_pad) * a.n_pad, mm = static_cast<int64_t>(a.m_pad) * a.m_pad;
      a.x[0] = reinterpret_cast<uint16_t*>(at);
      a.x[1] = a.x[0] + 2 * mn;
      a.a = a.x[1] + 2 * mn;
      a.b = a.a + 2 * mm;
      a.parts = reinterpret_cast<double*>(a.b + 2 * mm);
      at += bytes_of(x);
    }
  };
  for (int64_t at = 0; at < n;) {
    const int count = next_batch(m, n, true, &at, index);
    if (count == 0) break;
    fill(count, true);
    ns_small_kernel<<<count, kSmallThreads, 0, s>>>(t, k);
  }
  for (int64_t at = 0; at < n;) {
    const int count = next_batch(m, n, false, &at, index);
    if (count == 0) break;
    fill(count, false);
    uint32_t pieces = 0, tiles = 0;
    for (int i = 0; i < count; ++i) {
      t.first_piece[i] = pieces;
      pieces += static_cast<uint32_t>(piece_count(m[index[i]]));
    }
    const auto tables = [&] {          // the products write first_tile for tiles of their own
      tiles = 0;
      for (int i = 0; i < count; ++i) {
        t.first_tile[i] = tiles;
        tiles += static_cast<uint32_t>(t.m[i].m_pad / 64) * static_cast<uint32_t>(t.m[i].n_pad / 64);
      }
    };
    ns_measure_kernel<<<pieces, 256, 0, s>>>(t);
    tables();
    ns_split_kernel<<<tiles, 256, 0, s>>>(t);
    int from = 0;
    for (int i = 0; i < args.steps; ++i) {
      run_product<NS_GRAM>(t, k.gram, from, s);
      run_product<NS_SQUARE>(t, k.square[i], from, s);
      run_product<NS_APPLY>(t, k.apply[i], from, s);
      from ^= 1;
    }
    tables();
    ns_finish_kernel<<<tiles, 256, 0, s>>>(t, from);
  }
  return launched ? hipGetLastError() : hipSuccess;
}

}  // namespace qha
