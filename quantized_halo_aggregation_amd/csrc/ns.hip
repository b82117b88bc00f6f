// Orthogonalised updates: Newton-Schulz products of many matrices, and the optimiser's step around them.
//
// Mathematics, for a matrix of m x n values with m <= n (a tall one is taken as its transpose):
//   X = U / (|U| + eps),  then `steps` times  A = X X^T,  B = a I + b A + c A^2,  X = B X
// which moves every singular value s of X to a s + b s^3 + c s^5 and keeps the singular vectors.  U is the input, or the step's
// momentum: M = mu M + g, U = g + mu M (Nesterov) or M.  The step ends with p = decay p - step X.
//
// The host follows the largest singular value through the polynomials, which bounds X's entries and those of A and B: a power of two
// a step takes each bound to the end of half precision's range, and a float32 value is two f16 parts, hi + lo, to 2^-23 of
// itself above 2^-17 of the bound, below that to 2^-40 of the bound.  A product is rebuilt from hi hi, hi lo and lo hi (the dropped
// lo lo is below 2^-22 of a term, 2^-25 on the root mean square), summed in float32 by the matrix cores: half of what three bf16
// parts would cost (six products).  So a result has float32's precision with respect to its norm, which the smallest singular
// values amplify by up to a^steps either way, but not each row or column that is small by itself.  a X, the largest term of most values, is
// added to a product's result (on chip, where X's blocks stay in registers) or goes through the last product as B's diagonal, where
// it passes few additions: tiles take their own rows' steps last, and blocks straight from memory add that wavefront's sum last.  (Reading
// X for it instead took 3 to 6 % of a step in memory; the steps in their places left 5.0e-6 for the second 2.8e-6 below, 5.5e-6 for the third.)
// Measured, off by this share of the norm after five steps, in brackets the same with a library's float32 products: noise of 256 x 256
// 6e-7 (1.7e-6), of 4096 x 4096 2.5e-6 (4.8e-6); singular values falling to 1e-4, 128 x 128 2.8e-6 (3.6e-6), 1024 x 1024 2.8e-6
// (4.6e-6).  The worst row's share of itself where rows fade to 1e-6: 256 x 256 2.8e-5 (5e-6), 1024 x 1024 1.1e-4 (1.8e-5),
// 4096 x 4096 4.3e-4 (3.6e-5); with one scale for any coefficients 2.2e-4, 8.6e-4 and 3.5e-3.  Second parts with a scale of their own would
// need accumulators of their own, twice as many.
// What bounds it, and the forms that follow from it (five steps, float32, us a call):
//   - Large matrices: the matrix cores.  Tiles through LDS, A and B by their tiles on and below the diagonal (the others are stored
//     as their mirror), three launches a step for a batch of up to 40 matrices, whose tables the launches share.  4096 x 4096 3570 to 3790,
//     on a card where a plain library product in f16 reaches 1.31 PFLOP/s 3788, B X 343 (1.20 of part products), A and B 203 and 212 (1.1).  What is lost
//     is a step's wait and barrier, and the stores of a tile, with which nothing overlaps at one block a compute unit.
//   - Lists too small to fill the chip with tiles: the chain of loads and barriers of a launch.  Blocks of 32 x 32 whose wavefronts
//     share out the reduction, straight from memory, two or three launches a step: 8 of 256 x 256 98 to 100 in 17 launches of 5 to 8.
//   - Matrices that fit in one block's LDS (up to 32 x 896, 64 x 384, 96 x 192 and 128 x 128): one launch from the gradient to the updated
//     weight.  8 of 128 x 128 42, of which 5.5 a step: latency of LDS reads and of five barriers, the matrix cores are mostly idle.
#include "../../include/qha.h"
#include "qha_internal.hpp"
#include "tile_common.hpp"

#include <cmath>

namespace qha {
namespace {

// What the first X is multiplied by, whose values are at most 1 (see half_scale).
constexpr float kScaleX = 32768.0f;

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
// Four of 16 rows apart at once, from matrices whose rows are aligned to four values: all loads go out before the first is converted.
// Places past the end hold others' values.
template <typename E>
__device__ __forceinline__ void read_rows(const void* p, int64_t ld, int r, int rows, int c, int cols, f32x4 (&v)[4]) {
  typedef E vec __attribute__((ext_vector_type(4)));
  vec raw[4];
  const E* at = static_cast<const E*>(p) + (c < cols ? c : 0);
#pragma unroll
  for (int k = 0; k < 4; ++k) raw[k] = *reinterpret_cast<const vec*>(at + (r + 16 * k < rows ? r + 16 * k : rows - 1) * ld);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __builtin_convertvector(raw[k], f32x4);
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
__device__ __forceinline__ int matrix_of(const NsFirst& first, uint32_t block) {
  int i = 0;
#pragma unroll
  for (int k = 1; k < kNsBatch; ++k) i += k < first.n && first.block[k] <= block;
  return i;
}

__device__ __forceinline__ void split2(f32x4 x, f16x4& hi, f16x4& lo) {
  hi = __builtin_convertvector(x, f16x4);
  lo = __builtin_convertvector(x - __builtin_convertvector(hi, f32x4), f16x4);
}

// X, A and B in memory, in the order in which the matrix cores take them: blocks of 32 rows x 16 values along the reduction, 512 hi
// values, then their 512 lo values, those of lane l (row l % 32, values 8 (l / 32) .. + 7) together.  So a wavefront's operand is
// 1 KB without gaps, from memory or from LDS.  The rows of the four eights of 32 columns are turned by 0, 4, 8 and 12 places against
// each other: the transposing read, which takes four rows of all four at a time, then meets different banks.
// The place of value (r, c), hi, in rows of `cols` values:
constexpr int kBlock = 1024, kLo = 512;
__device__ __forceinline__ int64_t block_at(int64_t r, int64_t c, int64_t cols) {
  return ((r >> 5) * (cols >> 4) + (c >> 4)) * kBlock + ((c >> 3) & 1) * 256 + ((r + ((c >> 3) & 3) * 4) & 31) * 8 + (c & 7);
}
// A lane's place in an operand along the reduction: in blocks of even (h = 0) and odd (1) number of a row.
__device__ __forceinline__ int lane_at(int lane, int h) { return (lane >> 5) * 256 + ((lane + (lane >> 5) * 4 + h * 8) & 31) * 8; }
// A matrix's part of the workspace: A, B, X and the next one, (their transposes,) and the pieces' sums of squares.
struct NsParts {
  char* ws;
  int64_t mn, mm;                    // bytes of X and of A
  __device__ __forceinline__ explicit NsParts(const NsMat& a)
      : ws(a.ws), mn(4LL * a.m_pad * a.n_pad), mm(4LL * a.m_pad * a.m_pad) {}
  __device__ __forceinline__ uint16_t* x(int which) const { return reinterpret_cast<uint16_t*>(ws + 2 * mm + which * mn); }
  __device__ __forceinline__ uint16_t* xt(int which) const { return reinterpret_cast<uint16_t*>(ws + 2 * mm + (2 + which) * mn); }
  __device__ __forceinline__ uint16_t* a() const { return reinterpret_cast<uint16_t*>(ws); }
  __device__ __forceinline__ uint16_t* b() const { return reinterpret_cast<uint16_t*>(ws + mm); }
  __device__ __forceinline__ double* squares(bool transposes) const { return reinterpret_cast<double*>(ws + 2 * mm + (transposes ? 4 : 2) * mn); }
};
__device__ __forceinline__ void put4(uint16_t* p, int64_t at, f32x4 v) {
  f16x4 hi, lo;
  split2(v, hi, lo);
  *reinterpret_cast<f16x4*>(p + at) = hi;
  *reinterpret_cast<f16x4*>(p + at + kLo) = lo;
}
__device__ __forceinline__ void put8(uint16_t* p, int64_t at, f32x4 u, f32x4 v) {
  f16x4 hi[2], lo[2];
  split2(u, hi[0], lo[0]);
  split2(v, hi[1], lo[1]);
  *reinterpret_cast<f16x8*>(p + at) = __builtin_shufflevector(hi[0], hi[1], 0, 1, 2, 3, 4, 5, 6, 7);
  *reinterpret_cast<f16x8*>(p + at + kLo) = __builtin_shufflevector(lo[0], lo[1], 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x4 get4(const uint16_t* p, int64_t at) {
  return __builtin_convertvector(*reinterpret_cast<const f16x4*>(p + at), f32x4) +
         __builtin_convertvector(*reinterpret_cast<const f16x4*>(p + at + kLo), f32x4);
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

constexpr int kPieceCols = 256;

// Sum of squares of U by pieces of piece_rows x 256 values, in float64; the optimiser's momentum is updated here.  The first
// block leaves the table, which came with the arguments, in the workspace for the launches behind it.
__global__ __launch_bounds__(256) void ns_measure_kernel(NsTable t, NsFirst first, uint32_t* table) {
  __shared__ double buf[4];
  if (blockIdx.x == 0) {
    const uint32_t* words = reinterpret_cast<const uint32_t*>(&t);
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(NsTable) / 4); i += 256) table[i] = words[i];
  }
  const int i = matrix_of(first, blockIdx.x);
  const NsMat& a = t.m[i];
  const int piece = static_cast<int>(blockIdx.x - first.block[i]);
  const int col_pieces = (a.cols + kPieceCols - 1) / kPieceCols;
  const int c = piece % col_pieces * kPieceCols + (static_cast<int>(threadIdx.x) & 63) * 4;
  const int r0 = piece / col_pieces * t.piece_rows, r1 = r0 + t.piece_rows < a.rows ? r0 + t.piece_rows : a.rows;
  double s = 0.0;
  for (int r = r0 + static_cast<int>(threadIdx.x >> 6); r < r1; r += 8) {      // two rows' loads at once
    f32x4 g[2], m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      g[h] = m[h] = 0.0f;
      if (r + 4 * h >= r1) continue;
      g[h] = read4(a.src, a.lds, r + 4 * h, c, a.cols, t.type, a.vec_src);
      if (t.muon) m[h] = read4(a.mom, a.ldo, r + 4 * h, c, a.cols, QHA_F32, a.vec_mom);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (r + 4 * h >= r1) continue;
      if (t.muon) {
        m[h] = m[h] * t.mu + g[h] * t.grad_scale;
        write4(a.mom, a.ldo, r + 4 * h, c, a.cols, QHA_F32, a.vec_mom, m[h]);
      }
      const f32x4 u = update_of(t, g[h], m[h]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s += static_cast<double>(u[e]) * static_cast<double>(u[e]);
    }
  }
  s = block_sum(s, buf);
  if (threadIdx.x == 0) NsParts(a).squares(t.transposes)[piece] = s;
}

// X, and its transpose where the products read that, by tiles of 64 x 64, zero past the matrix's end.  Bound
// by memory: 24 of 4096 x 1024 with bf16 gradients and momentum 220 us, 1.0 GB at 4.6 TB/s (a row's loads after another's 265)
__global__ __launch_bounds__(256) void ns_split_kernel(const NsTable* table, NsFirst first) {
  const NsTable& t = *table;
  __shared__ double buf[4];
  __shared__ float tile[64][68];
  const int i = matrix_of(first, blockIdx.x);
  const NsMat& a = t.m[i];
  const int at = static_cast<int>(blockIdx.x - first.block[i]), wide = (a.n_pad + 63) / 64;
  const int x0 = at / wide * 64, y0 = at % wide * 64;            // of X
  const int r0 = a.tall ? y0 : x0, c0 = a.tall ? x0 : y0;        // of the matrix
  const int cl = (static_cast<int>(threadIdx.x) & 15) * 4, rl = static_cast<int>(threadIdx.x >> 4);
  f32x4 u[4], m[4];
  if (a.vec_src && (!t.muon || a.vec_mom)) {
    if (t.muon) read_rows<float>(a.mom, a.ldo, r0 + rl, a.rows, c0 + cl, a.cols, m);
    if (t.type == QHA_F32) read_rows<float>(a.src, a.lds, r0 + rl, a.rows, c0 + cl, a.cols, u);
    else if (t.type == QHA_BF16) read_rows<__bf16>(a.src, a.lds, r0 + rl, a.rows, c0 + cl, a.cols, u);
    else read_rows<_Float16>(a.src, a.lds, r0 + rl, a.rows, c0 + cl, a.cols, u);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[k] = m[k] = 0.0f;
      if (r0 + rl + 16 * k >= a.rows) continue;
      u[k] = read4(a.src, a.lds, r0 + rl + 16 * k, c0 + cl, a.cols, t.type, a.vec_src);
      if (t.muon) m[k] = read4(a.mom, a.ldo, r0 + rl + 16 * k, c0 + cl, a.cols, QHA_F32, a.vec_mom);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) u[k] = update_of(t, u[k], m[k]);
  const int pieces = ((a.rows + t.piece_rows - 1) / t.piece_rows) * ((a.cols + kPieceCols - 1) / kPieceCols);
  double s = 0.0;
  const NsParts w(a);
  for (int k = threadIdx.x; k < pieces; k += 256) s += w.squares(t.transposes)[k];
  const double by = scale_of(block_sum(s, buf), t.eps);
  // the tile as the matrix has it; a thread then takes four neighbours of X's rows, or of its transpose's
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = r0 + rl + 16 * k < a.rows && c0 + cl + e < a.cols;
      v[e] = in ? static_cast<float>(static_cast<double>(u[k][e]) * by) : 0.0f;
    }
    *reinterpret_cast<f32x4*>(&tile[rl + 16 * k][cl]) = v;
  }
  __syncthreads();
  uint16_t* xt = t.transposes ? w.xt(0) : nullptr;
  uint16_t* along = a.tall ? xt : w.x(0);                        // stored as the matrix is
  uint16_t* across = a.tall ? w.x(0) : xt;
  const int along_cols = a.tall ? a.m_pad : a.n_pad, across_cols = a.tall ? a.n_pad : a.m_pad;
  const int q = static_cast<int>(threadIdx.x) & 63;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = (static_cast<int>(threadIdx.x >> 6) + 4 * k) * 8;
    if (along && r0 + q < across_cols && c0 + c < along_cols)
      put8(along, block_at(r0 + q, c0 + c, along_cols), *reinterpret_cast<const f32x4*>(&tile[q][c]), *reinterpret_cast<const f32x4*>(&tile[q][c + 4]));
    if (across && c0 + q < along_cols && r0 + c < across_cols) {
      f32x4 v[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = tile[c + e][q];
      put8(across, block_at(c0 + q, r0 + c, across_cols), v[0], v[1]);
    }
  }
}

constexpr int kPartRow = 36;         // floats of a row of 32 in LDS, padded to spread columns over the banks

// The results from a block of 32 x 32 of the last X (times its scale) in LDS, rows x0 .., columns y0 ..: thread `id` of N takes four
// neighbours of the matrix's rows, so that eight threads write whole lines.  (Straight from the accumulators, 16 bytes of 32 rows
// at a time, the last product of 4096 x 4096 took 1638 us, the others 372.)
template <int N>
__device__ __forceinline__ void finish_block(const NsTable& t, const NsMat& a, const float* v, int64_t x0, int64_t y0, int id) {
  constexpr int K = 256 / N;
  const int64_t r0 = a.tall ? y0 : x0, c0 = a.tall ? x0 : y0;
  const auto four = [&](int k) {
    const int r = (id + k * N) >> 3, c = ((id + k * N) & 7) * 4;
    f32x4 o;
    if (a.tall) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = v[(c + e) * kPartRow + r];
    } else {
      o = *reinterpret_cast<const f32x4*>(v + r * kPartRow + c);
    }
    return o * t.result;
  };
  if (t.muon && a.vec_out && (!a.copy || a.vec_copy) && r0 + 32 <= a.rows && c0 + 32 <= a.cols) {
    // whole blocks of aligned weights: every weight on its way before the first is needed (24 of 4096 x 1024 with a copy,
    // one after the other 1108 us, 834)
    float* p = static_cast<float*>(a.dst) + r0 * a.ldo + c0;
    f32x4 w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = *reinterpret_cast<const f32x4*>(p + ((id + k * N) >> 3) * a.ldo + ((id + k * N) & 7) * 4);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t at = ((id + k * N) >> 3) * a.ldo + ((id + k * N) & 7) * 4;
      const f32x4 x = w[k] * t.decay - four(k) * a.step;
      *reinterpret_cast<f32x4*>(p + at) = x;
      if (a.copy) store4(a.copy, r0 * a.ldo + c0 + at, t.out_type, x);
    }
    return;
  }
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    const int r = (id + k * N) >> 3, c = ((id + k * N) & 7) * 4;
    if (r0 + r < a.rows) apply4(t, a, r0 + r, static_cast<int>(c0) + c, four(k));
  }
}

// ---------------------------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------------------------

enum { NS_GRAM = 0, NS_SQUARE = 1, NS_APPLY = 2, NS_LAST = 3 };      // NS_LAST: apply, with results in X's place
constexpr int BK = 32;               // steps of the reduction in LDS at once

// A thread's share of the loads of an operand's tile of a step: EXTENT rows, two blocks of each 32 rows (4 KB without gaps), or, ACROSS
// the reduction, 32 rows and EXTENT columns (without gaps in all).
template <bool ACROSS, int EXTENT, int NT>
struct Stager {
  static constexpr int N = EXTENT * 8 / NT;
  static constexpr int PER = ACROSS ? 128 : 256, RUNS = NT / PER;      // 16-byte pieces of a run, and runs that the threads take at once
  static_assert(EXTENT * 8 % NT == 0 && NT % PER == 0, "whole runs");
  const uint16_t* at[N];
  int64_t next_by;
  // The matrix has `rows` runs of 32 rows of `blocks` blocks; the tile begins at run (across: at block) `first`.  Those past the end
  // repeat the last one, whose results are not stored.
  // `id`: the thread's number of NT; the reduction begins at step `begin`.
  __device__ __forceinline__ Stager(const uint16_t* base, int64_t rows, int64_t blocks, int64_t first, int id, int64_t begin) {
    next_by = ACROSS ? blocks * kBlock : 2 * kBlock;
    base += begin * next_by;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t r = first + i * RUNS + id / PER;
      const int64_t run = ACROSS ? (r < blocks ? r : blocks - 1) : (r < rows ? r : rows - 1) * blocks;
      at[i] = base + run * kBlock + (id & (PER - 1)) * 8;
    }
  }
  __device__ __forceinline__ void move(int steps) {
#pragma unroll
    for (int i = 0; i < N; ++i) at[i] += steps * next_by;
  }
  // `lds`: the wavefront's part of the buffer
  __device__ __forceinline__ void load(const uint16_t* lds) {
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds_address(lds));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      load_to_lds(at[i], to + i * NT * 16);
      at[i] += next_by;
    }
  }
};

// Four neighbours of a row of B = a I + b A + c A^2 from c A^2's and A's.
__device__ __forceinline__ f32x4 square_terms(const NsCoef& k, f32x4 v, f32x4 of_a, int64_t row, int64_t col) {
  v += of_a * k.own;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] += col + e == row ? k.unit : 0.0f;
  return v;
}

// Tile of the lower triangle: row m of it begins at m (m + 1) / 2.
__device__ __forceinline__ void triangle(int tile, int* mt, int* nt) {
  int m = static_cast<int>((sqrtf(8.0f * static_cast<float>(tile) + 1.0f) - 1.0f) * 0.5f);
  while (m * (m + 1) / 2 > tile) --m;
  while ((m + 1) * (m + 2) / 2 <= tile) ++m;
  *mt = m;
  *nt = tile - m * (m + 1) / 2;
}

// A = X X^T (gram), B = a I + b A + c A A^T (square) or the next X = B X (apply): one tile of one matrix.  A wavefront owns MI x NI
// blocks of 32 x 32; X's columns in the last product come through the transposing read.  The matrix instruction's
// operands are swapped (C^T is formed), which leaves a lane four neighbouring columns of a row.  KS groups of WM x WN wavefronts share
// out the reduction, each with buffers of its own, and the first adds the second's sums to its own.  Bound by the matrix cores at 256 x 256 (63% of all cycles busy at 4096 x 4096, at the clock that their
// power leaves), by loads and barriers at 64 x 64 (19% at five of 1000 x 520), where three buffers of 32 steps were the best
// number (five of 1000 x 520 with three of 333 x 777, all steps: 269 us; two 286, four 275, five 277).
template <int KIND, int MI, int NI, int WM, int WN, int STAGES, int KS>
__global__ __launch_bounds__(WM * WN * KS * 64) void ns_product_kernel(const NsTable* table, NsFirst first, NsCoef k, int32_t from, uint32_t total) {
  constexpr int BM = MI * 32 * WM, BN = NI * 32 * WN, NT = WM * WN * 64;
  constexpr bool SYM = KIND == NS_GRAM || KIND == NS_SQUARE;
  static_assert(BM == BN, "square tiles, for symmetric results");
  constexpr int A_SIZE = BM * BK * 2, BUF = A_SIZE + BN * BK * 2;
  constexpr int PARTS = WM * WN * 32 * kPartRow;                     // floats: a block of 32 x 32 of each wavefront
  static_assert(KS == 1 || (KS == 2 && MI == 1 && NI == 1), "halves of the reduction in tiles of one block a wavefront");
  static_assert(PARTS * 4 * KS <= KS * STAGES * BUF * 2, "room for the transposes and for the other half's sums");
  __shared__ __attribute__((aligned(16))) uint16_t pool[KS * STAGES * BUF];
  // consecutive blocks go to the eight dies in turn: each takes a run of neighbouring tiles, which share operands
  const uint32_t band = (total + kXcds - 1) / kXcds;
  const uint32_t block = blockIdx.x % kXcds * band + blockIdx.x / kXcds;
  if (block >= total) return;
  const NsTable& t = *table;
  const int i = matrix_of(first, block);
  const NsMat& a = t.m[i];
  const int tile = static_cast<int>(block - first.block[i]);
  const int64_t m_pad = a.m_pad, n_pad = a.n_pad;
  int mt, nt;
  if constexpr (SYM) {
    triangle(tile, &mt, &nt);
  } else {                                     // down groups of eight row tiles before the next column tile
    const int m_tiles = static_cast<int>((m_pad + BM - 1) / BM), n_tiles = static_cast<int>((n_pad + BN - 1) / BN);
    const int g = tile / (8 * n_tiles), in = tile % (8 * n_tiles);
    const int rows = m_tiles - 8 * g < 8 ? m_tiles - 8 * g : 8;
    mt = 8 * g + in % rows;
    nt = in / rows;
  }
  const int lane = threadIdx.x & 63;
  const int group = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / NT);      // of the reduction's halves
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) - group * (NT / 64);
  const int id = static_cast<int>(threadIdx.x) - group * NT;
  const int wm = wave / WN, wn = wave % WN;
  uint16_t* lds = pool + group * STAGES * BUF;
  const NsParts w(a);
  const uint16_t* x = w.x(from);
  const uint16_t* P = KIND == NS_GRAM ? x : KIND == NS_SQUARE ? w.a() : w.b();
  const uint16_t* Q = KIND == NS_SQUARE ? w.a() : x;
  const int64_t depth = KIND == NS_GRAM ? n_pad : m_pad, cols = SYM ? m_pad : n_pad;

  f32x16 acc[MI][NI];
#pragma unroll
  for (int ii = 0; ii < MI; ++ii)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[ii][j] = 0.0f;
  const int whole = static_cast<int>(depth / BK), steps = (whole + KS - 1) / KS;
  const bool blank = KS == 2 && group == 1 && (whole & 1);           // a second half of one step fewer begins with zeros
  // In B X the steps of the tile's own rows, where B's diagonal brings a X in, come last: two jumps over the reduction's steps.  (A
  // reduction that begins behind them and turns took 2 % more.)  Tiles beside each other are then up to a tile's steps apart in X: at
  // 4096 x 4096 520 MB from memory instead of 403, and 0.7 % more time.
  const int mine = blank ? steps - 1 : steps;                        // of this group
  int first_step = group * steps, left = 0, jump = 0;      // loads left to the next jump, and its steps
  int after = 0, back = 0;             // the same of the jump behind it
  if constexpr (!SYM) {
    const int end = first_step + mine, own_end = (mt + 1) * (BM / BK);
    const int own_begin = mt * (BM / BK) > first_step ? mt * (BM / BK) : first_step;
    if (own_begin < own_end && own_end < end) {
      left = own_begin - first_step;
      jump = own_end - own_begin;
      after = end - own_end;
      back = own_begin - end;
      if (left == 0) {                 // they are the first ones
        first_step = own_end;
        left = after;
        jump = back;
      }
    }
  }
  Stager<false, BM, NT> sp(P, m_pad / 32, depth / 16, static_cast<int64_t>(mt) * (BM / 32), id, first_step);
  Stager<!SYM, BN, NT> sq(Q, m_pad / 32, (SYM ? depth : n_pad) / 16, static_cast<int64_t>(nt) * (SYM ? BN / 32 : BN / 16), id, first_step);
  const auto jump_over = [&] {
    if (SYM || --left != 0) return;
    sp.move(jump);
    sq.move(jump);
    left = jump == back ? 0 : after;
    jump = back;
  };
  constexpr int EACH = decltype(sp)::N + decltype(sq)::N;      // loads of a thread for a step
  // A step's operands come out of LDS in two halves of 16.  The first half of step s + 1 is read while the second half of step s is
  // multiplied: the wait for its loads and the barrier lie in the middle of step s, where they find the matrix cores busy.
  const int along[2] = {lane_at(lane, 0), lane_at(lane, 1)};
  // across: 16 lanes take 4 rows x 16 columns, lane j of them addresses row j / 4, columns 4 (j % 4), and receives four rows of
  // column j; rows 8 (l / 32) .. + 3 and the four behind them, columns 16 (l / 16 % 2) ..
  int across[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int j = lane & 15, r = (lane >> 5) * 8 + (j >> 2) + 4 * g, c = ((lane >> 4) & 1) * 16 + 4 * (j & 3);
    across[g] = static_cast<int>(block_at(r, c, 32));
  }
  const auto fetch = [&](int buffer, int h, s16x8 (&fp)[MI][2], s16x8 (&fq)[NI][2]) {
    const uint16_t* at = lds + buffer * BUF;
#pragma unroll
    for (int ii = 0; ii < MI; ++ii)
#pragma unroll
      for (int part = 0; part < 2; ++part)
        fp[ii][part] = *reinterpret_cast<const s16x8*>(at + along[h] + ((wm * MI + ii) * 2 + h) * kBlock + part * kLo);
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint16_t* from_q = at + A_SIZE + (wn * NI + j) * 2 * kBlock + part * kLo;
        if constexpr (SYM) {
          fq[j][part] = *reinterpret_cast<const s16x8*>(from_q + along[h] + h * kBlock);
        } else {                       // 16 rows on, a row's place changes by its fifth bit
          const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(from_q + (across[0] ^ h * 128)));
          const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(from_q + (across[1] ^ h * 128)));
          fq[j][part] = __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
        }
      }
  };
  const auto multiply_term = [&](const s16x8 (&fp)[MI][2], const s16x8 (&fq)[NI][2], int term) {      // lo hi, hi lo, hi hi
#pragma unroll
    for (int ii = 0; ii < MI; ++ii)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[ii][j] = mma<_Float16>(fq[j][term == 0], fp[ii][term == 1], acc[ii][j]);
  };
  const auto multiply = [&](const s16x8 (&fp)[MI][2], const s16x8 (&fq)[NI][2]) {
#pragma unroll
    for (int term = 0; term < 3; ++term) multiply_term(fp, fq, term);
  };
  uint16_t* to = lds + wave * 512;
  if (blank)
    for (int i = id * 8; i < BUF; i += NT * 8) *reinterpret_cast<s16x8*>(lds + i) = 0;
  for (int s = blank ? 1 : 0; s < STAGES && s < steps; ++s) {
    sp.load(to + s * BUF);
    sq.load(to + s * BUF + A_SIZE);
    jump_over();
  }
  if (steps >= STAGES) loads_left<(STAGES - 1) * EACH>();
  else loads_left<0>();
  __syncthreads();
  s16x8 p0[MI][2], q0[NI][2], p1[MI][2], q1[NI][2];
  fetch(0, 0, p0, q0);
  int now = 0;
  // the last step stands by itself: joined with the others it would make them wait for the reads of the half step behind
  for (int s = 0; s + 1 < steps; ++s) {
    fetch(now, 1, p1, q1);
    multiply(p0, q0);
    const int next = now + 1 == STAGES ? 0 : now + 1;
    // loads return in order: step s + 1 is there when only those of the steps behind it are on their way
    if (s + STAGES - 1 < steps) loads_left<(STAGES - 2) * EACH>();
    else loads_left<0>();
    __syncthreads();                 // for every wavefront, and everyone has read step s
    fetch(next, 0, p0, q0);
    // the loads of a later step go out between the products, which would otherwise wait for their issue
    const bool more = s + STAGES < steps;
    multiply_term(p1, q1, 0);
    if (more) sp.load(to + now * BUF);
    multiply_term(p1, q1, 1);
    if (more) {
      sq.load(to + now * BUF + A_SIZE);
      jump_over();
    }
    multiply_term(p1, q1, 2);
    now = next;
  }
  fetch(now, 1, p1, q1);
  multiply(p0, q0);
  multiply(p1, q1);

  // Element r of lane l: row l % 32, column 8 (r / 4) + 4 (l / 32) + r % 4 of its block.  The mirror of a symmetric result and rows of
  // the call's results pass through a piece of LDS of the wavefront's own.
  const bool turned = SYM ? mt != nt : KIND == NS_LAST;
  uint16_t* out = KIND == NS_GRAM ? w.a() : KIND == NS_SQUARE ? w.b() : w.x(from ^ 1);
  float* turn = reinterpret_cast<float*>(pool) + wave * 32 * kPartRow;
  if (KS == 2 || turned) __syncthreads();        // everyone has read the last step
  if constexpr (KS == 2) {
    f32x4* sums = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(pool) + PARTS) + wave * 256 + lane;
    if (group == 1) {
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[64 * q] = f32x4{acc[0][0][4 * q], acc[0][0][4 * q + 1], acc[0][0][4 * q + 2], acc[0][0][4 * q + 3]};
    }
    __syncthreads();
    if (group == 1) return;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][0][4 * q + e] += sums[64 * q][e];
  }
#pragma unroll
  for (int ii = 0; ii < MI; ++ii) {
    const int64_t row0 = static_cast<int64_t>(mt) * BM + (wm * MI + ii) * 32;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t col0 = static_cast<int64_t>(nt) * BN + (wn * NI + j) * 32;
      if (row0 >= m_pad || col0 >= cols) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = row0 + (lane & 31), col = col0 + 8 * q + 4 * (lane >> 5);
        f32x4 v = {acc[ii][j][4 * q], acc[ii][j][4 * q + 1], acc[ii][j][4 * q + 2], acc[ii][j][4 * q + 3]};
        v *= k.product;
        if constexpr (KIND == NS_SQUARE) v = square_terms(k, v, get4(w.a(), block_at(row, col, cols)), row, col);
        if constexpr (KIND != NS_LAST) put4(out, block_at(row, col, cols), v);
        if (turned) *reinterpret_cast<f32x4*>(turn + (lane & 31) * kPartRow + 8 * q + 4 * (lane >> 5)) = v;
      }
      if (!turned) continue;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if constexpr (KIND == NS_LAST) {
        finish_block<64>(t, a, turn, row0, col0, lane);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 8 * q + 4 * (lane >> 5);
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = turn[(c + e) * kPartRow + (lane & 31)];
          put4(out, block_at(col0 + (lane & 31), row0 + c, cols), v);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// ---------------------------------------------------------------------------------------------
// matrices that fit in LDS
// ---------------------------------------------------------------------------------------------

constexpr int kChipThreads = 512, kChipWaves = kChipThreads / 64;

// MB: rows of X by 32.  X's columns are padded to 64, A's rows to 64 or 128 values.
template <int MB>
struct Chip {
  static constexpr int CAP = MB == 1 ? 896 : MB == 2 ? 384 : MB == 3 ? 192 : 128;      // columns of X
  static constexpr int LDA = MB < 3 ? 64 : 128;
  static constexpr int X_SIZE = MB * 32 * CAP * 2, A_SIZE = MB * 32 * LDA * 2;         // 16-bit values
  static constexpr int PARTS = MB == 4 ? 0 : kChipWaves * 32 * kPartRow;               // floats
  static constexpr int BYTES = (X_SIZE + A_SIZE) * 2 + PARTS * 4;
};
constexpr int kChipBytes = Chip<1>::BYTES;
static_assert(Chip<2>::BYTES <= kChipBytes && Chip<3>::BYTES <= kChipBytes && Chip<4>::BYTES <= kChipBytes && kChipBytes <= 160000, "LDS");

// Places of 16-byte chunks in rows of a multiple of 256 bytes: rows r .. r + 15 fall on different sixteenths of 256 bytes, and so
// do every second chunk of four (hi or lo) of the rows 4 i .. 4 i + 3.  Rows 16 apart share a place, so that stores of 8 bytes by 32
// rows (chip_put) meet in pairs: 21 % of the LDS cycles of 8 of 128 x 128 are counted as conflicts.
__device__ __forceinline__ int place_chip(int row, int chunk) {
  return chunk ^ ((row & 1) | ((row & 2) << 2) | ((row & 12) >> 1));
}
__device__ __forceinline__ uint16_t* chip_at(uint16_t* lds, int ld, int row, int col, int part) {
  return lds + row * 2 * ld + place_chip(row, (col >> 3) * 2 + part) * 8 + (col & 7);
}
// A matrix in LDS as a lane reads operands of 32 rows or columns and 16 steps from it: lane l holds row (column) l % 32, steps
// 8 (l / 32) .. + 7.  The permutation acts on the low four bits of a chunk's number, of which a lane's own part is fixed: an
// address is one exclusive or and one addition away (addresses formed anew took longer than the products: 128 x 128 47 us).
struct ChipMatrix {
  const char* base;
  int row_bytes;
  int along_row, along_low;          // along the rows: byte of the lane's row, its bits of the place times 16
  int cross_row[2], cross_low[2], cross_in;
  __device__ __forceinline__ ChipMatrix(const uint16_t* lds, int ld, int lane) : base(reinterpret_cast<const char*>(lds)), row_bytes(4 * ld) {
    along_row = (lane & 31) * row_bytes;
    along_low = place_chip(lane & 31, (lane >> 5) * 2) * 16;
    const int j = lane & 15;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = (lane >> 5) * 8 + (j >> 2) + 4 * h;
      cross_row[h] = k * row_bytes + 8 * (j & 1);
      cross_low[h] = place_chip(k, ((lane >> 4) & 1) * 4 + ((j & 3) >> 1) * 2) * 16;
    }
  }
  // 32 steps from 32 kb on, as two times 16: rows 32 i .., as they are stored,
  __device__ __forceinline__ void along(int i, int kb, s16x8 (&f)[2][2]) const {
    const char* at = base + along_row + i * 32 * row_bytes + (kb >> 1) * 256;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int part = 0; part < 2; ++part)
        f[h][part] = *reinterpret_cast<const s16x8*>(at + (along_low ^ ((kb & 1) * 128 + h * 64 + part * 16)));
  }
  // columns 32 j .., across the rows,
  __device__ __forceinline__ void cross(int j, int kb, s16x8 (&f)[2][2]) const {
    const char* at = base + kb * 32 * row_bytes + (j >> 1) * 256;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int low = (j & 1) * 128 + part * 16;
        const char* p = at + h * 16 * row_bytes + cross_row[0] + (cross_low[0] ^ low);
        const char* q = at + h * 16 * row_bytes + cross_row[1] + (cross_low[1] ^ low);
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)q);
        f[h][part] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
      }
  }
  // and rows 32 i .. of a symmetric matrix of which the blocks on and below the diagonal are stored.
  __device__ __forceinline__ void rows(int i, int kb, s16x8 (&f)[2][2]) const {
    if (kb > i) cross(i, kb, f);
    else along(i, kb, f);
  }
};
__device__ __forceinline__ f32x16 three(const s16x8 (&q)[2], const s16x8 (&p)[2], f32x16 c) {
  c = mma<_Float16>(q[1], p[0], c);
  c = mma<_Float16>(q[0], p[1], c);
  return mma<_Float16>(q[0], p[0], c);
}
// A block's values to and from pairs: lane l has row l % 32, columns 8 g + 4 (l / 32) + e.
__device__ __forceinline__ char* chip_block(uint16_t* lds, int ld, int bi, int bj, int lane) {
  return reinterpret_cast<char*>(lds) + (bi * 32 + (lane & 31)) * 4 * ld + (bj >> 1) * 256 + (lane >> 5) * 8;
}
__device__ __forceinline__ void chip_put(uint16_t* lds, int ld, int bi, int bj, int lane, f32x16 v) {
  char* at = chip_block(lds, ld, bi, bj, lane);
  const int low = place_chip(lane & 31, 0) * 16 ^ (bj & 1) * 128;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    f16x4 hi, lo;
    split2(f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]}, hi, lo);
    *reinterpret_cast<f16x4*>(at + (low ^ (g * 32))) = hi;
    *reinterpret_cast<f16x4*>(at + (low ^ (g * 32 + 16))) = lo;
  }
}
__device__ __forceinline__ f32x4 chip_get4(uint16_t* lds, int ld, int row, int col) {
  return __builtin_convertvector(*reinterpret_cast<const f16x4*>(chip_at(lds, ld, row, col, 0)), f32x4) +
         __builtin_convertvector(*reinterpret_cast<const f16x4*>(chip_at(lds, ld, row, col, 1)), f32x4);
}
__device__ __forceinline__ f32x16 chip_get(uint16_t* lds, int ld, int bi, int bj, int lane) {
  const char* at = chip_block(lds, ld, bi, bj, lane);
  const int low = place_chip(lane & 31, 0) * 16 ^ (bj & 1) * 128;
  f32x16 v;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const f32x4 w = __builtin_convertvector(*reinterpret_cast<const f16x4*>(at + (low ^ (g * 32))), f32x4) +
                    __builtin_convertvector(*reinterpret_cast<const f16x4*>(at + (low ^ (g * 32 + 16))), f32x4);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * g + e] = w[e];
  }
  return v;
}

// On chip B is b A + c A^2: the wavefronts keep their blocks of X in registers as float32 from step to step, and a X is added to a
// product's result.

// The steps of a matrix of 97 to 128 rows and columns.  The ten blocks of a symmetric result go to the eight wavefronts so that
// each of the four SIMDs (wavefronts w and w + 4) has two or three; X's sixteen go two to each.  A wavefront keeps its blocks of
// A in registers for the term b A.
__device__ __forceinline__ void chip_steps_square(uint16_t* lx, uint16_t* la, const NsSteps& k, int lane, int wave) {
  constexpr int LD = 128;
  const ChipMatrix mx(lx, LD, lane), ma(la, LD, lane);
  // (0,0) and (1,1); (2,2) and (3,3); (1,0); (2,0); (3,0); (2,1); (3,1); (3,2)
  const int n_own = wave < 2 ? 2 : 1;
  const int bi[2] = {0x33232120 >> 4 * wave & 15, 2 * wave + 1}, bj[2] = {0x21100020 >> 4 * wave & 15, 2 * wave + 1};
  const int xi = (wave >> 2) * 2, xj = wave & 3;                     // X's blocks (xi, xj) and (xi + 1, xj)
  f32x16 own[2] = {chip_get(lx, LD, xi, xj, lane), chip_get(lx, LD, xi + 1, xj, lane)};
  for (int step = 0; step < k.steps; ++step) {
    f32x16 a[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      a[o] = 0.0f;
      if (o >= n_own) continue;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        s16x8 p[2][2], q[2][2];
        mx.along(bi[o], kb, p);
        if (wave < 2) {              // diagonal blocks
          a[o] = three(p[0], p[0], a[o]);
          a[o] = three(p[1], p[1], a[o]);
          continue;
        }
        mx.along(bj[o], kb, q);
        a[o] = three(q[0], p[0], a[o]);
        a[o] = three(q[1], p[1], a[o]);
      }
      a[o] *= k.gram[step];
      chip_put(la, LD, bi[o], bj[o], lane, a[o]);
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      if (o >= n_own) continue;
      f32x16 c = 0.0f;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        s16x8 p[2][2], q[2][2];
        ma.rows(bi[o], kb, p);
        if (wave < 2) {
          c = three(p[0], p[0], c);
          c = three(p[1], p[1], c);
          continue;
        }
        ma.rows(bj[o], kb, q);
        c = three(q[0], p[0], c);
        c = three(q[1], p[1], c);
      }
      a[o] = c * k.square[step].product + a[o] * k.square[step].own;
    }
    __syncthreads();                 // everyone has read A
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (o < n_own) chip_put(la, LD, bi[o], bj[o], lane, a[o]);
    __syncthreads();
    f32x16 x[2];
    x[0] = x[1] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      s16x8 p[2][2][2], q[2][2];
      mx.cross(xj, kb, q);
      ma.rows(xi, kb, p[0]);
      ma.rows(xi + 1, kb, p[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int o = 0; o < 2; ++o) x[o] = three(q[h], p[o][h], x[o]);
    }
    __syncthreads();                 // everyone has read X
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      own[o] = x[o] * k.apply[step] + own[o] * k.own[step];
      chip_put(lx, LD, xi + o, xj, lane, own[o]);
    }
    __syncthreads();
  }
}

// The steps of a matrix of fewer rows and up to CAP columns: for A the wavefronts share out the columns and each forms every
// block; a column block of X is a wavefront's own.
template <int MB>
__device__ __forceinline__ void chip_steps(uint16_t* lx, uint16_t* la, float* parts, int n64, const NsSteps& k, int lane, int wave) {
  constexpr int LDA = Chip<MB>::LDA, S = MB * (MB + 1) / 2, COLS = (Chip<MB>::CAP / 32 + kChipWaves - 1) / kChipWaves;
  const ChipMatrix mx(lx, n64, lane), ma(la, LDA, lane);
  f32x16 own[COLS][MB];              // column blocks wave, wave + 8 ..
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      own[c][i] = 0.0f;
      if (wave + c * kChipWaves < n64 / 32) own[c][i] = chip_get(lx, n64, i, wave + c * kChipWaves, lane);
    }
  for (int step = 0; step < k.steps; ++step) {
    f32x16 a[S];
#pragma unroll
    for (int s = 0; s < S; ++s) a[s] = 0.0f;
    for (int kb = wave; kb < n64 / 32; kb += kChipWaves) {
      s16x8 p[MB][2][2];
#pragma unroll
      for (int i = 0; i < MB; ++i) mx.along(i, kb, p[i]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0, s = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j <= i; ++j, ++s) a[s] = three(p[j][h], p[i][h], a[s]);
    }
    const int share = n64 / 32 < kChipWaves ? n64 / 32 : kChipWaves;       // wavefronts that have columns
#pragma unroll
    for (int i = 0, s = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j <= i; ++j, ++s) {
        if (s > 0) __syncthreads();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 v = {a[s][4 * g], a[s][4 * g + 1], a[s][4 * g + 2], a[s][4 * g + 3]};
          *reinterpret_cast<f32x4*>(parts + (wave * 32 + (lane & 31)) * kPartRow + 8 * g + 4 * (lane >> 5)) = v;
        }
        __syncthreads();
        if (threadIdx.x < 256) {
          const int r = static_cast<int>(threadIdx.x) >> 3, c = (static_cast<int>(threadIdx.x) & 7) * 4;
          f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int w = 0; w < share; ++w) v += *reinterpret_cast<const f32x4*>(parts + (w * 32 + r) * kPartRow + c);
          f16x4 hi, lo;
          split2(v * k.gram[step], hi, lo);
          *reinterpret_cast<f16x4*>(chip_at(la, LDA, i * 32 + r, j * 32 + c, 0)) = hi;
          *reinterpret_cast<f16x4*>(chip_at(la, LDA, i * 32 + r, j * 32 + c, 1)) = lo;
        }
      }
    __syncthreads();
    f32x16 b = 0.0f;
    int bi = 0, bj = wave;           // block `wave` of the lower triangle
    while (bj > bi) bj -= ++bi;
    if (wave < S) {
#pragma unroll
      for (int kb = 0; kb < MB; ++kb) {
        s16x8 p[2][2], q[2][2];
        ma.rows(bi, kb, p);
        ma.rows(bj, kb, q);
        b = three(q[0], p[0], b);
        b = three(q[1], p[1], b);
      }
      b = b * k.square[step].product + chip_get(la, LDA, bi, bj, lane) * k.square[step].own;
    }
    __syncthreads();
    if (wave < S) chip_put(la, LDA, bi, bj, lane, b);
    __syncthreads();
#pragma unroll
    for (int col = 0; col < COLS; ++col) {
      const int xj = wave + col * kChipWaves;
      if (xj >= n64 / 32) break;
      f32x16 x[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) x[i] = 0.0f;
#pragma unroll
      for (int kb = 0; kb < MB; ++kb) {
        s16x8 q[2][2];
        mx.cross(xj, kb, q);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          s16x8 p[2][2];
          ma.rows(i, kb, p);
          x[i] = three(q[0], p[0], x[i]);
          x[i] = three(q[1], p[1], x[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        own[col][i] = x[i] * k.apply[step] + own[col][i] * k.own[step];
        chip_put(lx, n64, i, xj, lane, own[col][i]);
      }
    }
    __syncthreads();
  }
}

// One matrix a block, from the gradient to the updated weight: X and, in turn, A and B as pairs in LDS.  SQUARE: those of 97
// to 128 rows and columns.  Measured (us a call, five steps): 128 x 128 39.5 (5.5 a step), 64 x 64 23.7, 32 x 32 13.2, 22 x 840 33.5,
// 96 x 192 57, 64 x 384 43.
template <bool SQUARE>
__global__ __launch_bounds__(kChipThreads) void ns_chip_kernel(NsTable t, NsSteps k) {
  __shared__ __attribute__((aligned(16))) char pool[SQUARE ? Chip<4>::BYTES : kChipBytes];
  __shared__ double buf[kChipWaves];
  const NsMat& a = t.m[blockIdx.x];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mb = a.m_pad / 32, n64 = a.n_pad;
  uint16_t* lx = reinterpret_cast<uint16_t*>(pool);
  // U as float32 in the places that its pairs will have: values 8 c .. + 3 of a row in its chunk 2 c, + 4 .. + 7 in the next
  const auto raw_at = [&](int row, int col) {
    return reinterpret_cast<float*>(lx + row * 2 * n64 + place_chip(row, (col >> 2)) * 8) + (col & 3);
  };
  if ((a.tall ? a.cols : a.rows) != mb * 32 || (a.tall ? a.rows : a.cols) != n64) {
    for (int i = threadIdx.x; i < mb * 32 * n64 / 4; i += kChipThreads) reinterpret_cast<f32x4*>(pool)[i] = 0.0f;
    __syncthreads();
  }
  const int groups = (a.cols + 3) / 4;                 // of four neighbours of the matrix's rows
  constexpr int AHEAD = 4;                             // groups whose loads are on their way together
  double s = 0.0;
  for (int i0 = threadIdx.x; i0 < a.rows * groups; i0 += AHEAD * kChipThreads) {
    f32x4 g[AHEAD], m[AHEAD];
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const int i = i0 + n * kChipThreads, r = i / groups, c = i % groups * 4;
      g[n] = m[n] = 0.0f;
      if (i >= a.rows * groups) continue;
      g[n] = read4(a.src, a.lds, r, c, a.cols, t.type, a.vec_src);
      if (t.muon) m[n] = read4(a.mom, a.ldo, r, c, a.cols, QHA_F32, a.vec_mom);
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const int i = i0 + n * kChipThreads, r = i / groups, c = i % groups * 4;
      if (i >= a.rows * groups) continue;
      if (t.muon) {
        m[n] = m[n] * t.mu + g[n] * t.grad_scale;
        write4(a.mom, a.ldo, r, c, a.cols, QHA_F32, a.vec_mom, m[n]);
      }
      f32x4 u = update_of(t, g[n], m[n]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c + e >= a.cols) u[e] = 0.0f;
        s += static_cast<double>(u[e]) * static_cast<double>(u[e]);
      }
      if (a.tall) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < a.cols) *raw_at(c + e, r) = u[e];
      } else {
        *reinterpret_cast<f32x4*>(raw_at(r, c)) = u;
      }
    }
  }
  const double by = scale_of(block_sum(s, buf), t.eps);      // its barriers make U whole
  for (int i = threadIdx.x; i < mb * 32 * n64 / 8; i += kChipThreads) {
    const int row = i / (n64 / 8), col = i % (n64 / 8) * 8;
    f32x4* at[2] = {reinterpret_cast<f32x4*>(raw_at(row, col)), reinterpret_cast<f32x4*>(raw_at(row, col + 4))};
    f16x4 hi[2], lo[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 v = *at[h];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(static_cast<double>(v[e]) * by);
      split2(v, hi[h], lo[h]);
    }
    *reinterpret_cast<f16x8*>(at[0]) = __builtin_shufflevector(hi[0], hi[1], 0, 1, 2, 3, 4, 5, 6, 7);
    *reinterpret_cast<f16x8*>(at[1]) = __builtin_shufflevector(lo[0], lo[1], 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __syncthreads();
  if constexpr (SQUARE) {
    chip_steps_square(lx, lx + Chip<4>::X_SIZE, k, lane, wave);
  } else if (mb == 3) {
    chip_steps<3>(lx, lx + Chip<3>::X_SIZE, reinterpret_cast<float*>(lx + Chip<3>::X_SIZE + Chip<3>::A_SIZE), n64, k, lane, wave);
  } else if (mb == 2) {
    chip_steps<2>(lx, lx + Chip<2>::X_SIZE, reinterpret_cast<float*>(lx + Chip<2>::X_SIZE + Chip<2>::A_SIZE), n64, k, lane, wave);
  } else {
    chip_steps<1>(lx, lx + Chip<1>::X_SIZE, reinterpret_cast<float*>(lx + Chip<1>::X_SIZE + Chip<1>::A_SIZE), n64, k, lane, wave);
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < a.rows * groups; i += kChipThreads) {
    const int r = i / groups, c = i % groups * 4;
    f32x4 v;
    if (a.tall) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = c + e < a.cols ? static_cast<float>(*reinterpret_cast<const _Float16*>(chip_at(lx, n64, c + e, r, 0))) +
                                    static_cast<float>(*reinterpret_cast<const _Float16*>(chip_at(lx, n64, c + e, r, 1)))
                              : 0.0f;
    } else {
      v = chip_get4(lx, n64, r, c);
    }
    apply4(t, a, r, c, v * t.result);
  }
}

// ---------------------------------------------------------------------------------------------
// products of few tiles
// ---------------------------------------------------------------------------------------------

constexpr int kDirectWaves = 4, kDirectChunks = 4, kFusedRows = 128, kFusedBlocks = 512;

// Operands of 32 rows and 32 steps straight from memory: p points to the rows' first block.
__device__ __forceinline__ void direct_load(const uint16_t* p, int lane, int64_t chunk, s16x8 (&f)[2][2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int part = 0; part < 2; ++part) f[h][part] = *reinterpret_cast<const s16x8*>(p + (2 * chunk + h) * kBlock + part * kLo + lane_at(lane, h));
}

// The same products for a batch whose tiles would leave most of the chip idle, where a launch's time is that of its chain of loads
// and barriers: a block owns 32 x 32 values, and its wavefronts share out the reduction by 32 steps, four of which they load at
// once straight from memory (X's transpose is kept for the last product).  Their sums meet in LDS and are added in order.
// FUSED (X of at most 128 rows): the last product's block forms its 32 rows of B itself, from A, which saves a launch.
template <int KIND, bool FUSED>
__global__ __launch_bounds__(kDirectWaves * 64) void ns_direct_kernel(const NsTable* table, NsFirst first, NsCoef sq, NsCoef k, int32_t from, uint32_t total) {
  constexpr bool SYM = KIND == NS_GRAM || KIND == NS_SQUARE;
  constexpr int W = kDirectWaves, CH = kDirectChunks;
  static_assert(!FUSED || (!SYM && kFusedRows <= 32 * W), "a block of B's rows for each wavefront");
  __shared__ float part[W][32][kPartRow];
  __shared__ __attribute__((aligned(16))) uint16_t panel[FUSED ? 32 * kFusedRows * 2 : 8];
  const uint32_t band = (total + kXcds - 1) / kXcds;
  const uint32_t block = blockIdx.x % kXcds * band + blockIdx.x / kXcds;
  if (block >= total) return;
  const NsTable& t = *table;
  const int i = matrix_of(first, block);
  const NsMat& a = t.m[i];
  const int tile = static_cast<int>(block - first.block[i]);
  const int m_pad = a.m_pad;
  int mt, nt;
  if constexpr (SYM) {
    triangle(tile, &mt, &nt);
  } else {
    mt = tile % (m_pad / 32);
    nt = tile / (m_pad / 32);
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const NsParts w(a);
  const uint16_t* x = w.x(from);
  const int64_t depth = KIND == NS_GRAM ? a.n_pad : m_pad;
  const auto rows_of = [&](const uint16_t* base, int block_row) {
    return base + block_row * (depth >> 4) * kBlock;
  };
  const uint16_t* p = rows_of(KIND == NS_GRAM ? x : KIND == NS_SQUARE || FUSED ? w.a() : w.b(), mt);
  const uint16_t* q = rows_of(KIND == NS_GRAM ? x : KIND == NS_SQUARE ? w.a() : w.xt(from), nt);
  static_assert(W * 64 == 256, "four of a block's values a thread");
  // four neighbours of a row a thread; A's for the square product are on their way early
  const int r = static_cast<int>(threadIdx.x) & 31, c = static_cast<int>(threadIdx.x >> 5) * 4;
  const int64_t row = mt * 32 + r, col = nt * 32 + c, cols = SYM ? m_pad : a.n_pad;
  f32x4 own = {0.0f, 0.0f, 0.0f, 0.0f};
  if (KIND == NS_SQUARE) own = get4(w.a(), block_at(row, col, cols));

  f32x16 acc[3];
#pragma unroll
  for (int e = 0; e < 3; ++e) acc[e] = 0.0f;
  const auto add = [&](const s16x8 (&fq)[2][2], const s16x8 (&fp)[2][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      acc[0] = mma<_Float16>(fq[h][1], fp[h][0], acc[0]);
      acc[1] = mma<_Float16>(fq[h][0], fp[h][1], acc[1]);
      acc[2] = mma<_Float16>(fq[h][0], fp[h][0], acc[2]);
    }
  };
  const int64_t chunks = depth / 32;
  if constexpr (FUSED) {
    s16x8 x_rows[2][2];
    if (wave < chunks) direct_load(q, lane, wave, x_rows);
    if (wave < chunks) {             // B's rows 32 mt .., columns 32 wave ..
      const uint16_t* other = rows_of(w.a(), wave);
      f32x4 a_own[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) a_own[g] = get4(w.a(), block_at(mt * 32 + (lane & 31), wave * 32 + 8 * g + 4 * (lane >> 5), m_pad));
      for (int64_t s = 0; s < chunks; s += CH) {
        s16x8 fp[CH][2][2], fq[CH][2][2];
#pragma unroll
        for (int n = 0; n < CH; ++n)
          if (s + n < chunks) {
            direct_load(p, lane, s + n, fp[n]);
            direct_load(other, lane, s + n, fq[n]);
          }
#pragma unroll
        for (int n = 0; n < CH; ++n)
          if (s + n < chunks) add(fq[n], fp[n]);
      }
      f32x16 b = (acc[0] + acc[1] + acc[2]) * sq.product;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 v = square_terms(sq, f32x4{b[4 * g], b[4 * g + 1], b[4 * g + 2], b[4 * g + 3]}, a_own[g],
                                     mt * 32 + (lane & 31), wave * 32 + 8 * g + 4 * (lane >> 5));
#pragma unroll
        for (int e = 0; e < 4; ++e) b[4 * g + e] = v[e];
      }
      chip_put(panel, kFusedRows, 0, wave, lane, b);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 3; ++e) acc[e] = 0.0f;
    if (wave < chunks) {
      s16x8 b_rows[2][2];
      ChipMatrix(panel, kFusedRows, lane).along(0, wave, b_rows);
      add(x_rows, b_rows);
    }
  } else {
    for (int64_t s = wave; s < chunks; s += W * CH) {
      s16x8 fp[CH][2][2], fq[CH][2][2];
#pragma unroll
      for (int n = 0; n < CH; ++n)
        if (s + n * W < chunks) {
          direct_load(p, lane, s + n * W, fp[n]);
          direct_load(q, lane, s + n * W, fq[n]);
        }
#pragma unroll
      for (int n = 0; n < CH; ++n)
        if (s + n * W < chunks) add(fq[n], fp[n]);
    }
  }
  acc[2] += acc[0] + acc[1];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const f32x4 v = {acc[2][4 * g], acc[2][4 * g + 1], acc[2][4 * g + 2], acc[2][4 * g + 3]};
    *reinterpret_cast<f32x4*>(&part[wave][lane & 31][8 * g + 4 * (lane >> 5)]) = v;
  }
  __syncthreads();
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int n = 1; n <= W; ++n) v += *reinterpret_cast<const f32x4*>(&part[((SYM ? 0u : static_cast<uint32_t>(mt)) + n) % W][r][c]);      // a X's last
  v *= k.product;
  if constexpr (KIND == NS_SQUARE) v = square_terms(k, v, own, row, col);
  if constexpr (KIND != NS_LAST) put4(KIND == NS_GRAM ? w.a() : KIND == NS_SQUARE ? w.b() : w.x(from ^ 1), block_at(row, col, cols), v);
  // the mirror of a symmetric result, the transpose of X, or the rows of the result
  if (SYM && mt == nt) return;
  *reinterpret_cast<f32x4*>(&part[0][r][c]) = v;         // each thread read its own four values of it alone
  __syncthreads();
  if constexpr (KIND == NS_LAST) {
    finish_block<256>(t, a, &part[0][0][0], mt * 32, nt * 32, threadIdx.x);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = part[0][c + e][r];
    put4(KIND == NS_GRAM ? w.a() : KIND == NS_SQUARE ? w.b() : w.xt(from ^ 1), block_at(nt * 32 + r, mt * 32 + c, m_pad), v);
  }
}

// ---------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------

constexpr int64_t kBatchValues = 1LL << 27;      // values of X in flight in a batch of several matrices

constexpr size_t kTableBytes = (sizeof(NsTable) + 255) / 256 * 256;

int64_t pad32(int64_t x) { return (x + 31) / 32 * 32; }
int64_t pad64(int64_t x) { return (x + 63) / 64 * 64; }
// Rows of X by 32 where the matrix fits in LDS, else 0.  (From memory, us for five steps: 128 x 128 73, on chip 40; 40 of them 108, 63;
// 96 x 192 69, 56; 64 x 384 70, 43; 22 x 840 72, 34; 32 x 32 55, 13.)
int chip_rows_of(const NsMatrix& m) {
  const int64_t s = m.rows < m.cols ? m.rows : m.cols, l = pad64(m.rows < m.cols ? m.cols : m.rows);
  if (s <= 32 && l <= Chip<1>::CAP) return 1;
  if (s <= 64 && l <= Chip<2>::CAP) return 2;
  if (s <= 96 && l <= Chip<3>::CAP) return 3;
  return s <= 128 && l <= Chip<4>::CAP ? 4 : 0;
}
int64_t piece_count(const NsMatrix& m, int64_t rows) {
  return (m.rows + rows - 1) / rows * ((m.cols + kPieceCols - 1) / kPieceCols);
}
int64_t short_side(const NsMatrix& m) { return pad32(m.rows < m.cols ? m.rows : m.cols); }
int64_t long_side(const NsMatrix& m) { return pad32(m.rows < m.cols ? m.cols : m.rows); }

// How a batch is worked: by tiles or directly, and rows of a piece to measure.
struct NsPlan {
  bool direct, fused;
  int piece_rows;
};
NsPlan plan_of(const NsMatrix* m, const int64_t* index, int count) {
  int64_t pieces = 0, tiles = 0, blocks = 0, deepest = 0, values = 0;
  bool fits = true;
  for (int i = 0; i < count; ++i) {
    const NsMatrix& x = m[index[i]];
    const int64_t s = short_side(x), l = long_side(x), rows = s / 32, cols = l / 32;
    pieces += piece_count(x, 8);
    fits = fits && s <= kFusedRows;
    tiles += (s + 63) / 64 * ((l + 63) / 64);
    blocks += rows * cols;
    deepest = l + 2 * s > deepest ? l + 2 * s : deepest;
    values += 64 * (rows * (rows + 1) / 2 * (l + (s <= kFusedRows ? 0 : s)) + rows * cols * s);
  }
  // us of a step: the operands that direct blocks read, at 13 TB/s; the tiles' steps of 32, one after the other.  Measured, direct and
  // tiled (us, five steps): 256 x 256 92, 104; 8 of them 102, 106; 16 148, 110; 512 x 512 115, 144; four 192, 154; 700 x 700 146, 162;
  // 800 x 800 183, 173; 1000 x 1000 270, 189; 39 x 3035 110, 161; 128 x 8000 235, 309; 300 x 8000 312, 345; 256 x 16000 488, 562; near each
  // other, and taken for direct: 520 x 4000 278, 268, four of 200 x 2000 182, 175, 12 of 96 x 2848 234, 222
  const double direct = static_cast<double>(values) * 4.0 / 13e6;
  const double tiled = 0.26 * static_cast<double>(deepest) / 32.0 * (tiles > 512 ? static_cast<double>(tiles) / 512.0 : 1.0);
  // each block forms B's rows: many of them lose more by it than a launch costs (12 of 96 x 2848 265 us, 237 unfused)
  NsPlan p = {direct < tiled, fits && blocks <= kFusedBlocks, 8};
  while (p.piece_rows < 64 && pieces > 1024) {
    p.piece_rows *= 2;
    pieces /= 2;
  }
  return p;
}
// a matrix's part of the workspace (NsParts)
size_t bytes_of(const NsMatrix& m, const NsPlan& p) {
  const int64_t s = short_side(m), l = long_side(m);
  return static_cast<size_t>((p.direct ? 4 : 2) * s * l + 2 * s * s) * 4 + static_cast<size_t>((piece_count(m, p.piece_rows) + 1) / 2 * 16);
}

enum { IN_MEMORY = 0, ON_CHIP = 1, ON_CHIP_SQUARE = 2 };
int place_of(const NsMatrix& m) {
  const int rows = chip_rows_of(m);
  return rows == 4 ? ON_CHIP_SQUARE : rows ? ON_CHIP : IN_MEMORY;
}

// The power of two that takes values of at most `most` to the end of half precision's range (65504, less what rounding may add), at most
// 2^largest, where steps have shrunk X to nothing.
double half_scale(double most, int largest) {
  const double bound = std::ldexp(1.0, largest);
  return most * bound > 60000.0 ? std::ldexp(1.0, std::ilogb(60000.0 / most)) : bound;
}

// The next batch of matrices of a place from *at on: their indices, at most kNsBatch.
int next_batch(const NsMatrix* m, int64_t n, int place, int64_t* at, int64_t* index) {
  int count = 0;
  int64_t values = 0;
  for (; *at < n && count < kNsBatch; ++*at) {
    const NsMatrix& x = m[*at];
    if (x.rows == 0 || x.cols == 0 || place_of(x) != place) continue;
    if (place == IN_MEMORY && count > 0 && values + x.rows * x.cols > kBatchValues) break;
    values += x.rows * x.cols;
    index[count++] = *at;
  }
  return count;
}

// Tiles of `side` of a batch's symmetric results, or of its X.
uint32_t tiles_of(const NsTable& t, bool sym, int side, NsFirst* first) {
  int64_t total = 0;
  if (first) first->n = t.n;
  for (int i = 0; i < t.n; ++i) {
    if (first) first->block[i] = static_cast<uint32_t>(total);
    const int64_t mt = (t.m[i].m_pad + side - 1) / side, nt = (t.m[i].n_pad + side - 1) / side;
    total += sym ? mt * (mt + 1) / 2 : mt * nt;
  }
  return static_cast<uint32_t>(total);
}

// The side of a launch's tiles, by the time that the busiest of the 256 compute units takes: its tiles' first loads and stores, and
// their steps.  Measured (us): gram products of 4096 x 4096: 192 222, 128 277, 256 281, 64 324; of 2528 x 3008: 128 89, 64 104, 192 137;
// of 24 of 1024 x 4096: 256 355, 128 393, 64 436, 192 447; of five of 544 x 1024: 64 14, 128 29.  Last products of the same: 256 335,
// 128 386, 64 494; 128 128, 64 159, 256 172; 256 585, 128 632, 64 839; 64 17, 128 19.
int side_of(const NsTable& t, bool sym, int64_t depth) {
  struct Speed {
    int side;
    double once, tile, step;         // us of a launch, of a tile, and of a step of the reduction in it
  };
  constexpr Speed speeds[] = {{64, 5.0, 1.0, 0.0078}, {128, 4.0, 3.0, 0.0235}, {192, 0.0, 10.0, 0.052}, {256, 0.0, 12.0, 0.083}};
  int best = 0;
  double least = 0.0;
  for (const Speed& v : speeds) {
    if (v.side == 192 && !sym) continue;
    const double most = static_cast<double>((tiles_of(t, sym, v.side, nullptr) + 255) / 256);
    // a unit holds two tiles of 128: one by itself runs slower
    const double step = v.side == 128 && most == 1.0 ? 0.0275 : v.step;
    const double time = v.once + most * (v.tile + step * static_cast<double>(depth));
    if (best == 0 || time < least) {
      best = v.side;
      least = time;
    }
  }
  return best;
}

// A launch's tiles: their side, their number, and each matrix's first.
struct NsTiles {
  int side;
  uint32_t total;
  NsFirst first;
  uint32_t grid() const { return (total + static_cast<uint32_t>(kXcds) - 1) / static_cast<uint32_t>(kXcds) * static_cast<uint32_t>(kXcds); }
};

template <int KIND>
void run_product(const NsTable* t, const NsTiles& b, int64_t depth, const NsCoef& k, int from, hipStream_t s) {
  constexpr bool SYM = KIND == NS_GRAM || KIND == NS_SQUARE;
  const uint32_t g = b.grid();
  if (b.side == 256) ns_product_kernel<KIND, 4, 2, 2, 4, 2, 1><<<g, 512, 0, s>>>(t, b.first, k, from, b.total);
  else if (b.side == 128) ns_product_kernel<KIND, 2, 2, 2, 2, 2, 1><<<g, 256, 0, s>>>(t, b.first, k, from, b.total);
  // two halves of the reduction where a compute unit has one tile at most, and steps enough (us, five steps, whole and halved:
  // 1024 x 4096 410, 362; 1300 x 1300 282, 268; 1000 x 1000 202, 189; four of 512 x 512 154, 158, 16 of 256 x 256 110, 118)
  else if (b.side == 64 && b.total <= 256 && depth > 512) ns_product_kernel<KIND, 1, 1, 2, 2, 3, 2><<<g, 512, 0, s>>>(t, b.first, k, from, b.total);
  else if (b.side == 64) ns_product_kernel<KIND, 1, 1, 2, 2, 3, 1><<<g, 256, 0, s>>>(t, b.first, k, from, b.total);
  else if constexpr (SYM) ns_product_kernel<KIND, 3, 3, 2, 2, 2, 1><<<g, 256, 0, s>>>(t, b.first, k, from, b.total);
}

// One step of a batch; the last one's results go where the call wants them.
void run_step(const NsTable* t, const NsPlan& plan, const NsTiles& gram, const NsTiles& square, const NsTiles& all,
              int64_t most_m, int64_t most_n, const NsSteps& k, int step, hipStream_t s) {
  const int from = step & 1;
  const bool last = step + 1 == k.steps;
  const NsCoef gr = {k.gram[step], 0.0f, 0.0f}, ap = {k.apply[step], 0.0f, 0.0f};
  if (plan.direct) {
    const NsCoef& sq = k.square[step];
    constexpr int NT = kDirectWaves * 64;
    ns_direct_kernel<NS_GRAM, false><<<gram.grid(), NT, 0, s>>>(t, gram.first, sq, gr, from, gram.total);
    if (!plan.fused) ns_direct_kernel<NS_SQUARE, false><<<square.grid(), NT, 0, s>>>(t, square.first, sq, sq, from, square.total);
    if (plan.fused && last) ns_direct_kernel<NS_LAST, true><<<all.grid(), NT, 0, s>>>(t, all.first, sq, ap, from, all.total);
    else if (plan.fused) ns_direct_kernel<NS_APPLY, true><<<all.grid(), NT, 0, s>>>(t, all.first, sq, ap, from, all.total);
    else if (last) ns_direct_kernel<NS_LAST, false><<<all.grid(), NT, 0, s>>>(t, all.first, sq, ap, from, all.total);
    else ns_direct_kernel<NS_APPLY, false><<<all.grid(), NT, 0, s>>>(t, all.first, sq, ap, from, all.total);
    return;
  }
  run_product<NS_GRAM>(t, gram, most_n, gr, from, s);
  run_product<NS_SQUARE>(t, square, most_m, k.square[step], from, s);
  if (last) run_product<NS_LAST>(t, all, most_m, ap, from, s);
  else run_product<NS_APPLY>(t, all, most_m, ap, from, s);
}

}  // namespace

size_t ns_workspace(const NsMatrix* m, int64_t n) {
  size_t most = 0;
  int64_t index[kNsBatch];
  for (int64_t at = 0; at < n;) {
    const int count = next_batch(m, n, IN_MEMORY, &at, index);
    size_t need = 0;
    const NsPlan plan = plan_of(m, index, count);
    for (int i = 0; i < count; ++i) need += bytes_of(m[index[i]], plan);
    if (count) need += kTableBytes;
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
  double scale_x = kScaleX;
  for (int i = 0; i < args.steps; ++i) {
    const double a = args.coefficients[3 * i], b = args.coefficients[3 * i + 1], c = args.coefficients[3 * i + 2];
    // X's and B's scales are float32 values, as are all ratios, which differ from their bounds' by less than 2^17
    const double scale_a = half_scale(args.most_x[i] * args.most_x[i], 240), scale_b = half_scale(args.most_b[i], 120);
    const double next = half_scale(args.most_x[i + 1], 120);
    k.gram[i] = static_cast<float>(scale_a / (scale_x * scale_x));
    k.square[i] = {static_cast<float>(c * (scale_b / (scale_a * scale_a))), static_cast<float>(b * (scale_b / scale_a)), static_cast<float>(a * scale_b)};
    k.apply[i] = static_cast<float>(next / (scale_b * scale_x));
    k.own[i] = static_cast<float>(a * (next / scale_x));
    scale_x = next;
  }
  t.result = static_cast<float>(1.0 / scale_x);
  int64_t index[kNsBatch];
  bool launched = false;
  NsPlan plan = {};
  const auto fill = [&](int count, bool small) {
    char* at = static_cast<char*>(ws) + kTableBytes;
    t.n = count;
    launched = true;
    for (int i = 0; i < count; ++i) {
      const NsMatrix& x = m[index[i]];
      NsMat& a = t.m[i];
      a.rows = static_cast<int32_t>(x.rows);
      a.cols = static_cast<int32_t>(x.cols);
      a.tall = x.rows > x.cols;
      const int64_t sh = a.tall ? x.cols : x.rows, lo = a.tall ? x.rows : x.cols;
      a.m_pad = static_cast<int32_t>(small ? 32 * chip_rows_of(x) : pad32(sh));
      a.n_pad = static_cast<int32_t>(small ? pad64(lo) : pad32(lo));
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
      a.ws = at;
      at += bytes_of(x, plan);
    }
  };
  for (int place : {ON_CHIP, ON_CHIP_SQUARE})
    for (int64_t at = 0; at < n;) {
      const int count = next_batch(m, n, place, &at, index);
      if (count == 0) break;
      fill(count, true);
      if (place == ON_CHIP) ns_chip_kernel<false><<<count, kChipThreads, 0, s>>>(t, k);
      else ns_chip_kernel<true><<<count, kChipThreads, 0, s>>>(t, k);
    }
  for (int64_t at = 0; at < n;) {
    const int count = next_batch(m, n, IN_MEMORY, &at, index);
    if (count == 0) break;
    plan = plan_of(m, index, count);
    fill(count, false);
    t.piece_rows = plan.piece_rows;
    t.transposes = plan.direct;
    NsFirst pieces = {};
    pieces.n = count;
    uint32_t n_pieces = 0;
    for (int i = 0; i < count; ++i) {
      pieces.block[i] = n_pieces;
      n_pieces += static_cast<uint32_t>(piece_count(m[index[i]], plan.piece_rows));
    }
    int64_t most_m = 0, most_n = 0;
    for (int i = 0; i < count; ++i) {
      most_m = t.m[i].m_pad > most_m ? t.m[i].m_pad : most_m;
      most_n = t.m[i].n_pad > most_n ? t.m[i].n_pad : most_n;
    }
    const auto tiles = [&](bool symmetric, int side) {
      NsTiles b;
      b.side = side;
      b.total = tiles_of(t, symmetric, side, &b.first);
      return b;
    };
    const NsTiles whole = tiles(false, 64);
    const NsTiles gram = tiles(true, plan.direct ? 32 : side_of(t, true, most_n));
    const NsTiles square = tiles(true, plan.direct ? 32 : side_of(t, true, most_m));
    const NsTiles all = tiles(false, plan.direct ? 32 : side_of(t, false, most_m));
    NsTable* table = static_cast<NsTable*>(ws);
    ns_measure_kernel<<<n_pieces, 256, 0, s>>>(t, pieces, reinterpret_cast<uint32_t*>(table));
    ns_split_kernel<<<whole.total, 256, 0, s>>>(table, whole.first);
    for (int i = 0; i < args.steps; ++i) run_step(table, plan, gram, square, all, most_m, most_n, k, i, s);
  }
  return launched ? hipGetLastError() : hipSuccess;
}

}  // namespace qha
