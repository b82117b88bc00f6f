// Gated projection H = act(A Wg^T) * (A Wu^T) and its gradients on the matrix cores.
//
// Mathematics: G = A Wg^T, U = A Wu^T, H = act(G) U.  Backward: dG = dH U act'(G), dU = dH act(G),
// dA = [dG dU] [Wg; Wu], [dWg; dWu] = [dG dU]^T A.  16-bit types multiply as they are; float32
// values are split exactly into three bf16 parts (hi, mid, lo) and a product is rebuilt from the six part
// products of weight >= 2^-16 of it (the dropped ones total below 2^-23 of the product).  [dG dU] of 16-bit types enters the
// float32 dW in three bf16 parts or two scaled f16 ones, and dA, a 16-bit result, in one.  All sums
// are float32 in the matrix cores' accumulators; a reduction that is split leaves float32 partials that
// are added in float64.
//
// One product kernel serves the three: a block owns a tile of C, steps through the reduction BK at a time
// with two LDS buffers per operand, and its wavefronts own pieces of the tile as 32x32 accumulators.
// Operands come in two orders.  Stored along the reduction (A and W in the forward, [dG dU] in dA)
// their tiles lie row by row in LDS and a lane reads its eight values at once; stored across it (W in
// dA, both operands of dW) the tile keeps the reduction index as its rows and the transposing LDS
// read hands a lane its values.  Tiles go from memory to LDS directly, 16 bytes a lane, into places
// permuted so that neither read meets bank conflicts; the last, partial step goes through registers,
// which write zeros where the reduction ends.  The forward's B tile interleaves 32 rows of Wg with
// 32 of Wu, so a wavefront holds G and U of the same columns and the activation and product happen in registers.
// The matrix instruction's operands are swapped (C^T is formed), which leaves a lane four neighbouring
// columns of a row to store at once.
// Bound: the matrix cores for wide layers (16384 x 2048 -> 8192 bf16 with all three results stored, 1.01 to 1.08 ms, 1.02 to
// 1.09 PFLOP/s, where a plain library product of that size class reaches 1.25), the order of loads, products
// and stores within a tile for narrow ones (300k x 128 -> 128 float32, 158 to 192 us against 123 us for its bytes).
#include "act_common.hpp"
#include "qha_internal.hpp"
#include "tile_common.hpp"

#include <type_traits>

namespace qha {
namespace {

// An operand of a product: rows of ld values, 16-bit ones in one or more planes `plane` values apart (the parts of
// float32 values), or float32 ones that are split on their way out of LDS.
struct Operand {
  const uint16_t* p0;
  const uint16_t* p1;  // the second matrix of pairs, or of the reduction's second segment
  int64_t ld, ld1;     // of p0 and p1
  int64_t plane;
  int64_t rows;        // stored rows
  int64_t cols;        // stored columns (a multiple of 16 bytes)
};

enum { ORDER_ROWS = 0, ORDER_PAIRS = 1, ORDER_CROSS = 2 };
// ORDER_ROWS:  stored along the reduction; tile row r is stored row r0 + r
// ORDER_PAIRS: the same, tile rows alternate between p0 and p1 by 32 (p0 and p1 hold `rows` rows each)
// ORDER_CROSS: stored across the reduction; tile rows are steps of the reduction, stored columns c0 + c

// Places of 16-byte chunks in a tile's LDS image, PER chunks a row.  LDS serves 256 bytes at a time, so the reads
// that go together must fall on different sixteenths of 256 bytes.  Along the reduction, 16 lanes read one
// chunk of as many rows (rows of 128 or 64 bytes, two or four to 256).  Across it, a transposing read (16-bit)
// takes 64 bytes of four rows at a time, and a read of float32 columns 128 bytes of two rows eight apart.
// The permutations are their own inverses.
template <int PER>
__device__ __forceinline__ int permute_along(int row, int chunk) {
  static_assert(PER == 8 || PER == 4, "rows of 128 or 64 bytes");
  return PER == 8 ? chunk ^ ((row >> 1) & 7) : chunk ^ ((row >> 2) & 3);
}
template <bool RAW, int PER>
__device__ __forceinline__ int permute_cross(int k, int chunk) {
  static_assert(PER >= (RAW ? 16 : 8), "rows of at least 256 bytes of float32, 128 of 16-bit values");
  if (RAW) return chunk ^ (k & 8);
  return PER == 8 ? chunk ^ ((k & 2) << 1) : chunk ^ ((k & 3) << 2);
}

// A thread's share of a tile of ROWS x COLS values (as stored): its N 16-byte chunks, one per NT.  RAW: float32.
template <int ORDER, int ROWS, int COLS, int NT, bool RAW>
struct Stager {
  static constexpr int W = RAW ? 4 : 8;            // values in a chunk
  static constexpr int HALVES = RAW ? 2 : 1;       // 16-bit halves of a value
  static constexpr int PER = COLS / W;
  static constexpr int N = ROWS * PER / NT;
  static_assert(ROWS * PER % NT == 0, "whole chunks per thread");
  const uint16_t* at[N];

  static __device__ __forceinline__ int row(int i) { return (i * NT + static_cast<int>(threadIdx.x)) / PER; }
  static __device__ __forceinline__ int chunk(int i) {
    const int q = (i * NT + static_cast<int>(threadIdx.x)) % PER;
    if constexpr (ORDER == ORDER_CROSS) return permute_cross<RAW, PER>(row(i), q);
    else return permute_along<PER>(row(i), q);
  }
  // base: the operand's (or segment's) matrix; k0: first step of the reduction; first: the tile's first stored
  // row (along) or column (across).  Rows and columns past the end repeat the last ones; their results
  // are not stored.
  __device__ __forceinline__ void start(const Operand& o, const uint16_t* base, int64_t ld, int64_t first, int64_t k0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (ORDER == ORDER_CROSS) {
        int64_t c = first + chunk(i) * W;
        c = c < o.cols ? c : o.cols - W;
        at[i] = base + ((k0 + row(i)) * ld + c) * HALVES;
      } else {
        int64_t r;
        const uint16_t* p = base;
        if (ORDER == ORDER_PAIRS) {
          const int b = row(i) >> 5;
          r = first + (b >> 1) * 32 + (row(i) & 31);
          if (b & 1) {
            p = o.p1;
            ld = o.ld1;
          } else {
            ld = o.ld;
          }
        } else {
          r = first + row(i);
        }
        r = r < o.rows ? r : o.rows - 1;
        at[i] = p + (r * ld + k0 + chunk(i) * W) * HALVES;
      }
    }
  }
  __device__ __forceinline__ void load(int64_t plane, const uint16_t* lds) const {
    const uint32_t to = lds_address(lds) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
#pragma unroll
    for (int i = 0; i < N; ++i) load_to_lds(at[i] + plane, to + i * NT * 16);
  }
  __device__ __forceinline__ void next(int64_t ld) {
#pragma unroll
    for (int i = 0; i < N; ++i) at[i] += (ORDER == ORDER_CROSS ? ROWS * ld : COLS) * HALVES;
  }
  // The last, partial step: `left` steps of the reduction remain, the others become zero.
  __device__ __forceinline__ void load_partial(int64_t plane, int64_t left, uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      u32x4 v = {0, 0, 0, 0};
      if ((ORDER == ORDER_CROSS ? row(i) : chunk(i) * W) < left) v = *reinterpret_cast<const u32x4*>(at[i] + plane);
      *reinterpret_cast<u32x4*>(lds + (i * NT + threadIdx.x) * 8) = v;
    }
  }
};

// The matrix operand of 32 tile rows (or columns) from `at` on, 16 steps of the reduction from ks on:
// lane l holds row l % 32, steps 8 (l / 32) .. + 7.
template <int ORDER, int COLS>
__device__ __forceinline__ s16x8 fragment(const uint16_t* lds, int at, int ks, int lane) {
  if constexpr (ORDER == ORDER_CROSS) {
    // the transposing read takes 4 steps x 16 columns per 16 lanes: lane j of them addresses step
    // j / 4, columns 4 (j % 4), and receives four steps of column j
    const int j = lane & 15;
    const int col = at + ((lane >> 4) & 1) * 16 + 4 * (j & 3);
    const int k = ks + (lane >> 5) * 8 + (j >> 2);
    const int off = (col & 7);
    const uint16_t* lo = lds + k * COLS + permute_cross<false, COLS / 8>(k, col >> 3) * 8 + off;
    const uint16_t* hi = lds + (k + 4) * COLS + permute_cross<false, COLS / 8>(k + 4, col >> 3) * 8 + off;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)lo);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)hi);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const int row = at + (lane & 31);
    const int c = permute_along<COLS / 8>(row, (ks >> 3) + (lane >> 5));
    return *reinterpret_cast<const s16x8*>(lds + row * COLS + c * 8);
  }
}

// x = hi + mid + lo exactly: each part is rounded to nearest even, the remainders are exact in float32.
__device__ __forceinline__ void split3(f32x4 x, bf16x4& h, bf16x4& m, bf16x4& l) {
  h = __builtin_convertvector(x, bf16x4);
  const f32x4 r = x - __builtin_convertvector(h, f32x4);
  m = __builtin_convertvector(r, bf16x4);
  l = __builtin_convertvector(r - __builtin_convertvector(m, f32x4), bf16x4);
}

__device__ __forceinline__ void split8(f32x4 a, f32x4 b, s16x8 (&part)[3]) {
  bf16x4 h[2], m[2], l[2];
  split3(a, h[0], m[0], l[0]);
  split3(b, h[1], m[1], l[1]);
  part[0] = __builtin_bit_cast(s16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
  part[1] = __builtin_bit_cast(s16x8, __builtin_shufflevector(m[0], m[1], 0, 1, 2, 3, 4, 5, 6, 7));
  part[2] = __builtin_bit_cast(s16x8, __builtin_shufflevector(l[0], l[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// The same of a float32 tile: the three parts of its values.
template <int ORDER, int COLS>
__device__ __forceinline__ void fragment_raw(const uint16_t* lds, int at, int ks, int lane, s16x8 (&part)[3]) {
  const float* x = reinterpret_cast<const float*>(lds);
  f32x4 a, b;
  if constexpr (ORDER == ORDER_CROSS) {
    const int col = at + (lane & 31);
    const int k = ks + (lane >> 5) * 8;              // bit 3 of k .. k + 7 is that of k
    const float* p = x + k * COLS + permute_cross<true, COLS / 4>(k, col >> 2) * 4 + (col & 3);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = p[e * COLS];
      b[e] = p[(e + 4) * COLS];
    }
  } else {
    const int row = at + (lane & 31);
    const int c = (ks >> 2) + (lane >> 5) * 2;
    a = *reinterpret_cast<const f32x4*>(x + row * COLS + permute_along<COLS / 4>(row, c) * 4);
    b = *reinterpret_cast<const f32x4*>(x + row * COLS + permute_along<COLS / 4>(row, c + 1) * 4);
  }
  split8(a, b, part);
}

// Half precision's exponents end at 2^15 and 2^-14, which gradients of either scale pass.  A row or column of [dG dU] whose
// largest finite magnitude has the float32 bits `size` enters its products times 2^scale_of(size), which puts that
// largest into [2^14, 2^15), and the result's row is multiplied by the inverse.  Both factors are normal float32 powers of two:
// products of f16 values stay below 2^33, and the upper bound keeps the inverse of vanishing sizes normal.
__device__ __forceinline__ int scale_of(uint32_t size) {
  const int s = 14 + 127 - static_cast<int>(size >> 23);
  return s < 100 ? s : 100;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

struct ProductArgs {
  Operand a, b;
  int64_t m, n;             // C is m x n (forward: n columns of H)
  int64_t k;                // reduction: `segments` of k steps; the second takes A's columns from k on and B's p1
  int32_t segments;
  int64_t k_each;           // steps of the reduction per split (a multiple of BK)
  int32_t m_tiles, n_tiles, splits;
  // forward
  void* h;
  void* gate;
  void* up;
  int64_t ldh, ldg, ldu;
  int32_t act;
  // dA: c (half = m); dW: c, with rows from `half` on in c1; or the split's partial
  void* c;
  float* c1;
  int64_t ldc, ldc1;
  int64_t half;
  float* partial;           // [splits][m][n] when splits > 1
  const uint32_t* sizes;    // f16 gradients: the size that each row of C was scaled by, or null
};

enum { OUT_GATED = 0, OUT_DA = 1, OUT_DW = 2 };

template <typename O>
__device__ __forceinline__ void store4(O* p, f32x4 v);
template <>
__device__ __forceinline__ void store4<float>(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
template <>
__device__ __forceinline__ void store4<__bf16>(__bf16* p, f32x4 v) {
  *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
}
template <>
__device__ __forceinline__ void store4<_Float16>(_Float16* p, f32x4 v) {
  *reinterpret_cast<f16x4*>(p) = __builtin_convertvector(v, f16x4);
}

// 32 rows x CW columns of results on their way out through a wavefront's own piece of LDS, as streaming stores
// (300k x 128 float32 forward 183 against 212 us on one card: the operands stay in the caches).  Rows are 16 bytes
// longer than their values, which spreads a column of lanes over the banks.
template <typename O, int CW>
struct RowWriter {
  static constexpr int STRIDE = CW * sizeof(O) + 16;
  static constexpr int PER = CW * sizeof(O) / 16;       // 16-byte pieces of a row
  char* mine;
  int lane;
  __device__ __forceinline__ RowWriter(uint16_t* lds, int wave, int ln)
      : mine(reinterpret_cast<char*>(lds) + wave * 32 * STRIDE), lane(ln) {}
  // four values of row lane % 32, from column c + 4 (lane / 32) on
  __device__ __forceinline__ void put(int c, f32x4 v) {
    store4<O>(reinterpret_cast<O*>(mine + (lane & 31) * STRIDE + (c + (lane >> 5) * 4) * sizeof(O)), v);
  }
  // rows r0 .. of the output that lie in [0, rows), columns c0 .. below cols
  __device__ __forceinline__ void flush(O* to, int64_t ld, int64_t r0, int64_t rows, int64_t c0, int64_t cols) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int E = 16 / sizeof(O);
#pragma unroll
    for (int s = 0; s < 32 * PER / 64; ++s) {
      const int r = (s * 64 + lane) / PER, q = (s * 64 + lane) % PER;
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * STRIDE + q * 16);
      const int64_t row = r0 + r, col = c0 + q * E;
      if (row >= 0 && row < rows && col < cols) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(to + row * ld + col));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
};

// Tiles dealt to the XCDs in bands: consecutive blocks go to the eight XCDs in turn, so block b takes
// position b / 8 of band b % 8; within a band, tiles run down groups of eight row tiles before the next
// column tile, so that both operands' tiles are found in that XCD's L2.
__device__ __forceinline__ bool tile_of(const ProductArgs& p, int64_t b, int64_t* mt, int64_t* nt, int64_t* sp) {
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles * p.splits;
  const int64_t band = (tiles + kXcds - 1) / kXcds;
  const int64_t t = (b % kXcds) * band + b / kXcds;
  if (b / kXcds >= band || t >= tiles) return false;
  const int64_t plane = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  *sp = t / plane;
  const int64_t r = t % plane;
  const int64_t group = 8 * p.n_tiles;
  const int64_t g = r / group, in = r % group;
  const int64_t rows = p.m_tiles - 8 * g < 8 ? p.m_tiles - 8 * g : 8;
  *mt = 8 * g + in % rows;
  *nt = in / rows;
  return true;
}

// T: 16-bit type of the planes; O: type of the stored result; PA, PB: parts of A's and B's values (1 and 1,
// 2 and 1, 3 and 1, or 3 and 3); RA, RB: they are split from float32 values in LDS (else stored as planes).
// BM x BN tile of C (forward: BN counts the rows of Wg and Wu together), wavefronts of WM x WN.
template <typename T, typename O, int PA, int PB, bool RA, bool RB, int OA, int OB, int OUT, int BM, int BN, int BK, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void product_kernel(ProductArgs p) {
  constexpr int NT = (BM / WM) * (BN / WN) * 64;
  constexpr int A_ROWS = OA == ORDER_CROSS ? BK : BM, A_COLS = OA == ORDER_CROSS ? BM : BK;
  constexpr int B_ROWS = OB == ORDER_CROSS ? BK : BN, B_COLS = OB == ORDER_CROSS ? BN : BK;
  constexpr int LA = RA ? 1 : PA, LB = RB ? 1 : PB;                   // planes in LDS
  constexpr int A_SIZE = BM * BK * (RA ? 2 : 1), B_SIZE = BN * BK * (RB ? 2 : 1), BUF = LA * A_SIZE + LB * B_SIZE;
  constexpr int MI = WM / 32, NI = WN / 32;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * BUF];

  int64_t mt, nt, sp;
  if (!tile_of(p, blockIdx.x, &mt, &nt, &sp)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / (BN / WN), wn = wave % (BN / WN);
  const int64_t m0 = mt * BM;
  const int64_t n0 = nt * (OUT == OUT_GATED ? BN / 2 : BN);
  const int64_t kbeg = sp * p.k_each;
  const int64_t kend = kbeg + p.k_each < p.k ? kbeg + p.k_each : p.k;

  f32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  auto multiply = [&](const uint16_t* at) {
    const uint16_t* bt = at + LA * A_SIZE;
    s16x8 fa[2][MI][PA], fb[2][NI][PB];
    auto fetch = [&](int ks, int to) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if constexpr (RA) {
          fragment_raw<OA, A_COLS>(at, wm * WM + i * 32, ks, lane, fa[to][i]);
        } else {
#pragma unroll
          for (int pl = 0; pl < PA; ++pl) fa[to][i][pl] = fragment<OA, A_COLS>(at + pl * A_SIZE, wm * WM + i * 32, ks, lane);
        }
      }
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        if constexpr (RB) {
          fragment_raw<OB, B_COLS>(bt, wn * WN + j * 32, ks, lane, fb[to][j]);
        } else {
#pragma unroll
          for (int pl = 0; pl < PB; ++pl) fb[to][j][pl] = fragment<OB, B_COLS>(bt + pl * B_SIZE, wn * WN + j * 32, ks, lane);
        }
      }
    };
    fetch(0, 0);
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      const int now = ks / 16 & 1;
      if (ks + 16 < BK) fetch(ks + 16, now ^ 1);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          f32x16 c = acc[i][j];
          // smallest part products first
          if constexpr (PB == 3) {
            c = mma<T>(fb[now][j][1], fa[now][i][1], c);
            c = mma<T>(fb[now][j][0], fa[now][i][2], c);
            c = mma<T>(fb[now][j][2], fa[now][i][0], c);
            c = mma<T>(fb[now][j][0], fa[now][i][1], c);
            c = mma<T>(fb[now][j][1], fa[now][i][0], c);
          } else if constexpr (PA > 1) {
            if constexpr (PA == 3) c = mma<T>(fb[now][j][0], fa[now][i][2], c);
            c = mma<T>(fb[now][j][0], fa[now][i][1], c);
          }
          acc[i][j] = mma<T>(fb[now][j][0], fa[now][i][0], c);
        }
    }
  };

  Stager<OA, A_ROWS, A_COLS, NT, RA> sa;
  Stager<OB, B_ROWS, B_COLS, NT, RB> sb;
  for (int seg = 0; seg < p.segments; ++seg) {
    const int64_t ldb = seg ? p.b.ld1 : p.b.ld;
    sa.start(p.a, p.a.p0 + (seg ? p.k * (RA ? 2 : 1) : 0), p.a.ld, m0, kbeg);
    sb.start(p.b, seg ? p.b.p1 : p.b.p0, ldb, n0, kbeg);
    auto load = [&](uint16_t* to) {
#pragma unroll
      for (int pl = 0; pl < LA; ++pl) sa.load(pl * p.a.plane, to + pl * A_SIZE);
#pragma unroll
      for (int pl = 0; pl < LB; ++pl) sb.load(pl * p.b.plane, to + LA * A_SIZE + pl * B_SIZE);
      sa.next(p.a.ld);
      sb.next(ldb);
    };
    const int64_t steps = kbeg < kend ? (kend - kbeg) / BK : 0, left = kbeg < kend ? (kend - kbeg) % BK : 0;
    // Two buffers.  Three or four with as many steps in flight cost a second block on the compute unit or a
    // larger tile, and lose: 300k x 128 float32 forward 248 and 262 us against 196, 16384 x 2048 -> 8192 bf16
    // 1128 us with steps of 32 against 1054.
    if (steps > 0) load(lds);
    for (int64_t t = 0; t < steps; ++t) {
      loads_done();
      __syncthreads();             // step t is there, and everyone has read step t - 1
      if (t + 1 < steps) load(lds + ((t + 1) & 1) * BUF);
      multiply(lds + (t & 1) * BUF);
    }
    __syncthreads();
    if (left > 0) {
#pragma unroll
      for (int pl = 0; pl < LA; ++pl) sa.load_partial(pl * p.a.plane, left, lds + pl * A_SIZE);
#pragma unroll
      for (int pl = 0; pl < LB; ++pl) sb.load_partial(pl * p.b.plane, left, lds + LA * A_SIZE + pl * B_SIZE);
      __syncthreads();
      multiply(lds);
      __syncthreads();
    }
  }

  // Element r of lane l is row l % 32, column 8 (r / 4) + 4 (l / 32) + r % 4 of its 32x32 block.  A
  // wavefront's 32 rows pass through a piece of LDS of its own (the loop's last barrier has freed it), so that a
  // row leaves in 16-byte stores of neighbouring lanes.
  constexpr int CW = OUT == OUT_GATED ? WN / 2 : WN;
  const int64_t row0 = m0 + wm * WM;
  const int64_t col0 = n0 + wn * CW;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t r0 = row0 + i * 32;
    if (r0 >= p.m) break;
    if constexpr (OUT != OUT_GATED && std::is_same<T, _Float16>::value) {
      if (p.sizes) {
        const int64_t row = r0 + (lane & 31);
        const float undo = power_of_two(-scale_of(p.sizes[row < p.m ? row : p.m - 1]));
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] *= undo;
      }
    }
    if constexpr (OUT == OUT_GATED) {
      RowWriter<O, CW> out(lds, wave, lane);
      auto put = [&](void* to, int64_t ld, auto value) {
#pragma unroll
        for (int j = 0; j < NI; j += 2)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = value(acc[i][j][4 * q + e], acc[i][j + 1][4 * q + e]);
            out.put(j * 16 + 8 * q, v);
          }
        out.flush(static_cast<O*>(to), ld, r0, p.m, col0, p.n);
      };
      put(p.h, p.ldh, [&](float g, float u) { return activate(g, p.act) * u; });
      if (p.gate) put(p.gate, p.ldg, [](float g, float) { return g; });
      if (p.up) put(p.up, p.ldu, [](float, float u) { return u; });
    } else if (OUT == OUT_DW || p.splits > 1) {
      RowWriter<float, CW> out(lds, wave, lane);
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
          out.put(j * 32 + 8 * q, v);
        }
      if (p.splits > 1) {
        out.flush(p.partial + sp * p.m * p.n, p.n, r0, p.m, col0, p.n);
      } else {
        // rows of dW_gate, then of dW_up
        out.flush(static_cast<float*>(p.c), p.ldc, r0, p.half, col0, p.n);
        out.flush(p.c1, p.ldc1, r0 - p.half, p.m - p.half, col0, p.n);
      }
    } else {
      RowWriter<O, CW> out(lds, wave, lane);
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
          out.put(j * 32 + 8 * q, v);
        }
      out.flush(static_cast<O*>(p.c), p.ldc, r0, p.m, col0, p.n);
    }
  }
}

// dA, or dWg and dWu (the rows below and from `half` on), from the splits' partials, added in order in float64.
template <typename O>
__global__ __launch_bounds__(256) void sum_splits_kernel(ProductArgs p, int64_t n4) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.m * n4) return;
  const int64_t row = i / n4, col = i % n4 * 4;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int k = 0; k < p.splits; ++k) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p.partial + (k * p.m + row) * p.n + col);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += static_cast<double>(v[e]);
  }
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = static_cast<float>(s[e]);
  if (row < p.half) store4<O>(static_cast<O*>(p.c) + row * p.ldc + col, r);
  else store4<float>(p.c1 + (row - p.half) * p.ldc1 + col, r);
}

// Planes [3][rows_out][cols_out] of the parts of a float32 matrix, zero where it ends.
__global__ __launch_bounds__(256) void split_kernel(const float* x, int64_t ld, int64_t rows, int64_t cols, __bf16* out,
                                                    int64_t rows_out, int64_t cols_out, int64_t plane) {
  const int64_t per = cols_out / 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < rows_out * per;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / per, c = i % per * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r < rows && c < cols) v = *reinterpret_cast<const f32x4*>(x + r * ld + c);
    bf16x4 h, m, l;
    split3(v, h, m, l);
    __bf16* o = out + r * cols_out + c;
    *reinterpret_cast<bf16x4*>(o) = h;
    *reinterpret_cast<bf16x4*>(o + plane) = m;
    *reinterpret_cast<bf16x4*>(o + 2 * plane) = l;
  }
}

// dG and dU of four values.
__device__ __forceinline__ void gate_terms(f32x4 dh, f32x4 g, f32x4 u, int32_t act, f32x4& dg, f32x4& du) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float slope;
    const float f = activate_both(g[e], act, &slope);
    dg[e] = dh[e] * u[e] * slope;
    du[e] = dh[e] * f;
  }
}

template <typename T>
__device__ __forceinline__ void gate_terms_at(const GatedArgs& p, int64_t r, int64_t c, f32x4& dg, f32x4& du) {
  typedef T vec __attribute__((ext_vector_type(4)));
  const f32x4 dh = __builtin_convertvector(*reinterpret_cast<const vec*>(static_cast<const T*>(p.dh) + r * p.lddh + c), f32x4);
  const f32x4 g = __builtin_convertvector(*reinterpret_cast<const vec*>(static_cast<const T*>(p.gate) + r * p.ldg + c), f32x4);
  const f32x4 u = __builtin_convertvector(*reinterpret_cast<const vec*>(static_cast<const T*>(p.up) + r * p.ldu + c), f32x4);
  gate_terms(dh, g, u, p.act, dg, du);
}

// [dG dU], 2n columns wide, as the products' operand: float32 values, or their three parts of bf16 in as many
// planes.  dA is stored in bf16 and takes the first part alone (one rounding of each term, as its own result has); dW is
// float32 and takes all three, which are the value exactly (two leave 2^-17 of a term: 2.6e-6 of dW at 8191 rows where
// float32 operands leave 1.6e-6).
template <typename T>
__global__ __launch_bounds__(256) void gate_grad_kernel(GatedArgs p, T* out) {
  typedef T vec __attribute__((ext_vector_type(4)));
  const int64_t per = p.n / 4, plane = p.m * 2 * p.n;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < p.m * per;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / per, c = i % per * 4;
    f32x4 d[2];
    gate_terms_at<T>(p, r, c, d[0], d[1]);
    T* o = out + r * 2 * p.n + c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<vec*>(o + h * p.n) = d[h];
      } else {
        vec first, second, third;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // finite values beyond bf16's largest start with it; an infinity is whole in its first part
          constexpr float top = 0x1.FEp127f;
          const float x = d[h][e], y = __builtin_isfinite(x) ? fminf(fmaxf(x, -top), top) : x;
          first[e] = static_cast<T>(y);
          const float rest = __builtin_isinf(x) ? 0.0f : x - static_cast<float>(first[e]);
          second[e] = static_cast<T>(rest);
          third[e] = static_cast<T>(rest - static_cast<float>(second[e]));
        }
        *reinterpret_cast<vec*>(o + h * p.n) = first;
        *reinterpret_cast<vec*>(o + h * p.n + plane) = second;
        *reinterpret_cast<vec*>(o + h * p.n + 2 * plane) = third;
      }
    }
  }
}

// f16: [dG dU] in three planes: two parts of its values scaled by columns for dW, which leave 2^-22 of a term or 2^-39 of its
// column's largest, and one rounding of its values scaled by rows for dA (2^-11 of a term or 2^-39 of its row's largest).
// Two launches in the same tiles of 4 `lanes` columns (a power of two of lanes) and rows_each rows: the first leaves
// each tile's largest finite magnitudes by row and column, the second adds them up, at most 256 of either, as it begins.
// A thread has four rows' loads in flight.  8191 x 4096, SiLU: 49 us (4.1 TB/s) and 121 us (5.0 TB/s).
constexpr int kGradThreads = 1024;
constexpr int64_t kGradTiles = 256;      // a block each: one for each compute unit

struct GradTiles {
  int32_t lanes, col_blocks, row_blocks;
  int64_t rows_each;
  uint32_t* by_row;        // [m], the final ones
  uint32_t* by_col;        // [2n]
  uint32_t* row_part;      // [col_blocks][m]
  uint32_t* col_part;      // [row_blocks][2n]
};

__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0;
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest of each x among a thread's `lanes` neighbours.
__device__ __forceinline__ void team_max(uint32_t (&x)[4], int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = larger(x[q], __shfl_xor(x[q], o, 64));
}

struct GradPlace {
  int tx, ty, rows_par;
  int64_t c, begin, end;
  __device__ __forceinline__ GradPlace(const GradTiles& t, int64_t m) {
    tx = static_cast<int>(threadIdx.x) % t.lanes;
    ty = static_cast<int>(threadIdx.x) / t.lanes;
    rows_par = kGradThreads / t.lanes;
    c = (static_cast<int64_t>(blockIdx.x) % t.col_blocks * t.lanes + tx) * 4;
    begin = static_cast<int64_t>(blockIdx.x) / t.col_blocks * t.rows_each;
    end = begin + t.rows_each < m ? begin + t.rows_each : m;
  }
};

// dG and dU of four columns from c on, of row r and the three rows `step` apart that follow it below `end`; zeros past it and past
// the last column.
__device__ __forceinline__ void gate_terms_of_rows(const GatedArgs& p, int64_t r, int64_t step, int64_t end, int64_t c,
                                                   f32x4 (&dg)[4], f32x4 (&du)[4]) {
  f16x4 dh[4], g[4], u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t row = r + q * step;
    if (row < end && c < p.n) {
      dh[q] = *reinterpret_cast<const f16x4*>(static_cast<const _Float16*>(p.dh) + row * p.lddh + c);
      g[q] = *reinterpret_cast<const f16x4*>(static_cast<const _Float16*>(p.gate) + row * p.ldg + c);
      u[q] = *reinterpret_cast<const f16x4*>(static_cast<const _Float16*>(p.up) + row * p.ldu + c);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    dg[q] = du[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (r + q * step < end && c < p.n)
      gate_terms(__builtin_convertvector(dh[q], f32x4), __builtin_convertvector(g[q], f32x4),
                 __builtin_convertvector(u[q], f32x4), p.act, dg[q], du[q]);
  }
}

__global__ __launch_bounds__(kGradThreads) void grad_sizes_kernel(GatedArgs p, GradTiles t) {
  __shared__ uint32_t top[8][kGradThreads];
  const GradPlace at(t, p.m);
  uint32_t col[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t r = at.begin + at.ty; r < at.end; r += 4 * at.rows_par) {      // the same rows for a whole team of lanes
    f32x4 dg[4], du[4];
    gate_terms_of_rows(p, r, at.rows_par, at.end, at.c, dg, du);
    uint32_t row[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = finite_bits(dg[q][e]), b = finite_bits(du[q][e]);
        col[e] = larger(col[e], a);
        col[4 + e] = larger(col[4 + e], b);
        row[q] = larger(row[q], larger(a, b));
      }
    if (!p.da) continue;
    team_max(row, t.lanes);
    if (at.tx == 0)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t to = r + q * at.rows_par;
        if (to < at.end) t.row_part[static_cast<int64_t>(blockIdx.x) % t.col_blocks * p.m + to] = row[q];
      }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) top[e][threadIdx.x] = col[e];
  __syncthreads();
  for (int i = threadIdx.x; i < t.lanes * 8; i += kGradThreads) {
    const int x = i / 8, e = i % 8;
    uint32_t most = 0;
#pragma unroll 8
    for (int y = 0; y < at.rows_par; ++y) most = larger(most, top[e][y * t.lanes + x]);
    const int64_t c = (static_cast<int64_t>(blockIdx.x) % t.col_blocks * t.lanes + x) * 4 + (e & 3);
    if (c < p.n) t.col_part[static_cast<int64_t>(blockIdx.x) / t.col_blocks * 2 * p.n + (e < 4 ? c : p.n + c)] = most;
  }
}

__global__ __launch_bounds__(kGradThreads) void gate_grad_f16_kernel(GatedArgs p, GradTiles t, _Float16* out) {
  __shared__ uint32_t size_of[512];                  // the tile's columns of dG, then of dU
  const GradPlace at(t, p.m);
  const int64_t plane = p.m * 2 * p.n;
  const int width = 4 * t.lanes, shares = kGradThreads / (2 * width);
  if (static_cast<int>(threadIdx.x) < 2 * width) size_of[threadIdx.x] = 0;
  __syncthreads();
  {
    const int i = static_cast<int>(threadIdx.x) % (2 * width);
    const int64_t c = static_cast<int64_t>(blockIdx.x) % t.col_blocks * width + i % width, col = i < width ? c : p.n + c;
    uint32_t most = 0;
    if (c < p.n) {
#pragma unroll 16
      for (int b = static_cast<int>(threadIdx.x) / (2 * width); b < t.row_blocks; b += shares)
        most = larger(most, t.col_part[static_cast<int64_t>(b) * 2 * p.n + col]);
    }
    atomicMax(size_of + i, most);
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < 2 * width && c < p.n && static_cast<int64_t>(blockIdx.x) < t.col_blocks)
      t.by_col[col] = size_of[i];
  }
  f32x4 by_col[2];
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int h = 0; h < 2; ++h) by_col[h][e] = power_of_two(scale_of(size_of[h * width + at.tx * 4 + e]));
  for (int64_t r = at.begin + at.ty; r < at.end; r += 4 * at.rows_par) {
    uint32_t size[4] = {0, 0, 0, 0};
    if (p.da) {
      for (int b = at.tx; b < t.col_blocks; b += t.lanes)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t row = r + q * at.rows_par;
          if (row < at.end) size[q] = larger(size[q], t.row_part[static_cast<int64_t>(b) * p.m + row]);
        }
      team_max(size, t.lanes);
    }
    f32x4 d[2][4];
    gate_terms_of_rows(p, r, at.rows_par, at.end, at.c, d[0], d[1]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t row = r + q * at.rows_par;
      if (row >= at.end) break;
      const float by_row = power_of_two(scale_of(size[q]));
      if (p.da && at.c == 0) t.by_row[row] = size[q];
      if (at.c >= p.n) continue;
      _Float16* o = out + row * 2 * p.n + at.c;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 x = d[h][q] * by_col[h];
        f16x4 second;
        const f16x4 first = __builtin_convertvector(x, f16x4);
#pragma unroll
        for (int e = 0; e < 4; ++e)        // an infinity is whole in its first part
          second[e] = static_cast<_Float16>(finite_bits(x[e]) ? x[e] - static_cast<float>(first[e]) : 0.0f);
        *reinterpret_cast<f16x4*>(o + h * p.n) = first;
        *reinterpret_cast<f16x4*>(o + h * p.n + plane) = second;
        if (p.da) store4<_Float16>(o + h * p.n + 2 * plane, d[h][q] * by_row);
      }
    }
  }
}

// Few rows (decoded tokens, queried nodes): the weights are read once at memory's rate and the tiles above
// would leave most of the chip idle.  A block owns 16 columns of H and all rows (16 MB of them); its eight
// wavefronts take every eighth 32-step piece of the reduction, read their 16 rows of Wg and Wu straight from
// memory as matrix operands (16 bytes a lane, four pieces in flight), and meet in LDS.  One row, 2048 -> 4096 bf16:
// 7.3 us, 4.6 TB/s of weights.
template <typename T, int MB>
__global__ __launch_bounds__(512) void few_rows_kernel(GatedArgs p) {
  constexpr bool F32 = sizeof(T) == 4;
  typedef typename std::conditional<F32, __bf16, T>::type P;       // the matrix cores' type
  constexpr int PL = F32 ? 3 : 1;
  __shared__ f32x4 sums[8][2][MB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 16;
  int64_t wrow = c0 + (lane & 15);
  wrow = wrow < p.n ? wrow : p.n - 1;                 // repeats the last row; its columns are not stored
  const int64_t kq = (lane >> 4) * 8;
  const T* gp = static_cast<const T*>(p.wg) + wrow * p.ldwg;
  const T* up = static_cast<const T*>(p.wu) + wrow * p.ldwu;
  const T* ap[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    int64_t r = b * 16 + (lane & 15);
    r = r < p.m ? r : p.m - 1;
    ap[b] = static_cast<const T*>(p.a) + r * p.lda;
  }
  f32x4 acc[2][MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[0][b] = acc[1][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  struct Piece {
    u32x4 w[F32 ? 2 : 1];
  };
  auto read = [&](const T* x, int64_t k) {
    Piece r;
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h) {
      r.w[h] = u32x4{0, 0, 0, 0};
      if (k + 4 * h < p.k) r.w[h] = *reinterpret_cast<const u32x4*>(x + k + 4 * h);
    }
    return r;
  };
  struct Parts {
    s16x8 p[PL];
  };
  auto parts = [&](const Piece& x) {
    Parts r;
    if constexpr (F32) {
      split8(__builtin_bit_cast(f32x4, x.w[0]), __builtin_bit_cast(f32x4, x.w[1]), r.p);
    } else {
      r.p[0] = __builtin_bit_cast(s16x8, x.w[0]);
    }
    return r;
  };
  auto madd = [&](const Parts& w, const Parts& a, f32x4 c) {
    if constexpr (F32) {
      c = mma16<P>(w.p[1], a.p[1], c);
      c = mma16<P>(w.p[0], a.p[2], c);
      c = mma16<P>(w.p[2], a.p[0], c);
      c = mma16<P>(w.p[0], a.p[1], c);
      c = mma16<P>(w.p[1], a.p[0], c);
    }
    return mma16<P>(w.p[0], a.p[0], c);
  };
  constexpr int AHEAD = MB <= 2 ? 4 : F32 && MB == 8 ? 1 : 2;
  for (int64_t k0 = wave * 32; k0 < p.k; k0 += 256 * AHEAD) {
    Piece g[AHEAD], u[AHEAD], a[AHEAD][MB];
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) {
      const int64_t k = k0 + 256 * t + kq;            // past the reduction's end everything reads as zero
      g[t] = read(gp, k);
      u[t] = read(up, k);
#pragma unroll
      for (int b = 0; b < MB; ++b) a[t][b] = read(ap[b], k);
    }
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) {
      const Parts wg = parts(g[t]), wu = parts(u[t]);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const Parts x = parts(a[t][b]);
        acc[0][b] = madd(wg, x, acc[0][b]);
        acc[1][b] = madd(wu, x, acc[1][b]);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    sums[wave][0][b][lane] = acc[0][b];
    sums[wave][1][b][lane] = acc[1][b];
  }
  __syncthreads();
  // element e of lane l is row l % 16, column 4 (l / 16) + e
  for (int i = threadIdx.x; i < MB * 64; i += 512) {
    const int b = i >> 6, l = i & 63;
    f32x4 g = sums[0][0][b][l], u = sums[0][1][b][l], h;
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      g += sums[w][0][b][l];
      u += sums[w][1][b][l];
    }
    const int64_t row = b * 16 + (l & 15), col = c0 + (l >> 4) * 4;
    if (row >= p.m || col >= p.n) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = activate(g[e], p.act) * u[e];
    store4<T>(static_cast<T*>(p.h) + row * p.ldh + col, h);
    if (p.gate_out) {
      store4<T>(static_cast<T*>(p.gate_out) + row * p.ldg + col, g);
      store4<T>(static_cast<T*>(p.up_out) + row * p.ldu + col, u);
    }
  }
}

uint32_t stride_blocks(int64_t items) {
  const int64_t b = (items + 255) / 256;
  return static_cast<uint32_t>(b < 16384 ? (b > 0 ? b : 1) : 16384);
}

int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }

template <typename T, typename O, int PA, int PB, bool RA, bool RB, int OA, int OB, int OUT, int BM, int BN, int BK, int WM, int WN>
hipError_t run_product(ProductArgs p, hipStream_t s) {
  p.m_tiles = static_cast<int32_t>((p.m + BM - 1) / BM);
  const int64_t wide = OUT == OUT_GATED ? BN / 2 : BN;
  p.n_tiles = static_cast<int32_t>((p.n + wide - 1) / wide);
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles * p.splits;
  const int64_t blocks = (tiles + kXcds - 1) / kXcds * kXcds;
  product_kernel<T, O, PA, PB, RA, RB, OA, OB, OUT, BM, BN, BK, WM, WN>
      <<<static_cast<uint32_t>(blocks), (BM / WM) * (BN / WN) * 64, 0, s>>>(p);
  return hipGetLastError();
}

constexpr int64_t kUnits = 256;          // compute units; a block with a large tile fills one

int64_t tiles_of(int64_t m, int64_t n, int64_t bm, int64_t bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); }

// Tile shapes, with medians of a kernel trace of both sides on one card.  Larger tiles read LDS less per product and need
// enough of them to occupy the compute units: forward of 16384 x 2048 -> 8192 bf16, 1044 us in 256 x 256 tiles (4096 of
// them) against 1225 us in 128 x 128; dA of 8191 x 8192 -> 1024, 206 us in 256 x 256 (128 tiles, half the chip) against
// 172 us in 128 x 128; its dW of two parts (f16) 261 us in 256 x 128 against 343 us, of three (bf16) 358 us in 128 x 128
// with steps of 32, two blocks to a compute unit, against 361 us in 256 x 128 and 455 us with steps of 64.
// Three-part products in 128 x 128, two blocks to a compute unit: forward, where one multiplies while the other stores,
// of 300k x 128 -> 128 148 against 168 us in 128 x 256, 20k x 384 -> 512 92 against 107 us.  dA and dW in tiles twice as
// large, one to a compute unit, where those make one round of blocks: of 4000 x 2048 -> 4096 652 and 758 us against 676
// and 773 us; 20k x 384 -> 512 would take two rounds of 314 and 336 blocks, 159 and 188 us against 93 and 107 us,
// and dA of 100k x 512 -> 512 seven, 584 against 549 us.  Where even tiles of 128 x 128 leave half the compute units idle, 64 x 64: forward of
// 512 x 1024 -> 2048 (128 tiles) bf16 12.2 against 15.4 us, float32 40 against 46 us; of 1500 x 1136 -> 1224
// (240 tiles) 21.1 against 18.9 us.
template <typename T, typename O, int PA, int PB, bool RA, bool RB, int OA, int OB, int OUT>
hipError_t product(const ProductArgs& p, hipStream_t s) {
  const int64_t n = OUT == OUT_GATED ? 2 * p.n : p.n;       // rows of the B operand
  [[maybe_unused]] const bool few = tiles_of(p.m, n, 128, 128) * p.splits <= kUnits / 2;
  if constexpr (PA == 1) {
    if (tiles_of(p.m, n, 256, 256) * p.splits >= 2 * kUnits) return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 256, 256, 64, 128, 64>(p, s);
    if (few) return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 64, 64, 64, 32, 64>(p, s);
    return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 128, 128, 64, 64, 64>(p, s);
  } else if constexpr (PA == 2) {
    if (p.m > 128 && tiles_of(p.m, n, 256, 128) * p.splits > kUnits / 2) return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 256, 128, 64, 64, 64>(p, s);
    return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 128, 128, 64, 64, 64>(p, s);
  } else if constexpr (PB == 1) {
    return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 128, 128, 32, 64, 64>(p, s);
  } else {
    if constexpr (OUT != OUT_GATED) {
      auto one_round = [&](int64_t bm, int64_t bn) {
        const int64_t blocks = tiles_of(p.m, n, bm, bn) * p.splits;
        return blocks > kUnits / 2 && blocks <= kUnits;
      };
      if (n > 128 && one_round(128, 256)) return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 128, 256, 32, 64, 64>(p, s);
      if (p.m > 128 && one_round(256, 128)) return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 256, 128, 32, 64, 64>(p, s);
    }
    if constexpr (OUT != OUT_DW) {
      if (few) return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 64, 64, 32, 32, 64>(p, s);
    }
    return run_product<T, O, PA, PB, RA, RB, OA, OB, OUT, 128, 128, 32, 64, 64>(p, s);
  }
}

Operand plain(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t plane = 0) {
  return {static_cast<const uint16_t*>(p), nullptr, ld, ld, plane, rows, cols};
}

constexpr int64_t kSplitStep = 64;       // a split's steps are a multiple of it

// Splits of dW's reduction over the rows: as many as keep the 256 x 128 tiles on the compute units at once (a few more
// would take a second round), each of at least 256 rows.
int32_t dw_splits(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = tiles_of(2 * n, k, 256, 128);
  int64_t s = kUnits / tiles;
  const int64_t most = (m + 255) / 256;
  s = s < most ? s : most;
  return static_cast<int32_t>(s < 1 ? 1 : s);
}

// Splits of dA's reduction over the gate's (and the up's) columns where its tiles are few.
int32_t da_splits(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = tiles_of(m, k, 128, 128);
  int64_t s = kUnits / (tiles > 0 ? tiles : 1);
  const int64_t most = (n + 255) / 256;
  s = s < most ? s : most;
  return static_cast<int32_t>(s < 1 ? 1 : s);
}

// Rows that few_rows_kernel takes.  Each of its n / 16 blocks reads all rows, padded to 16, 32, 64 or 128, so its time grows with
// both; the tiles' does not below 128 rows.  16-bit, few rows against tiles in us: 1 row of 2048 -> 4096 10.8 and 18.3,
// 16 rows of 4096 -> 8192 28.1 and 34.7, 32 rows 33.5 and 34.9, 64 rows of 2048 -> 4096 14.9 and 19.2, of 4096 -> 8192 47.5
// and 35.3, 128 rows of 1024 -> 2048 13.7 and 11.3.  float32, whose tiles split the weights first: 128 rows of
// 4096 -> 8192 167 and 276.
bool few_rows(int32_t type, int64_t m, int64_t n) {
  if (m <= 16) return true;
  if (type == QHA_F32) return m <= 128 && n < 16384;
  return m <= 64 && (m <= 32 ? 32 : 64) * n <= 1 << 18;
}

struct Space {
  int64_t w, grad, sizes, partial;        // bytes
};

int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }

// Tiles of the f16 gradients' two launches: up to 256 columns wide, and as many rows of tiles as make kGradTiles of them,
// with a row a thread at least.  Their sizes lie at `at`.
GradTiles grad_tiles(int64_t m, int64_t n, char* at) {
  GradTiles t = {};
  t.lanes = 1;
  while (t.lanes < 64 && t.lanes * 4 < n) t.lanes *= 2;
  t.col_blocks = static_cast<int32_t>((n + 4 * t.lanes - 1) / (4 * t.lanes));
  const int64_t rows_par = kGradThreads / t.lanes, most = (m + rows_par - 1) / rows_par;
  int64_t blocks = kGradTiles / t.col_blocks;
  blocks = blocks < most ? blocks : most;
  blocks = blocks > 0 ? blocks : 1;
  t.rows_each = (m + blocks - 1) / blocks;
  t.row_blocks = t.rows_each > 0 ? static_cast<int32_t>((m + t.rows_each - 1) / t.rows_each) : 0;
  t.by_row = reinterpret_cast<uint32_t*>(at);
  t.by_col = t.by_row + m;
  t.row_part = t.by_col + 2 * n;
  t.col_part = t.row_part + t.col_blocks * m;
  return t;
}

int64_t grad_tiles_space(int64_t m, int64_t n) {
  const GradTiles t = grad_tiles(m, n, nullptr);
  return up16(((1 + t.col_blocks) * m + (1 + t.row_blocks) * 2 * n) * 4);
}

Space gated_space(int32_t type, int64_t m, int64_t n, int64_t k, bool backward) {
  Space s = {0, 0, 0, 0};
  if (type == QHA_F32 && (backward || !few_rows(type, m, n))) s.w = up16(3 * 2 * up8(n) * up8(k) * 2);
  if (backward) {
    s.grad = up16(m * 2 * n * (type == QHA_F32 ? 4 : 6));      // float32, or three planes of 16 bits
    if (type == QHA_F16) s.sizes = grad_tiles_space(m, n);
    const int64_t splits = dw_splits(m, n, k);
    s.partial = splits > 1 ? up16(splits * 2 * n * k * 4) : 0;
    // dA's partials are read before dW writes its own to the same place
    const int64_t da = da_splits(m, n, k);
    const int64_t need = da > 1 ? up16(da * m * k * 4) : 0;
    s.partial = s.partial > need ? s.partial : need;
  }
  return s;
}

int64_t split_each(int64_t k, int32_t splits) { return ((k + splits - 1) / splits + kSplitStep - 1) / kSplitStep * kSplitStep; }

template <typename O>
hipError_t sum_splits(const ProductArgs& p, hipStream_t s) {
  const int64_t n4 = p.n / 4;
  sum_splits_kernel<O><<<static_cast<uint32_t>((p.m * n4 + 255) / 256), 256, 0, s>>>(p, n4);
  return hipGetLastError();
}

template <typename T>
hipError_t fwd_few(const GatedArgs& g, hipStream_t s) {
  const uint32_t blocks = static_cast<uint32_t>((g.n + 15) / 16);
  if (g.m <= 16) few_rows_kernel<T, 1><<<blocks, 512, 0, s>>>(g);
  else if (g.m <= 32) few_rows_kernel<T, 2><<<blocks, 512, 0, s>>>(g);
  else if (g.m <= 64) few_rows_kernel<T, 4><<<blocks, 512, 0, s>>>(g);
  else if constexpr (sizeof(T) == 4) few_rows_kernel<T, 8><<<blocks, 512, 0, s>>>(g);
  return hipGetLastError();
}

// The float32 weights in three bf16 planes [n8 rows of W_gate, n8 rows of W_up][k8], zero past n and k.
Operand weight_planes(const GatedArgs& g, void* ws, hipStream_t s) {
  const int64_t n8 = up8(g.n), k8 = up8(g.k), plane = 2 * n8 * k8;
  __bf16* w = static_cast<__bf16*>(ws);
  const uint32_t blocks = stride_blocks(n8 * k8 / 4);
  split_kernel<<<blocks, 256, 0, s>>>(static_cast<const float*>(g.wg), g.ldwg, g.n, g.k, w, n8, k8, plane);
  split_kernel<<<blocks, 256, 0, s>>>(static_cast<const float*>(g.wu), g.ldwu, g.n, g.k, w + n8 * k8, n8, k8, plane);
  return {reinterpret_cast<const uint16_t*>(w), reinterpret_cast<const uint16_t*>(w + n8 * k8), k8, k8, plane, n8, k8};
}

Operand weights16(const GatedArgs& g) {
  return {static_cast<const uint16_t*>(g.wg), static_cast<const uint16_t*>(g.wu), g.ldwg, g.ldwu, 0, g.n, g.k};
}

template <typename T, typename O, int PL>
hipError_t fwd(const GatedArgs& g, hipStream_t s) {
  ProductArgs p = {};
  p.a = plain(g.a, g.lda, g.m, g.k);
  p.b = PL == 3 ? weight_planes(g, g.ws, s) : weights16(g);
  p.m = g.m;
  p.n = g.n;
  p.k = p.k_each = g.k;
  p.splits = p.segments = 1;
  p.h = g.h;
  p.gate = g.gate_out;
  p.up = g.up_out;
  p.ldh = g.ldh;
  p.ldg = g.ldg;
  p.ldu = g.ldu;
  p.act = g.act;
  return product<T, O, PL, PL, PL == 3, false, ORDER_ROWS, ORDER_PAIRS, OUT_GATED>(p, s);
}

template <typename T, typename O, int PL>
hipError_t bwd(const GatedArgs& g, hipStream_t s) {
  const Space sp = gated_space(g.type, g.m, g.n, g.k, true);
  char* ws = static_cast<char*>(g.ws);
  O* grad = reinterpret_cast<O*>(ws + sp.w);
  float* partial = reinterpret_cast<float*>(ws + sp.w + sp.grad + sp.sizes);
  hipError_t e = hipSuccess;
  const int64_t plane = g.m * 2 * g.n;
  const Operand d = plain(grad, 2 * g.n, g.m, 2 * g.n, plane);
  Operand da_operand = d;
  const uint32_t *by_row = nullptr, *by_col = nullptr;
  if constexpr (std::is_same<T, _Float16>::value) {
    if (g.m > 0) {
      const GradTiles t = grad_tiles(g.m, g.n, ws + sp.w + sp.grad);
      grad_sizes_kernel<<<t.col_blocks * t.row_blocks, kGradThreads, 0, s>>>(g, t);
      gate_grad_f16_kernel<<<t.col_blocks * t.row_blocks, kGradThreads, 0, s>>>(g, t, grad);
      da_operand.p0 += 2 * plane;
      by_row = t.by_row;
      by_col = t.by_col;
    }
  } else {
    if (g.m > 0) gate_grad_kernel<O><<<stride_blocks(g.m * g.n / 4), 256, 0, s>>>(g, grad);
  }
  if (g.m > 0 && g.da) {
    ProductArgs p = {};
    p.a = da_operand;
    p.sizes = by_row;
    p.b = PL == 3 ? weight_planes(g, ws, s) : weights16(g);
    p.m = g.m;
    p.n = g.k;
    p.k = g.n;
    p.segments = 2;
    p.splits = da_splits(g.m, g.n, g.k);
    p.k_each = split_each(g.n, p.splits);
    p.half = g.m;
    p.c = g.da;
    p.ldc = g.ldda;
    p.partial = partial;
    e = product<T, O, PL, PL, PL == 3, false, ORDER_ROWS, ORDER_CROSS, OUT_DA>(p, s);
    if (e == hipSuccess && p.splits > 1) e = sum_splits<O>(p, s);
    if (e != hipSuccess) return e;
  }
  ProductArgs p = {};
  p.a = d;
  p.sizes = by_col;
  p.b = plain(g.a, g.lda, g.m, g.k);
  p.m = 2 * g.n;
  p.n = g.k;
  p.k = g.m;
  p.segments = 1;
  p.splits = dw_splits(g.m, g.n, g.k);
  p.k_each = split_each(g.m, p.splits);
  p.half = g.n;
  p.c = g.dwg;
  p.ldc = g.lddwg;
  p.c1 = g.dwu;
  p.ldc1 = g.lddwu;
  p.partial = partial;
  constexpr int parts = std::is_same<T, _Float16>::value ? 2 : 3;
  e = product<T, float, parts, PL, PL == 3, PL == 3, ORDER_CROSS, ORDER_CROSS, OUT_DW>(p, s);
  if (e == hipSuccess && p.splits > 1) e = sum_splits<float>(p, s);
  return e;
}

}  // namespace

size_t gated_workspace(int32_t type, int64_t m, int64_t n, int64_t k, bool backward) {
  const Space s = gated_space(type, m, n, k, backward);
  return static_cast<size_t>(s.w + s.grad + s.sizes + s.partial);
}

hipError_t launch_gated_fwd(const GatedArgs& g, hipStream_t s) {
  if (few_rows(g.type, g.m, g.n)) return g.type == QHA_F32 ? fwd_few<float>(g, s) : g.type == QHA_BF16 ? fwd_few<__bf16>(g, s) : fwd_few<_Float16>(g, s);
  if (g.type == QHA_F32) return fwd<__bf16, float, 3>(g, s);
  return g.type == QHA_BF16 ? fwd<__bf16, __bf16, 1>(g, s) : fwd<_Float16, _Float16, 1>(g, s);
}

hipError_t launch_gated_bwd(const GatedArgs& g, hipStream_t s) {
  if (g.type == QHA_F32) return bwd<__bf16, float, 3>(g, s);
  return g.type == QHA_BF16 ? bwd<__bf16, __bf16, 1>(g, s) : bwd<_Float16, _Float16, 1>(g, s);
}

}  // namespace qha
