// The norms around a block fused with its gate and the residual stream, and their gradients.
//
// Mathematics, per row: z = w_p hhat + b_p with hhat = (h - mean) rstd (layer norm), h rstd (RMS) or h;
//   x' = skip x + branch g z,   u = w_q xhat' + b_q with xhat' the same of x' (in float32, before it is rounded).
// Backward, with q = w_q du and t = dy + rstd (q - mean q - xhat' mean(q xhat')) (no mean q for RMS):
//   dx = skip t (the host sets skip to 1 where there is no block),  dg = sum of branch t z over the rows that share g,  dh the same form of q = w_p branch t g,
//   dw = sum dz xhat and db = sum dz over all rows, for both norms.
//
// Bound: memory, every array once.  A row belongs to a team of L threads (8 to a wavefront's 64, or a block of 256 or
// 512) that keeps it in registers, R vectors a thread (16 bytes of the branch's type), so that the statistics of both
// norms and both outputs come from one read; a thread's places, its weights and its share of the weights' gradients stay with
// it over many rows.  Sums over a row are float32 (at most 8192 values, means before squares).  Gradients of weights are
// float32 in a block, which leaves one partial; those of a shared gate one partial for each piece of a sample's rows; a second launch
// adds partials in float64 in a fixed order (a block by itself needs none).  A team loads its next row before it works on the
// present one, in the row's own type, and outputs are stored past the caches.
//
// Measured (kernel alone, in a loop over the same inputs): forward, 300k x 128 float32, both layer norms, 104 to 120 us (619 MB, 5.1 to 5.9 TB/s;
// a large copy here reaches 4.7); 16384 x 2048 bf16 on a float32 stream, four gates, 68 us (a call on new inputs 80, 5.0 TB/s); one row of
// 4096 3.4 us (8.5 a call: host).  Backward, 300001 x 256 float32 326 us and 6 for the partials (5.6 TB/s); 8191 x 2048 bf16, a gate a row,
// 46 and 5 (269 MB, 5.2 TB/s; a call on new inputs 58).
#include "act_common.hpp"
#include "qha_internal.hpp"

namespace qha {
namespace {

// Rows as V values a vector, whatever their type; loads ahead of their use stay in that type (half the registers).
template <typename E, int V>
struct Row {
  typedef E vec __attribute__((ext_vector_type(V), aligned(16)));
  typedef float wide __attribute__((ext_vector_type(V)));
  static __device__ __forceinline__ vec raw(const void* p, int64_t at) { return *reinterpret_cast<const vec*>(static_cast<const E*>(p) + at); }
  static __device__ __forceinline__ wide value(vec x) { return __builtin_convertvector(x, wide); }
  static __device__ __forceinline__ void store(void* p, int64_t at, wide x) {
    __builtin_nontemporal_store(__builtin_convertvector(x, vec), reinterpret_cast<vec*>(static_cast<E*>(p) + at));
  }
};

// The sum over W neighbouring lanes, in each of them: pairs, quads, halves and rows of 16 by the data paths of the vector
// unit, then the two swaps of rows and halves.
template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int W>
__device__ __forceinline__ float lanes_sum(float x) {
  static_assert(W >= 8 && W <= 64, "teams");
  x += moved<0xB1>(x);               // lanes 1 0 3 2
  x += moved<0x4E>(x);               // 2 3 0 1
  x += moved<0x141>(x);              // 7 .. 0
  if constexpr (W >= 16) x += moved<0x140>(x);      // 15 .. 0
  if constexpr (W >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (W >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return x;
}

template <int L>
constexpr int threads_of() { return L < 256 ? 256 : L; }

// Sums over the team; every thread gets them.  Blocks alternate between two LDS buffers, so that one barrier a sum is enough: a
// buffer is written again only after the barrier of the sum between.
template <int L, int N>
struct TeamSum {
  static constexpr int W = L < 64 ? L : 64;
  float (*lds)[8][N];
  int parity = 0;
  __device__ __forceinline__ void operator()(float (&s)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = lanes_sum<W>(s[i]);
    if constexpr (L > 64) {
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) lds[parity][threadIdx.x >> 6][i] = s[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < L / 64; ++k) s[i] += lds[parity][k][i];
      }
      parity ^= 1;
    }
  }
};

// Thread's places in a row.
template <int L, int R, int V>
struct Place {
  int col[R];
  bool in[R];
  __device__ __forceinline__ explicit Place(int c) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      col[r] = (static_cast<int>(threadIdx.x) % L + r * L) * V;
      in[r] = col[r] < c;
    }
  }
  typedef float wide __attribute__((ext_vector_type(V)));
  __device__ __forceinline__ wide weight(const float* w, float other, int r) const {
    wide x = other;
    if (w && in[r]) x = Row<float, V>::value(Row<float, V>::raw(w, col[r]));
    return x;
  }
  __device__ __forceinline__ void weights(const float* w, float other, wide (&to)[R]) const {
#pragma unroll
    for (int r = 0; r < R; ++r) to[r] = weight(w, other, r);
  }
};

template <typename S, typename T, int L, int R>
__global__ __launch_bounds__(threads_of<L>()) void residual_fwd_kernel(ResidualArgs a) {
  constexpr int V = 16 / sizeof(T);
  constexpr int TEAMS = threads_of<L>() / L;
  typedef float wide __attribute__((ext_vector_type(V)));
  __shared__ float lds[2][8][1];
  TeamSum<L, 1> team_sum{lds};
  const Place<L, R, V> at(a.c);
  const float n = static_cast<float>(a.c), eps = a.eps;
  wide pw[R], pb[R], qw[R], qb[R];
  at.weights(a.post_w, 1.0f, pw);
  at.weights(a.post_b, 0.0f, pb);
  at.weights(a.pre_w, 1.0f, qw);
  at.weights(a.pre_b, 0.0f, qb);
  const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
  typename Row<S, V>::vec next_x[R];
  typename Row<T, V>::vec next_h[R], next_g[R];
  auto fetch = [&](int64_t row) {
    const int64_t sample = a.positions == 1 ? row : static_cast<uint32_t>(row) / static_cast<uint32_t>(a.positions);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      next_x[r] = static_cast<S>(0.0f);
      next_h[r] = static_cast<T>(0.0f);
      next_g[r] = static_cast<T>(1.0f);
      if (row < a.rows && at.in[r]) {
        next_x[r] = Row<S, V>::raw(a.x, row * a.ldx + at.col[r]);
        if (a.h) next_h[r] = Row<T, V>::raw(a.h, row * a.ldh + at.col[r]);
        if (a.gate) next_g[r] = Row<T, V>::raw(a.gate, sample * a.ldg + at.col[r]);
      }
    }
  };
  // the norm's statistics of a row held as v[R]
  auto row_stats = [&](const wide (&v)[R], int kind, float* mean, float* rstd) {
    float s[1] = {0.0f};
    *mean = 0.0f;
    if (kind == QHA_ROW_LAYER) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += v[r][i];       // zeros past the row's end
      team_sum(s);
      *mean = s[0] / n;              // a quotient: rows of equal values have exactly that mean
    }
    s[0] = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = v[r][i] - *mean;
        s[0] += at.in[r] ? d * d : 0.0f;
      }
    team_sum(s);
    *rstd = 1.0f / sqrtf(s[0] / n + eps);
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / L;
  fetch(row);
  for (; row < a.rows; row += step) {
    wide x[R], z[R], g[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = Row<S, V>::value(next_x[r]);
      z[r] = Row<T, V>::value(next_h[r]);
      g[r] = Row<T, V>::value(next_g[r]);
    }
    fetch(row + step);
    if (a.h) {
      float mean = 0.0f, rstd = 1.0f;
      if (a.post != QHA_ROW_NONE) {
        row_stats(z, a.post, &mean, &rstd);
        if (a.post_stats && threadIdx.x % L == 0) *reinterpret_cast<float2*>(a.post_stats + 2 * row) = make_float2(mean, rstd);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[r] = a.skip * x[r] + a.branch * (g[r] * ((z[r] - mean) * rstd * pw[r] + pb[r]));
        if (!at.in[r]) x[r] = 0.0f;
        else Row<S, V>::store(a.y, row * a.ldy + at.col[r], x[r]);
      }
    }
    if (a.pre != QHA_ROW_NONE) {
      float mean, rstd;
      row_stats(x, a.pre, &mean, &rstd);
      if (a.pre_stats && threadIdx.x % L == 0) *reinterpret_cast<float2*>(a.pre_stats + 2 * row) = make_float2(mean, rstd);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (at.in[r]) Row<T, V>::store(a.u, row * a.ldu + at.col[r], (x[r] - mean) * rstd * qw[r] + qb[r]);
    }
  }
}

// A team's units of rows.  With a gate shared by the rows of a sample, a unit is `rows_each` consecutive rows of one sample (the last
// one of a sample shorter) and ends with its partial of dg; otherwise a team takes every n-th row.
template <typename S, typename T, int L, int R>
__global__ __launch_bounds__(threads_of<L>()) void residual_bwd_kernel(ResidualArgs a) {
  constexpr int V = 16 / sizeof(T);
  constexpr int NT = threads_of<L>(), TEAMS = NT / L;
  typedef float wide __attribute__((ext_vector_type(V)));
  __shared__ float lds[2][8][2];
  __shared__ float buf[L < 256 ? NT / 64 : 1][L < 256 ? L * R * V : 1];
  TeamSum<L, 2> team_sum{lds};
  const Place<L, R, V> at(a.c);
  const float inv = 1.0f / static_cast<float>(a.c);
  // 16 values a thread and array in blocks of 512 leave no registers for the next row's, and rows of 8192 float32 none for the
  // weights, which are then read again for every row
  constexpr bool AHEAD = L < 512 || R * V < 16, KEEP = AHEAD || sizeof(T) < 4;
  wide kept_pw[R], kept_pb[R], kept_qw[R], dpw[R], dpb[R], dqw[R], dqb[R], dg[R];
  if (KEEP) {
    at.weights(a.post_w, 1.0f, kept_pw);
    at.weights(a.post_b, 0.0f, kept_pb);
    at.weights(a.pre_w, 1.0f, kept_qw);
  }
  const auto pw = [&](int r) { return KEEP ? kept_pw[r] : at.weight(a.post_w, 1.0f, r); };
  const auto pb = [&](int r) { return KEEP ? kept_pb[r] : at.weight(a.post_b, 0.0f, r); };
  const auto qw = [&](int r) { return KEEP ? kept_qw[r] : at.weight(a.pre_w, 1.0f, r); };
#pragma unroll
  for (int r = 0; r < R; ++r) dpw[r] = dpb[r] = dqw[r] = dqb[r] = dg[r] = 0.0f;
  const int64_t teams = static_cast<int64_t>(gridDim.x) * TEAMS;
  const int64_t team = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / L;
  const bool shared = a.shared_gate;
  // q - mean q - xhat mean(q xhat), times rstd
  auto through_norm = [&](wide (&q)[R], const wide (&xhat)[R], int kind, float rstd) {
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[0] += q[r][i];
        s[1] += q[r][i] * xhat[r][i];
      }
    team_sum(s);
    const float level = kind == QHA_ROW_LAYER ? s[0] * inv : 0.0f, along = s[1] * inv;
#pragma unroll
    for (int r = 0; r < R; ++r) q[r] = rstd * (q[r] - level - xhat[r] * along);
  };
  // where a team is: a row of a unit
  struct Walk {
    int64_t unit, row, end, sample;
  };
  const int64_t step = shared ? 1 : teams;
  const auto begin = [&](Walk& w) {
    w.row = w.unit;
    w.end = w.unit < a.units ? a.rows : 0;
    w.sample = 0;
    if (shared && w.unit < a.units) {
      w.sample = static_cast<uint32_t>(w.unit) / static_cast<uint32_t>(a.chunks);
      const int64_t first = (w.unit - w.sample * a.chunks) * a.rows_each;
      w.row = w.sample * a.positions + first;
      w.end = w.sample * a.positions + (first + a.rows_each < a.positions ? first + a.rows_each : a.positions);
    }
  };
  typename Row<S, V>::vec next_t[R], next_y[R];
  typename Row<T, V>::vec next_q[R], next_h[R], next_g[R];
  float2 next_ps = make_float2(0.0f, 1.0f), next_qs = next_ps;
  const auto fetch = [&](const Walk& w) {
    const int64_t row = w.row;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      next_t[r] = next_y[r] = static_cast<S>(0.0f);
      next_q[r] = next_h[r] = static_cast<T>(0.0f);
      next_g[r] = static_cast<T>(1.0f);
      if (!at.in[r]) continue;
      if (a.pre != QHA_ROW_NONE) {
        next_q[r] = Row<T, V>::raw(a.du, row * a.lddu + at.col[r]);
        next_y[r] = Row<S, V>::raw(a.x, row * a.ldx + at.col[r]);
      }
      if (a.dy) next_t[r] = Row<S, V>::raw(a.dy, row * a.lddy + at.col[r]);
      if (a.h) next_h[r] = Row<T, V>::raw(a.h, row * a.ldh + at.col[r]);
      if (a.gate) next_g[r] = Row<T, V>::raw(a.gate, (shared ? w.sample : row) * a.ldg + at.col[r]);
    }
    if (a.post != QHA_ROW_NONE) next_ps = *reinterpret_cast<const float2*>(a.post_stats + 2 * row);
    if (a.pre != QHA_ROW_NONE) next_qs = *reinterpret_cast<const float2*>(a.pre_stats + 2 * row);
  };
  Walk now;
  now.unit = team;
  begin(now);
  if (AHEAD && now.row < now.end) fetch(now);
  while (now.row < now.end) {
    const int64_t row = now.row;
    Walk after = now;
    after.row += step;
    if (after.row >= after.end) {
      after.unit = shared ? after.unit + teams : a.units;
      begin(after);
    }
    if (!AHEAD) fetch(now);
    wide t[R], y[R], q[R], h[R], g[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      t[r] = Row<S, V>::value(next_t[r]);
      y[r] = Row<S, V>::value(next_y[r]);
      q[r] = Row<T, V>::value(next_q[r]);
      h[r] = Row<T, V>::value(next_h[r]);
      g[r] = Row<T, V>::value(next_g[r]);
    }
    const float2 ps = next_ps, qs = next_qs;
    if (AHEAD && after.row < after.end) fetch(after);
    if (a.pre != QHA_ROW_NONE) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        y[r] = at.in[r] ? (y[r] - qs.x) * qs.y : 0.0f;
        dqw[r] += q[r] * y[r];
        dqb[r] += q[r];
        q[r] *= qw(r);
      }
      through_norm(q, y, a.pre, qs.y);
#pragma unroll
      for (int r = 0; r < R; ++r) t[r] += q[r];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (at.in[r]) Row<S, V>::store(a.dx, row * a.lddx + at.col[r], a.skip * t[r]);
    if (a.h) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        t[r] = at.in[r] ? a.branch * t[r] : 0.0f;
        h[r] = at.in[r] ? (h[r] - ps.x) * ps.y : 0.0f;
        const wide e = t[r] * (h[r] * pw(r) + pb(r));
        if (shared) dg[r] += e;
        else if (a.dgate && at.in[r]) Row<T, V>::store(a.dgate, row * a.lddg + at.col[r], e);
        t[r] *= g[r];
        dpw[r] += t[r] * h[r];
        dpb[r] += t[r];
        t[r] *= pw(r);
      }
      if (a.post != QHA_ROW_NONE) through_norm(t, h, a.post, ps.y);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (at.in[r]) Row<T, V>::store(a.dh, row * a.lddh + at.col[r], t[r]);
    }
    if (shared && after.unit != now.unit) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (a.dgate && at.in[r]) {
          if (a.chunks == 1) Row<T, V>::store(a.dgate, now.sample * a.lddg + at.col[r], dg[r]);
          else Row<float, V>::store(a.gate_part, now.unit * a.c + at.col[r], dg[r]);
        }
        dg[r] = 0.0f;
      }
    }
    now = after;
  }
  // the block's partials: teams of a wavefront by exchanges, wavefronts through LDS
  const bool alone = gridDim.x == 1;
  auto leave = [&](wide (&v)[R], int which) {
    float* out = alone ? a.dvec[which] : a.vec_part + (static_cast<int64_t>(blockIdx.x) * 4 + which) * a.c;
    if constexpr (L >= 256) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (at.in[r])
#pragma unroll
          for (int i = 0; i < V; ++i) out[at.col[r] + i] = v[r][i];
    } else {
#pragma unroll
      for (int o = L; o < 64; o <<= 1)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < V; ++i) v[r][i] += __shfl_xor(v[r][i], o, 64);
      __syncthreads();
      if ((threadIdx.x & 63) < L)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < V; ++i) buf[threadIdx.x >> 6][at.col[r] + i] = v[r][i];
      __syncthreads();
      for (int i = threadIdx.x; i < a.c; i += NT) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NT / 64; ++k) s += buf[k][i];
        out[i] = s;
      }
    }
  };
  if (a.dvec[0]) leave(dpw, 0);
  if (a.dvec[1]) leave(dpb, 1);
  if (a.dvec[2]) leave(dqw, 2);
  if (a.dvec[3]) leave(dqb, 3);
  if (!alone || !shared || !a.dgate || a.chunks == 1) return;
  // a block by itself adds the pieces of a sample's gate, too
  __syncthreads();
  for (int64_t i = threadIdx.x; i < a.rows / a.positions * a.c; i += NT) {
    const int64_t sample = i / a.c, col = i % a.c;
    const float* part = a.gate_part + sample * a.chunks * a.c + col;
    double s = 0.0;
#pragma unroll 8
    for (int64_t k = 0; k < a.chunks; ++k) s += static_cast<double>(part[k * a.c]);
    static_cast<T*>(a.dgate)[sample * a.lddg + col] = static_cast<T>(static_cast<float>(s));
  }
}

// Adds partials in float64: blocks below 4 * col_blocks those of the weights, 32 columns each, the others those of
// a sample's gate.  Eight threads a column take every eighth partial and are added in order.
template <typename T>
__global__ __launch_bounds__(256) void residual_sums_kernel(ResidualArgs a, int32_t col_blocks) {
  __shared__ double buf[8][32];
  const int lane = static_cast<int>(threadIdx.x) & 31, k0 = static_cast<int>(threadIdx.x) >> 5;
  const int64_t set = static_cast<int64_t>(blockIdx.x) / col_blocks;      // 0 .. 3 the weights' gradients, then the samples
  const int col = static_cast<int>(static_cast<int64_t>(blockIdx.x) % col_blocks) * 32 + lane;
  const bool weights = set < 4;
  if (weights && !a.dvec[set]) return;
  const float* part = weights ? a.vec_part + set * a.c : a.gate_part + (set - 4) * a.chunks * a.c;
  const int64_t stride = weights ? 4LL * a.c : a.c, n = weights ? a.blocks : a.chunks;
  double s = 0.0;
  if (col < a.c) {
#pragma unroll 8
    for (int64_t k = k0; k < n; k += 8) s += static_cast<double>(part[k * stride + col]);
  }
  buf[k0][lane] = s;
  __syncthreads();
  if (k0 != 0 || col >= a.c) return;
  for (int k = 1; k < 8; ++k) s += buf[k][lane];
  if (weights) a.dvec[set][col] = static_cast<float>(s);
  else static_cast<T*>(a.dgate)[(set - 4) * a.lddg + col] = static_cast<T>(static_cast<float>(s));
}

// lanes of a team, by the vectors of a row
int team_of(int nvec) {
  return nvec <= 8 ? 8 : nvec <= 16 ? 16 : nvec <= 32 ? 32 : nvec <= 128 ? 64 : nvec <= 512 ? 256 : 512;
}
// Blocks of a launch: two a compute unit backward (its registers leave room for two or three: 300k x 256 float32 with 1024 blocks
// 400 us, with 512 322), four forward, more of the larger ones (300k x 128 float32 with 2048 blocks, which seven a unit
// do not divide, 122 us, with 1024 108; 4000 x 8192 float32 84 and 76).
int64_t most_blocks(int lanes) { return lanes == 512 ? 256 : 512; }
int64_t most_blocks_fwd(int lanes) { return lanes < 256 ? 1024 : 2048; }

template <typename S, typename T, int L, int R>
void run(const ResidualArgs& a, bool backward, hipStream_t s) {
  constexpr int TEAMS = threads_of<L>() / L;
  if (!backward) {
    const int64_t want = (a.rows + TEAMS - 1) / TEAMS;
    residual_fwd_kernel<S, T, L, R><<<static_cast<uint32_t>(want < most_blocks_fwd(L) ? want : most_blocks_fwd(L)), threads_of<L>(), 0, s>>>(a);
    return;
  }
  residual_bwd_kernel<S, T, L, R><<<static_cast<uint32_t>(a.blocks), threads_of<L>(), 0, s>>>(a);
}

template <typename S, typename T>
void run(const ResidualArgs& a, bool backward, hipStream_t s) {
  const int nvec = a.rows > 0 ? a.c / (16 / static_cast<int>(sizeof(T))) : 0;
  if (nvec == 0) {}                  // no rows: zeros alone
  else if (nvec <= 8) run<S, T, 8, 1>(a, backward, s);
  else if (nvec <= 16) run<S, T, 16, 1>(a, backward, s);
  else if (nvec <= 32) run<S, T, 32, 1>(a, backward, s);
  else if (nvec <= 64) run<S, T, 64, 1>(a, backward, s);
  else if (nvec <= 128) run<S, T, 64, 2>(a, backward, s);
  else if (nvec <= 256) run<S, T, 256, 1>(a, backward, s);
  else if (nvec <= 512) run<S, T, 256, 2>(a, backward, s);
  else if (nvec <= 1024) run<S, T, 512, 2>(a, backward, s);
  else if constexpr (sizeof(T) == 4) run<S, T, 512, 4>(a, backward, s);      // at most 8192 values
  if (!backward || a.blocks == 1) return;
  const bool gates = a.dgate && a.shared_gate && a.chunks > 1;
  const bool vectors = a.dvec[0] || a.dvec[1] || a.dvec[2] || a.dvec[3];
  if (!gates && !vectors) return;
  const int32_t col_blocks = (a.c + 31) / 32;
  const int64_t sets = 4 + (gates ? a.rows / a.positions : 0);
  residual_sums_kernel<T><<<static_cast<uint32_t>(sets * col_blocks), 256, 0, s>>>(a, col_blocks);
}

}  // namespace

// Blocks, units and pieces of samples of a backward, from a's rows, positions, c and type.
void residual_plan(ResidualArgs& a) {
  const int lanes = team_of(a.c / (a.type == QHA_F32 ? 4 : 8));
  const int teams = lanes < 256 ? 256 / lanes : 1;
  // one block alone, without a second launch, where its teams take at most three rows each (97 rows of 64 in three samples, ten each,
  // 17.6 us, with two launches 15; 4 rows of 64 12 and 15)
  const int64_t samples = a.rows / a.positions, most = a.rows <= 3 * teams ? 1 : most_blocks(lanes);
  a.chunks = 1;
  a.rows_each = a.positions;
  a.units = a.rows;
  if (a.shared_gate) {
    // whole samples where they fill the launch; otherwise pieces, at most one for each team
    const int64_t pieces = samples < most * teams ? most * teams / samples : 1;
    a.rows_each = (a.positions + pieces - 1) / pieces;
    a.chunks = (a.positions + a.rows_each - 1) / a.rows_each;
    a.units = samples * a.chunks;
  }
  const int64_t want = (a.units + teams - 1) / teams;
  a.blocks = want < most ? want : most;
  if (!a.shared_gate) a.units = a.blocks * teams < a.rows ? a.blocks * teams : a.rows;
}

size_t residual_workspace(const ResidualArgs& a) {
  size_t bytes = static_cast<size_t>(a.blocks) * 4 * static_cast<size_t>(a.c) * sizeof(float);
  if (a.shared_gate && a.chunks > 1) bytes += static_cast<size_t>(a.units) * static_cast<size_t>(a.c) * sizeof(float);
  return bytes;
}

hipError_t launch_residual(const ResidualArgs& a, bool backward, hipStream_t s) {
  if (a.type == QHA_F32) run<float, float>(a, backward, s);
  else if (a.type == QHA_BF16 && a.stream_type == QHA_F32) run<float, __bf16>(a, backward, s);
  else if (a.type == QHA_BF16) run<__bf16, __bf16>(a, backward, s);
  else if (a.stream_type == QHA_F32) run<float, _Float16>(a, backward, s);
  else run<_Float16, _Float16>(a, backward, s);
  return hipGetLastError();
}

}  // namespace qha
