// Group normalisation with an activation, channels last, and its gradients.
//
// Mathematics: per sample and group, mean and variance over positions and channels; y = act(w xhat + b)
// with xhat = (x - mean) rstd.  Backward with dz = dy act'(w xhat + b), q = w dz:
// dx = rstd (q - mean q - xhat mean(q xhat)), dw = sum dz xhat, db = sum dz.
//
// Bound: memory (x read and y written once at the least; dy, x and dx in the backward).
//
// Samples of at most 8192 values whose vectors lie in one group take one pass with the sample in registers
// (norm_rows.hip); the others two launches.  A block of 256 threads owns a chunk of a sample's rows
// and all channels: a thread keeps one 16-byte vector of channels (several where the row has more
// than 256 vectors) and walks down the rows, so loads are whole rows and nothing is exchanged until
// the chunk ends; then the vectors' sums meet in LDS and one pair per group goes to the workspace.
// The second launch adds the pairs of its sample's chunks in order and applies.  Forward sums are
// float64 (x and x^2: the float64 pipes idle in a memory-bound loop, and mean^2 >> variance costs
// nothing there); the backward's per-channel sums run in float32 over a chunk and meet in float64.
// 16 x 4096 x 512 bf16 in 32 groups, SiLU: 13 us for the sums (5.2 TB/s) and 33 us to apply (4.1 TB/s).
#include "act_common.hpp"
#include "qha_internal.hpp"

namespace qha {
namespace {

constexpr int NT = 256;

// Where a thread's vectors lie: with R = 1 a row has at most 256 vectors and the block takes
// 256 / nvec rows at a time; with R > 1 the block takes one row at a time, R vectors a thread.
template <int R>
struct Place {
  int nvec, tx, rl, rows_par;
  bool active;
  __device__ __forceinline__ explicit Place(int nv) : nvec(nv) {
    const int tid = threadIdx.x;
    if (R == 1) {
      rows_par = NT / nvec;
      rl = tid / nvec;
      tx = tid - rl * nvec;
      active = rl < rows_par;
    } else {
      rows_par = 1;
      rl = 0;
      tx = tid;
      active = true;
    }
  }
  __device__ __forceinline__ int vec(int r) const { return tx + r * NT; }
  __device__ __forceinline__ bool has(int r) const { return R == 1 ? active : vec(r) < nvec; }
  __device__ __forceinline__ int slot(int r) const { return rl * nvec + vec(r); }
};

__device__ __forceinline__ double shfl_xor_d(double x, int o) { return __shfl_xor(x, o, 64); }

// Threads per group when `entries` values are added per group: a power of two up to a wavefront.
__device__ __forceinline__ int team_size(int entries) {
  int ts = 1;
  while (ts < entries && ts < 64) ts <<= 1;
  return ts;
}

// Adds the block's per-channel pairs (s0, s1) by group and writes out[g] (two doubles each).  VG: every
// 16-byte vector lies in one group, and a thread's V channels are added before they meet in LDS;
// otherwise the channels go through LDS one lane of the vectors at a time.
template <int V, int R, bool VG, typename F>
__device__ __forceinline__ void reduce_groups(const Place<R>& at, int c, int groups, double2* buf, const F& pair,
                                              double* out) {
  const int per = c / groups;
  const int nv = per / V;
  const int entries = VG ? at.rows_par * nv : at.rows_par * ((per + V - 1) / V + 1);
  const int ts = team_size(entries);
  const int team = threadIdx.x / ts, ln = threadIdx.x % ts, teams = NT / ts;
  if (VG) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (at.has(r)) {
        double2 s = {0.0, 0.0};
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const double2 p = pair(r, v);
          s.x += p.x;
          s.y += p.y;
        }
        buf[at.slot(r)] = s;
      }
    __syncthreads();
  }
  for (int g0 = 0; g0 < groups; g0 += teams) {
    const int g = g0 + team;
    double a = 0.0, b = 0.0;
    if (VG) {
      if (g < groups)
        for (int e = ln; e < entries; e += ts) {
          const double2 s = buf[(e / nv) * at.nvec + g * nv + e % nv];
          a += s.x;
          b += s.y;
        }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (at.has(r)) buf[at.slot(r)] = pair(r, v);
        __syncthreads();
        if (g < groups) {
          // vectors whose lane v is a channel of group g
          const int lo = (g * per - v + V - 1) / V, hi = ((g + 1) * per - v + V - 1) / V;
          const int n = hi - lo;
          for (int e = ln; e < at.rows_par * n; e += ts) {
            const double2 s = buf[(e / n) * at.nvec + lo + e % n];
            a += s.x;
            b += s.y;
          }
        }
      }
    }
    for (int o = ts >> 1; o > 0; o >>= 1) {
      a += shfl_xor_d(a, o);
      b += shfl_xor_d(b, o);
    }
    if (g < groups && ln == 0) {
      out[2 * g] = a;
      out[2 * g + 1] = b;
    }
  }
}

struct Item {
  int64_t sample, row0, rows;
  __device__ __forceinline__ Item(const NormArgs& a, int64_t i) {
    sample = i / a.chunks;
    const int64_t ch = i - sample * a.chunks;
    row0 = sample * a.positions + ch * a.chunk_rows;
    const int64_t left = a.positions - ch * a.chunk_rows;
    rows = left < a.chunk_rows ? left : a.chunk_rows;
  }
};

template <typename T, int R, bool VG>
__global__ __launch_bounds__(NT) void norm_sums_kernel(NormArgs a) {
  constexpr int V = Pack<T>::N;
  __shared__ double2 buf[NT * R];
  const Place<R> at(a.c / V);
  for (int64_t item = blockIdx.x; item < a.samples * a.chunks; item += gridDim.x) {
    const Item it(a, item);
    const T* x = static_cast<const T*>(a.x) + it.row0 * a.ldx;
    double s0[R][V], s1[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int v = 0; v < V; ++v) s0[r][v] = s1[r][v] = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (at.has(r)) {
#pragma unroll 4
        for (int64_t i = at.rl; i < it.rows; i += at.rows_par) {
          const typename Pack<T>::wide q = Pack<T>::load(x + i * a.ldx + at.vec(r) * V);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const double d = static_cast<double>(q[v]);
            s0[r][v] += d;
            s1[r][v] += d * d;
          }
        }
      }
    reduce_groups<V, R, VG>(at, a.c, a.groups, buf, [&](int r, int v) { return make_double2(s0[r][v], s1[r][v]); },
                            a.group_part + item * a.groups * 2);
  }
}

// Adds the sample's chunk pairs per group, in a fixed order, and hands each to `put`.  Neighbouring threads
// read neighbouring groups of one chunk; the threads of a group then meet in LDS.
template <typename F>
__device__ __forceinline__ void combine_chunks(const NormArgs& a, int64_t sample, double2* buf, const F& put) {
  const int groups = a.groups;
  const double2* part = reinterpret_cast<const double2*>(a.group_part) + sample * a.chunks * groups;
  const int lanes = groups < NT ? NT / groups : 1;
  for (int g0 = 0; g0 < groups; g0 += NT) {
    const int lane = groups < NT ? static_cast<int>(threadIdx.x) / groups : 0;
    const int g = groups < NT ? static_cast<int>(threadIdx.x) % groups : g0 + static_cast<int>(threadIdx.x);
    double2 s = {0.0, 0.0};
    if (lane < lanes && g < groups) {
#pragma unroll 4
      for (int64_t k = lane; k < a.chunks; k += lanes) {
        const double2 p = part[k * groups + g];
        s.x += p.x;
        s.y += p.y;
      }
    }
    if (lanes > 1) {
      __syncthreads();
      buf[threadIdx.x] = s;
      __syncthreads();
      if (lane == 0)
        for (int k = 1; k < lanes; ++k) {
          s.x += buf[k * groups + g].x;
          s.y += buf[k * groups + g].y;
        }
    }
    if (lane == 0 && g < groups) put(g, s.x, s.y);
  }
}

template <typename T, int R, bool VG>
__global__ __launch_bounds__(NT) void norm_apply_kernel(NormArgs a) {
  constexpr int V = Pack<T>::N;
  extern __shared__ float2 stat[];           // mean, rstd per group
  __shared__ double2 buf[NT];
  const Place<R> at(a.c / V);
  const int per = a.c / a.groups;
  const double inv = 1.0 / (static_cast<double>(a.positions) * per);
  for (int64_t item = blockIdx.x; item < a.samples * a.chunks; item += gridDim.x) {
    const Item it(a, item);
    const bool first = item % a.chunks == 0;
    __syncthreads();                           // the last item's statistics have been used
    combine_chunks(a, it.sample, buf, [&](int g, double s, double q) {
      const double mean = s * inv, var = q * inv - mean * mean;
      const double rstd = 1.0 / sqrt((var < 0.0 ? 0.0 : var) + a.eps);
      stat[g] = make_float2(static_cast<float>(mean), static_cast<float>(rstd));
      if (first && a.mean) {
        a.mean[it.sample * a.groups + g] = static_cast<float>(mean);
        a.rstd[it.sample * a.groups + g] = static_cast<float>(rstd);
      }
    });
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (at.has(r)) {
        const int ch = at.vec(r) * V;
        float mean[V], scale[V], bias[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float2 st = stat[(VG ? ch : ch + v) / per];
          mean[v] = st.x;
          scale[v] = a.w ? st.y * a.w[ch + v] : st.y;
          bias[v] = a.b ? a.b[ch + v] : 0.0f;
        }
#pragma unroll 4
        for (int64_t i = at.rl; i < it.rows; i += at.rows_par) {
          const int64_t row = it.row0 + i;
          typename Pack<T>::wide q = Pack<T>::load(static_cast<const T*>(a.x) + row * a.ldx + ch);
#pragma unroll
          for (int v = 0; v < V; ++v) q[v] = activate((q[v] - mean[v]) * scale[v] + bias[v], a.act);
          Pack<T>::store(static_cast<T*>(a.y) + row * a.ldy + ch, q);
        }
      }
  }
}

// One block's items: per item the group sums of q and q xhat, over all of them the channel sums of dz and dz xhat.
template <typename T, int R, bool VG>
__global__ __launch_bounds__(NT) void norm_grad_sums_kernel(NormArgs a) {
  constexpr int V = Pack<T>::N;
  __shared__ double2 buf[R == 1 ? NT * V / 2 : NT * R];
  const Place<R> at(a.c / V);
  const int per = a.c / a.groups;
  const int64_t items = a.samples * a.chunks;
  const int64_t each = (items + a.sum_blocks - 1) / a.sum_blocks;
  const int64_t begin = blockIdx.x * each, end = begin + each < items ? begin + each : items;
  float db[R][V], dw[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) db[r][v] = dw[r][v] = 0.0f;
  for (int64_t i = begin; i < end; ++i) {
    const Item it(a, i);
    float s0[R][V], s1[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int v = 0; v < V; ++v) s0[r][v] = s1[r][v] = 0.0f;
      if (at.has(r)) {
        const int ch = at.vec(r) * V;
        float mean[V], rstd[V], w[V], b[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int64_t g = it.sample * a.groups + (VG ? ch : ch + v) / per;
          mean[v] = a.mean[g];
          rstd[v] = a.rstd[g];
          w[v] = a.w ? a.w[ch + v] : 1.0f;
          b[v] = a.b ? a.b[ch + v] : 0.0f;
        }
#pragma unroll 2
        for (int64_t k = at.rl; k < it.rows; k += at.rows_par) {
          const int64_t row = it.row0 + k;
          const typename Pack<T>::wide x = Pack<T>::load(static_cast<const T*>(a.x) + row * a.ldx + ch);
          const typename Pack<T>::wide dy = Pack<T>::load(static_cast<const T*>(a.dy) + row * a.lddy + ch);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float xhat = (x[v] - mean[v]) * rstd[v];
            const float dz = grad_z(dy[v], x[v], mean[v], rstd[v], xhat, w[v], b[v], a.act);
            s0[r][v] += dz;
            s1[r][v] += dz * xhat;
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          db[r][v] += s0[r][v];
          dw[r][v] += s1[r][v];
          s0[r][v] *= w[v];
          s1[r][v] *= w[v];
        }
      }
    }
    reduce_groups<V, R, VG>(at, a.c, a.groups, buf,
                            [&](int r, int v) { return make_double2(static_cast<double>(s0[r][v]), static_cast<double>(s1[r][v])); },
                            a.group_part + i * a.groups * 2);
  }
  if (!a.dw) return;
  float* out = a.chan_part + static_cast<int64_t>(blockIdx.x) * 2 * a.c;
  if constexpr (R > 1) {                     // a thread has its channels to itself
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (at.has(r))
#pragma unroll
        for (int v = 0; v < V; ++v) {
          out[at.vec(r) * V + v] = dw[r][v];
          out[a.c + at.vec(r) * V + v] = db[r][v];
        }
  } else {
    // [rows_par][c] pairs, then neighbouring lanes share a channel
    float2* pair = reinterpret_cast<float2*>(buf);
    __syncthreads();
    if (at.active)
#pragma unroll
      for (int v = 0; v < V; ++v) pair[at.rl * a.c + at.tx * V + v] = make_float2(dw[0][v], db[0][v]);
    __syncthreads();
    int lanes = 1;
    while (lanes < 64 && 2 * lanes * a.c <= NT) lanes *= 2;
    const int ln = threadIdx.x % lanes;
    for (int c0 = 0; c0 < a.c; c0 += NT / lanes) {
      const int ch = c0 + threadIdx.x / lanes;
      double s = 0.0, q = 0.0;
      if (ch < a.c)
#pragma unroll 4
        for (int k = ln; k < at.rows_par; k += lanes) {
          s += static_cast<double>(pair[k * a.c + ch].x);
          q += static_cast<double>(pair[k * a.c + ch].y);
        }
      for (int o = lanes >> 1; o > 0; o >>= 1) {
        s += shfl_xor_d(s, o);
        q += shfl_xor_d(q, o);
      }
      if (ln == 0 && ch < a.c) {
        out[ch] = static_cast<float>(s);
        out[a.c + ch] = static_cast<float>(q);
      }
    }
  }
}

// Channels [16 block ..) of dw and db (2c values laid end to end): the partials added in a fixed order.
__device__ __forceinline__ void sum_channels(const NormArgs& a, int block, double* buf) {
  const int col = block * 16 + threadIdx.x % 16, lane = threadIdx.x / 16;
  double s = 0.0;
  if (col < 2 * a.c) {
#pragma unroll 8
    for (int64_t k = lane; k < a.sum_blocks; k += 16) s += static_cast<double>(a.chan_part[k * 2 * a.c + col]);
  }
  buf[threadIdx.x] = s;
  __syncthreads();
  if (lane == 0 && col < 2 * a.c) {
    for (int k = 1; k < 16; ++k) s += buf[k * 16 + threadIdx.x];
    if (col < a.c) a.dw[col] = static_cast<float>(s);
    else a.db[col - a.c] = static_cast<float>(s);
  }
}

// The first blocks finish dw and db, the others apply dx to one item each.
template <typename T, int R, bool VG>
__global__ __launch_bounds__(NT) void norm_grad_apply_kernel(NormArgs a, int32_t sum_cols) {
  constexpr int V = Pack<T>::N;
  extern __shared__ float2 stat[];           // mean of q, mean of q xhat per group
  __shared__ double2 pairs[NT];
  if (static_cast<int32_t>(blockIdx.x) < sum_cols) {
    sum_channels(a, static_cast<int>(blockIdx.x), reinterpret_cast<double*>(pairs));
    return;
  }
  const Place<R> at(a.c / V);
  const int per = a.c / a.groups;
  const double inv = 1.0 / (static_cast<double>(a.positions) * per);
  const int64_t step = static_cast<int64_t>(gridDim.x) - sum_cols;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) - sum_cols; item < a.samples * a.chunks; item += step) {
    const Item it(a, item);
    __syncthreads();                           // the last item's means have been used
    combine_chunks(a, it.sample, pairs, [&](int g, double s, double q) {
      stat[g] = make_float2(static_cast<float>(s * inv), static_cast<float>(q * inv));
    });
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (at.has(r)) {
        const int ch = at.vec(r) * V;
        float mean[V], rstd[V], w[V], b[V], m0[V], m1[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int g = (VG ? ch : ch + v) / per;
          mean[v] = a.mean[it.sample * a.groups + g];
          rstd[v] = a.rstd[it.sample * a.groups + g];
          m0[v] = stat[g].x;
          m1[v] = stat[g].y;
          w[v] = a.w ? a.w[ch + v] : 1.0f;
          b[v] = a.b ? a.b[ch + v] : 0.0f;
        }
#pragma unroll 2
        for (int64_t k = at.rl; k < it.rows; k += at.rows_par) {
          const int64_t row = it.row0 + k;
          const typename Pack<T>::wide x = Pack<T>::load(static_cast<const T*>(a.x) + row * a.ldx + ch);
          const typename Pack<T>::wide dy = Pack<T>::load(static_cast<const T*>(a.dy) + row * a.lddy + ch);
          typename Pack<T>::wide dx;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float xhat = (x[v] - mean[v]) * rstd[v];
            const float q = w[v] * grad_z(dy[v], x[v], mean[v], rstd[v], xhat, w[v], b[v], a.act);
            dx[v] = rstd[v] * (q - m0[v] - xhat * m1[v]);
          }
          Pack<T>::store(static_cast<T*>(a.y) + row * a.ldy + ch, dx);
        }
      }
  }
}

// Blocks of one launch (a grid holds fewer than 2^32 threads); blocks step over further items.
uint32_t blocks_for(int64_t items) { return static_cast<uint32_t>(items < (1 << 22) ? items : (1 << 22)); }

int vectors(const NormArgs& a) { return a.c / (a.type == QHA_F32 ? 4 : 8); }

template <typename T, int R, bool VG>
void fwd(const NormArgs& a, hipStream_t s) {
  const uint32_t items = blocks_for(a.samples * a.chunks);
  norm_sums_kernel<T, R, VG><<<items, NT, 0, s>>>(a);
  norm_apply_kernel<T, R, VG><<<items, NT, a.groups * sizeof(float2), s>>>(a);
}

template <typename T, int R, bool VG>
void bwd(const NormArgs& a, hipStream_t s) {
  const uint32_t items = blocks_for(a.samples * a.chunks);
  const int32_t cols = a.dw ? (2 * a.c + 15) / 16 : 0;
  if (items) norm_grad_sums_kernel<T, R, VG><<<static_cast<uint32_t>(a.sum_blocks), NT, 0, s>>>(a);
  norm_grad_apply_kernel<T, R, VG><<<items + cols, NT, a.groups * sizeof(float2), s>>>(a, cols);
}

template <typename T, int R>
void go(const NormArgs& a, bool backward, hipStream_t s) {
  const bool whole = (a.c / a.groups) % Pack<T>::N == 0;
  if (backward) whole ? bwd<T, R, true>(a, s) : bwd<T, R, false>(a, s);
  else whole ? fwd<T, R, true>(a, s) : fwd<T, R, false>(a, s);
}

template <typename T>
void go(const NormArgs& a, bool backward, hipStream_t s) {
  const int nvec = vectors(a);
  if (nvec <= NT) go<T, 1>(a, backward, s);
  else if (nvec <= 2 * NT) go<T, 2>(a, backward, s);
  else if (nvec <= 4 * NT) go<T, 4>(a, backward, s);
  else if constexpr (sizeof(T) == 4) go<T, 8>(a, backward, s);      // at most 8192 channels
}

hipError_t launch(const NormArgs& a, bool backward, hipStream_t s) {
  if (a.type == QHA_F32) go<float>(a, backward, s);
  else if (a.type == QHA_BF16) go<__bf16>(a, backward, s);
  else go<_Float16>(a, backward, s);
  return hipGetLastError();
}

// Four blocks for each compute unit: with eight, the second launch of 16 x 4096 x 512 bf16 spends more on
// adding twice the chunks' pairs than it gains (57 against 39 us), with two it waits on memory (41 us).
constexpr int64_t kNormItems = 1024;

}  // namespace

// Chunks: enough items for kNormItems blocks, but no chunk of fewer than four rows per thread.
void norm_plan(NormArgs& a, bool backward) {
  if (norm_rows_fit(a)) {
    a.chunks = 0;
    a.chunk_rows = 1;
    a.sum_blocks = backward ? norm_rows_blocks(a) : 0;
    return;
  }
  const int nvec = vectors(a);
  const int64_t rows_par = nvec < NT ? NT / nvec : 1;
  int64_t chunks = (kNormItems + a.samples - 1) / a.samples;
  const int64_t most = (a.positions + 4 * rows_par - 1) / (4 * rows_par);
  if (chunks > most) chunks = most;
  a.chunk_rows = (a.positions + chunks - 1) / chunks;
  a.chunks = (a.positions + a.chunk_rows - 1) / a.chunk_rows;
  const int64_t items = a.samples * a.chunks;
  a.sum_blocks = backward ? (items < kNormItems ? items : kNormItems) : 0;
}

size_t norm_workspace(const NormArgs& a, bool backward) {
  const size_t chan = static_cast<size_t>(a.sum_blocks) * 2 * static_cast<size_t>(a.c) * sizeof(float);
  const size_t part = static_cast<size_t>(a.samples * a.chunks) * static_cast<size_t>(a.groups) * 2 * sizeof(double);
  return (chan + 15) / 16 * 16 + part;
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  return norm_rows_fit(a) ? launch_norm_rows(a, false, s) : launch(a, false, s);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  return a.samples > 0 && norm_rows_fit(a) ? launch_norm_rows(a, true, s) : launch(a, true, s);
}

}  // namespace qha
