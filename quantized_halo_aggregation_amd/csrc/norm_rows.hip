// Group normalisation of single rows (one position per sample) and its gradients, in one pass.
//
// Mathematics: as in the two-launch form: y = act(w xhat + b), xhat = (x - mean) rstd per row and group;
// dx = rstd (q - mean q - xhat mean(q xhat)) with q = w dy act'(.), dw = sum dz xhat, db = sum dz.
//
// Bound: memory, every array once.  A row belongs to a team of L threads (8 to a wavefront's 64, or a
// whole block of 256 for wide rows) that holds it in registers, R vectors of 16 bytes a thread, so
// the mean, the squares about it and the output come from one read.  Groups of a power of two of
// vectors are summed by exchanges between neighbouring lanes, whole rows by all of the team, other
// group sizes through LDS.  Teams walk over many rows with the next row's loads in flight and keep w, b
// and (backward) their share of dw and db in registers; a block leaves one partial of dw and db,
// and a second small launch adds those in float64.
#include "act_common.hpp"
#include "qha_internal.hpp"

namespace qha {
namespace {

constexpr int NT = 256;
constexpr int64_t kRowBlocks = 2048;     // forward: eight blocks for each compute unit
constexpr int64_t kGradBlocks = 1024;    // backward: each leaves a partial of dw and db

enum { SUM_LANES = 0, SUM_ROW = 1, SUM_LDS = 2 };

// How a group's vectors are summed: neighbouring lanes, the whole row, or through LDS.
int sum_mode(int nv, int groups, int lanes) {
  if (groups == 1) return SUM_ROW;
  return (nv & (nv - 1)) == 0 && nv <= (lanes < 64 ? lanes : 64) ? SUM_LANES : SUM_LDS;
}

// a[r] (one value per vector of the team's row) becomes its group's sum.  lds: one float per vector of
// every team of the block.
template <int L, int R>
__device__ __forceinline__ void group_sum(float (&a)[R], int mode, int nv, int nvec, float* lds) {
  constexpr int W = L < 64 ? L : 64;
  const int ln = threadIdx.x % L;
  if (mode == SUM_LANES) {
    for (int o = nv >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) a[r] += __shfl_xor(a[r], o, 64);
    return;
  }
  if (mode == SUM_ROW) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) t += a[r];
#pragma unroll
    for (int o = W >> 1; o > 0; o >>= 1) t += __shfl_xor(t, o, 64);
    if constexpr (L == 256) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = t;
      __syncthreads();
      t = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) a[r] = t;
    return;
  }
  float* mine = lds + (threadIdx.x / L) * L * R;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) mine[ln + r * L] = a[r];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = ln + r * L;
    if (j >= nvec) continue;
    const float* g = mine + j / nv * nv;
    float t = 0.0f;
    for (int k = 0; k < nv; ++k) t += g[k];
    a[r] = t;
  }
}

template <typename T, int L, int R>
__global__ __launch_bounds__(NT) void rows_fwd_kernel(NormArgs a, int mode) {
  constexpr int V = Pack<T>::N;
  typedef typename Pack<T>::wide wide;
  __shared__ float lds[NT * R];
  const int nvec = a.c / V, per = a.c / a.groups, nv = per / V;
  const int ln = threadIdx.x % L;
  const float inv = 1.0f / static_cast<float>(per);
  wide w[R], b[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = ln + r * L;
      w[r][v] = a.w && j < nvec ? a.w[j * V + v] : 1.0f;
      b[r][v] = a.b && j < nvec ? a.b[j * V + v] : 0.0f;
    }
  const int64_t step = static_cast<int64_t>(gridDim.x) * (NT / L);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (NT / L);
  // every team of the block runs the same number of turns (the LDS sums meet at barriers)
  wide next[R];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      next[r] = 0.0f;
      if (row < a.samples && ln + r * L < nvec) next[r] = Pack<T>::load(static_cast<const T*>(a.x) + row * a.ldx + (ln + r * L) * V);
    }
  };
  const int team = threadIdx.x / L;
  fetch(first + team);
  for (int64_t at = first; at < a.samples; at += step) {
    const int64_t row = at + team;
    wide x[R];
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = next[r];
      s[r] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) s[r] += x[r][v];
    }
    fetch(row + step);
    group_sum<L, R>(s, mode, nv, nvec, lds);
    float mean[R], q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = s[r] * inv;
      q[r] = 0.0f;
      const bool in = ln + r * L < nvec;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float d = x[r][v] - mean[r];
        q[r] += in ? d * d : 0.0f;
      }
    }
    group_sum<L, R>(q, mode, nv, nvec, lds);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int j = ln + r * L;
      if (row >= a.samples || j >= nvec) continue;
      const float rstd = 1.0f / sqrtf(q[r] * inv + static_cast<float>(a.eps));
      wide y;
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = activate((x[r][v] - mean[r]) * rstd * w[r][v] + b[r][v], a.act);
      Pack<T>::store(static_cast<T*>(a.y) + row * a.ldy + j * V, y);
      if (a.mean && j % nv == 0) {
        a.mean[row * a.groups + j / nv] = mean[r];
        a.rstd[row * a.groups + j / nv] = rstd;
      }
    }
  }
}

template <typename T, int L, int R>
__global__ __launch_bounds__(NT) void rows_bwd_kernel(NormArgs a, int mode) {
  constexpr int V = Pack<T>::N;
  typedef typename Pack<T>::wide wide;
  __shared__ float lds[2 * NT * R];
  const int nvec = a.c / V, per = a.c / a.groups, nv = per / V;
  const int ln = threadIdx.x % L;
  const float inv = 1.0f / static_cast<float>(per);
  wide w[R], b[R], dw[R], db[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    dw[r] = db[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = ln + r * L;
      w[r][v] = a.w && j < nvec ? a.w[j * V + v] : 1.0f;
      b[r][v] = a.b && j < nvec ? a.b[j * V + v] : 0.0f;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * (NT / L);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (NT / L);
  wide next_x[R], next_dy[R];
  float next_mean[R], next_rstd[R];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int j = ln + r * L;
      next_x[r] = next_dy[r] = 0.0f;
      next_mean[r] = next_rstd[r] = 0.0f;
      if (row < a.samples && j < nvec) {
        next_x[r] = Pack<T>::load(static_cast<const T*>(a.x) + row * a.ldx + j * V);
        next_dy[r] = Pack<T>::load(static_cast<const T*>(a.dy) + row * a.lddy + j * V);
        next_mean[r] = a.mean[row * a.groups + j / nv];
        next_rstd[r] = a.rstd[row * a.groups + j / nv];
      }
    }
  };
  const int team = threadIdx.x / L;
  fetch(first + team);
  for (int64_t at = first; at < a.samples; at += step) {
    const int64_t row = at + team;
    wide xhat[R], q[R];
    float rstd[R], s0[R], s1[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = next_rstd[r];
      s0[r] = s1[r] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float xh = (next_x[r][v] - next_mean[r]) * rstd[r];
        const float dz = grad_z(next_dy[r][v], next_x[r][v], next_mean[r], rstd[r], xh, w[r][v], b[r][v], a.act);
        dw[r][v] += dz * xh;
        db[r][v] += dz;
        xhat[r][v] = xh;
        q[r][v] = w[r][v] * dz;
        s0[r] += q[r][v];
        s1[r] += q[r][v] * xh;
      }
    }
    fetch(row + step);
    group_sum<L, R>(s0, mode, nv, nvec, lds);
    group_sum<L, R>(s1, mode, nv, nvec, lds + NT * R);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int j = ln + r * L;
      if (row >= a.samples || j >= nvec) continue;
      wide dx;
#pragma unroll
      for (int v = 0; v < V; ++v) dx[v] = rstd[r] * (q[r][v] - s0[r] * inv - xhat[r][v] * (s1[r] * inv));
      Pack<T>::store(static_cast<T*>(a.y) + row * a.ldy + j * V, dx);
    }
  }
  if (!a.dw) return;
  float* out = a.chan_part + static_cast<int64_t>(blockIdx.x) * 2 * a.c;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      __syncthreads();
      lds[threadIdx.x] = dw[r][v];
      lds[NT + threadIdx.x] = db[r][v];
      __syncthreads();
      const int j = threadIdx.x + r * L;
      if (threadIdx.x < L && j < nvec) {
        float s = 0.0f, q = 0.0f;
#pragma unroll
        for (int k = 0; k < NT / L; ++k) {
          s += lds[k * L + threadIdx.x];
          q += lds[NT + k * L + threadIdx.x];
        }
        out[j * V + v] = s;
        out[a.c + j * V + v] = q;
      }
    }
}

// dw and db (2c values laid end to end): 16 columns a block, the blocks' partials added by 64 threads a
// column and then in order.
__global__ __launch_bounds__(1024) void rows_channels_kernel(NormArgs a) {
  __shared__ double buf[1024];
  const int col = blockIdx.x * 16 + threadIdx.x % 16, lane = threadIdx.x / 16;
  double s = 0.0;
  if (col < 2 * a.c) {
#pragma unroll 8
    for (int64_t k = lane; k < a.sum_blocks; k += 64) s += static_cast<double>(a.chan_part[k * 2 * a.c + col]);
  }
  buf[threadIdx.x] = s;
  __syncthreads();
  if (lane < 4) {
    for (int k = lane + 4; k < 64; k += 4) s += buf[k * 16 + threadIdx.x % 16];
    buf[threadIdx.x] = s;
  }
  __syncthreads();
  if (lane == 0 && col < 2 * a.c) {
    s = (buf[threadIdx.x] + buf[16 + threadIdx.x]) + (buf[32 + threadIdx.x] + buf[48 + threadIdx.x]);
    (col < a.c ? a.dw[col] : a.db[col - a.c]) = static_cast<float>(s);
  }
}

int row_lanes(int nvec) { return nvec <= 8 ? 8 : nvec <= 16 ? 16 : nvec <= 32 ? 32 : nvec <= 256 ? 64 : 256; }

template <typename T, int L, int R>
void run(const NormArgs& a, bool backward, hipStream_t s) {
  const int nv = a.c / a.groups / Pack<T>::N;
  const int mode = sum_mode(nv, a.groups, L);
  const int64_t want = (a.samples + NT / L - 1) / (NT / L);
  if (backward) {
    rows_bwd_kernel<T, L, R><<<static_cast<uint32_t>(a.sum_blocks), NT, 0, s>>>(a, mode);
    if (a.dw) rows_channels_kernel<<<(2 * a.c + 15) / 16, 1024, 0, s>>>(a);
  } else {
    rows_fwd_kernel<T, L, R><<<static_cast<uint32_t>(want < kRowBlocks ? want : kRowBlocks), NT, 0, s>>>(a, mode);
  }
}

template <typename T>
void run(const NormArgs& a, bool backward, hipStream_t s) {
  const int nvec = a.c / Pack<T>::N;
  if (nvec <= 8) run<T, 8, 1>(a, backward, s);
  else if (nvec <= 16) run<T, 16, 1>(a, backward, s);
  else if (nvec <= 32) run<T, 32, 1>(a, backward, s);
  else if (nvec <= 64) run<T, 64, 1>(a, backward, s);
  else if (nvec <= 128) run<T, 64, 2>(a, backward, s);
  else if (nvec <= 256) run<T, 64, 4>(a, backward, s);
  else if (nvec <= 512) run<T, 256, 2>(a, backward, s);
  else if (nvec <= 1024) run<T, 256, 4>(a, backward, s);
  else if constexpr (sizeof(T) == 4) run<T, 256, 8>(a, backward, s);      // at most 8192 channels
}

}  // namespace

// Single rows whose vectors lie whole in one group.
bool norm_rows_fit(const NormArgs& a) { return a.positions == 1 && (a.c / a.groups) % (a.type == QHA_F32 ? 4 : 8) == 0; }

int64_t norm_rows_blocks(const NormArgs& a) {
  const int teams = NT / row_lanes(a.c / (a.type == QHA_F32 ? 4 : 8));
  const int64_t want = (a.samples + teams - 1) / teams;
  return want < kGradBlocks ? want : kGradBlocks;
}

hipError_t launch_norm_rows(const NormArgs& a, bool backward, hipStream_t s) {
  if (a.type == QHA_F32) run<float>(a, backward, s);
  else if (a.type == QHA_BF16) run<__bf16>(a, backward, s);
  else run<_Float16>(a, backward, s);
  return hipGetLastError();
}

}  // namespace qha
