// Group normalisation of samples that fit in registers (single rows, small maps), and its gradients, in one pass.
//
// Mathematics: as in the two-launch form: y = act(w xhat + b), xhat = (x - mean) rstd per sample and group;
// dx = rstd (q - mean q - xhat mean(q xhat)) with q = w dy act'(.), dw = sum dz xhat, db = sum dz.
//
// Bound: memory, every array once.  A sample of at most 8192 values belongs to a team of L threads (8 to a
// wavefront's 64, or a whole block of 256 for large ones) that holds it in registers, R vectors of 16 bytes
// a thread, so the mean, the squares about it and the output come from one read.  Vector j of a sample is
// vector j % nvec of its row j / nvec, the same for every sample, so a thread's places, its w and b and
// (backward) its share of dw and db stay with it while the team walks over many samples with the next one's loads in
// flight.  Groups of a power of two of vectors in rows of a power of two are summed by exchanges between lanes,
// one group by all of the team, others through LDS.  A block leaves one partial of dw and db, and a second small
// launch adds those in float64.
// 300k rows of 128 float32 in 8 groups: forward 55 us (5.9 TB/s; a large copy reaches 5.0), 300k rows of 256
// backward 162 to 178 us (5.2 to 5.7 TB/s).
#include "act_common.hpp"
#include "qha_internal.hpp"

namespace qha {
namespace {

constexpr int NT = 256;
constexpr int64_t kRowBlocks = 2048;     // forward: eight blocks for each compute unit
constexpr int64_t kGradBlocks = 1024;    // backward: each leaves a partial of dw and db

enum { SUM_LANES = 0, SUM_ALL = 1, SUM_LDS = 2 };

bool power_of_two(int x) { return (x & (x - 1)) == 0; }

// How a group's vectors are summed: between lanes of a wavefront, all of the team's, or through LDS.
int sum_mode(int nvec, int nv, int groups, int lanes) {
  if (groups == 1) return SUM_ALL;
  return power_of_two(nv) && power_of_two(nvec) && nvec <= (lanes < 64 ? lanes : 64) && lanes <= 64 ? SUM_LANES : SUM_LDS;
}

// a[r] (one value per vector of the team's sample, 0 past its end) becomes its group's sum.  nv: vectors of a group in a
// row; group[r]: the vector's group, -1 past the sample's end.  lds: 2 R floats per thread of the block.
template <int L, int R, bool LDS>
__device__ __forceinline__ void group_sum(float (&a)[R], int mode, int positions, int nvec, int nv, const int (&group)[R],
                                          float* lds) {
  constexpr int W = L < 64 ? L : 64;
  const int ln = threadIdx.x % L;
  if (!LDS && mode == SUM_LANES) {
    for (int o = nv >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) a[r] += __shfl_xor(a[r], o, 64);
    if (positions == 1) return;            // rows of nvec lanes: the same group of other positions
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) t += a[r];
    for (int o = nvec; o < W; o <<= 1) t += __shfl_xor(t, o, 64);
#pragma unroll
    for (int r = 0; r < R; ++r) a[r] = t;
    return;
  }
  if (!LDS) {
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
  // the team's vectors to LDS; `subs` neighbouring lanes add a group's, by positions or within rows, whichever are more
  const int groups = nvec / nv;
  int subs = 1;
  while (2 * subs * groups <= L && subs < W) subs *= 2;
  const int sub = ln % subs;
  float* mine = lds + (threadIdx.x / L) * 2 * L * R;
  float* sums = mine + L * R;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) mine[ln + r * L] = a[r];
  __syncthreads();
  for (int g0 = 0; g0 < groups; g0 += L / subs) {
    const int g = g0 + ln / subs;
    float t = 0.0f;
    if (g < groups) {
      const float* at = mine + g * nv;
      if (positions >= nv) {
        for (int p = sub; p < positions; p += subs)
          for (int k = 0; k < nv; ++k) t += at[p * nvec + k];
      } else {
        for (int k = sub; k < nv; k += subs)
          for (int p = 0; p < positions; ++p) t += at[p * nvec + k];
      }
    }
    for (int o = subs >> 1; o > 0; o >>= 1) t += __shfl_xor(t, o, 64);
    if (sub == 0 && g < groups) sums[g] = t;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (group[r] >= 0) a[r] = sums[group[r]];
}

// Thread `ln` of a team: the places of its vectors in a sample.
template <int L, int R, int V>
struct Places {
  int count, nvec, nv;          // vectors of a sample, of a row, of a group in a row
  int64_t pos[R];               // row in the sample
  int vec[R];                   // vector in the row
  int group[R];                 // its group
  bool in[R];
  __device__ __forceinline__ explicit Places(const NormArgs& a) {
    nvec = a.c / V;
    nv = nvec / a.groups;
    count = static_cast<int>(a.positions) * nvec;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int j = static_cast<int>(threadIdx.x) % L + r * L;
      in[r] = j < count;
      pos[r] = j / nvec;
      vec[r] = j % nvec;
      group[r] = in[r] ? vec[r] / nv : -1;
    }
  }
};

template <typename T, int L, int R, bool LDS>
__global__ __launch_bounds__(NT) void rows_fwd_kernel(NormArgs a, int mode) {
  constexpr int V = Pack<T>::N;
  typedef typename Pack<T>::wide wide;
  __shared__ float lds[2 * NT * R];
  const Places<L, R, V> at(a);
  const int positions = static_cast<int>(a.positions);
  const float n = static_cast<float>(positions * (a.c / a.groups));
  const int team = threadIdx.x / L;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (NT / L);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (NT / L);
  wide w[R], b[R];
  const T* xp[R];
  T* yp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    xp[r] = static_cast<const T*>(a.x) + ((first + team) * a.positions + at.pos[r]) * a.ldx + at.vec[r] * V;
    yp[r] = static_cast<T*>(a.y) + ((first + team) * a.positions + at.pos[r]) * a.ldy + at.vec[r] * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[r][v] = a.w && at.in[r] ? a.w[at.vec[r] * V + v] : 1.0f;
      b[r][v] = a.b && at.in[r] ? a.b[at.vec[r] * V + v] : 0.0f;
    }
  }
  // every team of the block takes the same number of turns (the LDS sums meet at barriers)
  wide next[R];
  const int64_t x_step = step * a.positions * a.ldx, y_step = step * a.positions * a.ldy;
  auto fetch = [&](int64_t sample) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      next[r] = 0.0f;
      if (sample < a.samples && at.in[r]) next[r] = Pack<T>::load(xp[r]);
      xp[r] += x_step;
    }
  };
  fetch(first + team);
  for (int64_t turn = first; turn < a.samples; turn += step) {
    const int64_t sample = turn + team;
    wide x[R];
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = next[r];
      s[r] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) s[r] += x[r][v];
    }
    fetch(sample + step);
    group_sum<L, R, LDS>(s, mode, positions, at.nvec, at.nv, at.group, lds);
    float mean[R], q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = s[r] / n;          // a quotient: groups of one value have exactly that mean
      q[r] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float d = x[r][v] - mean[r];
        q[r] += at.in[r] ? d * d : 0.0f;
      }
    }
    group_sum<L, R, LDS>(q, mode, positions, at.nvec, at.nv, at.group, lds);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      T* to = yp[r];
      yp[r] += y_step;
      if (sample >= a.samples || !at.in[r]) continue;
      const float rstd = 1.0f / sqrtf(q[r] / n + static_cast<float>(a.eps));
      wide y;
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = activate((x[r][v] - mean[r]) * rstd * w[r][v] + b[r][v], a.act);
      Pack<T>::store(to, y);
      if (a.mean && at.pos[r] == 0 && at.vec[r] == at.group[r] * at.nv) {
        a.mean[sample * a.groups + at.group[r]] = mean[r];
        a.rstd[sample * a.groups + at.group[r]] = rstd;
      }
    }
  }
}

template <typename T, int L, int R, bool LDS>
__global__ __launch_bounds__(NT) void rows_bwd_kernel(NormArgs a, int mode) {
  constexpr int V = Pack<T>::N;
  typedef typename Pack<T>::wide wide;
  __shared__ float lds[4 * NT * R];
  const Places<L, R, V> at(a);
  const int positions = static_cast<int>(a.positions);
  const float inv = 1.0f / static_cast<float>(positions * (a.c / a.groups));
  wide w[R], b[R], dw[R], db[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    dw[r] = db[r] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[r][v] = a.w && at.in[r] ? a.w[at.vec[r] * V + v] : 1.0f;
      b[r][v] = a.b && at.in[r] ? a.b[at.vec[r] * V + v] : 0.0f;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * (NT / L);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (NT / L);
  wide next_x[R], next_dy[R];
  float next_mean[R], next_rstd[R];
  auto fetch = [&](int64_t sample) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      next_x[r] = next_dy[r] = 0.0f;
      next_mean[r] = next_rstd[r] = 0.0f;
      if (sample < a.samples && at.in[r]) {
        const int64_t row = sample * a.positions + at.pos[r];
        next_x[r] = Pack<T>::load(static_cast<const T*>(a.x) + row * a.ldx + at.vec[r] * V);
        next_dy[r] = Pack<T>::load(static_cast<const T*>(a.dy) + row * a.lddy + at.vec[r] * V);
        next_mean[r] = a.mean[sample * a.groups + at.group[r]];
        next_rstd[r] = a.rstd[sample * a.groups + at.group[r]];
      }
    }
  };
  const int team = threadIdx.x / L;
  fetch(first + team);
  for (int64_t turn = first; turn < a.samples; turn += step) {
    const int64_t sample = turn + team;
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
    fetch(sample + step);
    group_sum<L, R, LDS>(s0, mode, positions, at.nvec, at.nv, at.group, lds);
    group_sum<L, R, LDS>(s1, mode, positions, at.nvec, at.nv, at.group, lds + 2 * NT * R);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (sample >= a.samples || !at.in[r]) continue;
      wide dx;
#pragma unroll
      for (int v = 0; v < V; ++v) dx[v] = rstd[r] * (q[r][v] - s0[r] * inv - xhat[r][v] * (s1[r] * inv));
      Pack<T>::store(static_cast<T*>(a.y) + (sample * a.positions + at.pos[r]) * a.ldy + at.vec[r] * V, dx);
    }
  }
  if (!a.dw) return;
  // Vector `vec` of a row is vector j of a sample for every j = vec (mod nvec): the block's shares of it lie in
  // lanes j - r L of each team.  Neighbouring lanes add them.
  constexpr int TEAMS = NT / L;
  float* out = a.chan_part + static_cast<int64_t>(blockIdx.x) * 2 * a.c;
  float* buf_w = lds;
  float* buf_b = lds + NT * R;
  int subs = 1;
  while (subs < 64 && 2 * subs * at.nvec <= NT) subs *= 2;
  const int sub = threadIdx.x % subs;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      buf_w[r * NT + threadIdx.x] = at.in[r] ? dw[r][v] : 0.0f;
      buf_b[r * NT + threadIdx.x] = at.in[r] ? db[r][v] : 0.0f;
    }
    __syncthreads();
    for (int vec0 = 0; vec0 < at.nvec; vec0 += NT / subs) {
      const int vec = vec0 + threadIdx.x / subs;
      float s = 0.0f, q = 0.0f;
      if (vec < at.nvec)
        for (int e = sub; e < positions * TEAMS; e += subs) {
          const int j = vec + e / TEAMS * at.nvec, k = e % TEAMS;
          s += buf_w[j / L * NT + k * L + j % L];
          q += buf_b[j / L * NT + k * L + j % L];
        }
      for (int o = subs >> 1; o > 0; o >>= 1) {
        s += __shfl_xor(s, o, 64);
        q += __shfl_xor(q, o, 64);
      }
      if (sub == 0 && vec < at.nvec) {
        out[vec * V + v] = s;
        out[a.c + vec * V + v] = q;
      }
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

int team_lanes(int count) { return count <= 8 ? 8 : count <= 16 ? 16 : count <= 32 ? 32 : count <= 256 ? 64 : 256; }

int row_vectors(const NormArgs& a) { return a.c / (a.type == QHA_F32 ? 4 : 8); }

template <typename T, int L, int R, bool LDS>
void run(const NormArgs& a, bool backward, int mode, hipStream_t s) {
  const int64_t want = (a.samples + NT / L - 1) / (NT / L);
  if (backward) {
    rows_bwd_kernel<T, L, R, LDS><<<static_cast<uint32_t>(a.sum_blocks), NT, 0, s>>>(a, mode);
    if (a.dw) rows_channels_kernel<<<(2 * a.c + 15) / 16, 1024, 0, s>>>(a);
  } else {
    rows_fwd_kernel<T, L, R, LDS><<<static_cast<uint32_t>(want < kRowBlocks ? want : kRowBlocks), NT, 0, s>>>(a, mode);
  }
}

// Sums through LDS are kernels of their own: beside them the others run slower (forward of 300k x 128 76 against 62 us).
template <typename T, int L, int R>
void run(const NormArgs& a, bool backward, hipStream_t s) {
  const int nvec = row_vectors(a);
  const int mode = sum_mode(nvec, nvec / a.groups, a.groups, L);
  if (mode == SUM_LDS) run<T, L, R, true>(a, backward, mode, s);
  else run<T, L, R, false>(a, backward, mode, s);
}

template <typename T>
void run(const NormArgs& a, bool backward, hipStream_t s) {
  const int count = static_cast<int>(a.positions) * row_vectors(a);
  if (count <= 8) run<T, 8, 1>(a, backward, s);
  else if (count <= 16) run<T, 16, 1>(a, backward, s);
  else if (count <= 32) run<T, 32, 1>(a, backward, s);
  else if (count <= 64) run<T, 64, 1>(a, backward, s);
  else if (count <= 128) run<T, 64, 2>(a, backward, s);
  else if (count <= 256) run<T, 64, 4>(a, backward, s);
  else if (count <= 512) run<T, 256, 2>(a, backward, s);
  else if (count <= 1024) run<T, 256, 4>(a, backward, s);
  else if constexpr (sizeof(T) == 4) run<T, 256, 8>(a, backward, s);      // at most 8192 values
}

}  // namespace

// Samples of at most 8192 values whose vectors lie whole in one group; of more than 256 vectors (a block each) only
// single rows, or many: a few blocks alone take longer than two launches that share the rows out (3 samples of
// 97 x 64 f16 backward, 24 against 19 us).
bool norm_rows_fit(const NormArgs& a) {
  if (a.positions > 8192 / a.c || (a.c / a.groups) % (a.type == QHA_F32 ? 4 : 8) != 0) return false;
  return a.positions == 1 || a.positions * row_vectors(a) <= 256 || a.samples >= 256;
}

int64_t norm_rows_blocks(const NormArgs& a) {
  const int teams = NT / team_lanes(static_cast<int>(a.positions) * row_vectors(a));
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
