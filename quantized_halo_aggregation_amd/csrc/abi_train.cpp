// C ABI of the training operators: host-side argument checks and kernel launches.
// Every check runs before anything is enqueued, so bad arguments never reach the GPU.
#include "../../include/qha.h"
#include "qha_internal.hpp"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>

using qha::fail;
using qha::ok;

namespace {

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(QHA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

constexpr int64_t kMaxRows = 2147483647LL;
constexpr int64_t kMaxWidth = 1 << 16;       // widths of a gated projection

bool known_type(int32_t t) { return t == QHA_F32 || t == QHA_BF16 || t == QHA_F16; }
uintptr_t type_bytes(int32_t t) { return t == QHA_F32 ? 4 : 2; }

}  // namespace

namespace {

// Checks the arguments both directions of the group norm share and fills the kernel arguments.
int take_norm(qha::NormArgs& a, int64_t n_samples, int64_t positions, int32_t c, int32_t n_groups, int32_t type,
              int32_t act, const float* weight, const float* bias) {
  std::memset(&a, 0, sizeof(a));
  if (n_samples < 0 || positions < 1 || n_samples > kMaxRows / positions) return fail(QHA_ERR_INVALID_ARG, "bad sizes");
  if (!known_type(type)) return fail(QHA_ERR_INVALID_ARG, "unknown element type %d", type);
  if (act < QHA_ACT_NONE || act > QHA_ACT_GELU) return fail(QHA_ERR_INVALID_ARG, "unknown activation %d", act);
  const int32_t vec = static_cast<int32_t>(16 / type_bytes(type));
  if (c < 1 || c % vec != 0) return fail(QHA_ERR_INVALID_ARG, "c=%d must be a multiple of %d", c, vec);
  if (c > 8192) return fail(QHA_ERR_UNSUPPORTED, "c=%d is above 8192", c);
  if (n_groups < 1 || c % n_groups != 0) return fail(QHA_ERR_INVALID_ARG, "%d groups do not divide c=%d", n_groups, c);
  if (!aligned(weight, 16) || !aligned(bias, 16)) return fail(QHA_ERR_INVALID_ARG, "weight / bias are not 16-byte aligned");
  a.samples = n_samples;
  a.positions = positions;
  a.c = c;
  a.groups = n_groups;
  a.type = type;
  a.act = act;
  a.w = weight;
  a.b = bias;
  return QHA_OK;
}

int check_rows(const char* name, const void* p, int64_t ld, int64_t c, int32_t type) {
  const int64_t vec = static_cast<int64_t>(16 / type_bytes(type));
  if (!p) return fail(QHA_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld < c || ld % vec != 0) return fail(QHA_ERR_INVALID_ARG, "%s: leading dimension %lld must be >= %lld and a multiple of %lld", name, (long long)ld, (long long)c, (long long)vec);
  if (!aligned(p, 16)) return fail(QHA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return QHA_OK;
}

int take_norm_workspace(qha::NormArgs& a, bool backward, void* ws, size_t bytes) {
  qha::norm_plan(a, backward);
  const size_t need = qha::norm_workspace(a, backward);
  if (need == 0) return QHA_OK;
  if (!ws || bytes < need) return fail(QHA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? bytes : (size_t)0);
  if (!aligned(ws, 16)) return fail(QHA_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  a.chan_part = static_cast<float*>(ws);
  const size_t chan = static_cast<size_t>(a.sum_blocks) * 2 * static_cast<size_t>(a.c) * sizeof(float);
  a.group_part = reinterpret_cast<double*>(static_cast<char*>(ws) + (chan + 15) / 16 * 16);
  return QHA_OK;
}

// Checks the arguments both directions of the residual norm share and fills the kernel arguments.
int take_residual(qha::ResidualArgs& a, int64_t n_rows, int64_t positions, int32_t c, int32_t stream_type, int32_t type,
                  int32_t post, int32_t pre, const float* const (&vectors)[4], double skip, double branch) {
  std::memset(&a, 0, sizeof(a));
  if (n_rows < 0 || n_rows > kMaxRows || positions < 1 || n_rows % positions != 0) return fail(QHA_ERR_INVALID_ARG, "bad sizes");
  if (!known_type(type)) return fail(QHA_ERR_INVALID_ARG, "unknown element type %d", type);
  if (stream_type != type && stream_type != QHA_F32) return fail(QHA_ERR_INVALID_ARG, "the stream's type %d is neither float32 nor %d", stream_type, type);
  if (post < QHA_ROW_NONE || post > QHA_ROW_LAYER || pre < QHA_ROW_NONE || pre > QHA_ROW_LAYER) return fail(QHA_ERR_INVALID_ARG, "unknown norm");
  const int32_t vec = static_cast<int32_t>(16 / type_bytes(type));
  if (c < 1 || c % vec != 0) return fail(QHA_ERR_INVALID_ARG, "c=%d must be a multiple of %d", c, vec);
  if (c > 8192) return fail(QHA_ERR_UNSUPPORTED, "c=%d is above 8192", c);
  if (!std::isfinite(static_cast<float>(skip)) || !std::isfinite(static_cast<float>(branch))) return fail(QHA_ERR_INVALID_ARG, "skip and branch must be finite in float32");
  for (const float* v : vectors)
    if (!aligned(v, 16)) return fail(QHA_ERR_INVALID_ARG, "a weight or bias is not 16-byte aligned");
  a.rows = n_rows;
  a.positions = positions;
  a.c = c;
  a.stream_type = stream_type;
  a.type = type;
  a.post = post;
  a.pre = pre;
  a.skip = static_cast<float>(skip);
  a.branch = static_cast<float>(branch);
  a.post_w = vectors[0];
  a.post_b = vectors[1];
  a.pre_w = vectors[2];
  a.pre_b = vectors[3];
  return QHA_OK;
}

}  // namespace

namespace {

int take_gated(qha::GatedArgs& g, int64_t m, int64_t n, int64_t k, int32_t type, int32_t act) {
  std::memset(&g, 0, sizeof(g));
  if (m < 0 || n < 0 || k < 0 || m > kMaxRows || n > kMaxWidth || k > kMaxWidth) return fail(QHA_ERR_INVALID_ARG, "bad sizes");
  if (!known_type(type)) return fail(QHA_ERR_INVALID_ARG, "unknown element type %d", type);
  if (act < QHA_ACT_NONE || act > QHA_ACT_GELU) return fail(QHA_ERR_INVALID_ARG, "unknown activation %d", act);
  const int64_t vec = static_cast<int64_t>(16 / type_bytes(type));
  if (n % vec || k % vec) return fail(QHA_ERR_INVALID_ARG, "n (%lld) and k (%lld) must be multiples of %lld", (long long)n, (long long)k, (long long)vec);
  // product tiles of 128 x 128 in one launch
  if ((m / 128 + 1) * (n / 64 + k / 128 + 2) > (1LL << 22)) return fail(QHA_ERR_UNSUPPORTED, "more than 2^22 tiles: cut the rows");
  g.m = m;
  g.n = n;
  g.k = k;
  g.type = type;
  g.act = act;
  return QHA_OK;
}

int take_gated_workspace(qha::GatedArgs& g, bool backward, void* ws, size_t bytes) {
  const size_t need = qha::gated_workspace(g.type, g.m, g.n, g.k, backward);
  if (need == 0) return QHA_OK;
  if (!ws || bytes < need) return fail(QHA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? bytes : (size_t)0);
  if (!aligned(ws, 16)) return fail(QHA_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  g.ws = ws;
  return QHA_OK;
}

constexpr int64_t kMaxSide = 1 << 16;       // rows and columns of a matrix to orthogonalise
constexpr double kMostCoefficient = 1e30;   // of a Newton-Schulz step: its products with the scales stay in float32's range

// The largest magnitude of f(r) = r (a + b r^2 + c r^4) on [0, 1]: at its end or where f' = a + 3 b t + 5 c t^2 = 0, t = r^2.
double largest_of(double a, double b, double c) {
  const auto f = [&](double r) { return std::fabs(r * (a + r * r * (b + r * r * c))); };
  double most = f(1.0);
  const double d = 9.0 * b * b - 20.0 * a * c;
  if (d < 0.0) return most;
  const double q = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));      // no difference of equals, whichever root is small
  for (double t : {q / (5.0 * c), a / q})
    if (t > 0.0 && t < 1.0) most = std::max(most, f(std::sqrt(t)));          // 0 / 0 and x / 0 are not
  return most;
}

// What a step (a, b, c) makes of singular values up to top: the largest |a + b s^2 + c s^4|, the largest value behind it, and the sum of
// its terms' sizes.
struct Reach {
  double inner, most, terms;
};
Reach reach_of(const double* k, double top) {
  // in units of top: with s = top r, a + b s^2 + c s^4 = a + (b top^2) r^2 + (c top^4) r^4
  const double t = top * top, a = k[0], b = k[1] * t, c = k[2] * t * t;
  Reach r = {std::max(std::fabs(a), std::fabs(a + b + c)), top * largest_of(a, b, c), std::fabs(a) + std::fabs(b) + std::fabs(c)};
  const double turn = -0.5 * (b / c);
  if (turn > 0.0 && turn < 1.0) r.inner = std::max(r.inner, std::fabs(a + 0.5 * b * turn));
  return r;
}

// The polynomials must keep X, A and B within the scaled parts' range, also where rounding takes a singular value past what the
// exact ones reach: a step's is taken for 2e-6 (16 units of float32) of its terms, and the next steps may grow it.  The bounds that X, A
// and B are scaled by allow for 16 times as much, or all that this check lets pass: steep steps of the largest matrices cannot overflow.
int check_steps(qha::NsArgs& args, int32_t steps, const double* coefficients, double eps) {
  constexpr double kRounding = 2e-6, kFar = 16.0, kMostX = 3.8, kMostB = 60.0;
  args.steps = steps;
  args.eps = eps;
  args.coefficients = coefficients;
  if (steps < 1 || steps > qha::kNsSteps) return fail(QHA_ERR_INVALID_ARG, "steps must lie in 1 .. %d, got %d", qha::kNsSteps, steps);
  if (!coefficients) return fail(QHA_ERR_INVALID_ARG, "coefficients is NULL");
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(QHA_ERR_INVALID_ARG, "eps must be finite and not negative");
  double top = 1.0, far = 1.0;
  args.most_x[0] = far;
  for (int32_t i = 0; i < steps; ++i) {
    const double* k = coefficients + 3 * i;
    for (int32_t e = 0; e < 3; ++e)
      if (!(std::fabs(k[e]) <= kMostCoefficient)) return fail(QHA_ERR_INVALID_ARG, "step %d: a coefficient is not finite or passes 1e30", i);
    const Reach r = reach_of(k, top), f = reach_of(k, far);
    if (!(r.inner <= kMostB)) return fail(QHA_ERR_INVALID_ARG, "step %d: a + b s^2 + c s^4 passes 60", i);
    if (!(r.most <= kMostX)) return fail(QHA_ERR_INVALID_ARG, "step %d: singular values pass 3.8", i);
    top = r.most + kRounding * top * r.terms;
    args.most_b[i] = std::min(f.inner + kFar * kRounding * f.terms, kMostB);
    args.most_x[i + 1] = far = std::min(f.most + kFar * kRounding * far * f.terms, kMostX);
  }
  return QHA_OK;
}

int check_sides(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return fail(QHA_ERR_INVALID_ARG, "a negative size");
  if (rows > kMaxSide || cols > kMaxSide) return fail(QHA_ERR_UNSUPPORTED, "%lld x %lld: more than 65536 rows or columns", (long long)rows, (long long)cols);
  return QHA_OK;
}

int check_ns_workspace(const qha::NsMatrix* m, int64_t n, const void* ws, size_t bytes) {
  const size_t need = qha::ns_workspace(m, n);
  if (need == 0) return QHA_OK;
  if (!ws || bytes < need) return fail(QHA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? bytes : (size_t)0);
  if (!aligned(ws, 16)) return fail(QHA_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  return QHA_OK;
}

// The library's list of a call's matrices; no exception crosses the C ABI.
std::unique_ptr<qha::NsMatrix[]> ns_list(int64_t n) {
  return std::unique_ptr<qha::NsMatrix[]>(n < (1LL << 32) ? new (std::nothrow) qha::NsMatrix[static_cast<size_t>(n)]() : nullptr);
}

}  // namespace

extern "C" {

size_t qha_gated_workspace(int32_t type, int64_t m, int64_t n, int64_t k, int32_t backward) {
  qha::GatedArgs g;
  if (take_gated(g, m, n, k, type, QHA_ACT_NONE) || n == 0 || k == 0) return 0;
  return qha::gated_workspace(type, m, n, k, backward != 0);
}

int qha_gated_project(int64_t m, int64_t n, int64_t k, int32_t type, const void* a, int64_t lda, const void* w_gate,
                      int64_t ldwg, const void* w_up, int64_t ldwu, int32_t act, void* h, int64_t ldh, void* gate,
                      int64_t ldg, void* up, int64_t ldu, void* workspace, size_t workspace_bytes, void* stream) {
  qha::GatedArgs g;
  int st = take_gated(g, m, n, k, type, act);
  if (st) return st;
  if ((gate == nullptr) != (up == nullptr)) return fail(QHA_ERR_INVALID_ARG, "gate and up come together");
  if (m == 0 || n == 0) return ok();
  if (k == 0) return fail(QHA_ERR_INVALID_ARG, "k = 0");
  if ((st = check_rows("a", a, lda, k, type)) || (st = check_rows("w_gate", w_gate, ldwg, k, type)) ||
      (st = check_rows("w_up", w_up, ldwu, k, type)) || (st = check_rows("h", h, ldh, n, type)))
    return st;
  if (gate && ((st = check_rows("gate", gate, ldg, n, type)) || (st = check_rows("up", up, ldu, n, type)))) return st;
  if ((st = take_gated_workspace(g, false, workspace, workspace_bytes))) return st;
  g.a = a;
  g.lda = lda;
  g.wg = w_gate;
  g.ldwg = ldwg;
  g.wu = w_up;
  g.ldwu = ldwu;
  g.h = h;
  g.ldh = ldh;
  g.gate_out = gate;
  g.up_out = up;
  g.ldg = ldg;
  g.ldu = ldu;
  return hip_status(qha::launch_gated_fwd(g, static_cast<hipStream_t>(stream)), "gated_project");
}

int qha_gated_backward(int64_t m, int64_t n, int64_t k, int32_t type, const void* dh, int64_t lddh, const void* gate,
                       int64_t ldg, const void* up, int64_t ldu, const void* a, int64_t lda, const void* w_gate,
                       int64_t ldwg, const void* w_up, int64_t ldwu, int32_t act, void* da, int64_t ldda, float* dw_gate,
                       int64_t lddwg, float* dw_up, int64_t lddwu, void* workspace, size_t workspace_bytes,
                       void* stream) {
  qha::GatedArgs g;
  int st = take_gated(g, m, n, k, type, act);
  if (st) return st;
  if (n == 0 || k == 0) return fail(QHA_ERR_INVALID_ARG, "n and k must be positive");
  if ((st = check_rows("w_gate", w_gate, ldwg, k, type)) || (st = check_rows("w_up", w_up, ldwu, k, type)) ||
      (st = check_rows("dw_gate", dw_gate, lddwg, k, QHA_F32)) || (st = check_rows("dw_up", dw_up, lddwu, k, QHA_F32)))
    return st;
  if (m > 0) {
    if ((st = check_rows("dh", dh, lddh, n, type)) || (st = check_rows("gate", gate, ldg, n, type)) ||
        (st = check_rows("up", up, ldu, n, type)) || (st = check_rows("a", a, lda, k, type)))
      return st;
    if (da && (st = check_rows("da", da, ldda, k, type))) return st;
  }
  if ((st = take_gated_workspace(g, true, workspace, workspace_bytes))) return st;
  g.dh = dh;
  g.lddh = lddh;
  g.gate = gate;
  g.ldg = ldg;
  g.up = up;
  g.ldu = ldu;
  g.a = a;
  g.lda = lda;
  g.wg = w_gate;
  g.ldwg = ldwg;
  g.wu = w_up;
  g.ldwu = ldwu;
  g.da = da;
  g.ldda = ldda;
  g.dwg = dw_gate;
  g.lddwg = lddwg;
  g.dwu = dw_up;
  g.lddwu = lddwu;
  return hip_status(qha::launch_gated_bwd(g, static_cast<hipStream_t>(stream)), "gated_backward");
}

size_t qha_group_norm_workspace(int64_t n_samples, int64_t positions, int32_t c, int32_t n_groups, int32_t backward) {
  if (n_samples <= 0 || positions <= 0 || n_samples > kMaxRows / positions || c <= 0 || c > 8192 || n_groups <= 0 || c % n_groups != 0) return 0;
  size_t need = 0;
  for (int32_t type : {QHA_F32, QHA_BF16}) {       // the element type is not asked for: room for each that c suits
    if (c % static_cast<int32_t>(16 / type_bytes(type)) != 0) continue;
    qha::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.samples = n_samples;
    a.positions = positions;
    a.c = c;
    a.groups = n_groups;
    a.type = type;
    qha::norm_plan(a, backward != 0);
    const size_t b = qha::norm_workspace(a, backward != 0);
    need = b > need ? b : need;
  }
  return need;
}

int qha_group_norm_fwd(int64_t n_samples, int64_t positions, int32_t c, int32_t n_groups, int32_t type, const void* x,
                       int64_t ldx, const float* weight, const float* bias, double eps, int32_t act, void* y,
                       int64_t ldy, float* mean, float* rstd, void* workspace, size_t workspace_bytes, void* stream) {
  qha::NormArgs a;
  int st = take_norm(a, n_samples, positions, c, n_groups, type, act, weight, bias);
  if (st) return st;
  if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(QHA_ERR_INVALID_ARG, "eps must be finite and not negative");
  if ((mean == nullptr) != (rstd == nullptr)) return fail(QHA_ERR_INVALID_ARG, "mean and rstd come together");
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return fail(QHA_ERR_INVALID_ARG, "mean / rstd misaligned");
  if (n_samples == 0) return ok();
  if ((st = check_rows("x", x, ldx, c, type)) || (st = check_rows("y", y, ldy, c, type))) return st;
  if ((st = take_norm_workspace(a, false, workspace, workspace_bytes))) return st;
  a.x = x;
  a.ldx = ldx;
  a.y = y;
  a.ldy = ldy;
  a.eps = eps;
  a.mean = mean;
  a.rstd = rstd;
  return hip_status(qha::launch_norm_fwd(a, static_cast<hipStream_t>(stream)), "group_norm_fwd");
}

int qha_group_norm_bwd(int64_t n_samples, int64_t positions, int32_t c, int32_t n_groups, int32_t type, const void* dy,
                       int64_t lddy, const void* x, int64_t ldx, const float* mean, const float* rstd,
                       const float* weight, const float* bias, int32_t act, void* dx, int64_t lddx, float* dweight,
                       float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  qha::NormArgs a;
  int st = take_norm(a, n_samples, positions, c, n_groups, type, act, weight, bias);
  if (st) return st;
  if ((dweight == nullptr) != (dbias == nullptr)) return fail(QHA_ERR_INVALID_ARG, "dweight and dbias come together");
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return fail(QHA_ERR_INVALID_ARG, "dweight / dbias misaligned");
  if (n_samples > 0) {
    if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return fail(QHA_ERR_INVALID_ARG, "mean / rstd out of contract");
    if ((st = check_rows("dy", dy, lddy, c, type)) || (st = check_rows("x", x, ldx, c, type)) ||
        (st = check_rows("dx", dx, lddx, c, type)))
      return st;
    if ((st = take_norm_workspace(a, true, workspace, workspace_bytes))) return st;
  } else if (!dweight) {
    return ok();
  }
  a.dy = dy;
  a.lddy = lddy;
  a.x = x;
  a.ldx = ldx;
  a.y = dx;
  a.ldy = lddx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dw = dweight;
  a.db = dbias;
  return hip_status(qha::launch_norm_bwd(a, static_cast<hipStream_t>(stream)), "group_norm_bwd");
}

size_t qha_residual_norm_workspace(int64_t n_rows, int64_t positions, int32_t c) {
  if (n_rows <= 0 || n_rows > kMaxRows || positions < 1 || n_rows % positions != 0 || c < 1 || c > 8192) return 0;
  size_t need = 0;
  for (int32_t type : {QHA_F32, QHA_BF16}) {       // the element type is not asked for: room for each that c suits
    if (c % static_cast<int32_t>(16 / type_bytes(type)) != 0) continue;
    for (int32_t gate = 0; gate < 2; ++gate) {
      qha::ResidualArgs a;
      std::memset(&a, 0, sizeof(a));
      a.rows = n_rows;
      a.positions = positions;
      a.c = c;
      a.type = type;
      a.shared_gate = gate && positions > 1;
      qha::residual_plan(a);
      const size_t b = qha::residual_workspace(a);
      need = b > need ? b : need;
    }
  }
  return need;
}

int qha_residual_norm_fwd(int64_t n_rows, int64_t positions, int32_t c, int32_t stream_type, int32_t type,
                          int32_t post, int32_t pre, const void* x, int64_t ldx, const void* h, int64_t ldh,
                          const void* gate, int64_t ldg, const float* post_weight, const float* post_bias,
                          const float* pre_weight, const float* pre_bias, double skip, double branch, double eps,
                          void* y, int64_t ldy, void* u, int64_t ldu, float* post_stats, float* pre_stats,
                          void* stream) {
  qha::ResidualArgs a;
  int st = take_residual(a, n_rows, positions, c, stream_type, type, post, pre, {post_weight, post_bias, pre_weight, pre_bias}, skip, branch);
  if (st) return st;
  if (!(eps >= 0.0) || !std::isfinite(static_cast<float>(eps))) return fail(QHA_ERR_INVALID_ARG, "eps must be finite in float32 and not negative");
  if (!aligned(post_stats, 8) || !aligned(pre_stats, 8)) return fail(QHA_ERR_INVALID_ARG, "statistics are not 8-byte aligned");
  if (pre == QHA_ROW_NONE && (u || pre_stats || pre_weight || pre_bias)) return fail(QHA_ERR_INVALID_ARG, "u, pre_stats or a pre vector without a pre norm");
  if (post == QHA_ROW_NONE && post_stats) return fail(QHA_ERR_INVALID_ARG, "post_stats without a post norm");
  if (!h && (post != QHA_ROW_NONE || pre == QHA_ROW_NONE || y || gate || post_weight || post_bias) && n_rows > 0)
    return fail(QHA_ERR_INVALID_ARG, "without h there is a pre norm alone: no y, gate, post norm or post vectors");
  if (n_rows == 0) return ok();
  if ((st = check_rows("x", x, ldx, c, stream_type))) return st;
  if (h && ((st = check_rows("h", h, ldh, c, type)) || (st = check_rows("y", y, ldy, c, stream_type)))) return st;
  if (gate && (st = check_rows("gate", gate, ldg, c, type))) return st;
  if (pre != QHA_ROW_NONE && (st = check_rows("u", u, ldu, c, type))) return st;
  a.eps = static_cast<float>(eps);
  a.x = x;
  a.ldx = ldx;
  a.h = h;
  a.ldh = ldh;
  a.gate = gate;
  a.ldg = ldg;
  a.y = y;
  a.ldy = ldy;
  a.u = u;
  a.ldu = ldu;
  a.post_stats = post_stats;
  a.pre_stats = pre_stats;
  return hip_status(qha::launch_residual(a, false, static_cast<hipStream_t>(stream)), "residual_norm_fwd");
}

int qha_residual_norm_bwd(int64_t n_rows, int64_t positions, int32_t c, int32_t stream_type, int32_t type,
                          int32_t post, int32_t pre, const void* dy, int64_t lddy, const void* du, int64_t lddu,
                          const void* y, int64_t ldy, const void* h, int64_t ldh, const void* gate, int64_t ldg,
                          const float* post_weight, const float* post_bias, const float* pre_weight, double skip,
                          double branch, const float* post_stats, const float* pre_stats, void* dx, int64_t lddx,
                          void* dh, int64_t lddh, void* dgate, int64_t lddg, float* dpost_weight, float* dpost_bias,
                          float* dpre_weight, float* dpre_bias, void* workspace, size_t workspace_bytes, void* stream) {
  qha::ResidualArgs a;
  int st = take_residual(a, n_rows, positions, c, stream_type, type, post, pre, {post_weight, post_bias, pre_weight, nullptr}, skip, branch);
  if (st) return st;
  float* const grads[4] = {dpost_weight, dpost_bias, dpre_weight, dpre_bias};
  for (float* v : grads)
    if (!aligned(v, 4)) return fail(QHA_ERR_INVALID_ARG, "a vector's gradient is misaligned");
  if (pre == QHA_ROW_NONE && (du || pre_stats || pre_weight || dpre_weight || dpre_bias)) return fail(QHA_ERR_INVALID_ARG, "du, pre_stats or a pre vector without a pre norm");
  if (post == QHA_ROW_NONE && post_stats) return fail(QHA_ERR_INVALID_ARG, "post_stats without a post norm");
  if (n_rows > 0) {
    if (!h && (post != QHA_ROW_NONE || pre == QHA_ROW_NONE || dh || gate || post_weight || post_bias || dpost_weight || dpost_bias))
      return fail(QHA_ERR_INVALID_ARG, "without h there is a pre norm alone: no dh, gate, post norm or post vectors");
    if (dgate && !gate) return fail(QHA_ERR_INVALID_ARG, "dgate without a gate");
    if (!dy && pre == QHA_ROW_NONE) return fail(QHA_ERR_INVALID_ARG, "dy is NULL");
    if (dy && (st = check_rows("dy", dy, lddy, c, stream_type))) return st;
    if ((st = check_rows("dx", dx, lddx, c, stream_type))) return st;
    if (h && ((st = check_rows("h", h, ldh, c, type)) || (st = check_rows("dh", dh, lddh, c, type)))) return st;
    if (gate && (st = check_rows("gate", gate, ldg, c, type))) return st;
    if (dgate && (st = check_rows("dgate", dgate, lddg, c, type))) return st;
    if (pre != QHA_ROW_NONE) {
      if ((st = check_rows("du", du, lddu, c, type)) || (st = check_rows("y", y, ldy, c, stream_type))) return st;
      if (!pre_stats || !aligned(pre_stats, 8)) return fail(QHA_ERR_INVALID_ARG, "pre_stats out of contract");
    }
    if (post != QHA_ROW_NONE && (!post_stats || !aligned(post_stats, 8))) return fail(QHA_ERR_INVALID_ARG, "post_stats out of contract");
  }
  bool partials = false;
  for (int i = 0; i < 4; ++i) {
    a.dvec[i] = grads[i];
    partials = partials || grads[i];
  }
  if (n_rows == 0 && !partials) return ok();
  a.shared_gate = n_rows > 0 && gate && positions > 1;
  qha::residual_plan(a);
  partials = n_rows > 0 && (partials || (a.shared_gate && dgate && a.chunks > 1));
  if (partials) {
    const size_t need = qha::residual_workspace(a);
    if (!workspace || workspace_bytes < need) return fail(QHA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : (size_t)0);
    if (!aligned(workspace, 16)) return fail(QHA_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    a.vec_part = static_cast<float*>(workspace);
    a.gate_part = a.vec_part + a.blocks * 4 * a.c;
  }
  if (!h) a.skip = 1.0f;             // without a block the forward's u is the norm of x itself, whatever skip is
  a.dy = dy;
  a.lddy = lddy;
  a.du = du;
  a.lddu = lddu;
  a.x = y;
  a.ldx = ldy;
  a.h = h;
  a.ldh = ldh;
  a.gate = gate;
  a.ldg = ldg;
  a.post_stats = const_cast<float*>(post_stats);
  a.pre_stats = const_cast<float*>(pre_stats);
  a.dx = dx;
  a.lddx = lddx;
  a.dh = dh;
  a.lddh = lddh;
  a.dgate = dgate;
  a.lddg = lddg;
  return hip_status(qha::launch_residual(a, true, static_cast<hipStream_t>(stream)), "residual_norm_bwd");
}

size_t qha_newton_schulz_workspace(const int64_t* sizes, int64_t n_matrices, int32_t steps) {
  if (!sizes || n_matrices <= 0 || steps < 1 || steps > qha::kNsSteps) return 0;
  const auto list = ns_list(n_matrices);
  if (!list) return 0;
  for (int64_t i = 0; i < n_matrices; ++i) {
    if (check_sides(sizes[2 * i], sizes[2 * i + 1])) return 0;
    list[i].rows = sizes[2 * i];
    list[i].cols = sizes[2 * i + 1];
  }
  return qha::ns_workspace(list.get(), n_matrices);
}

int qha_newton_schulz(const qha_ns_matrix* matrices, int64_t n_matrices, int32_t type, int32_t out_type, int32_t steps,
                      const double* coefficients, double eps, void* workspace, size_t workspace_bytes, void* stream) {
  if (n_matrices < 0) return fail(QHA_ERR_INVALID_ARG, "n_matrices < 0");
  if (!known_type(type) || !known_type(out_type)) return fail(QHA_ERR_INVALID_ARG, "unknown element type");
  qha::NsArgs a = {};
  int st = check_steps(a, steps, coefficients, eps);
  if (st) return st;
  if (n_matrices == 0) return ok();
  if (!matrices) return fail(QHA_ERR_INVALID_ARG, "matrices is NULL");
  const auto list = ns_list(n_matrices);
  if (!list) return fail(QHA_ERR_HIP, "no memory for %lld matrices", (long long)n_matrices);
  for (int64_t i = 0; i < n_matrices; ++i) {
    const qha_ns_matrix& m = matrices[i];
    if ((st = check_sides(m.rows, m.cols))) return st;
    if (m.rows == 0 || m.cols == 0) continue;
    if (!m.x || !m.out) return fail(QHA_ERR_INVALID_ARG, "matrix %lld: NULL pointer", (long long)i);
    if (m.ldx < m.cols || m.ldo < m.cols) return fail(QHA_ERR_INVALID_ARG, "matrix %lld: leading dimension below its %lld columns", (long long)i, (long long)m.cols);
    if (!aligned(m.x, type_bytes(type)) || !aligned(m.out, type_bytes(out_type))) return fail(QHA_ERR_INVALID_ARG, "matrix %lld: misaligned pointer", (long long)i);
    list[i].rows = m.rows;
    list[i].cols = m.cols;
    list[i].src = m.x;
    list[i].lds = m.ldx;
    list[i].dst = m.out;
    list[i].ldo = m.ldo;
  }
  if ((st = check_ns_workspace(list.get(), n_matrices, workspace, workspace_bytes))) return st;
  a.type = type;
  a.out_type = out_type;
  return hip_status(qha::launch_ns(list.get(), n_matrices, a, workspace, static_cast<hipStream_t>(stream)), "newton_schulz");
}

int qha_muon_step(const qha_muon_matrix* matrices, int64_t n_matrices, int32_t grad_type, int32_t copy_type, double lr,
                  double beta, int32_t nesterov, double weight_decay, double grad_scale, int32_t steps,
                  const double* coefficients, double eps, void* workspace, size_t workspace_bytes, void* stream) {
  if (n_matrices < 0) return fail(QHA_ERR_INVALID_ARG, "n_matrices < 0");
  if (!known_type(grad_type) || !known_type(copy_type)) return fail(QHA_ERR_INVALID_ARG, "unknown element type");
  if (!(lr >= 0.0) || !(weight_decay >= 0.0) || !std::isfinite(static_cast<float>(lr)) || !std::isfinite(static_cast<float>(lr * weight_decay)) ||
      !std::isfinite(weight_decay) || !std::isfinite(static_cast<float>(grad_scale)))
    return fail(QHA_ERR_INVALID_ARG, "lr and weight_decay must be finite and not negative, grad_scale finite");
  if (!(beta >= 0.0 && beta < 1.0)) return fail(QHA_ERR_INVALID_ARG, "beta must lie in [0, 1)");
  qha::NsArgs a = {};
  int st = check_steps(a, steps, coefficients, eps);
  if (st) return st;
  if (n_matrices == 0) return ok();
  if (!matrices) return fail(QHA_ERR_INVALID_ARG, "matrices is NULL");
  const auto list = ns_list(n_matrices);
  if (!list) return fail(QHA_ERR_HIP, "no memory for %lld matrices", (long long)n_matrices);
  for (int64_t i = 0; i < n_matrices; ++i) {
    const qha_muon_matrix& m = matrices[i];
    if ((st = check_sides(m.rows, m.cols))) return st;
    if (!(m.scale >= 0.0) || !std::isfinite(static_cast<float>(lr * m.scale))) return fail(QHA_ERR_INVALID_ARG, "matrix %lld: scale must be finite and not negative", (long long)i);
    if (m.rows == 0 || m.cols == 0) continue;
    if (!m.param || !m.grad || !m.momentum) return fail(QHA_ERR_INVALID_ARG, "matrix %lld: NULL pointer", (long long)i);
    if (!aligned(m.param, 4) || !aligned(m.momentum, 4) || !aligned(m.grad, type_bytes(grad_type)) || !aligned(m.copy, type_bytes(copy_type)))
      return fail(QHA_ERR_INVALID_ARG, "matrix %lld: misaligned pointer", (long long)i);
    list[i].rows = m.rows;
    list[i].cols = m.cols;
    list[i].src = m.grad;
    list[i].lds = list[i].ldo = m.cols;
    list[i].dst = m.param;
    list[i].mom = m.momentum;
    list[i].copy = m.copy;
    list[i].step = static_cast<float>(lr * m.scale);
  }
  if ((st = check_ns_workspace(list.get(), n_matrices, workspace, workspace_bytes))) return st;
  a.type = grad_type;
  a.out_type = copy_type;
  a.muon = 1;
  a.nesterov = nesterov != 0;
  a.mu = static_cast<float>(beta);
  a.grad_scale = static_cast<float>(grad_scale);
  a.decay = static_cast<float>(1.0 - lr * weight_decay);
  return hip_status(qha::launch_ns(list.get(), n_matrices, a, workspace, static_cast<hipStream_t>(stream)), "muon_step");
}

int qha_adamw_step(const qha_adamw_tensor* tensors, int64_t n_tensors, int32_t state_bits, int32_t grad_type,
                   int32_t copy_type, double lr, double beta1, double beta2, double eps, double weight_decay,
                   double grad_scale, int64_t step, void* stream) {
  if (n_tensors < 0) return fail(QHA_ERR_INVALID_ARG, "n_tensors < 0");
  if (state_bits != 8 && state_bits != 32) return fail(QHA_ERR_INVALID_ARG, "state_bits must be 8 or 32, got %d", state_bits);
  if (!known_type(grad_type) || !known_type(copy_type)) return fail(QHA_ERR_INVALID_ARG, "unknown element type");
  if (!(lr >= 0.0) || !std::isfinite(lr) || !(eps >= 0.0) || !std::isfinite(eps) || !(weight_decay >= 0.0) ||
      !std::isfinite(weight_decay) || !std::isfinite(grad_scale))
    return fail(QHA_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite and not negative, grad_scale finite");
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return fail(QHA_ERR_INVALID_ARG, "betas must lie in [0, 1)");
  if (step < 1) return fail(QHA_ERR_INVALID_ARG, "step counts from 1");
  if (n_tensors > 0 && !tensors) return fail(QHA_ERR_INVALID_ARG, "tensors is NULL");
  int64_t total = 0;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const qha_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (1LL << 35)) return fail(QHA_ERR_INVALID_ARG, "tensor %lld: bad size", (long long)i);
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale)))
      return fail(QHA_ERR_INVALID_ARG, "tensor %lld: NULL pointer", (long long)i);
    if (!aligned(t.param, 4) || !aligned(t.grad, type_bytes(grad_type)) || !aligned(t.copy, type_bytes(copy_type)) ||
        (state_bits == 32 && (!aligned(t.m, 4) || !aligned(t.v, 4))) ||
        (state_bits == 8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
      return fail(QHA_ERR_INVALID_ARG, "tensor %lld: misaligned pointer", (long long)i);
    total += t.n;
  }
  qha::AdamArgs a;
  std::memset(&a, 0, sizeof(a));
  a.grad_type = grad_type;
  a.copy_type = copy_type;
  const double c1 = 1.0 - std::pow(beta1, static_cast<double>(step));
  const double c2 = 1.0 - std::pow(beta2, static_cast<double>(step));
  a.decay = static_cast<float>(1.0 - lr * weight_decay);
  a.step_size = static_cast<float>(lr / c1);
  a.root_c2 = static_cast<float>(1.0 / std::sqrt(c2));
  a.eps = static_cast<float>(eps);
  a.grad_scale = static_cast<float>(grad_scale);
  a.beta1 = beta1;
  a.beta2 = beta2;
  a.passes = qha::adamw_passes(total);
  const int64_t chunk = 1024LL * a.passes;
  int64_t i = 0;
  while (i < n_tensors) {
    int32_t k = 0;
    int64_t blocks = 0;
    for (; i < n_tensors && k < qha::kAdamBatch; ++i) {
      const qha_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      const int64_t more = (t.n + chunk - 1) / chunk;
      if (k > 0 && blocks + more > qha::kMaxBlocks) break;
      a.t[k] = {t.n, t.param, t.grad, t.copy, t.m, t.v, t.m_scale, t.v_scale};
      a.first[k++] = static_cast<uint32_t>(blocks);
      blocks += more;
    }
    a.n_tensors = k;
    a.first[k] = static_cast<uint32_t>(blocks);
    if (k == 0) break;
    const int st = hip_status(qha::launch_adamw(a, state_bits, static_cast<hipStream_t>(stream)), "adamw_step");
    if (st) return st;
  }
  return ok();
}

int qha_adamw_values(const int8_t* m, const float* m_scale, float* m_out, const uint8_t* v, const float* v_scale,
                     float* v_out, int64_t n, void* stream) {
  if (n < 0 || n > (1LL << 33)) return fail(QHA_ERR_INVALID_ARG, "bad size");
  if (n == 0) return ok();
  const bool has_m = m || m_scale || m_out, has_v = v || v_scale || v_out;
  if ((has_m && !(m && m_scale && m_out)) || (has_v && !(v && v_scale && v_out))) return fail(QHA_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(m_scale, 4) || !aligned(v_scale, 4) || !aligned(m_out, 4) || !aligned(v_out, 4))
    return fail(QHA_ERR_INVALID_ARG, "misaligned pointer");
  if (!has_m && !has_v) return ok();
  return hip_status(qha::launch_adamw_values(m, m_scale, m_out, v, v_scale, v_out, n, static_cast<hipStream_t>(stream)),
                    "adamw_values");
}

}  // extern "C"
