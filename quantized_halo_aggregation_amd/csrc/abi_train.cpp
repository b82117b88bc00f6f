// C ABI of the training operators: host-side argument checks and kernel launches.
// Every check runs before anything is enqueued, so bad arguments never reach the GPU.
#include "../../include/qha.h"
#include "qha_internal.hpp"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

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
