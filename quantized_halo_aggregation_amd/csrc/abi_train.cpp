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

bool known_type(int32_t t) { return t == QHA_F32 || t == QHA_BF16 || t == QHA_F16; }
uintptr_t type_bytes(int32_t t) { return t == QHA_F32 ? 4 : 2; }

}  // namespace

extern "C" {

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
    if (t.n < 0 || t.n > (1LL << 40)) return fail(QHA_ERR_INVALID_ARG, "tensor %lld: bad size", (long long)i);
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale)))
      return fail(QHA_ERR_INVALID_ARG, "tensor %lld: NULL pointer", (long long)i);
    if (!aligned(t.param, 4) || !aligned(t.grad, type_bytes(grad_type)) || !aligned(t.copy, type_bytes(copy_type)) ||
        (state_bits == 32 && (!aligned(t.m, 4) || !aligned(t.v, 4))) ||
        (state_bits == 8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
      return fail(QHA_ERR_INVALID_ARG, "tensor %lld: misaligned pointer", (long long)i);
    total += t.n;
    if (total > (1LL << 42)) return fail(QHA_ERR_INVALID_ARG, "too many elements");
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
      if (k > 0 && blocks + more > 0x7FFFFFFFLL) break;
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
  if (n < 0 || n > (1LL << 40)) return fail(QHA_ERR_INVALID_ARG, "bad size");
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
