// C ABI of the state-space block (include/zo_block.h): argument checks and
// dispatch.  Nothing here synchronises, allocates or keeps state.
#include "../../include/zo_block.h"

#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "zo_block_internal.h"
#include "zo_internal.h"

using namespace zo;

namespace {

inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// ZO_FAULT=launch: the calls return ZO_ERR_CUDA before they enqueue anything
// (the host-side fault injection of the other calls).
bool injected_launch() {
  const char* f = getenv("ZO_FAULT");
  return f && strcmp(f, "launch") == 0;
}

int device_ok() {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
    cudaGetLastError();
    return ZO_ERR_NO_DEVICE;
  }
  return major == 10 ? ZO_OK : ZO_ERR_NO_DEVICE;
}

int launched(cudaError_t e) { return e == cudaSuccess ? ZO_OK : ZO_ERR_CUDA; }

int elem_bytes(int dtype) { return dtype == ZO_DTYPE_FP32 ? 4 : 2; }
bool dtype_ok(int d) { return d == ZO_DTYPE_FP32 || d == ZO_DTYPE_BF16 || d == ZO_DTYPE_FP16; }

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool here(const zo_tensor& t, int bytes) { return t.ptr && aligned(t.ptr, bytes); }
bool maybe(const zo_tensor& t, int bytes) { return aligned(t.ptr, bytes); }
bool here(const zo_f32& t) { return t.ptr && aligned(t.ptr, 4); }
bool maybe(const zo_f32& t) { return aligned(t.ptr, 4); }

// Sets divide the rows; steps and channels leave 32-bit arithmetic room for a tile more.
bool shape_ok(int32_t rows, int32_t seq, int32_t channels, int32_t sets, int32_t dtype) {
  constexpr int32_t kMost = 1 << 30;
  return rows >= 1 && seq >= 1 && seq <= kMost && channels >= 1 && channels <= kMost && sets >= 1 &&
         rows % sets == 0 && dtype_ok(dtype);
}

// An output with several rows (steps) must not lay one over another.
bool apart(const zo_tensor& t, int64_t rows, int64_t seq, int64_t width) {
  if (!t.ptr) return true;
  const int64_t r = t.row < 0 ? -t.row : t.row, s = t.step < 0 ? -t.step : t.step;
  if (rows > 1 && r < width) return false;
  if (seq > 1 && s < width) return false;
  if (rows > 1 && seq > 1) return r >= s * (seq - 1) + width || s >= r * (rows - 1) + width;
  return true;
}

bool apart(const zo_f32& t, int64_t rows, int64_t width) {
  return !t.ptr || rows == 1 || (t.stride < 0 ? -t.stride : t.stride) >= width;
}

int conv_sizes(const zo_conv_args* a) {
  if (!a || !shape_ok(a->rows, a->seq, a->channels, a->sets, a->dtype) || a->taps < 1 ||
      (a->flags & ~ZO_CONV_SILU))
    return ZO_ERR_INVALID_ARG;
  return a->taps > ZO_MAX_TAPS ? ZO_ERR_UNSUPPORTED : ZO_OK;
}

int conv_check(const zo_conv_args* a) {
  const int rc = conv_sizes(a);
  if (rc) return rc;
  const int e = elem_bytes(a->dtype);
  if (!here(a->x, e) || !here(a->weight) || !maybe(a->bias) || !maybe(a->state_in, e) ||
      !aligned(a->lengths, 4) || !aligned(a->status, 4))
    return ZO_ERR_INVALID_ARG;
  return ZO_OK;
}

// zo_conv and zo_conv_step after their own checks
int conv_forward(const zo_conv_args* a, void* stream) {
  const int e = elem_bytes(a->dtype);
  const zo_tensor &si = a->state_in, &so = a->state_out;
  if (!here(a->out, e) || !maybe(so, e) || a->out.ptr == a->x.ptr ||
      !apart(a->out, a->rows, a->seq, a->channels) ||
      !apart(so, a->rows, a->taps - 1, a->channels))
    return ZO_ERR_INVALID_ARG;
  // in place only element for element
  if (so.ptr && so.ptr == si.ptr && (so.row != si.row || so.step != si.step))
    return ZO_ERR_INVALID_ARG;
  if (const int rc = device_ok()) return rc;
  if (injected_launch()) return ZO_ERR_CUDA;
  return launched(launch_conv(*a, S(stream)));
}

int scan_sizes(const zo_scan_args* a) {
  if (!a || !shape_ok(a->rows, a->seq, a->channels, a->sets, a->dtype) || a->groups < 1 ||
      a->channels % a->groups || a->states < 1 || (a->flags & ~ZO_SCAN_SOFTPLUS))
    return ZO_ERR_INVALID_ARG;
  return a->states > ZO_MAX_STATES ? ZO_ERR_UNSUPPORTED : ZO_OK;
}

int scan_check(const zo_scan_args* a) {
  const int rc = scan_sizes(a);
  if (rc) return rc;
  const int e = elem_bytes(a->dtype);
  if (!here(a->u, e) || !here(a->delta, e) || !maybe(a->z, e) || !here(a->B, e) ||
      !here(a->C, e) || !here(a->A) || !maybe(a->skip) || !maybe(a->delta_bias) ||
      !aligned(a->lengths, 4) || !aligned(a->status, 4) || !aligned(a->checkpoints, 16))
    return ZO_ERR_INVALID_ARG;
  return ZO_OK;
}

int scan_forward_check(const zo_scan_args* a) {
  const int e = elem_bytes(a->dtype);
  const zo_f32 &si = a->state_in, &so = a->state_out;
  const int64_t DN = (int64_t)a->channels * a->states;
  if (!here(a->out, e) || !maybe(si) || !maybe(so) || a->out.ptr == a->u.ptr ||
      a->out.ptr == a->delta.ptr || (a->z.ptr && a->out.ptr == a->z.ptr) ||
      !apart(a->out, a->rows, a->seq, a->channels) || !apart(so, a->rows, DN))
    return ZO_ERR_INVALID_ARG;
  if (so.ptr && so.ptr == si.ptr && so.stride != si.stride) return ZO_ERR_INVALID_ARG;
  return ZO_OK;
}

int norm_check(const zo_norm_args* a) {
  if (!a || !shape_ok(a->rows, 1, a->channels, a->sets, a->dtype) || !dtype_ok(a->x_dtype) ||
      (a->x_dtype != a->dtype && a->x_dtype != ZO_DTYPE_FP32) ||
      (a->flags & ~ZO_NORM_GATE_FIRST) || !(a->eps > 0.f) || !isfinite(a->eps))
    return ZO_ERR_INVALID_ARG;
  if (a->channels > ZO_MAX_NORM_WIDTH) return ZO_ERR_UNSUPPORTED;
  const int e = elem_bytes(a->dtype);
  if (!maybe(a->o, e) || !maybe(a->gate, e) || !maybe(a->w_post) || !maybe(a->scale) ||
      !maybe(a->w_pre))
    return ZO_ERR_INVALID_ARG;
  if (!a->o.ptr && (a->gate.ptr || a->w_post.ptr || a->scale.ptr)) return ZO_ERR_INVALID_ARG;
  // "the norm after the block" is what the flag orders
  if ((a->flags & ZO_NORM_GATE_FIRST) && !a->gate.ptr) return ZO_ERR_INVALID_ARG;
  return ZO_OK;
}

bool workspace_ok(const void* ws, int64_t have, int64_t need) {
  return need <= 0 || (ws && aligned(ws, 16) && have >= need);
}

}  // namespace

extern "C" {

int zo_conv(const zo_conv_args* a, void* stream) {
  const int rc = conv_check(a);
  if (rc) return rc;
  return conv_forward(a, stream);
}

int zo_conv_step(const zo_conv_args* a, void* stream) {
  const int rc = conv_check(a);
  if (rc) return rc;
  if (a->seq != 1 || (a->taps > 1 && !a->state_in.ptr)) return ZO_ERR_INVALID_ARG;
  zo_conv_args b = *a;
  b.lengths = nullptr;
  return conv_forward(&b, stream);
}

int64_t zo_conv_backward_workspace(const zo_conv_args* a) {
  return conv_sizes(a) ? -1 : conv_backward_workspace(*a);
}

int zo_conv_backward(const zo_conv_args* a, const zo_conv_grads* g, void* ws, int64_t ws_bytes,
                     void* stream) {
  const int rc = conv_check(a);
  if (rc) return rc;
  if (!g) return ZO_ERR_INVALID_ARG;
  const int e = elem_bytes(a->dtype);
  if (!here(g->dout, e) || !here(g->dx, e) || !here(g->dweight) || !maybe(g->dbias) ||
      !maybe(g->dstate_out, e) || !maybe(g->dstate_in, e) || g->dx.ptr == a->x.ptr ||
      g->dx.ptr == g->dout.ptr || !apart(g->dx, a->rows, a->seq, a->channels) ||
      !apart(g->dstate_in, a->rows, a->taps - 1, a->channels) ||
      !apart(g->dweight, a->sets, (int64_t)a->taps * a->channels) ||
      !apart(g->dbias, a->sets, a->channels) ||
      !workspace_ok(ws, ws_bytes, conv_backward_workspace(*a)))
    return ZO_ERR_INVALID_ARG;
  if (const int dc = device_ok()) return dc;
  if (injected_launch()) return ZO_ERR_CUDA;
  return launched(launch_conv_backward(*a, *g, static_cast<float*>(ws), S(stream)));
}

int64_t zo_scan_workspace(const zo_scan_args* a) {
  return scan_sizes(a) ? -1 : scan_workspace(*a);
}

int64_t zo_scan_backward_workspace(const zo_scan_args* a) {
  return scan_sizes(a) ? -1 : scan_backward_workspace(*a);
}

int zo_scan(const zo_scan_args* a, void* ws, int64_t ws_bytes, void* stream) {
  int rc = scan_check(a);
  if (!rc) rc = scan_forward_check(a);
  if (rc) return rc;
  if (!workspace_ok(ws, ws_bytes, scan_workspace(*a))) return ZO_ERR_INVALID_ARG;
  if (const int dc = device_ok()) return dc;
  if (injected_launch()) return ZO_ERR_CUDA;
  return launched(launch_scan(*a, static_cast<float*>(ws), S(stream)));
}

int zo_scan_step(const zo_scan_args* a, void* stream) {
  int rc = scan_check(a);
  if (!rc) rc = scan_forward_check(a);
  if (rc) return rc;
  if (a->seq != 1 || !a->state_in.ptr) return ZO_ERR_INVALID_ARG;
  if (const int dc = device_ok()) return dc;
  if (injected_launch()) return ZO_ERR_CUDA;
  return launched(launch_scan_step(*a, S(stream)));
}

int zo_scan_backward(const zo_scan_args* a, const zo_scan_grads* g, void* ws, int64_t ws_bytes,
                     void* stream) {
  const int rc = scan_check(a);
  if (rc) return rc;
  if (!g) return ZO_ERR_INVALID_ARG;
  const int e = elem_bytes(a->dtype);
  const int64_t D = a->channels, DN = D * a->states, GN = (int64_t)a->groups * a->states;
  if (!a->checkpoints || !here(g->dout, e) || !here(g->du, e) || !here(g->ddelta, e) ||
      !here(g->dB, e) || !here(g->dC, e) || !here(g->dA) || !maybe(g->dskip) ||
      !maybe(g->ddelta_bias) || !maybe(g->dstate_out) || !maybe(g->dstate_in) ||
      !maybe(g->dz, e) || (a->z.ptr != nullptr) != (g->dz.ptr != nullptr) ||
      (g->dskip.ptr && !a->skip.ptr) || (g->ddelta_bias.ptr && !a->delta_bias.ptr))
    return ZO_ERR_INVALID_ARG;
  if (!apart(g->du, a->rows, a->seq, D) || !apart(g->ddelta, a->rows, a->seq, D) ||
      !apart(g->dz, a->rows, a->seq, D) || !apart(g->dB, a->rows, a->seq, GN) ||
      !apart(g->dC, a->rows, a->seq, GN) || !apart(g->dA, a->sets, DN) ||
      !apart(g->dskip, a->sets, D) || !apart(g->ddelta_bias, a->sets, D) ||
      !apart(g->dstate_in, a->rows, DN) ||
      !workspace_ok(ws, ws_bytes, scan_backward_workspace(*a)))
    return ZO_ERR_INVALID_ARG;
  if (const int dc = device_ok()) return dc;
  if (injected_launch()) return ZO_ERR_CUDA;
  return launched(launch_scan_backward(*a, *g, static_cast<float*>(ws), S(stream)));
}

int zo_block_norm(const zo_norm_args* a, void* stream) {
  const int rc = norm_check(a);
  if (rc) return rc;
  const int e = elem_bytes(a->dtype), ex = elem_bytes(a->x_dtype);
  if (!here(a->x, ex) || !maybe(a->x_out, ex) || !maybe(a->n_out, e) ||
      (!a->x_out.ptr && !a->n_out.ptr) || (a->n_out.ptr != nullptr) != (a->w_pre.ptr != nullptr) ||
      !apart(a->x_out, a->rows, 1, a->channels) || !apart(a->n_out, a->rows, 1, a->channels))
    return ZO_ERR_INVALID_ARG;
  if (a->x_out.ptr && a->x_out.ptr == a->x.ptr && a->x_out.row != a->x.row && a->rows > 1)
    return ZO_ERR_INVALID_ARG;
  if (a->n_out.ptr && (a->n_out.ptr == a->x.ptr || a->n_out.ptr == a->o.ptr ||
                       a->n_out.ptr == a->gate.ptr || a->n_out.ptr == a->x_out.ptr))
    return ZO_ERR_INVALID_ARG;
  if (const int dc = device_ok()) return dc;
  if (injected_launch()) return ZO_ERR_CUDA;
  return launched(launch_norm(*a, S(stream)));
}

int64_t zo_block_norm_backward_workspace(const zo_norm_args* a) {
  return !a || !shape_ok(a->rows, 1, a->channels, a->sets, ZO_DTYPE_FP32) ||
                 a->channels > ZO_MAX_NORM_WIDTH
             ? -1
             : norm_backward_workspace(*a);
}

int zo_block_norm_backward(const zo_norm_args* a, const zo_norm_grads* g, void* ws,
                           int64_t ws_bytes, void* stream) {
  const int rc = norm_check(a);
  if (rc) return rc;
  if (!g) return ZO_ERR_INVALID_ARG;
  const int e = elem_bytes(a->dtype), ex = elem_bytes(a->x_dtype);
  auto paired = [](const void* p, const void* q) { return (p != nullptr) == (q != nullptr); };
  if (!here(a->x_out, ex) || !maybe(g->dn, e) || !maybe(g->dx_out, ex) || !here(g->dx, ex) ||
      !maybe(g->d_o, e) || !maybe(g->dgate, e) || !maybe(g->dw_post) || !maybe(g->dscale) ||
      !maybe(g->dw_pre) || (!g->dn.ptr && !g->dx_out.ptr) || !paired(g->dn.ptr, a->w_pre.ptr) ||
      !paired(g->dw_pre.ptr, a->w_pre.ptr) || !paired(g->d_o.ptr, a->o.ptr) ||
      !paired(g->dgate.ptr, a->gate.ptr) || !paired(g->dw_post.ptr, a->w_post.ptr) ||
      !paired(g->dscale.ptr, a->scale.ptr))
    return ZO_ERR_INVALID_ARG;
  if (!apart(g->dx, a->rows, 1, a->channels) || !apart(g->d_o, a->rows, 1, a->channels) ||
      !apart(g->dgate, a->rows, 1, a->channels) || !apart(g->dw_post, a->sets, a->channels) ||
      !apart(g->dscale, a->sets, a->channels) || !apart(g->dw_pre, a->sets, a->channels))
    return ZO_ERR_INVALID_ARG;
  if (g->dx.ptr == a->x_out.ptr || (g->dx.ptr == g->dx_out.ptr && a->rows > 1 &&
                                    g->dx.row != g->dx_out.row))
    return ZO_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, norm_backward_workspace(*a))) return ZO_ERR_INVALID_ARG;
  if (const int dc = device_ok()) return dc;
  if (injected_launch()) return ZO_ERR_CUDA;
  return launched(launch_norm_backward(*a, *g, static_cast<float*>(ws), S(stream)));
}

}  // extern "C"
