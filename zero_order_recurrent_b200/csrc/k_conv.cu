// Short causal convolution over time, pre_t = b + sum_k w[k] x_{t-K+1+k} per
// channel, with its SiLU; its gradients; and the fixed-order sum of partial
// results that the block's backward passes share.
//
// Bound: memory.  The forward reads x and writes out once (2 K + 6 flops for 2
// values moved), the backward reads x and dout and writes dx.  A thread owns V
// neighbouring channels (16 bytes of a row in the forward, 8 in the backward,
// which keeps twice the windows) and walks a run of steps with the window in
// registers, so x is read once per run plus K - 1 steps of overlap.
#include "zo_block.cuh"
#include "zo_block_internal.h"
#include "zo_internal.h"

namespace zo {
namespace {

constexpr int kThreads = 128;

struct ConvDims {
  int64_t T;
  int D, rows_per_set, run, runs, ctiles;
};

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t row, int64_t T,
                                              int32_t* status, bool tell) {
  if (!lengths) return T;
  const int64_t n = lengths[row];
  if (n >= 0 && n <= T) return n;
  if (status && tell) *status = ZO_ERR_BOUNDS;
  return n < 0 ? 0 : T;
}

// The window value at step p (may be before 0): x, or the carried state, or 0.
template <class T, int V, int K>
__device__ __forceinline__ void load_step(const T* x, int64_t x_step, const T* s, int64_t s_step,
                                          int64_t p, int64_t len, float (&f)[V]) {
  if (p >= 0 && p < len) {
    load_vec<T, V>(x + p * x_step, f);
  } else if (p < 0 && s) {
    load_vec<T, V>(s + (p + K - 1) * s_step, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
  }
}

// U steps at a time: their loads are issued together.
template <class T, int V, int K, int U>
__global__ void __launch_bounds__(kThreads)
    conv_kernel(zo_conv_args a, ConvDims d) {
  const int ct = blockIdx.x % d.ctiles;
  const int64_t rest = blockIdx.x / d.ctiles;
  const int run = (int)(rest % d.runs);
  const int64_t row = rest / d.runs;
  const int64_t c = ((int64_t)ct * kThreads + threadIdx.x) * V;
  if (c >= d.D) return;
  const int64_t len = row_length(a.lengths, row, d.T, a.status, run == 0 && c == 0);
  const T* x = static_cast<const T*>(a.x.ptr) + row * a.x.row + c;
  const T* s = a.state_in.ptr ? static_cast<const T*>(a.state_in.ptr) + row * a.state_in.row + c
                              : nullptr;
  T* out = static_cast<T*>(a.out.ptr) + row * a.out.row + c;
  const int64_t set = row / d.rows_per_set;
  float w[K][V], b[V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) w[k][i] = a.weight.ptr[set * a.weight.stride + (int64_t)k * d.D + c + i];
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = a.bias.ptr ? a.bias.ptr[set * a.bias.stride + c + i] : 0.f;
  const int64_t t0 = (int64_t)run * d.run;
  const int64_t t1 = t0 + d.run < d.T ? t0 + d.run : d.T;
  float win[K - 1 + U][V];
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    load_step<T, V, K>(x, a.x.step, s, a.state_in.step, t0 - (K - 1) + j, len, win[j]);
  const bool silu = a.flags & ZO_CONV_SILU;
  for (int64_t t = t0; t < t1; t += U) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      load_step<T, V, K>(x, a.x.step, s, a.state_in.step, t + j, len, win[K - 1 + j]);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (t + j >= t1) break;
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float p = b[i];
#pragma unroll
        for (int k = 0; k < K; ++k) p = fmaf(w[k][i], win[j + k][i], p);
        y[i] = t + j < len ? (silu ? silu_f(p) : p) : 0.f;
      }
      store_vec<T, V>(out + (t + j) * a.out.step, y);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) win[j][i] = win[U + j][i];
  }
  // The window after the row's last step.  Only the first run reads state_in, so
  // the same thread may write it in place: all loads come before the stores.
  if (K > 1 && run == 0 && a.state_out.ptr) {
    T* so = static_cast<T*>(a.state_out.ptr) + row * a.state_out.row + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      load_step<T, V, K>(x, a.x.step, s, a.state_in.step, len - (K - 1) + j, len, win[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_vec<T, V>(so + j * a.state_out.step, win[j]);
  }
}

// d_t = dout_t silu'(pre_t);  dx_p = sum_k w[k] d_{p+K-1-k} (+ what state_out's
// gradient sends to p);  dw[k] += d_t x_{t-K+1+k};  db += d_t.
// The run of steps [t0, t1) owns d_t for the sums, and gives dx_p for
// p = t - (K - 1), t in [t0, t1 + K - 1 if it is the last run): p < 0 is the
// carried window's gradient.
template <class T, int V, int K, int U>
__global__ void __launch_bounds__(kThreads)
    conv_backward_kernel(zo_conv_args a, zo_conv_grads g, ConvDims d, float* part) {
  const int ct = blockIdx.x % d.ctiles;
  const int64_t rest = blockIdx.x / d.ctiles;
  const int run = (int)(rest % d.runs);
  const int64_t row = rest / d.runs;
  const int64_t c = ((int64_t)ct * kThreads + threadIdx.x) * V;
  if (c >= d.D) return;
  const int64_t len = row_length(a.lengths, row, d.T, a.status, run == 0 && c == 0);
  const T* x = static_cast<const T*>(a.x.ptr) + row * a.x.row + c;
  const T* s = a.state_in.ptr ? static_cast<const T*>(a.state_in.ptr) + row * a.state_in.row + c
                              : nullptr;
  const T* dout = static_cast<const T*>(g.dout.ptr) + row * g.dout.row + c;
  const T* dso = g.dstate_out.ptr
                     ? static_cast<const T*>(g.dstate_out.ptr) + row * g.dstate_out.row + c
                     : nullptr;
  T* dx = static_cast<T*>(g.dx.ptr) + row * g.dx.row + c;
  T* dsi = g.dstate_in.ptr ? static_cast<T*>(g.dstate_in.ptr) + row * g.dstate_in.row + c : nullptr;
  const int64_t set = row / d.rows_per_set;
  float w[K][V], b[V], dw[K][V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    b[i] = a.bias.ptr ? a.bias.ptr[set * a.bias.stride + c + i] : 0.f;
    db[i] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k][i] = a.weight.ptr[set * a.weight.stride + (int64_t)k * d.D + c + i];
      dw[k][i] = 0.f;
    }
  }
  const bool silu = a.flags & ZO_CONV_SILU;
  const int64_t t0 = (int64_t)run * d.run;
  const int64_t t1 = t0 + d.run < d.T ? t0 + d.run : d.T;
  // dx_p for p in [p0, p1): the first run begins with the carried window
  const int64_t p0 = run == 0 ? -(K - 1) : t0, p1 = t1;
  float xw[K - 1 + U][V], dd[K - 1 + U][V];  // x_{t-K+1..}, d_{t-K+1..}
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    load_step<T, V, K>(x, a.x.step, s, a.state_in.step, t0 - (K - 1) + j, len, xw[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) dd[j][i] = 0.f;
  }
  for (int64_t t = t0; t < t1 + K - 1; t += U) {
    float dy[U][V];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      load_step<T, V, K>(x, a.x.step, s, a.state_in.step, t + j, len, xw[K - 1 + j]);
      if (t + j < len) {
        load_vec<T, V>(dout + (t + j) * g.dout.step, dy[j]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) dy[j][i] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const bool mine = t + j < t1, on = t + j < len;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float p = b[i];
#pragma unroll
        for (int k = 0; k < K; ++k) p = fmaf(w[k][i], xw[j + k][i], p);
        const float v = on ? dy[j][i] * (silu ? dsilu_f(p) : 1.f) : 0.f;
        dd[K - 1 + j][i] = v;
        if (mine && on) {
          db[i] += v;
#pragma unroll
          for (int k = 0; k < K; ++k) dw[k][i] = fmaf(v, xw[j + k][i], dw[k][i]);
        }
      }
      const int64_t p = t + j - (K - 1);
      if (p >= p0 && p < p1) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) v = fmaf(w[k][i], dd[j + K - 1 - k][i], v);
          o[i] = v;
        }
        const int64_t q = p + K - 1 - len;  // which of the last inputs, if any
        if (dso && q >= 0 && q < K - 1) {
          float e[V];
          load_vec<T, V>(dso + q * g.dstate_out.step, e);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += e[i];
        }
        if (p >= 0) {
          store_vec<T, V>(dx + p * g.dx.step, o);
        } else if (dsi) {
          store_vec<T, V>(dsi + (p + K - 1) * g.dstate_in.step, o);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xw[j][i] = xw[U + j][i];
        dd[j][i] = dd[U + j][i];
      }
  }
  // partial sums of this run: [set][row of set, run][K + 1][D]
  float* out = part + ((set * d.rows_per_set + row % d.rows_per_set) * d.runs + run) * (K + 1) * d.D + c;
#pragma unroll
  for (int k = 0; k < K; ++k) store_vec<float, V>(out + (int64_t)k * d.D, dw[k]);
  store_vec<float, V>(out + (int64_t)K * d.D, db);
}

struct SumOuts {
  float* out[3];
  int64_t stride[3], n[3];
};

// 32 neighbouring values a block, by G warps that take every G-th part, eight loads at a time.
template <int G>
__global__ void __launch_bounds__(32 * G)
    sum_parts_kernel(const float* part, int64_t parts, int64_t n, SumOuts o) {
  __shared__ float sh[G][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane, set = blockIdx.y;
  const float* p = part + set * parts * n + i;
  float s = 0.f;
  if (i < n) {
    int64_t k = grp;
    for (; k + 7 * G < parts; k += 8 * G) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[(k + j * G) * n];
#pragma unroll
      for (int j = 4; j > 0; j /= 2)
#pragma unroll
        for (int m = 0; m < j; ++m) v[m] += v[m + j];
      s += v[0];
    }
    for (; k < parts; k += G) s += p[k * n];
  }
  sh[grp][lane] = s;
  __syncthreads();
  if (grp == 0 && i < n) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) v += sh[k][lane];
    int64_t j = i;
    int w = 0;
    while (w < 2 && j >= o.n[w]) j -= o.n[w++];
    if (o.out[w]) o.out[w][set * o.stride[w] + j] = v;
  }
}

// Steps of one run: whole rows where there are rows enough for about eight
// blocks an SM, else as many runs as give that, but not under 16 steps (and so
// never under the K - 1 steps by which neighbouring runs overlap).
ConvDims conv_dims(const zo_conv_args& a, int v) {
  ConvDims d;
  d.T = a.seq;
  d.D = a.channels;
  d.rows_per_set = a.rows / a.sets;
  d.ctiles = (int)ceil_div(ceil_div(a.channels, v), kThreads);
  const int64_t want = ceil_div(8 * kBlockSMs, (int64_t)d.ctiles * a.rows);
  int64_t run = ceil_div(a.seq, want);
  if (run < 16) run = 16;
  d.run = (int)run;
  d.runs = (int)ceil_div(a.seq, run);
  return d;
}

// As conv_dims for the backward pass, whose partial sums are laid out by run:
// v = 1, so that the workspace does not go by alignment.
ConvDims conv_backward_dims(const zo_conv_args& a, int v) {
  ConvDims d = conv_dims(a, 4);
  d.ctiles = (int)ceil_div(ceil_div(a.channels, v), kThreads);
  return d;
}

template <class T, int V, int K>
cudaError_t run_conv(const zo_conv_args& a, cudaStream_t st) {
  const ConvDims d = conv_dims(a, V);
  const int64_t blocks = (int64_t)d.ctiles * d.runs * a.rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  conv_kernel<T, V, K, 4><<<(unsigned)blocks, kThreads, 0, st>>>(a, d);
  count_launch();
  return cudaGetLastError();
}

template <class T, int V, int K>
cudaError_t run_conv_backward(const zo_conv_args& a, const zo_conv_grads& g, float* ws,
                              cudaStream_t st) {
  const ConvDims d = conv_backward_dims(a, V);
  const int64_t blocks = (int64_t)d.ctiles * d.runs * a.rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  conv_backward_kernel<T, V, K, 4><<<(unsigned)blocks, kThreads, 0, st>>>(a, g, d, ws);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const SumOut outs[2] = {{g.dweight, (int64_t)K * d.D}, {g.dbias, d.D}};
  return launch_sum_parts(ws, a.sets, (int64_t)d.rows_per_set * d.runs, (int64_t)(K + 1) * d.D, outs, 2, st);
}

template <template <class, int, int> class F, class T, int V, class... A>
cudaError_t by_taps(int taps, A&&... x) {
  switch (taps) {
    case 1: return F<T, V, 1>::run(x...);
    case 2: return F<T, V, 2>::run(x...);
    case 3: return F<T, V, 3>::run(x...);
    case 4: return F<T, V, 4>::run(x...);
    case 5: return F<T, V, 5>::run(x...);
    case 6: return F<T, V, 6>::run(x...);
    case 7: return F<T, V, 7>::run(x...);
    default: return F<T, V, 8>::run(x...);
  }
}

template <class T, int V, int K> struct Forward {
  static cudaError_t run(const zo_conv_args& a, cudaStream_t st) { return run_conv<T, V, K>(a, st); }
};
template <class T, int V, int K> struct Backward {
  static cudaError_t run(const zo_conv_args& a, const zo_conv_grads& g, float* ws, cudaStream_t st) {
    return run_conv_backward<T, V, K>(a, g, ws, st);
  }
};

template <class T>
cudaError_t conv_typed(const zo_conv_args& a, cudaStream_t st) {
  constexpr int W = 16 / sizeof(T);
  int v = W;
  for (const zo_tensor* t : {&a.x, &a.out, &a.state_in, &a.state_out}) {
    const int u = vec_width(*t, sizeof(T), a.channels, W);
    v = u < v ? u : v;
  }
  return v == W ? by_taps<Forward, T, W>(a.taps, a, st) : by_taps<Forward, T, 1>(a.taps, a, st);
}

template <class T>
cudaError_t conv_backward_typed(const zo_conv_args& a, const zo_conv_grads& g, float* ws,
                                cudaStream_t st) {
  int v = 4;
  for (const zo_tensor* t : {&a.x, &a.state_in, &g.dout, &g.dx, &g.dstate_out, &g.dstate_in}) {
    const int u = vec_width(*t, sizeof(T), a.channels, 4);
    v = u < v ? u : v;
  }
  return v == 4 ? by_taps<Backward, T, 4>(a.taps, a, g, ws, st)
                : by_taps<Backward, T, 1>(a.taps, a, g, ws, st);
}

}  // namespace

cudaError_t launch_sum_parts(const float* part, int sets, int64_t parts, int64_t n,
                             const SumOut* outs, int count, cudaStream_t st) {
  SumOuts o{};
  for (int i = 0; i < count; ++i) {
    o.out[i] = outs[i].out.ptr;
    o.stride[i] = outs[i].out.stride;
    o.n[i] = outs[i].n;
  }
  const int64_t bx = ceil_div(n, 32);
  if (bx > INT32_MAX) return cudaErrorInvalidConfiguration;
  for (int s0 = 0; s0 < sets; s0 += 65535) {  // grid.y holds 16 bits
    const int ns = sets - s0 < 65535 ? sets - s0 : 65535;
    const dim3 grid((unsigned)bx, (unsigned)ns);
    const float* p = part + (int64_t)s0 * parts * n;
    if (parts > 64)
      sum_parts_kernel<32><<<grid, 1024, 0, st>>>(p, parts, n, o);
    else
      sum_parts_kernel<8><<<grid, 256, 0, st>>>(p, parts, n, o);
    count_launch();
    for (int i = 0; i < count; ++i)
      if (o.out[i]) o.out[i] += 65535 * o.stride[i];
  }
  return cudaGetLastError();
}

cudaError_t launch_conv(const zo_conv_args& a, cudaStream_t st) {
  switch (a.dtype) {
    case ZO_DTYPE_BF16: return conv_typed<__nv_bfloat16>(a, st);
    case ZO_DTYPE_FP16: return conv_typed<__half>(a, st);
    default: return conv_typed<float>(a, st);
  }
}

int64_t conv_backward_workspace(const zo_conv_args& a) {
  const ConvDims d = conv_backward_dims(a, 1);
  return (int64_t)a.rows * d.runs * (a.taps + 1) * a.channels * (int64_t)sizeof(float);
}

cudaError_t launch_conv_backward(const zo_conv_args& a, const zo_conv_grads& g, float* ws,
                                 cudaStream_t st) {
  switch (a.dtype) {
    case ZO_DTYPE_BF16: return conv_backward_typed<__nv_bfloat16>(a, g, ws, st);
    case ZO_DTYPE_FP16: return conv_backward_typed<__half>(a, g, ws, st);
    default: return conv_backward_typed<float>(a, g, ws, st);
  }
}

}  // namespace zo
