// Short causal convolution over time, pre_t = b + sum_k w[k] x_{t-K+1+k} per
// channel, with its SiLU; its gradients; and the fixed-order sum of partial
// results that the block's backward passes share.
//
// Bound: memory.  The forward reads x and writes out once (2 K + 6 flops for 2
// values moved), the backward reads x and dout and writes dx.  A thread owns four
// neighbouring channels and walks a run of steps with the window in registers, in
// pairs of channels for the packed fp32 instructions, so x is read once per run plus
// K - 1 steps of overlap; the next U steps are on their way while U are computed.
// Measured at 8 rows x 2048 steps x 4096 channels, K = 4, bf16: forward 68 us (4.0 TB/s),
// backward 168 us (2.4 TB/s).  Both wait for loads, with no pipe above 55%.  Neither wider
// accesses nor more steps ahead nor more blocks an SM change the forward by more than a tenth.
#include <initializer_list>
#include <type_traits>

#include "zo_block.cuh"
#include "zo_block_internal.h"
#include "zo_internal.h"

namespace zo {
namespace {

constexpr int kThreads = 128;

// Blocks of an SM that the registers allow.  At the sizes above, in us by blocks an SM; forward:
// 4 taps 70 with 7, 72 with 6, 74 with 5; 6 taps 118, 83 and 84; 8 taps 97 with 5, 98 with 4, 113
// with 3.  Backward: 2, 3 and 4 taps 131, 150 and 168 with 4, 153, 166 and 177 with 3 (fp32 4 taps
// 177 and 151, channels one by one 211 and 147: they spill); 5 taps 191, 189 and 226 with 4, 3 and
// 2; 6 taps 316, 212 and 249; 8 taps 709, 283 and 264.
constexpr int held_forward(int taps) { return taps <= 4 ? 7 : taps <= 6 ? 5 : 4; }
constexpr int held_backward(int taps) { return taps <= 4 ? 4 : taps <= 5 ? 3 : 2; }

struct ConvDims {
  int T, D, rows_per_set, run, runs, ctiles;
  bool params;  // the parameters' rows can be accessed by vectors
};

__device__ __forceinline__ int row_length(const int32_t* lengths, int64_t row, int T,
                                          int32_t* status, bool tell) {
  if (!lengths) return T;
  const int n = lengths[row];
  if (n >= 0 && n <= T) return n;
  if (status && tell) *status = ZO_ERR_BOUNDS;
  return n < 0 ? 0 : T;
}

// V channels from p, of which `have` exist (VEC: always all, on a vector's boundary); zeros
// where `on` is false.
template <class T, int V, bool VEC>
__device__ __forceinline__ Vec<T, V> load_channels(const T* p, int have, bool on) {
  if constexpr (VEC) {
    return load_if<T, V>(p, on);
  } else {
    Vec<T, V> x;
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = load_if<T, 1>(p + i, on && i < have).v[0];
    return x;
  }
}

template <class T, bool VEC, int P>
__device__ __forceinline__ void store_channels(T* p, int have, const float2 (&f)[P]) {
  Vec<T, 2 * P> x;
#pragma unroll
  for (int i = 0; i < P; ++i) x.v[2 * i] = from_f<T>(f[i].x), x.v[2 * i + 1] = from_f<T>(f[i].y);
  if constexpr (VEC) {
    *reinterpret_cast<Vec<T, 2 * P>*>(p) = x;
  } else {
#pragma unroll
    for (int i = 0; i < 2 * P; ++i)
      if (i < have) p[i] = x.v[i];
  }
}

template <class T, int P>
__device__ __forceinline__ void pairs_of(const Vec<T, 2 * P>& x, float2 (&f)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) f[i] = make_float2(to_f(x.v[2 * i]), to_f(x.v[2 * i + 1]));
}

template <int P>
__device__ __forceinline__ void load_params(const float* p, int have, bool vec, float2 (&f)[P]) {
  Vec<float, 2 * P> x;
  if (vec) {
    x = *reinterpret_cast<const Vec<float, 2 * P>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) x.v[i] = i < have ? p[i] : 0.f;
  }
  pairs_of(x, f);
}

template <int P>
__device__ __forceinline__ void zero(float2 (&f)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) f[i] = two(0.f);
}

// Where a thread works.
struct Place {
  int run, c, have;
  int64_t row, set;
};
template <int V>
__device__ __forceinline__ Place place(const ConvDims& d) {
  Place p;
  const unsigned rest = blockIdx.x / (unsigned)d.ctiles;
  p.c = (int)((blockIdx.x % (unsigned)d.ctiles * kThreads + threadIdx.x) * V);
  p.have = d.D - p.c;
  p.run = rest % (unsigned)d.runs;
  p.row = rest / (unsigned)d.runs;
  p.set = (int)p.row / d.rows_per_set;
  return p;
}

// One row's inputs: x, before it the carried window (or 0), after its length 0.
template <class T, int K, int V, bool VEC>
struct Inputs {
  const T *x, *s;
  int64_t x_step, s_step;
  int len, have;
  __device__ __forceinline__ Inputs(const zo_conv_args& a, const Place& p, int n) {
    x = static_cast<const T*>(a.x.ptr) + p.row * a.x.row + p.c;
    s = K > 1 && a.state_in.ptr ? static_cast<const T*>(a.state_in.ptr) + p.row * a.state_in.row + p.c : nullptr;
    x_step = a.x.step;
    s_step = a.state_in.step;
    len = n;
    have = p.have;
  }
  __device__ __forceinline__ Vec<T, V> at(int t) const {  // any step
    const T* p = t >= 0 ? x + t * x_step : s + (t + K - 1) * s_step;
    return load_channels<T, V, VEC>(p, have, t >= 0 ? t < len : s != nullptr);
  }
  __device__ __forceinline__ Vec<T, V> from_x(int t) const {  // t >= 0
    return load_channels<T, V, VEC>(x + t * x_step, have, t < len);
  }
};

template <class T, int K, int V, int U, bool VEC>
__global__ void __launch_bounds__(kThreads, held_forward(K)) conv_kernel(zo_conv_args a, ConvDims d) {
  constexpr int P = V / 2;
  const Place p = place<V>(d);
  if (p.have <= 0) return;
  const int len = row_length(a.lengths, p.row, d.T, a.status, p.run == 0 && p.c == 0);
  const Inputs<T, K, V, VEC> in(a, p, len);
  float2 w[K][P], b[P];
#pragma unroll
  for (int k = 0; k < K; ++k)
    load_params(a.weight.ptr + p.set * a.weight.stride + (int64_t)k * d.D + p.c, p.have, d.params, w[k]);
  zero(b);
  if (a.bias.ptr) load_params(a.bias.ptr + p.set * a.bias.stride + p.c, p.have, d.params, b);
  const int t0 = p.run * d.run, t1 = t0 + d.run < d.T ? t0 + d.run : d.T;
  Vec<T, V> next[U];
#pragma unroll
  for (int j = 0; j < U; ++j) next[j] = in.from_x(t0 + j);
  float2 win[K - 1 + U][P];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) pairs_of(in.at(t0 - (K - 1) + j), win[j]);
  const bool silu = a.flags & ZO_CONV_SILU;
  T* out = static_cast<T*>(a.out.ptr) + p.row * a.out.row + (int64_t)t0 * a.out.step + p.c;
  for (int t = t0; t < t1; t += U) {
#pragma unroll
    for (int j = 0; j < U; ++j) pairs_of(next[j], win[K - 1 + j]);
    if (t + U < t1)
#pragma unroll
      for (int j = 0; j < U; ++j) next[j] = in.from_x(t + U + j);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (t + j >= t1) break;
      float2 y[P];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        y[i] = b[i];
#pragma unroll
        for (int k = 0; k < K; ++k) y[i] = __ffma2_rn(w[k][i], win[j + k][i], y[i]);
        if (silu) y[i] = silu_2(y[i]);
        if (t + j >= len) y[i] = two(0.f);
      }
      store_channels<T, VEC>(out, p.have, y);
      out += a.out.step;
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) win[j][i] = win[U + j][i];
  }
  // The window after the row's last step.  Only the first run reads state_in, so
  // the same thread may write it in place: all loads come before the stores.
  if (K > 1 && p.run == 0 && a.state_out.ptr) {
    T* so = static_cast<T*>(a.state_out.ptr) + p.row * a.state_out.row + p.c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) pairs_of(in.at(len - (K - 1) + j), win[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_channels<T, VEC>(so + j * a.state_out.step, p.have, win[j]);
  }
}

// d_t = dout_t silu'(pre_t);  dx_p = sum_k w[k] d_{p+K-1-k} (+ what state_out's
// gradient sends to p);  dw[k] += d_t x_{t-K+1+k};  db += d_t.
// The run of steps [t0, t1) owns d_t for the sums, and gives dx_p for p in [t0, t1);
// the first run also for p < 0, which is the carried window's gradient.
template <class T, int K, int V, int U, bool VEC>
__global__ void __launch_bounds__(kThreads, held_backward(K))
    conv_backward_kernel(zo_conv_args a, zo_conv_grads g, ConvDims d, float* part) {
  constexpr int P = V / 2;
  const Place p = place<V>(d);
  if (p.have <= 0) return;
  const int len = row_length(a.lengths, p.row, d.T, a.status, p.run == 0 && p.c == 0);
  const Inputs<T, K, V, VEC> in(a, p, len);
  const T* dout = static_cast<const T*>(g.dout.ptr) + p.row * g.dout.row + p.c;
  const T* dso = K > 1 && g.dstate_out.ptr
                     ? static_cast<const T*>(g.dstate_out.ptr) + p.row * g.dstate_out.row + p.c
                     : nullptr;
  T* dx = static_cast<T*>(g.dx.ptr) + p.row * g.dx.row + p.c;
  T* dsi = K > 1 && g.dstate_in.ptr ? static_cast<T*>(g.dstate_in.ptr) + p.row * g.dstate_in.row + p.c : nullptr;
  auto dout_at = [&](int t) { return load_channels<T, V, VEC>(dout + t * g.dout.step, p.have, t < len); };
  float2 w[K][P], b[P], dw[K][P], db[P];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    load_params(a.weight.ptr + p.set * a.weight.stride + (int64_t)k * d.D + p.c, p.have, d.params, w[k]);
    zero(dw[k]);
  }
  zero(b);
  zero(db);
  if (a.bias.ptr) load_params(a.bias.ptr + p.set * a.bias.stride + p.c, p.have, d.params, b);
  const bool silu = a.flags & ZO_CONV_SILU;
  const int t0 = p.run * d.run, t1 = t0 + d.run < d.T ? t0 + d.run : d.T;
  const int p0 = p.run == 0 ? -(K - 1) : t0, last = t1 + K - 1;
  Vec<T, V> nx[U], ny[U];
#pragma unroll
  for (int j = 0; j < U; ++j) nx[j] = in.from_x(t0 + j), ny[j] = dout_at(t0 + j);
  float2 xw[K - 1 + U][P], dd[K - 1 + U][P];  // x_{t-K+1..}, d_{t-K+1..}
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    pairs_of(in.at(t0 - (K - 1) + j), xw[j]);
    zero(dd[j]);
  }
  for (int t = t0; t < last; t += U) {
    float2 dy[U][P];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      pairs_of(nx[j], xw[K - 1 + j]);
      pairs_of(ny[j], dy[j]);
    }
    if (t + U < last)
#pragma unroll
      for (int j = 0; j < U; ++j) nx[j] = in.from_x(t + U + j), ny[j] = dout_at(t + U + j);
#pragma unroll
    for (int j = 0; j < U; ++j) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float2 v = dy[j][i];  // 0 behind the row's end
        if (silu) {
          float2 pre = b[i], s, slope;
#pragma unroll
          for (int k = 0; k < K; ++k) pre = __ffma2_rn(w[k][i], xw[j + k][i], pre);
          silu_slope_2(pre, s, slope);
          v = t + j < len ? __fmul2_rn(v, slope) : two(0.f);
        }
        dd[K - 1 + j][i] = v;
        if (t + j < t1) {
          db[i] = __fadd2_rn(db[i], v);
#pragma unroll
          for (int k = 0; k < K; ++k) dw[k][i] = __ffma2_rn(v, xw[j + k][i], dw[k][i]);
        }
      }
      const int q = t + j - (K - 1);  // whose gradient is now complete
      if (q >= p0 && q < t1) {
        float2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          o[i] = two(0.f);
#pragma unroll
          for (int k = 0; k < K; ++k) o[i] = __ffma2_rn(w[k][i], dd[j + K - 1 - k][i], o[i]);
        }
        const int r = t + j - len;  // which of the last inputs, if any
        if (dso && r >= 0 && r < K - 1) {
          float2 e[P];
          pairs_of(load_channels<T, V, VEC>(dso + r * g.dstate_out.step, p.have, true), e);
#pragma unroll
          for (int i = 0; i < P; ++i) o[i] = __fadd2_rn(o[i], e[i]);
        }
        if (q >= 0)
          store_channels<T, VEC>(dx + q * g.dx.step, p.have, o);
        else if (dsi)
          store_channels<T, VEC>(dsi + (q + K - 1) * g.dstate_in.step, p.have, o);
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        xw[j][i] = xw[U + j][i];
        dd[j][i] = dd[U + j][i];
      }
  }
  // partial sums of this run: [set][row of set, run][K + 1][D]
  float* out = part + (p.row * d.runs + p.run) * (K + 1) * d.D + p.c;
#pragma unroll
  for (int k = 0; k <= K; ++k) store_channels<float, VEC>(out + (int64_t)k * d.D, p.have, k < K ? dw[k < K ? k : K - 1] : db);
}

struct SumOuts {
  float* out[3];
  int64_t stride[3], n[3];
};

// 32 neighbouring values a block, by G warps that take every G-th part, eight loads at a time.
// Eight warps, or 32 where there are few values or many parts for each: 74 parts of 24576
// values take 6 us with eight and 15 with 32.
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

// Steps of one run.  Neighbouring runs both read K - 1 steps and the backward pass sums over
// runs, so they should be long; and all blocks together should nearly fill a whole number of
// waves, `held` blocks an SM each: two waves where that leaves runs of 24 steps, else one, and
// 16 steps at least.  At most 256 steps, so that the backward pass's sums have two stages.
ConvDims conv_dims(const zo_conv_args& a, int V, int held) {
  ConvDims d;
  d.T = a.seq;
  d.D = a.channels;
  d.rows_per_set = a.rows / a.sets;
  d.ctiles = (int)ceil_div(ceil_div(a.channels, V), kThreads);
  const int64_t per_run = (int64_t)d.ctiles * a.rows, wave = held * kBlockSMs;
  auto steps = [&](int64_t blocks) { return ceil_div(a.seq, blocks < per_run ? 1 : blocks / per_run); };
  int64_t run = steps(2 * wave);
  if (run < 24) run = steps(wave);
  run = run < 16 ? 16 : run > 256 ? 256 : run;
  d.run = (int)run;
  d.runs = (int)ceil_div(a.seq, run);
  d.params = a.channels % V == 0;
  for (const zo_f32* p : {&a.weight, &a.bias})
    d.params = d.params && p->stride % V == 0 && reinterpret_cast<uintptr_t>(p->ptr) % 16 == 0;
  return d;
}
// Channels a thread: with eight, the forward of 8 x 2048 x 4096 takes 83 us instead of 70.
constexpr int kChannels = 4;
ConvDims backward_dims(const zo_conv_args& a) { return conv_dims(a, kChannels, held_backward(a.taps)); }

template <class T, int K, bool VEC>
cudaError_t run_conv(const zo_conv_args& a, cudaStream_t st) {
  const ConvDims d = conv_dims(a, kChannels, held_forward(K));
  const int64_t blocks = (int64_t)d.ctiles * d.runs * a.rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  conv_kernel<T, K, kChannels, 4, VEC><<<(unsigned)blocks, kThreads, 0, st>>>(a, d);
  count_launch();
  return cudaGetLastError();
}

template <class T, int K, bool VEC>
cudaError_t run_conv_backward(const zo_conv_args& a, const zo_conv_grads& g, float* ws,
                              cudaStream_t st) {
  const ConvDims d = backward_dims(a);
  const int64_t blocks = (int64_t)d.ctiles * d.runs * a.rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  conv_backward_kernel<T, K, kChannels, 4, VEC><<<(unsigned)blocks, kThreads, 0, st>>>(a, g, d, ws);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const SumOut outs[2] = {{g.dweight, (int64_t)K * d.D}, {g.dbias, d.D}};
  return launch_sum_parts(ws, a.sets, (int64_t)d.rows_per_set * d.runs, (int64_t)(K + 1) * d.D, outs, 2, st);
}

template <class F>
cudaError_t by_taps(int taps, F&& f) {
  using std::integral_constant;
  switch (taps) {
    case 1: return f(integral_constant<int, 1>());
    case 2: return f(integral_constant<int, 2>());
    case 3: return f(integral_constant<int, 3>());
    case 4: return f(integral_constant<int, 4>());
    case 5: return f(integral_constant<int, 5>());
    case 6: return f(integral_constant<int, 6>());
    case 7: return f(integral_constant<int, 7>());
    default: return f(integral_constant<int, 8>());
  }
}

// Whether V channels of all of these can be accessed together.
bool vectors(std::initializer_list<const zo_tensor*> tensors, int elem, int channels, int V) {
  for (const zo_tensor* t : tensors)
    if (vec_width(*t, elem, channels, V) != V) return false;
  return true;
}

template <class T>
cudaError_t conv_typed(const zo_conv_args& a, cudaStream_t st) {
  const bool vec = vectors({&a.x, &a.out, &a.state_in, &a.state_out}, sizeof(T), a.channels, kChannels);
  return by_taps(a.taps, [&](auto k) {
    return vec ? run_conv<T, decltype(k)::value, true>(a, st) : run_conv<T, decltype(k)::value, false>(a, st);
  });
}

template <class T>
cudaError_t conv_backward_typed(const zo_conv_args& a, const zo_conv_grads& g, float* ws,
                                cudaStream_t st) {
  const bool vec = vectors({&a.x, &a.state_in, &g.dout, &g.dx, &g.dstate_out, &g.dstate_in}, sizeof(T), a.channels, kChannels);
  return by_taps(a.taps, [&](auto k) {
    return vec ? run_conv_backward<T, decltype(k)::value, true>(a, g, ws, st)
               : run_conv_backward<T, decltype(k)::value, false>(a, g, ws, st);
  });
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
    if (parts > 64 && (bx * ns < kBlockSMs || parts > 256))  // more threads a value
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
  const ConvDims d = backward_dims(a);
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
