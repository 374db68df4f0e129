// Selective scan: per row, channel and state h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,
// y_t = sum_n C_t h_t + skip u_t, out_t = y_t silu(z_t), d_t = softplus(delta_t + bias);
// its gradients; and its single-token form.
//
// A channel's states lie on LN lanes, four each; a warp walks 32 / LN channels
// through time.
#include <type_traits>

#include "zo_block.cuh"
#include "zo_block_internal.h"
#include "zo_internal.h"

namespace zo {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = ZO_SCAN_CHUNK;

struct ScanDims {
  int64_t T;
  int D, N, G, Dg;        // channels, states, groups, channels of a group
  int rows_per_set;
  int tiles;              // channel tiles of a group
  int64_t chunks;
};

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t row, int64_t T,
                                              int32_t* status, bool tell) {
  if (!lengths) return T;
  const int64_t n = lengths[row];
  if (n >= 0 && n <= T) return n;
  if (status && tell) *status = ZO_ERR_BOUNDS;
  return n < 0 ? 0 : T;
}

// log(1 + exp(x)); above 20 it is x to fp32
__device__ __forceinline__ float softplus_f(float x) { return x > 20.f ? x : log1pf(expf(x)); }

template <int LN>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int m = LN / 2; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Where a thread works: its row, group, channel and first state.
struct Place {
  int64_t row, set;
  int g, c, n0, tile;
  bool on;  // its channel exists (its lanes take part in shuffles either way)
};

template <int LN>
__device__ __forceinline__ Place place(const ScanDims& d, int64_t block) {
  Place p;
  constexpr int CT = kThreads / LN;
  p.tile = (int)(block % d.tiles);
  block /= d.tiles;
  p.g = (int)(block % d.G);
  p.row = block / d.G;
  p.set = p.row / d.rows_per_set;
  const int k = p.tile * CT + (int)threadIdx.x / LN;
  p.on = k < d.Dg;
  p.c = p.g * d.Dg + (p.on ? k : 0);
  p.n0 = ((int)threadIdx.x % LN) * 4;
  return p;
}

template <class T>
__device__ __forceinline__ void load_states(const T* p, int n0, int N, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = n0 + i < N ? to_f(p[n0 + i]) : 0.f;
}

template <class T, int LN>
__global__ void __launch_bounds__(kThreads) scan_kernel(zo_scan_args a, ScanDims d) {
  const Place p = place<LN>(d, blockIdx.x);
  const int64_t len = row_length(a.lengths, p.row, d.T, a.status, p.tile == 0 && threadIdx.x == 0);
  const int lane = (int)threadIdx.x % LN;
  float A[4], h[4];
  load_states(a.A.ptr + p.set * a.A.stride + (int64_t)p.c * d.N, p.n0, d.N, A);
  if (a.state_in.ptr)
    load_states(a.state_in.ptr + p.row * a.state_in.stride + (int64_t)p.c * d.N, p.n0, d.N, h);
  else
    h[0] = h[1] = h[2] = h[3] = 0.f;
  const float skip = a.skip.ptr ? a.skip.ptr[p.set * a.skip.stride + p.c] : 0.f;
  const float bias = a.delta_bias.ptr ? a.delta_bias.ptr[p.set * a.delta_bias.stride + p.c] : 0.f;
  const T* u = static_cast<const T*>(a.u.ptr) + p.row * a.u.row + p.c;
  const T* dl = static_cast<const T*>(a.delta.ptr) + p.row * a.delta.row + p.c;
  const T* z = a.z.ptr ? static_cast<const T*>(a.z.ptr) + p.row * a.z.row + p.c : nullptr;
  const T* B = static_cast<const T*>(a.B.ptr) + p.row * a.B.row + (int64_t)p.g * d.N;
  const T* C = static_cast<const T*>(a.C.ptr) + p.row * a.C.row + (int64_t)p.g * d.N;
  T* out = static_cast<T*>(a.out.ptr) + p.row * a.out.row + p.c;
  for (int64_t t = 0; t < d.T; ++t) {
    if (a.checkpoints && t % kChunk == 0 && p.on) {
      float* k = a.checkpoints + ((p.row * d.chunks + t / kChunk) * d.D + p.c) * d.N;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p.n0 + i < d.N) k[p.n0 + i] = h[i];
    }
    if (t >= len) {
      if (p.on && lane == 0) out[t * a.out.step] = from_f<T>(0.f);
      continue;
    }
    const float ut = to_f(u[t * a.u.step]);
    const float raw = to_f(dl[t * a.delta.step]) + bias;
    const float dt = a.flags & ZO_SCAN_SOFTPLUS ? softplus_f(raw) : raw;
    float Bt[4], Ct[4], y = 0.f;
    load_states(B + t * a.B.step, p.n0, d.N, Bt);
    load_states(C + t * a.C.step, p.n0, d.N, Ct);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(expf(dt * A[i]), h[i], dt * ut * Bt[i]);
      y = fmaf(Ct[i], h[i], y);
    }
    y = fmaf(skip, ut, sum_lanes<LN>(y));
    if (p.on && lane == 0)
      out[t * a.out.step] = from_f<T>(z ? y * silu_f(to_f(z[t * a.z.step])) : y);
  }
  if (a.state_out.ptr && p.on) {
    float* k = a.state_out.ptr + p.row * a.state_out.stride + (int64_t)p.c * d.N;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p.n0 + i < d.N) k[p.n0 + i] = h[i];
  }
}

// Backwards through time, chunk by chunk: the states of a chunk are run again
// from its checkpoint, then g_t = C_t dy_t + a_{t+1} g_{t+1} comes back through
// it.  With a_t h_{t-1} = w:
//   dC_t = sum_c dy h;  dB_t = sum_c g d u;  du = d sum_n g B + skip dy
//   dd = sum_n g (A w + u B);  ddelta = dd softplus'(raw);  dA = sum_t g w d
template <class T, int LN>
__global__ void __launch_bounds__(kThreads)
    scan_backward_kernel(zo_scan_args a, zo_scan_grads g, ScanDims d, float* part_bc, float* part_a,
                         float* part_skip, float* part_bias) {
  extern __shared__ float sh[];  // [warp][step][dB, dC][4 LN]
  const Place p = place<LN>(d, blockIdx.x);
  const int64_t len = row_length(a.lengths, p.row, d.T, a.status, p.tile == 0 && threadIdx.x == 0);
  const int lane = (int)threadIdx.x % LN, warp = (int)threadIdx.x / 32;
  const int64_t cn = (int64_t)p.c * d.N;
  float A[4], gr[4], dA[4] = {0.f, 0.f, 0.f, 0.f}, ds = 0.f, db = 0.f;
  load_states(a.A.ptr + p.set * a.A.stride + cn, p.n0, d.N, A);
  if (g.dstate_out.ptr)
    load_states(g.dstate_out.ptr + p.row * g.dstate_out.stride + cn, p.n0, d.N, gr);
  else
    gr[0] = gr[1] = gr[2] = gr[3] = 0.f;
  const float skip = a.skip.ptr ? a.skip.ptr[p.set * a.skip.stride + p.c] : 0.f;
  const float bias = a.delta_bias.ptr ? a.delta_bias.ptr[p.set * a.delta_bias.stride + p.c] : 0.f;
  const T* u = static_cast<const T*>(a.u.ptr) + p.row * a.u.row + p.c;
  const T* dl = static_cast<const T*>(a.delta.ptr) + p.row * a.delta.row + p.c;
  const T* z = a.z.ptr ? static_cast<const T*>(a.z.ptr) + p.row * a.z.row + p.c : nullptr;
  const T* B = static_cast<const T*>(a.B.ptr) + p.row * a.B.row + (int64_t)p.g * d.N;
  const T* C = static_cast<const T*>(a.C.ptr) + p.row * a.C.row + (int64_t)p.g * d.N;
  const T* dout = static_cast<const T*>(g.dout.ptr) + p.row * g.dout.row + p.c;
  T* du = static_cast<T*>(g.du.ptr) + p.row * g.du.row + p.c;
  T* dd = static_cast<T*>(g.ddelta.ptr) + p.row * g.ddelta.row + p.c;
  T* dz = z ? static_cast<T*>(g.dz.ptr) + p.row * g.dz.row + p.c : nullptr;
  for (int64_t k = d.chunks - 1; k >= 0; --k) {
    const int64_t t0 = k * kChunk;
    float h[kChunk + 1][4];
    load_states(a.checkpoints + (p.row * d.chunks + k) * d.D * d.N + cn, p.n0, d.N, h[0]);
    for (int j = 0; j < kChunk; ++j) {
      const int64_t t = t0 + j;
      if (t < len) {
        const float raw = to_f(dl[t * a.delta.step]) + bias;
        const float dt = a.flags & ZO_SCAN_SOFTPLUS ? softplus_f(raw) : raw;
        const float x = dt * to_f(u[t * a.u.step]);
        float Bt[4];
        load_states(B + t * a.B.step, p.n0, d.N, Bt);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[j + 1][i] = fmaf(expf(dt * A[i]), h[j][i], x * Bt[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[j + 1][i] = h[j][i];
      }
    }
    for (int j = kChunk - 1; j >= 0; --j) {
      const int64_t t = t0 + j;
      if (t >= d.T) continue;
      float bc[2][4] = {};
      if (t >= len) {
        if (p.on && lane == 0) {
          du[t * g.du.step] = from_f<T>(0.f);
          dd[t * g.ddelta.step] = from_f<T>(0.f);
          if (z) dz[t * g.dz.step] = from_f<T>(0.f);
        }
      } else {
        const float ut = to_f(u[t * a.u.step]);
        const float raw = to_f(dl[t * a.delta.step]) + bias;
        const float dt = a.flags & ZO_SCAN_SOFTPLUS ? softplus_f(raw) : raw;
        float Bt[4], Ct[4], y = 0.f;
        load_states(B + t * a.B.step, p.n0, d.N, Bt);
        load_states(C + t * a.C.step, p.n0, d.N, Ct);
        float dy = to_f(dout[t * g.dout.step]);
        if (z) {
          const float zt = to_f(z[t * a.z.step]);
#pragma unroll
          for (int i = 0; i < 4; ++i) y = fmaf(Ct[i], h[j + 1][i], y);
          y = fmaf(skip, ut, sum_lanes<LN>(y));
          if (p.on && lane == 0) dz[t * g.dz.step] = from_f<T>(dy * y * dsilu_f(zt));
          dy *= silu_f(zt);
        }
        float gB = 0.f, gA = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float at = expf(dt * A[i]);
          gr[i] = fmaf(Ct[i], dy, gr[i]);
          bc[0][i] = p.on ? gr[i] * dt * ut : 0.f;
          bc[1][i] = p.on ? dy * h[j + 1][i] : 0.f;
          gB = fmaf(gr[i], Bt[i], gB);
          const float w = gr[i] * at * h[j][i];
          gA = fmaf(w, A[i], gA);
          dA[i] = fmaf(w, dt, dA[i]);
          gr[i] *= at;
        }
        gB = sum_lanes<LN>(gB);
        gA = sum_lanes<LN>(gA);
        const float sp = a.flags & ZO_SCAN_SOFTPLUS ? sigmoid_f(raw) : 1.f;
        const float dr = fmaf(gB, ut, gA) * sp;
        ds = fmaf(dy, ut, ds);
        db += dr;
        if (p.on && lane == 0) {
          du[t * g.du.step] = from_f<T>(fmaf(gB, dt, skip * dy));
          dd[t * g.ddelta.step] = from_f<T>(dr);
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int m = LN; m < 32; m *= 2) bc[q][i] += __shfl_xor_sync(0xffffffffu, bc[q][i], m);
          if ((int)threadIdx.x % 32 < LN)
            sh[((warp * kChunk + j) * 2 + q) * 4 * LN + p.n0 + i] = bc[q][i];
        }
    }
    __syncthreads();
    // [tile][row][t][g][dB, dC][N]
    for (int i = threadIdx.x; i < kChunk * 2 * d.N; i += kThreads) {
      const int n = i % d.N, q = i / d.N % 2, j = i / d.N / 2;
      if (t0 + j < d.T) {
        float v = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) v += sh[((w * kChunk + j) * 2 + q) * 4 * LN + n];
        part_bc[((((int64_t)p.tile * a.rows + p.row) * d.T + t0 + j) * d.G + p.g) * 2 * d.N +
                q * d.N + n] = v;
      }
    }
    __syncthreads();
  }
  if (!p.on) return;
  float* pa = part_a + p.row * d.D * d.N + cn;
  float* di = g.dstate_in.ptr ? g.dstate_in.ptr + p.row * g.dstate_in.stride + cn : nullptr;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (p.n0 + i < d.N) {
      pa[p.n0 + i] = dA[i];
      if (di) di[p.n0 + i] = gr[i];
    }
  if (lane == 0) {
    part_skip[p.row * d.D + p.c] = ds;
    part_bias[p.row * d.D + p.c] = db;
  }
}

template <class T>
__global__ void __launch_bounds__(256)
    sum_bc_kernel(zo_scan_args a, zo_scan_grads g, ScanDims d, const float* part) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per_step = (int64_t)d.G * 2 * d.N, n = a.rows * d.T * per_step;
  if (i >= n) return;
  float v = 0.f;
  for (int t = 0; t < d.tiles; ++t) v += part[t * n + i];
  const int64_t row = i / per_step / d.T, t = i / per_step % d.T;
  const int j = (int)(i % per_step), grp = j / (2 * d.N), q = j / d.N % 2, k = j % d.N;
  const zo_tensor& o = q ? g.dC : g.dB;
  static_cast<T*>(o.ptr)[row * o.row + t * o.step + (int64_t)grp * d.N + k] = from_f<T>(v);
}

template <int LN>
ScanDims scan_dims(const zo_scan_args& a) {
  ScanDims d;
  d.T = a.seq;
  d.D = a.channels;
  d.N = a.states;
  d.G = a.groups;
  d.Dg = a.channels / a.groups;
  d.rows_per_set = a.rows / a.sets;
  d.tiles = (int)ceil_div(d.Dg, kThreads / LN);
  d.chunks = ceil_div(a.seq, kChunk);
  return d;
}

template <class T, int LN>
cudaError_t run_scan(const zo_scan_args& a, cudaStream_t st) {
  const ScanDims d = scan_dims<LN>(a);
  const int64_t blocks = (int64_t)d.tiles * d.G * a.rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  scan_kernel<T, LN><<<(unsigned)blocks, kThreads, 0, st>>>(a, d);
  count_launch();
  return cudaGetLastError();
}

template <class T, int LN>
cudaError_t run_scan_backward(const zo_scan_args& a, const zo_scan_grads& g, float* ws,
                              cudaStream_t st) {
  const ScanDims d = scan_dims<LN>(a);
  const int64_t blocks = (int64_t)d.tiles * d.G * a.rows, DN = (int64_t)d.D * d.N;
  const int64_t bc = (int64_t)a.rows * d.T * d.G * 2 * d.N;
  if (blocks > INT32_MAX || ceil_div(bc, 256) > INT32_MAX) return cudaErrorInvalidConfiguration;
  float* pa = ws + d.tiles * bc;
  float* ps = pa + a.rows * DN;
  float* pb = ps + (int64_t)a.rows * d.D;
  const int smem = kThreads / 32 * kChunk * 2 * 4 * LN * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(scan_backward_kernel<T, LN>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  scan_backward_kernel<T, LN><<<(unsigned)blocks, kThreads, smem, st>>>(a, g, d, ws, pa, ps, pb);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  sum_bc_kernel<T><<<(unsigned)ceil_div(bc, 256), 256, 0, st>>>(a, g, d, ws);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t rows = d.rows_per_set;
  e = launch_sum_parts(pa, a.sets, rows, DN, DN, g.dA.ptr, g.dA.stride, st);
  if (e == cudaSuccess && g.dskip.ptr)
    e = launch_sum_parts(ps, a.sets, rows, d.D, d.D, g.dskip.ptr, g.dskip.stride, st);
  if (e == cudaSuccess && g.ddelta_bias.ptr)
    e = launch_sum_parts(pb, a.sets, rows, d.D, d.D, g.ddelta_bias.ptr, g.ddelta_bias.stride, st);
  return e;
}

// Lanes of a channel: four states each, a power of two.
int lanes_of(int states) {
  int n = 1;
  while (4 * n < states) n *= 2;
  return n;
}

template <class F>
auto by_lanes(int states, F&& f) {
  switch (lanes_of(states)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    default: return f(std::integral_constant<int, 32>());
  }
}

template <class F>
cudaError_t by_type(int dtype, F&& f) {
  switch (dtype) {
    case ZO_DTYPE_BF16: return f(__nv_bfloat16());
    case ZO_DTYPE_FP16: return f(__half());
    default: return f(float());
  }
}

}  // namespace

int64_t scan_workspace(const zo_scan_args&) { return 0; }

int64_t scan_backward_workspace(const zo_scan_args& a) {
  return by_lanes(a.states, [&](auto ln) {
    const ScanDims d = scan_dims<decltype(ln)::value>(a);
    return (int64_t)sizeof(float) * ((int64_t)d.tiles * a.rows * d.T * d.G * 2 * d.N +
                                     (int64_t)a.rows * d.D * (d.N + 2));
  });
}

cudaError_t launch_scan(const zo_scan_args& a, float*, cudaStream_t st) {
  return by_type(a.dtype, [&](auto t) {
    return by_lanes(a.states, [&](auto ln) {
      return run_scan<decltype(t), decltype(ln)::value>(a, st);
    });
  });
}

cudaError_t launch_scan_step(const zo_scan_args& a, cudaStream_t st) {
  zo_scan_args b = a;
  b.lengths = nullptr;
  b.checkpoints = nullptr;
  return launch_scan(b, nullptr, st);
}

cudaError_t launch_scan_backward(const zo_scan_args& a, const zo_scan_grads& g, float* ws,
                                 cudaStream_t st) {
  return by_type(a.dtype, [&](auto t) {
    return by_lanes(a.states, [&](auto ln) {
      return run_scan_backward<decltype(t), decltype(ln)::value>(a, g, ws, st);
    });
  });
}

}  // namespace zo
