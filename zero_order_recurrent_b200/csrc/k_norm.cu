// The join of two blocks: p = rms(o) w_post silu(gate) (or the gate before that
// norm), x' = x + s p, n = rms(x') w_pre, and its gradients.
//
// Bound: memory.  A row is read once into registers, both norms' sums are taken
// over it there, and it is written once: the forward moves x, o, gate -> x', n,
// the backward x', o, gate, dn, dx' -> dx, do, dgate and adds the four columns'
// gradients up in registers over all rows that a block walks.
#include "zo_block.cuh"
#include "zo_block_internal.h"
#include "zo_internal.h"

namespace zo {
namespace {

// Sums of NV values over the W threads of a row (W = 32: a warp; else a block of
// W threads).  sh: NV x (W / 32) floats; every thread gets the result.
template <int W, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* sh) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int m = 16; m > 0; m /= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
  if (W > 32) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    __syncthreads();  // the last use of sh
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) sh[i * (W / 32) + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int k = 0; k < W / 32; ++k) v[i] += sh[i * (W / 32) + k];
    }
  }
}

template <int W>
constexpr int block_of() {
  return W < 128 ? 128 : W;
}

// Parameters of set `set` at channel c, or 1 where there are none.
template <int V>
__device__ __forceinline__ void load_param(const zo_f32& p, int64_t set, int64_t c, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = p.ptr ? p.ptr[set * p.stride + c + i] : 1.f;
}

// A thread holds E vectors of V channels, W vectors apart.
template <class T, class XT, int V, int E, int W>
__global__ void __launch_bounds__(block_of<W>())
    norm_kernel(zo_norm_args a, int rows_per_set) {
  __shared__ float sh[W / 32];
  const int tid = threadIdx.x % W;
  const int64_t row = (int64_t)blockIdx.x * (block_of<W>() / W) + threadIdx.x / W;
  if (row >= a.rows) return;  // whole warps (W = 32) or none
  const int64_t set = row / rows_per_set;
  const int D = a.channels;
  const bool first = a.flags & ZO_NORM_GATE_FIRST;
  float x[E][V], p[E][V];
  float s[1] = {0.f};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t c = ((int64_t)e * W + tid) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) x[e][i] = p[e][i] = 0.f;
    if (c < D) {
      load_vec<XT, V>(static_cast<const XT*>(a.x.ptr) + row * a.x.row + c, x[e]);
      if (a.o.ptr) load_vec<T, V>(static_cast<const T*>(a.o.ptr) + row * a.o.row + c, p[e]);
      if (first) {
        float z[V];
        load_vec<T, V>(static_cast<const T*>(a.gate.ptr) + row * a.gate.row + c, z);
#pragma unroll
        for (int i = 0; i < V; ++i) p[e][i] *= silu_f(z[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] = fmaf(p[e][i], p[e][i], s[0]);
    }
  }
  float r = 1.f;
  if (a.w_post.ptr) {
    row_sums<W, 1>(s, sh);
    r = 1.f / sqrtf(s[0] / D + a.eps);
  }
  s[0] = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t c = ((int64_t)e * W + tid) * V;
    if (c < D) {
      if (a.o.ptr) {
        float w[V], k[V];
        load_param<V>(a.w_post, set, c, w);
        load_param<V>(a.scale, set, c, k);
        if (a.gate.ptr && !first) {
          float z[V];
          load_vec<T, V>(static_cast<const T*>(a.gate.ptr) + row * a.gate.row + c, z);
#pragma unroll
          for (int i = 0; i < V; ++i) w[i] *= silu_f(z[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) x[e][i] = fmaf(k[i], p[e][i] * r * w[i], x[e][i]);
      }
      if (a.x_out.ptr) store_vec<XT, V>(static_cast<XT*>(a.x_out.ptr) + row * a.x_out.row + c, x[e]);
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] = fmaf(x[e][i], x[e][i], s[0]);
    }
  }
  if (!a.n_out.ptr) return;
  row_sums<W, 1>(s, sh);
  r = 1.f / sqrtf(s[0] / D + a.eps);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t c = ((int64_t)e * W + tid) * V;
    if (c < D) {
      float w[V];
      load_param<V>(a.w_pre, set, c, w);
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] *= x[e][i] * r;
      store_vec<T, V>(static_cast<T*>(a.n_out.ptr) + row * a.n_out.row + c, w);
    }
  }
}

// With y = x', rn = 1 / rms(y), r = 1 / rms(v), v = o (or o act), act = silu(gate):
//   G  = dx' + rn (dn w_pre - y rn^2 mean(dn w_pre y))          -> dx
//   dw_pre += dn y rn;  ds += G p;  dp = G s
//   dw_post += dp' v r, dp' = dp act (or dp);  dv = r (e - v r mean(e v r)), e = dp' w_post
//   do = dv (or dv act);  dgate = silu'(gate) (dp p / act, or dv o)
template <class T, class XT, int V, int E, int W>
__global__ void __launch_bounds__(block_of<W>())
    norm_backward_kernel(zo_norm_args a, zo_norm_grads g, int rows_per_set, int groups, float* part) {
  __shared__ float sh[3 * (W / 32)];
  constexpr int kRows = block_of<W>() / W;  // row groups of a block
  const int tid = threadIdx.x % W;
  const int D = a.channels;
  const int set = blockIdx.x / (groups / kRows);
  const int group = (blockIdx.x % (groups / kRows)) * kRows + threadIdx.x / W;
  const bool first = a.flags & ZO_NORM_GATE_FIRST;
  const float inv_d = 1.f / D;
  float s_pre[E][V], s_post[E][V], s_scale[E][V];
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int i = 0; i < V; ++i) s_pre[e][i] = s_post[e][i] = s_scale[e][i] = 0.f;
  for (int64_t k = group; k < rows_per_set; k += groups) {
    const int64_t row = (int64_t)set * rows_per_set + k;
    float y[E][V], o[E][V], z[E][V], dn[E][V], G[E][V];
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t c = ((int64_t)e * W + tid) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) y[e][i] = o[e][i] = z[e][i] = dn[e][i] = G[e][i] = 0.f;
      if (c < D) {
        load_vec<XT, V>(static_cast<const XT*>(a.x_out.ptr) + row * a.x_out.row + c, y[e]);
        if (g.dn.ptr) load_vec<T, V>(static_cast<const T*>(g.dn.ptr) + row * g.dn.row + c, dn[e]);
        if (g.dx_out.ptr)
          load_vec<XT, V>(static_cast<const XT*>(g.dx_out.ptr) + row * g.dx_out.row + c, G[e]);
        if (a.o.ptr) load_vec<T, V>(static_cast<const T*>(a.o.ptr) + row * a.o.row + c, o[e]);
        if (a.gate.ptr)
          load_vec<T, V>(static_cast<const T*>(a.gate.ptr) + row * a.gate.row + c, z[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t c = ((int64_t)e * W + tid) * V;
      if (c < D) {
        float w[V];
        load_param<V>(a.w_pre, set, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s[0] = fmaf(y[e][i], y[e][i], s[0]);
          s[1] = fmaf(dn[e][i] * w[i], y[e][i], s[1]);
          const float v = first ? o[e][i] * silu_f(z[e][i]) : o[e][i];
          s[2] = fmaf(v, v, s[2]);
        }
      }
    }
    row_sums<W, 3>(s, sh);
    const float rn = 1.f / sqrtf(s[0] * inv_d + a.eps);
    const float r = a.w_post.ptr ? 1.f / sqrtf(s[2] * inv_d + a.eps) : 1.f;
    const float back = g.dn.ptr ? rn * rn * s[1] * inv_d : 0.f;
    float q[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t c = ((int64_t)e * W + tid) * V;
      if (c < D) {
        float w[V], wp[V], sc[V];
        load_param<V>(a.w_pre, set, c, w);
        load_param<V>(a.w_post, set, c, wp);
        load_param<V>(a.scale, set, c, sc);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (g.dn.ptr) {
            s_pre[e][i] = fmaf(dn[e][i], y[e][i] * rn, s_pre[e][i]);
            G[e][i] = fmaf(rn, dn[e][i] * w[i] - y[e][i] * back, G[e][i]);
          }
          const float act = a.gate.ptr ? silu_f(z[e][i]) : 1.f;
          const float vh = (first ? o[e][i] * act : o[e][i]) * r;
          const float after = first ? 1.f : act;
          s_scale[e][i] = fmaf(G[e][i], vh * wp[i] * after, s_scale[e][i]);
          const float dp = G[e][i] * sc[i];
          s_post[e][i] = fmaf(dp * after, vh, s_post[e][i]);
          q[0] = fmaf(dp * after * wp[i], vh, q[0]);
        }
        store_vec<XT, V>(static_cast<XT*>(g.dx.ptr) + row * g.dx.row + c, G[e]);
      }
    }
    if (!a.o.ptr) continue;
    float m = 0.f;
    if (a.w_post.ptr) {
      row_sums<W, 1>(q, sh);
      m = q[0] * inv_d;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t c = ((int64_t)e * W + tid) * V;
      if (c < D) {
        float wp[V], sc[V], d_o[V], dz[V];
        load_param<V>(a.w_post, set, c, wp);
        load_param<V>(a.scale, set, c, sc);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float act = a.gate.ptr ? silu_f(z[e][i]) : 1.f;
          const float vh = (first ? o[e][i] * act : o[e][i]) * r;
          const float dp = G[e][i] * sc[i];
          const float dvh = dp * wp[i] * (first ? 1.f : act);
          const float dv = a.w_post.ptr ? r * (dvh - vh * m) : dvh;
          d_o[i] = first ? dv * act : dv;
          dz[i] = (first ? dv * o[e][i] : dp * vh * wp[i]) * dsilu_f(z[e][i]);
        }
        store_vec<T, V>(static_cast<T*>(g.d_o.ptr) + row * g.d_o.row + c, d_o);
        if (g.dgate.ptr) store_vec<T, V>(static_cast<T*>(g.dgate.ptr) + row * g.dgate.row + c, dz);
      }
    }
  }
  // [set][group][w_pre, w_post, scale][D]
  float* out = part + ((int64_t)set * groups + group) * 3 * D;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t c = ((int64_t)e * W + tid) * V;
    if (c < D)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        out[c + i] = s_pre[e][i];
        out[D + c + i] = s_post[e][i];
        out[2 * (int64_t)D + c + i] = s_scale[e][i];
      }
  }
}

// Row groups of one set in the backward pass (a multiple of 4, the most that a
// block holds): about 512 threads an SM, and no more groups than rows.
int norm_groups(const zo_norm_args& a) {
  const int64_t w = a.channels <= 512 ? 32 : a.channels <= 2048 ? 128 : a.channels <= 8192 ? 512 : 1024;
  int64_t g = ceil_div((int64_t)kBlockSMs * 512 / w, a.sets);
  const int64_t rows = a.rows / a.sets;
  if (g > rows) g = rows;
  return (int)(ceil_div(g, 4) * 4);
}

template <class T, class XT, int V, int E, int W>
cudaError_t run_norm(const zo_norm_args& a, cudaStream_t st) {
  const int64_t blocks = ceil_div(a.rows, block_of<W>() / W);
  norm_kernel<T, XT, V, E, W><<<(unsigned)blocks, block_of<W>(), 0, st>>>(a, a.rows / a.sets);
  count_launch();
  return cudaGetLastError();
}

template <class T, class XT, int V, int E, int W>
cudaError_t run_norm_backward(const zo_norm_args& a, const zo_norm_grads& g, float* ws,
                              cudaStream_t st) {
  const int groups = norm_groups(a);
  const int64_t blocks = (int64_t)groups / (block_of<W>() / W) * a.sets;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  norm_backward_kernel<T, XT, V, E, W>
      <<<(unsigned)blocks, block_of<W>(), 0, st>>>(a, g, a.rows / a.sets, groups, ws);
  count_launch();
  cudaError_t e = cudaGetLastError();
  const int64_t D = a.channels;
  if (e != cudaSuccess) return e;
  const SumOut outs[3] = {{g.dw_pre, D}, {g.dw_post, D}, {g.dscale, D}};
  return launch_sum_parts(ws, a.sets, groups, 3 * D, outs, 3, st);
}

// Whether all rows start on 16 bytes.
bool on_16_bytes(const zo_tensor& t, int bytes) {
  return !t.ptr || (t.row % (16 / bytes) == 0 && reinterpret_cast<uintptr_t>(t.ptr) % 16 == 0);
}

// Widths of 8 channels a vector where everything allows it, else of one.  The
// forward holds 32 channels a thread, the backward 16 (with three sums each).
template <class T, class XT>
cudaError_t norm_typed(const zo_norm_args& a, cudaStream_t st) {
  bool wide = a.channels % 8 == 0;
  for (const zo_tensor* t : {&a.x, &a.x_out}) wide = wide && on_16_bytes(*t, sizeof(XT));
  for (const zo_tensor* t : {&a.o, &a.gate, &a.n_out}) wide = wide && on_16_bytes(*t, sizeof(T));
  const int D = a.channels;
  if (wide) {
    if (D <= 256) return run_norm<T, XT, 8, 1, 32>(a, st);
    if (D <= 1024) return run_norm<T, XT, 8, 4, 32>(a, st);
    if (D <= 4096) return run_norm<T, XT, 8, 4, 128>(a, st);
    if (D <= 8192) return run_norm<T, XT, 8, 4, 256>(a, st);
    return run_norm<T, XT, 8, 4, 512>(a, st);
  }
  if (D <= 256) return run_norm<T, XT, 1, 8, 32>(a, st);
  if (D <= 1024) return run_norm<T, XT, 1, 32, 32>(a, st);
  if (D <= 4096) return run_norm<T, XT, 1, 32, 128>(a, st);
  return run_norm<T, XT, 1, 32, 512>(a, st);
}

template <class T, class XT>
cudaError_t norm_backward_typed(const zo_norm_args& a, const zo_norm_grads& g, float* ws,
                                cudaStream_t st) {
  bool wide = a.channels % 8 == 0;
  for (const zo_tensor* t : {&a.x_out, &g.dx_out, &g.dx}) wide = wide && on_16_bytes(*t, sizeof(XT));
  for (const zo_tensor* t : {&a.o, &a.gate, &g.dn, &g.d_o, &g.dgate})
    wide = wide && on_16_bytes(*t, sizeof(T));
  const int D = a.channels;
  if (wide) {
    if (D <= 512) return run_norm_backward<T, XT, 8, 2, 32>(a, g, ws, st);
    if (D <= 2048) return run_norm_backward<T, XT, 8, 2, 128>(a, g, ws, st);
    if (D <= 8192) return run_norm_backward<T, XT, 8, 2, 512>(a, g, ws, st);
    return run_norm_backward<T, XT, 8, 2, 1024>(a, g, ws, st);
  }
  if (D <= 512) return run_norm_backward<T, XT, 1, 16, 32>(a, g, ws, st);
  if (D <= 2048) return run_norm_backward<T, XT, 1, 16, 128>(a, g, ws, st);
  if (D <= 8192) return run_norm_backward<T, XT, 1, 16, 512>(a, g, ws, st);
  return run_norm_backward<T, XT, 1, 16, 1024>(a, g, ws, st);
}

template <class F>
cudaError_t norm_by_types(const zo_norm_args& a, F&& f) {
  if (a.dtype == ZO_DTYPE_FP32) return f(float(), float());
  const bool same = a.x_dtype == a.dtype;
  if (a.dtype == ZO_DTYPE_BF16)
    return same ? f(__nv_bfloat16(), __nv_bfloat16()) : f(__nv_bfloat16(), float());
  return same ? f(__half(), __half()) : f(__half(), float());
}

}  // namespace

cudaError_t launch_norm(const zo_norm_args& a, cudaStream_t st) {
  return norm_by_types(a, [&](auto t, auto x) { return norm_typed<decltype(t), decltype(x)>(a, st); });
}

int64_t norm_backward_workspace(const zo_norm_args& a) {
  return (int64_t)a.sets * norm_groups(a) * 3 * a.channels * (int64_t)sizeof(float);
}

cudaError_t launch_norm_backward(const zo_norm_args& a, const zo_norm_grads& g, float* ws,
                                 cudaStream_t st) {
  return norm_by_types(a, [&](auto t, auto x) {
    return norm_backward_typed<decltype(t), decltype(x)>(a, g, ws, st);
  });
}

}  // namespace zo
