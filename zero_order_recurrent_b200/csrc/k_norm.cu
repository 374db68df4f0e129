// The join of two blocks: p = rms(o) w_post silu(gate) (or the gate before that
// norm), x' = x + s p, n = rms(x') w_pre, and its gradients.
//
// Bound: memory.  A row is read once into registers, both norms' sums are taken
// over it there, and it is written once: the forward moves x, o, gate -> x', n,
// the backward x', o, gate, dn, dx' -> dx, do, dgate and adds the columns' gradients
// up in registers over all rows that a block walks.  A thread has 16 channels of a
// row in the forward and 8 in the backward (16 in wide rows), so that enough bytes are on
// their way; all of a row's loads are issued before anything waits for one.  The
// activations pass by the first-level cache, which then keeps the parameters.
// Measured with fp32 residuals and bf16: forward of 16384 x 4096 188 us (5.0 TB/s), backward of
// 8192 x 2048 90 us (4.1 TB/s).
#include <initializer_list>

#include "zo_block.cuh"
#include "zo_block_internal.h"
#include "zo_internal.h"

namespace zo {
namespace {

// Threads of a block: rows of under 128 threads go several to a block.
template <int W>
constexpr int block_of() {
  return W < 128 ? 128 : W;
}

// Sums of NV values over the W threads of a row.  sh: NV x (threads / 32) floats;
// every thread gets the result.  With W > 32 all threads of the block take part.
template <int W, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* sh) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int m = 16; m > 0; m /= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
  if constexpr (W > 32) {
    constexpr int N = block_of<W>() / 32, R = W / 32;  // warps of the block, of the row
    const int warp = threadIdx.x / 32, first = warp / R * R;
    __syncthreads();  // the last use of sh
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) sh[i * N + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int k = 0; k < R; ++k) v[i] += sh[i * N + first + k];
    }
  }
}

// A thread's share of a row: E vectors of V channels, W vectors apart.
template <int V, int E, int W>
struct Share {
  static constexpr int N = V * E;
  int tid, D;
  __device__ __forceinline__ int channel(int e) const { return (e * W + tid) * V; }
  __device__ __forceinline__ bool has(int e) const { return channel(e) < D; }  // V divides D

  template <class T>
  __device__ __forceinline__ void load(const zo_tensor& t, int64_t row, Vec<T, V> (&x)[E]) const {
    const T* p = static_cast<const T*>(t.ptr) + row * t.row;  // zeros where there is no tensor
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = load_if<T, V>(p + channel(e), t.ptr && has(e));
  }
  template <class T>
  __device__ __forceinline__ static void floats(const Vec<T, V> (&x)[E], float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f(x[i / V].v[i % V]);
  }
  template <class T>
  __device__ __forceinline__ void store(T* row, const float (&f)[N]) const {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (has(e)) {
        Vec<T, V> x;
#pragma unroll
        for (int v = 0; v < V; ++v) x.v[v] = from_f<T>(f[e * V + v]);
        *reinterpret_cast<Vec<T, V>*>(row + channel(e)) = x;
      }
  }
  // A parameter's values at vector e, 1 where there is none.  vec: rows start on 16 bytes.
  __device__ __forceinline__ void param(const zo_f32& p, int64_t set, bool vec, int e, float* f) const {
    const float* q = p.ptr + set * p.stride + channel(e);
    if (!p.ptr || !has(e)) {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = p.ptr ? 0.f : 1.f;
    } else if (V >= 4 && vec) {
#pragma unroll
      for (int v = 0; v + 3 < V; v += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(q + v));
        f[v] = x.x, f[v + 1] = x.y, f[v + 2] = x.z, f[v + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = __ldg(q + v);
    }
  }
  __device__ __forceinline__ void params(const zo_f32& p, int64_t set, bool vec, float (&f)[N]) const {
#pragma unroll
    for (int e = 0; e < E; ++e) param(p, set, vec, e, f + e * V);
  }
  template <class T>
  __device__ __forceinline__ void store_at(T* row, int e, const float (&f)[V]) const {
    Vec<T, V> x;
#pragma unroll
    for (int v = 0; v < V; ++v) x.v[v] = from_f<T>(f[v]);
    if (has(e)) *reinterpret_cast<Vec<T, V>*>(row + channel(e)) = x;
  }
};

// silu of all values, two at a time
template <int N>
__device__ __forceinline__ void silus(const float (&z)[N], float (&act)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 s = silu_2(make_float2(z[i], z[i + 1]));
    act[i] = s.x, act[i + 1] = s.y;
  }
}

template <class T, class XT, int V, int E, int W>
__global__ void __launch_bounds__(block_of<W>())
    norm_kernel(zo_norm_args a, int rows_per_set, bool pvec) {
  __shared__ float sh[block_of<W>() / 32];
  using S = Share<V, E, W>;
  constexpr int N = S::N;
  const S me{(int)threadIdx.x % W, a.channels};
  const int64_t r = (int64_t)blockIdx.x * (block_of<W>() / W) + threadIdx.x / W;
  const bool on = r < a.rows;
  const int64_t row = on ? r : a.rows - 1, set = row / rows_per_set;
  const bool first = a.flags & ZO_NORM_GATE_FIRST, block = a.o.ptr, gate = a.gate.ptr;
  Vec<XT, V> rx[E];
  Vec<T, V> ro[E], rg[E];
  me.load(a.x, row, rx);
  me.load(a.o, row, ro);
  me.load(a.gate, row, rg);
  float x[N];
  S::floats(rx, x);
  if (block) {
    float p[N], act[N], w[N];
    S::floats(ro, p);
    if (gate) {
      S::floats(rg, w);
      silus<N>(w, act);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (first) p[i] *= act[i];
      s[0] = fmaf(p[i], p[i], s[0]);
    }
    if (a.w_post.ptr) {
      row_sums<W, 1>(s, sh);
      const float k = 1.f / sqrtf(s[0] / me.D + a.eps);
      me.params(a.w_post, set, pvec, w);
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] *= k * w[i];
    }
    me.params(a.scale, set, pvec, w);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(w[i], gate && !first ? p[i] * act[i] : p[i], x[i]);
  }
  if (a.x_out.ptr && on) me.store(static_cast<XT*>(a.x_out.ptr) + row * a.x_out.row, x);
  if (!a.n_out.ptr) return;
  float s[1] = {0.f}, w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[0] = fmaf(x[i], x[i], s[0]);
  row_sums<W, 1>(s, sh);
  const float k = 1.f / sqrtf(s[0] / me.D + a.eps);
  me.params(a.w_pre, set, pvec, w);
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] *= x[i] * k;
  if (on) me.store(static_cast<T*>(a.n_out.ptr) + row * a.n_out.row, w);
}

// With y = x', rn = 1 / rms(y), r = 1 / rms(v), v = o (or o act), act = silu(gate):
//   G  = dx' + rn (dn w_pre - y rn^2 mean(dn w_pre y))          -> dx
//   dw_pre += dn y rn;  ds += G p;  dp = G s
//   dw_post += dp' v r, dp' = dp act (or dp);  dv = r (e - v r mean(e v r)), e = dp' w_post
//   do = dv (or dv act);  dgate = silu'(gate) (dp v r w_post, or dv o)
// A group of W threads walks the rows group, group + groups, ... of one set.  With 8
// channels a thread the parameters and the columns' sums stay in registers; with 16 (wide
// rows) the sums are in shared memory, each thread's its own, and the parameters are loaded
// again from the first-level cache.
template <class T, class XT, int V, int E, int W>
__global__ void __launch_bounds__(block_of<W>(), V * E <= 8 ? 512 / block_of<W>() : 1)
    norm_backward_kernel(zo_norm_args a, zo_norm_grads g, int rows_per_set, int groups, bool pvec, float* part) {
  constexpr int kRows = block_of<W>() / W;  // groups of a block
  __shared__ float sh[3 * (block_of<W>() / 32)];
  extern __shared__ float columns[];        // [3][N][W] with 16 channels a thread
  using S = Share<V, E, W>;
  constexpr int N = S::N;
  constexpr bool kKeep = N <= 8;
  const S me{(int)threadIdx.x % W, a.channels};
  const int set = blockIdx.x / (unsigned)(groups / kRows);
  const int group0 = blockIdx.x % (unsigned)(groups / kRows) * kRows, group = group0 + (int)threadIdx.x / W;
  const bool first = a.flags & ZO_NORM_GATE_FIRST, block = a.o.ptr, gate = a.gate.ptr, next = g.dn.ptr;
  const float inv_d = 1.f / me.D;
  float k_pre[kKeep ? N : V], k_post[kKeep ? N : V], k_scale[kKeep ? N : V];  // [vector e's]
  if constexpr (kKeep) {
    me.params(a.w_pre, set, pvec, k_pre);
    me.params(a.w_post, set, pvec, k_post);
    me.params(a.scale, set, pvec, k_scale);
  }
  float s_pre[kKeep ? N : 1], s_post[kKeep ? N : 1], s_scale[kKeep ? N : 1];
  auto add = [&](float* reg, int which, int i, float v) {
    if constexpr (kKeep)
      reg[i] += v;
    else
      columns[(which * N + i) * W + me.tid] += v;
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (kKeep) {
      s_pre[i] = s_post[i] = s_scale[i] = 0.f;
    } else {
#pragma unroll
      for (int w = 0; w < 3; ++w) columns[(w * N + i) * W + me.tid] = 0.f;
    }
  }
  constexpr auto at = [](int e) { return kKeep ? e * V : 0; };  // vector e's parameters
  // all groups of a block go round as often as its first one: they share barriers
  for (int64_t k0 = group0; k0 < rows_per_set; k0 += groups) {
    const int64_t k = k0 + (group - group0);
    const bool on = k < rows_per_set;
    const int64_t row = (int64_t)set * rows_per_set + (on ? k : rows_per_set - 1);
    Vec<XT, V> ry[E], rG[E];
    Vec<T, V> ro[E], rz[E], rn_[E];
    me.load(a.x_out, row, ry);
    me.load(g.dx_out, row, rG);
    me.load(g.dn, row, rn_);
    me.load(a.o, row, ro);
    me.load(a.gate, row, rz);
    // v and, where there is a gate, its activation and slope, for channels i, i + 1 of a thread
    // (pairs reach across vectors where those have one channel)
    auto pair = [&](const auto& x, int i) {
      return make_float2(to_f(x[i / V].v[i % V]), to_f(x[(i + 1) / V].v[(i + 1) % V]));
    };
    float s[3] = {0.f, 0.f, 0.f};
    if (next)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if constexpr (!kKeep) me.param(a.w_pre, set, pvec, e, k_pre);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float y = to_f(ry[e].v[v]);
          s[0] = fmaf(y, y, s[0]);
          s[1] = fmaf(to_f(rn_[e].v[v]) * k_pre[at(e) + v], y, s[1]);
        }
      }
    if (block)
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float2 v = pair(ro, i);
        if (first) v = __fmul2_rn(v, silu_2(pair(rz, i)));
        s[2] = fmaf(v.x, v.x, fmaf(v.y, v.y, s[2]));
      }
    row_sums<W, 3>(s, sh);
    const float rn = next ? 1.f / sqrtf(s[0] * inv_d + a.eps) : 0.f, back = rn * rn * s[1] * inv_d;
    const float r = a.w_post.ptr ? 1.f / sqrtf(s[2] * inv_d + a.eps) : 1.f;
    float G[N];
    XT* dx = static_cast<XT*>(g.dx.ptr) + row * g.dx.row;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (!kKeep) me.param(a.w_pre, set, pvec, e, k_pre);
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = e * V + v;
        G[i] = to_f(rG[e].v[v]);
        if (next) {
          const float y = to_f(ry[e].v[v]), dn = to_f(rn_[e].v[v]);
          if (on) add(s_pre, 0, i, dn * (y * rn));
          G[i] = fmaf(rn, dn * k_pre[at(e) + v] - y * back, G[i]);
        }
        o[v] = G[i];
      }
      if (on) me.store_at(dx, e, o);
    }
    if (!block) continue;
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const int e = i / V;
      if constexpr (!kKeep)
        if (i % V == 0) {
          me.param(a.w_post, set, pvec, e, k_post);
          me.param(a.scale, set, pvec, e, k_scale);
        }
      const float2 act = gate ? silu_2(pair(rz, i)) : two(1.f);
      float2 v = __fmul2_rn(pair(ro, i), two(r));
      if (first) v = __fmul2_rn(v, act);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float vi = h ? v.y : v.x, after = first ? 1.f : h ? act.y : act.x;
        if constexpr (!kKeep && V == 1)
          if (h) {
            me.param(a.w_post, set, pvec, e + 1, k_post);
            me.param(a.scale, set, pvec, e + 1, k_scale);
          }
        const float kp = k_post[kKeep ? i + h : (i + h) % V], ks = k_scale[kKeep ? i + h : (i + h) % V];
        if (on) add(s_scale, 2, i + h, G[i + h] * (vi * kp * after));
        const float t = G[i + h] * ks * after;
        if (on) add(s_post, 1, i + h, t * vi);
        q[0] = fmaf(t * kp, vi, q[0]);
      }
    }
    float m = 0.f;
    if (a.w_post.ptr) {
      row_sums<W, 1>(q, sh);
      m = q[0] * inv_d;
    }
    if (!on) continue;
    T* d_o = static_cast<T*>(g.d_o.ptr) + row * g.d_o.row;
    T* dg = static_cast<T*>(g.dgate.ptr) + (gate ? row * g.dgate.row : 0);
    float fo[V < 2 ? 2 : V], fz[V < 2 ? 2 : V];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const int e = i / V;
      if constexpr (!kKeep)
        if (i % V == 0) {
          me.param(a.w_post, set, pvec, e, k_post);
          me.param(a.scale, set, pvec, e, k_scale);
        }
      float2 act = two(1.f), slope = two(0.f);
      if (gate) silu_slope_2(pair(rz, i), act, slope);
      const float2 o = pair(ro, i);
      float2 v = __fmul2_rn(o, two(r));
      if (first) v = __fmul2_rn(v, act);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (!kKeep && V == 1)
          if (h) {
            me.param(a.w_post, set, pvec, e + 1, k_post);
            me.param(a.scale, set, pvec, e + 1, k_scale);
          }
        const float kp = k_post[kKeep ? i + h : (i + h) % V], ks = k_scale[kKeep ? i + h : (i + h) % V];
        const float vi = h ? v.y : v.x, ai = h ? act.y : act.x, si = h ? slope.y : slope.x;
        const float dp = G[i + h] * ks;
        float t = dp * (first ? 1.f : ai) * kp;
        if (a.w_post.ptr) t = r * (t - vi * m);
        const int j = V < 2 ? h : (i + h) % V;
        fz[j] = first ? t * (h ? o.y : o.x) * si : dp * vi * kp * si;
        fo[j] = first ? t * ai : t;
      }
      if constexpr (V < 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float to[1] = {fo[h]}, tz[1] = {fz[h]};
          me.store_at(d_o, e + h, to);
          if (gate) me.store_at(dg, e + h, tz);
        }
      } else if ((i + 2) % V == 0) {
        me.store_at(d_o, e, fo);
        if (gate) me.store_at(dg, e, fz);
      }
    }
  }
  // [set][group][w_pre, w_post, scale][D]
  float* out = part + ((int64_t)set * groups + group) * 3 * me.D;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float f[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (kKeep)
          f[v] = w == 0 ? s_pre[e * V + v] : w == 1 ? s_post[e * V + v] : s_scale[e * V + v];
        else
          f[v] = columns[(w * N + e * V + v) * W + me.tid];
      }
      if constexpr (V >= 4) {
        if (me.has(e))
#pragma unroll
          for (int v = 0; v < V; v += 4)
            *reinterpret_cast<float4*>(out + (int64_t)w * me.D + me.channel(e) + v) = make_float4(f[v], f[v + 1], f[v + 2], f[v + 3]);
      } else {
        me.store_at(out + (int64_t)w * me.D, e, f);
      }
    }
}

// Threads of a row in the backward pass.  Rows of more than 8192 channels take 1024 threads with 64
// registers each, some of them spilled; with 512 threads and 32 channels a thread 2048 x 16384 takes
// 580 instead of 845 us (but 8 x 16384 55 instead of 49; the forward 161 instead of 139).
int backward_width(int channels) {
  return channels <= 256 ? 32 : channels <= 512 ? 64 : channels <= 1024 ? 128 : channels <= 2048 ? 256
         : channels <= 8192 ? 512 : 1024;
}

// Row groups of one set in the backward pass: no more than fill the SMs once, at 512 threads an
// SM, nor more than there are rows; a multiple of those that a block holds.
int norm_groups(const zo_norm_args& a) {
  const int w = backward_width(a.channels), held = w < 128 ? 128 / w : 1;
  int64_t g = (int64_t)kBlockSMs * 512 / w / a.sets;
  const int64_t rows = a.rows / a.sets;
  if (g > rows) g = ceil_div(rows, held) * held;
  g = g / held * held;
  return (int)(g < held ? held : g);
}

// Whether a parameter's rows start on 16 bytes.
bool params_aligned(std::initializer_list<const zo_f32*> params) {
  for (const zo_f32* p : params)
    if (p->stride % 4 || reinterpret_cast<uintptr_t>(p->ptr) % 16) return false;
  return true;
}

template <class T, class XT, int V, int E, int W>
cudaError_t run_norm(const zo_norm_args& a, cudaStream_t st) {
  const int64_t blocks = ceil_div(a.rows, block_of<W>() / W);
  norm_kernel<T, XT, V, E, W><<<(unsigned)blocks, block_of<W>(), 0, st>>>(
      a, a.rows / a.sets, params_aligned({&a.w_post, &a.scale, &a.w_pre}));
  count_launch();
  return cudaGetLastError();
}

template <class T, class XT, int V, int E, int W>
cudaError_t run_norm_backward(const zo_norm_args& a, const zo_norm_grads& g, float* ws,
                              cudaStream_t st) {
  const int groups = norm_groups(a);
  const int64_t blocks = (int64_t)groups / (block_of<W>() / W) * a.sets, D = a.channels;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  constexpr int kSmem = V * E > 8 ? 3 * V * E * W * (int)sizeof(float) : 0;
  cudaError_t e = allow_shared(norm_backward_kernel<T, XT, V, E, W>, kSmem);
  if (e != cudaSuccess) return e;
  norm_backward_kernel<T, XT, V, E, W><<<(unsigned)blocks, block_of<W>(), kSmem, st>>>(
      a, g, a.rows / a.sets, groups, params_aligned({&a.w_post, &a.scale, &a.w_pre}), ws);
  count_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const SumOut outs[3] = {{g.dw_pre, D}, {g.dw_post, D}, {g.dscale, D}};
  return launch_sum_parts(ws, a.sets, groups, 3 * D, outs, 3, st);
}

// Channels that all rows can be accessed by: 8, or 2, or 1.
template <class T, class XT>
int norm_vector(std::initializer_list<const zo_tensor*> xs, std::initializer_list<const zo_tensor*> os, int channels) {
  int v = 8;
  auto limit = [&](zo_tensor t, int bytes) {
    t.step = 0;
    const int most = 16 / bytes;  // 8 channels of fp32 are two accesses
    int w = vec_width(t, bytes, channels, most);
    if (w == most && channels % 8 == 0) w = 8;
    v = w < v ? w : v;
  };
  for (const zo_tensor* t : xs) limit(*t, sizeof(XT));
  for (const zo_tensor* t : os) limit(*t, sizeof(T));
  return v == 8 ? 8 : v >= 2 ? 2 : 1;
}

template <class T, class XT, int V>
cudaError_t norm_width(const zo_norm_args& a, cudaStream_t st) {
  const int D = a.channels;
  if (D <= 256) return run_norm<T, XT, V, 8 / V, 32>(a, st);
  if (D <= 512) return run_norm<T, XT, V, 16 / V, 32>(a, st);
  if (D <= 1024) return run_norm<T, XT, V, 16 / V, 64>(a, st);
  if (D <= 2048) return run_norm<T, XT, V, 16 / V, 128>(a, st);
  if (D <= 4096) return run_norm<T, XT, V, 16 / V, 256>(a, st);
  if (D <= 8192) return run_norm<T, XT, V, 16 / V, 512>(a, st);
  return run_norm<T, XT, V, 16 / V, 1024>(a, st);
}

template <class T, class XT, int V>
cudaError_t norm_backward_width(const zo_norm_args& a, const zo_norm_grads& g, float* ws, cudaStream_t st) {
  switch (backward_width(a.channels)) {
    case 32: return run_norm_backward<T, XT, V, 8 / V, 32>(a, g, ws, st);
    case 64: return run_norm_backward<T, XT, V, 8 / V, 64>(a, g, ws, st);
    case 128: return run_norm_backward<T, XT, V, 8 / V, 128>(a, g, ws, st);
    case 256: return run_norm_backward<T, XT, V, 8 / V, 256>(a, g, ws, st);
    case 512:
      return a.channels <= 4096 ? run_norm_backward<T, XT, V, 8 / V, 512>(a, g, ws, st)
                                : run_norm_backward<T, XT, V, 16 / V, 512>(a, g, ws, st);
    default: return run_norm_backward<T, XT, V, 16 / V, 1024>(a, g, ws, st);
  }
}

template <class T, class XT>
cudaError_t norm_typed(const zo_norm_args& a, cudaStream_t st) {
  switch (norm_vector<T, XT>({&a.x, &a.x_out}, {&a.o, &a.gate, &a.n_out}, a.channels)) {
    case 8: return norm_width<T, XT, 8>(a, st);
    case 2: return norm_width<T, XT, 2>(a, st);
    default: return norm_width<T, XT, 1>(a, st);
  }
}

template <class T, class XT>
cudaError_t norm_backward_typed(const zo_norm_args& a, const zo_norm_grads& g, float* ws,
                                cudaStream_t st) {
  switch (norm_vector<T, XT>({&a.x_out, &g.dx_out, &g.dx}, {&a.o, &a.gate, &g.dn, &g.d_o, &g.dgate}, a.channels)) {
    case 8: return norm_backward_width<T, XT, 8>(a, g, ws, st);
    case 2: return norm_backward_width<T, XT, 2>(a, g, ws, st);
    default: return norm_backward_width<T, XT, 1>(a, g, ws, st);
  }
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
