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

// x sigmoid(x); the quotient is off by 2 units in the last place
__device__ __forceinline__ float fast_silu(float x) { return __fdividef(x, 1.f + expf(-x)); }

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_1(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 exp2_2(float2 x) { return make_float2(exp2_1(x.x), exp2_1(x.y)); }

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

template <bool WIDE>
__device__ __forceinline__ void load_states4(const float* p, int n0, int N, float (&f)[4]) {
  if constexpr (WIDE) {  // N is a multiple of 4
    f[0] = f[1] = f[2] = f[3] = 0.f;
    if (n0 < N) load_vec<float, 4>(p + n0, f);
  } else {
    load_states(p, n0, N, f);
  }
}

template <bool WIDE>
__device__ __forceinline__ void store_states4(float* p, int n0, int N, const float (&f)[4]) {
  if constexpr (WIDE) {
    if (n0 < N) store_vec<float, 4>(p + n0, f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < N) p[n0 + i] = f[i];
  }
}

__device__ __forceinline__ void store_states(float* p, int n0, int N, const float2 (&h)[2]) {
  const float f[4] = {h[0].x, h[0].y, h[1].x, h[1].y};
  if (N % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0)
    store_states4<true>(p, n0, N, f);
  else
    store_states4<false>(p, n0, N, f);
}

// ---- forward -------------------------------------------------------------------

// Sum over the LN lanes of a channel of y[j], j < min(LN, 4) steps: exchanges
// that halve the number of steps a lane keeps, then plain ones.  Lane q gets
// the sum of step q % 4 (q % LN for fewer lanes).
template <int LN>
constexpr int steps_per_sum() {
  return LN < 4 ? LN : 4;
}

template <int LN>
__device__ __forceinline__ float sum_steps(const float (&y)[steps_per_sum<LN>()], int q) {
  float v;
  if constexpr (LN == 1) {
    v = y[0];
  } else if constexpr (LN == 2) {
    const float keep = q & 1 ? y[1] : y[0], give = q & 1 ? y[0] : y[1];
    v = keep + __shfl_xor_sync(0xffffffffu, give, 1);
  } else {
    float k0 = q & 1 ? y[1] : y[0], g0 = q & 1 ? y[0] : y[1];
    float k1 = q & 1 ? y[3] : y[2], g1 = q & 1 ? y[2] : y[3];
    k0 += __shfl_xor_sync(0xffffffffu, g0, 1);
    k1 += __shfl_xor_sync(0xffffffffu, g1, 1);
    v = (q & 2 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, q & 2 ? k0 : k1, 2);
#pragma unroll
    for (int m = 4; m < LN; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  }
  return v;
}

// A tile of TT steps in shared memory.
template <int LN, int WT, int WC>
struct Tile {
  static constexpr int kSteps = kChunk * WT;
  static constexpr int kChannels = WC * 32 / LN;
  static constexpr int kThreads = 32 * WT * WC;
  static constexpr int kStates = 4 * LN;
  float2 dx[kSteps][kChannels];   // d, d u (0 behind the row's length)
  float2 out[kSteps][kChannels];  // skip u, silu(z)
  float B[kSteps][kStates], C[kSteps][kStates];
  float decay[WT][kChannels][kStates], state[WT][kChannels][kStates];  // WT > 1
};

// WT warps divide a tile of time among them (kChunk steps each) and WC warps its
// channels.  With WT > 1 every warp first runs its steps from the state 0 and
// keeps their decays exp(d A) in registers; the warps then exchange (decay of
// the whole chunk, state at its end), so each knows the state that it starts
// from, and run the steps again, this time without exponentials.  That costs one
// more multiply-add a state and step and makes WT times as many warps, which a
// few long rows need to fill the SMs.
//
// Bound: the special function unit, 16 results a clock and SM.  A value with 16
// states needs 16 exponentials and 4 for softplus and silu, 20 / 16 clocks; its
// 8 bytes in bf16 take 0.34 clocks of an SM's share of the memory.
template <class T, int LN, int WT, int WC, int V>
__global__ void __launch_bounds__(32 * WT * WC)
    scan_kernel(zo_scan_args a, ScanDims d) {
  using S = Tile<LN, WT, WC>;
  extern __shared__ __align__(16) unsigned char smem[];
  S& sh = *reinterpret_cast<S*>(smem);
  int64_t block = blockIdx.x;
  const int tile = (int)(block % d.tiles);
  block /= d.tiles;
  const int g = (int)(block % d.G);
  const int64_t row = block / d.G, set = row / d.rows_per_set;
  const int warp = threadIdx.x / 32, wt = warp % WT, wc = warp / WT;
  const int q = (int)threadIdx.x % LN, ch = wc * (32 / LN) + (int)threadIdx.x % 32 / LN;
  const int k0 = tile * S::kChannels;  // first channel of the tile in its group
  const int left = d.Dg - k0;          // channels of the group from there on
  const bool on = ch < left;
  const int64_t c0 = (int64_t)g * d.Dg + k0;
  const int n0 = q * 4;
  const int64_t len = row_length(a.lengths, row, d.T, a.status, tile == 0 && threadIdx.x == 0);

  float2 A2[2], h[2];
  {
    float A[4] = {0.f, 0.f, 0.f, 0.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) {
      load_states(a.A.ptr + set * a.A.stride + (c0 + ch) * d.N, n0, d.N, A);
      if (a.state_in.ptr)
        load_states(a.state_in.ptr + row * a.state_in.stride + (c0 + ch) * d.N, n0, d.N, s);
    }
    A2[0] = make_float2(A[0] * kLog2e, A[1] * kLog2e);
    A2[1] = make_float2(A[2] * kLog2e, A[3] * kLog2e);
    h[0] = make_float2(s[0], s[1]);
    h[1] = make_float2(s[2], s[3]);
  }
  const T* u = static_cast<const T*>(a.u.ptr) + row * a.u.row + c0;
  const T* dl = static_cast<const T*>(a.delta.ptr) + row * a.delta.row + c0;
  const T* z = a.z.ptr ? static_cast<const T*>(a.z.ptr) + row * a.z.row + c0 : nullptr;
  const T* B = static_cast<const T*>(a.B.ptr) + row * a.B.row + (int64_t)g * d.N;
  const T* C = static_cast<const T*>(a.C.ptr) + row * a.C.row + (int64_t)g * d.N;
  T* out = static_cast<T*>(a.out.ptr) + row * a.out.row + c0;
  const float* skip = a.skip.ptr ? a.skip.ptr + set * a.skip.stride + c0 : nullptr;
  const float* bias = a.delta_bias.ptr ? a.delta_bias.ptr + set * a.delta_bias.stride + c0 : nullptr;
  const bool softplus = a.flags & ZO_SCAN_SOFTPLUS;

  for (int64_t t0 = 0; t0 < d.T; t0 += S::kSteps) {
    if (t0 >= len) {  // behind the row's end: zeros, and the state as it is
      if (on && a.checkpoints && t0 + wt * kChunk < d.T)
        store_states(a.checkpoints + ((row * d.chunks + t0 / kChunk + wt) * d.D + c0 + ch) * d.N,
                     n0, d.N, h);
      for (int i = threadIdx.x; i < S::kSteps * S::kChannels; i += S::kThreads) {
        const int t = i / S::kChannels, c = i % S::kChannels;
        if (c < left && t0 + t < d.T) out[(t0 + t) * a.out.step + c] = from_f<T>(0.f);
      }
      continue;
    }
    // The tile's inputs, V channels a thread.
    for (int i = threadIdx.x; i < S::kSteps * S::kChannels / V; i += S::kThreads) {
      const int t = i / (S::kChannels / V), c = i % (S::kChannels / V) * V;
      const bool in = t0 + t < len && c < left;
      float fu[V], fd[V], fz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) fu[v] = fd[v] = fz[v] = 0.f;
      if (in) {
        load_vec<T, V>(u + (t0 + t) * a.u.step + c, fu);
        load_vec<T, V>(dl + (t0 + t) * a.delta.step + c, fd);
        if (z) load_vec<T, V>(z + (t0 + t) * a.z.step + c, fz);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float dt = fd[v] + (bias && in ? bias[c + v] : 0.f);
        if (softplus) dt = softplus_f(dt);
        if (!in) dt = 0.f;
        sh.dx[t][c + v] = make_float2(dt, dt * fu[v]);
        sh.out[t][c + v] = make_float2(skip && in ? skip[c + v] * fu[v] : 0.f,
                                       !in ? 0.f : z ? fast_silu(fz[v]) : 1.f);
      }
    }
    for (int i = threadIdx.x; i < S::kSteps * S::kStates; i += S::kThreads) {
      const int t = i / S::kStates, n = i % S::kStates;
      const bool in = t0 + t < len && n < d.N;
      sh.B[t][n] = in ? to_f(B[(t0 + t) * a.B.step + n]) : 0.f;
      sh.C[t][n] = in ? to_f(C[(t0 + t) * a.C.step + n]) : 0.f;
    }
    __syncthreads();

    const int s0 = wt * kChunk;  // the warp's first step in the tile
    float2 decay[kChunk][2];
    if constexpr (WT > 1) {
      float2 l[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const float2 dx = sh.dx[s0 + j][ch];
        const float4 b = *reinterpret_cast<const float4*>(&sh.B[s0 + j][n0]);
        decay[j][0] = exp2_2(__fmul2_rn(make_float2(dx.x, dx.x), A2[0]));
        decay[j][1] = exp2_2(__fmul2_rn(make_float2(dx.x, dx.x), A2[1]));
        const float2 x = make_float2(dx.y, dx.y);
        l[0] = __ffma2_rn(decay[j][0], l[0], __fmul2_rn(x, make_float2(b.x, b.y)));
        l[1] = __ffma2_rn(decay[j][1], l[1], __fmul2_rn(x, make_float2(b.z, b.w)));
        sum += dx.x;
      }
      const float2 p0 = exp2_2(__fmul2_rn(make_float2(sum, sum), A2[0]));
      const float2 p1 = exp2_2(__fmul2_rn(make_float2(sum, sum), A2[1]));
      *reinterpret_cast<float4*>(&sh.decay[wt][ch][n0]) = make_float4(p0.x, p0.y, p1.x, p1.y);
      *reinterpret_cast<float4*>(&sh.state[wt][ch][n0]) = make_float4(l[0].x, l[0].y, l[1].x, l[1].y);
      __syncthreads();
    }
    float2 r[2] = {h[0], h[1]};  // the state that the warp starts from
    if constexpr (WT > 1) {
#pragma unroll
      for (int w = 0; w < WT; ++w) {
        if (w == wt) r[0] = h[0], r[1] = h[1];
        const float4 p = *reinterpret_cast<const float4*>(&sh.decay[w][ch][n0]);
        const float4 l = *reinterpret_cast<const float4*>(&sh.state[w][ch][n0]);
        h[0] = __ffma2_rn(make_float2(p.x, p.y), h[0], make_float2(l.x, l.y));
        h[1] = __ffma2_rn(make_float2(p.z, p.w), h[1], make_float2(l.z, l.w));
      }
    }
    if (a.checkpoints && on && t0 + s0 < d.T) {
      float* k = a.checkpoints + ((row * d.chunks + t0 / kChunk + wt) * d.D + c0 + ch) * d.N;
      store_states(k, n0, d.N, r);
    }
    constexpr int U = steps_per_sum<LN>();
#pragma unroll
    for (int j0 = 0; j0 < kChunk; j0 += U) {
      if (t0 + s0 + j0 >= d.T) break;
      float y[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const float2 dx = sh.dx[s0 + j0 + j][ch];
        const float4 b = *reinterpret_cast<const float4*>(&sh.B[s0 + j0 + j][n0]);
        const float4 c = *reinterpret_cast<const float4*>(&sh.C[s0 + j0 + j][n0]);
        const float2 x = make_float2(dx.y, dx.y);
        if constexpr (WT == 1) {
          decay[j0 + j][0] = exp2_2(__fmul2_rn(make_float2(dx.x, dx.x), A2[0]));
          decay[j0 + j][1] = exp2_2(__fmul2_rn(make_float2(dx.x, dx.x), A2[1]));
        }
        r[0] = __ffma2_rn(decay[j0 + j][0], r[0], __fmul2_rn(x, make_float2(b.x, b.y)));
        r[1] = __ffma2_rn(decay[j0 + j][1], r[1], __fmul2_rn(x, make_float2(b.z, b.w)));
        const float2 s = __ffma2_rn(make_float2(c.z, c.w), r[1], __fmul2_rn(make_float2(c.x, c.y), r[0]));
        y[j] = s.x + s.y;
      }
      const float v = sum_steps<LN>(y, q);
      const int t = s0 + j0 + q % U;
      if (q < U && on && t0 + t < d.T) {
        const float2 o = sh.out[t][ch];
        out[(t0 + t) * a.out.step + ch] = from_f<T>(t0 + t < len ? (v + o.x) * o.y : 0.f);
      }
    }
    if constexpr (WT == 1) h[0] = r[0], h[1] = r[1];
    __syncthreads();
  }
  if (a.state_out.ptr && on && wt == 0)
    store_states(a.state_out.ptr + row * a.state_out.stride + (c0 + ch) * d.N, n0, d.N, h);
}

// One token.  A thread holds four states of a channel and walks RG rows of a
// set, so that A is read once for them.  Bound: the states, read and written.
template <class T, int LN, int RG, bool WIDE>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(zo_scan_args a, ScanDims d, int64_t groups) {
  const int64_t nb = ((int64_t)d.D * LN + kThreads - 1) / kThreads;  // blocks of a row
  const int64_t i = blockIdx.x % nb * kThreads + threadIdx.x;       // (channel, lane)
  const int q = (int)(i % LN), n0 = q * 4;
  const bool on = i / LN < d.D;
  const int64_t c = on ? i / LN : 0;
  const int64_t first = blockIdx.x / nb * RG, set = first / groups;
  const int64_t r0 = set * d.rows_per_set + first % groups;
  const int g = (int)(c / d.Dg);
  float A[4];
  load_states4<WIDE>(a.A.ptr + set * a.A.stride + c * d.N, n0, d.N, A);
  const float skip = a.skip.ptr ? a.skip.ptr[set * a.skip.stride + c] : 0.f;
  const float bias = a.delta_bias.ptr ? a.delta_bias.ptr[set * a.delta_bias.stride + c] : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] *= kLog2e;
#pragma unroll
  for (int k = 0; k < RG; ++k) {
    const int64_t row = r0 + k;
    if (RG > 1 && first % groups + k >= d.rows_per_set) break;
    float h[4] = {0.f, 0.f, 0.f, 0.f}, B[4], C[4], y = 0.f;
    if (on) load_states4<WIDE>(a.state_in.ptr + row * a.state_in.stride + c * d.N, n0, d.N, h);
    load_states(static_cast<const T*>(a.B.ptr) + row * a.B.row + (int64_t)g * d.N, n0, d.N, B);
    load_states(static_cast<const T*>(a.C.ptr) + row * a.C.row + (int64_t)g * d.N, n0, d.N, C);
    const float u = to_f(static_cast<const T*>(a.u.ptr)[row * a.u.row + c]);
    float dt = to_f(static_cast<const T*>(a.delta.ptr)[row * a.delta.row + c]) + bias;
    if (a.flags & ZO_SCAN_SOFTPLUS) dt = softplus_f(dt);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(exp2_1(dt * A[i]), h[i], dt * u * B[i]);
      y = fmaf(C[i], h[i], y);
    }
    if (on && a.state_out.ptr)
      store_states4<WIDE>(a.state_out.ptr + row * a.state_out.stride + c * d.N, n0, d.N, h);
    y = fmaf(skip, u, sum_lanes<LN>(y));
    if (on && q == 0) {
      if (a.z.ptr) y *= fast_silu(to_f(static_cast<const T*>(a.z.ptr)[row * a.z.row + c]));
      static_cast<T*>(a.out.ptr)[row * a.out.row + c] = from_f<T>(y);
    }
  }
}

// ---- backward ------------------------------------------------------------------

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

template <class T, int LN, int WT, int WC, int V>
cudaError_t run_scan_tiled(const zo_scan_args& a, cudaStream_t st) {
  using S = Tile<LN, WT, WC>;
  ScanDims d = scan_dims<LN>(a);
  d.tiles = (int)ceil_div(d.Dg, S::kChannels);
  const int64_t blocks = (int64_t)d.tiles * d.G * a.rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(
      scan_kernel<T, LN, WT, WC, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S));
  if (e != cudaSuccess) return e;
  scan_kernel<T, LN, WT, WC, V><<<(unsigned)blocks, S::kThreads, sizeof(S), st>>>(a, d);
  count_launch();
  return cudaGetLastError();
}

template <class T, int LN, int WT, int WC>
cudaError_t run_scan_vec(const zo_scan_args& a, cudaStream_t st) {
  // the thread's channels of a tile are kChunk / LN; a vector of them at most 16 bytes
  constexpr int W = kChunk / LN < 1 ? 1 : kChunk / LN;
  constexpr int V = W * (int)sizeof(T) <= 16 ? W : 16 / (int)sizeof(T);
  int v = V;
  for (const zo_tensor* t : {&a.u, &a.delta, &a.z}) {
    const int w = vec_width(*t, sizeof(T), a.channels / a.groups, V);
    v = w < v ? w : v;
  }
  return v == V ? run_scan_tiled<T, LN, WT, WC, V>(a, st) : run_scan_tiled<T, LN, WT, WC, 1>(a, st);
}

template <class T, int LN>
cudaError_t run_scan(const zo_scan_args& a, cudaStream_t st) {
  return a.seq <= 2 * kChunk ? run_scan_vec<T, LN, 1, 4>(a, st) : run_scan_vec<T, LN, 4, 2>(a, st);
}

template <class T, int LN, int RG>
cudaError_t run_scan_step(const zo_scan_args& a, cudaStream_t st) {
  const ScanDims d = scan_dims<LN>(a);
  const int64_t groups = ceil_div(d.rows_per_set, RG) * RG;  // rows of a set, whole groups
  const int64_t blocks = ceil_div((int64_t)d.D * LN, kThreads) * (groups / RG) * a.sets;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  bool wide = d.N % 4 == 0;
  for (const zo_f32* p : {&a.A, &a.state_in, &a.state_out})
    wide = wide && p->stride % 4 == 0 && reinterpret_cast<uintptr_t>(p->ptr) % 16 == 0;
  if (wide)
    scan_step_kernel<T, LN, RG, true><<<(unsigned)blocks, kThreads, 0, st>>>(a, d, groups);
  else
    scan_step_kernel<T, LN, RG, false><<<(unsigned)blocks, kThreads, 0, st>>>(a, d, groups);
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
  return by_type(a.dtype, [&](auto t) {
    return by_lanes(a.states, [&](auto ln) {
      using T = decltype(t);
      constexpr int LN = decltype(ln)::value;
      // several rows a thread once that leaves enough threads for the memory's latency
      const int64_t threads = (int64_t)a.rows * a.channels * LN;
      return threads >= 4ll * kBlockSMs * 2048 ? run_scan_step<T, LN, 4>(a, st)
                                               : run_scan_step<T, LN, 1>(a, st);
    });
  });
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
