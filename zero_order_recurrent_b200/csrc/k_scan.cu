// Selective scan: per row, channel and state h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,
// y_t = sum_n C_t h_t + skip u_t, out_t = y_t silu(z_t), d_t = softplus(delta_t + bias);
// its gradients; and its single-token form.
//
// A channel's states lie on LN lanes, four each; a warp walks 32 / LN channels
// through time.
#include <initializer_list>
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

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.92596299e-8f;  // log2(e) - kLog2e
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float exp2_1(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_1(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 exp2_2(float2 x) { return make_float2(exp2_1(x.x), exp2_1(x.y)); }
__device__ __forceinline__ float2 rcp_2(float2 x) { return make_float2(rcp_1(x.x), rcp_1(x.y)); }

// max(x, 0), NaN for NaN
__device__ __forceinline__ float relu_nan(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// log(1 + exp(x)) = max(x, 0) + log(1 + e), e = exp(-|x|), with the series
// log(1 + e) = 2 atanh(s) = 2 s (1 + s^2 / 3 + s^4 / 5 + ...), s = e / (2 + e) <= 1/3: what
// follows the eighth term is under 2e-9 of it.  Relative accuracy down to the smallest
// steps, which log(1 + e) of a rounded 1 + e has not.  e = 2^t (1 + r ln 2) where t + r is
// |x| log2(e) to twice the precision.
__device__ __forceinline__ float2 softplus_2(float2 x) {
  // (beyond -126, e is 0 either way, and an infinite t would leave no r)
  const float2 m = make_float2(fmaxf(-fabsf(x.x), -126.f), fmaxf(-fabsf(x.y), -126.f));
  const float2 t = __fmul2_rn(m, two(kLog2e));
  float2 r = __ffma2_rn(m, two(kLog2e), make_float2(-t.x, -t.y));
  r = __ffma2_rn(m, two(kLog2eLow), r);
  float2 e = exp2_2(t);
  e = __ffma2_rn(e, __fmul2_rn(r, two(kLn2)), e);
  const float2 s = __fmul2_rn(e, rcp_2(__fadd2_rn(e, two(2.f))));
  const float2 w = __fmul2_rn(s, s), s2 = __fadd2_rn(s, s);
  float2 p = __ffma2_rn(w, two(1.f / 15.f), two(1.f / 13.f));
  p = __ffma2_rn(w, p, two(1.f / 11.f));
  p = __ffma2_rn(w, p, two(1.f / 9.f));
  p = __ffma2_rn(w, p, two(1.f / 7.f));
  p = __ffma2_rn(w, p, two(1.f / 5.f));
  p = __ffma2_rn(w, p, two(1.f / 3.f));
  const float2 l = __ffma2_rn(s2, __fmul2_rn(w, p), s2);
  return __fadd2_rn(make_float2(relu_nan(x.x), relu_nan(x.y)), l);
}
__device__ __forceinline__ float softplus_f(float x) { return softplus_2(two(x)).x; }

// x sigmoid(x)
__device__ __forceinline__ float2 silu_2(float2 x) {
  const float2 e = exp2_2(__fmul2_rn(x, two(-kLog2e)));
  return __fmul2_rn(x, rcp_2(__fadd2_rn(e, two(1.f))));
}

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

// Lanes: the 32 / LN channels of a warp are neighbours and a channel's LN lanes
// 32 / LN apart.  A shared-memory access of 16 bytes a lane takes two clocks when
// neighbouring lanes ask for the same address (B and C here) and four when they
// do not; the other order made those the bound.
template <int LN>
constexpr int kWidth = 32 / LN;

// Sum over the LN lanes of a channel of y[j], j < min(LN, 4) steps: exchanges
// that halve the number of steps a lane keeps, then plain ones.  Lane q of the
// channel gets the sum of step q % 4 (q % LN for fewer lanes).
template <int LN>
constexpr int steps_per_sum() {
  return LN < 4 ? LN : 4;
}

template <int LN>
__device__ __forceinline__ float sum_steps(const float (&y)[steps_per_sum<LN>()], int q) {
  constexpr int W = kWidth<LN>;
  float v;
  if constexpr (LN == 1) {
    v = y[0];
  } else if constexpr (LN == 2) {
    const float keep = q & 1 ? y[1] : y[0], give = q & 1 ? y[0] : y[1];
    v = keep + __shfl_xor_sync(0xffffffffu, give, W);
  } else {
    float k0 = q & 1 ? y[1] : y[0], g0 = q & 1 ? y[0] : y[1];
    float k1 = q & 1 ? y[3] : y[2], g1 = q & 1 ? y[2] : y[3];
    k0 += __shfl_xor_sync(0xffffffffu, g0, W);
    k1 += __shfl_xor_sync(0xffffffffu, g1, W);
    v = (q & 2 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, q & 2 ? k0 : k1, 2 * W);
#pragma unroll
    for (int m = 4; m < LN; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m * W);
  }
  return v;
}

// A tile of time in shared memory.
template <class T, int LN, int WT, int WC>
struct Tile {
  static constexpr int kSteps = kChunk * WT;
  static constexpr int kChannels = WC * kWidth<LN>;
  static constexpr int kThreads = 32 * WT * WC;
  static constexpr int kStates = 4 * LN;
  // as in memory, on their way while the tile before is computed
  alignas(16) T u[kSteps][kChannels];
  alignas(16) T d[kSteps][kChannels];
  alignas(16) T z[kSteps][kChannels];
  alignas(16) T b[kSteps][kStates];
  alignas(16) T c[kSteps][kStates];
  // what the scan reads
  alignas(16) float2 dx[kSteps][kChannels];   // d, d u (0 behind the row's length)
  alignas(16) float2 out[kSteps][kChannels];  // skip u, silu(z)
  alignas(16) float B[kSteps][kStates], C[kSteps][kStates];
  // what the time warps exchange (WT > 1)
  float decay[WT][kChannels][kStates], state[WT][kChannels][kStates], end[kChannels][kStates];
  alignas(16) float2 set[kChannels];  // delta's bias, skip
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const unsigned s = (unsigned)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Copies `steps` rows of the first `width` of PITCH elements, asynchronously
// `bytes` at a time (16, 8 or 4, which divide a row; 0: element by element).
template <class T, int PITCH, int THREADS>
__device__ __forceinline__ void fetch_rows(T* to, const T* from, int64_t step, int steps, int width,
                                           int bytes) {
  auto run = [&](auto size) {
    constexpr int B = decltype(size)::value, E = B / (int)sizeof(T), P = PITCH / E;
    if constexpr (E >= 1 && P >= 1) {
      for (int i = threadIdx.x; i < steps * P; i += THREADS) {
        const int t = i / P, c = i % P * E;
        if (c < width) copy_async<B>(to + t * PITCH + c, from + t * step + c);
      }
    }
  };
  if (bytes == 16)
    run(std::integral_constant<int, 16>());
  else if (bytes == 8)
    run(std::integral_constant<int, 8>());
  else if (bytes == 4)
    run(std::integral_constant<int, 4>());
  else
    for (int i = threadIdx.x; i < steps * PITCH; i += THREADS) {
      const int t = i / PITCH, c = i % PITCH;
      if (c < width) to[i] = from[t * step + c];
    }
}

// Blocks of an SM that the registers must allow.
template <int LN, int WT>
constexpr int scan_residency() {
  return WT == 1 ? (LN < 16 ? 6 : 4) : 2;
}

// WT warps divide a tile of time among them (kChunk steps each) and WC warps its
// channels.  With WT > 1 every warp first runs its steps from the state 0 and
// keeps their decays exp(d A) in registers; the warps then exchange (decay of
// the whole chunk, state at its end), so each knows the state that it starts
// from, and run the steps again, this time without exponentials.  That costs one
// more multiply-add a state and step and makes WT times as many warps, which a
// few long rows need to fill the SMs.
//
// A block walks the tiles of `rows` rows of one set, one row after the other;
// the next tile's inputs are on their way while a tile is computed.
//
// Bound: the special function unit, 16 results a clock and SM.  A value with 16
// states needs 16 exponentials and 5 for softplus and silu, 21 / 16 clocks; its
// 8 bytes in bf16 take 0.34 clocks of an SM's share of the memory.
template <class T, int LN, int WT, int WC>
__global__ void __launch_bounds__(32 * WT * WC, scan_residency<LN, WT>())
    scan_kernel(zo_scan_args a, ScanDims d, int rows, int copy, int copy_bc) {
  using S = Tile<T, LN, WT, WC>;
  extern __shared__ __align__(16) unsigned char smem[];
  S& sh = *reinterpret_cast<S*>(smem);
  const unsigned tiles = d.tiles * d.G, blocks = (d.rows_per_set + rows - 1) / rows;
  const unsigned tile_g = blockIdx.x % tiles, rest = blockIdx.x / tiles;
  const int tile = tile_g % d.tiles, g = tile_g / d.tiles;
  const int set = rest / blocks, first = (int)(rest % blocks) * rows;
  const int row0 = set * d.rows_per_set + first;
  const int row1 = row0 + (first + rows < d.rows_per_set ? rows : d.rows_per_set - first);

  const int tid = threadIdx.x, warp = tid / 32, wt = warp % WT, wc = warp / WT;
  const int q = tid % 32 / kWidth<LN>, n0 = q * 4, ch = wc * kWidth<LN> + tid % kWidth<LN>;
  const int left = d.Dg - tile * S::kChannels;  // channels of the group from the tile on
  const bool on = ch < left;
  const int64_t c0 = (int64_t)g * d.Dg + tile * S::kChannels;
  const int T_ = (int)d.T;
  float2 A2[2];
  {
    float A[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) load_states(a.A.ptr + set * a.A.stride + (c0 + ch) * d.N, n0, d.N, A);
    A2[0] = make_float2(A[0] * kLog2e, A[1] * kLog2e);
    A2[1] = make_float2(A[2] * kLog2e, A[3] * kLog2e);
  }
  const bool softplus = a.flags & ZO_SCAN_SOFTPLUS, gate = a.z.ptr != nullptr;
  if (tid < S::kChannels)
    sh.set[tid] = make_float2(
        a.delta_bias.ptr && tid < left ? a.delta_bias.ptr[set * a.delta_bias.stride + c0 + tid] : 0.f,
        a.skip.ptr && tid < left ? a.skip.ptr[set * a.skip.stride + c0 + tid] : 0.f);

  // Sets the tile at step t0 of a row on its way; `valid` steps of it exist.
  const int width = left < S::kChannels ? left : S::kChannels;
  auto fetch = [&](int64_t row, int64_t t0, int valid) {
    constexpr int C = S::kChannels, N = S::kStates, H = S::kThreads;
    fetch_rows<T, C, H>(&sh.u[0][0], static_cast<const T*>(a.u.ptr) + row * a.u.row + t0 * a.u.step + c0,
                        a.u.step, valid, width, copy);
    fetch_rows<T, C, H>(&sh.d[0][0], static_cast<const T*>(a.delta.ptr) + row * a.delta.row + t0 * a.delta.step + c0,
                        a.delta.step, valid, width, copy);
    if (gate)
      fetch_rows<T, C, H>(&sh.z[0][0], static_cast<const T*>(a.z.ptr) + row * a.z.row + t0 * a.z.step + c0,
                          a.z.step, valid, width, copy);
    const int64_t gn = (int64_t)g * d.N;
    fetch_rows<T, N, H>(&sh.b[0][0], static_cast<const T*>(a.B.ptr) + row * a.B.row + t0 * a.B.step + gn,
                        a.B.step, valid, d.N, copy_bc);
    fetch_rows<T, N, H>(&sh.c[0][0], static_cast<const T*>(a.C.ptr) + row * a.C.row + t0 * a.C.step + gn,
                        a.C.step, valid, d.N, copy_bc);
  };
  // Steps of the tile at t0 that a row of length n has.
  auto steps_of = [&](int n, int t0) { return n - t0 < S::kSteps ? n > t0 ? n - t0 : 0 : S::kSteps; };
  auto load_state = [&](int64_t row, float2 (&h)[2]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (on && a.state_in.ptr)
      load_states(a.state_in.ptr + row * a.state_in.stride + (c0 + ch) * d.N, n0, d.N, s);
    h[0] = make_float2(s[0], s[1]);
    h[1] = make_float2(s[2], s[3]);
  };
  const bool tell = tile == 0 && tid == 0;
  int len = (int)row_length(a.lengths, row0, d.T, a.status, tell);
  fetch(row0, 0, steps_of(len, 0));
  float2 next[2];  // the next row's first state
  load_state(row0, next);

  for (int row = row0; row < row1; ++row) {
    float2 h[2] = {next[0], next[1]};
    T* out = static_cast<T*>(a.out.ptr) + row * a.out.row + c0;
    const int next_len = row + 1 < row1 ? (int)row_length(a.lengths, row + 1, d.T, a.status, tell) : 0;
    for (int t0 = 0; t0 < T_; t0 += S::kSteps) {
      const int steps = steps_of(T_, t0), valid = steps_of(len, t0);
      const bool last = t0 + S::kSteps >= T_;
      copies_done();
      __syncthreads();
      if (valid == 0) {  // behind the row's end: zeros, and the state as it is
        if (last && row + 1 < row1) {
          fetch(row + 1, 0, steps_of(next_len, 0));
          load_state(row + 1, next);
        }
        if (WT > 1 && len > 0) {  // a tile came before
          const float4 e = *reinterpret_cast<const float4*>(&sh.end[ch][n0]);
          h[0] = make_float2(e.x, e.y);
          h[1] = make_float2(e.z, e.w);
        }
        if (on && a.checkpoints && wt * kChunk < steps)
          store_states(a.checkpoints + ((row * d.chunks + t0 / kChunk + wt) * d.D + c0 + ch) * d.N,
                       n0, d.N, h);
        for (int i = tid; i < steps * S::kChannels; i += S::kThreads) {
          const int t = i / S::kChannels, c = i % S::kChannels;
          if (c < left) out[(t0 + t) * a.out.step + c] = from_f<T>(0.f);
        }
        continue;
      }
      // Everything that is one channel's and step's is computed once, for two
      // channels at a time.
      constexpr int P = S::kChannels / 2;
#pragma unroll 2
      for (int i = tid; i < S::kSteps * P; i += S::kThreads) {
        const int t = i / P, c = i % P * 2;
        float4 dx = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < valid) {
          const float4 k = *reinterpret_cast<const float4*>(&sh.set[c]);
          const float2 u = make_float2(to_f(sh.u[t][c]), to_f(sh.u[t][c + 1]));
          float2 dt = make_float2(to_f(sh.d[t][c]) + k.x, to_f(sh.d[t][c + 1]) + k.z);
          if (softplus) dt = softplus_2(dt);
          const float2 x = __fmul2_rn(dt, u), su = __fmul2_rn(make_float2(k.y, k.w), u);
          const float2 sz = gate ? silu_2(make_float2(to_f(sh.z[t][c]), to_f(sh.z[t][c + 1]))) : two(1.f);
          dx = make_float4(dt.x, x.x, dt.y, x.y);
          *reinterpret_cast<float4*>(&sh.out[t][c]) = make_float4(su.x, sz.x, su.y, sz.y);
        }
        *reinterpret_cast<float4*>(&sh.dx[t][c]) = dx;  // of channels behind the last: not read
      }
#pragma unroll 2
      for (int i = tid; i < S::kSteps * LN; i += S::kThreads) {
        const int t = i / LN, n = i % LN * 4;
        float fb[4] = {0.f, 0.f, 0.f, 0.f}, fc[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < valid) {
          load_vec<T, 4>(&sh.b[t][n], fb);
          load_vec<T, 4>(&sh.c[t][n], fc);
          if (n + 4 > d.N)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (n + k >= d.N) fb[k] = fc[k] = 0.f;
        }
        store_vec<float, 4>(&sh.B[t][n], fb);
        store_vec<float, 4>(&sh.C[t][n], fc);
      }
      __syncthreads();
      if (!last) {
        fetch(row, t0 + S::kSteps, steps_of(len, t0 + S::kSteps));
      } else if (row + 1 < row1) {
        fetch(row + 1, 0, steps_of(next_len, 0));
        load_state(row + 1, next);
      }

      const int s0 = wt * kChunk;  // the warp's first step in the tile
      float2 decay[kChunk][2];
      if constexpr (WT > 1) {
        float2 l[2] = {two(0.f), two(0.f)};
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          const float2 dx = sh.dx[s0 + j][ch];
          const float4 b = *reinterpret_cast<const float4*>(&sh.B[s0 + j][n0]);
          decay[j][0] = exp2_2(__fmul2_rn(two(dx.x), A2[0]));
          decay[j][1] = exp2_2(__fmul2_rn(two(dx.x), A2[1]));
          l[0] = __ffma2_rn(decay[j][0], l[0], __fmul2_rn(two(dx.y), make_float2(b.x, b.y)));
          l[1] = __ffma2_rn(decay[j][1], l[1], __fmul2_rn(two(dx.y), make_float2(b.z, b.w)));
          sum += dx.x;
        }
        if (wt < WT - 1) {
          const float2 p0 = exp2_2(__fmul2_rn(two(sum), A2[0])), p1 = exp2_2(__fmul2_rn(two(sum), A2[1]));
          *reinterpret_cast<float4*>(&sh.decay[wt][ch][n0]) = make_float4(p0.x, p0.y, p1.x, p1.y);
          *reinterpret_cast<float4*>(&sh.state[wt][ch][n0]) = make_float4(l[0].x, l[0].y, l[1].x, l[1].y);
        }
        if (t0 > 0) {  // where the tile before ended; written again only after the barrier
          const float4 e = *reinterpret_cast<const float4*>(&sh.end[ch][n0]);
          h[0] = make_float2(e.x, e.y);
          h[1] = make_float2(e.z, e.w);
        }
        __syncthreads();
        for (int w = 0; w < wt; ++w) {
          const float4 p = *reinterpret_cast<const float4*>(&sh.decay[w][ch][n0]);
          const float4 e = *reinterpret_cast<const float4*>(&sh.state[w][ch][n0]);
          h[0] = __ffma2_rn(make_float2(p.x, p.y), h[0], make_float2(e.x, e.y));
          h[1] = __ffma2_rn(make_float2(p.z, p.w), h[1], make_float2(e.z, e.w));
        }
      }
      if (a.checkpoints && on && s0 < steps) {
        float* k = a.checkpoints + ((row * d.chunks + t0 / kChunk + wt) * d.D + c0 + ch) * d.N;
        store_states(k, n0, d.N, h);
      }
      constexpr int U = steps_per_sum<LN>();
      T* o = out + (t0 + s0 + q % U) * a.out.step + ch;
#pragma unroll
      for (int j0 = 0; j0 < kChunk; j0 += U) {
        float y[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const float2 dx = sh.dx[s0 + j0 + j][ch];
          const float4 b = *reinterpret_cast<const float4*>(&sh.B[s0 + j0 + j][n0]);
          const float4 c = *reinterpret_cast<const float4*>(&sh.C[s0 + j0 + j][n0]);
          if constexpr (WT == 1) {
            decay[j0 + j][0] = exp2_2(__fmul2_rn(two(dx.x), A2[0]));
            decay[j0 + j][1] = exp2_2(__fmul2_rn(two(dx.x), A2[1]));
          }
          h[0] = __ffma2_rn(decay[j0 + j][0], h[0], __fmul2_rn(two(dx.y), make_float2(b.x, b.y)));
          h[1] = __ffma2_rn(decay[j0 + j][1], h[1], __fmul2_rn(two(dx.y), make_float2(b.z, b.w)));
          const float2 e = __ffma2_rn(make_float2(c.z, c.w), h[1], __fmul2_rn(make_float2(c.x, c.y), h[0]));
          y[j] = e.x + e.y;
        }
        const float v = sum_steps<LN>(y, q);
        const int t = s0 + j0 + q % U;
        if (q < U && on && t < steps) {
          const float2 e = sh.out[t][ch];
          *o = from_f<T>(t < valid ? (v + e.x) * e.y : 0.f);
        }
        o += U * a.out.step;
        if (s0 + j0 + U >= steps) break;
      }
      if (WT > 1 && wt == WT - 1)
        *reinterpret_cast<float4*>(&sh.end[ch][n0]) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    }
    if (a.state_out.ptr && on && wt == WT - 1)
      store_states(a.state_out.ptr + row * a.state_out.stride + (c0 + ch) * d.N, n0, d.N, h);
    len = next_len;
  }
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
      if (a.z.ptr) y *= silu_2(two(to_f(static_cast<const T*>(a.z.ptr)[row * a.z.row + c]))).x;
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

// Bytes of an asynchronous copy that all rows of these tensors keep to: 16, 8
// or 4, or 0.
int copy_bytes(std::initializer_list<const zo_tensor*> tensors, int elem, int64_t width) {
  int bytes = 16;
  for (const zo_tensor* t : tensors) {
    const int b = vec_width(*t, elem, width, 16 / elem) * elem;
    bytes = b < bytes ? b : bytes;
  }
  return bytes < 4 ? 0 : bytes;
}

template <class T, int LN, int WT, int WC>
cudaError_t run_scan_tiled(const zo_scan_args& a, cudaStream_t st) {
  using S = Tile<T, LN, WT, WC>;
  ScanDims d = scan_dims<LN>(a);
  d.tiles = (int)ceil_div(d.Dg, S::kChannels);
  // Rows that fit one tile go several to a block, as long as that leaves 16
  // blocks an SM: the block's first loads are waited for once for all of them.
  int64_t rows = 1;
  if (a.seq <= S::kSteps) rows = (int64_t)d.tiles * d.G * a.rows / (16 * kBlockSMs);
  rows = rows < 1 ? 1 : rows > d.rows_per_set ? d.rows_per_set : rows;
  const int64_t blocks = (int64_t)d.tiles * d.G * ceil_div(d.rows_per_set, rows) * a.sets;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  constexpr int kRow = S::kChannels * (int)sizeof(T);
  int copy = copy_bytes({&a.u, &a.delta, &a.z}, sizeof(T), d.Dg);
  if (copy > kRow) copy = kRow;
  const int copy_bc = copy_bytes({&a.B, &a.C}, sizeof(T), d.N);
  const cudaError_t e = cudaFuncSetAttribute(
      scan_kernel<T, LN, WT, WC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S));
  if (e != cudaSuccess) return e;
  scan_kernel<T, LN, WT, WC>
      <<<(unsigned)blocks, S::kThreads, sizeof(S), st>>>(a, d, (int)rows, copy, copy_bc);
  count_launch();
  return cudaGetLastError();
}

// Rows of at most two chunks are walked by one warp a channel group; longer ones
// by several along time (eight where a warp's channels still fill sectors).
template <class T, int LN>
cudaError_t run_scan(const zo_scan_args& a, cudaStream_t st) {
  if (a.seq <= 2 * kChunk) return run_scan_tiled<T, LN, 1, 4>(a, st);
  if constexpr (LN <= 4)
    return run_scan_tiled<T, LN, 8, 1>(a, st);
  else
    return run_scan_tiled<T, LN, 4, 2>(a, st);
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
