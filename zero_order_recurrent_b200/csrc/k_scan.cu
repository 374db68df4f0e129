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

// ---- forward -------------------------------------------------------------------

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
template <class T, int PITCH>
__device__ __forceinline__ void fetch_rows(T* to, const T* from, int64_t step, int steps, int width,
                                           int bytes) {
  auto run = [&](auto size) {
    constexpr int B = decltype(size)::value, E = B / (int)sizeof(T), P = PITCH / E;
    if constexpr (E >= 1 && P >= 1) {
      for (int i = threadIdx.x; i < steps * P; i += blockDim.x) {
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
    for (int i = threadIdx.x; i < steps * PITCH; i += blockDim.x) {
      const int t = i / PITCH, c = i % PITCH;
      if (c < width) to[i] = from[t * step + c];
    }
}

// S states from n0 on, as S / 2 pairs.
template <int S>
__device__ __forceinline__ void load_pairs(const float* p, int n0, int N, bool wide, float2 (&h)[S / 2]) {
#pragma unroll
  for (int i = 0; i < S; i += 4) {
    float f[4];
    if (wide)
      load_states4<true>(p, n0 + i, N, f);
    else
      load_states4<false>(p, n0 + i, N, f);
    h[i / 2] = make_float2(f[0], f[1]);
    h[i / 2 + 1] = make_float2(f[2], f[3]);
  }
}

template <int S>
__device__ __forceinline__ void store_pairs(float* p, int n0, int N, bool wide, const float2 (&h)[S / 2]) {
#pragma unroll
  for (int i = 0; i < S; i += 4) {
    const float f[4] = {h[i / 2].x, h[i / 2].y, h[i / 2 + 1].x, h[i / 2 + 1].y};
    if (wide)
      store_states4<true>(p, n0 + i, N, f);
    else
      store_states4<false>(p, n0 + i, N, f);
  }
}

// How time is divided among blocks: `n` parts of `steps` steps (whole chunks).
// Part k starts from state[row][k] and sum[row][k] holds its sum of d.
struct Parts {
  int n, steps;
  float *state, *sum;
};

constexpr int kTile = kChunk;  // steps of B and C in shared memory

template <class T, int NP>
struct BC {
  alignas(16) T raw[2][2][kTile][NP];     // [buffer][B, C]: as in memory, on their way
  alignas(16) float f[2][2][kTile][NP];   // [buffer][B, C]: what the scan reads
};

// A lane holds S states of one channel (LN lanes a channel where there are more
// than 16), a warp 32 / LN neighbouring channels, and everything of a channel and
// step - softplus, silu, loads, the output - is done once, by that lane.  B and C,
// which all channels of a group share, come through shared memory a tile ahead;
// u, delta and z come straight into registers kAhead steps ahead.
//
// Bound: the special function unit, 16 results a clock and SM.  A value with 16
// states takes 16 exponentials and 5 for softplus and silu, so 21 / 16 clocks; its
// 8 bytes in bf16 take 0.34 clocks of an SM's share of the memory.  The 16
// exponentials of one step are independent, so a warp a scheduler nearly fills the
// unit.  Fewer lanes a state (four states a lane) make more warps, but were bound
// by shared-memory accesses and issue: 2.5 times the instructions a value.
//
// Where rows and channels are too few for the SMs, time is divided as well: LOCAL
// runs each part but the last from the state 0, scan_join_kernel passes the states
// on from part to part, and then all parts run from the states they start with.
// That takes the exponentials twice.
//
// A block takes `rows` rows of one set one after the other.
constexpr int kAhead = 4;

template <class T, int S, int LN, bool LOCAL>
__global__ void __launch_bounds__(128, 4)
    scan_kernel(zo_scan_args a, ScanDims d, Parts parts, int rows, int copy_bc, bool wide) {
  constexpr int NP = S * LN, W = 32 / LN, H = S / 2;
  extern __shared__ __align__(16) unsigned char smem[];
  BC<T, NP>& sh = *reinterpret_cast<BC<T, NP>*>(smem);
  const unsigned tiles = d.tiles * d.G, row_blocks = (d.rows_per_set + rows - 1) / rows;
  const unsigned nparts = LOCAL ? parts.n - 1 : parts.n;
  const unsigned tile_g = blockIdx.x % tiles, r1_ = blockIdx.x / tiles;
  const int part = r1_ % nparts;
  const unsigned rest = r1_ / nparts;
  const int tile = tile_g % d.tiles, g = tile_g / d.tiles;
  const int set = rest / row_blocks, first = (int)(rest % row_blocks) * rows;
  const int row0 = set * d.rows_per_set + first;
  const int row1 = row0 + (first + rows < d.rows_per_set ? rows : d.rows_per_set - first);
  const int tb = part * parts.steps, te = tb + parts.steps < d.T ? tb + parts.steps : (int)d.T;

  const int lane = threadIdx.x % 32, q = lane / W, n0 = q * S;
  const int k = (tile * (int)(blockDim.x / 32) + (int)threadIdx.x / 32) * W + lane % W;
  const bool on = k < d.Dg;
  const int64_t c = (int64_t)g * d.Dg + (on ? k : 0);
  float2 A2[H];
  load_pairs<S>(a.A.ptr + set * a.A.stride + c * d.N, n0, d.N, false, A2);
#pragma unroll
  for (int i = 0; i < H; ++i) A2[i] = __fmul2_rn(A2[i], two(kLog2e));
  const float bias = a.delta_bias.ptr ? a.delta_bias.ptr[set * a.delta_bias.stride + c] : 0.f;
  const float skip = !LOCAL && a.skip.ptr ? a.skip.ptr[set * a.skip.stride + c] : 0.f;
  const bool softplus = a.flags & ZO_SCAN_SOFTPLUS, gate = !LOCAL && a.z.ptr;

  const bool tell = tile == 0 && part == 0 && threadIdx.x == 0 && !LOCAL;
  auto end_of = [&](int row) {  // of the part, or of the row where that comes first
    const int n = (int)row_length(a.lengths, row, d.T, a.status, tell);
    return n < te ? n : te;
  };
  // B and C of the tile at step t of a row
  auto fetch = [&](int row, int t, int end, int buf) {
    const int n = end - t < kTile ? end - t : kTile;
    const int64_t gn = (int64_t)g * d.N;
    fetch_rows<T, NP>(&sh.raw[buf][0][0][0],
                      static_cast<const T*>(a.B.ptr) + row * a.B.row + t * a.B.step + gn, a.B.step, n, d.N, copy_bc);
    if (!LOCAL)
      fetch_rows<T, NP>(&sh.raw[buf][1][0][0],
                        static_cast<const T*>(a.C.ptr) + row * a.C.row + t * a.C.step + gn, a.C.step, n, d.N, copy_bc);
  };
  auto convert = [&](int buf) {  // states beyond N multiply zeros: h is 0 there
    constexpr int M = (LOCAL ? 1 : 2) * kTile * NP / 4;
    for (int i = threadIdx.x; i < M; i += blockDim.x) {
      const int n = i % (NP / 4) * 4;
      float f[4];
      load_vec<T, 4>(&sh.raw[buf][0][0][0] + i * 4, f);
      if (n + 4 > d.N)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j >= d.N) f[j] = 0.f;
      store_vec<float, 4>(&sh.f[buf][0][0][0] + i * 4, f);
    }
  };
  T ru[kAhead], rd[kAhead], rz[kAhead];
  const T *pu, *pd, *pz = nullptr;  // the next steps to load
  auto at = [&](int row) {
    pu = static_cast<const T*>(a.u.ptr) + row * a.u.row + tb * a.u.step + c;
    pd = static_cast<const T*>(a.delta.ptr) + row * a.delta.row + tb * a.delta.step + c;
    if (gate) pz = static_cast<const T*>(a.z.ptr) + row * a.z.row + tb * a.z.step + c;
  };
  auto load = [&](int n) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j < n) {
        ru[j] = pu[j * a.u.step];
        rd[j] = pd[j * a.delta.step];
        if (gate) rz[j] = pz[j * a.z.step];
      }
    pu += kAhead * a.u.step;
    pd += kAhead * a.delta.step;
    if (gate) pz += kAhead * a.z.step;
  };

  int end = end_of(row0), buf = 0;
  at(row0);
  load(end - tb);
  fetch(row0, tb, end, 0);
  for (int row = row0; row < row1; ++row) {
    const bool more = row + 1 < row1;
    const int next_end = more ? end_of(row + 1) : 0;
    float2 h[H];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < H; ++i) h[i] = two(0.f);
    if (!LOCAL) {
      if (parts.n > 1)
        load_pairs<S>(parts.state + (((int64_t)row * parts.n + part) * d.D + c) * d.N, n0, d.N, wide, h);
      else if (a.state_in.ptr)
        load_pairs<S>(a.state_in.ptr + row * a.state_in.stride + c * d.N, n0, d.N, wide, h);
    }
    T* out = LOCAL ? nullptr : static_cast<T*>(a.out.ptr) + row * a.out.row + tb * a.out.step + c;
    int t = tb;
    for (; t < end; t += kTile) {
      copies_done();
      __syncthreads();
      convert(buf);
      __syncthreads();
      const bool last = t + kTile >= end;
      if (!last)
        fetch(row, t + kTile, end, buf ^ 1);
      else if (more)
        fetch(row + 1, tb, next_end, buf ^ 1);
      if (!LOCAL && a.checkpoints && on)
        store_pairs<S>(a.checkpoints + ((row * d.chunks + t / kChunk) * d.D + c) * d.N, n0, d.N, wide, h);
#pragma unroll 1
      for (int s = 0; s < kTile && t + s < end; s += kAhead) {
        const int n = end - t - s;  // steps left
        float du[kAhead], dd[kAhead], dz[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          du[j] = to_f(ru[j]);
          dd[j] = to_f(rd[j]);
          dz[j] = gate ? to_f(rz[j]) : 0.f;
        }
        if (n > kAhead) {
          load(n - kAhead);
        } else if (more) {
          at(row + 1);
          load(next_end - tb);
        }
        auto run = [&](auto all) {  // the steps; all: kAhead of them, with no checks in between
          constexpr bool whole = decltype(all)::value;
#pragma unroll
          for (int j = 0; j < kAhead; j += 2) {
            if (!whole && j >= n) break;
            float2 dt = __fadd2_rn(make_float2(dd[j], dd[j + 1]), two(bias));
            if (softplus) dt = softplus_2(dt);
            if (!whole && j + 1 >= n) dt.y = 0.f;
            const float2 u = make_float2(du[j], whole || j + 1 < n ? du[j + 1] : 0.f);
            const float2 x = __fmul2_rn(dt, u);
            const float2 gz = gate ? silu_2(make_float2(dz[j], dz[j + 1])) : two(1.f);
            if (LOCAL) sum += dt.x + dt.y;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (!whole && e == 1 && j + 1 >= n) break;
              const float2 d1 = two(e ? dt.y : dt.x), x1 = two(e ? x.y : x.x);
              const float4* B = reinterpret_cast<const float4*>(&sh.f[buf][0][s + j + e][n0]);
              const float4* C = reinterpret_cast<const float4*>(&sh.f[buf][1][s + j + e][n0]);
              float2 y = two(0.f);
#pragma unroll
              for (int i = 0; i < H; i += 2) {
                const float4 b = B[i / 2];
                h[i] = __ffma2_rn(exp2_2(__fmul2_rn(d1, A2[i])), h[i], __fmul2_rn(x1, make_float2(b.x, b.y)));
                h[i + 1] = __ffma2_rn(exp2_2(__fmul2_rn(d1, A2[i + 1])), h[i + 1], __fmul2_rn(x1, make_float2(b.z, b.w)));
                if (!LOCAL) {
                  const float4 v = C[i / 2];
                  y = __ffma2_rn(make_float2(v.x, v.y), h[i], y);
                  y = __ffma2_rn(make_float2(v.z, v.w), h[i + 1], y);
                }
              }
              if (!LOCAL) {
                float v = y.x + y.y;
#pragma unroll
                for (int m = W; m < 32; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
                v = fmaf(skip, e ? u.y : u.x, v) * (e ? gz.y : gz.x);
                if (on && q == 0) out[(j + e) * a.out.step] = from_f<T>(v);
              }
            }
          }
        };
        if (n >= kAhead)
          run(std::true_type());
        else
          run(std::false_type());
        out += kAhead * a.out.step;
      }
      buf ^= 1;
    }
    if (LOCAL) {
      if (on) {
        const int64_t at = ((int64_t)row * parts.n + part) * d.D + c;
        store_pairs<S>(parts.state + at * d.N, n0, d.N, wide, h);
        if (q == 0) parts.sum[at] = sum;
      }
    } else {
      if (on && end < te) {  // behind the row's end: zeros, and the state as it is
        const int from = end > tb ? end : tb;
        if (q == 0)
          for (int i = from; i < te; ++i)
            static_cast<T*>(a.out.ptr)[row * a.out.row + i * a.out.step + c] = from_f<T>(0.f);
        if (a.checkpoints)
          for (int i = (from + kChunk - 1) / kChunk; i * kChunk < te; ++i)
            store_pairs<S>(a.checkpoints + ((row * d.chunks + i) * d.D + c) * d.N, n0, d.N, wide, h);
      }
      if (a.state_out.ptr && on && te == d.T)
        store_pairs<S>(a.state_out.ptr + row * a.state_out.stride + c * d.N, n0, d.N, wide, h);
      if (end <= tb && more) {  // nothing was computed that would have fetched this
        at(row + 1);
        load(next_end - tb);
        __syncthreads();
        fetch(row + 1, tb, next_end, buf);
      }
    }
    end = next_end;
  }
}

// state[row][k] becomes the state that part k starts from.
__global__ void __launch_bounds__(256) scan_join_kernel(zo_scan_args a, ScanDims d, Parts parts) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, DN = (int64_t)d.D * d.N;
  if (i >= a.rows * DN) return;
  const int64_t row = i / DN, cn = i % DN, c = cn / d.N, set = row / d.rows_per_set;
  const float A2 = a.A.ptr[set * a.A.stride + cn] * kLog2e;
  float h = a.state_in.ptr ? a.state_in.ptr[row * a.state_in.stride + cn] : 0.f;
  for (int k = 0; k < parts.n; ++k) {
    const int64_t at = row * parts.n + k;
    float l = 0.f, s = 0.f;
    if (k + 1 < parts.n) {
      l = parts.state[at * DN + cn];
      s = parts.sum[at * d.D + c];
    }
    parts.state[at * DN + cn] = h;
    h = fmaf(exp2_1(s * A2), h, l);
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

// States a lane and lanes a channel.
int states_per_lane(int N) { return N <= 4 ? 4 : N <= 8 ? 8 : 16; }
int lanes_per_channel(int N) {
  int n = 1;
  while (n * states_per_lane(N) < N) n *= 2;
  return n;
}

// Warps of a block (at most four, and no more than a group's channels fill),
// and the parts of time.  One pass over time with w warps a scheduler (592 of
// them) runs at about min(w, 1) of the special function unit's rate; in parts the
// exponentials come twice (37 instead of 21 results a value).  So time is divided
// where there are under half as many warps as schedulers, into as many parts as
// make four blocks an SM at most (which is what stays there), of 64 steps at least.
struct ScanPlan {
  int warps, tiles, parts, steps;
};
ScanPlan scan_plan(const zo_scan_args& a) {
  ScanPlan p;
  const int64_t Dg = a.channels / a.groups, per_warp = 32 / lanes_per_channel(a.states);
  const int64_t w = ceil_div(Dg, per_warp);
  p.warps = w < 4 ? (int)w : 4;
  p.tiles = (int)ceil_div(w, p.warps);
  const int64_t all = w * a.groups * a.rows;
  const int64_t blocks = (int64_t)p.tiles * a.groups * a.rows;
  int64_t n = all * 2 < 4 * kBlockSMs ? 4 * kBlockSMs / blocks : 1;
  int64_t steps = ceil_div(ceil_div(a.seq, n), kChunk) * kChunk;
  if (n > 1 && steps < 64) steps = 64;
  p.parts = (int)ceil_div(a.seq, steps);
  p.steps = p.parts > 1 ? (int)steps : (int)(ceil_div(a.seq, kChunk) * kChunk);
  return p;
}

template <class T, int S, int LN>
cudaError_t run_scan(const zo_scan_args& a, float* ws, cudaStream_t st) {
  const ScanPlan plan = scan_plan(a);
  ScanDims d = scan_dims<LN>(a);
  d.tiles = plan.tiles;
  const int64_t DN = (int64_t)d.D * d.N;
  const Parts parts{plan.parts, plan.steps, ws, ws + (int64_t)a.rows * plan.parts * DN};
  // Short rows go several to a block, as long as that leaves 16 blocks an SM: A
  // and the block's first loads are waited for once for all of them.
  const int64_t per_row = (int64_t)d.tiles * d.G;
  int64_t rows = plan.parts == 1 && a.seq <= 4 * kTile ? per_row * a.rows / (16 * kBlockSMs) : 1;
  rows = rows < 1 ? 1 : rows > d.rows_per_set ? d.rows_per_set : rows;
  const int64_t row_blocks = ceil_div(d.rows_per_set, rows) * a.sets;
  const int64_t blocks = per_row * row_blocks * plan.parts;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int copy = copy_bytes({&a.B, &a.C}, sizeof(T), d.N);
  bool wide = d.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.checkpoints) % 16 == 0;
  for (const zo_f32* p : {&a.state_in, &a.state_out})
    wide = wide && p->stride % 4 == 0 && reinterpret_cast<uintptr_t>(p->ptr) % 16 == 0;
  const int threads = 32 * plan.warps;
  constexpr int kSmem = (int)sizeof(BC<T, S * LN>);
  cudaError_t e = cudaSuccess;
  if (plan.parts > 1) {
    if ((e = cudaFuncSetAttribute(scan_kernel<T, S, LN, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kSmem)) != cudaSuccess)
      return e;
    scan_kernel<T, S, LN, true><<<(unsigned)(per_row * row_blocks * (plan.parts - 1)), threads, kSmem, st>>>(
        a, d, parts, (int)rows, copy, d.N % 4 == 0);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    scan_join_kernel<<<(unsigned)ceil_div(a.rows * DN, 256), 256, 0, st>>>(a, d, parts);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = cudaFuncSetAttribute(scan_kernel<T, S, LN, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmem)) != cudaSuccess)
    return e;
  scan_kernel<T, S, LN, false><<<(unsigned)blocks, threads, kSmem, st>>>(a, d, parts, (int)rows, copy, wide);
  count_launch();
  return cudaGetLastError();
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
cudaError_t by_states(int states, F&& f) {
  using std::integral_constant;
  switch (lanes_per_channel(states)) {
    case 1:
      return states <= 4   ? f(integral_constant<int, 4>(), integral_constant<int, 1>())
             : states <= 8 ? f(integral_constant<int, 8>(), integral_constant<int, 1>())
                           : f(integral_constant<int, 16>(), integral_constant<int, 1>());
    case 2: return f(integral_constant<int, 16>(), integral_constant<int, 2>());
    case 4: return f(integral_constant<int, 16>(), integral_constant<int, 4>());
    default: return f(integral_constant<int, 16>(), integral_constant<int, 8>());
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

int64_t scan_workspace(const zo_scan_args& a) {
  const ScanPlan p = scan_plan(a);
  return p.parts == 1 ? 0 : (int64_t)a.rows * p.parts * a.channels * (a.states + 1) * (int64_t)sizeof(float);
}

int64_t scan_backward_workspace(const zo_scan_args& a) {
  return by_lanes(a.states, [&](auto ln) {
    const ScanDims d = scan_dims<decltype(ln)::value>(a);
    return (int64_t)sizeof(float) * ((int64_t)d.tiles * a.rows * d.T * d.G * 2 * d.N +
                                     (int64_t)a.rows * d.D * (d.N + 2));
  });
}

cudaError_t launch_scan(const zo_scan_args& a, float* ws, cudaStream_t st) {
  return by_type(a.dtype, [&](auto t) {
    return by_states(a.states, [&](auto s, auto ln) {
      return run_scan<decltype(t), decltype(s)::value, decltype(ln)::value>(a, ws, st);
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
