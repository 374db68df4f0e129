// What the forward and the backward pass of the selective scan share: exponentials and softplus, states
// in memory and tiles in shared memory, parts of time, and the choice of template arguments.
#pragma once

#include <cuda_runtime.h>
#include <float.h>

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
  int tiles = 0;          // channel tiles of a group
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

// 2^x, near 1 to fp32's own precision.  The special function unit's results there (for x < 0) are
// too small on average: by 5e-9 of themselves up to |x| = 2^-10, by 2.4e-8 from 2^-8 to 2^-5.  A decay
// of 2^x lasts 1 / |x| steps and so adds 4e-6 to a state's relative error at |x| = 2^-8, 1.5e-5 at
// 2^-12 (measured with varied steps; CUDA's expf: 7e-7 and 4e-5; a correctly rounded 2^x: 3e-7 and
// 1e-6).  So up to 1/8 a polynomial of degree 4 that is 1 at 0 and has the least largest relative
// error (3.1e-9; its coefficients are the solution of that linear programme): 3.4e-7 and 1.1e-6.
__device__ __forceinline__ float2 exp2_slow_2(float2 x) {
  const float2 e = exp2_2(x);
  float2 p = __ffma2_rn(x, two(0.009628420695662498f), two(0.05553207919001579f));
  p = __ffma2_rn(x, p, two(0.24022643268108368f));
  p = __ffma2_rn(x, p, two(0.6931470632553101f));
  p = __ffma2_rn(x, p, two(1.f));
  return make_float2(fabsf(x.x) < 0.125f ? p.x : e.x, fabsf(x.y) < 0.125f ? p.y : e.y);
}

// The decay of a step, 2^(d A2).  With fp32 activations as above, which takes a fifth of the forward
// pass's time (1 row x 16384 steps x 2048 channels 401 and 494 us).  With narrower ones, whose d, u and
// B are already rounded to 2^-9 or 2^-12, the unit's own result with its argument moved by 8e-9, which
// costs nothing (decays of 1 stay 1): up to |x| = 2^-10 it is then right on average (a state's error
// at 2^-12 falls from 1.5e-5 to 1.6e-6), from 2^-8 on still 1.8e-8 too small (3e-6 at 2^-8).
template <class T>
__device__ __forceinline__ float2 decay_2(float2 d, float2 A2) {
  if constexpr (sizeof(T) == 4)
    return exp2_slow_2(__fmul2_rn(d, A2));
  else
    return exp2_2(__ffma2_rn(d, A2, two(8e-9f)));
}

// A log2(e), kept finite: the lowest fp32 as a decay rate gives decays of 0 and, at steps of
// length 0, of 1.
__device__ __forceinline__ float rate(float A) {
  const float v = A * kLog2e;
  return fabsf(v) > FLT_MAX ? copysignf(FLT_MAX, v) : v;
}
__device__ __forceinline__ float2 rate_2(float2 A) { return make_float2(rate(A.x), rate(A.y)); }

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

template <int LN>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int m = LN / 2; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
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
constexpr int kAhead = 4;     // steps of a channel's inputs in registers ahead

constexpr int kJoin = 8;  // parts whose results are loaded together

// local + 2^x h: the state behind a part whose decays are 2^x together, as its steps would leave
// it one after the other: a large growth of a small state stays finite, that of the state 0 is 0, and
// an infinite state stays so though no fp32 is as small as its decays together.
__device__ __forceinline__ float carried(float x, float h, float local) {
  const float half = exp2_slow_2(two(0.5f * x)).x;
  if (h == 0.f) return local;
  if (fabsf(h) > FLT_MAX && x >= -FLT_MAX) return h + local;
  return fmaf(half * h, half, local);
}

ScanDims scan_dims(const zo_scan_args& a) {
  ScanDims d;
  d.T = a.seq;
  d.D = a.channels;
  d.N = a.states;
  d.G = a.groups;
  d.Dg = a.channels / a.groups;
  d.rows_per_set = a.rows / a.sets;
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
// and the parts of time.  A warp alone on its scheduler keeps the special function
// unit busy a third of the time, and in parts the exponentials come twice (38 instead of
// 20 results a value), so time is divided where there are under 4/3 warps for each of the 592
// schedulers, into as many parts as make four blocks an SM at most (which is what stays there),
// of 32 steps at least.  2048 steps of 2048 channels in one pass and in parts: 2 rows (128
// warps) 452 and 131 us, 4 rows 455 and 223, 8 rows 457 and 408, 12 rows 578 and 543.
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
  int64_t n = 3 * all < 16 * kBlockSMs ? 4 * kBlockSMs / blocks : 1;
  if (n < 1) n = 1;  // blocks of one warp
  int64_t steps = ceil_div(ceil_div(a.seq, n), kChunk) * kChunk;
  if (n > 1 && steps < 32) steps = 32;
  p.parts = (int)ceil_div(a.seq, steps);
  p.steps = p.parts > 1 ? (int)steps : (int)(ceil_div(a.seq, kChunk) * kChunk);
  return p;
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
}  // namespace zo
