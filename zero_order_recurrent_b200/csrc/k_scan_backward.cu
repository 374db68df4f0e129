// Gradients of the selective scan (k_scan.cu has its formulas and the forward pass).  States, carries
// and sums are fp32; times are at 16 states and bf16.
//
// With a_t h_{t-1} = w_t and g_t = C_t dy_t + a_{t+1} g_{t+1}, dy = dout silu(z):
//   dC_t = sum_c dy h;  dB_t = sum_c g d u;  du = d sum_n g B + skip dy
//   dd = sum_n g (A w + u B);  ddelta = dd softplus'(raw);  dA = sum_t g w d
//   dskip = sum_t dy u;  dbias = sum_t ddelta;  dz = dout y silu'(z)

#include "k_scan.cuh"

namespace zo {
namespace {

// The lanes' sums of NV values: lane l gets, in v[0 ..], those of the values whose index has
// the bits of l / STRIDE on top (lowest bit first); where lanes outnumber values, several
// lanes get the same.
template <int NV, int LANES, int STRIDE>
__device__ __forceinline__ void sum_over(float* v, int lane) {
  if constexpr (LANES > 1) {
    if constexpr (NV > 1) {
      const bool up = lane & STRIDE;
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        const float keep = up ? v[i + NV / 2] : v[i], give = up ? v[i] : v[i + NV / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, STRIDE);
      }
      sum_over<NV / 2, LANES / 2, STRIDE * 2>(v, lane);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], STRIDE);
      sum_over<1, LANES / 2, STRIDE * 2>(v, lane);
    }
  }
}

// The same for three values of each of four channels, over LN lanes: lane q gets, in v[0 ..],
// the three of channel 2 (q & 1) + (q >> 1 & 1) (of two or four channels where LN is 2 or 1).
template <int LN>
__device__ __forceinline__ void sum_over12(float* v, int lane) {
  if constexpr (LN >= 2) sum_over<12, 2, 1>(v, lane);
  if constexpr (LN >= 4) sum_over<6, 2, 2>(v, lane);
  if constexpr (LN >= 8)
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int m = 4; m < LN; m *= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
}

// A lane's carry over one part of time from the carry 0 at its end:
// carry <- a_t (carry + C_t dy_t), t backwards; parts 1 .. n-1, into parts.state and sum.
template <class T, int S, int LN>
__global__ void __launch_bounds__(128, 4)
    scan_carry_kernel(zo_scan_args a, zo_scan_grads g, ScanDims d, Parts parts, int copy) {
  constexpr int NP = S * LN, W = 32 / LN, H = S / 2;
  __shared__ __align__(16) float C[kTile][NP];
  __shared__ __align__(16) T raw[kTile][NP];
  const unsigned tiles = d.tiles * d.G;
  const unsigned tile_g = blockIdx.x % tiles, rest = blockIdx.x / tiles;
  const int part = 1 + rest % (parts.n - 1), row = rest / (parts.n - 1);
  const int tile = tile_g % d.tiles, grp = tile_g / d.tiles, set = row / d.rows_per_set;
  const int tb = part * parts.steps, te = tb + parts.steps < d.T ? tb + parts.steps : (int)d.T;
  const int lane = threadIdx.x % 32, q = lane / W, n0 = q * S;
  const int k = (tile * (int)(blockDim.x / 32) + (int)threadIdx.x / 32) * W + lane % W;
  const bool on = k < d.Dg;
  const int64_t c = (int64_t)grp * d.Dg + (on ? k : 0);
  float2 A2[H], v[H];
  load_pairs<S>(a.A.ptr + set * a.A.stride + c * d.N, n0, d.N, false, A2);
#pragma unroll
  for (int i = 0; i < H; ++i) {
    A2[i] = rate_2(A2[i]);
    v[i] = two(0.f);
  }
  const float bias = a.delta_bias.ptr ? a.delta_bias.ptr[set * a.delta_bias.stride + c] : 0.f;
  const bool softplus = a.flags & ZO_SCAN_SOFTPLUS, gate = a.z.ptr;
  const int len = (int)row_length(a.lengths, row, d.T, nullptr, false), end = len < te ? len : te;
  const int t1 = tb + (end > tb ? (end - 1 - tb) / kTile * kTile : -kTile);  // the last tile
  const T* pd = static_cast<const T*>(a.delta.ptr) + row * a.delta.row + (int64_t)(t1 + kTile) * a.delta.step + c;
  const T* po = static_cast<const T*>(g.dout.ptr) + row * g.dout.row + (int64_t)(t1 + kTile) * g.dout.step + c;
  const T* pz = gate ? static_cast<const T*>(a.z.ptr) + row * a.z.row + (int64_t)(t1 + kTile) * a.z.step + c : nullptr;
  const T* pc = static_cast<const T*>(a.C.ptr) + row * a.C.row + (int64_t)grp * d.N;
  T rd[kAhead], ro[kAhead], rz[kAhead];
  auto load = [&](int t) {  // steps t .. t + kAhead - 1, those before the last loaded ones
    pd -= kAhead * a.delta.step;
    po -= kAhead * g.dout.step;
    if (gate) pz -= kAhead * a.z.step;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (t >= tb && t + j < end) {
        rd[j] = pd[j * a.delta.step];
        ro[j] = po[j * g.dout.step];
        if (gate) rz[j] = pz[j * a.z.step];
      }
  };
  auto fetch = [&](int t) {
    fetch_rows<T, NP>(&raw[0][0], pc + t * a.C.step, a.C.step, end - t < kTile ? end - t : kTile, d.N, copy);
  };
  float sum = 0.f;
  if (t1 >= tb) {
    load(t1 + kTile - kAhead);
    fetch(t1);
  }
  for (int t = t1; t >= tb; t -= kTile) {
    copies_done();
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * NP / 4; i += blockDim.x) {
      const int n = i % (NP / 4) * 4;
      float f[4];
      load_vec<T, 4>(&raw[0][0] + i * 4, f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j >= d.N || t + i / (NP / 4) >= end) f[j] = 0.f;
      store_vec<float, 4>(&C[0][0] + i * 4, f);
    }
    __syncthreads();
    if (t > tb) fetch(t - kTile);
#pragma unroll 1
    for (int s = kTile - kAhead; s >= 0; s -= kAhead) {
      const int n = end - t - s;  // steps that exist
      float2 dt[kAhead / 2], dy[kAhead / 2];
#pragma unroll
      for (int j = 0; j < kAhead; j += 2) {
        dt[j / 2] = __fadd2_rn(make_float2(to_f(rd[j]), to_f(rd[j + 1])), two(bias));
        dy[j / 2] = make_float2(j < n ? to_f(ro[j]) : 0.f, j + 1 < n ? to_f(ro[j + 1]) : 0.f);
        if (gate)
          dy[j / 2] = __fmul2_rn(dy[j / 2], silu_2(make_float2(j < n ? to_f(rz[j]) : 0.f, j + 1 < n ? to_f(rz[j + 1]) : 0.f)));
      }
      load(t + s - kAhead);
#pragma unroll
      for (int j = kAhead - 1; j >= 0; --j) {
        if (j % 2) {
          if (softplus) dt[j / 2] = softplus_2(dt[j / 2]);
          if (j - 1 >= n) dt[j / 2].x = 0.f;
          if (j >= n) dt[j / 2].y = 0.f;
          sum += dt[j / 2].x + dt[j / 2].y;
        }
        const float2 d1 = two(j % 2 ? dt[j / 2].y : dt[j / 2].x), y1 = two(j % 2 ? dy[j / 2].y : dy[j / 2].x);
        const float4* cs = reinterpret_cast<const float4*>(&C[s + j][n0]);
#pragma unroll
        for (int i = 0; i < H; i += 2) {
          const float4 f = cs[i / 2];
          v[i] = __fmul2_rn(decay_2<T>(d1, A2[i]), __ffma2_rn(y1, make_float2(f.x, f.y), v[i]));
          v[i + 1] = __fmul2_rn(decay_2<T>(d1, A2[i + 1]), __ffma2_rn(y1, make_float2(f.z, f.w), v[i + 1]));
        }
      }
    }
  }
  if (on) {
    const int64_t at = ((int64_t)row * parts.n + part) * d.D + c;
    store_pairs<S>(parts.state + at * d.N, n0, d.N, d.N % 4 == 0, v);
    if (q == 0) parts.sum[at] = sum;
  }
}

// state[row][k] becomes the carry that comes into part k at its end.
__global__ void __launch_bounds__(256) carry_join_kernel(zo_scan_args a, zo_scan_grads g, ScanDims d, Parts parts) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, DN = (int64_t)d.D * d.N;
  if (i >= a.rows * DN) return;
  const int64_t row = i / DN, cn = i % DN, c = cn / d.N, set = row / d.rows_per_set;
  const float A2 = rate(a.A.ptr[set * a.A.stride + cn]);
  float v = g.dstate_out.ptr ? g.dstate_out.ptr[row * g.dstate_out.stride + cn] : 0.f;
  float* state = parts.state + row * parts.n * DN + cn;
  const float* sum = parts.sum + row * parts.n * d.D + c;
  for (int k0 = parts.n - 1; k0 >= 0; k0 -= kJoin) {
    float l[kJoin], s[kJoin];
#pragma unroll
    for (int j = 0; j < kJoin; ++j)
      if (k0 - j > 0) {
        l[j] = state[(k0 - j) * DN];
        s[j] = sum[(int64_t)(k0 - j) * d.D];
      }
#pragma unroll
    for (int j = 0; j < kJoin; ++j)
      if (k0 - j >= 0) {
        state[(k0 - j) * DN] = v;
        v = carried(s[j] * A2, v, l[j]);
      }
  }
}

constexpr int kSub = 2;      // steps whose states and decays are in registers together
constexpr int kBlock = 4;    // steps between states kept in shared memory
constexpr int kFlush = 64;   // chunks after which the parameters' sums are put away

// Warps of a block at most: 128 channels.
template <int LN>
constexpr int kBackWarps = LN >= 4 ? 4 : LN;

template <int LN, int WARPS, int ZEROS>
struct BackTile {
  static constexpr int kWarps = WARPS, kThreads = 32 * kWarps;
  static constexpr int kWarpChannels = 128 / LN, kChannels = kWarps * kWarpChannels;
  static constexpr int NP = 4 * LN, kMid = kChunk / kBlock - 1;
  static constexpr int kRows = kChunk + ZEROS;             // ZEROS: a row of zeros behind the steps
  alignas(16) float d[kRows][kChannels], u[kRows][kChannels], dy[kRows][kChannels];
  float slope[kChunk][kChannels], zf[kChunk][kChannels];   // softplus'(raw), dout silu'(z)
  alignas(16) float2 B[kChunk][NP], C[kChunk][NP];         // each twice, for pairs of channels
  alignas(16) float4 mid[kMid][4][kThreads];               // the states before the later blocks
  float bc[kWarps][kChunk / 2][2 * NP];                    // the warps' sums for dB and dC, half a chunk
};

// What the backward pass leaves to be summed up: dB and dC by channel tile, the parameters'
// gradients by row, part and flush.
struct BackSums {
  float *bc, *param;  // param: [row, part, flush][D N of A, D of skip, D of the bias]
  int flushes;        // of a row's part
};

// A lane holds 4 neighbouring channels x 4 states, in pairs of channels: so the sums
// over a channel's states (12 values: two for the gradients, one for y) and those over
// channels (8 values: dB, dC) are both half done in the lane, and take 16 shuffles a step
// and warp where 16 states a lane would take 31 and 4 states of one channel a lane 37.
//
// Chunk by chunk backwards: the states are run forward from the chunk's checkpoint,
// keeping those before each block of kBlock steps in shared memory; then, backwards over the
// blocks and kSub steps at a time, states and decays are run again into registers and the carry
// comes back through them.  The exponentials are so done 2.25 times, which costs less than to
// keep every state in memory.  More steps in registers, or all states before kSub steps in
// shared memory, leave two blocks an SM instead of three (576 against 561 us, 649 against 561).
//
// Bound: latency.  It takes 570 instructions for 32 channels, 16 states and a step and 42 results
// of the special function unit a value, but no pipe is above 32% and 53% of the issue slots are used:
// 2.4 warps a scheduler do not hide the waits between dependent products and for a chunk's inputs.
// 4 rows x 2048 steps x 2048 channels: 562 us, and 124 us for the carries (their unit 67% busy),
// against 42 us of memory traffic for the whole training step.  Up to 8 states six warps an SM stay,
// at 254 registers a thread: with twelve and 168, and parts of time to match, 4 and 8 states take
// 531 and 578 us instead of 612 and 618 for those rows, and 1058 and 817 instead of 841 and 762
// for 32 x 512.  Blocks of one warp
// serve narrow groups: 12 rows x 2288 steps x 40 channels in 4 groups, forward and backward,
// 581 us with blocks of four warps only and 335 with either.
//
// GUARD: there are states beyond N (1 - whole lanes of them, if any; 2 - parts of lanes too), or there
// is no skip.  Those states and their carries and that skip are 0, but 0 times an infinite d u or dy is
// NaN.  So such lanes read zeros for these, and single states are left out of all sums.  It takes 1 to
// 2% of the time, 4% at 12 states and 7% at 3.
template <class T, int LN, int WARPS, int GUARD>
__global__ void __launch_bounds__(32 * WARPS, LN >= 4 ? 12 / WARPS : 6 / WARPS)
    scan_backward_kernel(zo_scan_args a, zo_scan_grads g, ScanDims d, Parts parts, BackSums sums, bool vec) {
  using S = BackTile<LN, WARPS, GUARD != 0>;
  extern __shared__ __align__(16) unsigned char smem[];
  S& sh = *reinterpret_cast<S*>(smem);
  const unsigned tiles = d.tiles * d.G;
  const unsigned tile_g = blockIdx.x % tiles, rest = blockIdx.x / tiles;
  const int part = rest % parts.n, row = rest / parts.n;
  const int tile = tile_g % d.tiles, grp = tile_g / d.tiles, set = row / d.rows_per_set;
  const int tb = part * parts.steps, te = tb + parts.steps < d.T ? tb + parts.steps : (int)d.T;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, q = lane % LN, n0 = 4 * q;
  const int ch = warp * S::kWarpChannels + lane / LN * 4;  // the lane's first channel in the tile
  const int left = d.Dg - tile * S::kChannels;             // channels of the group from the tile on
  const int64_t c0 = (int64_t)grp * d.Dg + tile * S::kChannels;
  const bool softplus = a.flags & ZO_SCAN_SOFTPLUS, gate = a.z.ptr;
  const int len = (int)row_length(a.lengths, row, d.T, a.status, tile == 0 && part == 0 && tid == 0);
  const int end = len < te ? len : te;

  // [state][pair of channels]
  float2 A2[4][2], gr[4][2], dA[4][2];
  auto load_lane = [&](const float* p, float2 (&f)[4][2]) {  // [channel][N] from the tile's first channel
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (ch + i < left) {
        const float* s = p + (int64_t)(ch + i) * d.N;
        if (d.N % 4 == 0 && reinterpret_cast<uintptr_t>(s) % 16 == 0)
          load_states4<true>(s, n0, d.N, v);
        else
          load_states4<false>(s, n0, d.N, v);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) (i % 2 ? f[n][i / 2].y : f[n][i / 2].x) = v[n];
    }
  };
  auto store_lane = [&](float* p, const float2 (&f)[4][2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (ch + i < left) {
        float v[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) v[n] = i % 2 ? f[n][i / 2].y : f[n][i / 2].x;
        store_states4<false>(p + (int64_t)(ch + i) * d.N, n0, d.N, v);
      }
  };
  load_lane(a.A.ptr + set * a.A.stride + c0 * d.N, A2);
  if (parts.n > 1)
    load_lane(parts.state + (((int64_t)row * parts.n + part) * d.D + c0) * d.N, gr);
  else if (g.dstate_out.ptr)
    load_lane(g.dstate_out.ptr + row * g.dstate_out.stride + c0 * d.N, gr);
  else
#pragma unroll
    for (int n = 0; n < 4; ++n) gr[n][0] = gr[n][1] = two(0.f);
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      A2[n][p] = rate_2(A2[n][p]);
      dA[n][p] = two(0.f);
    }

  // After the sums over states a lane has MC of its four channels, from `mine` on.
  constexpr int MC = LN >= 4 ? 1 : 4 / LN;
  const int mine = ch + (LN == 1 ? 0 : LN == 2 ? 2 * (q & 1) : 2 * (q & 1) + (q >> 1 & 1));
  float skip[MC], ds[MC], db[MC];
#pragma unroll
  for (int i = 0; i < MC; ++i) {
    skip[i] = a.skip.ptr && mine + i < left ? a.skip.ptr[set * a.skip.stride + c0 + mine + i] : 0.f;
    ds[i] = db[i] = 0.f;
  }
  const bool writes = LN < 4 || q < 4;
  T* pdu = static_cast<T*>(g.du.ptr) + row * g.du.row + c0 + mine;
  T* pdd = static_cast<T*>(g.ddelta.ptr) + row * g.ddelta.row + c0 + mine;
  T* pdz = static_cast<T*>(g.dz.ptr) + (gate ? row * g.dz.row + c0 + mine : 0);

  // behind the row's end
  if (writes)
    for (int t = end > tb ? end : tb; t < te; ++t)
#pragma unroll
      for (int i = 0; i < MC; ++i)
        if (mine + i < left) {
          pdu[t * g.du.step + i] = from_f<T>(0.f);
          pdd[t * g.ddelta.step + i] = from_f<T>(0.f);
          if (gate) pdz[t * g.dz.step + i] = from_f<T>(0.f);
        }

  int flush = 0;
  auto put_away = [&] {  // the parameters' sums so far
    const int64_t at = ((int64_t)row * parts.n + part) * sums.flushes + flush++;
    float* p = sums.param + at * ((int64_t)d.D * (d.N + 2));
    store_lane(p + c0 * d.N, dA);
#pragma unroll
    for (int n = 0; n < 4; ++n) dA[n][0] = dA[n][1] = two(0.f);
#pragma unroll
    for (int i = 0; i < MC; ++i) {
      if (writes && mine + i < left) {
        p[(int64_t)d.D * d.N + c0 + mine + i] = ds[i];
        p[(int64_t)d.D * (d.N + 1) + c0 + mine + i] = db[i];
      }
      ds[i] = db[i] = 0.f;
    }
  };

  const T* bu = static_cast<const T*>(a.u.ptr) + row * a.u.row + c0;
  const T* bd = static_cast<const T*>(a.delta.ptr) + row * a.delta.row + c0;
  const T* bz = static_cast<const T*>(a.z.ptr) + (gate ? row * a.z.row + c0 : 0);
  const T* bo = static_cast<const T*>(g.dout.ptr) + row * g.dout.row + c0;
  const T* bB = static_cast<const T*>(a.B.ptr) + row * a.B.row + (int64_t)grp * d.N;
  const T* bC = static_cast<const T*>(a.C.ptr) + row * a.C.row + (int64_t)grp * d.N;

  // A thread takes the same four channels of every step that it prepares.
  constexpr int kQuads = S::kChannels / 4;
  const int pc = tid % kQuads * 4;
  float bias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    bias[e] = a.delta_bias.ptr && pc + e < left ? a.delta_bias.ptr[set * a.delta_bias.stride + c0 + pc + e] : 0.f;

  const bool none = GUARD && LN > 2 && n0 >= d.N;  // a lane without states
  if (GUARD)
    for (int i = tid; i < S::kChannels; i += S::kThreads) sh.d[S::kRows - 1][i] = sh.u[S::kRows - 1][i] = sh.dy[S::kRows - 1][i] = 0.f;
  int chunks = 0;
  for (int t0 = end > tb ? tb + (end - 1 - tb) / kChunk * kChunk : tb - 1; t0 >= tb; t0 -= kChunk) {
    __syncthreads();
    // The chunk's inputs and what is one channel's and step's, four channels at a time.
#pragma unroll 2
    for (int s = tid / kQuads; s < kChunk; s += S::kThreads / kQuads) {
      const int c = pc;
      const int64_t t = t0 + s;
      float fu[4] = {}, fd[4] = {}, fz[4] = {}, fo[4] = {};
      if (t < end) {
        if (vec && c < left) {
          load_vec<T, 4>(bu + t * a.u.step + c, fu);
          load_vec<T, 4>(bd + t * a.delta.step + c, fd);
          load_vec<T, 4>(bo + t * g.dout.step + c, fo);
          if (gate) load_vec<T, 4>(bz + t * a.z.step + c, fz);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < left) {
              fu[e] = to_f(bu[t * a.u.step + c + e]);
              fd[e] = to_f(bd[t * a.delta.step + c + e]);
              fo[e] = to_f(bo[t * g.dout.step + c + e]);
              if (gate) fz[e] = to_f(bz[t * a.z.step + c + e]);
            }
        }
      }
      float o[5][4];
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 k = make_float2(bias[e], bias[e + 1]);
        const float2 raw = __fadd2_rn(make_float2(fd[e], fd[e + 1]), k);
        float2 dt = raw, slope = two(1.f), dy = make_float2(fo[e], fo[e + 1]), zf = two(0.f);
        if (softplus) {
          dt = softplus_2(raw);
          slope = sigmoid_2(raw);
        }
        if (gate) {
          float2 v;  // silu(z)
          silu_slope_2(make_float2(fz[e], fz[e + 1]), v, zf);
          zf = __fmul2_rn(dy, zf);
          dy = __fmul2_rn(dy, v);
        }
        const bool in = t < end;
        o[0][e] = in ? dt.x : 0.f, o[0][e + 1] = in ? dt.y : 0.f;
        o[1][e] = fu[e], o[1][e + 1] = fu[e + 1];
        o[2][e] = dy.x, o[2][e + 1] = dy.y;
        o[3][e] = slope.x, o[3][e + 1] = slope.y;
        o[4][e] = zf.x, o[4][e + 1] = zf.y;
      }
      store_vec<float, 4>(&sh.d[s][c], o[0]);
      store_vec<float, 4>(&sh.u[s][c], o[1]);
      store_vec<float, 4>(&sh.dy[s][c], o[2]);
      store_vec<float, 4>(&sh.slope[s][c], o[3]);
      store_vec<float, 4>(&sh.zf[s][c], o[4]);
    }
    for (int i = tid; i < kChunk * S::NP; i += S::kThreads) {
      const int s = i / S::NP, n = i % S::NP;
      const bool in = t0 + s < end && n < d.N;
      sh.B[s][n] = two(in ? to_f(bB[(t0 + s) * a.B.step + n]) : 0.f);
      sh.C[s][n] = two(in ? to_f(bC[(t0 + s) * a.C.step + n]) : 0.f);
    }
    float2 h0[4][2];
    load_lane(a.checkpoints + ((row * d.chunks + t0 / kChunk) * d.D + c0) * d.N, h0);
    if (t0 - kChunk >= tb) {  // the chunk before: its inputs come nearer meanwhile
      constexpr int kLine = 128 / (int)sizeof(T), kLines = (S::kChannels + kLine - 1) / kLine;
      for (int i = tid; i < 4 * kChunk * kLines; i += S::kThreads) {
        const int c = i % kLines * kLine, which = i / kLines % 4;
        const int64_t t = t0 - kChunk + i / (4 * kLines);
        const T* p = which == 0 ? bu + t * a.u.step : which == 1 ? bd + t * a.delta.step
                     : which == 2 ? bo + t * g.dout.step : bz + t * a.z.step;
        if (c < left && (which < 3 || gate)) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c));
      }
    }
    __syncthreads();

    auto load4 = [&](const float2* p, float2 (&f)[4]) {
      const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
      f[0] = make_float2(x.x, x.y), f[1] = make_float2(x.z, x.w);
      f[2] = make_float2(y.x, y.y), f[3] = make_float2(y.z, y.w);
    };
    auto step = [&](auto slow, int s, float2 (&h)[4][2], float2 (&at)[4][2]) {
      const int at_s = none ? S::kRows - 1 : s;
      const float4 dt = *reinterpret_cast<const float4*>(&sh.d[at_s][ch]);
      const float4 u = *reinterpret_cast<const float4*>(&sh.u[at_s][ch]);
      float2 b[4];
      load4(&sh.B[s][n0], b);
      const float2 d2[2] = {make_float2(dt.x, dt.y), make_float2(dt.z, dt.w)};
      const float2 x2[2] = {__fmul2_rn(d2[0], make_float2(u.x, u.y)), __fmul2_rn(d2[1], make_float2(u.z, u.w))};
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float2 x = __fmul2_rn(d2[p], A2[n][p]);
          at[n][p] = decltype(slow)::value ? exp2_slow_2(x) : exp2_2(x);
          h[n][p] = __ffma2_rn(at[n][p], h[n][p], __fmul2_rn(x2[p], b[n]));
        }
    };
    float2 hs[kSub + 1][4][2], at[kSub][4][2];
    const int blocks = (end - t0 < kChunk ? end - t0 + kBlock - 1 : kChunk) / kBlock;
    const int subs = (end - t0 < kChunk ? end - t0 + kSub - 1 : kChunk) / kSub;
#pragma unroll 1
    for (int m = 0; m + 1 < blocks; ++m) {
#pragma unroll
      for (int j = 0; j < kBlock; ++j) step(std::false_type(), m * kBlock + j, h0, at[0]);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        sh.mid[m][n][tid] = make_float4(h0[n][0].x, h0[n][0].y, h0[n][1].x, h0[n][1].y);
    }
    float cs[MC] = {}, cb[MC] = {};  // the chunk's sums for dskip and dbias
    const int64_t after = t0 + subs * kSub;
    T *wu = pdu + after * g.du.step, *wd = pdd + after * g.ddelta.step, *wz = pdz + (gate ? after * g.dz.step : 0);
#pragma unroll 1
    for (int m = subs - 1; m >= 0; --m) {
      constexpr int R = kBlock / kSub;
      if (m >= R) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float4 f = sh.mid[m / R - 1][n][tid];
          hs[0][n][0] = make_float2(f.x, f.y);
          hs[0][n][1] = make_float2(f.z, f.w);
        }
      } else {
        load_lane(a.checkpoints + ((row * d.chunks + t0 / kChunk) * d.D + c0) * d.N, hs[0]);
      }
#pragma unroll 1
      for (int k = m / R * R; k < m; ++k)  // from the block's first step
#pragma unroll
        for (int j = 0; j < kSub; ++j) step(std::false_type(), k * kSub + j, hs[0], at[0]);
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
#pragma unroll
        for (int n = 0; n < 4; ++n) hs[j + 1][n][0] = hs[j][n][0], hs[j + 1][n][1] = hs[j][n][1];
        step(std::true_type(), m * kSub + j, hs[j + 1], at[j]);
      }
#pragma unroll
      for (int j = kSub - 1; j >= 0; --j) {
        const int s = m * kSub + j;
        const int at_s = none ? S::kRows - 1 : s;
        const float4 d4 = *reinterpret_cast<const float4*>(&sh.d[at_s][ch]);
        const float4 u4 = *reinterpret_cast<const float4*>(&sh.u[at_s][ch]);
        const float4 y4 = *reinterpret_cast<const float4*>(&sh.dy[at_s][ch]);
        float2 b[4], c[4];
        load4(&sh.B[s][n0], b);
        load4(&sh.C[s][n0], c);
        const float2 d2[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
        const float2 x2[2] = {__fmul2_rn(d2[0], make_float2(u4.x, u4.y)), __fmul2_rn(d2[1], make_float2(u4.z, u4.w))};
        const float2 y2[2] = {make_float2(y4.x, y4.y), make_float2(y4.z, y4.w)};
        float2 gA[2] = {two(0.f), two(0.f)}, gB[2] = {two(0.f), two(0.f)}, y[2] = {two(0.f), two(0.f)};
        float v[8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int p = 0; p < 2; ++p) gr[n][p] = __ffma2_rn(c[n], y2[p], gr[n][p]);
          const float2 tb2 = __ffma2_rn(x2[1], gr[n][1], __fmul2_rn(x2[0], gr[n][0]));
          const float2 tc2 = __ffma2_rn(y2[1], hs[j + 1][n][1], __fmul2_rn(y2[0], hs[j + 1][n][0]));
          v[n] = tb2.x + tb2.y;
          v[4 + n] = tc2.x + tc2.y;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const bool real = GUARD < 2 || n0 + n < d.N;
            if (real) y[p] = __ffma2_rn(c[n], hs[j + 1][n][p], y[p]);
            if (real) gB[p] = __ffma2_rn(b[n], gr[n][p], gB[p]);
            gr[n][p] = __fmul2_rn(gr[n][p], at[j][n][p]);
            const float2 w = __fmul2_rn(gr[n][p], hs[j][n][p]);
            if (real) gA[p] = __ffma2_rn(w, A2[n][p], gA[p]);
            dA[n][p] = __ffma2_rn(w, d2[p], dA[n][p]);
          }
        }
        constexpr int CG = 32 / LN;
        sum_over<8, CG, LN>(v, lane);
        {
          constexpr int NB = CG < 8 ? 8 / CG : 1;  // values the lane now has
          const int cg = lane / LN;
          int idx = 0;
#pragma unroll
          for (int bit = 0; (1 << bit) < (CG < 8 ? CG : 8); ++bit) idx += (cg >> bit & 1) * (4 >> bit);
          if (CG <= 8 || cg < 8)
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              const int id = idx + i;  // B or C, state
              sh.bc[warp][s % (kChunk / 2)][id / 4 * S::NP + n0 + id % 4] = v[i];
            }
        }
        float r[12];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[3 * i] = i % 2 ? gA[i / 2].y : gA[i / 2].x;
          r[3 * i + 1] = i % 2 ? gB[i / 2].y : gB[i / 2].x;
          r[3 * i + 2] = i % 2 ? y[i / 2].y : y[i / 2].x;
        }
        sum_over12<LN>(r, lane);
        wu -= g.du.step;
        wd -= g.ddelta.step;
        if (gate) wz -= g.dz.step;
        if (writes && t0 + s < end)
#pragma unroll
          for (int i = 0; i < MC; ++i) {
            const int k = mine + i;
            const float u = sh.u[s][k], dyk = sh.dy[s][k];
            const float dr = fmaf(r[3 * i], kLn2, r[3 * i + 1] * u) * sh.slope[s][k];
            cs[i] = fmaf(dyk, u, cs[i]);
            cb[i] += dr;
            if (k < left) {
              const bool skips = !GUARD || a.skip.ptr;
              wu[i] = from_f<T>(fmaf(r[3 * i + 1], sh.d[s][k], skips ? skip[i] * dyk : 0.f));
              wd[i] = from_f<T>(dr);
              if (gate) wz[i] = from_f<T>(sh.zf[s][k] * (skips ? fmaf(skip[i], u, r[3 * i + 2]) : r[3 * i + 2]));
            }
          }
      }
      if (m * kSub % (kChunk / 2) == 0) {  // [tile][row][t][group][dB, dC][N]
        __syncthreads();
        for (int i = tid; i < kChunk / 2 * 2 * d.N; i += S::kThreads) {
          const int n = i % d.N, k = i / d.N % 2, s = i / d.N / 2;
          const int64_t t = t0 + m * kSub + s;
          if (t < end) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) v += sh.bc[w][s][k * S::NP + n];
            sums.bc[((((int64_t)tile * a.rows + row) * d.T + t) * d.G + grp) * 2 * d.N + k * d.N + n] = v;
          }
        }
        __syncthreads();
      }
    }
#pragma unroll
    for (int i = 0; i < MC; ++i) {
      ds[i] += cs[i];
      db[i] += cb[i];
    }
    if (++chunks % kFlush == 0) put_away();
  }
  while (flush < sums.flushes) put_away();
  if (part == 0 && g.dstate_in.ptr)
    store_lane(g.dstate_in.ptr + row * g.dstate_in.stride + c0 * d.N, gr);
}

template <class T>
__global__ void __launch_bounds__(256)
    sum_bc_kernel(zo_scan_args a, zo_scan_grads g, ScanDims d, const float* part) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per_step = (int64_t)d.G * 2 * d.N, n = a.rows * d.T * per_step;
  if (i >= n) return;
  float v = 0.f;
  const int64_t row = i / per_step / d.T, t = i / per_step % d.T;
  if (t < row_length(a.lengths, row, d.T, nullptr, false))
    for (int k = 0; k < d.tiles; ++k) v += part[k * n + i];
  const int j = (int)(i % per_step), grp = j / (2 * d.N), q = j / d.N % 2, k = j % d.N;
  const zo_tensor& o = q ? g.dC : g.dB;
  static_cast<T*>(o.ptr)[row * o.row + t * o.step + (int64_t)grp * d.N + k] = from_f<T>(v);
}

// The backward pass's division of time: parts, which cost a pass over the carries, wherever the
// SMs hold twice the blocks.  2048 steps of 2048 channels in one pass and in parts: 2 rows
// (32 blocks) 2050 and 328 us, 8 rows 2073 and 1255, 12 rows 2518 and 1859.
struct BackPlan {
  int warps, tiles, parts, steps, flushes;
  int64_t bc, param, state, sum;  // floats of workspace
};
template <int LN>
BackPlan back_plan(const zo_scan_args& a) {
  BackPlan p;
  // Blocks of several warps share B and C and leave fewer partial sums; blocks of one where the
  // others would leave a fifth of their warps without channels.
  const int64_t w = ceil_div(a.channels / a.groups, 128 / LN), most = kBackWarps<LN>;
  p.warps = 5 * ceil_div(w, most) * most > 6 * w ? 1 : (int)most;
  p.tiles = (int)ceil_div(w, p.warps);
  const int64_t blocks = (int64_t)p.tiles * a.groups * a.rows;
  const int64_t room = (LN >= 4 ? 12 : 6) / p.warps * kBlockSMs;  // blocks that the SMs hold
  int64_t n = blocks * 2 < room ? room / blocks : 1;
  int64_t steps = ceil_div(ceil_div(a.seq, n), kChunk) * kChunk;
  if (n > 1 && steps < 32) steps = 32;
  p.parts = (int)ceil_div(a.seq, steps);
  p.steps = (int)steps;
  p.flushes = (int)ceil_div(steps / kChunk, kFlush);
  const int64_t DN = (int64_t)a.channels * a.states, each = (int64_t)a.rows * p.parts;
  p.bc = (int64_t)p.tiles * a.rows * a.seq * a.groups * 2 * a.states;
  p.param = each * p.flushes * (DN + 2 * a.channels);
  p.state = p.parts > 1 ? each * DN : 0;
  p.sum = p.parts > 1 ? each * a.channels : 0;
  return p;
}

template <class T, int LN, int S, int LC>
cudaError_t run_scan_backward(const zo_scan_args& a, const zo_scan_grads& g, float* ws,
                              cudaStream_t st) {
  const BackPlan p = back_plan<LN>(a);
  ScanDims d = scan_dims(a);
  d.tiles = p.tiles;
  const int64_t DN = (int64_t)d.D * d.N, blocks = (int64_t)p.tiles * d.G * a.rows * p.parts;
  const int64_t bc = (int64_t)a.rows * d.T * d.G * 2 * d.N;
  if (blocks > INT32_MAX || ceil_div(bc, 256) > INT32_MAX) return cudaErrorInvalidConfiguration;
  float* state = ws;  // first, for its alignment
  float* param = state + ceil_div(p.state, 4) * 4;
  const BackSums sums{param + p.param, param, p.flushes};
  const Parts parts{p.parts, p.steps, state, param + p.param + p.bc};
  cudaError_t e = cudaSuccess;
  if (p.parts > 1) {
    const ScanPlan f = scan_plan(a);  // its blocks' shape
    ScanDims dc = d;
    dc.tiles = f.tiles;
    const int64_t carry = (int64_t)f.tiles * d.G * a.rows * (p.parts - 1);
    if (carry > INT32_MAX) return cudaErrorInvalidConfiguration;
    scan_carry_kernel<T, S, LC><<<(unsigned)carry, 32 * f.warps, 0, st>>>(
        a, g, dc, parts, copy_bytes({&a.C}, sizeof(T), d.N));
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    carry_join_kernel<<<(unsigned)ceil_div(a.rows * DN, 256), 256, 0, st>>>(a, g, d, parts);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  bool vec = true;
  for (const zo_tensor* t : {&a.u, &a.delta, &a.z, &g.dout})
    vec = vec && vec_width(*t, sizeof(T), d.Dg, 4) == 4;
  auto launch = [&](auto warps) {
    constexpr int W = decltype(warps)::value;
    const int guard = d.N % 4 ? 2 : d.N < 4 * LN || !a.skip.ptr ? 1 : 0;
    const int smem = guard ? (int)sizeof(BackTile<LN, W, 1>) : (int)sizeof(BackTile<LN, W, 0>);
    auto kernel = guard == 2 ? scan_backward_kernel<T, LN, W, 2>
                  : guard ? scan_backward_kernel<T, LN, W, 1> : scan_backward_kernel<T, LN, W, 0>;
    const cudaError_t r = allow_shared(kernel, smem);
    if (r != cudaSuccess) return r;
    kernel<<<(unsigned)blocks, 32 * W, smem, st>>>(a, g, d, parts, sums, vec);
    count_launch();
    return cudaGetLastError();
  };
  e = p.warps == 1 ? launch(std::integral_constant<int, 1>()) : launch(std::integral_constant<int, kBackWarps<LN>>());
  if (e != cudaSuccess) return e;
  sum_bc_kernel<T><<<(unsigned)ceil_div(bc, 256), 256, 0, st>>>(a, g, d, sums.bc);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const SumOut outs[3] = {{g.dA, DN}, {g.dskip, d.D}, {g.ddelta_bias, d.D}};
  return launch_sum_parts(sums.param, a.sets, (int64_t)d.rows_per_set * p.parts * p.flushes, DN + 2 * d.D, outs, 3, st);
}

}  // namespace

int64_t scan_backward_workspace(const zo_scan_args& a) {
  return by_lanes(a.states, [&](auto ln) {
    const BackPlan p = back_plan<decltype(ln)::value>(a);
    return (int64_t)sizeof(float) * (p.bc + p.param + ceil_div(p.state, 4) * 4 + p.sum);
  });
}

cudaError_t launch_scan_backward(const zo_scan_args& a, const zo_scan_grads& g, float* ws,
                                 cudaStream_t st) {
  return by_type(a.dtype, [&](auto t) {
    return by_lanes(a.states, [&](auto ln) {
      constexpr int L = decltype(ln)::value;  // four states a lane; the carry's kernel has up to 16
      return run_scan_backward<decltype(t), L, L == 1 ? 4 : L == 2 ? 8 : 16, L <= 4 ? 1 : L / 4>(a, g, ws, st);
    });
  });
}

}  // namespace zo
