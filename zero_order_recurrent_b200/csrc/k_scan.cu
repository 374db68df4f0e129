// Selective scan: per row, channel and state h_t = exp(d_t A) h_{t-1} + d_t u_t B_t,
// y_t = sum_n C_t h_t + skip u_t, out_t = y_t silu(z_t), d_t = softplus(delta_t + bias);
// and its single-token form.  States, carries and sums are fp32.  (Gradients: k_scan_backward.cu.)
//
// exp(d A) is 2^(d A log2(e)) by the special function unit (2^-22 relative) and, near 1 where such
// errors add up over a state's memory, a polynomial (decay_2).  It is not the tensor cores' work:
// every channel and state has its own decay at every step, so no step is a matrix product.  Times
// below are at 16 states and bf16.
#include "k_scan.cuh"

namespace zo {
namespace {

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
// states takes 16 exponentials and 4 for softplus and silu, so 20 / 16 clocks; its
// 8 bytes in bf16 take 0.34 clocks of an SM's share of the memory.  The 16
// exponentials of one step are independent.  Four states a lane and four warps along
// time, each keeping its decays in registers for a second run, make more warps without parts,
// but took 7.6 instructions a value, which bound them, against 3.6 here.
//
// Where rows and channels are too few for the SMs, time is divided as well: LOCAL
// runs each part but the last from the state 0, scan_join_kernel passes the states
// on from part to part, and then all parts run from the states they start with.
// That takes the exponentials and softplus twice.
//
// Measured: 4096 rows x 10 steps x 1024 channels with states in and out 333 us (2.6 TB/s; by
// the unit's count 186, which is 56% busy: the rest waits between dependent products, for a row's
// state and at a tile's barriers, with 4 warps a scheduler); 1 row x 16384 steps x 2048 channels in
// 37 parts 397 us (by its count 280, 77% busy from the state 0 and 70% with the states).  With fp32
// activations 374 and 494 us.
//
// A block takes `rows` rows of one set one after the other.
//
// GUARD: there are lanes with states beyond N, or there is no skip.  Those states are 0, as B is there,
// and so is that skip, but 0 times an infinite d u or u is NaN: such a step puts the states back and
// takes its y again, and adds no skip.  It takes 2 to 3% of the time.
template <class T, int S, int LN, bool LOCAL, bool GUARD>
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
  for (int i = 0; i < H; ++i) A2[i] = rate_2(A2[i]);
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
    if (!LOCAL && more && a.state_in.ptr && n0 < d.N)  // on its way while this row is computed
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.state_in.ptr + (row + 1) * a.state_in.stride + c * d.N + n0));
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
                h[i] = __ffma2_rn(decay_2<T>(d1, A2[i]), h[i], __fmul2_rn(x1, make_float2(b.x, b.y)));
                h[i + 1] = __ffma2_rn(decay_2<T>(d1, A2[i + 1]), h[i + 1], __fmul2_rn(x1, make_float2(b.z, b.w)));
                if (!LOCAL) {
                  const float4 v = C[i / 2];
                  y = __ffma2_rn(make_float2(v.x, v.y), h[i], y);
                  y = __ffma2_rn(make_float2(v.z, v.w), h[i + 1], y);
                }
              }
              if (GUARD && !(fabsf(x1.x) <= FLT_MAX)) {
                y = two(0.f);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                  if (n0 + 2 * i >= d.N) h[i].x = 0.f;
                  if (n0 + 2 * i + 1 >= d.N) h[i].y = 0.f;
                  y = __ffma2_rn(reinterpret_cast<const float2*>(C)[i], h[i], y);
                }
              }
              if (!LOCAL) {
                float v = y.x + y.y;
#pragma unroll
                for (int m = W; m < 32; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
                if (!GUARD || a.skip.ptr) v = fmaf(skip, e ? u.y : u.x, v);
                v *= e ? gz.y : gz.x;
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
  const float A2 = rate(a.A.ptr[set * a.A.stride + cn]);
  float h = a.state_in.ptr ? a.state_in.ptr[row * a.state_in.stride + cn] : 0.f;
  float* state = parts.state + row * parts.n * DN + cn;
  const float* sum = parts.sum + row * parts.n * d.D + c;
  for (int k0 = 0; k0 < parts.n; k0 += kJoin) {
    float l[kJoin], s[kJoin];
#pragma unroll
    for (int j = 0; j < kJoin; ++j)
      if (k0 + j + 1 < parts.n) {
        l[j] = state[(k0 + j) * DN];
        s[j] = sum[(int64_t)(k0 + j) * d.D];
      }
#pragma unroll
    for (int j = 0; j < kJoin; ++j)
      if (k0 + j < parts.n) {
        state[(k0 + j) * DN] = h;
        h = carried(s[j] * A2, h, l[j]);
      }
  }
}

// One token.  A thread holds four states of a channel and walks RG rows of a
// set, so that A is read once for them; all its loads are issued before the first result is
// waited for.  Bound: the states, read and written: 512 rows x 4096 channels take 60 us, 4.8 TB/s.
// HOW: 2 - there is a skip, and every lane has four states, which, like those of A, B and C, are on
// 16 (8) bytes; 3 - so, without skip; 1 - so, but lanes behind the last state may have none;
// 0 - states one at a time.
template <class T, int LN, int RG, int HOW>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(zo_scan_args a, ScanDims d, unsigned groups) {
  const unsigned nb = ((unsigned)d.D * LN + kThreads - 1) / kThreads;  // blocks of a row
  const unsigned i = blockIdx.x % nb * kThreads + threadIdx.x;        // (channel, lane)
  const int q = (int)(i % LN), n0 = q * 4;
  const bool on = i / LN < (unsigned)d.D;
  const int c = on ? (int)(i / LN) : 0;
  const unsigned first = blockIdx.x / nb * RG, set = first / groups, in_set = first % groups;
  const int have = d.rows_per_set - (int)in_set;  // rows of the set from the first on
  const int64_t r0 = (int64_t)set * d.rows_per_set + in_set;
  const int64_t g = c / d.Dg, cn = (int64_t)c * d.N;
  auto four = [&](auto* p, auto& x) {  // p[n0 ..], zeros from N on
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    if constexpr (HOW >= 2) {
      x = *reinterpret_cast<const Vec<E, 4>*>(p + n0);
    } else if constexpr (HOW == 1) {
      x = load_if<E, 4>(p + n0, n0 < d.N);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x.v[j] = load_if<E, 1>(p + n0 + j, n0 + j < d.N).v[0];
    }
  };
  Vec<float, 4> A, h[RG];
  Vec<T, 4> B[RG], C[RG];
  T u[RG], dl[RG], z[RG];
  const T* pz = static_cast<const T*>(a.z.ptr ? a.z.ptr : a.u.ptr);
  const int64_t z_row = a.z.ptr ? a.z.row : a.u.row;
#pragma unroll
  for (int k = 0; k < RG; ++k) {
    const int64_t row = r0 + (k < have ? k : have - 1);  // the last row again behind it
    four(static_cast<const float*>(a.state_in.ptr) + row * a.state_in.stride + cn, h[k]);
    four(static_cast<const T*>(a.B.ptr) + row * a.B.row + g * d.N, B[k]);
    four(static_cast<const T*>(a.C.ptr) + row * a.C.row + g * d.N, C[k]);
    u[k] = static_cast<const T*>(a.u.ptr)[row * a.u.row + c];
    dl[k] = static_cast<const T*>(a.delta.ptr)[row * a.delta.row + c];
    z[k] = pz[row * z_row + c];
  }
  four(static_cast<const float*>(a.A.ptr) + set * a.A.stride + cn, A);
  const float2 A2[2] = {make_float2(rate(A.v[0]), rate(A.v[1])), make_float2(rate(A.v[2]), rate(A.v[3]))};
  const float skip = a.skip.ptr ? a.skip.ptr[set * a.skip.stride + c] : 0.f;
  const float bias = a.delta_bias.ptr ? a.delta_bias.ptr[set * a.delta_bias.stride + c] : 0.f;
#pragma unroll
  for (int k0 = 0; k0 < RG; k0 += 2) {  // two rows at a time where one channel's work is done
    constexpr int P = RG > 1 ? 2 : 1;
    if (k0 >= have) break;
    const int k1 = k0 + P - 1;
    const float2 uu = make_float2(to_f(u[k0]), to_f(u[k1]));
    float2 dt = __fadd2_rn(make_float2(to_f(dl[k0]), to_f(dl[k1])), two(bias));
    if (a.flags & ZO_SCAN_SOFTPLUS) dt = softplus_2(dt);
    const float2 xx = __fmul2_rn(dt, uu);
    const float2 gate = a.z.ptr ? silu_2(make_float2(to_f(z[k0]), to_f(z[k1]))) : two(1.f);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const int k = k0 + e;
      if (k >= have) break;
      const float2 x = two(e ? xx.y : xx.x), d2 = two(e ? dt.y : dt.x);
      float2 y = two(0.f);
      float f[4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 v = __ffma2_rn(decay_2<T>(d2, A2[p]), make_float2(h[k].v[2 * p], h[k].v[2 * p + 1]),
                                    __fmul2_rn(x, make_float2(to_f(B[k].v[2 * p]), to_f(B[k].v[2 * p + 1]))));
        float2 in_y = v;  // states beyond N (of lanes, or one by one) add nothing, not even where d u is infinite
        if (HOW == 0 && n0 + 2 * p >= d.N) in_y.x = 0.f;
        if (HOW == 0 && n0 + 2 * p + 1 >= d.N) in_y.y = 0.f;
        if (HOW == 1 && n0 >= d.N) in_y = two(0.f);
        y = __ffma2_rn(make_float2(to_f(C[k].v[2 * p]), to_f(C[k].v[2 * p + 1])), in_y, y);
        f[2 * p] = v.x, f[2 * p + 1] = v.y;
      }
      const int64_t row = r0 + k;
      if (on && a.state_out.ptr)
        store_states4<HOW != 0>(a.state_out.ptr + row * a.state_out.stride + cn, n0, d.N, f);
      float out = sum_lanes<LN>(y.x + y.y);
      if (HOW == 2 || (HOW < 2 && a.skip.ptr)) out = fmaf(skip, e ? uu.y : uu.x, out);
      out *= e ? gate.y : gate.x;
      if (on && q == 0) static_cast<T*>(a.out.ptr)[row * a.out.row + c] = from_f<T>(out);
    }
  }
}

template <class T, int S, int LN>
cudaError_t run_scan(const zo_scan_args& a, float* ws, cudaStream_t st) {
  const ScanPlan plan = scan_plan(a);
  ScanDims d = scan_dims(a);
  d.tiles = plan.tiles;
  const int64_t DN = (int64_t)d.D * d.N;
  const Parts parts{plan.parts, plan.steps, ws, ws + (int64_t)a.rows * plan.parts * DN};
  // Short rows go several to a block, as long as that leaves 16 blocks an SM: A
  // and the block's first loads are waited for once for all of them.  4096 rows x 1024 channels
  // with one row and with several a block: 10 steps 416 and 337 us, 40 steps 1039 and 1052.
  const int64_t per_row = (int64_t)d.tiles * d.G;
  int64_t rows = plan.parts == 1 && a.seq <= 2 * kTile ? per_row * a.rows / (16 * kBlockSMs) : 1;
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
    if ((e = allow_shared(scan_kernel<T, S, LN, true, false>, kSmem)) != cudaSuccess) return e;
    scan_kernel<T, S, LN, true, false><<<(unsigned)(per_row * row_blocks * (plan.parts - 1)), threads, kSmem, st>>>(
        a, d, parts, (int)rows, copy, d.N % 4 == 0);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    scan_join_kernel<<<(unsigned)ceil_div(a.rows * DN, 256), 256, 0, st>>>(a, d, parts);
    count_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  auto kernel = d.N < S * LN || !a.skip.ptr ? scan_kernel<T, S, LN, false, true> : scan_kernel<T, S, LN, false, false>;
  if ((e = allow_shared(kernel, kSmem)) != cudaSuccess) return e;
  kernel<<<(unsigned)blocks, threads, kSmem, st>>>(a, d, parts, (int)rows, copy, wide);
  count_launch();
  return cudaGetLastError();
}

template <class T, int LN, int RG>
cudaError_t run_scan_step(const zo_scan_args& a, cudaStream_t st) {
  const ScanDims d = scan_dims(a);
  const int64_t groups = ceil_div(d.rows_per_set, RG) * RG;  // rows of a set, whole groups
  const int64_t blocks = ceil_div((int64_t)d.D * LN, kThreads) * (groups / RG) * a.sets;
  if (blocks > INT32_MAX || (int64_t)d.D * LN > INT32_MAX || groups * a.sets > UINT32_MAX)
    return cudaErrorInvalidConfiguration;
  bool wide = d.N % 4 == 0;
  for (const zo_f32* p : {&a.A, &a.state_in, &a.state_out})
    wide = wide && p->stride % 4 == 0 && reinterpret_cast<uintptr_t>(p->ptr) % 16 == 0;
  for (const zo_tensor* t : {&a.B, &a.C}) wide = wide && vec_width(*t, sizeof(T), 4, 4) == 4;
  if (wide && d.N == 4 * LN && a.skip.ptr)
    scan_step_kernel<T, LN, RG, 2><<<(unsigned)blocks, kThreads, 0, st>>>(a, d, (unsigned)groups);
  else if (wide && d.N == 4 * LN)
    scan_step_kernel<T, LN, RG, 3><<<(unsigned)blocks, kThreads, 0, st>>>(a, d, (unsigned)groups);
  else if (wide)
    scan_step_kernel<T, LN, RG, 1><<<(unsigned)blocks, kThreads, 0, st>>>(a, d, (unsigned)groups);
  else
    scan_step_kernel<T, LN, RG, 0><<<(unsigned)blocks, kThreads, 0, st>>>(a, d, (unsigned)groups);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

int64_t scan_workspace(const zo_scan_args& a) {
  const ScanPlan p = scan_plan(a);
  return p.parts == 1 ? 0 : (int64_t)a.rows * p.parts * a.channels * (a.states + 1) * (int64_t)sizeof(float);
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
      // Several rows a thread once that leaves enough threads for the memory's latency: one and
      // four rows a thread take 93 and 62 us for 512 rows of 4096 channels in one set, 22 and 23 for
      // 64.  A set's last thread loads its last row again for those that it lacks: in sets of four
      // and five rows 95 and 68, 95 and 83, of two 97 either way, and of one row 99 and 161.
      const int64_t threads = (int64_t)a.rows * a.channels * LN;
      return threads >= 4ll * kBlockSMs * 2048 ? run_scan_step<T, LN, 4>(a, st)
                                               : run_scan_step<T, LN, 1>(a, st);
    });
  });
}

}  // namespace zo
