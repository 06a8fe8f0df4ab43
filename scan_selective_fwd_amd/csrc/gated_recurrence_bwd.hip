// Gated linear recurrence, backward.  With g_t the gradient at the state h_t:
//   g_t = dh_t + a_{t+1} g_{t+1}      (dh_t = dout_t, times z_t s(z_t) with z)
//   dx = g m s(i),  di = g u (1 - s(i)),  with m = sqrt(1 - a^2), u = m s(i) x
//   d(log a) = g (a h_{t-1} - s(i) x a^2 / m),  dr = d(log a) A s(r) (1 - s(r))
//   dA = sum of d(log a) s(r),  dz = dout h (silu)'(z),  dh0 = a_0 g_0
// The recurrence of g runs from the last step to the first; it is joined over waves and
// tiles as the forward's is (rec_chain, tiles taken from the last on).  The states are
// formed again from the forward's checkpoints, 64 steps apart, which is a tile: no tile
// waits for the states of another.  (A call without them runs the forward first, without
// its outputs.)
//
// A lane takes one channel, a wave 8 steps, a block 8 waves: what a step's gradients take
// of its gates (seven values) then fits 128 registers beside the loads, and two blocks
// share a CU.  Every tensor is read once and written once.  2 x 2048 x 5120 in bfloat16
// with z take 95 to 97 us (378 MB, 4.0 TB/s; without the joining and the gates' arithmetic the
// same loads and stores take 94), 4 x 777 x 1025 in float32 with flags 24 (884 tiles, 1.7
// times those that fit at once); a SIMD issues VALU for 57 us of the first.  A block lives 9 us: 0.6 for its ticket, 2.6 until its gates
// are formed, 2.6 for the states and both sums of maps, 1.9 for the tiles behind it, 1.3
// for the gradients.  Tried: two channels a lane (243 us, spills), the gates formed a
// second time instead of kept (132), tiles of 128 steps and one block a CU (158), three
// blocks a CU by spilling (199).
#include "recurrent_common.hpp"

namespace mscan {

namespace {

constexpr int S = (int)kRecBwdRun;
constexpr int kMaxWaves = (int)(kRecBwdOneTile / kRecBwdRun);
constexpr int kTileWaves = (int)(kRecBwdTile / kRecBwdRun);
constexpr int kMarkWaves = (int)kRecTile / S;   // waves between checkpoints

template <typename T, int V, bool Z, bool RESET, bool CHAIN>
__global__ __launch_bounds__(CHAIN ? kTileWaves * 64 : kMaxWaves * 64, 4) void rec_bwd_kernel(const RecParams p) {
  constexpr int C = 64 * V;                       // channels of a strip
  constexpr int G = (int)kRecGroup;
  constexpr int W = CHAIN ? kTileWaves : kMaxWaves;
  __shared__ float sA[W][C], sH[W][C], sB[W][C];
  __shared__ int sCut[W];
  __shared__ uint64_t sMap[CHAIN ? G : 1][CHAIN ? C : 1];
  __shared__ uint32_t sTicket;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = CHAIN ? kTileWaves : blockDim.x >> 6;
  const uint32_t strips = (uint32_t)((p.dim + C - 1) / C);
  const uint32_t across = strips * (uint32_t)p.batch;
  const uint32_t tiles = CHAIN ? (uint32_t)((p.L + kRecBwdTile - 1) / kRecBwdTile) : 1;
  const int64_t marks = (p.L + kRecTile - 1) / kRecTile;
  const uint32_t at = rec_strip(across, p.by_die);
  if (at >= across) return;
  const uint32_t q = CHAIN ? rec_ticket(p.ticket, at, &sTicket) : 0;
  if (CHAIN && q >= tiles) return;      // another call took tickets here: none of ours is left
  const uint32_t tile = tiles - 1 - q;                        // the last tile first
  const int64_t b = uniform(at / strips);
  const uint32_t c0 = (at - (uint32_t)b * strips) * C, c = c0 + lane * V;
  const bool on = c < p.dim;
  // a lane past the last channel reads, and waits for, the first of its own strip
  const uint32_t cl = on ? c : c0, cb = cl * (uint32_t)sizeof(T);
  const int64_t t0 = ((int64_t)tile * waves + wave) * S;      // the wave's first step
  const int64_t left = p.L - t0;
  const int n = uniform(left >= S ? S : left > 0 ? (int)left : 0);   // its steps

  // every load of the run is in flight at once
  RecRaw<T, V> xr[S], rr[S], ir[S], yr[S], zr[Z ? S : 1];
  const int64_t ts = n ? t0 : p.L - 1;
  RecWalk<T> x(p.x, b, ts), r(p.r, b, ts), i(p.i, b, ts), z(p.z, b, ts),
      dy({p.dout, p.L * p.dim, p.dim}, b, ts);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    rr[s].load(r.p, cb);
    ir[s].load(i.p, cb);
    xr[s].load(x.p, cb);
    yr[s].load(dy.p, cb);
    if constexpr (Z) zr[s].load(z.p, cb);
    r.next(s, n);
    i.next(s, n);
    x.next(s, n);
    dy.next(s, n);
    z.next(s, n);
  }
  // the state at the checkpoint before the run (a run past the end has none)
  float h[V];
  const int64_t mark = t0 / kRecTile < marks ? t0 / kRecTile : marks - 1;
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = p.kept[(b * marks + mark) * p.dim + cl + v];
  if (n < S) {                                               // steps past the end
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s >= n) {
        rr[s].fill(-INFINITY);
        ir[s].fill(0.0f);
        xr[s].fill(0.0f);
        yr[s].fill(0.0f);
        if constexpr (Z) zr[s].fill(0.0f);
      }
  }
  uint32_t flags = 0;
  if constexpr (RESET) {
    const bool f = lane < n && p.reset[b * p.L + t0 + lane];
    flags = (uint32_t)__ballot(f);
  }
  float A2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A2[v] = rec_log2(p.A[cl + v]);

  // the run's map of the states, and what the gradients take of the gates: with g the
  // gradient at a state and y the log of its decay
  //   dx = g m s(i),  di = g u (1 - s(i)),  u = m s(i) x
  //   d(log a) y = g a (y before - u a y / m^2),  dr of it times 1 - s(r)
  // y / m^2 is -1/2 where the decay is 1, and u vanishes there; m^2 is held at float32's
  // smallest normal value, below which y loses its digits
  float a[S][V], u[S][V], A[V], H[V];
  float by_x[S][V], by_i[S][V], y[S][V], own[S][V], by_r[S][V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    H[v] = 0.0f;
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const bool cut = RESET && (flags >> s & 1);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const RecGate g = rec_gate(rr[s].get(v), ir[s].get(v), A2[v]);
      a[s][v] = g.a;
      by_x[s][v] = rec_sqrt(g.m2) * g.si;
      u[s][v] = by_x[s][v] * xr[s].get(v);
      by_i[s][v] = u[s][v] * g.i.complement();
      y[s][v] = g.lg * kLn2;
      const float ym = y[s][v] * fast_rcp(__builtin_fmaxf(g.m2, 0x1p-126f));
      own[s][v] = u[s][v] * g.a * ym;
      by_r[s][v] = g.r.complement();
      H[v] = rec_apply(g.a, u[s][v], cut, H[v]);
      A[v] *= g.a;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sA[wave][lane * V + v] = A[v];
    sH[wave][lane * V + v] = H[v];
  }
  if (lane == 0) sCut[wave] = flags != 0;
  __syncthreads();
  for (int w = wave / kMarkWaves * kMarkWaves; w < wave; ++w) {
    const bool cw = sCut[w] != 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = rec_apply(sA[w][lane * V + v], sH[w][lane * V + v], cw, h[v]);
  }

  // the states before each step (in the inputs' place), the gate on the output, and
  // the run's map of the gradient that comes to the state from later steps
  float dh[S][V], B[V];
  const int64_t row = p.dim * (int64_t)sizeof(T), row0 = (b * p.L + t0) * row;
  auto states = [&](const int steps) {
    char* to = static_cast<char*>(p.dz) + row0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool cut = RESET && (flags >> s & 1);
      float dz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float before = h[v];
        h[v] = rec_apply(a[s][v], u[s][v], cut, before);
        u[s][v] = before;
        dh[s][v] = yr[s].get(v);
        if constexpr (Z) {
          const float z = zr[s].get(v), sz = sigmoid(z);
          dz[v] = dh[s][v] * h[v] * (sz * __builtin_fmaf(z, 1.0f - sz, 1.0f));
          dh[s][v] *= z * sz;
        }
      }
      if constexpr (Z) {
        if (on && s < steps) rec_store<T, V>(to, cb, dz);
        to += row;
      }
    }
  };
  if (n == S) states(S);
  else states(n);
#pragma unroll
  for (int v = 0; v < V; ++v) B[v] = 0.0f;
#pragma unroll
  for (int s = S - 1; s >= 0; --s) {
    const bool cut = RESET && (flags >> s & 1);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float y = a[s][v] * (dh[s][v] + B[v]);
      B[v] = cut ? 0.0f : y;
    }
  }
  // the first run of the walk starts from dlast
  const bool first = q == 0 && wave == waves - 1 && p.dlast;
  float after[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    after[v] = first ? p.dlast[b * p.dim + cl + v] : 0.0f;
    sB[wave][lane * V + v] = first ? rec_apply(A[v], B[v], flags != 0, after[v]) : B[v];
  }
  __syncthreads();
  float Ab[V], Bb[V], At[V], Bt[V];
  bool cutb = false, cutt = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    Ab[v] = At[v] = 1.0f;
    Bb[v] = Bt[v] = 0.0f;
  }
  for (int w = waves - 1; w >= 0; --w) {
    if (w == wave) {
      cutb = cutt;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Ab[v] = At[v];
        Bb[v] = Bt[v];
      }
    }
    const bool cw = sCut[w] != 0 || (q == 0 && w == waves - 1 && p.dlast);
    cutt = cutt || cw;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float Aw = sA[w][lane * V + v];
      Bt[v] = rec_apply(Aw, sB[w][lane * V + v], cw, Bt[v]);
      At[v] *= Aw;
    }
  }
  if constexpr (CHAIN) {
    const uint32_t groups = (tiles + G - 1) / G;
    rec_chain<V, G, kTileWaves>(p.maps + ((uint64_t)b * tiles + q) * p.dim + cl,
                    p.heads + ((uint64_t)b * groups + q / G) * p.dim + cl, p.dim, q, At, Bt, cutt,
                    on, wave, lane, sMap, after);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) after[v] = rec_apply(Ab[v], Bb[v], cutb, after[v]);

  float sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = 0.0f;
  auto grads = [&](const int steps) {
    char* dx_to = static_cast<char*>(p.dx) + row0 + (S - 1) * row;
    char* dr_to = static_cast<char*>(p.dr) + row0 + (S - 1) * row;
    char* di_to = static_cast<char*>(p.di) + row0 + (S - 1) * row;
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
      const bool cut = RESET && (flags >> s & 1);
      float dx[V], dr[V], di[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float g = dh[s][v] + after[v], ag = a[s][v] * g;
        const float kept = __builtin_fmaf(y[s][v], u[s][v], -own[s][v]);
        const float e = ag * (cut ? -own[s][v] : kept);
        after[v] = cut ? 0.0f : ag;
        dx[v] = g * by_x[s][v];
        di[v] = g * by_i[s][v];
        dr[v] = e * by_r[s][v];
        sum[v] += e;
      }
      if (s < steps) {
        rec_store<T, V>(dx_to, cb, dx);
        rec_store<T, V>(dr_to, cb, dr);
        rec_store<T, V>(di_to, cb, di);
      }
      dx_to -= row;
      dr_to -= row;
      di_to -= row;
    }
  };
  if (on) {
    if (n == S) grads(S);
    else grads(n);
  }
  // the lane's channel again, from the lane's number: kept over the gates, it would be spilled
  const uint32_t zero = opaque_int(0);
  const uint32_t end = c0 + __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero)) * V;
  if (t0 == 0 && p.dh0 && on)
#pragma unroll
    for (int v = 0; v < V; ++v) p.dh0[b * p.dim + end + v] = after[v];
  // the tile's share of dA, its runs added in order
#pragma unroll
  for (int v = 0; v < V; ++v) sH[wave][lane * V + v] = sum[v];
  __syncthreads();
  if (wave == 0 && on)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float s = sum[v];
      for (int w = 1; w < waves; ++w) s += sH[w][lane * V + v];
      p.part[((int64_t)b * tiles + tile) * p.dim + end + v] = s;
    }
}

// dA: the tiles' shares added in a fixed order, in 64 bits; 32 slices of them by 32
// channels, from channel c0 on.
constexpr int kSumChannels = 32, kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void rec_sum_kernel(const RecParams p, const int64_t parts,
                                                              const int64_t c0) {
  __shared__ double red[32][33];
  const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t c = c0 + (int64_t)blockIdx.x * kSumChannels + cl;
  double sum = 0.0;
  if (c < p.dim) {
#pragma unroll 4
    for (int64_t k = sl; k < parts; k += 32) sum += p.part[k * p.dim + c];
  }
  red[cl][sl] = sum;
  __syncthreads();
  // a wave takes two channels' slices
  const int ch = threadIdx.x >> 5, at = threadIdx.x & 31;
  sum = red[ch][at];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  const int64_t to = c0 + (int64_t)blockIdx.x * kSumChannels + ch;
  if (at == 0 && to < p.dim) p.dA[to] = (float)sum / p.A[to];   // the shares are A times too large
}

template <typename T, int V, bool Z, bool RESET>
hipError_t go(RecParams p, hipStream_t s) {
  const int64_t tiles = rec_bwd_tiles(p.L);
  const int64_t grid = rec_grid(&p, p.batch * rec_strips(p.dim, V == 2), tiles, sizeof(T));
  hipError_t e;
  if (!p.ticket) {
    hipLaunchKernelGGL((rec_bwd_kernel<T, V, Z, RESET, false>), dim3((unsigned)grid),
                       dim3((unsigned)((p.L + S - 1) / S * 64)), 0, s, p);
  } else {
    e = rec_clear(p, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((rec_bwd_kernel<T, V, Z, RESET, true>), dim3((unsigned)grid),
                       dim3(kTileWaves * 64), 0, s, p);
  }
  e = hipGetLastError();
  // as many launches as hold the channels: one, up to 2^27 - 32 of them
  constexpr int64_t most = kSumChannels * max_blocks(kSumThreads);
  for (int64_t c0 = 0; c0 < p.dim && e == hipSuccess; c0 += most) {
    const int64_t n = p.dim - c0 < most ? p.dim - c0 : most;
    hipLaunchKernelGGL(rec_sum_kernel, dim3((unsigned)((n + kSumChannels - 1) / kSumChannels)),
                       dim3(kSumThreads), 0, s, p, p.batch * tiles, c0);
    e = hipGetLastError();
  }
  return e;
}

// Single elements: pairs would take more registers than let two blocks share a CU.
template <typename T>
hipError_t by_form(const RecParams& p, hipStream_t s) {
  if (p.reset) return p.z.p ? go<T, 1, true, true>(p, s) : go<T, 1, false, true>(p, s);
  return p.z.p ? go<T, 1, true, false>(p, s) : go<T, 1, false, false>(p, s);
}

}  // namespace

hipError_t dispatch_rec_bwd(const RecParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? by_form<float>(p, s) : by_form<bf16_t>(p, s);
}

}  // namespace mscan
