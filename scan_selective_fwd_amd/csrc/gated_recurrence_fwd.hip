// Gated linear recurrence, forward.  Per channel, with s the logistic function:
//   a_t = exp(A s(r_t)),  u_t = sqrt(1 - a_t^2) s(i_t) x_t,  h_t = a_t h_{t-1} + u_t
//   out_t = h_t  (h_t z_t s(z_t) with z)
// A step is an affine map of the state, h -> a h + u, and a run of steps is one too:
// (a1, u1) then (a2, u2) is (a2 a1, a2 u1 + u2).
//
// A lane takes two bfloat16 channels (one of float32, or where rows do not allow pairs),
// a wave 64 lanes and 16 steps, kept in registers: every tensor is read once and written
// once.  The waves of a block take one run after another of a strip of channels and join
// their maps in LDS.  Up to 256 steps are one block's; longer sequences take tiles of 128
// steps, whose blocks publish their maps and fetch those before them (rec_chain), so that
// all of a row's tiles are worked on at once.  Tickets, not block numbers, say which tile a
// block takes: a tile then waits only for tiles that run already.
//
// Bound by HBM and by what joins the tiles: 8 x 2048 x 1536 in bfloat16 with z take 59 us
// (252 MB, 4.3 TB/s; without the joining and the gates' arithmetic the same loads and
// stores take 55), 131072 x 1536 without z 360 (1.61 GB, 4.5 TB/s; 312), 2 x 2048 x 5120
// with z 49, 3 x 1000 x 1003 in float32 with z and flags 15 (384 tiles on 256 CUs).  A SIMD issues VALU for 28 us
// of the first (36 instructions and 8 transcendental ones an element).  Tried: tiles of 64
// steps (four blocks a CU, 509 us for the long one), of 256 (one block a CU, 436), groups
// of 8 and 32 tiles (380, 442), blocks that take tile after tile (88 us for 49: a loop's
// loads wait for the stores before them), loads begun before the ticket is known (443 for
// 377: at the start half of the guesses are wrong).
#include "recurrent_common.hpp"

namespace mscan {

namespace {

constexpr int S = (int)kRecRun;
constexpr int kMaxWaves = (int)(kRecOneTile / kRecRun);
constexpr int kTileWaves = (int)(kRecFwdTile / kRecRun);

template <typename T, int V, bool Z, bool RESET, bool CHAIN>
__global__ __launch_bounds__(CHAIN ? kTileWaves * 64 : kMaxWaves * 64, 4) void rec_fwd_kernel(
    const RecParams p) {
  constexpr int C = 64 * V;                       // channels of a strip
  constexpr int G = (int)kRecGroup;
  constexpr int W = CHAIN ? kTileWaves : kMaxWaves;
  __shared__ float sA[W][C], sH[W][C];
  __shared__ int sCut[W];
  __shared__ uint64_t sMap[CHAIN ? G : 1][CHAIN ? C : 1];
  __shared__ uint32_t sTicket;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = CHAIN ? kTileWaves : blockDim.x >> 6;
  const uint32_t strips = (uint32_t)((p.dim + C - 1) / C);
  const uint32_t across = strips * (uint32_t)p.batch;
  const int64_t marks = (p.L + kRecTile - 1) / kRecTile;

  const uint32_t at = rec_strip(across, p.by_die);
  if (at >= across) return;
  const uint32_t tiles = CHAIN ? (uint32_t)((p.L + kRecFwdTile - 1) / kRecFwdTile) : 1;
  const uint32_t tile = CHAIN ? rec_ticket(p.ticket, at, &sTicket) : 0;
  if (CHAIN && tile >= tiles) return;   // another call took tickets here: none of ours is left
  const int64_t b = uniform(at / strips);
  const uint32_t c0 = (at - (uint32_t)b * strips) * C, c = c0 + lane * V;
  const bool on = c < p.dim;
  // a lane past the last channel reads, and waits for, the first of its own strip
  const uint32_t cl = on ? c : c0, cb = cl * (uint32_t)sizeof(T);
  const int64_t t0 = ((int64_t)tile * waves + wave) * S;      // the wave's first step
  const int64_t left = p.L - t0;
  const int n = uniform(left >= S ? S : left > 0 ? (int)left : 0);   // its steps

  // every load of the run is in flight at once
  RecRaw<T, V> xr[S], rr[S], ir[S], zr[Z ? S : 1];
  const int64_t ts = n ? t0 : p.L - 1;
  RecWalk<T> x(p.x, b, ts), r(p.r, b, ts), i(p.i, b, ts), z(p.z, b, ts);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    rr[s].load(r.p, cb);
    ir[s].load(i.p, cb);
    xr[s].load(x.p, cb);
    if constexpr (Z) zr[s].load(z.p, cb);
    r.next(s, n);
    i.next(s, n);
    x.next(s, n);
    z.next(s, n);
  }
  if (n < S) {                                               // those leave the state
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s >= n) {
        rr[s].fill(-INFINITY);
        ir[s].fill(0.0f);
        xr[s].fill(0.0f);
      }
  }
  uint32_t flags = 0;                                        // of the wave's steps
  if constexpr (RESET) {
    const bool f = lane < n && p.reset[b * p.L + t0 + lane];
    flags = (uint32_t)__ballot(f);
  }
  float A2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A2[v] = rec_log2(p.A[cl + v]);

  // the run's own map.  Decay and input of each step stay for the second pass, which is
  // one multiply-add a step
  float a[S][V], u[S][V], A[V], H[V];
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
      u[s][v] = rec_sqrt(g.m2) * (g.si * xr[s].get(v));
      H[v] = rec_apply(a[s][v], u[s][v], cut, H[v]);
      A[v] *= a[s][v];
    }
  }
  // the first run starts from h0, and says so by a map that leaves out what is before
  // it: h0 is read here alone, before anything that last (h0's place, it may be) waits for
  const bool first = t0 == 0 && p.h0;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = first ? p.h0[b * p.dim + cl + v] : 0.0f;
    sA[wave][lane * V + v] = A[v];
    sH[wave][lane * V + v] = first ? rec_apply(A[v], H[v], flags != 0, h[v]) : H[v];
  }
  if (lane == 0) sCut[wave] = first || flags != 0;
  __syncthreads();

  // the map of the waves before this one, and the tile's
  float Ab[V], Hb[V], At[V], Ht[V];
  bool cutb = false, cutt = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    Ab[v] = At[v] = 1.0f;
    Hb[v] = Ht[v] = 0.0f;
  }
  for (int w = 0; w < waves; ++w) {
    if (w == wave) {
      cutb = cutt;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Ab[v] = At[v];
        Hb[v] = Ht[v];
      }
    }
    const bool cw = sCut[w] != 0;
    cutt = cutt || cw;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float Aw = sA[w][lane * V + v];
      Ht[v] = rec_apply(Aw, sH[w][lane * V + v], cw, Ht[v]);
      At[v] *= Aw;
    }
  }

  // the state that enters the tile
  if constexpr (CHAIN) {
    const uint32_t groups = (tiles + G - 1) / G;
    rec_chain<V, G, kTileWaves>(p.maps + ((uint64_t)b * tiles + tile) * p.dim + cl,
                    p.heads + ((uint64_t)b * groups + tile / G) * p.dim + cl, p.dim, tile, At, Ht,
                    cutt, on, wave, lane, sMap, h);
  }
  // and the wave's run
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = rec_apply(Ab[v], Hb[v], cutb, h[v]);
  if (p.ckpt && on && t0 % kRecTile == 0 && n)
#pragma unroll
    for (int v = 0; v < V; ++v) p.ckpt[(b * marks + t0 / kRecTile) * p.dim + c + v] = h[v];
  if (!on || !(p.out || p.last)) return;
  char* out = static_cast<char*>(p.out) + (b * p.L + t0) * p.dim * (int64_t)sizeof(T);
  auto outputs = [&](const int steps) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool cut = RESET && (flags >> s & 1);
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = rec_apply(a[s][v], u[s][v], cut, h[v]);
        y[v] = Z ? h[v] * silu(zr[Z ? s : 0].get(v)) : h[v];
      }
      if (s < steps) rec_store<T, V>(out, cb, y);
      out += p.dim * (int64_t)sizeof(T);
    }
  };
  if (n == S && p.out) outputs(S);
  else outputs(p.out ? n : 0);
  if (p.last && left > 0 && left <= S)
#pragma unroll
    for (int v = 0; v < V; ++v) p.last[b * p.dim + c + v] = h[v];
}

template <typename T, int V, bool Z, bool RESET>
hipError_t go(RecParams p, hipStream_t s) {
  const int64_t grid = rec_grid(&p, p.batch * rec_strips(p.dim, V == 2), rec_fwd_tiles(p.L), sizeof(T));
  if (!p.ticket) {
    hipLaunchKernelGGL((rec_fwd_kernel<T, V, Z, RESET, false>), dim3((unsigned)grid),
                       dim3((unsigned)((p.L + S - 1) / S * 64)), 0, s, p);
    return hipGetLastError();
  }
  const hipError_t e = rec_clear(p, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((rec_fwd_kernel<T, V, Z, RESET, true>), dim3((unsigned)grid),
                     dim3(kTileWaves * 64), 0, s, p);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t by_form(const RecParams& p, hipStream_t s) {
  if (p.reset) return p.z.p ? go<T, V, true, true>(p, s) : go<T, V, false, true>(p, s);
  return p.z.p ? go<T, V, true, false>(p, s) : go<T, V, false, false>(p, s);
}

__global__ __launch_bounds__(256) void rec_clear_kernel(uint64_t* p, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += step) p[k] = 0;
}

}  // namespace

// Clears what the tiles publish.  A kernel: it may be captured into a graph.
hipError_t rec_clear(const RecParams& p, hipStream_t s) {
  const int64_t n = (p.words + 255) / 256;
  hipLaunchKernelGGL(rec_clear_kernel, dim3((unsigned)(n < 4096 ? n : 4096)), dim3(256), 0, s,
                     reinterpret_cast<uint64_t*>(p.ticket), p.words);
  return hipGetLastError();
}

hipError_t dispatch_rec_fwd(const RecParams& p, int dtype, hipStream_t s) {
  if (dtype == 0) return by_form<float, 1>(p, s);
  return p.pairs ? by_form<bf16_t, 2>(p, s) : by_form<bf16_t, 1>(p, s);
}

}  // namespace mscan
