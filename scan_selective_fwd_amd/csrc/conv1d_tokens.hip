// Short causal depthwise convolution + SiLU over token-major rows:
//   pre_t = b + sum_k w[k] x_{t-k} over the lags k < W that stay in t's
//   sequence, out_t = pre_t sigmoid(pre_t)
// and its backward, dpre_t = dout_t silu'(pre_t):
//   dx_s = sum_k w[k] dpre_{s+k},  dw[k] = sum_t dpre_t x_{t-k},  db = sum_t dpre_t.
//
// Channels are contiguous, so a lane owns four of them and marches along a run
// of tokens with the last three inputs (and, backwards, the open sums of dx) in
// registers: every row is read once by its run and the three rows between runs
// twice.  Rows are loaded ahead in groups and kept packed until used.  In
// bfloat16 at width 4 the forward of 8 x 2048 x 1792 takes 24 us (118 MB at
// 4.9 TB/s: HBM), the backward of 2 x 2047 x 5376 with flags 52 us (132 MB at
// 2.6 TB/s; 45 with its inputs in the last-level cache, for 33 of which a SIMD issues
// VALU: per value the activation's derivative, the shares of dw and the flags'
// selects) and its sum 4 us.  With the width at run time they took 8 and 13 more.
#include "heads_common.hpp"

namespace mscan {

namespace {

constexpr int kAhead = 4;     // rows the backward loads ahead

// Weights by lag: w4[k] multiplies x_{t-k}.  The width W is a template argument:
// an input at a lag past it must not be multiplied, not even by zero.
template <int W, int V>
__device__ __forceinline__ void load_lags(const float* w, int64_t c, float (&w4)[W][V]) {
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < W; ++k) w4[k][v] = w[(c + v) * W + (W - 1 - k)];
}

// Input row s of batch row b, s in [-3, L): from x, the window before it, or zero.
template <typename T, int V>
__device__ __forceinline__ void input_row(const TokConvParams& p, int64_t b, int64_t s, int64_t c,
                                          float (&v)[V]) {
  if (s >= 0) {
    load_vec<T, V>(p.x.p, b * p.x.batch + s * p.x.token + c, v);
  } else if (p.window && s + p.W - 1 >= 0) {
    load_vec<T, V>(p.window, (b * (p.W - 1) + s + p.W - 1) * p.dim + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
  }
}

// The inputs at lags 1..3 of step t0: h[k] = x_{t0-1-k}, zero outside the
// sequence that reaches t0 - 1.
template <typename T, int V, bool RST>
__device__ __forceinline__ void history(const TokConvParams& p, const uint8_t* rst, int64_t b,
                                        int64_t t0, int64_t c, float (&h)[3][V]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) input_row<T, V>(p, b, t0 - 1 - k, c, h[k]);
  if constexpr (RST) {
    // a flag at t0 - 1 - k hides the inputs before that step
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (t0 - 1 - k >= 0 && rst[t0 - 1 - k] != 0)
#pragma unroll
        for (int j = k + 1; j < 3; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) h[j][v] = 0.0f;
  }
}

template <int V>
__device__ __forceinline__ void clear(float (&h)[3][V]) {
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) h[k][v] = 0.0f;
}

template <int V>
__device__ __forceinline__ void push(float (&h)[3][V], const float (&x)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[2][v] = h[1][v];
    h[1][v] = h[0][v];
    h[0][v] = x[v];
  }
}

template <int W, int V>
__device__ __forceinline__ void pre_act(const float (&w4)[W][V], const float (&cb)[V],
                                        const float (&x)[V], const float (&h)[3][V],
                                        float (&pre)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a = __builtin_fmaf(w4[0][v], x[v], cb[v]);
#pragma unroll
    for (int k = 1; k < W; ++k) a = __builtin_fmaf(w4[k][v], h[k - 1][v], a);
    pre[v] = a;
  }
}

template <typename T, int V, int W, bool RST>
__global__ __launch_bounds__(256) void tokconv_fwd_kernel(const TokConvParams p) {
  const int64_t nvec = p.dim / V;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t run = i / nvec;
  if (run >= p.batch * p.tiles) return;
  const int64_t c = (i - run * nvec) * V;
  const int64_t b = run / p.tiles;
  const int64_t t0 = (run - b * p.tiles) * kTokConvFwdRun;
  const uint8_t* rst = RST ? p.reset + b * p.L : nullptr;
  float w4[W][V], cb[V], h[3][V];
  load_lags<W, V>(p.w, c, w4);
#pragma unroll
  for (int v = 0; v < V; ++v) cb[v] = p.b ? p.b[c + v] : 0.0f;
  history<T, V, RST>(p, rst, b, t0, c, h);
  const int64_t n = p.L - t0 < kTokConvFwdRun ? p.L - t0 : kTokConvFwdRun;
  const int64_t x0 = b * p.x.batch + t0 * p.x.token + c;
  const int64_t o0 = (b * p.L + t0) * p.dim + c;
  auto step = [&](int64_t j, const Raw<T, V>& r) {
    if constexpr (RST)
      if (rst[t0 + j] != 0) clear<V>(h);
    float x[V], pre[V];
    r.get(x);
    pre_act<W, V>(w4, cb, x, h, pre);
    push<V>(h, x);
#pragma unroll
    for (int v = 0; v < V; ++v) pre[v] = silu(pre[v]);
    store_vec<T, V>(p.out, o0 + j * p.dim, pre);
  };
  if (n == kTokConvFwdRun) {
    Raw<T, V> x[kTokConvFwdRun];
#pragma unroll
    for (int j = 0; j < kTokConvFwdRun; ++j) x[j].load(p.x.p, x0 + j * p.x.token);
#pragma unroll
    for (int j = 0; j < kTokConvFwdRun; ++j) step(j, x[j]);
  } else {
    for (int64_t j = 0; j < n; ++j) {
      Raw<T, V> x;
      x.load(p.x.p, x0 + j * p.x.token);
      step(j, x);
    }
  }
  if (p.window_out && t0 + n == p.L) {
    // h holds the last three inputs of the sequence that goes on
    for (int k = 0; k < W - 1; ++k)
      store_vec<T, V>(p.window_out, (b * (W - 1) + (W - 2 - k)) * p.dim + c,
                      k == 0 ? h[0] : k == 1 ? h[1] : h[2]);
  }
}

// d silu(a) / da.
__device__ __forceinline__ float dsilu(float a) {
  const float sg = sigmoid(a);
  return sg * __builtin_fmaf(a, 1.0f - sg, 1.0f);
}

// A block: 64 lanes of channels by 4 waves, each a run of kTokConvRun tokens.
template <typename T, int V, int W, bool RST>
__global__ __launch_bounds__(256) void tokconv_bwd_kernel(const TokConvParams p) {
  __shared__ float red[4][W + 1][64 * V];
  const int64_t ctiles = (p.dim + 64 * V - 1) / (64 * V);
  const int64_t tile = blockIdx.x / ctiles;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (blockIdx.x - tile * ctiles) * (64 * V) + lane * V;
  const int64_t b = tile / p.tiles;
  const int64_t t0 = (tile - b * p.tiles) * kTokConvTile + wave * kTokConvRun;
  float dw[W][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][v] = 0.0f;
  }
  if (c < p.dim && t0 < p.L) {
    const uint8_t* rst = RST ? p.reset + b * p.L : nullptr;
    float w4[W][V], cb[V], h[3][V], acc[3][V];   // acc[k]: dx_{t-1-k} so far
    load_lags<W, V>(p.w, c, w4);
#pragma unroll
    for (int v = 0; v < V; ++v) cb[v] = p.b ? p.b[c + v] : 0.0f;
    history<T, V, RST>(p, rst, b, t0, c, h);
    clear<V>(acc);
    // lags of step t that stay in its sequence: up to `age`
    int age = 3;
    if constexpr (RST)
      for (int k = 3; k >= 1; --k)
        if (t0 - k >= 0) age = rst[t0 - k] != 0 ? 0 : (age < 3 ? age + 1 : 3);
    const int64_t x0 = b * p.x.batch + c, o0 = b * p.L * p.dim + c;
    // one step: t = t0 + j, own ones below kTokConvRun
    auto step = [&](int j, const Raw<T, V>& xr, const Raw<T, V>& gr) {
      const int64_t t = t0 + j;
      float x[V], g[V], pre[V];
      xr.get(x);
      gr.get(g);
      if (t < p.L) {
        if constexpr (RST) {
          if (rst[t] != 0) {
            clear<V>(h);
            age = 0;
          } else {
            age = age < 3 ? age + 1 : 3;
          }
        }
        pre_act<W, V>(w4, cb, x, h, pre);
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] *= dsilu(pre[v]);
        if (j < kTokConvRun) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            db[v] += g[v];
            dw[0][v] = __builtin_fmaf(g[v], x[v], dw[0][v]);
#pragma unroll
            for (int k = 1; k < W; ++k) dw[k][v] = __builtin_fmaf(g[v], h[k - 1][v], dw[k][v]);
          }
        }
      }
      // dx_{t-3} is complete with this step's share
      float done[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        done[v] = acc[2][v];
        if constexpr (W > 3) done[v] = (!RST || age >= 3) ? __builtin_fmaf(w4[3][v], g[v], done[v]) : done[v];
        acc[2][v] = acc[1][v];
        if constexpr (W > 2) acc[2][v] = (!RST || age >= 2) ? __builtin_fmaf(w4[2][v], g[v], acc[2][v]) : acc[2][v];
        acc[1][v] = (!RST || age >= 1) ? __builtin_fmaf(w4[1][v], g[v], acc[0][v]) : acc[0][v];
        acc[0][v] = w4[0][v] * g[v];
      }
      push<V>(h, x);
      const int64_t s = t - 3;
      if (j >= 3) {
        if (s < p.L) store_vec<T, V>(p.dx, o0 + s * p.dim, done);
      } else if (t0 == 0 && p.dwindow && s + W - 1 >= 0) {
        store_vec<T, V>(p.dwindow, (b * (W - 1) + s + W - 1) * p.dim + c, done);
      }
    };
    auto load = [&](int j, Raw<T, V>& x, Raw<T, V>& g) {
      const int64_t t = t0 + j;
      x.zero();
      g.zero();
      if (t < p.L) {
        x.load(p.x.p, x0 + t * p.x.token);
        g.load(p.dout, o0 + t * p.dim);
      }
    };
    static_assert(kTokConvRun % kAhead == 0, "whole groups");
    Raw<T, V> xr[2][kAhead], gr[2][kAhead], xe[3], ge[3];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, xr[0][i], gr[0][i]);
#pragma unroll
    for (int j = 0; j < kTokConvRun; j += kAhead) {
      const int k = (j / kAhead) & 1;
      if (j + kAhead < kTokConvRun) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(j + kAhead + i, xr[k ^ 1][i], gr[k ^ 1][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) load(kTokConvRun + i, xe[i], ge[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) step(j + i, xr[k][i], gr[k][i]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) step(kTokConvRun + i, xe[i], ge[i]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W; ++k) red[wave][k][v * 64 + lane] = dw[k][v];
    red[wave][W][v * 64 + lane] = db[v];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 256) {
    const int k = i / (64 * V), r = i - k * (64 * V);
    const int64_t ch = (blockIdx.x - tile * ctiles) * (64 * V) + (r & 63) * V + (r >> 6);
    const float sum = (red[0][k][r] + red[1][k][r]) + (red[2][k][r] + red[3][k][r]);
    // rows 0..W-1: dw by position (lag W-1-row), row W: db
    if (ch < p.dim) p.part[(tile * (W + 1) + (k == W ? W : W - 1 - k)) * p.dim + ch] = sum;
  }
}

// dw, db: the tiles' shares summed in order, 8 slices of them by 32 channels.
__global__ __launch_bounds__(256) void tokconv_sum_kernel(const TokConvParams p) {
  __shared__ float red[8][32];
  const int64_t ctiles = (p.dim + 31) / 32;
  const int k = (int)(blockIdx.x / ctiles);
  const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t c = (blockIdx.x - (int64_t)k * ctiles) * 32 + cl;
  const int64_t n = p.batch * p.tiles;
  float sum = 0.0f;
  if (c < p.dim)
    for (int64_t i = sl; i < n; i += 8) sum += p.part[(i * (p.W + 1) + k) * p.dim + c];
  red[sl][cl] = sum;
  __syncthreads();
  if (sl == 0 && c < p.dim) {
    for (int j = 1; j < 8; ++j) sum += red[j][cl];
    if (k < p.W) p.dw[c * p.W + k] = sum;
    else if (p.db) p.db[c] = sum;
  }
}

// One token of every sequence (256 x 5376 channels: 11 us).  What it costs is its
// latency, so it rounds each product and sum by itself, the oldest input first,
// and takes the library's exp and a true division: the bits that a chain of
// elementwise float operations gives.  The result is rounded to the stored type
// and enters a state, where one unit of bfloat16 would show.  The forward over many
// tokens is bound by HBM only with fused operations and the fast sigmoid, so 4 of
// 100 thousand results differ between the two by that unit; both are as near to 64
// bits (1.67e-3 in bfloat16, 7e-8 in float32).
template <int W, int V>
__device__ __forceinline__ void step_act(const float (&w4)[W][V], const float (&cb)[V],
                                         const float (&x)[V], const float (&h)[3][V],
                                         float (&out)[V]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a = w4[W - 1][v] * h[W - 2][v];
#pragma unroll
    for (int k = W - 2; k >= 1; --k) a = a + w4[k][v] * h[k - 1][v];
    a = a + w4[0][v] * x[v];
    a = a + cb[v];
    out[v] = a * (1.0f / (1.0f + expf(-a)));
  }
}

template <typename T, int V, int W>
__global__ __launch_bounds__(256) void tokconv_step_kernel(const TokConvStepParams p) {
  const int64_t nvec = p.dim / V;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t b = i / nvec;
  if (b >= p.batch) return;
  const int64_t c = (i - b * nvec) * V;
  const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
  float out[V];
  if (slot < 0 || slot >= p.pool) {
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.0f;
    store_vec<T, V>(p.out, b * p.dim + c, out);
    return;
  }
  const int64_t w0 = slot * (W - 1) * p.dim + c;
  float w4[W][V], cb[V], x[V], h[3][V];
  load_vec<T, V>(p.x, b * p.x_batch + c, x);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) load_vec<T, V>(p.window, w0 + (W - 2 - k) * p.dim, h[k]);
  load_lags<W, V>(p.w, c, w4);
#pragma unroll
  for (int v = 0; v < V; ++v) cb[v] = p.b ? p.b[c + v] : 0.0f;
  step_act<W, V>(w4, cb, x, h, out);
  store_vec<T, V>(p.out, b * p.dim + c, out);
  // the window moves on by one token
#pragma unroll
  for (int k = W - 2; k >= 1; --k) store_vec<T, V>(p.window, w0 + (W - 2 - k) * p.dim, h[k - 1]);
  store_vec<T, V>(p.window, w0 + (W - 2) * p.dim, x);
}

unsigned blocks_of(int64_t threads) { return (unsigned)((threads + 255) / 256); }

template <typename T, int V, int W>
hipError_t fwd_go(TokConvParams p, hipStream_t s) {
  p.tiles = (p.L + kTokConvFwdRun - 1) / kTokConvFwdRun;
  const dim3 grid(blocks_of(p.batch * p.tiles * (p.dim / V)));
  if (p.reset) hipLaunchKernelGGL((tokconv_fwd_kernel<T, V, W, true>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((tokconv_fwd_kernel<T, V, W, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, int V, int W>
hipError_t bwd_go(const TokConvParams& p, hipStream_t s) {
  const int64_t ctiles = (p.dim + 64 * V - 1) / (64 * V);
  const dim3 grid((unsigned)(p.batch * p.tiles * ctiles));
  if (p.reset) hipLaunchKernelGGL((tokconv_bwd_kernel<T, V, W, true>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((tokconv_bwd_kernel<T, V, W, false>), grid, dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned sums = (unsigned)((W + 1) * ((p.dim + 31) / 32));
  hipLaunchKernelGGL(tokconv_sum_kernel, dim3(sums), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, int V, int W>
hipError_t step_go(const TokConvStepParams& p, hipStream_t s) {
  hipLaunchKernelGGL((tokconv_step_kernel<T, V, W>), dim3(blocks_of(p.batch * (p.dim / V))),
                     dim3(256), 0, s, p);
  return hipGetLastError();
}

// f.go<T, V, W>() for the call's type, vector length and width (2 to 4).
template <typename T, int V, typename F>
hipError_t by_width(int64_t W, const F& f) {
  switch (W) {
    case 2: return f.template go<T, V, 2>();
    case 3: return f.template go<T, V, 3>();
    case 4: return f.template go<T, V, 4>();
  }
  return hipErrorInvalidValue;
}
template <typename F>
hipError_t by_type(int dtype, bool vec, int64_t W, const F& f) {
  if (dtype == 0) return vec ? by_width<float, 4>(W, f) : by_width<float, 1>(W, f);
  return vec ? by_width<bf16_t, 4>(W, f) : by_width<bf16_t, 1>(W, f);
}

struct Fwd {
  const TokConvParams& p;
  hipStream_t s;
  template <typename T, int V, int W>
  hipError_t go() const { return fwd_go<T, V, W>(p, s); }
};
struct Bwd {
  const TokConvParams& p;
  hipStream_t s;
  template <typename T, int V, int W>
  hipError_t go() const { return bwd_go<T, V, W>(p, s); }
};
struct Token {
  const TokConvStepParams& p;
  hipStream_t s;
  template <typename T, int V, int W>
  hipError_t go() const { return step_go<T, V, W>(p, s); }
};

}  // namespace

hipError_t dispatch_tokconv_fwd(const TokConvParams& p, int dtype, hipStream_t s) {
  return by_type(dtype, p.vec, p.W, Fwd{p, s});
}

hipError_t dispatch_tokconv_bwd(const TokConvParams& p, int dtype, hipStream_t s) {
  return by_type(dtype, p.vec, p.W, Bwd{p, s});
}

hipError_t dispatch_tokconv_step(const TokConvStepParams& p, int dtype, hipStream_t s) {
  return by_type(dtype, p.vec, p.W, Token{p, s});
}

}  // namespace mscan
