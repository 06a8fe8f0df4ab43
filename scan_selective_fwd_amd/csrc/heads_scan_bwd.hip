// The backward of the multi-head scan, one token after the other: per (batch row, head)
//   h_t = a_t h_{t-1} + w_t u_t B_t^T,   out_t = h_t C_t + D u_t,   h (P, N)
// with the adjoint g_t = dout_t C_t^T + a_{t+1} g_{t+1},
//   du = w g B + D dout,  dB = w g^T u,  dC = h^T dout,  dw = u . (g B),
//   dlog_t = <a_t g_t, h_{t-1}>, the gradient of the log decay.
// The backward keeps every state of its forward sweep in the workspace.
//
// A block of 256 threads holds one head's state in registers: thread (row
// pi, quarter nq) holds rows pi and pi + 64, states nq, nq + 4, ...
#include "heads_common.hpp"

namespace mscan {

namespace {

template <typename T>
__device__ __forceinline__ float elem(const Rows& r, int64_t b, int64_t t, int64_t i) {
  return Elem<T>::load1(static_cast<const T*>(r.p) + b * r.batch + t * r.token + i);
}

// Sums over the block's 64 rows of v[j] (state n = nq + 4 j): result in sh[n].
template <int J>
__device__ __forceinline__ void sum_rows(float (&v)[J], float (*sh)[4 * J]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int off = 4; off < 64; off <<= 1) v[j] += __shfl_xor(v[j], off);
    if (lane < 4) sh[wave][lane + 4 * j] = v[j];
  }
  __syncthreads();
  for (int n = threadIdx.x; n < 4 * J; n += 256)
    sh[0][n] = (sh[0][n] + sh[1][n]) + (sh[2][n] + sh[3][n]);
  __syncthreads();
}

__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

template <typename T, int J>
__global__ __launch_bounds__(256) void heads_bwd_kernel(const HeadsBwdParams p) {
  __shared__ float shn[4][4 * J];
  __shared__ float sh4[4];
  const int64_t b = blockIdx.x / p.H;
  const int hd = (int)(blockIdx.x - b * p.H), g = hd / (p.H / p.G);
  const int pi = threadIdx.x >> 2, nq = threadIdx.x & 3;
  const uint8_t* rst = reset_row(p.reset, b, p.L);
  const float A = p.A[hd], bias = p.bias ? p.bias[hd] : 0.0f, D = p.D ? p.D[hd] : 0.0f;
  const int64_t s0 = (b * p.H + hd) * (int64_t)p.P * p.N;
  // this thread's share of the state after each step, 2 J floats at a stride of 256
  float* keep = p.states + (b * p.H + hd) * p.L * (512 * J) + threadIdx.x;
  float h[2][J], v[J];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int pp = pi + 64 * i, n = nq + 4 * j;
      h[i][j] = p.h0 && pp < p.P && n < p.N ? p.h0[s0 + (int64_t)pp * p.N + n] : 0.0f;
    }
  auto dyv = [&](int64_t t, int i) {
    return pi + 64 * i < p.P
               ? Elem<T>::load1(static_cast<const T*>(p.dout) +
                                ((b * p.L + t) * p.H + hd) * p.P + pi + 64 * i)
               : 0.0f;
  };
  auto uv = [&](int64_t t, int i) {
    return pi + 64 * i < p.P ? elem<T>(p.u, b, t, (int64_t)hd * p.P + pi + 64 * i) : 0.0f;
  };
  // forward in time: the states, dC and z
  for (int64_t t = 0; t < p.L; ++t) {
    const Step q = make_step(elem<T>(p.delta, b, t, hd) + bias, A, p.softplus, p.zoh);
    const float a = exp2f(q.lg);
    const bool cut = rst && rst[t] != 0;
    const float u[2] = {uv(t, 0), uv(t, 1)}, dy[2] = {dyv(t, 0), dyv(t, 1)};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = nq + 4 * j;
      const float Bn = n < p.N ? elem<T>(p.B, b, t, (int64_t)g * p.N + n) : 0.0f;
      v[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[i][j] = __builtin_fmaf(u[i] * q.w, Bn, cut ? 0.0f : a * h[i][j]);
        v[j] = __builtin_fmaf(h[i][j], dy[i], v[j]);
        keep[t * (512 * J) + (i * J + j) * 256] = h[i][j];
      }
    }
    sum_rows<J>(v, shn);
    for (int n = threadIdx.x; n < p.N; n += 256)
      p.dC_part[((b * p.L + t) * p.H + hd) * p.N + n] = shn[0][n];
  }
  // backward in time: the adjoint
  float gr[2][J];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int pp = pi + 64 * i, n = nq + 4 * j;
      gr[i][j] = p.dlast && pp < p.P && n < p.N ? p.dlast[s0 + (int64_t)pp * p.N + n] : 0.0f;
    }
  float dA = 0.0f, dD = 0.0f, dbias = 0.0f;
  for (int64_t t = p.L - 1; t >= 0; --t) {
    const float raw = elem<T>(p.delta, b, t, hd) + bias;
    const Step q = make_step(raw, A, p.softplus, p.zoh);
    const float a = exp2f(q.lg);
    const bool cut = rst && rst[t] != 0;
    const float u[2] = {uv(t, 0), uv(t, 1)}, dy[2] = {dyv(t, 0), dyv(t, 1)};
    float gB[2] = {0.0f, 0.0f}, F = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = nq + 4 * j;
      const float Bn = n < p.N ? elem<T>(p.B, b, t, (int64_t)g * p.N + n) : 0.0f;
      const float Cn = n < p.N ? elem<T>(p.C, b, t, (int64_t)g * p.N + n) : 0.0f;
      v[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        gr[i][j] = __builtin_fmaf(dy[i], Cn, gr[i][j]);
        gB[i] = __builtin_fmaf(gr[i][j], Bn, gB[i]);
        v[j] = __builtin_fmaf(gr[i][j], u[i] * q.w, v[j]);
        gr[i][j] = cut ? 0.0f : a * gr[i][j];
        const int pp = pi + 64 * i;
        const float before =
            t > 0 ? keep[(t - 1) * (512 * J) + (i * J + j) * 256]
                  : (p.h0 && pp < p.P && n < p.N ? p.h0[s0 + (int64_t)pp * p.N + n] : 0.0f);
        F = __builtin_fmaf(gr[i][j], before, F);
      }
    }
    F = block_sum(F, sh4);
    float W = 0.0f, ud = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      gB[i] += __shfl_xor(gB[i], 1);
      gB[i] += __shfl_xor(gB[i], 2);
      const int pp = pi + 64 * i;
      if (nq == 0) {
        W = __builtin_fmaf(gB[i], u[i], W);
        ud = __builtin_fmaf(u[i], dy[i], ud);
        if (pp < p.P)
          Elem<T>::store1(static_cast<T*>(p.du) + ((b * p.L + t) * p.H + hd) * p.P + pp,
                          __builtin_fmaf(D, dy[i], gB[i] * q.w));
      }
    }
    W = block_sum(W, sh4);
    ud = block_sum(ud, sh4);
    sum_rows<J>(v, shn);
    for (int n = threadIdx.x; n < p.N; n += 256)
      p.dB_part[((b * p.L + t) * p.H + hd) * p.N + n] = shn[0][n];
    float by_dt, by_A;
    step_weight_grad(q.dt, A, p.zoh, by_dt, by_A);
    const float ddt = (A * F + W * by_dt) * q.draw;
    dA += q.dt * F + W * by_A;
    dD += ud;
    dbias += ddt;
    if (threadIdx.x == 0)
      Elem<T>::store1(static_cast<T*>(p.ddelta) + (b * p.L + t) * p.H + hd, ddt);
  }
  if (p.dh0)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int pp = pi + 64 * i, n = nq + 4 * j;
        if (pp < p.P && n < p.N) p.dh0[s0 + (int64_t)pp * p.N + n] = gr[i][j];
      }
  if (threadIdx.x == 0) {
    float* hp = p.head_part + (b * p.H + hd) * 3;
    hp[0] = dA;
    hp[1] = dD;
    hp[2] = dbias;
  }
}

// dB, dC: the heads of a group summed in order.
template <typename T>
__global__ __launch_bounds__(256) void heads_bwd_sum_kernel(const HeadsBwdParams p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / (p.G * p.N);
  if (row >= p.batch * p.L) return;
  const int gn = (int)(i - row * (p.G * p.N)), g = gn / p.N, n = gn - g * p.N;
  const int per = p.H / p.G;
  float sB = 0.0f, sC = 0.0f;
  for (int k = 0; k < per; ++k) {
    const int64_t at = (row * p.H + g * per + k) * p.N + n;
    sB += p.dB_part[at];
    sC += p.dC_part[at];
  }
  Elem<T>::store1(static_cast<T*>(p.dB) + i, sB);
  Elem<T>::store1(static_cast<T*>(p.dC) + i, sC);
}

__global__ __launch_bounds__(256) void heads_bwd_head_kernel(const HeadsBwdParams p) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h >= p.H) return;
  float s[3] = {0.0f, 0.0f, 0.0f};
  for (int64_t b = 0; b < p.batch; ++b)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += p.head_part[(b * p.H + h) * 3 + k];
  p.dA[h] = s[0];
  if (p.dD) p.dD[h] = s[1];
  if (p.dbias) p.dbias[h] = s[2];
}

template <typename T, int J>
hipError_t bwd_go(const HeadsBwdParams& p, hipStream_t s) {
  hipLaunchKernelGGL((heads_bwd_kernel<T, J>), dim3((unsigned)(p.batch * p.H)), dim3(256), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t n = p.batch * p.L * p.G * p.N;
  hipLaunchKernelGGL((heads_bwd_sum_kernel<T>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(heads_bwd_head_kernel, dim3((unsigned)((p.H + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_t(const HeadsBwdParams& p, hipStream_t s) {
  if (p.N <= 16) return bwd_go<T, 4>(p, s);
  if (p.N <= 64) return bwd_go<T, 16>(p, s);
  if (p.N <= 128) return bwd_go<T, 32>(p, s);
  return bwd_go<T, 64>(p, s);
}

}  // namespace

hipError_t dispatch_heads_bwd(const HeadsBwdParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? bwd_t<float>(p, s) : bwd_t<bf16_t>(p, s);
}

}  // namespace mscan
