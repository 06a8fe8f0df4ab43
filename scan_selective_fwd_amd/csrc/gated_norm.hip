// Group norm under a SiLU gate, rows of token-major activations.  With
// g = silu(z), per row and group:
//   gate first: v = x g, out = v r w;  else: v = x, out = v r w g
//   r = 1 / sqrt(mean(v^2) + eps)
// Backward, with dhat = dout w (times g when the gate comes last):
//   dv = r (dhat - v r^2 mean(dhat v));
//   gate first: dx = dv g, dg = dv x;  else: dx = dv, dg = dout w v r
//   dz = dg silu'(z);  dw = sum over rows of dout v r (times g)
//
// A team of 64 or 256 threads takes one group of one row and keeps it in
// registers: every tensor is read once and written once, and the two sums of
// the backward come from the same pass.  Groups too long for the registers,
// or rows not on 16 bytes, are walked twice (the second time from the cache).
// The forward is bound by HBM: 16384 rows of 1536 in bfloat16 take 28 us (151 MB,
// 5.3 TB/s).  The backward of 4096 rows of 5120 in 8 groups takes 50 us (210 MB at
// 4.2 TB/s), for about 36 of which a SIMD issues VALU (gate, its derivative and the
// two passes over a value), and 42 with its inputs in the last-level cache; the sum
// of dw takes 6.
#include "heads_common.hpp"

namespace mscan {

namespace {

constexpr int kNormBlocks = 1024;   // blocks of the backward: four a CU

// Sums of a and b over a team of TEAM threads (64: the wave; 256: the block).
template <int TEAM>
__device__ __forceinline__ void team_sum(float& a, float& b, float (*sh)[2]) {
  a = row_sum_to_last(a);
  b = row_sum_to_last(b);
  a = rs_pair32(rs_pair16(a, a), rs_pair16(a, a));   // over the rows, in their last lanes
  b = rs_pair32(rs_pair16(b, b), rs_pair16(b, b));
  a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, a), 63));
  b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, b), 63));
  if constexpr (TEAM == 256) {
    __syncthreads();   // the previous row's sums have been read
    if ((threadIdx.x & 63) == 0) {
      sh[threadIdx.x >> 6][0] = a;
      sh[threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    a = (sh[0][0] + sh[1][0]) + (sh[2][0] + sh[3][0]);
    b = (sh[0][1] + sh[1][1]) + (sh[2][1] + sh[3][1]);
  }
}

struct Gate {
  float g, dg;   // silu(z) and its derivative
};

__device__ __forceinline__ Gate gate_of(float z) {
  const float sg = sigmoid(z);
  return {z * sg, sg * __builtin_fmaf(z, 1.0f - sg, 1.0f)};
}

template <typename T, int V, int TEAM, int NV>
__global__ __launch_bounds__(256) void norm_fwd_kernel(const NormParams p) {
  __shared__ float sh[4][2];
  constexpr int TEAMS = 256 / TEAM;
  const int tid = threadIdx.x & (TEAM - 1);
  const int64_t i = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM;
  const bool on = i < p.rows * p.groups;       // whole teams
  const int64_t row = on ? i / p.groups : 0;
  const int64_t c0 = on ? (i - row * p.groups) * p.gs : 0;
  float x[NV][V], g[NV][V];
  float s2 = 0.0f, unused = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t k = (int64_t)(j * TEAM + tid) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[j][v] = 0.0f;
      g[j][v] = 1.0f;
    }
    if (on && k < p.gs) {
      load_vec<T, V>(p.x, row * p.x_row + c0 + k, x[j]);
      if (p.z) load_vec<T, V>(p.z, row * p.z_row + c0 + k, g[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (p.z) g[j][v] = silu(g[j][v]);
      const float t = p.gate_first ? x[j][v] * g[j][v] : x[j][v];
      s2 = __builtin_fmaf(t, t, s2);
    }
  team_sum<TEAM>(s2, unused, sh);
  const float r = 1.0f / __builtin_sqrtf(s2 / (float)p.gs + p.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t k = (int64_t)(j * TEAM + tid) * V;
    if (on && k < p.gs) {
      float w[V], o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = 1.0f;
      if (p.w) load_f32<V>(p.w, c0 + k, w);
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = x[j][v] * g[j][v] * r * w[v];
      store_vec<T, V>(p.out, row * p.dim + c0 + k, o);
    }
  }
}

// Any length and alignment: the group is walked twice.
template <typename T, int V, int TEAM>
__global__ __launch_bounds__(256) void norm_fwd_walk_kernel(const NormParams p) {
  __shared__ float sh[4][2];
  constexpr int TEAMS = 256 / TEAM;
  const int tid = threadIdx.x & (TEAM - 1);
  const int64_t i = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM;
  const bool on = i < p.rows * p.groups;
  const int64_t row = on ? i / p.groups : 0;
  const int64_t c0 = on ? (i - row * p.groups) * p.gs : 0;
  const int64_t n = on ? p.gs : 0;
  float s2 = 0.0f, unused = 0.0f;
  for (int64_t k = (int64_t)tid * V; k < n; k += TEAM * V) {
    float x[V], z[V];
    load_vec<T, V>(p.x, row * p.x_row + c0 + k, x);
    if (p.z && p.gate_first) load_vec<T, V>(p.z, row * p.z_row + c0 + k, z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float t = p.z && p.gate_first ? x[v] * silu(z[v]) : x[v];
      s2 = __builtin_fmaf(t, t, s2);
    }
  }
  team_sum<TEAM>(s2, unused, sh);
  const float r = 1.0f / __builtin_sqrtf(s2 / (float)p.gs + p.eps);
  for (int64_t k = (int64_t)tid * V; k < n; k += TEAM * V) {
    float x[V], z[V], w[V], o[V];
    load_vec<T, V>(p.x, row * p.x_row + c0 + k, x);
    if (p.z) load_vec<T, V>(p.z, row * p.z_row + c0 + k, z);
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = 1.0f;
    if (p.w) load_f32<V>(p.w, c0 + k, w);
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = (p.z ? x[v] * silu(z[v]) : x[v]) * r * w[v];
    store_vec<T, V>(p.out, row * p.dim + c0 + k, o);
  }
}

// What an element gives to the two sums of its row.
__device__ __forceinline__ void bwd_sums(const NormParams& p, float x, float g, float dy, float w,
                                         float& s2, float& sv) {
  const float t = p.gate_first ? x * g : x;
  const float dhat = p.gate_first ? dy * w : dy * w * g;
  s2 = __builtin_fmaf(t, t, s2);
  sv = __builtin_fmaf(dhat, t, sv);
}

// The element's gradients; k = r^2 mean(dhat v).  Adds its share of dw.
__device__ __forceinline__ void bwd_elem(const NormParams& p, float x, Gate q, float dy, float w,
                                         float r, float k, float& dx, float& dz, float& dw) {
  const float t = p.gate_first ? x * q.g : x;
  const float dhat = p.gate_first ? dy * w : dy * w * q.g;
  const float dv = r * __builtin_fmaf(-t, k, dhat);
  const float hat = t * r;
  dx = p.gate_first ? dv * q.g : dv;
  dz = (p.gate_first ? dv * x : dy * w * hat) * q.dg;
  dw = __builtin_fmaf(p.gate_first ? dy : dy * q.g, hat, dw);
}

// Block (part, group): its teams take every (parts * TEAMS)-th row, and leave
// the block's share of dw in part.
template <typename T, int V, int TEAM, int NV>
__global__ __launch_bounds__(256) void norm_bwd_kernel(const NormParams p) {
  constexpr int TEAMS = 256 / TEAM;
  __shared__ float sh[4][2];
  __shared__ float red[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? TEAM * NV * V : 1];
  const int tid = threadIdx.x & (TEAM - 1), team = threadIdx.x / TEAM;
  const int64_t part = blockIdx.x / p.groups;
  const int64_t c0 = (blockIdx.x - part * p.groups) * p.gs;
  float w[NV][V], dw[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t k = (int64_t)(j * TEAM + tid) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[j][v] = 1.0f;
      dw[j][v] = 0.0f;
    }
    if (p.w && k < p.gs) load_f32<V>(p.w, c0 + k, w[j]);
  }
  // the next row's loads are in flight while this one is worked on
  Raw<T, V> xr[NV], zr[NV], yr[NV];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t k = (int64_t)(j * TEAM + tid) * V;
      xr[j].zero();
      zr[j].zero();
      yr[j].zero();
      if (k < p.gs && row < p.rows) {
        xr[j].load(p.x, row * p.x_row + c0 + k);
        if (p.z) zr[j].load(p.z, row * p.z_row + c0 + k);
        yr[j].load(p.dout, row * p.dim + c0 + k);
      }
    }
  };
  const int64_t step = p.parts * TEAMS;
  load(part * TEAMS + team);
  for (int64_t row = part * TEAMS + team; row < p.rows; row += step) {
    float x[NV][V], dy[NV][V];
    Gate q[NV][V];
    float s2 = 0.0f, sv = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float z[V];
      xr[j].get(x[j]);
      zr[j].get(z);
      yr[j].get(dy[j]);
#pragma unroll
      for (int v = 0; v < V; ++v) q[j][v] = p.z ? gate_of(z[v]) : Gate{1.0f, 0.0f};
    }
    load(row + step);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) bwd_sums(p, x[j][v], q[j][v].g, dy[j][v], w[j][v], s2, sv);
    team_sum<TEAM>(s2, sv, sh);
    const float r = 1.0f / __builtin_sqrtf(s2 / (float)p.gs + p.eps);
    const float kk = r * r * (sv / (float)p.gs);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t k = (int64_t)(j * TEAM + tid) * V;
      float dx[V], dz[V];
#pragma unroll
      for (int v = 0; v < V; ++v)
        bwd_elem(p, x[j][v], q[j][v], dy[j][v], w[j][v], r, kk, dx[v], dz[v], dw[j][v]);
      if (k < p.gs) {
        store_vec<T, V>(p.dx, row * p.dim + c0 + k, dx);
        if (p.z) store_vec<T, V>(p.dz, row * p.dim + c0 + k, dz);
      }
    }
  }
  if (!p.dw) return;
  if constexpr (TEAMS > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) red[team][(j * V + v) * TEAM + tid] = dw[j][v];
    __syncthreads();
    for (int i = threadIdx.x; i < TEAM * NV * V; i += 256) {
      const int jv = i / TEAM, lane = i - jv * TEAM;
      const int64_t k = (int64_t)((jv / V) * TEAM + lane) * V + jv % V;
      float sum = 0.0f;
#pragma unroll
      for (int m = 0; m < TEAMS; ++m) sum += red[m][i];
      if (k < p.gs) p.part[part * p.dim + c0 + k] = sum;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t k = (int64_t)(j * TEAM + tid) * V + v;
        if (k < p.gs) p.part[part * p.dim + c0 + k] = dw[j][v];
      }
  }
}

// Any length and alignment: rows are walked twice by the block, dw is added
// up in the block's own row of part.
template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_walk_kernel(const NormParams p) {
  __shared__ float sh[4][2];
  const int64_t part = blockIdx.x / p.groups;
  const int64_t c0 = (blockIdx.x - part * p.groups) * p.gs;
  float* mine = p.dw ? p.part + part * p.dim + c0 : nullptr;
  if (mine)
    for (int64_t k = threadIdx.x; k < p.gs; k += 256) mine[k] = 0.0f;
  for (int64_t row = part; row < p.rows; row += p.parts) {
    float s2 = 0.0f, sv = 0.0f;
    float x[1], z[1] = {0.0f}, dy[1];
    for (int64_t k = threadIdx.x; k < p.gs; k += 256) {
      load_vec<T, 1>(p.x, row * p.x_row + c0 + k, x);
      if (p.z) load_vec<T, 1>(p.z, row * p.z_row + c0 + k, z);
      load_vec<T, 1>(p.dout, row * p.dim + c0 + k, dy);
      bwd_sums(p, x[0], p.z ? silu(z[0]) : 1.0f, dy[0], p.w ? p.w[c0 + k] : 1.0f, s2, sv);
    }
    team_sum<256>(s2, sv, sh);
    const float r = 1.0f / __builtin_sqrtf(s2 / (float)p.gs + p.eps);
    const float kk = r * r * (sv / (float)p.gs);
    for (int64_t k = threadIdx.x; k < p.gs; k += 256) {
      load_vec<T, 1>(p.x, row * p.x_row + c0 + k, x);
      if (p.z) load_vec<T, 1>(p.z, row * p.z_row + c0 + k, z);
      load_vec<T, 1>(p.dout, row * p.dim + c0 + k, dy);
      const Gate q = p.z ? gate_of(z[0]) : Gate{1.0f, 0.0f};
      float dx[1], dz[1], dw = mine ? mine[k] : 0.0f;
      bwd_elem(p, x[0], q, dy[0], p.w ? p.w[c0 + k] : 1.0f, r, kk, dx[0], dz[0], dw);
      store_vec<T, 1>(p.dx, row * p.dim + c0 + k, dx);
      if (p.z) store_vec<T, 1>(p.dz, row * p.dim + c0 + k, dz);
      if (mine) mine[k] = dw;
    }
  }
}

// dw: the parts summed in order, 8 slices of them by 32 channels.
__global__ __launch_bounds__(256) void norm_sum_kernel(const NormParams p) {
  __shared__ float red[8][32];
  const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float sum = 0.0f;
  if (c < p.dim)
    for (int64_t i = sl; i < p.parts; i += 8) sum += p.part[i * p.dim + c];
  red[sl][cl] = sum;
  __syncthreads();
  if (sl == 0 && c < p.dim) {
    for (int j = 1; j < 8; ++j) sum += red[j][cl];
    p.dw[c] = sum;
  }
}

// The rows in as few launches as hold them.
template <typename T>
hipError_t by_rows(void (*kernel)(const NormParams), NormParams p, int64_t per, hipStream_t s) {
  const int64_t most = norm_launch_rows(p.groups, per);
  for (int64_t left = p.rows; left > 0; left -= p.rows) {
    p.rows = left < most ? left : most;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((p.rows * p.groups + per - 1) / per)), dim3(256), 0,
                       s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.x = static_cast<const T*>(p.x) + p.rows * p.x_row;
    if (p.z) p.z = static_cast<const T*>(p.z) + p.rows * p.z_row;
    p.out = static_cast<T*>(p.out) + p.rows * p.dim;
  }
  return hipSuccess;
}

template <typename T, int V, int TEAM, int NV>
hipError_t fwd_go(const NormParams& p, hipStream_t s) {
  return by_rows<T>(norm_fwd_kernel<T, V, TEAM, NV>, p, 256 / TEAM, s);
}

template <typename T, int V, int TEAM>
hipError_t fwd_walk(const NormParams& p, hipStream_t s) {
  return by_rows<T>(norm_fwd_walk_kernel<T, V, TEAM>, p, 256 / TEAM, s);
}

template <typename T, int V>
hipError_t fwd_t(const NormParams& p, hipStream_t s) {
  const int64_t nv = p.vec ? (p.gs + V - 1) / V : 0;
  if (!p.vec) return p.gs <= 512 ? fwd_walk<T, 1, 64>(p, s) : fwd_walk<T, 1, 256>(p, s);
  if (nv <= 64) return fwd_go<T, V, 64, 1>(p, s);
  if (nv <= 128) return fwd_go<T, V, 64, 2>(p, s);
  if (nv <= 192) return fwd_go<T, V, 64, 3>(p, s);
  if (nv <= 256) return fwd_go<T, V, 64, 4>(p, s);
  if (nv <= 512) return fwd_go<T, V, 256, 2>(p, s);
  if (nv <= 1024) return fwd_go<T, V, 256, 4>(p, s);
  return fwd_walk<T, V, 256>(p, s);
}

template <typename T, int V, int TEAM, int NV>
hipError_t bwd_go(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_bwd_kernel<T, V, TEAM, NV>), dim3((unsigned)(p.parts * p.groups)),
                     dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_t(const NormParams& p, hipStream_t s) {
  constexpr int V = 4;
  const int64_t nv = (p.gs + V - 1) / V;
  hipError_t e;
  if (!p.vec || nv > 2048) {
    hipLaunchKernelGGL((norm_bwd_walk_kernel<T>), dim3((unsigned)(p.parts * p.groups)), dim3(256),
                       0, s, p);
    e = hipGetLastError();
  } else if (nv <= 64) {
    e = bwd_go<T, V, 64, 1>(p, s);
  } else if (nv <= 128) {
    e = bwd_go<T, V, 64, 2>(p, s);
  } else if (nv <= 192) {
    e = bwd_go<T, V, 64, 3>(p, s);
  } else if (nv <= 256) {
    e = bwd_go<T, V, 256, 1>(p, s);
  } else if (nv <= 512) {
    e = bwd_go<T, V, 256, 2>(p, s);
  } else if (nv <= 1024) {
    e = bwd_go<T, V, 256, 4>(p, s);
  } else {
    e = bwd_go<T, V, 256, 8>(p, s);
  }
  if (e != hipSuccess || !p.dw) return e;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((p.dim + 31) / 32)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t groups) {
  int64_t n = kNormBlocks / groups;
  if (n < 1) n = 1;
  return n < rows ? n : rows;
}

hipError_t dispatch_norm_fwd(const NormParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? fwd_t<float, 4>(p, s) : fwd_t<bf16_t, 8>(p, s);
}

hipError_t dispatch_norm_bwd(const NormParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? bwd_t<float>(p, s) : bwd_t<bf16_t>(p, s);
}

}  // namespace mscan
