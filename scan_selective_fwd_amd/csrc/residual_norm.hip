// Root-mean-square norm with the residual's addition, rows of token-major activations:
//   res = x + residual (as it is stored),  out = res r w,  r = 1 / sqrt(mean(res^2) + eps)
// in the activations' type, or in 8 bits under the row's scale max|out| / 448.
// Backward, with dhat = dout w:
//   d = dres + r (dhat - res r^2 mean(dhat res)),  dw = sum over rows of dout res r
//
// A team of 64 to 512 threads takes a row and keeps it in registers: every tensor is
// read once and written once, and the largest value of 8 bits is found on the way.  Rows
// too long for that are walked again from the cache.  Bound by HBM: the forward of 16384
// rows of 1536 in bfloat16 takes 38 us (201 MB, 5.3 TB/s), of 4096 of 5120 on a float32
// stream into 8 bits 47 (231 MB, 4.9 TB/s); the backward of 4096 of 5120 in bfloat16 29 to
// 34 (168 MB, 5.0 TB/s or more), and 4 for the sum of dw.  Rows that do not start on 16
// bytes are read element by element (4096 of 6001 take 118 us for 39).
#include "recurrent_common.hpp"

namespace mscan {

namespace {

constexpr int kParts = 512;        // blocks of the backward: two a CU
constexpr int kFwdBlocks = (1 << 22) - 1;   // of up to 1024 threads in one launch
constexpr int kWalk = 1024;

// Where row `row` of a view starts.
__device__ __forceinline__ int64_t row_at(const ResNormParams& p, int64_t row, int64_t batch,
                                          int64_t step) {
  if (!p.inner) return row * step;
  const int64_t b = row / p.inner;
  return b * batch + (row - b * p.inner) * step;
}

// Element k of the row that starts `row` elements behind p.  The row is the block's, the
// place in it 32 bits: the access forms the sum.
template <typename E>
__device__ __forceinline__ const void* place(const void* p, int64_t row, uint32_t k) {
  return static_cast<const char*>(p) + row * (int64_t)sizeof(E) + (uint32_t)(k * sizeof(E));
}
template <typename E>
__device__ __forceinline__ void* place(void* p, int64_t row, uint32_t k) {
  return static_cast<char*>(p) + row * (int64_t)sizeof(E) + (uint32_t)(k * sizeof(E));
}

template <bool MAX>
__device__ __forceinline__ float join(float a, float b) {
  return MAX ? __builtin_fmaxf(a, b) : a + b;
}

// Sum (or largest value) over a team of TEAM threads of a block, in every thread.  `sh`
// holds a float for each wave of the block.
template <int TEAM, bool MAX>
__device__ __forceinline__ float team_join(float a, float* sh) {
  a = join<MAX>(a, dpp_mov<0xB1>(a, a));     // quad_perm 1,0,3,2
  a = join<MAX>(a, dpp_mov<0x4E>(a, a));     // quad_perm 2,3,0,1
  a = join<MAX>(a, dpp_mov<0x141>(a, a));    // row_half_mirror
  a = join<MAX>(a, dpp_mov<0x140>(a, a));    // row_mirror
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(a), false, false);
  a = join<MAX>(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(a), false, false);
  a = join<MAX>(__uint_as_float(r[0]), __uint_as_float(r[1]));
  if constexpr (TEAM > 64) {
    constexpr int W = TEAM / 64;
    __syncthreads();   // what was joined before has been read
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = a;
    __syncthreads();
    const int w0 = threadIdx.x / TEAM * W;
    a = sh[w0];
#pragma unroll
    for (int w = 1; w < W; ++w) a = join<MAX>(a, sh[w0 + w]);
  }
  return a;
}

// 1 / sqrt(mean of squares + eps) from their sum.  Where that passes float32's range (or
// vanishes beside an eps that does), `again` forms it from values times a scale.
template <typename F>
__device__ __forceinline__ float root_of(float s2, const ResNormParams& p, F again) {
  const float n = (float)p.dim;
  if (__builtin_expect(s2 < 3e38f && (s2 > 0x1p-80f || p.eps > 0x1p-90f), 1))
    return 1.0f / __builtin_sqrtf(s2 / n + p.eps);
  const float sc = s2 < 1.0f ? 0x1p70f : 0x1p-70f;
  return sc / __builtin_sqrtf(again(sc) / n + p.eps * sc * sc);
}

// V values of x + residual as they are stored: the norm is of what the stream keeps, so
// that the backward, which has only that, forms the same statistics.
template <typename R, int V>
__device__ __forceinline__ void add_stored(float (&x)[V], const float (&r)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] += r[v];
  if constexpr (sizeof(R) == 2) {
    if constexpr (V == 1) {
      x[0] = bf16_lo(pack_bf16(x[0], x[0]));
    } else {
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const uint32_t w = pack_bf16(x[v], x[v + 1]);
        x[v] = bf16_lo(w);
        x[v + 1] = bf16_hi(w);
      }
    }
  }
}

// To the nearest of e4m3, ties to even (v_cvt_pk_fp8_f32): |y| is at most 448 and one
// unit of float32 in its last place, which rounds to 448; a NaN stays one.
template <int V>
__device__ __forceinline__ void store_e4m3(void* out, int64_t at, const float (&y)[V]) {
  uint8_t* q = static_cast<uint8_t*>(out) + at;
  if constexpr (V == 1) {
    *q = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[0], 0, false);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
      int t = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k], y[4 * k + 1], 0, false);
      w[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k + 2], y[4 * k + 3], t, true);
    }
    if constexpr (V == 4) *reinterpret_cast<uint32_t*>(q) = w[0];
    else *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  }
}

template <int V>
__device__ __forceinline__ void load_weight(const float* w, int64_t at, float (&v)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = 1.0f;
  if (w) load_f32<V>(w, at, v);
}

template <typename T, typename R, bool FP8, int V, int TEAM, int NV>
__global__ __launch_bounds__(256) void res_norm_fwd_kernel(const ResNormParams p) {
  __shared__ float sh[4];
  constexpr int TEAMS = 256 / TEAM;
  const int tid = threadIdx.x & (TEAM - 1);
  const int64_t n = p.dim;
  for (int64_t row0 = (int64_t)blockIdx.x * TEAMS; row0 < p.rows; row0 += (int64_t)gridDim.x * TEAMS) {
    const int64_t row = row0 + threadIdx.x / TEAM;
    const bool on = row < p.rows;                 // whole teams
    const int64_t x0 = row_at(p, row, p.x_batch, p.x_row);
    const int64_t r0 = row_at(p, row, p.res_batch, p.res_row);
    float x[NV][V], r[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t k = (int64_t)(j * TEAM + tid) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) x[j][v] = r[j][v] = 0.0f;
      if (on && k < n) {
        load_vec<T, V>(p.x, x0 + k, x[j]);
        if (p.res) load_vec<R, V>(p.res, r0 + k, r[j]);
      }
    }
    float s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (p.res) add_stored<R, V>(x[j], r[j]);
#pragma unroll
      for (int v = 0; v < V; ++v) s2 = __builtin_fmaf(x[j][v], x[j][v], s2);
    }
    s2 = team_join<TEAM, false>(s2, sh);
    const float root = root_of(s2, p, [&](float sc) {
      float t2 = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float t = x[j][v] * sc;
          t2 = __builtin_fmaf(t, t, t2);
        }
      return team_join<TEAM, false>(t2, sh);
    });
    float y[NV][V], most = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t k = (int64_t)(j * TEAM + tid) * V;
      if (on && k < n) {
        if (p.res) store_vec<R, V>(p.res_out, row * n + k, x[j]);
        float w[V];
        load_weight<V>(p.w, k, w);
#pragma unroll
        for (int v = 0; v < V; ++v) y[j][v] = x[j][v] * root * w[v];
        if constexpr (!FP8) store_vec<T, V>(p.out, row * n + k, y[j]);
        else
#pragma unroll
          for (int v = 0; v < V; ++v) most = __builtin_fmaxf(most, __builtin_fabsf(y[j][v]));
      }
    }
    if constexpr (FP8) {
      most = __builtin_fmaxf(team_join<TEAM, true>(most, sh), 0x1p-100f);
      const float inv = 448.0f / most;
      if (on && tid == 0) p.scale[row] = most / 448.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int64_t k = (int64_t)(j * TEAM + tid) * V;
        if (on && k < n) {
#pragma unroll
          for (int v = 0; v < V; ++v) y[j][v] *= inv;
          store_e4m3<V>(p.out, row * n + k, y[j]);
        }
      }
    }
  }
}

// Rows too long for the registers: walked two or three times by a block.
template <typename T, typename R, bool FP8, int V>
__global__ __launch_bounds__(kWalk) void res_norm_fwd_walk_kernel(const ResNormParams p) {
  __shared__ float sh[kWalk / 64];
  const int64_t n = p.dim;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t x0 = row_at(p, row, p.x_batch, p.x_row);
    const int64_t r0 = row_at(p, row, p.res_batch, p.res_row);
    auto sum = [&](int64_t k, float (&x)[V]) {
      float r[V];
      load_vec<T, V>(p.x, x0 + k, x);
      if (p.res) {
        load_vec<R, V>(p.res, r0 + k, r);
        add_stored<R, V>(x, r);
      }
    };
    auto squares = [&](float sc) {
      float s2 = 0.0f;
      for (int64_t k = (int64_t)threadIdx.x * V; k < n; k += kWalk * V) {
        float x[V];
        sum(k, x);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float t = x[v] * sc;
          s2 = __builtin_fmaf(t, t, s2);
        }
      }
      return team_join<kWalk, false>(s2, sh);
    };
    const float root = root_of(squares(1.0f), p, squares);
    auto normed = [&](int64_t k, float (&x)[V], float (&y)[V]) {
      float w[V];
      sum(k, x);
      load_weight<V>(p.w, k, w);
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = x[v] * root * w[v];
    };
    float inv = 1.0f;
    if constexpr (FP8) {
      float most = 0.0f;
      for (int64_t k = (int64_t)threadIdx.x * V; k < n; k += kWalk * V) {
        float x[V], y[V];
        normed(k, x, y);
#pragma unroll
        for (int v = 0; v < V; ++v) most = __builtin_fmaxf(most, __builtin_fabsf(y[v]));
      }
      most = __builtin_fmaxf(team_join<kWalk, true>(most, sh), 0x1p-100f);
      inv = 448.0f / most;
      if (threadIdx.x == 0) p.scale[row] = most / 448.0f;
    }
    for (int64_t k = (int64_t)threadIdx.x * V; k < n; k += kWalk * V) {
      float x[V], y[V];
      normed(k, x, y);
      if (p.res) store_vec<R, V>(p.res_out, row * n + k, x);
      if constexpr (FP8) {
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] *= inv;
        store_e4m3<V>(p.out, row * n + k, y);
      } else {
        store_vec<T, V>(p.out, row * n + k, y);
      }
    }
  }
}

// Block `part`: its teams take every (parts * TEAMS)-th row, the next row's loads in
// flight while one is worked on (where the registers hold both), and leave the block's
// share of dw in part.
template <typename T, typename R, int V, int TEAM, int NV>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void res_norm_bwd_kernel(
    const ResNormParams p) {
  constexpr bool AHEAD = NV * V <= (V == 1 ? 8 : 24);
  constexpr int THREADS = TEAM > 256 ? TEAM : 256, TEAMS = THREADS / TEAM;
  __shared__ float sh[THREADS / 64];
  __shared__ float red[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? TEAM * NV * V : 1];
  const int tid = threadIdx.x & (TEAM - 1), team = threadIdx.x / TEAM;
  const int64_t n = p.dim;         // at most 16384 here
  float w[NV][V], dw[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t k = (uint32_t)(j * TEAM + tid) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[j][v] = 1.0f;
      dw[j][v] = 0.0f;
    }
    if (AHEAD && p.w && k < n) load_f32<V>(static_cast<const float*>(place<float>(p.w, 0, k)), 0, w[j]);
  }
  Raw<R, V> xr[NV], gr[NV];
  Raw<T, V> yr[NV];
  auto load = [&](int64_t row) {
    const int64_t r0 = row_at(p, row, p.res_batch, p.res_row);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t k = (uint32_t)(j * TEAM + tid) * V;
      xr[j].zero();
      yr[j].zero();
      if (k < n && row < p.rows) {
        xr[j].load(place<R>(p.res, r0, k), 0);
        yr[j].load(place<T>(p.dout, row * n, k), 0);
      }
    }
  };
  auto load_dres = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t k = (uint32_t)(j * TEAM + tid) * V;
      gr[j].zero();
      if (p.dres && k < n && row < p.rows) gr[j].load(place<R>(p.dres, row * n, k), 0);
    }
  };
  const int64_t step = p.parts * TEAMS;
  if (AHEAD) {
    load(blockIdx.x * (int64_t)TEAMS + team);
    load_dres(blockIdx.x * (int64_t)TEAMS + team);
  }
  // every team walks as long as the first: the joins wait for whole blocks
  for (int64_t row0 = blockIdx.x * (int64_t)TEAMS; row0 < p.rows; row0 += step) {
    const int64_t row = row0 + team;
    float x[NV][V], dy[NV][V], g[NV][V];
    float s2 = 0.0f, sv = 0.0f;
    if (!AHEAD) load(row);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xr[j].get(x[j]);
      yr[j].get(dy[j]);
      if (AHEAD) gr[j].get(g[j]);
    }
    if (AHEAD) {
      load(row + step);
      load_dres(row + step);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {       // from the cache, row by row
        const uint32_t k = (uint32_t)(j * TEAM + tid) * V;
        if (p.w && k < n) load_f32<V>(static_cast<const float*>(place<float>(p.w, 0, k)), 0, w[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s2 = __builtin_fmaf(x[j][v], x[j][v], s2);
        sv = __builtin_fmaf(dy[j][v] * w[j][v], x[j][v], sv);
      }
    s2 = team_join<TEAM, false>(s2, sh);
    sv = team_join<TEAM, false>(sv, sh);
    const float r = root_of(s2, p, [&](float sc) {
      float t2 = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float t = x[j][v] * sc;
          t2 = __builtin_fmaf(t, t, t2);
        }
      return team_join<TEAM, false>(t2, sh);
    });
    const float kk = r * (sv / (float)p.dim);
    if (!AHEAD) {
      mem_fence_compiler();                // not before the sums, which need registers
      load_dres(row);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t k = (uint32_t)(j * TEAM + tid) * V;
      float d[V];
      if (!AHEAD) gr[j].get(g[j]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float hat = x[j][v] * r;
        d[v] = __builtin_fmaf(r, __builtin_fmaf(-hat, kk, dy[j][v] * w[j][v]), g[j][v]);
        dw[j][v] = __builtin_fmaf(dy[j][v], hat, dw[j][v]);
      }
      if (k < n && row < p.rows) {
        store_vec<T, V>(place<T>(p.dx, row * n, k), 0, d);
        if (sizeof(T) != sizeof(R) && p.dresidual) store_vec<R, V>(place<R>(p.dresidual, row * n, k), 0, d);
      }
    }
  }
  if (!p.dw) return;
  float* mine = p.part + blockIdx.x * n;
  if constexpr (TEAMS > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) red[team][(j * V + v) * TEAM + tid] = dw[j][v];
    __syncthreads();
    for (int i = threadIdx.x; i < TEAM * NV * V; i += THREADS) {
      const int jv = i / TEAM, lane = i - jv * TEAM;
      const int64_t k = (int64_t)((jv / V) * TEAM + lane) * V + jv % V;
      float sum = red[0][i];
#pragma unroll
      for (int m = 1; m < TEAMS; ++m) sum += red[m][i];
      if (k < n) mine[k] = sum;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t k = (uint32_t)(j * TEAM + tid) * V;
      if (k < n) store_vec<float, V>(mine, k, dw[j]);
    }
  }
}

// Any length and alignment: rows are walked twice by the block, dw is added up in the
// block's own row of part.
template <typename T, typename R>
__global__ __launch_bounds__(kWalk) void res_norm_bwd_walk_kernel(const ResNormParams p) {
  __shared__ float sh[kWalk / 64];
  const int64_t n = p.dim;
  float* mine = p.dw ? p.part + blockIdx.x * n : nullptr;
  if (mine)
    for (int64_t k = threadIdx.x; k < n; k += kWalk) mine[k] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.rows; row += p.parts) {
    const R* res = static_cast<const R*>(p.res) + row_at(p, row, p.res_batch, p.res_row);
    const T* dout = static_cast<const T*>(p.dout) + row * n;
    float s2 = 0.0f, sv = 0.0f;
    for (int64_t k = threadIdx.x; k < n; k += kWalk) {
      const float v = Elem<R>::load1(res + k);
      s2 = __builtin_fmaf(v, v, s2);
      sv = __builtin_fmaf(Elem<T>::load1(dout + k) * (p.w ? p.w[k] : 1.0f), v, sv);
    }
    s2 = team_join<kWalk, false>(s2, sh);
    sv = team_join<kWalk, false>(sv, sh);
    const float r = root_of(s2, p, [&](float sc) {
      float t2 = 0.0f;
      for (int64_t k = threadIdx.x; k < n; k += kWalk) {
        const float v = Elem<R>::load1(res + k) * sc;
        t2 = __builtin_fmaf(v, v, t2);
      }
      return team_join<kWalk, false>(t2, sh);
    });
    const float kk = r * (sv / (float)p.dim);
    for (int64_t k = threadIdx.x; k < n; k += kWalk) {
      const float hat = Elem<R>::load1(res + k) * r, dy = Elem<T>::load1(dout + k);
      const float g = p.dres ? Elem<R>::load1(static_cast<const R*>(p.dres) + row * n + k) : 0.0f;
      const float d = __builtin_fmaf(
          r, __builtin_fmaf(-hat, kk, dy * (p.w ? p.w[k] : 1.0f)), g);
      Elem<T>::store1(static_cast<T*>(p.dx) + row * n + k, d);
      if (p.dresidual) Elem<R>::store1(static_cast<R*>(p.dresidual) + row * n + k, d);
      if (mine) mine[k] = __builtin_fmaf(dy, hat, mine[k]);
    }
  }
}

// dw: the parts summed in order, 16 slices of them by 64 channels.
__global__ __launch_bounds__(1024) void res_norm_sum_kernel(const ResNormParams p) {
  __shared__ float red[16][64];
  const int cl = threadIdx.x & 63, sl = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + cl;
  float sum = 0.0f;
  if (c < p.dim) {
#pragma unroll 8
    for (int64_t i = sl; i < p.parts; i += 16) sum += p.part[i * p.dim + c];
  }
  red[sl][cl] = sum;
  __syncthreads();
  if (sl == 0 && c < p.dim) {
    for (int j = 1; j < 16; ++j) sum += red[j][cl];
    p.dw[c] = sum;
  }
}

template <typename T, typename R, bool FP8, int V, int TEAM, int NV>
hipError_t fwd_go(const ResNormParams& p, hipStream_t s) {
  const int64_t blocks = (p.rows + 256 / TEAM - 1) / (256 / TEAM);
  hipLaunchKernelGGL((res_norm_fwd_kernel<T, R, FP8, V, TEAM, NV>),
                     dim3((unsigned)(blocks < kFwdBlocks ? blocks : kFwdBlocks)), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R, bool FP8, int V>
hipError_t fwd_v(const ResNormParams& p, hipStream_t s) {
  const int64_t nv = (p.dim + V - 1) / V;
  if (nv <= 64) return fwd_go<T, R, FP8, V, 64, 1>(p, s);
  if (nv <= 128) return fwd_go<T, R, FP8, V, 64, 2>(p, s);
  if (nv <= 192) return fwd_go<T, R, FP8, V, 64, 3>(p, s);
  if (nv <= 256) return fwd_go<T, R, FP8, V, 64, 4>(p, s);
  if (nv <= 512) return fwd_go<T, R, FP8, V, 256, 2>(p, s);
  if (nv <= 768) return fwd_go<T, R, FP8, V, 256, 3>(p, s);
  if (nv <= 1024) return fwd_go<T, R, FP8, V, 256, 4>(p, s);
  if (nv <= 2048) return fwd_go<T, R, FP8, V, 256, 8>(p, s);
  if constexpr (V == 1) {
    if (nv <= 4096) return fwd_go<T, R, FP8, V, 256, 16>(p, s);
    if (nv <= 8192) return fwd_go<T, R, FP8, V, 256, 32>(p, s);
  }
  hipLaunchKernelGGL((res_norm_fwd_walk_kernel<T, R, FP8, V>),
                     dim3((unsigned)(p.rows < kFwdBlocks ? p.rows : kFwdBlocks)), dim3(kWalk), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R>
hipError_t fwd_t(const ResNormParams& p, bool fp8, hipStream_t s) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  if (p.vec) return fp8 ? fwd_v<T, R, true, V>(p, s) : fwd_v<T, R, false, V>(p, s);
  return fp8 ? fwd_v<T, R, true, 1>(p, s) : fwd_v<T, R, false, 1>(p, s);
}

template <typename T, typename R, int V, int TEAM, int NV>
hipError_t bwd_go(const ResNormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((res_norm_bwd_kernel<T, R, V, TEAM, NV>), dim3((unsigned)p.parts),
                     dim3(TEAM > 256 ? TEAM : 256), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R, int V>
hipError_t bwd_v(const ResNormParams& p, hipStream_t s) {
  const int64_t nv = (p.dim + V - 1) / V;
  if (nv <= 64) return bwd_go<T, R, V, 64, 1>(p, s);
  if (nv <= 128) return bwd_go<T, R, V, 64, 2>(p, s);
  if (nv <= 192) return bwd_go<T, R, V, 64, 3>(p, s);
  if (nv <= 256) return bwd_go<T, R, V, 256, 1>(p, s);
  if (nv <= 512) return bwd_go<T, R, V, 256, 2>(p, s);
  if (nv <= 768) return bwd_go<T, R, V, 256, 3>(p, s);
  if (nv <= 1024) return bwd_go<T, R, V, 256, 4>(p, s);
  if (nv <= 1280) return bwd_go<T, R, V, 256, 5>(p, s);
  if (nv <= 1536) return bwd_go<T, R, V, 256, 6>(p, s);
  if (nv <= 2048) return bwd_go<T, R, V, 512, 4>(p, s);
  if (nv <= 4096) return bwd_go<T, R, V, 512, 8>(p, s);
  if constexpr (V == 1)
    if (nv <= 8192) return bwd_go<T, R, V, 512, 16>(p, s);
  hipLaunchKernelGGL((res_norm_bwd_walk_kernel<T, R>), dim3((unsigned)p.parts), dim3(kWalk), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R>
hipError_t bwd_t(const ResNormParams& p, hipStream_t s) {
  const hipError_t e = p.vec ? bwd_v<T, R, 4>(p, s) : bwd_v<T, R, 1>(p, s);
  if (e != hipSuccess || !p.dw) return e;
  hipLaunchKernelGGL(res_norm_sum_kernel, dim3((unsigned)((p.dim + 63) / 64)), dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace

int64_t res_norm_parts(int64_t rows) { return rows < kParts ? rows : kParts; }

hipError_t dispatch_res_norm_fwd(const ResNormParams& p, ResNormKind kind, bool fp8,
                                 hipStream_t s) {
  switch (kind) {
    case kResF32: return fwd_t<float, float>(p, fp8, s);
    case kResBf16: return fwd_t<bf16_t, bf16_t>(p, fp8, s);
    default: return fwd_t<bf16_t, float>(p, fp8, s);
  }
}

hipError_t dispatch_res_norm_bwd(const ResNormParams& p, ResNormKind kind, hipStream_t s) {
  switch (kind) {
    case kResF32: return bwd_t<float, float>(p, s);
    case kResBf16: return bwd_t<bf16_t, bf16_t>(p, s);
    default: return bwd_t<bf16_t, float>(p, s);
  }
}

}  // namespace mscan
