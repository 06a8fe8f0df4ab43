// Root-mean-square norm with the residual's addition, rows of token-major activations:
//   res = x + residual (as it is stored),  out = res r w,  r = 1 / sqrt(mean(res^2) + eps)
// in the activations' type, or in 8 bits under the row's scale max|out| / 448.
// Backward, with dhat = dout w:
//   d = dres + r (dhat - res r^2 mean(dhat res)),  dw = sum over rows of dout res r
//
// A team of 64 to 512 threads takes a row and keeps it in registers: every tensor is
// read once and written once, all of a row's loads are in flight together, and the largest
// value of 8 bits is found on the way.  Rows too long for that are walked again from the
// cache.  Bound by HBM: the forward of 16384 rows of 1536 in bfloat16 takes 31 to 34 us (201
// MB, 5.9 TB/s or more; 36 to 37 where each group's loads wait for those before), of 4096 of
// 5120 on a float32 stream into 8 bits 39 to 41 (231 MB, 5.7; 47); the backward of 4096 of 5120
// in bfloat16 29 to 32 (168 MB, 5.2), and 4 for the sum of dw.  Rows that start anywhere are
// read as wide: 4096 of 6001 in bfloat16 take 32 us forward, 52 backward (element by element
// 122 and 120), 2000 of 8191 24 and 36 (75 and 75).
#include "recurrent_common.hpp"

namespace mscan {

namespace {

constexpr int kParts = 512;        // blocks of the backward: two a CU
constexpr int kFwdBlocks = (1 << 22) - 1;   // of up to 1024 threads in one launch
constexpr int kWalk = 1024;
// Rows up to here go by single elements, one a lane: 27941 of 38 in bfloat16 take 8.0 us
// forward and 13.5 backward (11.2 and 15.6 in groups; their bytes 1.7 at 5.0 TB/s), 16000 of
// 64 5.5 and 9.6 (6.7 and 10.4; 1.6); 64000 of 128 24 and 30 by two elements a lane, 20 and
// 29 in groups (13).  What is left above the bytes is lanes without work: a row is a wave's.
constexpr int kNarrow = 64;

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
// vanishes beside an eps that does), `again` forms it from values times a scale: 2^28
// squares of up to (2^128 2^-90)^2 stay below 2^104, and of a sum past the range the root
// mean square is 2^50 at least, times the scale 2^-40.
__device__ __forceinline__ bool in_range(float s2, const ResNormParams& p) {
  return __builtin_expect(s2 < 3e38f && (s2 > 0x1p-80f || p.eps > 0x1p-90f), 1);
}
template <typename F>
__device__ __forceinline__ float root_of(float s2, const ResNormParams& p, F again) {
  const float n = (float)p.dim;
  if (in_range(s2, p))
    return 1.0f / __builtin_sqrtf(s2 / n + p.eps);
  const float sc = s2 < 1.0f ? 0x1p70f : 0x1p-90f;
  return sc / __builtin_sqrtf(again(sc) / n + p.eps * sc * sc);
}

// What the backward takes of a row's two sums: r = 1 / sqrt(mean(res^2) + eps), and
// mean(dhat res) r, the mean of dhat times the normed row.  Where the squares' sum passes
// float32's range, `squares` forms r as root_of does, and `normed` the second sum from res r,
// whose values are sqrt(dim) at most.  `on`: whether there is a row; the zeros of none have
// no root without eps, and are to add nothing to dw.
struct RowGrad {
  float r, kk;
  template <typename F, typename G>
  __device__ __forceinline__ RowGrad(float s2, float sv, const ResNormParams& p, bool on, F squares,
                                     G normed) {
    const float n = (float)p.dim;
    if (in_range(s2, p)) {
      r = 1.0f / __builtin_sqrtf(s2 / n + p.eps);
      kk = r * (sv / n);
    } else {
      r = root_of(s2, p, squares);
      if (!on) r = 0.0f;
      kk = normed(r) / n;
    }
  }
};

// V elements of a row.  EVEN: every row starts on 16 bytes and is whole groups of V.
// Otherwise the place is any element's: the memory takes wide accesses there too.
template <bool EVEN, typename T, int V>
struct Words {   // as they lie in memory: kept so while loads are in flight
  static constexpr int N = V * sizeof(T) <= 4 ? 1 : V * sizeof(T) / 4;
  uint32_t w[N];
  __device__ __forceinline__ void load(const void* p) {
    constexpr int bytes = V * sizeof(T);
    const void* q = __builtin_assume_aligned(p, !EVEN ? sizeof(T) : bytes < 16 ? bytes : 16);
    if constexpr (bytes == 2) {
      uint16_t one;
      __builtin_memcpy(&one, q, 2);
      w[0] = one;
    } else {
      __builtin_memcpy(w, q, bytes);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
      else v[i] = i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
  }
};

template <bool EVEN, typename T, int V>
__device__ __forceinline__ void load_row(const void* p, int64_t at, float (&v)[V]) {
  Words<EVEN, T, V> r;
  r.load(static_cast<const T*>(p) + at);
  r.get(v);
}

template <bool EVEN, typename T, int V>
__device__ __forceinline__ void store_row(void* p, int64_t at, const float (&v)[V]) {
  if constexpr (EVEN || V == 1) {
    store_vec<T, V>(p, at, v);
  } else if constexpr (sizeof(T) == 4) {
    __builtin_memcpy(static_cast<T*>(p) + at, v, V * sizeof(T));
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    __builtin_memcpy(static_cast<T*>(p) + at, w, V * sizeof(T));
  }
}

// The group of V elements that a thread takes: `k0` by its number.  A row's last group ends
// with the row, whatever that leaves of it: its first `drop` elements are another thread's
// too, which counts them in its sums; both store the same values.
template <bool EVEN, int V>
struct Group {
  uint32_t k;
  int drop;
  bool in;
  __device__ __forceinline__ Group(uint32_t k0, uint32_t n) : k(k0), drop(0), in(k0 < n) {
    if constexpr (!EVEN && V > 1) {
      drop = (int)k0 - (int)(n - V);
      if (drop > 0) k = n - V;
    }
  }
  __device__ __forceinline__ float own(int v, float x) const {
    return !EVEN && V > 1 && v < drop ? 0.0f : x;
  }
};

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

// To the nearest of e4m3, ties to even (v_cvt_pk_fp8_f32): |y| is at most 448 and two
// units of float32 in its last place, which rounds to 448; a NaN stays one.
template <bool EVEN, int V>
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
    if constexpr (!EVEN) __builtin_memcpy(q, w, V);
    else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(q) = w[0];
    else *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  }
}

// What a row's values are divided by for 8 bits: its scale, at least 2^-100 / 448.  The
// quotient is the sum of the products with a reciprocal in two floats, rounded once (the
// product with one took 2.4 % of rows of quarters up to 7 to the other neighbour of a
// middle).  Over an infinite scale finite values are zeros, infinities NaN.
struct RowScale {
  float scale, hi, lo;
  __device__ __forceinline__ explicit RowScale(float most)
      : scale(__builtin_fmaxf(most, 0x1p-100f) / 448.0f) {
    const float by = scale < __builtin_inff() ? scale : 0.0f, first = fast_rcp(scale);
    hi = __builtin_fmaf(__builtin_fmaf(-by, first, 1.0f), first, first);
    lo = __builtin_fmaf(-by, hi, 1.0f) * hi;
  }
  __device__ __forceinline__ float over(float y) const { return __builtin_fmaf(y, hi, y * lo); }
};

template <bool EVEN, int V>
__device__ __forceinline__ void load_weight(const float* w, int64_t at, float (&v)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = 1.0f;
  if (w) load_row<EVEN, float, V>(w, at, v);
}

template <typename T, typename R, bool FP8, bool EVEN, int V, int TEAM, int NV>
__global__ __launch_bounds__(256) void res_norm_fwd_kernel(const ResNormParams p) {
  __shared__ float sh[4];
  constexpr int TEAMS = 256 / TEAM;
  constexpr bool EARLY = NV * V <= 32;
  const int tid = threadIdx.x & (TEAM - 1);
  const int64_t n = p.dim;
  const int64_t step = (int64_t)gridDim.x * TEAMS;
  for (int64_t row0 = (int64_t)blockIdx.x * TEAMS; row0 < p.rows; row0 += step) {
    const int64_t row = row0 + threadIdx.x / TEAM;
    const bool on = row < p.rows;                 // whole teams
    const int64_t x0 = row_at(p, row, p.x_batch, p.x_row);
    const int64_t r0 = row_at(p, row, p.res_batch, p.res_row);
    // every load of the row is in flight at once, the weights' too where there is room
    Words<EVEN, T, V> xr[NV];
    Words<EVEN, R, V> rr[NV];
    float x[NV][V], w[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      xr[j].zero();
      if (on && g.in) xr[j].load(place<T>(p.x, x0, g.k));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      rr[j].zero();
      if (p.res && on && g.in) rr[j].load(place<R>(p.res, r0, g.k));
    }
    auto weights = [&](int j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
#pragma unroll
      for (int v = 0; v < V; ++v) w[j][v] = 1.0f;
      if (p.w && g.in) load_row<EVEN, float, V>(place<float>(p.w, 0, g.k), 0, w[j]);
    };
    if constexpr (EARLY)
#pragma unroll
      for (int j = 0; j < NV; ++j) weights(j);
    float s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      xr[j].get(x[j]);
      if (p.res) {
        float r[V];
        rr[j].get(r);
        add_stored<R, V>(x[j], r);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float t = g.own(v, x[j][v]);
        s2 = __builtin_fmaf(t, t, s2);
      }
    }
    s2 = team_join<TEAM, false>(s2, sh);
    const float root = root_of(s2, p, [&](float sc) {
      float t2 = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float t = g.own(v, x[j][v]) * sc;
          t2 = __builtin_fmaf(t, t, t2);
        }
      }
      return team_join<TEAM, false>(t2, sh);
    });
    float y[NV][V], most = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      if (on && g.in) {
        if (p.res) store_row<EVEN, R, V>(p.res_out, row * n + g.k, x[j]);
        if constexpr (!EARLY) weights(j);
#pragma unroll
        for (int v = 0; v < V; ++v) y[j][v] = x[j][v] * root * w[j][v];
        if constexpr (!FP8) store_row<EVEN, T, V>(p.out, row * n + g.k, y[j]);
        else
#pragma unroll
          for (int v = 0; v < V; ++v) most = __builtin_fmaxf(most, __builtin_fabsf(y[j][v]));
      }
    }
    if constexpr (FP8) {
      const RowScale to(team_join<TEAM, true>(most, sh));
      if (on && tid == 0) p.scale[row] = to.scale;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
        if (on && g.in) {
#pragma unroll
          for (int v = 0; v < V; ++v) y[j][v] = to.over(y[j][v]);
          store_e4m3<EVEN, V>(p.out, row * n + g.k, y[j]);
        }
      }
    }
  }
}

// Rows too long for the registers: walked two or three times by a block.  A thread's share
// of a sum has no bound on its terms and is held in 64 bits (in 32 a row of 2^28 squares lost
// 6e-5 of their sum: small ones beside a large sum are rounded to nothing).
template <typename T, typename R, bool FP8, bool EVEN, int V>
__global__ __launch_bounds__(kWalk) void res_norm_fwd_walk_kernel(const ResNormParams p) {
  __shared__ float sh[kWalk / 64];
  const int64_t n = p.dim;
  // every group of V elements, and one by one what is left behind the last
  auto walk = [&](auto step) {
    float x[V], one[1];
    int64_t k = (int64_t)threadIdx.x * V;
    for (; k + V <= n; k += kWalk * V) step(k, x);
    if constexpr (!EVEN) {
      k = n / V * V + threadIdx.x;
      if (k < n) step(k, one);
    }
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t x0 = row_at(p, row, p.x_batch, p.x_row);
    const int64_t r0 = row_at(p, row, p.res_batch, p.res_row);
    auto sum = [&](int64_t k, auto& x) {
      constexpr int W = sizeof(x) / 4;
      float r[W];
      load_row<EVEN, T, W>(p.x, x0 + k, x);
      if (p.res) {
        load_row<EVEN, R, W>(p.res, r0 + k, r);
        add_stored<R, W>(x, r);
      }
    };
    auto squares = [&](float sc) {
      double s2 = 0.0;
      walk([&](int64_t k, auto& x) {
        float t = 0.0f;
        sum(k, x);
        for (float v : x) t = __builtin_fmaf(v * sc, v * sc, t);
        s2 += t;
      });
      return team_join<kWalk, false>((float)s2, sh);
    };
    const float root = root_of(squares(1.0f), p, squares);
    auto normed = [&](int64_t k, auto& x, auto& y) {
      constexpr int W = sizeof(x) / 4;
      float w[W];
      sum(k, x);
      load_weight<EVEN, W>(p.w, k, w);
#pragma unroll
      for (int v = 0; v < W; ++v) y[v] = x[v] * root * w[v];
    };
    float most = 0.0f;
    if constexpr (FP8) {
      walk([&](int64_t k, auto& x) {
        normed(k, x, x);
        for (float v : x) most = __builtin_fmaxf(most, __builtin_fabsf(v));
      });
      most = team_join<kWalk, true>(most, sh);
    }
    const RowScale to(most);
    if (FP8 && threadIdx.x == 0) p.scale[row] = to.scale;
    walk([&](int64_t k, auto& x) {
      constexpr int W = sizeof(x) / 4;
      float y[W];
      normed(k, x, y);
      if (p.res) store_row<EVEN, R, W>(p.res_out, row * n + k, x);
      if constexpr (FP8) {
#pragma unroll
        for (int v = 0; v < W; ++v) y[v] = to.over(y[v]);
        store_e4m3<EVEN, W>(p.out, row * n + k, y);
      } else {
        store_row<EVEN, T, W>(p.out, row * n + k, y);
      }
    });
  }
}

// Block `part`: its teams take every (parts * TEAMS)-th row, the next row's loads in
// flight while one is worked on (where the registers hold both), and leave the block's
// share of dw in part.
template <typename T, typename R, bool EVEN, int V, int TEAM, int NV>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void res_norm_bwd_kernel(
    const ResNormParams p) {
  constexpr bool AHEAD = NV * V <= 24;
  static_assert(EVEN || AHEAD, "a row is read whole before any of it is written");
  constexpr int THREADS = TEAM > 256 ? TEAM : 256, TEAMS = THREADS / TEAM;
  __shared__ float sh[THREADS / 64];
  __shared__ float red[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? TEAM * NV * V : 1];
  const int tid = threadIdx.x & (TEAM - 1), team = threadIdx.x / TEAM;
  const int64_t n = p.dim;         // at most 16384 here
  float w[NV][V], dw[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[j][v] = 1.0f;
      dw[j][v] = 0.0f;
    }
    if (AHEAD && p.w && g.in) load_row<EVEN, float, V>(place<float>(p.w, 0, g.k), 0, w[j]);
  }
  Words<EVEN, R, V> xr[NV], gr[NV];
  Words<EVEN, T, V> yr[NV];
  auto load = [&](int64_t row) {
    const int64_t r0 = row_at(p, row, p.res_batch, p.res_row);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      xr[j].zero();
      yr[j].zero();
      if (g.in && row < p.rows) {
        xr[j].load(place<R>(p.res, r0, g.k));
        yr[j].load(place<T>(p.dout, row * n, g.k));
      }
    }
  };
  auto load_dres = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      gr[j].zero();
      if (p.dres && g.in && row < p.rows) gr[j].load(place<R>(p.dres, row * n, g.k));
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
    float x[NV][V], dy[NV][V], ds[NV][V];
    float s2 = 0.0f, sv = 0.0f;
    if (!AHEAD) load(row);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xr[j].get(x[j]);
      yr[j].get(dy[j]);
      if (AHEAD) gr[j].get(ds[j]);
    }
    if (AHEAD) {
      load(row + step);
      load_dres(row + step);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {       // from the cache, row by row
        const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
        if (p.w && g.in) load_row<EVEN, float, V>(place<float>(p.w, 0, g.k), 0, w[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float t = g.own(v, x[j][v]);
        s2 = __builtin_fmaf(t, t, s2);
        sv = __builtin_fmaf(g.own(v, dy[j][v] * w[j][v]), t, sv);
      }
    }
    s2 = team_join<TEAM, false>(s2, sh);
    sv = team_join<TEAM, false>(sv, sh);
    const RowGrad row_grad(
        s2, sv, p, TEAMS == 1 || row < p.rows,
        [&](float sc) {
          float t2 = 0.0f;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
#pragma unroll
            for (int v = 0; v < V; ++v) {
              const float t = g.own(v, x[j][v]) * sc;
              t2 = __builtin_fmaf(t, t, t2);
            }
          }
          return team_join<TEAM, false>(t2, sh);
        },
        [&](float r) {
          float t = 0.0f;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
#pragma unroll
            for (int v = 0; v < V; ++v)
              t = __builtin_fmaf(g.own(v, dy[j][v] * w[j][v]), x[j][v] * r, t);
          }
          return team_join<TEAM, false>(t, sh);
        });
    const float r = row_grad.r, kk = row_grad.kk;
    if (!AHEAD) {
      mem_fence_compiler();                // not before the sums, which need registers
      load_dres(row);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      float d[V];
      if (!AHEAD) gr[j].get(ds[j]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float hat = x[j][v] * r;
        d[v] = __builtin_fmaf(r, __builtin_fmaf(-hat, kk, dy[j][v] * w[j][v]), ds[j][v]);
        dw[j][v] = __builtin_fmaf(dy[j][v], hat, dw[j][v]);
      }
      if (g.in && row < p.rows) {
        store_row<EVEN, T, V>(place<T>(p.dx, row * n, g.k), 0, d);
        if (sizeof(T) != sizeof(R) && p.dresidual)
          store_row<EVEN, R, V>(place<R>(p.dresidual, row * n, g.k), 0, d);
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
      const Group<EVEN, V> g(((jv / V) * TEAM + lane) * V, (uint32_t)n);
      float sum = red[0][i];
#pragma unroll
      for (int m = 1; m < TEAMS; ++m) sum += red[m][i];
      if (g.in) mine[g.k + jv % V] = sum;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Group<EVEN, V> g((j * TEAM + tid) * V, (uint32_t)n);
      if (g.in) store_row<EVEN, float, V>(mine, g.k, dw[j]);
    }
  }
}

// Any length and alignment: rows are walked twice by the block, sums held as in the
// forward's walk; dw is added up in the block's own row of part, each thread at its own
// places.
template <typename T, typename R>
__global__ __launch_bounds__(kWalk) void res_norm_bwd_walk_kernel(const ResNormParams p) {
  constexpr int V = 4;
  __shared__ float sh[kWalk / 64];
  const int64_t n = p.dim;
  float* mine = p.dw ? p.part + blockIdx.x * n : nullptr;
  // every group of V elements, and one by one what is left behind the last
  auto walk = [&](auto step) {
    float x[V], one[1];
    int64_t k = (int64_t)threadIdx.x * V;
    for (; k + V <= n; k += kWalk * V) step(k, x);
    k = n / V * V + threadIdx.x;
    if (k < n) step(k, one);
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += p.parts) {
    const int64_t r0 = row_at(p, row, p.res_batch, p.res_row), d0 = row * n;
    double s2d = 0.0, svd = 0.0;
    walk([&](int64_t k, auto& x) {
      constexpr int W = sizeof(x) / 4;
      float dy[W], w[W], t2 = 0.0f, tv = 0.0f;
      load_row<false, R, W>(p.res, r0 + k, x);
      load_row<false, T, W>(p.dout, d0 + k, dy);
      load_weight<false, W>(p.w, k, w);
#pragma unroll
      for (int v = 0; v < W; ++v) {
        t2 = __builtin_fmaf(x[v], x[v], t2);
        tv = __builtin_fmaf(dy[v] * w[v], x[v], tv);
      }
      s2d += t2;
      svd += tv;
    });
    const float s2 = team_join<kWalk, false>((float)s2d, sh);
    const float sv = team_join<kWalk, false>((float)svd, sh);
    const RowGrad row_grad(
        s2, sv, p, true,
        [&](float sc) {
          double t2 = 0.0;
          walk([&](int64_t k, auto& x) {
            float t = 0.0f;
            load_row<false, R, sizeof(x) / 4>(p.res, r0 + k, x);
            for (float v : x) t = __builtin_fmaf(v * sc, v * sc, t);
            t2 += t;
          });
          return team_join<kWalk, false>((float)t2, sh);
        },
        [&](float r) {
          double t = 0.0;
          walk([&](int64_t k, auto& x) {
            constexpr int W = sizeof(x) / 4;
            float dy[W], w[W], tv = 0.0f;
            load_row<false, R, W>(p.res, r0 + k, x);
            load_row<false, T, W>(p.dout, d0 + k, dy);
            load_weight<false, W>(p.w, k, w);
#pragma unroll
            for (int v = 0; v < W; ++v) tv = __builtin_fmaf(dy[v] * w[v], x[v] * r, tv);
            t += tv;
          });
          return team_join<kWalk, false>((float)t, sh);
        });
    const float r = row_grad.r, kk = row_grad.kk;
    walk([&](int64_t k, auto& x) {
      constexpr int W = sizeof(x) / 4;
      float dy[W], w[W], ds[W], dw[W], d[W];
      load_row<false, R, W>(p.res, r0 + k, x);
      load_row<false, T, W>(p.dout, d0 + k, dy);
      load_weight<false, W>(p.w, k, w);
#pragma unroll
      for (int v = 0; v < W; ++v) ds[v] = dw[v] = 0.0f;
      if (p.dres) load_row<false, R, W>(p.dres, d0 + k, ds);
      if (mine && row != blockIdx.x) load_row<false, float, W>(mine, k, dw);
#pragma unroll
      for (int v = 0; v < W; ++v) {
        const float hat = x[v] * r;
        d[v] = __builtin_fmaf(r, __builtin_fmaf(-hat, kk, dy[v] * w[v]), ds[v]);
        dw[v] = __builtin_fmaf(dy[v], hat, dw[v]);
      }
      store_row<false, T, W>(p.dx, d0 + k, d);
      if (p.dresidual) store_row<false, R, W>(p.dresidual, d0 + k, d);
      if (mine) store_row<false, float, W>(mine, k, dw);
    });
  }
}

// dw: the parts summed in order, 16 slices of them by 64 channels, from channel c0 on.
constexpr int kSumChannels = 64, kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void res_norm_sum_kernel(const ResNormParams p,
                                                                   const int64_t c0) {
  __shared__ float red[16][64];
  const int cl = threadIdx.x & 63, sl = threadIdx.x >> 6;
  const int64_t c = c0 + (int64_t)blockIdx.x * kSumChannels + cl;
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

template <typename T, typename R, bool FP8, bool EVEN, int V, int TEAM, int NV>
hipError_t fwd_go(const ResNormParams& p, hipStream_t s) {
  const int64_t blocks = (p.rows + 256 / TEAM - 1) / (256 / TEAM);
  hipLaunchKernelGGL((res_norm_fwd_kernel<T, R, FP8, EVEN, V, TEAM, NV>),
                     dim3((unsigned)(blocks < kFwdBlocks ? blocks : kFwdBlocks)), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R, bool FP8, bool EVEN>
hipError_t fwd_v(const ResNormParams& p, hipStream_t s) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  const int64_t nv = (p.dim + V - 1) / V;
  if (nv <= 64) return fwd_go<T, R, FP8, EVEN, V, 64, 1>(p, s);
  if (nv <= 128) return fwd_go<T, R, FP8, EVEN, V, 64, 2>(p, s);
  if (nv <= 192) return fwd_go<T, R, FP8, EVEN, V, 64, 3>(p, s);
  if (nv <= 256) return fwd_go<T, R, FP8, EVEN, V, 64, 4>(p, s);
  if (nv <= 512) return fwd_go<T, R, FP8, EVEN, V, 256, 2>(p, s);
  if (nv <= 768) return fwd_go<T, R, FP8, EVEN, V, 256, 3>(p, s);
  if (nv <= 1024) return fwd_go<T, R, FP8, EVEN, V, 256, 4>(p, s);
  if (nv <= 2048) return fwd_go<T, R, FP8, EVEN, V, 256, 8>(p, s);
  hipLaunchKernelGGL((res_norm_fwd_walk_kernel<T, R, FP8, EVEN, V>),
                     dim3((unsigned)(p.rows < kFwdBlocks ? p.rows : kFwdBlocks)), dim3(kWalk), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R>
hipError_t fwd_t(const ResNormParams& p, bool fp8, hipStream_t s) {
  if (p.dim <= kNarrow)
    return fp8 ? fwd_go<T, R, true, false, 1, 64, 1>(p, s)
               : fwd_go<T, R, false, false, 1, 64, 1>(p, s);
  if (p.vec) return fp8 ? fwd_v<T, R, true, true>(p, s) : fwd_v<T, R, false, true>(p, s);
  return fp8 ? fwd_v<T, R, true, false>(p, s) : fwd_v<T, R, false, false>(p, s);
}

template <typename T, typename R, bool EVEN, int V, int TEAM, int NV>
hipError_t bwd_go(const ResNormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((res_norm_bwd_kernel<T, R, EVEN, V, TEAM, NV>), dim3((unsigned)p.parts),
                     dim3(TEAM > 256 ? TEAM : 256), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R, bool EVEN>
hipError_t bwd_v(const ResNormParams& p, hipStream_t s) {
  constexpr int V = 4;
  const int64_t nv = (p.dim + V - 1) / V;
  if (nv <= 64) return bwd_go<T, R, EVEN, V, 64, 1>(p, s);
  if (nv <= 128) return bwd_go<T, R, EVEN, V, 64, 2>(p, s);
  if (nv <= 192) return bwd_go<T, R, EVEN, V, 64, 3>(p, s);
  if (nv <= 256) return bwd_go<T, R, EVEN, V, 256, 1>(p, s);
  if (nv <= 512) return bwd_go<T, R, EVEN, V, 256, 2>(p, s);
  if (nv <= 768) return bwd_go<T, R, EVEN, V, 256, 3>(p, s);
  if (nv <= 1024) return bwd_go<T, R, EVEN, V, 256, 4>(p, s);
  if (nv <= 1280) return bwd_go<T, R, EVEN, V, 256, 5>(p, s);
  if (nv <= 1536) return bwd_go<T, R, EVEN, V, 256, 6>(p, s);
  if (nv <= 2048) return bwd_go<T, R, EVEN, V, 512, 4>(p, s);
  if constexpr (EVEN)    // the others would spill
    if (nv <= 4096) return bwd_go<T, R, EVEN, V, 512, 8>(p, s);
  hipLaunchKernelGGL((res_norm_bwd_walk_kernel<T, R>), dim3((unsigned)p.parts), dim3(kWalk), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R>
hipError_t bwd_t(const ResNormParams& p, hipStream_t s) {
  hipError_t e = p.dim <= kNarrow ? bwd_go<T, R, false, 1, 64, 1>(p, s)
                 : p.vec          ? bwd_v<T, R, true>(p, s)
                                  : bwd_v<T, R, false>(p, s);
  if (!p.dw) return e;
  // as many launches as hold the channels: one, up to 2^28 - 64 of them
  constexpr int64_t most = kSumChannels * max_blocks(kSumThreads);
  for (int64_t c0 = 0; c0 < p.dim && e == hipSuccess; c0 += most) {
    const int64_t n = p.dim - c0 < most ? p.dim - c0 : most;
    hipLaunchKernelGGL(res_norm_sum_kernel, dim3((unsigned)((n + kSumChannels - 1) / kSumChannels)),
                       dim3(kSumThreads), 0, s, p, c0);
    e = hipGetLastError();
  }
  return e;
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
