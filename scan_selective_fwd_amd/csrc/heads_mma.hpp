// Matrix-product building blocks of the multi-head scan kernels (gfx950).
//
// A chunk of kQ tokens turns the recurrence into products: with S_t the sum of
// the log decays up to t inside the chunk,
//   out_q = sum_{s <= q} (C_q . B_s) e^{S_q - S_s} w_s u_s + e^{S_q} h_in C_q
//   h_out = e^{S_end} h_in + sum_s e^{S_end - S_s} w_s u_s B_s^T
// All of them run on v_mfma_f32_16x16x32_bf16.  An operand of 16 outer by 32
// inner elements is a fragment: lane (i = lane & 15, g = lane >> 4) holds outer
// element i and the inner elements 4g..4g+3 and 16+4g..16+4g+3.  The order of
// the inner elements is free as long as both operands use the same, and with
// this one a result (lane i, g: column i, rows 4g..4g+3) is itself half a
// fragment with its rows as inner elements: the state goes from the update that
// accumulates it to the products that read it without leaving its registers.
//
// Precision.  bfloat16 inputs are exact operands.  A float32 operand (states,
// decay-weighted inputs, float32 inputs) is the exact sum of three bfloat16
// parts of 8 bits each; products of parts are kept down to 2^-24 of the whole,
// so such a product is as good as float32's.  Where a result is stored in
// bfloat16 one rounded part is used instead and said so.
#pragma once

#include "heads_common.hpp"

namespace mscan {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kCols = 64;      // channels of a head a block takes: 16 a wave

// Per type: tokens a chunk, parts of an input operand, row padding of a tile.
// Padding by 16 bytes spreads the rows of a fragment's read over the banks.
template <typename T>
struct Mx;
template <>
struct Mx<bf16_t> {
  static constexpr int Q = 64, PARTS = 1, PAD = 8, V = 8;
};
template <>
struct Mx<float> {
  static constexpr int Q = 32, PARTS = 3, PAD = 4, V = 4;
};

template <int NP>
struct Frag {
  bf16x8 v[NP];
};

__device__ __forceinline__ bf16x8 as_frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// The upper halves of two floats as a bfloat16 pair (a in the low half).
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float top8(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
}

// Eight floats as one rounded part, or as three exact ones.
template <int NP>
__device__ __forceinline__ Frag<NP> to_frag(const float (&x)[8]) {
  Frag<NP> f;
  if constexpr (NP == 1) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
    f.v[0] = as_frag(r);
  } else {
    static_assert(NP == 3, "NP");
    u32x4 r[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      const float a1 = a - top8(a), b1 = b - top8(b);
      const float a2 = a1 - top8(a1), b2 = b1 - top8(b1);
      r[0][j] = pack_hi(a, b);
      r[1][j] = pack_hi(a1, b1);
      r[2][j] = pack_hi(a2, b2);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) f.v[k] = as_frag(r[k]);
  }
  return f;
}

// Two result tiles (inner elements 0..15 and 16..31) as a fragment.
template <int NP>
__device__ __forceinline__ Frag<NP> acc_frag(const f32x4& lo, const f32x4& hi) {
  const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return to_frag<NP>(x);
}

// acc += A B^T over 32 inner elements, part products down to 2^-24.
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const Frag<NA>& a, const Frag<NB>& b) {
  constexpr int NM = NA > NB ? NA : NB;
#pragma unroll
  for (int s = NM - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NB)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[j], acc, 0, 0, 0);
    }
}

__device__ __forceinline__ int lane_i() { return threadIdx.x & 15; }
__device__ __forceinline__ int lane_g() { return (threadIdx.x >> 4) & 3; }

// Fragment of a tile whose rows are the outer elements: rows o0 + i, inner
// elements k0 + ...
template <typename T>
__device__ __forceinline__ Frag<Mx<T>::PARTS> load_rows(const T* tile, int stride, int o0, int k0) {
  const T* q = tile + (o0 + lane_i()) * stride + k0 + 4 * lane_g();
  if constexpr (sizeof(T) == 2) {
    const u32x2 a = *reinterpret_cast<const u32x2*>(q);
    const u32x2 b = *reinterpret_cast<const u32x2*>(q + 16);
    Frag<1> f;
    f.v[0] = as_frag(u32x4{a[0], a[1], b[0], b[1]});
    return f;
  } else {
    return acc_frag<3>(*reinterpret_cast<const f32x4*>(q), *reinterpret_cast<const f32x4*>(q + 16));
  }
}

// The eight values of a fragment of a tile whose rows are the inner elements:
// rows k0 + ..., outer element o0 + i.  bfloat16 tiles use the transposing LDS
// read: a group of 16 lanes reads 4 rows of 16 elements and lane i gets column i.
__device__ __forceinline__ bf16x8 load_cols_raw(const bf16_t* tile, int stride, int o0, int k0) {
  typedef s16x4 __attribute__((address_space(3))) * lds_ptr;
  const int i = lane_i();
  const bf16_t* q = tile + (k0 + 4 * lane_g() + (i >> 2)) * stride + o0 + 4 * (i & 3);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)q);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(q + 16 * stride));
  const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
  return as_frag(u32x4{ua[0], ua[1], ub[0], ub[1]});
}

__device__ __forceinline__ void load_cols_f32(const float* tile, int stride, int o0, int k0,
                                              float (&x)[8]) {
  const float* q = tile + (k0 + 4 * lane_g()) * stride + o0 + lane_i();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = q[j * stride];
    x[4 + j] = q[(16 + j) * stride];
  }
}

template <typename T>
__device__ __forceinline__ Frag<Mx<T>::PARTS> load_cols(const T* tile, int stride, int o0, int k0) {
  if constexpr (sizeof(T) == 2) {
    Frag<1> f;
    f.v[0] = load_cols_raw(tile, stride, o0, k0);
    return f;
  } else {
    float x[8];
    load_cols_f32(tile, stride, o0, k0, x);
    return to_frag<3>(x);
  }
}

// The same fragment with its inner elements weighted by c, as three parts; an
// inner element of weight 0 counts as zero whatever it holds.
template <typename T>
__device__ __forceinline__ Frag<3> load_cols_weighted(const T* tile, int stride, int o0, int k0,
                                                      const float* c) {
  float x[8];
  if constexpr (sizeof(T) == 2) {
    const u32x4 r = __builtin_bit_cast(u32x4, load_cols_raw(tile, stride, o0, k0));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf16_lo(r[j]);
      x[2 * j + 1] = bf16_hi(r[j]);
    }
  } else {
    load_cols_f32(tile, stride, o0, k0, x);
  }
  const f32x4 c0 = *reinterpret_cast<const f32x4*>(c + k0 + 4 * lane_g());
  const f32x4 c1 = *reinterpret_cast<const f32x4*>(c + k0 + 16 + 4 * lane_g());
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = c0[j] == 0.0f ? 0.0f : x[j] * c0[j];
    x[4 + j] = c1[j] == 0.0f ? 0.0f : x[4 + j] * c1[j];
  }
  return to_frag<3>(x);
}

// ---------------------------------------------------------------------------
// Staging: ROWS tokens by COLS elements from global rows to an LDS tile, in
// 16-byte pieces held in registers between the two.
// ---------------------------------------------------------------------------
template <typename T, int ROWS, int COLS>
struct Stage {
  static constexpr int V = 16 / sizeof(T);
  static constexpr int PER_ROW = COLS / V;
  static constexpr int COUNT = (ROWS * PER_ROW + 255) / 256;
  static_assert(COLS % V == 0, "COLS");
  u32x4 v[COUNT];

  // Rows t0 .. t0 + len - 1 of batch row b, elements [at, at + n) of each; the
  // rest of the tile is zero.  VEC: rows start on 16 bytes and n is whole
  // pieces.
  template <bool VEC>
  __device__ __forceinline__ void load(const Rows& r, int64_t b, int64_t t0, int len, int64_t at,
                                       int n) {
    const T* base = static_cast<const T*>(r.p) + b * r.batch + t0 * r.token + at;
#pragma unroll
    for (int k = 0; k < COUNT; ++k) {
      const int idx = k * 256 + threadIdx.x;
      const int row = idx / PER_ROW, c = (idx % PER_ROW) * V;
      v[k] = u32x4{0, 0, 0, 0};
      if (row < len && c < n) {
        const T* q = base + row * r.token + c;
        if constexpr (VEC) {
          v[k] = *reinterpret_cast<const u32x4*>(q);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            if (c + e < n) {
              if constexpr (sizeof(T) == 2) v[k][e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
              else v[k][e] = __builtin_bit_cast(uint32_t, q[e]);
            }
          }
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* tile, int stride) const {
#pragma unroll
    for (int k = 0; k < COUNT; ++k) {
      const int idx = k * 256 + threadIdx.x;
      const int row = idx / PER_ROW, c = (idx % PER_ROW) * V;
      if (ROWS * PER_ROW % 256 == 0 || row < ROWS)
        *reinterpret_cast<u32x4*>(tile + row * stride + c) = v[k];
    }
  }
  // Nonzero when an infinity or a NaN is among the values.
  __device__ __forceinline__ uint32_t non_finite() const {
    constexpr uint32_t e = sizeof(T) == 2 ? 0x7F807F80u : 0x7F800000u;
    constexpr uint32_t one = sizeof(T) == 2 ? 0x00800080u : 0x00800000u;
    constexpr uint32_t top = sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < COUNT; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) bad |= (v[k][j] & e) + one;
    return bad & top;
  }
};

// ---------------------------------------------------------------------------
// The scalars of a chunk, one token a lane of one wave.
// ---------------------------------------------------------------------------
template <int Q>
struct alignas(16) Scal {
  float S[Q];    // sum of the log2 decays from the chunk's start, or from the last flag
  float w[Q];    // weight of the token's input
  float c[Q];    // its weight in the state at the chunk's end (0 if a flag follows)
  float e[Q];    // weight of the entering state in the token's row (0 after a flag)
  int id[Q];     // flags up to the token
  float dec;     // weight of the entering state in the state at the chunk's end
  float pad[3];
};

// Raw step and flag of this lane's token of a chunk, loaded ahead of time.
struct StepIn {
  float raw;
  int flag;
};

template <typename T>
__device__ __forceinline__ StepIn load_step(const HeadsParams& p, int64_t b, int h, float bias,
                                            int64_t t0, int len) {
  const int l = threadIdx.x & 63;
  StepIn s = {0.0f, 0};
  if (l < len) {
    s.raw = Elem<T>::load1(static_cast<const T*>(p.delta.p) + b * p.delta.batch +
                           (t0 + l) * p.delta.token + h) +
            bias;
    if (p.reset) s.flag = p.reset[b * p.L + t0 + l] != 0;
  }
  return s;
}

template <int Q>
__device__ __forceinline__ void chunk_scalars(const HeadsParams& p, const StepIn& in, float A,
                                              int len, Scal<Q>* o) {
  const int l = threadIdx.x & 63;
  const Step st = make_step(in.raw, A, p.softplus != 0, p.zoh != 0);
  float S = l < len ? st.lg : 0.0f;
  const float w = l < len ? st.w : 0.0f;
  const uint64_t flags = __ballot(in.flag && l < len);
  const uint64_t upto = flags & ((2ull << l) - 1ull);
  const int start = upto ? 63 - __builtin_clzll(upto) : 0;
  const int id = __builtin_popcountll(upto), id_end = __builtin_popcountll(flags);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const float t = __shfl_up(S, off);
    if (l - off >= start) S += t;
  }
  const float end = __shfl(S, 63);
  if (l < Q) {
    o->S[l] = S;
    o->w[l] = w;
    o->c[l] = id == id_end ? fast_exp2(end - S) * w : 0.0f;
    o->e[l] = id == 0 ? fast_exp2(S) : 0.0f;
    o->id[l] = id;
  }
  if (l == 0) o->dec = id_end == 0 ? fast_exp2(end) : 0.0f;
}

// x weighted by f; 0 for a weight of 0, whatever x holds.
__device__ __forceinline__ float weigh(float x, float f) { return f == 0.0f ? 0.0f : x * f; }

// ---------------------------------------------------------------------------
// Infinities and NaN.  A matrix product spreads one over its whole row and
// column even where the other factor's weight is zero, so in a chunk that holds
// one, u's are taken out (zeros in their place, and a mark by column), and the
// rows of B that a flag keeps from the state at the chunk's end are cleared.
// What the marked values reach is then set to NaN: the rows of the same
// sequence from the mark on, and the state if the sequence goes on.  All other
// rows keep the bits they have without it.  Called by the whole block, between
// barriers of its own; B's rows must not be read for M afterwards.
// ---------------------------------------------------------------------------
template <typename T, int Q, int NP>
__device__ __forceinline__ void take_out(T* Xs, int xstride, T* Bs, int bstride,
                                         const Scal<Q>& sc, uint64_t* marks) {
  const int id_end = sc.id[Q - 1];
  if (threadIdx.x < kCols) {
    uint64_t m = 0;
    for (int q = 0; q < Q; ++q) {
      const float x = Elem<T>::load1(Xs + q * xstride + threadIdx.x);
      if (!(__builtin_fabsf(x) < __builtin_inff())) {
        m |= 1ull << q;
        Xs[q * xstride + threadIdx.x] = T(0);
      }
    }
    marks[threadIdx.x] = m;
  }
  for (int i = threadIdx.x; i < Q * NP; i += 256)
    if (sc.id[i / NP] != id_end) Bs[(i / NP) * bstride + i % NP] = T(0);
  __syncthreads();
}

// The marks that reach token q: those of its sequence up to it.
template <int Q>
__device__ __forceinline__ bool marked(uint64_t marks, const Scal<Q>& sc, int q) {
  for (int s = 0; s <= q; ++s)
    if ((marks >> s & 1) != 0 && sc.id[s] == sc.id[q]) return true;
  return false;
}

// ---------------------------------------------------------------------------
// The state of a head's 64 columns, rows n, columns p: wave w holds columns
// 16 w + i and, in tile nt, states 16 nt + 4 g + (0..3).
// ---------------------------------------------------------------------------
// Between kernels a state is kept in this order, kCols * 32 NK floats.
template <int NK>
__device__ __forceinline__ int64_t frag_at(int nt) {
  return (((threadIdx.x >> 6) * (2 * NK) + nt) * 64 + (threadIdx.x & 63)) * 4;
}

// From or to (batch, heads, headdim, dstate) arrays; c0: the block's first channel.
template <int NK>
__device__ __forceinline__ void load_state(const float* st, int c0, int P, int N, f32x4 (&h)[2 * NK]) {
  const int pp = c0 + 16 * (threadIdx.x >> 6) + lane_i();
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt) {
    const int n = 16 * nt + 4 * lane_g();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[nt][j] = st && pp < P && n + j < N ? st[(int64_t)pp * N + n + j] : 0.0f;
  }
}

template <int NK>
__device__ __forceinline__ void store_state(float* st, int c0, int P, int N,
                                            const f32x4 (&h)[2 * NK]) {
  const int pp = c0 + 16 * (threadIdx.x >> 6) + lane_i();
  if (pp >= P) return;
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt) {
    const int n = 16 * nt + 4 * lane_g();
    if (N % 4 == 0 && (reinterpret_cast<uintptr_t>(st) & 15) == 0) {
      if (n < N) *reinterpret_cast<f32x4*>(st + (int64_t)pp * N + n) = h[nt];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < N) st[(int64_t)pp * N + n + j] = h[nt][j];
    }
  }
}

// h <- dec h + sum_t c_t keys_t vals_t^T over a chunk's tiles.
template <typename T, int NK>
__device__ __forceinline__ void update_state(f32x4 (&h)[2 * NK], float dec, const T* keys,
                                             int kstride, const T* vals, int vstride,
                                             const float* c) {
  constexpr int Q = Mx<T>::Q;
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) h[nt][j] = weigh(h[nt][j], dec);
#pragma unroll
  for (int ks = 0; ks < Q / 32; ++ks) {
    const Frag<3> x = load_cols_weighted<T>(vals, vstride, 16 * (threadIdx.x >> 6), 32 * ks, c);
#pragma unroll
    for (int nt = 0; nt < 2 * NK; ++nt)
      mma(h[nt], load_cols<T>(keys, kstride, 16 * nt, 32 * ks), x);
  }
}

}  // namespace mscan
