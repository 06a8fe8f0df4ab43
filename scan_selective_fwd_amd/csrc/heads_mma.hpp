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
// so such a product is as good as float32's.  Where the result is stored in
// bfloat16 two parts are used instead, which keep 2^-17 of the operand: the
// result's own rounding, 2^-9, is then all that shows.
#pragma once

#include "heads_common.hpp"

namespace mscan {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Channels: a wave takes a slice of 32 of one head (two tiles of 16), a block
// four slices.  With two tiles a fragment of B or C read from LDS feeds two
// matrix instructions; with one, the LDS reads took longer than the products.
constexpr int kSlice = 32;
constexpr int kCols = 4 * kSlice;

// Per type: tokens a chunk, parts of an input operand, row padding of a tile.
// The LDS serves 16 lanes of 8 bytes at a time over 128 bytes of banks: rows 8
// bytes apart there (PAD) serve fragments along the rows without conflicts,
// rows 32 bytes apart (PADT) the transposing reads; 16 (PADB) serves both in two.
template <typename T>
struct Mx;
template <>
struct Mx<bf16_t> {
  static constexpr int Q = 64, PARTS = 1, PAD = 4, PADT = 16, PADB = 8, V = 8;
};
template <>
struct Mx<float> {
  static constexpr int Q = 32, PARTS = 3, PAD = 4, PADT = 4, PADB = 4, V = 4;
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

// Eight floats as two parts (2^-17 of each is lost) or as three exact ones.
template <int NP>
__device__ __forceinline__ Frag<NP> to_frag(const float (&x)[8]) {
  Frag<NP> f;
  if constexpr (NP == 2) {
    u32x4 r[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      r[0][j] = pack_hi(a, b);
      r[1][j] = pack_bf16(a - top8(a), b - top8(b));
    }
    f.v[0] = as_frag(r[0]);
    f.v[1] = as_frag(r[1]);
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

// acc[r][c] += A[r] B[c]^T over 32 inner elements, part products down to 2^-24.
// The accumulators alternate, so that no instruction waits for the one before.
template <int NA, int NB, int R, int C>
__device__ __forceinline__ void mma(f32x4 (&acc)[R][C], const Frag<NA> (&a)[R],
                                    const Frag<NB> (&b)[C]) {
  constexpr int NM = NA > NB ? NA : NB;
#pragma unroll
  for (int s = NM - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NB)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < C; ++c)
            acc[r][c] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[r].v[i], b[c].v[j], acc[r][c], 0, 0, 0);
    }
}

// A thread's place among the 256 that stage a tile together.
__device__ __forceinline__ int tid256() { return (int)(threadIdx.x & 255); }

__device__ __forceinline__ bool not_finite(float x) {
  return !(__builtin_fabsf(x) < __builtin_inff());
}

// Keeps the scheduler from moving one phase's loads into another, where they
// would only hold registers.
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ int lane_i() { return threadIdx.x & 15; }
__device__ __forceinline__ int lane_g() { return (threadIdx.x >> 4) & 3; }

// A lane's place in a fragment.  lane_fresh() hides it from the optimizer, so
// that addresses made from it are formed again where they are used instead of
// being kept, and spilled, across a loop.
struct Lane {
  int i, g;
};
__device__ __forceinline__ Lane lane_kept() { return {lane_i(), lane_g()}; }
__device__ __forceinline__ Lane lane_fresh() {
  const int t = opaque_int((int)threadIdx.x);
  return {t & 15, (t >> 4) & 3};
}

// Fragment of a tile whose rows are the outer elements: rows o0 + i, inner
// elements k0 + ...
template <typename T>
__device__ __forceinline__ Frag<Mx<T>::PARTS> load_rows(const T* tile, int stride, int o0, int k0,
                                                           Lane ln = lane_kept()) {
  const T* q = tile + ln.i * stride + 4 * ln.g + (o0 * stride + k0);
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
__device__ __forceinline__ bf16x8 load_cols_raw(const bf16_t* tile, int stride, int o0, int k0,
                                                Lane ln = lane_kept()) {
  typedef s16x4 __attribute__((address_space(3))) * lds_ptr;
  const bf16_t* q = tile + (4 * ln.g + (ln.i >> 2)) * stride + 4 * (ln.i & 3) + (k0 * stride + o0);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)q);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(q + 16 * stride));
  const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
  return as_frag(u32x4{ua[0], ua[1], ub[0], ub[1]});
}

__device__ __forceinline__ void load_cols_f32(const float* tile, int stride, int o0, int k0,
                                              float (&x)[8], Lane ln = lane_kept()) {
  const float* q = tile + 4 * ln.g * stride + ln.i + (k0 * stride + o0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = q[j * stride];
    x[4 + j] = q[(16 + j) * stride];
  }
}

template <typename T>
__device__ __forceinline__ Frag<Mx<T>::PARTS> load_cols(const T* tile, int stride, int o0, int k0,
                                                           Lane ln = lane_kept()) {
  if constexpr (sizeof(T) == 2) {
    Frag<1> f;
    f.v[0] = load_cols_raw(tile, stride, o0, k0, ln);
    return f;
  } else {
    float x[8];
    load_cols_f32(tile, stride, o0, k0, x, ln);
    return to_frag<3>(x);
  }
}

// The values of such a fragment, and the fragment weighted by c along its
// inner elements, as three parts.
template <typename T>
struct Cols {
  bf16x8 raw;    // bfloat16
  float x[8];    // float32
  __device__ __forceinline__ void load(const T* tile, int stride, int o0, int k0) {
    if constexpr (sizeof(T) == 2) raw = load_cols_raw(tile, stride, o0, k0);
    else load_cols_f32(tile, stride, o0, k0, x);
  }
  __device__ __forceinline__ Frag<3> weighted(const float* c, int k0) const {
    const f32x4 c0 = *reinterpret_cast<const f32x4*>(c + k0 + 4 * lane_g());
    const f32x4 c1 = *reinterpret_cast<const f32x4*>(c + k0 + 16 + 4 * lane_g());
    float y[8];
    if constexpr (sizeof(T) == 2) {
      const u32x4 r = __builtin_bit_cast(u32x4, raw);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = bf16_lo(r[j]);
        y[2 * j + 1] = bf16_hi(r[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] *= c0[j];
      y[4 + j] *= c1[j];
    }
    return to_frag<3>(y);
  }
  // Part of an operand that is NaN or infinite wherever a value is.
  __device__ __forceinline__ bf16x8 top() const {
    if constexpr (sizeof(T) == 2) {
      return raw;
    } else {
      u32x4 r;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = pack_hi(x[2 * j], x[2 * j + 1]);
      return as_frag(r);
    }
  }
};

// ---------------------------------------------------------------------------
// A range of global memory read with the hardware's range check: 16 bytes at an
// offset, zeros from `bytes` on.  The base and the range are uniform.
// ---------------------------------------------------------------------------
struct Buffer {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Buffer(const void* base, uint32_t bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00027000)) {}
  __device__ __forceinline__ u32x4 load(uint32_t off) const {
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
  }
};
constexpr uint32_t kOutside = 0x80000000u;   // beyond every range: they stay below 2^31

// ---------------------------------------------------------------------------
// Staging: ROWS tokens by COLS elements from global rows to an LDS tile, in
// 16-byte pieces held in registers between the two.
// ---------------------------------------------------------------------------
// The tile's columns are `sub` wide parts (heads); part j's elements are the
// row's [at + j * run, at + j * run + n), n <= run, n <= sub.
template <typename T, int ROWS, int COLS, bool VEC>
struct Stage {
  static constexpr int V = 16 / sizeof(T);
  static constexpr int PER_ROW = COLS / V;
  static constexpr int COUNT = (ROWS * PER_ROW + 255) / 256;
  static_assert(COLS % V == 0 && ROWS * PER_ROW % 256 == 0, "whole pieces a thread");
  static constexpr int STEP = 256 / PER_ROW;   // rows between a thread's pieces
  static_assert(256 % PER_ROW == 0, "a thread keeps its column");
  u32x4 v[COUNT];
  uint32_t off;    // bytes from the chunk's first row to the thread's first piece
  int n_;          // elements of the thread's piece inside the row
  int part, cc;    // the piece's place

  __device__ __forceinline__ void init(const Rows& r, int64_t at, int sub, int run, int n,
                                       int parts) {
    const int c = (tid256() % PER_ROW) * V;
    part = c / sub;
    cc = c - part * sub;
    n_ = part < parts && cc < n ? n - cc : 0;
    // a piece outside the row is out of the buffer's range
    off = n_ > 0 ? (uint32_t)((at + (int64_t)part * run + cc +
                               (int64_t)(tid256() / PER_ROW) * r.token) * (int)sizeof(T))
                 : kOutside;
  }
  // Rows t0 .. t0 + len - 1 of batch row b.  VEC: rows start on 16 bytes, n is
  // whole pieces, and a chunk spans less than 2^31 bytes (the caller's check);
  // the loads carry the chunk's range, and outside it they give zeros.
  __device__ __forceinline__ void load(const Rows& r, int64_t b, int64_t t0, int len, int64_t at,
                                       int run, int width) {
    const char* base = static_cast<const char*>(r.p) + (b * r.batch + t0 * r.token) * (int)sizeof(T);
    if constexpr (VEC) {
      const uint32_t stride = (uint32_t)(r.token * (int)sizeof(T));
      // width: elements from the row's start that belong to the tile's rows
      const Buffer buf(base, (uint32_t)(len - 1) * stride + (uint32_t)(width * (int)sizeof(T)));
      const uint32_t o = (uint32_t)opaque_int((int)off);
#pragma unroll
      for (int k = 0; k < COUNT; ++k) v[k] = buf.load(o + (uint32_t)(k * STEP) * stride);
    } else {
      const int row0 = tid256() / PER_ROW;
      const T* q0 = reinterpret_cast<const T*>(base) + at + (int64_t)part * run + cc;
#pragma unroll
      for (int k = 0; k < COUNT; ++k) {
        const int row = row0 + k * STEP;
        const T* q = q0 + row * r.token;
        v[k] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (e < n_ && row < len) {
            if constexpr (sizeof(T) == 2) v[k][e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
            else v[k][e] = __builtin_bit_cast(uint32_t, q[e]);
          }
        }
      }
    }
  }
  // The same of rows at `base` (the chunk's first, at the tile's first element)
  // that are `stride` elements apart, n elements each.
  __device__ __forceinline__ void load_at(const T* base, int64_t stride, int len, int n) {
    const int t = opaque_int(tid256());
    const int c = (t % PER_ROW) * V, row0 = t / PER_ROW;
    if constexpr (VEC) {
      const uint32_t bytes = (uint32_t)(stride * (int)sizeof(T));
      const Buffer buf(base, (uint32_t)(len - 1) * bytes + (uint32_t)(n * (int)sizeof(T)));
      const uint32_t o =
          c < n ? (uint32_t)row0 * bytes + (uint32_t)(c * (int)sizeof(T)) : kOutside;
#pragma unroll
      for (int k = 0; k < COUNT; ++k) v[k] = buf.load(o + (uint32_t)(k * STEP) * bytes);
    } else {
#pragma unroll
      for (int k = 0; k < COUNT; ++k) {
        const int row = row0 + k * STEP;
        const T* q = base + row * stride + c;
        v[k] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (c + e < n && row < len) {
            if constexpr (sizeof(T) == 2) v[k][e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
            else v[k][e] = __builtin_bit_cast(uint32_t, q[e]);
          }
        }
      }
    }
  }
  // Whether a value is infinite or NaN.
  __device__ __forceinline__ bool odd() const {
    bool r = false;
#pragma unroll
    for (int k = 0; k < COUNT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r = r || not_finite(__uint_as_float(v[k][i]));     // bfloat16: the upper one
        if constexpr (sizeof(T) == 2) r = r || not_finite(bf16_lo(v[k][i]));
      }
    return r;
  }
  __device__ __forceinline__ void store(T* tile, int stride) const {
    const int t = opaque_int(tid256());
    T* q = tile + (t / PER_ROW) * stride + (t % PER_ROW) * V;
#pragma unroll
    for (int k = 0; k < COUNT; ++k) {
      if constexpr (sizeof(T) == 2) {   // rows may start on 8 bytes
        u32x2* o = reinterpret_cast<u32x2*>(q + k * STEP * stride);
        o[0] = u32x2{v[k][0], v[k][1]};
        o[1] = u32x2{v[k][2], v[k][3]};
      } else {
        *reinterpret_cast<u32x4*>(q + k * STEP * stride) = v[k];
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Weights of what crosses a chunk.  One that a flag makes nothing is kBlocked:
// nothing passes, whatever it would weigh.  A decay that underflows is 0 and still
// multiplies, so that an infinity or NaN before it stays, as it does step by step.
// ---------------------------------------------------------------------------
constexpr float kBlocked = -0.0f;
__device__ __forceinline__ bool blocked(float f) { return __float_as_uint(f) == 0x80000000u; }
__device__ __forceinline__ float weigh(float x, float f) { return blocked(f) ? 0.0f : x * f; }
// The weight of passing two.
__device__ __forceinline__ float join(float a, float b) {
  return blocked(a) || blocked(b) ? kBlocked : a * b;
}

// ---------------------------------------------------------------------------
// The scalars of a head's chunk.  They are prepared once for all passes, one
// token a lane: in the passes themselves the softplus, the exponentials and the
// sum over the chunk kept three waves waiting for one.
// ---------------------------------------------------------------------------
template <int Q>
struct alignas(16) Scal {
  float S[Q];    // sum of the log2 decays from the chunk's start, or from the last flag
  float w[Q];    // weight of the token's input
  float c[Q];    // its weight in the state at the chunk's end (blocked if a flag follows)
  float e[Q];    // weight of the entering state in the token's row (blocked after a flag)
  float g[Q];    // forward: w times the decay to the end of the token's tile of 16;
                 // backward: what S lost when it was rounded
  float r[Q];    // forward: what S lost; backward: decay to the chunk's end (blocked if
                 // a flag follows)
  int id[Q];     // flags up to the token
  float dec;     // weight of the entering state in the state at the chunk's end
  int flags;     // flags in the chunk
  float pad[2];
};

// The heads' scalars of one chunk, on their way from global memory to LDS.
template <int Q, int HEADS = 4>
struct ScalStage {
  static constexpr int PIECES = sizeof(Scal<Q>) / 16;
  static constexpr int COUNT = (HEADS * PIECES + 255) / 256;   // two at most
  u32x4 v[COUNT];
  __device__ __forceinline__ void load(const void* scal, int64_t at, int heads) {
    const Buffer buf(static_cast<const Scal<Q>*>(scal) + at, (uint32_t)(heads * PIECES * 16));
    const uint32_t o = 16u * (uint32_t)opaque_int((int)tid256());
    v[0] = buf.load(o);
    if constexpr (COUNT == 2) {
      v[1] = u32x4{0, 0, 0, 0};
      if (heads * PIECES > 256) v[1] = buf.load(o + 256 * 16);
    }
  }
  // Whether a scalar is infinite or NaN (the numbers of flags never look so).
  __device__ __forceinline__ bool odd() const {
    bool r = false;
#pragma unroll
    for (int k = 0; k < COUNT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) r = r || not_finite(__uint_as_float(v[k][i]));
    return r;
  }
  __device__ __forceinline__ void store(Scal<Q>* lds, int heads) const {
    u32x4* q = reinterpret_cast<u32x4*>(lds);
    const int n = heads * PIECES;
    const int i = tid256();
    if (i < n) q[i] = v[0];
    if constexpr (COUNT == 2)
      if (i + 256 < n) q[i + 256] = v[1];
  }
};

// ---------------------------------------------------------------------------
// Infinities and NaN.  A matrix product spreads one over its whole row and
// column even where the other factor's weight is zero.  Where a wave's columns
// of a chunk hold one, they are taken out (zeros in their place) and kept as
// marks by column; what they reach is then set to NaN: the rows of the same
// sequence from the mark on, and the state if the sequence goes on.  In a chunk
// with flags the rows of B that a flag keeps from the state are cleared when
// they hold one.  All other rows keep the bits they have without it.
// ---------------------------------------------------------------------------
// The marks of column c of a tile (bit q: row q), its values taken out.
template <typename T, int Q>
__device__ __forceinline__ uint64_t take_out(T* tile, int stride, int c) {
  uint64_t m = 0;
#pragma unroll 1
  for (int q = 0; q < Q; ++q)
    if (not_finite(Elem<T>::load1(tile + q * stride + c))) {
      m |= 1ull << q;
      tile[q * stride + c] = T(0);
    }
  return m;
}

// Whether a mark reaches token q: one of its sequence up to it.
template <int Q>
__device__ __forceinline__ bool marked_upto(uint64_t marks, const int* id, int q) {
#pragma unroll 1
  for (int s = 0; s <= q; ++s)
    if ((marks >> s & 1) != 0 && id[s] == id[q]) return true;
  return false;
}

// Whether a mark is in sequence number n.
template <int Q>
__device__ __forceinline__ bool marked(uint64_t marks, const int* id, int n) {
#pragma unroll 1
  for (int s = 0; s < Q; ++s)
    if ((marks >> s & 1) != 0 && id[s] == n) return true;
  return false;
}

// Whether the wave's 32 columns from c0 of a tile hold an infinity or a NaN:
// zero times anything else is zero.
template <typename T, int Q>
__device__ __forceinline__ bool tile_odd(const T* tile, int stride, int c0) {
  const bf16x8 zero = as_frag(u32x4{0, 0, 0, 0});
  f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int ks = 0; ks < Q / 32; ++ks)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) {
      Cols<T> x;
      x.load(tile, stride, c0 + 16 * pt, 32 * ks);
      r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(zero, x.top(), r, 0, 0, 0);
    }
  return __any(r[0] != 0.0f);
}

// Clears the non-finite values of the rows of other sequences than number
// `stays`.  Called by the whole block.
template <typename T, int Q, int NP>
__device__ __forceinline__ void clear_kept(T* tile, int stride, const int* id, int stays) {
#pragma unroll 1
  for (int i = threadIdx.x; i < Q * NP; i += 256) {
    T* x = tile + (i / NP) * stride + i % NP;
    if (id[i / NP] != stays && not_finite(Elem<T>::load1(x))) *x = T(0);
  }
}

// ---------------------------------------------------------------------------
// The state of a slice, rows n, columns p: tile (nt, pt) holds states
// 16 nt + 4 g + (0..3) of column 16 pt + i.
// ---------------------------------------------------------------------------
// Between kernels a slice's state is 32 NK kSlice floats in this order.
template <int NK>
__device__ __forceinline__ int frag_at(int nt, int pt, int lane = (int)(threadIdx.x & 63)) {
  return lane * 4 + (nt * 2 + pt) * 256;
}
template <int NK>
constexpr int64_t slice_floats() { return 32 * NK * kSlice; }

template <int NK>
__device__ __forceinline__ void load_frags(const float* st, f32x4 (&h)[2 * NK][2]) {
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) h[nt][pt] = *reinterpret_cast<const f32x4*>(st + frag_at<NK>(nt, pt));
}

template <int NK>
__device__ __forceinline__ void store_frags(float* st, const f32x4 (&h)[2 * NK][2]) {
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) *reinterpret_cast<f32x4*>(st + frag_at<NK>(nt, pt)) = h[nt][pt];
}

template <int NK>
__device__ __forceinline__ void fill(f32x4 (&h)[2 * NK][2], float v) {
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) h[nt][pt] = f32x4{v, v, v, v};
}

// From or to one head's (headdim, dstate) state; c0: the slice's first channel.
template <int NK>
__device__ __forceinline__ void load_state(const float* st, int c0, int P, int N,
                                           f32x4 (&h)[2 * NK][2]) {
#pragma unroll
  for (int pt = 0; pt < 2; ++pt) {
    const int pp = c0 + 16 * pt + lane_i();
#pragma unroll
    for (int nt = 0; nt < 2 * NK; ++nt) {
      const int n = 16 * nt + 4 * lane_g();
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[nt][pt][j] = st && pp < P && n + j < N ? st[(int64_t)pp * N + n + j] : 0.0f;
    }
  }
}

template <int NK>
__device__ __forceinline__ void store_state(float* st, int c0, int P, int N,
                                            const f32x4 (&h)[2 * NK][2]) {
  const bool whole = N % 4 == 0 && (reinterpret_cast<uintptr_t>(st) & 15) == 0;
#pragma unroll
  for (int pt = 0; pt < 2; ++pt) {
    const int pp = c0 + 16 * pt + lane_i();
    if (pp >= P) continue;
#pragma unroll
    for (int nt = 0; nt < 2 * NK; ++nt) {
      const int n = 16 * nt + 4 * lane_g();
      if (whole) {
        if (n < N) *reinterpret_cast<f32x4*>(st + (int64_t)pp * N + n) = h[nt][pt];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) st[(int64_t)pp * N + n + j] = h[nt][pt][j];
      }
    }
  }
}

// h <- dec h.  dec is the wave's.
template <int NK>
__device__ __forceinline__ void decay_state(f32x4 (&h)[2 * NK][2], float dec) {
  if (blocked(dec)) {
    fill<NK>(h, 0.0f);
  } else {
#pragma unroll
    for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) h[nt][pt] *= dec;
  }
}

// h += sum_t c_t keys_t x_t^T over 32 tokens, x given as fragments.
template <typename T, int NK, int NX>
__device__ __forceinline__ void add_outer(f32x4 (&h)[2 * NK][2], const T* keys, int kstride, int k0,
                                          const Frag<NX> (&x)[2]) {
  Frag<Mx<T>::PARTS> b[2][2];
  b[0][0] = load_cols<T>(keys, kstride, 0, k0);
  b[0][1] = load_cols<T>(keys, kstride, 16, k0);
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    if (i + 1 < NK) {
      b[(i + 1) & 1][0] = load_cols<T>(keys, kstride, 32 * i + 32, k0);
      b[(i + 1) & 1][1] = load_cols<T>(keys, kstride, 32 * i + 48, k0);
    }
    phase();
    f32x4 (&pair)[2][2] = *reinterpret_cast<f32x4(*)[2][2]>(&h[2 * i]);
    mma(pair, b[i & 1], x);
  }
}

// A chunk's step of a slice's state: h <- dec h + sum_t c_t keys_t vals_t^T.
template <typename T, int NK>
__device__ __forceinline__ void step_state(f32x4 (&h)[2 * NK][2], float dec, const float* c,
                                           const T* keys, int kstride, const T* vals, int vstride,
                                           int col) {
  constexpr int Q = Mx<T>::Q;
  decay_state<NK>(h, dec);
#pragma unroll
  for (int ks = 0; ks < Q / 32; ++ks) {
    Frag<3> x[2];
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) {
      Cols<T> v;
      v.load(vals, vstride, col + 16 * pt, 32 * ks);
      x[pt] = v.weighted(c, 32 * ks);
    }
    add_outer<T, NK>(h, keys, kstride, 32 * ks, x);
  }
}

// A lane's column of tile column pt becomes NaN.
template <int NK>
__device__ __forceinline__ void spoil(f32x4 (&h)[2 * NK][2], int pt) {
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) (pt == 0 ? h[nt][0] : h[nt][1])[j] = __builtin_nanf("");
}

// Which heads and columns a block and its waves take.
struct Place {
  int64_t b;
  int seg, g, h0;      // first head of the block
  int heads;           // heads of the block
  int h, slice;        // the wave's
  bool on;             // whether the wave has columns
  int c0, ncol;        // its first channel in the head, channels left there
  int col;             // its first column in the block's tile
};

// Blocks in order: batch row, segment, group, head block; contiguous ranges
// share an XCD, whose L2 then serves B and C to all heads of a row.
__device__ __forceinline__ Place place_at(const HeadsParams& p, int nseg, int block) {
  int id = xcd_remap(block, (int)(p.batch * nseg * p.G * p.hblocks));
  Place k;
  const int per = p.H / p.G, hb = id % p.hblocks;
  id /= p.hblocks;
  k.g = id % p.G;
  id /= p.G;
  k.seg = id % nseg;
  k.b = id / nseg;
  const int first = hb * p.hpw, left = per - first;
  k.heads = left < p.hpw ? left : p.hpw;
  k.h0 = k.g * per + first;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hh = wave / p.slices;
  k.slice = wave - hh * p.slices;
  k.on = hh < k.heads;
  k.h = k.h0 + (k.on ? hh : 0);
  k.c0 = k.slice * kSlice;
  k.ncol = p.P - k.c0;
  k.col = wave * kSlice;
  return k;
}

__device__ __forceinline__ Place place_of(const HeadsParams& p, int nseg) {
  return place_at(p, nseg, (int)blockIdx.x);
}

__device__ __forceinline__ int64_t slice_slot(const HeadsParams& p, const Place& k, int n, int i) {
  return ((k.b * p.H + k.h) * p.slices + k.slice) * n + i;
}

}  // namespace mscan
