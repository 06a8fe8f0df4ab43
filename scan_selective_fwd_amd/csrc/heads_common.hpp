// Device helpers shared by the multi-head operators.
#pragma once

#include "device_common.hpp"
#include "heads.hpp"

namespace mscan {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two floats as a packed bfloat16 pair, round to nearest even (one
// v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Four consecutive elements as they lie in memory (8 or 16 aligned bytes), or,
// with V = 1, one: kept so while loads are in flight, unpacked where used.
template <typename T, int V>
struct Raw {
  static constexpr int WORDS = V * sizeof(T) <= 4 ? 1 : V * sizeof(T) / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const T* q = static_cast<const T*>(p) + at;
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 2) w[0] = *q;
      else w[0] = __float_as_uint(*q);
    } else if constexpr (WORDS == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(q);
      w[0] = x.x; w[1] = x.y;
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(q);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
      v[0] = bf16_lo(w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
};

// V consecutive elements at p: V = 1, or 16 bytes of them at a 16-byte aligned p.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const void* p, int64_t at, float (&v)[V]) {
  const T* q = static_cast<const T*>(p) + at;
  if constexpr (V == 8) {
    Elem<T>::template load_k<V>(q, v);
  } else {
    Raw<T, V> r;
    r.load(q, 0);
    r.get(v);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(void* p, int64_t at, const float (&v)[V]) {
  T* q = static_cast<T*>(p) + at;
  if constexpr (sizeof(T) == 2) {
    if constexpr (V == 1) {
      *q = (bf16_t)pack_bf16(v[0], v[0]);
    } else if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else {
      static_assert(V == 8, "V");
      uint4 x;
      x.x = pack_bf16(v[0], v[1]);
      x.y = pack_bf16(v[2], v[3]);
      x.z = pack_bf16(v[4], v[5]);
      x.w = pack_bf16(v[6], v[7]);
      *reinterpret_cast<uint4*>(q) = x;
    }
  } else {
    if constexpr (V == 1) *q = v[0];
    else Elem<T>::template store_k<V>(q, v);
  }
}

template <int V>
__device__ __forceinline__ void load_f32(const float* p, int64_t at, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = p[at];
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 x = reinterpret_cast<const float4*>(p + at)[i];
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
  }
}

// What one step of one head is made of: the step delta, its derivative to
// the raw step, the log2 of the decay and the input's weight.  These are one
// scalar a (token, head), against P N products, so they take the library's
// accurate functions.
struct Step {
  float dt, draw, lg, w;
};

constexpr float kTinyA = 1e-30f;   // below it the ZOH weight is its limit, delta

// The log2 decay is held at -150: 2^-150 is zero in float32, and sums of them, made
// in 64 bits and kept as two floats, stay finite with bits to spare.
constexpr float kLgMin = -150.0f;

__device__ __forceinline__ float step_weight(float dt, float A, bool zoh) {
  if (!zoh || __builtin_fabsf(A) < kTinyA) return dt;
  return expm1f(dt * A) / A;
}

__device__ __forceinline__ Step make_step(float raw, float A, bool soft, bool zoh) {
  Step s;
  s.dt = raw;
  s.draw = 1.0f;
  if (soft) {
    const float e = expf(-__builtin_fabsf(raw));
    s.dt = __builtin_fmaxf(raw, 0.0f) + log1pf(e);
    s.draw = raw >= 0.0f ? 1.0f / (1.0f + e) : e / (1.0f + e);
  }
  const float lg = s.dt * A * kLog2e;
  s.lg = lg < kLgMin ? kLgMin : lg;     // a NaN stays
  s.w = step_weight(s.dt, A, zoh);
  return s;
}

// dw/d(delta) and dw/dA of the input's weight.
__device__ __forceinline__ void step_weight_grad(float dt, float A, bool zoh, float& by_dt,
                                                 float& by_A) {
  by_dt = 1.0f;
  by_A = 0.0f;
  if (!zoh) return;
  const float x = dt * A;
  if (__builtin_fabsf(x) < 0.05f) {
    // delta^2 (1/2 + x/3 + x^2/8 + x^3/30 + x^4/144 + ...): the first term left out
    // is below 5e-9 of the sum
    by_dt = __builtin_fabsf(A) < kTinyA ? 1.0f : expf(x);
    by_A = dt * dt *
           (0.5f + x * (1.0f / 3.0f + x * (0.125f + x * (1.0f / 30.0f + x * (1.0f / 144.0f)))));
    return;
  }
  const float e = expf(x);
  by_dt = e;
  by_A = (dt * e - expm1f(x) / A) / A;
}

}  // namespace mscan
