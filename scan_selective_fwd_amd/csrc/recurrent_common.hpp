// Device helpers of the gated linear recurrence.
#pragma once

#include "heads_common.hpp"
#include "recurrent.hpp"

// Products and sums are fused only where written so: a row gives the same bits in every
// variant of a kernel, whatever its alignment.
#pragma clang fp contract(off)

namespace mscan {

// 1 - exp2(z) for z in [-kSmallZ, 0]: -z times a polynomial of degree 4 in z, the
// least largest relative error over the interval (8e-8; coefficients of
// (e^w - 1) / w on [-1/2, 0], scaled by powers of ln 2).
constexpr float kSmallZ = 0.72134752f;   // 0.5 / ln 2
constexpr float kOneMinus0 = 0.6931471229f;
constexpr float kOneMinus1 = 0.2402229011f;
constexpr float kOneMinus2 = 0.0554646403f;
constexpr float kOneMinus3 = 0.0094645340f;
constexpr float kOneMinus4 = 0.0010833843f;

// The gates of one step and what they make of it.
struct RecGate {
  float sr, si;   // sigmoids of r and i
  float lg;       // log2 of the decay
  float a;        // the decay
  float m2;       // 1 - a^2
};

// Within one unit in the last place, as the exponentials here are.
__device__ __forceinline__ float rec_sqrt(float x) { return __builtin_amdgcn_sqrtf(x); }

// A2 = A log2(e).  1 - a^2 is formed without cancellation: from the polynomial where
// a^2 is above e^(-1/2), from a itself below, where it keeps at least 0.39.
__device__ __forceinline__ RecGate rec_gate(float r, float i, float A2) {
  RecGate g;
  g.sr = sigmoid(r);
  g.si = sigmoid(i);
  g.lg = A2 * g.sr;
  g.a = fast_exp2(g.lg);
  const float z = g.lg + g.lg;
  float q = __builtin_fmaf(z, kOneMinus4, kOneMinus3);
  q = __builtin_fmaf(z, q, kOneMinus2);
  q = __builtin_fmaf(z, q, kOneMinus1);
  q = __builtin_fmaf(z, q, kOneMinus0);
  const float far = __builtin_fmaf(-g.a, g.a, 1.0f);
  g.m2 = z < -kSmallZ ? far : -z * q;
  return g;
}

// A value that is the same in every lane, but was formed where lanes have their own
// (quotients are): from here on it is kept, and what is made of it formed, once a wave.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// V channels of one token as they lie in memory: two bfloat16, or one element.
template <typename T, int V>
struct RecRaw {
  static_assert(V == 1 || (V == 2 && sizeof(T) == 2), "V");
  uint32_t w;
  // The row's address is the same in every lane, the lane's place in it 32 bits: then
  // the sum is formed by the load itself.
  __device__ __forceinline__ void load(const char* row, uint32_t at) {
    const char* q = row + at;
    if constexpr (V == 2) w = *reinterpret_cast<const uint32_t*>(q);
    else if constexpr (sizeof(T) == 2) w = *reinterpret_cast<const T*>(q);
    else w = __float_as_uint(*reinterpret_cast<const T*>(q));
  }
  __device__ __forceinline__ void fill(float v) {   // a value that bfloat16 holds
    w = __float_as_uint(v);
    if constexpr (sizeof(T) == 2) w = w >> 16 | w;
  }
  __device__ __forceinline__ float get(int v) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    else return v ? bf16_hi(w) : bf16_lo(w);
  }
};

template <typename T, int V>
__device__ __forceinline__ void rec_store(char* row, uint32_t at, const float (&y)[V]) {
  char* q = row + at;
  if constexpr (V == 2) *reinterpret_cast<uint32_t*>(q) = pack_bf16(y[0], y[1]);
  else if constexpr (sizeof(T) == 2) *reinterpret_cast<T*>(q) = (T)pack_bf16(y[0], y[0]);
  else *reinterpret_cast<T*>(q) = y[0];
}

// The rows of a run of n steps, one after another; behind the last it stays there.
template <typename T>
struct RecWalk {
  const char* p;
  int64_t step;
  __device__ __forceinline__ RecWalk(const Rows& q, int64_t b, int64_t t)
      : p(static_cast<const char*>(q.p) + (b * q.batch + t * q.token) * (int64_t)sizeof(T)),
        step(q.token * (int64_t)sizeof(T)) {}
  __device__ __forceinline__ void next(int s, int n) { p += s + 1 < n ? step : 0; }
};

// The affine map h -> A h + H of a run of steps; `cut`: a flag in it leaves h out
// whatever it holds.
__device__ __forceinline__ float rec_apply(float A, float H, bool cut, float h) {
  const float y = __builtin_fmaf(A, h, H);
  return cut ? H : y;
}

// A run's map in one 64-bit word, whose store makes it valid: the sign of A, which is
// never negative, says that it is there, an A of infinity that it is cut.
constexpr uint32_t kThere = 0x80000000u, kCutBits = 0x7F800000u;

__device__ __forceinline__ uint64_t rec_pack(float A, float H, bool cut) {
  const uint32_t a = cut ? kCutBits : __float_as_uint(A);
  return (uint64_t)(a | kThere) << 32 | __float_as_uint(H);
}

__device__ __forceinline__ void rec_publish(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Waits for the word at p.  Who writes it took an earlier ticket, so it runs already
// and waits only for earlier tickets itself: the wait ends.
__device__ __forceinline__ uint64_t rec_wait(uint64_t* p) {
  uint64_t v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  while (!(v >> 63)) {
    __builtin_amdgcn_s_sleep(1);
    v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  return v;
}

// The value that enters tile q (counted in the order of the tickets) of a row: the
// maps of its group's earlier tiles joined, then the value behind the group before.
// Publishes the tile's own map (At, Ht, cutt), or for the last of a group the value
// behind it.  h: in, what enters tile 0; out, what enters this one.  The order of
// the products does not depend on who was first, so equal inputs give equal bits.
// maps, heads: this tile's and its group's words; `on`: whether the lane's channels exist.
template <int V, int G>
__device__ __forceinline__ void rec_chain(uint64_t* maps, uint64_t* heads, int64_t dim, uint32_t q,
                                          const float (&At)[V], const float (&Ht)[V], bool cutt,
                                          bool on, int wave, int waves, int lane,
                                          uint64_t (*sMap)[64 * V], float* sHead, float (&h)[V]) {
  const int j = q % G;
  const bool later = q >= G;
  if (wave == 0 && on && j != G - 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) rec_publish(maps + v, rec_pack(At[v], Ht[v], cutt));
  }
  for (int k = wave; k < j; k += waves)
#pragma unroll
    for (int v = 0; v < V; ++v) sMap[k][lane * V + v] = rec_wait(maps - (int64_t)(j - k) * dim + v);
  __syncthreads();
  float A[V], H[V];
  bool cut[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    H[v] = 0.0f;
    cut[v] = false;
  }
  for (int k = 0; k < j; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint64_t m = sMap[k][lane * V + v];
      const uint32_t hi = (uint32_t)(m >> 32) & ~kThere;
      const bool c = hi == kCutBits;
      H[v] = rec_apply(__uint_as_float(hi), __uint_as_float((uint32_t)m), c, H[v]);
      cut[v] = cut[v] || c;
      A[v] *= c ? 1.0f : __uint_as_float(hi);
    }
  if (later) {
    // joined before the wait: the next group waits for two products after this one
    if (wave == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = __uint_as_float((uint32_t)rec_wait(heads - dim + v));
        sHead[lane * V + v] = h[v] = rec_apply(A[v], H[v], cut[v], h[v]);
      }
  } else if (j) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = H[v];
  }
  if (j == G - 1 && wave == 0 && on)
#pragma unroll
    for (int v = 0; v < V; ++v)
      rec_publish(heads + v, rec_pack(0.0f, rec_apply(At[v], Ht[v], cutt, h[v]), false));
  if (later) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = sHead[lane * V + v];
  }
}

// The next tile of a strip: the first block to come takes its first, and so on.  Each
// strip counts for itself, on a cache line of its own.
__device__ __forceinline__ uint32_t rec_ticket(uint32_t* tickets, uint32_t strip,
                                               uint32_t* sTicket) {
  if (threadIdx.x == 0)
    *sTicket = __hip_atomic_fetch_add(tickets + (size_t)strip * kTicketWords, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*sTicket);
}

}  // namespace mscan
