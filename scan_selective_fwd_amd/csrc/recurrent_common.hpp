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

// A sigmoid s(v) = 1 / (1 + e), e = exp(-v), and its complement 1 - s(v) = e s(v): the
// difference would keep few digits of an open gate's, or none.  A gate so far shut that e is
// infinite and s is 0 gives 0, which stands beside factors that are 0 there.
struct RecSigmoid {
  float s, e;
  __device__ __forceinline__ explicit RecSigmoid(float v) : e(fast_exp(-v)) {
    s = fast_rcp(1.0f + e);
  }
  __device__ __forceinline__ float complement() const { return __builtin_fminf(e, 1e38f) * s; }
};

// The gates of one step and what they make of it.
struct RecGate {
  RecSigmoid r, i;
  float sr, si;   // sigmoids of r and i
  float lg;       // log2 of the decay
  float a;        // the decay
  float m2;       // 1 - a^2
};

// Within one unit in the last place, as the exponentials here are.
__device__ __forceinline__ float rec_sqrt(float x) { return __builtin_amdgcn_sqrtf(x); }

// A in the units of exp2, held in range: a step past the end has a gate of 0 and keeps the
// state whatever A is.  A NaN stays.
__device__ __forceinline__ float rec_log2(float A) {
  const float a = A * kLog2e;
  return a < -3e38f ? -3e38f : a;
}

// A2 = rec_log2(A).  1 - a^2 is formed without cancellation: from the polynomial where
// a^2 is above e^(-1/2), from a itself below, where it keeps at least 0.39.
__device__ __forceinline__ RecGate rec_gate(float r, float i, float A2) {
  RecGate g{RecSigmoid(r), RecSigmoid(i)};
  g.sr = g.r.s;
  g.si = g.i.s;
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

// Outputs pass by the second-level cache (backward of 2 x 2048 x 5120 with its gate 104 ->
// 102 us, forward 57 -> 53).  Inputs do not: that gains 5 % where they come from memory and
// loses up to 27 % where they are in the last-level cache.
template <typename T, int V>
__device__ __forceinline__ void rec_store(char* row, uint32_t at, const float (&y)[V]) {
  char* q = row + at;
  if constexpr (V == 2) __builtin_nontemporal_store(pack_bf16(y[0], y[1]), reinterpret_cast<uint32_t*>(q));
  else if constexpr (sizeof(T) == 2) __builtin_nontemporal_store((T)pack_bf16(y[0], y[0]), reinterpret_cast<T*>(q));
  else __builtin_nontemporal_store((T)y[0], reinterpret_cast<T*>(q));
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

__device__ __forceinline__ uint64_t rec_look(uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Waits for the word at p, v what was seen there.  Who writes it took an earlier ticket of
// the same strip, so it runs already and waits only for earlier tickets of that strip
// itself: the wait ends.  Where the words are lost, which takes another call on the same
// workspace at the same time, it ends after many seconds, with a NaN.
constexpr uint32_t kRecPatience = 1u << 24;
__device__ __forceinline__ uint64_t rec_wait(uint64_t* p, uint64_t v) {
  for (uint32_t n = 0; !(v >> 63); ++n) {
    if (n == kRecPatience) return (uint64_t)(kThere | kCutBits) << 32 | 0x7FC00000u;
    __builtin_amdgcn_s_sleep(1);
    v = rec_look(p);
  }
  return v;
}

// The value that enters tile q (counted in the order of the tickets) of a row: that
// behind the group before, and the maps of its group's earlier tiles.
// Publishes the tile's own map (At, Ht, cutt), or for the last of a group the value
// behind it.  h: in, what enters tile 0; out, what enters this one.  The order of
// the products does not depend on who was first, so equal inputs give equal bits.
// maps, heads: this tile's and its group's words; `on`: whether the lane's channels exist;
// W: the block's waves.
template <int V, int G, int W>
__device__ __forceinline__ void rec_chain(uint64_t* maps, uint64_t* heads, int64_t dim, uint32_t q,
                                          const float (&At)[V], const float (&Ht)[V], bool cutt,
                                          bool on, int wave, int lane, uint64_t (*sMap)[64 * V],
                                          float (&h)[V]) {
  static_assert(G <= 2 * W, "a wave fetches two words at most");
  const int j = q % G;
  const bool later = q >= G;
  if (wave == 0 && on && j != G - 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) rec_publish(maps + v, rec_pack(At[v], Ht[v], cutt));
  }
  // word k < j is the map of the group's tile k, word j the value behind the group before;
  // all are asked for at once
  const int items = later ? j + 1 : j;
  uint64_t m[2][V];
  uint64_t* from[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int k = wave + e * W;
    from[e] = k < j ? maps - (int64_t)(j - k) * dim : heads - dim;
    if (k < items)
#pragma unroll
      for (int v = 0; v < V; ++v) m[e][v] = rec_look(from[e] + v);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int k = wave + e * W;
    if (k < items)
#pragma unroll
      for (int v = 0; v < V; ++v) sMap[k][lane * V + v] = rec_wait(from[e] + v, m[e][v]);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (later) h[v] = __uint_as_float((uint32_t)sMap[j][lane * V + v]);
  for (int k = 0; k < j; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint64_t w = sMap[k][lane * V + v];
      const uint32_t hi = (uint32_t)(w >> 32) & ~kThere;
      h[v] = rec_apply(__uint_as_float(hi), __uint_as_float((uint32_t)w), hi == kCutBits, h[v]);
    }
  if (j == G - 1 && wave == 0 && on)
#pragma unroll
    for (int v = 0; v < V; ++v)
      rec_publish(heads + v, rec_pack(0.0f, rec_apply(At[v], Ht[v], cutt, h[v]), false));
}

// The strip of a block; one past the last for the few blocks that have none.
__device__ __forceinline__ uint32_t rec_strip(uint32_t across, uint32_t by_die) {
  if (!by_die) return uniform(blockIdx.x % across);
  const uint32_t at = uniform(blockIdx.x % (8 * by_die));
  return at % 8 * by_die + at / 8;
}

// The tile of a block, by the tickets of its strip: who comes first takes the first, and
// so on.  Each strip counts for itself, on a cache line of its own (with one counter for
// all a tile took 27 to 40 ns of it).
__device__ __forceinline__ uint32_t rec_ticket(uint32_t* tickets, uint32_t strip,
                                               uint32_t* sTicket) {
  if (threadIdx.x == 0)
    *sTicket = __hip_atomic_fetch_add(tickets + (size_t)strip * kTicketWords, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return uniform(*sTicket);
}

}  // namespace mscan
