// The scalars of every chunk of the multi-head scan (Scal, heads_mma.hpp): one
// wave a (batch row, chunk, head), one token a lane.  Made once here, they cost
// each pass one load instead of a scan and its exponentials a wave.  Bound by its
// writes, 28 bytes a token and head: 8 x 2048 tokens of 24 heads take 6.9 us,
// 131072 of one row 30 us (88 MB, 2.9 TB/s).
#include "heads_mma.hpp"

namespace mscan {

namespace {

template <typename T, bool BWD>
__global__ __launch_bounds__(256) void heads_scal_kernel(const HeadsParams p) {
  constexpr int Q = Mx<T>::Q;
  const int64_t chunks = (p.L + Q - 1) / Q;
  const int l = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= p.batch * chunks * p.H) return;
  const int h = (int)(id % p.H);
  const int64_t bc = id / p.H, b = bc / chunks, t0 = (bc - b * chunks) * Q;
  const int len = p.L - t0 < Q ? (int)(p.L - t0) : Q;
  const int64_t t = t0 + (l < len ? l : len - 1);
  const float raw =
      Elem<T>::load1(static_cast<const T*>(p.delta.p) + b * p.delta.batch + t * p.delta.token + h) +
      (p.bias ? p.bias[h] : 0.0f);
  const int flag = p.reset ? p.reset[b * p.L + t] : 0;
  const Step st = make_step(raw, p.A[h], p.softplus != 0, p.zoh != 0);
  // Sums in 64 bits: of two near each other far below zero the difference is the
  // exponent of a weight near 1, and 32 bits would lose 1e-6 of it.
  double S = l < len ? (double)st.lg : 0.0;
  const float w = l < len ? st.w : 0.0f;
  const uint64_t flags = __ballot(flag != 0 && l < len);
  const uint64_t upto = flags & ((2ull << l) - 1ull);
  const int start = upto ? 63 - __builtin_clzll(upto) : 0;
  const int n = __builtin_popcountll(upto), n_end = __builtin_popcountll(flags);
  // sums restart at a flag: no value of one sequence enters another's
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double x = __shfl_up(S, off);
    if (l - off >= start) S += x;
  }
  const double end = __shfl(S, 63), tile_end = __shfl(S, l | 15);
  const float high = (float)S, to_end = fast_exp2((float)(end - S));
  Scal<Q>* o = static_cast<Scal<Q>*>(p.scal) + id;
  if (l < Q) {
    o->S[l] = high;
    o->w[l] = w;
    // (the sum turns a -0 of a weight below zero into 0: that one underflowed)
    o->c[l] = n == n_end ? to_end * w + 0.0f : kBlocked;
    o->e[l] = n == 0 ? fast_exp2(high) : kBlocked;
    const float low = (float)(S - (double)high);
    o->g[l] = BWD ? low : fast_exp2((float)(tile_end - S)) * w;
    o->r[l] = !BWD ? low : n == n_end ? to_end : kBlocked;
    o->id[l] = n;
  }
  if (l == 0) {
    o->dec = n_end == 0 ? fast_exp2((float)end) : kBlocked;
    o->flags = n_end;
    o->pad[0] = o->pad[1] = 0.0f;
  }
}

}  // namespace

hipError_t dispatch_heads_scal(const HeadsParams& p, int dtype, bool bwd, hipStream_t s) {
  const int q = dtype == 0 ? Mx<float>::Q : Mx<bf16_t>::Q;
  const int64_t waves = p.batch * ((p.L + q - 1) / q) * p.H;
  const dim3 grid((unsigned)((waves + 3) / 4));
  if (dtype == 0) {
    if (bwd) hipLaunchKernelGGL((heads_scal_kernel<float, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((heads_scal_kernel<float, false>), grid, dim3(256), 0, s, p);
  } else {
    if (bwd) hipLaunchKernelGGL((heads_scal_kernel<bf16_t, true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((heads_scal_kernel<bf16_t, false>), grid, dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace mscan
