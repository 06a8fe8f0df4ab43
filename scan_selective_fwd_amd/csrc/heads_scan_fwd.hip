// Forward of the multi-head scan over a prompt (the formulas: heads_mma.hpp).
//
// A block of 4 waves walks one head's 64 columns along a segment of the
// sequence, chunk by chunk, the (64, N) state in its registers: what is read is
// u, delta, B, C, what is written is out.  Where the heads alone do not fill
// the chip the sequence is cut into segments: a first pass over the segments
// leaves each one's end state from zero and its decay, a carry joins them, and
// the output pass starts each segment from the state entering it.
#include "heads_mma.hpp"

namespace mscan {

namespace {

struct Block {
  int64_t b;
  int h, pb, seg, g;
};

// Blocks in order: batch row, segment, head, column block; contiguous ranges
// share an XCD, whose L2 then serves B and C to all heads of a row.
__device__ __forceinline__ Block block_of(const HeadsParams& p, int nseg) {
  int id = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  Block k;
  k.pb = id % p.PB;
  id /= p.PB;
  k.h = id % p.H;
  id /= p.H;
  k.seg = id % nseg;
  k.b = id / nseg;
  k.g = k.h / (p.H / p.G);
  return k;
}

__device__ __forceinline__ int64_t slot_of(const HeadsParams& p, int64_t b, int h, int pb, int n,
                                           int k) {
  return ((b * p.H + h) * p.PB + pb) * n + k;
}

template <int NK>
__device__ __forceinline__ void spoil(f32x4 (&h)[2 * NK]) {
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) h[nt][j] = __builtin_nanf("");
}

template <typename T, int NK, bool VEC>
__global__ __launch_bounds__(256, 2) void heads_fwd_kernel(const HeadsFwdParams p) {
  constexpr int Q = Mx<T>::Q, PAD = Mx<T>::PAD, NP = 32 * NK;
  constexpr int SX = kCols + PAD, SN = NP + PAD, SM = Q + PAD, QT = Q / 16;
  constexpr int PARTS = Mx<T>::PARTS;
  __shared__ __align__(16) T Xs[Q * SX];
  __shared__ __align__(16) T Bs[Q * SN];
  __shared__ __align__(16) T Cs[Q * SN];
  __shared__ __align__(16) T Ms[Q * SM];
  __shared__ Scal<Q> scal[2];
  __shared__ uint32_t bad[2];
  __shared__ uint64_t marks[kCols];
  const Block k = block_of(p, p.nseg);
  const int wave = threadIdx.x >> 6;
  const int c0 = k.pb * kCols, ncol = p.P - c0 < kCols ? p.P - c0 : kCols;
  const float A = p.A[k.h], bias = p.bias ? p.bias[k.h] : 0.0f, D = p.D ? p.D[k.h] : 0.0f;
  const int64_t begin = (int64_t)k.seg * p.seg_len;
  const int64_t end = k.seg + 1 == p.nseg ? p.L : begin + p.seg_len;
  const int64_t ucol = (int64_t)k.h * p.P + c0, ncols = (int64_t)k.g * p.N;

  f32x4 h[2 * NK];
  if (k.seg == 0) {
    load_state<NK>(p.h0 ? p.h0 + (k.b * p.H + k.h) * (int64_t)p.P * p.N : nullptr, c0, p.P, p.N, h);
  } else {
    const float* st = p.seg_state + slot_of(p, k.b, k.h, k.pb, p.nseg - 1, k.seg - 1) * (kCols * NP);
#pragma unroll
    for (int nt = 0; nt < 2 * NK; ++nt)
      h[nt] = *reinterpret_cast<const f32x4*>(st + frag_at<NK>(nt));
  }
  // tiles above the diagonal are read as part of a 32-step and stay zero
  for (int i = threadIdx.x; i < Q * SM; i += 256) Ms[i] = T(0);
  if (threadIdx.x < 2) bad[threadIdx.x] = 0;

  Stage<T, Q, kCols> sx;
  Stage<T, Q, NP> sb, sc;
  StepIn in{};
  auto fetch = [&](int64_t t) {
    const int len = end - t < Q ? (int)(end - t) : Q;
    sx.template load<VEC>(p.u, k.b, t, len, ucol, ncol);
    sb.template load<VEC>(p.B, k.b, t, len, ncols, p.N);
    sc.template load<VEC>(p.C, k.b, t, len, ncols, p.N);
    if (wave == 3) in = load_step<T>(p, k.b, k.h, bias, t, len);
  };
  fetch(begin);
  if (wave == 3) chunk_scalars<Q>(p, in, A, end - begin < Q ? (int)(end - begin) : Q, &scal[0]);
  int buf = 0;
  __syncthreads();
  for (int64_t t = begin; t < end;) {
    const int len = end - t < Q ? (int)(end - t) : Q;
    sx.store(Xs, SX);
    sb.store(Bs, SN);
    sc.store(Cs, SN);
    if (sx.non_finite() | sb.non_finite()) bad[buf] = 1;
    __syncthreads();
    const int64_t next = t + Q;
    if (next < end) fetch(next);
    const Scal<Q>& sc_ = scal[buf];

    // M^T tiles (rows s, columns q) on and below the diagonal, stored as M rows
    {
      constexpr int TILES = QT * (QT + 1) / 2;
      // wave 3 also prepares the next chunk's scalars
      const int t0 = wave * (TILES / 3), t1 = wave == 3 ? TILES : t0 + TILES / 3;
      for (int i = t0; i < t1; ++i) {
        int qt = 0, st = i;
        while (st > qt) st -= ++qt;
        f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < NK; ++kk)
          mma(a, load_rows<T>(Bs, SN, 16 * st, 32 * kk), load_rows<T>(Cs, SN, 16 * qt, 32 * kk));
        const int q = 16 * qt + lane_i(), s = 16 * st + 4 * lane_g();
        const float Sq = sc_.S[q];
        const int idq = sc_.id[q];
        float m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool on = s + j <= q && sc_.id[s + j] == idq;
          m[j] = on ? a[j] * (fast_exp2(Sq - sc_.S[s + j]) * sc_.w[s + j]) : 0.0f;
        }
        if constexpr (sizeof(T) == 2) {
          // rounded to bfloat16, as out is
          *reinterpret_cast<u32x2*>(Ms + q * SM + s) =
              u32x2{pack_bf16(m[0], m[1]), pack_bf16(m[2], m[3])};
        } else {
          *reinterpret_cast<f32x4*>(Ms + q * SM + s) = f32x4{m[0], m[1], m[2], m[3]};
        }
      }
    }
    // out^T (rows p, columns q): the entering state's share.  The state is
    // rounded to bfloat16 for it where out is.
    f32x4 y[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) y[qt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      const Frag<PARTS> hf = acc_frag<PARTS>(h[2 * kk], h[2 * kk + 1]);
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) mma(y[qt], hf, load_rows<T>(Cs, SN, 16 * qt, 32 * kk));
    }
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
      const float e = sc_.e[16 * qt + lane_i()];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[qt][j] = weigh(y[qt][j], e);
    }
    if (wave == 3 && next < end)
      chunk_scalars<Q>(p, in, A, end - next < Q ? (int)(end - next) : Q, &scal[buf ^ 1]);
    if (threadIdx.x == 0) bad[buf ^ 1] = 0;
    __syncthreads();
    const bool odd = bad[buf] != 0;
    if (odd) take_out<T, Q, NP>(Xs, SX, Bs, SN, sc_, marks);
    // ... and the chunk's own inputs'
#pragma unroll
    for (int ks = 0; ks < Q / 32; ++ks) {
      const Frag<PARTS> x = load_cols<T>(Xs, SX, 16 * wave, 32 * ks);
#pragma unroll
      for (int qt = 2 * ks; qt < QT; ++qt) mma(y[qt], x, load_rows<T>(Ms, SM, 16 * qt, 32 * ks));
    }
    update_state<T, NK>(h, sc_.dec, Bs, SN, Xs, SX, sc_.c);
    // four columns of a token a lane
    const int col = 16 * wave + 4 * lane_g();
    if (odd) {
      if (marked(marks[16 * wave + lane_i()], sc_, Q - 1)) spoil<NK>(h);
      for (int qt = 0; qt < QT; ++qt)
        for (int j = 0; j < 4; ++j)
          if (marked(marks[col + j], sc_, 16 * qt + lane_i()))
#pragma unroll
            for (int a = 0; a < QT; ++a)
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if (a == qt && b == j) y[a][b] = __builtin_nanf("");
    }
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
      const int q = 16 * qt + lane_i();
      if (q < len && col < ncol) {
        const T* ur = Xs + q * SX + col;
        T* o = static_cast<T*>(p.out) + ((k.b * p.L + t + q) * p.H + k.h) * (int64_t)p.P + c0 + col;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(D, Elem<T>::load1(ur + j), y[qt][j]);
        if constexpr (VEC) {
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
          else
            *reinterpret_cast<f32x4*>(o) = f32x4{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j < ncol) Elem<T>::store1(o + j, v[j]);
        }
      }
    }
    t = next;
    buf ^= 1;
    __syncthreads();
  }
  if (p.last && k.seg + 1 == p.nseg)
    store_state<NK>(p.last + (k.b * p.H + k.h) * (int64_t)p.P * p.N, c0, p.P, p.N, h);
}

// A segment's end state from zero and its decay.
template <typename T, int NK, bool VEC>
__global__ __launch_bounds__(256, 2) void heads_seg_kernel(const HeadsFwdParams p) {
  constexpr int Q = Mx<T>::Q, PAD = Mx<T>::PAD, NP = 32 * NK;
  constexpr int SX = kCols + PAD, SN = NP + PAD;
  __shared__ __align__(16) T Xs[Q * SX];
  __shared__ __align__(16) T Bs[Q * SN];
  __shared__ Scal<Q> scal[2];
  __shared__ uint32_t bad[2];
  __shared__ uint64_t marks[kCols];
  const Block k = block_of(p, p.nseg - 1);
  const int wave = threadIdx.x >> 6;
  const int c0 = k.pb * kCols, ncol = p.P - c0 < kCols ? p.P - c0 : kCols;
  const float A = p.A[k.h], bias = p.bias ? p.bias[k.h] : 0.0f;
  const int64_t begin = (int64_t)k.seg * p.seg_len, end = begin + p.seg_len;
  const int64_t ucol = (int64_t)k.h * p.P + c0, ncols = (int64_t)k.g * p.N;
  f32x4 h[2 * NK];
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt) h[nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float dec = 1.0f;
  Stage<T, Q, kCols> sx;
  Stage<T, Q, NP> sb;
  StepIn in{};
  if (threadIdx.x < 2) bad[threadIdx.x] = 0;
  auto fetch = [&](int64_t t) {
    const int len = end - t < Q ? (int)(end - t) : Q;
    sx.template load<VEC>(p.u, k.b, t, len, ucol, ncol);
    sb.template load<VEC>(p.B, k.b, t, len, ncols, p.N);
    if (wave == 3) in = load_step<T>(p, k.b, k.h, bias, t, len);
  };
  fetch(begin);
  if (wave == 3) chunk_scalars<Q>(p, in, A, end - begin < Q ? (int)(end - begin) : Q, &scal[0]);
  int buf = 0;
  __syncthreads();
  for (int64_t t = begin; t < end;) {
    sx.store(Xs, SX);
    sb.store(Bs, SN);
    if (sx.non_finite() | sb.non_finite()) bad[buf] = 1;
    __syncthreads();
    const int64_t next = t + Q;
    if (next < end) fetch(next);
    if (threadIdx.x == 0) bad[buf ^ 1] = 0;
    const bool odd = bad[buf] != 0;
    if (odd) take_out<T, Q, NP>(Xs, SX, Bs, SN, scal[buf], marks);
    update_state<T, NK>(h, scal[buf].dec, Bs, SN, Xs, SX, scal[buf].c);
    if (odd && marked(marks[16 * wave + lane_i()], scal[buf], Q - 1)) spoil<NK>(h);
    dec = weigh(dec, scal[buf].dec);
    if (wave == 3 && next < end)
      chunk_scalars<Q>(p, in, A, end - next < Q ? (int)(end - next) : Q, &scal[buf ^ 1]);
    t = next;
    buf ^= 1;
    __syncthreads();
  }
  const int64_t slot = slot_of(p, k.b, k.h, k.pb, p.nseg - 1, k.seg);
  float* st = p.seg_state + slot * (kCols * NP);
#pragma unroll
  for (int nt = 0; nt < 2 * NK; ++nt) *reinterpret_cast<f32x4*>(st + frag_at<NK>(nt)) = h[nt];
  if (threadIdx.x == 0) p.seg_dec[slot] = dec;
}

// The state entering each segment, in place of the one before's end state.
template <int NK>
__global__ __launch_bounds__(256) void heads_carry_kernel(const HeadsFwdParams p) {
  constexpr int NP = 32 * NK, PER = kCols * NP / 4 / 256;   // blocks a column block
  const int64_t id = blockIdx.x / PER;
  const int e = (int)(blockIdx.x - id * PER) * 256 + threadIdx.x;   // float4 of the state
  const int pb = (int)(id % p.PB);
  const int64_t bh = id / p.PB;
  const int nt = (e >> 6) % (2 * NK), w = (e >> 6) / (2 * NK), l = e & 63;
  const int pp = pb * kCols + 16 * w + (l & 15), n = 16 * nt + 4 * (l >> 4);
  f32x4 h = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.h0 && pp < p.P)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < p.N) h[j] = p.h0[(bh * p.P + pp) * p.N + n + j];
  const int segs = p.nseg - 1;
  f32x4* st = reinterpret_cast<f32x4*>(p.seg_state + id * segs * (int64_t)(kCols * NP)) + e;
  constexpr int64_t STEP = kCols * NP / 4;
#pragma unroll 4
  for (int k = 0; k < segs; ++k) {
    const f32x4 s = st[k * STEP];
    const float d = p.seg_dec[id * segs + k];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = weigh(h[j], d) + s[j];
    st[k * STEP] = h;
  }
}

template <typename T, int NK, bool VEC>
hipError_t fwd_go(const HeadsFwdParams& p, hipStream_t s) {
  const int64_t cols = p.batch * p.H * p.PB;
  if (p.nseg > 1) {
    hipLaunchKernelGGL((heads_seg_kernel<T, NK, VEC>), dim3((unsigned)(cols * (p.nseg - 1))), dim3(256),
                       0, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((heads_carry_kernel<NK>), dim3((unsigned)(cols * (kCols * 32 * NK / 1024))),
                       dim3(256), 0, s, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((heads_fwd_kernel<T, NK, VEC>), dim3((unsigned)(cols * p.nseg)), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, int NK>
hipError_t fwd_nk(const HeadsFwdParams& p, hipStream_t s) {
  return p.vec ? fwd_go<T, NK, true>(p, s) : fwd_go<T, NK, false>(p, s);
}

template <typename T>
hipError_t fwd_t(const HeadsFwdParams& p, hipStream_t s) {
  if (p.N <= 32) return fwd_nk<T, 1>(p, s);
  if (p.N <= 64) return fwd_nk<T, 2>(p, s);
  if (p.N <= 128) return fwd_nk<T, 4>(p, s);
  return fwd_nk<T, 8>(p, s);
}

}  // namespace

hipError_t dispatch_heads_fwd(const HeadsFwdParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? fwd_t<float>(p, s) : fwd_t<bf16_t>(p, s);
}

}  // namespace mscan
