// One step of the multi-head scan for a batch of sequences, in place on a
// pool of states:
//   h <- exp(delta A) h + w u B^T,   out = h C + D u     per head, h (P, N).
//
// The states are the traffic: each is read and written once (8 P N bytes a
// head against 6 P N flops), so the kernel is bound by HBM for large batches
// and by one trip to it for small ones.  LPR lanes share a row of N states,
// four states a lane (one 16-byte load and store where N allows), and each
// thread takes four rows, all of whose loads are in flight together.  256 rows
// of 80 heads of 64 x 128 take 271 us (1.34 GB, 5.0 TB/s, a large copy's rate);
// one row of 24 heads 5.6 us, of which the launch and one trip are most.
#include "heads_common.hpp"

namespace mscan {

namespace {

constexpr int kStepRows = 4;   // rows of a head's state per thread

template <typename T, int LPR, bool VEC>
__global__ __launch_bounds__(256) void heads_step_kernel(const HeadsStepParams p) {
  constexpr int PASS = 256 / LPR;                // rows of one pass of the block
  const int lane = threadIdx.x & (LPR - 1), r0 = threadIdx.x / LPR;
  const int tiles = (p.P + PASS * kStepRows - 1) / (PASS * kStepRows);
  const int64_t bh = blockIdx.x / tiles;
  const int p0 = (int)(blockIdx.x - bh * tiles) * PASS * kStepRows + r0;
  const int64_t b = bh / p.H;
  const int h = (int)(bh - b * p.H), g = h / (p.H / p.G);
  const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
  const bool on = slot >= 0 && slot < p.pool;    // the whole block
  T* out = static_cast<T*>(p.out) + bh * p.P;
  if (!on) {
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const int pp = p0 + i * PASS;
      if (pp < p.P && lane == 0) out[pp] = T(0);
    }
    return;
  }
  float* st = p.state + (slot * p.H + h) * (int64_t)p.P * p.N;
  auto col = [&](int j) { return VEC ? lane * 4 + j : lane + j * LPR; };
  float s[kStepRows][4], Bv[4], Cv[4], uv[kStepRows];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int pp = p0 + i * PASS;
    const bool row = pp < p.P;
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
    if constexpr (VEC) {
      if (row && lane * 4 < p.N) load_f32<4>(st, (int64_t)pp * p.N + lane * 4, s[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (row && col(j) < p.N) s[i][j] = st[(int64_t)pp * p.N + col(j)];
    }
    uv[i] = row ? Elem<T>::load1(static_cast<const T*>(p.u.p) + b * p.u.batch +
                                 (int64_t)h * p.P + pp)
                : 0.0f;
  }
  const T* Bp = static_cast<const T*>(p.B.p) + b * p.B.batch + (int64_t)g * p.N;
  const T* Cp = static_cast<const T*>(p.C.p) + b * p.C.batch + (int64_t)g * p.N;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = col(j) < p.N;
    Bv[j] = in ? Elem<T>::load1(Bp + col(j)) : 0.0f;
    Cv[j] = in ? Elem<T>::load1(Cp + col(j)) : 0.0f;
  }
  const float A = p.A[h];
  const float raw = Elem<T>::load1(static_cast<const T*>(p.delta.p) + b * p.delta.batch + h) +
                    (p.bias ? p.bias[h] : 0.0f);
  const Step q = make_step(raw, A, p.softplus != 0, p.zoh != 0);
  const float a = exp2f(q.lg), D = p.D ? p.D[h] : 0.0f;
  float y[kStepRows];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int pp = p0 + i * PASS;
    const float xw = uv[i] * q.w;
    float acc = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[i][j] = __builtin_fmaf(a, s[i][j], xw * Bv[j]);
      acc = __builtin_fmaf(s[i][j], Cv[j], acc);
    }
    y[i] = acc;
    if (pp < p.P) {
      if constexpr (VEC) {
        if (lane * 4 < p.N)
          *reinterpret_cast<float4*>(st + (int64_t)pp * p.N + lane * 4) =
              make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col(j) < p.N) st[(int64_t)pp * p.N + col(j)] = s[i][j];
      }
    }
  }
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) y[i] += __shfl_xor(y[i], off);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const int pp = p0 + i * PASS;
      if (pp < p.P) Elem<T>::store1(out + pp, __builtin_fmaf(D, uv[i], y[i]));
    }
  }
}

template <typename T, int LPR>
hipError_t step_go(const HeadsStepParams& p, bool vec, hipStream_t s) {
  static_assert(step_rows(4 * LPR) == 256 / LPR * kStepRows, "the ABI layer's count of blocks");
  const int64_t rows = step_rows(p.N);
  const int64_t blocks = p.batch * p.H * ((p.P + rows - 1) / rows);
  if (vec)
    hipLaunchKernelGGL((heads_step_kernel<T, LPR, true>), dim3((unsigned)blocks), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((heads_step_kernel<T, LPR, false>), dim3((unsigned)blocks), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t step_t(const HeadsStepParams& p, hipStream_t s) {
  const bool vec = p.N % 4 == 0 && (reinterpret_cast<uintptr_t>(p.state) & 15) == 0;
  if (p.N <= 16) return step_go<T, 4>(p, vec, s);
  if (p.N <= 32) return step_go<T, 8>(p, vec, s);
  if (p.N <= 64) return step_go<T, 16>(p, vec, s);
  if (p.N <= 128) return step_go<T, 32>(p, vec, s);
  return step_go<T, 64>(p, vec, s);
}

}  // namespace

hipError_t dispatch_heads_step(const HeadsStepParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? step_t<float>(p, s) : step_t<bf16_t>(p, s);
}

}  // namespace mscan
