// Gated linear recurrence, backward: a thread walks one channel of one
// batch row, neighbours on neighbouring channels.
#include "recurrent_common.hpp"

namespace mscan {

namespace {

template <typename T>
__device__ __forceinline__ float at(const Rows& q, int64_t b, int64_t t, int64_t d) {
  return Elem<T>::load1(static_cast<const T*>(q.p) + b * q.batch + t * q.token + d);
}

template <typename T>
__global__ __launch_bounds__(256) void rec_bwd_kernel(const RecParams p) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= p.batch * p.dim) return;
  const int64_t b = n / p.dim, d = n - b * p.dim;
  const int64_t tiles = (p.L + kRecTile - 1) / kRecTile;
  const float A = p.A[d], A2 = A * kLog2e;
  float* st = p.states + b * kRecTile * p.dim + d;
  float after = p.dlast ? p.dlast[n] : 0.0f, sum = 0.0f;
  for (int64_t k = tiles - 1; k >= 0; --k) {
    const int64_t t0 = k * kRecTile, t1 = t0 + kRecTile < p.L ? t0 + kRecTile : p.L;
    float h = p.kept[(b * tiles + k) * p.dim + d];
    for (int64_t t = t0; t < t1; ++t) {
      st[(t - t0) * p.dim] = h;
      const RecGate g = rec_gate(at<T>(p.r, b, t, d), at<T>(p.i, b, t, d), A2);
      const float v = __builtin_sqrtf(g.m2) * g.si * at<T>(p.x, b, t, d);
      h = p.reset && p.reset[b * p.L + t] ? v : __builtin_fmaf(g.a, h, v);
    }
    for (int64_t t = t1 - 1; t >= t0; --t) {
      const int64_t o = (b * p.L + t) * p.dim + d;
      const float x = at<T>(p.x, b, t, d), before = st[(t - t0) * p.dim];
      const RecGate g = rec_gate(at<T>(p.r, b, t, d), at<T>(p.i, b, t, d), A2);
      const bool cut = p.reset && p.reset[b * p.L + t];
      const float m = __builtin_sqrtf(g.m2), ix = g.si * x;
      float dy = Elem<T>::load1(static_cast<const T*>(p.dout) + o);
      if (p.z.p) {
        const float z = at<T>(p.z, b, t, d), sz = sigmoid(z);
        const float hh = cut ? m * ix : __builtin_fmaf(g.a, before, m * ix);
        Elem<T>::store1(static_cast<T*>(p.dz) + o,
                        dy * hh * (sz * __builtin_fmaf(z, 1.0f - sz, 1.0f)));
        dy = dy * (z * sz);
      }
      const float gh = dy + after;
      after = cut ? 0.0f : g.a * gh;
      const float y = g.lg * kLn2;
      const float ym = g.m2 < 1e-37f ? 0.0f : y / m;
      const float kept = cut ? 0.0f : g.a * before * y;
      const float s = gh * __builtin_fmaf(-ix * ym, g.a * g.a, kept);
      const float gm = gh * m * g.si;
      Elem<T>::store1(static_cast<T*>(p.dx) + o, gm);
      Elem<T>::store1(static_cast<T*>(p.di) + o, gm * x * (1.0f - g.si));
      Elem<T>::store1(static_cast<T*>(p.dr) + o, s * (1.0f - g.sr));
      sum += s;
    }
  }
  p.part[n] = sum / A;
  if (p.dh0) p.dh0[n] = after;
}

__global__ __launch_bounds__(256) void rec_sum_kernel(const RecParams p) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (d >= p.dim) return;
  double s = 0.0;
  for (int64_t b = 0; b < p.batch; ++b) s += p.part[b * p.dim + d];
  p.dA[d] = (float)s;
}

unsigned blocks(int64_t n) { return (unsigned)((n + 255) / 256); }

template <typename T>
hipError_t bwd_t(const RecParams& p, hipStream_t s) {
  if (p.ckpt) {   // the states at the tiles' starts
    RecParams f = p;
    f.out = nullptr;
    f.last = nullptr;
    f.z.p = nullptr;
    const hipError_t e = dispatch_rec_fwd(f, sizeof(T) == 4 ? 0 : 1, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((rec_bwd_kernel<T>), dim3(blocks(p.batch * p.dim)), dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rec_sum_kernel, dim3(blocks(p.dim)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t dispatch_rec_bwd(const RecParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? bwd_t<float>(p, s) : bwd_t<bf16_t>(p, s);
}

}  // namespace mscan
