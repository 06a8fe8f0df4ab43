// One step of the gated linear recurrence for a batch of sequences, in place on a
// pool of states:  h <- a h + sqrt(1 - a^2) s(i) x,  out = h (or h silu(z)).
// A thread takes one channel of one row.
#include "recurrent_common.hpp"

namespace mscan {

namespace {

template <typename T>
__global__ __launch_bounds__(256) void rec_step_kernel(const RecStepParams p) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= p.batch * p.dim) return;
  const int64_t b = n / p.dim, d = n - b * p.dim;
  const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
  T* out = static_cast<T*>(p.out) + n;
  if (slot < 0 || slot >= p.pool) {
    *out = T(0);
    return;
  }
  auto in = [&](const void* q, int64_t row) {
    return Elem<T>::load1(static_cast<const T*>(q) + b * row + d);
  };
  float* st = p.state + slot * p.dim + d;
  const RecGate g = rec_gate(in(p.r, p.r_row), in(p.i, p.i_row), p.A[d] * kLog2e);
  const float h = __builtin_fmaf(g.a, *st, __builtin_sqrtf(g.m2) * g.si * in(p.x, p.x_row));
  *st = h;
  Elem<T>::store1(out, p.z ? h * silu(in(p.z, p.z_row)) : h);
}

}  // namespace

hipError_t dispatch_rec_step(const RecStepParams& p, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)((p.batch * p.dim + 255) / 256));
  if (dtype == 0)
    hipLaunchKernelGGL((rec_step_kernel<float>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((rec_step_kernel<bf16_t>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace mscan
