// Root-mean-square norm with the residual's addition: a block takes a row.
#include "recurrent_common.hpp"

namespace mscan {

namespace {

constexpr int kParts = 512;

// Sum (or largest value) over the block's 256 threads, in every thread.
template <bool MAX>
__device__ __forceinline__ float block_join(float a, float* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float o = __shfl_xor(a, off);
    a = MAX ? __builtin_fmaxf(a, o) : a + o;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = a;
  __syncthreads();
  return MAX ? __builtin_fmaxf(__builtin_fmaxf(sh[0], sh[1]), __builtin_fmaxf(sh[2], sh[3]))
             : (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

template <typename T>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32((bf16_t)pack_bf16(v, v));
  else return v;
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false);
}

// 1 / sqrt(mean of squares + eps) from their sum.  Where that passes float32's range (or
// vanishes beside an eps that does), `again` forms it from values times a scale.
template <typename F>
__device__ __forceinline__ float root_of(float s2, const ResNormParams& p, F again) {
  const float n = (float)p.dim;
  if (__builtin_expect(s2 < 3e38f && (s2 > 0x1p-80f || p.eps > 0x1p-90f), 1))
    return 1.0f / __builtin_sqrtf(s2 / n + p.eps);
  const float sc = s2 < 1.0f ? 0x1p70f : 0x1p-70f;
  return sc / __builtin_sqrtf(again(sc) / n + p.eps * sc * sc);
}

template <typename T, typename R, bool FP8>
__global__ __launch_bounds__(256) void res_norm_fwd_kernel(const ResNormParams p) {
  __shared__ float sh[4];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.x_row;
    const R* res = p.res ? static_cast<const R*>(p.res) + row * p.res_row : nullptr;
    R* keep = p.res_out ? static_cast<R*>(p.res_out) + row * p.dim : nullptr;
    auto sum = [&](int64_t k) {
      const float v = Elem<T>::load1(x + k);
      return res ? rounded<R>(v + Elem<R>::load1(res + k)) : v;
    };
    float s2 = 0.0f;
    for (int64_t k = threadIdx.x; k < p.dim; k += 256) {
      const float v = sum(k);
      s2 = __builtin_fmaf(v, v, s2);
    }
    s2 = block_join<false>(s2, sh);
    const float r = root_of(s2, p, [&](float sc) {
      float t2 = 0.0f;
      for (int64_t k = threadIdx.x; k < p.dim; k += 256) {
        const float v = sum(k) * sc;
        t2 = __builtin_fmaf(v, v, t2);
      }
      return block_join<false>(t2, sh);
    });
    float inv = 1.0f;
    if constexpr (FP8) {
      float most = 0.0f;
      for (int64_t k = threadIdx.x; k < p.dim; k += 256)
        most = __builtin_fmaxf(most, __builtin_fabsf(sum(k) * r * (p.w ? p.w[k] : 1.0f)));
      most = __builtin_fmaxf(block_join<true>(most, sh), 0x1p-100f);
      inv = 448.0f / most;
      if (threadIdx.x == 0) p.scale[row] = most / 448.0f;
    }
    for (int64_t k = threadIdx.x; k < p.dim; k += 256) {
      const float v = sum(k), y = v * r * (p.w ? p.w[k] : 1.0f);
      if constexpr (FP8) static_cast<uint8_t*>(p.out)[row * p.dim + k] = to_e4m3(y * inv);
      else Elem<T>::store1(static_cast<T*>(p.out) + row * p.dim + k, y);
      if (keep) Elem<R>::store1(keep + k, v);
    }
  }
}

template <typename T, typename R>
__global__ __launch_bounds__(256) void res_norm_bwd_kernel(const ResNormParams p) {
  __shared__ float sh[4];
  float* mine = p.dw ? p.part + blockIdx.x * p.dim : nullptr;
  if (mine)
    for (int64_t k = threadIdx.x; k < p.dim; k += 256) mine[k] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.rows; row += p.parts) {
    const R* res = static_cast<const R*>(p.res) + row * p.res_row;
    const T* dout = static_cast<const T*>(p.dout) + row * p.dim;
    float s2 = 0.0f, sv = 0.0f;
    for (int64_t k = threadIdx.x; k < p.dim; k += 256) {
      const float v = Elem<R>::load1(res + k);
      s2 = __builtin_fmaf(v, v, s2);
      sv = __builtin_fmaf(Elem<T>::load1(dout + k) * (p.w ? p.w[k] : 1.0f), v, sv);
    }
    s2 = block_join<false>(s2, sh);
    sv = block_join<false>(sv, sh);
    const float r = root_of(s2, p, [&](float sc) {
      float t2 = 0.0f;
      for (int64_t k = threadIdx.x; k < p.dim; k += 256) {
        const float v = Elem<R>::load1(res + k) * sc;
        t2 = __builtin_fmaf(v, v, t2);
      }
      return block_join<false>(t2, sh);
    });
    const float kk = r * (r * (sv / (float)p.dim));
    for (int64_t k = threadIdx.x; k < p.dim; k += 256) {
      const float v = Elem<R>::load1(res + k), dy = Elem<T>::load1(dout + k);
      float d = r * __builtin_fmaf(-v, kk, dy * (p.w ? p.w[k] : 1.0f));
      if (p.dres) d += Elem<R>::load1(static_cast<const R*>(p.dres) + row * p.dim + k);
      Elem<T>::store1(static_cast<T*>(p.dx) + row * p.dim + k, d);
      if (p.dresidual) Elem<R>::store1(static_cast<R*>(p.dresidual) + row * p.dim + k, d);
      if (mine) mine[k] = __builtin_fmaf(dy, v * r, mine[k]);
    }
  }
}

__global__ __launch_bounds__(256) void res_norm_sum_kernel(const ResNormParams p) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.dim) return;
  float s = 0.0f;
  for (int64_t i = 0; i < p.parts; ++i) s += p.part[i * p.dim + c];
  p.dw[c] = s;
}

template <typename T, typename R>
hipError_t fwd_go(const ResNormParams& p, bool fp8, hipStream_t s) {
  const dim3 grid((unsigned)(p.rows < 65536 ? p.rows : 65536));
  if (fp8)
    hipLaunchKernelGGL((res_norm_fwd_kernel<T, R, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((res_norm_fwd_kernel<T, R, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename R>
hipError_t bwd_go(const ResNormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((res_norm_bwd_kernel<T, R>), dim3((unsigned)p.parts), dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.dw) return e;
  hipLaunchKernelGGL(res_norm_sum_kernel, dim3((unsigned)((p.dim + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

int64_t res_norm_parts(int64_t rows) { return rows < kParts ? rows : kParts; }

hipError_t dispatch_res_norm_fwd(const ResNormParams& p, ResNormKind kind, bool fp8,
                                 hipStream_t s) {
  switch (kind) {
    case kResF32: return fwd_go<float, float>(p, fp8, s);
    case kResBf16: return fwd_go<bf16_t, bf16_t>(p, fp8, s);
    default: return fwd_go<bf16_t, float>(p, fp8, s);
  }
}

hipError_t dispatch_res_norm_bwd(const ResNormParams& p, ResNormKind kind, hipStream_t s) {
  switch (kind) {
    case kResF32: return bwd_go<float, float>(p, s);
    case kResBf16: return bwd_go<bf16_t, bf16_t>(p, s);
    default: return bwd_go<bf16_t, float>(p, s);
  }
}

}  // namespace mscan
