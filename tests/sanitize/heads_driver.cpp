// Drives the C ABI layer of the multi-head operators on the host, the
// dispatchers replaced by stand-ins that check what they are given.
#include <stdio.h>
#include <stdlib.h>

#include "heads.hpp"
#include "mamba_scan.h"

static long launched = 0;

#define REQUIRE(c)                                          \
  do {                                                      \
    if (!(c)) {                                             \
      printf("line %d: %s\n", __LINE__, #c);                \
      exit(1);                                              \
    }                                                       \
  } while (0)

namespace mscan {

static void common(const HeadsParams& p) {
  ++launched;
  REQUIRE(p.slices * 32 >= p.P && (p.slices - 1) * 32 < p.P);
  REQUIRE(p.hpw >= 1 && p.hpw * p.slices <= 4 && (long)p.hblocks * p.hpw >= p.H / p.G);
  REQUIRE(p.nseg >= 1 && p.seg_len * p.nseg >= p.L && p.seg_len * (p.nseg - 1) < p.L);
}
hipError_t dispatch_heads_fwd(const HeadsFwdParams& p, int, hipStream_t) {
  common(p);
  return hipSuccess;
}
hipError_t dispatch_heads_bwd(const HeadsBwdParams& p, int, hipStream_t) {
  common(p);
  REQUIRE(p.splits >= 1);
  return hipSuccess;
}
hipError_t dispatch_heads_step(const HeadsStepParams&, int, hipStream_t) {
  ++launched;
  return hipSuccess;
}
hipError_t dispatch_tokconv_fwd(const TokConvParams&, int, hipStream_t) { ++launched; return hipSuccess; }
hipError_t dispatch_tokconv_bwd(const TokConvParams& p, int, hipStream_t) {
  ++launched;
  REQUIRE(p.tiles >= 1);
  return hipSuccess;
}
hipError_t dispatch_tokconv_step(const TokConvStepParams&, int, hipStream_t) { ++launched; return hipSuccess; }
int64_t norm_parts(int64_t rows, int64_t groups) {
  const int64_t n = 1024 / groups < 1 ? 1 : 1024 / groups;
  return n < rows ? n : rows;
}
hipError_t dispatch_norm_fwd(const NormParams&, int, hipStream_t) { ++launched; return hipSuccess; }
hipError_t dispatch_norm_bwd(const NormParams& p, int, hipStream_t) {
  ++launched;
  REQUIRE(p.parts >= 1);
  return hipSuccess;
}

}  // namespace mscan

int main() {
  const int64_t sizes[] = {-1, 0, 1, 2, 3, 17, 64, 100, 128, 129, 256, 257, 4096, (int64_t)1 << 24,
                           (int64_t)1 << 31, (int64_t)1 << 40, (int64_t)1 << 61, INT64_MAX};
  char* const buf = reinterpret_cast<char*>((uintptr_t)1 << 20);   // never followed
  float* const f = reinterpret_cast<float*>(buf);
  long tried = 0;
  for (int64_t batch : sizes)
    for (int64_t L : sizes)
      for (int64_t heads : sizes)
        for (int64_t P : {(int64_t)1, (int64_t)33, (int64_t)64, (int64_t)128, INT64_MAX})
          for (int64_t N : {(int64_t)1, (int64_t)16, (int64_t)256, INT64_MAX})
            for (int64_t stride : {(int64_t)0, (int64_t)512, INT64_MAX})
              for (int dt : {0, 1}) {
                mamba_heads_shape s = {};
                s.batch = batch; s.seqlen = L; s.heads = heads; s.headdim = P; s.dstate = N;
                s.groups = heads % 4 == 0 ? 4 : 1;
                s.u_batch_stride = s.B_batch_stride = stride;
                s.u_token_stride = s.B_token_stride = s.delta_token_stride = stride;
                s.C_token_stride = s.C_batch_stride = s.delta_batch_stride = stride;
                s.dtype = dt; s.delta_softplus = 1; s.segments = (int)(L & 7);
                const size_t nf = mamba_heads_scan_fwd_workspace_size(&s);
                const size_t nb = mamba_heads_scan_bwd_workspace_size(&s);
                const int rf = mamba_heads_scan_fwd(&s, buf, buf, f, buf, buf, f, f, f, nullptr,
                                                    buf, f, buf, SIZE_MAX - 1, nullptr);
                const int rb = mamba_heads_scan_bwd(&s, buf, buf, f, buf, buf, f, f, f, nullptr, buf,
                                                    f, buf, buf, f, buf, buf, f, f, f, buf,
                                                    SIZE_MAX - 1, nullptr);
                REQUIRE((nf == SIZE_MAX) == (rf != MAMBA_OK) && (nb == SIZE_MAX) == (rb != MAMBA_OK));
                s.seqlen = 1;
                mamba_heads_state_update(&s, f, nullptr, L, buf, buf, f, buf, buf, f, f, buf, nullptr);
                ++tried;
              }
  for (int64_t batch : sizes)
    for (int64_t dim : sizes)
      for (int64_t L : sizes)
        for (int64_t W : {(int64_t)-1, (int64_t)2, (int64_t)4, INT64_MAX})
          for (int dt : {0, 1}) {
            const mamba_dtype t = (mamba_dtype)dt;
            const size_t n = mamba_conv1d_tokens_bwd_workspace_size(batch, dim, L, W);
            mamba_conv1d_tokens_fwd(buf, L, dim, f, f, buf, nullptr, W, t, batch, dim, L, buf,
                                    buf + 256, nullptr);
            const int r = mamba_conv1d_tokens_bwd(buf, 0, 0, f, f, buf, nullptr, buf, W, t, batch,
                                                  dim, L, buf, f, f, buf, buf, SIZE_MAX - 1, nullptr);
            REQUIRE((n == SIZE_MAX) == (r != MAMBA_OK));
            mamba_conv1d_tokens_update(buf, dim, buf, nullptr, L, f, f, W, t, batch, dim, buf, nullptr);
            const size_t m = mamba_gated_norm_bwd_workspace_size(batch, dim, L);
            mamba_gated_norm_fwd(buf, dim, buf, dim, f, batch, dim, L, 1e-5f, 1, t, buf, nullptr);
            const int q = mamba_gated_norm_bwd(buf, 0, buf, 0, f, buf, batch, dim, L, 1e-5f, 0, t,
                                               buf, buf, f, buf, SIZE_MAX - 1, nullptr);
            REQUIRE((m == SIZE_MAX) == (q != MAMBA_OK));
            ++tried;
          }
  REQUIRE(launched > 1000);
  printf("heads ok: %ld tried, %ld launched\n", tried, launched);
  return 0;
}
