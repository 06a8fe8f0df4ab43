// The largest sizes that the ABI layer of the multi-head operators lets through to a
// launch, and the next ones, which it refuses: a launch takes less than 2^32 threads.
// The dispatchers are stand-ins; nothing is launched or followed.
#include <stdio.h>
#include <stdlib.h>

#include "heads.hpp"
#include "mamba_scan.h"

#define REQUIRE(c)                                          \
  do {                                                      \
    if (!(c)) {                                             \
      printf("line %d: %s\n", __LINE__, #c);                \
      exit(1);                                              \
    }                                                       \
  } while (0)

namespace mscan {
hipError_t dispatch_heads_fwd(const HeadsFwdParams&, int, hipStream_t) { return hipSuccess; }
hipError_t dispatch_heads_bwd(const HeadsBwdParams&, int, hipStream_t) { return hipSuccess; }
hipError_t dispatch_heads_step(const HeadsStepParams&, int, hipStream_t) { return hipSuccess; }
hipError_t dispatch_tokconv_fwd(const TokConvParams&, int, hipStream_t) { return hipSuccess; }
hipError_t dispatch_tokconv_bwd(const TokConvParams&, int, hipStream_t) { return hipSuccess; }
hipError_t dispatch_tokconv_step(const TokConvStepParams&, int, hipStream_t) { return hipSuccess; }
hipError_t dispatch_norm_fwd(const NormParams&, int, hipStream_t) { return hipSuccess; }
hipError_t dispatch_norm_bwd(const NormParams&, int, hipStream_t) { return hipSuccess; }
int64_t norm_parts(int64_t rows, int64_t groups) {
  const int64_t n = 1024 / groups < 1 ? 1 : 1024 / groups;
  return n < rows ? n : rows;
}
}  // namespace mscan

static char* const buf = reinterpret_cast<char*>((uintptr_t)1 << 20);
static float* const f32 = reinterpret_cast<float*>((uintptr_t)1 << 20);

static mamba_heads_shape shape(int64_t batch, int64_t L, int64_t heads, int64_t P, int64_t N) {
  mamba_heads_shape s = {};
  s.batch = batch; s.seqlen = L; s.heads = heads; s.groups = 1; s.headdim = P; s.dstate = N;
  s.dtype = MAMBA_BF16; s.segments = 1;
  return s;
}

static int fwd(const mamba_heads_shape& s) {
  const int r = mamba_heads_scan_fwd(&s, buf, buf, f32, buf, buf, nullptr, nullptr, nullptr, nullptr,
                                     buf, nullptr, buf, SIZE_MAX - 1, nullptr);
  REQUIRE((mamba_heads_scan_fwd_workspace_size(&s) == SIZE_MAX) == (r != MAMBA_OK));
  return r;
}
static int bwd(const mamba_heads_shape& s) {
  const int r = mamba_heads_scan_bwd(&s, buf, buf, f32, buf, buf, nullptr, nullptr, nullptr, nullptr,
                                     buf, nullptr, buf, buf, f32, buf, buf, nullptr, nullptr, nullptr,
                                     buf, SIZE_MAX - 1, nullptr);
  REQUIRE((mamba_heads_scan_bwd_workspace_size(&s) == SIZE_MAX) == (r != MAMBA_OK));
  return r;
}
static int step(const mamba_heads_shape& s) {
  return mamba_heads_state_update(&s, f32, nullptr, s.batch, buf, buf, f32, buf, buf, nullptr,
                                  nullptr, buf, nullptr);
}
static int conv(int64_t batch, int64_t dim, int64_t L, char* x) {
  return mamba_conv1d_tokens_fwd(x, 0, 0, f32, nullptr, nullptr, nullptr, 4, MAMBA_BF16, batch, dim,
                                 L, buf + 4096, nullptr, nullptr);
}
static int conv_one(int64_t batch, int64_t dim, char* x) {
  return mamba_conv1d_tokens_update(x, 0, buf, nullptr, batch, f32, nullptr, 4, MAMBA_BF16, batch,
                                    dim, buf, nullptr);
}
static int norm(int64_t rows, int64_t dim, int64_t groups) {
  return mamba_gated_norm_fwd(buf, 0, nullptr, 0, nullptr, rows, dim, groups, 0.0f, 1, MAMBA_BF16,
                              buf, nullptr);
}

int main() {
  const int H = 1 << 16, BAD = MAMBA_ERR_UNSUPPORTED;
  REQUIRE(mscan::max_blocks(256) == (1 << 24) - 1 && mscan::max_blocks(512) == (1 << 23) - 1);
  // the output pass: a block a head of 128 channels and segment
  REQUIRE(fwd(shape(255, 1, H, 128, 16)) == MAMBA_OK && fwd(shape(256, 1, H, 128, 16)) == BAD);
  // the scalars: four (chunk, head) a block
  REQUIRE(fwd(shape(255, 4 * 64, H, 128, 16)) == MAMBA_OK);
  REQUIRE(fwd(shape(255, 4 * 64 + 65, H, 128, 16)) == BAD);
  // the carry over more segments than the output pass joins, 8 blocks a slice of 32
  mamba_heads_shape s = shape(1, 64 * 9, 1 << 14, 128, 256);
  s.segments = 9;
  REQUIRE(fwd(s) == MAMBA_OK);
  s.batch = 32;
  REQUIRE(fwd(s) == BAD);
  // the backward's carry, both directions
  REQUIRE(bwd(shape(31, 1, H, 128, 16)) == MAMBA_OK && bwd(shape(32, 1, H, 128, 16)) == BAD);
  // its chunks, 512 threads a block at N = 128
  REQUIRE(bwd(shape(1, 64ll * ((1 << 23) - 1), 1, 32, 128)) == MAMBA_OK);
  REQUIRE(bwd(shape(1, 64ll * (1 << 23), 1, 32, 128)) == BAD);
  // the single-token forms
  REQUIRE(step(shape(255, 1, H, 1, 1)) == MAMBA_OK && step(shape(256, 1, H, 1, 1)) == BAD);
  REQUIRE(step(shape(31, 1, H, 128, 256)) == MAMBA_OK && step(shape(32, 1, H, 128, 256)) == BAD);
  // the convolution: four channels a thread, or one off 16 bytes
  const int64_t wide = 1 << 24, rows16 = 1 << 21;
  REQUIRE(conv_one(8191, rows16, buf) == MAMBA_OK && conv_one(8192, rows16, buf) == BAD);
  REQUIRE(conv_one(255, wide, buf + 2) == MAMBA_OK && conv_one(256, wide, buf + 2) == BAD);
  REQUIRE(conv(8191, rows16, 16, buf) == MAMBA_OK && conv(8191, rows16, 17, buf) == BAD);
  REQUIRE(conv(255, wide, 16, buf + 2) == MAMBA_OK && conv(256, wide, 1, buf + 2) == BAD);
  REQUIRE(mamba_conv1d_tokens_bwd_workspace_size(63, wide, 64, 4) != SIZE_MAX);
  REQUIRE(mamba_conv1d_tokens_bwd_workspace_size(64, wide, 64, 4) == SIZE_MAX);
  // the norm takes more rows in more launches
  REQUIRE(norm(1ll << 32, 8, 1) == MAMBA_OK);
  REQUIRE(norm(1, (1 << 24) - 1, (1 << 24) - 1) == MAMBA_OK);
  REQUIRE(norm(1, 1 << 24, 1 << 24) == BAD);
  for (int64_t groups : {(int64_t)1, (int64_t)3, (int64_t)1000, (int64_t)(1 << 24) - 1})
    for (int64_t per : {(int64_t)1, (int64_t)4}) {
      const int64_t rows = mscan::norm_launch_rows(groups, per);
      REQUIRE(rows >= 1 && (rows * groups + per - 1) / per <= mscan::max_blocks(256));
    }
  printf("limits ok\n");
  return 0;
}
