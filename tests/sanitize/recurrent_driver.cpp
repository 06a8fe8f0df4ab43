// Drives the C ABI layer of the recurrent block's operators on the host, the
// dispatchers replaced by stand-ins that check what they are given.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "mamba_scan.h"
#include "recurrent.hpp"

static long launched = 0;
static const char* ws_begin = nullptr;
static size_t ws_bytes = 0;

#define REQUIRE(c)                                          \
  do {                                                      \
    if (!(c)) {                                             \
      printf("line %d: %s\n", __LINE__, #c);                \
      exit(1);                                              \
    }                                                       \
  } while (0)

// Whether [p, p + n) lies in the workspace of the call.
static bool inside(const void* p, size_t n) {
  const char* q = static_cast<const char*>(p);
  return q >= ws_begin && n <= ws_bytes && (size_t)(q - ws_begin) <= ws_bytes - n;
}

namespace mscan {

static void chain(const RecParams& p, int64_t tiles) {
  ++launched;
  REQUIRE(p.batch > 0 && p.L > 0 && p.dim > 0);
  REQUIRE((p.ticket != nullptr) == (tiles > 1));
  RecParams q = p;
  const int64_t across = p.batch * rec_strips(p.dim, p.pairs), grid = rec_grid(&q, across, tiles, 4);
  REQUIRE(grid > 0 && grid <= max_blocks(64) && (!q.by_die || 8 * (int64_t)q.by_die >= across));
  if (!p.ticket) return;
  const size_t row = (size_t)(p.batch * p.dim) * 8;
  const int64_t groups = (tiles + kRecGroup - 1) / kRecGroup;
  REQUIRE(inside(p.ticket, (size_t)p.words * 8));
  REQUIRE(inside(p.ticket, (size_t)across * kTicketWords * 4));
  REQUIRE(inside(p.maps, row * (size_t)tiles) && inside(p.heads, row * (size_t)groups));
  REQUIRE((const char*)p.maps >= (const char*)p.ticket + across * kTicketWords * 4);
  REQUIRE((const char*)p.heads >= (const char*)p.maps + row * (size_t)tiles);
  // what is cleared ends with the last of the heads
  REQUIRE((const char*)p.ticket + p.words * 8 == (const char*)p.heads + row * (size_t)groups);
}
hipError_t dispatch_rec_fwd(const RecParams& p, int, hipStream_t) {
  chain(p, rec_fwd_tiles(p.L));
  REQUIRE(p.out || inside(p.ckpt, (size_t)(p.batch * p.dim) * 4 * (size_t)((p.L + 63) / 64)));
  return hipSuccess;
}
hipError_t dispatch_rec_bwd(const RecParams& p, int, hipStream_t) {
  chain(p, rec_bwd_tiles(p.L));
  REQUIRE(p.kept && inside(p.part, (size_t)(p.batch * p.dim) * 4 * (size_t)rec_bwd_tiles(p.L)));
  if (p.ticket) REQUIRE((const char*)p.part >= (const char*)p.ticket + p.words * 8);
  return hipSuccess;
}
hipError_t dispatch_rec_step(const RecStepParams&, int, hipStream_t) { ++launched; return hipSuccess; }
int64_t res_norm_parts(int64_t rows) { return rows < 512 ? rows : 512; }
hipError_t dispatch_res_norm_fwd(const ResNormParams& p, ResNormKind, bool fp8, hipStream_t) {
  ++launched;
  REQUIRE(p.out && (!fp8 || p.scale));
  return hipSuccess;
}
hipError_t dispatch_res_norm_bwd(const ResNormParams& p, ResNormKind, hipStream_t) {
  ++launched;
  REQUIRE(p.parts >= 1 && inside(p.part, (size_t)(p.parts * p.dim) * 4));
  return hipSuccess;
}

}  // namespace mscan

int main() {
  // pointers that are never followed, far enough from each other
  char* base = reinterpret_cast<char*>((uintptr_t)1 << 50);
  auto at = [&](int k) { return base + ((uintptr_t)k << 44); };
  const int64_t sizes[] = {1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4096,
                           70000, (int64_t)1 << 27, (int64_t)1 << 40};
  const int64_t dims[] = {1, 2, 63, 64, 65, 128, 1003, 5120, (int64_t)1 << 28, ((int64_t)1 << 28) + 1};
  const int64_t batches[] = {1, 3, 300, 70000, (int64_t)1 << 33};
  long refused = 0, ran = 0;
  for (int64_t b : batches)
    for (int64_t L : sizes)
      for (int64_t d : dims)
        for (int dt = 0; dt < 2; ++dt) {
          mamba_recurrence_shape s{};
          s.batch = b; s.seqlen = L; s.dim = d; s.dtype = dt;
          const bool small = b < (int64_t)1 << 20 && L < (int64_t)1 << 30 && d < (int64_t)1 << 30;
          const int64_t row = small ? d : 0;
          s.x_token_stride = s.r_token_stride = s.i_token_stride = s.z_token_stride = row;
          s.x_batch_stride = s.r_batch_stride = s.i_batch_stride = s.z_batch_stride = row * (small ? L : 0);
          const bool fits = (double)b * (double)L * (double)d * 4 < 1e13;   // under 2^44 bytes
          const size_t nf = mamba_gated_recurrence_fwd_workspace_size(&s);
          const size_t n0 = mamba_gated_recurrence_bwd_workspace_size(&s, 0);
          const size_t n1 = mamba_gated_recurrence_bwd_workspace_size(&s, 1);
          const size_t nc = mamba_gated_recurrence_checkpoint_size(&s);
          REQUIRE(nc == SIZE_MAX || nc == (size_t)(b * d) * (size_t)((L + 63) / 64) * 4);
          REQUIRE(n0 >= n1 || n1 == SIZE_MAX);
          void* ws = at(9);
          for (int z = 0; z < 2; ++z)
            for (int kept = 0; kept < 2; ++kept) {
              ws_begin = at(9); ws_bytes = nf == SIZE_MAX ? 0 : nf;
              mamba_status st = mamba_gated_recurrence_fwd(
                  &s, at(1), at(2), at(3), (const float*)at(4), z ? at(5) : nullptr, nullptr, nullptr,
                  at(6), (float*)at(7), kept ? (float*)at(8) : nullptr, ws, ws_bytes, nullptr);
              REQUIRE(!fits || (st == MAMBA_OK) == (nf != SIZE_MAX));
              if (st == MAMBA_OK) ++ran; else ++refused;
              if (nf != SIZE_MAX && nf > 0 && fits)
                REQUIRE(mamba_gated_recurrence_fwd(&s, at(1), at(2), at(3), (const float*)at(4), nullptr,
                                                   nullptr, nullptr, at(6), nullptr, nullptr, ws, nf - 1,
                                                   nullptr) == MAMBA_ERR_WORKSPACE);
              const size_t nb = kept ? n1 : n0;
              ws_bytes = nb == SIZE_MAX ? 0 : nb;
              st = mamba_gated_recurrence_bwd(
                  &s, at(1), at(2), at(3), (const float*)at(4), z ? at(5) : nullptr, nullptr, nullptr,
                  at(6), nullptr, kept ? (const float*)at(8) : nullptr, at(10), at(11), at(12),
                  (float*)at(13), z ? at(14) : nullptr, nullptr, ws, ws_bytes, nullptr);
              REQUIRE(!fits || (st == MAMBA_OK) == (nb != SIZE_MAX));
              if (nb != SIZE_MAX && fits)
                REQUIRE(mamba_gated_recurrence_bwd(&s, at(1), at(2), at(3), (const float*)at(4), nullptr,
                                                   nullptr, nullptr, at(6), nullptr,
                                                   kept ? (const float*)at(8) : nullptr, at(10), at(11),
                                                   at(12), (float*)at(13), nullptr, nullptr, ws, nb - 1,
                                                   nullptr) == MAMBA_ERR_WORKSPACE);
            }
          s.seqlen = 1;
          mamba_gated_recurrence_update(&s, (float*)at(4), nullptr, b, at(1), at(2), at(3),
                                        (const float*)at(8), nullptr, at(6), nullptr);
        }
  for (int64_t rows : sizes)
    for (int64_t d : dims)
      for (int dt = 0; dt < 2; ++dt)
        for (int rdt = 0; rdt < 2; ++rdt) {
          const bool fits = (double)rows * (double)d * 4 < 1e13;
          const size_t n = mamba_residual_norm_bwd_workspace_size(rows, d);
          mamba_status st = mamba_residual_norm_fwd(at(1), d, d, at(2), d, d, (const float*)at(3), 1, rows, d, 1e-5f,
                                                    (mamba_dtype)dt, (mamba_dtype)rdt, at(4), at(5), nullptr);
          REQUIRE(dt == 0 && rdt == 1 ? st == MAMBA_ERR_DTYPE
                                      : !fits || (st == MAMBA_OK) == (n != SIZE_MAX));
          mamba_residual_norm_fp8(at(1), d, d, nullptr, 0, 0, nullptr, 3, rows, d, 1e-5f, (mamba_dtype)dt,
                                  (mamba_dtype)dt, (uint8_t*)at(4), (float*)at(5), nullptr, nullptr);
          ws_begin = at(9); ws_bytes = n == SIZE_MAX ? 0 : n;
          mamba_residual_norm_bwd(at(1), d, d, (const float*)at(2), at(3), at(4), 1, rows, d, 1e-5f,
                                  (mamba_dtype)dt, (mamba_dtype)rdt, at(5),
                                  dt != rdt ? at(6) : nullptr, (float*)at(7), at(9), ws_bytes, nullptr);
        }
  REQUIRE(launched > 1000 && ran > 100 && refused > 100);
  printf("recurrent ok: %ld launches\n", launched);
  return 0;
}
