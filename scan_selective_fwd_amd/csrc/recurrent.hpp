// Parameters and dispatchers of the recurrent block's operators: the gated
// linear recurrence and the norm with the residual's addition.
#pragma once

#include "heads.hpp"

namespace mscan {

struct RecParams {
  Rows x, r, i, z;       // z.p nullable
  const float* A;
  const float* h0;       // nullable
  const uint8_t* reset;  // nullable
  int64_t batch, L, dim;
  // forward
  void* out;
  float* last;           // nullable
  float* ckpt;           // nullable, (batch, tiles, dim): the state entering each kRecTile steps
  bool pairs;            // rows start on 4 bytes and hold whole pairs of bfloat16
  // workspace where the sequence takes several tiles
  uint32_t* ticket;      // (batch * strips) counters, kTicketWords apart
  uint64_t* maps;        // (batch, tiles, dim): the tiles' maps
  uint64_t* heads;       // (batch, groups of tiles, dim): the state after each group
  int64_t words;         // of ticket, maps and heads together, in 64 bits: cleared first
  uint32_t by_die;       // strips that a die takes one after another; 0: in turn
  // backward
  const void* dout;
  const float* dlast;    // nullable
  const float* kept;     // the checkpoints
  void* dx;
  void* dr;
  void* di;
  void* dz;              // nullable
  float* dA;
  float* dh0;            // nullable
  float* part;           // workspace, (batch, tiles, dim): the tiles' shares of dA
};

constexpr int64_t kRecTile = 64;   // steps between checkpoints

// The forward: a wave takes kRecRun steps, a block up to 16 waves of one row, in one launch;
// longer sequences take tiles of kRecFwdTile steps, joined kRecGroup at a time, and a
// launch before that clears the words that join them.
constexpr int64_t kRecRun = 16;
constexpr int64_t kRecOneTile = 16 * kRecRun;
constexpr int64_t kRecFwdTile = 8 * kRecRun;
constexpr int64_t kRecGroup = 16;

// The backward: the same with runs of kRecBwdRun steps.
constexpr int64_t kRecBwdRun = 8;
constexpr int64_t kRecBwdOneTile = 16 * kRecBwdRun;
constexpr int64_t kRecBwdTile = 8 * kRecBwdRun;
static_assert(kRecBwdTile % kRecTile == 0 && kRecFwdTile % kRecTile == 0, "tiles between checkpoints");

// Tiles of a sequence in either pass.
constexpr int64_t rec_fwd_tiles(int64_t L) {
  return L <= kRecOneTile ? 1 : (L + kRecFwdTile - 1) / kRecFwdTile;
}
constexpr int64_t rec_bwd_tiles(int64_t L) {
  return L <= kRecBwdOneTile ? 1 : (L + kRecBwdTile - 1) / kRecBwdTile;
}

constexpr int kTicketWords = 32;

constexpr int64_t rec_strips(int64_t dim, bool pairs) {
  return pairs ? (dim + 127) / 128 : (dim + 63) / 64;
}

// Blocks go to the chip's eight dies in turn.  Neighbouring strips share the cache lines
// between them where rows do not start on one, and then go to the same die, as long as
// that leaves no die without work (backward of 8 x 2048 x 1538 187 -> 120 us, forward 66 ->
// 56, bfloat16).  Returns the blocks of a launch over `tiles` tiles of `across` strips.
inline int64_t rec_grid(RecParams* p, int64_t across, int64_t tiles, int es) {
  const bool apart = p->dim * es % 128 == 0;
  const bool by_die = across % 8 == 0 || (!apart && across >= 32);
  p->by_die = by_die ? (uint32_t)((across + 7) / 8) : 0;
  return (by_die ? 8 * (int64_t)p->by_die : across) * tiles;
}

hipError_t rec_clear(const RecParams& p, hipStream_t s);
hipError_t dispatch_rec_fwd(const RecParams& p, int dtype, hipStream_t s);
hipError_t dispatch_rec_bwd(const RecParams& p, int dtype, hipStream_t s);

struct RecStepParams {
  const void* x;
  const void* r;
  const void* i;
  const void* z;         // nullable
  int64_t x_row, r_row, i_row, z_row;
  const float* A;
  float* state;
  const int32_t* slots;  // nullable
  int64_t pool, batch, dim;
  bool vec;              // groups of four channels: one load of each tensor
  void* out;
};

hipError_t dispatch_rec_step(const RecStepParams& p, int dtype, hipStream_t s);

struct ResNormParams {
  const void* x;         // the backward's: nothing
  const void* res;       // nullable in the forward; the kept sum in the backward
  const float* w;        // nullable
  int64_t x_row, res_row;
  int64_t inner;         // rows of a batch row where x_batch, res_batch part them; 0: one run
  int64_t x_batch, res_batch;
  int64_t rows, dim;     // rows in all
  float eps;
  bool vec;              // every row starts on 16 bytes
  void* out;
  float* scale;          // 8 bits
  void* res_out;         // nullable
  // backward
  const void* dout;
  const void* dres;      // nullable
  void* dx;
  void* dresidual;       // nullable
  float* dw;             // nullable
  float* part;           // (parts, dim)
  int64_t parts;
};

// Types of a call: x, residual and out.
enum ResNormKind { kResF32, kResBf16, kResBf16F32 };   // x and residual alike, or bf16 on float32

// Blocks that share the rows in the norm's backward.
int64_t res_norm_parts(int64_t rows);

hipError_t dispatch_res_norm_fwd(const ResNormParams& p, ResNormKind kind, bool fp8, hipStream_t s);
hipError_t dispatch_res_norm_bwd(const ResNormParams& p, ResNormKind kind, hipStream_t s);

}  // namespace mscan
