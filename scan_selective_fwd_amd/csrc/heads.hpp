// Parameters and dispatchers of the multi-head operators: the scan with one
// decay a head, its single-token form, the token-major convolution and the
// gated group norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mscan {

// Blocks of one launch: HIP takes less than 2^32 threads along a dimension.
constexpr int64_t max_blocks(int threads) { return (int64_t)0xFFFFFFFF / threads; }

// A batch of token rows: element (b, t, i) at p[b * batch + t * token + i].
struct Rows {
  const void* p;
  int64_t batch, token;
};

struct HeadsParams {
  Rows u, delta, B, C;
  const float* A;
  const float* D;        // nullable
  const float* bias;     // nullable
  const float* h0;       // nullable
  const uint8_t* reset;  // nullable
  int64_t batch, L;
  int H, P, G, N;
  int softplus, zoh;
  int vec;               // rows of u, B, C (and dout, out) start 16-byte aligned
  // a block's four waves take slices of 32 channels: of one head, or of hpw
  int slices, hpw, hblocks;   // slices a head, heads a block, blocks a group
  // the sequence in nseg segments of seg_len steps (whole chunks)
  int nseg;
  int64_t seg_len;
  void* scal;            // workspace, (batch, chunks, H) chunk scalars
  float* seg_state;      // workspace, (batch, H, slices, nseg - 1) states
  float* seg_dec;        // and their segments' decays
};

// Segments up to which the forward's output pass carries the state itself: its
// blocks then read (nseg - 1) / 2 states each on average, where a carry pass
// reads and writes every state once more.
constexpr int kSelfCarry = 8;

struct HeadsFwdParams : HeadsParams {
  bool carried;          // a carry pass joins the segments
  void* out;
  float* last;           // nullable
  float* h0_kept;        // nullable workspace, (batch, H, slices) states: h0 before last
                         // takes its place
};

struct HeadsBwdParams : HeadsParams {
  const void* dout;
  const float* dlast;    // nullable
  void* du;
  void* ddelta;
  float* dA;
  void* dB;
  void* dC;
  float* dD;             // nullable
  float* dbias;          // nullable
  float* dh0;            // nullable
  int splits;            // blocks that share the heads of a chunk
  int chunk;             // its tokens
  // workspace
  float* h_chunk;        // (batch, chunks, H, slices) states at the chunks' starts,
  float* g_chunk;        // adjoints behind their ends: from zero within a segment
  float* h_pre;          // (batch, chunks, H): weight in them of what enters the segment
  float* g_pre;
  float* h_seg;          // (batch, H, slices, nseg): the same of the segments
  float* g_seg;
  float* h_dec;
  float* g_dec;
  float* F;              // (batch, H, blocks of 64 channels, L): gradient of the log decay
  float* W;              // and of the inputs' weight
  float* dB_part;        // (splits, batch, L, G, N)
  float* dC_part;
  float* ud_part;        // (batch, chunks, H, blocks of 64 channels): sum of u dout
  float* head_part;      // (batch, chunks, H, 3): dA, dD, dbias
};

struct HeadsStepParams : HeadsParams {
  float* state;
  const int32_t* slots;  // nullable
  int64_t pool;
  void* out;
};

// Rows of a head's state that a block of the single-token form takes.
constexpr int64_t step_rows(int64_t N) {
  return N <= 16 ? 256 : N <= 32 ? 128 : N <= 64 ? 64 : N <= 128 ? 32 : 16;
}

// Heads that a block of the backward's chunks takes side by side, by the state's
// width in 32s, and the blocks that sum dB and dC at most.
constexpr int chunk_sides(int nk) { return nk == 4 ? 2 : 1; }
constexpr int64_t kMaxSumBlocks = 1 << 20;

hipError_t dispatch_heads_scal(const HeadsParams& p, int dtype, bool bwd, hipStream_t s);
hipError_t dispatch_heads_fwd(const HeadsFwdParams& p, int dtype, hipStream_t s);
hipError_t dispatch_heads_bwd(const HeadsBwdParams& p, int dtype, hipStream_t s);
hipError_t dispatch_heads_step(const HeadsStepParams& p, int dtype, hipStream_t s);

struct TokConvParams {
  Rows x;
  const float* w;
  const float* b;        // nullable
  const void* window;    // nullable
  const uint8_t* reset;  // nullable
  int64_t batch, dim, L;
  int W;
  bool vec;              // rows start 16-byte aligned: 16-byte loads
  int64_t tiles;         // token tiles of the launch
  // forward
  void* out;
  void* window_out;      // nullable
  // backward
  const void* dout;
  void* dx;
  float* dw;
  float* db;             // nullable
  void* dwindow;         // nullable
  float* part;           // (batch * tiles, W + 1, dim): the tiles' shares of dw, db
};

// Tokens a thread of the forward takes.
constexpr int kTokConvFwdRun = 16;
// Token tile of the backward: a block's 4 waves take kTokConvRun tokens each.
constexpr int kTokConvRun = 16;
constexpr int kTokConvTile = 4 * kTokConvRun;

hipError_t dispatch_tokconv_fwd(const TokConvParams& p, int dtype, hipStream_t s);
hipError_t dispatch_tokconv_bwd(const TokConvParams& p, int dtype, hipStream_t s);

struct TokConvStepParams {
  const void* x;
  int64_t x_batch;
  void* window;
  const int32_t* slots;  // nullable
  int64_t pool, batch, dim;
  const float* w;
  const float* b;        // nullable
  void* out;
  int W;
  bool vec;
};

hipError_t dispatch_tokconv_step(const TokConvStepParams& p, int dtype, hipStream_t s);

struct NormParams {
  const void* x;
  const void* z;         // nullable
  const float* w;        // nullable
  int64_t x_row, z_row;
  int64_t rows, dim, gs; // gs = dim / groups
  int groups;
  float eps;
  bool gate_first, vec;
  void* out;
  // backward
  const void* dout;
  void* dx;
  void* dz;              // nullable
  float* dw;             // nullable
  float* part;           // (parts, dim)
  int64_t parts;
};

// Rows that one launch of the norm's forward takes, with `per` groups a block.
inline int64_t norm_launch_rows(int64_t groups, int64_t per) {
  return max_blocks(256) * per / groups;
}

// Blocks that share the rows of one group in the norm's backward.
int64_t norm_parts(int64_t rows, int64_t groups);

hipError_t dispatch_norm_fwd(const NormParams& p, int dtype, hipStream_t s);
hipError_t dispatch_norm_bwd(const NormParams& p, int dtype, hipStream_t s);

}  // namespace mscan
