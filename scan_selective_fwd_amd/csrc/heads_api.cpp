// C ABI of the multi-head operators: argument checks, workspace carving and
// dispatch.  Nothing here allocates, frees or synchronizes; every launch goes
// on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "heads.hpp"
#include "mamba_scan.h"

namespace {

constexpr int64_t kMaxHeadDim = 128;
constexpr int64_t kMaxHeadState = 256;
constexpr int64_t kLim = (int64_t)1 << 62;
constexpr int64_t kGridLim = 0x7FFFFFFF;

int esize(int dt) { return dt == MAMBA_F32 ? 4 : 2; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Nullable pointers pass.
bool aligned_f32(const void* p) { return aligned(p, 4); }

mamba_status hip_status(hipError_t e) { return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// a * b <= kLim for a, b >= 0.
bool mul_ok(int64_t a, int64_t b) { return b == 0 || a <= kLim / b; }

// Whether (batch, tokens) rows at these strides stay inside 2^62 elements.
bool span_ok(int64_t batch, int64_t sb, int64_t tokens, int64_t st) {
  return mul_ok(batch, sb) && mul_ok(tokens, st) && batch * sb <= kLim - tokens * st;
}

// Whether rows at p with these strides can be read in 16-byte pieces.
// (a chunk of 64 rows and one more within 2^31 bytes: the kernels' offsets inside one).
bool rows16(const void* p, int64_t sb, int64_t st, int64_t run, int es) {
  const int64_t v = 16 / es;
  return aligned(p, 16) && sb % v == 0 && st % v == 0 && run % v == 0 && st <= (1 << 21) &&
         run <= (1 << 21);
}

mamba_status check_shape(const mamba_heads_shape* s) {
  if (!s) return MAMBA_ERR_NULL_PTR;
  if (s->dtype != MAMBA_F32 && s->dtype != MAMBA_BF16) return MAMBA_ERR_DTYPE;
  if (s->disc != MAMBA_DISC_ZOH && s->disc != MAMBA_DISC_EULER) return MAMBA_ERR_DTYPE;
  if (s->batch <= 0 || s->seqlen <= 0 || s->heads <= 0 || s->headdim <= 0 || s->groups <= 0 ||
      s->dstate <= 0)
    return MAMBA_ERR_SHAPE;
  if (s->heads % s->groups != 0) return MAMBA_ERR_SHAPE;
  if (s->segments < 0) return MAMBA_ERR_INVALID;
  if (s->headdim > kMaxHeadDim || s->dstate > kMaxHeadState) return MAMBA_ERR_UNSUPPORTED;
  if (s->heads > (1 << 16) || s->batch > kGridLim / s->heads) return MAMBA_ERR_UNSUPPORTED;
  // dense (batch, seqlen, heads, headdim or dstate) arrays, in bytes
  if (s->seqlen > kLim / 1024 / (s->batch * s->heads)) return MAMBA_ERR_UNSUPPORTED;
  const int64_t strides[] = {s->u_batch_stride, s->u_token_stride, s->delta_batch_stride,
                             s->delta_token_stride, s->B_batch_stride, s->B_token_stride,
                             s->C_batch_stride, s->C_token_stride};
  for (int i = 0; i < 8; i += 2) {
    if (strides[i] < 0 || strides[i + 1] < 0) return MAMBA_ERR_SHAPE;
    if (!span_ok(s->batch, strides[i], s->seqlen, strides[i + 1])) return MAMBA_ERR_UNSUPPORTED;
  }
  return MAMBA_OK;
}

// The parameters all forms share; `vec` covers u, B and C only.
mscan::HeadsParams common(const mamba_heads_shape* s, const void* u, const void* delta,
                          const float* A, const void* B, const void* C, const float* D,
                          const float* bias, const float* h0, const uint8_t* reset) {
  mscan::HeadsParams p{};
  p.u = {u, s->u_batch_stride, s->u_token_stride};
  p.delta = {delta, s->delta_batch_stride, s->delta_token_stride};
  p.B = {B, s->B_batch_stride, s->B_token_stride};
  p.C = {C, s->C_batch_stride, s->C_token_stride};
  p.A = A; p.D = D; p.bias = bias; p.h0 = h0; p.reset = reset;
  p.batch = s->batch; p.L = s->seqlen;
  p.H = (int)s->heads; p.P = (int)s->headdim; p.G = (int)s->groups; p.N = (int)s->dstate;
  p.softplus = s->delta_softplus != 0; p.zoh = s->disc == MAMBA_DISC_ZOH;
  const int es = esize(s->dtype);
  p.vec = rows16(u, p.u.batch, p.u.token, p.P, es) && rows16(B, p.B.batch, p.B.token, p.N, es) &&
          rows16(C, p.C.batch, p.C.token, p.N, es) &&
          s->heads * s->headdim <= (1 << 21);   // a chunk of dense rows within 2^31 bytes too
  return p;
}

mamba_status check_inputs(const mamba_heads_shape* s, const void* u, const void* delta,
                          const float* A, const void* B, const void* C, const float* D,
                          const float* bias, const float* h0) {
  if (!u || !delta || !A || !B || !C) return MAMBA_ERR_NULL_PTR;
  const size_t es = (size_t)esize(s->dtype);
  if (!aligned(u, es) || !aligned(delta, es) || !aligned(B, es) || !aligned(C, es))
    return MAMBA_ERR_ALIGNMENT;
  if (!aligned_f32(A) || !aligned_f32(D) || !aligned_f32(bias) || !aligned_f32(h0))
    return MAMBA_ERR_ALIGNMENT;
  return MAMBA_OK;
}

constexpr int64_t kSlice = 32;   // channels a wave takes

int64_t chunk_len(const mamba_heads_shape* s) { return s->dtype == MAMBA_BF16 ? 64 : 32; }

// How heads map to the four waves of a block.
struct Map {
  int64_t slices, hpw, hblocks;
};

Map map_of(const mamba_heads_shape* s) {
  Map m;
  m.slices = (s->headdim + kSlice - 1) / kSlice;
  m.hpw = m.slices == 1 ? 4 : m.slices == 2 ? 2 : 1;
  const int64_t per = s->heads / s->groups;
  m.hblocks = (per + m.hpw - 1) / m.hpw;
  return m;
}

// dstate as the kernels hold it.
int64_t pad_state(const mamba_heads_shape* s) {
  return s->dstate <= 32 ? 32 : s->dstate <= 64 ? 64 : s->dstate <= 128 ? 128 : 256;
}

// Segments: as many as fit `target` blocks, the ones the chip holds at once (one
// more and they take two rounds), each of at least `least` chunks.  The forward
// takes 1: 200 steps of 24 heads take 23.9 us in four segments and 32.1 in one,
// 1000 steps 35.2 in 16, 38.6 in 8, 48.3 in 4.  The backward, whose segments
// serve its states pass alone, takes 2: 512 steps take 59.3 us in four segments,
// 61.9 in two, 57.2 in eight; 4 x 512 take 78.8 in two, 83.7 in four, 94.9 in
// eight.
constexpr int64_t kTargetBlocks = 512;
// The backward's states pass runs both directions at once.  In bfloat16 with
// N > 64 it is bound by the states it writes, more blocks gain nothing, and the
// chunks add an entering state where a segment does not begin the row.  With 160
// blocks for 256, of 64 channels and N = 128: 2 x 2048 x 80 heads take 319 us for
// 332, 8 x 2048 x 24 362 for 370, 4 x 4096 x 4 94 for 103, 65536 x 4 352 for 358,
// 16384 x 2 101 for 101, 16384 x 24 417 for 409, 65536 x 24 1512 for 1495; N = 256:
// 8192 x 8 in two groups 214 for 254, 2 x 8192 x 12 of 128 channels 1132 for 1055.
// Otherwise the products bound it: N = 64 takes 210 us for 204 (2 x 2048 x 80);
// float32 648 for 677 there, 158 for 158 with 16 heads, 102 for 99 (4 x 777 x 16,
// N = 64).
int64_t state_blocks(const mamba_heads_shape* s) {
  return s->dtype == MAMBA_BF16 && s->dstate > 64 ? 160 : kTargetBlocks / 2;
}
// Blocks of the backward's chunks that run at once: one a CU, two where N <= 64
// leaves them the LDS.
int64_t chunk_blocks(const mamba_heads_shape* s) { return s->dstate <= 64 ? 512 : 256; }

void split(const mamba_heads_shape* s, int64_t target, int64_t least, int* nseg,
           int64_t* seg_len) {
  const int64_t q = chunk_len(s), chunks = (s->seqlen + q - 1) / q;
  const int64_t blocks = s->batch * s->groups * map_of(s).hblocks;
  int64_t n = s->segments;
  if (n == 0) {
    n = target / blocks;
    if (n > chunks / least) n = chunks / least;
  }
  if (n > chunks) n = chunks;
  if (n > 4096) n = 4096;
  if (n < 1) n = 1;
  const int64_t per = (chunks + n - 1) / n;
  *seg_len = per * q;
  *nseg = (int)((chunks + per - 1) / per);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace of the forward: the segments' states and decays.
struct FwdLayout {
  int nseg;
  int64_t seg_len;
  size_t scal, state, dec, h0, total;
};

bool fwd_layout(const mamba_heads_shape* s, FwdLayout* l) {
  split(s, kTargetBlocks, 1, &l->nseg, &l->seg_len);
  const int64_t cols = s->batch * s->heads * map_of(s).slices;
  if (cols > kGridLim / l->nseg || cols > kGridLim / 16) return false;
  const int64_t most = mscan::max_blocks(256), bh = s->batch * s->heads;
  if (s->batch * s->groups * map_of(s).hblocks > most / l->nseg) return false;
  if (l->nseg > mscan::kSelfCarry && cols > most / (pad_state(s) / 32)) return false;
  const size_t n = (size_t)cols * (size_t)(l->nseg - 1);
  const int64_t q = chunk_len(s), chunks = (s->seqlen + q - 1) / q;
  if (chunks > kGridLim / bh || bh * chunks > 4 * most) return false;
  l->scal = 0;
  l->state = up256((size_t)(s->batch * s->heads * chunks) * (size_t)(28 * q + 16));
  l->dec = l->state + up256(n * (size_t)(kSlice * pad_state(s)) * 4);
  l->h0 = l->dec + up256(n * 4);
  // used where last_state is h0: another segment's block may write one before this
  // segment's reads the other
  l->total = l->h0 + (l->nseg > 1 ? up256((size_t)cols * (size_t)(kSlice * pad_state(s)) * 4) : 0);
  return true;
}

// Workspace of the backward: see HeadsBwdParams.
struct BwdLayout {
  int nseg, splits;
  int64_t seg_len;
  size_t scal, h_chunk, g_chunk, h_pre, g_pre, h_seg, g_seg, h_dec, g_dec, F, W, dB_part, dC_part,
      ud_part, head_part, total;
};

bool bwd_layout(const mamba_heads_shape* s, BwdLayout* l) {
  split(s, state_blocks(s), 2, &l->nseg, &l->seg_len);
  const int64_t q = chunk_len(s), chunks = (s->seqlen + q - 1) / q;
  const Map m = map_of(s);
  const int64_t bh = s->batch * s->heads, cols = bh * m.slices;
  const int64_t cb = (s->headdim + 63) / 64, units = s->heads / s->groups * cb;
  if (chunks > kGridLim / 16 / cols || cols > kGridLim / 32 / l->nseg) return false;
  if (s->batch * s->seqlen > kGridLim * 128 / (s->groups * s->dstate)) return false;
  const int64_t most = mscan::max_blocks(256), nk = pad_state(s) / 32;
  if (s->batch * s->groups * m.hblocks > most / 2 / l->nseg || cols > most / 2 / nk ||
      bh * chunks > 4 * (most - mscan::kMaxSumBlocks))
    return false;
  // The heads of a chunk are shared among as many blocks as run at once, each
  // with at least one: 2 x 2048 x 80 heads took 308 us with 256 blocks (336
  // and 387 against 330 with 512 and 1024); their shares of dB and dC are summed after.
  const int64_t blocks = s->batch * s->groups * chunks;
  int64_t sp = chunk_blocks(s) / blocks;
  if (sp > units) sp = units;
  if (sp < 1) sp = 1;
  l->splits = (int)sp;
  if (blocks > mscan::max_blocks(256 * mscan::chunk_sides((int)nk)) / sp) return false;
  const size_t state = (size_t)(kSlice * pad_state(s)) * 4;
  const size_t bch = (size_t)(bh * chunks), bl = (size_t)s->batch * (size_t)s->seqlen;
  const size_t gn = (size_t)(s->groups * s->dstate);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += up256(bytes);
    return o;
  };
  l->scal = take(bch * (size_t)(28 * q + 16));
  l->h_chunk = take(bch * (size_t)m.slices * state);
  l->g_chunk = take(bch * (size_t)m.slices * state);
  l->h_pre = take(bch * 4);
  l->g_pre = take(bch * 4);
  l->h_seg = take((size_t)cols * (size_t)l->nseg * state);
  l->g_seg = take((size_t)cols * (size_t)l->nseg * state);
  l->h_dec = take((size_t)cols * (size_t)l->nseg * 4);
  l->g_dec = take((size_t)cols * (size_t)l->nseg * 4);
  l->F = take(bl * (size_t)(s->heads * cb) * 4);
  l->W = take(bl * (size_t)(s->heads * cb) * 4);
  l->dB_part = take((size_t)sp * bl * gn * 4);
  l->dC_part = take((size_t)sp * bl * gn * 4);
  l->ud_part = take(bch * (size_t)cb * 4);
  l->head_part = take(bch * 12);
  l->total = at;
  return true;
}

mamba_status check_conv(const void* x, const float* w, const float* b, int64_t width,
                        mamba_dtype dt, int64_t batch, int64_t dim, int64_t L) {
  if (dt != MAMBA_F32 && dt != MAMBA_BF16) return MAMBA_ERR_DTYPE;
  if (batch <= 0 || dim <= 0 || L <= 0 || width <= 0) return MAMBA_ERR_SHAPE;
  if (width < 2 || width > 4) return MAMBA_ERR_UNSUPPORTED;
  // dense (batch, L, dim) arrays in bytes; a 32-bit grid of channel tiles
  if (batch > kGridLim / 4 || L > kLim / 16 / batch || dim > kLim / 16 / (batch * L) ||
      dim > (int64_t)1 << 24)
    return MAMBA_ERR_UNSUPPORTED;
  if (!x || !w) return MAMBA_ERR_NULL_PTR;
  if (!aligned(x, (size_t)esize(dt)) || !aligned_f32(w) || !aligned_f32(b))
    return MAMBA_ERR_ALIGNMENT;
  return MAMBA_OK;
}

int64_t conv_tiles(int64_t L, int64_t tile) { return (L + tile - 1) / tile; }

// Whether (tiles of tokens) x (batch rows) x (channel tiles) is a legal grid.
bool conv_grid_ok(int64_t batch, int64_t dim, int64_t tiles) {
  const int64_t cb = (dim + 63) / 64, most = mscan::max_blocks(256);
  return tiles <= most / batch && tiles * batch <= most / cb;
}

// The same of one thread a run of tokens and `v` channels.
bool conv_threads_ok(int64_t batch, int64_t dim, int64_t runs, int v) {
  const int64_t most = mscan::max_blocks(256) * 256;
  return runs <= most / batch && dim / v <= most / (runs * batch);
}

mamba_status check_norm(const void* x, int64_t x_row, const void* z, int64_t z_row,
                        const float* weight, int64_t rows, int64_t dim, int64_t groups, float eps,
                        mamba_dtype dt) {
  if (dt != MAMBA_F32 && dt != MAMBA_BF16) return MAMBA_ERR_DTYPE;
  if (rows <= 0 || dim <= 0 || groups <= 0 || dim % groups != 0) return MAMBA_ERR_SHAPE;
  if (x_row < 0 || (z && z_row < 0)) return MAMBA_ERR_SHAPE;
  if (!(eps >= 0.0f)) return MAMBA_ERR_INVALID;
  if (dim > (1 << 28) || rows > kLim / 16 / dim || groups > mscan::max_blocks(256) ||
      !mul_ok(rows, x_row) || !mul_ok(rows, z_row))
    return MAMBA_ERR_UNSUPPORTED;
  if (!x) return MAMBA_ERR_NULL_PTR;
  const size_t es = (size_t)esize(dt);
  if (!aligned(x, es) || !aligned(z, es) || !aligned_f32(weight)) return MAMBA_ERR_ALIGNMENT;
  return MAMBA_OK;
}

mscan::NormParams norm_params(const void* x, int64_t x_row, const void* z, int64_t z_row,
                              const float* weight, int64_t rows, int64_t dim, int64_t groups,
                              float eps, int gate_first, mamba_dtype dt) {
  mscan::NormParams p{};
  p.x = x; p.z = z; p.w = weight; p.x_row = x_row; p.z_row = z_row;
  p.rows = rows; p.dim = dim; p.gs = dim / groups; p.groups = (int)groups; p.eps = eps;
  p.gate_first = gate_first != 0;
  const int es = esize(dt);
  // every group starts on 16 bytes in x, z, the weights and the dense outputs
  p.vec = rows16(x, 0, x_row, p.gs, es) && (!z || rows16(z, 0, z_row, p.gs, es)) &&
          aligned(weight, 16);
  return p;
}

}  // namespace

extern "C" {

size_t mamba_heads_scan_fwd_workspace_size(const mamba_heads_shape* shape) {
  FwdLayout l;
  return check_shape(shape) == MAMBA_OK && fwd_layout(shape, &l) ? l.total : SIZE_MAX;
}

mamba_status mamba_heads_scan_fwd(const mamba_heads_shape* shape, const void* u,
                                  const void* delta, const float* A, const void* B,
                                  const void* C, const float* D, const float* delta_bias,
                                  const float* h0, const uint8_t* reset, void* out,
                                  float* last_state, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  mamba_status st = check_shape(shape);
  if (st != MAMBA_OK) return st;
  st = check_inputs(shape, u, delta, A, B, C, D, delta_bias, h0);
  if (st != MAMBA_OK) return st;
  if (!out) return MAMBA_ERR_NULL_PTR;
  if (!aligned(out, (size_t)esize(shape->dtype)) || !aligned_f32(last_state))
    return MAMBA_ERR_ALIGNMENT;
  FwdLayout l;
  if (!fwd_layout(shape, &l)) return MAMBA_ERR_UNSUPPORTED;
  if (h0 && last_state && last_state != h0) {   // in place, or apart
    const uintptr_t a = reinterpret_cast<uintptr_t>(h0), b = reinterpret_cast<uintptr_t>(last_state);
    if ((a < b ? b - a : a - b) <
        (size_t)(shape->batch * shape->heads) * (size_t)(shape->headdim * shape->dstate) * 4)
      return MAMBA_ERR_INVALID;
  }
  if (!workspace || workspace_bytes < l.total) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MAMBA_ERR_ALIGNMENT;
  mscan::HeadsFwdParams p{};
  static_cast<mscan::HeadsParams&>(p) =
      common(shape, u, delta, A, B, C, D, delta_bias, h0, reset);
  const Map m = map_of(shape);
  p.slices = (int)m.slices; p.hpw = (int)m.hpw; p.hblocks = (int)m.hblocks;
  p.nseg = l.nseg; p.seg_len = l.seg_len;
  p.scal = workspace;
  p.seg_state = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.state);
  p.seg_dec = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.dec);
  if (last_state && last_state == h0 && p.nseg > 1)
    p.h0_kept = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.h0);
  p.out = out; p.last = last_state; p.carried = p.nseg > mscan::kSelfCarry;
  p.vec = p.vec && aligned(out, 16);
  return hip_status(mscan::dispatch_heads_fwd(p, shape->dtype == MAMBA_F32 ? 0 : 1,
                                              as_stream(stream)));
}

size_t mamba_heads_scan_bwd_workspace_size(const mamba_heads_shape* shape) {
  BwdLayout l;
  return check_shape(shape) == MAMBA_OK && bwd_layout(shape, &l) ? l.total : SIZE_MAX;
}

mamba_status mamba_heads_scan_bwd(const mamba_heads_shape* shape, const void* u,
                                  const void* delta, const float* A, const void* B,
                                  const void* C, const float* D, const float* delta_bias,
                                  const float* h0, const uint8_t* reset, const void* dout,
                                  const float* dlast_state, void* du, void* ddelta, float* dA,
                                  void* dB, void* dC, float* dD, float* ddelta_bias, float* dh0,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  mamba_status st = check_shape(shape);
  if (st != MAMBA_OK) return st;
  st = check_inputs(shape, u, delta, A, B, C, D, delta_bias, h0);
  if (st != MAMBA_OK) return st;
  if (!dout || !du || !ddelta || !dA || !dB || !dC) return MAMBA_ERR_NULL_PTR;
  if ((dD && !D) || (ddelta_bias && !delta_bias) || (dh0 && !h0)) return MAMBA_ERR_INVALID;
  const size_t es = (size_t)esize(shape->dtype);
  if (!aligned(dout, es) || !aligned(du, es) || !aligned(ddelta, es) || !aligned(dB, es) ||
      !aligned(dC, es) || !aligned_f32(dlast_state) || !aligned_f32(dA) || !aligned_f32(dD) ||
      !aligned_f32(ddelta_bias) || !aligned_f32(dh0))
    return MAMBA_ERR_ALIGNMENT;
  BwdLayout l;
  if (!bwd_layout(shape, &l)) return MAMBA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < l.total) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MAMBA_ERR_ALIGNMENT;
  mscan::HeadsBwdParams p{};
  static_cast<mscan::HeadsParams&>(p) =
      common(shape, u, delta, A, B, C, D, delta_bias, h0, reset);
  p.dout = dout; p.dlast = dlast_state; p.du = du; p.ddelta = ddelta; p.dA = dA; p.dB = dB;
  p.dC = dC; p.dD = dD; p.dbias = ddelta_bias; p.dh0 = dh0;
  p.vec = p.vec && aligned(dout, 16) && aligned(du, 16) && aligned(dB, 16) && aligned(dC, 16);
  char* ws = static_cast<char*>(workspace);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  const Map m = map_of(shape);
  p.slices = (int)m.slices; p.hpw = (int)m.hpw; p.hblocks = (int)m.hblocks;
  p.nseg = l.nseg; p.seg_len = l.seg_len; p.splits = l.splits;
  p.chunk = (int)chunk_len(shape);
  p.scal = ws + l.scal;
  p.h_chunk = f(l.h_chunk); p.g_chunk = f(l.g_chunk); p.h_pre = f(l.h_pre); p.g_pre = f(l.g_pre);
  p.h_seg = f(l.h_seg); p.g_seg = f(l.g_seg); p.h_dec = f(l.h_dec); p.g_dec = f(l.g_dec);
  p.F = f(l.F); p.W = f(l.W); p.dB_part = f(l.dB_part); p.dC_part = f(l.dC_part);
  p.ud_part = f(l.ud_part); p.head_part = f(l.head_part);
  return hip_status(mscan::dispatch_heads_bwd(p, shape->dtype == MAMBA_F32 ? 0 : 1,
                                              as_stream(stream)));
}

mamba_status mamba_heads_state_update(const mamba_heads_shape* shape, float* state,
                                      const int32_t* slots, int64_t pool, const void* u,
                                      const void* delta, const float* A, const void* B,
                                      const void* C, const float* D, const float* delta_bias,
                                      void* out, void* stream) {
  mamba_status st = check_shape(shape);
  if (st != MAMBA_OK) return st;
  if (shape->seqlen != 1 || pool <= 0 || (!slots && pool < shape->batch)) return MAMBA_ERR_SHAPE;
  if (pool > kLim / (kMaxHeadDim * kMaxHeadState * 4) / shape->heads) return MAMBA_ERR_UNSUPPORTED;
  const int64_t rows = mscan::step_rows(shape->dstate);
  if (shape->batch * shape->heads > mscan::max_blocks(256) / ((shape->headdim + rows - 1) / rows))
    return MAMBA_ERR_UNSUPPORTED;
  st = check_inputs(shape, u, delta, A, B, C, D, delta_bias, nullptr);
  if (st != MAMBA_OK) return st;
  if (!state || !out) return MAMBA_ERR_NULL_PTR;
  if (!aligned(out, (size_t)esize(shape->dtype)) || !aligned_f32(state) || !aligned(slots, 4))
    return MAMBA_ERR_ALIGNMENT;
  mscan::HeadsStepParams p{};
  static_cast<mscan::HeadsParams&>(p) =
      common(shape, u, delta, A, B, C, D, delta_bias, nullptr, nullptr);
  p.state = state; p.slots = slots; p.pool = pool; p.out = out;
  return hip_status(mscan::dispatch_heads_step(p, shape->dtype == MAMBA_F32 ? 0 : 1,
                                               as_stream(stream)));
}

mamba_status mamba_conv1d_tokens_fwd(const void* x, int64_t x_batch_stride,
                                     int64_t x_token_stride, const float* w, const float* b,
                                     const void* window, const uint8_t* reset, int64_t width,
                                     mamba_dtype dt, int64_t batch, int64_t dim, int64_t seqlen,
                                     void* out, void* window_out, void* stream) {
  mamba_status st = check_conv(x, w, b, width, dt, batch, dim, seqlen);
  if (st != MAMBA_OK) return st;
  if (x_batch_stride < 0 || x_token_stride < 0) return MAMBA_ERR_SHAPE;
  if (!span_ok(batch, x_batch_stride, seqlen, x_token_stride)) return MAMBA_ERR_UNSUPPORTED;
  if (!out) return MAMBA_ERR_NULL_PTR;
  const int es = esize(dt);
  if (!aligned(out, (size_t)es) || !aligned(window, (size_t)es) || !aligned(window_out, (size_t)es))
    return MAMBA_ERR_ALIGNMENT;
  if (window && window == window_out) return MAMBA_ERR_INVALID;
  // a run of tokens reads the last inputs of the one before, which may have written by then
  if (out == x) return MAMBA_ERR_INVALID;
  mscan::TokConvParams p{};
  p.x = {x, x_batch_stride, x_token_stride};
  p.w = w; p.b = b; p.window = window; p.reset = reset;
  p.batch = batch; p.dim = dim; p.L = seqlen; p.W = (int)width;
  p.out = out; p.window_out = window_out;
  p.vec = rows16(x, x_batch_stride, x_token_stride, dim, es) && aligned(out, 16) &&
          aligned(window, 16) && aligned(window_out, 16) && aligned(w, 16) && aligned(b, 16);
  if (!conv_threads_ok(batch, dim, conv_tiles(seqlen, mscan::kTokConvFwdRun), p.vec ? 4 : 1))
    return MAMBA_ERR_UNSUPPORTED;
  return hip_status(mscan::dispatch_tokconv_fwd(p, dt == MAMBA_F32 ? 0 : 1, as_stream(stream)));
}

size_t mamba_conv1d_tokens_bwd_workspace_size(int64_t batch, int64_t dim, int64_t seqlen,
                                              int64_t width) {
  static const float dummy[4] = {};
  if (check_conv(dummy, dummy, nullptr, width, MAMBA_F32, batch, dim, seqlen) != MAMBA_OK)
    return SIZE_MAX;
  const int64_t tiles = conv_tiles(seqlen, mscan::kTokConvTile);
  if (!conv_grid_ok(batch, dim, tiles)) return SIZE_MAX;
  return up256((size_t)(batch * tiles) * (size_t)(width + 1) * (size_t)dim * 4);
}

mamba_status mamba_conv1d_tokens_bwd(const void* x, int64_t x_batch_stride,
                                     int64_t x_token_stride, const float* w, const float* b,
                                     const void* window, const uint8_t* reset, const void* dout,
                                     int64_t width, mamba_dtype dt, int64_t batch, int64_t dim,
                                     int64_t seqlen, void* dx, float* dw, float* db,
                                     void* dwindow, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  mamba_status st = check_conv(x, w, b, width, dt, batch, dim, seqlen);
  if (st != MAMBA_OK) return st;
  if (x_batch_stride < 0 || x_token_stride < 0) return MAMBA_ERR_SHAPE;
  if (!span_ok(batch, x_batch_stride, seqlen, x_token_stride)) return MAMBA_ERR_UNSUPPORTED;
  if (!dout || !dx || !dw) return MAMBA_ERR_NULL_PTR;
  if ((db && !b) || (dwindow && !window)) return MAMBA_ERR_INVALID;
  const int es = esize(dt);
  if (!aligned(dout, (size_t)es) || !aligned(dx, (size_t)es) || !aligned(window, (size_t)es) ||
      !aligned(dwindow, (size_t)es) || !aligned_f32(dw) || !aligned_f32(db))
    return MAMBA_ERR_ALIGNMENT;
  const size_t need = mamba_conv1d_tokens_bwd_workspace_size(batch, dim, seqlen, width);
  if (need == SIZE_MAX) return MAMBA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MAMBA_ERR_ALIGNMENT;
  mscan::TokConvParams p{};
  p.x = {x, x_batch_stride, x_token_stride};
  p.w = w; p.b = b; p.window = window; p.reset = reset;
  p.batch = batch; p.dim = dim; p.L = seqlen; p.W = (int)width;
  p.tiles = conv_tiles(seqlen, mscan::kTokConvTile);
  p.dout = dout; p.dx = dx; p.dw = dw; p.db = db; p.dwindow = dwindow;
  p.part = static_cast<float*>(workspace);
  p.vec = rows16(x, x_batch_stride, x_token_stride, dim, es) && aligned(dout, 16) &&
          aligned(dx, 16) && aligned(window, 16) && aligned(dwindow, 16) && aligned(w, 16) &&
          aligned(b, 16);
  return hip_status(mscan::dispatch_tokconv_bwd(p, dt == MAMBA_F32 ? 0 : 1, as_stream(stream)));
}

mamba_status mamba_conv1d_tokens_update(const void* x, int64_t x_batch_stride, void* window,
                                        const int32_t* slots, int64_t pool, const float* w,
                                        const float* b, int64_t width, mamba_dtype dt,
                                        int64_t batch, int64_t dim, void* out, void* stream) {
  mamba_status st = check_conv(x, w, b, width, dt, batch, dim, 1);
  if (st != MAMBA_OK) return st;
  if (x_batch_stride < 0 || pool <= 0 || (!slots && pool < batch)) return MAMBA_ERR_SHAPE;
  if (!mul_ok(batch, x_batch_stride) || pool > kLim / 64 / dim) return MAMBA_ERR_UNSUPPORTED;
  if (!window || !out) return MAMBA_ERR_NULL_PTR;
  const int es = esize(dt);
  if (!aligned(out, (size_t)es) || !aligned(window, (size_t)es) || !aligned(slots, 4))
    return MAMBA_ERR_ALIGNMENT;
  mscan::TokConvStepParams p{};
  p.x = x; p.x_batch = x_batch_stride; p.window = window; p.slots = slots; p.pool = pool;
  p.batch = batch; p.dim = dim; p.w = w; p.b = b; p.out = out; p.W = (int)width;
  p.vec = rows16(x, x_batch_stride, 0, dim, es) && aligned(window, 16) && aligned(out, 16) &&
          aligned(w, 16) && aligned(b, 16);
  if (!conv_threads_ok(batch, dim, 1, p.vec ? 4 : 1)) return MAMBA_ERR_UNSUPPORTED;
  return hip_status(mscan::dispatch_tokconv_step(p, dt == MAMBA_F32 ? 0 : 1, as_stream(stream)));
}

mamba_status mamba_gated_norm_fwd(const void* x, int64_t x_row_stride, const void* z,
                                  int64_t z_row_stride, const float* weight, int64_t rows,
                                  int64_t dim, int64_t groups, float eps, int gate_first,
                                  mamba_dtype dt, void* out, void* stream) {
  mamba_status st = check_norm(x, x_row_stride, z, z_row_stride, weight, rows, dim, groups, eps, dt);
  if (st != MAMBA_OK) return st;
  if (!out) return MAMBA_ERR_NULL_PTR;
  if (!aligned(out, (size_t)esize(dt))) return MAMBA_ERR_ALIGNMENT;
  mscan::NormParams p = norm_params(x, x_row_stride, z, z_row_stride, weight, rows, dim, groups,
                                    eps, gate_first, dt);
  p.out = out;
  p.vec = p.vec && aligned(out, 16);
  return hip_status(mscan::dispatch_norm_fwd(p, dt == MAMBA_F32 ? 0 : 1, as_stream(stream)));
}

size_t mamba_gated_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups) {
  static const float dummy[4] = {};
  if (check_norm(dummy, dim, nullptr, 0, nullptr, rows, dim, groups, 0.0f, MAMBA_F32) != MAMBA_OK)
    return SIZE_MAX;
  return up256((size_t)mscan::norm_parts(rows, groups) * (size_t)dim * 4);
}

mamba_status mamba_gated_norm_bwd(const void* x, int64_t x_row_stride, const void* z,
                                  int64_t z_row_stride, const float* weight, const void* dout,
                                  int64_t rows, int64_t dim, int64_t groups, float eps,
                                  int gate_first, mamba_dtype dt, void* dx, void* dz,
                                  float* dweight, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  mamba_status st = check_norm(x, x_row_stride, z, z_row_stride, weight, rows, dim, groups, eps, dt);
  if (st != MAMBA_OK) return st;
  if (!dout || !dx) return MAMBA_ERR_NULL_PTR;
  if ((z != nullptr) != (dz != nullptr) || (weight != nullptr) != (dweight != nullptr))
    return MAMBA_ERR_INVALID;
  const size_t es = (size_t)esize(dt);
  if (!aligned(dout, es) || !aligned(dx, es) || !aligned(dz, es) || !aligned_f32(dweight))
    return MAMBA_ERR_ALIGNMENT;
  const size_t need = mamba_gated_norm_bwd_workspace_size(rows, dim, groups);
  if (need == SIZE_MAX) return MAMBA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MAMBA_ERR_ALIGNMENT;
  mscan::NormParams p = norm_params(x, x_row_stride, z, z_row_stride, weight, rows, dim, groups,
                                    eps, gate_first, dt);
  p.dout = dout; p.dx = dx; p.dz = dz; p.dw = dweight;
  p.part = static_cast<float*>(workspace);
  p.parts = mscan::norm_parts(rows, groups);
  p.vec = p.vec && aligned(dout, 16) && aligned(dx, 16) && aligned(dz, 16);
  return hip_status(mscan::dispatch_norm_bwd(p, dt == MAMBA_F32 ? 0 : 1, as_stream(stream)));
}

}  // extern "C"
