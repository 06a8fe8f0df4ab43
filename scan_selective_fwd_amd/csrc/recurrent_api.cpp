// C ABI of the recurrent block's operators: argument checks, workspace carving
// and dispatch.  Nothing here allocates, frees or synchronizes; every launch goes
// on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "mamba_scan.h"
#include "recurrent.hpp"

namespace {

constexpr int64_t kLim = (int64_t)1 << 60;   // elements: their bytes fit 64 bits

int esize(int dt) { return dt == MAMBA_F32 ? 4 : 2; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Nullable pointers pass.
bool aligned_f32(const void* p) { return aligned(p, 4); }

mamba_status hip_status(hipError_t e) { return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// a * b <= kLim for a, b >= 0.
bool mul_ok(int64_t a, int64_t b) { return b == 0 || a <= kLim / b; }

// Whether (batch, tokens) rows at these strides stay inside 2^60 elements.
bool span_ok(int64_t batch, int64_t sb, int64_t tokens, int64_t st) {
  return mul_ok(batch, sb) && mul_ok(tokens, st) && batch * sb <= kLim - tokens * st;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Whether [a, a + n) and [b, b + n) overlap without being the same.
bool partly(const void* a, const void* b, size_t n) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p != q && (p < q ? q - p : p - q) < n;
}

// Whether [a, a + na) and [b, b + nb) overlap; absent ones do not.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return a && b && (p < q ? q - p < na : p - q < nb);
}

mamba_status check_shape(const mamba_recurrence_shape* s) {
  if (!s) return MAMBA_ERR_NULL_PTR;
  if (s->dtype != MAMBA_F32 && s->dtype != MAMBA_BF16) return MAMBA_ERR_DTYPE;
  if (s->batch <= 0 || s->seqlen <= 0 || s->dim <= 0) return MAMBA_ERR_SHAPE;
  if (s->x_batch_stride < 0 || s->x_token_stride < 0 || s->r_batch_stride < 0 ||
      s->r_token_stride < 0 || s->i_batch_stride < 0 || s->i_token_stride < 0 ||
      s->z_batch_stride < 0 || s->z_token_stride < 0)
    return MAMBA_ERR_SHAPE;
  if (s->dim > (int64_t)1 << 28 || s->seqlen > kLim / 64 / s->batch ||
      s->dim > kLim / 64 / (s->batch * s->seqlen))
    return MAMBA_ERR_UNSUPPORTED;
  if (!span_ok(s->batch, s->x_batch_stride, s->seqlen, s->x_token_stride) ||
      !span_ok(s->batch, s->r_batch_stride, s->seqlen, s->r_token_stride) ||
      !span_ok(s->batch, s->i_batch_stride, s->seqlen, s->i_token_stride) ||
      !span_ok(s->batch, s->z_batch_stride, s->seqlen, s->z_token_stride))
    return MAMBA_ERR_UNSUPPORTED;
  return MAMBA_OK;
}

// Whether a pass in `tiles` tiles of up to `waves` waves is a legal grid, with the blocks
// that may be without a strip.
bool grid_ok(const mamba_recurrence_shape* s, int64_t tiles, int64_t waves) {
  return s->batch <= mscan::max_blocks((int)(64 * waves)) / 2 /
                         mscan::rec_strips(s->dim, false) / tiles;
}
bool fwd_ok(const mamba_recurrence_shape* s) {
  const int64_t tiles = mscan::rec_fwd_tiles(s->seqlen);
  return grid_ok(s, tiles, tiles > 1 ? mscan::kRecFwdTile / mscan::kRecRun
                                     : (s->seqlen + mscan::kRecRun - 1) / mscan::kRecRun);
}
bool bwd_ok(const mamba_recurrence_shape* s) {
  const int64_t tiles = mscan::rec_bwd_tiles(s->seqlen);
  return grid_ok(s, tiles, tiles > 1 ? mscan::kRecBwdTile / mscan::kRecBwdRun
                                     : (s->seqlen + mscan::kRecBwdRun - 1) / mscan::kRecBwdRun);
}

mamba_status check_inputs(const mamba_recurrence_shape* s, const void* x, const void* r,
                          const void* i, const float* A, const void* z, const float* h0) {
  if (!x || !r || !i || !A) return MAMBA_ERR_NULL_PTR;
  const size_t es = (size_t)esize(s->dtype);
  if (!aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(z, es) ||
      !aligned_f32(A) || !aligned_f32(h0))
    return MAMBA_ERR_ALIGNMENT;
  return MAMBA_OK;
}

// Bytes that a call reads or writes; of an absent tensor p is null.
struct Region {
  const void* p;
  size_t n;
};

// Whether one of the outputs lies over one of the inputs.
bool over_inputs(std::initializer_list<Region> outputs, std::initializer_list<Region> inputs) {
  for (const Region& o : outputs)
    for (const Region& i : inputs)
      if (overlap(o.p, o.n, i.p, i.n)) return true;
  return false;
}

// Whether two of the outputs lie over one another.
bool over_each_other(std::initializer_list<Region> outputs) {
  for (const Region* a = outputs.begin(); a != outputs.end(); ++a)
    for (const Region* b = a + 1; b != outputs.end(); ++b)
      if (overlap(a->p, a->n, b->p, b->n)) return true;
  return false;
}

size_t sequence_bytes(const mamba_recurrence_shape* s) {
  return (size_t)(s->batch * s->seqlen * s->dim) * (size_t)esize(s->dtype);
}

size_t state_bytes(const mamba_recurrence_shape* s) { return (size_t)(s->batch * s->dim) * 4; }

// From the first element of a view of rows to the end of its last.
Region rows(const mamba_recurrence_shape* s, const void* p, int64_t sb, int64_t st) {
  return {p, (size_t)((s->batch - 1) * sb + (s->seqlen - 1) * st + s->dim) *
                 (size_t)esize(s->dtype)};
}

// Whether one of the outputs lies over what every call of the recurrence reads.
bool over_shared(std::initializer_list<Region> outputs, const mamba_recurrence_shape* s,
                 const void* x, const void* r, const void* i, const float* A, const void* z) {
  return over_inputs(outputs, {rows(s, x, s->x_batch_stride, s->x_token_stride),
                               rows(s, r, s->r_batch_stride, s->r_token_stride),
                               rows(s, i, s->i_batch_stride, s->i_token_stride),
                               rows(s, z, s->z_batch_stride, s->z_token_stride),
                               {A, (size_t)s->dim * 4}});
}

int64_t tiles(const mamba_recurrence_shape* s) {
  return (s->seqlen + mscan::kRecTile - 1) / mscan::kRecTile;
}

mscan::RecParams common(const mamba_recurrence_shape* s, const void* x, const void* r,
                        const void* i, const float* A, const void* z, const float* h0,
                        const uint8_t* reset) {
  mscan::RecParams p{};
  p.x = {x, s->x_batch_stride, s->x_token_stride};
  p.r = {r, s->r_batch_stride, s->r_token_stride};
  p.i = {i, s->i_batch_stride, s->i_token_stride};
  p.z = {z, s->z_batch_stride, s->z_token_stride};
  p.A = A; p.h0 = h0; p.reset = reset;
  p.batch = s->batch; p.L = s->seqlen; p.dim = s->dim;
  return p;
}

// Whether bfloat16 rows can be taken in pairs.  One tile a row on fewer blocks than CUs is
// bound by the work of each, and takes single elements (200 steps of 1536 channels 12 us in
// pairs, 9 so); elsewhere pairs halve the loads (131072 x 1536 411 us, 432 without them).
bool pairs(const mamba_recurrence_shape* s, const void* x, const void* r, const void* i,
           const void* z) {
  auto ok = [](const void* p, int64_t sb, int64_t st) {
    return aligned(p, 4) && sb % 2 == 0 && st % 2 == 0;
  };
  const bool few = s->seqlen <= mscan::kRecOneTile && s->batch * mscan::rec_strips(s->dim, true) < 256;
  return s->dtype == MAMBA_BF16 && !few && s->dim % 2 == 0 &&
         ok(x, s->x_batch_stride, s->x_token_stride) &&
         ok(r, s->r_batch_stride, s->r_token_stride) &&
         ok(i, s->i_batch_stride, s->i_token_stride) &&
         (!z || ok(z, s->z_batch_stride, s->z_token_stride));
}

// Workspace of a pass in `n` tiles, none where one tile holds the sequence.
struct ChainLayout {
  size_t maps, heads, total;
};

ChainLayout chain_layout(const mamba_recurrence_shape* s, int64_t n) {
  if (n == 1) return {0, 0, 0};
  const int64_t g = (n + mscan::kRecGroup - 1) / mscan::kRecGroup;
  const size_t row = (size_t)(s->batch * s->dim) * 8;
  ChainLayout l;
  l.maps = (size_t)(s->batch * mscan::rec_strips(s->dim, false)) * mscan::kTicketWords * 4;
  l.heads = l.maps + row * (size_t)n;
  l.total = l.heads + row * (size_t)g;
  return l;
}

ChainLayout fwd_layout(const mamba_recurrence_shape* s) {
  return chain_layout(s, mscan::rec_fwd_tiles(s->seqlen));
}

ChainLayout bwd_chain(const mamba_recurrence_shape* s) {
  return chain_layout(s, mscan::rec_bwd_tiles(s->seqlen));
}

void carve(mscan::RecParams* p, const ChainLayout& l, void* workspace) {
  p->ticket = nullptr;
  if (!l.total) return;
  char* ws = static_cast<char*>(workspace);
  p->ticket = reinterpret_cast<uint32_t*>(ws);
  p->maps = reinterpret_cast<uint64_t*>(ws + l.maps);
  p->heads = reinterpret_cast<uint64_t*>(ws + l.heads);
  p->words = (int64_t)(l.total / 8);
}

// Workspace of the backward.
struct BwdLayout {
  size_t chain, part, ckpt, fwd, total;
};

BwdLayout bwd_layout(const mamba_recurrence_shape* s, bool given) {
  const size_t row = (size_t)(s->batch * s->dim) * 4;
  BwdLayout l;
  l.chain = 0;
  l.part = up256(bwd_chain(s).total);
  l.ckpt = l.part + up256(row * (size_t)mscan::rec_bwd_tiles(s->seqlen));
  l.fwd = l.ckpt + (given ? 0 : up256(row * (size_t)tiles(s)));
  l.total = l.fwd + (given ? 0 : up256(fwd_layout(s).total));
  return l;
}

// Rows of a view: element (b, t, i) at p[b * batch + t * row + i].
struct View {
  const void* p;
  int64_t batch, row;
};

mamba_status check_norm(const View& x, const View& res, const float* weight, int64_t batch,
                        int64_t rows, int64_t dim, float eps, mamba_dtype dt, mamba_dtype rdt,
                        mscan::ResNormKind* kind) {
  if ((dt != MAMBA_F32 && dt != MAMBA_BF16) || (rdt != MAMBA_F32 && rdt != dt))
    return MAMBA_ERR_DTYPE;
  *kind = dt == MAMBA_F32 ? mscan::kResF32 : rdt == MAMBA_F32 ? mscan::kResBf16F32 : mscan::kResBf16;
  if (batch <= 0 || rows <= 0 || dim <= 0 || x.batch < 0 || x.row < 0 || res.batch < 0 || res.row < 0)
    return MAMBA_ERR_SHAPE;
  if (!(eps >= 0.0f)) return MAMBA_ERR_INVALID;
  if (dim > (1 << 28) || rows > kLim / 16 / dim || batch > kLim / 16 / dim / rows ||
      !span_ok(batch, x.batch, rows, x.row) || !span_ok(batch, res.batch, rows, res.row))
    return MAMBA_ERR_UNSUPPORTED;
  if (!x.p) return MAMBA_ERR_NULL_PTR;
  if (!aligned(x.p, (size_t)esize(dt)) || !aligned(res.p, (size_t)esize(rdt)) || !aligned_f32(weight))
    return MAMBA_ERR_ALIGNMENT;
  return MAMBA_OK;
}

// Bytes from the first element to the end of the last row.
size_t span(const View& v, int64_t batch, int64_t rows, int64_t dim, int es) {
  return (size_t)((batch - 1) * v.batch + (rows - 1) * v.row + dim) * (size_t)es;
}

bool one_run(const View& v, int64_t batch, int64_t rows) {
  return !v.p || batch == 1 || v.batch == rows * v.row;
}

// Whether every row starts on 16 bytes.
bool rows16(const View& v, int es) {
  return aligned(v.p, 16) && v.batch % (16 / es) == 0 && v.row % (16 / es) == 0;
}

mamba_status norm_fwd(const View& x, View res, const float* weight, int64_t batch, int64_t rows,
                      int64_t dim, float eps, mamba_dtype dt, mamba_dtype rdt, void* out,
                      float* scale, bool fp8, void* residual_out, void* stream) {
  mscan::ResNormKind kind;
  if (!res.p) res = {nullptr, 0, 0};
  const mamba_status st = check_norm(x, res, weight, batch, rows, dim, eps, dt, rdt, &kind);
  if (st != MAMBA_OK) return st;
  if (!out || (fp8 && !scale) || (res.p && !residual_out)) return MAMBA_ERR_NULL_PTR;
  if (!res.p && residual_out) return MAMBA_ERR_INVALID;
  const int es = esize(dt), er = esize(rdt);
  if ((!fp8 && !aligned(out, (size_t)es)) || !aligned_f32(scale) ||
      !aligned(residual_out, (size_t)er))
    return MAMBA_ERR_ALIGNMENT;
  const size_t n = (size_t)(batch * rows * dim), no = n * (fp8 ? 1 : (size_t)es), nr = n * (size_t)er;
  const size_t sx = span(x, batch, rows, dim, es), sr = span(res, batch, rows, dim, er);
  const Region o = {out, no}, sc = {scale, (size_t)(batch * rows) * 4}, k = {residual_out, nr};
  if (over_inputs({o, sc, k}, {{x.p, sx}, {weight, (size_t)dim * 4}}) ||
      over_inputs({o, sc}, {{res.p, sr}}) || over_each_other({o, sc, k}))
    return MAMBA_ERR_INVALID;
  // the stream is carried in place row on row, or apart
  const bool dense = (rows == 1 || res.row == dim) && (batch == 1 || res.batch == rows * dim);
  if (overlap(residual_out, nr, res.p, sr) && (residual_out != res.p || !dense))
    return MAMBA_ERR_INVALID;
  mscan::ResNormParams p{};
  p.x = x.p; p.x_batch = x.batch; p.x_row = x.row;
  p.res = res.p; p.res_batch = res.batch; p.res_row = res.row;
  p.inner = one_run(x, batch, rows) && one_run(res, batch, rows) ? 0 : rows;
  p.w = weight; p.rows = batch * rows; p.dim = dim; p.eps = eps;
  p.out = out; p.scale = scale; p.res_out = residual_out;
  p.vec = dim % (16 / es) == 0 && rows16(x, es) && (!res.p || rows16(res, er)) &&
          aligned(weight, 16) && aligned(out, fp8 ? (size_t)(16 / es) : 16) &&
          aligned(residual_out, 16);
  return hip_status(mscan::dispatch_res_norm_fwd(p, kind, fp8, as_stream(stream)));
}

}  // namespace

extern "C" {

size_t mamba_gated_recurrence_checkpoint_size(const mamba_recurrence_shape* shape) {
  if (check_shape(shape) != MAMBA_OK || !fwd_ok(shape)) return SIZE_MAX;
  return (size_t)(shape->batch * shape->dim) * (size_t)tiles(shape) * 4;
}

size_t mamba_gated_recurrence_fwd_workspace_size(const mamba_recurrence_shape* shape) {
  return check_shape(shape) == MAMBA_OK && fwd_ok(shape) ? fwd_layout(shape).total : SIZE_MAX;
}

size_t mamba_gated_recurrence_bwd_workspace_size(const mamba_recurrence_shape* shape,
                                                 int with_checkpoints) {
  return check_shape(shape) == MAMBA_OK && bwd_ok(shape) && (with_checkpoints || fwd_ok(shape))
             ? bwd_layout(shape, with_checkpoints != 0).total
             : SIZE_MAX;
}

mamba_status mamba_gated_recurrence_fwd(const mamba_recurrence_shape* shape, const void* x,
                                        const void* r, const void* i, const float* A,
                                        const void* z, const float* h0, const uint8_t* reset,
                                        void* out, float* last_state, float* checkpoints,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  mamba_status st = check_shape(shape);
  if (st != MAMBA_OK) return st;
  st = check_inputs(shape, x, r, i, A, z, h0);
  if (st != MAMBA_OK) return st;
  if (!out) return MAMBA_ERR_NULL_PTR;
  if (!aligned(out, (size_t)esize(shape->dtype)) || !aligned_f32(last_state) ||
      !aligned_f32(checkpoints))
    return MAMBA_ERR_ALIGNMENT;
  if (h0 && last_state && partly(h0, last_state, (size_t)(shape->batch * shape->dim) * 4))
    return MAMBA_ERR_INVALID;
  const size_t need = mamba_gated_recurrence_fwd_workspace_size(shape);
  if (need == SIZE_MAX) return MAMBA_ERR_UNSUPPORTED;
  const size_t seq = sequence_bytes(shape), state = state_bytes(shape);
  const size_t marks = mamba_gated_recurrence_checkpoint_size(shape);
  const Region o = {out, seq}, l = {last_state, state}, c = {checkpoints, marks};
  const Region w = {need ? workspace : nullptr, need};
  const Region flags = {reset, (size_t)(shape->batch * shape->seqlen)};
  if (over_shared({o, l, c}, shape, x, r, i, A, z) || over_inputs({o, l, c}, {flags}) ||
      over_inputs({o, c}, {{h0, state}}) || over_each_other({o, l, c}))
    return MAMBA_ERR_INVALID;
  if (need && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return MAMBA_ERR_ALIGNMENT;
  if (over_shared({w}, shape, x, r, i, A, z) || over_inputs({w}, {flags, {h0, state}, o, l, c}))
    return MAMBA_ERR_INVALID;
  mscan::RecParams p = common(shape, x, r, i, A, z, h0, reset);
  p.out = out; p.last = last_state; p.ckpt = checkpoints;
  p.pairs = pairs(shape, x, r, i, z) && aligned(out, 4);
  carve(&p, fwd_layout(shape), workspace);
  return hip_status(mscan::dispatch_rec_fwd(p, shape->dtype == MAMBA_F32 ? 0 : 1,
                                            as_stream(stream)));
}

mamba_status mamba_gated_recurrence_bwd(const mamba_recurrence_shape* shape, const void* x,
                                        const void* r, const void* i, const float* A,
                                        const void* z, const float* h0, const uint8_t* reset,
                                        const void* dout, const float* dlast_state,
                                        const float* checkpoints, void* dx, void* dr, void* di,
                                        float* dA, void* dz, float* dh0, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  mamba_status st = check_shape(shape);
  if (st != MAMBA_OK) return st;
  st = check_inputs(shape, x, r, i, A, z, h0);
  if (st != MAMBA_OK) return st;
  if (!dout || !dx || !dr || !di || !dA) return MAMBA_ERR_NULL_PTR;
  if ((z != nullptr) != (dz != nullptr) || (dh0 && !h0)) return MAMBA_ERR_INVALID;
  const size_t es = (size_t)esize(shape->dtype);
  if (!aligned(dout, es) || !aligned(dx, es) || !aligned(dr, es) || !aligned(di, es) ||
      !aligned(dz, es) || !aligned_f32(dlast_state) || !aligned_f32(checkpoints) ||
      !aligned_f32(dA) || !aligned_f32(dh0))
    return MAMBA_ERR_ALIGNMENT;
  if (!bwd_ok(shape) || (!checkpoints && !fwd_ok(shape))) return MAMBA_ERR_UNSUPPORTED;
  const size_t seq = sequence_bytes(shape), state = state_bytes(shape);
  const size_t marks = (size_t)(shape->batch * shape->dim) * (size_t)tiles(shape) * 4;
  const Region x_ = {dx, seq}, r_ = {dr, seq}, i_ = {di, seq}, z_ = {dz, seq};
  const Region a_ = {dA, (size_t)shape->dim * 4}, h_ = {dh0, state};
  const Region h = {h0, state}, flags = {reset, (size_t)(shape->batch * shape->seqlen)};
  const Region d = {dout, seq}, l_ = {dlast_state, state}, c = {checkpoints, marks};
  if (over_shared({x_, r_, i_, z_, a_, h_}, shape, x, r, i, A, z) ||
      over_inputs({x_, r_, i_, z_, a_, h_}, {h, flags, d, l_, c}) ||
      over_each_other({x_, r_, i_, z_, a_, h_}))
    return MAMBA_ERR_INVALID;
  const BwdLayout l = bwd_layout(shape, checkpoints != nullptr);
  if (!workspace || workspace_bytes < l.total) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MAMBA_ERR_ALIGNMENT;
  const Region w = {workspace, l.total};
  if (over_shared({w}, shape, x, r, i, A, z) ||
      over_inputs({w}, {h, flags, d, l_, c, x_, r_, i_, z_, a_, h_}))
    return MAMBA_ERR_INVALID;
  mscan::RecParams p = common(shape, x, r, i, A, z, h0, reset);
  char* ws = static_cast<char*>(workspace);
  p.dout = dout; p.dlast = dlast_state;
  p.dx = dx; p.dr = dr; p.di = di; p.dz = dz; p.dA = dA; p.dh0 = dh0;
  p.part = reinterpret_cast<float*>(ws + l.part);
  p.kept = checkpoints;
  if (!checkpoints) {   // the forward's pass over the states alone
    mscan::RecParams f = common(shape, x, r, i, A, nullptr, h0, reset);
    f.pairs = pairs(shape, x, r, i, nullptr);
    f.ckpt = reinterpret_cast<float*>(ws + l.ckpt);
    carve(&f, fwd_layout(shape), ws + l.fwd);
    st = hip_status(mscan::dispatch_rec_fwd(f, shape->dtype == MAMBA_F32 ? 0 : 1, as_stream(stream)));
    if (st != MAMBA_OK) return st;
    p.kept = f.ckpt;
  }
  carve(&p, bwd_chain(shape), ws + l.chain);
  return hip_status(mscan::dispatch_rec_bwd(p, shape->dtype == MAMBA_F32 ? 0 : 1,
                                            as_stream(stream)));
}

mamba_status mamba_gated_recurrence_update(const mamba_recurrence_shape* shape, float* state,
                                           const int32_t* slots, int64_t pool, const void* x,
                                           const void* r, const void* i, const float* A,
                                           const void* z, void* out, void* stream) {
  mamba_status st = check_shape(shape);
  if (st != MAMBA_OK) return st;
  if (shape->seqlen != 1 || pool <= 0 || (!slots && pool < shape->batch)) return MAMBA_ERR_SHAPE;
  if (pool > kLim / 16 / shape->dim || shape->batch > mscan::max_blocks(256) * 256 / shape->dim)
    return MAMBA_ERR_UNSUPPORTED;
  st = check_inputs(shape, x, r, i, A, z, nullptr);
  if (st != MAMBA_OK) return st;
  if (!state || !out) return MAMBA_ERR_NULL_PTR;
  if (!aligned(out, (size_t)esize(shape->dtype)) || !aligned_f32(state) || !aligned(slots, 4))
    return MAMBA_ERR_ALIGNMENT;
  const Region o = {out, sequence_bytes(shape)}, st_ = {state, (size_t)(pool * shape->dim) * 4};
  if (over_shared({o, st_}, shape, x, r, i, A, z) ||
      over_inputs({o, st_}, {{slots, (size_t)shape->batch * 4}}) || over_inputs({o}, {st_}))
    return MAMBA_ERR_INVALID;
  mscan::RecStepParams p{};
  p.x = x; p.r = r; p.i = i; p.z = z;
  p.x_row = shape->x_batch_stride; p.r_row = shape->r_batch_stride;
  p.i_row = shape->i_batch_stride; p.z_row = shape->z_batch_stride;
  p.A = A; p.state = state; p.slots = slots; p.pool = pool;
  p.batch = shape->batch; p.dim = shape->dim; p.out = out;
  const int es = esize(shape->dtype);
  auto four = [&](const void* q, int64_t row) {
    return aligned(q, (size_t)(4 * es)) && row % 4 == 0;
  };
  p.vec = four(x, p.x_row) && four(r, p.r_row) && four(i, p.i_row) && (!z || four(z, p.z_row)) &&
          four(out, p.dim) && aligned(state, 16) && aligned(A, 16);
  return hip_status(mscan::dispatch_rec_step(p, shape->dtype == MAMBA_F32 ? 0 : 1,
                                             as_stream(stream)));
}

mamba_status mamba_residual_norm_fwd(const void* x, int64_t x_batch_stride, int64_t x_row_stride,
                                     const void* residual, int64_t residual_batch_stride,
                                     int64_t residual_row_stride, const float* weight,
                                     int64_t batch, int64_t rows, int64_t dim, float eps,
                                     mamba_dtype dt, mamba_dtype residual_dt, void* out,
                                     void* residual_out, void* stream) {
  return norm_fwd({x, x_batch_stride, x_row_stride},
                  {residual, residual_batch_stride, residual_row_stride}, weight, batch, rows, dim,
                  eps, dt, residual_dt, out, nullptr, false, residual_out, stream);
}

mamba_status mamba_residual_norm_fp8(const void* x, int64_t x_batch_stride, int64_t x_row_stride,
                                     const void* residual, int64_t residual_batch_stride,
                                     int64_t residual_row_stride, const float* weight,
                                     int64_t batch, int64_t rows, int64_t dim, float eps,
                                     mamba_dtype dt, mamba_dtype residual_dt, uint8_t* out8,
                                     float* scale, void* residual_out, void* stream) {
  return norm_fwd({x, x_batch_stride, x_row_stride},
                  {residual, residual_batch_stride, residual_row_stride}, weight, batch, rows, dim,
                  eps, dt, residual_dt, out8, scale, true, residual_out, stream);
}

size_t mamba_residual_norm_bwd_workspace_size(int64_t rows, int64_t dim) {
  static const float dummy[4] = {};
  mscan::ResNormKind kind;
  if (check_norm({dummy, 0, 0}, {dummy, 0, 0}, nullptr, 1, rows, dim, 0.0f, MAMBA_F32, MAMBA_F32,
                 &kind) != MAMBA_OK)
    return SIZE_MAX;
  return up256((size_t)mscan::res_norm_parts(rows) * (size_t)dim * 4);
}

mamba_status mamba_residual_norm_bwd(const void* res, int64_t res_batch_stride,
                                     int64_t res_row_stride, const float* weight,
                                     const void* dout, const void* dres, int64_t batch,
                                     int64_t rows, int64_t dim, float eps, mamba_dtype dt,
                                     mamba_dtype residual_dt, void* dx, void* dresidual,
                                     float* dweight, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  mscan::ResNormKind kind;
  const View r = {res, res_batch_stride, res_row_stride};
  const mamba_status st =
      check_norm({dout, 0, 0}, r, weight, batch, rows, dim, eps, dt, residual_dt, &kind);
  if (st != MAMBA_OK) return st;
  if (!res || !dx) return MAMBA_ERR_NULL_PTR;
  if ((weight != nullptr) != (dweight != nullptr) || (dresidual && residual_dt == dt))
    return MAMBA_ERR_INVALID;
  const int es = esize(dt), er = esize(residual_dt);
  if (!aligned(dres, (size_t)er) || !aligned(dx, (size_t)es) || !aligned(dresidual, (size_t)er) ||
      !aligned_f32(dweight))
    return MAMBA_ERR_ALIGNMENT;
  const size_t n = (size_t)(batch * rows * dim), sr = span(r, batch, rows, dim, er);
  const size_t wide = (size_t)dim * 4;
  const Region x_ = {dx, n * (size_t)es}, r_ = {dresidual, n * (size_t)er}, w_ = {dweight, wide};
  const Region in = {res, sr}, g = {weight, wide}, d = {dout, n * (size_t)es}, s = {dres, n * (size_t)er};
  if (over_inputs({x_, r_, w_}, {in, g, d, s}) || over_each_other({x_, r_, w_}))
    return MAMBA_ERR_INVALID;
  const size_t need = mamba_residual_norm_bwd_workspace_size(batch * rows, dim);
  if (need == SIZE_MAX) return MAMBA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MAMBA_ERR_ALIGNMENT;
  if (over_inputs({{workspace, need}}, {in, g, d, s, x_, r_, w_})) return MAMBA_ERR_INVALID;
  mscan::ResNormParams p{};
  p.res = res; p.res_batch = r.batch; p.res_row = r.row;
  p.inner = one_run(r, batch, rows) ? 0 : rows;
  p.w = weight; p.rows = batch * rows; p.dim = dim; p.eps = eps;
  p.dout = dout; p.dres = dres; p.dx = dx; p.dresidual = dresidual; p.dw = dweight;
  p.part = static_cast<float*>(workspace);
  p.parts = mscan::res_norm_parts(p.rows);
  p.vec = dim % (16 / es) == 0 && rows16(r, er) && aligned(dout, 16) && aligned(dres, 16) &&
          aligned(weight, 16) && aligned(dx, 16) && aligned(dresidual, 16);
  return hip_status(mscan::dispatch_res_norm_bwd(p, kind, as_stream(stream)));
}

}  // extern "C"
