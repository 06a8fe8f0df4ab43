// Backward of the multi-head scan.  With the adjoint g of the state (what
// everything after a step makes of it),
//   du_s = w_s g_s B_s + D dout_s,  dB_s = w_s g_s^T u_s,  dC_q = h_q^T dout_q,
//   dw_s = u_s . (g_s B_s),  F_t = <a_t g_t, h_{t-1}>, the gradient of the log decay.
// Within a chunk, with the entering state h, the adjoint g behind its end, the
// decays L_qs = e^{S_q - S_s}, r_s to the chunk's end and e_q from its start:
//   g_s B_s  = sum_{q >= s} L_qs (C_q . B_s) dout_q + r_s g B_s
//   g_s^T u_s = sum_{q >= s} L_qs (dout_q . u_s) C_q + r_s g^T u_s
//   dC_q     = sum_{s <= q} L_qs w_s (dout_q . u_s) B_s + e_q h^T dout_q
//   F_t = dec <g, h> + sum_{q >= t} e_q dout_q . (h C_q) + sum_{s < t} w_s r_s u_s . (g B_s)
//         + sum_{s < t <= q} K_qs,   K_qs = L_qs w_s (C_q . B_s)(dout_q . u_s):
// the paths through step t from before the chunk or inside it to inside or
// behind it.  Summing whole rows and taking differences over the sequence
// instead would lose F to cancellation.
//
// Passes: the chunks' scalars; the states at every chunk's start and the
// adjoints behind every chunk's end (segments of the sequence in parallel from
// zero, then their carries); the chunks, all independent, each block looping
// over heads with dB and dC in registers; sums over the blocks' shares.
//
// 2 x 2048 tokens, 80 heads of 64, N = 128, bfloat16: 319 us in all.  Bound by the
// states (335 MB written, then read) and by the phases of the chunks.  In bfloat16 the
// states are multiplied in two parts for dB and dC (rounded once, up to 1.46 times the
// error of the results' own rounding; now 1.0, for 5 % of the time).
#include <type_traits>

#include "heads_mma.hpp"

namespace mscan {

namespace {

template <typename T, int NK>
struct BwdTiles {
  static constexpr int Q = Mx<T>::Q, PAD = Mx<T>::PAD, PADT = Mx<T>::PADT;
  static constexpr int NP = 32 * NK, QT = Q / 16;
  static constexpr int PARTS = Mx<T>::PARTS;
  static constexpr int SX = 64 + PAD, SN = NP + PAD, SM = Q + PAD;
  // region that holds a head's states, then its two matrices
  static constexpr int ZSTATE = 64 * SN, ZM = 2 * Q * SM;
  static constexpr int Z = ZSTATE > ZM ? ZSTATE : ZM;
};

// ---------------------------------------------------------------------------
// States at the chunks' starts (REV false: keys B, inputs u) or adjoints behind
// their ends (REV true: keys C, inputs dout), from zero within a segment; pre:
// the weight in them of the segment's entering state or adjoint.
// ---------------------------------------------------------------------------
template <typename T, int NK, bool VEC, bool REV>
__device__ __forceinline__ void states_of(const HeadsBwdParams& p, int block, T* Xs, T* Ks,
                                          Scal<Mx<T>::Q>* scal) {
  using F = BwdTiles<T, NK>;
  constexpr int Q = F::Q, NP = F::NP, SX = kCols + F::PADT, SN = NP + F::PADT;
  const Place k = place_at(p, p.nseg, block);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t begin = (int64_t)k.seg * p.seg_len;
  const int64_t end = k.seg + 1 == p.nseg ? p.L : begin + p.seg_len;
  const int64_t ucol = (int64_t)k.h0 * p.P, ncols = (int64_t)k.g * p.N;
  const int uwidth = (k.h0 + k.heads) * p.P, nwidth = (k.g + 1) * p.N;
  const int sub = p.slices * kSlice, hh = wave / p.slices;
  const int64_t chunks = (p.L + Q - 1) / Q;
  const Rows vals = REV ? Rows{p.dout, p.L * p.H * p.P, (int64_t)p.H * p.P} : p.u;
  const Rows keys = REV ? p.C : p.B;
  f32x4 h[2 * NK][2];
  fill<NK>(h, 0.0f);
  float pre = 1.0f;
  Stage<T, Q, kCols, VEC> sx;
  Stage<T, Q, NP, VEC> sk;
  ScalStage<Q> ss;
  sx.init(vals, ucol, sub, p.P, p.P, k.heads);
  sk.init(keys, ncols, NP, 0, p.N, 1);
  auto fetch = [&](int64_t t) {
    const int len = end - t < Q ? (int)(end - t) : Q;
    ss.load(p.scal, (k.b * chunks + t / Q) * p.H + k.h0, k.heads);
    sx.load(vals, k.b, t, len, ucol, p.P, uwidth);
    sk.load(keys, k.b, t, len, ncols, 0, nwidth);
  };
  const int64_t n = (end - begin + Q - 1) / Q;
  auto at = [&](int64_t i) { return begin + (REV ? n - 1 - i : i) * Q; };
  fetch(at(0));
  for (int64_t i = 0; i < n; ++i) {
    sx.store(Xs, SX);
    sk.store(Ks, SN);
    ss.store(scal, k.heads);
    __syncthreads();
    if (i + 1 < n) fetch(at(i + 1));
    const Scal<Q>& me = scal[k.on ? hh : 0];
    if (scal[0].flags != 0) {
      clear_kept<T, Q, NP>(Ks, SN, scal[0].id, REV ? 0 : scal[0].flags);
      __syncthreads();
    }
    if (k.on) {
      const int64_t c = (k.b * chunks + at(i) / Q) * p.H + k.h;
      float* st = (REV ? p.g_chunk : p.h_chunk) + (c * p.slices + k.slice) * slice_floats<NK>();
      store_frags<NK>(st, h);
      if (k.slice == 0 && (threadIdx.x & 63) == 0) (REV ? p.g_pre : p.h_pre)[c] = pre;
      uint64_t marks[2] = {0, 0};
      if (tile_odd<T, Q>(Xs, SX, k.col)) {
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
          marks[pt] = take_out<T, Q>(Xs, SX, k.col + 16 * pt + lane_i());
      }
      step_state<T, NK>(h, me.dec, REV ? me.e : me.c, Ks, SN, Xs, SX, k.col);
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
        if (marks[pt] != 0 && marked<Q>(marks[pt], me.id, REV ? 0 : me.flags)) spoil<NK>(h, pt);
      pre = join(pre, me.dec);
    }
    __syncthreads();
  }
  if (!k.on) return;
  const int64_t slot = slice_slot(p, k, p.nseg, k.seg);
  store_frags<NK>((REV ? p.g_seg : p.h_seg) + slot * slice_floats<NK>(), h);
  if ((threadIdx.x & 63) == 0) (REV ? p.g_dec : p.h_dec)[slot] = pre;
}

// Both directions in one launch, the update of the forward's pass; the state in
// registers is written at every chunk: 100 us of the 319 (357 MB at 3.6 TB/s).
template <typename T, int NK, bool VEC>
__global__ __launch_bounds__(256, NK == 8 ? 1 : 2) void heads_states_kernel(const HeadsBwdParams p) {
  using F = BwdTiles<T, NK>;
  __shared__ __align__(16) T Xs[F::Q * (kCols + F::PADT)];
  __shared__ __align__(16) T Ks[F::Q * (F::NP + F::PADT)];
  extern __shared__ __align__(16) char dyn[];
  Scal<F::Q>* const scal = reinterpret_cast<Scal<F::Q>*>(dyn);
  // both directions in one launch
  const int half = gridDim.x / 2;
  if ((int)blockIdx.x < half) states_of<T, NK, VEC, false>(p, (int)blockIdx.x, Xs, Ks, scal);
  else states_of<T, NK, VEC, true>(p, (int)blockIdx.x - half, Xs, Ks, scal);
}

// The chunks leave out an entering state whose weight is 0, blocked or underflowed
// (8 us of 328).  A non-finite one must still reach them: the underflowed weights of
// its segment become the least float above 0.  Blocks of one head may write the same
// weight, all of them this value.
template <bool REV>
__device__ __forceinline__ void let_pass(const HeadsBwdParams& p, int64_t bh, int seg) {
  const int64_t b = bh / p.H, h = bh - b * p.H;
  const int64_t q = p.chunk, chunks = (p.L + q - 1) / q, per = p.seg_len / q;
  const int64_t end = (seg + 1) * per < chunks ? (seg + 1) * per : chunks;
  float* const pre = (REV ? p.g_pre : p.h_pre) + b * chunks * p.H + h;
  for (int64_t c = seg * per + (threadIdx.x & 63); c < end; c += 64)
    if (__float_as_uint(pre[c * p.H]) == 0) pre[c * p.H] = __uint_as_float(1);
}

// What enters each segment, in place of what the one before left: states from
// h0 on, or adjoints from the last state's gradient back, and dh0 behind them.
template <int NK, bool REV>
__device__ __forceinline__ void carry_of(const HeadsBwdParams& p, int64_t block) {
  constexpr int PER = NK;
  const int64_t id = block / PER;
  const int e = (int)(block - id * PER) * 256 + threadIdx.x;
  const int slice = (int)(id % p.slices);
  const int64_t bh = id / p.slices;
  const int nt = e >> 7, pt = (e >> 6) & 1, l = e & 63;
  const int pp = slice * kSlice + 16 * pt + (l & 15), n = 16 * nt + 4 * (l >> 4);
  const float* first = REV ? p.dlast : p.h0;
  f32x4 h = {0.0f, 0.0f, 0.0f, 0.0f};
  if (first && pp < p.P)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < p.N) h[j] = first[(bh * p.P + pp) * p.N + n + j];
  f32x4* st = reinterpret_cast<f32x4*>((REV ? p.g_seg : p.h_seg) + id * p.nseg * slice_floats<NK>()) + e;
  const float* dec = (REV ? p.g_dec : p.h_dec) + id * p.nseg;
  constexpr int64_t STEP = slice_floats<NK>() / 4;
#pragma unroll 4
  for (int i = 0; i < p.nseg; ++i) {
    const int k = REV ? p.nseg - 1 - i : i;
    const f32x4 s = st[k * STEP];
    const float d = dec[k];
    st[k * STEP] = h;
    if (__any(not_finite(h[0]) || not_finite(h[1]) || not_finite(h[2]) || not_finite(h[3])))
      let_pass<REV>(p, bh, k);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = weigh(h[j], d) + s[j];
  }
  if (REV && p.dh0 && pp < p.P)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < p.N) p.dh0[(bh * p.P + pp) * p.N + n + j] = h[j];
}

// Two segments of 2 x 80 heads, both ways: 7 us, trips to memory.
template <int NK>
__global__ __launch_bounds__(256) void heads_bwd_carry_kernel(const HeadsBwdParams p) {
  const int half = gridDim.x / 2;
  if ((int)blockIdx.x < half) carry_of<NK, false>(p, blockIdx.x);
  else carry_of<NK, true>(p, (int64_t)blockIdx.x - half);
}

// ---------------------------------------------------------------------------
// The chunks.
// ---------------------------------------------------------------------------
// Sums over the lanes of equal column (g = 0..3), in all of them.
__device__ __forceinline__ float sum_g(float v) {
  v = rs_pair16(v, v);
  return rs_pair32(v, v);
}
// Sum over the wave, in the last lane of every 16.
__device__ __forceinline__ float sum_wave(float v) { return sum_g(row_sum_to_last(v)); }

// Inclusive sums over the lanes, in order.
__device__ __forceinline__ float prefix(float v) {
  v += dpp_mov<kRowShr1>(0.0f, v);
  v += dpp_mov<kRowShr2>(0.0f, v);
  v += dpp_mov<kRowShr4>(0.0f, v);
  v += dpp_mov<kRowShr8>(0.0f, v);
  v += dpp_mov<kRowBcast15, 0xA>(0.0f, v);
  v += dpp_mov<kRowBcast31, 0xC>(0.0f, v);
  return v;
}

// The same over the 16 lanes of a row, and from its end.
enum : int { kRowShl1 = 0x101, kRowShl2 = 0x102, kRowShl4 = 0x104, kRowShl8 = 0x108 };
__device__ __forceinline__ float prefix16(float v) {
  v += dpp_mov<kRowShr1>(0.0f, v);
  v += dpp_mov<kRowShr2>(0.0f, v);
  v += dpp_mov<kRowShr4>(0.0f, v);
  v += dpp_mov<kRowShr8>(0.0f, v);
  return v;
}
__device__ __forceinline__ float suffix16(float v) {
  v += dpp_mov<kRowShl1>(0.0f, v);
  v += dpp_mov<kRowShl2>(0.0f, v);
  v += dpp_mov<kRowShl4>(0.0f, v);
  v += dpp_mov<kRowShl8>(0.0f, v);
  return v;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// Four consecutive elements of a tile as floats.
template <typename T>
__device__ __forceinline__ f32x4 four(const T* q) {
  if constexpr (sizeof(T) == 2) {
    const u32x2 u = *reinterpret_cast<const u32x2*>(q);
    return f32x4{bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1])};
  } else {
    return *reinterpret_cast<const f32x4*>(q);
  }
}
template <typename T>
__device__ __forceinline__ void put4(T* q, const f32x4& v) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<u32x2*>(q) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  else
    *reinterpret_cast<f32x4*>(q) = v;
}

template <int Q>
struct alignas(16) BwdSums {
  float row[Q / 16][Q];   // by tile of s: sum over s < q of K_qs
  float col[Q / 16][Q];   // by tile of q: sum over q > s of K_qs / w_s
  float diag[Q];          // K_ss / w_s
  float in[4][Q];         // by wave: u_s . (g B_s)
  float out[4][Q];        // by wave: dout_q . (h C_q)
  float gh[4], ud[4];     // by wave: <g, h>, sum of u dout
};

// Heads a block takes side by side, 4 waves each.  With two, a wave holds half
// of dB and dC and keeps its registers (2 x 2048 x 80 x 64, N = 128: 207 us when tried, one
// head 244).  N <= 64 has a tile of dB and dC for 4 waves at most, and two blocks
// of one head fit a CU (4 x 777 x 16 in float32: 112 -> 100 us; 2 x 2048 x 80 in
// bfloat16: 210 -> 201); N > 128 leaves LDS for one.
template <int NK>
constexpr int kSide = chunk_sides(NK);

// One chunk, its heads in turn: 205 us of the 319, 20 us a pair of heads, of which
// the matrix units are busy 3.5 and VALU is issued for 8; the waits for the next states (up to 3) and the
// phases between barriers, one block a CU, are the rest.
template <typename T, int NK, bool VEC>
__global__ __launch_bounds__(256 * kSide<NK>, NK == 8 ? 1 : 2)
void heads_chunk_kernel(const HeadsBwdParams p) {
  using F = BwdTiles<T, NK>;
  constexpr int Q = F::Q, NP = F::NP, QT = F::QT, SX = F::SX, SN = F::SN, SM = F::SM;
  constexpr int PARTS = F::PARTS, SIDE = kSide<NK>, WAVES = 4 * SIDE;
  constexpr int NTW = 2 * NK > WAVES ? 2 * NK / WAVES : 1;   // tiles of dB, dC a wave
  constexpr int ZP = PARTS == 1 ? 2 : PARTS;   // parts of a state, of a chunk's matrix
  __shared__ __align__(16) T Bs[Q * SN];
  __shared__ __align__(16) T Cs[Q * SN];
  __shared__ __align__(16) T Xall[SIDE][Q * SX];
  __shared__ __align__(16) T Yall[SIDE][Q * SX];   // dout
  __shared__ __align__(16) T Zall[SIDE][F::Z];     // g, then h, then the matrices
  // in bfloat16 the states' low parts, then the second matrix's
  constexpr int LSIZE = F::ZSTATE > Q * SM ? F::ZSTATE : Q * SM;
  __shared__ __align__(16) T Lall[PARTS == 1 ? SIDE : 1][PARTS == 1 ? LSIZE : 8];
  __shared__ Scal<Q> scall[SIDE];
  __shared__ BwdSums<Q> sums_all[SIDE];
  __shared__ int odd_all[WAVES];
  const int wave8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int side = wave8 >> 2, wave = wave8 & 3;
  const int lane = threadIdx.x & 63, li = lane_i(), lg = 4 * lane_g();
  T* const Xs = Xall[side];
  T* const Ys = Yall[side];
  T* const Zs = Zall[side];
  Scal<Q>* const sc = &scall[side];
  BwdSums<Q>& sums = sums_all[side];
  const int64_t chunks = (p.L + Q - 1) / Q;
  // blocks: split, chunk, group, batch row
  int id = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int split = id % p.splits;
  id /= p.splits;
  const int64_t chunk = id % (int)chunks;
  id /= (int)chunks;
  const int grp = id % p.G;
  const int64_t b = id / p.G;
  const int64_t t0 = chunk * Q;
  const int len = p.L - t0 < Q ? (int)(p.L - t0) : Q;
  const int seg = (int)(t0 / p.seg_len);
  const int per = p.H / p.G, CB = (p.P + 63) / 64;
  const int units = per * CB;                      // (head, 64 columns)
  const int u0 = (int)((int64_t)units * split / p.splits);
  const int u1 = (int)((int64_t)units * (split + 1) / p.splits);
  const int64_t row = (int64_t)p.H * p.P;
  const T* const ub = static_cast<const T*>(p.u.p) + b * p.u.batch + t0 * p.u.token;
  const T* const yb = static_cast<const T*>(p.dout) + (b * p.L + t0) * row;
  const int64_t ch0 = (b * chunks + chunk) * p.H;

  Stage<T, Q, 64, VEC> sx, sy;
  ScalStage<Q, 1> ss;
  f32x4 g[2 * NK], h[2 * NK];
  auto head_of = [&](int u) { return grp * per + (CB == 1 ? u : u / CB); };
  // the side's unit, its last one again where there is none: nothing of that is kept
  auto mine = [&](int u) { return u + side < u1 ? u + side : u1 - 1; };
  auto fetch = [&](int u) {
    const int hd = head_of(u), c0 = (u % CB) * 64;
    const int n = p.P - c0 < 64 ? p.P - c0 : 64;
    const int64_t at = (int64_t)hd * p.P + c0;
    ss.load(p.scal, ch0 + hd, 1);
    sx.load_at(ub + at, p.u.token, len, n);
    sy.load_at(yb + at, row, len, n);
  };
  // A wave's 16 columns of a state: half of a slice.
  auto slice_of = [&](int u) { return (u % CB) * 2 + (wave >> 1); };
  auto fetch_state = [&](const float* base, int u, f32x4 (&r)[2 * NK]) {
    if (slice_of(u) < p.slices) {
      const float* st = base + ((ch0 + head_of(u)) * p.slices + slice_of(u)) * slice_floats<NK>() +
                        frag_at<NK>(0, wave & 1, 0);
      const uint32_t o = 4u * (uint32_t)(opaque_int((int)threadIdx.x) & 63);
#pragma unroll
      for (int nt = 0; nt < 2 * NK; ++nt)
        r[nt] = *reinterpret_cast<const f32x4*>(st + o + frag_at<NK>(nt, 0, 0));
    } else {
#pragma unroll
      for (int nt = 0; nt < 2 * NK; ++nt) r[nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  // adds the segment's entering state or adjoint, unless its weight is nothing
  auto add_entering = [&](const float* base, float pre, int u, f32x4 (&r)[2 * NK]) {
    if (pre != 0.0f && slice_of(u) < p.slices) {
      const float* st = base + (((b * p.H + head_of(u)) * p.slices + slice_of(u)) * (int64_t)p.nseg + seg) *
                                   slice_floats<NK>() + frag_at<NK>(0, wave & 1, 0);
      const uint32_t o = 4u * (uint32_t)(opaque_int((int)threadIdx.x) & 63);
#pragma unroll
      for (int nt = 0; nt < 2 * NK; ++nt) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(st + o + frag_at<NK>(nt, 0, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) r[nt][j] = __builtin_fmaf(pre, x[j], r[nt][j]);
      }
    }
  };
  const int flags = static_cast<const Scal<Q>*>(p.scal)[ch0 + head_of(u0)].flags;   // the batch row's
  const bool flagged = flags != 0;
  const bool enters = seg > 0 || p.h0 != nullptr;
  const bool enters_back = seg + 1 < p.nseg || p.dlast != nullptr;

  const T* const kb = static_cast<const T*>(p.B.p) + b * p.B.batch + t0 * p.B.token + (int64_t)grp * p.N;
  const T* const kc = static_cast<const T*>(p.C.p) + b * p.C.batch + t0 * p.C.token + (int64_t)grp * p.N;
  bool keys_odd = false;
  {
    Stage<T, Q, NP, VEC> sb;
    if (SIDE == 1 || side == 0) {
      sb.load_at(kb, p.B.token, len, p.N);
      sb.store(Bs, SN);
      if (flagged) keys_odd = sb.odd();
    }
    if (SIDE == 1 || side == 1) {
      sb.load_at(kc, p.C.token, len, p.N);
      sb.store(Cs, SN);
      if (flagged) keys_odd = sb.odd() || keys_odd;
    }
  }
  keys_odd = __any(keys_odd);
  fetch(mine(u0));
  fetch_state(p.g_chunk, mine(u0), g);
  fetch_state(p.h_chunk, mine(u0), h);
  __syncthreads();

  // C_q . B_s (rows q, columns s): the diagonal tile of the wave and up to two
  // below it, the same for all heads
  constexpr int OFF = QT == 4 ? 2 : 1;
  int qt[1 + OFF], st[1 + OFF];
  bool on[1 + OFF];
  on[0] = wave < QT;
  qt[0] = st[0] = on[0] ? wave : 0;
  if constexpr (QT == 4) {
    qt[1] = wave < 3 ? 3 : 1;
    st[1] = wave < 3 ? wave : 0;
    on[1] = true;
    qt[2] = 2;
    st[2] = wave & 1;
    on[2] = wave < 2;
  } else {
    qt[1] = 1;
    st[1] = 0;
    on[1] = wave == 2;
  }
  f32x4 cb[1 + OFF][1][1];
#pragma unroll
  for (int i = 0; i <= OFF; ++i) cb[i][0][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int kk = 0; kk < NK; ++kk)
#pragma unroll
    for (int i = 0; i <= OFF; ++i) {
      const Frag<PARTS> cf[1] = {load_rows<T>(Cs, SN, 16 * qt[i], 32 * kk)};
      const Frag<PARTS> bf[1] = {load_rows<T>(Bs, SN, 16 * st[i], 32 * kk)};
      mma(cb[i], cf, bf);
    }

  // dB, dC (rows n, columns tokens) of the wave's state tiles, all heads
  const bool has_n = wave8 * NTW < 2 * NK;
  const int n0 = has_n ? 16 * wave8 * NTW : 0;
  f32x4 dB[NTW][QT], dC[NTW][QT];
#pragma unroll
  for (int i = 0; i < NTW; ++i)
#pragma unroll
    for (int j = 0; j < QT; ++j) dB[i][j] = dC[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // acc += f Z^T tile^T of every side's unit (rows n, columns tokens), weighted
  // by token: what reaches dB from behind the chunk, dC from before it
  auto inter = [&](int u, const T (*tiles)[Q * SX], bool second, f32x4 (&acc)[NTW][QT]) {
#pragma unroll
    for (int x = 0; x < SIDE; ++x) {
      if (u + x >= u1) break;
      const Lane ln = lane_fresh();
      const int li = ln.i;
      f32x4 t[NTW][QT];
#pragma unroll
      for (int i = 0; i < NTW; ++i)
#pragma unroll
        for (int j = 0; j < QT; ++j) t[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        Frag<ZP> zf[NTW];
        Frag<PARTS> xf[QT];
#pragma unroll
        for (int i = 0; i < NTW; ++i) {
          if constexpr (PARTS == 1) {
            zf[i].v[0] = load_cols<T>(Zall[x] + n0, SN, 16 * i, 32 * kk, ln).v[0];
            zf[i].v[1] = load_cols<T>(Lall[x] + n0, SN, 16 * i, 32 * kk, ln).v[0];
          } else {
            zf[i] = load_cols<T>(Zall[x] + n0, SN, 16 * i, 32 * kk, ln);
          }
        }
#pragma unroll
        for (int j = 0; j < QT; ++j) xf[j] = load_rows<T>(tiles[x], SX, 16 * j, 32 * kk, ln);
        phase();
        mma(t, zf, xf);
      }
      if (flagged) {
#pragma unroll
        for (int j = 0; j < QT; ++j) {
          const bool off = blocked(second ? scall[x].e[16 * j + li] : scall[x].c[16 * j + li]);
#pragma unroll
          for (int i = 0; i < NTW; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[i][j][e] = off ? 0.0f : t[i][j][e];
        }
      }
#pragma unroll
      for (int j = 0; j < QT; ++j) {
        const float f = second ? scall[x].e[16 * j + li] : scall[x].c[16 * j + li];
#pragma unroll
        for (int i = 0; i < NTW; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(f, t[i][j][e], acc[i][j][e]);
      }
      phase();
    }
  };
  // acc = state fragments (rows p) times tile rows (columns), three exact parts
  auto project = [&](const f32x4 (&r)[2 * NK], const T* tile, f32x4 (&acc)[1][QT]) {
#pragma unroll
    for (int j = 0; j < QT; ++j) acc[0][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const Lane ln = lane_fresh();
    Frag<PARTS> bf[2][QT];
#pragma unroll
    for (int j = 0; j < QT; ++j) bf[0][j] = load_rows<T>(tile, SN, 16 * j, 0, ln);
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      if (kk + 1 < NK) {
#pragma unroll
        for (int j = 0; j < QT; ++j)
          bf[(kk + 1) & 1][j] = load_rows<T>(tile, SN, 16 * j, 32 * kk + 32, ln);
      }
      const Frag<3> rf[1] = {acc_frag<3>(r[2 * kk], r[2 * kk + 1])};
      phase();
      mma(acc, rf, bf[kk & 1]);
    }
  };
  // a state's tile, rows p
  auto put_state = [&](const f32x4 (&r)[2 * NK]) {
    const Lane ln = lane_fresh();
    const int o = 16 * wave * SN + ln.i * SN + 4 * ln.g;
#pragma unroll
    for (int nt = 0; nt < 2 * NK; ++nt) {
      if constexpr (PARTS == 1) {
        // rounded, not cut as in project(): the compiler would keep the rests for both
        const f32x4& v = r[nt];
        const u32x2 hi = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        *reinterpret_cast<u32x2*>(Zs + o + 16 * nt) = hi;
        *reinterpret_cast<u32x2*>(Lall[side] + o + 16 * nt) =
            u32x2{pack_bf16(v[0] - bf16_lo(hi[0]), v[1] - bf16_hi(hi[0])),
                  pack_bf16(v[2] - bf16_lo(hi[1]), v[3] - bf16_hi(hi[1]))};
      } else {
        put4<T>(Zs + o + 16 * nt, r[nt]);
      }
    }
  };

  // B and C of sequence number n of the chunk alone, zeros for the others' rows; of
  // all for n < 0.  Element by element: seldom used.
  auto copy_keys = [&](int n) {
#pragma unroll 1
    for (int i = opaque_int((int)threadIdx.x); i < Q * NP; i += 256 * SIDE) {
      const int r = i / NP, c = i - r * NP;
      const bool keep = r < len && c < p.N && (n < 0 || scall[0].id[r] == n);
      Bs[r * SN + c] = keep ? kb[r * p.B.token + c] : T(0);
      Cs[r * SN + c] = keep ? kc[r * p.C.token + c] : T(0);
    }
  };

  // Where a chunk with flags holds an infinity or NaN the products would carry it
  // into the other sequences' rows: such a chunk's sequences are taken one by one,
  // the others' rows zero and their weights blocked.
  int pass = 0;
  for (int u = u0; u < u1;) {
    const int mu = mine(u);
    const bool live = u + side < u1;
    const int hd = head_of(mu), c0 = (mu % CB) * 64;
    const float D = p.D ? p.D[hd] : 0.0f;
    if (enters_back) add_entering(p.g_seg, p.g_pre[ch0 + hd], mu, g);
    if (enters) add_entering(p.h_seg, p.h_pre[ch0 + hd], mu, h);
    float gh = 0.0f;    // <g, h>
#pragma unroll
    for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) gh = __builtin_fmaf(g[nt][j], h[nt][j], gh);
    if (flagged) {
      const int odd = __any(keys_odd || sx.odd() || sy.odd() || ss.odd() || not_finite(gh));
      if ((opaque_int((int)threadIdx.x) & 63) == 0) odd_all[wave8] = odd;
    }
    sx.store(Xs, SX);
    sy.store(Ys, SX);
    ss.store(sc, 1);
    __syncthreads();
    if (u + SIDE < u1) fetch(mine(u + SIDE));
    bool odd = false;
    if (flagged) {
#pragma unroll
      for (int i = 0; i < WAVES; ++i) odd = odd || odd_all[i] != 0;
      odd = __builtin_amdgcn_readfirstlane(odd);
    }
    if (odd) {
      const int t = opaque_int(tid256());
#pragma unroll 1
      for (int i = t; i < Q * 64; i += 256)
        if (sc->id[i / 64] != pass) Xs[i / 64 * SX + i % 64] = Ys[i / 64 * SX + i % 64] = T(0);
      if (t < Q && sc->id[t] != pass) {
        sc->e[t] = sc->c[t] = sc->r[t] = kBlocked;
        sc->S[t] = sc->g[t] = sc->w[t] = 0.0f;
      }
      copy_keys(pass);
      if (pass < flags) fetch(mu);    // once more, for the next sequence
      __syncthreads();
    }
    const bool again = odd && pass < flags;
    const int next = again ? u : u + SIDE;
    const bool more = next < u1;
    put_state(g);    // for dB
    // (g B_s)^T (rows p, columns s)
    f32x4 du[1][QT];
    project(g, Bs, du);
    float ud = 0.0f;
    {
    const Lane ln = lane_fresh();
    const int li = ln.i, lg = 4 * ln.g, lane = li + 16 * ln.g;
#pragma unroll
    for (int s = 0; s < QT; ++s) {
      const f32x4 x = four<T>(Xs + (16 * s + li) * SX + 16 * wave + lg);
      const f32x4 y = four<T>(Ys + (16 * s + li) * SX + 16 * wave + lg);
      float v = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v = __builtin_fmaf(x[j], du[0][s][j], v);
        ud = __builtin_fmaf(x[j], y[j], ud);
      }
      v = sum_g(v);
      if (lane < 16) sums.in[wave][16 * s + li] = v;
      const float r = sc->r[16 * s + li];
#pragma unroll
      for (int j = 0; j < 4; ++j) du[0][s][j] = weigh(du[0][s][j], r);
    }
    gh = sum_wave(gh);
    ud = sum_wave(ud);
    if (lane == 15) {
      sums.gh[wave] = gh;
      sums.ud[wave] = ud;
    }
    }
    phase();
    // (h C_q)^T (rows p, columns q)
    auto from_before = [&]() {
      f32x4 y[1][QT];
      project(h, Cs, y);
    const Lane ln = lane_fresh();
    const int li = ln.i, lg = 4 * ln.g, lane = li + 16 * ln.g;

#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const f32x4 d = four<T>(Ys + (16 * q + li) * SX + 16 * wave + lg);
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) v = __builtin_fmaf(d[j], y[0][q][j], v);
        v = sum_g(v);
        if (lane < 16) sums.out[wave][16 * q + li] = v;
      }
    };
    if constexpr (PARTS == 1) from_before();
    // dout_q . u_s, and from it K's sums and the two matrices of the chunk
    u32x2 lg_hi[1 + OFF], lg_lo[1 + OFF], lr_hi[1 + OFF], lr_lo[1 + OFF];   // bfloat16, packed
    f32x4 lg_f[1 + OFF], lr_f[1 + OFF];                     // float32
    {
    const Lane ln = lane_fresh();
    const int li = ln.i, lg = 4 * ln.g, lane = li + 16 * ln.g;
      f32x4 a[1 + OFF][1][1];
      Frag<PARTS> yf[2][1 + OFF][1], xf[2][1 + OFF][1];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i <= OFF; ++i) {
          a[i][0][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          yf[kk][i][0] = load_rows<T>(Ys + 16 * qt[i] * SX, SX, 0, 32 * kk, ln);
          xf[kk][i][0] = load_rows<T>(Xs + 16 * st[i] * SX, SX, 0, 32 * kk, ln);
        }
      phase();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i <= OFF; ++i) mma(a[i], yf[kk][i], xf[kk][i]);
#pragma unroll
      for (int i = 0; i <= OFF; ++i) {
        const int s = 16 * st[i] + li, q = 16 * qt[i] + lg;
        const float Ss = sc->S[s], Ls = sc->g[s], ws = sc->w[s];
        const f32x4 Sq = *reinterpret_cast<const f32x4*>(sc->S + q);
        const f32x4 Lq = *reinterpret_cast<const f32x4*>(sc->g + q);
        bool in[4];     // whether s reaches q: not before it, nor across a flag
        f32x4 L;
#pragma unroll
        for (int j = 0; j < 4; ++j) in[j] = i > 0 || q + j >= s;
        if (flagged)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            in[j] = in[j] && sc->id[q + j] == sc->id[s] && (!odd || sc->id[s] == pass);
#pragma unroll
        for (int j = 0; j < 4; ++j) L[j] = fast_exp2((Sq[j] - Ss) + (Lq[j] - Ls));
        float colsum = 0.0f, dg = 0.0f;
        f32x4 k, m1, m2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float G = cb[i][0][0][j], R = a[i][0][0][j];
          m1[j] = in[j] ? G * L[j] : 0.0f;
          m2[j] = in[j] ? R * L[j] * ws : 0.0f;
          const float kn = in[j] ? m1[j] * R : 0.0f;
          if (i == 0 && q + j == s) {
            dg = kn;
            k[j] = 0.0f;
          } else {
            colsum += kn;
            k[j] = kn * ws;
          }
        }
        colsum = sum_g(colsum);
        if (i == 0) dg = sum_g(dg);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = row_sum_to_last(k[j]);
        if (on[i]) {
          if (lane < 16) {
            sums.col[qt[i]][s] = colsum;
            if (i == 0) sums.diag[s] = dg;
          }
          if (li == 15) *reinterpret_cast<f32x4*>(&sums.row[st[i]][q]) = k;
        }
        if constexpr (PARTS == 1) {
          lg_hi[i] = u32x2{pack_bf16(m1[0], m1[1]), pack_bf16(m1[2], m1[3])};
          lg_lo[i] = u32x2{pack_bf16(m1[0] - bf16_lo(lg_hi[i][0]), m1[1] - bf16_hi(lg_hi[i][0])),
                           pack_bf16(m1[2] - bf16_lo(lg_hi[i][1]), m1[3] - bf16_hi(lg_hi[i][1]))};
          lr_hi[i] = u32x2{pack_bf16(m2[0], m2[1]), pack_bf16(m2[2], m2[3])};
          lr_lo[i] = u32x2{pack_bf16(m2[0] - bf16_lo(lr_hi[i][0]), m2[1] - bf16_hi(lr_hi[i][0])),
                           pack_bf16(m2[2] - bf16_lo(lr_hi[i][1]), m2[3] - bf16_hi(lr_hi[i][1]))};
        } else {
          lg_f[i] = m1;
          lr_f[i] = m2;
        }
      }
    }
    __syncthreads();
    // the next heads' states take these registers as soon as they are free:
    // their loads are the longest and come for all blocks at about one time
    if (more) fetch_state(p.g_chunk, mine(next), g);
    if (has_n) inter(u, Xall, false, dB);
    if constexpr (PARTS != 1) from_before();
    __syncthreads();
    put_state(h);
    phase();
    if (more) fetch_state(p.h_chunk, mine(next), h);
    __syncthreads();
    if (has_n) inter(u, Yall, true, dC);
    __syncthreads();
    // the chunk's matrices, rows s, columns q; the tiles beside the diagonal
    // that a 32-step also reads are zero.  Both in two parts: du weighs heads of
    // very different steps, and a matrix rounded once shows in the larger terms;
    // of dB and dC it is nearly all, and rounded once made their error 1.4 times
    // that of the stored type (for 3 % of the time).
    T* const M1 = Zs;
    T* const M2 = Zs + Q * SM;
    T* const M1b = Xs;          // u's tile is done with
    T* const M2b = Lall[PARTS == 1 ? side : 0];
    static_assert(SX >= SM, "the second part fits u's tile");
    {
    const Lane ln = lane_fresh();
    const int li = ln.i, lg = 4 * ln.g, lane = li + 16 * ln.g;
#pragma unroll
    for (int i = 0; i <= OFF; ++i)
      if (on[i]) {
        const int o = (16 * st[i] + li) * SM + 16 * qt[i] + lg;
        if constexpr (PARTS == 1) {
          *reinterpret_cast<u32x2*>(M1 + o) = lg_hi[i];
          *reinterpret_cast<u32x2*>(M1b + o) = lg_lo[i];
          *reinterpret_cast<u32x2*>(M2 + o) = lr_hi[i];
          *reinterpret_cast<u32x2*>(M2b + o) = lr_lo[i];
        } else {
          put4<T>(M1 + o, lg_f[i]);
          put4<T>(M2 + o, lr_f[i]);
        }
      }
    if (wave >= 4 - QT / 2) {
      const int z = wave - (4 - QT / 2);           // tiles (q, s) = (2 z, 2 z + 1)
      const int o = (32 * z + 16 + li) * SM + 32 * z + lg;
      const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
      put4<T>(M1 + o, zero);
      if constexpr (PARTS == 1) {
        put4<T>(M1b + o, zero);
        put4<T>(M2b + o, zero);
      }
      put4<T>(M2 + o, zero);
    }
    }
    __syncthreads();
    // du within the chunk
    {
    const Lane ln = lane_fresh();
#pragma unroll
    for (int ks = 0; ks < Q / 32; ++ks) {
      const Frag<PARTS> yf[1] = {load_cols<T>(Ys + 16 * wave, SX, 0, 32 * ks, ln)};
      constexpr int MP = PARTS == 1 ? 2 : PARTS;
      Frag<MP> mf[QT];
#pragma unroll
      for (int s = 0; s < 2 * ks + 2; ++s) {
        if constexpr (PARTS == 1) {
          mf[s].v[0] = load_rows<T>(M1, SM, 16 * s, 32 * ks, ln).v[0];
          mf[s].v[1] = load_rows<T>(M1b, SM, 16 * s, 32 * ks, ln).v[0];
        } else {
          mf[s] = load_rows<T>(M1, SM, 16 * s, 32 * ks, ln);
        }
      }
      phase();
      if (ks == 0) {
        f32x4 (&d)[1][2] = *reinterpret_cast<f32x4(*)[1][2]>(&du[0][0]);
        mma(d, yf, *reinterpret_cast<const Frag<MP>(*)[2]>(&mf[0]));
      } else {
        mma(du, yf, mf);
      }
    }
    }
    // dB (from C, rows of M2) and dC (from B, columns of M2) within the chunk
    // of one sequence alone the others' columns are left as they are: zeros times what
    // it holds may not be zero
    auto within = [&](auto apart) {
      auto put = [&](f32x4& to, const f32x4& v, bool keep) {
#pragma unroll
        for (int e = 0; e < 4; ++e) to[e] = !apart || keep ? v[e] : to[e];
      };
#pragma unroll
      for (int x = 0; x < SIDE; ++x) {
        if (u + x >= u1) break;
        const Lane ln = lane_fresh();
        // in bfloat16 its low part too: of a few tokens the matrix is all of dB, dC
#pragma unroll
        for (int part = 0; part < (PARTS == 1 ? 2 : 1); ++part) {
        const T* const m2 = part == 0 ? Zall[x] + Q * SM : Lall[x];
#pragma unroll
        for (int ks = 0; ks < Q / 32; ++ks) {
          Frag<PARTS> cf[NTW], bf[NTW], rf[QT], kf[QT];
#pragma unroll
          for (int i = 0; i < NTW; ++i) {
            cf[i] = load_cols<T>(Cs + n0, SN, 16 * i, 32 * ks, ln);
            bf[i] = load_cols<T>(Bs + n0, SN, 16 * i, 32 * ks, ln);
          }
#pragma unroll
          for (int s = 0; s < 2 * ks + 2; ++s) rf[s] = load_rows<T>(m2, SM, 16 * s, 32 * ks, ln);
#pragma unroll
          for (int q = 2 * ks; q < QT; ++q) kf[q] = load_cols<T>(m2, SM, 16 * q, 32 * ks, ln);
          phase();
#pragma unroll
          for (int i = 0; i < NTW; ++i) {
#pragma unroll
            for (int s = 0; s < QT; ++s) {
              const bool keep = !apart || scall[x].id[16 * s + ln.i] == pass;
              if (s < 2 * ks + 2) {
                f32x4 d[1][1] = {{dB[i][s]}};
                mma(d, *reinterpret_cast<const Frag<PARTS>(*)[1]>(&cf[i]),
                    *reinterpret_cast<const Frag<PARTS>(*)[1]>(&rf[s]));
                put(dB[i][s], d[0][0], keep);
              }
              if (s >= 2 * ks) {
                f32x4 d[1][1] = {{dC[i][s]}};
                mma(d, *reinterpret_cast<const Frag<PARTS>(*)[1]>(&bf[i]),
                    *reinterpret_cast<const Frag<PARTS>(*)[1]>(&kf[s]));
                put(dC[i][s], d[0][0], keep);
              }
            }
          }
          phase();
        }
        }
      }
    };
    if (has_n) {
      // (N > 128 has no registers for a copy of its own: 2 x 1024 x 12 heads of 128,
      // N = 256: 183 us for 234)
      if constexpr (NK == 8) within(odd);
      else if (odd) within(std::true_type{});
      else within(std::false_type{});
    }
    // du: four columns of a token a lane
    if (live) {
    const Lane ln = lane_fresh();
    const int li = ln.i, lg = 4 * ln.g, lane = li + 16 * ln.g;
      const int c = 16 * wave + lg, ncol = p.P - c0;
      T* const o0 = static_cast<T*>(p.du) + (b * p.L + t0) * row + (int64_t)hd * p.P + c0;
      const uint32_t off = (uint32_t)opaque_int(
          (int)((uint32_t)li * (uint32_t)(row * sizeof(T)) + (uint32_t)(c * sizeof(T))));
#pragma unroll
      for (int s = 0; s < QT; ++s) {
        const f32x4 y = four<T>(Ys + (16 * s + li) * SX + c);
        const float w = sc->w[16 * s + li];
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(D, y[j], w * du[0][s][j]);
        if (16 * s + li < len && c < ncol && (!odd || sc->id[16 * s + li] == pass)) {
          if constexpr (VEC) {
            put4<T>(reinterpret_cast<T*>(reinterpret_cast<char*>(o0 + 16 * s * row) + off), v);
          } else {
            T* o = o0 + (16 * s + li) * row + c;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (c + j < ncol) Elem<T>::store1(o + j, v[j]);
          }
        }
      }
    }
    // F and dw of every token, one a lane
    if (wave == 0 && live) {
    const Lane ln = lane_fresh();
    const int li = ln.i, lg = 4 * ln.g, lane = li + 16 * ln.g;
      const int t = lane < Q ? lane : Q - 1, tr = Q - 1 - t;   // and from the end
      const bool in = lane < Q;
      const int tile = t / 16;
      float row[QT], col[QT], rowO = 0.0f, colO = 0.0f, rowD = 0.0f, colD = 0.0f;
      float zi = 0.0f, wi = 0.0f;
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        row[i] = sums.row[i][t];
        col[i] = sums.col[i][t];
      }
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        rowO += i < tile ? row[i] : 0.0f;
        colO += i > tile ? col[i] : 0.0f;
        rowD = i == tile ? row[i] : rowD;
        colD = i == tile ? col[i] : colD;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        zi += sums.out[i][tr];
        wi += sums.in[i][t];
      }
      const float w = sc->w[t];
      zi = in ? weigh(zi, sc->e[tr]) : 0.0f;
      wi = weigh(wi, sc->r[t]);
      const float dw = (colO + colD) + sums.diag[t] + wi;
      // F: the paths that cross into t.  Those that leave the chunk from before t
      // and those that enter it and end from t on; those between t's tile and others,
      // and over it: sums without cancellation (starts less ends over the whole chunk
      // lost 2e-6 of dA); and within it, those that start before t less those that
      // end there.
      const float leave = in ? w * wi : 0.0f, starts = in ? w * colO : 0.0f;
      const float ends = in ? rowO : 0.0f, x = in ? w * colD - rowD : 0.0f;
      auto crossing = [&](float leave, float zi, float starts, float ends, float x, float row0,
                          float row1) {
        float F = prefix(leave) - leave + __shfl(prefix(zi), tr);
        F += suffix16(ends) + (prefix16(starts) - starts);
        if constexpr (QT == 4) {
          // read outside any branch: a lane that is off there may hold no value
          const float r0 = prefix16(tile >= 2 ? row0 : 0.0f);
          const float r1 = prefix16(tile == 3 ? row1 : 0.0f);
          const float r02 = lane_value(r0, 47), r03 = lane_value(r0, 63), r13 = lane_value(r1, 63);
          F += tile == 1 ? r02 + r03 : tile == 2 ? r03 + r13 : 0.0f;
        }
        return F + (prefix16(x) - x);
      };
      float F;
      if (flagged && __any(not_finite(leave) || not_finite(zi) || not_finite(starts) ||
                           not_finite(ends) || not_finite(x))) {
        // these sums run over all the chunk's sequences: each by itself
        F = 0.0f;
#pragma unroll 1
        for (int n = 0; n <= flags; ++n) {
          const bool m = sc->id[t] == n;
          const float f = crossing(m ? leave : 0.0f, sc->id[tr] == n ? zi : 0.0f, m ? starts : 0.0f,
                                   m ? ends : 0.0f, m ? x : 0.0f, m ? row[0] : 0.0f,
                                   m ? row[QT == 4 ? 1 : 0] : 0.0f);
          if (m) F = f;
        }
      } else {
        F = crossing(leave, zi, starts, ends, x, row[0], row[QT == 4 ? 1 : 0]);
      }
      const float T4 =
          weigh((sums.gh[0] + sums.gh[1]) + (sums.gh[2] + sums.gh[3]), sc->dec);
      float Fv = T4 + F;
      if (flagged && sc->id[t] != (t > 0 ? sc->id[t - 1] : 0)) Fv = 0.0f;
      if (lane < len && (!odd || sc->id[t] == pass)) {
        const int64_t o = ((b * p.H + hd) * CB + mu % CB) * p.L + t0 + lane;
        p.F[o] = Fv;
        p.W[o] = dw;
      }
      if (lane == 0) {
        float* const o = p.ud_part + (ch0 + hd) * CB + mu % CB;
        const float v = (sums.ud[0] + sums.ud[1]) + (sums.ud[2] + sums.ud[3]);
        *o = pass == 0 ? v : *o + v;
      }
    }
    __syncthreads();
    if (odd && !again && more) copy_keys(-1);
    pass = again ? pass + 1 : 0;
    u = next;
  }
  // the block's shares of dB, dC
  if (has_n) {
    const int64_t o = (((int64_t)split * p.batch + b) * p.L + t0) * p.G * p.N + (int64_t)grp * p.N;
#pragma unroll
    for (int j = 0; j < QT; ++j) {
      const int t = 16 * j + li;
      if (t < len)
#pragma unroll
        for (int i = 0; i < NTW; ++i) {
          const int n = n0 + 16 * i + lg;
          const int64_t at = o + (int64_t)t * p.G * p.N + n;
          if (p.N % 4 == 0) {
            if (n < p.N) {
              *reinterpret_cast<f32x4*>(p.dB_part + at) = dB[i][j];
              *reinterpret_cast<f32x4*>(p.dC_part + at) = dC[i][j];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < p.N) {
                p.dB_part[at + e] = dB[i][j][e];
                p.dC_part[at + e] = dC[i][j][e];
              }
          }
        }
    }
  }
}

// dB, dC: the splits' shares summed in order, V elements a thread and step.
template <typename T, int V>
__device__ __forceinline__ void sum_splits(const HeadsBwdParams& p, int64_t n, int64_t i) {
  float sB[V] = {}, sC[V] = {};
  for (int k = 0; k < p.splits; ++k) {
    float b[V], c[V];
    load_vec<float, V>(p.dB_part, k * n + i, b);
    load_vec<float, V>(p.dC_part, k * n + i, c);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sB[j] += b[j];
      sC[j] += c[j];
    }
  }
  store_vec<T, V>(p.dB, i, sB);
  store_vec<T, V>(p.dC, i, sC);
}

// One launch for what the chunks leave: dB and dC, and, in the blocks from `sums`
// on, ddelta of every token from F and dw with a chunk's shares of dA, dD, dbias,
// one wave a (batch row, chunk, head): 9 us of the 319.  Two launches took 3 us more.
template <typename T, int V>
__global__ __launch_bounds__(256) void heads_bwd_tail_kernel(const HeadsBwdParams p, int sums) {
  constexpr int Q = Mx<T>::Q;
  if ((int)blockIdx.x < sums) {
    const int64_t n = p.batch * p.L * p.G * p.N;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < n;
         i += (int64_t)sums * 256 * V)
      sum_splits<T, V>(p, n, i);
    return;
  }
  const int64_t chunks = (p.L + Q - 1) / Q;
  const int l = threadIdx.x & 63, CB = (p.P + 63) / 64;
  const int64_t id =
      ((int64_t)blockIdx.x - sums) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= p.batch * chunks * p.H) return;
  const int hd = (int)(id % p.H);
  const int64_t bc = id / p.H, b = bc / chunks, t = (bc - b * chunks) * Q + l;
  const bool in = l < Q && t < p.L;
  float dA = 0.0f, dbias = 0.0f;
  if (in) {
    const float raw =
        Elem<T>::load1(static_cast<const T*>(p.delta.p) + b * p.delta.batch + t * p.delta.token + hd) +
        (p.bias ? p.bias[hd] : 0.0f);
    const float A = p.A[hd];
    const Step q = make_step(raw, A, p.softplus != 0, p.zoh != 0);
    float by_dt, by_A, F = 0.0f, W = 0.0f;
    step_weight_grad(q.dt, A, p.zoh != 0, by_dt, by_A);
    for (int c = 0; c < CB; ++c) {
      F += p.F[((b * p.H + hd) * CB + c) * p.L + t];
      W += p.W[((b * p.H + hd) * CB + c) * p.L + t];
    }
    dbias = (A * F + W * by_dt) * q.draw;
    dA = q.dt * F + W * by_A;
    Elem<T>::store1(static_cast<T*>(p.ddelta) + (b * p.L + t) * p.H + hd, dbias);
  }
  dA = sum_wave(dA);
  dbias = sum_wave(dbias);
  if (l == 15) {
    float ud = 0.0f;
    for (int c = 0; c < CB; ++c) ud += p.ud_part[id * CB + c];
    p.head_part[id * 3] = dA;
    p.head_part[id * 3 + 1] = ud;
    p.head_part[id * 3 + 2] = dbias;
  }
}

// dA, dD, dbias of a head: its chunks' shares, in a fixed order (4 us: one trip).
__global__ __launch_bounds__(256) void heads_bwd_head_kernel(const HeadsBwdParams p, int64_t rows) {
  __shared__ float red[4][3];
  const int h = blockIdx.x;
  float s[3] = {0.0f, 0.0f, 0.0f};
  for (int64_t i = threadIdx.x; i < rows; i += 256)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += p.head_part[(i * p.H + h) * 3 + k];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    s[k] = sum_wave(s[k]);
    if ((threadIdx.x & 63) == 15) red[threadIdx.x >> 6][k] = s[k];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] = (red[0][k] + red[1][k]) + (red[2][k] + red[3][k]);
    p.dA[h] = s[0];
    if (p.dD) p.dD[h] = s[1];
    if (p.dbias) p.dbias[h] = s[2];
  }
}

template <typename T, int NK, bool VEC>
hipError_t bwd_go(const HeadsBwdParams& p, hipStream_t s) {
  constexpr int Q = Mx<T>::Q;
  const int dtype = sizeof(T) == 4 ? 0 : 1;
  hipError_t e = dispatch_heads_scal(p, dtype, true, s);
  if (e != hipSuccess) return e;
  const int64_t chunks = (p.L + Q - 1) / Q;
  const int64_t seg_blocks = p.batch * p.G * p.hblocks * p.nseg;
  const size_t lds = (size_t)p.hpw * sizeof(Scal<Q>);
  hipLaunchKernelGGL((heads_states_kernel<T, NK, VEC>), dim3((unsigned)(2 * seg_blocks)), dim3(256),
                     lds, s, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((heads_bwd_carry_kernel<NK>),
                     dim3((unsigned)(2 * p.batch * p.H * p.slices * NK)), dim3(256), 0, s, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((heads_chunk_kernel<T, NK, VEC>),
                     dim3((unsigned)(p.batch * p.G * chunks * p.splits)), dim3(256 * kSide<NK>), 0, s, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t n = p.batch * p.L * p.G * p.N, waves = p.batch * chunks * p.H;
  // four elements a thread where they stay together
  const bool four = n % 4 == 0 &&
                    ((uintptr_t)p.dB | (uintptr_t)p.dC) % (4 * sizeof(T)) == 0;
  const int64_t per = four ? 1024 : 256;
  const int64_t sums = (n + per - 1) / per < kMaxSumBlocks ? (n + per - 1) / per : kMaxSumBlocks;
  const dim3 grid((unsigned)(sums + (waves + 3) / 4));
  if (four)
    hipLaunchKernelGGL((heads_bwd_tail_kernel<T, 4>), grid, dim3(256), 0, s, p, (int)sums);
  else
    hipLaunchKernelGGL((heads_bwd_tail_kernel<T, 1>), grid, dim3(256), 0, s, p, (int)sums);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(heads_bwd_head_kernel, dim3((unsigned)p.H), dim3(256), 0, s, p,
                     p.batch * chunks);
  return hipGetLastError();
}

template <typename T, int NK>
hipError_t bwd_nk(const HeadsBwdParams& p, hipStream_t s) {
  return p.vec ? bwd_go<T, NK, true>(p, s) : bwd_go<T, NK, false>(p, s);
}

template <typename T>
hipError_t bwd_t(const HeadsBwdParams& p, hipStream_t s) {
  if (p.N <= 32) return bwd_nk<T, 1>(p, s);
  if (p.N <= 64) return bwd_nk<T, 2>(p, s);
  if (p.N <= 128) return bwd_nk<T, 4>(p, s);
  return bwd_nk<T, 8>(p, s);
}

}  // namespace

hipError_t dispatch_heads_bwd(const HeadsBwdParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? bwd_t<float>(p, s) : bwd_t<bf16_t>(p, s);
}

}  // namespace mscan
