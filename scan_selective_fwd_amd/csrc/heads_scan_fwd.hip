// Forward of the multi-head scan over a prompt (the formulas: heads_mma.hpp).
//
// A block of 4 waves walks along a segment of the sequence, chunk by chunk, a
// slice of 32 channels a wave, the slice's (N, 32) state in its registers: what
// is read is u, delta, B, C, what is written is out.  The heads of a block
// share B, C and the products C_q . B_s.  Where the heads alone do not fill the
// chip the sequence is cut into segments: a first pass over the segments leaves
// each one's end state from zero and its decay, a carry joins them, and the
// output pass starts each segment from the state entering it.  Up to
// kSelfCarry segments the output pass joins those before its own by itself.
//
// What bounds it: the phases of a chunk (stage, products of C and B, the state's
// share, M, the chunk's own, the update), not HBM or the matrix units.  Two blocks
// share a CU and a chunk of both takes 23 thousand clocks, of which a SIMD issues
// VALU for 12, its matrix unit is busy 6.4 and the LDS serves 4.  One block of four
// slices fills two heads of 64 channels, so that B and C are read by half as many
// blocks (with the scalars made once: 167 -> 110 us when built).  In bfloat16 M and
// the entering state are multiplied in two parts: rounded once each, as out is, they
// made out's error 1.2 to 1.4 times that of its own rounding; it is 1.0 with them,
// for 10 % of the time.  8 x 2048 tokens, 24 heads of 64, N = 128, bfloat16: 107 us in
// all (1.1 TB/s of what has to move, 120 TFLOP/s); 131072 tokens of one row 681 us
// (1.3 TB/s).
#include "heads_mma.hpp"

namespace mscan {

namespace {

template <typename T, int NK>
struct FwdTiles {
  static constexpr int Q = Mx<T>::Q, PAD = Mx<T>::PAD, NP = 32 * NK;
  static constexpr int PADT = Mx<T>::PADT;
  static constexpr int SX = kCols + PADT, SB = NP + Mx<T>::PADB, SN = NP + PAD, SM = Q + PAD, QT = Q / 16;
  static constexpr int TILES = QT * (QT + 1) / 2;
  static constexpr int PARTS = Mx<T>::PARTS;
  static constexpr int HP = PARTS == 1 ? 2 : 3;   // parts of the entering state
  static constexpr int MP = PARTS == 1 ? 2 : 3;   // and of M
  static constexpr int OFF = QT == 4 ? 2 : 1;     // M's tiles of a wave below the diagonal
  // Where M's low parts wait (bfloat16): with N <= 64 in registers, to take the high
  // parts' place after those are multiplied, as two blocks of four heads fit a CU only
  // so (8 x 2048 x 48 heads of 32, N = 64: 89 us for 118); else C's place.
  static constexpr bool TWICE = PARTS == 1 && NK <= 2;
  using Low = u32x2[TWICE ? 4 : 1][1 + OFF];
};

// Dynamic LDS: the heads' scalars and, in the output pass, their M tiles, then C's
// tile, whose place M's low parts (bfloat16) take once C is done with.
template <typename T>
size_t scal_bytes(int hpw) {
  return (size_t)hpw * sizeof(Scal<Mx<T>::Q>);
}
template <typename T, int NK>
size_t m_bytes(int hpw) {
  return (size_t)hpw * FwdTiles<T, NK>::Q * FwdTiles<T, NK>::SM * sizeof(T);
}
template <typename T, int NK>
size_t c_bytes(int hpw) {
  const size_t c = (size_t)FwdTiles<T, NK>::Q * FwdTiles<T, NK>::SN * sizeof(T);
  const size_t m = FwdTiles<T, NK>::MP == 2 && !FwdTiles<T, NK>::TWICE ? m_bytes<T, NK>(hpw) : 0;
  return c > m ? c : m;
}

// The tiles of M that a wave takes: the diagonal tile of its number and up to two
// below: (3, wave) for waves 0..2 and (1, 0); then (2, wave) for waves 0, 1.
template <int QT>
struct MTiles {
  static constexpr int OFF = QT == 4 ? 2 : 1;
  int qt[1 + OFF], st[1 + OFF];
  bool on[1 + OFF];
  __device__ __forceinline__ explicit MTiles(int wave) {
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
  }
};

// C_q . B_s of the wave's tiles (columns q, rows s).
template <typename T, int NK>
__device__ __forceinline__ void products(const T* Bs, const T* Cs,
                                         f32x4 (&a)[1 + FwdTiles<T, NK>::OFF][1][1]) {
  using F = FwdTiles<T, NK>;
  constexpr int SN = F::SN, QT = F::QT, PARTS = F::PARTS, OFF = F::OFF;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MTiles<QT> tiles(wave);
  const int (&qt)[1 + OFF] = tiles.qt, (&st)[1 + OFF] = tiles.st;
  Frag<PARTS> bf[2][1 + OFF][1], cf[2][1 + OFF][1];
#pragma unroll
  for (int i = 0; i <= OFF; ++i) {
    a[i][0][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    bf[0][i][0] = load_rows<T>(Bs, F::SB, 16 * st[i], 0);
    cf[0][i][0] = load_rows<T>(Cs, SN, 16 * qt[i], 0);
  }
#pragma unroll
  for (int kk = 0; kk < NK; ++kk) {
    if (kk + 1 < NK) {
#pragma unroll
      for (int i = 0; i <= OFF; ++i) {
        bf[(kk + 1) & 1][i][0] = load_rows<T>(Bs, F::SB, 16 * st[i], 32 * kk + 32);
        cf[(kk + 1) & 1][i][0] = load_rows<T>(Cs, SN, 16 * qt[i], 32 * kk + 32);
      }
    }
    phase();
#pragma unroll
    for (int i = 0; i <= OFF; ++i) mma(a[i], bf[kk & 1][i], cf[kk & 1][i]);
  }
}

// The block's M tiles from these, weighted for each head, as M's rows; in bfloat16
// M's high parts, and its low ones to Low.
template <typename T, int NK>
__device__ __forceinline__ void decayed_products(
    const HeadsParams& p, int heads, bool flagged,
    const f32x4 (&a)[1 + FwdTiles<T, NK>::OFF][1][1], const Scal<Mx<T>::Q>* scal, T* Mall, T* Low,
    typename FwdTiles<T, NK>::Low& low) {
  using F = FwdTiles<T, NK>;
  constexpr int Q = F::Q, SM = F::SM, QT = F::QT, OFF = F::OFF;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MTiles<QT> tiles(wave);
  const int (&qt)[1 + OFF] = tiles.qt, (&st)[1 + OFF] = tiles.st;
  const bool (&on)[1 + OFF] = tiles.on;
  const Lane ln = lane_fresh();
  const int li = ln.i, lg = 4 * ln.g;
  auto weight = [&](int x) {
    const Scal<Q>& o = scal[x];
    float m[1 + OFF][4], Sq[1 + OFF], Lq[1 + OFF], Se[1 + OFF], Le[1 + OFF];
    f32x4 g[1 + OFF];
    // differences of the sums with what their rounding lost: after a step that
    // forgets nearly all the sums are large and the weights near 1 again
    const f32x4 Ss = *reinterpret_cast<const f32x4*>(o.S + 16 * st[0] + lg);
    const f32x4 Ls = *reinterpret_cast<const f32x4*>(o.r + 16 * st[0] + lg);
    const f32x4 w = *reinterpret_cast<const f32x4*>(o.w + 16 * st[0] + lg);
#pragma unroll
    for (int i = 0; i <= OFF; ++i) {
      Sq[i] = o.S[16 * qt[i] + li];
      Lq[i] = o.r[16 * qt[i] + li];
      Se[i] = o.S[16 * st[i] + 15];
      Le[i] = o.r[16 * st[i] + 15];
      g[i] = *reinterpret_cast<const f32x4*>(o.g + 16 * st[i] + lg);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m[0][j] = lg + j <= li
                    ? a[0][0][0][j] * (fast_exp2((Sq[0] - Ss[j]) + (Lq[0] - Ls[j])) * w[j])
                    : 0.0f;
    // Below the diagonal the decay is the product of two, to the end of s's
    // tile and on to q: with steps that are never negative neither leaves the
    // range that their product keeps.
#pragma unroll
    for (int i = 1; i <= OFF; ++i) {
      const float f = fast_exp2((Sq[i] - Se[i]) + (Lq[i] - Le[i]));
#pragma unroll
      for (int j = 0; j < 4; ++j) m[i][j] = a[i][0][0][j] * (g[i][j] * f);
    }
    if (!p.softplus) {
#pragma unroll
      for (int i = 1; i <= OFF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = 16 * st[i] + lg + j;
          m[i][j] = a[i][0][0][j] * (fast_exp2((Sq[i] - o.S[s]) + (Lq[i] - o.r[s])) * o.w[s]);
        }
    }
    if (flagged) {
#pragma unroll
      for (int i = 0; i <= OFF; ++i) {
        const int idq = o.id[16 * qt[i] + li];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[i][j] = o.id[16 * st[i] + lg + j] == idq ? m[i][j] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i <= OFF; ++i) {
      u32x2 rest = {0, 0};
      if constexpr (F::MP == 2)
        rest = u32x2{pack_bf16(m[i][0] - top8(m[i][0]), m[i][1] - top8(m[i][1])),
                     pack_bf16(m[i][2] - top8(m[i][2]), m[i][3] - top8(m[i][3]))};
      if constexpr (F::TWICE) low[x][i] = rest;
      if (on[i]) {
        const int o = x * Q * SM + (16 * qt[i] + li) * SM + 16 * st[i] + lg;
        if constexpr (F::MP == 2) {
          *reinterpret_cast<u32x2*>(Mall + o) =
              u32x2{pack_hi(m[i][0], m[i][1]), pack_hi(m[i][2], m[i][3])};
          if constexpr (!F::TWICE) *reinterpret_cast<u32x2*>(Low + o) = rest;
        } else {
          *reinterpret_cast<f32x4*>(Mall + o) = f32x4{m[i][0], m[i][1], m[i][2], m[i][3]};
        }
      }
    }
    // Low's tiles above the diagonal that a 32-step reads with the others
    if constexpr (F::MP == 2 && !F::TWICE) {
      if (wave >= 4 - QT / 2) {
        const int z = 2 * (wave - (4 - QT / 2));
        *reinterpret_cast<u32x2*>(Low + x * Q * SM + (16 * z + li) * SM + 16 * z + 16 + lg) =
            u32x2{0, 0};
      }
    }
  };
  // two heads at a time: their reads and exponentials overlap
  if constexpr (F::TWICE) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x < heads) weight(x);
  } else {
#pragma unroll 1
    for (int x = 0; x < heads; x += 2) {
      weight(x);
      if (x + 1 < heads) weight(x + 1);
    }
  }
}

// M's low parts in place of the high ones.
template <typename T, int NK>
__device__ __forceinline__ void store_low(int heads, T* Mall,
                                          const typename FwdTiles<T, NK>::Low& low) {
  using F = FwdTiles<T, NK>;
  const MTiles<F::QT> tiles(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  const Lane ln = lane_fresh();
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (x < heads)
#pragma unroll
      for (int i = 0; i <= F::OFF; ++i)
        if (tiles.on[i])
          *reinterpret_cast<u32x2*>(Mall + x * F::Q * F::SM + (16 * tiles.qt[i] + ln.i) * F::SM +
                                    16 * tiles.st[i] + 4 * ln.g) = low[x][i];
}


// The output pass; 80 us of 118 in the kernels' trace, 503 of 735.
template <typename T, int NK, bool VEC>
__global__ __launch_bounds__(256, NK == 8 ? 1 : 2) void heads_fwd_kernel(const HeadsFwdParams p) {
  using F = FwdTiles<T, NK>;
  constexpr int Q = F::Q, NP = F::NP, SX = F::SX, SB = F::SB, SN = F::SN, SM = F::SM, QT = F::QT;
  constexpr int PARTS = F::PARTS;
  __shared__ __align__(16) T Xs[Q * SX];
  __shared__ __align__(16) T Bs[Q * SB];
  extern __shared__ __align__(16) char dyn[];
  Scal<Q>* const scal = reinterpret_cast<Scal<Q>*>(dyn);
  T* const Mall = reinterpret_cast<T*>(dyn + p.hpw * sizeof(Scal<Q>));
  T* const Cs = Mall + p.hpw * Q * SM;
  const Place k = place_of(p, p.nseg);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t begin = (int64_t)k.seg * p.seg_len;
  const int64_t end = k.seg + 1 == p.nseg ? p.L : begin + p.seg_len;
  const int64_t ucol = (int64_t)k.h0 * p.P, ncols = (int64_t)k.g * p.N;
  const int uwidth = (k.h0 + k.heads) * p.P;
  const int sub = p.slices * kSlice, hh = wave / p.slices;
  const float D = p.D ? p.D[k.h] : 0.0f;
  const int64_t chunks = (p.L + Q - 1) / Q;

  f32x4 h[2 * NK][2];
  if (!k.on) {
    fill<NK>(h, 0.0f);
  } else if (p.carried && k.seg > 0) {
    load_frags<NK>(p.seg_state + slice_slot(p, k, p.nseg - 1, k.seg - 1) * slice_floats<NK>(), h);
  } else {
    if (p.h0_kept)
      load_frags<NK>(p.h0_kept + slice_slot(p, k, 1, 0) * slice_floats<NK>(), h);
    else
      load_state<NK>(p.h0 ? p.h0 + (k.b * p.H + k.h) * (int64_t)p.P * p.N : nullptr, k.c0, p.P, p.N, h);
    // few segments: each joins the ones before it by itself
    const int64_t slot = slice_slot(p, k, p.nseg - 1, 0);
    for (int i = 0; i < k.seg; ++i) {
      f32x4 x[2 * NK][2];
      load_frags<NK>(p.seg_state + (slot + i) * slice_floats<NK>(), x);
      decay_state<NK>(h, p.seg_dec[slot + i]);
#pragma unroll
      for (int nt = 0; nt < 2 * NK; ++nt)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) h[nt][pt] += x[nt][pt];
    }
  }
  // tiles above the diagonal are read as part of a 32-step and stay zero
  for (int i = threadIdx.x; i < p.hpw * Q * SM; i += 256) Mall[i] = T(0);

  Stage<T, Q, kCols, VEC> sx;
  Stage<T, Q, NP, VEC> sb, sc;
  ScalStage<Q> ss;
  sx.init(p.u, ucol, sub, p.P, p.P, k.heads);
  auto rows = [&](int64_t t) { return end - t < Q ? (int)(end - t) : Q; };
  auto row_of = [&](const Rows& r, int64_t t) {
    return static_cast<const T*>(r.p) + k.b * r.batch + t * r.token + ncols;
  };
  auto fetch = [&](int64_t t) {
    const int len = rows(t);
    ss.load(p.scal, (k.b * chunks + t / Q) * p.H + k.h0, k.heads);
    sx.load(p.u, k.b, t, len, ucol, p.P, uwidth);
    sb.load_at(row_of(p.B, t), p.B.token, len, p.N);
    sc.load_at(row_of(p.C, t), p.C.token, len, p.N);
  };
  fetch(begin);
  __syncthreads();
  for (int64_t t = begin; t < end; t += Q) {
    const int len = rows(t);
    sx.store(Xs, SX);
    sb.store(Bs, SB);
    sc.store(Cs, SN);
    ss.store(scal, k.heads);
    __syncthreads();
    // the next chunk's loads have this whole one to arrive
    if (t + Q < end) fetch(t + Q);
    const Scal<Q>& me = scal[k.on ? hh : 0];
    const bool flagged = scal[0].flags != 0;   // flags are the batch row's

    // M^T tiles (rows s, columns q) on and below the diagonal: C_q . B_s once for
    // the block, weighted for each head
    f32x4 cb[1 + F::OFF][1][1];
    products<T, NK>(Bs, Cs, cb);
    typename F::Low low;
    constexpr bool IN_C = F::MP == 2 && !F::TWICE;   // M's low parts take C's place
    if constexpr (!IN_C)
      decayed_products<T, NK>(p, k.heads, flagged, cb, scal, Mall, nullptr, low);
    phase();
    // out^T (rows p, columns q): the entering state's share
    f32x4 y[2][QT];
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) y[pt][qt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (k.on) {
      // two tiles of rows a step, their fragments loaded a step ahead
      constexpr int PAIRS = QT / 2, STEPS = NK * PAIRS;
      Frag<PARTS> cf[2][2];
      auto load_c = [&](int i, Frag<PARTS> (&f)[2]) {
        f[0] = load_rows<T>(Cs, SN, 32 * (i % PAIRS), 32 * (i / PAIRS));
        f[1] = load_rows<T>(Cs, SN, 32 * (i % PAIRS) + 16, 32 * (i / PAIRS));
      };
      load_c(0, cf[0]);
      Frag<F::HP> hf[2];
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int kk = i / PAIRS, qt = 2 * (i % PAIRS);
        if (i + 1 < STEPS) load_c(i + 1, cf[(i + 1) & 1]);
        if (i % PAIRS == 0) {
          hf[0] = acc_frag<F::HP>(h[2 * kk][0], h[2 * kk + 1][0]);
          hf[1] = acc_frag<F::HP>(h[2 * kk][1], h[2 * kk + 1][1]);
        }
        phase();
        f32x4 yy[2][2] = {{y[0][qt], y[0][qt + 1]}, {y[1][qt], y[1][qt + 1]}};
        mma(yy, hf, cf[i & 1]);
        y[0][qt] = yy[0][0];
        y[0][qt + 1] = yy[0][1];
        y[1][qt] = yy[1][0];
        y[1][qt + 1] = yy[1][1];
      }
      if (flagged) {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
          const float e = me.e[16 * qt + lane_i()];
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[pt][qt][j] = weigh(y[pt][qt][j], e);
        }
      } else {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
          const float e = me.e[16 * qt + lane_i()];
          y[0][qt] *= e;
          y[1][qt] *= e;
        }
      }
    }
    __syncthreads();
    if constexpr (IN_C) decayed_products<T, NK>(p, k.heads, flagged, cb, scal, Mall, Cs, low);
    if (flagged) clear_kept<T, Q, NP>(Bs, SB, scal[0].id, scal[0].flags);
    if (IN_C || flagged) __syncthreads();
    // ... and the chunk's own inputs'
    uint64_t marks[2] = {0, 0};
    bool odd = false;
    if (k.on) {
      odd = tile_odd<T, Q>(Xs, SX, k.col);
      if (odd) {
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
          marks[pt] = take_out<T, Q>(Xs, SX, k.col + 16 * pt + lane_i());
      }
    }
    // (tile pair, 32-step): the first step reaches all rows, the second the last half
    constexpr int STEPS = Q == 64 ? 3 : 1, MR = IN_C ? 2 : PARTS;   // parts read at a time
    const T* const Ms = Mall + (k.on ? hh : 0) * Q * SM;
    Frag<PARTS> xf[Q / 32][2];
    auto within = [&]() {
      Frag<MR> mf[2][2];
      auto load_m = [&](int i, Frag<MR> (&f)[2]) {
        const int qt = i == 0 ? 0 : 2, ks = i == 2 ? 1 : 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if constexpr (IN_C) {
            f[c].v[0] = load_rows<T>(Ms, SM, 16 * qt + 16 * c, 32 * ks).v[0];
            f[c].v[1] = load_rows<T>(Cs + hh * Q * SM, SM, 16 * qt + 16 * c, 32 * ks).v[0];
          } else {
            f[c] = load_rows<T>(Ms, SM, 16 * qt + 16 * c, 32 * ks);
          }
        }
      };
      load_m(0, mf[0]);
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int qt = i == 0 ? 0 : 2, ks = i == 2 ? 1 : 0;
        if (i + 1 < STEPS) load_m(i + 1, mf[(i + 1) & 1]);
        phase();
        f32x4 yy[2][2] = {{y[0][qt], y[0][qt + 1]}, {y[1][qt], y[1][qt + 1]}};
        mma(yy, xf[ks], mf[i & 1]);
        y[0][qt] = yy[0][0];
        y[0][qt + 1] = yy[0][1];
        y[1][qt] = yy[1][0];
        y[1][qt + 1] = yy[1][1];
      }
    };
    if (k.on) {
#pragma unroll
      for (int ks = 0; ks < Q / 32; ++ks)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
          xf[ks][pt] = load_cols<T>(Xs, SX, k.col + 16 * pt, 32 * ks);
      within();
    }
    if constexpr (F::TWICE) {
      __syncthreads();
      store_low<T, NK>(k.heads, Mall, low);
      __syncthreads();
      if (k.on) within();
    }
    if (k.on) {
      if (odd) {
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // column 4 g + j's marks are with the lane of that column
            const int from = 4 * lane_g() + j;
            const uint64_t m = (uint64_t)(uint32_t)__shfl((int)(uint32_t)marks[pt], from) |
                               (uint64_t)(uint32_t)__shfl((int)(uint32_t)(marks[pt] >> 32), from) << 32;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
              if (marked_upto<Q>(m, me.id, 16 * qt + lane_i())) y[pt][qt][j] = __builtin_nanf("");
          }
      }
      phase();
      // four columns of a token a lane
      const int64_t row = (int64_t)p.H * p.P;
      T* const o0 = static_cast<T*>(p.out) + (k.b * p.L + t) * row + (int64_t)k.h * p.P + k.c0;
      // one offset a lane, the tiles' bases uniform; a chunk of out spans less
      // than 2^31 bytes
      const Lane ln = lane_fresh();
      const uint32_t off =
          (uint32_t)ln.i * (uint32_t)(row * sizeof(T)) + 4u * (uint32_t)ln.g * sizeof(T);
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) {
        const int q = 16 * qt + ln.i;
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) {
          const int c = 16 * pt + 4 * ln.g;
          const T* ur = Xs + q * SX + k.col + c;
          float v[4];
          if constexpr (sizeof(T) == 2) {
            const u32x2 u = *reinterpret_cast<const u32x2*>(ur);
            v[0] = bf16_lo(u[0]); v[1] = bf16_hi(u[0]); v[2] = bf16_lo(u[1]); v[3] = bf16_hi(u[1]);
          } else {
            const f32x4 u = *reinterpret_cast<const f32x4*>(ur);
            v[0] = u[0]; v[1] = u[1]; v[2] = u[2]; v[3] = u[3];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(D, v[j], y[pt][qt][j]);
          if (q < len && c < k.ncol) {
            if constexpr (VEC) {
              char* o = reinterpret_cast<char*>(o0 + 16 * qt * row + 16 * pt) + off;
              if constexpr (sizeof(T) == 2)
                *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
              else
                *reinterpret_cast<f32x4*>(o) = f32x4{v[0], v[1], v[2], v[3]};
            } else {
              T* o = o0 + q * row + c;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (c + j < k.ncol) Elem<T>::store1(o + j, v[j]);
            }
          }
        }
        phase();
      }
      phase();
      step_state<T, NK>(h, me.dec, me.c, Bs, SB, Xs, SX, k.col);
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
        if (marks[pt] != 0 && marked<Q>(marks[pt], me.id, me.flags)) spoil<NK>(h, pt);
    }
    __syncthreads();
  }
  if (p.last && k.on && k.seg + 1 == p.nseg)
    store_state<NK>(p.last + (k.b * p.H + k.h) * (int64_t)p.P * p.N, k.c0, p.P, p.N, h);
}

// A segment's end state from zero and its decay: the output pass's update alone,
// which reads u and B and writes a state a segment; 31 us of the 118, 188 of the 735.
template <typename T, int NK, bool VEC>
__global__ __launch_bounds__(256, NK == 8 ? 1 : 2) void heads_seg_kernel(const HeadsFwdParams p) {
  using F = FwdTiles<T, NK>;
  constexpr int Q = F::Q, NP = F::NP, SX = F::SX, SB = NP + F::PADT;   // only read transposed
  __shared__ __align__(16) T Xs[Q * SX];
  __shared__ __align__(16) T Bs[Q * SB];
  extern __shared__ __align__(16) char dyn[];
  Scal<Q>* const scal = reinterpret_cast<Scal<Q>*>(dyn);
  const Place k = place_of(p, p.nseg - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t begin = (int64_t)k.seg * p.seg_len, end = begin + p.seg_len;   // whole chunks
  const int64_t ucol = (int64_t)k.h0 * p.P, ncols = (int64_t)k.g * p.N;
  const int uwidth = (k.h0 + k.heads) * p.P, nwidth = (k.g + 1) * p.N;
  const int sub = p.slices * kSlice, hh = wave / p.slices;
  const int64_t chunks = (p.L + Q - 1) / Q;
  f32x4 h[2 * NK][2];
  if (p.h0_kept && k.on && k.seg == 0) {
    load_state<NK>(p.h0 + (k.b * p.H + k.h) * (int64_t)p.P * p.N, k.c0, p.P, p.N, h);
    store_frags<NK>(p.h0_kept + slice_slot(p, k, 1, 0) * slice_floats<NK>(), h);
  }
  fill<NK>(h, 0.0f);
  float dec = 1.0f;
  Stage<T, Q, kCols, VEC> sx;
  Stage<T, Q, NP, VEC> sb;
  ScalStage<Q> ss;
  sx.init(p.u, ucol, sub, p.P, p.P, k.heads);
  sb.init(p.B, ncols, NP, 0, p.N, 1);
  auto fetch = [&](int64_t t) {
    ss.load(p.scal, (k.b * chunks + t / Q) * p.H + k.h0, k.heads);
    sx.load(p.u, k.b, t, Q, ucol, p.P, uwidth);
    sb.load(p.B, k.b, t, Q, ncols, 0, nwidth);
  };
  fetch(begin);
  for (int64_t t = begin; t < end; t += Q) {
    sx.store(Xs, SX);
    sb.store(Bs, SB);
    ss.store(scal, k.heads);
    __syncthreads();
    if (t + Q < end) fetch(t + Q);
    const Scal<Q>& me = scal[k.on ? hh : 0];
    if (scal[0].flags != 0) {
      clear_kept<T, Q, NP>(Bs, SB, scal[0].id, scal[0].flags);
      __syncthreads();
    }
    if (k.on) {
      uint64_t marks[2] = {0, 0};
      if (tile_odd<T, Q>(Xs, SX, k.col)) {
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
          marks[pt] = take_out<T, Q>(Xs, SX, k.col + 16 * pt + lane_i());
      }
      step_state<T, NK>(h, me.dec, me.c, Bs, SB, Xs, SX, k.col);
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
        if (marks[pt] != 0 && marked<Q>(marks[pt], me.id, me.flags)) spoil<NK>(h, pt);
      dec = join(dec, me.dec);
    }
    __syncthreads();
  }
  if (!k.on) return;
  const int64_t slot = slice_slot(p, k, p.nseg - 1, k.seg);
  store_frags<NK>(p.seg_state + slot * slice_floats<NK>(), h);
  if ((threadIdx.x & 63) == 0) p.seg_dec[slot] = dec;
}

// The state entering each segment, in place of the one before's end state: four
// floats a thread, bound by the trips to memory (42 segments of 24 heads: 13 us).
template <int NK>
__global__ __launch_bounds__(256) void heads_carry_kernel(const HeadsFwdParams p) {
  constexpr int PER = NK;   // blocks a slice: 1024 NK floats, four a thread
  const int64_t id = blockIdx.x / PER;
  const int e = (int)(blockIdx.x - id * PER) * 256 + threadIdx.x;   // float4 of the state
  const int slice = (int)(id % p.slices);
  const int64_t bh = id / p.slices;
  const int nt = e >> 7, pt = (e >> 6) & 1, l = e & 63;
  const int pp = slice * kSlice + 16 * pt + (l & 15), n = 16 * nt + 4 * (l >> 4);
  f32x4 h = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.h0 && pp < p.P)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < p.N) h[j] = p.h0[(bh * p.P + pp) * p.N + n + j];
  const int segs = p.nseg - 1;
  f32x4* st = reinterpret_cast<f32x4*>(p.seg_state + id * segs * slice_floats<NK>()) + e;
  constexpr int64_t STEP = slice_floats<NK>() / 4;
  // a group's loads are out together (16 segments 10 us -> 6)
  constexpr int GROUP = 8;
  for (int k0 = 0; k0 < segs; k0 += GROUP) {
    f32x4 s[GROUP];
    float d[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      const int k = k0 + i < segs ? k0 + i : segs - 1;
      s[i] = st[k * STEP];
      d[i] = p.seg_dec[id * segs + k];
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i)
      if (k0 + i < segs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = weigh(h[j], d[i]) + s[i][j];
        st[(k0 + i) * STEP] = h;
      }
  }
}

template <typename T, int NK, bool VEC>
hipError_t fwd_go(const HeadsFwdParams& p, hipStream_t s) {
  {
    const hipError_t e = dispatch_heads_scal(p, sizeof(T) == 4 ? 0 : 1, false, s);
    if (e != hipSuccess) return e;
  }
  const int64_t blocks = p.batch * p.G * p.hblocks;
  if (p.nseg > 1) {
    const size_t lds = scal_bytes<T>(p.hpw);
    hipLaunchKernelGGL((heads_seg_kernel<T, NK, VEC>), dim3((unsigned)(blocks * (p.nseg - 1))),
                       dim3(256), lds, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.carried) {
      hipLaunchKernelGGL((heads_carry_kernel<NK>), dim3((unsigned)(p.batch * p.H * p.slices * NK)),
                         dim3(256), 0, s, p);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  const size_t lds = scal_bytes<T>(p.hpw) + m_bytes<T, NK>(p.hpw) + c_bytes<T, NK>(p.hpw);
  hipLaunchKernelGGL((heads_fwd_kernel<T, NK, VEC>), dim3((unsigned)(blocks * p.nseg)), dim3(256),
                     lds, s, p);
  return hipGetLastError();
}

template <typename T, int NK>
hipError_t fwd_nk(const HeadsFwdParams& p, hipStream_t s) {
  return p.vec ? fwd_go<T, NK, true>(p, s) : fwd_go<T, NK, false>(p, s);
}

template <typename T>
hipError_t fwd_t(const HeadsFwdParams& p, hipStream_t s) {
  if (p.N <= 32) return fwd_nk<T, 1>(p, s);
  if (p.N <= 64) return fwd_nk<T, 2>(p, s);
  if (p.N <= 128) return fwd_nk<T, 4>(p, s);
  return fwd_nk<T, 8>(p, s);
}

}  // namespace

hipError_t dispatch_heads_fwd(const HeadsFwdParams& p, int dtype, hipStream_t s) {
  return dtype == 0 ? fwd_t<float>(p, s) : fwd_t<bf16_t>(p, s);
}

}  // namespace mscan
