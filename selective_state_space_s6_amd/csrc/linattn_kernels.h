// linattn_kernels.h -- linear attention with a decay for each head: the chunk walk.
//
// With a_t = exp(g_t), S_t = a_t S_{t-1} + k_t v_t^T and o_t = scale q_t^T S_t.  Over a chunk of C
// tokens with c_i = g_1 + .. + g_i, c its total, S the state before it:
//     o_i = scale ( sum_{j<=i} e^{c_i - c_j} (q_i . k_j) v_j + e^{c_i} q_i S )
//     S'  = e^c S + sum_j e^{c - c_j} k_j v_j^T
// and backwards, R the gradient of the state behind the chunk:
//     o_j = sum_{i>=j} e^{c_i - c_j} (q_j . k_i) v_i + e^{c - c_j} q_j R
//     R'  = e^c R + sum_i e^{c_i} k_i v_i^T
// The gradients are these two walks on other operands: dq = forward(do, v, k),
// dk = backward(v, do, q), dv = backward(k, q, do).
//
// A chunk has 64 tokens: the pairs cost as many products as the state does at 64 channels, and the tiles of two
// workgroups of eight wavefronts fit the LDS of a compute unit (256 fp32 channels: chunks of 32, one workgroup).  The
// state never leaves the accumulators: their layout is, with the channels counted as 8 (l / 16) + 4 u + r, that
// of the operand which meets the queries, so only its rounding into parts lies between.  Long sequences of few heads
// are cut into segments; a pass over k and v forms each one's own state, a prefix what enters it.
// What bounds it (1 x 32 heads x 16384, 128 x 128 bf16, 243 us; 105 us of bytes): the state pass takes 81 us, of which 52
// are its bytes, the prefix 13, the walk 149.  In the walk the matrix units are busy 29 % of the time, the vector
// units 52 %, and a wavefront waits 42 % of it: the products of one chunk hang on one another, three barriers part them, and
// registers (128) and LDS hold four wavefronts a SIMD; 37 % of the LDS's cycles are bank conflicts.  Four wavefronts of 32 columns, which read half as much from
// the LDS, are slower (walk 169 us), as are two tiles of k and v in turns in the state pass (no gain).
#pragma once

#include <cmath>
#include <type_traits>

#include "device_common.h"
#include "linattn_device.h"
#include "scan_launch.h"

namespace selscan {
namespace {

// x as a sum of N values of the matrix cores' type (the first rounds x, the next what that left).  Where x is
// not finite, neither is the sum.
template <typename T, int N>
__device__ __forceinline__ void lin_split(f32x8 x, typename lin_io<T>::frag* out) {
  if constexpr (sizeof(T) == 4) {
    out[0] = x;
  } else {
    u32x4 part[N];
    // A pair's product with (-1, 0) or (0, -1) takes one of the two off without unpacking it.  (The constants
    // go through registers: as literals the compiler writes them in a form that the instruction reads otherwise.)
    uint32_t first = 0x0000bf80u, second = 0xbf800000u;
    asm volatile("" : "+s"(first), "+s"(second));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const bf16x2 r = __builtin_convertvector(f32x2{a, b}, bf16x2);
        part[n][i] = __builtin_bit_cast(uint32_t, r);
        a = __builtin_amdgcn_fdot2_f32_bf16(r, __builtin_bit_cast(bf16x2, first), a, false);
        b = __builtin_amdgcn_fdot2_f32_bf16(r, __builtin_bit_cast(bf16x2, second), b, false);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) out[n] = __builtin_bit_cast(bf16x8, part[n]);
  }
}

// What rounding to bfloat16 leaves of a value.
__device__ __forceinline__ float lin_rest(float v) { return v - float(__bf16(v)); }

// A token's decay, 2^-150 and more: only a token that starts anew ends an infinity.  (Of finite values, what a product
// of decays leaves below fp32's smallest value is nothing; one that is not finite is walked token by token.)
__device__ __forceinline__ float lin_decay(float log2d) {
  const float d = lin_exp2(log2d);
  return d < kTiny ? kTiny : d;
}

// Wavefronts that a SIMD is to hold, NW of them a workgroup: as many as the LDS of a compute unit holds tiles for.
template <typename T, int KD, int NW, bool DOT> constexpr int lin_waves() {
  return sizeof(T) == 4 || KD == 256 ? (NW == 8 ? 2 : 1) : NW == 8 ? 4 : KD == 128 && DOT ? 2 : 3;
}

// What the tokens of a chunk are to one another.
template <int C> struct alignas(16) LinDecays {
  float hi[C], lo[C];       // log2 of the decays since the chunk's start, in two parts
  float f[C], w[C];         // factor of a row's product with the state; of a row's share in the new state
  int lim[C];               // the row's first visible key (forward), its last (backward)
  float mul;                // what the held state is multiplied by (1 as a rule: see `scale` in the walk)
  float before, after;      // the held state's scale before the chunk, and behind it
};

template <typename T, int KD, int NW, int HP, int C, bool STATE, bool DOT>
struct alignas(16) LinShared {
  static constexpr int NPP = sizeof(T) == 4 ? 1 : 2;      // parts of the pairs on the matrix cores
  static constexpr int IT = C / 16, kPairs = IT * (IT + 1) / 2 * 256;
  T q[STATE ? 8 : C * KD];
  T k[C * KD];
  T v[C * 16 * NW];
  T p[STATE ? 8 : HP * NPP * kPairs + 8];                          // (8 zeros behind them)
  LinDecays<C> dec[HP][2];  // this chunk's, and the next one's
  float dot[DOT ? NW : 1][DOT ? C : 1];
  float cross[NW];
  int bad;
};

template <LinWalk WALK> struct LinWalks { LinParams p[WALK == LinWalk::states || WALK == LinWalk::grads ? 2 : 1]; };

// One of a kernel's LinWalks, its first argument, read anew: what comes of it is not kept from before.
__device__ __forceinline__ const LinParams& lin_again(int i) {
  auto at = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return ((const LinParams*)at)[i];
}

// A workgroup's part of a walk: head `part` of its heads, a block of columns, a segment.
template <int C, int HP, int COLS, bool STATE, bool REV> struct LinPlace {
  int nb, seg, chunks, col0;
  int64_t h, b, bh, chunk0, L;
  __device__ __forceinline__ LinPlace(const LinParams& p, int item, int part) {
    // (32 bits, unsigned: a division of 64 takes a hundred instructions and more)
    const uint32_t segs = uint32_t(STATE ? p.nseg - 1 : p.nseg);    // (nothing is behind the last segment)
    const uint32_t H = uint32_t(p.H), heads = H / HP, rest = uint32_t(item) / heads, blk = uint32_t(p.nblk);
    const uint32_t segments = rest / blk, row = segments / segs;
    const int sidx = int(segments - row * segs);
    nb = int(rest - segments * blk);
    h = (uint32_t(item) - rest * heads) * HP + part;
    b = row;
    bh = b * H + h;
    seg = STATE && REV ? sidx + 1 : sidx;
    chunk0 = int64_t(seg) * p.seg_chunks;
    chunks = int(p.nchunks - chunk0 < p.seg_chunks ? p.nchunks - chunk0 : p.seg_chunks);
    col0 = nb * COLS;
    L = p.L;
  }
  __device__ __forceinline__ int64_t start_of(int ci) const { return (chunk0 + (REV ? chunks - 1 - ci : ci)) * C; }
  __device__ __forceinline__ int tokens_of(int64_t t0) const { return int(L - t0 < C ? L - t0 : C); }
  // column `col` of a row of `out`, and of x
  __device__ __forceinline__ char* out_at(const LinParams& p, int64_t t, int col, int size) const {
    return static_cast<char*>(p.out) + (b * p.o_sb + h * p.o_sh + t * p.o_sl + col) * size;
  }
  template <typename T> __device__ __forceinline__ const T* x_at(const LinParams& p, int64_t t, int col) const {
    return static_cast<const T*>(p.x.p) + b * p.x.sb + int64_t(uint32_t(h) / uint32_t(p.x.share)) * p.x.sh + t * p.x.sl + col;
  }
};

// One workgroup of NW wavefronts walks the chunks of one segment of HP heads of one batch row that share their
// queries and keys, for 16 NW / HP columns of v each: a wavefront owns 16 of them, and the state's [KD][16] in
// its accumulators, which are at once the operand of its product with the queries.
// STATE: only the state at the segment's end, from zero.
// DOT: the products of x with the rows' parts of the state too, the state between every lin_span() chunks, and a mark for
// chunks that need it themselves (lin_between_kernel).  For the spans that have one, with a span in a segment's place:
// KEEP: only the state before each chunk.  CROSS: only its products with the backward walk's behind the chunk.
// bf16: pairs and state go to the matrix cores with 16 bits, twice the result's own (pairs of 8 bits would add as
// much again to its rounding), the state with 24 where its products give the decays' gradient, an fp32 result.
template <typename T, int KD, int NW, int HP, int C, LinWalk WALK>
__global__ __launch_bounds__(64 * NW, (lin_waves<T, KD, NW, WALK == LinWalk::grads>())) void lin_kernel(LinWalks<WALK> walks) {
  constexpr bool CROSS = WALK == LinWalk::cross, KEEP = WALK == LinWalk::keep;
  constexpr bool STATE = WALK == LinWalk::state || WALK == LinWalk::states || CROSS || KEEP, OWN = STATE && !CROSS && !KEEP;
  constexpr bool DOT = WALK == LinWalk::grads;
  using io = lin_io<T>;
  using frag = typename io::frag;
  constexpr int NP = sizeof(T) == 4 ? 1 : DOT ? 3 : 2;   // parts of the state on the matrix cores
  constexpr bool kBoth = WALK == LinWalk::states || WALK == LinWalk::grads;
  constexpr int NX = sizeof(T) == 2 ? 3 : 1;      // the state is held in fp32: what is added to it keeps 24 bits
  using Sh = LinShared<T, KD, NW, HP, C, STATE, DOT>;
  constexpr int NPP = Sh::NPP;
  __shared__ Sh sh;

  if constexpr (KEEP || CROSS) {
    // nothing to do where no chunk has a mark
    const LinParams& p = walks.p[0];
    const int item = xcd_contiguous_block(blockIdx.x, gridDim.x), heads = int(p.H) / HP, seg = item / heads / p.nblk % p.nseg;
    const int64_t bh = int64_t(item / heads / p.nblk / p.nseg) * p.H + item % heads * HP, chunk0 = int64_t(seg) * p.seg_chunks;
    const int each = int(p.nchunks - chunk0 < p.seg_chunks ? p.nchunks - chunk0 : p.seg_chunks) * p.marks_each;
    int any = 0;
    for (int i = threadIdx.x; i < 2 * HP * each; i += 64 * NW)
      any |= p.marks[(((i / each & 1) * p.batch * p.H + bh + i / each / 2) * p.nchunks + chunk0) * p.marks_each + i % each];
    if (!__syncthreads_or(any)) return;
  }
  auto segment = [&](auto reversed, const int item) __attribute__((always_inline)) {
    constexpr bool REV = decltype(reversed)::value;
    constexpr int kWaves = NW / HP;                 // of a head
    constexpr int KK = KD / 32, KS = C / 32, IT = C / 16, kWV = 16 * kWaves, kPairs = Sh::kPairs, kThreads = 64 * NW;
    constexpr int kDecayWave = kWaves - 1;          // has the least to do with the pairs

    const int all_wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6), part = all_wave / kWaves, wave = all_wave % kWaves;
    using Place = LinPlace<C, HP, kWV, OWN, REV>;
    f32x4 S[KK][2];
    int begin = 0;                                  // the chunk that the walk begins with (again, behind one that was walked token by token)
    do {
    // (Parameters and places are formed anew here, and behind the walk: kept, they would not leave its registers room.)
    const LinParams& p = lin_again(kBoth && REV ? 1 : 0);
    int it = item;
    asm volatile("" : "+s"(it), "+s"(begin));
    int lane = lin_lane(), tid = 64 * all_wave + lane, l16 = lane & 15, g = lane >> 4;
    const Place place(p, it, part);
    const int nb = place.nb, chunks = place.chunks, col0 = place.col0, wcol = wave * 16;
    const int64_t h = place.h, b = place.b, bh = place.bh;

    // f(four state values, which of them, its place in a head's state in bytes): beyond the state for what is not there, where loads give
    // zero and stores are dropped
    auto each_state = [&](const LinParams& p, int col0, int row, int col, auto&& f) __attribute__((always_inline)) {
      const int lane = lin_lane(), l16 = lane & 15, g = lane >> 4, n = col0 + wcol + l16, left = p.kd - 8 * g;
      row *= 4;
      col = n < p.vd ? 4 * col * n : kNowhere;
#pragma unroll
      for (int a = 0; a < KK; ++a)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int kd = 32 * a + 4 * u + r;
            f(S[a][u], r, kd < left ? row * (8 * g + kd) + col : kNowhere);
          }
    };
    auto load_state = [&](const LinParams& p, int col0, const float* at, int row, int col, int size) __attribute__((always_inline)) {
      const auto from = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(at), (short)0, size * 4, 0x00020000);
      each_state(p, col0, row, col, [&](f32x4& s, int r, int at) { s[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(from, at, 0, 0)); });
    };
    auto store_state = [&](const LinParams& p, int col0, float* at) __attribute__((always_inline)) {
      const auto to = __builtin_amdgcn_make_buffer_rsrc(at, (short)0, p.kd * p.vd * 4, 0x00020000);
      each_state(p, col0, int(p.s_row), int(p.s_col),
                 [&](f32x4& s, int r, int at) { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s[r]), to, at, 0, 0); });
    };

    auto start_of = [&](int ci) { return place.start_of(ci); };
    auto tokens_of = [&](int64_t t0) { return place.tokens_of(t0); };

    LinTile<T, KD, C, kThreads> tq, tk;
    LinTile<T, kWV, C, 64 * kWaves> tv;
    T* const sv = sh.v + part * C * kWV;
    T* const sp = STATE ? sh.p : sh.p + part * NPP * kPairs;
    const int nothing = (HP - part) * NPP * kPairs;
    constexpr int64_t kOn = REV ? -C : C;           // tokens from a chunk to the next
    // the log decays of a chunk, a chunk ahead of its operands
    const float* gates = nullptr;
    const int gsl = int(p.g_sl);
    float gate = 0.f;
    auto load_gate = [&](int64_t t0) {
      if (wave == kDecayWave) {
        const int n = tokens_of(t0), lane = lin_lane();
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(gates), (short)0, ((n - 1) * gsl + 1) * 4, 0x00020000);
        gate = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, lane < n ? lane * gsl * 4 : 0x7ffffff0, 0, 0));
        gates += kOn * gsl;
      }
    };

    double total = 0.0;                             // STATE: log2 of the segment's decay
    bool anew = false;
    // The state is held as a multiple `scale` (its logarithm, base 2) of the accumulators, which takes up the
    // chunks' decays until it leaves 2^-16 .. 2^16: most chunks then leave the accumulators as they are.
    double scale = 0.0;
    // the factors of a chunk's tokens, of the gates that kDecayWave has loaded
    auto mark = [&](const LinParams& p, const Place& place, int64_t chunk, bool marked) {
      p.marks[(((REV ? p.batch * p.H : 0) + place.bh) * p.nchunks + chunk) * p.nblk + place.nb] = marked;
    };
    auto decays = [&](LinDecays<C>& d, int64_t chunk) {
      const int lane = lin_lane();
      double c = double(gate) * 1.4426950408889634;
      const bool start = c < -150.0;                // a decay below 2^-150 is none at all
      const bool any_strong = DOT && !REV && __ballot(c < kStrong) != 0;
      if (start) c = 0.0;
#pragma unroll
      for (int s = 1; s < 64; s *= 2) {
        const double o = __shfl_up(c, s);
        if (lane >= s) c += o;
      }
      const uint64_t starts = __ballot(start);
      const double all = __shfl(c, 63);
      const uint64_t upto = (uint64_t(2) << lane) - 1;
      const uint64_t before = starts & upto, after = starts & ~upto;
      const double next = scale + all;
      const bool fold = starts != 0 || !(next > -16.0 && next < 16.0);
      const double held = fold ? 0.0 : next;
      const float f = REV ? (after ? 0.f : lin_exp2(float(all - c + scale))) : (before ? 0.f : lin_exp2(float(c + scale)));
      const float w = REV ? (before ? 0.f : lin_exp2(float(c - held))) : (after ? 0.f : lin_exp2(float(all - c - held)));
      if (lane < C) {
        d.hi[lane] = float(c);
        d.lo[lane] = float(c - double(float(c)));
        d.f[lane] = f * p.fscale;
        d.w[lane] = w * p.wscale;
        d.lim[lane] = REV ? (after ? __builtin_ctzll(after) - 1 : C) : (before ? 63 - __builtin_clzll(before) : 0);
      }
      if (lane == 0) {
        d.mul = starts ? 0.f : fold ? lin_exp2(float(next)) : 1.f;
        d.before = __builtin_amdgcn_exp2f(float(scale));
        d.after = __builtin_amdgcn_exp2f(float(held));
      }
      scale = held;
      if (DOT && p.marks && lane == 0)
        mark(p, place, chunk, !REV && starts == 0 && all > kGone && any_strong && (chunk > 0 || p.ends & 1) && (chunk + 1 < p.nchunks || p.ends & 2));
      if (STATE) {
        total += all;
        anew |= starts != 0;
      }
    };

    // whether any of the 32 channels are there (the first are; of a width that is no power of two the last may not be)
    auto there = [&](int a) { return a <= KK / 2 || 32 * a < p.kd; };
    // ---- the pairs: P_ij = e^{c_i - c_j} (q_i . k_j), as its transpose's tiles (lane: one i, four j)
    auto pairs = [&](const LinDecays<C>& dec) {
      constexpr int kUnits = C == 64 ? 6 : 2;       // 16 rows by 32 keys, those that see each other
#pragma unroll 1
      for (int unit = wave; unit < kUnits; unit += kWaves) {
        // C = 64 forward: (0,0) (1,0) (2,0) (2,1) (3,0) (3,1); backward: (3,1) (2,1) (1,1) (1,0) (0,1) (0,0)
        int it = C == 32 ? unit : unit < 2 ? unit : unit / 2 + 1, ks = C == 32 || unit < 2 ? 0 : unit & 1;
        if (REV) { it = IT - 1 - it; ks = KS - 1 - ks; }
        f32x4 acc[2] = {};
        frag fq[2], fk[2][2];                       // (those of the next product on their way during this one)
        auto ask = [&](int a) {
          fq[a & 1] = io::template row<KD>(sh.q, 16 * it + l16, 32 * a + 8 * g);
#pragma unroll
          for (int u = 0; u < 2; ++u) fk[a & 1][u] = io::template row<KD>(sh.k, 32 * ks + 16 * u + l16, 32 * a + 8 * g);
        };
        ask(0);
#pragma unroll
        for (int a = 0; a < KK; ++a) {
          if (a + 1 < KK) ask(a + 1);
          __builtin_amdgcn_sched_barrier(0);
          if (there(a)) {
#pragma unroll
            for (int u = 0; u < 2; ++u) acc[u] = io::mma(fk[a & 1][u], fq[a & 1], acc[u]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        const int i = 16 * it + l16;
        const float chi = dec.hi[i], clo = dec.lo[i];
        const int lim = dec.lim[i];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j0 = 32 * ks + 16 * u + 4 * g;
          const int pi = REV ? IT - 1 - it : it, pj = REV ? IT - 1 - 2 * ks - u : 2 * ks + u;
          if (pj > pi) continue;                    // (the block beyond the diagonal's)
          f32x4 val;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = j0 + r;
            const float d = (chi - dec.hi[j]) + (clo - dec.lo[j]);
            const bool seen = REV ? j >= i && j <= lim : j <= i && j >= lim;
            val[r] = acc[u][r] * (__builtin_amdgcn_exp2f(seen ? (REV ? -d : d) : -1e30f) * p.pscale);
          }
#pragma unroll
          for (int x = 0; x < NPP; ++x) {
            io::store(sp + x * kPairs + lin_pair_at<T>(pi, pj, l16, 4 * g), val);
            if (x + 1 < NPP)
#pragma unroll
              for (int r = 0; r < 4; ++r) val[r] = lin_rest(val[r]);
          }
        }
      }
    };
    // ---- out^T, columns of v down, tokens across: the part of the state
    f32x4 acc[IT];
    auto from_state = [&](const LinDecays<C>& dec) {
#pragma unroll
      for (int it = 0; it < IT; ++it) acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
      constexpr int kTwo = IT / 2;
      frag fq[2][2], fs[NP];
      auto ask = [&](int i) {
#pragma unroll
        for (int x = 0; x < 2; ++x) fq[i & 1][x] = io::template row<KD>(sh.q, 16 * (2 * (i % kTwo) + x) + l16, 32 * (i / kTwo) + 8 * g);
      };
      ask(0);
#pragma unroll
      for (int i = 0; i < KK * kTwo; ++i) {
        const int a = i / kTwo, it = 2 * (i % kTwo);
        if (i + 1 < KK * kTwo) ask(i + 1);
        __builtin_amdgcn_sched_barrier(0);
        if (there(a)) {
          if (it == 0) lin_split<T, NP>(__builtin_shufflevector(S[a][0], S[a][1], 0, 1, 2, 3, 4, 5, 6, 7), fs);
#pragma unroll
          for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) acc[it + x] = io::mma(fs[n], fq[i & 1][x], acc[it + x]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const float f = dec.f[16 * it + l16];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[it][r] *= f;
      }
    };
    frag fv[KS];
    auto values = [&] {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) fv[ks] = io::template column<kWV>(sv, 32 * ks + 8 * g, wcol, 4, l16);
    };
    // ... and that of the pairs; false if something of it is not finite
    auto from_pairs = [&] {
      float chk = 0.f;
      auto seen = [](int it, int ks) { return REV ? 32 * ks + 31 >= 16 * it : 32 * ks <= 16 * it + 15; };
#pragma unroll
      for (int x = 0; x < NPP; ++x) {
        if (x > 0) __builtin_amdgcn_sched_barrier(0);
        frag fp[IT][KS];
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            if (seen(it, ks)) {
              // (lane groups 0 and 1 have the first block's values, 2 and 3 the second's: of the diagonal's, one is not kept)
              const int pi = REV ? IT - 1 - it : it, pj = REV ? IT - 1 - 2 * ks : 2 * ks, more = REV ? -(g >> 1) : g >> 1;
              const int at = lin_pair_at<T>(pi, pj, 16 * more + l16, 8 * (g & 1));
              const bool whole = REV ? pj <= pi : pj < pi;
              fp[it][ks] = io::pair(sp, whole || pj + more <= pi ? x * kPairs + at : nothing);
            }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int it = 0; it < IT; ++it)
            if (seen(it, ks)) acc[it] = io::mma(fv[ks], fp[it][ks], acc[it]);
      }
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) chk = fmaf(acc[it][r], 0.f, chk);
      return __all(chk == 0.f);
    };
    // Four columns of a row of the chunk's tile of `out`; rows and columns that are not there are beyond it,
    // and dropped.
    const int ocols = p.vd - (col0 + wcol), osl = int(p.o_sl), xsl = int(p.x.sl), oes = p.out_f32 ? 4 : int(sizeof(T));
    char* out = nullptr;
    const T* xs = nullptr;
    // x's rows, asked for before they meet the result (16 bits a value: two a register)
    constexpr int kXRegs = sizeof(T) == 2 ? 2 : 4;
    uint32_t xv[DOT ? IT : 1][kXRegs];
    auto load_x = [&](int n) {
      constexpr int kOutside = 0x7ffffff0;
      const int room = ocols - 4 * g, es = int(sizeof(T));
      const auto from = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(xs), (short)0,
                                                          ocols > 0 ? ((n - 1) * xsl + ocols) * es : 0, 0x00020000);
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int i = 16 * it + l16, at = i < n ? (i * xsl + 4 * g) * es : kOutside;
        if (ocols >= 16) {
          if constexpr (sizeof(T) == 2) {
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(from, at, 0, 0);
            xv[it][0] = v[0]; xv[it][1] = v[1];
          } else {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(from, at, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) xv[it][r] = v[r];
          }
        } else {
#pragma unroll
          for (int r = 0; r < kXRegs; ++r) xv[it][r] = 0;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int to = r < room ? at + r * es : kOutside;
            if constexpr (sizeof(T) == 2)
              xv[it][r / 2] |= uint32_t(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(from, to, 0, 0))) << (16 * (r % 2));
            else
              xv[it][r] = __builtin_amdgcn_raw_buffer_load_b32(from, to, 0, 0);
          }
        }
      }
    };
    // the products of x with what a row has of the state
    auto dots = [&] {
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = sizeof(T) == 4 ? __uint_as_float(xv[it][r % kXRegs])
                                         : __uint_as_float(r % 2 ? xv[it][r / 2] & 0xffff0000u : xv[it][r / 2] << 16);
          sum = fmaf(acc[it][r], x, sum);
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (g == 0) sh.dot[all_wave][16 * it + l16] = sum;
      }
    };
    // A state kept at `to`, a block of [the walk of dq's rows][c_row]: a lane of the backward walk, whose rows and columns are
    // exchanged, then has four values in one access.
    auto kept_at = [&](const LinParams& p, float* at) {
      return __builtin_amdgcn_make_buffer_rsrc(at, (short)0, int(CROSS ? p.vd : p.kd) * int(p.c_row) * 4, 0x00020000);
    };
    auto keep = [&](const LinParams& p, const Place& place, float* at, float scale) __attribute__((always_inline)) {
      const auto to = kept_at(p, at);
      const int lane = lin_lane(), n = place.col0 + wcol + (lane & 15), kd0 = 8 * (lane >> 4), row = 4 * int(p.c_row);
      const int off = n < int(p.c_row) ? row * kd0 + 4 * n : kNowhere;
#pragma unroll
      for (int a = 0; a < KK; ++a)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            __builtin_amdgcn_raw_buffer_store_b32(n < p.vd ? __float_as_uint(S[a][u][r] * scale) : 0u, to, off + row * (32 * a + 4 * u + r), 0, 0);
    };
    auto kept_block = [&](const LinParams& p, const Place& place, int64_t chunk) {
      return p.kept + (place.bh * p.nchunks + chunk) * (int64_t(CROSS ? p.vd : p.kd) * p.c_row);
    };
    // what a walk keeps before chunk `chunk` of its direction: the states between every lin_span() chunks, or (KEEP) the others
    auto keep_some = [&](const LinParams& p, const Place& place, int64_t chunk, float scale) __attribute__((always_inline)) {
      if (KEEP || (DOT && !REV)) {
        if ((chunk % lin_span() == 0) != KEEP) keep(p, place, kept_block(p, place, chunk), scale);
      } else if (DOT && (chunk + 1) % lin_span() == 0 && chunk + 1 < p.nchunks) {
        keep(p, place, p.back + (place.bh * ((p.nchunks + lin_span() - 1) / lin_span()) + (chunk + 1) / lin_span()) * (int64_t(p.kd) * p.c_row), scale);
      }
    };
    // ... and the sum of its products with the walk's
    f32x4 kept[CROSS ? KK : 1][2];
    auto load_kept = [&](const LinParams& p, const Place& place, int64_t chunk, int half) __attribute__((always_inline)) {
      const auto from = kept_at(p, kept_block(p, place, chunk));
      const int lane = lin_lane(), n = place.col0 + wcol + (lane & 15), kd0 = 8 * (lane >> 4);
      const int at = n < p.vd ? 4 * (n * int(p.c_row) + kd0) : kNowhere;
#pragma unroll
      for (int a = KK / 2 * half; a < KK / 2 * (half + 1); ++a)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          kept[a][u] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, at + 4 * (32 * a + 4 * u), 0, 0));
    };
    auto cross = [&](const LinParams& p, float scale) __attribute__((always_inline)) {
      const int left = p.kd - 8 * (lin_lane() >> 4);
      float sum = 0.f;
#pragma unroll
      for (int a = 0; a < KK; ++a)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = kept[a][u][r];
            sum = fmaf(32 * a + 4 * u + r < left ? x : 0.f, S[a][u][r] * scale, sum);      // (behind a row's end lies the next one)
          }
#pragma unroll
      for (int x = 32; x > 0; x /= 2) sum += __shfl_xor(sum, x);
      if (lin_lane() == 0) sh.cross[all_wave] = sum;
    };
    auto store_cross = [&](const LinParams& p, const Place& place, int64_t chunk) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += sh.cross[part * kWaves + w];
      if (lin_lane() == 0) p.cross[(place.nb * p.batch * p.H + place.bh) * p.nchunks + chunk] = sum;
    };
    auto write = [&](int n) {
      constexpr int kOutside = 0x7ffffff0;
      const int room = ocols - 4 * g;               // columns that are there
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(out, (short)0,
                                                          ocols > 0 ? ((n - 1) * osl + ocols) * oes : 0, 0x00020000);
      const int at = (l16 * osl + 4 * g) * oes, step = 16 * osl * oes;
      auto put = [&](f32x4 v, int to) {
        if (sizeof(T) == 4 || p.out_f32) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, to, 0, 0);
        } else {
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4)), rsrc, to, 0, 0);
        }
      };
      if (n == C && ocols >= 16) {
#pragma unroll
        for (int it = 0; it < IT; ++it) put(acc[it], at + it * step);
      } else {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const int to = 16 * it + l16 < n ? at + it * step : kOutside;
          put(acc[it], room >= 4 ? to : kOutside);
          if (room > 0 && room < 4) {
#pragma unroll
            for (int r = 0; r < 3; ++r) {
              const int one = r < room ? to + r * oes : kOutside;
              if (sizeof(T) == 4 || p.out_f32)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[it][r]), rsrc, one, 0, 0);
              else
                __builtin_amdgcn_raw_buffer_store_b16((short)bf16_rne(acc[it][r]), rsrc, one, 0, 0);
            }
          }
        }
      }
    };
    auto multiply = [&](float m) {
      if (__builtin_amdgcn_readfirstlane(__float_as_int(m)) == __float_as_int(1.f)) return;
#pragma unroll
      for (int a = 0; a < KK; ++a)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[a][u][r] *= m;
    };
    // ---- the new state: w_j v_j in parts, so that nothing of what is added to fp32 is lost
    auto update = [&](const LinDecays<C>& dec) {
      multiply(dec.mul);
      frag fk[2][2], fw[NX];
      auto ask = [&](int i) {
#pragma unroll
        for (int u = 0; u < 2; ++u) fk[i & 1][u] = io::template column<KD>(sh.k, 32 * (i / KK) + 8 * g, 32 * (i % KK) + 4 * u, 8, l16);
      };
      ask(0);
#pragma unroll
      for (int i = 0; i < KS * KK; ++i) {
        const int ks = i / KK, a = i % KK;
        if (i + 1 < KS * KK) ask(i + 1);
        if (a == 0) {
          f32x8 x = io::wide(fv[ks]);
          const f32x4* const w = reinterpret_cast<const f32x4*>(dec.w + 32 * ks + 8 * g);
          x *= __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7);
          lin_split<T, NX>(x, fw);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (there(a)) {
#pragma unroll
          for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u) S[a][u] = io::mma(fk[i & 1][u], fw[n], S[a][u]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    auto first_state = [&](const LinParams& p, const Place& place) __attribute__((always_inline)) {
      const int block = p.kd * p.vd;                // of a head's state
      const float* from = p.s0 ? p.s0 + place.bh * block : nullptr;
      int row = int(p.s_row), col = int(p.s_col), size = block;
      if (OWN) {
        from = nullptr;
      } else if (KEEP || CROSS) {
        if (place.seg != (CROSS ? p.nseg - 1 : 0)) {
          row = CROSS ? 1 : int(p.c_row);
          col = CROSS ? int(p.c_row) : 1;
          size = (CROSS ? p.vd : p.kd) * int(p.c_row);
          from = CROSS ? p.back + (place.bh * p.nseg + place.seg + 1) * size : p.kept + (place.bh * p.nchunks + place.chunk0) * size;
        }
      } else if (p.nseg > 1) {
        from = p.seg + (place.bh * p.nseg + place.seg) * block;
      }
      if (from) {
        load_state(p, place.col0, from, row, col, size);
      } else {
#pragma unroll
        for (int a = 0; a < KK; ++a) S[a][0] = S[a][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    };
    if (begin == 0) first_state(p, place);

    // Inside a chunk a token is kept from another by a zero factor, which an infinity or a NaN turns into a
    // NaN.  If anything that comes out is not finite, what the wavefront has formed of the chunk is dropped, and it and
    // those behind it are walked token by token until the state is finite.  Where the state before the chunk is not, it may be
    // by the multiple that it is held as (up to 2^16 of it): all of the segment is walked so then, from its first token.
    // whether anything takes the state behind the last chunk
    const bool wanted = OWN || (p.s1 && place.seg == (REV ? 0 : p.nseg - 1));
    const bool with = DOT && p.dot != nullptr;     // the decays' gradient is
    bool done = true;
    int ci = begin;
    int64_t t0 = start_of(ci);
    if (!STATE) tq.init(p.q, b, h, t0, 0, p.kd);
    tk.init(p.k, b, h, t0, 0, p.kd);
    tv.init(p.v, b, h, t0, col0, p.vd);
    gates = p.g + b * p.g_sb + h * p.g_sh + t0 * p.g_sl;
    if (!STATE) out = place.out_at(p, t0, col0 + wcol, oes);
    if (DOT) xs = place.template x_at<T>(p, t0, col0 + wcol);
    begin = 0;
    const T *now_q = tq.at, *now_k = tk.at, *now_v = tv.at;
    if (CROSS) load_kept(p, place, t0 / C, 0);
    load_gate(t0);
    if (!STATE) tq.template load<REV>(tid, tokens_of(t0));
    tk.template load<REV>(tid, tokens_of(t0));
    tv.template load<REV>(64 * wave + lane, tokens_of(t0));
    if (wave == kDecayWave) decays(sh.dec[part][ci & 1], t0 / C);
    if (ci + 1 < chunks) load_gate(t0 + kOn);
    if (!STATE && tid == 0) sh.bad = 0;
    if (!STATE && tid < 8) sh.p[HP * NPP * kPairs + tid] = T(0);
    for (;; ++ci, t0 += kOn) {
      LinDecays<C>& dec = sh.dec[part][ci & 1];
      const int n = tokens_of(t0);
      lane = lin_lane();
      tid = 64 * all_wave + lane;
      const int vid = 64 * wave + lane;             // of the head's threads
      l16 = lane & 15;
      g = lane >> 4;
      // (half of what is kept is on its way through the update, half from here on)
      if (CROSS) load_kept(p, place, t0 / C, 1);
      if (!STATE) tq.store(sh.q, tid, now_q, n);
      tk.store(sh.k, tid, now_k, n);
      tv.store(sv, vid, now_v, n);
      __syncthreads();
      const bool more = ci + 1 < chunks;
      const int next = more ? tokens_of(t0 + kOn) : 0;
      if (!STATE) now_q = tq.at;
      now_k = tk.at;
      now_v = tv.at;
      if (wave == kDecayWave && more) decays(sh.dec[part][(ci + 1) & 1], t0 / C + (REV ? -1 : 1));
      if (!STATE) {
        // (the next chunk's operands are asked for one by one, and not all of them at a time)
        if (more) tq.template load<REV>(tid, next);
        if (DOT && with) keep_some(p, place, t0 / C, dec.before);
        pairs(dec);
        if (more) tk.template load<REV>(tid, next);
        from_state(dec);
        __syncthreads();
      }
      if (KEEP) keep_some(p, place, t0 / C, dec.before);
      if (CROSS) {
        cross(p, dec.before);
        if (more) load_kept(p, place, t0 / C - 1, 0);
      }
      if (STATE && more) tk.template load<REV>(tid, next);
      if (more) tv.template load<REV>(vid, next);
      if (ci + 2 < chunks) load_gate(t0 + 2 * kOn);
      values();
      if (DOT && with) {
        load_x(n);
        dots();
      }
      if (!STATE) {
        done = from_pairs();
        if (done)
          write(n);
        else if (lane == 0)
          sh.bad = 1;
        out += kOn * osl * oes;
        if (DOT) xs += kOn * xsl;
      }
      if (done && (more || wanted)) update(dec);
      __syncthreads();
      if (!STATE && sh.bad != 0) break;
      if (CROSS && wave == 0) store_cross(p, place, t0 / C);
      if (DOT && with && vid < n) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += sh.dot[part * kWaves + w][vid];
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(p.dot + (nb * p.batch * p.H + bh) * p.L + t0, (short)0, n * 4, 0x00020000);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sum), rsrc, vid * 4, 0, 0);
      }
      if (ci + 1 == chunks) break;
    }
    // the accumulators as the state itself
    multiply(STATE || done ? sh.dec[part][ci & 1].after : sh.dec[part][ci & 1].before);
    {
      const LinParams& p = lin_again(kBoth && REV ? 1 : 0);
      int it = item;
      asm volatile("" : "+s"(it), "+s"(ci));
      const Place place(p, it, part);
      const int col0 = place.col0, chunks = place.chunks;
      const int64_t h = place.h, b = place.b, bh = place.bh;
      const bool bad = !STATE && sh.bad != 0, ends = STATE || (p.s1 && place.seg == (REV ? 0 : p.nseg - 1));
      bool again = false;
      if (STATE || bad || ends) {
        float chk = 0.f;
#pragma unroll
        for (int a = 0; a < KK; ++a)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) chk = fmaf(S[a][u][r], 0.f, chk);
        again = __syncthreads_or(chk != 0.f);
      }
      // ---- token by token, with choices in the place of zero factors; the chunks before `from` stand, `done`: that one too
      if (bad || again) {
        const int from = STATE ? 0 : bad ? ci : chunks, oes = p.out_f32 ? 4 : int(sizeof(T));
        if (again) first_state(p, place);
        float* const row_q = reinterpret_cast<float*>(sh.k);         // [KD], and of k
        float* const row_k = row_q + KD;
        const T* const base_q = STATE ? nullptr : tq.head(p.q, b, h, 0);
        const T *const base_k = tk.head(p.k, b, h, 0), *const base_v = tv.head(p.v, b, h, col0);
        const float* const base_g = p.g + b * p.g_sb + h * p.g_sh;
#pragma unroll 1
        for (int ci = again ? 0 : from; ci < chunks; ++ci) {
          const int64_t t0 = place.start_of(ci);
          const int n = place.tokens_of(t0);
          const bool stands = !STATE && (ci < from || (ci == from && done));
          const bool with = ci >= from && DOT && p.dot != nullptr;
          // (a wavefront whose first chunk stands holds the state behind it by now, and has kept the one before it)
          if (((DOT && with) || KEEP) && (!stands || again)) keep_some(p, place, t0 / C, 1.f);
          if (DOT && with && wave == kDecayWave && lin_lane() == 0) mark(p, place, t0 / C, true);
          if (CROSS) {
            load_kept(p, place, t0 / C, 0);
            load_kept(p, place, t0 / C, 1);
            cross(p, 1.f);
            __syncthreads();
            if (wave == 0) store_cross(p, place, t0 / C);
          }
          // the state before the chunk, what the tokens since have left of it, and whether that is none
          f32x4 S0[DOT ? KK : 1][2];
          if constexpr (DOT)
#pragma unroll
            for (int a = 0; a < KK; ++a) S0[a][0] = S[a][0], S0[a][1] = S[a][1];
          float left = p.fscale;
          bool gone = false;
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
            const int64_t t = t0 + (REV ? n - 1 - i : i);
            const int lane = lin_lane(), tid = 64 * all_wave + lane, l16 = lane & 15, g = lane >> 4;
            __syncthreads();
            for (int c = tid; c < KD; c += kThreads) {
              row_q[c] = !STATE && c < p.kd ? io::widen(base_q[t * p.q.sl + c]) : 0.f;
              row_k[c] = c < p.kd ? io::widen(base_k[t * p.k.sl + c]) : 0.f;
            }
            __syncthreads();
            const int col = col0 + wcol + l16;
            const float v = col < p.vd ? io::widen(base_v[t * p.v.sl + wcol + l16]) * p.wscale : 0.f;
            const double c = double(base_g[t * p.g_sl]) * 1.4426950408889634;
            const bool start = c < -150.0;
            const float d = start ? 0.f : lin_decay(float(c));
            float out = 0.f, of_state = 0.f;
            if (DOT && !REV) {
              gone |= start;
              left *= d;
            }
            if (!stands || again) {
#pragma unroll
              for (int a = 0; a < KK; ++a)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int r = 0; r < 4; ++r) {
                    const int kd = 32 * a + 8 * g + 4 * u + r;
                    float s = S[a][u][r];
                    if (!REV) s = start ? 0.f : s * d;
                    if (kd < p.kd) {
                      s = fmaf(row_k[kd], v, s);
                      out = fmaf(row_q[kd], s, out);
                      if (DOT) of_state = fmaf(row_q[kd], S0[a][u][r], of_state);
                    }
                    if (REV) s = start ? 0.f : s * d;
                    S[a][u][r] = s;
                  }
            }
            if (!STATE) {
              out += __shfl_xor(out, 16);
              out += __shfl_xor(out, 32);
              out *= p.fscale;
              if (!stands && col < p.vd) {
                if (g == 0) {
                  char* const to = place.out_at(p, t, col, oes);
                  if (p.out_f32)
                    *reinterpret_cast<float*>(to) = out;
                  else
                    io::narrow(reinterpret_cast<T*>(to), out);
                }
              }
              if (DOT && with) {
                float dot = 0.f;
                if (!gone && col < p.vd) dot = of_state * left * io::widen(*place.template x_at<T>(p, t, col));
                // (what a wavefront whose first chunk stands has left there is that chunk's)
                for (int x = 32; x > 0; x /= 2) dot += __shfl_xor(dot, x);
                if (lane == 0 && !stands) sh.dot[all_wave][t - t0] = dot;
                __syncthreads();
                if (wave == 0 && lane == 0) {
                  float sum = 0.f;
                  for (int w = 0; w < kWaves; ++w) sum += sh.dot[part * kWaves + w][t - t0];
                  p.dot[(place.nb * p.batch * p.H + bh) * p.L + t] = sum;
                }
              }
            }
            if (DOT && REV) {
              gone |= start;
              left *= d;
            }
          }
          if (!STATE && !(again && from > 0) && ci >= from && ci + 1 < chunks) {
            // back to chunks
            float chk = 0.f;
#pragma unroll
            for (int a = 0; a < KK; ++a)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) chk = fmaf(S[a][u][r], 0.f, chk);
            if (!__syncthreads_or(chk != 0.f)) {
              begin = ci + 1;
              break;
            }
          }
        }
        if (begin > 0) continue;
      }

      const int block = p.kd * p.vd;
      if (OWN) {
        store_state(p, col0, p.seg + (bh * p.nseg + place.seg) * block);
        if (wave == kDecayWave && lin_lane() == 0 && place.nb == 0)
          p.seg_decay[bh * p.nseg + place.seg] = anew ? -HUGE_VAL : total;
      } else if (!STATE && ends) {
        store_state(p, col0, p.s1 + bh * block);
      }
    }
    } while (begin > 0);
  };

  // The heads of a token lie next to one another, so the rows of one head are a power of two apart as a
  // rule, in one channel of the L2: an XCD takes the heads side by side.
  const int item = xcd_contiguous_block(blockIdx.x, gridDim.x);
  // (Two walks at once fill the compute units where one does not: 2 x 6 heads x 333 fp32, forward and backward, 118 us
  // one after the other, 86 so; where each fills them the time is the same.)
  constexpr std::true_type backward;
  constexpr std::false_type forward;
  if constexpr (WALK == LinWalk::backward || WALK == LinWalk::cross) {
    segment(backward, item);
  } else if constexpr (!kBoth) {
    segment(forward, item);
  } else {
    if (item & 1)
      segment(backward, item >> 1);
    else
      segment(forward, item >> 1);
  }
}

template <typename T, int KD, int NW, int HP, int C, LinWalk WALK>
hipError_t lin_start(const LinParams* p, int64_t segs, hipStream_t stream) {
  constexpr int kWalks = sizeof(LinWalks<WALK>) / sizeof(LinParams);
  const int64_t items = kWalks * p->batch * (p->H / HP) * p->nblk * segs;
  if (items == 0) return hipSuccess;
  LinWalks<WALK> walks;
  for (int i = 0; i < kWalks; ++i) walks.p[i] = p[i];
  lin_kernel<T, KD, NW, HP, C, WALK><<<dim3(uint32_t(items)), dim3(64 * NW), 0, stream>>>(walks);
  return hipGetLastError();
}

template <typename T, int KD, int NW, int HP>
hipError_t lin_launch(LinWalk walk, const LinParams* p, hipStream_t stream) {
  constexpr int C = lin_chunk(sizeof(T) == 2, KD);
  switch (walk) {
    case LinWalk::forward: return lin_start<T, KD, NW, HP, C, LinWalk::forward>(p, p->nseg, stream);
    case LinWalk::backward: return lin_start<T, KD, NW, HP, C, LinWalk::backward>(p, p->nseg, stream);
    case LinWalk::state: return lin_start<T, KD, NW, HP, C, LinWalk::state>(p, p->nseg - 1, stream);
    case LinWalk::states: return lin_start<T, KD, NW, HP, C, LinWalk::states>(p, p->nseg - 1, stream);
    case LinWalk::cross: return lin_start<T, KD, NW, HP, C, LinWalk::cross>(p, p->nseg, stream);
    // (the keys of these walks, and the queries, are do and v, each head's own)
    case LinWalk::keep:
      if constexpr (HP == 1) return lin_start<T, KD, NW, 1, C, LinWalk::keep>(p, p->nseg, stream);
      break;
    case LinWalk::grads:
      if constexpr (HP == 1) return lin_start<T, KD, NW, 1, C, LinWalk::grads>(p, p->nseg, stream);
  }
  return hipErrorInvalidValue;
}

template <typename T, int KD> hipError_t lin_choose(LinWalk walk, const LinParams* p, hipStream_t stream) {
  // (Gradients whose other width is above 128 have its chunks, and v's columns are more than 128 then.)
  if constexpr (sizeof(T) == 4 && KD < 256)
    if (p->chunk == 32) {
      if (walk == LinWalk::grads) return lin_start<T, KD, 8, 1, 32, LinWalk::grads>(p, p->nseg, stream);
      if (walk == LinWalk::keep) return lin_start<T, KD, 8, 1, 32, LinWalk::keep>(p, p->nseg, stream);
      if (walk == LinWalk::cross) return lin_start<T, KD, 8, 1, 32, LinWalk::cross>(p, p->nseg, stream);
      return hipErrorInvalidValue;
    }
  // Eight wavefronts for 128 columns; of at most 64 columns a workgroup has four, or takes two heads that share their
  // queries and keys, which it then stages once (4 x 80 heads on one q and k x 8192, 128 x 64 bf16: 660 us with
  // a head each, 560 so).
  if (p->vd > 64) return lin_launch<T, KD, 8, 1>(walk, p, stream);
  return p->pairs ? lin_launch<T, KD, 8, 2>(walk, p, stream) : lin_launch<T, KD, 4, 1>(walk, p, stream);
}

}  // namespace
}  // namespace selscan
