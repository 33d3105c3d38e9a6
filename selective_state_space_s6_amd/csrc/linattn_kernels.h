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
#pragma once

#include "device_common.h"
#include "scan_launch.h"

namespace selscan {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) float f32x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr float kTiny = 1.401298464e-45f;      // 2^-149

// What the walk needs of an element type: eight consecutive values of a contraction in one
// fragment (lane l: row or column l % 16, values 8 (l / 16) ..), and the product of two.
template <typename T> struct lin_io;
template <> struct lin_io<uint16_t> {
  using frag = bf16x8;
  static constexpr int kVec = 8;               // elements of 16 bytes
  static constexpr int kPad = 8;               // elements between LDS rows
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ frag row(const uint16_t* p) { return *reinterpret_cast<const frag*>(p); }
  // a column: values at rows r0 .. r0 + 7; the 16 lanes of a group ask for 4 rows of four 4-element
  // pieces, and the transposing read hands each lane its column
  static __device__ __forceinline__ frag column(const uint16_t* tile, int ld, int r0, int piece, int lane16) {
    const uint16_t* p = tile + (r0 + (lane16 >> 2)) * ld + piece;
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * ld));
    struct { s16x4 a, b; } v = {a, b};
    return __builtin_bit_cast(frag, v);
  }
  static __device__ __forceinline__ f32x8 wide(frag a) { return __builtin_convertvector(a, f32x8); }
  static __device__ __forceinline__ frag round(f32x8 a) { return __builtin_convertvector(a, frag); }
  static __device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
  // N consecutive values (N = 4, 8) to p: in LDS (aligned), or to global memory (on any element's boundary),
  // the first `room` of them
  template <int N> static __device__ __forceinline__ void store(uint16_t* p, const float* v) {
    typedef __attribute__((ext_vector_type(N))) __bf16 b;
    typedef __attribute__((ext_vector_type(N))) float f;
    f x;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v[i];
    *reinterpret_cast<b*>(p) = __builtin_convertvector(x, b);
  }
  template <int N> static __device__ __forceinline__ void put(uint16_t* p, const float* v, int room) {
    typedef __attribute__((ext_vector_type(N))) __bf16 b;
    typedef __attribute__((ext_vector_type(N))) float f;
    typedef b loose __attribute__((aligned(2)));
    f x;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v[i];
    if (room >= N)
      *reinterpret_cast<loose*>(p) = __builtin_convertvector(x, b);
    else
      for (int i = 0; i < N; ++i)
        if (i < room) p[i] = bf16_rne(v[i]);
  }
};
template <> struct lin_io<float> {
  using frag = f32x8;
  static constexpr int kVec = 4;
  static constexpr int kPad = 4;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ frag row(const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ frag column(const float* tile, int ld, int r0, int col) {
    frag v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[(r0 + e) * ld + col];
    return v;
  }
  static __device__ __forceinline__ f32x8 wide(frag a) { return a; }
  static __device__ __forceinline__ frag round(f32x8 a) { return a; }
  static __device__ __forceinline__ float widen(float b) { return b; }
  template <int N> static __device__ __forceinline__ void store(float* p, const float* v) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  }
  template <int N> static __device__ __forceinline__ void put(float* p, const float* v, int room) {
    typedef f32x4 loose __attribute__((aligned(4)));
    if (room >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) *reinterpret_cast<loose*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
      for (int i = 0; i < N; ++i)
        if (i < room) p[i] = v[i];
    }
  }
};

// Column l % 16 of a tile of 16 (piece 4 wide at `spread` elements): where the lane's column is,
// and where its transposing read begins.
template <typename T>
__device__ __forceinline__ typename lin_io<T>::frag lin_column(const T* tile, int ld, int r0, int first, int spread, int lane16) {
  if constexpr (sizeof(T) == 2)
    return lin_io<T>::column(tile, ld, r0, first + spread * (lane16 & 3), lane16);
  else
    return lin_io<T>::column(tile, ld, r0, first + spread * (lane16 >> 2) + (lane16 & 3));
}

// x as a sum of `N` values of the matrix cores' type (the first rounds x, the next what that
// left).  Where the first is not finite nothing is left.
template <typename T, int N>
__device__ __forceinline__ void lin_split(f32x8 x, typename lin_io<T>::frag* out) {
  out[0] = lin_io<T>::round(x);
#pragma unroll
  for (int n = 1; n < N; ++n) {
    const f32x8 w = lin_io<T>::wide(out[n - 1]);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fabsf(w[e]) < __builtin_inff() ? x[e] - w[e] : 0.f;
    out[n] = lin_io<T>::round(x);
  }
}

// What rounding to bfloat16 leaves of a value.
__device__ __forceinline__ float lin_rest(float v) {
  const float w = __uint_as_float(uint32_t(bf16_rne(v)) << 16);
  return fabsf(w) < __builtin_inff() ? v - w : 0.f;
}

// A product of decays that fp32 cannot hold is held at its smallest value: only a token that starts
// anew ends an infinity.
__device__ __forceinline__ float lin_decay(float log2d) {
  const float d = __builtin_amdgcn_exp2f(log2d);
  return d < kTiny ? kTiny : d;
}

// Tokens of a chunk: the LDS of a compute unit holds the tiles of a chunk of 64, but not those of 256
// fp32 channels.
template <typename T, int KD> constexpr int lin_chunk_of() { return sizeof(T) == 4 && KD == 256 ? 32 : 64; }

// Wavefronts a SIMD is to hold: two workgroups of a compute unit hide each other's waits; states of 256 x 32
// and more in a wavefront's registers leave room for one.
template <typename T, int KD, int NT> constexpr int lin_waves() { return KD * NT * (sizeof(T) == 4 ? 2 : 1) <= 256 ? 2 : 1; }

// What the tokens of a chunk are to one another.
template <int C> struct LinDecays {
  float hi[C], lo[C];       // log2 of the decays since the chunk's start, in two parts
  float f[C], w[C];         // factor of a row's product with the state; of a row's share in the new state
  int lim[C];               // the row's first visible key (forward), its last (backward)
  float carry;
  int fresh;                // a token of the chunk starts anew
};

template <typename T, int KD, int NT, bool STATE, int NPP>
struct alignas(16) LinShared {
  static constexpr int C = lin_chunk_of<T, KD>();
  static constexpr int kLdK = KD + lin_io<T>::kPad, kLdV = 64 * NT + lin_io<T>::kPad, kLdP = C + lin_io<T>::kPad;
  T q[STATE ? 8 : C * kLdK];
  T k[C * kLdK];
  T v[C * kLdV];
  T p[STATE ? 8 : NPP * C * kLdP];
  LinDecays<C> dec[2];      // this job's, and the next one's
  float dot[4][C];
  int bad;
};

// An operand's tile of C rows and W columns on its way: rows lo .. hi - 1 of `rows` tokens, zeros
// elsewhere.  A thread has 16-byte pieces of a row (on any element's boundary); where the width is
// not a multiple of a piece, the end of row `lane` is a piece of wavefront `tail`'s own.
template <typename T, int W, int LD, int C>
struct LinTile {
  static constexpr int V = lin_io<T>::kVec, kPieces = W / V, kRows = 256 / kPieces, N = C / kRows;
  u32x4 piece[N];
  T end[V - 1];

  __device__ __forceinline__ void load(const LinTensor& x, int64_t b, int64_t h, int64_t t0, int n, int lo, int hi, int col0,
                                       int width, int tail) {
    const int tid = threadIdx.x;
    const T* base = static_cast<const T*>(x.p) + b * x.sb + t0 * x.sl + (h / x.share) * x.sh + col0;
    const int sl = int(x.sl), cols = width - col0 < W ? width - col0 : W;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), (short)0, int(((n - 1) * sl + cols) * int(sizeof(T))),
                                                        0x00020000);
    const int row0 = tid / kPieces, c = (tid % kPieces) * V;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = row0 + i * kRows;
      const bool in = row >= lo && row < hi && c + V <= cols;
      piece[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, in ? (row * sl + c) * int(sizeof(T)) : kOutside, 0, 0);
    }
    if (cols % V != 0 && (tid >> 6) == tail) {
      const int row = tid & 63, first = cols - cols % V;
#pragma unroll
      for (int e = 0; e < V - 1; ++e) {
        const bool in = row >= lo && row < hi && first + e < cols;
        const int at = in ? (row * sl + first + e) * int(sizeof(T)) : kOutside;
        if constexpr (sizeof(T) == 2)
          end[e] = T(__builtin_amdgcn_raw_buffer_load_b16(rsrc, at, 0, 0));
        else
          end[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0));
      }
    }
  }
  __device__ __forceinline__ void store(T* tile, int col0, int width, int tail) const {
    const int tid = threadIdx.x, cols = width - col0 < W ? width - col0 : W;
    const int row0 = tid / kPieces, c = (tid % kPieces) * V;
    // (the piece of a row's end is its owner's)
    if (cols % V == 0 || c != cols - cols % V) {
#pragma unroll
      for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(tile + (row0 + i * kRows) * LD + c) = piece[i];
    }
    if (cols % V != 0 && (tid >> 6) == tail && (tid & 63) < C) {
      union { u32x4 v; T e[V]; } u;
      u.v = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < V - 1; ++e) u.e[e] = end[e];
      *reinterpret_cast<u32x4*>(tile + (tid & 63) * LD + cols - cols % V) = u.v;
    }
  }
  static constexpr int kOutside = 0x7ffffff0;    // beyond any tile: reads as zero
};

// What a workgroup does at once: the tokens lo .. hi - 1 of a chunk (all of it, or one token).
struct LinJob {
  int ci, lo, hi;
  bool single;
};

// One workgroup of four wavefronts walks the chunks of one segment of one (batch row, head) for 64 NT
// columns of v: wavefront w owns 16 NT of them, and the state's [KD][16 NT] in its accumulators,
// which are at once the operand of its product with the queries.
// STATE: only the state at the segment's end, from zero.
// NS: parts that a fp32 value is split into where it meets the matrix cores (the state; 3: the pairs too).
template <typename T, int KD, int NT, bool REV, bool STATE, int NS>
__global__ __launch_bounds__(256, (lin_waves<T, KD, NT>())) void lin_kernel(LinParams p) {
  using io = lin_io<T>;
  using frag = typename io::frag;
  constexpr int NP = sizeof(T) == 2 ? NS : 1, NPP = NP == 3 ? 3 : 1;
  using Sh = LinShared<T, KD, NT, STATE, NPP>;
  constexpr int C = Sh::C, KK = KD / 32, KS = C / 32, IT = C / 16;
  constexpr int NW = sizeof(T) == 2 ? 3 : 1;      // the state is held in fp32: what is added to it keeps 24 bits
  __shared__ Sh sh;

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int item = xcd_contiguous_block(blockIdx.x, gridDim.x);
  const int segs = STATE ? p.nseg - 1 : p.nseg;   // (nothing is behind the last segment)
  const int sidx = item % segs;
  const int seg = STATE && REV ? sidx + 1 : sidx;
  const int nb = (item / segs) % p.nblk;
  const int64_t bh = item / segs / p.nblk, b = bh / p.H, h = bh % p.H;
  const int64_t chunk0 = int64_t(seg) * p.seg_chunks;
  const int chunks = int(p.nchunks - chunk0 < p.seg_chunks ? p.nchunks - chunk0 : p.seg_chunks);
  const int col0 = nb * 64 * NT;
  // columns of v: tile nt, row or column m of it
  constexpr int kSpread = 4 * NT;
  const int wcol = wave * 16 * NT;

  f32x4 S[KK][2][NT];
  float* const seg_at = p.seg + ((bh * p.nblk + nb) * p.nseg + seg) * (KD * 64 * NT);
  const int64_t sbase = bh * p.kd * p.vd;
  auto zero_state = [&] {
#pragma unroll
    for (int a = 0; a < KK; ++a)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t) S[a][u][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  // f(four state values, which of them, its place in the head's state)
  auto each_state = [&](auto&& f) {
#pragma unroll
    for (int a = 0; a < KK; ++a)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int kd = 32 * a + 8 * g + 4 * u + r, n = col0 + wcol + kSpread * (l16 >> 2) + 4 * t + (l16 & 3);
            if (kd < p.kd && n < p.vd) f(S[a][u][t], r, p.s_row * kd + p.s_col * n);
          }
  };

  auto start_of = [&](int ci) { return (chunk0 + (REV ? chunks - 1 - ci : ci)) * C; };
  auto tokens_of = [&](int64_t t0) { return int(p.L - t0 < C ? p.L - t0 : C); };
  auto whole = [&](int ci) { return LinJob{ci, 0, tokens_of(start_of(ci)), false}; };
  auto first_token = [&](int ci) {
    const int t = REV ? tokens_of(start_of(ci)) - 1 : 0;
    return LinJob{ci, t, t + 1, true};
  };

  LinTile<T, KD, Sh::kLdK, C> tq, tk;
  LinTile<T, 64 * NT, Sh::kLdV, C> tv;
  float gate = 0.f;
  auto load = [&](const LinJob& j) {
    const int64_t t0 = start_of(j.ci);
    const int n = tokens_of(t0);
    if (!STATE) tq.load(p.q, b, h, t0, n, j.lo, j.hi, 0, p.kd, 0);
    tk.load(p.k, b, h, t0, n, j.lo, j.hi, 0, p.kd, 1);
    tv.load(p.v, b, h, t0, n, j.lo, j.hi, col0, p.vd, 2);
    if (wave == 3) {
      gate = 0.f;
      if (lane >= j.lo && lane < j.hi) gate = p.g[b * p.g_sb + (t0 + lane) * p.g_sl + h * p.g_sh];
    }
  };

  double total = 0.0;                             // STATE: log2 of the segment's decay
  bool anew = false;
  // the factors of a job's tokens, of the gates that wavefront 3 has loaded
  auto decays = [&](LinDecays<C>& d) {
    double c = double(gate) * 1.4426950408889634;
    const bool start = c < -150.0;                // a decay below 2^-150 is none at all
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
    const float in = before ? 0.f : lin_decay(float(c));
    const float out = after ? 0.f : lin_decay(float(all - c));
    if (lane < C) {
      d.hi[lane] = float(c);
      d.lo[lane] = float(c - double(float(c)));
      d.f[lane] = (REV ? out : in) * p.fscale;
      d.w[lane] = (REV ? in : out) * p.wscale;
      d.lim[lane] = REV ? (after ? __builtin_ctzll(after) - 1 : C) : (before ? 63 - __builtin_clzll(before) : 0);
    }
    if (lane == 0) {
      d.carry = lin_decay(float(all));
      d.fresh = starts != 0;
    }
    if (STATE) {
      total += all;
      anew |= starts != 0;
    }
  };

  LinJob job = whole(0);
  zero_state();
  if (!STATE) {
    if (p.nseg > 1) {
#pragma unroll
      for (int a = 0; a < KK; ++a)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            S[a][u][t] = *reinterpret_cast<const f32x4*>(seg_at + (((a * 2 + u) * NT + t) * 256 + tid) * 4);
    } else if (p.s0) {
      each_state([&](f32x4& s, int r, int64_t at) { s[r] = p.s0[sbase + at]; });
    }
  }

  // A chunk is first walked as a whole.  Inside it a token is kept from another by a zero factor, which
  // an infinity or a NaN would turn into a NaN: if anything that comes out is not finite, what the
  // wavefront has formed is dropped and the chunk is walked token by token.  `done`: what this
  // wavefront formed of the whole chunk stands.
  bool done = false, retry = false, ahead = false;
  for (int cur = 0;; cur ^= 1) {
    LinDecays<C>& dec = sh.dec[cur];
    if (!ahead) {
      load(job);
      if (wave == 3) decays(dec);
    }
    const int64_t t0 = start_of(job.ci);
    if (!STATE) tq.store(sh.q, 0, p.kd, 0);
    tk.store(sh.k, 0, p.kd, 1);
    tv.store(sh.v, col0, p.vd, 2);
    __syncthreads();
    // ---- the next job's operands are asked for
    LinJob next = job;
    if (job.single && (REV ? job.lo > 0 : job.hi < tokens_of(t0))) {
      next.lo += REV ? -1 : 1;
      next.hi = next.lo + 1;
    } else if (job.ci + 1 < chunks) {
      next = STATE && retry ? first_token(job.ci + 1) : whole(job.ci + 1);
    } else {
      next.ci = chunks;
    }
    if (next.ci < chunks) load(next);
    if (!STATE && tid == 0) sh.bad = 0;

    // ---- the pairs: P_ij = e^{c_i - c_j} (q_i . k_j), as its transpose's tiles (lane: one i, four j)
    if (!STATE) {
      constexpr int kUnits = C == 64 ? 6 : 2;     // 16 rows by 32 keys, those that see each other
#pragma unroll 1
      for (int unit = wave; unit < kUnits; unit += 4) {
        // C = 64 forward: (0,0) (1,0) (2,0) (2,1) (3,0) (3,1); backward: (3,1) (2,1) (1,1) (1,0) (0,1) (0,0)
        int it = C == 32 ? unit : unit < 2 ? unit : unit / 2 + 1, ks = C == 32 || unit < 2 ? 0 : unit & 1;
        if (REV) { it = IT - 1 - it; ks = KS - 1 - ks; }
        f32x4 acc[2] = {};
#pragma unroll
        for (int a = 0; a < KK; ++a) {
          const frag fq = io::row(sh.q + (16 * it + l16) * Sh::kLdK + 32 * a + 8 * g);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            acc[u] = io::mma(io::row(sh.k + (32 * ks + 16 * u + l16) * Sh::kLdK + 32 * a + 8 * g), fq, acc[u]);
        }
        const int i = 16 * it + l16;
        const float chi = dec.hi[i], clo = dec.lo[i];
        const int lim = dec.lim[i];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j0 = 32 * ks + 16 * u + 4 * g;
          float val[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = j0 + r;
            const float d = (chi - dec.hi[j]) + (clo - dec.lo[j]);
            const bool seen = REV ? j >= i && j <= lim : j <= i && j >= lim;
            val[r] = seen ? acc[u][r] * (__builtin_amdgcn_exp2f(REV ? -d : d) * p.pscale) : 0.f;
          }
#pragma unroll
          for (int x = 0; x < NPP; ++x) {
            io::template store<4>(sh.p + (x * C + i) * Sh::kLdP + j0, val);
            if (x + 1 < NPP)
#pragma unroll
              for (int r = 0; r < 4; ++r) val[r] = lin_rest(val[r]);
          }
        }
      }
      __syncthreads();
    }

    if (!done) {
      frag fv[KS][NT];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          fv[ks][t] = lin_column<T>(sh.v, Sh::kLdV, 32 * ks + 8 * g, wcol + 4 * t, kSpread, l16);

      bool fine = true;
      if (!STATE) {
        // ---- out^T: columns of v down, tokens across
        f32x4 acc[IT][NT] = {};
#pragma unroll
        for (int a = 0; a < KK; ++a) {
          frag fs[NT][NP];
#pragma unroll
          for (int t = 0; t < NT; ++t)
            lin_split<T, NP>(__builtin_shufflevector(S[a][0][t], S[a][1][t], 0, 1, 2, 3, 4, 5, 6, 7), fs[t]);
#pragma unroll
          for (int it = 0; it < IT; ++it) {
            const frag fq = io::row(sh.q + (16 * it + l16) * Sh::kLdK + 32 * a + 8 * g);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < NP; ++x) acc[it][t] = io::mma(fs[t][x], fq, acc[it][t]);
          }
        }
        float chk = 0.f;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const float f = dec.f[16 * it + l16];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[it][t][r] = f == 0.f ? 0.f : acc[it][t][r] * f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (REV ? 32 * ks + 31 < 16 * it : 32 * ks > 16 * it + 15) continue;
#pragma unroll
            for (int x = 0; x < NPP; ++x) {
              const frag fp = io::row(sh.p + (x * C + 16 * it + l16) * Sh::kLdP + 32 * ks + 8 * g);
#pragma unroll
              for (int t = 0; t < NT; ++t) acc[it][t] = io::mma(fv[ks][t], fp, acc[it][t]);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) chk = fmaf(acc[it][t][r], 0.f, chk);
        }
        fine = job.single || __all(chk == 0.f);
        if (fine) {
          const int cbase = wcol + 4 * NT * g, room = p.vd - col0 - cbase;   // columns that are there
#pragma unroll
          for (int it = 0; it < IT; ++it) {
            const int i = 16 * it + l16;
            const bool in = i >= job.lo && i < job.hi;
            float val[4 * NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int r = 0; r < 4; ++r) val[4 * t + r] = acc[it][t][r];
            if (in) {
              const int64_t at = b * p.o_sb + (t0 + i) * p.o_sl + h * p.o_sh + col0 + cbase;
              if (p.out_f32)
                lin_io<float>::template put<4 * NT>(static_cast<float*>(p.out) + at, val, room);
              else
                io::template put<4 * NT>(static_cast<T*>(p.out) + at, val, room);
            }
            if (p.dot) {                          // out_i . x_i, for the decays' gradient
              float sum = 0.f;
              if (in) {
                const T* x = static_cast<const T*>(p.x.p) + b * p.x.sb + (t0 + i) * p.x.sl + (h / p.x.share) * p.x.sh + col0 + cbase;
                for (int e = 0; e < 4 * NT; ++e)
                  if (e < room) sum = fmaf(val[e], io::widen(x[e]), sum);
              }
              sum += __shfl_xor(sum, 16);
              sum += __shfl_xor(sum, 32);
              if (g == 0) sh.dot[wave][i] = sum;
            }
          }
        } else if (lane == 0) {
          sh.bad = 1;
        }
      }
      if (fine) {
        // ---- the new state: w_j v_j in parts, so that nothing of what is added to fp32 is lost
        const float keep = dec.carry;
        const bool fresh = dec.fresh != 0;
#pragma unroll
        for (int a = 0; a < KK; ++a)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int r = 0; r < 4; ++r) S[a][u][t][r] = fresh ? 0.f : S[a][u][t][r] * keep;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          frag fw[NT][NW];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            f32x8 x = io::wide(fv[ks][t]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float w = dec.w[32 * ks + 8 * g + e];
              x[e] = w == 0.f ? 0.f : w * x[e];
            }
            lin_split<T, NW>(x, fw[t]);
          }
#pragma unroll
          for (int a = 0; a < KK; ++a)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const frag fk = lin_column<T>(sh.k, Sh::kLdK, 32 * ks + 8 * g, 32 * a + 4 * u, 8, l16);
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < NW; ++x) S[a][u][t] = io::mma(fk, fw[t][x], S[a][u][t]);
            }
        }
        done = !job.single;
      }
    }
    if (wave == 3 && next.ci < chunks) decays(sh.dec[cur ^ 1]);
    __syncthreads();
    const bool bad = !STATE && !job.single && sh.bad != 0;
    if (!STATE && p.dot && !bad && tid >= job.lo && tid < job.hi)
      p.dot[((int64_t(nb) * p.batch + b) * p.L + t0 + tid) * p.H + h] = sh.dot[0][tid] + sh.dot[1][tid] + sh.dot[2][tid] + sh.dot[3][tid];
    ahead = true;
    if (bad) {
      next = first_token(job.ci);
      ahead = false;
    } else if (next.ci == chunks) {
      if (!STATE || retry) break;
      // the same for a segment's state: from its start again, token by token
      float chk = 0.f;
#pragma unroll
      for (int a = 0; a < KK; ++a)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) chk = fmaf(S[a][u][t][r], 0.f, chk);
      if (!__syncthreads_or(chk != 0.f)) break;
      retry = true;
      total = 0.0;
      zero_state();
      next = first_token(0);
      ahead = false;
    }
    if (!next.single || STATE) done = false;
    job = next;
  }

  if (STATE) {
#pragma unroll
    for (int a = 0; a < KK; ++a)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          *reinterpret_cast<f32x4*>(seg_at + (((a * 2 + u) * NT + t) * 256 + tid) * 4) = S[a][u][t];
    if (tid == 192 && nb == 0)
      p.seg_decay[bh * p.nseg + seg] = anew ? -1.f : lin_decay(float(total));
  } else if (p.s1 && seg == (REV ? 0 : p.nseg - 1)) {
    each_state([&](f32x4& s, int r, int64_t at) { p.s1[sbase + at] = s[r]; });
  }
}

template <typename T, int KD, int NT, bool REV, bool STATE, int NS>
hipError_t lin_launch(const LinParams& p, hipStream_t stream) {
  const int64_t items = p.batch * p.H * p.nblk * (STATE ? p.nseg - 1 : p.nseg);
  if (items == 0) return hipSuccess;
  lin_kernel<T, KD, NT, REV, STATE, NS><<<dim3(uint32_t(items)), dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T, int KD, int NT, int NS>
hipError_t lin_dispatch(bool rev, bool state, const LinParams& p, hipStream_t stream) {
  if (state) return rev ? lin_launch<T, KD, NT, true, true, 1>(p, stream) : lin_launch<T, KD, NT, false, true, 1>(p, stream);
  return rev ? lin_launch<T, KD, NT, true, false, NS>(p, stream) : lin_launch<T, KD, NT, false, false, NS>(p, stream);
}

}  // namespace
}  // namespace selscan
