// gated_kernels.hip -- the gated linear recurrence: forward, backward and decode step.
//
// A token is the map h -> a h + b with a = e^la, b = m sigmoid(g) x, and maps compose:
// (A', H') after (A, H) is (A' A, A' H + H').  So a run of tokens is worked on by one wavefront in
// registers, runs meet in LDS, and chunks of them in the workspace, without a second pass over
// the inputs.  Composition always takes the same order, so results do not depend on timing.
#include <type_traits>

#include "gated_device.h"

#include "scan_launch.h"
#include "selscan.h"

namespace selscan {
namespace {

constexpr int kTile = SELSCAN_GATED_TILE;

template <typename IO> __device__ __forceinline__ IO narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float v) { return bf16_rne(v); }

// ---- tiles of 128 channels: a lane owns a channel pair, a wavefront a run of S tokens

constexpr int kCh = 128;                   // channels of a workgroup
constexpr int kLinkGroup = 8;              // chunks between two chunks that publish their end state

// Two channels of one token, through a buffer descriptor on the chunk: the row's offset in a
// scalar register, the channels' in one (pairs) or two vector registers.  The descriptor ends
// with the chunk's last row and kNoChannel lies behind any: loads out of range give zero and
// stores are dropped, so neither the last tokens nor the last channels need a branch.
constexpr uint32_t kNoChannel = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const void* p, int rows, int row_bytes, int cols_bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (rows - 1) * row_bytes + cols_bytes, 0x00020000);
}
// How a lane's two channels are moved.  kPairs: in one access, on any element's boundary (the
// memory system takes those).  kOddPairs, where D is odd: the same, but the last channel is
// loaded as the second one of the pair that ends there (`last` moves it into place) and stored
// by itself, both behind a branch that only the last tile of channels takes; for every D that
// branch costs 6 % (4 x 16384 x 2560 in bf16).  kSingle: one by one, for D = 1, which has no pair.
// Forward and backward of 2 x 16384 x 2560 in bf16 take 172 and 385 us in pairs, 229 and 431
// where these straddle words, 552 and 961 one by one; D = 2559: 197 and 450.
enum { kSingle, kPairs, kOddPairs };
template <typename IO> struct pair_io;
template <> struct pair_io<float> {
  typedef uint32_t raw_t __attribute__((ext_vector_type(2)));
  template <int VEC> static __device__ __forceinline__ raw_t load(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row) {
    if constexpr (VEC != kSingle) return __builtin_bit_cast(raw_t, __builtin_amdgcn_raw_buffer_load_b64(r, o0, row, 0));
    else return raw_t{__builtin_amdgcn_raw_buffer_load_b32(r, o0, row, 0), __builtin_amdgcn_raw_buffer_load_b32(r, o1, row, 0)};
  }
  // the compiler no longer knows what v holds, so nothing formed from it before is kept for after
  static __device__ __forceinline__ void forget(raw_t& v) { asm("" : "+v"(v)); }
  static __device__ __forceinline__ void last(raw_t& v, bool lane) { v.x = lane ? v.y : v.x; }
  static __device__ __forceinline__ float lo(raw_t v) { return __uint_as_float(v.x); }
  static __device__ __forceinline__ float hi(raw_t v) { return __uint_as_float(v.y); }
  template <int VEC>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row, float a, float b, bool odd) {
    const raw_t v = {__float_as_uint(a), __float_as_uint(b)};
    if constexpr (VEC != kSingle) {
      __builtin_amdgcn_raw_buffer_store_b64(v, r, o0, row, 0);
      if (VEC == kOddPairs && odd) __builtin_amdgcn_raw_buffer_store_b32(v.x, r, o1, row, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b32(v.x, r, o0, row, 0);
      __builtin_amdgcn_raw_buffer_store_b32(v.y, r, o1, row, 0);
    }
  }
};
template <> struct pair_io<uint16_t> {
  using raw_t = uint32_t;
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  template <int VEC> static __device__ __forceinline__ raw_t load(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row) {
    if constexpr (VEC != kSingle) return __builtin_amdgcn_raw_buffer_load_b32(r, o0, row, 0);
    else return uint32_t(__builtin_amdgcn_raw_buffer_load_b16(r, o0, row, 0)) |
                (uint32_t(__builtin_amdgcn_raw_buffer_load_b16(r, o1, row, 0)) << 16);
  }
  static __device__ __forceinline__ void forget(raw_t& v) { asm("" : "+v"(v)); }
  static __device__ __forceinline__ void last(raw_t& v, bool lane) { v = lane ? v >> 16 : v; }
  static __device__ __forceinline__ float lo(raw_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(raw_t v) { return __uint_as_float(v & 0xffff0000u); }
  template <int VEC>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row, float a, float b, bool odd) {
    const f32x2_t f = {a, b};                              // to nearest even
    const uint32_t v = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
    if constexpr (VEC != kSingle) {
      __builtin_amdgcn_raw_buffer_store_b32(v, r, o0, row, 0);
      if (VEC == kOddPairs && odd) __builtin_amdgcn_raw_buffer_store_b16(uint16_t(v), r, o1, row, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b16(uint16_t(v), r, o0, row, 0);
      __builtin_amdgcn_raw_buffer_store_b16(uint16_t(v >> 16), r, o1, row, 0);
    }
  }
};

// The offsets of a lane's channels c, c + 1 in a row of D, for loads and for stores.
template <int VEC> struct Columns {
  uint32_t l0, l1, s0, s1;
  bool odd, lane;                          // (kOddPairs) the last tile of channels, the last channel's lane
  __device__ __forceinline__ Columns(int c, int D, int es, bool last_tile) {
    odd = VEC == kOddPairs && last_tile;
    lane = c + 1 == D;
    l0 = s0 = c < D ? c * es : kNoChannel;
    l1 = s1 = c + 1 < D ? (c + 1) * es : kNoChannel;
    if constexpr (VEC == kOddPairs) {
      l0 = c + 1 < D ? c * es : c < D ? (c - 1) * es : kNoChannel;
      s0 = c + 1 < D ? c * es : kNoChannel;
      s1 = lane ? c * es : kNoChannel;
    }
  }
};

// The links between the chunks of one chain (a batch row's 128 channels), in the workspace: zero
// until written, each word whole or absent, so a reader needs no other order between writes.
//   map [items][2][64]: the chunk's map h -> A h + H as {A with its sign bit set, H} (A >= 0),
//     the even channels before the odd ones;
//   end [groups][2][64]: the state behind the chunk as {1, h}, by the last chunk of a group.
__device__ __forceinline__ void put_word(uint64_t* p, uint32_t tag, float v) {
  __hip_atomic_store(p, (uint64_t(tag) << 32) | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_word(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The wait ends (see the kernels' tickets).  It is bounded all the same (some seconds); a word
// that never comes reads as NaN.
constexpr int kMaxPolls = 1 << 21;
__device__ __forceinline__ uint64_t wait_word(const uint64_t* p, uint64_t first) {
  uint64_t w = first;
  for (int n = 0; w == 0 && n < kMaxPolls; ++n) {
    __builtin_amdgcn_s_sleep(1);
    w = get_word(p);
  }
  return w != 0 ? w : (uint64_t(0xffc00000u) << 32) | 0x7fc00000u;
}

// h behind a map (A, H); with CUT a map that takes nothing from h takes not even an infinity.
template <bool CUT> __device__ __forceinline__ float through(float A, float H, float h) {
  const float v = fmaf(A, h, H);
  return CUT && A == 0.f ? H : v;
}

// The product of decays.  One that leaves fp32 is held at its least number, so an infinity does not
// end there (in 0 * inf); with CUT it is zero behind a reset alone.  (Of the largest state that
// leaves 2^-21, what a product rounded to fp32 may be off by; the least normal number would
// leave 4.)
constexpr float kLeastDecay = 0x1p-149f;
template <bool CUT> __device__ __forceinline__ float decays(float A, float a) {
  if (CUT && (A == 0.f || a == 0.f)) return 0.f;
  return fmaxf(A * a, kLeastDecay);
}

// The links of one chunk, the pos-th of its chain (counted from the end in the backward pass).
struct Link {
  uint64_t* map;                           // of this chunk and lane
  uint64_t* end;                           // of this chunk's group
  int64_t next;                            // words between a chain's chunks
  int pos, in_group;
  bool last;
  __device__ __forceinline__ Link(const GatedParams& p, uint32_t order, uint32_t chain, uint32_t chains, int lane) {
    next = int64_t(chains) * kCh;
    uint64_t* const base = p.links + kTicketWords + int64_t(chain) * kCh + lane;
    map = base + order * next;
    end = base + (int64_t(p.n_chunks) + order / kLinkGroup) * next;
    pos = int(order);
    in_group = pos % kLinkGroup;
    last = pos == p.n_chunks - 1;
  }
  __device__ __forceinline__ void publish(float A0, float A1, float H0, float H1) const {
    if (last) return;
    put_word(map, __float_as_uint(A0) | 0x80000000u, H0);
    put_word(map + 64, __float_as_uint(A1) | 0x80000000u, H1);
  }
  __device__ __forceinline__ void publish_end(float h0, float h1) const {
    if (last || in_group != kLinkGroup - 1) return;
    put_word(end, 1u, h0);
    put_word(end + 64, 1u, h1);
  }
  // Wavefront 0 reads the state behind the group before (none: zero, the first chunk's map
  // takes nothing from it), wavefront j the map of the group's chunk j - 1.
  __device__ __forceinline__ void read(int wave, float4* to) const {
    if (pos == 0 || wave > in_group) return;
    if (wave == 0 && pos < kLinkGroup) {
      *to = make_float4(0.f, 0.f, 0.f, 0.f);
      return;
    }
    const uint64_t* const q = wave == 0 ? end - next : map - (in_group - wave + 1) * next;
    const uint64_t f0 = get_word(q), f1 = get_word(q + 64);
    const uint64_t w0 = wait_word(q, f0), w1 = wait_word(q + 64, f1);
    *to = make_float4(fabsf(__uint_as_float(uint32_t(w0 >> 32))), fabsf(__uint_as_float(uint32_t(w1 >> 32))),
                      __uint_as_float(uint32_t(w0)), __uint_as_float(uint32_t(w1)));
  }
};

// What a ticket stands for: one chunk of one chain.  Tickets run over all chains' first chunks,
// then their second ones, and so on.
struct Chunk {
  uint32_t chunk, chain, b, ct;
  int64_t t0;
  int rest;                                // tokens
};
// c softplus(lam) of a channel, zero behind the last
__device__ __forceinline__ float gated_rate(const GatedParams& p, int c) {
  if (c >= int(p.D)) return 0.f;
  return p.kd != nullptr ? p.kd[c] : p.c * softplus_f32(p.lam[c]);
}

template <int LEN>
__device__ __forceinline__ Chunk chunk_of(const GatedParams& p, uint32_t ticket, uint32_t chains, uint32_t ctiles) {
  // (the quotients come from the vector unit: back into scalar registers, or every address
  // after them stays out of them)
  Chunk k;
  k.chunk = __builtin_amdgcn_readfirstlane(ticket / chains);
  k.chain = ticket - k.chunk * chains;
  k.b = __builtin_amdgcn_readfirstlane(k.chain / ctiles);
  k.ct = k.chain - k.b * ctiles;
  k.t0 = int64_t(k.chunk) * LEN;
  k.rest = int(p.L - k.t0 < LEN ? p.L - k.t0 : LEN);
  return k;
}

// The map of a run of S tokens, and the states before each of them.
template <int S, bool CUT>
__device__ __forceinline__ void run_map(const float (&a)[S], const float (&b)[S], uint32_t cuts, float& A, float& H) {
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (CUT && (cuts >> i & 1)) A = H = 0.f;
    H = fmaf(a[i], H, b[i]);
    A *= a[i];
  }
}
template <int S, bool CUT>
__device__ __forceinline__ void run_states(const float (&a)[S], float (&b)[S], uint32_t cuts, float& h) {
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const float before = h;
    if (CUT && (cuts >> i & 1)) h = 0.f;
    h = fmaf(a[i], h, b[i]);
    b[i] = before;
  }
}

// Chunks of NW S tokens and 128 channels.  Each wavefront forms the map of its S tokens in
// registers; the maps meet in LDS, the workgroup's in the links, where the maps of the chunks
// since the last published state and that state are read, one by each wavefront; every
// wavefront then walks its tokens from the state that enters them, composed in a fixed order.
// The inputs are read once.  A workgroup takes chunk after chunk by ticket, the next one's
// inputs in flight while it waits for the links of this one.  A chunk's predecessors have
// lower tickets, so whoever holds them works on them or on still lower ones: every wait ends.
//
// Four tensors pass through HBM once: 4 x 16384 tokens x 2560 channels in bf16 are 1342 MB and take
// 270 us, 5.0 TB/s where a large copy reaches 5.9.  Without the links (and so with wrong
// states) it is 250, without the arithmetic 246: bytes, arithmetic (55 % of the vector
// instructions' slots) and the exchange hide one another but for some 10 % each.  One, two and
// four sequences take 102, 171 and 277 a call: up to 65 us of it do not shrink with the bytes
// (start, drain, the clearing launch, links between chunks in work at once; not told apart).
// 128 tokens of bf16 a chunk, 64 of fp32, are what two chunks' raw inputs leave room for.
// Measured against a state of this kernel that took 281 (25 at 3 x 1537 x 771 in fp32): chunks
// of 64 tokens in bf16, twice the links, slower; two chunks ahead, which spills, 314;
// workgroups of 64 channels and four wavefronts, three a compute unit, 294 (32); one wavefront
// that reads all links for the others, 347.
template <typename IO, int NW, int S, int VEC, bool RESET>
__global__ __launch_bounds__(NW * 64) void gated_fwd_kernel(GatedParams p) {
  using T = pair_io<IO>;
  constexpr int kLen = NW * S;
  static_assert(kLinkGroup <= NW, "a wavefront reads one link");
  __shared__ float4 maps[2][NW][kCh / 2];          // of the wavefronts' tokens
  __shared__ float4 links[2][kLinkGroup][kCh / 2];    // of the chunks before; [0] the state behind their group
  __shared__ uint32_t tickets[3];                  // by turns; [2] the first
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t ctiles = uint32_t((p.D + kCh - 1) / kCh), chains = uint32_t(p.batch) * ctiles;
  const uint32_t total = chains * uint32_t(p.n_chunks);
  constexpr int es = int(sizeof(IO));
  const int xs = int(p.x_sl) * es, rs = int(p.r_sl) * es, gs = int(p.g_sl) * es, ys = int(p.y_sl) * es;   // bytes
  const int D = int(p.D), s0 = wave * S;           // this wavefront's first token in a chunk
  uint32_t* const counter = reinterpret_cast<uint32_t*>(p.links);
  uint32_t now = blockIdx.x, next = total;         // the first chunk's ticket and the following one's
  if (p.links != nullptr) {
    if (tid == 0) tickets[2] = atomicAdd(counter, 1u);
    __syncthreads();
    now = __builtin_amdgcn_readfirstlane(tickets[2]);
    if (now >= total) return;
  }

  struct Raw {
    typename T::raw_t x[S], r[S], g[S];
    uint32_t first;                                // lane i: token i starts a sequence
    float k0, k1;
  };
  // the gates of a chunk, and its x
  auto load_gates = [&](const Chunk& k, Raw& w) __attribute__((always_inline)) {
    const auto rp = chunk_rsrc(static_cast<const IO*>(p.r) + k.b * p.r_sb + k.t0 * p.r_sl, k.rest, rs, D * es);
    const auto gp = chunk_rsrc(static_cast<const IO*>(p.g) + k.b * p.g_sb + k.t0 * p.g_sl, k.rest, gs, D * es);
    const int c = int(k.ct) * kCh + 2 * lane;
    w.first = 0;
    if constexpr (RESET) {
      const int t = s0 + lane;
      if (lane < S && t < k.rest) w.first = p.reset[k.b * p.reset_sb + k.t0 + t];
    }
    w.k0 = gated_rate(p, c);
    w.k1 = gated_rate(p, c + 1);
    const Columns<VEC> col(c, D, es, k.ct == ctiles - 1);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      w.r[i] = T::template load<VEC>(rp, col.l0, col.l1, (s0 + i) * rs);
      w.g[i] = T::template load<VEC>(gp, col.l0, col.l1, (s0 + i) * gs);
    }
  };
  auto load_x = [&](const Chunk& k, Raw& w) __attribute__((always_inline)) {
    const auto xp = chunk_rsrc(static_cast<const IO*>(p.x) + k.b * p.x_sb + k.t0 * p.x_sl, k.rest, xs, D * es);
    const int c = int(k.ct) * kCh + 2 * lane;
    const Columns<VEC> col(c, D, es, k.ct == ctiles - 1);
#pragma unroll
    for (int i = 0; i < S; ++i) w.x[i] = T::template load<VEC>(xp, col.l0, col.l1, (s0 + i) * xs);
  };

  Chunk k = chunk_of<kLen>(p, now, chains, ctiles);
  // Chunk k from `w`, the following one's inputs on their way into `wn`; false after the last.
  auto step = [&](Raw& w, Raw& wn, const int par) __attribute__((always_inline)) -> bool {
    const bool more = next < total;
    const Chunk kn = chunk_of<kLen>(p, more ? next : 0, chains, ctiles);
    if (more) load_gates(kn, wn);
    uint32_t after = total;
    if (more && tid == 0) after = atomicAdd(counter, 1u);
    const Columns<VEC> col(int(k.ct) * kCh + 2 * lane, D, es, k.ct == ctiles - 1);
    if (VEC == kOddPairs && col.odd) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        T::last(w.x[i], col.lane);
        T::last(w.r[i], col.lane);
        T::last(w.g[i], col.lane);
      }
    }
    float a0[S], a1[S], b0[S], b1[S];
    uint32_t cuts = 0;                             // bit i: token i starts a sequence
    if constexpr (RESET) cuts = uint32_t(__ballot(w.first != 0));
    // |log a| is at most k: where that is small for the whole wavefront, no exp2 is needed (2 x
    // 16384 x 2560 in bf16: 173 us so, 186 with both forms formed and one chosen).  (The
    // branch is taken four tokens at a time: around all of them, the compiler keeps every
    // gate's sigmoid in registers across it.)
    const bool small = __all(w.k0 < kGatedSmall && w.k1 < kGatedSmall);
#pragma unroll
    for (int i0 = 0; i0 < S; i0 += 4) {
      float m0[4], m1[4];
      if (small) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gated_decay_small(-w.k0 * sigmoid_f32(T::lo(w.r[i0 + i])), a0[i0 + i], m0[i]);
          gated_decay_small(-w.k1 * sigmoid_f32(T::hi(w.r[i0 + i])), a1[i0 + i], m1[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gated_decay(-w.k0 * sigmoid_f32(T::lo(w.r[i0 + i])), a0[i0 + i], m0[i]);
          gated_decay(-w.k1 * sigmoid_f32(T::hi(w.r[i0 + i])), a1[i0 + i], m1[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (RESET && (cuts >> i0 & 15) != 0 && (cuts >> (i0 + i) & 1)) {
          a0[i0 + i] = a1[i0 + i] = 0.f;
          m0[i] = m1[i] = 1.f;
        }
        b0[i0 + i] = m0[i] * (sigmoid_f32(T::lo(w.g[i0 + i])) * T::lo(w.x[i0 + i]));
        b1[i0 + i] = m1[i] * (sigmoid_f32(T::hi(w.g[i0 + i])) * T::hi(w.x[i0 + i]));
      }
    }
    if (k.rest < kLen) {                           // behind the last token: the map that changes nothing
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (s0 + i >= k.rest) { a0[i] = a1[i] = 1.f; b0[i] = b1[i] = 0.f; }
    }
    float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f;
    if (RESET && cuts != 0) {                      // (rare)
      run_map<S, true>(a0, b0, cuts, A0, H0);
      run_map<S, true>(a1, b1, cuts, A1, H1);
    } else {
      run_map<S, false>(a0, b0, 0, A0, H0);
      run_map<S, false>(a1, b1, 0, A1, H1);
      A0 = fmaxf(A0, kLeastDecay);
      A1 = fmaxf(A1, kLeastDecay);
    }
    const int c = int(k.ct) * kCh + 2 * lane;
    const bool ok0 = c < D, ok1 = c + 1 < D, last = int(k.chunk) == p.n_chunks - 1;
    if (wave == 0 && k.chunk == 0) {
      // the initial state enters through the first map, and nobody else reads it: it may lie
      // where the last chunk writes the last state
      float h0 = 0.f, h1 = 0.f;
      if (p.h0 != nullptr) {
        if (ok0) h0 = p.h0[int64_t(k.b) * D + c];
        if (ok1) h1 = p.h0[int64_t(k.b) * D + c + 1];
      }
      links[par][0][lane] = make_float4(0.f, 0.f, h0, h1);
      H0 = through<RESET>(A0, H0, h0);
      H1 = through<RESET>(A1, H1, h1);
      A0 = A1 = 0.f;
    }
    maps[par][wave][lane] = make_float4(A0, A1, H0, H1);
    if (tid == 0) tickets[par] = after;
    __syncthreads();
    const Link link(p, k.chunk, k.chain, chains, lane);
    if (wave == NW - 1 && p.links != nullptr) {    // the chunk's map, before any wait
      float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const float4 m = maps[par][j][lane];
        H0 = through<RESET>(m.x, m.z, H0);
        H1 = through<RESET>(m.y, m.w, H1);
        A0 = decays<RESET>(A0, m.x);
        A1 = decays<RESET>(A1, m.y);
      }
      link.publish(A0, A1, H0, H1);
    }
    link.read(wave, &links[par][wave][lane]);
    if (more) load_x(kn, wn);
    __syncthreads();
    after = __builtin_amdgcn_readfirstlane(tickets[par]);
    float h0 = links[par][0][lane].z, h1 = links[par][0][lane].w;
    // (the first map holds the initial state: an infinite one, taken again times its A = 0, would be NaN)
    if (k.chunk == 0 && wave != 0) h0 = h1 = 0.f;
    for (int j = 1; j <= link.in_group; ++j) {
      const float4 m = links[par][j][lane];
      h0 = through<RESET>(m.x, m.z, h0);
      h1 = through<RESET>(m.y, m.w, h1);
    }
    for (int j = 0; j < wave; ++j) {
      const float4 m = maps[par][j][lane];
      h0 = through<RESET>(m.x, m.z, h0);
      h1 = through<RESET>(m.y, m.w, h1);
    }
    if (p.ckpt != nullptr && (k.t0 + s0) % kTile == 0 && s0 < k.rest) {
      float* const o = p.ckpt + (k.b * p.ntiles + (k.t0 + s0) / kTile) * p.D + c;
      if (ok0) o[0] = h0;
      if (ok1) o[1] = h1;
    }
    const auto yp = chunk_rsrc(static_cast<IO*>(p.y) + k.b * p.y_sb + k.t0 * p.y_sl, k.rest, ys, D * es);
    if (RESET && cuts != 0) {
      run_states<S, true>(a0, b0, cuts, h0);
      run_states<S, true>(a1, b1, cuts, h1);
    } else {
      run_states<S, false>(a0, b0, 0, h0);
      run_states<S, false>(a1, b1, 0, h1);
    }
    if (p.y != nullptr) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const bool end = i == S - 1;               // b holds the state before each token
        T::template store<VEC>(yp, col.s0, col.s1, (s0 + i) * ys, end ? h0 : b0[i + 1 < S ? i + 1 : i],
                               end ? h1 : b1[i + 1 < S ? i + 1 : i], col.odd);
      }
    }
    if (wave == NW - 1) {                          // the state behind the chunk
      if (p.links != nullptr) link.publish_end(h0, h1);
      if (last && p.last != nullptr) {
        float* const o = p.last + int64_t(k.b) * D + c;
        if (ok0) o[0] = h0;
        if (ok1) o[1] = h1;
      }
    }
    if (!more) return false;
    k = kn;
    next = after;
    return true;
  };

  Raw w0, w1;
  load_gates(k, w0);
  load_x(k, w0);
  if (p.persistent) {
    if (tid == 0) tickets[1] = atomicAdd(counter, 1u);
    __syncthreads();
    next = __builtin_amdgcn_readfirstlane(tickets[1]);
  }
  while (step(w0, w1, 0) && step(w1, w0, 1)) {
  }
}

// What the chunks of one call share: the links, empty, and the channels' c softplus(lam).  A
// kernel, not a memset: calls may be captured.  (11 MB of links take 6 us.)
__global__ __launch_bounds__(256) void gated_begin_kernel(ulonglong2* links, int64_t pairs, const float* lam, float c, float* kd,
                                                          int64_t D) {
  const int64_t i0 = blockIdx.x * int64_t(256) + threadIdx.x, n = int64_t(gridDim.x) * 256;
  for (int64_t i = i0; i < pairs; i += n) links[i] = make_ulonglong2(0, 0);
  for (int64_t i = i0; i < D; i += n) kd[i] = c * softplus_f32(lam[i]);
}

// The backward pass over chunks of NW S tokens and 128 channels, from the last one on.  With
// G_t = a_t l_t, what token t hands to the adjoint l_{t-1} = dy_{t-1} + G_t, the map of a token
// is G -> a (G + dy): the same kind as the forward pass's, joined in the same way along the
// reversed sequence.  The states are formed again from the chunk's checkpoint.  The gates'
// sigmoids are computed twice, before the exchange of maps (the decays stay in registers)
// and after it: keeping them takes 32 registers, which fp32 (236 of 256 at its two wavefronts a
// SIMD) has not and bf16 (204) has; that is not built.
//
// Seven tensors pass through HBM once: 4 x 4096 x 2560 in bf16 are 587 MB and take 184 us,
// 3.2 TB/s.  The loads alone take 113 and the arithmetic fills 55 % of its slots, 84 vector
// instructions an element of which ten are transcendental, four of those the sigmoids formed
// again.  The three phases of a chunk (map, wait, gradients) follow one another with one
// workgroup on a compute unit, since the raw inputs of two chunks fill its registers; but
// workgroups of half as many channels, three a compute unit, took 183 (in fp32 42 against 38),
// so the phases alone are not what it waits for.
template <typename IO, int NW, int S, int VEC, bool RESET>
__global__ __launch_bounds__(NW * 64) void gated_bwd_kernel(GatedParams p) {
  using T = pair_io<IO>;
  constexpr int kLen = NW * S, es = int(sizeof(IO));
  static_assert(kLinkGroup <= NW && kLen % kTile == 0, "a wavefront reads one link; a chunk starts at a checkpoint");
  __shared__ float4 maps[2][NW][kCh / 2];          // of the wavefronts' tokens, forward
  __shared__ float2 backs[2][NW][kCh / 2];         // and backward (with the same A)
  __shared__ float4 links[2][kLinkGroup][kCh / 2]; // of the chunks behind; [0] what their group receives
  __shared__ float2 sums[2][NW][kCh / 2];
  __shared__ uint32_t tickets[3];                  // by turns; [2] the first
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t ctiles = uint32_t((p.D + kCh - 1) / kCh), chains = uint32_t(p.batch) * ctiles;
  const uint32_t total = chains * uint32_t(p.n_chunks);
  const int D = int(p.D);
  uint32_t* const counter = reinterpret_cast<uint32_t*>(p.links);
  uint32_t now = blockIdx.x, next = total;         // the first chunk's ticket and the following one's
  if (p.links != nullptr) {
    if (tid == 0) tickets[2] = atomicAdd(counter, 1u);
    __syncthreads();
    now = __builtin_amdgcn_readfirstlane(tickets[2]);
    if (now >= total) return;
  }
  struct Raw {
    typename T::raw_t x[S], r[S], g[S], y[S];
    uint32_t first;                                // lane i: token i starts a sequence
    float k0, k1, h0, h1;                          // the channels' rates, the state entering the chunk
  };
  // the chunk of a ticket: the order-th from the end
  auto chunk_back = [&](uint32_t ticket, uint32_t& order) __attribute__((always_inline)) {
    Chunk k = chunk_of<kLen>(p, ticket, chains, ctiles);
    order = k.chunk;
    k.chunk = uint32_t(p.n_chunks) - 1 - order;
    k.t0 = int64_t(k.chunk) * kLen;
    k.rest = int(p.L - k.t0 < kLen ? p.L - k.t0 : kLen);
    return k;
  };
  // The gates of a chunk, and the rest of its inputs.  (The rows' offsets are formed anew for every
  // chunk: kept over all of them, they fill the scalar registers and spill into vector ones.)
  auto load_gates = [&](const Chunk& k, Raw& w) __attribute__((always_inline)) {
    int s0 = wave * S;
    asm("" : "+s"(s0));
    const int rs = int(p.r_sl) * es, gs = int(p.g_sl) * es;
    const int c = int(k.ct) * kCh + 2 * lane;
    const Columns<VEC> col(c, D, es, k.ct == ctiles - 1);
    w.first = 0;
    if constexpr (RESET) {
      const int t = s0 + lane;
      if (lane < S && t < k.rest) w.first = p.reset[k.b * p.reset_sb + k.t0 + t];
    }
    w.k0 = gated_rate(p, c);
    w.k1 = gated_rate(p, c + 1);
    w.h0 = w.h1 = 0.f;
    const float* const q = p.ckpt + (k.b * p.ntiles + k.t0 / kTile) * p.D + c;
    if (c < D) w.h0 = q[0];
    if (c + 1 < D) w.h1 = q[1];
    const auto rp = chunk_rsrc(static_cast<const IO*>(p.r) + k.b * p.r_sb + k.t0 * p.r_sl, k.rest, rs, D * es);
    const auto gp = chunk_rsrc(static_cast<const IO*>(p.g) + k.b * p.g_sb + k.t0 * p.g_sl, k.rest, gs, D * es);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      w.r[i] = T::template load<VEC>(rp, col.l0, col.l1, (s0 + i) * rs);
      w.g[i] = T::template load<VEC>(gp, col.l0, col.l1, (s0 + i) * gs);
    }
  };
  auto load_rest = [&](const Chunk& k, Raw& w) __attribute__((always_inline)) {
    int s0 = wave * S;
    asm("" : "+s"(s0));
    const int xs = int(p.x_sl) * es, ys = int(p.y_sl) * es;
    const Columns<VEC> col(int(k.ct) * kCh + 2 * lane, D, es, k.ct == ctiles - 1);
    const auto xp = chunk_rsrc(static_cast<const IO*>(p.x) + k.b * p.x_sb + k.t0 * p.x_sl, k.rest, xs, D * es);
    const auto yp = chunk_rsrc(static_cast<const IO*>(p.dy) + k.b * p.y_sb + k.t0 * p.y_sl, k.rest, ys, D * es);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      w.x[i] = T::template load<VEC>(xp, col.l0, col.l1, (s0 + i) * xs);
      w.y[i] = T::template load<VEC>(yp, col.l0, col.l1, (s0 + i) * ys);
    }
  };

  uint32_t order;
  Chunk k = chunk_back(now, order);
  // Chunk k from `w`, the following one's inputs on their way into `wn`; false after the last.
  auto step = [&](Raw& w, Raw& wn, const int par) __attribute__((always_inline)) -> bool {
    const bool more = next < total;
    uint32_t order_n;
    const Chunk kn = chunk_back(more ? next : 0, order_n);
    if (more) load_gates(kn, wn);
    uint32_t after = total;
    if (more && tid == 0) after = atomicAdd(counter, 1u);
    const Link link(p, order, k.chain, chains, lane);
    const int c = int(k.ct) * kCh + 2 * lane, s0 = wave * S;
    const bool ok0 = c < D, ok1 = c + 1 < D;
    const Columns<VEC> col(c, D, es, k.ct == ctiles - 1);
    auto& xr = w.x;
    auto& rr = w.r;
    auto& gr = w.g;
    auto& yr = w.y;
    if (VEC == kOddPairs && col.odd) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        T::last(xr[i], col.lane);
        T::last(rr[i], col.lane);
        T::last(gr[i], col.lane);
        T::last(yr[i], col.lane);
      }
    }
    const float k0 = w.k0, k1 = w.k1;
    float h0 = w.h0, h1 = w.h1;
    uint32_t cuts = 0;                             // bit i: token i starts a sequence
    if constexpr (RESET) cuts = uint32_t(__ballot(w.first != 0));
    float a0[S], a1[S], m0[S], m1[S], b0[S], b1[S];
    float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f;
    const bool small = __all(k0 < kGatedSmall && k1 < kGatedSmall);
#pragma unroll
    for (int i0 = 0; i0 < S; i0 += 4) {
      if (small) {
#pragma unroll
        for (int i = i0; i < i0 + 4; ++i) {
          gated_decay_small(-k0 * sigmoid_f32(T::lo(rr[i])), a0[i], m0[i]);
          gated_decay_small(-k1 * sigmoid_f32(T::hi(rr[i])), a1[i], m1[i]);
        }
      } else {
#pragma unroll
        for (int i = i0; i < i0 + 4; ++i) {
          gated_decay(-k0 * sigmoid_f32(T::lo(rr[i])), a0[i], m0[i]);
          gated_decay(-k1 * sigmoid_f32(T::hi(rr[i])), a1[i], m1[i]);
        }
      }
      // (rare: a token that starts a sequence or lies behind the last)
      if ((RESET && (cuts >> i0 & 15) != 0) || s0 + i0 + 4 > k.rest) {
#pragma unroll
        for (int i = i0; i < i0 + 4; ++i) {
          if (RESET && (cuts >> i & 1)) {
            a0[i] = a1[i] = 0.f;
            m0[i] = m1[i] = 1.f;
          }
          if (s0 + i >= k.rest) {                  // the map that changes nothing
            a0[i] = a1[i] = 1.f;
            m0[i] = m1[i] = 0.f;
            xr[i] = yr[i] = typename T::raw_t{};   // (where rows overlap, theirs lie in range)
          }
        }
      }
#pragma unroll
      for (int i = i0; i < i0 + 4; ++i) {
        b0[i] = m0[i] * (sigmoid_f32(T::lo(gr[i])) * T::lo(xr[i]));
        b1[i] = m1[i] * (sigmoid_f32(T::hi(gr[i])) * T::hi(xr[i]));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    float G0 = 0.f, G1 = 0.f;
    if (RESET && cuts != 0) {                      // (rare)
      run_map<S, true>(a0, b0, cuts, A0, H0);
      run_map<S, true>(a1, b1, cuts, A1, H1);
#pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        const bool cut = cuts >> i & 1;
        G0 = cut ? 0.f : a0[i] * (G0 + T::lo(yr[i]));
        G1 = cut ? 0.f : a1[i] * (G1 + T::hi(yr[i]));
      }
    } else {
      run_map<S, false>(a0, b0, 0, A0, H0);
      run_map<S, false>(a1, b1, 0, A1, H1);
      A0 = fmaxf(A0, kLeastDecay);
      A1 = fmaxf(A1, kLeastDecay);
#pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        G0 = a0[i] * (G0 + T::lo(yr[i]));
        G1 = a1[i] * (G1 + T::hi(yr[i]));
      }
    }
    maps[par][wave][lane] = make_float4(A0, A1, H0, H1);
    backs[par][wave][lane] = make_float2(G0, G1);
    if (tid == 0) tickets[par] = after;
    __syncthreads();
    after = __builtin_amdgcn_readfirstlane(tickets[par]);
    if (wave == 0) {
      float P0 = 1.f, P1 = 1.f, R0 = 0.f, R1 = 0.f;
      if (link.pos == 0) {
        // The last chunk knows what it receives; nobody else reads dlast, and it is read before
        // anything is published: it may lie where the first chunk writes dh0.
        if (p.dlast != nullptr) {
          if (ok0) R0 = p.dlast[int64_t(k.b) * D + c];
          if (ok1) R1 = p.dlast[int64_t(k.b) * D + c + 1];
        }
        links[par][0][lane] = make_float4(0.f, 0.f, R0, R1);
      }
      if (p.links != nullptr) {                    // the chunk's map, before any wait
#pragma unroll 2
        for (int j = NW - 1; j >= 0; --j) {
          const float4 m = maps[par][j][lane];
          const float2 g = backs[par][j][lane];
          R0 = through<RESET>(m.x, g.x, R0);
          R1 = through<RESET>(m.y, g.y, R1);
          P0 = decays<RESET>(P0, m.x);
          P1 = decays<RESET>(P1, m.y);
        }
        if (link.pos == 0) P0 = P1 = 0.f;
        link.publish(P0, P1, R0, R1);
      }
    }
    if (link.pos != 0) link.read(wave, &links[par][wave][lane]);
    if (more) load_rest(kn, wn);
    // the states before this wavefront's tokens, while the links arrive
#pragma unroll 2
    for (int j = 0; j < wave; ++j) {
      const float4 m = maps[par][j][lane];
      h0 = through<RESET>(m.x, m.z, h0);
      h1 = through<RESET>(m.y, m.w, h1);
    }
    // b becomes the state before its token
    if (RESET && cuts != 0) {
      run_states<S, true>(a0, b0, cuts, h0);
      run_states<S, true>(a1, b1, cuts, h1);
    } else {
      run_states<S, false>(a0, b0, 0, h0);
      run_states<S, false>(a1, b1, 0, h1);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {                  // the gates anew, not their sigmoids from before the exchange
      T::forget(rr[i]);
      T::forget(gr[i]);
    }
    __syncthreads();
    G0 = links[par][0][lane].z;
    G1 = links[par][0][lane].w;
#pragma unroll 2
    for (int j = 1; j <= link.in_group; ++j) {
      const float4 m = links[par][j][lane];
      G0 = through<RESET>(m.x, m.z, G0);
      G1 = through<RESET>(m.y, m.w, G1);
    }
#pragma unroll 2
    for (int j = NW - 1; j > wave; --j) {
      const float4 m = maps[par][j][lane];
      const float2 g = backs[par][j][lane];
      G0 = through<RESET>(m.x, g.x, G0);
      G1 = through<RESET>(m.y, g.y, G1);
    }
    float e0 = 0.f, e1 = 0.f;
    {
      const int64_t o = (int64_t(k.b) * p.L + k.t0) * p.D;
      const int os = D * es;
      const auto dxp = chunk_rsrc(static_cast<IO*>(p.dx) + o, k.rest, os, os);
      const auto drp = chunk_rsrc(static_cast<IO*>(p.dr) + o, k.rest, os, os);
      const auto dgp = chunk_rsrc(static_cast<IO*>(p.dg) + o, k.rest, os, os);
      // one token and channel: its adjoint l, the gradients of x, r and g, and G to hand on
      auto token = [&](float r, float g, float x, float dy, float k, float a, float m, float h, bool cut, float& G, float& sum,
                       float& dx, float& dr, float& dg) __attribute__((always_inline)) {
        float s, s1, sg, sg1;
        sigmoid_pair(r, s, s1);
        sigmoid_pair(g, sg, sg1);
        const float l = G + dy, v = sg * x, la = -k * s, dv = l * m;
        const float w = m > 0.f ? la * __builtin_amdgcn_rcpf(m) : 0.f;
        G = a * l;
        float e = G * fmaf(-a * w, v, la * h);
        if (RESET && cut) G = e = 0.f;             // (a scalar branch)
        dx = dv * sg;
        dg = dv * v * sg1;
        dr = e * s1;
        sum += e;
      };
#pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        const bool cut = RESET && (cuts >> i & 1);
        float dx0, dx1, dr0, dr1, dg0, dg1;
        token(T::lo(rr[i]), T::lo(gr[i]), T::lo(xr[i]), T::lo(yr[i]), k0, a0[i], m0[i], b0[i], cut, G0, e0, dx0, dr0, dg0);
        token(T::hi(rr[i]), T::hi(gr[i]), T::hi(xr[i]), T::hi(yr[i]), k1, a1[i], m1[i], b1[i], cut, G1, e1, dx1, dr1, dg1);
        if (s0 + i >= k.rest) e0 = e1 = 0.f;       // (nothing before it in this walk)
        T::template store<VEC>(dxp, col.s0, col.s1, (s0 + i) * os, dx0, dx1, col.odd);
        T::template store<VEC>(drp, col.s0, col.s1, (s0 + i) * os, dr0, dr1, col.odd);
        T::template store<VEC>(dgp, col.s0, col.s1, (s0 + i) * os, dg0, dg1, col.odd);
        __builtin_amdgcn_sched_barrier(0);         // a token at a time: all at once take twice the registers
      }
    }
    if (wave == 0) {                               // what the chunk before receives
      if (p.links != nullptr) link.publish_end(G0, G1);
      if (k.chunk == 0 && p.dh0 != nullptr) {
        float* const q = p.dh0 + int64_t(k.b) * D + c;
        if (ok0) q[0] = G0;
        if (ok1) q[1] = G1;
      }
    }
    sums[par][wave][lane] = make_float2(e0, e1);
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int j = 1; j < NW; ++j) {
        e0 += sums[par][j][lane].x;
        e1 += sums[par][j][lane].y;
      }
      float* const q = p.plam + (int64_t(k.chunk) * p.batch + k.b) * p.D + c;
      if (ok0) q[0] = e0;
      if (ok1) q[1] = e1;
    }
    if (!more) return false;
    k = kn;
    order = order_n;
    next = after;
    return true;
  };

  Raw w0, w1;
  load_gates(k, w0);
  load_rest(k, w0);
  if (p.persistent) {
    if (tid == 0) tickets[1] = atomicAdd(counter, 1u);
    __syncthreads();
    next = __builtin_amdgcn_readfirstlane(tickets[1]);
  }
  while (step(w0, w1, 0) && step(w1, w0, 1)) {
  }
}

// dlam: the sum of the parts [nparts][D] in a fixed order, times sigmoid(lam) / softplus(lam).
// (256 parts of 2560 channels: 4.7 us, a launch and its latencies.)
__global__ __launch_bounds__(1024) void gated_dlam_kernel(GatedParams p, int64_t nparts) {
  __shared__ float part[32][33];
  const int col = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t d = int64_t(blockIdx.x) * 32 + col;
  float sum = 0.f;
  if (d < p.D) {
#pragma unroll 8
    for (int64_t j = row; j < nparts; j += 32) sum += p.plam[j * p.D + d];
  }
  part[row][col] = sum;
  __syncthreads();
  if (row == 0 && d < p.D) {
    for (int j = 1; j < 32; ++j) sum += part[j][col];
    p.dlam[d] = sum * gated_lam_ratio(p.lam[d]);
  }
}

// One token: V channels a thread.  V = 4 where every operand can be moved in whole vectors (aligned,
// sizes and strides a multiple of 4), else 1.  512 rows of 2560 channels in bf16 (21 MB): 6.1 us
// (a call takes 8.5 on the host); 8192 rows: 52.0 us with 4, 69.4 with 1, in fp32 81.8 and 92.2.
template <typename IO, int V>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedParams p, float* __restrict__ state) {
  using T = io_traits<IO>;
  struct alignas(V * sizeof(IO)) Vec { IO v[V]; };
  struct alignas(V * 4) Vec32 { float v[V]; };
  const uint32_t per = uint32_t(p.D / V);                            // threads a batch row
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.batch * per) return;
  const int64_t b = i / per, d = (i - b * per) * V;
  const Vec x = *reinterpret_cast<const Vec*>(static_cast<const IO*>(p.x) + b * p.x_sb + d);
  const Vec r = *reinterpret_cast<const Vec*>(static_cast<const IO*>(p.r) + b * p.r_sb + d);
  const Vec g = *reinterpret_cast<const Vec*>(static_cast<const IO*>(p.g) + b * p.g_sb + d);
  Vec32 h = *reinterpret_cast<const Vec32*>(state + b * p.D + d);
  const Vec32 lam = *reinterpret_cast<const Vec32*>(p.lam + d);
  Vec y;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float a, m;
    gated_decay(-p.c * softplus_f32(lam.v[j]) * sigmoid_f32(T::widen(r.v[j])), a, m);
    h.v[j] = fmaf(a, h.v[j], m * (sigmoid_f32(T::widen(g.v[j])) * T::widen(x.v[j])));
    y.v[j] = narrow<IO>(h.v[j]);
  }
  *reinterpret_cast<Vec32*>(state + b * p.D + d) = h;
  *reinterpret_cast<Vec*>(static_cast<IO*>(p.y) + b * p.y_sb + d) = y;
}

constexpr int kGatedWaves = 8;
template <typename IO> constexpr int kGatedRun = gated_chunk(sizeof(IO) == 2) / kGatedWaves;   // tokens of a run
static_assert(kTile % kGatedRun<float> == 0 && kTile % kGatedRun<uint16_t> == 0, "checkpoints lie at the starts of runs");

unsigned blocks_for(int64_t n, int per) { return unsigned((n + per - 1) / per); }

}  // namespace

// Clears the links and, with them, forms the channels' rates; with one chunk each workgroup
// forms its own.
static hipError_t launch_gated_begin(GatedParams& p, hipStream_t stream) {
  if (p.links == nullptr) {
    p.kd = nullptr;
    return hipSuccess;
  }
  const int64_t pairs = gated_link_words(p.batch, p.D, p.n_chunks) / 2;       // (an even number of words)
  const int64_t blocks = ((pairs > p.D ? pairs : p.D) + 255) / 256;
  hipLaunchKernelGGL(gated_begin_kernel, dim3(unsigned(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream,
                     reinterpret_cast<ulonglong2*>(p.links), pairs, p.lam, p.c, p.kd, p.D);
  return hipGetLastError();
}

template <typename IO, int VEC, bool RESET>
static hipError_t launch_gated_fwd_t(GatedParams p, int cus, hipStream_t stream) {
  const int64_t items = p.batch * ((p.D + kCh - 1) / kCh) * p.n_chunks;
  const int64_t resident = cus;                    // a workgroup of eight wavefronts fills a compute unit's registers
  p.persistent = p.links != nullptr && items > resident;
  const dim3 grid(unsigned(p.persistent ? resident : items));
  hipLaunchKernelGGL((gated_fwd_kernel<IO, kGatedWaves, kGatedRun<IO>, VEC, RESET>), grid, dim3(kGatedWaves * 64), 0, stream, p);
  return hipGetLastError();
}

template <typename IO, int VEC, bool RESET>
static hipError_t launch_gated_bwd_t(GatedParams p, int cus, hipStream_t stream) {
  const int64_t items = p.batch * ((p.D + kCh - 1) / kCh) * p.n_chunks;
  const int64_t resident = cus;
  p.persistent = p.links != nullptr && items > resident;
  const dim3 grid(unsigned(p.persistent ? resident : items));
  hipLaunchKernelGGL((gated_bwd_kernel<IO, kGatedWaves, kGatedBwdChunk / kGatedWaves, VEC, RESET>), grid, dim3(kGatedWaves * 64),
                     0, stream, p);
  hipLaunchKernelGGL(gated_dlam_kernel, dim3(unsigned((p.D + 31) / 32)), dim3(1024), 0, stream, p, p.batch * p.n_chunks);
  return hipGetLastError();
}

template <typename F> static hipError_t by_type(bool bf16, const GatedParams& p, F f) {
  const bool reset = p.reset != nullptr;
  auto with = [&](auto io, auto vec) {
    return reset ? f(io, vec, std::true_type{}) : f(io, vec, std::false_type{});
  };
  auto typed = [&](auto io) {
    if (p.D == 1) return with(io, std::integral_constant<int, kSingle>{});
    if (p.D % 2 != 0) return with(io, std::integral_constant<int, kOddPairs>{});
    return with(io, std::integral_constant<int, kPairs>{});
  };
  return bf16 ? typed(uint16_t{}) : typed(float{});
}

hipError_t launch_gated_fwd(bool bf16, GatedParams p, int cus, hipStream_t stream) {
  const hipError_t e = launch_gated_begin(p, stream);
  if (e != hipSuccess) return e;
  return by_type(bf16, p, [&](auto io, auto vec, auto reset) {
    return launch_gated_fwd_t<decltype(io), decltype(vec)::value, decltype(reset)::value>(p, cus, stream);
  });
}

hipError_t launch_gated_bwd(bool bf16, GatedParams p, int cus, hipStream_t stream) {
  const hipError_t e = launch_gated_begin(p, stream);
  if (e != hipSuccess) return e;
  return by_type(bf16, p, [&](auto io, auto vec, auto reset) {
    return launch_gated_bwd_t<decltype(io), decltype(vec)::value, decltype(reset)::value>(p, cus, stream);
  });
}

hipError_t launch_gated_step(bool bf16, const GatedParams& p, float* state, hipStream_t stream) {
  const uintptr_t ptrs = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.r) | reinterpret_cast<uintptr_t>(p.g) |
                         reinterpret_cast<uintptr_t>(p.y);
  const uintptr_t floats = reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(p.lam);
  const bool vec = (p.D | p.x_sb | p.r_sb | p.g_sb | p.y_sb) % 4 == 0 && ptrs % (bf16 ? 8 : 16) == 0 && floats % 16 == 0;
  auto with = [&](auto io, auto v) {
    constexpr int V = decltype(v)::value;
    hipLaunchKernelGGL((gated_step_kernel<decltype(io), V>), dim3(blocks_for(p.batch * (p.D / V), 256)), dim3(256), 0, stream, p,
                       state);
    return hipGetLastError();
  };
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  if (bf16) return vec ? with(uint16_t{}, Four{}) : with(uint16_t{}, One{});
  return vec ? with(float{}, Four{}) : with(float{}, One{});
}

}  // namespace selscan
