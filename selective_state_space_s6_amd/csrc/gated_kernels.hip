// gated_kernels.hip -- the gated linear recurrence: forward, backward and decode step.
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
// scalar register, the channels' in one (VEC) or two vector registers.  The descriptor ends
// with the chunk's last row and kNoChannel lies behind any: loads out of range give zero and
// stores are dropped, so neither the last tokens nor the last channels need a branch.
constexpr uint32_t kNoChannel = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const void* p, int rows, int row_bytes, int cols_bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (rows - 1) * row_bytes + cols_bytes, 0x00020000);
}
template <typename IO> struct pair_io;
template <> struct pair_io<float> {
  typedef uint32_t raw_t __attribute__((ext_vector_type(2)));
  template <bool VEC> static __device__ __forceinline__ raw_t load(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row) {
    if constexpr (VEC) return __builtin_bit_cast(raw_t, __builtin_amdgcn_raw_buffer_load_b64(r, o0, row, 0));
    else return raw_t{__builtin_amdgcn_raw_buffer_load_b32(r, o0, row, 0), __builtin_amdgcn_raw_buffer_load_b32(r, o1, row, 0)};
  }
  static __device__ __forceinline__ float lo(raw_t v) { return __uint_as_float(v.x); }
  static __device__ __forceinline__ float hi(raw_t v) { return __uint_as_float(v.y); }
  template <bool VEC>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row, float a, float b) {
    const raw_t v = {__float_as_uint(a), __float_as_uint(b)};
    if constexpr (VEC) {
      __builtin_amdgcn_raw_buffer_store_b64(v, r, o0, row, 0);
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
  template <bool VEC> static __device__ __forceinline__ raw_t load(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row) {
    if constexpr (VEC) return __builtin_amdgcn_raw_buffer_load_b32(r, o0, row, 0);
    else return uint32_t(__builtin_amdgcn_raw_buffer_load_b16(r, o0, row, 0)) |
                (uint32_t(__builtin_amdgcn_raw_buffer_load_b16(r, o1, row, 0)) << 16);
  }
  static __device__ __forceinline__ float lo(raw_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(raw_t v) { return __uint_as_float(v & 0xffff0000u); }
  template <bool VEC>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t o0, uint32_t o1, int row, float a, float b) {
    const f32x2_t f = {a, b};                              // to nearest even
    const uint32_t v = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
    if constexpr (VEC) {
      __builtin_amdgcn_raw_buffer_store_b32(v, r, o0, row, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b16(uint16_t(v), r, o0, row, 0);
      __builtin_amdgcn_raw_buffer_store_b16(uint16_t(v >> 16), r, o1, row, 0);
    }
  }
};

// The links between the chunks of one chain (a batch row's 64 channels), in the workspace: zero
// until written, each word whole or absent, so a reader needs no other order between writes.
//   map [items][2][64]: the chunk's map h -> A h + H as {A with its sign bit set, H} (A >= 0),
//     the even channels before the odd ones;
//   end [groups][2][64]: the state behind the chunk as {1, h}, by every kLinkGroup-th chunk.
__device__ __forceinline__ void put_word(uint64_t* p, uint32_t tag, float v) {
  __hip_atomic_store(p, (uint64_t(tag) << 32) | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_word(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The wait ends (see the kernels' tickets).  It is bounded all the same; a word that never comes
// reads as NaN.
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

// What a ticket stands for: one chunk of one chain.  Tickets run over all chains' first chunks,
// then their second ones, and so on.
struct Chunk {
  uint32_t chunk, chain, b, ct;
  int64_t t0;
  int rest;                                // tokens
};
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

// Chunks of NW S tokens and 128 channels.  Each wavefront forms the map of its S tokens in
// registers; the maps meet in LDS, the workgroup's in the links, where the maps of the chunks
// since the last published state and that state are read, one by each wavefront; every
// wavefront then walks its tokens from the state that enters them, composed in a fixed order.
// The inputs are read once.  A workgroup takes chunk after chunk by ticket, the next one's
// inputs in flight while it waits for the links of this one.  A chunk's predecessors have
// lower tickets, so whoever holds them works on them or on still lower ones: every wait ends.
template <typename IO, int NW, int S, bool VEC, bool RESET>
__global__ __launch_bounds__(NW * 64) void gated_fwd_kernel(GatedParams p) {
  using T = pair_io<IO>;
  constexpr int kLen = NW * S, kGroup = kLinkGroup;
  static_assert(kGroup <= NW, "a wavefront reads one link");
  __shared__ float4 maps[2][NW][kCh / 2];          // of the wavefronts' tokens
  __shared__ float4 links[2][kGroup][kCh / 2];        // of the chunks before; [0] the state behind their group
  __shared__ uint32_t tickets[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t ctiles = uint32_t((p.D + kCh - 1) / kCh), chains = uint32_t(p.batch) * ctiles;
  const uint32_t total = chains * uint32_t(p.n_chunks);
  constexpr int es = int(sizeof(IO));
  const int xs = int(p.x_sl) * es, rs = int(p.r_sl) * es, gs = int(p.g_sl) * es, ys = int(p.y_sl) * es;   // bytes
  const int D = int(p.D), s0 = wave * S;           // this wavefront's first token in a chunk
  uint32_t* const counter = reinterpret_cast<uint32_t*>(p.links);
  uint32_t now = blockIdx.x, next = total;         // the first chunk's ticket and the following one's
  if (p.links != nullptr) {
    if (tid == 0) tickets[0] = atomicAdd(counter, 1u);
    __syncthreads();
    now = __builtin_amdgcn_readfirstlane(tickets[0]);
    if (now >= total) return;
  }

  struct Raw {
    typename T::raw_t x[S], r[S], g[S];
    uint32_t firsts;                               // bit i: token i starts a sequence
    float k0, k1;
  };
  auto load = [&](const Chunk& k, Raw& w) __attribute__((always_inline)) {
    const auto xp = chunk_rsrc(static_cast<const IO*>(p.x) + k.b * p.x_sb + k.t0 * p.x_sl, k.rest, xs, D * es);
    const auto rp = chunk_rsrc(static_cast<const IO*>(p.r) + k.b * p.r_sb + k.t0 * p.r_sl, k.rest, rs, D * es);
    const auto gp = chunk_rsrc(static_cast<const IO*>(p.g) + k.b * p.g_sb + k.t0 * p.g_sl, k.rest, gs, D * es);
    const int c = int(k.ct) * kCh + 2 * lane;
    w.k0 = c < D ? p.kd[c] : 0.f;
    w.k1 = c + 1 < D ? p.kd[c + 1] : 0.f;
    const uint32_t o0 = c < D ? c * es : kNoChannel, o1 = c + 1 < D ? (c + 1) * es : kNoChannel;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      w.r[i] = T::template load<VEC>(rp, o0, o1, (s0 + i) * rs);
      w.g[i] = T::template load<VEC>(gp, o0, o1, (s0 + i) * gs);
      w.x[i] = T::template load<VEC>(xp, o0, o1, (s0 + i) * xs);
    }
    if constexpr (RESET) {
      const int t = s0 + (lane & (S - 1));
      const bool f = t < k.rest && p.reset[k.b * p.reset_sb + k.t0 + t] != 0;
      w.firsts = uint32_t(__ballot(f)) & ((1u << S) - 1u);
    }
  };

  Chunk k = chunk_of<kLen>(p, now, chains, ctiles);
  // Chunk k from `w`, the following one's inputs on their way into `wn`; false after the last.
  auto step = [&](Raw& w, Raw& wn, const int par) __attribute__((always_inline)) -> bool {
    const bool more = next < total;
    const Chunk kn = chunk_of<kLen>(p, more ? next : 0, chains, ctiles);
    if (more) load(kn, wn);
    uint32_t after = total;
    if (more && tid == 0) after = atomicAdd(counter, 1u);
    float a0[S], a1[S], b0[S], b1[S];
    // |log a| is at most k: where that is small for the whole wavefront, no exp2 is needed.  (The
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
        if (RESET && (w.firsts >> (i0 + i) & 1)) { a0[i0 + i] = a1[i0 + i] = 0.f; m0[i] = m1[i] = 1.f; }
        b0[i0 + i] = m0[i] * (sigmoid_f32(T::lo(w.g[i0 + i])) * T::lo(w.x[i0 + i]));
        b1[i0 + i] = m1[i] * (sigmoid_f32(T::hi(w.g[i0 + i])) * T::hi(w.x[i0 + i]));
      }
    }
    if (k.rest < kLen) {                           // behind the last token: the map that changes nothing
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (s0 + i >= k.rest) { a0[i] = a1[i] = 1.f; b0[i] = b1[i] = 0.f; }
    }
    const uint32_t cuts = w.firsts;
    float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (RESET && (cuts >> i & 1)) { A0 = A1 = H0 = H1 = 0.f; }
      H0 = fmaf(a0[i], H0, b0[i]);
      H1 = fmaf(a1[i], H1, b1[i]);
      A0 *= a0[i];
      A1 *= a1[i];
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
    const int pos = int(k.chunk) % kGroup;         // maps between the last published state and this chunk
    uint64_t* const map = p.links + kTicketWords + (int64_t(k.chunk) * chains + k.chain) * kCh + lane;
    uint64_t* const end = p.links + kTicketWords +
                          (int64_t(p.n_chunks) * chains + int64_t(k.chunk / kGroup) * chains + k.chain) * kCh + lane;
    if (wave == NW - 1 && !last) {                 // the chunk's map, before any wait
      float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const float4 m = maps[par][j][lane];
        H0 = through<RESET>(m.x, m.z, H0);
        H1 = through<RESET>(m.y, m.w, H1);
        A0 = RESET && m.x == 0.f ? 0.f : A0 * m.x;
        A1 = RESET && m.y == 0.f ? 0.f : A1 * m.y;
      }
      put_word(map, __float_as_uint(A0) | 0x80000000u, H0);
      put_word(map + 64, __float_as_uint(A1) | 0x80000000u, H1);
    }
    if (k.chunk > 0 && wave <= pos && wave < kGroup) {
      // wavefront 0 reads the state behind the group before, wavefront j the map of the group's
      // chunk j - 1
      const uint64_t* const q = wave == 0 ? end - int64_t(chains) * kCh : map - int64_t(pos - wave + 1) * chains * kCh;
      if (wave > 0 || int(k.chunk) >= kGroup) {
        const uint64_t f0 = get_word(q), f1 = get_word(q + 64);
        const uint64_t w0 = wait_word(q, f0), w1 = wait_word(q + 64, f1);
        links[par][wave][lane] = make_float4(fabsf(__uint_as_float(uint32_t(w0 >> 32))), fabsf(__uint_as_float(uint32_t(w1 >> 32))),
                                        __uint_as_float(uint32_t(w0)), __uint_as_float(uint32_t(w1)));
      } else {
        links[par][0][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    __syncthreads();
    after = __builtin_amdgcn_readfirstlane(tickets[par]);
    float h0 = links[par][0][lane].z, h1 = links[par][0][lane].w;
    for (int j = 1; j <= pos; ++j) {
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
    const uint32_t o0 = ok0 ? c * es : kNoChannel, o1 = ok1 ? (c + 1) * es : kNoChannel;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (RESET && (cuts >> i & 1)) h0 = h1 = 0.f;
      h0 = fmaf(a0[i], h0, b0[i]);
      h1 = fmaf(a1[i], h1, b1[i]);
      if (p.y != nullptr) T::template store<VEC>(yp, o0, o1, (s0 + i) * ys, h0, h1);
    }
    if (wave == NW - 1) {                          // the state behind the chunk
      if (!last && pos == kGroup - 1) {
        put_word(end, 1u, h0);
        put_word(end + 64, 1u, h1);
      }
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
  load(k, w0);
  if (p.persistent) {
    if (tid == 0) tickets[1] = atomicAdd(counter, 1u);
    __syncthreads();
    next = __builtin_amdgcn_readfirstlane(tickets[1]);
  }
  while (step(w0, w1, 0) && step(w1, w0, 1)) {
  }
}

// What the chunks of one call share: the links, empty, and the channels' c softplus(lam).
__global__ __launch_bounds__(256) void gated_begin_kernel(uint64_t* links, int64_t words, const float* lam, float c, float* kd,
                                                          int64_t D) {
  const int64_t i0 = blockIdx.x * int64_t(256) + threadIdx.x, n = int64_t(gridDim.x) * 256;
  for (int64_t i = i0; i < words; i += n) links[i] = 0;
  for (int64_t i = i0; i < D; i += n) kd[i] = c * softplus_f32(lam[i]);
}

// One thread walks one channel of one batch row backwards, tile by tile; a tile's states are
// formed again from its checkpoint.
template <typename IO>
__global__ __launch_bounds__(64) void gated_bwd_kernel(GatedParams p) {
  using T = io_traits<IO>;
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= p.batch * p.D) return;
  const int64_t b = i / p.D, d = i % p.D;
  const IO* x = static_cast<const IO*>(p.x) + b * p.x_sb + d;
  const IO* r = static_cast<const IO*>(p.r) + b * p.r_sb + d;
  const IO* g = static_cast<const IO*>(p.g) + b * p.g_sb + d;
  const IO* dy = static_cast<const IO*>(p.dy) + b * p.y_sb + d;
  const int64_t o = b * p.L * p.D + d;
  IO* dx = static_cast<IO*>(p.dx) + o;
  IO* dr = static_cast<IO*>(p.dr) + o;
  IO* dg = static_cast<IO*>(p.dg) + o;
  float* hb = p.hbuf + b * kTile * p.D + d;               // state before each token of the tile
  const float k = p.c * softplus_f32(p.lam[d]);
  float adj = p.dlast ? p.dlast[i] : 0.f, sum = 0.f;
  for (int64_t tile = p.ntiles - 1; tile >= 0; --tile) {
    const int64_t t0 = tile * kTile, t1 = t0 + kTile < p.L ? t0 + kTile : p.L;
    float h = p.ckpt[(b * p.ntiles + tile) * p.D + d];
    for (int64_t t = t0; t < t1; ++t) {
      hb[(t - t0) * p.D] = h;
      float a, m;
      gated_decay(-k * sigmoid_f32(T::widen(r[t * p.r_sl])), a, m);
      if (p.reset && p.reset[b * p.reset_sb + t]) { a = h = 0.f; m = 1.f; }
      h = fmaf(a, h, m * (sigmoid_f32(T::widen(g[t * p.g_sl])) * T::widen(x[t * p.x_sl])));
    }
    for (int64_t t = t1 - 1; t >= t0; --t) {
      float s, s1, sg, sg1;
      sigmoid_pair(T::widen(r[t * p.r_sl]), s, s1);
      sigmoid_pair(T::widen(g[t * p.g_sl]), sg, sg1);
      const float v = sg * T::widen(x[t * p.x_sl]), la = -k * s;
      float a, m;
      gated_decay(la, a, m);
      const bool first = p.reset && p.reset[b * p.reset_sb + t];
      if (first) { a = 0.f; m = 1.f; }
      adj += T::widen(dy[t * p.y_sl]);
      const float w = m > 0.f ? la / m : 0.f, dv = adj * m;
      const float e = first ? 0.f : adj * a * (la * hb[(t - t0) * p.D] - a * w * v);
      dx[t * p.D] = narrow<IO>(dv * sg);
      dr[t * p.D] = narrow<IO>(e * s1);
      dg[t * p.D] = narrow<IO>(dv * v * sg1);
      sum += e;
      adj = first ? 0.f : adj * a;
    }
  }
  if (p.dh0) p.dh0[i] = adj;
  p.plam[i] = sum;
}

__global__ __launch_bounds__(64) void gated_dlam_kernel(GatedParams p) {
  const int64_t d = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (d >= p.D) return;
  float sum = 0.f;
  for (int64_t b = 0; b < p.batch; ++b) sum += p.plam[b * p.D + d];
  p.dlam[d] = sum * gated_lam_ratio(p.lam[d]);
}

template <typename IO>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedParams p, float* state) {
  using T = io_traits<IO>;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.batch * p.D) return;
  const int64_t b = i / p.D, d = i % p.D;
  float a, m;
  gated_decay(-p.c * softplus_f32(p.lam[d]) * sigmoid_f32(T::widen(static_cast<const IO*>(p.r)[b * p.r_sb + d])), a, m);
  const float v = sigmoid_f32(T::widen(static_cast<const IO*>(p.g)[b * p.g_sb + d])) *
                  T::widen(static_cast<const IO*>(p.x)[b * p.x_sb + d]);
  const float h = fmaf(a, state[i], m * v);
  state[i] = h;
  static_cast<IO*>(p.y)[b * p.y_sb + d] = narrow<IO>(h);
}

constexpr int kGatedWaves = 8;
template <typename IO> constexpr int kGatedRun = gated_chunk(sizeof(IO) == 2) / kGatedWaves;   // tokens of a run
static_assert(kTile % kGatedRun<float> == 0 && kTile % kGatedRun<uint16_t> == 0, "checkpoints lie at the starts of runs");

unsigned blocks_for(int64_t n, int per) { return unsigned((n + per - 1) / per); }

}  // namespace

template <typename IO, bool VEC, bool RESET>
static hipError_t launch_gated_fwd_t(GatedParams p, int cus, hipStream_t stream) {
  const int64_t items = p.batch * ((p.D + kCh - 1) / kCh) * p.n_chunks;
  const int64_t resident = cus;                    // a workgroup of eight wavefronts fills a compute unit's registers
  p.persistent = p.links != nullptr && items > resident;
  const dim3 grid(unsigned(p.persistent ? resident : items));
  hipLaunchKernelGGL((gated_fwd_kernel<IO, kGatedWaves, kGatedRun<IO>, VEC, RESET>), grid, dim3(kGatedWaves * 64), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_gated_fwd(bool bf16, const GatedParams& p, int cus, hipStream_t stream) {
  const int64_t words = p.links ? gated_link_words(p.batch, p.D, p.n_chunks) : 0;
  const int64_t blocks = ((words > p.D ? words : p.D) + 1023) / 1024;
  hipLaunchKernelGGL(gated_begin_kernel, dim3(unsigned(blocks < 1024 ? blocks : 1024)), dim3(256), 0, stream, p.links, words,
                     p.lam, p.c, p.kd, p.D);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool reset = p.reset != nullptr;
  if (bf16)
    return p.vec ? (reset ? launch_gated_fwd_t<uint16_t, true, true>(p, cus, stream) : launch_gated_fwd_t<uint16_t, true, false>(p, cus, stream))
                 : (reset ? launch_gated_fwd_t<uint16_t, false, true>(p, cus, stream) : launch_gated_fwd_t<uint16_t, false, false>(p, cus, stream));
  return p.vec ? (reset ? launch_gated_fwd_t<float, true, true>(p, cus, stream) : launch_gated_fwd_t<float, true, false>(p, cus, stream))
               : (reset ? launch_gated_fwd_t<float, false, true>(p, cus, stream) : launch_gated_fwd_t<float, false, false>(p, cus, stream));
}

hipError_t launch_gated_bwd(bool bf16, const GatedParams& p, hipStream_t stream) {
  const dim3 grid(blocks_for(p.batch * p.D, 64));
  if (bf16) hipLaunchKernelGGL(gated_bwd_kernel<uint16_t>, grid, dim3(64), 0, stream, p);
  else hipLaunchKernelGGL(gated_bwd_kernel<float>, grid, dim3(64), 0, stream, p);
  hipLaunchKernelGGL(gated_dlam_kernel, dim3(blocks_for(p.D, 64)), dim3(64), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_gated_step(bool bf16, const GatedParams& p, float* state, hipStream_t stream) {
  const dim3 grid(blocks_for(p.batch * p.D, 256));
  if (bf16) hipLaunchKernelGGL(gated_step_kernel<uint16_t>, grid, dim3(256), 0, stream, p, state);
  else hipLaunchKernelGGL(gated_step_kernel<float>, grid, dim3(256), 0, stream, p, state);
  return hipGetLastError();
}

}  // namespace selscan
