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

// ---- tiles of 64 channels: a lane owns a channel pair, a half wavefront a run of S tokens

constexpr int kCh = 64;                    // channels of a workgroup
constexpr int kLinkGroup = 16;             // chunks between two chunks that publish their end state

// Two channels of one token as loaded.
template <typename IO> struct pair_io;
template <> struct pair_io<float> {
  using raw_t = float2;
  template <bool VEC>
  static __device__ __forceinline__ raw_t load(const float* p, uint32_t o0, uint32_t o1) {
    if constexpr (VEC) return *reinterpret_cast<const float2*>(p + o0);
    else return make_float2(p[o0], p[o1]);
  }
  static __device__ __forceinline__ float lo(raw_t v) { return v.x; }
  static __device__ __forceinline__ float hi(raw_t v) { return v.y; }
  template <bool VEC>
  static __device__ __forceinline__ void store(float* p, uint32_t o, float a, float b, bool ok0, bool ok1) {
    if constexpr (VEC) {
      if (ok0) *reinterpret_cast<float2*>(p + o) = make_float2(a, b);
    } else {
      if (ok0) p[o] = a;
      if (ok1) p[o + 1] = b;
    }
  }
};
template <> struct pair_io<uint16_t> {
  using raw_t = uint32_t;
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  template <bool VEC>
  static __device__ __forceinline__ raw_t load(const uint16_t* p, uint32_t o0, uint32_t o1) {
    if constexpr (VEC) return *reinterpret_cast<const uint32_t*>(p + o0);
    else return uint32_t(p[o0]) | (uint32_t(p[o1]) << 16);
  }
  static __device__ __forceinline__ float lo(raw_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(raw_t v) { return __uint_as_float(v & 0xffff0000u); }
  template <bool VEC>
  static __device__ __forceinline__ void store(uint16_t* p, uint32_t o, float a, float b, bool ok0, bool ok1) {
    const f32x2_t f = {a, b};                              // to nearest even
    const uint32_t v = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
    if constexpr (VEC) {
      if (ok0) *reinterpret_cast<uint32_t*>(p + o) = v;
    } else {
      if (ok0) p[o] = uint16_t(v);
      if (ok1) p[o + 1] = uint16_t(v >> 16);
    }
  }
};

// The links between the chunks of one chain (a batch row's 64 channels), in the workspace: zero
// until written, each word whole or absent, so a reader needs no other order between writes.
//   map [items][64]: the chunk's map h -> A h + H as {A with its sign bit set, H} (A >= 0);
//   end [groups][64]: the state behind the chunk as {1, h}, by every kLinkGroup-th chunk.
__device__ __forceinline__ void put_word(uint64_t* p, uint32_t tag, float v) {
  __hip_atomic_store(p, (uint64_t(tag) << 32) | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_word(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The writer holds a lower ticket, so it has started and waits for no later one: the wait
// ends.  It is bounded all the same; a word that never comes reads as NaN.
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

// State entering a chunk, from the maps of the chunks before it in its group and the state
// behind the group before (a fixed order of operations whatever the timing).
template <bool CUT>
__device__ __forceinline__ float link_state(const uint64_t* map, const uint64_t* end, int64_t chain, int64_t chains,
                                            int pos, int ch, float h0) {
  if (pos == 0) return h0;
  const int base = pos / kLinkGroup * kLinkGroup, n = pos - base;
  uint64_t w[kLinkGroup], e = 0;
  const uint64_t* const m = map + (int64_t(base) * chains + chain) * kCh + ch;
  const uint64_t* const ep = end + (int64_t(base / kLinkGroup - 1) * chains + chain) * kCh + ch;
  if (base > 0) e = get_word(ep);
#pragma unroll
  for (int j = 0; j < kLinkGroup - 1; ++j)
    if (j < n) w[j] = get_word(m + int64_t(j) * chains * kCh);
  float h = base > 0 ? __uint_as_float(uint32_t(wait_word(ep, e))) : h0;
#pragma unroll
  for (int j = 0; j < kLinkGroup - 1; ++j)
    if (j < n) {
      const uint64_t v = wait_word(m + int64_t(j) * chains * kCh, w[j]);
      h = through<CUT>(fabsf(__uint_as_float(uint32_t(v >> 32))), __uint_as_float(uint32_t(v)), h);
    }
  return h;
}

// One workgroup per chunk of 2 NW S tokens and 64 channels.  Each half wavefront forms the map
// of its S tokens in registers; the maps meet in LDS, the workgroup's in the links; every half
// wavefront then walks its tokens from the state that enters them.  The inputs are read once.
// Workgroups take their chunks by ticket, all chains' first chunks first, so that a chunk's
// predecessors have been started before it.
template <typename IO, int NW, int S, bool VEC, bool RESET>
__global__ __launch_bounds__(NW * 64) void gated_fwd_kernel(GatedParams p) {
  using T = pair_io<IO>;
  constexpr int NSB = 2 * NW, kLen = NSB * S;
  __shared__ float4 maps[NSB][kCh / 2];
  __shared__ float2 enter[kCh / 2];
  __shared__ uint32_t ticket;
  const int tid = threadIdx.x, lane = tid & 31, sb = tid >> 5;
  uint32_t item = blockIdx.x;
  if (p.links != nullptr) {
    if (tid == 0) ticket = atomicAdd(reinterpret_cast<uint32_t*>(p.links), 1u);
    __syncthreads();
    item = ticket;
  }
  const uint32_t ctiles = uint32_t((p.D + kCh - 1) / kCh), chains = uint32_t(p.batch) * ctiles;
  const uint32_t chunk = item / chains, chain = item % chains, b = chain / ctiles, ct = chain % ctiles;
  const int64_t t0 = int64_t(chunk) * kLen;
  const int rest = int(p.L - t0 < kLen ? p.L - t0 : kLen);       // tokens of this chunk
  const int c = int(ct) * kCh + 2 * lane, D = int(p.D);
  const bool ok0 = c < D, ok1 = c + 1 < D;
  const uint32_t c0 = ok0 ? c : (VEC ? D - 2 : D - 1), c1 = ok1 ? c + 1 : D - 1;
  const IO* const xp = static_cast<const IO*>(p.x) + b * p.x_sb + t0 * p.x_sl;
  const IO* const rp = static_cast<const IO*>(p.r) + b * p.r_sb + t0 * p.r_sl;
  const IO* const gp = static_cast<const IO*>(p.g) + b * p.g_sb + t0 * p.g_sl;
  const uint32_t xs = uint32_t(p.x_sl), rs = uint32_t(p.r_sl), gs = uint32_t(p.g_sl);
  const int s0 = sb * S;                                        // this run's first token in the chunk

  typename T::raw_t xr[S], rr[S], gr[S];
  bool first[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const uint32_t t = s0 + i < rest ? s0 + i : rest - 1;
    rr[i] = T::template load<VEC>(rp, t * rs + c0, t * rs + c1);
    gr[i] = T::template load<VEC>(gp, t * gs + c0, t * gs + c1);
    xr[i] = T::template load<VEC>(xp, t * xs + c0, t * xs + c1);
    first[i] = RESET ? p.reset[b * p.reset_sb + t0 + t] != 0 : false;
  }
  const float k0 = p.c * softplus_f32(p.lam[c0]), k1 = p.c * softplus_f32(p.lam[c1]);

  float a0[S], a1[S], b0[S], b1[S];
  auto tokens = [&](auto decay) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float m0, m1;
      decay(-k0 * sigmoid_f32(T::lo(rr[i])), a0[i], m0);
      decay(-k1 * sigmoid_f32(T::hi(rr[i])), a1[i], m1);
      if (RESET && first[i]) { a0[i] = a1[i] = 0.f; m0 = m1 = 1.f; }
      b0[i] = m0 * (sigmoid_f32(T::lo(gr[i])) * T::lo(xr[i]));
      b1[i] = m1 * (sigmoid_f32(T::hi(gr[i])) * T::hi(xr[i]));
    }
  };
  // |log a| is at most k: where that is small for the whole wavefront, no exp2 is needed
  if (__all(k0 < kGatedSmall && k1 < kGatedSmall)) tokens([](float y, float& a, float& m) { gated_decay_small(y, a, m); });
  else tokens([](float y, float& a, float& m) { gated_decay(y, a, m); });
  if (rest < kLen) {                                            // tokens behind the last: the map that changes nothing
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (s0 + i >= rest) { a0[i] = a1[i] = 1.f; b0[i] = b1[i] = 0.f; first[i] = false; }
  }

  float A0 = 1.f, A1 = 1.f, H0 = 0.f, H1 = 0.f;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (RESET && first[i]) { A0 = A1 = H0 = H1 = 0.f; }
    H0 = fmaf(a0[i], H0, b0[i]);
    H1 = fmaf(a1[i], H1, b1[i]);
    A0 *= a0[i];
    A1 *= a1[i];
  }
  maps[sb][lane] = make_float4(A0, A1, H0, H1);
  __syncthreads();
  if (tid < kCh) {                                              // the first wavefront, a lane a channel
    const float* const col = reinterpret_cast<const float*>(&maps[0][tid >> 1]) + (tid & 1);
    const int ch = int(ct) * kCh + tid;
    float A = 1.f, H = 0.f;
#pragma unroll
    for (int j = 0; j < NSB; ++j) {
      const float Aj = col[j * kCh * 2], Hj = col[j * kCh * 2 + 2];
      H = through<RESET>(Aj, Hj, H);
      A = RESET && Aj == 0.f ? 0.f : A * Aj;
    }
    float h = p.h0 != nullptr && ch < D ? p.h0[int64_t(b) * D + ch] : 0.f;
    if (p.links != nullptr) {
      uint64_t* const map = p.links + kCh;
      uint64_t* const end = map + int64_t(p.n_chunks) * chains * kCh;
      const bool last = int(chunk) == p.n_chunks - 1;
      if (!last) put_word(map + int64_t(item) * kCh + tid, __float_as_uint(A) | 0x80000000u, H);
      h = link_state<RESET>(map, end, chain, chains, int(chunk), tid, h);
      if (!last && chunk % kLinkGroup == kLinkGroup - 1)
        put_word(end + (int64_t(chunk / kLinkGroup) * chains + chain) * kCh + tid, 1u, through<RESET>(A, H, h));
    }
    reinterpret_cast<float*>(enter)[tid] = h;
    if (p.last != nullptr && ch < D && int(chunk) == p.n_chunks - 1) p.last[int64_t(b) * D + ch] = through<RESET>(A, H, h);
  }
  __syncthreads();
  float h0 = enter[lane].x, h1 = enter[lane].y;
  for (int j = 0; j < sb; ++j) {
    const float4 m = maps[j][lane];
    h0 = through<RESET>(m.x, m.z, h0);
    h1 = through<RESET>(m.y, m.w, h1);
  }
  if (p.ckpt != nullptr && s0 % kTile == 0 && s0 < rest) {
    float* const o = p.ckpt + (b * p.ntiles + (t0 + s0) / kTile) * p.D + c;
    if (ok0) o[0] = h0;
    if (ok1) o[1] = h1;
  }
  if (p.y == nullptr) return;
  IO* const yp = static_cast<IO*>(p.y) + b * p.y_sb + t0 * p.y_sl;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (RESET && first[i]) h0 = h1 = 0.f;
    h0 = fmaf(a0[i], h0, b0[i]);
    h1 = fmaf(a1[i], h1, b1[i]);
    if (s0 + i < rest) T::template store<VEC>(yp, uint32_t(s0 + i) * uint32_t(p.y_sl) + uint32_t(c), h0, h1, ok0, ok1);
  }
}

__global__ __launch_bounds__(256) void clear_links_kernel(uint64_t* p, int64_t n) {
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = 0;
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

constexpr int kGatedWaves = 8, kGatedRun = 16;      // wavefronts and tokens of a run
static_assert(kGatedChunk == 2 * kGatedWaves * kGatedRun, "chunk length");
static_assert(kTile % kGatedRun == 0 && kGatedChunk % kTile == 0, "checkpoints lie at the starts of runs");

unsigned blocks_for(int64_t n, int per) { return unsigned((n + per - 1) / per); }

}  // namespace

hipError_t launch_clear_links(const GatedParams& p, int64_t words, hipStream_t stream) {
  const int64_t blocks = (words + 1023) / 1024;
  hipLaunchKernelGGL(clear_links_kernel, dim3(unsigned(blocks < 1024 ? blocks : 1024)), dim3(256), 0, stream, p.links, words);
  return hipGetLastError();
}

template <typename IO, bool VEC, bool RESET>
static hipError_t launch_gated_fwd_t(const GatedParams& p, hipStream_t stream) {
  const dim3 grid(unsigned(p.batch * ((p.D + kCh - 1) / kCh) * p.n_chunks));
  hipLaunchKernelGGL((gated_fwd_kernel<IO, kGatedWaves, kGatedRun, VEC, RESET>), grid, dim3(kGatedWaves * 64), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_gated_fwd(bool bf16, const GatedParams& p, hipStream_t stream) {
  if (p.links != nullptr) {
    const hipError_t e = launch_clear_links(p, gated_link_words(p.batch, p.D, p.n_chunks), stream);
    if (e != hipSuccess) return e;
  }
  const bool reset = p.reset != nullptr;
  if (bf16)
    return p.vec ? (reset ? launch_gated_fwd_t<uint16_t, true, true>(p, stream) : launch_gated_fwd_t<uint16_t, true, false>(p, stream))
                 : (reset ? launch_gated_fwd_t<uint16_t, false, true>(p, stream) : launch_gated_fwd_t<uint16_t, false, false>(p, stream));
  return p.vec ? (reset ? launch_gated_fwd_t<float, true, true>(p, stream) : launch_gated_fwd_t<float, true, false>(p, stream))
               : (reset ? launch_gated_fwd_t<float, false, true>(p, stream) : launch_gated_fwd_t<float, false, false>(p, stream));
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
