// cache_kernels.hip -- the 8-bit state cache: writing, reading, and the decode steps of the
// selective scan and of the scalar-decay layer on cached states.  Reading is bound by its bytes;
// the others stand between their bytes and the arithmetic on each value, which therefore is
// kept short: a code is the integer part of a sum (seeded) or rounded and packed in one instruction
// (v_cvt_pk_u8_f32), both biased by 128, and a pair of values shares one 32-bit mix for its rounding.
#include <type_traits>

#include "device_common.h"
#include "scan_launch.h"

namespace selscan {
namespace {

constexpr float kTinyRow = 0x1p-100f;     // rows whose largest magnitude is below are zero
constexpr float kCodes = 127.f;
constexpr uint32_t kBias = 0x80808080u;   // code + 128 in each byte

// ---- the 16 random bits of a value: whole-number mixing of the seed, the row's index and the
// value's place in the row.  Rounding needs no more than that neighbouring values, rows and
// seeds do not follow one another, which two multiplications by odd numbers with the high
// half folded back before each give (tests count the bits).
__device__ __forceinline__ uint32_t mix_bits(uint32_t v) {
  v ^= v >> 16;
  v *= 0xBB67AE85u;
  return v ^ (v >> 15);
}
__device__ __forceinline__ uint32_t row_key(int64_t seed, uint32_t row) {
  const uint32_t k = mix_bits(uint32_t(uint64_t(seed)) ^ (row * 0x9E3779B9u));
  return mix_bits(k ^ uint32_t(uint64_t(seed) >> 32));
}
// of the values 2 pair (low half) and 2 pair + 1 (high half)
__device__ __forceinline__ uint32_t pair_bits(uint32_t key, uint32_t pair) { return mix_bits(key + pair * 0x9E3779B9u); }

struct RowScale {
  float scale, inv;
  bool bad;                               // an infinity or a NaN in the row: a NaN scale, zero codes
};
// The scale amax / 127 and the codes' factor 1 / scale, each within half an ulp (a Newton step after
// the product with 1 / 127 and after v_rcp_f32): |h| inv stays below 127 (1 + 2^-23), 127 + 2^-16.
__device__ __forceinline__ RowScale row_scale(float amax, bool bad) {
  constexpr float kOne127 = 1.f / kCodes;
  const float s0 = amax * kOne127, s = fmaf(fmaf(-kCodes, s0, amax), kOne127, s0);
  const float r0 = __builtin_amdgcn_rcpf(s);
  RowScale r{s, fmaf(fmaf(-s, r0, 1.f), r0, r0), bad};
  if (!(amax >= kTinyRow)) r.scale = r.inv = 0.f;
  if (bad) r.scale = __builtin_nanf("");
  return r;
}
// Four codes of values 4 quad .. 4 quad + 3 of a row.
// Seeded: floor(t + u), t = h inv, u = (k + 1/2) / 65536, from the sum t + 384 + j / 32768, j = k / 2
// rounded down.  It lies in (256, 512), where numbers are 2^-15 apart, so its bits 15 to 22 are the
// floor + 128, and t's rounding to 2^-15 stands for the rest of u.  A t within 2^-16 of a code is
// that code's whatever k is: a state that a token leaves as it was, c scale, is off by half an ulp
// like inv, 127 2^-23 < 2^-16 together, and keeps c.  (With 128 in place of 384 and a rounding
// conversion, one in 2^16 of the odd codes fell by one a token, and 127 cannot rise again.)
// To nearest: v_cvt_pk_u8_f32 rounds ties to even, 2^-16 more sends them up.
template <bool SEEDED>
__device__ __forceinline__ uint32_t pack_codes(const float (&h)[4], const RowScale& r, uint32_t key, uint32_t quad) {
  uint32_t q = 0;
  if constexpr (SEEDED) {
    const uint32_t w0 = pair_bits(key, 2 * quad), w1 = pair_bits(key, 2 * quad + 1);
    auto sum = [&](float v, uint32_t j) { return __float_as_uint(fmaf(v, r.inv, __uint_as_float(j | 0x43c00000u))); };
    const uint32_t s0 = sum(h[0], (w0 >> 1) & 0x7fffu), s1 = sum(h[1], w0 >> 17);
    const uint32_t s2 = sum(h[2], (w1 >> 1) & 0x7fffu), s3 = sum(h[3], w1 >> 17);
    // bytes 1 and 2 of two sums side by side, shifted to whole bytes
    const uint32_t p0 = __builtin_amdgcn_perm(s1, s0, 0x06050201u) >> 7, p1 = __builtin_amdgcn_perm(s3, s2, 0x06050201u) >> 7;
    q = __builtin_amdgcn_perm(p1, p0, 0x06040200u);
  } else {
    constexpr float kOff = 128.f + 0x1p-16f;
    q = __builtin_amdgcn_cvt_pk_u8_f32(fmaf(h[0], r.inv, kOff), 0, q);
    q = __builtin_amdgcn_cvt_pk_u8_f32(fmaf(h[1], r.inv, kOff), 1, q);
    q = __builtin_amdgcn_cvt_pk_u8_f32(fmaf(h[2], r.inv, kOff), 2, q);
    q = __builtin_amdgcn_cvt_pk_u8_f32(fmaf(h[3], r.inv, kOff), 3, q);
  }
  return r.bad ? 0u : q ^ kBias;
}
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// the slot that batch row b names, or -1
__device__ __forceinline__ int64_t slot_of(const int32_t* ids, int64_t b, int64_t slots) {
  const int64_t s = ids ? int64_t(ids[b]) : b;
  return s >= 0 && s < slots ? s : -1;
}

// Over the L lanes (a power of two) that share a row.  After the exchanges within a quad all its
// lanes agree, so mirrors of 8 and of 16 lanes join quads and halves of a row of 16.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, false));
}
template <int L, typename F> __device__ __forceinline__ float group_all(float v, F f) {
  if constexpr (L >= 2) v = f(v, dpp<0xB1>(v));
  if constexpr (L >= 4) v = f(v, dpp<0x4E>(v));
  if constexpr (L >= 8) v = f(v, dpp<0x141>(v));
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v));
  if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16));
  return v;
}
__device__ __forceinline__ float fmax2(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float fadd2(float a, float b) { return a + b; }

// whether a lane of the row found one
template <int L> __device__ __forceinline__ bool row_bad(bool bad) {
  return __any(bad) ? group_all<L>(bad ? 1.f : 0.f, fmax2) != 0.f : false;
}

// Four codes of a row, n of them present, and back; WORDS: whole and on a 4-byte boundary.
template <bool WORDS> __device__ __forceinline__ uint32_t load_codes(const int8_t* q, int n) {
  if constexpr (WORDS) return n > 0 ? *reinterpret_cast<const uint32_t*>(q) : 0u;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) w |= uint32_t(uint8_t(q[j])) << (8 * j);
  return w;
}
template <bool WORDS> __device__ __forceinline__ void store_codes(int8_t* q, int n, uint32_t w) {
  if constexpr (WORDS) {
    if (n > 0) *reinterpret_cast<uint32_t*>(q) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) q[j] = int8_t(w >> (8 * j));
  }
}
// two floats as bf16, to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}
// Code j of four.  (Written out: the compiler takes the byte apart first, two instructions a code.)
__device__ __forceinline__ float code_value(uint32_t w, int j) {
  float v;
  if (j == 0) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(v) : "v"(w));
  else if (j == 1) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(v) : "v"(w));
  else if (j == 2) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(v) : "v"(w));
  else asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(v) : "v"(w));
  return v;
}

// Writing: four values a lane, L lanes a row, whole lines in and out; a workgroup stays within one
// state, so its slot and the division for it are scalar.  256 states of 2560 x 16 (55 MB): 11.2 us,
// 4.9 TB/s, seeded 11.8 (with a vector division for every lane's state 12.4, in 64 bits 14.1).
// WORDS: rows of whole fours, codes on 4-byte and states on 16-byte boundaries; 1024 states take
// 36.0 us (seeded 37.1), value by value 48.0.
template <int L, bool WORDS, bool SEEDED>
__global__ __launch_bounds__(256) void cache_write_kernel(const float* __restrict__ state, CacheParams p) {
  const uint32_t rows = uint32_t(p.rows), len = uint32_t(p.row_len), elems = uint32_t(p.elems);
  const uint32_t per = (rows + 256 / L - 1) / (256 / L);            // workgroups a state
  const uint32_t b = __builtin_amdgcn_readfirstlane(blockIdx.x / per);
  const int64_t slot = slot_of(p.write_slots, b, p.slots);
  if (slot < 0) return;                            // padding
  const uint32_t row = (blockIdx.x - b * per) * (256 / L) + threadIdx.x / L, quad = threadIdx.x % L;
  const uint32_t e0 = row * len + 4 * quad;        // (below 2^31 + 2^15)
  const int left = row < rows ? int(row * len + len < elems ? row * len + len : elems) - int(e0) : 0;
  const int n = left < 0 ? 0 : left < 4 ? left : 4;
  const float* const src = state + int64_t(b) * elems;
  float h[4] = {0.f, 0.f, 0.f, 0.f};
  if (WORDS && n == 4) {
    const float4 v = *reinterpret_cast<const float4*>(src + e0);
    h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) h[j] = src[e0 + j];
  }
  const float amax = group_all<L>(fmaxf(fmaxf(fabsf(h[0]), fabsf(h[1])), fmaxf(fabsf(h[2]), fabsf(h[3]))), fmax2);
  const bool ok = finite(h[0]) && finite(h[1]) && finite(h[2]) && finite(h[3]);
  const RowScale r = row_scale(amax, row_bad<L>(!ok));
  const uint32_t key = SEEDED ? row_key(*p.seed, b * rows + row) : 0;
  const uint32_t w = pack_codes<SEEDED>(h, r, key, quad);
  store_codes<WORDS>(p.q + slot * elems + e0, n, w);
  if (quad == 0 && row < rows) p.scale[slot * rows + row] = r.scale;
}

// Reading: eight values a thread (VEC: row_len % 8 == 0 and everything aligned), else one.  64 states
// of 80 heads x 64 x 128 into bf16 (127 MB): 18.5 us, 6.9 TB/s (partly from the last-level cache).
// 1024 states of 2560 x 16: 22.2 us by eights, 80.8 one by one.
template <typename OUT, bool VEC>
__global__ __launch_bounds__(256) void cache_read_kernel(OUT* __restrict__ out, CacheParams p) {
  constexpr int W = VEC ? 8 : 1;
  const uint32_t elems = uint32_t(p.elems), per = (elems + 256 * W - 1) / (256 * W);   // workgroups a state
  const int64_t b = blockIdx.x / per, slot = slot_of(p.read_slots, b, p.slots);
  const uint32_t e = ((blockIdx.x % per) * 256u + threadIdx.x) * W;
  if (e >= elems) return;
  float v[W];
  if (slot < 0) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = 0.f;
  } else {
    const float scale = p.scale[slot * p.rows + e / uint32_t(p.row_len)];
    const int8_t* const q = p.q + slot * p.elems + e;
    if constexpr (VEC) {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = code_value(j < 4 ? w.x : w.y, j & 3) * scale;
    } else {
      v[0] = float(*q) * scale;
    }
  }
  OUT* const o = out + b * p.elems + e;
  if constexpr (!VEC) {
    if constexpr (sizeof(OUT) == 2) *o = bf16_rne(v[0]);
    else *o = v[0];
  } else if constexpr (sizeof(OUT) == 2) {
    uint4 w;
    w.x = pack_bf16(v[0], v[1]); w.y = pack_bf16(v[2], v[3]); w.z = pack_bf16(v[4], v[5]); w.w = pack_bf16(v[6], v[7]);
    *reinterpret_cast<uint4*>(o) = w;
  } else {
    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The 16 states of a lane behind one token, their part of the readout and their largest
// magnitude: h = keep q + a b, where `coeff(j, keep, a, b)` gives the factors.  A NaN or an
// infinity among the states shows in the readout (0 * inf is NaN); only then is it looked for.
struct LaneStates {
  float h[16], y, amax;
  bool bad;
};
template <typename F>
__device__ __forceinline__ void advance(const uint32_t (&w)[4], const float (&C)[16], LaneStates& s, F coeff) {
  float y = 0.f, amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float keep, a, b;
    coeff(j, keep, a, b);
    s.h[j] = fmaf(a, b, keep * code_value(w[j >> 2], j & 3));
    y = fmaf(C[j], s.h[j], y);
    amax = fmaxf(amax, fabsf(s.h[j]));
  }
  s.y = y;
  s.amax = amax;
  s.bad = false;
  if (__any(!finite(y))) {
    bool ok = true;
#pragma unroll
    for (int j = 0; j < 16; ++j) ok = ok && finite(s.h[j]);
    s.bad = !ok;
  }
}
// 1 / a to half an ulp (v_rcp_f32 and a Newton step); 0 for 0
__device__ __forceinline__ float reciprocal(float a) {
  const float r = __builtin_amdgcn_rcpf(a);
  return a == 0.f ? 0.f : fmaf(fmaf(-a, r, 1.f), r, r);
}

__device__ __forceinline__ float silu(float z) {
  return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// One token of the selective scan.  L lanes a channel, 16 states a lane; B and C of the batch row
// are staged in LDS.  WORDS: dstate % 4 == 0, codes on 4-byte and rates on 16-byte boundaries; LINES:
// dstate % 16 == 0, both on 16-byte boundaries (a lane whose states all lie behind the last works
// on its channel's first rates and zero codes, and stores nothing).  512 rows x 2560 x 16
// and x 64 in bf16, seeded: 22.8 and 69.6 us with LINES, 24.4 and 77.8 with WORDS; 1024 rows x
// 16 on other values: 44 with either, 143 value by value.
// Some 27 vector instructions a state (decay, input coefficient, readout, rounding; two of them at
// a quarter of the rate) stand against 2 bytes of codes: 512 rows (63 MB) take 23.6 us in bf16 and
// 22.8 in fp32, 16 of which the instructions fill and 11 the bytes; rounded to nearest 21.0 and
// 20.1.  A workgroup loads, waits and works once, so only others on the unit fill its wait:
// that is taken to be the rest.  Walking two batch rows with a channel's rates
// kept in registers measured the same, four slower (three wavefronts a SIMD).
template <typename IO, int L, bool WORDS, bool LINES, bool SEEDED>
__global__ __launch_bounds__(256) void step_cached_kernel(StepParams s, CacheParams p) {
  using T = io_traits<IO>;
  constexpr int kN = 16 * L;
  __shared__ float bc[2][kN];
  const int N = int(s.N), l = threadIdx.x % L;
  const uint32_t groups = uint32_t((p.rows * L + 255) / 256);       // workgroups a batch row
  const int64_t b = blockIdx.x / groups, d = int64_t(blockIdx.x % groups) * (256 / L) + threadIdx.x / L;
  const int64_t to = slot_of(p.write_slots, b, p.slots), from = slot_of(p.read_slots, b, p.slots);
  if (to < 0) return;                              // padding
  const bool live = d < p.rows;
  const int n0 = 16 * l;                           // this lane's first state
  // everything is asked for before anything is waited for (and converted when it is used)
  uint32_t w[4] = {0, 0, 0, 0};
  float scale = 0.f;
  IO u_raw = 0, dt_raw = 0, z_raw = 0;
  if (live) {
    u_raw = static_cast<const IO*>(s.u)[b * s.u_sb + d];
    dt_raw = static_cast<const IO*>(s.delta)[b * s.delta_sb + d];
    if (s.z) z_raw = static_cast<const IO*>(s.z)[b * s.z_sb + d];
  }
  if (live && from >= 0) {
    const int8_t* const q = p.q + (from * p.rows + d) * N + n0;
    scale = p.scale[from * p.rows + d];
    if constexpr (LINES) {
      if (n0 < N) {
        const uint4 t = *reinterpret_cast<const uint4*>(q);
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = load_codes<WORDS>(q + 4 * k, N - n0 - 4 * k);
    }
  }
  float A[16];
  if constexpr (LINES) {
    const float4* const q = reinterpret_cast<const float4*>(s.A + (live ? d * N + (n0 < N ? n0 : 0) : 0));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = q[k];
      A[4 * k] = v.x; A[4 * k + 1] = v.y; A[4 * k + 2] = v.z; A[4 * k + 3] = v.w;
    }
  } else if constexpr (WORDS) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live && n0 + 4 * k < N) v = *reinterpret_cast<const float4*>(s.A + d * N + n0 + 4 * k);
      A[4 * k] = v.x; A[4 * k + 1] = v.y; A[4 * k + 2] = v.z; A[4 * k + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) A[j] = live && n0 + j < N ? s.A[d * N + n0 + j] : 0.f;
  }
  const float skip = live && s.Dskip ? s.Dskip[d] : 0.f, bias = live && s.delta_bias ? s.delta_bias[d] : 0.f;
  const uint32_t key = SEEDED ? row_key(*p.seed, uint32_t(b * p.rows + d)) : 0;
  if (threadIdx.x < 2 * kN) {
    const int i = threadIdx.x / kN, n = threadIdx.x % kN;
    float v = 0.f;
    if (n < N) v = T::widen(i == 0 ? static_cast<const IO*>(s.B)[b * s.B_sb + n] : static_cast<const IO*>(s.C)[b * s.C_sb + n]);
    bc[i][n] = v;
  }
  __syncthreads();
  const float u = T::widen(u_raw), x = T::widen(dt_raw) + bias, dt = s.softplus ? softplus_f32(x) : x, du = dt * u;
  if constexpr (!LINES) {                          // no state: any rate that decays (a zero must stay one)
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (n0 + j >= N) A[j] = -copysignf(1.f, dt);
  }
  float C[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) C[j] = bc[1][n0 + j];
  LaneStates st;
  if (s.euler) {
    advance(w, C, st, [&](int j, float& keep, float& a, float& b) {
      keep = __builtin_amdgcn_exp2f(dt * A[j] * kLog2e) * scale;
      a = du;
      b = bc[0][n0 + j];
    });
  } else {
    // (e^x - 1) / A u, x = dt A, y = x log2 e.  From |y| = 1/12 down the series of dt u (e^x - 1) / x to
    // x^3 / 24, whose next term is 9e-8 of it; above it (2^y - 1) / A, where the difference and
    // v_rcp_f32 leave 1.3e-6.  (dt enters that through the exponential alone: an infinite step
    // gives -u / A, a product with dt would be 0 * inf.)
    constexpr float kLn2 = 0.693147181f;
    const float lt = dt * kLog2e, k1 = du * (kLn2 / 2.f), k2 = du * (kLn2 * kLn2 / 6.f), k3 = du * (kLn2 * kLn2 * kLn2 / 24.f);
    advance(w, C, st, [&](int j, float& keep, float& a, float& b) {
      const float y = lt * A[j], ab = __builtin_amdgcn_exp2f(y), ia = __builtin_amdgcn_rcpf(A[j]);
      const float ser = fmaf(y, fmaf(y, fmaf(y, k3, k2), k1), du);
      keep = ab * scale;
      a = fabsf(y) < 1.f / 12.f ? ser : fmaf(ab, ia, -ia) * u;
      b = bc[0][n0 + j];
    });
  }
  float y = group_all<L>(st.y, fadd2);
  const RowScale rs = row_scale(group_all<L>(st.amax, fmax2), row_bad<L>(st.bad));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float h4[4] = {st.h[4 * k], st.h[4 * k + 1], st.h[4 * k + 2], st.h[4 * k + 3]};
    w[k] = pack_codes<SEEDED>(h4, rs, key, uint32_t(4 * l + k));
  }
  if (!live) return;
  int8_t* const q = p.q + (to * p.rows + d) * N + n0;
  if constexpr (LINES) {
    if (n0 < N) *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) store_codes<WORDS>(q + 4 * k, N - n0 - 4 * k, w[k]);
  }
  if (l == 0) {
    p.scale[to * p.rows + d] = rs.scale;
    y = fmaf(skip, u, y);
    if (s.z) y *= silu(T::widen(z_raw));
    IO* const o = static_cast<IO*>(s.y) + b * s.y_sb + d;
    if constexpr (sizeof(IO) == 2) *o = bf16_rne(y);
    else *o = y;
  }
}

// A view of n bytes from p on; loads behind its end give zero and stores there are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t view(const void* p, int64_t n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, int(p != nullptr ? n : 0), 0x00020000);
}

// One token of the scalar-decay layer.  N / 16 lanes a row (head and channel), 16 states a
// lane; a workgroup walks `passes` groups of rows of one batch row, whose B and C stay in
// registers.  A group lies within one head.  All of a batch row is reached through views whose
// ends stand for its bounds, at offsets of which only a scalar part changes from group to group.
// LINES: the codes on 16-byte boundaries (128 rows: 42.0 us), else byte by byte (150).
// 64 rows x 80 heads x 64 x 128 (88 MB): 23.6 us, 17 of which the instructions fill (16 a state,
// the coefficient formed once a row) and 15 the bytes; to nearest 18.0, 64 states 14.3.  With
// 64-bit addresses and branches at the bounds it took 26.2.
template <int N, bool LINES, bool SEEDED>
__global__ __launch_bounds__(256) void ssd_step_cached_kernel(SsdParams s, CacheParams p, int passes) {
  using T = io_traits<uint16_t>;
  typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
  constexpr int L = N / 16, RP = 256 / L;
  static_assert(64 % RP == 0, "a group of rows lies within one head");
  const int l = threadIdx.x % L;
  const uint32_t groups = uint32_t((p.rows + RP * passes - 1) / (RP * passes));     // workgroups a batch row
  const uint32_t b = __builtin_amdgcn_readfirstlane(blockIdx.x / groups);
  const int64_t to = slot_of(p.write_slots, b, p.slots), from = slot_of(p.read_slots, b, p.slots);
  if (to < 0) return;                              // padding
  const uint32_t row0 = (blockIdx.x - b * groups) * uint32_t(passes) * RP;          // of the workgroup
  float B[16], C[16];
  {
    const uint4* const bp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(s.B) + int64_t(b) * N + 16 * l);
    const uint4* const cp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(s.C) + int64_t(b) * N + 16 * l);
    const uint4 b0 = bp[0], b1 = bp[1], c0 = cp[0], c1 = cp[1];
    const uint32_t bw[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
    const uint32_t cw[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      B[2 * j] = __uint_as_float(bw[j] << 16);
      B[2 * j + 1] = __uint_as_float(bw[j] & 0xffff0000u);
      C[2 * j] = __uint_as_float(cw[j] << 16);
      C[2 * j + 1] = __uint_as_float(cw[j] & 0xffff0000u);
    }
  }
  const int64_t seed = SEEDED ? *p.seed : 0;
  const auto xv = view(static_cast<const uint16_t*>(s.x) + b * p.rows, p.rows * 2);
  const auto zv = view(s.z ? static_cast<const uint16_t*>(s.z) + b * p.rows : nullptr, p.rows * 2);
  const auto dv = view(static_cast<const uint16_t*>(s.delta) + b * s.H, s.H * 2);
  const auto av = view(s.A, s.H * 4), kv = view(s.Dskip, p.rows * 4);
  const auto qv = view(from >= 0 ? p.q + from * p.elems : nullptr, p.elems);
  const auto sv = view(from >= 0 ? p.scale + from * p.rows : nullptr, p.rows * 4);
  const auto yv = view(static_cast<uint16_t*>(s.y) + b * p.rows, p.rows * 2);
  const auto qo = view(p.q + to * p.elems, p.elems), so = view(p.scale + to * p.rows, p.rows * 4);
  const uint32_t own = threadIdx.x / L, codes = own * N + 16 * l;                   // in a group
  const uint32_t first2 = l == 0 ? own * 2 : 0x80000000u, first4 = l == 0 ? own * 4 : 0x80000000u;
  struct Row {                                     // (as loaded: a conversion here would wait for it)
    u32x4_t w;
    uint32_t scale, a, skip;
    uint16_t x, z, dt;
  };
  auto load = [&](uint32_t row, Row& v) __attribute__((always_inline)) {
    v.x = __builtin_amdgcn_raw_buffer_load_b16(xv, own * 2, row * 2, 0);
    v.dt = __builtin_amdgcn_raw_buffer_load_b16(dv, 0, (row >> 6) * 2, 0);
    v.a = __builtin_amdgcn_raw_buffer_load_b32(av, 0, (row >> 6) * 4, 0);
    v.z = __builtin_amdgcn_raw_buffer_load_b16(zv, own * 2, row * 2, 0);
    v.skip = __builtin_amdgcn_raw_buffer_load_b32(kv, own * 4, row * 4, 0);
    v.scale = __builtin_amdgcn_raw_buffer_load_b32(sv, own * 4, row * 4, 0);
    if constexpr (LINES) {
      v.w = __builtin_amdgcn_raw_buffer_load_b128(qv, codes, row * N, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v.w[k] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v.w[k] |= uint32_t(__builtin_amdgcn_raw_buffer_load_b8(qv, codes + 4 * k + j, row * N, 0)) << (8 * j);
      }
    }
  };
  auto work = [&](uint32_t row, const Row& v) __attribute__((always_inline)) {
    const float x = T::widen(v.x), dt = T::widen(v.dt), A = __uint_as_float(v.a);
    const float ab = __builtin_amdgcn_exp2f(dt * A * kLog2e);
    const float drive = (s.euler ? dt : zoh_coeff_exact(dt, A, reciprocal(A), ab)) * x;
    const float keep = ab * __uint_as_float(v.scale);
    uint32_t w[4] = {v.w[0], v.w[1], v.w[2], v.w[3]};
    LaneStates st;
    advance(w, C, st, [&](int j, float& k, float& a, float& c) {
      k = keep;
      a = drive;
      c = B[j];
    });
    float y = group_all<L>(st.y, fadd2);
    const RowScale rs = row_scale(group_all<L>(st.amax, fmax2), row_bad<L>(st.bad));
    const uint32_t key = SEEDED ? row_key(seed, uint32_t(b * p.rows) + row + own) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float h4[4] = {st.h[4 * k], st.h[4 * k + 1], st.h[4 * k + 2], st.h[4 * k + 3]};
      w[k] = pack_codes<SEEDED>(h4, rs, key, uint32_t(4 * l + k));
    }
    if constexpr (LINES) {
      __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{w[0], w[1], w[2], w[3]}, qo, codes, row * N, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) __builtin_amdgcn_raw_buffer_store_b8(uint8_t(w[k / 4] >> (8 * (k % 4))), qo, codes + k, row * N, 0);
    }
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(rs.scale), so, first4, row * 4, 0);
    y = fmaf(__uint_as_float(v.skip), x, y);
    if (s.z) y *= silu(T::widen(v.z));
    __builtin_amdgcn_raw_buffer_store_b16(bf16_rne(y), yv, first2, row * 2, 0);
  };
  Row r0, r1;
  load(row0, r0);
  for (int t = 0;;) {                              // the next group's loads ahead of this one's work
    if (t + 1 < passes) load(row0 + (t + 1) * RP, r1);
    work(row0 + t * RP, r0);
    if (++t == passes) break;
    if (t + 1 < passes) load(row0 + (t + 1) * RP, r0);
    work(row0 + t * RP, r1);
    if (++t == passes) break;
  }
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int L, bool WORDS>
hipError_t launch_write_t(const float* state, const CacheParams& p, hipStream_t stream) {
  const dim3 grid(unsigned((p.rows + 256 / L - 1) / (256 / L) * p.count));
  if (p.seed) hipLaunchKernelGGL((cache_write_kernel<L, WORDS, true>), grid, dim3(256), 0, stream, state, p);
  else hipLaunchKernelGGL((cache_write_kernel<L, WORDS, false>), grid, dim3(256), 0, stream, state, p);
  return hipGetLastError();
}

template <typename IO, int L, bool WORDS, bool LINES>
hipError_t launch_step_t(const StepParams& s, const CacheParams& p, hipStream_t stream) {
  const dim3 grid(unsigned((p.rows * L + 255) / 256 * s.batch));
  if (p.seed) hipLaunchKernelGGL((step_cached_kernel<IO, L, WORDS, LINES, true>), grid, dim3(256), 0, stream, s, p);
  else hipLaunchKernelGGL((step_cached_kernel<IO, L, WORDS, LINES, false>), grid, dim3(256), 0, stream, s, p);
  return hipGetLastError();
}

template <typename IO, int L>
hipError_t launch_step_l(const StepParams& s, const CacheParams& p, hipStream_t stream) {
  const bool words = s.N % 4 == 0 && on(p.q, 4) && on(s.A, 16), lines = s.N % 16 == 0 && on(p.q, 16) && on(s.A, 16);
  if (lines) return launch_step_t<IO, L, true, true>(s, p, stream);
  if (words) return launch_step_t<IO, L, true, false>(s, p, stream);
  return launch_step_t<IO, L, false, false>(s, p, stream);
}

template <int N>
hipError_t launch_ssd_n(const SsdParams& s, const CacheParams& p, hipStream_t stream) {
  constexpr int RP = 256 / (N / 16);
  const int64_t groups = (p.rows + RP - 1) / RP;
  // A power of two that leaves at least 1024 workgroups, at most 4 (64 rows x 80 heads, with the
  // read-back: 48.6 us with 1, 45.6 with 2, 45.0 with 4, 47.3 with 8).
  int passes = 1;
  while (passes < 4 && groups * p.count >= 2048 * int64_t(passes)) passes *= 2;
  const dim3 grid(unsigned((p.rows + RP * passes - 1) / (RP * passes) * p.count));
  const bool lines = on(p.q, 16);
  if (lines) {
    if (p.seed) hipLaunchKernelGGL((ssd_step_cached_kernel<N, true, true>), grid, dim3(256), 0, stream, s, p, passes);
    else hipLaunchKernelGGL((ssd_step_cached_kernel<N, true, false>), grid, dim3(256), 0, stream, s, p, passes);
  } else {
    if (p.seed) hipLaunchKernelGGL((ssd_step_cached_kernel<N, false, true>), grid, dim3(256), 0, stream, s, p, passes);
    else hipLaunchKernelGGL((ssd_step_cached_kernel<N, false, false>), grid, dim3(256), 0, stream, s, p, passes);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const float* state, const CacheParams& p, hipStream_t stream) {
  const bool words = p.row_len % 4 == 0 && p.elems % 4 == 0 && on(p.q, 4) && on(state, 16);
  auto with = [&](auto w) {
    constexpr bool W = decltype(w)::value;
    if (p.row_len <= 4) return launch_write_t<1, W>(state, p, stream);
    if (p.row_len <= 8) return launch_write_t<2, W>(state, p, stream);
    if (p.row_len <= 16) return launch_write_t<4, W>(state, p, stream);
    if (p.row_len <= 32) return launch_write_t<8, W>(state, p, stream);
    if (p.row_len <= 64) return launch_write_t<16, W>(state, p, stream);
    return launch_write_t<32, W>(state, p, stream);
  };
  return words ? with(std::true_type{}) : with(std::false_type{});
}

hipError_t launch_cache_read(bool bf16, void* out, const CacheParams& p, hipStream_t stream) {
  const bool vec = p.row_len % 8 == 0 && p.elems % 8 == 0 && on(p.q, 8) && on(out, 16);
  const int64_t per = vec ? 2048 : 256;
  const dim3 grid(unsigned((p.elems + per - 1) / per * p.count));
  auto with = [&](auto io, auto v) {
    using OUT = decltype(io);
    hipLaunchKernelGGL((cache_read_kernel<OUT, decltype(v)::value>), grid, dim3(256), 0, stream, static_cast<OUT*>(out), p);
    return hipGetLastError();
  };
  if (bf16) return vec ? with(uint16_t{}, std::true_type{}) : with(uint16_t{}, std::false_type{});
  return vec ? with(float{}, std::true_type{}) : with(float{}, std::false_type{});
}

hipError_t launch_step_cached(bool bf16, const StepParams& s, const CacheParams& p, hipStream_t stream) {
  auto with = [&](auto io) {
    using IO = decltype(io);
    if (s.N <= 16) return launch_step_l<IO, 1>(s, p, stream);
    if (s.N <= 32) return launch_step_l<IO, 2>(s, p, stream);
    return launch_step_l<IO, 4>(s, p, stream);
  };
  return bf16 ? with(uint16_t{}) : with(float{});
}

hipError_t launch_ssd_step_cached(const SsdParams& s, const CacheParams& p, hipStream_t stream) {
  return s.N == 64 ? launch_ssd_n<64>(s, p, stream) : launch_ssd_n<128>(s, p, stream);
}

}  // namespace selscan
