// cache_kernels.hip -- the 8-bit state cache: writing, reading, and the decode steps of the
// selective scan and of the scalar-decay layer on cached states.
#include "device_common.h"
#include "scan_launch.h"

namespace selscan {
namespace {

constexpr float kTinyRow = 0x1p-100f;     // rows whose largest magnitude is below are zero
constexpr float kCodes = 127.f;

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
__device__ __forceinline__ float rounding_offset(bool seeded, uint32_t key, uint32_t j) {
  if (!seeded) return 0.5f;
  const uint32_t w = pair_bits(key, j >> 1);
  return (float((j & 1) ? w >> 16 : w & 0xffffu) + 0.5f) * 0x1p-16f;
}

struct RowScale {
  float scale, inv;
};
// NaN or infinity anywhere in the row (bad): a NaN scale and zero codes
__device__ __forceinline__ RowScale row_scale(float amax, bool bad) {
  if (bad) return {__builtin_nanf(""), 0.f};
  if (!(amax >= kTinyRow)) return {0.f, 0.f};
  return {amax / kCodes, kCodes / amax};
}
__device__ __forceinline__ int8_t code(float h, float inv, float off, bool bad) {
  if (bad) return 0;
  return int8_t(fminf(fmaxf(floorf(fmaf(h, inv, off)), -kCodes), kCodes));
}
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// the slot that batch row b names, or -1
__device__ __forceinline__ int64_t slot_of(const int32_t* ids, int64_t b, int64_t slots) {
  const int64_t s = ids ? int64_t(ids[b]) : b;
  return s >= 0 && s < slots ? s : -1;
}

// One thread per row.
__global__ __launch_bounds__(64) void cache_write_kernel(const float* state, CacheParams p) {
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= p.count * p.rows) return;
  const int64_t b = i / p.rows, row = i % p.rows, slot = slot_of(p.write_slots, b, p.slots);
  if (slot < 0) return;
  const int64_t e0 = row * p.row_len, n = e0 + p.row_len < p.elems ? p.row_len : p.elems - e0;
  const float* h = state + b * p.elems + e0;
  float amax = 0.f;
  bool bad = false;
  for (int64_t j = 0; j < n; ++j) {
    amax = fmaxf(amax, fabsf(h[j]));
    bad |= !finite(h[j]);
  }
  const RowScale s = row_scale(amax, bad);
  const uint32_t key = p.seed ? row_key(*p.seed, uint32_t(i)) : 0;
  int8_t* q = p.q + slot * p.elems + e0;
  for (int64_t j = 0; j < n; ++j) q[j] = code(h[j], s.inv, rounding_offset(p.seed != nullptr, key, uint32_t(j)), bad);
  p.scale[slot * p.rows + row] = s.scale;
}

template <typename OUT>
__global__ __launch_bounds__(64) void cache_read_kernel(OUT* out, CacheParams p) {
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= p.count * p.rows) return;
  const int64_t b = i / p.rows, row = i % p.rows, slot = slot_of(p.read_slots, b, p.slots);
  const int64_t e0 = row * p.row_len, n = e0 + p.row_len < p.elems ? p.row_len : p.elems - e0;
  const float scale = slot < 0 ? 0.f : p.scale[slot * p.rows + row];
  for (int64_t j = 0; j < n; ++j) {
    const float v = slot < 0 ? 0.f : float(p.q[slot * p.elems + e0 + j]) * scale;
    if constexpr (sizeof(OUT) == 2) out[b * p.elems + e0 + j] = bf16_rne(v);
    else out[b * p.elems + e0 + j] = v;
  }
}

// One thread per channel: a first walk over its states for the readout and the largest
// magnitude, a second one for the codes.
template <typename IO>
__global__ __launch_bounds__(64) void step_cached_kernel(StepParams s, CacheParams p) {
  using T = io_traits<IO>;
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= p.count * p.rows) return;
  const int64_t b = i / p.rows, d = i % p.rows;
  const int64_t from = slot_of(p.read_slots, b, p.slots), to = slot_of(p.write_slots, b, p.slots);
  if (to < 0) return;
  const float u = T::widen(static_cast<const IO*>(s.u)[b * s.u_sb + d]);
  const float dt = step_size(T::widen(static_cast<const IO*>(s.delta)[b * s.delta_sb + d]),
                             s.delta_bias ? s.delta_bias[d] : 0.f, s.softplus != 0);
  const float scale = from < 0 ? 0.f : p.scale[from * p.rows + d];
  const IO* const B = static_cast<const IO*>(s.B) + b * s.B_sb;
  const IO* const C = static_cast<const IO*>(s.C) + b * s.C_sb;
  auto state = [&](int64_t j) {
    const float a = s.A[d * s.N + j], ab = __builtin_amdgcn_exp2f(dt * a * kLog2e);
    const float coeff = (s.euler || a == 0.f) ? dt : zoh_coeff_exact(dt, a, 1.f / a, ab);
    const float h = from < 0 ? 0.f : float(p.q[(from * p.rows + d) * s.N + j]) * scale;
    return fmaf(ab, h, coeff * (T::widen(B[j]) * u));
  };
  float y = s.Dskip ? s.Dskip[d] * u : 0.f, amax = 0.f;
  bool bad = false;
  for (int64_t j = 0; j < s.N; ++j) {
    const float h = state(j);
    y = fmaf(T::widen(C[j]), h, y);
    amax = fmaxf(amax, fabsf(h));
    bad |= !finite(h);
  }
  const RowScale rs = row_scale(amax, bad);
  const uint32_t key = p.seed ? row_key(*p.seed, uint32_t(i)) : 0;
  for (int64_t j = 0; j < s.N; ++j)
    p.q[(to * p.rows + d) * s.N + j] = code(state(j), rs.inv, rounding_offset(p.seed != nullptr, key, uint32_t(j)), bad);
  p.scale[to * p.rows + d] = rs.scale;
  if (s.z) {
    const float z = T::widen(static_cast<const IO*>(s.z)[b * s.z_sb + d]);
    y *= z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
  }
  IO* const yo = static_cast<IO*>(s.y) + b * s.y_sb + d;
  if constexpr (sizeof(IO) == 2) *yo = bf16_rne(y);
  else *yo = y;
}

// One thread per (head, channel) row of N states.
__global__ __launch_bounds__(64) void ssd_step_cached_kernel(SsdParams s, CacheParams p) {
  using T = io_traits<uint16_t>;
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= p.count * p.rows) return;
  const int64_t b = i / p.rows, row = i % p.rows, head = row / 64;
  const int64_t from = slot_of(p.read_slots, b, p.slots), to = slot_of(p.write_slots, b, p.slots);
  if (to < 0) return;
  const float x = T::widen(static_cast<const uint16_t*>(s.x)[i]);
  const float dt = T::widen(static_cast<const uint16_t*>(s.delta)[b * s.H + head]), a = s.A[head];
  const float ab = __builtin_amdgcn_exp2f(dt * a * kLog2e);
  const float drive = ((s.euler || a == 0.f) ? dt : zoh_coeff_exact(dt, a, 1.f / a, ab)) * x;
  const float scale = from < 0 ? 0.f : p.scale[from * p.rows + row];
  const uint16_t* const B = static_cast<const uint16_t*>(s.B) + b * s.N;
  const uint16_t* const C = static_cast<const uint16_t*>(s.C) + b * s.N;
  auto state = [&](int64_t j) {
    const float h = from < 0 ? 0.f : float(p.q[(from * p.rows + row) * s.N + j]) * scale;
    return fmaf(ab, h, drive * T::widen(B[j]));
  };
  float y = s.Dskip ? s.Dskip[row] * x : 0.f, amax = 0.f;
  bool bad = false;
  for (int64_t j = 0; j < s.N; ++j) {
    const float h = state(j);
    y = fmaf(T::widen(C[j]), h, y);
    amax = fmaxf(amax, fabsf(h));
    bad |= !finite(h);
  }
  const RowScale rs = row_scale(amax, bad);
  const uint32_t key = p.seed ? row_key(*p.seed, uint32_t(i)) : 0;
  for (int64_t j = 0; j < s.N; ++j)
    p.q[(to * p.rows + row) * s.N + j] =
        code(state(j), rs.inv, rounding_offset(p.seed != nullptr, key, uint32_t(j)), bad);
  p.scale[to * p.rows + row] = rs.scale;
  if (s.z) {
    const float z = T::widen(static_cast<const uint16_t*>(s.z)[i]);
    y *= z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
  }
  static_cast<uint16_t*>(s.y)[i] = bf16_rne(y);
}

unsigned row_blocks(const CacheParams& p, int per) { return unsigned((p.count * p.rows + per - 1) / per); }

}  // namespace

hipError_t launch_cache_write(const float* state, const CacheParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(cache_write_kernel, dim3(row_blocks(p, 64)), dim3(64), 0, stream, state, p);
  return hipGetLastError();
}

hipError_t launch_cache_read(bool bf16, void* out, const CacheParams& p, hipStream_t stream) {
  const dim3 grid(row_blocks(p, 64));
  if (bf16) hipLaunchKernelGGL(cache_read_kernel<uint16_t>, grid, dim3(64), 0, stream, static_cast<uint16_t*>(out), p);
  else hipLaunchKernelGGL(cache_read_kernel<float>, grid, dim3(64), 0, stream, static_cast<float*>(out), p);
  return hipGetLastError();
}

hipError_t launch_step_cached(bool bf16, const StepParams& s, const CacheParams& p, hipStream_t stream) {
  const dim3 grid(row_blocks(p, 64));
  if (bf16) hipLaunchKernelGGL(step_cached_kernel<uint16_t>, grid, dim3(64), 0, stream, s, p);
  else hipLaunchKernelGGL(step_cached_kernel<float>, grid, dim3(64), 0, stream, s, p);
  return hipGetLastError();
}

hipError_t launch_ssd_step_cached(const SsdParams& s, const CacheParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(ssd_step_cached_kernel, dim3(row_blocks(p, 64)), dim3(64), 0, stream, s, p);
  return hipGetLastError();
}

}  // namespace selscan
