// norm_kernels.hip -- group norm with an activation, token by token, channels last.
//
//     xh = (x - mean) / sqrt(var + eps) over the channels of a token's group,  n = xh w + b,
//     y = act(n), or with a gate y = n act(z);   act(t) = t sigmoid(t), or t
// Backward, dn = dy act'(n) (gate: dy act(z), dz = dy n act'(z)), u = dn w, r = 1 / sqrt(var + eps):
//     dx = r (u - mean(u) - xh mean(u xh)),  dw = sum dn xh,  db = sum dn
//
// A group lies in the registers of up to 64 lanes, or of four wavefronts, 16 bytes of each operand a lane and
// piece, so that a row is read once: the mean, then the squares of what is off it (not E x^2 - mean^2, which cancels),
// both in fp32.  Results are rounded once.  Memory bounds the forward (16384 x 32 x 128 bf16, gate: 80 us, 5.0
// TB/s; a large copy 5.2); the backward (16384 x 40 x 64: 110 us for 420 MB, 3.8 TB/s) also waits for its
// two sums in a row, one after the other, with three to seven wavefronts a SIMD.
#include <hip/hip_runtime.h>

#include <cmath>

#include "device_common.h"
#include "scan_launch.h"

namespace selscan {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// VEC consecutive elements as they lie in memory: 16 bytes (EVEN: on a boundary of 16, else on any element's), or one
// element.
template <typename T, int VEC, bool EVEN> struct NormRaw {
  using type = u32x4;
  static __device__ __forceinline__ type load(const T* p) {
    if constexpr (EVEN) return *reinterpret_cast<const u32x4*>(p);
    u32x4 r;
    __builtin_memcpy(&r, p, 16);
    return r;
  }
  static __device__ __forceinline__ void widen(type r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(r[i]);
      }
    }
  }
};
template <typename T, bool EVEN> struct NormRaw<T, 1, EVEN> {
  using type = T;
  static __device__ __forceinline__ type load(const T* p) { return *p; }
  static __device__ __forceinline__ void widen(type r, float* v) { v[0] = io_traits<T>::widen(r); }
};
template <int VEC, bool EVEN> __device__ __forceinline__ void norm_load_f32(const float* p, float* v) {
  constexpr int N = VEC < 4 ? 1 : 4;
#pragma unroll
  for (int i = 0; i < VEC; i += N) NormRaw<float, N, EVEN>::widen(NormRaw<float, N, EVEN>::load(p + i), v + i);
}
template <typename T, int VEC, bool EVEN> __device__ __forceinline__ void norm_store(T* p, const float* v) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(T) == 2) *p = bf16_rne(v[0]); else *p = v[0];
  } else if constexpr (sizeof(T) == 2) {
    typedef __attribute__((ext_vector_type(VEC))) __bf16 b;
    typedef __attribute__((ext_vector_type(VEC))) float f;
    f x;
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = v[i];
    const b r = __builtin_convertvector(x, b);
    if constexpr (EVEN) *reinterpret_cast<b*>(p) = r; else __builtin_memcpy(p, &r, 16);
  } else {
    typedef __attribute__((ext_vector_type(4))) float f;
    const f r = {v[0], v[1], v[2], v[3]};
    if constexpr (EVEN) *reinterpret_cast<f*>(p) = r; else __builtin_memcpy(p, &r, 16);
  }
}

// Where a thread's i-th piece of a group begins.  Of a width that is no multiple of VEC the last piece ends where the
// group does: its first `had` values are the piece before's too, which counts them (both form and store the same bits).
template <int VEC, bool EVEN> struct NormPlace {
  int c, had;
  bool in;
  __device__ __forceinline__ NormPlace(int i, int lanes, int lane, int width) {
    const int at = (i * lanes + lane) * VEC;
    in = at < width;
    c = EVEN || at + VEC <= width ? at : width - VEC;
    had = at - c;
  }
  __device__ __forceinline__ bool counts(int e) const { return EVEN || e >= had; }
};

// What a thread has of a group of channels of one row, on its way: all that a row needs is asked for before
// anything of it is waited for.
template <typename T, int VEC, int EPT, bool EVEN> struct NormPiece {
  using Raw = NormRaw<T, VEC, EVEN>;
  typename Raw::type raw[EPT];
  __device__ __forceinline__ void load(const T* src, int lanes, int lane, int width) {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const NormPlace<VEC, EVEN> at(i, lanes, lane, width);
      raw[i] = typename Raw::type{};
      if (at.in) raw[i] = Raw::load(src + at.c);
    }
  }
  __device__ __forceinline__ void widen(int i, float* v) const { Raw::widen(raw[i], v); }
  // everything has come
  __device__ __forceinline__ void wait() {
#pragma unroll
    for (int i = 0; i < EPT; ++i) asm volatile("" : "+v"(raw[i]));
  }
};

template <int CTRL> __device__ __forceinline__ float norm_dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, false));
}

// The sum over the `lanes` threads of a group, in every one of them and with the same bits.  Up to 16 lanes exchange in
// the vector unit (by pairs, twos, fours, and mirrored halves of 8 and 16: what the halves hold is uniform by then); an
// exchange through the LDS, as the wider ones are, takes some 100 cycles (backward, 16384 x 32 x 128 with a gate:
// 187 us with all of them there, 169 so).
__device__ __forceinline__ float norm_sum(float v, int lanes, float* tmp) {
  if (lanes > 1) v += norm_dpp<0xb1>(v);          // quad_perm 1 0 3 2
  if (lanes > 2) v += norm_dpp<0x4e>(v);          // quad_perm 2 3 0 1
  if (lanes > 4) v += norm_dpp<0x141>(v);         // row_half_mirror
  if (lanes > 8) v += norm_dpp<0x140>(v);         // row_mirror
  if (lanes > 16) v += __shfl_xor(v, 16);
  if (lanes > 32) v += __shfl_xor(v, 32);
  if (lanes > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
  }
  return v;
}

// act(t) and act'(t).  The exponent -t log2 e is off by 2^-24 of itself when it is rounded, and the sigmoid by |t| times as
// much; the reciprocal instruction by 2^-23.  Results in bf16 keep nothing of that; in fp32 the exponent's rest (and
// that of log2 e) and a step of Newton's put it right.
template <typename T> __device__ __forceinline__ float norm_act(float t, bool silu, float& slope) {
  if (!silu) { slope = 1.f; return t; }
  if constexpr (sizeof(T) == 2) {
    const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-t * kLog2e));
    slope = fmaf(t * s, 1.f - s, s);
    return t * s;
  }
  constexpr float kLow = 1.92596302e-8f;          // log2 e less its fp32 value
  const float x = fminf(-t * kLog2e, 127.9f);     // (beyond it the sigmoid is zero, and 1 + e^-t a number)
  const float rest = x < 127.9f && x > -200.f ? fmaf(-t, kLog2e, -x) - t * kLow : 0.f;
  const float e0 = __builtin_amdgcn_exp2f(x), e = fmaf(e0, rest * 0.693147181f, e0), d = 1.f + e;
  const float r = __builtin_amdgcn_rcpf(d), s = x < 127.9f ? fmaf(fmaf(-d, r, 1.f), r, r) : 0.f;
  slope = fmaf(t * s, e * s, s);                  // (1 - s is e s)
  return t * s;
}

template <typename T, int VEC, int EPT, bool EVEN>
struct NormRow {
  float x[EPT * VEC];      // (x - mean) / sqrt(var + eps)
  float r;
  __device__ __forceinline__ void form(const NormPiece<T, VEC, EPT, EVEN>& raw, int lanes, int lane, int width, float eps, float* tmp) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const NormPlace<VEC, EVEN> at(i, lanes, lane, width);
      raw.widen(i, x + i * VEC);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += at.counts(e) ? x[i * VEC + e] : 0.f;
    }
    const float inv = 1.f / float(width);
    const float mean = norm_sum(s, lanes, tmp) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const NormPlace<VEC, EVEN> at(i, lanes, lane, width);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[i * VEC + e] = at.in ? x[i * VEC + e] - mean : 0.f;
        q = at.counts(e) ? fmaf(x[i * VEC + e], x[i * VEC + e], q) : q;
      }
    }
    r = 1.f / sqrtf(fmaf(norm_sum(q, lanes, tmp), inv, eps));
#pragma unroll
    for (int i = 0; i < EPT * VEC; ++i) x[i] *= r;
  }
};

// A row's place: token l of batch row b.
struct NormToken {
  int64_t b, l;
  __device__ __forceinline__ NormToken(const NormParams& p, uint32_t row) {
    const uint32_t L = uint32_t(p.L), n = p.L == p.rows ? 0 : row / L;
    b = n;
    l = row - n * L;
  }
};

template <typename T, int VEC, int EPT, bool EVEN>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormParams p) {
  __shared__ float tmp[4];
  const int lanes = 1 << p.log_lanes, lane = threadIdx.x & (lanes - 1);
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x, groups = uint32_t(p.groups);
  const uint32_t gi = block * (256u >> p.log_lanes) + (threadIdx.x >> p.log_lanes);
  if (gi >= uint32_t(p.rows) * groups) return;
  // (32 bits hold rows and groups; divisions of 64 take as many instructions as the row's arithmetic: 91 us in the place
  // of 82, 16384 rows of 32 x 128 with a gate)
  const uint32_t row = gi / groups;
  const NormToken at_row(p, row);
  const int64_t b = at_row.b, l = at_row.l;
  const int64_t c0 = int64_t(gi - row * groups) * p.width;
  const bool gate = p.z != nullptr;
  NormPiece<T, VEC, EPT, EVEN> x, z;
  x.load(static_cast<const T*>(p.x) + b * p.x_sb + l * p.x_sl + c0, lanes, lane, p.width);
  if (gate) z.load(static_cast<const T*>(p.z) + b * p.z_sb + l * p.z_sl + c0, lanes, lane, p.width);
  T* y = static_cast<T*>(p.y) + b * p.y_sb + l * p.y_sl + c0;
  // (y may lie where z does, and another wavefront's piece may begin within this one's: z is there before the barriers)
  if (!EVEN && gate && lanes > 64) z.wait();
  NormRow<T, VEC, EPT, EVEN> n;
  n.form(x, lanes, lane, p.width, p.eps, tmp);
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const NormPlace<VEC, EVEN> at(i, lanes, lane, p.width);
    const int c = at.c;
    if (!at.in) break;
    float w[VEC], o[VEC], t[VEC];
    if (p.weight) norm_load_f32<VEC, EVEN>(p.weight + c0 + c, w);
    if (p.bias) norm_load_f32<VEC, EVEN>(p.bias + c0 + c, o);
    if (gate) z.widen(i, t);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float v = fmaf(n.x[i * VEC + e], p.weight ? w[e] : 1.f, p.bias ? o[e] : 0.f);
      float slope;
      o[e] = gate ? v * norm_act<T>(t[e], p.silu, slope) : norm_act<T>(v, p.silu, slope);
    }
    norm_store<T, VEC, EVEN>(y + c, o);
  }
}

// A workgroup keeps to `256 / lanes` groups of channels (of several rows at once where there are fewer groups)
// and walks every `splits`-th row, so that the sums for weight and bias stay in registers.  (The next row
// asked for ahead takes registers that more wavefronts make better use of: 16384 x 32 x 128 fp32 271 us, 262 without.)
template <typename T, int VEC, int EPT, bool EVEN>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormParams p) {
  __shared__ float tmp[4];
  const int lanes = 1 << p.log_lanes, lane = threadIdx.x & (lanes - 1), slot = threadIdx.x >> p.log_lanes;
  const int gslot = slot & int(p.gper - 1), rslot = slot / int(p.gper), rows_at_once = (256 >> p.log_lanes) / int(p.gper);
  const int64_t split = blockIdx.x / uint32_t(p.cblocks), cb = blockIdx.x - uint32_t(split) * uint32_t(p.cblocks);
  const int64_t group = cb * p.gper + gslot;
  if (group >= p.groups) return;                  // (a group's threads all leave, or none)
  const int64_t c0 = group * p.width;
  const int64_t part = split * rows_at_once + rslot, step = p.splits * rows_at_once;
  const bool gate = p.z != nullptr;
  float w[EPT * VEC], o[EPT * VEC], dw[EPT * VEC], db[EPT * VEC];
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const NormPlace<VEC, EVEN> at(i, lanes, lane, p.width);
#pragma unroll
    for (int e = 0; e < VEC; ++e) { w[i * VEC + e] = 1.f; o[i * VEC + e] = dw[i * VEC + e] = db[i * VEC + e] = 0.f; }
    if (at.in) {
      if (p.weight) norm_load_f32<VEC, EVEN>(p.weight + c0 + at.c, w + i * VEC);
      if (p.bias) norm_load_f32<VEC, EVEN>(p.bias + c0 + at.c, o + i * VEC);
    }
  }
  const float inv = 1.f / float(p.width);
  NormPiece<T, VEC, EPT, EVEN> x, z, dy;
  auto ask = [&](int64_t row) {
    const NormToken at_row(p, uint32_t(row));
    const int64_t b = at_row.b, l = at_row.l;
    x.load(static_cast<const T*>(p.x) + b * p.x_sb + l * p.x_sl + c0, lanes, lane, p.width);
    if (gate) z.load(static_cast<const T*>(p.z) + b * p.z_sb + l * p.z_sl + c0, lanes, lane, p.width);
    dy.load(static_cast<const T*>(p.dy) + b * p.y_sb + l * p.y_sl + c0, lanes, lane, p.width);
  };
  for (int64_t row = part; row < p.rows; row += step) {
    ask(row);
    const int64_t out = row * p.groups * p.width + c0;
    NormRow<T, VEC, EPT, EVEN> n;
    n.form(x, lanes, lane, p.width, p.eps, tmp);
    float u[EPT * VEC], m1 = 0.f, m2 = 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const NormPlace<VEC, EVEN> at(i, lanes, lane, p.width);
      float d[VEC], t[VEC], dz[VEC];
      dy.widen(i, d);                         // (zero behind the group's end: nothing comes of it there)
      if (gate) z.widen(i, t);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int k = i * VEC + e;
        const float v = fmaf(n.x[k], w[k], o[k]);
        float slope, dn;
        if (gate) {
          dn = d[e] * norm_act<T>(t[e], p.silu, slope);
          dz[e] = d[e] * v * slope;
        } else {
          norm_act<T>(v, p.silu, slope);
          dn = d[e] * slope;
        }
        u[k] = dn * w[k];
        dw[k] = fmaf(dn, n.x[k], dw[k]);
        db[k] += dn;
        m1 += at.counts(e) ? u[k] : 0.f;
        m2 = at.counts(e) ? fmaf(u[k], n.x[k], m2) : m2;
      }
      if (gate && at.in) norm_store<T, VEC, EVEN>(static_cast<T*>(p.dz) + out + at.c, dz);
    }
    m1 = norm_sum(m1, lanes, tmp) * inv;
    m2 = norm_sum(m2, lanes, tmp) * inv;
    // two channels: what is left of u - mean(u) beside xh is eps / (var + eps) of it
    const float two = p.width == 2 ? n.r * n.r * p.eps : 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const NormPlace<VEC, EVEN> at(i, lanes, lane, p.width);
      float d[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float a = u[i * VEC + e] - m1;
        d[e] = n.r * (p.width == 2 ? a * two : fmaf(-n.x[i * VEC + e], m2, a));
      }
      if (at.in) norm_store<T, VEC, EVEN>(static_cast<T*>(p.dx) + out + at.c, d);
    }
  }
  if (!p.part) return;
  // the rows that a wavefront takes at once, into its first threads
  for (int d = lanes * p.gper; d < 64; d *= 2) {
#pragma unroll
    for (int k = 0; k < EPT * VEC; ++k) {
      dw[k] += __shfl_xor(dw[k], d);
      db[k] += __shfl_xor(db[k], d);
    }
  }
  const int span = lanes * p.gper < 64 ? 64 : lanes * p.gper;      // threads of one part
  if (int(threadIdx.x) % span >= lanes * p.gper) return;
  const int64_t C = p.groups * p.width;
  float* const own = p.part + 2 * C * (split * (256 / span) + threadIdx.x / span);
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const NormPlace<VEC, EVEN> at(i, lanes, lane, p.width);
    if (!at.in) break;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (!at.counts(e)) continue;
      own[c0 + at.c + e] = dw[i * VEC + e];
      own[C + c0 + at.c + e] = db[i * VEC + e];
    }
  }
}

// dweight and dbias: 8 columns a workgroup, every 32nd part a row of threads; eight parts asked for at once.  The parts, sums of
// some tens of rows in fp32 (in the registers that a row leaves), are added up in 64 bits.
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* part, int64_t parts, int64_t C, float* dw, float* db) {
  __shared__ double s[2][32][9];
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t c = int64_t(blockIdx.x) * 8 + x;
  double a = 0.0, b = 0.0;
  if (c < C) {
    for (int64_t i = y; i < parts; i += 256) {
      float u[8], v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t j = i + 32 * k < parts ? i + 32 * k : i;
        u[k] = part[2 * j * C + c];
        v[k] = part[(2 * j + 1) * C + c];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        a += i + 32 * k < parts ? double(u[k]) : 0.0;
        b += i + 32 * k < parts ? double(v[k]) : 0.0;
      }
    }
  }
  s[0][y][x] = a;
  s[1][y][x] = b;
  __syncthreads();
  if (y < 2 && c < C) {
    double t = 0.0;
    for (int i = 0; i < 32; ++i) t += s[y][i][x];
    float* const out = y == 0 ? dw : db;
    if (out) out[c] = float(t);
  }
}

template <typename T, int VEC, int EPT, bool EVEN>
hipError_t norm_launch(bool bwd, const NormParams& p, hipStream_t stream) {
  if (bwd) {
    norm_bwd_kernel<T, VEC, EPT, EVEN><<<dim3(uint32_t(p.cblocks * p.splits)), dim3(256), 0, stream>>>(p);
  } else {
    const int64_t per = 256 >> p.log_lanes;
    const int64_t blocks = (p.rows * p.groups + per - 1) / per, kSide = 1 << 20;     // (2^32 threads a side at most)
    const dim3 grid(uint32_t(blocks < kSide ? blocks : kSide), uint32_t((blocks + kSide - 1) / kSide));
    norm_fwd_kernel<T, VEC, EPT, EVEN><<<grid, dim3(256), 0, stream>>>(p);
  }
  return hipGetLastError();
}

template <typename T, bool EVEN>
hipError_t norm_pieces(bool bwd, const NormParams& p, hipStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  switch (p.ept) {
    case 1: return norm_launch<T, VEC, 1, EVEN>(bwd, p, stream);
    case 2: return norm_launch<T, VEC, 2, EVEN>(bwd, p, stream);
  }
  if (VEC == 8 || p.ept <= 4) return norm_launch<T, VEC, 4, EVEN>(bwd, p, stream);
  return norm_launch<T, VEC, VEC == 8 ? 4 : 8, EVEN>(bwd, p, stream);
}

template <typename T>
hipError_t norm_dispatch(bool bwd, const NormParams& p, hipStream_t stream) {
  if (p.width < 16 / int(sizeof(T))) return norm_launch<T, 1, 1, false>(bwd, p, stream);
  // (The masks of a last piece cost 16384 x 32 x 128 bf16 92 -> 97 us forward, x 40 x 64 117 -> 129 backward.)
  return p.even ? norm_pieces<T, true>(bwd, p, stream) : norm_pieces<T, false>(bwd, p, stream);
}

}  // namespace

NormPlan norm_plan(bool bf16, bool bwd, int64_t rows, int64_t groups, int64_t width) {
  NormPlan pl{};
  const int64_t vec = bf16 ? 8 : 4, per = width < vec ? 1 : vec, pieces = (width + per - 1) / per;
  while (pl.log_lanes < 6 && 1 << pl.log_lanes < pieces) ++pl.log_lanes;
  // Four wavefronts for a group that would be more than four pieces a lane of one; in the backward, which holds six
  // values for each of the forward's two, more than two (16384 x 2 x 2048 bf16, a gate: forward 81 us with one
  // wavefront a group, 85 with four, backward 223 and 157; 8192 x 2 x 2048 fp32 81 and 73, 201 and 148; 16384 x 4 x 1024
  // bf16 77 and 112, 167 and 225).
  if (pieces > (bwd ? 128 : 256)) pl.log_lanes = 8;
  const int64_t lanes = 1 << pl.log_lanes, slots = 256 / lanes;
  pl.ept = int32_t((pieces + lanes - 1) / lanes);
  pl.gper = 1;
  while (pl.gper < slots && pl.gper < groups) pl.gper *= 2;
  pl.cblocks = (groups + pl.gper - 1) / pl.gper;
  // The backward's workgroups: four a compute unit.  Fewer where the rows are few: a workgroup takes 2.1 us for each
  // of its rows, one after the other, and its part of the sums costs 12 us for every million of its channels, to
  // write and to add up, so the rows of one are about sqrt(rows * channels / 2^18) (512 rows of 4096
  // channels: one row a workgroup 34.9 us, 3 24.2, 8 28.3; 2048 rows 38.2, 6 35.7; 64 rows 12.2, 3 14.5).
  const int64_t at_once = slots / pl.gper, each = at_once * int64_t(std::ceil(std::sqrt(double(rows * groups * width) / 262144.0)));
  const int64_t most = each > 0 ? (rows + each - 1) / each : 1;
  pl.splits = (1024 + pl.cblocks - 1) / pl.cblocks;
  if (pl.splits > most) pl.splits = most;
  if (pl.splits < 1) pl.splits = 1;
  const int64_t span = lanes * pl.gper < 64 ? 64 : lanes * pl.gper;
  pl.parts = pl.splits * (256 / span);
  return pl;
}

hipError_t launch_norm(bool bf16, bool bwd, const NormParams& p, hipStream_t stream) {
  hipError_t e = bf16 ? norm_dispatch<uint16_t>(bwd, p, stream) : norm_dispatch<float>(bwd, p, stream);
  if (e == hipSuccess && bwd && p.part) {
    const int64_t C = p.groups * p.width;
    norm_sums_kernel<<<dim3(uint32_t((C + 7) / 8)), dim3(256), 0, stream>>>(p.part, p.parts, C, p.dweight, p.dbias);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace selscan
