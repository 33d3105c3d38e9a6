// linattn_kernels.hip -- linear attention: what surrounds the chunk walk of linattn_kernels.h (the
// states that enter the segments, sums over shared heads, the decays' gradient) and the decode step.
#include <hip/hip_runtime.h>

#include <cmath>

#include "device_common.h"
#include "scan_launch.h"

namespace selscan {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;

// Memory bounds all of these.  Segment states, from zero, into the states that enter the segments, in place: s := e^c s + own.  A thread has
// one value of a head's state; eight segments' are asked for at once.  The product with a segment's decay is formed in
// 64 bits, where neither overflows nor vanishes what meets a state that is small, zero or large.
__global__ __launch_bounds__(256) void lin_prefix_kernel(LinParams fwd, LinParams rev, int blocks) {
  const bool REV = blockIdx.y != 0;
  const LinParams& p = REV ? rev : fwd;
  const int block = p.kd * p.vd, at = int(blockIdx.x % blocks) * 256 + int(threadIdx.x);
  const int64_t bh = blockIdx.x / blocks;
  if (at >= block) return;
  float s = p.s0 ? p.s0[bh * block + at] : 0.f;
  float* const ws = p.seg + bh * p.nseg * block + at;
  const double* const decay = p.seg_decay + bh * p.nseg;
  for (int first = 0; first < p.nseg; first += 8) {
    const int n = p.nseg - first < 8 ? p.nseg - first : 8;
    float own[8];
    double d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = first + i + 1 < p.nseg ? first + i : 0;        // (nothing was left behind the last segment)
      const int seg = REV ? p.nseg - 1 - k : k;
      own[i] = ws[int64_t(seg) * block];
      d[i] = decay[seg];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        const int seg = REV ? p.nseg - 1 - first - i : first + i;
        ws[int64_t(seg) * block] = s;
        // (beyond 2^+-1000 whatever is not zero is infinite, and what is finite vanishes)
        const double whole = fmin(fmax(rint(d[i]), -1000.0), 1000.0);
        const double by = ldexp(double(__builtin_amdgcn_exp2f(float(fmax(d[i] - whole, -1.0)))), int(whole));
        s = d[i] == -HUGE_VAL ? own[i] : float(fma(by, double(s), double(own[i])));
      }
  }
}

// 2^log_lanes threads for a row of `width` columns.
template <typename T>
__global__ __launch_bounds__(256) void lin_heads_kernel(const float* part, T* out0, T* out1, int64_t rows, int share, int width,
                                                        int log_lanes) {
  T* const out = blockIdx.y ? out1 : out0;
  part += blockIdx.y * rows * share * width;
  const int c = threadIdx.x & ((1 << log_lanes) - 1), per = 256 >> log_lanes;
  if (c >= width) return;
  for (int64_t row = int64_t(blockIdx.x) * per + (threadIdx.x >> log_lanes); row < rows; row += int64_t(gridDim.x) * per) {
    const float* const src = part + row * share * width + c;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < share; ++k) s += src[int64_t(k) * width];
    if constexpr (sizeof(T) == 2)
      out[row * width + c] = bf16_rne(s);
    else
      out[row * width + c] = s;
  }
}

// One workgroup per segment of a (batch row, head), its threads' four tokens each at a time, from the last.  The sums run
// in 64 bits: what a token's decay passes is the small difference of what follows it and what precedes it.  Two things
// cut them short, since what is left out would add up to nothing but its rounding: a token that starts anew ends the
// sums of those before it, and what passes from a segment to the next is the product of the state there and its
// gradient (4 x 16 heads x 4096 packed tokens in 8 segments: relative error
// 1.5e-6 with neither, 1.2e-6 with the first, 5.8e-7; 1 x 4 heads x 131072, whose sums also run side by side then: the
// backward 990 us, and 764).
template <int kDecayThreads>
__global__ __launch_bounds__(kDecayThreads) void lin_decay_kernel(LinDecayParams p) {
  __shared__ double tmp[kDecayThreads / 64];
  __shared__ int ends[kDecayThreads / 64];
  const int nseg = p.nseg, seg = int(blockIdx.x) % nseg;
  const int64_t bh = int(blockIdx.x) / nseg, b = bh / p.H, h = bh % p.H;
  const int64_t first = seg * p.seg_len, L = seg + 1 < nseg ? first + p.seg_len : p.L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto block_sum = [&](double v) {
    for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
    __syncthreads();
    if (lane == 0) tmp[wave] = v;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kDecayThreads / 64; ++w) s += tmp[w];
    return s;
  };
  double carry = 0.0;
  const bool behind = seg + 1 == nseg;
  const float* const state = behind ? (p.last ? p.last + bh * p.state : nullptr) : p.states + (bh * nseg + seg + 1) * p.state;
  const float* const grad = behind ? (p.dlast ? p.dlast + bh * p.state : nullptr) : p.grads + (bh * nseg + seg) * p.state;
  if (state && grad) {
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = tid; i < p.state; i += kDecayThreads) s += double(state[i]) * double(grad[i]);
    carry = block_sum(s);
  }
  double sum = 0.0;
  const int64_t part = p.batch * p.L * p.H;
  constexpr int64_t kStep = 4 * kDecayThreads;
  for (int64_t t1 = first + (L - first + kStep - 1) / kStep * kStep; t1 > first; t1 -= kStep) {
    const int64_t t = t1 - 4 * tid - 4;           // thread 0 has the last four tokens
    double v[4];
    bool start[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = 0.0;
      start[e] = false;
      if (t + e < L) {
        const int64_t at = bh * p.L + t + e;
        for (int i = 0; i < p.nq; ++i) v[e] += double(p.qdq[i * part + at]);
        for (int i = 0; i < p.nk; ++i) v[e] -= double(p.kdk[i * part + at]);
        start[e] = double(p.g[b * p.g_sb + (t + e) * p.g_sl + h * p.g_sh]) * 1.4426950408889634 < -150.0;
      }
    }
#pragma unroll
    for (int e = 2; e >= 0; --e) v[e] += start[e + 1] ? 0.0 : v[e + 1];
    // what this thread and those with later tokens add to an earlier token, and whether one of them starts anew
    double all = start[0] ? 0.0 : v[0];
    int end = start[0] || start[1] || start[2] || start[3];
    for (int d = 1; d < 64; d *= 2) {
      const double o = __shfl_up(all, d);
      const int oe = __shfl_up(end, d);
      if (lane >= d) {
        if (!end) all += o;
        end |= oe;
      }
    }
    __syncthreads();
    if (lane == 63) {
      tmp[wave] = all;
      ends[wave] = end;
    }
    __syncthreads();
    double later = carry;                         // of the wavefronts with later tokens
    for (int w = 0; w < kDecayThreads / 64; ++w) {
      carry = ends[w] ? tmp[w] : carry + tmp[w];
      if (w + 1 == wave) later = carry;
    }
    const double o = __shfl_up(all, 1);
    const int oe = __shfl_up(end, 1);
    if (lane > 0) later = oe ? o : later + o;
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      const double g = start[e] ? 0.0 : v[e] + later;
      if (start[e]) later = 0.0;
      if (t + e < L) {
        if (p.dg) p.dg[(b * p.L + t + e) * p.H + h] = float(g);
        sum += g;
      }
    }
  }
  if (p.dg_heads) {
    sum = block_sum(sum);
    if (tid == 0) p.sums[blockIdx.x] = sum;
  }
}

__global__ __launch_bounds__(256) void lin_decay_heads_kernel(const double* sums, float* out, int64_t batch, int64_t H, int nseg) {
  const int64_t h = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (h >= H) return;
  double s = 0.0;
  for (int64_t b = 0; b < batch; ++b)
    for (int seg = 0; seg < nseg; ++seg) s += sums[(b * H + h) * nseg + seg];
  out[h] = float(s);
}

// One workgroup per (batch row, head): S := a S + k v^T, o = scale q^T S, on a state of [K][V].  A row
// of the state is taken by `lanes` lanes of 4 columns, 16 bytes on any boundary of 4; the 256 / lanes rows of a pass are
// summed through LDS.  Memory bounds it: 64 x 80 heads x 128 x 64 take 53 us for 336 MB (6.3 TB/s, some of it from the
// last-level cache; 65 us where slots are shared out and the states do not fit it).  Of a V that is no multiple of 4 the last lane's columns end where the row does: some are the lane
// before's too, and both form and store the same bits (one instruction reads a row, a later one writes it).
template <typename T>
__global__ __launch_bounds__(256) void lin_step_kernel(LinStepParams p, int lanes) {
  __shared__ float sq[256], sk[256];
  __shared__ f32x4 part[256];
  const int64_t b = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int64_t src = p.read_slots ? int64_t(p.read_slots[b]) : b, dst = p.write_slots ? int64_t(p.write_slots[b]) : b;
  if (dst < 0 || dst >= p.slots) return;          // padding
  const bool from = src >= 0 && src < p.slots;
  const int tid = threadIdx.x, first = (tid % lanes) * 4, row0 = tid / lanes, rows = 256 / lanes;
  const bool wide = p.vd >= 4, in = first < p.vd;
  const int col = wide && first + 4 > p.vd ? p.vd - 4 : first;
  const int64_t hk = h / p.share;
  auto at = [](const void* t, int64_t i) { return io_traits<T>::widen(static_cast<const T*>(t)[i]); };
  if (tid < p.kd) {
    sq[tid] = at(p.q, b * p.q_sb + hk * p.q_sh + tid) * p.scale;
    sk[tid] = at(p.k, b * p.k_sb + hk * p.k_sh + tid);
  }
  f32x4 v = {0.f, 0.f, 0.f, 0.f}, o = v;
  for (int e = 0; e < 4; ++e)
    if (in && col + e < p.vd) v[e] = at(p.v, b * p.v_sb + h * p.v_sh + col + e);
  const float lg = p.g[b * p.g_sb + h * p.g_sh];
  const bool keep = from && !(double(lg) * 1.4426950408889634 < -150.0);
  const float a = expf(lg);
  const int64_t block = int64_t(p.kd) * p.vd;
  const float* s_in = p.state + (src * p.H + h) * block + col;
  float* s_out = p.state + (dst * p.H + h) * block + col;
  __syncthreads();
  for (int r = row0; r < p.kd; r += rows) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (keep && in) {
      if (wide)
        __builtin_memcpy(&s, s_in + int64_t(r) * p.vd, 16);
      else
        for (int e = 0; e < 4; ++e)
          if (col + e < p.vd) s[e] = s_in[int64_t(r) * p.vd + e];
    }
    const float k = sk[r], q = sq[r];
    for (int e = 0; e < 4; ++e) {
      s[e] = keep ? fmaf(a, s[e], k * v[e]) : k * v[e];
      o[e] = fmaf(q, s[e], o[e]);
    }
    if (in) {
      if (wide)
        __builtin_memcpy(s_out + int64_t(r) * p.vd, &s, 16);
      else
        for (int e = 0; e < 4; ++e)
          if (col + e < p.vd) s_out[int64_t(r) * p.vd + e] = s[e];
    }
  }
  part[tid] = o;
  __syncthreads();
  if (tid < lanes && in) {
    for (int r = 1; r < rows; ++r) o += part[r * lanes + tid];
    T* dsto = static_cast<T*>(p.o) + b * p.o_sb + h * p.o_sh + col;
    for (int e = 0; e < 4; ++e)
      if (col + e < p.vd) {
        if constexpr (sizeof(T) == 2)
          dsto[e] = bf16_rne(o[e]);
        else
          dsto[e] = o[e];
      }
  }
}

}  // namespace

hipError_t launch_lin(bool bf16, LinWalk walk, const LinParams* p, hipStream_t stream) {
  switch (lin_kd(p->kd)) {
    case 64: return bf16 ? launch_lin_bf16_64(walk, p, stream) : launch_lin_f32_64(walk, p, stream);
    case 128: return bf16 ? launch_lin_bf16_128(walk, p, stream) : launch_lin_f32_128(walk, p, stream);
    default: return bf16 ? launch_lin_bf16_256(walk, p, stream) : launch_lin_f32_256(walk, p, stream);
  }
}

hipError_t launch_lin_states(bool bf16, bool both, const LinParams* p, hipStream_t stream) {
  if (p->nseg == 1) return hipSuccess;
  const hipError_t e = launch_lin(bf16, both ? LinWalk::states : LinWalk::state, p, stream);
  if (e != hipSuccess) return e;
  const int blocks = (p->kd * p->vd + 255) / 256;
  lin_prefix_kernel<<<dim3(uint32_t(p->batch * p->H * blocks), both ? 2 : 1), dim3(256), 0, stream>>>(p[0], p[both], blocks);
  return hipGetLastError();
}

hipError_t launch_lin_heads(bool bf16, const float* part, void* out0, void* out1, int64_t tokens, int64_t H, int share,
                            int width, hipStream_t stream) {
  int log_lanes = 0;
  while (1 << log_lanes < width) ++log_lanes;
  const int64_t rows = tokens * (H / share), per = 256 >> log_lanes, blocks = (rows + per - 1) / per;
  const dim3 grid(uint32_t(blocks < (1 << 20) ? blocks : 1 << 20), 2);
  if (bf16)
    lin_heads_kernel<uint16_t><<<grid, dim3(256), 0, stream>>>(part, static_cast<uint16_t*>(out0),
                                                               static_cast<uint16_t*>(out1), rows, share, width, log_lanes);
  else
    lin_heads_kernel<float><<<grid, dim3(256), 0, stream>>>(part, static_cast<float*>(out0), static_cast<float*>(out1), rows,
                                                            share, width, log_lanes);
  return hipGetLastError();
}

hipError_t launch_lin_decay(const LinDecayParams& p, hipStream_t stream) {
  // As many threads as one step of the tokens takes (4096 heads of 64 tokens: 1024 threads 74 us, 256 17; 1024 heads
  // of 1024 tokens 31 and 20; of more tokens, fewer threads have more steps, each of which waits for its sums).
  const dim3 grid(uint32_t(p.batch * p.H * p.nseg));
  if (p.seg_len <= 1024)
    lin_decay_kernel<256><<<grid, dim3(256), 0, stream>>>(p);
  else
    lin_decay_kernel<1024><<<grid, dim3(1024), 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.dg_heads) {
    lin_decay_heads_kernel<<<dim3(uint32_t((p.H + 255) / 256)), dim3(256), 0, stream>>>(p.sums, p.dg_heads, p.batch, p.H, p.nseg);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_lin_step(bool bf16, const LinStepParams& p, hipStream_t stream) {
  int lanes = 1;
  while (lanes * 4 < p.vd) lanes *= 2;
  const dim3 grid(uint32_t(p.batch * p.H));
  if (bf16)
    lin_step_kernel<uint16_t><<<grid, dim3(256), 0, stream>>>(p, lanes);
  else
    lin_step_kernel<float><<<grid, dim3(256), 0, stream>>>(p, lanes);
  return hipGetLastError();
}

}  // namespace selscan
