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

// One thread walks one channel of one batch row.
template <typename IO>
__global__ __launch_bounds__(64) void gated_fwd_kernel(GatedParams p) {
  using T = io_traits<IO>;
  const int64_t i = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (i >= p.batch * p.D) return;
  const int64_t b = i / p.D, d = i % p.D;
  const IO* x = static_cast<const IO*>(p.x) + b * p.x_sb + d;
  const IO* r = static_cast<const IO*>(p.r) + b * p.r_sb + d;
  const IO* g = static_cast<const IO*>(p.g) + b * p.g_sb + d;
  IO* y = p.y ? static_cast<IO*>(p.y) + b * p.y_sb + d : nullptr;
  const float k = p.c * softplus_f32(p.lam[d]);
  float h = p.h0 ? p.h0[i] : 0.f;
  for (int64_t t = 0; t < p.L; ++t) {
    if (p.ckpt && t % kTile == 0) p.ckpt[(b * p.ntiles + t / kTile) * p.D + d] = h;
    float a, m;
    gated_decay(-k * sigmoid_f32(T::widen(r[t * p.r_sl])), a, m);
    // a first token takes nothing from the state, not even an infinity (also below)
    if (p.reset && p.reset[b * p.reset_sb + t]) { a = h = 0.f; m = 1.f; }
    h = fmaf(a, h, m * (sigmoid_f32(T::widen(g[t * p.g_sl])) * T::widen(x[t * p.x_sl])));
    if (y) y[t * p.y_sl] = narrow<IO>(h);
  }
  if (p.last) p.last[i] = h;
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

unsigned blocks_for(int64_t n, int per) { return unsigned((n + per - 1) / per); }

}  // namespace

hipError_t launch_gated_fwd(bool bf16, const GatedParams& p, hipStream_t stream) {
  const dim3 grid(blocks_for(p.batch * p.D, 64));
  if (bf16) hipLaunchKernelGGL(gated_fwd_kernel<uint16_t>, grid, dim3(64), 0, stream, p);
  else hipLaunchKernelGGL(gated_fwd_kernel<float>, grid, dim3(64), 0, stream, p);
  return hipGetLastError();
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
