// linattn_kernels.hip -- linear attention: what surrounds the chunk walk of linattn_kernels.h (the
// states that enter the segments, sums over shared heads, the decays' gradient) and the decode step.
#include <hip/hip_runtime.h>

#include <cmath>

#include "device_common.h"
#include "linattn_device.h"
#include "scan_launch.h"

namespace selscan {
namespace {

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

// Running sums over the lanes of a wavefront, in the vector unit: within rows of 16 lanes, then from row to row.
template <int CTRL, int ROWS> __device__ __forceinline__ float lin_moved(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS> __device__ __forceinline__ double lin_moved(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b)), CTRL, ROWS, 0xf, false));
  const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(b >> 32)), CTRL, ROWS, 0xf, false));
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
template <typename V> __device__ __forceinline__ V lin_running(V v) {
  v += lin_moved<0x111, 0xf>(v);                  // row_shr:1, 2, 4, 8
  v += lin_moved<0x112, 0xf>(v);
  v += lin_moved<0x114, 0xf>(v);
  v += lin_moved<0x118, 0xf>(v);
  v += lin_moved<0x142, 0xa>(v);                  // row_bcast:15, into the second and the fourth row
  v += lin_moved<0x143, 0xc>(v);                  // row_bcast:31, into the upper two
  return v;
}
template <typename V> __device__ __forceinline__ V lin_before(V v) { return lin_moved<0x138, 0xf>(v); }      // wave_shr:1

// The decays' gradient.  A token's decay meets what passes it: from its chunk's tokens before it, or from the state S before
// the chunk, to its chunk's tokens from itself on, or to the gradient R of the state behind the chunk:
//     dg_t = sum_{j < t <= i} P_ij (q_i . k_j) (do_i . v_j) + sum_{i >= t} X_i + sum_{j < t} Y_j + e^c <S, R>,
//     P_ij = scale e^{c_i - c_j},  X_i = scale e^{c_i} q_i S do_i,  Y_j = e^{c - c_j} k_j R v_j
// Every addend has the token's decay in it, and none of them a token that does not meet it, so neither strong decays nor what
// is not finite elsewhere cost a gradient its bits.  (The sum over all later tokens of q . dq - k . dk is the same and needs no
// products, but what cancels in it is of the size of the gradients of q and k: at decays of e^-6 its relative error was 1e-3,
// of e^-20 it had no digit.)  X and Y come from the walks, the products of rows with their parts of the state.
//
// Z = e^c <S, R>.  Beside a chunk, <S', R'> = Z + sum Y behind it (S' the state there) and Z + sum X before it, so that from one such
// product Z follows from chunk to chunk.  What that loses is 2^-24 of the X and Y on the way, of which a token's gradient is
// a share of the size of its decay: 1/64 of it still leaves more than four digits.  So the walks keep S and R between every lin_span() chunks only; a chunk in which a token starts anew,
// or whose decay is below fp32's smallest, 2^-149, has Z = 0.  A chunk with a stronger decay that is neither is
// marked, and so is one with a value that is not finite: in such spans S is formed before each chunk (the walk `keep`)
// and met by R behind it (`cross`).
// One workgroup for lin_span() chunks of a head (4 x 4096 tokens of 16 heads, 128 x 128: 20 us).
__global__ __launch_bounds__(256) void lin_between_kernel(LinBetweenParams p) {
  constexpr int kSpan = lin_span();
  __shared__ double sum_x[kSpan], sum_y[kSpan], total[kSpan], tmp[4];
  __shared__ int begins[kSpan];
  const int64_t spans = (p.nchunks + kSpan - 1) / kSpan;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t item = blockIdx.x; item < p.batch * p.H * spans; item += gridDim.x) {
    const int64_t bh = item / spans, m = item % spans, b = bh / p.H, h = bh % p.H, c0 = m * kSpan;
    const int n = int(p.nchunks - c0 < kSpan ? p.nchunks - c0 : kSpan);
    int any = 0;
    for (int i = tid; i < 2 * n * p.marks_each; i += 256)
      any |= p.marks[((i & 1) * p.batch * p.H + bh) * p.nchunks * p.marks_each + c0 * p.marks_each + (i >> 1)];
    const bool marked = __syncthreads_or(any);
    const int64_t rows = p.batch * p.H * p.L;
    for (int c = wave; c < n; c += 4) {
      const int64_t t0 = (c0 + c) * p.chunk;
      const bool in = lane < p.chunk && t0 + lane < p.L;
      double g = in ? double(p.g[b * p.g_sb + (t0 + lane) * p.g_sl + h * p.g_sh]) * 1.4426950408889634 : 0.0, x = 0.0, y = 0.0;
      const bool start = g < -150.0;
      const uint64_t starts = __ballot(start), upto = (uint64_t(2) << lane) - 1;
      if (in)
        for (int i = 0; i < p.nq; ++i) {
          x += double(p.qdq[i * rows + bh * p.L + t0 + lane]);
          y += double(p.kdk[i * rows + bh * p.L + t0 + lane]);
        }
      if (start) g = 0.0;
      if (starts & upto) x = 0.0;
      if (starts & ~upto) y = 0.0;
      for (int d = 32; d > 0; d /= 2) {
        x += __shfl_xor(x, d);
        y += __shfl_xor(y, d);
        g += __shfl_xor(g, d);
      }
      if (lane == 0) {
        sum_x[c] = x;
        sum_y[c] = y;
        total[c] = g;
        begins[c] = starts != 0;
      }
    }
    __syncthreads();
    double* const out = p.between + bh * p.nchunks + c0;
    if (marked) {
      if (tid < n) {
        double z = 0.0;
        for (int i = 0; i < p.nz; ++i) z += double(p.cross[(i * p.batch * p.H + bh) * p.nchunks + c0 + tid]);
        const double whole = fmin(fmax(rint(total[tid]), -1000.0), 1000.0);
        z *= ldexp(double(__builtin_amdgcn_exp2f(float(fmax(total[tid] - whole, -1.0)))), int(whole));
        out[tid] = begins[tid] ? 0.0 : z;
      }
    } else {
      // <S, R> behind the last of the chunks
      const float *s = nullptr, *r = nullptr;
      int64_t size = p.kept_state;
      if (m + 1 < spans) {
        s = p.kept + (bh * p.nchunks + (m + 1) * kSpan) * size;
        r = p.back + (bh * spans + m + 1) * size;
      } else if (p.dlast) {
        size = p.state;
        s = p.last + bh * size;
        r = p.dlast + bh * size;
      }
      double sum = 0.0;
      if (s && m + 1 < spans) {                     // (rows of a multiple of four)
#pragma unroll 4
        for (int64_t i = tid; i < size / 4; i += 256) {
          const f32x4 x = reinterpret_cast<const f32x4*>(s)[i], y = reinterpret_cast<const f32x4*>(r)[i];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += double(x[e]) * double(y[e]);
        }
      } else if (s) {
#pragma unroll 8
        for (int64_t i = tid; i < size; i += 256) sum += double(s[i]) * double(r[i]);
      }
      for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d);
      if (lane == 0) tmp[wave] = sum;
      __syncthreads();
      if (tid == 0) {
        double beside = (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
        for (int c = n - 1; c >= 0; --c) {
          const bool first = c0 + c == 0 && !p.initial, last = c0 + c + 1 == p.nchunks && !p.dlast;   // (one of the two is zero)
          const double z = begins[c] || total[c] < kGone || first || last ? 0.0 : beside - sum_y[c];
          beside = z + sum_x[c];
          out[c] = z;
        }
      }
    }
    __syncthreads();
  }
}

// One workgroup a chunk of a head.  Memory bounds it: 4 x 4096 tokens of 16 heads, 128 x 128 bf16, 68 us for the 268 MB of q, k,
// v and do.  (Its tiles and sums leave room for six workgroups a compute unit; with two of them, and sums through the LDS
// in the place of the vector unit's, 160 us.)
template <typename T, int C>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 6 : 4) void lin_decay_kernel(LinDecayParams p, int64_t items) {
  using io = lin_io<T>;
  using Tile = LinTile<T, 64, C, 256>;
  constexpr int IT = C / 16, kTiles = IT * (IT + 1) / 2, kOwn = (kTiles + 3) / 4, kRow = C + 4;
  union Shared {
    struct { T rows[C * 64], cols[C * 64]; } t;
    float pairs[C * kRow];
  };
  __shared__ alignas(16) Shared sh;
  __shared__ float hi[C], lo[C], part[4][C];
  __shared__ int lim[C];
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int first = xcd_contiguous_block(blockIdx.x, gridDim.x);
  for (int64_t item = first; item < items; item += gridDim.x) {
    // (the heads of a chunk side by side: those that share queries and keys find them in the L2)
    const int64_t h = item % p.H, chunk = item / p.H % p.nchunks, b = item / p.H / p.nchunks, bh = b * p.H + h, t0 = chunk * C;
    const int n = int(p.L - t0 < C ? p.L - t0 : C);
    int lane = lin_lane(), tid = 64 * wave + lane, l16 = lane & 15, g = lane >> 4;
    auto again = [&] {
      lane = lin_lane();
      tid = 64 * wave + lane;
      l16 = lane & 15;
      g = lane >> 4;
    };
    // the decays: every wavefront has them, a token a lane
    double c = lane < n ? double(p.g[b * p.g_sb + (t0 + lane) * p.g_sl + h * p.g_sh]) * 1.4426950408889634 : 0.0;
    const bool start = c < -150.0;
    if (start) c = 0.0;
    c = lin_running(c);
    const uint64_t starts = __ballot(start);
    const uint64_t upto = (uint64_t(2) << lane) - 1, before = starts & upto, after = starts & ~upto;
    __syncthreads();                                // (what the item before has left there is no longer read)
    if (wave == 0 && lane < C) {
      hi[lane] = float(c);
      lo[lane] = float(c - double(float(c)));
      lim[lane] = before ? 63 - __builtin_clzll(before) : 0;
    }
    // q . k and do . v of the blocks that see each other, 64 channels at a time, the next ones on their way
    f32x4 qk[kOwn], dov[kOwn];
    // block x of a wavefront: row of blocks, and column
    auto block_row = [&](int x) { const int i = wave + 4 * x; return i >= 6 ? 3 : i >= 3 ? 2 : i >= 1 ? 1 : 0; };
    auto block_col = [&](int x) { const int r = block_row(x); return wave + 4 * x - r * (r + 1) / 2; };
#pragma unroll
    for (int x = 0; x < kOwn; ++x) dov[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int of = 0; of < 2; ++of) {
      // q . k first, do . v then, each in dov
#pragma unroll
      for (int x = 0; x < kOwn; ++x) {
        qk[x] = dov[x];
        dov[x] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      const int width = of ? p.dv : p.dk;
      Tile rows, cols;
      const T *now_r, *now_c;
      auto load = [&](int col0) {
        rows.init(p.rows[of], b, h, t0, col0, width);
        cols.init(p.cols[of], b, h, t0, col0, width);
        now_r = rows.at;
        now_c = cols.at;
        rows.template load<false>(tid, n);
        cols.template load<false>(tid, n);
      };
      again();
      load(0);
#pragma unroll 1
      for (int col0 = 0; col0 < width; col0 += 64) {
        again();
        rows.store(sh.t.rows, tid, now_r, n);
        cols.store(sh.t.cols, tid, now_c, n);
        __syncthreads();
        if (col0 + 64 < width) load(col0 + 64);
#pragma unroll
        for (int x = 0; x < kOwn; ++x) {
          __builtin_amdgcn_sched_barrier(0);
          again();
          if (wave + 4 * x >= kTiles) continue;
#pragma unroll
          for (int a = 0; a < 2; ++a)
            dov[x] = io::mma(io::template row<64>(sh.t.cols, 16 * block_col(x) + l16, 32 * a + 8 * g),
                             io::template row<64>(sh.t.rows, 16 * block_row(x) + l16, 32 * a + 8 * g), dov[x]);
        }
        __syncthreads();
      }
    }
    // the pairs: a lane has row i and columns j0 ..; nothing of what does not see each other
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      if (wave + 4 * x >= kTiles) continue;
      again();
      const int i = 16 * block_row(x) + l16, j0 = 16 * block_col(x) + 4 * g;
      f32x4 val;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = j0 + r;
        const float d = (hi[i] - hi[j]) + (lo[i] - lo[j]);
        const bool seen = j < i && j >= lim[i] && i < n;
        val[r] = seen ? qk[x][r] * (lin_exp2(d) * p.scale) * dov[x][r] : 0.f;
      }
      *reinterpret_cast<f32x4*>(sh.pairs + i * kRow + j0) = val;
    }
    __syncthreads();
    // sums over the pairs that pass a token, a token a lane: j < t by a running sum over each row, i >= t by choice
    float sum = 0.f;
    for (int i = wave; i < C; i += 4) {
      float v = lane < (i & ~15) + 16 ? sh.pairs[i * kRow + lane] : 0.f;
      v = lin_before(lin_running(v));
      if (lane <= i) sum += v;
    }
    if (lane < C) part[wave][lane] = sum;
    __syncthreads();
    if (wave == 0) {
      double x = 0.0, y = 0.0, z = 0.0;
      const int64_t at = bh * p.L + t0 + lane, rows_all = p.batch * p.H * p.L;
      if (lane < n) {
        for (int i = 0; i < p.nq; ++i) x += double(p.qdq[i * rows_all + at]);
        for (int i = 0; i < p.nq; ++i) y += double(p.kdk[i * rows_all + at]);
      }
      if (before) x = 0.0;                          // the state before the chunk does not reach it
      if (after) y = 0.0;                           // it does not reach the state behind the chunk
      if (!starts && p.between) z = p.between[bh * p.nchunks + chunk];
      x = __shfl(lin_running(__shfl(x, 63 - lane)), 63 - lane);
      y = lin_before(lin_running(y));
      double dg = 0.0;
      if (lane < n && !start)
        dg = double((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane])) + x + y + z;
      if (p.dg && lane < n) p.dg[(b * p.L + t0 + lane) * p.H + h] = float(dg);
      if (p.dg_heads) {
        for (int s = 32; s > 0; s /= 2) dg += __shfl_xor(dg, s);
        if (lane == 0) p.sums[(h * p.batch + b) * p.nchunks + chunk] = dg;
      }
    }
  }
}

// One workgroup a head: its chunks' sums, in a fixed order.
__global__ __launch_bounds__(256) void lin_decay_heads_kernel(const double* sums, float* out, int64_t each) {
  __shared__ double tmp[4];
  const double* const own = sums + blockIdx.x * each;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < each; i += 256) s += own[i];
  for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = float((tmp[0] + tmp[1]) + (tmp[2] + tmp[3]));
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
  const float a = fmaxf(expf(lg), kTiny);         // (2^-150 and more, as in lin_decay(): only a token that starts anew ends an infinity)
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

hipError_t launch_lin_between(const LinBetweenParams& p, hipStream_t stream) {
  const int64_t items = p.batch * p.H * ((p.nchunks + lin_span() - 1) / lin_span()), most = 1 << 20;
  lin_between_kernel<<<dim3(uint32_t(items < most ? items : most)), dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_lin_decay(bool bf16, const LinDecayParams& p, hipStream_t stream) {
  const int64_t items = p.batch * p.H * p.nchunks, most = 1 << 20;
  const dim3 grid(uint32_t(items < most ? items : most));
  if (bf16)
    lin_decay_kernel<uint16_t, 64><<<grid, dim3(256), 0, stream>>>(p, items);
  else if (p.chunk == 64)
    lin_decay_kernel<float, 64><<<grid, dim3(256), 0, stream>>>(p, items);
  else
    lin_decay_kernel<float, 32><<<grid, dim3(256), 0, stream>>>(p, items);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.dg_heads) {
    lin_decay_heads_kernel<<<dim3(uint32_t(p.H)), dim3(256), 0, stream>>>(p.sums, p.dg_heads, p.batch * p.nchunks);
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
