// linattn_device.h -- linear attention: what the chunk walk (linattn_kernels.h) and the decays' gradient
// (linattn_kernels.hip) share: element types, tiles in the LDS and on their way there.
#pragma once

#include <cmath>
#include <type_traits>

#include "device_common.h"
#include "scan_launch.h"

namespace selscan {
namespace {

typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) float f32x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr float kTiny = 1.401298464e-45f;      // 2^-149
// Where the decays' gradient takes the product of a state and its gradient from the chunks beside it, and where not
// (lin_between_kernel): log2 of a token's decay, and of a chunk's.
constexpr double kStrong = -6.0, kGone = -149.0;
constexpr int kNowhere = 0x3ffffff0;            // a place in bytes beyond any state, another state's added to it too

// Place of (row, column) in an LDS tile of W columns.  A row's 16-byte pieces are exchanged with one another by
// bits of the row, so that both ways of reading, sixteen rows of one column of pieces and four neighbouring rows of four
// neighbouring pieces, spread over the banks more than plain rows would.  (Rows of 128 bytes share 256 in pairs.)
template <typename T, int W> __device__ __forceinline__ int lin_at(int row, int col) {
  constexpr int V = 16 / int(sizeof(T)), kPieces = W / V;
  static_assert(kPieces >= 8, "");
  const int f = kPieces >= 16 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  return row * W + ((col / V) ^ f) * V + col % V;
}

// Place of the pairs of row i and keys j .. in their tile: of the 16 x 16 blocks only those that see each other are
// kept, by rows of blocks (the backward's mirrored, `it` and `jt` counted from the end).  A row of fp32 has four 16-byte pieces, exchanged by bits
// of the row; one of bf16 has two, and a block's sixteen rows lie on all banks as they are.
template <typename T> __device__ __forceinline__ int lin_pair_at(int it, int jt, int row, int col) {
  constexpr int V = 16 / int(sizeof(T)), f = sizeof(T) == 4 ? 3 : 0;
  return ((it * (it + 1) / 2 + jt) * 16 + row) * 16 + ((col / V) ^ ((row >> 2) & f)) * V + col % V;
}

// What the walk needs of an element type: eight consecutive values of a contraction in one
// fragment (lane l: row or column l % 16, values 8 (l / 16) ..), and the product of two.
template <typename T> struct lin_io;
template <> struct lin_io<uint16_t> {
  using frag = bf16x8;
  static constexpr int kVec = 8;               // elements of 16 bytes
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // a column: values at rows r0 .. r0 + 7 of a tile; the 16 lanes of a group ask for 4 rows of four 4-element
  // pieces (lane i: row i / 4, piece i % 4), and the transposing read hands each lane its column
  template <int W>
  static __device__ __forceinline__ frag column(const uint16_t* tile, int r0, int first, int spread, int l16) {
    const int col = first + spread * (l16 & 3), r = r0 + (l16 >> 2);
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(tile + lin_at<uint16_t, W>(r, col)));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(tile + lin_at<uint16_t, W>(r + 4, col)));
    struct { s16x4 a, b; } v = {a, b};
    return __builtin_bit_cast(frag, v);
  }
  template <int W> static __device__ __forceinline__ frag row(const uint16_t* tile, int r, int c) {
    return *reinterpret_cast<const frag*>(tile + lin_at<uint16_t, W>(r, c));
  }
  static __device__ __forceinline__ frag pair(const uint16_t* tile, int at) { return *reinterpret_cast<const frag*>(tile + at); }
  static __device__ __forceinline__ f32x8 wide(frag a) { return __builtin_convertvector(a, f32x8); }
  static __device__ __forceinline__ frag round(f32x8 a) { return __builtin_convertvector(a, frag); }
  static __device__ __forceinline__ void narrow(uint16_t* p, float v) { *p = bf16_rne(v); }
  static __device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
  static __device__ __forceinline__ void store(uint16_t* p, f32x4 v) { *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4); }
};
template <> struct lin_io<float> {
  using frag = f32x8;
  static constexpr int kVec = 4;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  template <int W> static __device__ __forceinline__ frag row(const float* tile, int r, int c) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(tile + lin_at<float, W>(r, c));
    const f32x4 b = *reinterpret_cast<const f32x4*>(tile + lin_at<float, W>(r, c + 4));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  template <int W>
  static __device__ __forceinline__ frag column(const float* tile, int r0, int first, int spread, int l16) {
    const int col = first + spread * (l16 >> 2) + (l16 & 3);
    frag v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[lin_at<float, W>(r0 + e, col)];
    return v;
  }
  static __device__ __forceinline__ frag pair(const float* tile, int at) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(tile + at);
    const f32x4 b = *reinterpret_cast<const f32x4*>(tile + (at ^ 4));       // (the piece beside it)
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f32x8 wide(frag a) { return a; }
  static __device__ __forceinline__ frag round(f32x8 a) { return a; }
  static __device__ __forceinline__ void narrow(float* p, float v) { *p = v; }
  static __device__ __forceinline__ float widen(float b) { return b; }
  static __device__ __forceinline__ void store(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
};

// The lane's number, formed anew wherever it is asked for: kept, what is formed of it (places in tiles and
// tensors) would not leave the walk's registers room.
__device__ __forceinline__ int lin_lane() {
  int zero = 0;
  asm volatile("" : "+s"(zero));
  return int(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, uint32_t(zero))));
}

// 2^x, its subnormal values too (the instruction gives zero in their place).
__device__ __forceinline__ float lin_exp2(float x) {
  return x < -100.f ? __builtin_amdgcn_exp2f(x + 64.f) * 5.421010862e-20f : __builtin_amdgcn_exp2f(x);
}
// An operand's tile of C rows and W columns on its way: the n tokens of a chunk, zeros elsewhere.  A
// thread has 16-byte pieces of a row (on any element's boundary).  Where the width is not a multiple of a
// piece, the last one is read so that it ends where the row does, and its values are moved when they are
// stored; rows shorter than a piece are read element by element then.
// (What a call forms of `tid`, it forms again at each chunk: kept, it would not leave the registers room.)
template <typename T, int W, int C, int THREADS>
struct LinTile {
  static constexpr int V = lin_io<T>::kVec, kPieces = W / V, kRows = THREADS / kPieces, N = C / kRows;
  static_assert(N >= 1 && N * kRows == C, "");
  static constexpr int kOutside = 0x7ffffff0;    // beyond any tile: reads as zero
  u32x4 piece[N];
  const T* at;            // the next chunk's first token
  int sl, cols;
  bool even;

  static __device__ __forceinline__ const T* head(const LinTensor& x, int64_t b, int64_t h, int col0) {
    return static_cast<const T*>(x.p) + b * x.sb + int64_t(uint32_t(h) / uint32_t(x.share)) * x.sh + col0;
  }
  __device__ __forceinline__ void init(const LinTensor& x, int64_t b, int64_t h, int64_t t0, int col0, int width) {
    at = head(x, b, h, col0) + t0 * x.sl;
    sl = int(x.sl);
    cols = width - col0 < W ? width - col0 : W;
    even = cols % V == 0;
  }
  // asks for the pieces of a chunk and goes on to the next
  template <bool REV> __device__ __forceinline__ void load(int tid, int n) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(at), (short)0,
                                                        ((n - 1) * sl + cols) * int(sizeof(T)), 0x00020000);
    const int row0 = tid / kPieces, step = kRows * sl * int(sizeof(T));
    int c = (tid % kPieces) * V;
    const bool in = c < cols;
    if (c + V > cols) c = cols - V;
    const int to = in && c >= 0 ? (row0 * sl + c) * int(sizeof(T)) : kOutside;
    if (n == C) {
#pragma unroll
      for (int i = 0; i < N; ++i) piece[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, to + i * step, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        piece[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, row0 + i * kRows < n ? to + i * step : kOutside, 0, 0);
    }
    at += (REV ? -int64_t(C) : int64_t(C)) * sl;
  }
  // ... and their place in the tile; `now`: the chunk's first token
  __device__ __forceinline__ void store(T* tile, int tid, const T* now, int n) {
    const int row0 = tid / kPieces, c = (tid % kPieces) * V;
    if (!even) {
      int cols = this->cols;
      asm volatile("" : "+s"(cols));
      const int by = (V - cols % V) * int(sizeof(T));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        u32x4 x = piece[i];
        if (by & 2) x = u32x4{(x[0] >> 16) | (x[1] << 16), (x[1] >> 16) | (x[2] << 16), (x[2] >> 16) | (x[3] << 16), x[3] >> 16};
        if (by & 4) x = u32x4{x[1], x[2], x[3], 0};
        if (by & 8) x = u32x4{x[2], x[3], 0, 0};
        if (c + V > cols) piece[i] = x;           // the end of a row: down by V - cols % V values
      }
      if (cols < V) {
        if (c == 0)
#pragma unroll 1
          for (int i = 0; i < N; ++i)
#pragma unroll 1
            for (int e = 0; e < V; ++e) {
              const int row = row0 + i * kRows;
              tile[lin_at<T, W>(row, e)] = e < cols && row < n ? now[int64_t(row) * sl + e] : T(0);
            }
        if (c == 0) return;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(tile + lin_at<T, W>(row0 + i * kRows, c)) = piece[i];
  }
};

}  // namespace
}  // namespace selscan
