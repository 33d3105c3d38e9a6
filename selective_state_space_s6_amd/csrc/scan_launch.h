// scan_launch.h -- internal interface between the C ABI (selscan_api.cpp) and the
// kernels (scan_kernels.h and the units that instantiate it).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace selscan {

constexpr int kWavesPerBlock = 4;
enum { kPassSingle = 0, kPassState = 1, kPassApply = 2 };

// Everything one scan-kernel launch needs.  Strides are in elements.
struct ScanParams {
  const void* u;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* Dskip;   // may be null
  const void* z;        // may be null
  void* y;
  float* last_state;    // may be null
  const float* h0;      // initial state [batch][D][N], may be null (zero); selective only
  const float* delta_bias;   // [D], may be null (zero)
  int32_t euler;        // 1: Bbar = delta * B (first-order input coefficient)
  int32_t dxf;          // 1: the step size is transformed: delta + delta_bias, then softplus if
  int32_t softplus;     //    softplus is 1
  int64_t batch, L, D, N;
  int64_t u_sb, u_sl, delta_sb, delta_sl, z_sb, z_sl, y_sb, y_sl;
  int64_t B_sb, B_sl, B_sd, C_sb, C_sl, C_sd;
  int64_t chunk_len;    // tokens per chunk (L for the single pass)
  int32_t n_chunks;     // 1 for the single pass
  int32_t groups;       // channel groups per batch row: ceil(D / channels-per-wave)
  int32_t total_items;  // batch * n_chunks * groups (one wavefront each)
  float* ws_state;      // chunked: [batch][D][N][n_chunks] end states, then carries
  float* ws_dsum;       // chunked: [batch][D][n_chunks] sum of delta per chunk
  int32_t pipelined;    // 1: scan_kernel_coop (16 lanes per channel, D % 4 == 0, u/delta/z/y
                        //    rows and B/C rows readable four elements at a time); 0: scan_kernel
  // state pass of scan_kernel_coop, selective coefficients, optional: the state from a zero
  // start and the running sum of delta at the start of every 16-token tile of the chunk
  float* ckpt;          // [batch][ck_ntiles][D][N], tile index l / 16, or null
  float* ck_dsum;       // [batch][ck_ntiles][D]
  int64_t ck_ntiles;
  int32_t state_all;    // scan_kernel_coop: the state pass runs the last chunk too (its end
                        //    state is never carried; wanted for its checkpoints)
  int32_t sched_round;  // workgroups the GPU deals out per round (its compute units; 0 if
                        //    unknown: no rotation): workgroup b arrives on its compute unit in
                        //    round b / sched_round, which sets its turn in scan_kernel_coop's
                        //    issue-priority rotation
};

struct PrefixParams {
  const float* A;
  const float* dsum;
  const float* h0;      // initial state [batch][D][N], may be null (zero)
  float* state;
  int64_t batch, D, N;
  int32_t n_chunks;
  int32_t seg_width;    // power of two >= n_chunks, <= 64
};

// Lanes per channel (S) and states per lane (K) for N states.
void lanes_for_states(int64_t N, int* S, int* K);

hipError_t launch_scan_pass(int pass, bool bf16, bool ti, int S, int K, const ScanParams& p, hipStream_t stream);
// one scan pass of one element type (scan_inst_<io>_<pass>.hip); launch_scan_pass picks one
hipError_t launch_scan_f32_single(bool ti, int S, int K, const ScanParams& p, hipStream_t stream);
hipError_t launch_scan_f32_state(bool ti, int S, int K, const ScanParams& p, hipStream_t stream);
hipError_t launch_scan_f32_apply(bool ti, int S, int K, const ScanParams& p, hipStream_t stream);
hipError_t launch_scan_bf16_single(bool ti, int S, int K, const ScanParams& p, hipStream_t stream);
hipError_t launch_scan_bf16_state(bool ti, int S, int K, const ScanParams& p, hipStream_t stream);
hipError_t launch_scan_bf16_apply(bool ti, int S, int K, const ScanParams& p, hipStream_t stream);
hipError_t launch_chunk_prefix(const PrefixParams& p, hipStream_t stream);
hipError_t launch_fill_zero(float* x, int64_t n, hipStream_t stream);
hipError_t launch_copy(float* dst, const float* src, int64_t n, hipStream_t stream);

// One decode step (seqlen 1), state updated in place.
struct StepParams {
  const void* u;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* Dskip;   // may be null
  const void* z;        // may be null
  void* y;
  float* state;         // [batch][D][N]
  const float* delta_bias;   // [D], may be null (zero)
  int32_t euler;        // 1: Bbar = delta * B
  int32_t dxf;          // 1: step size delta + delta_bias, then softplus if softplus is 1
  int32_t softplus;
  int64_t batch, D, N;
  int64_t u_sb, delta_sb, z_sb, y_sb, B_sb, B_sd, C_sb, C_sd;
  int32_t vec;          // 1: N % 4 == 0, state and per-token B/C rows aligned to 4 elements
};
hipError_t launch_step(bool bf16, bool ti, const StepParams& p, hipStream_t stream);

// The convolution mode of fixed coefficients (conv_kernels.hip): delta [D], B/C [D][*] with
// channel strides B_sd / C_sd; u, z, y rows of D channels, D % 4 == 0, rows 16-byte (fp32) or
// 8-byte (bf16) aligned.
struct ConvParams {
  const void* u;
  const void* delta;
  const float* delta_bias;   // may be null
  const float* A;
  const void* B;
  const void* C;
  const float* Dskip;        // may be null
  const void* z;             // may be null
  void* y;
  float* last_state;         // may be null
  int32_t euler, dxf, softplus;
  int64_t batch, L, D, N;
  int64_t u_sb, u_sl, z_sb, z_sl, y_sb, y_sl, B_sd, C_sd;
  int32_t sched_round;       // compute units of the GPU (0 if unknown): the workgroup's dispatch
                             //    round, blockIdx / sched_round, sets its issue-priority turn
};
hipError_t launch_conv_ti(bool bf16, const ConvParams& p, hipStream_t stream);

}  // namespace selscan

namespace selscan {

// The backward pass (selective coefficients).  Strides in elements; the gradients du,
// ddelta, dz are contiguous [batch][L][D] in the I/O type.
struct BwdParams {
  const void* u;
  const void* delta;
  const float* delta_bias;   // may be null
  const float* A;
  const void* B;
  const void* C;
  const float* Dskip;   // may be null
  const void* z;        // may be null
  const float* h0;      // may be null
  const void* dy;
  const float* dlast;   // may be null
  void* du;
  void* ddelta;
  void* dz;             // may be null (then not written)
  float* dh0;           // may be null
  float* ckpt;          // [batch][ntiles][D][N] state at the start of every tile
  float* pB;            // [groups][batch][L][N] per-channel-group partial sums of dB
  float* pC;            // [groups][batch][L][N] per-group partial sums of dC
  float* pA;            // [batch][n_chunks][D][N] partial sums of dA
  float* pD;            // [batch][n_chunks][D] partial sums of dDskip
  float* pbias;         // [batch][n_chunks][D] partial sums of the bias gradient
  float* carry;         // [batch][D][N][n_chunks] state entering each chunk (n_chunks > 1)
  float* adjG;          // [batch][D][N][n_chunks] adjoint a chunk hands back from a zero start
  float* adjS;          // [batch][D][n_chunks] sum of delta over each chunk
  float* adj_in;        // [batch][D][N][n_chunks] adjoint reaching each chunk's end
  int64_t batch, L, D, N;
  int64_t u_sb, u_sl, delta_sb, delta_sl, z_sb, z_sl, dy_sb, dy_sl, B_sb, B_sl, C_sb, C_sl;
  int64_t ntiles;       // ceil(L / 16)
  int64_t chunk_len;    // tokens per chunk, a multiple of 16
  int32_t n_chunks;
  int32_t groups;       // ceil(D / channels per workgroup)
  int32_t euler;
  int32_t dxf;
  int32_t softplus;
  // 1: the forward state pass wrote each tile's zero-start state into ckpt and its running
  // sum of delta into ck_dsum, for every chunk
  int32_t ck_fwd;
  const float* ck_dsum; // [batch][ntiles][D]
  // fixed coefficients: [batch][D][n_chunks] each chunk's sum of delta (the chunk state pass
  // writes it for chunk_prefix_kernel)
  float* sdsum;
  // fixed coefficients: B_sd, C_sd (element stride between channels of B[d][n], C[d][n])
  int64_t B_sd, C_sd;
  // 1: u, delta, dy, z and du, ddelta, dz move as 4-channel vectors (D % 4 == 0; their row
  // and batch strides multiples of 4 elements, rows at least D long; bases aligned to 4
  // elements; a chunk's span under 2^31 bytes)
  int32_t vec;
};
// lanes per channel of the backward kernel (4 states per lane): 4, 8 or 16
int bwd_lanes_per_channel(int64_t N);
hipError_t launch_bwd(bool bf16, const BwdParams& p, hipStream_t stream);
// backward of fixed coefficients (bwd_ti_kernels.hip): the chunk end states from zero (for
// chunk_prefix_kernel), the chunk adjoints from zero (for bwd_adjoint_combine_kernel), or the
// main pass
enum { kTiPassState = 0, kTiPassAdjoint = 1, kTiPassMain = 2 };
hipError_t launch_bwd_ti(bool bf16, int pass, const BwdParams& p, hipStream_t stream);
// the adjoint combine of the selective backward, on its own (fixed coefficients)
hipError_t launch_bwd_adjoint_combine(const BwdParams& p, hipStream_t stream);
// out[i] = sum_{j < nparts} part[j * stride + i], i < m; out in the I/O type when bf16
hipError_t launch_sum_partials(const float* part, int64_t nparts, int64_t stride, void* out, int64_t m, bool bf16,
                               hipStream_t stream);

}  // namespace selscan

namespace selscan {

// The scalar-decay (Mamba-2) layer: bf16 x, delta, B, C, z, y; fp32 A [H], Dskip [H*P],
// states.  Contiguous: x, z, y [batch][L][H][64]; delta [batch][L][H]; B, C [batch][L][N].
struct SsdParams {
  const void* x;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* Dskip;   // may be null
  const void* z;        // may be null
  void* y;
  const float* h0;      // [batch][H][64][N], may be null
  float* last_state;    // [batch][H][64][N], may be null
  float* state;         // workspace [batch][H][n_chunks][64][N]: chunk states (transposed)
  uint16_t* carry;      // workspace [batch][H][n_chunks][64][N]: bf16 state entering each chunk
  float* decay;         // workspace [batch][H][n_chunks]: exp(A sum delta) of each chunk
  float* seg_state;     // workspace [batch][H][n_seg][64][N]: segment end states, then carried-in states
  float* seg_decay;     // workspace [batch][H][n_seg]: exp(A sum delta) of each segment
  int64_t batch, L, H, N;
  int64_t n_chunks;     // ceil(L / 64)
  int64_t n_seg;        // on-chip path: sequence segments (1: the whole sequence per workgroup)
  int64_t seg_chunks;   // chunks per segment (the last may have fewer)
  int32_t euler;
  int32_t fused;        // 1: on chip, one workgroup per (batch, segment, head), the state in registers
};
hipError_t launch_ssd(const SsdParams& p, hipStream_t stream);

}  // namespace selscan

namespace selscan {

// The gated linear recurrence (gated_kernels.hip).  Strides in elements; dx, dr, dg contiguous
// [batch][L][D] in the I/O type.
struct GatedParams {
  const void* x;
  const void* r;
  const void* g;
  const float* lam;
  const uint8_t* reset;  // may be null
  void* y;               // may be null (only the checkpoints are wanted)
  const float* h0;       // [batch][D], may be null (zero)
  float* last;           // [batch][D], may be null
  float* ckpt;           // [batch][ntiles][D] state entering each tile, may be null
  const void* dy;        // backward only, with y's strides
  const float* dlast;    // may be null
  void* dx;
  void* dr;
  void* dg;
  float* dlam;           // [D]
  float* dh0;            // may be null
  int64_t batch, L, D;
  int64_t x_sb, x_sl, r_sb, r_sl, g_sb, g_sl, y_sb, y_sl, reset_sb;
  int64_t ntiles;        // ceil(L / SELSCAN_GATED_TILE)
  float c;
  uint64_t* links;       // workspace: gated_link_words() words, or null (one chunk)
  float* kd;             // workspace [D]: c softplus(lam) (links)
  int32_t n_chunks;      // chunks of the pass: ceil(L / gated_chunk()), ceil(L / kGatedBwdChunk)
  int32_t persistent;    // workgroups take chunks by ticket (links)
  float* plam;           // workspace [n_chunks][batch][D]: partial sums of dlam
};
// tokens of a workgroup: eight runs of as many as its registers hold twice over
constexpr int gated_chunk(bool bf16) { return bf16 ? 128 : 64; }
constexpr int kGatedBwdChunk = 64;     // of the backward pass
constexpr int kTicketWords = 16;       // a cache line for the ticket counter
// words of the links between chunks: the ticket, a map per chunk and an end state per 8
// chunks, for every 128 channels
constexpr int64_t gated_link_words(int64_t batch, int64_t D, int64_t n_chunks) {
  return kTicketWords + batch * ((D + 127) / 128) * 128 * (n_chunks + n_chunks / 8);
}
hipError_t launch_gated_fwd(bool bf16, GatedParams p, int cus, hipStream_t stream);
hipError_t launch_gated_bwd(bool bf16, GatedParams p, int cus, hipStream_t stream);
hipError_t launch_gated_step(bool bf16, const GatedParams& p, float* state, hipStream_t stream);

// The 8-bit state cache (cache_kernels.hip): q [slots][elems], scale [slots][rows].
struct CacheParams {
  int8_t* q;
  float* scale;
  const int32_t* read_slots;   // may be null (0, 1, 2, ...)
  const int32_t* write_slots;  // may be null
  const int64_t* seed;         // may be null (round to nearest)
  int64_t slots, elems, row_len, rows;
  int64_t count;               // batch rows
};
hipError_t launch_cache_write(const float* state, const CacheParams& p, hipStream_t stream);
hipError_t launch_cache_read(bool bf16, void* out, const CacheParams& p, hipStream_t stream);
// one decode step of the selective scan / of the scalar-decay layer on cached states
hipError_t launch_step_cached(bool bf16, const StepParams& s, const CacheParams& p, hipStream_t stream);
hipError_t launch_ssd_step_cached(const SsdParams& s, const CacheParams& p, hipStream_t stream);

}  // namespace selscan

namespace selscan {

// Linear attention with a decay for each head (linattn_kernels.h, linattn_kernels.hip).
// A [batch][tokens][heads / share][width] operand; strides in elements.
struct LinTensor {
  const void* p;
  int64_t sb, sl, sh;
  int32_t share;        // heads that share one row
};
// One walk over the chunks (the header of linattn_kernels.h): the operands in the roles that they have in it.
struct LinParams {
  LinTensor q, k, v;
  void* out;            // [batch][tokens][H][vd] in the I/O type, or fp32 (out_f32)
  int64_t o_sb, o_sl, o_sh;
  int32_t out_f32;
  const float* g;       // logarithms of the decays
  int64_t g_sb, g_sl, g_sh;
  const float* s0;      // state that the walk begins with, (batch, head) blocks of kd * vd; may be null (zero)
  float* s1;            // state that it ends with, or null
  int64_t s_row, s_col; // strides of s0 and s1 within a block
  float* seg;           // workspace: [batch][H][nseg] blocks of kd * vd, laid out as s0's
  double* seg_decay;    // workspace: [batch][H][nseg], log2 of the segment's decay, -infinity where the state starts anew
  LinTensor x;          // grads: the products of x with the rows' parts of the state, [nblk][batch][H][L] (null: not wanted)
  float* dot;
  float* kept;          // the states before chunks, [batch][H][nchunks] blocks of [dv][c_row]: written by grads (forward,
  int64_t c_row;        // every lin_span()-th) and keep (the others), read by cross; c_row: dk to a multiple of 4
  float* back;          // grads, backward: the gradients between every lin_span() chunks, [batch][H][ceil(nchunks / lin_span())] blocks
  int32_t* marks;       // [2][batch][H][nchunks][marks_each]: written by grads, read by keep and cross, which leave spans without one
  int32_t marks_each;   // blocks of columns of grads
  int32_t ends;         // grads: 1: there is an initial state, 2: a gradient of the last one
  float* cross;         // cross: its product with the gradient behind the chunk, [nblk][batch][H][nchunks]
  int64_t batch, L, H;
  int32_t kd, vd;       // width of q and k, of v and out (1 .. 256)
  float pscale, fscale, wscale;   // of the pairs, of a row's product with the state, of its share in the state
  int32_t chunk;        // tokens of a chunk
  int64_t nchunks;      // ceil(L / chunk)
  int64_t seg_chunks;   // chunks of a segment
  int32_t nseg, nblk;   // segments; blocks of lin_cols() columns
  int32_t pairs;        // 1: heads 2 i and 2 i + 1 share their q and k and vd is at most 64: a workgroup takes both
};
constexpr int lin_kd(int64_t kd) { return kd <= 64 ? 64 : kd <= 128 ? 128 : 256; }
constexpr int lin_cols(int64_t vd) { return vd <= 64 ? 64 : 128; }
// Chunks between states that the decays' gradient starts from.
constexpr int lin_span() { return 8; }
// Tokens of a chunk: the LDS of a compute unit holds the tiles of a chunk of 64, but not those of 256
// fp32 channels.  (Chunks of 32 for all of fp32, two workgroups a compute unit: 2 x 16 heads x 4096, 64 x 64, 79 us in
// the place of 80; 128 x 128, whose registers then spill, 231 in the place of 198.)
constexpr int lin_chunk(bool bf16, int64_t kd) { return !bf16 && kd > 128 ? 32 : 64; }
// What a launch walks: forward or backward; the segments' states only, forward, or in both directions (p[0] forward,
// p[1] backward); a forward and a backward walk of what shares no queries and keys (pairs == 0), with their rows' products if wanted;
// of spans with a mark (segments of lin_span() chunks) the states before all chunks (forward), and their products with the
// gradients behind them (backward).
enum class LinWalk { forward, backward, state, states, grads, keep, cross };
// one launch, from s0 or (nseg > 1) from the states that enter the segments
hipError_t launch_lin(bool bf16, LinWalk walk, const LinParams* p, hipStream_t stream);
// nseg > 1: the states that enter the segments, from k, v and s0 (kd x vd, rows s_row apart, s_col == 1 or the
// other way round); of both directions, or forward only
hipError_t launch_lin_states(bool bf16, bool both, const LinParams* p, hipStream_t stream);
// units of one element type and width of q and k
hipError_t launch_lin_bf16_64(LinWalk walk, const LinParams* p, hipStream_t stream);
hipError_t launch_lin_bf16_128(LinWalk walk, const LinParams* p, hipStream_t stream);
hipError_t launch_lin_bf16_256(LinWalk walk, const LinParams* p, hipStream_t stream);
hipError_t launch_lin_f32_64(LinWalk walk, const LinParams* p, hipStream_t stream);
hipError_t launch_lin_f32_128(LinWalk walk, const LinParams* p, hipStream_t stream);
hipError_t launch_lin_f32_256(LinWalk walk, const LinParams* p, hipStream_t stream);

// Sums over the heads that share one, for two gradients: part [2][tokens][H][width] fp32 ->
// out0 and out1 [tokens][H / share][width]
hipError_t launch_lin_heads(bool bf16, const float* part, void* out0, void* out1, int64_t tokens, int64_t H, int share,
                            int width, hipStream_t stream);

// The decays' gradient, from the pairs of each chunk and what the walks have left of the states before and behind it.
struct LinDecayParams {
  LinTensor rows[2], cols[2];     // q and do; k and v
  int32_t dk, dv;
  const float* qdq;     // [nq][batch][H][L]: q . (the state's part of dq)
  const float* kdk;     // [nq][batch][H][L]: k . (the state's part of dk)
  const double* between;  // [batch][H][nchunks]: e^c <S, R>, or null (zero)
  const float* g;
  int64_t g_sb, g_sl, g_sh;
  float scale;
  float* dg;            // [batch][L][H], or null: the heads' sums only
  double* sums;         // workspace [H][batch][nchunks]
  float* dg_heads;      // [H], or null
  int64_t batch, L, H, nchunks;
  int32_t chunk, nq;
};
// e^c <S, R> of each chunk, S the state before it and R the gradient behind it
struct LinBetweenParams {
  const float* qdq;     // as LinDecayParams
  const float* kdk;
  const float* cross;   // [nz][batch][H][nchunks]: <S, R> of spans with a mark
  const float* kept;    // as LinParams
  const float* back;
  const int32_t* marks;
  const float* last;    // [batch][H][state]: the last state and its gradient, or null (zero)
  const float* dlast;
  const float* g;
  int64_t g_sb, g_sl, g_sh;
  double* between;
  int64_t batch, L, H, nchunks;
  int64_t state, kept_state;      // values of a state, and of a kept one
  int32_t chunk, nq, nz, marks_each;
  int32_t initial;      // there is an initial state
};
hipError_t launch_lin_between(const LinBetweenParams& p, hipStream_t stream);
hipError_t launch_lin_decay(bool bf16, const LinDecayParams& p, hipStream_t stream);

// One token per batch row, states in slots.
struct LinStepParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  void* o;
  float* state;               // [slots][H][K][V]
  const int32_t* read_slots;  // may be null (0, 1, 2, ...)
  const int32_t* write_slots;
  int64_t slots, batch, H;
  int32_t share, kd, vd;
  int64_t q_sb, q_sh, k_sb, k_sh, v_sb, v_sh, o_sb, o_sh, g_sb, g_sh;
  float scale;
};
hipError_t launch_lin_step(bool bf16, const LinStepParams& p, hipStream_t stream);

// Group norm with an activation (norm_kernels.hip).
struct NormPlan {
  int32_t log_lanes;    // threads of a group: a power of two up to 64, or 256
  int32_t ept;          // accesses of a thread
  int64_t gper, cblocks, splits, parts;  // backward: groups side by side in a workgroup, blocks of them, workgroups
                        // that share the rows, partial sums of dweight and dbias
};
NormPlan norm_plan(bool bf16, bool bwd, int64_t rows, int64_t groups, int64_t width);
struct NormParams {
  const void* x;
  const float* weight;  // [C], may be null
  const float* bias;    // [C], may be null
  const void* z;        // may be null (no gate)
  void* y;
  const void* dy;       // backward, with y's strides
  void* dx;
  void* dz;
  float* dweight;
  float* dbias;
  float* part;          // workspace [parts][2][C], or null (neither is wanted)
  int64_t rows, L, groups;
  int32_t width, silu;
  int32_t even;         // every group of channels begins and ends on 16 bytes
  int64_t x_sb, x_sl, z_sb, z_sl, y_sb, y_sl;
  float eps;
  int32_t log_lanes, ept;
  int64_t gper, cblocks, splits, parts;
};
hipError_t launch_norm(bool bf16, bool bwd, const NormParams& p, hipStream_t stream);

}  // namespace selscan
