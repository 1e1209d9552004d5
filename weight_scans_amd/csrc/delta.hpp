// delta.hpp -- argument blocks and launchers of the gated delta rule and of the
// query / key norms, shared by gl_delta.cpp and the kernels.  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "internal.hpp"

namespace gls {

struct Str3 {
  int64_t b, h, t;
};

// One call of the gated delta rule.  N sequences: b = 0..B-1 of T tokens each,
// or (cu != NULL) n = 0..N-1 of the packed axis of T tokens.
struct DeltaArgs {
  const void* q = nullptr;
  const void* k = nullptr;
  const void* v = nullptr;
  const void* la = nullptr;
  const void* be = nullptr;
  const void* state_in = nullptr;
  const int32_t* cu = nullptr;
  void* y = nullptr;
  void* state_out = nullptr;
  const void* dy = nullptr;
  const void* dstate_out = nullptr;
  void* dq = nullptr;
  void* dk_ = nullptr;
  void* dv_ = nullptr;
  void* dla = nullptr;
  void* dbe = nullptr;
  void* dstate_in = nullptr;
  int64_t N = 0, B = 0, T = 0;
  int H = 0, Hk = 0, dk = 0, dv = 0;
  bool gate_io = false;  // gates in the io dtype, not the compute type
  double scale = 1.0;
  Str3 sq, sk, sv, sy, sg, sdq, sdk, sdv, sdy, sdg;
  // token-serial kernels: states before every kSerialCk-th token
  // [slot][H][dv][dk], slot = serial_slot() + chunk
  void* ckpt = nullptr;
  // token-serial backward: sums over 16 rows of S, [tiles][H][B*T][dk] and [tiles][H][B*T]
  void* part_dq = nullptr;
  void* part_dk = nullptr;
  void* part_la = nullptr;
  void* part_be = nullptr;
  // step
  const int32_t* slots = nullptr;
  int64_t n_slots = 0;
};

// Slot of the first chunk of sequence n: sequences get consecutive, disjoint
// runs of slots for any lengths (a sequence of `len` tokens from t0 needs
// ceil(len / chunk) <= (t0 + len) / chunk - t0 / chunk + 1 of them).
__host__ __device__ inline int64_t chunk_slot0(bool packed, int64_t n, int64_t t0, int64_t T, int chunk) {
  return packed ? t0 / chunk + n : n * ((T + chunk - 1) / chunk);
}
inline int64_t chunk_slots(bool packed, int64_t N, int64_t T, int chunk) {
  return packed ? T / chunk + N : N * ((T + chunk - 1) / chunk);
}

// Batch row, first token and length of sequence n; cu's values are clamped to
// 0..T, so that a wrong table cannot lead outside the tensors.
struct SeqRange {
  int64_t b, t0, len;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* cu, int64_t n, int64_t T) {
  if (!cu) return {n, 0, T};
  int64_t lo = cu[n], hi = cu[n + 1];
  lo = lo < 0 ? 0 : lo > T ? T : lo;
  hi = hi < lo ? lo : hi > T ? T : hi;
  return {0, lo, hi - lo};
}

constexpr int kSerialRows = 16;  // rows of S per work-group of the token-serial kernels
inline int serial_ck(int io) { return io == IO_F64 ? 8 : 16; }
hipError_t launch_delta_serial_fwd(int io, const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_serial_bwd(int io, const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_step(int io, const DeltaArgs& a, hipStream_t s);

// Chunked matrix-core path (bf16, dk and dv multiples of 8, at most 128).  Per
// chunk of 64 tokens and value head (record = slot * H + h) the preparation
// leaves, as fragments of 64 lanes x 8 bf16 in the order in which the
// recurrences use them:
//   yf   Y  = (I + L beta)^-1 L, rows i     [6 blocks][hi, lo]
//   ytf, ptf   Y and P = scale (decayed q_i.k_j) with rows j   [6][hi, lo] each (training)
// and gates [9][64] fp32: e^l, beta, e^(l_C - l), the cumulative log2 decay l in
// two parts (whole and fraction), and the decay between blocks of 16 tokens as
// a product of two factors <= 1, with m_x the l before block x: e^(l_i - m_x)
// of i in block x, and e^(m_x - l_j) of j before it (x = 1, 2, 3).  The recurrences leave (training),
// in the form in which the gradients take them as operands:
//   sf, lf   the state before, the adjoint after the chunk: (rt, kb / 2) has
//            [lane (g, l)][kb % 2][q] = S[index(rt, 4 g + q)][index(kb, l)]  (delta_mfma.hpp)
//   yb       y before its rounding: (rt, tb) has [lane (g, l)][4] fp32 = y[token 16 tb + l][index(rt, 4 g + q)]
//   st       the last state [N][H][dv][dk] fp32
// and, as two fragments a row tile (row l in lanes, tokens in order; rows and
// halves exchanged as raw_at says),
//   ef, gf   e and dL/d(beta e)
//   zf, bf   dL/dlog_alpha and dL/dbeta over the tile's rows [64] fp32
constexpr int kDeltaChunk = 64;
constexpr int kFrag = 512;                       // bf16 per fragment
constexpr int kYf = 12 * kFrag;                  // per record
constexpr int kGates = 9 * 64;
constexpr int kPiece = 256;                      // bf16 per piece
constexpr int kY32 = 10 * 256;                   // fp32 per record
struct ChunkArgs {
  DeltaArgs a;
  uint16_t* yf = nullptr;
  uint16_t* ytf = nullptr;
  uint16_t* ptf = nullptr;
  float* gates = nullptr;
  uint16_t* sf = nullptr;
  uint16_t* ef = nullptr;
  float* yb = nullptr;
  float* st = nullptr;
  float* zf = nullptr;
  float* bf = nullptr;
  // fp32 chunks: Y and P by blocks of 16, [10][256] each, rows i in lanes, and
  // (training) rows j; the states before and the adjoints after the chunks by
  // blocks [row tile][dk / 16][256], row index 4g + q, column l in lanes; e, y
  // (yb) and dL/d(beta e), [64][16 row tiles] each
  float* y32 = nullptr;
  float* p32 = nullptr;
  float* yt32 = nullptr;
  float* pt32 = nullptr;
  float* s32 = nullptr;
  float* l32 = nullptr;
  float* e32 = nullptr;
  float* g32 = nullptr;
  uint16_t* lf = nullptr;
  uint16_t* gf = nullptr;
  int64_t slots = 0;    // chunk slots of the call
  int n_seg = 1;        // segments per sequence
  float* seg_s = nullptr;  // [head][n_seg][dv][dk] their first states (the first's: state_in, if given)
  float* seg_m = nullptr;  // [head][n_seg][dk][dk] what they do to a state
  float* seg_l = nullptr;  // backward: [head][n_seg][dv][dk] their last adjoints (the last's: dstate_out, if given)
};
inline int delta_wide(int d) { return d <= 64 ? 64 : 128; }
__host__ __device__ inline int delta_row_tiles(int dv) { return (dv + 31) / 32 * 2; }
bool delta_chunk_ok(int io, const DeltaArgs& a);  // sizes and strides of q, k, v
bool delta_rows_ok(const Str3& s, int d);         // strides of the other row tensors
hipError_t launch_delta_prep(const ChunkArgs& c, hipStream_t s);
hipError_t launch_delta_chunk_fwd(const ChunkArgs& c, hipStream_t s);
hipError_t launch_delta_chunk_bwd(const ChunkArgs& c, hipStream_t s);
hipError_t launch_delta_join(const ChunkArgs& c, bool back, hipStream_t s);
// The same in fp32 (dk and dv multiples of 4).
bool delta_chunk_f32_ok(int io, const DeltaArgs& a);  // sizes and strides of q, k, v
bool delta_rows_f32_ok(const Str3& s, int d);         // strides of the other row tensors
hipError_t launch_delta_chunk_f32(const ChunkArgs& c, hipStream_t s);
hipError_t launch_delta_chunk_f32_bwd(const ChunkArgs& c, hipStream_t s);

// Norms of queries and keys with the rotation.
struct QkArgs {
  const void* x[2];    // q, k
  const void* w[2];
  void* out[2];        // forward: normed rows; backward: dq, dk
  const void* dout[2]; // backward: gradients of the normed rows
  Str3 sx[2], so[2], sdo[2];
  int Hn[2];
  double scale[2];
  const void* cos;
  const void* sin;
  const int32_t* pos;
  int64_t B, T, n_pos, pos0;
  int d, rot;
  bool interleaved;
  double eps;
  void* part;          // backward: [2][groups][d] sums for dw
  void* dw[2];
  int64_t n_part;      // work-groups (parts)
  int hpg;             // heads per group of lanes (vector kernels)
};
// Work-groups of the backward (parts of the dw sums) for B*T tokens.
int64_t qknorm_bwd_parts(int io, const QkArgs& a);
hipError_t launch_qknorm_fwd(int io, const QkArgs& a, hipStream_t s);
hipError_t launch_qknorm_bwd(int io, const QkArgs& a, hipStream_t s);

}  // namespace gls
