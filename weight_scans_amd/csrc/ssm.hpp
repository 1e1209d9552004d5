// ssm.hpp -- argument blocks and launchers of the selective scan, the short
// convolution and the norms around a block, shared by gl_ssm.cpp and the kernels.
// Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "delta.hpp"  // SeqRange, chunk_slot0: packed sequences

namespace gls {

struct Rows {
  int64_t b, t, g;
};
// A launch counts its threads in 32 bits.  A call's launchers return
// hipErrorInvalidConfiguration for one that would not fit before they launch any.
inline bool launch_fits(int64_t threads) { return threads <= 0xffffffffLL - 1024; }

// ---- convolution
struct ConvArgs {
  const void* x = nullptr;
  const void* w = nullptr;
  const void* bias = nullptr;
  const void* state_in = nullptr;
  const int32_t* cu = nullptr;
  void* y = nullptr;
  void* state_out = nullptr;
  const void* dy = nullptr;
  const void* dstate_out = nullptr;
  void* dx = nullptr;
  void* dw = nullptr;
  void* dbias = nullptr;
  void* dstate_in = nullptr;
  void* part = nullptr;  // backward: [parts][K + 1][D] sums for dw and dbias
  const int32_t* slots = nullptr;
  int64_t n_slots = 0;
  int64_t n_seq = 0;     // packed sequences, 0 = none
  int64_t N = 0, B = 0, T = 0;
  int D = 0, K = 0;
  bool silu = false;
  Rows sx{}, sy{}, sdy{}, sdx{};
};
size_t conv_bwd_ws(int io, const ConvArgs& a);
hipError_t launch_conv_fwd(int io, const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd(int io, const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(int io, const ConvArgs& a, hipStream_t s);

// ---- selective scan
struct SsmArgs {
  const void* x = nullptr;
  const void* dt = nullptr;
  const void* A = nullptr;
  const void* Bm = nullptr;
  const void* Cm = nullptr;
  const void* skip = nullptr;
  const void* z = nullptr;
  const void* bias = nullptr;
  const void* state_in = nullptr;
  const int32_t* cu = nullptr;
  void* y = nullptr;
  void* state_out = nullptr;
  void* ckpt = nullptr;  // states before every ssm_ck-th token, [slot][N][D] par
  const void* dy = nullptr;
  const void* dstate_out = nullptr;
  void* dx = nullptr;
  void* ddt = nullptr;
  void* dA = nullptr;
  void* dB = nullptr;
  void* dC = nullptr;
  void* dskip = nullptr;
  void* dz = nullptr;
  void* dbias = nullptr;
  void* dstate_in = nullptr;
  void* part_bc = nullptr;   // backward: sums over a work-group's channels (k_ssm_bwd.hip)
  void* part_par = nullptr;  // backward: [sequence][N + 2][D], sums over a sequence: dA, dskip, dbias
  const int32_t* slots = nullptr;
  int64_t n_slots = 0;
  int64_t N = 0, B = 0, T = 0;  // sequences, batch, tokens
  int D = 0, Ns = 0, G = 0;     // channels, states, groups
  bool packed = false, softplus = false;
  bool vec_bc = false;          // rows of B and C in vectors of 16 bytes (set by the launchers)
  Rows sx{}, sdt{}, sz{}, sB{}, sC{}, sy{};
  Rows sdy{}, sdx{}, sddt{}, sdz{}, sdB{}, sdC{};
};
inline int64_t ssm_blocks(const SsmArgs& a, int CH) {
  const int dg = a.D / a.G;
  return static_cast<int64_t>((dg + CH - 1) / CH) * a.G;
}
// Channels a work-group and tokens a slot; tiles are of 8 * 64 / channels slots.
constexpr int kSsmWaves = 8;  // of a work-group
struct SsmShape {
  int channels, tokens;
  int tile() const { return tokens * kSsmWaves * (64 / channels); }
  bool fits(const SsmArgs& a) const { return launch_fits(a.N * ssm_blocks(a, channels) * 64 * kSsmWaves); }
};
SsmShape ssm_shape(const SsmArgs& a, int io, int most);
// Those of the backward: at most as many channels as leave the LDS room for N states of
// each (32 to 64 states, 16 to 128, 8 to 256; half these states in fp64), and more than the
// rounds of tiles ask for where the parts of the sums over channels, which are fewer then,
// would take more than 2^30 bytes.  That bounds them only as far as those most channels
// do: 8 * 8192 tokens of 4096 channels and 64 states leave 4 GiB, 4 * 4096 of 2048 and 256
// 8 GiB.  It costs time: one sequence of 2048 channels and 16 states in bf16, 32896 tokens:
// 16 channels 3.25 ms (0.5 GiB), 8 channels 2.10 ms (1.0 GiB); 131072 tokens: 32 channels 20.5 ms
// (1 GiB), 8 channels 8.1 ms (4 GiB).  A forward that trains keeps the states before its tiles.
SsmShape ssm_bwd_shape(int io, const SsmArgs& a);
inline int ssm_ck(int io, const SsmArgs& a) { return ssm_bwd_shape(io, a).tile(); }
size_t ssm_bc_bytes(int io, const SsmArgs& a);
bool ssm_bwd_fits(int io, const SsmArgs& a);
hipError_t launch_ssm_fwd(int io, const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_bwd(int io, const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_step(int io, const SsmArgs& a, hipStream_t s);

// ---- norms around a block
struct AddNormArgs {
  const void* x = nullptr;
  const void* r = nullptr;
  const void* w = nullptr;
  const void* wx = nullptr;
  const void* scale = nullptr;
  void* n = nullptr;
  void* r_out = nullptr;
  const void* dn = nullptr;
  const void* dro = nullptr;
  void* dx = nullptr;
  void* dr = nullptr;
  void* dw[3] = {nullptr, nullptr, nullptr};  // dw, dwx, dscale
  void* part = nullptr;                       // [3][parts][d]
  int64_t B = 0, T = 0;
  int d = 0;
  bool res_f32 = false;  // residual in fp32 with bf16 io
  double eps = 0;
  Rows sx{}, sr{}, sn{}, sro{}, sdn{}, sdro{}, sdx{}, sdr{};
};
int64_t addnorm_parts(const AddNormArgs& a);
hipError_t launch_addnorm_fwd(int io, const AddNormArgs& a, hipStream_t s);
hipError_t launch_addnorm_bwd(int io, const AddNormArgs& a, hipStream_t s);

struct GateNormArgs {
  const void* x = nullptr;
  const void* z = nullptr;
  const void* w = nullptr;
  void* y = nullptr;
  const void* dy = nullptr;
  void* dx = nullptr;
  void* dz = nullptr;
  void* dw = nullptr;
  void* part = nullptr;  // [parts][d], per group if the weights are
  int64_t B = 0, T = 0;
  int G = 0, d = 0;
  bool first = false, group_w = false;
  double eps = 0;
  Rows sx{}, sz{}, sy{}, sdy{}, sdx{}, sdz{};
};
int64_t gatenorm_parts(const GateNormArgs& a);
hipError_t launch_gatenorm_fwd(int io, const GateNormArgs& a, hipStream_t s);
hipError_t launch_gatenorm_bwd(int io, const GateNormArgs& a, hipStream_t s);

// Sums over `rows` rows (none: zeros) of `cols` elements in a fixed order, for each
// z < nz with a place: out[z].p[c * out[z].stride] = sum_r part[z][r][c] (par type).
struct SumOut {
  void* p;
  int64_t stride;
};
constexpr int kMaxSums = 9;
constexpr int kSumCols = 64, kSumRows = 16;  // threads of a work-group
inline bool sums_fit(int64_t cols) { return launch_fits((cols + kSumCols - 1) / kSumCols * (kSumCols * kSumRows)); }
hipError_t launch_sum_rows(int io, const void* part, const SumOut* out, int nz, int64_t rows, int64_t cols,
                           hipStream_t s);

}  // namespace gls
