// k_delta_prep.hip -- what a chunk of the gated delta rule is in itself, for all
// chunks in parallel: with l the cumulative log decay of the chunk's 64 tokens,
//
//   L_ij = e^(l_i - l_j) k_i.k_j  (j < i)
//   Y = (I + L beta)^-1 L,  so that  e = r - Y (beta r)  for  r = v - e^l S k
//
// the gates' factors, and for training P_ij = scale e^(l_i - l_j) q_i.k_j
// (j <= i) with rows j.  One work-group of four waves per chunk and value head.  The scores run in both orientations (operands exchanged) on the bf16
// matrix cores, straight from global memory: each orientation is the operand
// form of one later product.  Y in fp32: wave w inverts its 16 x 16 diagonal
// block I + B (B = L beta) by substitution, a column per lane; then wave j
// takes column block j down its rows, Y_ij = N_i (L_ij - sum_k B_ik Y_kj), with
// v_mfma_f32_16x16x4_f32, each result feeding the next product in registers.
//
// The cumulative decay is kept as whole part and fraction (log2): whole parts
// add exactly, so that differences stay exact to 2^-19 however many tokens of
// the chunk forget everything (log_alpha = -inf counts as 2^-200).
//
// Y and P leave as two bf16 terms (16 significand bits), what the recurrences
// multiply.  Bound by these stores and by the solve's chain: training 4 x 16 x
// 4096 x 128 moves 294 MB in 71 us (4.1 TB/s), 8 x 16 x 4096 x 64 454 MB in 96 us
// (4.7; a large copy reaches 5.2).  A wave loads only the row blocks that it
// multiplies, so that three work-groups fit a CU (with all of K and Q: 92 / 119).
#include "delta_solve.hpp"
#include "dev_common.hpp"

namespace gls {
namespace {

constexpr int kThreads = 256;

template <int DK>
__global__ __launch_bounds__(kThreads, 3) void delta_prep(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NS = DK / 32;
  __shared__ SolveLds s;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = static_cast<int>(blockIdx.x % a.H);
  const int64_t slot = blockIdx.x / a.H, rec = slot * a.H + h;
  const int hk = h / (a.H / a.Hk);
  SeqRange sr;
  int64_t t0;
  if (!chunk_of_slot(a, slot, sr, t0)) return;
  const int nt = static_cast<int>(sr.len - t0 < 64 ? sr.len - t0 : 64);

  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + (sr.t0 + t0) * a.sk.t;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + (sr.t0 + t0) * a.sq.t;
  // rows past the chunk's end and columns past dk read as zeros
  // Row blocks 0 .. w of K, then w .. 3 of Q (training only): all that the wave
  // multiplies
  bf16x8 m[5][NS];
  uint32_t at[NS];
#pragma unroll
  for (int c = 0; c < NS; ++c) {
    const int col = 32 * c + 8 * g;
    at[c] = col < a.dk ? static_cast<uint32_t>(col * 2) : kPastEnd;
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const bool k = i <= w, in = k || ca.ptf;
    const __amdgpu_buffer_rsrc_t r = buffer_rsrc(
        k ? kp : qp, in ? static_cast<int>(((nt - 1) * (k ? a.sk.t : a.sq.t) + a.dk) * 2) : 0);
    const uint32_t o = (16 * (k ? i : i - 1) + l) * static_cast<uint32_t>(k ? a.sk.t : a.sq.t) * 2;
#pragma unroll
    for (int c = 0; c < NS; ++c) m[i][c] = load16(r, at[c] + o);
  }
  float la = 0.f, be = 0.f;
  if (lane < nt) {
    const int64_t o = sr.b * a.sg.b + h * a.sg.h + (sr.t0 + t0 + lane) * a.sg.t;
    la = a.gate_io ? bf16_to_f32(static_cast<const uint16_t*>(a.la)[o]) : static_cast<const float*>(a.la)[o];
    be = a.gate_io ? bf16_to_f32(static_cast<const uint16_t*>(a.be)[o]) : static_cast<const float*>(a.be)[o];
  }
  chunk_gate_factors(s, ca.gates + rec * kGates, la, be, ca.ytf != nullptr, w, lane);
  lds_barrier();

  const auto put = [&](uint16_t* dst, const bf16x8& f) {
    *reinterpret_cast<bf16x8*>(dst + lane * 8) = f;
  };
  const auto put2 = [&](uint16_t* dst, int f, const f32x4& u, const f32x4& v) {
    const Pair8 p = split8(u, v);
    put(dst + (2 * f) * kFrag, p.hi);
    put(dst + (2 * f + 1) * kFrag, p.lo);
  };
  // L: row block w, in both orientations; for training P's column block w (rows j
  // in lanes)
  const float sc = static_cast<float>(a.scale);
#pragma unroll
  for (int wc = 0; wc < 4; ++wc) {
    if (wc != w) continue;
    const auto& kw = m[wc];
#pragma unroll
    for (int j = 0; j <= wc; ++j) {
      f32x4 x = zero4(), xt = zero4();
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        x = mfma16x16x32(kw[c], m[j][c], x);
        xt = mfma16x16x32(m[j][c], kw[c], xt);
      }
      put_scores(s, wc, j, x, xt, lane);
    }
    if (ca.ptf) {
      f32x4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = zero4();
        if (i < wc) continue;
#pragma unroll
        for (int c = 0; c < NS; ++c) p[i] = mfma16x16x32(m[i + 1][c], kw[c], p[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) p[i][q] *= sc * s.decay(16 * i + 4 * g + q, 16 * wc + l, false);
      }
#pragma unroll
      for (int c = wc / 2; c < 2; ++c) put2(ca.ptf + rec * kYf, wc < 2 ? 2 * wc + c : wc + 2, p[2 * c], p[2 * c + 1]);
    }
  }
  invert_diagonal(s, w, lane);
  lds_barrier();
  f32x4 y[4];
  solve_column(s, w, lane, y);
  lds_barrier();  // Lr is free
  if (ca.ytf) {  // rows j = this wave's columns: the results as they are
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (c < w / 2) continue;
      put2(ca.ytf + rec * kYf, w < 2 ? 2 * w + c : w + 2, y[2 * c], y[2 * c + 1]);
    }
  }
  turn_column(s, w, lane, y);
  lds_barrier();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (c > w / 2) continue;
    const f32x4 u = *reinterpret_cast<const f32x4*>(&s.Lr[SolveLds::tri(w, 2 * c)][lane * 4]);
    const f32x4 v =
        2 * c + 1 <= w ? *reinterpret_cast<const f32x4*>(&s.Lr[SolveLds::tri(w, 2 * c + 1)][lane * 4]) : zero4();
    put2(ca.yf + rec * kYf, w < 2 ? w : 2 * w - 2 + c, u, v);
  }
}

}  // namespace

bool delta_rows_ok(const Str3& s, int d) {
  constexpr int64_t most = 1 << 23;  // 64 rows within the 2 GiB of a buffer
  return s.b % 8 == 0 && s.h % 8 == 0 && s.t % 8 == 0 && s.t >= d && s.t < most;
}

bool delta_chunk_ok(int io, const DeltaArgs& a) {
  return io == IO_BF16 && a.dk % 8 == 0 && a.dv % 8 == 0 && delta_rows_ok(a.sq, a.dk) &&
         delta_rows_ok(a.sk, a.dk) && delta_rows_ok(a.sv, a.dv);
}

hipError_t launch_delta_prep(const ChunkArgs& c, hipStream_t s) {
  const int64_t n = c.slots * c.a.H;
  if (n == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(n));
  if (c.a.dk <= 64) delta_prep<64><<<grid, kThreads, 0, s>>>(c);
  else delta_prep<128><<<grid, kThreads, 0, s>>>(c);
  return hipGetLastError();
}

}  // namespace gls
