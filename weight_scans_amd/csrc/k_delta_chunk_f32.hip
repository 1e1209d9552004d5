// k_delta_chunk_f32.hip -- the gated delta rule over the chunks of a sequence in
// fp32, forward.  Per chunk of 64 tokens, with S the state before it and Y, P as
// the bf16 chunks have them:
//
//   R = V - e^l (K S^T),  E = R - Y (beta R),  U = beta E
//   y = scale e^l (Q S^T) + P U,   S <- e^(l_C) S + U^T (e^(l_C - l) K)
//
// All products are v_mfma_f32_16x16x4_f32, whose results chain as operands in
// registers (delta_f32.hpp): a wave carries 16 rows of S through the sequence,
// as in bf16.  Bound by the fp32 matrix rate of the one wave that has a row tile's
// chain (64 x 64: 3.7 us a chunk, 2.2 of them matrix instructions): 4 x 8 x 1024 x
// 64 takes 15 us to prepare and 59 us (token by token: 340).
#include "delta_f32.hpp"
#include "dev_common.hpp"

namespace gls {
namespace {

// Y and P of a chunk: blocks (i, j <= i) of 16 x 16, row 16 i + l in lanes,
// columns 16 j + 4g .. + 3; for training also with column 16 j + l in lanes, rows
// 16 i + 4g .. + 3; and the gates' factors.
template <int DK>
__global__ __launch_bounds__(256) void delta_prep_f32(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16;
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
  const float* kp = static_cast<const float*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + (sr.t0 + t0) * a.sk.t;
  const float* qp = static_cast<const float*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + (sr.t0 + t0) * a.sq.t;
  // rows past the chunk's end and columns past dk read as zeros
  const __amdgpu_buffer_rsrc_t rk = buffer_rsrc(kp, static_cast<int>(((nt - 1) * a.sk.t + a.dk) * 4));
  const __amdgpu_buffer_rsrc_t rq = buffer_rsrc(qp, static_cast<int>(((nt - 1) * a.sq.t + a.dk) * 4));
  const auto row = [&](const __amdgpu_buffer_rsrc_t& r, int64_t st, int tb, int b) {
    const int c = 16 * b + 4 * g;
    return load_f32x4(r, c < a.dk ? static_cast<uint32_t>(((16 * tb + l) * static_cast<int>(st) + c) * 4) : kPastEnd);
  };
  // this wave's rows of K and Q, and row block j of K in turn
  f32x4 kw[NB], qw[NB], kj[2][NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) kw[b] = row(rk, a.sk.t, w, b);
#pragma unroll
  for (int b = 0; b < NB; ++b) kj[0][b] = row(rk, a.sk.t, 0, b);
  float la = 0.f, be = 0.f;
  if (lane < nt) {
    const int64_t o = sr.b * a.sg.b + h * a.sg.h + (sr.t0 + t0 + lane) * a.sg.t;
    la = static_cast<const float*>(a.la)[o];
    be = static_cast<const float*>(a.be)[o];
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) qw[b] = row(rq, a.sq.t, w, b);
  chunk_gate_factors(s, ca.gates + rec * kGates, la, be, false, w, lane);
  lds_barrier();

  const float sc = static_cast<float>(a.scale);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j > w) break;
    if (j < 3) {
#pragma unroll
      for (int b = 0; b < NB; ++b) kj[(j + 1) & 1][b] = row(rk, a.sk.t, j + 1, b);
    }
    f32x4 x = zero4(), xt = zero4(), p = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      x = mul16(kw[b], kj[j & 1][b], x);
      xt = mul16(kj[j & 1][b], kw[b], xt);
      p = mul16(kj[j & 1][b], qw[b], p);
    }
    put_scores(s, w, j, x, xt, lane);
#pragma unroll
    for (int q = 0; q < 4; ++q) p[q] *= sc * s.decay(16 * w + l, 16 * j + 4 * g + q, false);
    *reinterpret_cast<f32x4*>(ca.p32 + rec * kY32 + SolveLds::tri(w, j) * 256 + lane * 4) = p;
  }
  if (ca.pt32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < w) continue;
      f32x4 x = zero4();
#pragma unroll
      for (int b = 0; b < NB; ++b) x = mul16(row(rq, a.sq.t, i, b), kw[b], x);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] *= sc * s.decay(16 * i + 4 * g + q, 16 * w + l, false);
      *reinterpret_cast<f32x4*>(ca.pt32 + rec * kY32 + SolveLds::tri(i, w) * 256 + lane * 4) = x;
    }
  }
  invert_diagonal(s, w, lane);
  lds_barrier();
  f32x4 y[4];
  solve_column(s, w, lane, y);
  lds_barrier();  // Lr is free
  turn_column(s, w, lane, y);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i >= w && ca.yt32)
      *reinterpret_cast<f32x4*>(ca.yt32 + rec * kY32 + SolveLds::tri(i, w) * 256 + lane * 4) = y[i];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i >= w)
      *reinterpret_cast<f32x4*>(ca.y32 + rec * kY32 + SolveLds::tri(i, w) * 256 + lane * 4) =
          *reinterpret_cast<const f32x4*>(&s.Lr[SolveLds::tri(i, w)][lane * 4]);
}

template <int DK, int NW>
struct F32Lds {
  alignas(16) char k[2][64 * DK * 4];
  alignas(16) float gt[2][192];
  alignas(16) float sx[2][NW][DK * 16];
  alignas(16) float ux[2][NW][64 * 16];
};

// A work-group is NW state waves, NW output waves one chunk behind, and a wave
// that loads the next chunk's K; V, Y, Q and P go straight to registers.
template <int DK, int NW, bool SAVE>
__global__ __launch_bounds__(64 * (2 * NW + 1)) void delta_chunk_f32(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16, VW = 16 * NW;
  __shared__ F32Lds<DK, NW> lds;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (a.dv + VW - 1) / VW;
  int64_t head;
  int tile;
  if (!head_of_block(blockIdx.x, tiles, a.N * a.H, head, tile)) return;
  const int h = static_cast<int>(head % a.H);
  const int64_t n = head / a.H;
  const int hk = h / (a.H / a.Hk), r0 = tile * VW;
  const SeqRange sr = seq_range(a.cu, n, a.T);
  const int nc = static_cast<int>((sr.len + kDeltaChunk - 1) / kDeltaChunk);
  const int64_t slot0 = chunk_slot0(a.cu != nullptr, n, sr.t0, a.T, kDeltaChunk);
  const int64_t rec0 = slot0 * a.H + h;

  if (wave == 2 * NW) {  // ---- loads: K and gates, one chunk ahead
    constexpr int NK = DK / 4;
    const float* kp = static_cast<const float*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
    uint32_t ko[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) ko[i] = tile_off_f32<DK>(i, lane, a.sk.t, a.dk);
    const auto issue = [&](int c) {
      const bool in = c < nc;
      const __amdgpu_buffer_rsrc_t rk = rows_f32(kp, c * 64LL, in ? sr.len : 0, a.sk.t, a.dk);
      const __amdgpu_buffer_rsrc_t rg =
          buffer_rsrc(ca.gates + (in ? (rec0 + static_cast<int64_t>(c) * a.H) * kGates : 0), in ? 768 : 0);
#pragma unroll
      for (int i = 0; i < NK; ++i) dma16(rk, ko[i], lds.k[c & 1] + i * 1024);
#pragma unroll
      for (int i = 0; i < 3; ++i) dma4(rg, (i * 64 + lane) * 4, lds.gt[c & 1] + i * 64);
    };
    issue(0);
    for (int c = 0; c <= nc; ++c) {
      wait_vm<0>();
      lds_barrier();
      if (c < nc) issue(c + 1);  // into the slot of chunk c - 1
    }
    wait_vm<0>();
    return;
  }

  if (wave >= NW) {  // ---- outputs, one chunk behind
    const int w = wave - NW;
    const int rr = r0 + 16 * w + 4 * g, rt = tile * NW + w, n_rt = delta_row_tiles(a.dv);
    float* yp = static_cast<float*>(a.y) + sr.b * a.sy.b + h * a.sy.h + sr.t0 * a.sy.t + rr;
    const float* qp = static_cast<const float*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
    const float sc = static_cast<float>(a.scale);
    uint32_t qo[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      qo[b] = 16 * b + 4 * g < a.dk ? static_cast<uint32_t>((l * static_cast<int>(a.sq.t) + 16 * b + 4 * g) * 4)
                                    : kPastEnd;
    f32x4 qf[4][NB], pf[10];
    float gs[4];
    const auto fetch = [&](int c) {
      const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
      const __amdgpu_buffer_rsrc_t rq = rows_f32(qp, c * 64LL, sr.len, a.sq.t, a.dk);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          qf[tb][b] = load_f32x4(rq, qo[b] + static_cast<uint32_t>(tb * 64 * static_cast<int>(a.sq.t)));
#pragma unroll
      for (int f = 0; f < 10; ++f) pf[f] = *reinterpret_cast<const f32x4*>(ca.p32 + rec * kY32 + f * 256 + lane * 4);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) gs[tb] = ca.gates[rec * kGates + 16 * tb + l];
    };
    if (nc > 0) fetch(0);
    lds_barrier();
    for (int c = 0; c < nc; ++c) {
      lds_barrier();
      const float* sx = lds.sx[c & 1][w] + lane * 4;
      const float* ux = lds.ux[c & 1][w] + lane * 4;
      f32x4 o[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) o[tb] = zero4();
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4 sf = *reinterpret_cast<const f32x4*>(sx + b * 256);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int tb = 0; tb < 4; ++tb) o[tb] = mfma_f32(sf[q], qf[tb][b][q], o[tb]);
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const float f = sc * gs[tb];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[tb][q] *= f;
      }
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        const f32x4 uf = *reinterpret_cast<const f32x4*>(ux + jb * 256);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int tb = jb; tb < 4; ++tb) o[tb] = mfma_f32(uf[q], pf[SolveLds::tri(tb, jb)][q], o[tb]);
      }
      fetch(min(c + 1, nc - 1));
      if constexpr (SAVE) {
        const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
#pragma unroll
        for (int b = 0; b < NB; ++b)
          *reinterpret_cast<f32x4*>(ca.s32 + ((rec * n_rt + rt) * NB + b) * 256 + lane * 4) =
              turned_f32(lds.sx[c & 1][w] + b * 256, lane);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
          *reinterpret_cast<f32x4*>(ca.yb + (rec * 64 + 16 * tb + l) * (16 * n_rt) + rr) = o[tb];
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const int64_t t = 64LL * c + 16 * tb + l;
        if (a.y && t < sr.len && rr < a.dv) *reinterpret_cast<f32x4*>(yp + t * a.sy.t) = o[tb];
      }
    }
    return;
  }

  // ---- states
  const int r = r0 + 16 * wave + l;
  const int64_t so = (head * a.dv + r) * a.dk;
  const __amdgpu_buffer_rsrc_t first = state_rsrc(
      a.state_in ? static_cast<const float*>(a.state_in) + head * a.dv * a.dk : nullptr, a.dv, a.dk);
  f32x4 S[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) S[b] = load_f32x4(first, state_off(r, 16 * b + 4 * g, a.dk));
  const float* vp = static_cast<const float*>(a.v) + sr.b * a.sv.b + h * a.sv.h + sr.t0 * a.sv.t;
  uint32_t vo[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    vo[q] = r < a.dv ? static_cast<uint32_t>(((4 * g + q) * static_cast<int>(a.sv.t) + r) * 4) : kPastEnd;
  f32x4 V[4], yf[10];
  const auto fetch = [&](int c) {
    const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
    const __amdgpu_buffer_rsrc_t rv = rows_f32(vp, c * 64LL, sr.len, a.sv.t, a.dv);
#pragma unroll
    for (int tb = 0; tb < 4; ++tb)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        V[tb][q] = load4(rv, vo[q] + static_cast<uint32_t>(tb * 64 * static_cast<int>(a.sv.t)));
#pragma unroll
    for (int f = 0; f < 10; ++f) yf[f] = *reinterpret_cast<const f32x4*>(ca.y32 + rec * kY32 + f * 256 + lane * 4);
  };
  if (nc > 0) fetch(0);
  const uint32_t ka = row_at<DK>(lane);
  const uint32_t kc[4] = {col_at<DK>(lane, 0), col_at<DK>(lane, 1), col_at<DK>(lane, 2), col_at<DK>(lane, 3)};
  for (int c = 0; c < nc; ++c) {
    lds_barrier();
    const char* kt = lds.k[c & 1];
    const float* gt = lds.gt[c & 1] + 4 * g;
    const auto gate = [&](int m, int tb) { return *reinterpret_cast<const f32x4*>(gt + 64 * m + 16 * tb); };
    float* sx = lds.sx[c & 1][wave] + lane * 4;
    float* ux = lds.ux[c & 1][wave] + lane * 4;
    f32x4 E[4], Z[4], be[4];
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) E[tb] = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f32x4 kf[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) kf[tb] = row_frag<DK>(kt, ka, tb, b);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) E[tb] = mfma_f32(kf[tb][q], S[b][q], E[tb]);
      *reinterpret_cast<f32x4*>(sx + b * 256) = S[b];  // for the output wave
    }
    const float whole = lds.gt[c & 1][63];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) S[b][q] *= whole;
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      const f32x4 gm = gate(0, tb);
      be[tb] = gate(1, tb);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        E[tb][q] = fmaf(-gm[q], E[tb][q], V[tb][q]);
        Z[tb][q] = -be[tb][q] * E[tb][q];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = j; i < 4; ++i) E[i] = mfma_f32(yf[SolveLds::tri(i, j)][q], Z[j][q], E[i]);
    fetch(min(c + 1, nc - 1));
    if constexpr (SAVE) {
      const int VP = 16 * delta_row_tiles(a.dv);
      const __amdgpu_buffer_rsrc_t re =
          buffer_rsrc(ca.e32 + (rec0 + static_cast<int64_t>(c) * a.H) * 64 * VP, 256 * VP);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) store_rows(re, static_cast<uint32_t>((4 * g * VP + r) * 4), VP, tb, E[tb]);
    }
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      const f32x4 rs = gate(2, tb);
#pragma unroll
      for (int q = 0; q < 4; ++q) E[tb][q] *= be[tb][q];
      *reinterpret_cast<f32x4*>(ux + tb * 256) = E[tb];
#pragma unroll
      for (int q = 0; q < 4; ++q) E[tb][q] *= rs[q];
    }
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      f32x4 kf[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) kf[b] = col_frag<DK>(kt, kc, tb, b);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int b = 0; b < NB; ++b) S[b] = mfma_f32(kf[b][q], E[tb][q], S[b]);
    }
  }
  lds_barrier();
  if (r < a.dv) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int c = 16 * b + 4 * g;
      if (c >= a.dk) continue;
      if (a.state_out) *reinterpret_cast<f32x4*>(static_cast<float*>(a.state_out) + so + c) = S[b];
      if constexpr (SAVE) *reinterpret_cast<f32x4*>(ca.st + so + c) = S[b];
    }
  }
}

template <int DK, int NW>
hipError_t launch(const ChunkArgs& c, hipStream_t s) {
  const int64_t n = c.slots * c.a.H;
  if (n > 0) {
    delta_prep_f32<DK><<<dim3(static_cast<unsigned>(n)), 256, 0, s>>>(c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int tiles = (c.a.dv + 16 * NW - 1) / (16 * NW);
  const dim3 grid(static_cast<unsigned>(head_blocks(c.a.N * c.a.H, tiles)));
  if (c.s32) delta_chunk_f32<DK, NW, true><<<grid, 64 * (2 * NW + 1), 0, s>>>(c);
  else delta_chunk_f32<DK, NW, false><<<grid, 64 * (2 * NW + 1), 0, s>>>(c);
  return hipGetLastError();
}

}  // namespace

bool delta_rows_f32_ok(const Str3& s, int d) {
  constexpr int64_t most = 1 << 22;  // 64 rows within the 2 GiB of a buffer
  return s.b % 4 == 0 && s.h % 4 == 0 && s.t % 4 == 0 && s.t >= d && s.t < most;
}

bool delta_chunk_f32_ok(int io, const DeltaArgs& a) {
  return io == IO_F32 && a.dk % 4 == 0 && a.dv % 4 == 0 && delta_rows_f32_ok(a.sq, a.dk) &&
         delta_rows_f32_ok(a.sk, a.dk) && delta_rows_f32_ok(a.sv, a.dv);
}

hipError_t launch_delta_chunk_f32(const ChunkArgs& c, hipStream_t s) {
  if (c.a.N * c.a.H == 0) return hipSuccess;
  return c.a.dk <= 64 ? launch<64, 2>(c, s) : launch<128, 2>(c, s);
}

}  // namespace gls
