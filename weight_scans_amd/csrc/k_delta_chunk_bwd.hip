// k_delta_chunk_bwd.hip -- the gated delta rule's gradients over chunks (bf16 on
// the matrix cores), from what the forward left.  With Lam the adjoint of the
// state after the chunk:
//
//   dU = P^T dO + e^(l_C - l) (K Lam^T),  G = dU - Y^T (beta dU),  F = beta G
//   Lam <- e^(l_C) Lam + (scale e^l dO)^T Q - (e^l F)^T K
//
// is again a recurrence of independent rows (delta_chunk_rev, the mirror of the
// forward kernel: state waves with Lam^T in their accumulators; helper waves
// form the two products with dO one chunk ahead and hand them over in fp32).  As
// there the chain of a chunk in one wave bounds it, 3.4 us a step at 128 x 128:
// 4 x 16 x 4096 x 128 takes 222 us (860 MB, 3.9 TB/s), 8 x 16 x 4096 x 64 190 us (898
// MB, 4.7 TB/s: near what a copy reaches).  P^T is read, not formed here: the
// helpers would outlast the state waves (before dv left here too: 205 and 175 us, so
// 252 and 207).  Segments as in the forward, from the right: Lam_begin = Lam_end M^T +
// Z, with M the forward's (1 x 16 x 32768 x 128: the whole backward 952 us in four,
// 1588 in one).
//
// The rest is one work-group per chunk and key head (delta_chunk_grad):
//
//   dq = scale e^l dO S + dP K,              dP_ij = scale D_ij beta_j dO_i.e_j  (j <= i)
//   dk = beta (e^(l_C - l) E Lam - e^l G S) + dP^T Q - (H + H^T) K,
//                                            H_ij = D_ij beta_i beta_j G_i.e_j   (j < i)
//   D_ij = e^(l_i - l_j)
//
// and dv = beta G leaves the recurrence, rounded once from its fp32 (from the bf16 G
// that the gradients take it was 2.4e-3 off instead of 1.7e-3).
//
// The decay's gradient is dlog_alpha_t = <dL/dS_{t-1}, S_{t-1}>.  Scaling a row
// of S and of v together scales that row of y, so this product changes from
// token to token only by dy.y - dv.v (Euler), row by row:
//   dlog_alpha_t = <dL/dS_T, S_T> + sum_{s >= t} (dy_s.y_s - dv_s.v_s).
// The sum runs over the whole sequence while its value stays a few tokens'
// terms in size, so its terms must not be rounded to bf16: the reverse
// recurrence forms dv.v from its fp32 accumulators and dy.y from the forward's
// fp32 y, and carries the sum for its 16 rows.  (The same gradient from the
// rounded states and e, as the sum of the flows past token t, has no long sum,
// but the rounding of each flow left errors of up to 7e-3.  It is what tokens that keep
// little of the state get, where the difference of the terms is lost in their own
// rounding: delta_chunk_decay.)  dbeta = G.e is formed there too, from the fp32 G and
// the rounded e.
#include "delta_solve.hpp"
#include "dev_common.hpp"

namespace gls {
namespace {

template <int DK, int NW>
struct RevLds {
  static constexpr int NS = DK / 32, NB = DK / 16, VW = 16 * NW;
  alignas(16) char k[3][64 * DK * 2];
  alignas(16) char q[3][64 * DK * 2];
  alignas(16) char o[3][64 * VW * 2];
  alignas(16) char v[3][64 * VW * 2];
  alignas(16) float gt[4][192];
  float dyy[NW][3][64], vdv[NW][2][64];   // dy.y, v.dv over the wave's rows
  alignas(16) float x1[NW][4 * 256];      // P^T dO
  alignas(16) float x2[NW][NB * 256];     // (scale e^l dO)^T Q
  alignas(16) uint16_t turn[NW][NS * kFrag];
};

// STATES: only what segments 1 .. n_seg - 1 do to an adjoint of zero.
template <int DK, int NW, bool STATES>
__global__ __launch_bounds__(64 * (2 * NW + 2)) void delta_chunk_rev(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NS = DK / 32, NB = DK / 16, VW = 16 * NW;
  __shared__ RevLds<DK, NW> lds;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (a.dv + VW - 1) / VW;
  int64_t head;
  int tile;
  const int runs = STATES ? ca.n_seg - 1 : ca.n_seg;
  if (!head_of_block(blockIdx.x, tiles, a.N * a.H * runs, head, tile)) return;
  const int seg = static_cast<int>(static_cast<uint32_t>(head) % static_cast<uint32_t>(runs)) + (STATES ? 1 : 0);
  head = static_cast<uint32_t>(head) / static_cast<uint32_t>(runs);
  const bool last = seg == ca.n_seg - 1;
  const int h = static_cast<int>(head % a.H);
  const int64_t n = head / a.H;
  const int hk = h / (a.H / a.Hk), r0 = tile * VW;
  SeqRange sr = seq_range(a.cu, n, a.T);
  int64_t slot0 = chunk_slot0(a.cu != nullptr, n, sr.t0, a.T, kDeltaChunk);
  const int nc = segment_of(sr, slot0, seg, ca.n_seg);
  const int64_t rec0 = slot0 * a.H + h;
  // the adjoint after the last chunk and the state there
  const int64_t dd = static_cast<int64_t>(a.dv) * a.dk;
  // (in segments the call's last adjoint too comes from seg_l, where the STATES pass
  // leaves it: the first segment writes dstate_in, which may be the same memory)
  float* seg_l = ca.seg_l + (head * ca.n_seg + seg) * dd;
  const float* given = last && a.dstate_out ? static_cast<const float*>(a.dstate_out) + head * dd : nullptr;
  const float* lam_end = last     ? (given && !STATES && ca.n_seg > 1 ? seg_l : given)
                         : STATES ? nullptr
                                  : seg_l;
  const float* state_end = last ? ca.st + head * dd : ca.seg_s + (head * ca.n_seg + seg + 1) * dd;

  // Step i: the helpers take chunk nc - 1 - i, the state waves the one before
  // (nc - i), and the helpers finish the decay's gradient of the one before
  // that.  Barrier A begins the step; between A and B the state waves take the
  // helpers' results of the step before, after B they may be overwritten.
  if (wave == 2 * NW) {  // ---- loads for the helpers: Q, dO; gates and V
    constexpr int NK = DK / 8, NV = VW / 8, PER = NK + 2 * NV + 3;
    const uint16_t* vp = static_cast<const uint16_t*>(a.v) + sr.b * a.sv.b + h * a.sv.h + sr.t0 * a.sv.t + r0;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
    const uint16_t* op = static_cast<const uint16_t*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t + r0;
    uint32_t qo[NK], oo[NV], vo[NV];
#pragma unroll
    for (int i = 0; i < NK; ++i) qo[i] = tile_off<DK>(i, lane, a.sq.t, 0, a.dk);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      oo[i] = tile_off<VW>(i, lane, a.sdy.t, 0, a.dv - r0);
      vo[i] = tile_off<VW>(i, lane, a.sv.t, 0, a.dv - r0);
    }
    const auto issue = [&](int i) {
      const int c = nc - 1 - i, s = i % 3;
      const bool in = c >= 0;
      const __amdgpu_buffer_rsrc_t rq = rows_rsrc(qp, in ? c * 64LL : 0, in ? sr.len : 0, a.sq.t, a.dk);
      const __amdgpu_buffer_rsrc_t ro = rows_rsrc(op, in ? c * 64LL : 0, in ? sr.len : 0, a.sdy.t, min(VW, a.dv - r0));
      const __amdgpu_buffer_rsrc_t rv = rows_rsrc(vp, in ? c * 64LL : 0, in ? sr.len : 0, a.sv.t, min(VW, a.dv - r0));
      const __amdgpu_buffer_rsrc_t rg =
          buffer_rsrc(ca.gates + (in ? (rec0 + static_cast<int64_t>(c) * a.H) * kGates : 0), in ? 768 : 0);
#pragma unroll
      for (int j = 0; j < NK; ++j) dma16(rq, qo[j], lds.q[s] + j * 1024);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        dma16(ro, oo[j], lds.o[s] + j * 1024);
        dma16(rv, vo[j], lds.v[s] + j * 1024);
      }
#pragma unroll
      for (int j = 0; j < 3; ++j) dma4(rg, (j * 64 + lane) * 4, lds.gt[i & 3] + j * 64);
    };
    issue(0);
    issue(1);
    for (int i = 0; i <= nc + 1; ++i) {
      wait_vm<PER>();
      lds_barrier();
      lds_barrier();
      // slot (i + 2) % 3 held index i - 1: its Q and dO are done with, and its V
      // was read by the state waves between A and B of this step (gates: four
      // slots, index i - 2's is done with)
      issue(i + 2);
    }
    wait_vm<0>();
    return;
  }
  if (wave == 2 * NW + 1) {  // ---- loads for the state waves: K
    constexpr int NK = DK / 8;
    const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
    uint32_t ko[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) ko[i] = tile_off<DK>(i, lane, a.sk.t, 0, a.dk);
    const auto issue = [&](int i) {  // index i is used in step i + 1
      const int c = nc - 1 - i;
      const __amdgpu_buffer_rsrc_t rk = rows_rsrc(kp, c >= 0 ? c * 64LL : 0, c >= 0 ? sr.len : 0, a.sk.t, a.dk);
#pragma unroll
      for (int j = 0; j < NK; ++j) dma16(rk, ko[j], lds.k[i % 3] + j * 1024);
    };
    issue(0);
    lds_barrier();
    lds_barrier();
    issue(1);
    for (int i = 1; i <= nc + 1; ++i) {
      wait_vm<NK>();  // index i - 1 is there
      lds_barrier();
      lds_barrier();
      issue(i + 1);   // into the slot of index i - 2
    }
    wait_vm<0>();
    return;
  }

  const TileLane<DK> tk = tile_lane<DK>(lane);
  if (wave >= NW) {  // ---- helpers: the products with dO
    const int w = wave - NW;
    const TileLane<VW> to = tile_lane<VW>(lane);
    const float sc = static_cast<float>(a.scale);
    const int rt = tile * NW + w, n_rt = delta_row_tiles(a.dv);
    bf16x8 pf[12];
    f32x4 yb[4];
    const auto fetch = [&](int c) {
      const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
      const uint16_t* p = ca.ptf + rec * kYf + lane * 8;
#pragma unroll
      for (int f = 0; f < 12; ++f) pf[f] = *reinterpret_cast<const bf16x8*>(p + f * kFrag);
      if constexpr (!STATES)
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
          yb[tb] = *reinterpret_cast<const f32x4*>(ca.yb + ((rec * n_rt + rt) * 4 + tb) * 256 + lane * 4);
    };
    if (nc > 0) fetch(nc - 1);
    float z = 0.f;  // <dL/dS, S> after the chunk, over this wave's rows
    if (!STATES && lam_end) {
      const __amdgpu_buffer_rsrc_t ru = state_rsrc(lam_end, a.dv, a.dk), rs = state_rsrc(state_end, a.dv, a.dk);
      f32x4 u[NB], s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t o = state_off(r0 + index1(w, l), index4(b, g), a.dk);
        u[b] = load_f32x4(ru, o);
        s[b] = load_f32x4(rs, o);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) z = fmaf(u[b][q], s[b][q], z);
    }
    z = wave_sum(z);
    wait_vm<0>();  // dstate_in may be dstate_out
    float lw = 0.f;
    for (int i = 0; i <= nc + 1; ++i) {
      lds_barrier();  // A
      lds_barrier();  // B: the results of the step before have been taken
      if (!STATES && i >= 2) {
        const int64_t rec = rec0 + static_cast<int64_t>(nc + 1 - i) * a.H;
        const float x = lds.dyy[w][(i - 2) % 3][lane] - lds.vdv[w][i & 1][lane];
        const float y = decay_sum(wave_reverse(x, lane), z, tokens_below(lw, kForget), lane);
        ca.zf[(rec * n_rt + rt) * 64 + 63 - lane] = y;
        z = readlane_f(y, 63);
      }
      f32x4 x1[4], x2[NB];
      if (i < nc) {
        const int sl = i % 3;
        if constexpr (!STATES)
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {  // dy.y: token 16 tb + l
          const f32x4 d = widen(row4<VW>(lds.o[sl], to, tb, w));
          const float x = sum_rows((d[0] * yb[tb][0] + d[1] * yb[tb][1]) + (d[2] * yb[tb][2] + d[3] * yb[tb][3]));
          if (g == 0) lds.dyy[w][i % 3][16 * tb + l] = x;
        }
        s16x4 o[4];
        f32x4 d[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          o[tb] = col4<VW>(lds.o[sl], to, tb, w);
          d[tb] = widen(o[tb]);
          const f32x4 gm = *reinterpret_cast<const f32x4*>(&lds.gt[i & 3][16 * tb + 4 * g]);
#pragma unroll
          for (int q = 0; q < 4; ++q) d[tb][q] *= sc * gm[q];
          x1[tb] = zero4();
        }
        const bf16x8 o0 = join(o[0], o[1]), o1 = join(o[2], o[3]);
#pragma unroll
        for (int jb = 0; jb < 4; ++jb)
#pragma unroll
          for (int s = jb / 2; s < 2; ++s) {
            const int f = jb < 2 ? 2 * jb + s : jb + 2;
            x1[jb] = mfma16x16x32(pf[2 * f + 1], s ? o1 : o0, x1[jb]);
            x1[jb] = mfma16x16x32(pf[2 * f], s ? o1 : o0, x1[jb]);
          }
        if (i + 1 < nc) fetch(nc - 2 - i);
        const Pair8 d0 = split8(d[0], d[1]), d1 = split8(d[2], d[3]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const bf16x8 q0 = frag_c<DK>(lds.q[sl], tk, 0, b), q1 = frag_c<DK>(lds.q[sl], tk, 1, b);
          x2[b] = mfma16x16x32(q0, d0.hi, zero4());
          x2[b] = mfma16x16x32(q0, d0.lo, x2[b]);
          x2[b] = mfma16x16x32(q1, d1.hi, x2[b]);
          x2[b] = mfma16x16x32(q1, d1.lo, x2[b]);
        }
      }
      if (i < nc) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) *reinterpret_cast<f32x4*>(&lds.x1[w][tb * 256 + lane * 4]) = x1[tb];
#pragma unroll
        for (int b = 0; b < NB; ++b) *reinterpret_cast<f32x4*>(&lds.x2[w][b * 256 + lane * 4]) = x2[b];
      }
      if (!STATES && i >= 1 && i <= nc)  // the decay of the chunk whose sum the next step takes
        lw = ca.gates[(rec0 + static_cast<int64_t>(nc - i) * a.H) * kGates + 192 + lane];
    }
    return;
  }

  // ---- adjoint states
  const TileLane<VW> tv = tile_lane<VW>(lane);
  const int r = r0 + index1(wave, l);
  const __amdgpu_buffer_rsrc_t first = state_rsrc(lam_end, a.dv, a.dk);
  f32x4 S[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) S[b] = load_f32x4(first, state_off(r, index4(b, g), a.dk));
  if (STATES && given && r < a.dv) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (index4(b, g) < a.dk)
        *reinterpret_cast<f32x4*>(seg_l + static_cast<int64_t>(r) * a.dk + index4(b, g)) = S[b];
  }
  bf16x8 yf[12], ef[2];
  const int rt = tile * NW + wave, n_rt = delta_row_tiles(a.dv);
  const auto fetch = [&](int c) {
    const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
    const uint16_t* p = ca.ytf + rec * kYf + lane * 8;
#pragma unroll
    for (int f = 0; f < 12; ++f) yf[f] = *reinterpret_cast<const bf16x8*>(p + f * kFrag);
  };
  const auto fetch_e = [&](int c) {
    if constexpr (STATES) return;
    const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      ef[s] = *reinterpret_cast<const bf16x8*>(ca.ef + ((rec * n_rt + rt) * 2 + s) * kFrag + raw_at(lane));
  };
  if (nc > 0) {
    fetch(nc - 1);
    fetch_e(nc - 1);
  }
  Pair8 sp[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) sp[s] = split8(S[2 * s], S[2 * s + 1]);
  uint16_t* turn = lds.turn[wave];
  // dv: rows index4(wave, g) .. + 3 of token l of a block
  uint16_t* dvp = static_cast<uint16_t*>(a.dv_) + sr.b * a.sdv.b + h * a.sdv.h + sr.t0 * a.sdv.t + r0;
  const uint32_t dvo = r0 + index4(wave, g) < a.dv ? static_cast<uint32_t>((l * a.sdv.t + index4(wave, g)) * 2) : kPastEnd;
  lds_barrier();
  lds_barrier();
  for (int i = 1; i <= nc; ++i) {
    const int c = nc - i;
    const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
    if constexpr (!STATES)
#pragma unroll
      for (int s = 0; s < NS; ++s) *reinterpret_cast<bf16x8*>(&turn[s * kFrag + lane * 8]) = sp[s].hi;
    lds_barrier();  // A
    const int sl = (i - 1) % 3;
    const char* kt = lds.k[sl];
    const float* gt = lds.gt[(i - 1) & 3];
    const auto gate = [&](int m, int tb) { return *reinterpret_cast<const f32x4*>(gt + 64 * m + 16 * tb + 4 * g); };
    f32x4 x1[4], x2[NB], G[4], x[4];
    s16x4 vv[4];
    bf16x8 kf[2][NS], kc[NB], gf[2], lf[NB / 2];
    Pair8 z[2], u;
    float xe[16], yv[16];
    const auto read_k = [&](int half) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int s = 0; s < NS; ++s) kf[i][s] = frag_n<DK>(kt, tk, 2 * half + i, s);
    };
    const auto ks = [&](int half) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          G[2 * half + i] = mfma16x16x32(kf[i][s], sp[s].hi, s ? G[2 * half + i] : zero4());
          G[2 * half + i] = mfma16x16x32(kf[i][s], sp[s].lo, G[2 * half + i]);
        }
    };
    // dU, and the operand beta dU
    const auto residual = [&](int half) {
      f32x4 Z[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tb = 2 * half + i;
        const f32x4 rs = gate(2, tb), be = gate(1, tb);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          G[tb][q] = fmaf(rs[q], G[tb][q], x1[tb][q]);
          Z[i][q] = be[q] * G[tb][q];
        }
      }
      z[half] = split8(Z[0], Z[1]);
    };
    // Y^T (beta dU): tokens of the first half also take the second's
    const auto solve = [&](int half) {
#pragma unroll
      for (int s = 1; s >= half; --s)
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int jb = 2 * half + i, f = half ? jb + 2 : 2 * jb + s;
            x[jb] = mfma16x16x32(yf[2 * f + (m == 0)], m == 1 ? z[s].lo : z[s].hi, m || s == 0 ? x[jb] : zero4());
          }
    };
    // G, its products with e and v, and the operand -e^l F
    const auto errors = [&](int half) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) G[2 * half + i][q] -= x[2 * half + i][q];
      if constexpr (!STATES) gf[half] = raw_order(round8(G[2 * half], G[2 * half + 1]), lane);
      const s16x8 e = STATES ? s16x8{} : __builtin_bit_cast(s16x8, raw_order(ef[half], lane));
      const f32x4 ee[2] = {widen(__builtin_shufflevector(e, e, 0, 1, 2, 3)), widen(__builtin_shufflevector(e, e, 4, 5, 6, 7))};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tb = 2 * half + i;
        const f32x4 v = widen(vv[tb]), be = gate(1, tb);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (!STATES) xe[4 * tb + q] = G[tb][q] * ee[i][q];
          G[tb][q] *= be[q];
          if constexpr (!STATES) yv[4 * tb + q] = v[q] * G[tb][q];
        }
      }
      // dv, rounded once: to be turned to rows of tokens
      if constexpr (!STATES)
        *reinterpret_cast<bf16x8*>(&turn[half * kFrag + lane * 8]) = round8(G[2 * half], G[2 * half + 1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x4 gm = gate(0, 2 * half + i);
#pragma unroll
        for (int q = 0; q < 4; ++q) G[2 * half + i][q] *= -gm[q];
      }
      u = split8(G[2 * half], G[2 * half + 1]);
    };
    const auto read_kc = [&](int half) {
#pragma unroll
      for (int b = 0; b < NB; ++b) kc[b] = frag_c<DK>(kt, tk, half, b);
    };

#pragma unroll
    for (int b = 0; b < NB; ++b) x2[b] = *reinterpret_cast<const f32x4*>(&lds.x2[wave][b * 256 + lane * 4]);
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      vv[tb] = col4<VW>(lds.v[sl], tv, tb, wave);
      x1[tb] = *reinterpret_cast<const f32x4*>(&lds.x1[wave][tb * 256 + lane * 4]);
    }
    const float whole = gt[63];
    read_k(1);
    lds_barrier();  // B
    if constexpr (!STATES)
#pragma unroll
      for (int b = 0; b < NB; b += 2) lf[b / 2] = join(turned(turn, b, lane), turned(turn, b + 1, lane));
    ks(1);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) S[b][q] = fmaf(whole, S[b][q], x2[b][q]);
    read_k(0);
    interleave<4 * NS, 1, 2>();
    ks(0);
    residual(1);
    interleave<4 * NS, 1, 40 / (4 * NS)>();
    solve(1);
    residual(0);
    interleave<6, 1, 7>();
    read_kc(1);
    solve(0);
    errors(1);
    interleave<12, 1, 7>();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      S[b] = mfma16x16x32(kc[b], u.hi, S[b]);
      S[b] = mfma16x16x32(kc[b], u.lo, S[b]);
    }
    errors(0);
    interleave<2 * NB, 1, 80 / (2 * NB)>();
    // the next chunk's, before this one's stores (waited for in order of issue)
    fetch(max(c - 1, 0));
    fetch_e(max(c - 1, 0));
    read_kc(0);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      S[b] = mfma16x16x32(kc[b], u.hi, S[b]);
      S[b] = mfma16x16x32(kc[b], u.lo, S[b]);
    }
    const int tok = 16 * (l >> 2) + 4 * g + (l & 3);
    float be_ = 0.f;
    if constexpr (!STATES) {
      be_ = row_sums(xe, l);
      lds.vdv[wave][(i - 1) & 1][tok] = row_sums(yv, l);
    }
    interleave<2 * NB, 1, 96 / (2 * NB)>();
#pragma unroll
    for (int s = 0; s < NS; ++s) sp[s] = split8(S[2 * s], S[2 * s + 1]);
    if constexpr (!STATES) {
#pragma unroll
      for (int b = 0; b < NB; b += 2)
        *reinterpret_cast<bf16x8*>(ca.lf + ((rec * n_rt + rt) * NB + b) * kPiece + lane * 8) = lf[b / 2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        *reinterpret_cast<bf16x8*>(ca.gf + ((rec * n_rt + rt) * 2 + s) * kFrag + raw_at(lane)) = gf[s];
      ca.bf[(rec * n_rt + rt) * 64 + tok] = be_;
      s16x4 dvf[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) dvf[tb] = turned(turn, tb, lane);
      const __amdgpu_buffer_rsrc_t rd = rows_rsrc(dvp, c * 64LL, sr.len, a.sdv.t, min(VW, a.dv - r0));
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
        store8(rd, dvo + static_cast<uint32_t>(tb * 32 * a.sdv.t), __builtin_bit_cast(uint2, dvf[tb]));
    }
  }
  lds_barrier();
  lds_barrier();
  float* to = STATES     ? ca.seg_l + (head * ca.n_seg + seg - 1) * a.dv * a.dk
              : seg == 0 ? static_cast<float*>(a.dstate_in)
                         : nullptr;
  if (to && r < a.dv) {
    to += (STATES ? 0 : head * a.dv * a.dk) + static_cast<int64_t>(r) * a.dk;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (index4(b, g) < a.dk) *reinterpret_cast<f32x4*>(to + index4(b, g)) = S[b];
  }
}

// ---- the gradients of one chunk, for the value heads of one key head in turn
// (their sums stay in registers), on four waves.
//
// Scores: dO e^T and G e^T below the diagonal, each in both orientations (every
// later product wants its operand with another index in lanes), one kind a
// wave, handed on through LDS.  Off the diagonal the decay is a product of two
// factors; on it, exact per element.
//
// Then a wave takes two column blocks of dq and dk (for a share of the tokens
// where there are fewer than eight blocks): operands of tokens (dO, e, G,
// scores) come from LDS and serve both blocks, S and Lam straight from global
// memory.  Loading a chunk's 160 KB (128 x 128) and multiplying take about as
// long: dO, e and G are done with before K and Q are needed, which take their
// place, so that two work-groups fit a CU and one loads while the other
// multiplies.  Bound by HBM: 4 x 16 x 4096 x 128 moves 766 MB in 154 us, 8 x 16 x
// 4096 x 64 642 MB in 129 us, 5.0 TB/s both, what a large copy reaches.  S, Lam, e
// and G were rounded once to bf16 by the recurrences (dq, dk: 3e-3 against 1.7e-3 of
// their own rounding); as two terms each they would add half to that traffic.
template <int DK, int DV>
struct GradLds {
  static constexpr int kCols = 64 * DK * 2;
  union {
    struct {
      alignas(16) char o[64 * DV * 2];
      alignas(16) uint16_t e[64 * DV];
      alignas(16) uint16_t g[64 * DV];
    };
    struct {
      alignas(16) char k[kCols];
      alignas(16) char q[kCols];
    };
  };
  // operand pieces (lane block, contraction block): dP [i][j], dP^T [j][i], and
  // H + H^T with the two halves of its diagonal blocks apart (48.. 51: the other)
  alignas(16) uint16_t sc[52 * kPiece];
  alignas(16) float gt[kGates];
};

constexpr int kGradThreads = 256;

template <int DK, int DV, bool SHARED>
__global__ __launch_bounds__(kGradThreads) __attribute__((amdgpu_waves_per_eu(2))) void
delta_chunk_grad(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16, NP = NB / 2, NT = NP, NR = DV / 32;  // NT blocks of 16 tokens a wave
  __shared__ GradLds<DK, DV> lds;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = static_cast<int>(blockIdx.x % a.Hk), grp = SHARED ? a.H / a.Hk : 1;
  const int64_t slot = blockIdx.x / a.Hk;
  SeqRange sr;
  int64_t t0;
  if (!chunk_of_slot(a, slot, sr, t0)) return;
  const int nt = static_cast<int>(sr.len - t0 < 64 ? sr.len - t0 : 64);
  const int n_rt = delta_row_tiles(a.dv), nr = n_rt / 2;
  const int kb0 = 2 * (w % NP), tb0 = NT * (w / NP);
  const float sc = static_cast<float>(a.scale);
  const s16x4 none = {0, 0, 0, 0};

  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
  f32x4 dq[2][NT], dk[2][NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) dq[0][t] = dq[1][t] = dk[0][t] = dk[1][t] = zero4();

  for (int gi = 0; gi < grp; ++gi) {
    const int h = hk * grp + gi;
    const int64_t rec = slot * a.H + h;
    int lane = threadIdx.x & 63;
    // Anew for each head: addresses kept over the loop cost more registers than there are.
    if constexpr (SHARED) asm volatile("" : "+v"(lane));
    const int l = lane & 15, g = lane >> 4;
    const TileLane<DK> tk = tile_lane<DK>(lane);
    const TileLane<DV> to = tile_lane<DV>(lane);
    const uint32_t ra = raw_turned(lane);
    if (gi) __syncthreads();  // the head before is done with the tiles
    {
      const uint16_t* op = static_cast<const uint16_t*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t;
      const __amdgpu_buffer_rsrc_t ro = rows_rsrc(op, t0, sr.len, a.sdy.t, a.dv);
      const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(ca.gates + rec * kGates, kGates * 4);
      const int eb = n_rt * 2 * kFrag * 2;  // bytes of e's fragments
      const __amdgpu_buffer_rsrc_t re = buffer_rsrc(ca.ef + rec * 2 * n_rt * kFrag, eb);
      const __amdgpu_buffer_rsrc_t rr = buffer_rsrc(ca.gf + rec * 2 * n_rt * kFrag, eb);
      if (w < 3) {
#pragma unroll
        for (int i = 0; i < 3; ++i) dma4(rg, ((3 * w + i) * 64 + lane) * 4, lds.gt + (3 * w + i) * 64);
      }
#pragma unroll
      for (int j = 0; j < DV / 32; ++j) {
        const int i = w * (DV / 32) + j;
        dma16(re, i * 1024 + lane * 16, reinterpret_cast<char*>(lds.e) + i * 1024);
        dma16(ro, tile_off<DV>(i, lane, a.sdy.t, 0, a.dv), lds.o + i * 1024);
        dma16(rr, i * 1024 + lane * 16, reinterpret_cast<char*>(lds.g) + i * 1024);
      }
    }
    // columns of this wave, of Lam and of S
    s16x8 lc[2 * NR], sc_[2 * NR];
    const auto columns = [&](const uint16_t* p, s16x8 (&st)[2 * NR]) {
      const __amdgpu_buffer_rsrc_t r = buffer_rsrc(p + rec * n_rt * (NB * kPiece), n_rt * NB * kPiece * 2);
#pragma unroll
      for (int rt = 0; rt < 2 * NR; ++rt)
        st[rt] = __builtin_bit_cast(s16x8, load16(r, (rt * NB + kb0) * (kPiece * 2) + lane * 16));
    };
    columns(ca.lf, lc);
    // gates: dlog_alpha and dbeta of token `lane`, over the row tiles
    float dl = 0.f, ge = 0.f;
    if (w == 3) {
      const __amdgpu_buffer_rsrc_t rz = buffer_rsrc(ca.zf + rec * n_rt * 64, n_rt * 256);
      const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(ca.bf + rec * n_rt * 64, n_rt * 256);
      float z[2 * NR], b[2 * NR];
#pragma unroll
      for (int i = 0; i < 2 * NR; ++i) {
        z[i] = load4(rz, (i * 64 + lane) * 4);
        b[i] = load4(rb, (i * 64 + lane) * 4);
      }
#pragma unroll
      for (int i = 0; i < 2 * NR; ++i) {
        dl += z[i];
        ge += b[i];
      }
    }
    wait_vm<0>();
    __syncthreads();
    const float* gam = lds.gt;
    const float* bet = lds.gt + 64;
    const float* rst = lds.gt + 128;
    const auto four = [&](const float* p, int b) { return *reinterpret_cast<const f32x4*>(p + 16 * b + 4 * g); };
    // e and G turned: tokens 16 tb + l in lanes, rows 32 R.. in order O
    const auto piece = [&](const uint16_t* p, int tb, int R) {
      return join(turned_raw(p + (4 * R) * kFrag, ra, tb), turned_raw(p + (4 * R + 2) * kFrag, ra, tb));
    };

    // ---- scores: wave w has kind w: dO e^T as [j][i] and [i][j], G e^T as
    // [j][i] and [i][j] (result rows first; the piece has the result's columns
    // in lanes).
    {
      const int kind = w;
      const bool isG = kind >= 2, ij = kind & 1;
      f32x4 v[10];
#pragma unroll
      for (int b = 0; b < 10; ++b) v[b] = zero4();
#pragma unroll 1
      for (int R = 0; R < nr; ++R) {
        bf16x8 i[4], j[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          i[b] = isG ? piece(lds.g, b, R) : frag_n<DV>(lds.o, to, b, R);
          j[b] = piece(lds.e, b, R);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y <= x; ++y) {
            f32x4& acc = v[x * (x + 1) / 2 + y];
            acc = ij ? mfma16x16x32(i[x], j[y], acc) : mfma16x16x32(j[y], i[x], acc);
          }
      }
      const auto finish = [&](int x, int y, f32x4 o) {  // block row x, column y <= x
        const int rb = ij ? x : y, cb = ij ? y : x;     // of the result
        if (x > y) {
          const float* ai = lds.gt + 320;
          const float* bj = lds.gt + 320 + 64 * x;
          const float fl = (ij ? bj : ai)[16 * cb + l] * (ij || isG ? bet[16 * cb + l] : 1.f) * (isG ? 1.f : sc);
          f32x4 fr = four(ij ? ai : bj, rb);
          if (!ij || isG) fr *= four(bet, rb);
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] *= fr[q] * fl;
        } else {
          const float lw = lds.gt[192 + 16 * x + l], lf = lds.gt[256 + 16 * x + l], bl = bet[16 * x + l];
          const f32x4 rw = four(lds.gt + 192, x), rf = four(lds.gt + 256, x), rbt = four(bet, x);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 4 * g + q, i = ij ? r : l, j = ij ? l : r;
            const float d = fexp2(ij ? (rw[q] - lw) + (rf[q] - lf) : (lw - rw[q]) + (lf - rf[q]));
            const float f = isG ? rbt[q] * bl : sc * (ij ? bl : rbt[q]);
            o[q] = j < i || (j == i && !isG) ? o[q] * d * f : 0.f;
          }
        }
        const int at = (isG ? 32 : 16 * kind) + (isG && ij && x == y ? 16 + x : 4 * cb + rb);
        *reinterpret_cast<uint2*>(&lds.sc[at * kPiece + lane * 4]) = make_uint2(pack2(o[0], o[1]), pack2(o[2], o[3]));
      };
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y <= x; ++y) finish(x, y, v[x * (x + 1) / 2 + y]);
    }
    columns(ca.sf, sc_);
    // ---- products with the states: result layout [column k: 4g + q][token l]
    f32x4 x[2][NT];
    const auto states = [&](const s16x8 (&st)[2 * NR], auto&& operand) {
#pragma unroll
      for (int t = 0; t < NT; ++t) x[0][t] = x[1][t] = zero4();
#pragma unroll
      for (int R = 0; R < NR; ++R) {
        if (R >= nr) break;
        const bf16x8 s0 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(st[2 * R], st[2 * R + 1], 0, 1, 2, 3, 8, 9, 10, 11));
        const bf16x8 s1 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(st[2 * R], st[2 * R + 1], 4, 5, 6, 7, 12, 13, 14, 15));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8 f = operand(tb0 + t, R);
          x[0][t] = mfma16x16x32(s0, f, x[0][t]);
          x[1][t] = mfma16x16x32(s1, f, x[1][t]);
        }
      }
    };
    const auto add = [&](f32x4 (&d)[2][NT], auto&& factor) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f = factor(16 * (tb0 + t) + l);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          d[0][t][q] = fmaf(f, x[0][t][q], d[0][t][q]);
          d[1][t][q] = fmaf(f, x[1][t][q], d[1][t][q]);
        }
      }
    };
    states(lc, [&](int tb, int R) { return piece(lds.e, tb, R); });
    add(dk, [&](int tok) { return rst[tok] * bet[tok]; });
    states(sc_, [&](int tb, int R) { return frag_n<DV>(lds.o, to, tb, R); });
    add(dq, [&](int tok) { return sc * gam[tok]; });
    states(sc_, [&](int tb, int R) { return piece(lds.g, tb, R); });
    add(dk, [&](int tok) { return -gam[tok] * bet[tok]; });
    __syncthreads();  // dO, e and G are done with, the scores are there
    {
      const __amdgpu_buffer_rsrc_t rk = rows_rsrc(kp, t0, sr.len, a.sk.t, a.dk);
      const __amdgpu_buffer_rsrc_t rq = rows_rsrc(qp, t0, sr.len, a.sq.t, a.dk);
#pragma unroll
      for (int j = 0; j < DK / 32; ++j) {
        const int i = w * (DK / 32) + j;
        dma16(rk, tile_off<DK>(i, lane, a.sk.t, 0, a.dk), lds.k + i * 1024);
        dma16(rq, tile_off<DK>(i, lane, a.sq.t, 0, a.dk), lds.q + i * 1024);
      }
      wait_vm<0>();
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {  // tokens 32 s.. as the contraction index
      bf16x8 kf[2], kn[2], qf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        kf[i] = frag_c<DK>(lds.k, tk, s, kb0 + i);
        qf[i] = frag_c<DK>(lds.q, tk, s, kb0 + i);
        kn[i] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(s16x8, kf[i]) ^ static_cast<short>(0x8000));
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tb = tb0 + t;
        const auto pc = [&](int m, int at) { return *reinterpret_cast<const s16x4*>(lds.sc + (16 * m + at) * kPiece + lane * 4); };
        if (s <= tb / 2) {  // j <= i
          const bf16x8 f = join(pc(0, tb * 4 + 2 * s), 2 * s + 1 <= tb ? pc(0, tb * 4 + 2 * s + 1) : none);
          dq[0][t] = mfma16x16x32(kf[0], f, dq[0][t]);
          dq[1][t] = mfma16x16x32(kf[1], f, dq[1][t]);
        }
        if (s >= tb / 2) {  // i >= j
          const bf16x8 f = join(2 * s >= tb ? pc(1, tb * 4 + 2 * s) : none, pc(1, tb * 4 + 2 * s + 1));
          dk[0][t] = mfma16x16x32(qf[0], f, dk[0][t]);
          dk[1][t] = mfma16x16x32(qf[1], f, dk[1][t]);
        }
        // a diagonal block's halves have their zeros where the other has not
        s16x4 m0 = pc(2, tb * 4 + 2 * s), m1 = pc(2, tb * 4 + 2 * s + 1);
        if (2 * s == tb) m0 |= pc(2, 16 + tb);
        if (2 * s + 1 == tb) m1 |= pc(2, 16 + tb);
        const bf16x8 f = join(m0, m1);
        dk[0][t] = mfma16x16x32(kn[0], f, dk[0][t]);
        dk[1][t] = mfma16x16x32(kn[1], f, dk[1][t]);
      }
    }
    if (w == 3) {
      if (lane < nt) {
        const int64_t o = sr.b * a.sdg.b + h * a.sdg.h + (sr.t0 + t0 + lane) * a.sdg.t;
        if (a.gate_io) {
          static_cast<uint16_t*>(a.dla)[o] = f32_to_bf16(dl);
          static_cast<uint16_t*>(a.dbe)[o] = f32_to_bf16(ge);
        } else {
          static_cast<float*>(a.dla)[o] = dl;
          static_cast<float*>(a.dbe)[o] = ge;
        }
      }
    }
  }
  // blocks kb0 and kb0 + 1 are eight neighbouring columns
  const int l = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const int col = index4(kb0, g);
  if (col < a.dk) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = 16 * (tb0 + t) + l;
      if (tok >= nt) continue;
      const int64_t tt = sr.t0 + t0 + tok;
      const auto put = [&](void* p, const Str3& s, const f32x4& u, const f32x4& v) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + sr.b * s.b + hk * s.h + tt * s.t + col) =
            make_uint4(pack2(u[0], u[1]), pack2(u[2], u[3]), pack2(v[0], v[1]), pack2(v[2], v[3]));
      };
      put(a.dq, a.sdq, dq[0][t], dq[1][t]);
      put(a.dk_, a.sdk, dk[0][t], dk[1][t]);
    }
  }
}

// ---- dlog_alpha of the tokens that keep little (delta_solve.hpp), for chunks
// that have one, after the gradients above: one work-group per chunk and value head,
// four waves.
//   m_ij = D_ij beta_j (scale q_i.k_j dO_i.e_j - beta_i k_i.k_j G_i.e_j)
//   a_i = e^l_i (scale q_i.(dO S)_i - beta_i k_i.(G S)_i)
//   b_j = e^(l_C - l_j) beta_j k_j.(e Lam)_j,  c = e^l_C <S, Lam>
// from the same rounded S, Lam, e and G: relative errors of some 3e-3 of a gradient
// that the running sum would lose.  Products as in delta_chunk_grad.  Where no chunk
// has such a token a launch that reads 256 bytes a head and chunk, 4.5 us; where every
// one has, 235 us at 8 x 16 x 4096 x 64 and at 4 x 16 x 4096 x 128.
template <int DV>
struct DecayLds {
  alignas(16) char o[64 * DV * 2];
  alignas(16) uint16_t e[64 * DV];
  alignas(16) uint16_t g[64 * DV];
  alignas(16) float gt[kGates];
  float a[4][64], b[4][64], c[4];  // parts of the waves
  Crossing x;
  uint64_t found[16];
};

template <int DK, int DV>
__global__ __launch_bounds__(kGradThreads) __attribute__((amdgpu_waves_per_eu(2))) void
delta_chunk_decay(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16, NP = NB / 2, NT = NP, NR = DV / 32, NS = DK / 32;
  __shared__ DecayLds<DV> lds;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for_strong(ca, lds.found, w, lane, [&](int64_t rec, uint64_t strong) {
    const int h = static_cast<int>(static_cast<uint32_t>(rec) % static_cast<uint32_t>(a.H));
    const int64_t slot = static_cast<uint32_t>(rec) / static_cast<uint32_t>(a.H);
    const int hk = h / (a.H / a.Hk);
    SeqRange sr;
    int64_t t0;
    if (!chunk_of_slot(a, slot, sr, t0)) return;
    __syncthreads();  // the one before is done with the tiles
    const int nt = static_cast<int>(sr.len - t0 < 64 ? sr.len - t0 : 64);
    const int n_rt = delta_row_tiles(a.dv), nr = n_rt / 2;
    const int kb0 = 2 * (w % NP), tb0 = NT * (w / NP);
    const float sc = static_cast<float>(a.scale);
    const uint16_t* op = static_cast<const uint16_t*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t;
    const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
    const __amdgpu_buffer_rsrc_t rk = rows_rsrc(kp, t0, sr.len, a.sk.t, a.dk);
    const __amdgpu_buffer_rsrc_t rq = rows_rsrc(qp, t0, sr.len, a.sq.t, a.dk);
    {
      const __amdgpu_buffer_rsrc_t ro = rows_rsrc(op, t0, sr.len, a.sdy.t, a.dv);
      const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(ca.gates + rec * kGates, kGates * 4);
      const int eb = n_rt * 2 * kFrag * 2;
      const __amdgpu_buffer_rsrc_t re = buffer_rsrc(ca.ef + rec * 2 * n_rt * kFrag, eb);
      const __amdgpu_buffer_rsrc_t rr = buffer_rsrc(ca.gf + rec * 2 * n_rt * kFrag, eb);
      if (w < 3) {
#pragma unroll
        for (int i = 0; i < 3; ++i) dma4(rg, ((3 * w + i) * 64 + lane) * 4, lds.gt + (3 * w + i) * 64);
      }
#pragma unroll
      for (int j = 0; j < DV / 32; ++j) {
        const int i = w * (DV / 32) + j;
        dma16(re, i * 1024 + lane * 16, reinterpret_cast<char*>(lds.e) + i * 1024);
        dma16(ro, tile_off<DV>(i, lane, a.sdy.t, 0, a.dv), lds.o + i * 1024);
        dma16(rr, i * 1024 + lane * 16, reinterpret_cast<char*>(lds.g) + i * 1024);
      }
    }
    s16x8 lc[2 * NR], st[2 * NR];  // this wave's columns of Lam and of S
    const auto columns = [&](const uint16_t* p, s16x8 (&to)[2 * NR]) {
      const __amdgpu_buffer_rsrc_t r = buffer_rsrc(p + rec * n_rt * (NB * kPiece), n_rt * NB * kPiece * 2);
#pragma unroll
      for (int rt = 0; rt < 2 * NR; ++rt)
        to[rt] = __builtin_bit_cast(s16x8, load16(r, (rt * NB + kb0) * (kPiece * 2) + lane * 16));
    };
    columns(ca.lf, lc);
    columns(ca.sf, st);
    wait_vm<0>();
    __syncthreads();
    const TileLane<DV> to = tile_lane<DV>(lane);
    const uint32_t ra = raw_turned(lane);
    const auto piece = [&](const uint16_t* p, int tb, int R) {
      return join(turned_raw(p + (4 * R) * kFrag, ra, tb), turned_raw(p + (4 * R + 2) * kFrag, ra, tb));
    };
    const auto half = [](const s16x8& v, int i) {
      return widen(i ? __builtin_shufflevector(v, v, 4, 5, 6, 7) : __builtin_shufflevector(v, v, 0, 1, 2, 3));
    };
    const auto dot = [](const f32x4& u, const f32x4& v) { return (u[0] * v[0] + u[1] * v[1]) + (u[2] * v[2] + u[3] * v[3]); };

    // ---- from the first state and to the end: products with the states, [column
    // 4g + q of this wave's two blocks][token l], times the rows of q or k
    const int col = index4(kb0, g);  // eight neighbouring columns
    const auto product = [&](const s16x8 (&s)[2 * NR], auto&& operand, __amdgpu_buffer_rsrc_t rows, int64_t stride,
                             int t) {
      f32x4 x[2] = {zero4(), zero4()};
#pragma unroll
      for (int R = 0; R < NR; ++R) {
        if (R >= nr) break;
        const bf16x8 s0 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(s[2 * R], s[2 * R + 1], 0, 1, 2, 3, 8, 9, 10, 11));
        const bf16x8 s1 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(s[2 * R], s[2 * R + 1], 4, 5, 6, 7, 12, 13, 14, 15));
        const bf16x8 f = operand(tb0 + t, R);
        x[0] = mfma16x16x32(s0, f, x[0]);
        x[1] = mfma16x16x32(s1, f, x[1]);
      }
      const uint32_t at = static_cast<uint32_t>((16 * (tb0 + t) + l) * stride * 2);
      const s16x8 v = __builtin_bit_cast(s16x8, load16(rows, col < a.dk ? at + col * 2 : kPastEnd));
      return sum_rows(dot(x[0], half(v, 0)) + dot(x[1], half(v, 1)));
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = 16 * (tb0 + t) + l;
      const float gam = lds.gt[tok], bet = lds.gt[64 + tok], rst = lds.gt[128 + tok];
      const float oq = product(st, [&](int tb, int R) { return frag_n<DV>(lds.o, to, tb, R); }, rq, a.sq.t, t);
      const float gk = product(st, [&](int tb, int R) { return piece(lds.g, tb, R); }, rk, a.sk.t, t);
      const float ek = product(lc, [&](int tb, int R) { return piece(lds.e, tb, R); }, rk, a.sk.t, t);
      if (g == 0) {
        lds.a[w][tok] = gam * (sc * oq - bet * gk);
        lds.b[w][tok] = rst * bet * ek;
      }
    }
    {
      float c = 0.f;
      if (tb0 == 0) {
#pragma unroll
        for (int rt = 0; rt < 2 * NR; ++rt)
#pragma unroll
          for (int i = 0; i < 2; ++i) c += dot(half(st[rt], i), half(lc[rt], i));
      }
      c = wave_sum(c);
      if (lane == 0) lds.c[w] = c;
    }
    // ---- from token to token: blocks of 16 x 16 of the lower triangle in turn
    for (int b = w; b < 10; b += 4) {
      const int x = tri_i(b), y = tri_j(b);
      f32x4 oe = zero4(), ge = zero4(), qk = zero4(), kk = zero4();
      for (int R = 0; R < nr; ++R) {
        const bf16x8 e = piece(lds.e, y, R);
        oe = mfma16x16x32(frag_n<DV>(lds.o, to, x, R), e, oe);
        ge = mfma16x16x32(piece(lds.g, x, R), e, ge);
      }
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        const uint32_t cc = 32 * c + 8 * g < a.dk ? static_cast<uint32_t>((32 * c + 8 * g) * 2) : kPastEnd;
        const auto row = [&](__amdgpu_buffer_rsrc_t r, int64_t stride, int tb) {
          return load16(r, cc + static_cast<uint32_t>((16 * tb + l) * stride * 2));
        };
        const bf16x8 kj = row(rk, a.sk.t, y);
        qk = mfma16x16x32(row(rq, a.sq.t, x), kj, qk);
        kk = mfma16x16x32(row(rk, a.sk.t, x), kj, kk);
      }
      const int j = 16 * y + l;
      const float lw = lds.gt[192 + j], lf = lds.gt[256 + j], bj = lds.gt[64 + j];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = 16 * x + 4 * g + q;
        const float d = bj * fexp2((lds.gt[192 + i] - lw) + (lds.gt[256 + i] - lf));
        lds.x.m[i * 65 + j] = d * (sc * qk[q] * oe[q] - lds.gt[64 + i] * kk[q] * ge[q]);
      }
    }
    __syncthreads();
    if (w == 0) lds.x.gather(lane);
    __syncthreads();
    if (w != 0) return;
    float from = 0.f, into = 0.f, all = 0.f;
    const int w0 = (lane >> 4) / NT * NP;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      from += lds.a[w0 + i][lane];
      into += lds.b[w0 + i][lane];
      all += lds.c[i];
    }
    const float z = lds.x.at(from, into, lds.gt[63] * all, lane);
    if (lane < nt && ((strong >> lane) & 1)) {
      const int64_t o = sr.b * a.sdg.b + h * a.sdg.h + (sr.t0 + t0 + lane) * a.sdg.t;
      if (a.gate_io) static_cast<uint16_t*>(a.dla)[o] = f32_to_bf16(z);
      else static_cast<float*>(a.dla)[o] = z;
    }
  });
}

template <int DK>
hipError_t launch(const ChunkArgs& c, hipStream_t s) {
  constexpr int NW = 2;
  const int tiles = (c.a.dv + 16 * NW - 1) / (16 * NW);
  const auto blocks = [&](int runs) { return dim3(static_cast<unsigned>(head_blocks(c.a.N * c.a.H * runs, tiles))); };
  hipError_t e = hipSuccess;
  if (c.n_seg > 1) {
    delta_chunk_rev<DK, NW, true><<<blocks(c.n_seg - 1), 64 * (2 * NW + 2), 0, s>>>(c);
    if ((e = hipGetLastError()) != hipSuccess || (e = launch_delta_join(c, true, s)) != hipSuccess) return e;
  }
  delta_chunk_rev<DK, NW, false><<<blocks(c.n_seg), 64 * (2 * NW + 2), 0, s>>>(c);
  e = hipGetLastError();
  if (e != hipSuccess || c.slots == 0) return e;
  const dim3 grid(static_cast<unsigned>(c.slots * c.a.Hk));
  const bool shared = c.a.H != c.a.Hk;
  if (c.a.dv <= 64) {
    if (shared) delta_chunk_grad<DK, 64, true><<<grid, kGradThreads, 0, s>>>(c);
    else delta_chunk_grad<DK, 64, false><<<grid, kGradThreads, 0, s>>>(c);
  } else {
    if (shared) delta_chunk_grad<DK, 128, true><<<grid, kGradThreads, 0, s>>>(c);
    else delta_chunk_grad<DK, 128, false><<<grid, kGradThreads, 0, s>>>(c);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (c.a.dv <= 64) delta_chunk_decay<DK, 64><<<seek_groups(c, 2), kGradThreads, 0, s>>>(c);
  else delta_chunk_decay<DK, 128><<<seek_groups(c, 2), kGradThreads, 0, s>>>(c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunk_bwd(const ChunkArgs& c, hipStream_t s) {
  if (c.a.N * c.a.H == 0) return hipSuccess;
  return c.a.dk <= 64 ? launch<64>(c, s) : launch<128>(c, s);
}

}  // namespace gls
