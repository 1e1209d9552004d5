// k_delta_chunk_bwd.hip -- the gated delta rule's gradients over chunks (bf16 on
// the matrix cores), from what the forward left.  With Lam the adjoint of the
// state after the chunk:
//
//   dU = P^T dO + e^(l_C - l) (K Lam^T),  G = dU - Y^T (beta dU),  F = beta G
//   Lam <- e^(l_C) Lam + (scale e^l dO)^T Q - (e^l F)^T K
//
// is again a recurrence of independent rows (delta_chunk_rev, the mirror of the
// forward kernel: state waves with Lam^T in their accumulators; helper waves
// form the two products with dO one chunk ahead and hand them over in fp32).
// The rest is one work-group per chunk and key head (delta_chunk_grad):
//
//   dq = scale e^l dO S + dP K,              dP_ij = scale D_ij beta_j dO_i.e_j  (j <= i)
//   dk = beta (e^(l_C - l) E Lam - e^l G S) + dP^T Q - (H + H^T) K,
//                                            H_ij = D_ij beta_i beta_j G_i.e_j   (j < i)
//   dv = beta G,   D_ij = e^(l_i - l_j)
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
// but the rounding of each flow left errors of up to 7e-3.)  dbeta = G.e is
// formed there too, from the fp32 G.
#include "delta_mfma.hpp"
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

template <int DK, int NW>
__global__ __launch_bounds__(64 * (2 * NW + 2)) void delta_chunk_rev(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NS = DK / 32, NB = DK / 16, VW = 16 * NW;
  __shared__ RevLds<DK, NW> lds;
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
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
        yb[tb] = *reinterpret_cast<const f32x4*>(ca.yb + ((rec * n_rt + rt) * 4 + tb) * 256 + lane * 4);
    };
    if (nc > 0) fetch(nc - 1);
    float z = 0.f;  // <dL/dS, S> after the chunk, over this wave's rows
    if (a.dstate_out && r0 + index1(w, l) < a.dv) {
      const int64_t so = (head * a.dv + r0 + index1(w, l)) * a.dk;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (index4(b, g) < a.dk) {
          const f32x4 u = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.dstate_out) + so + index4(b, g));
          const f32x4 s = *reinterpret_cast<const f32x4*>(ca.st + so + index4(b, g));
#pragma unroll
          for (int q = 0; q < 4; ++q) z = fmaf(u[q], s[q], z);
        }
    }
    z = wave_sum(z);
    for (int i = 0; i <= nc + 1; ++i) {
      lds_barrier();
      if (i >= 2) {
        const int64_t rec = rec0 + static_cast<int64_t>(nc + 1 - i) * a.H;
        const float x = lds.dyy[w][(i - 2) % 3][lane] - lds.vdv[w][i & 1][lane];
        const float y = wave_scan_add(wave_reverse(x, lane));
        ca.zf[(rec * n_rt + rt) * 64 + 63 - lane] = z + y;
        z += readlane_f(y, 63);
      }
      f32x4 x1[4], x2[NB];
      if (i < nc) {
        const int sl = i % 3;
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
      lds_barrier();
      if (i < nc) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) *reinterpret_cast<f32x4*>(&lds.x1[w][tb * 256 + lane * 4]) = x1[tb];
#pragma unroll
        for (int b = 0; b < NB; ++b) *reinterpret_cast<f32x4*>(&lds.x2[w][b * 256 + lane * 4]) = x2[b];
      }
    }
    return;
  }

  // ---- adjoint states
  const TileLane<VW> tv = tile_lane<VW>(lane);
  const int r = r0 + index1(wave, l);
  const int64_t so = (head * a.dv + r) * a.dk;
  f32x4 S[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    S[b] = a.dstate_out && r < a.dv && index4(b, g) < a.dk
               ? *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.dstate_out) + so + index4(b, g))
               : zero4();
  bf16x8 yf[12], ef[2];
  const int rt = tile * NW + wave, n_rt = delta_row_tiles(a.dv);
  const auto fetch = [&](int c) {
    const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
    const uint16_t* p = ca.ytf + rec * kYf + lane * 8;
#pragma unroll
    for (int f = 0; f < 12; ++f) yf[f] = *reinterpret_cast<const bf16x8*>(p + f * kFrag);
  };
  const auto fetch_e = [&](int c) {
    const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      ef[s] = *reinterpret_cast<const bf16x8*>(ca.ef + ((rec * n_rt + rt) * 2 + s) * kFrag + raw_at(lane));
  };
  if (nc > 0) {
    fetch(nc - 1);
    fetch_e(nc - 1);
  }
  lds_barrier();
  lds_barrier();
  for (int i = 1; i <= nc; ++i) {
    const int c = nc - i;
    const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
    Pair8 sp[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) sp[s] = split8(S[2 * s], S[2 * s + 1]);
    uint16_t* turn = lds.turn[wave];
#pragma unroll
    for (int s = 0; s < NS; ++s) *reinterpret_cast<bf16x8*>(&turn[s * kFrag + lane * 8]) = sp[s].hi;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      *reinterpret_cast<s16x4*>(ca.lf + ((rec * n_rt + rt) * NB + b) * kPiece + lane * 4) = turned(turn, b, lane);
    lds_barrier();  // A
    const int sl = (i - 1) % 3;
    const char* kt = lds.k[sl];
    const float* gt = lds.gt[(i - 1) & 3];
    const auto gate = [&](int m, int tb) { return *reinterpret_cast<const f32x4*>(gt + 64 * m + 16 * tb + 4 * g); };
    f32x4 x1[4];
    s16x4 vv[4];
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      vv[tb] = col4<VW>(lds.v[sl], tv, tb, wave);
      x1[tb] = *reinterpret_cast<const f32x4*>(&lds.x1[wave][tb * 256 + lane * 4]);
    }
    const float whole = gt[63];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const f32x4 x2 = *reinterpret_cast<const f32x4*>(&lds.x2[wave][b * 256 + lane * 4]);
#pragma unroll
      for (int q = 0; q < 4; ++q) S[b][q] = fmaf(whole, S[b][q], x2[q]);
    }
    lds_barrier();  // B
    f32x4 G[4], Z[4];
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) G[tb] = zero4();
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const bf16x8 kf = frag_n<DK>(kt, tk, tb, s);
        G[tb] = mfma16x16x32(kf, sp[s].hi, G[tb]);
        G[tb] = mfma16x16x32(kf, sp[s].lo, G[tb]);
      }
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      const f32x4 rs = gate(2, tb), be = gate(1, tb);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        G[tb][q] = fmaf(rs[q], G[tb][q], x1[tb][q]);
        Z[tb][q] = be[q] * G[tb][q];
      }
    }
    {
      const Pair8 z0 = split8(Z[0], Z[1]), z1 = split8(Z[2], Z[3]);
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        f32x4 x = zero4();
#pragma unroll
        for (int s = jb / 2; s < 2; ++s) {
          const int f = jb < 2 ? 2 * jb + s : jb + 2;
          const Pair8& z = s ? z1 : z0;
          x = mfma16x16x32(yf[2 * f + 1], z.hi, x);
          x = mfma16x16x32(yf[2 * f], z.lo, x);
          x = mfma16x16x32(yf[2 * f], z.hi, x);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) G[jb][q] -= x[q];
      }
    }
    if (i < nc) fetch(c - 1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
      *reinterpret_cast<bf16x8*>(ca.gf + ((rec * n_rt + rt) * 2 + s) * kFrag + raw_at(lane)) =
          raw_order(round8(G[2 * s], G[2 * s + 1]), lane);
    {  // G.e and v.dv: token 16 (l / 4) + 4 g + l % 4
      float x[16], y[16];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const s16x8 e = __builtin_bit_cast(s16x8, raw_order(ef[s], lane));
        const f32x4 e0 = widen(__builtin_shufflevector(e, e, 0, 1, 2, 3));
        const f32x4 e1 = widen(__builtin_shufflevector(e, e, 4, 5, 6, 7));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x[8 * s + q] = G[2 * s][q] * e0[q];
          x[8 * s + 4 + q] = G[2 * s + 1][q] * e1[q];
        }
      }
      if (i < nc) fetch_e(c - 1);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const f32x4 v = widen(vv[tb]), be = gate(1, tb);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          G[tb][q] *= be[q];
          y[4 * tb + q] = v[q] * G[tb][q];
        }
      }
      const int tok = 16 * (l >> 2) + 4 * g + (l & 3);
      ca.bf[(rec * n_rt + rt) * 64 + tok] = row_sums(x, l);
      lds.vdv[wave][(i - 1) & 1][tok] = row_sums(y, l);
    }
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      const f32x4 gm = gate(0, tb);
#pragma unroll
      for (int q = 0; q < 4; ++q) G[tb][q] *= -gm[q];
    }
    const Pair8 u0 = split8(G[0], G[1]), u1 = split8(G[2], G[3]);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bf16x8 k0 = frag_c<DK>(kt, tk, 0, b), k1 = frag_c<DK>(kt, tk, 1, b);
      S[b] = mfma16x16x32(k0, u0.hi, S[b]);
      S[b] = mfma16x16x32(k0, u0.lo, S[b]);
      S[b] = mfma16x16x32(k1, u1.hi, S[b]);
      S[b] = mfma16x16x32(k1, u1.lo, S[b]);
    }
  }
  lds_barrier();
  lds_barrier();
  if (a.dstate_in && r < a.dv) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (index4(b, g) < a.dk)
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.dstate_in) + so + index4(b, g)) = S[b];
  }
}

// ---- the gradients of one chunk, for the value heads of one key head in turn
// (their sums stay in registers).  Eight waves: first the score blocks dP, dP^T
// and H + H^T, dealt over the waves and handed on through LDS as operands;
// then wave w takes 16 columns of dq and dk (S and Lam enter as operands
// straight from global memory, each column block once).
template <int DK, int DV>
struct GradLds {
  alignas(16) char k[64 * DK * 2];
  alignas(16) char q[64 * DK * 2];
  alignas(16) char o[64 * DV * 2];
  alignas(16) uint16_t e[DV / 16 * 4 * kPiece];
  alignas(16) uint16_t g[DV / 16 * 4 * kPiece];
  alignas(16) uint16_t sc[3][16 * kPiece];   // dP [i][j], dP^T [j][i], H + H^T [a][b]
  alignas(16) float gt[kGates];
};

constexpr int kGradThreads = 512;

template <int DK, int DV>
__global__ __launch_bounds__(kGradThreads) void delta_chunk_grad(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16, NT = DK == 128 ? 4 : 2, NR = DV / 32;
  __shared__ GradLds<DK, DV> lds;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = static_cast<int>(blockIdx.x % a.Hk), grp = a.H / a.Hk;
  const int64_t slot = blockIdx.x / a.Hk;
  int64_t n, c;
  if (a.cu) {
    int64_t lo = 0, hi = a.N - 1;
    while (lo < hi) {
      const int64_t m = (lo + hi + 1) / 2;
      if (chunk_slot0(true, m, seq_range(a.cu, m, a.T).t0, a.T, kDeltaChunk) <= slot) lo = m;
      else hi = m - 1;
    }
    n = lo;
    c = slot - chunk_slot0(true, n, seq_range(a.cu, n, a.T).t0, a.T, kDeltaChunk);
  } else {
    const int64_t nc = (a.T + kDeltaChunk - 1) / kDeltaChunk;
    n = slot / nc;
    c = slot % nc;
  }
  const SeqRange sr = seq_range(a.cu, n, a.T);
  const int64_t t0 = c * kDeltaChunk;
  if (c < 0 || t0 >= sr.len) return;
  const int nt = static_cast<int>(sr.len - t0 < 64 ? sr.len - t0 : 64);
  const int n_rt = delta_row_tiles(a.dv);
  const int kb = w % NB, tb0 = DK == 128 ? 0 : 2 * (w / NB);
  const TileLane<DK> tk = tile_lane<DK>(lane);
  const TileLane<DV> to = tile_lane<DV>(lane);
  const uint32_t ra = raw_turned(lane);
  const float sc = static_cast<float>(a.scale);

  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
  {
    const __amdgpu_buffer_rsrc_t rk = rows_rsrc(kp, t0, sr.len, a.sk.t, a.dk);
    const __amdgpu_buffer_rsrc_t rq = rows_rsrc(qp, t0, sr.len, a.sq.t, a.dk);
#pragma unroll
    for (int i = w; i < DK / 8; i += 8) {
      dma16(rk, tile_off<DK>(i, lane, a.sk.t, 0, a.dk), lds.k + i * 1024);
      dma16(rq, tile_off<DK>(i, lane, a.sq.t, 0, a.dk), lds.q + i * 1024);
    }
  }
  f32x4 dq[NT], dk[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) dq[t] = dk[t] = zero4();

  for (int gi = 0; gi < grp; ++gi) {
    const int h = hk * grp + gi;
    const int64_t rec = slot * a.H + h;
    if (gi) __syncthreads();  // the head before is done with the tiles
    {
      const uint16_t* op = static_cast<const uint16_t*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t;
      const __amdgpu_buffer_rsrc_t ro = rows_rsrc(op, t0, sr.len, a.sdy.t, a.dv);
      const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(ca.gates + rec * kGates, kGates * 4);
      const int eb = n_rt * 2 * kFrag * 2;  // bytes of e's fragments
      const __amdgpu_buffer_rsrc_t re = buffer_rsrc(ca.ef + rec * 2 * n_rt * kFrag, eb);
      const __amdgpu_buffer_rsrc_t rr = buffer_rsrc(ca.gf + rec * 2 * n_rt * kFrag, eb);
#pragma unroll
      for (int i = w; i < DV / 8; i += 8) {
        dma16(ro, tile_off<DV>(i, lane, a.sdy.t, 0, a.dv), lds.o + i * 1024);
        dma16(re, i * 1024 + lane * 16, reinterpret_cast<char*>(lds.e) + i * 1024);
        dma16(rr, i * 1024 + lane * 16, reinterpret_cast<char*>(lds.g) + i * 1024);
      }
      if (w < 5) dma4(rg, (w * 64 + lane) * 4, lds.gt + w * 64);
    }
    // S and Lam, columns of this wave
    s16x4 sp[2 * NR], lp[2 * NR];
#pragma unroll
    for (int rt = 0; rt < 2 * NR; ++rt) {
      const s16x4 none = {0, 0, 0, 0};
      sp[rt] = rt < n_rt ? *reinterpret_cast<const s16x4*>(ca.sf + ((rec * n_rt + rt) * NB + kb) * kPiece + lane * 4) : none;
      lp[rt] = rt < n_rt ? *reinterpret_cast<const s16x4*>(ca.lf + ((rec * n_rt + rt) * NB + kb) * kPiece + lane * 4) : none;
    }
    wait_vm<0>();
    __syncthreads();
    const float* gam = lds.gt;
    const float* bet = lds.gt + 64;
    const float* rst = lds.gt + 128;
    const auto decay = [&](int i, int j) {
      return fexp2((lds.gt[192 + i] - lds.gt[192 + j]) + (lds.gt[256 + i] - lds.gt[256 + j]));
    };
    // e and G turned: tokens 16 tb + l in lanes, rows 32 R.. in order O
    const auto piece = [&](const uint16_t* p, int tb, int R) {
      return join(turned_raw(p + (4 * R) * kFrag, ra, tb), turned_raw(p + (4 * R + 2) * kFrag, ra, tb));
    };
    // ---- scores.  Result layout [row block index 4g + q][column l]; the piece
    // of (column block, row block) is then an operand with the column in lanes.
    const int nr = n_rt / 2;
    for (int b = w; b < 36; b += 8) {
      const bool sym = b >= 20;
      int x, y;  // row and column block of the result
      const int tb = b < 10 ? b : b - 10;
      if (sym) { x = (b - 20) >> 2; y = (b - 20) & 3; }
      else if (b < 10) { x = tri_j(tb); y = tri_i(tb); }   // [j][i]
      else { x = tri_i(tb); y = tri_j(tb); }               // [i][j]
      f32x4 v = zero4(), v2 = zero4();
      for (int R = 0; R < nr; ++R) {
        if (!sym) {
          const bf16x8 of = frag_n<DV>(lds.o, to, b < 10 ? y : x, R);
          const bf16x8 ef = piece(lds.e, b < 10 ? x : y, R);
          v = b < 10 ? mfma16x16x32(ef, of, v) : mfma16x16x32(of, ef, v);
        } else {
          if (x <= y) v = mfma16x16x32(piece(lds.e, x, R), piece(lds.g, y, R), v);   // H[y][x]
          if (x >= y) v2 = mfma16x16x32(piece(lds.g, x, R), piece(lds.e, y, R), v2);  // H[x][y]
        }
      }
      f32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int p = 16 * x + 4 * g + q, m = 16 * y + l;  // tokens of row and column
        if (!sym) {
          const int i = b < 10 ? m : p, j = b < 10 ? p : m;
          o[q] = j <= i ? sc * bet[j] * decay(i, j) * v[q] : 0.f;
        } else {
          const float bb = bet[p] * bet[m];
          o[q] = p < m ? bb * decay(m, p) * v[q] : p > m ? bb * decay(p, m) * v2[q] : 0.f;
        }
      }
      uint16_t* dst = lds.sc[sym ? 2 : b < 10 ? 0 : 1] + (y * 4 + x) * kPiece + lane * 4;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(o[0], o[1]), pack2(o[2], o[3]));
    }
    // ---- dv: row tiles w, w + 8, .. of 16 columns of v
    for (int rt = w; rt < n_rt; rt += 8) {
      const int r = index4(rt, g);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const int t = 16 * tb + l;
        const f32x4 gv = widen(turned_raw(lds.g + 2 * rt * kFrag, ra, tb));
        const float b = bet[t];
        if (t < nt && r < a.dv)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dv_) + sr.b * a.sdv.b + h * a.sdv.h +
                                    (sr.t0 + t0 + t) * a.sdv.t + r) =
              make_uint2(pack2(b * gv[0], b * gv[1]), pack2(b * gv[2], b * gv[3]));
      }
    }
    // ---- products with the states: result layout [column k: 4g + q][token l]
    f32x4 a1[NT], a2[NT], a3[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) a1[t] = a2[t] = a3[t] = zero4();
#pragma unroll
    for (int R = 0; R < NR; ++R) {
      if (R >= nr) break;
      const bf16x8 sf = join(sp[2 * R], sp[2 * R + 1]), lf = join(lp[2 * R], lp[2 * R + 1]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        a1[t] = mfma16x16x32(sf, frag_n<DV>(lds.o, to, tb0 + t, R), a1[t]);
        a2[t] = mfma16x16x32(lf, piece(lds.e, tb0 + t, R), a2[t]);
        a3[t] = mfma16x16x32(sf, piece(lds.g, tb0 + t, R), a3[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = 16 * (tb0 + t) + l;
      const float ga = gam[tok], rb = rst[tok] * bet[tok], gb = ga * bet[tok];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a1[t][q] *= sc * ga;
        dk[t][q] += rb * a2[t][q] - gb * a3[t][q];
      }
    }
    __syncthreads();  // the scores are there
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      // tokens 32 s.. as the contraction index
      const bf16x8 kf = frag_c<DK>(lds.k, tk, s, kb), qf = frag_c<DK>(lds.q, tk, s, kb);
      const bf16x8 kn = __builtin_bit_cast(bf16x8, __builtin_bit_cast(s16x8, kf) ^ static_cast<short>(0x8000));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tb = tb0 + t;
        const s16x4 none = {0, 0, 0, 0};
        const auto pc = [&](int m, int b) { return *reinterpret_cast<const s16x4*>(lds.sc[m] + (tb * 4 + b) * kPiece + lane * 4); };
        if (s <= tb / 2) {  // j <= i
          const s16x4 p0 = pc(0, 2 * s), p1 = 2 * s + 1 <= tb ? pc(0, 2 * s + 1) : none;
          a1[t] = mfma16x16x32(kf, join(p0, p1), a1[t]);
        }
        if (s >= tb / 2) {  // i >= j
          const s16x4 p0 = 2 * s >= tb ? pc(1, 2 * s) : none, p1 = pc(1, 2 * s + 1);
          dk[t] = mfma16x16x32(qf, join(p0, p1), dk[t]);
        }
        dk[t] = mfma16x16x32(kn, join(pc(2, 2 * s), pc(2, 2 * s + 1)), dk[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int q = 0; q < 4; ++q) dq[t][q] += a1[t][q];
    }
    if (w == 0) {  // gates, lane = token
      float ge = 0.f, dl = 0.f;
      for (int i = 0; i < n_rt; ++i) {
        ge += ca.bf[(rec * n_rt + i) * 64 + lane];
        dl += ca.zf[(rec * n_rt + i) * 64 + lane];
      }
      // a token that forgets everything has no gradient to its decay
      const float lw = lds.gt[192 + lane];
      if (lw - wave_shift_up(lw, 0.f) < -149.f) dl = 0.f;
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
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int tok = 16 * (tb0 + t) + l, col = index4(kb, g);
    if (tok < nt && col < a.dk) {
      const int64_t tt = sr.t0 + t0 + tok;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dq) + sr.b * a.sdq.b + hk * a.sdq.h + tt * a.sdq.t + col) =
          make_uint2(pack2(dq[t][0], dq[t][1]), pack2(dq[t][2], dq[t][3]));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dk_) + sr.b * a.sdk.b + hk * a.sdk.h + tt * a.sdk.t + col) =
          make_uint2(pack2(dk[t][0], dk[t][1]), pack2(dk[t][2], dk[t][3]));
    }
  }
}

template <int DK>
hipError_t launch(const ChunkArgs& c, hipStream_t s) {
  constexpr int NW = 2;
  const int tiles = (c.a.dv + 16 * NW - 1) / (16 * NW);
  delta_chunk_rev<DK, NW><<<dim3(static_cast<unsigned>(head_blocks(c.a.N * c.a.H, tiles))), 64 * (2 * NW + 2), 0, s>>>(c);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || c.slots == 0) return e;
  const dim3 grid(static_cast<unsigned>(c.slots * c.a.Hk));
  if (c.a.dv <= 64) delta_chunk_grad<DK, 64><<<grid, kGradThreads, 0, s>>>(c);
  else delta_chunk_grad<DK, 128><<<grid, kGradThreads, 0, s>>>(c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunk_bwd(const ChunkArgs& c, hipStream_t s) {
  if (c.a.N * c.a.H == 0) return hipSuccess;
  return c.a.dk <= 64 ? launch<64>(c, s) : launch<128>(c, s);
}

}  // namespace gls
