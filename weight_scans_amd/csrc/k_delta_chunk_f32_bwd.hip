// k_delta_chunk_f32_bwd.hip -- the gated delta rule's gradients over chunks in
// fp32, from what the forward left: the formulas of the bf16 chunks
// (k_delta_chunk_bwd.hip), every product on v_mfma_f32_16x16x4_f32.
//
// The decay's gradient is again dlog_alpha_t = <dL/dS_T, S_T> + sum_{s >= t}
// (dy_s.y_s - dv_s.v_s); here both states are kept in fp32, so the product
// <Lam, S> is taken anew at every chunk's end and the sum runs over the chunk's
// tokens only.  Tokens that keep little of the state get it as in bf16 from what
// crosses them (delta_decay_f32).
//
// The recurrence is bound by the matrix rate of the waves that have a row tile's
// chain, the gradients by the matrix cores and HBM: 4 x 8 x 1024 x 64 takes 56 us
// and 32 us, 128 x 128 heads 78 us and 73 us, and 4 us to look for tokens that keep
// little (token by token all together: 1058 and 1728 us).  With one wave to a row
// tile's chain the recurrence took 106 and 150 us; where heads fill the card by
// themselves the two are level (256 heads of 64: 439 us with the gradients, before
// 435).
#include <type_traits>

#include "delta_f32.hpp"
#include "dev_common.hpp"

namespace gls {
namespace {

// The recurrence of Lam from the last chunk to the first.  A work-group has 16
// rows; two waves share the products of a chunk (token blocks as Part, columns of
// Lam in halves; the fp32 matrix rate of one SIMD bounds their chain) and exchange
// Lam, beta dU and G through LDS, three barriers a chunk: every buffer's reads end
// one barrier before its next write.  A third wave has what is no part of the
// chain: Lam turned for the gradients, dbeta and the decay's terms.  The last one
// loads the next chunk's K, Q and gates; dO, V, y, e go straight to registers.
template <int DK>
struct RevLds {
  alignas(16) char k[2][64 * DK * 4];
  alignas(16) char q[2][64 * DK * 4];
  alignas(16) float gt[2][192];
  alignas(16) float lx[DK * 16];  // Lam^T after the chunk, blocks of 16
  alignas(16) float zx[64 * 16];  // -beta dU
  alignas(16) float gx[64 * 16];  // G
  float xs[64];
};
constexpr int kRevThreads = 4 * 64;

template <int DK>
__global__ __launch_bounds__(kRevThreads) void delta_rev_f32(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16, HB = NB / 2;
  __shared__ RevLds<DK> lds;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_rt = delta_row_tiles(a.dv), VP = 16 * n_rt;
  int64_t head;
  int rt;
  if (!head_of_block(blockIdx.x, n_rt, a.N * a.H, head, rt)) return;
  const int h = static_cast<int>(head % a.H);
  const int64_t n = head / a.H;
  const int hk = h / (a.H / a.Hk), r = 16 * rt + l;
  const SeqRange sr = seq_range(a.cu, n, a.T);
  const int nc = static_cast<int>((sr.len + kDeltaChunk - 1) / kDeltaChunk);
  const int64_t slot0 = chunk_slot0(a.cu != nullptr, n, sr.t0, a.T, kDeltaChunk);
  const int64_t rec0 = slot0 * a.H + h;
  const auto rec_of = [&](int c) { return rec0 + static_cast<int64_t>(c) * a.H; };
  const auto block = [&](const float* x, int b) { return *reinterpret_cast<const f32x4*>(x + b * 256 + lane * 4); };
  const auto put = [&](float* x, int b, const f32x4& v) { *reinterpret_cast<f32x4*>(x + b * 256 + lane * 4) = v; };

  if (wave == 3) {  // ---- loads
    constexpr int NK = DK / 4;
    const float* kp = static_cast<const float*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
    const float* qp = static_cast<const float*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
    uint32_t ko[NK], qo[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      ko[i] = tile_off_f32<DK>(i, lane, a.sk.t, a.dk);
      qo[i] = tile_off_f32<DK>(i, lane, a.sq.t, a.dk);
    }
    const auto issue = [&](int c) {
      const int s = c & 1;
      const __amdgpu_buffer_rsrc_t rk = rows_f32(kp, c * 64LL, sr.len, a.sk.t, a.dk);
      const __amdgpu_buffer_rsrc_t rq = rows_f32(qp, c * 64LL, sr.len, a.sq.t, a.dk);
      const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(ca.gates + rec_of(c) * kGates, 768);
#pragma unroll
      for (int i = 0; i < NK; ++i) dma16(rk, ko[i], lds.k[s] + i * 1024);
#pragma unroll
      for (int i = 0; i < NK; ++i) dma16(rq, qo[i], lds.q[s] + i * 1024);
#pragma unroll
      for (int i = 0; i < 3; ++i) dma4(rg, (i * 64 + lane) * 4, lds.gt[s] + i * 64);
    };
    if (nc > 0) issue(nc - 1);
    for (int c = nc - 1; c >= 0; --c) {
      wait_vm<0>();
      lds_barrier();
      if (c > 0) issue(c - 1);  // into the slot of chunk c + 1
      lds_barrier();
      lds_barrier();
    }
    return;
  }

  const float* vp = static_cast<const float*>(a.v) + sr.b * a.sv.b + h * a.sv.h + sr.t0 * a.sv.t;
  const float* op = static_cast<const float*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t;
  uint32_t vo[4], oo[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    vo[q] = r < a.dv ? static_cast<uint32_t>(((4 * g + q) * static_cast<int>(a.sv.t) + r) * 4) : kPastEnd;
    oo[q] = r < a.dv ? static_cast<uint32_t>(((4 * g + q) * static_cast<int>(a.sdy.t) + r) * 4) : kPastEnd;
  }
  const int64_t all = head * a.dv * a.dk;
  const __amdgpu_buffer_rsrc_t ru =
      state_rsrc(a.dstate_out ? static_cast<const float*>(a.dstate_out) + all : nullptr, a.dv, a.dk);

  if (wave == 2) {  // ---- Lam for the gradients, dbeta, the decay's terms
    float z = 0.f;  // <Lam, state> after the chunk, over these rows
    {
      const __amdgpu_buffer_rsrc_t rs = state_rsrc(a.dstate_out ? ca.st + all : nullptr, a.dv, a.dk);
      f32x4 u[NB], s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u[b] = load_f32x4(ru, state_off(r, 16 * b + 4 * g, a.dk));
        s[b] = load_f32x4(rs, state_off(r, 16 * b + 4 * g, a.dk));
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) z = fmaf(u[b][q], s[b][q], z);
    }
    z = wave_sum(z);
    wait_vm<0>();  // dstate_in may be dstate_out
    const uint32_t ra = static_cast<uint32_t>((4 * g * VP + r) * 4);
    f32x4 sn[NB];  // the state after the chunk, turned
    for (int c = nc - 1; c >= 0; --c) {
      const int64_t rec = rec_of(c);
      const float lw = ca.gates[rec * kGates + 192 + lane];
      f32x4 dO[4], V[4], Y[4], E[4];
      {
        const __amdgpu_buffer_rsrc_t ro = rows_f32(op, c * 64LL, sr.len, a.sdy.t, a.dv);
        const __amdgpu_buffer_rsrc_t rv = rows_f32(vp, c * 64LL, sr.len, a.sv.t, a.dv);
        const __amdgpu_buffer_rsrc_t re = buffer_rsrc(ca.e32 + rec * 64 * VP, 256 * VP);
        const __amdgpu_buffer_rsrc_t ry = buffer_rsrc(ca.yb + rec * 64 * VP, 256 * VP);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            dO[tb][q] = load4(ro, oo[q] + static_cast<uint32_t>(tb * 64 * static_cast<int>(a.sdy.t)));
            V[tb][q] = load4(rv, vo[q] + static_cast<uint32_t>(tb * 64 * static_cast<int>(a.sv.t)));
          }
          E[tb] = load_rows(re, ra, VP, tb);
          Y[tb] = load_rows(ry, ra, VP, tb);
        }
      }
      lds_barrier();
      float zz = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4 x = turned_f32(lds.lx + b * 256, lane);
        *reinterpret_cast<f32x4*>(ca.l32 + ((rec * n_rt + rt) * NB + b) * 256 + lane * 4) = x;
        if (c + 1 < nc)
#pragma unroll
          for (int q = 0; q < 4; ++q) zz = fmaf(x[q], sn[b][q], zz);
      }
      if (c + 1 < nc) z = wave_sum(zz);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        sn[b] = *reinterpret_cast<const f32x4*>(ca.s32 + ((rec * n_rt + rt) * NB + b) * 256 + lane * 4);
      lds_barrier();
      lds_barrier();
      float xe[16], xv[16];
      const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(ca.g32 + rec * 64 * VP, 256 * VP);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const f32x4 be = *reinterpret_cast<const f32x4*>(lds.gt[c & 1] + 64 + 16 * tb + 4 * g);
        const f32x4 G = block(lds.gx, tb);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          xe[4 * tb + q] = G[q] * E[tb][q];
          xv[4 * tb + q] = dO[tb][q] * Y[tb][q] - V[tb][q] * (be[q] * G[q]);
        }
        store_rows(rg, ra, VP, tb, G);
      }
      const int tok = 16 * (l >> 2) + 4 * g + (l & 3);
      const float db = row_sums(xe, l);
      lds.xs[tok] = row_sums(xv, l);
      const float sum = decay_sum(lds.xs[63 - lane], z, tokens_below(lw, kForget), lane);
      ca.bf[(rec * n_rt + rt) * 64 + tok] = db;
      ca.zf[(rec * n_rt + rt) * 64 + 63 - lane] = sum;
    }
    return;
  }

  const auto chain = [&](auto part) {
    constexpr int B0 = HB * decltype(part)::value, OB = HB - B0;  // own columns, the other's
    using Pt = Part<decltype(part)::value>;
    const float sc = static_cast<float>(a.scale);
    f32x4 S[HB];  // Lam^T
#pragma unroll
    for (int b = 0; b < HB; ++b) S[b] = load_f32x4(ru, state_off(r, 16 * (B0 + b) + 4 * g, a.dk));
#pragma unroll
    for (int b = 0; b < HB; ++b) put(lds.lx, B0 + b, S[b]);
    f32x4 dO[4], pt[5], yt[5];
    const auto fetch_o = [&](int c) {  // dO and P^T
      const __amdgpu_buffer_rsrc_t ro = rows_f32(op, c * 64LL, sr.len, a.sdy.t, a.dv);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          dO[tb][q] = load4(ro, oo[q] + static_cast<uint32_t>(tb * 64 * static_cast<int>(a.sdy.t)));
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = Pt::tb(x); i < 4; ++i)
          pt[Pt::below(x, i)] = *reinterpret_cast<const f32x4*>(ca.pt32 + rec_of(c) * kY32 +
                                                                SolveLds::tri(i, Pt::tb(x)) * 256 + lane * 4);
    };
    const auto fetch_y = [&](int c) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = Pt::tb(x); i < 4; ++i)
          yt[Pt::below(x, i)] = *reinterpret_cast<const f32x4*>(ca.yt32 + rec_of(c) * kY32 +
                                                                SolveLds::tri(i, Pt::tb(x)) * 256 + lane * 4);
    };
    if (nc > 0) {
      fetch_o(nc - 1);
      fetch_y(nc - 1);
    }
    const uint32_t ka = row_at<DK>(lane);
    const uint32_t kc[4] = {col_at<DK>(lane, 0), col_at<DK>(lane, 1), col_at<DK>(lane, 2), col_at<DK>(lane, 3)};
    for (int c = nc - 1; c >= 0; --c) {
      lds_barrier();
      const char* kt = lds.k[c & 1];
      const char* qt = lds.q[c & 1];
      const float* gt = lds.gt[c & 1] + 4 * g;
      const auto gate = [&](int m, int tb) { return *reinterpret_cast<const f32x4*>(gt + 64 * m + 16 * tb); };
      // K Lam^T of the own tokens
      f32x4 D[2] = {zero4(), zero4()};
      const auto scores = [&](int b, const f32x4& s) {
        f32x4 kf[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) kf[x] = row_frag<DK>(kt, ka, Pt::tb(x), b);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int x = 0; x < 2; ++x) D[x] = mfma_f32(kf[x][q], s[q], D[x]);
      };
#pragma unroll
      for (int b = 0; b < HB; ++b) scores(B0 + b, S[b]);
#pragma unroll
      for (int b = 0; b < HB; ++b) scores(OB + b, block(lds.lx, OB + b));
      // dU = e^(l_C - l) K Lam^T + P^T dO
#pragma unroll
      for (int x = 0; x < 2; ++x) D[x] *= gate(2, Pt::tb(x));
#pragma unroll
      for (int i = 3; i >= 0; --i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (i >= Pt::tb(x)) D[x] = mfma_f32(pt[Pt::below(x, i)][q], dO[i][q], D[x]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const f32x4 be = gate(1, Pt::tb(x));
        f32x4 z;
#pragma unroll
        for (int q = 0; q < 4; ++q) z[q] = -be[q] * D[x][q];
        put(lds.zx, Pt::tb(x), z);
      }
      // Q's part of the own columns before the others' beta dU is waited for
      const float whole = lds.gt[c & 1][63];
#pragma unroll
      for (int b = 0; b < HB; ++b) S[b] *= whole;
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const f32x4 o = dO[tb] * (gate(0, tb) * sc);
        f32x4 qf[HB];
#pragma unroll
        for (int b = 0; b < HB; ++b) qf[b] = col_frag<DK>(qt, kc, tb, B0 + b);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int b = 0; b < HB; ++b) S[b] = mfma_f32(qf[b][q], o[q], S[b]);
      }
      fetch_o(max(c - 1, 0));
      lds_barrier();
      // G = dU - Y^T (beta dU)
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        if (i < Pt::tb(0)) continue;
        const f32x4 z = block(lds.zx, i);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (i >= Pt::tb(x)) D[x] = mfma_f32(yt[Pt::below(x, i)][q], z[q], D[x]);
      }
      fetch_y(max(c - 1, 0));
#pragma unroll
      for (int x = 0; x < 2; ++x) put(lds.gx, Pt::tb(x), D[x]);
      lds_barrier();
      // K's part
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const f32x4 f = block(lds.gx, tb) * (gate(0, tb) * gate(1, tb));
        f32x4 kf[HB];
#pragma unroll
        for (int b = 0; b < HB; ++b) kf[b] = col_frag<DK>(kt, kc, tb, B0 + b);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int b = 0; b < HB; ++b) S[b] = mfma_f32(kf[b][q], -f[q], S[b]);
      }
#pragma unroll
      for (int b = 0; b < HB; ++b) put(lds.lx, B0 + b, S[b]);
    }
    if (a.dstate_in && r < a.dv) {
#pragma unroll
      for (int b = 0; b < HB; ++b) {
        const int col = 16 * (B0 + b) + 4 * g;
        if (col < a.dk)
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.dstate_in) + (head * a.dv + r) * a.dk + col) = S[b];
      }
    }
  };
  if (wave == 0) chain(std::integral_constant<int, 0>{});
  else chain(std::integral_constant<int, 1>{});
}

// The gradients of one chunk, for the value heads of one key head in turn.  Wave
// w has the 16 tokens of block w, of dq and of dk: every block of scores that it
// needs comes out of the matrix cores with the index in lanes that the next
// product wants, so the waves share K and Q in LDS and nothing else.
template <int DK>
struct GradLds {
  alignas(16) char k[64 * DK * 4];
  alignas(16) char q[64 * DK * 4];
};

template <int DK, int W>
__device__ __forceinline__ void grad_block(const ChunkArgs& ca, const GradLds<DK>& lds, int64_t slot, const SeqRange& sr,
                                           int64_t t0, int hk, int lane) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16;
  const int grp = a.H / a.Hk;
  const int nt = static_cast<int>(sr.len - t0 < 64 ? sr.len - t0 : 64);
  const int n_rt = delta_row_tiles(a.dv), VP = 16 * n_rt;
  const float sc = static_cast<float>(a.scale);
  f32x4 dq[NB], dk[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) dq[b] = dk[b] = zero4();
  for (int gi = 0; gi < grp; ++gi) {
    const int h = hk * grp + gi;
    const int64_t rec = slot * a.H + h;
    // anew for each head: addresses kept over the loop cost more registers than there are
    asm volatile("" : "+v"(lane));
    const int l = lane & 15, g = lane >> 4;
    const float* gt = ca.gates + rec * kGates;
    const __amdgpu_buffer_rsrc_t ro =
        rows_f32(static_cast<const float*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t, t0, sr.len, a.sdy.t,
                 a.dv);
    float* dvp = static_cast<float*>(a.dv_) + sr.b * a.sdv.b + h * a.sdv.h + (sr.t0 + t0 + 16 * W + l) * a.sdv.t;
    const float* ep = ca.e32 + (rec * 64 + l) * VP + 4 * g;
    const float* gp = ca.g32 + (rec * 64 + l) * VP + 4 * g;
    const float* sp = ca.s32 + rec * n_rt * (NB * 256) + lane * 4;
    const float* lp = ca.l32 + rec * n_rt * (NB * 256) + lane * 4;
    const float bet = gt[64 + 16 * W + l], gam = gt[16 * W + l], rst = gt[128 + 16 * W + l];
    // e_j dO_i and e_j G_i below and on the diagonal: rows j of column i = W's
    // tokens (pq, h2), rows i of column j = W's (pk, h1)
    f32x4 pq[4], pk[4], h1[4], h2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pq[i] = pk[i] = h1[i] = h2[i] = zero4();
#pragma unroll 1
    for (int rt = 0; rt < n_rt; ++rt) {
      f32x4 d[4], e[4], G[4];
      const int c = 16 * rt + 4 * g;
      const uint32_t co = c < a.dv ? static_cast<uint32_t>(c * 4) : kPastEnd;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= W) {
          d[i] = load_f32x4(ro, co + static_cast<uint32_t>((16 * i + l) * static_cast<int>(a.sdy.t) * 4));
          G[i] = *reinterpret_cast<const f32x4*>(gp + 16 * i * VP + 16 * rt);
        }
        if (i <= W) e[i] = *reinterpret_cast<const f32x4*>(ep + 16 * i * VP + 16 * rt);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i <= W) {
          pq[i] = mul16(e[i], d[W], pq[i]);
          h2[i] = mul16(e[i], G[W], h2[i]);
        }
        if (i >= W) {
          pk[i] = mul16(d[i], e[W], pk[i]);
          h1[i] = mul16(G[i], e[W], h1[i]);
        }
      }
      const f32x4 dw = d[W] * (sc * gam), ew = e[W] * (rst * bet), gw = G[W] * (-gam * bet);
      if (16 * W + l < nt && c < a.dv) *reinterpret_cast<f32x4*>(dvp + c) = G[W] * bet;
      // four column blocks at a time
#pragma unroll
      for (int b0 = 0; b0 < NB; b0 += 4) {
        f32x4 s[4], lam[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          s[b] = *reinterpret_cast<const f32x4*>(sp + (rt * NB + b0 + b) * 256);
          lam[b] = *reinterpret_cast<const f32x4*>(lp + (rt * NB + b0 + b) * 256);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            dq[b0 + b] = mfma_f32(dw[q], s[b][q], dq[b0 + b]);
            dk[b0 + b] = mfma_f32(ew[q], lam[b][q], dk[b0 + b]);
            dk[b0 + b] = mfma_f32(gw[q], s[b][q], dk[b0 + b]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // decay, beta and the triangle
    const float lw = gt[192 + 16 * W + l], lf = gt[256 + 16 * W + l];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 rw = *reinterpret_cast<const f32x4*>(gt + 192 + 16 * i + 4 * g);
      const f32x4 rf = *reinterpret_cast<const f32x4*>(gt + 256 + 16 * i + 4 * g);
      const f32x4 rb = *reinterpret_cast<const f32x4*>(gt + 64 + 16 * i + 4 * g);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int x = 16 * i + 4 * g + q, y = 16 * W + l;  // the row's token, the column's
        const float up = fexp2((lw - rw[q]) + (lf - rf[q])), down = fexp2((rw[q] - lw) + (rf[q] - lf));
        if (i <= W) {
          pq[i][q] = x <= y ? pq[i][q] * (sc * rb[q] * up) : 0.f;
          h2[i][q] = x < y ? h2[i][q] * (rb[q] * bet * up) : 0.f;
        }
        if (i >= W) {
          pk[i][q] = x >= y ? pk[i][q] * (sc * bet * down) : 0.f;
          h1[i][q] = x > y ? h1[i][q] * (rb[q] * bet * down) : 0.f;
        }
        h1[i][q] = -(h1[i][q] + h2[i][q]);
      }
    }
    const uint32_t kc[4] = {col_at<DK>(lane, 0), col_at<DK>(lane, 1), col_at<DK>(lane, 2), col_at<DK>(lane, 3)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4 kf = col_frag<DK>(lds.k, kc, i, b);
        if (i <= W) dq[b] = mul16(pq[i], kf, dq[b]);
        dk[b] = mul16(h1[i], kf, dk[b]);
        if (i >= W) dk[b] = mul16(pk[i], col_frag<DK>(lds.q, kc, i, b), dk[b]);
        if (b % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (W == 3) {  // gates: token `lane`, over the row tiles
      const __amdgpu_buffer_rsrc_t rz = buffer_rsrc(ca.zf + rec * n_rt * 64, n_rt * 256);
      const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(ca.bf + rec * n_rt * 64, n_rt * 256);
      float z[8], b[8], dl = 0.f, db = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[i] = load4(rz, (i * 64 + lane) * 4);
        b[i] = load4(rb, (i * 64 + lane) * 4);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dl += z[i];
        db += b[i];
      }
      if (lane < nt) {
        const int64_t o = sr.b * a.sdg.b + h * a.sdg.h + (sr.t0 + t0 + lane) * a.sdg.t;
        static_cast<float*>(a.dla)[o] = dl;
        static_cast<float*>(a.dbe)[o] = db;
      }
    }
  }
  const int l = lane & 15, g = lane >> 4;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int tok = 16 * W + 4 * g + q;
    if (tok >= nt) continue;
    float* pq = static_cast<float*>(a.dq) + sr.b * a.sdq.b + hk * a.sdq.h + (sr.t0 + t0 + tok) * a.sdq.t;
    float* pk = static_cast<float*>(a.dk_) + sr.b * a.sdk.b + hk * a.sdk.h + (sr.t0 + t0 + tok) * a.sdk.t;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (16 * b + l < a.dk) {
        pq[16 * b + l] = dq[b][q];
        pk[16 * b + l] = dk[b][q];
      }
  }
}

template <int DK>
__global__ __launch_bounds__(256, 2) void delta_grad_f32(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  __shared__ GradLds<DK> lds;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = static_cast<int>(blockIdx.x % a.Hk);
  const int64_t slot = blockIdx.x / a.Hk;
  SeqRange sr;
  int64_t t0;
  if (!chunk_of_slot(a, slot, sr, t0)) return;
  {
    const float* kp = static_cast<const float*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
    const float* qp = static_cast<const float*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
    const __amdgpu_buffer_rsrc_t rk = rows_f32(kp, t0, sr.len, a.sk.t, a.dk);
    const __amdgpu_buffer_rsrc_t rq = rows_f32(qp, t0, sr.len, a.sq.t, a.dk);
#pragma unroll
    for (int j = 0; j < DK / 16; ++j) {
      const int i = w * (DK / 16) + j;
      dma16(rk, tile_off_f32<DK>(i, lane, a.sk.t, a.dk), lds.k + i * 1024);
      dma16(rq, tile_off_f32<DK>(i, lane, a.sq.t, a.dk), lds.q + i * 1024);
    }
    wait_vm<0>();
  }
  __syncthreads();
  if (w == 0) grad_block<DK, 0>(ca, lds, slot, sr, t0, hk, lane);
  else if (w == 1) grad_block<DK, 1>(ca, lds, slot, sr, t0, hk, lane);
  else if (w == 2) grad_block<DK, 2>(ca, lds, slot, sr, t0, hk, lane);
  else grad_block<DK, 3>(ca, lds, slot, sr, t0, hk, lane);
}

// dlog_alpha of the tokens that keep little (delta_solve.hpp), for chunks that have
// one: the terms of the bf16 form (delta_chunk_decay) in fp32, one work-group per
// chunk and value head, wave w with the tokens of block w.
template <int DK>
struct DecayLds {
  alignas(16) char k[64 * DK * 4];
  alignas(16) char q[64 * DK * 4];
  float a[64], b[64], c;
  Crossing x;
  uint64_t found[16];
};

template <int DK>
__global__ __launch_bounds__(256) void delta_decay_f32(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16;
  __shared__ DecayLds<DK> lds;
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
    const float* gt = ca.gates + rec * kGates;
    const int nt = static_cast<int>(sr.len - t0 < 64 ? sr.len - t0 : 64);
    const int n_rt = delta_row_tiles(a.dv), VP = 16 * n_rt;
    const float sc = static_cast<float>(a.scale);
    {
      const float* kp = static_cast<const float*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
      const float* qp = static_cast<const float*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
      const __amdgpu_buffer_rsrc_t rk = rows_f32(kp, t0, sr.len, a.sk.t, a.dk);
      const __amdgpu_buffer_rsrc_t rq = rows_f32(qp, t0, sr.len, a.sq.t, a.dk);
#pragma unroll
      for (int j = 0; j < DK / 16; ++j) {
        const int i = w * (DK / 16) + j;
        dma16(rk, tile_off_f32<DK>(i, lane, a.sk.t, a.dk), lds.k + i * 1024);
        dma16(rq, tile_off_f32<DK>(i, lane, a.sq.t, a.dk), lds.q + i * 1024);
      }
    }
    const __amdgpu_buffer_rsrc_t ro = rows_f32(
        static_cast<const float*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t, t0, sr.len, a.sdy.t, a.dv);
    const float* ep = ca.e32 + (rec * 64 + l) * VP + 4 * g;
    const float* gp = ca.g32 + (rec * 64 + l) * VP + 4 * g;
    const float* sp = ca.s32 + rec * n_rt * (NB * 256) + lane * 4;
    const float* lp = ca.l32 + rec * n_rt * (NB * 256) + lane * 4;
    f32x4 oe[4], ge[4], os[NB], gs[NB], el[NB];
    float c = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) oe[j] = ge[j] = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) os[b] = gs[b] = el[b] = zero4();
#pragma unroll 1
    for (int rt = 0; rt < n_rt; ++rt) {
      const int r = 16 * rt + 4 * g;
      const f32x4 d = load_f32x4(ro, r < a.dv ? static_cast<uint32_t>(((16 * w + l) * static_cast<int>(a.sdy.t) + r) * 4)
                                              : kPastEnd);
      const f32x4 G = *reinterpret_cast<const f32x4*>(gp + 16 * w * VP + 16 * rt);
      const f32x4 own = *reinterpret_cast<const f32x4*>(ep + 16 * w * VP + 16 * rt);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > w) break;
        const f32x4 e = *reinterpret_cast<const f32x4*>(ep + 16 * j * VP + 16 * rt);
        oe[j] = mul16(d, e, oe[j]);
        ge[j] = mul16(G, e, ge[j]);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4 s = *reinterpret_cast<const f32x4*>(sp + (rt * NB + b) * 256);
        const f32x4 lam = *reinterpret_cast<const f32x4*>(lp + (rt * NB + b) * 256);
        os[b] = mul16(d, s, os[b]);
        gs[b] = mul16(G, s, gs[b]);
        el[b] = mul16(own, lam, el[b]);
#pragma unroll
        for (int q = 0; q < 4; ++q) c = fmaf(s[q], lam[q], c);
      }
    }
    c = wave_sum(c);
    if (w == 0 && lane == 0) lds.c = c;
    wait_vm<0>();
    __syncthreads();
    const uint32_t ra = row_at<DK>(lane);
    const uint32_t kc[4] = {col_at<DK>(lane, 0), col_at<DK>(lane, 1), col_at<DK>(lane, 2), col_at<DK>(lane, 3)};
    // tokens 16 w + 4g + q, columns in lanes
    f32x4 oq = zero4(), gk = zero4(), ek = zero4();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const f32x4 q = col_frag<DK>(lds.q, kc, w, b), k = col_frag<DK>(lds.k, kc, w, b);
      oq += os[b] * q;
      gk += gs[b] * k;
      ek += el[b] * k;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int tok = 16 * w + 4 * g + q;
      const float x = gt[tok] * (sc * row_sum(oq[q]) - gt[64 + tok] * row_sum(gk[q]));
      const float y = gt[128 + tok] * gt[64 + tok] * row_sum(ek[q]);
      if (l == 0) {
        lds.a[tok] = x;
        lds.b[tok] = y;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > w) break;
      f32x4 qk = zero4(), kk = zero4();
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4 kj = row_frag<DK>(lds.k, ra, j, b);
        qk = mul16(row_frag<DK>(lds.q, ra, w, b), kj, qk);
        kk = mul16(row_frag<DK>(lds.k, ra, w, b), kj, kk);
      }
      const int y = 16 * j + l;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int x = 16 * w + 4 * g + q;
        const float f = gt[64 + y] * fexp2((gt[192 + x] - gt[192 + y]) + (gt[256 + x] - gt[256 + y]));
        lds.x.m[x * 65 + y] = f * (sc * qk[q] * oe[j][q] - gt[64 + x] * kk[q] * ge[j][q]);
      }
    }
    __syncthreads();
    if (w == 0) lds.x.gather(lane);
    __syncthreads();
    if (w != 0) return;
    const float z = lds.x.at(lds.a[lane], lds.b[lane], gt[63] * lds.c, lane);
    if (lane < nt && ((strong >> lane) & 1))
      static_cast<float*>(a.dla)[sr.b * a.sdg.b + h * a.sdg.h + (sr.t0 + t0 + lane) * a.sdg.t] = z;
  });
}

template <int DK>
hipError_t launch(const ChunkArgs& c, hipStream_t s) {
  delta_rev_f32<DK><<<dim3(static_cast<unsigned>(head_blocks(c.a.N * c.a.H, delta_row_tiles(c.a.dv)))), kRevThreads, 0,
                      s>>>(c);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || c.slots == 0) return e;
  delta_grad_f32<DK><<<dim3(static_cast<unsigned>(c.slots * c.a.Hk)), 256, 0, s>>>(c);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  delta_decay_f32<DK><<<seek_groups(c, DK <= 64 ? 2 : 1), 256, 0, s>>>(c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunk_f32_bwd(const ChunkArgs& c, hipStream_t s) {
  if (c.a.N * c.a.H == 0) return hipSuccess;
  return c.a.dk <= 64 ? launch<64>(c, s) : launch<128>(c, s);
}

}  // namespace gls
