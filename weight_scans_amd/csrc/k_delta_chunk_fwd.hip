// k_delta_chunk_fwd.hip -- the gated delta rule over the chunks of a sequence,
// forward (bf16 on the matrix cores).  Per chunk, with S the state before it:
//
//   R = V - e^l (K S^T),  E = R - Y (beta R),  U = beta E
//   y = scale e^l (Q S^T) + P U,   S <- e^(l_C) S + U^T (e^(l_C - l) K)
//
// The rows of S are independent, so one wave carries 16 of them through the
// whole sequence without meeting another: S^T stays in its accumulators, and
// every product's result is the next product's operand in registers (see
// delta_mfma.hpp); only the chunk's K, V and Y come from outside.  Operands that
// are not exact bf16 inputs are split into two bf16 terms.
//
// A work-group is NW state waves, NW output waves (they get S and U of the
// chunk before through LDS and form y one chunk behind, so that y is off the
// chain) and two waves that keep the direct loads of the next two chunks in
// flight: one barrier per chunk.  The output waves also form the chunk's P, in
// the step before they use it (with P left in memory by the preparation both took
// 293 instead of 246 us together, training 8 x 16 x 4096 x 64).
//
// Bound by the chain of a chunk's products in one wave (128 x 128: 2.3 us a step,
// of which its matrix instructions take 0.6; vector work that splits operands
// stands between them, so nothing else fills the gaps of a SIMD that one wave
// has), and in training by what is kept for the backward.  Work-groups of 32 rows,
// two state waves: LDS holds one of them a CU, and 64 rows would leave half the
// CUs idle at 64 sequence-heads.  4 x 16 x 4096 x 128: 145 us, training 197 us
// (664 MB, 3.4 TB/s); 8 x 16 x 4096 x 64: 111 us, training 150 us (650 MB, 4.3 TB/s).
//
// Few heads and many chunks: the chunks of a sequence are cut into n_seg
// segments that run at once.  What a segment does to the state is
//   S_end = S_begin M + Z
// row by row; a first pass (STATES: no outputs) gets Z as the end of the
// segment from S = 0 and M as its end from S = I without values, delta_join
// forms the segments' first states one after another, and the pass over the
// tokens then starts every segment from its own.  1 x 16 x 32768 x 128, four
// segments: 198 us + 8 us + 252 us for the passes, 940 us in one.
#include "delta_mfma.hpp"
#include "dev_common.hpp"

namespace gls {
namespace {

enum { OUTPUTS, TRAINING, STATES };  // y; y and what the backward needs; M and Z of segments

template <int DK, int NW, int MODE>
struct FwdLds {
  static constexpr int NS = DK / 32, VW = 16 * NW, OUT = MODE != STATES;
  alignas(16) char k[3][64 * DK * 2];
  alignas(16) char q[OUT ? 3 : 1][OUT ? 64 * DK * 2 : 16];
  alignas(16) char v[2][64 * VW * 2];
  alignas(16) float gt[2][192];
  alignas(16) float fo[2][OUT ? 384 : 4];  // the decay's factors for P, [6][64]
  alignas(16) uint16_t sx[2][NW][OUT ? 2 * NS * kFrag : 8];  // hi, then lo
  alignas(16) uint16_t ux[2][NW][OUT ? 4 * kFrag : 8];
};
template <int NW, int MODE>
constexpr int kFwdThreads = 64 * (MODE == STATES ? NW + 1 : 2 * NW + 2);

template <int DK, int NW, int MODE>
__global__ __launch_bounds__((kFwdThreads<NW, MODE>)) void delta_chunk_fwd(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr bool SAVE = MODE == TRAINING, OUT = MODE != STATES;
  constexpr int NS = DK / 32, NB = DK / 16, VW = 16 * NW, LOADER = OUT ? 2 * NW : NW;
  __shared__ FwdLds<DK, NW, MODE> lds;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ztiles = (a.dv + VW - 1) / VW, tiles = ztiles + (OUT ? 0 : (a.dk + VW - 1) / VW);
  const int runs = OUT ? ca.n_seg : ca.n_seg - 1;  // segments of this pass
  int64_t head;
  int tile;
  if (!head_of_block(blockIdx.x, tiles, a.N * a.H * runs, head, tile)) return;
  const int seg = static_cast<int>(static_cast<uint32_t>(head) % static_cast<uint32_t>(runs));
  head = static_cast<uint32_t>(head) / static_cast<uint32_t>(runs);
  const bool ident = !OUT && tile >= ztiles;  // rows of M, not of Z
  if (ident) {
    if (seg == 0) return;  // its first state is known: Z is its end from there
    tile -= ztiles;
  }
  const int h = static_cast<int>(head % a.H);
  const int64_t n = head / a.H;
  const int hk = h / (a.H / a.Hk), r0 = tile * VW;
  SeqRange sr = seq_range(a.cu, n, a.T);
  int64_t slot0 = chunk_slot0(a.cu != nullptr, n, sr.t0, a.T, kDeltaChunk);
  const int nc = segment_of(sr, slot0, seg, ca.n_seg);
  const int64_t rec0 = slot0 * a.H + h;

  if (wave == LOADER) {  // ---- loads: K two chunks ahead, V and gates one
    constexpr int NK = DK / 8, NV = VW / 8;
    const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
    const uint16_t* vp = static_cast<const uint16_t*>(a.v) + sr.b * a.sv.b + h * a.sv.h + sr.t0 * a.sv.t + r0;
    uint32_t ko[NK], vo[NV];
#pragma unroll
    for (int i = 0; i < NK; ++i) ko[i] = tile_off<DK>(i, lane, a.sk.t, 0, a.dk);
#pragma unroll
    for (int i = 0; i < NV; ++i) vo[i] = tile_off<VW>(i, lane, a.sv.t, 0, a.dv - r0);
    const auto issue_k = [&](int c) {
      const __amdgpu_buffer_rsrc_t rk = rows_rsrc(kp, c * 64LL, c < nc ? sr.len : 0, a.sk.t, a.dk);
#pragma unroll
      for (int i = 0; i < NK; ++i) dma16(rk, ko[i], lds.k[c % 3] + i * 1024);
    };
    const auto issue_v = [&](int c) {
      const bool in = c < nc;
      const __amdgpu_buffer_rsrc_t rv = rows_rsrc(vp, c * 64LL, in && !ident ? sr.len : 0, a.sv.t, min(VW, a.dv - r0));
      const __amdgpu_buffer_rsrc_t rg =
          buffer_rsrc(ca.gates + (in ? (rec0 + static_cast<int64_t>(c) * a.H) * kGates : 0), in ? 768 : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) dma16(rv, vo[i], lds.v[c & 1] + i * 1024);
#pragma unroll
      for (int i = 0; i < 3; ++i) dma4(rg, (i * 64 + lane) * 4, lds.gt[c & 1] + i * 64);
    };
    issue_v(0);
    issue_k(0);
    issue_k(1);
    for (int c = 0; c <= nc; ++c) {
      wait_vm<NK>();  // chunk c is there, K of c + 1 in flight
      lds_barrier();
      issue_v(c + 1);  // into the slots of chunk c - 1
      issue_k(c + 2);
    }
    wait_vm<0>();
    return;
  }
  if (OUT && wave == LOADER + 1) {  // ---- loads: Q, two chunks ahead
    constexpr int NK = DK / 8;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
    uint32_t qo[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) qo[i] = tile_off<DK>(i, lane, a.sq.t, 0, a.dk);
    const auto issue = [&](int c) {
      const __amdgpu_buffer_rsrc_t rq = rows_rsrc(qp, c * 64LL, c < nc ? sr.len : 0, a.sq.t, a.dk);
#pragma unroll
      for (int i = 0; i < NK; ++i) dma16(rq, qo[i], lds.q[c % 3] + i * 1024);
    };
    const auto gates = [&](int c) { return ca.gates + (rec0 + static_cast<int64_t>(c) * a.H) * kGates; };
    DecayFactors df(static_cast<float>(a.scale), lane);
    if (nc > 0) df.fetch(gates(0));
    issue(0);
    issue(1);
    if (nc > 0) df.put(lds.fo[0]);
    // Training: this wave also keeps the states (it has the time), two row tiles
    // of the chunk before
    constexpr int ST = SAVE ? NW * NB / 2 : 0;
    const int n_rt = delta_row_tiles(a.dv);
    const auto keep = [&](int c) {
      uint16_t* to = ca.sf + ((rec0 + static_cast<int64_t>(c) * a.H) * n_rt + tile * NW) * NB * kPiece + lane * 8;
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int b = 0; b < NB; b += 2)
          *reinterpret_cast<bf16x8*>(to + (w * NB + b) * kPiece) =
              join(turned(lds.sx[c & 1][w], b, lane), turned(lds.sx[c & 1][w], b + 1, lane));
    };
    for (int c = 0; c <= nc; ++c) {
      // chunk c is there; newer are the loads of c + 1 and the stores of c - 2
      if (SAVE && c >= 2) wait_vm<NK + ST>();
      else wait_vm<NK>();
      lds_barrier();
      if (c + 1 < nc) df.fetch(gates(c + 1));  // before the loads that need not be waited for
      issue(c + 2);                            // into the slot of chunk c - 1
      if (c + 1 < nc) df.put(lds.fo[(c + 1) & 1]);
      if constexpr (SAVE)
        if (c > 0) keep(c - 1);
    }
    wait_vm<0>();
    return;
  }

  const TileLane<DK> tk = tile_lane<DK>(lane);
  if (OUT && wave >= NW) {  // ---- outputs, one chunk behind
    const int w = wave - NW;
    const int rr = r0 + index4(w, g);
    uint16_t* yp = static_cast<uint16_t*>(a.y) + sr.b * a.sy.b + h * a.sy.h + sr.t0 * a.sy.t + rr;
    const float sc = static_cast<float>(a.scale);
    const int rt = tile * NW + w, n_rt = delta_row_tiles(a.dv);
    // P and Q of the chunk, formed and read in its own step, used in the next
    Pair8 pf[6];
    bf16x8 qf[4][NS];
    float gs[4];
    const auto scores = [&](int c) {
      const char* qt = lds.q[c % 3];
      const char* kt = lds.k[c % 3];
      const float* fo = lds.fo[c & 1];
      const auto row = [&](int at) { return *reinterpret_cast<const f32x4*>(fo + at + 4 * g); };
#pragma unroll
      for (int x = 0; x < 4; ++x) gs[x] = sc * lds.gt[c & 1][16 * x + l];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int s = 0; s < NS; ++s) qf[tb][s] = frag_n<DK>(qt, tk, tb, s);
#pragma unroll
      for (int jp = 0; jp < 2; ++jp) {
        bf16x8 kf[2][NS];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int s = 0; s < NS; ++s) kf[h][s] = frag_n<DK>(kt, tk, 2 * jp + h, s);
#pragma unroll
        for (int tb = 2 * jp; tb < 4; ++tb) {
          f32x4 p[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = 2 * jp + h;
            p[h] = zero4();
            if (j > tb) continue;
#pragma unroll
            for (int s = 0; s < NS; ++s) p[h] = mfma16x16x32(kf[h][s], qf[tb][s], p[h]);
            if (j < tb) {
              const f32x4 f = row(64 * tb + 16 * j) * fo[16 * tb + l];
#pragma unroll
              for (int q = 0; q < 4; ++q) p[h][q] *= f[q];
            } else {
              const f32x4 rw = row(256 + 16 * tb), rf = row(320 + 16 * tb);
              const float lw = fo[256 + 16 * tb + l], lf = fo[320 + 16 * tb + l];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float d = sc * fexp2((lw - rw[q]) + (lf - rf[q]));
                p[h][q] = 4 * g + q <= l ? p[h][q] * d : 0.f;
              }
            }
          }
          pf[tb < 2 ? tb : 2 * tb - 2 + jp] = split8(p[0], p[1]);
        }
      }
    };
    lds_barrier();
    if (nc > 0) scores(0);
    for (int c = 0; c < nc; ++c) {
      lds_barrier();
      const uint16_t* sx = lds.sx[c & 1][w];
      const uint16_t* ux = lds.ux[c & 1][w];
      f32x4 o[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) o[tb] = zero4();
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const bf16x8 sh = *reinterpret_cast<const bf16x8*>(sx + s * kFrag + lane * 8);
        const bf16x8 sl = *reinterpret_cast<const bf16x8*>(sx + (NS + s) * kFrag + lane * 8);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          o[tb] = mfma16x16x32(sl, qf[tb][s], o[tb]);
          o[tb] = mfma16x16x32(sh, qf[tb][s], o[tb]);
        }
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
#pragma unroll
        for (int q = 0; q < 4; ++q) o[tb][q] *= gs[tb];
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bf16x8 uh = *reinterpret_cast<const bf16x8*>(ux + s * kFrag + lane * 8);
        const bf16x8 ul = *reinterpret_cast<const bf16x8*>(ux + (2 + s) * kFrag + lane * 8);
#pragma unroll
        for (int tb = 2 * s; tb < 4; ++tb) {
          const int f = tb < 2 ? tb : 2 * tb - 2 + s;
          o[tb] = mfma16x16x32(uh, pf[f].lo, o[tb]);
          o[tb] = mfma16x16x32(ul, pf[f].hi, o[tb]);
          o[tb] = mfma16x16x32(uh, pf[f].hi, o[tb]);
        }
      }
      if constexpr (SAVE) {
        const int64_t rec = rec0 + static_cast<int64_t>(c) * a.H;
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
          *reinterpret_cast<f32x4*>(ca.yb + ((rec * n_rt + rt) * 4 + tb) * 256 + lane * 4) = o[tb];
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const int64_t t = 64LL * c + 16 * tb + l;
        if (a.y && t < sr.len && rr < a.dv)
          *reinterpret_cast<uint2*>(yp + t * a.sy.t) = make_uint2(pack2(o[tb][0], o[tb][1]), pack2(o[tb][2], o[tb][3]));
      }
      if (c + 1 < nc) scores(c + 1);
    }
    return;
  }

  // ---- states
  const TileLane<VW> tv = tile_lane<VW>(lane);
  const int r = r0 + index1(wave, l);
  const int64_t so = (head * a.dv + r) * a.dk;
  // segment states [head][n_seg][dv][dk], M [head][n_seg][dk][dk]
  const auto seg_at = [&](int s) { return (head * ca.n_seg + s) * a.dv * a.dk; };
  // A pass over the tokens in segments takes the call's first state from seg_s too,
  // where the STATES pass leaves it: its first segment would read it while the last
  // one writes the final state, which may be the same memory
  const float* given = a.state_in ? static_cast<const float*>(a.state_in) + head * a.dv * a.dk : nullptr;
  const float* from = ident                                  ? nullptr
                      : seg == 0 && (!OUT || ca.n_seg == 1)  ? given
                      : OUT && (seg > 0 || given != nullptr) ? ca.seg_s + seg_at(seg)
                                                             : nullptr;
  const __amdgpu_buffer_rsrc_t first = state_rsrc(from, a.dv, a.dk);
  f32x4 S[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) S[b] = load_f32x4(first, state_off(r, index4(b, g), a.dk));
  if (ident) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) S[b][q] = index4(b, g) + q == r ? 1.f : 0.f;
  }
  if (!OUT && seg == 0 && given && r < a.dv) {
    float* keep = ca.seg_s + seg_at(0) + static_cast<int64_t>(r) * a.dk;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (index4(b, g) < a.dk) *reinterpret_cast<f32x4*>(keep + index4(b, g)) = S[b];
  }
  bf16x8 yf[12];
  const uint16_t* yp = ca.yf + rec0 * kYf + lane * 8;
#pragma unroll
  for (int f = 0; f < 12; ++f)
    if (nc > 0) yf[f] = *reinterpret_cast<const bf16x8*>(yp + f * kFrag);
  const int rt = tile * NW + wave, n_rt = delta_row_tiles(a.dv);
  Pair8 sp[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) sp[s] = split8(S[2 * s], S[2 * s + 1]);
  for (int c = 0; c < nc; ++c) {
    lds_barrier();
    const int sl = c % 3;
    const char* kt = lds.k[sl];
    const float* gt = lds.gt[c & 1] + 4 * g;
    const auto gate = [&](int m, int tb) { return *reinterpret_cast<const f32x4*>(gt + 64 * m + 16 * tb); };
    // the next chunk's Y, fetched as this one's is used up
    yp += (c + 1 < nc ? static_cast<int64_t>(a.H) : 0) * kYf;
    uint16_t* sx = OUT ? lds.sx[c & 1][wave] + lane * 8 : nullptr;
    uint16_t* ux = OUT ? lds.ux[c & 1][wave] + lane * 8 : nullptr;
    f32x4 E[4], be[4], gm[4], rs[4];
    s16x4 vv[4];
    bf16x8 kf[2][NS], kc[NB];
    Pair8 z[2], u;
    bf16x8 ef[2];
    f32x4 x[4];
    // R = V - e^l (K S^T) and the operand beta R, a half of the tokens at a time
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
          E[2 * half + i] = mfma16x16x32(kf[i][s], sp[s].hi, s ? E[2 * half + i] : zero4());
          E[2 * half + i] = mfma16x16x32(kf[i][s], sp[s].lo, E[2 * half + i]);
        }
    };
    const auto residual = [&](int half) {
      f32x4 Z[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tb = 2 * half + i;
        const f32x4 v = widen(vv[tb]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          E[tb][q] = fmaf(-gm[tb][q], E[tb][q], v[q]);
          Z[i][q] = be[tb][q] * E[tb][q];
        }
      }
      z[half] = split8(Z[0], Z[1]);
    };
    // Y (beta R)
    const auto solve = [&](int half) {
#pragma unroll
      for (int s = 0; s <= half; ++s)
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ib = 2 * half + i, f = half ? 2 * ib - 2 + s : ib;
            x[ib] = mfma16x16x32(yf[2 * f + (m == 0)], m == 1 ? z[s].lo : z[s].hi, m + s ? x[ib] : zero4());
          }
    };
    // e, U for the output wave, and the operand e^(l_C - l) U
    const auto errors = [&](int half) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) E[2 * half + i][q] -= x[2 * half + i][q];
      if constexpr (SAVE) ef[half] = raw_order(round8(E[2 * half], E[2 * half + 1]), lane);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) E[2 * half + i][q] *= be[2 * half + i][q];
      if constexpr (OUT) {
        const Pair8 p = split8(E[2 * half], E[2 * half + 1]);
        *reinterpret_cast<bf16x8*>(ux + half * kFrag) = p.hi;
        *reinterpret_cast<bf16x8*>(ux + (2 + half) * kFrag) = p.lo;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) E[2 * half + i][q] *= rs[2 * half + i][q];
      u = split8(E[2 * half], E[2 * half + 1]);
    };
    const auto read_kc = [&](int half) {
#pragma unroll
      for (int b = 0; b < NB; ++b) kc[b] = frag_c<DK>(kt, tk, half, b);
    };
    const auto update = [&](const Pair8& p) {
#pragma unroll
      for (int b = 0; b < NB; ++b) S[b] = mfma16x16x32(kc[b], p.hi, S[b]);
#pragma unroll
      for (int b = 0; b < NB; ++b) S[b] = mfma16x16x32(kc[b], p.lo, S[b]);
    };

    read_k(0);
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      gm[tb] = gate(0, tb);
      be[tb] = gate(1, tb);
      rs[tb] = gate(2, tb);
      vv[tb] = col4<VW>(lds.v[c & 1], tv, tb, wave);
    }
    const float whole = lds.gt[c & 1][63];
    ks(0);
    if constexpr (OUT) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {  // S of this chunk for the output wave
        *reinterpret_cast<bf16x8*>(sx + s * kFrag) = sp[s].hi;
        *reinterpret_cast<bf16x8*>(sx + (NS + s) * kFrag) = sp[s].lo;
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) S[b][q] *= whole;
    read_k(1);
    interleave<4 * NS, 1, 2>();
    ks(1);
    residual(0);
    interleave<4 * NS, 1, 48 / (4 * NS)>();
    solve(0);
    residual(1);
    interleave<6, 1, 8>();
    read_kc(0);
    solve(1);
    errors(0);
#pragma unroll
    for (int f = 0; f < 4; ++f) yf[f] = *reinterpret_cast<const bf16x8*>(yp + f * kFrag);
    interleave<12, 1, 6>();
    const Pair8 u0 = u;
    update(u0);
    errors(1);
#pragma unroll
    for (int f = 4; f < 12; ++f) yf[f] = *reinterpret_cast<const bf16x8*>(yp + f * kFrag);
    interleave<2 * NB, 1, 72 / (2 * NB)>();
    read_kc(1);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      S[b] = mfma16x16x32(kc[b], u.hi, S[b]);
      S[b] = mfma16x16x32(kc[b], u.lo, S[b]);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) sp[s] = split8(S[2 * s], S[2 * s + 1]);
    __builtin_amdgcn_sched_group_barrier(0x8, 6, 0);
    interleave<(2 * NB - 6) / 2, 2, 12>();
    if constexpr (SAVE) {
      // after the loads of the next chunk's Y: these are waited for in the order
      // of issue, and a store before them would be waited for as well
      uint16_t* p = ca.ef + ((rec0 + static_cast<int64_t>(c) * a.H) * n_rt + rt) * 2 * kFrag + raw_at(lane);
      *reinterpret_cast<bf16x8*>(p) = ef[0];
      *reinterpret_cast<bf16x8*>(p + kFrag) = ef[1];
    }
  }
  lds_barrier();
  float* to = OUT ? (seg == ca.n_seg - 1 && a.state_out ? static_cast<float*>(a.state_out) + so : nullptr)
              : ident ? ca.seg_m + ((head * ca.n_seg + seg) * a.dk + r) * a.dk
                      : ca.seg_s + seg_at(seg + 1) + static_cast<int64_t>(r) * a.dk;
  if (r < (ident ? a.dk : a.dv)) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (index4(b, g) < a.dk) {
        if (to) *reinterpret_cast<f32x4*>(to + index4(b, g)) = S[b];
        if (SAVE && seg == ca.n_seg - 1) *reinterpret_cast<f32x4*>(ca.st + so + index4(b, g)) = S[b];
      }
  }
}

// First states of the segments: S_(s+1) = S_s M_s + Z_s, s = 1 .. n_seg - 2, in
// fp32; Z_s stands where S_(s+1) goes.  BACK: their last adjoints, Lam_(s-1) =
// Lam_s M_s^T + Z_s, s = n_seg - 2 .. 1.  A work-group has 16 rows of a head,
// which stay in LDS between the segments; wave w forms the column blocks w and
// w + 4 of 16.  Bound by latency: about 2 us a segment.
template <int DK, bool BACK>
__global__ __launch_bounds__(256) void delta_join(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16, P = DK + 4;
  __shared__ __align__(16) float rows[2][16 * P];
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (a.dv + 15) / 16;
  const int64_t head = blockIdx.x / tiles;
  const int r0 = static_cast<int>(blockIdx.x % tiles) * 16;
  const int nr = min(16, a.dv - r0);
  // rows r0.. of a segment's state or adjoint, zeros past dv and dk
  const auto at = [&](int s) { return (BACK ? ca.seg_l : ca.seg_s) + ((head * ca.n_seg + s) * a.dv + r0) * a.dk; };
  const auto states = [&](int s) { return buffer_rsrc(at(s), nr * a.dk * 4); };
  const __amdgpu_buffer_rsrc_t r1 = states(BACK ? ca.n_seg - 2 : 1);
  for (int i = threadIdx.x; i < 16 * DK; i += 256) {
    const int r = i / DK, c = i % DK;
    rows[0][r * P + c] = load4(r1, c < a.dk ? static_cast<uint32_t>((r * a.dk + c) * 4) : kPastEnd);
  }
  for (int n = 0; n + 2 < ca.n_seg; ++n) {
    const int s = BACK ? ca.n_seg - 2 - n : n + 1, next = BACK ? s - 1 : s + 1;
    const __amdgpu_buffer_rsrc_t rm = buffer_rsrc(ca.seg_m + (head * ca.n_seg + s) * a.dk * a.dk, a.dk * a.dk * 4);
    const __amdgpu_buffer_rsrc_t rz = states(next);
    const float* from = rows[n & 1];
    float* to = rows[(n + 1) & 1];
    float m[(NB + 3) / 4][NB][4];
    f32x4 x[(NB + 3) / 4];
#pragma unroll
    for (int i = 0; i < (NB + 3) / 4; ++i) {
      const int c = 16 * (w + 4 * i) + l;
      const uint32_t o = c < a.dk ? static_cast<uint32_t>(c * 4) : kPastEnd;
#pragma unroll
      for (int kb = 0; kb < NB; ++kb)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int k = 16 * kb + 4 * g + q;
          m[i][kb][q] = BACK ? load4(rm, c < a.dk && k < a.dk ? static_cast<uint32_t>((c * a.dk + k) * 4) : kPastEnd)
                             : load4(rm, o + k * a.dk * 4);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) x[i][q] = load4(rz, o + (4 * g + q) * a.dk * 4);
    }
    lds_barrier();
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
      const f32x4 sf = *reinterpret_cast<const f32x4*>(from + l * P + 16 * kb + 4 * g);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < (NB + 3) / 4; ++i)
          x[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(sf[q], m[i][kb][q], x[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < (NB + 3) / 4; ++i) {
      const int c = 16 * (w + 4 * i) + l;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 4 * g + q;
        to[r * P + c] = x[i][q];
        if (r < nr && c < a.dk) at(next)[r * a.dk + c] = x[i][q];
      }
    }
  }
}

template <int DK, int NW, int MODE>
hipError_t launch(const ChunkArgs& c, hipStream_t s) {
  constexpr int VW = 16 * NW;
  const int tiles = (c.a.dv + VW - 1) / VW + (MODE == STATES ? (c.a.dk + VW - 1) / VW : 0);
  const int64_t runs = c.a.N * c.a.H * (MODE == STATES ? c.n_seg - 1 : c.n_seg);
  const dim3 grid(static_cast<unsigned>(head_blocks(runs, tiles)));
  delta_chunk_fwd<DK, NW, MODE><<<grid, kFwdThreads<NW, MODE>, 0, s>>>(c);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_all(const ChunkArgs& c, hipStream_t s) {
  if (c.n_seg > 1) {
    hipError_t e = launch<DK, 4, STATES>(c, s);
    if (e != hipSuccess) return e;
    if ((e = launch_delta_join(c, false, s)) != hipSuccess) return e;
  }
  return c.sf ? launch<DK, 2, TRAINING>(c, s) : launch<DK, 2, OUTPUTS>(c, s);
}

}  // namespace

hipError_t launch_delta_join(const ChunkArgs& c, bool back, hipStream_t s) {
  if (c.n_seg <= 2) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(c.a.N * c.a.H * ((c.a.dv + 15) / 16)));
  if (c.a.dk <= 64) {
    if (back) delta_join<64, true><<<grid, 256, 0, s>>>(c);
    else delta_join<64, false><<<grid, 256, 0, s>>>(c);
  } else {
    if (back) delta_join<128, true><<<grid, 256, 0, s>>>(c);
    else delta_join<128, false><<<grid, 256, 0, s>>>(c);
  }
  return hipGetLastError();
}

hipError_t launch_delta_chunk_fwd(const ChunkArgs& c, hipStream_t s) {
  if (c.a.N * c.a.H == 0) return hipSuccess;
  return c.a.dk <= 64 ? launch_all<64>(c, s) : launch_all<128>(c, s);
}

}  // namespace gls
