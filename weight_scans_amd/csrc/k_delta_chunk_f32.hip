// k_delta_chunk_f32.hip -- the gated delta rule over the chunks of a sequence in
// fp32, forward.  Per chunk of 64 tokens, with S the state before it and Y, P as
// the bf16 chunks have them:
//
//   R = V - e^l (K S^T),  E = R - Y (beta R),  U = beta E
//   y = scale e^l (Q S^T) + P U,   S <- e^(l_C) S + U^T (e^(l_C - l) K)
//
// All products are v_mfma_f32_16x16x4_f32, whose results chain as operands in
// registers (delta_f32.hpp): 16 rows of S go through the sequence in one
// work-group, as in bf16, here in two waves: at the fp32 matrix rate a chunk's
// chain in one wave took 3.6 us (64 x 64), in two with their exchanges 2.3.  4 x 8 x
// 1024 x 64 takes 15 us to prepare and 37 us (in one wave 58; token by token both
// 340); at 8 x 16 x 4096 x 64, where all CUs are busy, 447 us against 414 in all.
#include <type_traits>

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

// A work-group has 16 rows of S.  The products of a chunk are shared by two state
// waves (the fp32 matrix rate of one SIMD bounds their chain), two output waves
// follow one chunk behind, and one wave loads the next chunk's K; V, Y, Q and P
// go straight to registers.  Part p of either pair has the token blocks 0 and 3,
// or 1 and 2 (five of the ten blocks of Y or P each), and the columns of S in
// halves.  Three barriers a chunk: S, R and U are exchanged through LDS.
template <int DK>
struct F32Lds {
  alignas(16) char k[2][64 * DK * 4];
  alignas(16) float gt[2][192];
  alignas(16) float sx[3][DK * 16];  // S^T before the chunk, blocks of 16
  alignas(16) float zx[64 * 16];     // -beta R
  alignas(16) float ux[2][64 * 16];  // U
};
constexpr int kF32Threads = 5 * 64;

template <int DK, bool SAVE>
__global__ __launch_bounds__(kF32Threads) void delta_chunk_f32(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NB = DK / 16, HB = NB / 2;
  __shared__ F32Lds<DK> lds;
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = SAVE ? delta_row_tiles(a.dv) : (a.dv + 15) / 16;
  int64_t head;
  int rt;
  if (!head_of_block(blockIdx.x, tiles, a.N * a.H, head, rt)) return;
  const int h = static_cast<int>(head % a.H);
  const int64_t n = head / a.H;
  const int hk = h / (a.H / a.Hk), r0 = 16 * rt, n_rt = delta_row_tiles(a.dv);
  const SeqRange sr = seq_range(a.cu, n, a.T);
  const int nc = static_cast<int>((sr.len + kDeltaChunk - 1) / kDeltaChunk);
  const int64_t slot0 = chunk_slot0(a.cu != nullptr, n, sr.t0, a.T, kDeltaChunk);
  const int64_t rec0 = slot0 * a.H + h;
  const auto rec_of = [&](int c) { return rec0 + static_cast<int64_t>(c) * a.H; };

  if (wave == 4) {  // ---- loads: K and gates, one chunk ahead
    constexpr int NK = DK / 4;
    const float* kp = static_cast<const float*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
    uint32_t ko[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) ko[i] = tile_off_f32<DK>(i, lane, a.sk.t, a.dk);
    const auto issue = [&](int c) {
      const bool in = c < nc;
      const __amdgpu_buffer_rsrc_t rk = rows_f32(kp, c * 64LL, in ? sr.len : 0, a.sk.t, a.dk);
      const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(ca.gates + (in ? rec_of(c) * kGates : 0), in ? 768 : 0);
#pragma unroll
      for (int i = 0; i < NK; ++i) dma16(rk, ko[i], lds.k[c & 1] + i * 1024);
#pragma unroll
      for (int i = 0; i < 3; ++i) dma4(rg, (i * 64 + lane) * 4, lds.gt[c & 1] + i * 64);
    };
    issue(0);
    for (int c = 0; c <= nc; ++c) {
      wait_vm<0>();
      lds_barrier();
      if (c == nc) break;
      issue(c + 1);  // into the slot of chunk c - 1
      lds_barrier();
      lds_barrier();
    }
    wait_vm<0>();
    return;
  }

  const auto outputs = [&](auto part) {  // ---- one chunk behind
    using Pt = Part<decltype(part)::value>;
    const int rr = r0 + 4 * g;
    float* yp = static_cast<float*>(a.y) + sr.b * a.sy.b + h * a.sy.h + sr.t0 * a.sy.t + rr;
    const float* qp = static_cast<const float*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
    const float sc = static_cast<float>(a.scale);
    uint32_t qo[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      qo[b] = 16 * b + 4 * g < a.dk ? static_cast<uint32_t>((l * static_cast<int>(a.sq.t) + 16 * b + 4 * g) * 4)
                                    : kPastEnd;
    f32x4 qf[2][NB], pf[5];
    float gs[2];
    const auto fetch = [&](int c) {
      const int64_t rec = rec_of(c);
      const __amdgpu_buffer_rsrc_t rq = rows_f32(qp, c * 64LL, sr.len, a.sq.t, a.dk);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          qf[x][b] = load_f32x4(rq, qo[b] + static_cast<uint32_t>(Pt::tb(x) * 64 * static_cast<int>(a.sq.t)));
#pragma unroll
        for (int j = 0; j < Pt::count(x); ++j)
          pf[Pt::block(x, j)] = *reinterpret_cast<const f32x4*>(ca.p32 + rec * kY32 +
                                                                SolveLds::tri(Pt::tb(x), j) * 256 + lane * 4);
        gs[x] = sc * ca.gates[rec * kGates + 16 * Pt::tb(x) + l];
      }
    };
    if (nc > 0) fetch(0);
    lds_barrier();
    for (int c = 0; c < nc; ++c) {
      // the two inner barriers of step c, then the one that begins step c + 1;
      // the work on chunk c stands between those of step c + 1
      if (c == 0) {
        lds_barrier();
        lds_barrier();
      }
      lds_barrier();
      const float* sx = lds.sx[c % 3] + lane * 4;
      const float* ux = lds.ux[c & 1] + lane * 4;
      f32x4 o[2] = {zero4(), zero4()};
      const auto states = [&](int b) {
        const f32x4 sf = *reinterpret_cast<const f32x4*>(sx + b * 256);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int x = 0; x < 2; ++x) o[x] = mfma_f32(sf[q], qf[x][b][q], o[x]);
      };
      const bool more = c + 1 < nc;  // step c + 1 has inner barriers
#pragma unroll
      for (int b = 0; b < HB; ++b) states(b);
      if (more) lds_barrier();
#pragma unroll
      for (int b = HB; b < NB; ++b) states(b);
      if (more) lds_barrier();
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[x][q] *= gs[x];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 uf = *reinterpret_cast<const f32x4*>(ux + j * 256);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (j >= Pt::count(x)) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[x] = mfma_f32(uf[q], pf[Pt::block(x, j)][q], o[x]);
        }
      }
      fetch(min(c + 1, nc - 1));
      if constexpr (SAVE) {
#pragma unroll
        for (int b = HB * decltype(part)::value; b < HB * decltype(part)::value + HB; ++b)
          *reinterpret_cast<f32x4*>(ca.s32 + ((rec_of(c) * n_rt + rt) * NB + b) * 256 + lane * 4) =
              turned_f32(lds.sx[c % 3] + b * 256, lane);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int64_t t = 64LL * c + 16 * Pt::tb(x) + l;
        if constexpr (SAVE)
          *reinterpret_cast<f32x4*>(ca.yb + (rec_of(c) * 64 + 16 * Pt::tb(x) + l) * (16 * n_rt) + rr) = o[x];
        if (a.y && t < sr.len && rr < a.dv) *reinterpret_cast<f32x4*>(yp + t * a.sy.t) = o[x];
      }
    }
  };
  if (wave == 2) return outputs(std::integral_constant<int, 0>{});
  if (wave == 3) return outputs(std::integral_constant<int, 1>{});

  const auto states = [&](auto part) {
    constexpr int P = decltype(part)::value, B0 = HB * P, OB = HB - B0;  // own columns, the other's
    using Pt = Part<P>;
    const int r = r0 + l;
    const __amdgpu_buffer_rsrc_t first = state_rsrc(
        a.state_in ? static_cast<const float*>(a.state_in) + head * a.dv * a.dk : nullptr, a.dv, a.dk);
    f32x4 S[HB];
#pragma unroll
    for (int b = 0; b < HB; ++b) S[b] = load_f32x4(first, state_off(r, 16 * (B0 + b) + 4 * g, a.dk));
#pragma unroll
    for (int b = 0; b < HB; ++b) *reinterpret_cast<f32x4*>(lds.sx[0] + (B0 + b) * 256 + lane * 4) = S[b];
    const float* vp = static_cast<const float*>(a.v) + sr.b * a.sv.b + h * a.sv.h + sr.t0 * a.sv.t;
    uint32_t vo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      vo[q] = r < a.dv ? static_cast<uint32_t>(((4 * g + q) * static_cast<int>(a.sv.t) + r) * 4) : kPastEnd;
    f32x4 V[2], yf[5];
    const auto fetch = [&](int c) {
      const __amdgpu_buffer_rsrc_t rv = rows_f32(vp, c * 64LL, sr.len, a.sv.t, a.dv);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          V[x][q] = load4(rv, vo[q] + static_cast<uint32_t>(Pt::tb(x) * 64 * static_cast<int>(a.sv.t)));
#pragma unroll
        for (int j = 0; j < Pt::count(x); ++j)
          yf[Pt::block(x, j)] = *reinterpret_cast<const f32x4*>(ca.y32 + rec_of(c) * kY32 +
                                                                SolveLds::tri(Pt::tb(x), j) * 256 + lane * 4);
      }
    };
    if (nc > 0) fetch(0);
    const uint32_t ka = row_at<DK>(lane);
    const uint32_t kc[4] = {col_at<DK>(lane, 0), col_at<DK>(lane, 1), col_at<DK>(lane, 2), col_at<DK>(lane, 3)};
    for (int c = 0; c < nc; ++c) {
      lds_barrier();
      const char* kt = lds.k[c & 1];
      const float* gt = lds.gt[c & 1] + 4 * g;
      const auto gate = [&](int m, int tb) { return *reinterpret_cast<const f32x4*>(gt + 64 * m + 16 * tb); };
      const auto block = [&](const float* x, int b) { return *reinterpret_cast<const f32x4*>(x + b * 256 + lane * 4); };
      const auto put = [&](float* x, int b, const f32x4& v) { *reinterpret_cast<f32x4*>(x + b * 256 + lane * 4) = v; };
      const float* sx = lds.sx[c % 3];
      // R and -beta R of the own tokens
      f32x4 E[2] = {zero4(), zero4()}, be[2];
      const auto scores = [&](int b, const f32x4& s) {
        f32x4 kf[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) kf[x] = row_frag<DK>(kt, ka, Pt::tb(x), b);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int x = 0; x < 2; ++x) E[x] = mfma_f32(kf[x][q], s[q], E[x]);
      };
#pragma unroll
      for (int b = 0; b < HB; ++b) scores(B0 + b, S[b]);
#pragma unroll
      for (int b = 0; b < HB; ++b) scores(OB + b, block(sx, OB + b));
      const float whole = lds.gt[c & 1][63];
#pragma unroll
      for (int b = 0; b < HB; ++b) S[b] *= whole;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const f32x4 gm = gate(0, Pt::tb(x));
        be[x] = gate(1, Pt::tb(x));
        f32x4 z;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          E[x][q] = fmaf(-gm[q], E[x][q], V[x][q]);
          z[q] = -be[x][q] * E[x][q];
        }
        put(lds.zx, Pt::tb(x), z);
      }
      lds_barrier();
      // E = R - Y (beta R)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= Pt::count(0) && j >= Pt::count(1)) continue;
        const f32x4 z = block(lds.zx, j);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (j < Pt::count(x)) E[x] = mfma_f32(yf[Pt::block(x, j)][q], z[q], E[x]);
      }
      fetch(min(c + 1, nc - 1));
#pragma unroll
      for (int x = 0; x < 2; ++x) put(lds.ux[c & 1], Pt::tb(x), E[x] * be[x]);
      if constexpr (SAVE) {
        const int VP = 16 * n_rt;
        const __amdgpu_buffer_rsrc_t re = buffer_rsrc(ca.e32 + rec_of(c) * 64 * VP, 256 * VP);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          store_rows(re, static_cast<uint32_t>((4 * g * VP + r) * 4), VP, Pt::tb(x), E[x]);
      }
      lds_barrier();
      // the own columns of S
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const f32x4 u = block(lds.ux[c & 1], tb) * gate(2, tb);
        f32x4 kf[HB];
#pragma unroll
        for (int b = 0; b < HB; ++b) kf[b] = col_frag<DK>(kt, kc, tb, B0 + b);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int b = 0; b < HB; ++b) S[b] = mfma_f32(kf[b][q], u[q], S[b]);
      }
#pragma unroll
      for (int b = 0; b < HB; ++b) put(lds.sx[(c + 1) % 3], B0 + b, S[b]);
    }
    lds_barrier();
    if (r < a.dv) {
      const int64_t so = (head * a.dv + r) * a.dk;
#pragma unroll
      for (int b = 0; b < HB; ++b) {
        const int c = 16 * (B0 + b) + 4 * g;
        if (c >= a.dk) continue;
        if (a.state_out) *reinterpret_cast<f32x4*>(static_cast<float*>(a.state_out) + so + c) = S[b];
        if constexpr (SAVE) *reinterpret_cast<f32x4*>(ca.st + so + c) = S[b];
      }
    }
  };
  if (wave == 0) states(std::integral_constant<int, 0>{});
  else states(std::integral_constant<int, 1>{});
}

template <int DK>
hipError_t launch(const ChunkArgs& c, hipStream_t s) {
  const int64_t n = c.slots * c.a.H;
  if (n > 0) {
    delta_prep_f32<DK><<<dim3(static_cast<unsigned>(n)), 256, 0, s>>>(c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int tiles = c.s32 ? delta_row_tiles(c.a.dv) : (c.a.dv + 15) / 16;
  const dim3 grid(static_cast<unsigned>(head_blocks(c.a.N * c.a.H, tiles)));
  if (c.s32) delta_chunk_f32<DK, true><<<grid, kF32Threads, 0, s>>>(c);
  else delta_chunk_f32<DK, false><<<grid, kF32Threads, 0, s>>>(c);
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
  return c.a.dk <= 64 ? launch<64>(c, s) : launch<128>(c, s);
}

}  // namespace gls
