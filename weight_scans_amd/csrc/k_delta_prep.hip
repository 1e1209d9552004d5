// k_delta_prep.hip -- what a chunk of the gated delta rule is in itself, for all
// chunks in parallel: with l the cumulative log decay of the chunk's 64 tokens,
//
//   L_ij = e^(l_i - l_j) k_i.k_j  (j < i),   P_ij = scale e^(l_i - l_j) q_i.k_j  (j <= i)
//   Y = (I + L beta)^-1 L,  so that  e = r - Y (beta r)  for  r = v - e^l S k
//
// and the gates' factors.  One work-group of four waves per chunk and value
// head.  The scores run in both orientations (operands exchanged) on the bf16
// matrix cores, straight from global memory: each orientation is the operand
// form of one later product.  Y in fp32: wave w inverts its 16 x 16 diagonal
// block I + B (B = L beta) by substitution, a column per lane; then wave j
// takes column block j down its rows, Y_ij = N_i (L_ij - sum_k B_ik Y_kj), with
// v_mfma_f32_16x16x4_f32, each result feeding the next product in registers.
//
// The cumulative decay is kept as whole part and fraction (log2): whole parts
// add exactly, so that differences stay exact to 2^-19 however many tokens of
// the chunk forget everything (log_alpha = -inf counts as 2^-200).
#include "delta_mfma.hpp"
#include "dev_common.hpp"

namespace gls {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// c + A B of 16 x 16 blocks: A with rows in lanes (value q: column 4g + q), B
// in result layout.
__device__ __forceinline__ f32x4 mul16(const f32x4& a, const f32x4& b, f32x4 c) {
#pragma unroll
  for (int q = 0; q < 4; ++q) c = mfma_f32(a[q], b[q], c);
  return c;
}

template <int DK>
__global__ __launch_bounds__(kThreads) void delta_prep(ChunkArgs ca) {
  const DeltaArgs& a = ca.a;
  constexpr int NS = DK / 32;
  __shared__ float gw[64], gf[64], gb[64];
  __shared__ __align__(16) float Lr[10][256], Ba[6][256], Na[4][256], Bd[4][16 * 20], Yt[4][16 * 20];
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = static_cast<int>(blockIdx.x % a.H);
  const int64_t slot = blockIdx.x / a.H, rec = slot * a.H + h;
  const int hk = h / (a.H / a.Hk);

  // the slot's sequence and first token
  int64_t n, c;
  if (a.cu) {
    int64_t lo = 0, hi = a.N - 1;  // last n with slot0(n) <= slot
    while (lo < hi) {
      const int64_t m = (lo + hi + 1) / 2;
      if (chunk_slot0(true, m, seq_range(a.cu, m, a.T).t0, a.T, kDeltaChunk) <= slot) lo = m;
      else hi = m - 1;
    }
    n = lo;
    c = slot - chunk_slot0(true, n, seq_range(a.cu, n, a.T).t0, a.T, kDeltaChunk);
  } else {
    const uint32_t nc = static_cast<uint32_t>((a.T + kDeltaChunk - 1) / kDeltaChunk);
    n = static_cast<uint32_t>(slot) / nc;
    c = static_cast<uint32_t>(slot) % nc;
  }
  const SeqRange sr = seq_range(a.cu, n, a.T);
  const int64_t t0 = c * kDeltaChunk;
  if (c < 0 || t0 >= sr.len) return;
  const int nt = static_cast<int>(sr.len - t0 < 64 ? sr.len - t0 : 64);

  // gates: lane = token (every wave the same)
  float x2 = 0.f, be = 0.f;
  if (lane < nt) {
    const int64_t o = sr.b * a.sg.b + h * a.sg.h + (sr.t0 + t0 + lane) * a.sg.t;
    const float la = a.gate_io ? bf16_to_f32(static_cast<const uint16_t*>(a.la)[o]) : static_cast<const float*>(a.la)[o];
    be = a.gate_io ? bf16_to_f32(static_cast<const uint16_t*>(a.be)[o]) : static_cast<const float*>(a.be)[o];
    x2 = fmaxf(la * 1.44269504088896f, -200.f);
  }
  const float xw = rintf(x2);
  const float lw = wave_scan_add(xw), lf = wave_scan_add(x2 - xw);
  if (w == 0) {
    gw[lane] = lw;
    gf[lane] = lf;
    gb[lane] = be;
    float* gt = ca.gates + rec * kGates;
    gt[lane] = fexp2(lw + lf);
    gt[64 + lane] = be;
    gt[128 + lane] = fexp2((readlane_f(lw, 63) - lw) + (readlane_f(lf, 63) - lf));
    gt[192 + lane] = lw;
    gt[256 + lane] = lf;
    if (ca.ytf) {  // training only
#pragma unroll
      for (int x = 1; x < 4; ++x) {
        const float mw = readlane_f(lw, 16 * x - 1), mf = readlane_f(lf, 16 * x - 1);
        if (lane >> 4 == x) gt[320 + lane] = fexp2((lw - mw) + (lf - mf));
        if (lane < 16 * x) gt[320 + 64 * x + lane] = fexp2((mw - lw) + (mf - lf));
      }
    }
  }
  __syncthreads();

  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + (sr.t0 + t0) * a.sk.t;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + (sr.t0 + t0) * a.sq.t;
  // rows past the chunk's end and columns past dk read as zeros
  const __amdgpu_buffer_rsrc_t rk = buffer_rsrc(kp, static_cast<int>(((nt - 1) * a.sk.t + a.dk) * 2));
  const __amdgpu_buffer_rsrc_t rq = buffer_rsrc(qp, static_cast<int>(((nt - 1) * a.sq.t + a.dk) * 2));
  const auto row = [&](const __amdgpu_buffer_rsrc_t& r, int64_t st, int tb, int s) {
    const int col = 32 * s + 8 * g;
    return load16(r, col < a.dk ? static_cast<uint32_t>(((16 * tb + l) * static_cast<int>(st) + col) * 2) : kPastEnd);
  };
  bf16x8 kf[4][NS];
#pragma unroll
  for (int tb = 0; tb < 4; ++tb)
#pragma unroll
    for (int s = 0; s < NS; ++s) kf[tb][s] = row(rk, a.sk.t, tb, s);

  // decay e^(l_i - l_j), zero above the diagonal (and on it for `strict`)
  const auto decay = [&](int i, int j, bool strict) {
    const float d = fexp2((gw[i] - gw[j]) + (gf[i] - gf[j]));
    return j < i || (j == i && !strict) ? d : 0.f;
  };
  const auto tri = [](int i, int j) { return i * (i + 1) / 2 + j; };

  // L: row block w.  Result form [i][j] -> Lr; exchanged [j][i], times -beta_j,
  // is the operand form of -B.
#pragma unroll
  for (int wc = 0; wc < 4; ++wc) {
    if (wc != w) continue;
#pragma unroll
    for (int j = 0; j <= wc; ++j) {
      f32x4 x = zero4(), xt = zero4();
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        x = mfma16x16x32(kf[wc][s], kf[j][s], x);
        xt = mfma16x16x32(kf[j][s], kf[wc][s], xt);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] *= decay(16 * wc + 4 * g + q, 16 * j + l, true);
        xt[q] *= -gb[16 * j + 4 * g + q] * decay(16 * wc + l, 16 * j + 4 * g + q, true);
      }
      *reinterpret_cast<f32x4*>(&Lr[tri(wc, j)][lane * 4]) = x;
      if (j < wc) *reinterpret_cast<f32x4*>(&Ba[wc * (wc - 1) / 2 + j][lane * 4]) = xt;
      else *reinterpret_cast<f32x4*>(&Bd[w][l * 20 + 4 * g]) = xt;  // -B, row-major
    }
  }
  // inverse of the diagonal block: lane l has column l; N_r = delta - sum B_rk N_k
  {
    float nn[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == l ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < r; ++k) s = fmaf(Bd[w][r * 20 + k], nn[k], s);
      nn[r] = s;
    }
    // operand form: lane l has row l, columns 4g..4g+3 (all four g hold the same columns)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if ((r >> 2) == g) Yt[w][r * 20 + l] = nn[r];
    *reinterpret_cast<f32x4*>(&Na[w][lane * 4]) = *reinterpret_cast<const f32x4*>(&Yt[w][l * 20 + 4 * g]);
  }
  __syncthreads();

  // Y, column block w
  f32x4 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = zero4();
    if (i < w) continue;
    f32x4 t = *reinterpret_cast<const f32x4*>(&Lr[tri(i, w)][lane * 4]);
#pragma unroll
    for (int k = 0; k < i; ++k)
      if (k >= w) t = mul16(*reinterpret_cast<const f32x4*>(&Ba[i * (i - 1) / 2 + k][lane * 4]), y[k], t);
    y[i] = mul16(*reinterpret_cast<const f32x4*>(&Na[i][lane * 4]), t, zero4());
  }
  __syncthreads();  // Lr is free
  const auto put = [&](uint16_t* dst, const bf16x8& f) {
    *reinterpret_cast<bf16x8*>(dst + lane * 8) = f;
  };
  if (ca.ytf) {  // rows j = this wave's columns: the results as they are
    uint16_t* o = ca.ytf + rec * kYf;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s < w / 2) continue;
      const Pair8 p = split8(y[2 * s], y[2 * s + 1]);
      const int f = w < 2 ? 2 * w + s : w + 2;
      put(o + (2 * f) * kFrag, p.hi);
      put(o + (2 * f + 1) * kFrag, p.lo);
    }
  }
  // the other orientation through LDS: block (i, w) row-major in Lr
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) Yt[w][(4 * g + q) * 20 + l] = y[i][q];
    *reinterpret_cast<f32x4*>(&Lr[tri(i, w)][lane * 4]) = *reinterpret_cast<const f32x4*>(&Yt[w][l * 20 + 4 * g]);
  }
  __syncthreads();
  {
    uint16_t* o = ca.yf + rec * kYf;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s > w / 2) continue;
      const f32x4 u = *reinterpret_cast<const f32x4*>(&Lr[tri(w, 2 * s)][lane * 4]);
      const f32x4 v = 2 * s + 1 <= w ? *reinterpret_cast<const f32x4*>(&Lr[tri(w, 2 * s + 1)][lane * 4]) : zero4();
      const Pair8 p = split8(u, v);
      const int f = w < 2 ? w : 2 * w - 2 + s;
      put(o + (2 * f) * kFrag, p.hi);
      put(o + (2 * f + 1) * kFrag, p.lo);
    }
  }

  // P: row block w (rows i in lanes), and for training column block w (rows j
  // in lanes)
  const float sc = static_cast<float>(a.scale);
  bf16x8 qf[4][NS];
#pragma unroll
  for (int tb = 0; tb < 4; ++tb)
#pragma unroll
    for (int s = 0; s < NS; ++s)
      qf[tb][s] = row(rq, a.sq.t, tb, s);
#pragma unroll
  for (int wc = 0; wc < 4; ++wc) {
    if (wc != w) continue;
    f32x4 p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = zero4();
      if (j > wc) continue;
#pragma unroll
      for (int s = 0; s < NS; ++s) p[j] = mfma16x16x32(kf[j][s], qf[wc][s], p[j]);
#pragma unroll
      for (int q = 0; q < 4; ++q) p[j][q] *= sc * decay(16 * wc + l, 16 * j + 4 * g + q, false);
    }
    uint16_t* o = ca.pf + rec * kYf;
#pragma unroll
    for (int s = 0; s <= wc / 2; ++s) {
      const Pair8 pr = split8(p[2 * s], p[2 * s + 1]);
      const int f = wc < 2 ? wc : 2 * wc - 2 + s;
      put(o + (2 * f) * kFrag, pr.hi);
      put(o + (2 * f + 1) * kFrag, pr.lo);
    }
    if (ca.ptf) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = zero4();
        if (i < wc) continue;
#pragma unroll
        for (int s = 0; s < NS; ++s) p[i] = mfma16x16x32(qf[i][s], kf[wc][s], p[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) p[i][q] *= sc * decay(16 * i + 4 * g + q, 16 * wc + l, false);
      }
      uint16_t* ot = ca.ptf + rec * kYf;
#pragma unroll
      for (int s = wc / 2; s < 2; ++s) {
        const Pair8 pr = split8(p[2 * s], p[2 * s + 1]);
        const int f = wc < 2 ? 2 * wc + s : wc + 2;
        put(ot + (2 * f) * kFrag, pr.hi);
        put(ot + (2 * f + 1) * kFrag, pr.lo);
      }
    }
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
