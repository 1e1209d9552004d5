// delta_solve.hpp -- what the chunk preparations share: the gates' factors, and
// Y = (I + B)^-1 L of a 64 x 64 chunk in fp32 by blocks of 16 (four waves).
#pragma once

#include "delta_mfma.hpp"

namespace gls {

// Sequence and chunk of a slot; false if the slot holds none.
__device__ __forceinline__ bool chunk_of_slot(const DeltaArgs& a, int64_t slot, SeqRange& sr, int64_t& t0) {
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
  sr = seq_range(a.cu, n, a.T);
  t0 = c * kDeltaChunk;
  return c >= 0 && t0 < sr.len;
}

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

struct SolveLds {
  float gw[64], gf[64], gb[64];  // cumulative log2 decay, whole and fraction; beta
  // L by blocks (result layout), -B below the diagonal and the inverses of the
  // diagonal blocks (operand layout), -B on the diagonal and a turning place
  // (row-major)
  alignas(16) float Lr[10][256], Ba[6][256], Na[4][256], Bd[4][16 * 20], Yt[4][16 * 20];
  __device__ static constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }
  // e^(l_i - l_j), zero above the diagonal (and on it for `strict`)
  __device__ __forceinline__ float decay(int i, int j, bool strict) const {
    const float d = fexp2((gw[i] - gw[j]) + (gf[i] - gf[j]));
    return j < i || (j == i && !strict) ? d : 0.f;
  }
};

// Gates of a chunk (every wave; lane = token): into LDS and, by wave 0, into
// the record.  la and be are log_alpha and beta (0 past the chunk's end).
__device__ __forceinline__ void chunk_gate_factors(SolveLds& s, float* gt, float la, float be, bool between, int w,
                                                   int lane) {
  // not fmaxf: a log_alpha that is no number stays one
  const float la2 = la * 1.44269504088896f, x2 = la2 < -200.f ? -200.f : la2;
  const float xw = rintf(x2);
  const float lw = wave_scan_add(xw), lf = wave_scan_add(x2 - xw);
  if (w != 0) return;
  s.gw[lane] = lw;
  s.gf[lane] = lf;
  s.gb[lane] = be;
  gt[lane] = fexp2(lw + lf);
  gt[64 + lane] = be;
  gt[128 + lane] = fexp2((readlane_f(lw, 63) - lw) + (readlane_f(lf, 63) - lf));
  gt[192 + lane] = lw;
  gt[256 + lane] = lf;
  if (between) {
#pragma unroll
    for (int x = 1; x < 4; ++x) {
      const float mw = readlane_f(lw, 16 * x - 1), mf = readlane_f(lf, 16 * x - 1);
      if (lane >> 4 == x) gt[320 + lane] = fexp2((lw - mw) + (lf - mf));
      if (lane < 16 * x) gt[320 + 64 * x + lane] = fexp2((mw - lw) + (mf - lf));
    }
  }
}

// Scores k_i.k_j of block (w, j) in both orientations (x: [i][j], xt: [j][i])
// -> L and -B in LDS.
__device__ __forceinline__ void put_scores(SolveLds& s, int w, int j, f32x4 x, f32x4 xt, int lane) {
  const int l = lane & 15, g = lane >> 4;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    x[q] *= s.decay(16 * w + 4 * g + q, 16 * j + l, true);
    xt[q] *= -s.gb[16 * j + 4 * g + q] * s.decay(16 * w + l, 16 * j + 4 * g + q, true);
  }
  *reinterpret_cast<f32x4*>(&s.Lr[SolveLds::tri(w, j)][lane * 4]) = x;
  if (j < w) *reinterpret_cast<f32x4*>(&s.Ba[w * (w - 1) / 2 + j][lane * 4]) = xt;
  else *reinterpret_cast<f32x4*>(&s.Bd[w][l * 20 + 4 * g]) = xt;
}

// Inverse of I + B's diagonal block w by substitution: lane l has column l,
// N_r = delta - sum_k B_rk N_k.
__device__ __forceinline__ void invert_diagonal(SolveLds& s, int w, int lane) {
  const int l = lane & 15, g = lane >> 4;
  float nn[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float x = r == l ? 1.f : 0.f;
#pragma unroll
    for (int k = 0; k < r; ++k) x = fmaf(s.Bd[w][r * 20 + k], nn[k], x);
    nn[r] = x;
  }
  // operand form: lane l has row l, columns 4g..4g+3 (all four g hold the same columns)
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if ((r >> 2) == g) s.Yt[w][r * 20 + l] = nn[r];
  *reinterpret_cast<f32x4*>(&s.Na[w][lane * 4]) = *reinterpret_cast<const f32x4*>(&s.Yt[w][l * 20 + 4 * g]);
}

// Column block w of Y in result layout (after a barrier): Y_ij = N_i (L_ij - sum_k B_ik Y_kj).
__device__ __forceinline__ void solve_column(const SolveLds& s, int w, int lane, f32x4 (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = zero4();
    if (i < w) continue;
    f32x4 t = *reinterpret_cast<const f32x4*>(&s.Lr[SolveLds::tri(i, w)][lane * 4]);
#pragma unroll
    for (int k = 0; k < i; ++k)
      if (k >= w) t = mul16(*reinterpret_cast<const f32x4*>(&s.Ba[i * (i - 1) / 2 + k][lane * 4]), y[k], t);
    y[i] = mul16(*reinterpret_cast<const f32x4*>(&s.Na[i][lane * 4]), t, zero4());
  }
}

// The other orientation: block (i, w) with rows i in lanes, into Lr (free after
// a barrier behind solve_column).
__device__ __forceinline__ void turn_column(SolveLds& s, int w, int lane, const f32x4 (&y)[4]) {
  const int l = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) s.Yt[w][(4 * g + q) * 20 + l] = y[i][q];
    *reinterpret_cast<f32x4*>(&s.Lr[SolveLds::tri(i, w)][lane * 4]) =
        *reinterpret_cast<const f32x4*>(&s.Yt[w][l * 20 + 4 * g]);
  }
}

}  // namespace gls
