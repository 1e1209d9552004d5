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

// ---- the decay's gradient.  dlog_alpha_t = <dL/dS_{t-1}, S_{t-1}>, and this
// product changes from token to token by dy.y - dv.v (k_delta_chunk_bwd.hip), so
// the recurrences carry it as a sum.  Its terms do not shrink with alpha_t, what
// they add up to does: where a token keeps little, rounding is all that is left of
// the difference (bf16, 330 tokens of uniform log_alpha: relative error 1.6e-2 at
// -5, 0.15 at -8, 150 at -15).  So
//   - a token that keeps less than 2^kForget starts the sum anew at zero (what is
//     dropped is below its rounding): nothing of later tokens' rounding reaches
//     earlier ones, and
//   - tokens that keep less than 2^kStrong get the sum of everything that crosses
//     them, every term of which has their factor (Crossing).
// Both ways at uniform log_alpha, bf16, 16 heads of 128, relative error of a head
// (median): 4096 tokens -3.3 sum 2.2e-3 / crossing 1.0e-3, -4 5.1e-3 / 6.5e-4, -5
// 1.1e-2 / 4e-4; 330 tokens 6e-4 / 9e-4, 2.0e-3 / 6e-4, 4.1e-3 / 4e-4.  kStrong (0.022)
// is where the sum's reaches what dq and dk have, not where the two are equal: the
// crossings cost a second pass over a chunk.  Steps of the decay are told from their
// whole parts (exact).
constexpr float kStrong = -5.5f, kForget = -23.5f;
__device__ __forceinline__ uint64_t tokens_below(float lw, float least) {
  return __ballot(lw - wave_shift_up(lw, 0.f) < least);
}
// The sum from the right over a chunk, x of token 63 - lane and z from the right of
// the chunk: what it is before token 63 - lane.
__device__ __forceinline__ float decay_sum(float x, float z, uint64_t forget, int lane) {
  if (forget == 0) return z + wave_scan_add(x);
  const bool anew = (forget >> (63 - lane)) & 1;
  float a = anew ? 0.f : 1.f, b = anew ? 0.f : x;
  wave_scan_affine(a, b);
  return fmaf(a, z, b);
}

// Work-groups of four waves look for the heads' chunks that have such tokens, 16
// at a time with all loads in flight (a work-group to each of 8 x 16 x 4096 / 64 took
// 9 us where there are none, this takes 4), and take those in turn: work(record, its
// tokens as bits).  A slot that holds no chunk may show any bits.
template <typename F>
__device__ __forceinline__ void for_strong(const ChunkArgs& ca, uint64_t (&found)[16], int w, int lane, F&& work) {
  const uint32_t n = static_cast<uint32_t>(ca.slots * ca.a.H), step = gridDim.x;
  for (uint32_t first = blockIdx.x; first < n; first = n - first > 16 * step ? first + 16 * step : n) {
    const auto record = [&](int i) { return first + static_cast<uint64_t>(i) * step; };
    float lw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint64_t r = record(4 * w + u);
      lw[u] = ca.gates[(r < n ? r : n - 1) * kGates + 192 + lane];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint64_t bits = tokens_below(lw[u], kStrong);
      if (lane == 0) found[4 * w + u] = record(4 * w + u) < n ? bits : 0;
    }
    __syncthreads();
    for (uint64_t left = __ballot(lane < 16 && found[lane & 15] != 0); left != 0; left &= left - 1) {
      const int i = __builtin_ctzll(left);
      work(static_cast<int64_t>(record(i)), found[i]);
    }
    __syncthreads();
  }
}
// Their number: as many as the card holds at once, per_cu of 256.
inline dim3 seek_groups(const ChunkArgs& c, int per_cu) {
  const int64_t n = c.slots * c.a.H, most = 256 * per_cu;
  return dim3(static_cast<unsigned>(n < most ? n : most));
}

// What crosses a token of a chunk: with m_ij (j < i) what goes from the write of
// token j to what token i makes of it, a_i from the chunk's first state to token i, b_j
// from token j to the chunk's end and c from end to end, before token t
//   sum_{i >= t > j} m_ij + sum_{i >= t} a_i + sum_{j < t} b_j + c.
// No term is taken off again: each sum takes in only what has the factors of all
// tokens that it crosses.
struct Crossing {
  float m[64 * 65];
  // m_ij -> sums over i' >= i, by one wave (lane = j); m is set below the diagonal
  __device__ __forceinline__ void gather(int lane) {
    float x = 0.f;
#pragma unroll 8
    for (int i = 63; i > 0; --i) {
      x += i > lane ? m[i * 65 + lane] : 0.f;
      if (i > lane) m[i * 65 + lane] = x;
    }
  }
  // after a barrier, by one wave (lane = t)
  __device__ __forceinline__ float at(float a, float b, float c, int lane) const {
    float x = 0.f;
#pragma unroll 8
    for (int j = 0; j < 63; ++j) x += j < lane ? m[lane * 65 + j] : 0.f;
    const float from = wave_reverse(wave_scan_add(wave_reverse(a, lane)), lane);
    return ((x + from) + wave_shift_up(wave_scan_add(b), 0.f)) + c;
  }
};

}  // namespace gls
