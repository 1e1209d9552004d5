// ssm_scan.hpp -- what the forward and the backward of the selective scan share:
// how a work-group cuts a sequence's tokens and channels among its lanes, and the
// scan over the lanes.
//
// A work-group owns CH neighbouring channels of one sequence and walks it in tiles
// of SL x TT tokens: a lane has one channel and TT consecutive tokens (a slot).
// Lanes c, c + CH, ... of a wave and the waves hold the tile's SL slots in order.
// Per state, a slot's effect on what enters it is h -> P h + H, with H the state that
// it makes of zero and P = exp(A sum D); effects compose along the slots by
//   (P2, H2) o (P1, H1) = (P2 P1, P2 H1 + H2),
// first across a wave's slots by shuffles, then across the waves in LDS.
#pragma once

#include "ssm_dev.hpp"

namespace gls {

template <typename S_, int CH_, int W_, int TT_, int NS_, int NB_>
struct SsmTile {
  using S = S_;
  static constexpr int CH = CH_;          // channels
  static constexpr int W = W_;            // waves
  static constexpr int TT = TT_;          // tokens a slot
  static constexpr int NS = NS_;          // states at a time
  static constexpr int NB = NB_;          // states whose B and C are in LDS at a time
  static constexpr int TS = 64 / CH;      // slots a wave
  static constexpr int SL = W * TS;       // slots
  static constexpr int TILE = SL * TT;    // tokens a tile
  static constexpr int THREADS = 64 * W;
  // B, C [token][NB]; slots are a vector further apart than their tokens, so that a
  // wave's slots read other banks
  static constexpr int PAD = 16 / sizeof(S);
  static constexpr int BC = TILE * NB + SL * PAD;
  __device__ static __forceinline__ int at(int token, int n) { return token * NB + token / TT * PAD + n; }
  __host__ __device__ static constexpr int npad(int N) { return (N + NB - 1) / NB * NB; }
  // LDS: B, C of the tile; A log2 e and the state that enters it (two: this tile's and the
  // next one's) per channel; what the waves pass on (two turns of (P, H))
  static size_t lds(int N) {
    return sizeof(S) * (2 * BC + 3 * static_cast<size_t>(npad(N)) * CH + 2 * W * CH * 2 * NS);
  }
};

// The work-group's channels and sequence.
struct SsmPlace {
  int g, d0, nch;   // group, first channel, channels
  int64_t n;        // sequence
};
__device__ __forceinline__ SsmPlace ssm_place(const SsmArgs& a, int CH, int64_t i) {
  const int dg = a.D / a.G, nb = (dg + CH - 1) / CH;
  const int64_t blocks = static_cast<int64_t>(nb) * a.G;
  const int cb = static_cast<int>(i % blocks);
  SsmPlace p;
  p.g = cb / nb;
  const int c0 = cb % nb * CH;
  p.d0 = p.g * dg + c0;
  p.nch = dg - c0 < CH ? dg - c0 : CH;
  p.n = i / blocks;
  return p;
}
inline int64_t ssm_blocks(const SsmArgs& a, int CH) {
  const int dg = a.D / a.G;
  return static_cast<int64_t>((dg + CH - 1) / CH) * a.G;
}

// B and C of states n0 .. n0 + NB - 1 for the tile's tokens into LDS, zero past N
// and past the sequence.
template <typename IO, typename L>
__device__ __forceinline__ void ssm_load_bc(const SsmArgs& a, const SsmPlace& p, const SeqRange& r, int64_t tile0, int n0,
                                            typename L::S* sB, typename L::S* sC) {
  using S = typename L::S;
  const IO* B = static_cast<const IO*>(a.Bm) + r.b * a.sB.b + p.g * a.sB.g;
  const IO* C = static_cast<const IO*>(a.Cm) + r.b * a.sC.b + p.g * a.sC.g;
  constexpr int per = L::TILE * L::NB / L::THREADS;
  static_assert(L::TILE * L::NB % L::THREADS == 0, "whole turns");
#pragma unroll 8
  for (int k = 0; k < per; ++k) {
    const int i = k * L::THREADS + threadIdx.x, tok = i / L::NB, nn = i % L::NB;
    const int64_t t = tile0 + tok;
    const bool in = t < r.len && n0 + nn < a.Ns;
    const int64_t tc = r.t0 + (in ? t : 0), nc = in ? n0 + nn : 0;
    const S b = load_as<S>(B, tc * a.sB.t + nc), c = load_as<S>(C, tc * a.sC.t + nc);
    sB[L::at(tok, nn)] = in ? b : S(0);
    sC[L::at(tok, nn)] = in ? c : S(0);
  }
}

template <typename S, int NS>
__device__ __forceinline__ void lds_get(const S* p, S (&v)[NS]) {
  if constexpr (sizeof(S) * NS == 16) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    __builtin_memcpy(v, &t, 16);
  } else if constexpr (sizeof(S) * NS == 8) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    __builtin_memcpy(v, &t, 8);
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j) v[j] = p[j];
  }
}

// Scan over the slots of (P, H), forward or (BACK) from the last slot: on return
// H is what enters the lane's slot, given that h enters the tile's first (last).
// One barrier; agg is [2][W][CH][2 NS], `turn` changes with every call.
template <typename L, bool BACK>
__device__ __forceinline__ void ssm_scan(typename L::S (&P)[L::NS], typename L::S (&H)[L::NS], typename L::S (&h)[L::NS],
                                         typename L::S* agg, int& turn) {
  using S = typename L::S;
  constexpr int CH = L::CH, TS = L::TS, W = L::W, NS = L::NS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane % CH;
  const int ts = BACK ? TS - 1 - lane / CH : lane / CH;  // order of the scan
#pragma unroll
  for (int m = 1; m < TS; m <<= 1) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const S p = BACK ? __shfl_down(P[j], m * CH, 64) : __shfl_up(P[j], m * CH, 64);
      const S h = BACK ? __shfl_down(H[j], m * CH, 64) : __shfl_up(H[j], m * CH, 64);
      if (ts >= m) {
        H[j] = fma_(P[j], h, H[j]);
        P[j] *= p;
      }
    }
  }
  S* mine = agg + ((turn * W + wave) * CH + c) * 2 * NS;
  if (ts == TS - 1) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      mine[j] = P[j];
      mine[NS + j] = H[j];
    }
  }
  // exclusive within the wave
  if constexpr (TS > 1) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const S p = BACK ? __shfl_down(P[j], CH, 64) : __shfl_up(P[j], CH, 64);
      const S h = BACK ? __shfl_down(H[j], CH, 64) : __shfl_up(H[j], CH, 64);
      P[j] = ts ? p : S(1);
      H[j] = ts ? h : S(0);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      P[j] = S(1);
      H[j] = S(0);
    }
  }
  __syncthreads();
  const int before = BACK ? W - 1 - wave : wave;
  for (int k = 0; k < before; ++k) {
    const int w = BACK ? W - 1 - k : k;
    const S* o = agg + ((turn * W + w) * CH + c) * 2 * NS;
    S p[NS], q[NS];
    lds_get<S, NS>(o, p);
    lds_get<S, NS>(o + NS, q);
#pragma unroll
    for (int j = 0; j < NS; ++j) h[j] = fma_(p[j], h[j], q[j]);
  }
#pragma unroll
  for (int j = 0; j < NS; ++j) H[j] = fma_(P[j], h[j], H[j]);
  turn ^= 1;
}

}  // namespace gls
