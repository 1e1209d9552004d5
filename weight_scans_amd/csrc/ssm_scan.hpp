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
  // B, C by groups of NS states, [group][token][NS]; slots are a vector further apart
  // than their tokens, so that a wave's slots read other banks
  static constexpr int PAD = 16 / sizeof(S);
  static constexpr int GROUP = TILE * NS + SL * PAD;
  static constexpr int BC = GROUP * (NB / NS);
  __device__ static __forceinline__ int at(int token, int n) {
    return n / NS * GROUP + token * NS + token / TT * PAD + n % NS;
  }
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

// A tensor of rows as a work-group reads it: one base for the tile (the same in all
// lanes, so that it is kept and moved on by the scalar unit), and the lane's offset
// in bytes, which stays (below 2^32: the host bounds the strides).
template <typename IO, typename L>
struct SlotRows {
  const char* base;  // the tile's first token, at channel d0
  int64_t step;      // bytes a token
  uint32_t off, col; // the lane's first token and channel; its channel
  __device__ __forceinline__ SlotRows(const void* p, const Rows& s, const SeqRange& r, int d0, int c, int slot, int64_t tile0)
      : base(static_cast<const char*>(p) + (r.b * s.b + (r.t0 + tile0) * s.t + d0) * static_cast<int64_t>(sizeof(IO))),
        step(s.t * static_cast<int64_t>(sizeof(IO))),
        off(static_cast<uint32_t>(slot * L::TT * step) + c * static_cast<uint32_t>(sizeof(IO))),
        col(c * static_cast<uint32_t>(sizeof(IO))) {
    // known only here: multiples of it for 16 tokens and seven tensors, kept over the
    // loop over the tiles, are more than the scalar registers
    asm volatile("" : "+s"(step));
  }
  // The lane's TT tokens of a tile that has `left` (past its end: the last one again).
  template <typename S>
  __device__ __forceinline__ void ld(int left, int slot, S (&v)[L::TT]) const {
    if (left >= L::TILE) {
#pragma unroll
      for (int i = 0; i < L::TT; ++i) v[i] = load_as<S>(reinterpret_cast<const IO*>(base + i * step + off), 0);
    } else {
      int first = slot * L::TT;
      asm volatile("" : "+v"(first));  // likewise: not kept for the next use
#pragma unroll
      for (int i = 0; i < L::TT; ++i) {
        const int tok = min(first + i, left - 1);
        v[i] = load_as<S>(reinterpret_cast<const IO*>(base + static_cast<uint32_t>(tok) * step + col), 0);
      }
    }
  }
  __device__ __forceinline__ IO* out(int i) const {
    return reinterpret_cast<IO*>(const_cast<char*>(base) + i * step + off);
  }
};

// D of the slot's tokens from dt and its bias; zero, as nothing then changes, past its end.
template <typename S, int TT>
__device__ __forceinline__ void ssm_steps(bool softplus, S bias, int here, S (&D)[TT]) {
  if (softplus) {
#pragma unroll
    for (int i = 0; i < TT; ++i) D[i] = softplus_(D[i] + bias);
  } else {
#pragma unroll
    for (int i = 0; i < TT; ++i) D[i] += bias;
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) D[i] = i < here ? D[i] : S(0);
}

inline bool ssm_vec_bc(int io, const SsmArgs& a) {
  return a.Ns % vec_of(io) == 0 && aligned16(a.Bm) && aligned16(a.Cm) && aligned16(io, a.sB) && aligned16(io, a.sC);
}

// B and C of states n0 .. n0 + NB - 1 for the tile's tokens into LDS, zero past N and
// past the sequence; in vectors where rows begin on 16 bytes and N is whole vectors.
template <typename IO, typename L>
__device__ __forceinline__ void ssm_load_bc(const SsmArgs& a, const SsmPlace& p, const SeqRange& r, int64_t tile0, int n0,
                                            typename L::S* sB, typename L::S* sC) {
  using S = typename L::S;
  const IO* B = static_cast<const IO*>(a.Bm) + r.b * a.sB.b + (r.t0 + tile0) * a.sB.t + p.g * a.sB.g + n0;
  const IO* C = static_cast<const IO*>(a.Cm) + r.b * a.sC.b + (r.t0 + tile0) * a.sC.t + p.g * a.sC.g + n0;
  const int left = static_cast<int>(r.len - tile0 < L::TILE ? r.len - tile0 : L::TILE), states = a.Ns - n0;
  constexpr int V = Vec<IO>::n < L::NB ? Vec<IO>::n : L::NB;
  if (a.vec_bc) {
    constexpr int per = L::TILE * L::NB / V;
    constexpr int rounds = (per + L::THREADS - 1) / L::THREADS;
    S b[rounds][V], c[rounds][V];
#pragma unroll
    for (int k = 0; k < rounds; ++k) {
      const int i = k * L::THREADS + threadIdx.x, tok = i * V / L::NB, nn = i * V % L::NB;
      const bool in = tok < left && nn < states;
      const int64_t tc = in ? tok : 0, nc = in ? nn : 0;
      load_w<IO, S, V>(B + tc * a.sB.t + nc, b[k]);
      load_w<IO, S, V>(C + tc * a.sC.t + nc, c[k]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        b[k][e] = in ? b[k][e] : S(0);
        c[k][e] = in ? c[k][e] : S(0);
      }
    }
#pragma unroll
    for (int k = 0; k < rounds; ++k) {
      const int i = k * L::THREADS + threadIdx.x, tok = i * V / L::NB, nn = i * V % L::NB;
      if (per % L::THREADS == 0 || i < per) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sB[L::at(tok, nn + e)] = b[k][e];
          sC[L::at(tok, nn + e)] = c[k][e];
        }
      }
    }
    return;
  }
#pragma unroll 4
  for (int k = 0; k < L::TILE * L::NB / L::THREADS; ++k) {
    const int i = k * L::THREADS + threadIdx.x, tok = i / L::NB, nn = i % L::NB;
    const bool in = tok < left && nn < states;
    const int64_t tc = in ? tok : 0, nc = in ? nn : 0;
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

// NS values of each of K = 16 bytes / NS tokens from token i on.
template <typename L>
struct SlotBC {
  using S = typename L::S;
  static constexpr int K = 16 / (sizeof(S) * L::NS);
  S v[K][L::NS];
  __device__ __forceinline__ SlotBC(const S* p, int i) {
    const uint4 t = *reinterpret_cast<const uint4*>(p + i * L::NS);
    __builtin_memcpy(v, &t, 16);
  }
};

// The lanes' values of the other half of the wave: a from lanes 0..31, b from 32..63.
template <typename S>
__device__ __forceinline__ void halves(S x, S& lo, S& hi) {
  if constexpr (sizeof(S) == 4) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(r[0]);
    hi = __uint_as_float(r[1]);
  } else {
    const int l = threadIdx.x & 31;
    lo = __shfl(x, l, 64);
    hi = __shfl(x, l + 32, 64);
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
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane % CH;
  const int ts = BACK ? TS - 1 - lane / CH : lane / CH;  // order of the scan
  S* const mine = agg + ((turn * W + wave) * CH + c) * 2 * NS;
  S wp[NS], wh[NS];  // of the whole wave, in the lanes that hold it
  if constexpr (TS == 2) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      S p0, p1, h0, h1;
      if constexpr (BACK) {
        halves(P[j], p1, p0);
        halves(H[j], h1, h0);
      } else {
        halves(P[j], p0, p1);
        halves(H[j], h0, h1);
      }
      wp[j] = p0 * p1;
      wh[j] = fma_(p1, h0, h1);
      P[j] = ts ? p0 : S(1);
      H[j] = ts ? h0 : S(0);
    }
  } else {
#pragma unroll
    for (int m = 1; m < TS; m <<= 1) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const S p = BACK ? __shfl_down(P[j], m * CH, 64) : __shfl_up(P[j], m * CH, 64);
        const S q = BACK ? __shfl_down(H[j], m * CH, 64) : __shfl_up(H[j], m * CH, 64);
        if (ts >= m) {
          H[j] = fma_(P[j], q, H[j]);
          P[j] *= p;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      wp[j] = P[j];
      wh[j] = H[j];
      if constexpr (TS > 1) {
        const S p = BACK ? __shfl_down(P[j], CH, 64) : __shfl_up(P[j], CH, 64);
        const S q = BACK ? __shfl_down(H[j], CH, 64) : __shfl_up(H[j], CH, 64);
        P[j] = ts ? p : S(1);
        H[j] = ts ? q : S(0);
      } else {
        P[j] = S(1);
        H[j] = S(0);
      }
    }
  }
  if (ts == TS - 1) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      mine[j] = wp[j];
      mine[NS + j] = wh[j];
    }
  }
  __syncthreads();
  // the waves before, in order
  const int before = BACK ? W - 1 - wave : wave;
  S p[W - 1][NS], q[W - 1][NS];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int w = BACK ? W - 1 - k : k;
    const S* o = agg + ((turn * W + w) * CH + c) * 2 * NS;
    if (k < before) {
      lds_get<S, NS>(o, p[k]);
      lds_get<S, NS>(o + NS, q[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    if (k < before) {
#pragma unroll
      for (int j = 0; j < NS; ++j) h[j] = fma_(p[k][j], h[j], q[k][j]);
    }
#pragma unroll
  for (int j = 0; j < NS; ++j) H[j] = fma_(P[j], h[j], H[j]);
  turn ^= 1;
}

// Keeps the compiler from moving instructions across: loads of later tokens that are
// issued all at once take more registers than there are.
__device__ __forceinline__ void fence_order() { __builtin_amdgcn_sched_barrier(0); }

}  // namespace gls
