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
//
// Tokens in a lane, not in a matrix product: decays differ per channel and state, so
// that a product over tokens would need one matrix of them each.  States one after
// another in groups of NS, not side by side in lanes: a lane's x, D and y then serve all
// states, and only B and C are read per state, from LDS.  Longer slots cost less in
// exchanges (16 tokens: 690 us the backward at 4 x 4096 x 2048 x 16; 8 with twice the states
// at once: 903), shorter ones leave less of a short sequence's tile empty.
#pragma once

#include "ssm_dev.hpp"

namespace gls {

constexpr int kSsmShort = 4;  // tokens a slot where sequences are short (16 else, 8 in fp64)

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
  static constexpr int AGG = W * CH * 2 * NS;
  // LDS: B, C of the tile; A log2 e and the state that enters it (two: this tile's and the
  // next one's) per channel; what the waves pass on (two turns of (P, H))
  static size_t lds(int N) {
    return sizeof(S) * (2 * BC + 3 * static_cast<size_t>(npad(N)) * CH + 2 * AGG);
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
// The rows behind the last packed sequence belong to none: the last sequence's work-groups
// make them zeros.
template <typename IO, typename L>
__device__ __forceinline__ void clear_behind(const SsmArgs& a, const SsmPlace& p, const SeqRange& r, void* out, const Rows& s) {
  if (!a.packed || p.n + 1 < a.N || !out) return;
  const int c = threadIdx.x % L::CH;
  if (c >= p.nch) return;
  for (int64_t t = r.t0 + r.len + threadIdx.x / L::CH; t < a.T; t += L::THREADS / L::CH)
    store_from(static_cast<IO*>(out) + t * s.t, p.d0 + c, typename L::S(0));
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
  // The lane's TT tokens of a tile that has `left` (past its end: the last one again), as
  // they lie in memory: what is not yet converted is not yet waited for.
  template <int n>
  __device__ __forceinline__ void fetch(int left, int slot, IO (&v)[n]) const {
    static_assert(n == L::TT, "a slot's tokens");
    if (left >= L::TILE) {
#pragma unroll
      for (int i = 0; i < L::TT; ++i) v[i] = *reinterpret_cast<const IO*>(base + i * step + off);
    } else {
      int first = slot * L::TT;
      asm volatile("" : "+v"(first));  // likewise: not kept for the next use
#pragma unroll
      for (int i = 0; i < L::TT; ++i) {
        const int tok = min(first + i, left - 1);
        v[i] = *reinterpret_cast<const IO*>(base + static_cast<uint32_t>(tok) * step + col);
      }
    }
  }
  __device__ __forceinline__ IO* out(int i) const {
    return reinterpret_cast<IO*>(const_cast<char*>(base) + i * step + off);
  }
};

// D of the slot's tokens from dt and its bias.
template <typename S, int TT>
__device__ __forceinline__ void ssm_steps(bool softplus, S bias, S (&D)[TT]) {
  if (softplus) {
#pragma unroll
    for (int i = 0; i < TT; ++i) D[i] = softplus_(D[i] + bias);
  } else {
#pragma unroll
    for (int i = 0; i < TT; ++i) D[i] += bias;
  }
}

inline bool ssm_vec_bc(int io, const SsmArgs& a) {
  return a.Ns % vec_of(io) == 0 && aligned16(a.Bm) && aligned16(a.Cm) && aligned16(io, a.sB) && aligned16(io, a.sC);
}

// B and C of states n0 .. n0 + NB - 1 for the tile's tokens into LDS, zero past N and
// past the sequence: `fetch` asks for them (in vectors, where rows begin on 16 bytes
// and N is whole vectors), `store` puts them there.
template <typename IO, typename L>
struct TileBC {
  using S = typename L::S;
  static constexpr int V = Vec<IO>::n < L::NB ? Vec<IO>::n : L::NB;
  static constexpr int PER = L::TILE * L::NB / V, ROUNDS = (PER + L::THREADS - 1) / L::THREADS;
  uint4 b[ROUNDS], c[ROUNDS];

  __device__ static __forceinline__ const IO* first(const void* p, const Rows& s, const SsmPlace& w, const SeqRange& r,
                                                    int64_t tile0, int n0) {
    return static_cast<const IO*>(p) + r.b * s.b + (r.t0 + tile0) * s.t + w.g * s.g + n0;
  }
  __device__ __forceinline__ void fetch(const SsmArgs& a, const SsmPlace& w, const SeqRange& r, int64_t tile0, int left, int n0) {
    if (!a.vec_bc) return;
    const IO *B = first(a.Bm, a.sB, w, r, tile0, n0), *C = first(a.Cm, a.sC, w, r, tile0, n0);
    const int states = a.Ns - n0;
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      const int i = (k * L::THREADS + threadIdx.x) * V, tok = i / L::NB, nn = i % L::NB;
      const bool in = tok < left && nn < states;
      const int64_t tc = in ? tok : 0, nc = in ? nn : 0;
      b[k] = *reinterpret_cast<const uint4*>(B + tc * a.sB.t + nc);
      c[k] = *reinterpret_cast<const uint4*>(C + tc * a.sC.t + nc);
    }
  }
  __device__ __forceinline__ void store(const SsmArgs& a, const SsmPlace& w, const SeqRange& r, int64_t tile0, int left, int n0,
                                        S* sB, S* sC) const {
    const int states = a.Ns - n0;
    if (a.vec_bc) {
#pragma unroll
      for (int k = 0; k < ROUNDS; ++k) {
        const int i = (k * L::THREADS + threadIdx.x) * V, tok = i / L::NB, nn = i % L::NB;
        const bool in = tok < left && nn < states;
        S vb[Vec<IO>::n], vc[Vec<IO>::n];
        Vec<IO>::ld(reinterpret_cast<const IO*>(&b[k]), vb);
        Vec<IO>::ld(reinterpret_cast<const IO*>(&c[k]), vc);
        if (PER % L::THREADS == 0 || k * L::THREADS + static_cast<int>(threadIdx.x) < PER) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sB[L::at(tok, nn + e)] = in ? vb[e] : S(0);
            sC[L::at(tok, nn + e)] = in ? vc[e] : S(0);
          }
        }
      }
      return;
    }
    const IO *B = first(a.Bm, a.sB, w, r, tile0, n0), *C = first(a.Cm, a.sC, w, r, tile0, n0);
#pragma unroll 4
    for (int k = 0; k < L::TILE * L::NB / L::THREADS; ++k) {
      const int i = k * L::THREADS + threadIdx.x, tok = i / L::NB, nn = i % L::NB;
      const bool in = tok < left && nn < states;
      const int64_t tc = in ? tok : 0, nc = in ? nn : 0;
      const S vb = load_as<S>(B, tc * a.sB.t + nc), vc = load_as<S>(C, tc * a.sC.t + nc);
      sB[L::at(tok, nn)] = in ? vb : S(0);
      sC[L::at(tok, nn)] = in ? vc : S(0);
    }
  }
};

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

// A slot's B or C of one state group, four tokens at a time (two in fp64).  BUFS = 2:
// the next block is on its way while one is used.
template <typename L, int BUFS>
struct SlotBC {
  using S = typename L::S;
  static constexpr int BLOCK = 16 / sizeof(S);
  static_assert(L::TT % BLOCK == 0, "whole blocks");
  const S* p;
  S v[BUFS][BLOCK][L::NS];
  __device__ __forceinline__ explicit SlotBC(const S* first) : p(first) {}
  __device__ __forceinline__ void load(int i) {  // tokens i .. i + BLOCK - 1
    const uint4* s = reinterpret_cast<const uint4*>(p + i * L::NS);
    uint4 t[L::NS];
#pragma unroll
    for (int k = 0; k < L::NS; ++k) t[k] = s[k];
    __builtin_memcpy(v[i / BLOCK % BUFS], t, sizeof(t));
  }
  __device__ __forceinline__ S at(int i, int j) const { return v[i / BLOCK % BUFS][i % BLOCK][j]; }
};

// x of the lower and of the upper of the two groups of m lanes that a lane's pair of groups
// is (m = 8, 16 or 32), lane by lane.
template <int m, typename S>
__device__ __forceinline__ void pair_of(S x, S& lo, S& hi) {
  if constexpr (sizeof(S) == 4 && m == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(r[0]);
    hi = __uint_as_float(r[1]);
  } else if constexpr (sizeof(S) == 4 && m == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(r[0]);
    hi = __uint_as_float(r[1]);
  } else if constexpr (sizeof(S) == 4 && m == 8) {
    const float o = __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x128, 0xf, 0xf, true));  // row_ror:8
    const bool up = threadIdx.x & 8;
    lo = up ? o : x;
    hi = up ? x : o;
  } else {
    const S o = __shfl_xor(x, m, 64);
    const bool up = threadIdx.x & m;
    lo = up ? o : x;
    hi = up ? x : o;
  }
}

// Scan over the slots of (P, H), forward or (BACK) from the last slot, in two halves with
// a barrier of the caller between them: `leave` composes a wave's slots and leaves the
// whole in LDS; `take` returns in H what enters the lane's slot, given that h enters
// the tile's first (last).  agg: [W][CH][2 NS].
template <typename L, bool BACK>
struct SsmScan {
  using S = typename L::S;
  static constexpr int CH = L::CH, TS = L::TS, W = L::W, NS = L::NS;

  __device__ static __forceinline__ int order(int lane) { return BACK ? TS - 1 - lane / CH : lane / CH; }

  __device__ static __forceinline__ void leave(S (&P)[NS], S (&H)[NS], S* agg) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    S pe[NS], he[NS];  // of the slots before the lane's
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      pe[j] = S(1);
      he[j] = S(0);
    }
    level<CH>(P, H, pe, he);  // P, H: now of the whole wave
    if (order(lane) == TS - 1) {
      S* const mine = agg + (wave * CH + lane % CH) * 2 * NS;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        mine[j] = P[j];
        mine[NS + j] = H[j];
      }
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      P[j] = pe[j];
      H[j] = he[j];
    }
  }

  // Groups of m lanes into groups of 2 m.
  template <int m>
  __device__ static __forceinline__ void level(S (&P)[NS], S (&H)[NS], S (&pe)[NS], S (&he)[NS]) {
    if constexpr (m < 64) {
      const bool second = ((threadIdx.x & m) != 0) != BACK;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        S p0, p1, h0, h1;
        if constexpr (BACK) {
          pair_of<m>(P[j], p1, p0);
          pair_of<m>(H[j], h1, h0);
        } else {
          pair_of<m>(P[j], p0, p1);
          pair_of<m>(H[j], h0, h1);
        }
        he[j] = second ? fma_(pe[j], h0, he[j]) : he[j];
        pe[j] = second ? pe[j] * p0 : pe[j];
        P[j] = p0 * p1;
        H[j] = fma_(p1, h0, h1);
      }
      level<2 * m>(P, H, pe, he);
    }
  }

  __device__ static __forceinline__ void take(const S (&P)[NS], S (&H)[NS], S (&h)[NS], const S* agg) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int before = BACK ? W - 1 - wave : wave;  // waves, in order
    S p[W - 1][NS], q[W - 1][NS];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int w = BACK ? W - 1 - k : k;
      const S* o = agg + (w * CH + lane % CH) * 2 * NS;
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
  }
};

// Keeps the compiler from moving instructions across: loads of later tokens that are
// issued all at once take more registers than there are.
__device__ __forceinline__ void fence_order() { __builtin_amdgcn_sched_barrier(0); }

}  // namespace gls
