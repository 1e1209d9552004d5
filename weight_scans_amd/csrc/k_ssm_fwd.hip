// k_ssm_fwd.hip -- selective scan, forward (training and prefill).
//
//   D = softplus(dt + bias),  h = e h + (D x) B,  e = exp(D A),  y = (C h + skip x) silu(z)
//
// The decays differ per channel and state, so nothing of this is a matrix product:
// per token, channel and state it is a product and an exponential (four cycles of
// the vector ALU to a product's one) for e, and two products and two sums of products.
// How the lanes cut the work: ssm_scan.hpp.  A slot keeps its decays in registers
// between the two passes over its tokens: from zero, for its effect, and from what
// enters it, for y.
//
// Bound by the vector ALU, not by memory.  4 x 4096 tokens of 2048 channels and 16
// states in bf16, gated, with the states for a backward: 257 us, 12 instructions per token,
// channel and state (15 of the ALU's slots; eight are the least), the ALU busy three
// quarters of the time; its bytes alone would take 52 us.  One sequence of 32768 tokens: 690
// (8 channels: the only ones that spill, 3 registers in bf16, 27 in fp32 and fp64).
#include <algorithm>

#include "ssm_scan.hpp"

namespace gls {
namespace {

template <typename IO, typename L, bool Z>
__global__ __launch_bounds__(L::THREADS) void ssm_fwd(SsmArgs a, int ck) {
  using S = typename L::S;
  using BC = SlotBC<L, 1>;
  constexpr int CH = L::CH, TT = L::TT, NS = L::NS, NB = L::NB, BL = BC::BLOCK;
  extern __shared__ __align__(16) char lds[];
  const int np = L::npad(a.Ns);
  S* const sB = reinterpret_cast<S*>(lds);
  S* const sC = sB + L::BC;
  S* const agg = sC + L::BC;                     // [2][W][CH][2 NS]
  S* const sA = agg + 2 * L::AGG;                // [np][CH]
  S* sh = sA + np * CH;                          // [2][np][CH]
  const SsmPlace p = ssm_place(a, CH, xcd_order(blockIdx.x, gridDim.x));
  const SeqRange r = seq_range(a.cu, p.n, a.T);
  clear_behind<IO, L>(a, p, r, a.y, a.sy);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int slot = wave * L::TS + lane / CH;
  const bool in = lane % CH < p.nch;
  const int c = lane % CH, cc = in ? c : 0, d = p.d0 + cc;
  for (int i = threadIdx.x; i < np * CH; i += L::THREADS) {
    const int n = i / CH, ch = i % CH;
    const bool there = n < a.Ns && ch < p.nch;
    const int64_t o = static_cast<int64_t>(p.d0 + (there ? ch : 0)) * a.Ns + (there ? n : 0);
    sA[i] = there ? static_cast<const S*>(a.A)[o] * static_cast<S>(kLog2e) : S(0);
    sh[i] = there && a.state_in ? static_cast<const S*>(a.state_in)[p.n * a.D * a.Ns + o] : S(0);
  }
  const S skip = a.skip ? static_cast<const S*>(a.skip)[d] : S(0);
  const S bias = a.bias ? static_cast<const S*>(a.bias)[d] : S(0);
  const int64_t ck0 = chunk_slot0(a.packed, p.n, r.t0, a.T, ck);
  int turn = 0;
  S* sh1 = sh + np * CH;
  for (int64_t tile0 = 0; tile0 < r.len; tile0 += L::TILE) {
    const int left = static_cast<int>(r.len - tile0 < L::TILE ? r.len - tile0 : L::TILE);
    const int here = left - slot * TT;  // the slot's tokens that are there, if positive
    S D[TT], u[TT], y[TT], sum = S(0);
    TileBC<IO, L> bc;
    {
      IO x[TT], dt[TT];
      SlotRows<IO, L>(a.x, a.sx, r, p.d0, cc, slot, tile0).fetch(left, slot, x);
      SlotRows<IO, L>(a.dt, a.sdt, r, p.d0, cc, slot, tile0).fetch(left, slot, dt);
      bc.fetch(a, p, r, tile0, left, 0);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        u[i] = load_as<S>(&x[i], 0);
        D[i] = load_as<S>(&dt[i], 0);
      }
    }
    ssm_steps<S, TT>(a.softplus, bias, D);
    if (left < L::TILE) {  // past the end nothing changes
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        D[i] = i < here ? D[i] : S(0);
        u[i] = i < here ? u[i] : S(0);
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      y[i] = skip * u[i];
      u[i] *= D[i];
      sum += D[i];
    }
    const bool work = left > wave * (L::TS * TT);  // a wave past the end only hands on
    for (int n0 = 0; n0 < np; n0 += NB) {
      if (n0) bc.fetch(a, p, r, tile0, left, n0);
      __syncthreads();
      bc.store(a, p, r, tile0, left, n0, sB, sC);
      __syncthreads();
      for (int n1 = 0; n1 < NB; n1 += NS) {
        if (n0 + n1 >= a.Ns) break;
        BC B(sB + L::at(slot * TT, n1)), C(sC + L::at(slot * TT, n1));
        S A[NS], P[NS], h[NS], h0[NS], e[TT][NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          A[j] = sA[(n0 + n1 + j) * CH + c];
          P[j] = exp2_(A[j] * sum);
          h[j] = S(0);
          h0[j] = sh[(n0 + n1 + j) * CH + c];
        }
        if (work) {
#pragma unroll
          for (int i = 0; i < TT; i += BL) {
            B.load(i);
#pragma unroll
            for (int k = i; k < i + BL; ++k)
#pragma unroll
              for (int j = 0; j < NS; ++j) {
                e[k][j] = exp2_(D[k] * A[j]);
                h[j] = fma_(e[k][j], h[j], u[k] * B.at(k, j));
              }
            fence_order();
          }
        }
        S* const at = agg + turn * L::AGG;
        turn ^= 1;
        SsmScan<L, false>::leave(P, h, at);
        __syncthreads();
        SsmScan<L, false>::take(P, h, h0, at);
        if (a.ckpt && in && here > 0 && (tile0 + slot * TT) % ck == 0) {
          S* o = static_cast<S*>(a.ckpt) + ((ck0 + (tile0 + slot * TT) / ck) * a.Ns + n0 + n1) * a.D + d;
#pragma unroll
          for (int j = 0; j < NS; ++j)
            if (n0 + n1 + j < a.Ns) o[static_cast<int64_t>(j) * a.D] = h[j];
        }
        fence_order();
        if (work) {
#pragma unroll
          for (int i = 0; i < TT; i += BL) {
            B.load(i);
            C.load(i);
#pragma unroll
            for (int k = i; k < i + BL; ++k)
#pragma unroll
              for (int j = 0; j < NS; ++j) {
                h[j] = fma_(e[k][j], h[j], u[k] * B.at(k, j));
                y[k] = fma_(C.at(k, j), h[j], y[k]);
              }
            fence_order();
          }
        }
        if (slot == L::SL - 1) {
#pragma unroll
          for (int j = 0; j < NS; ++j) sh1[(n0 + n1 + j) * CH + c] = h[j];
        }
      }
    }
    S* const other = sh;
    sh = sh1;
    sh1 = other;
    IO raw[Z ? TT : 1];
    if constexpr (Z) SlotRows<IO, L>(a.z, a.sz, r, p.d0, cc, slot, tile0).fetch(left, slot, raw);
    if (!a.y) continue;
    if constexpr (Z) {
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const S z = load_as<S>(&raw[i], 0);
        y[i] *= z * sigmoid_(z);
      }
    }
    const SlotRows<IO, L> out(a.y, a.sy, r, p.d0, cc, slot, tile0);
    if (left >= L::TILE) {
      if (in) {
#pragma unroll
        for (int i = 0; i < TT; ++i) put(out.out(i), y[i]);
      }
    } else if (in) {
#pragma unroll
      for (int i = 0; i < TT; ++i)
        if (i < here) put(out.out(i), y[i]);
    }
  }
  if (!a.state_out) return;
  __syncthreads();
  for (int i = threadIdx.x; i < np * CH; i += L::THREADS) {
    const int n = i % np, ch = i / np;
    if (n < a.Ns && ch < p.nch)
      static_cast<S*>(a.state_out)[(p.n * a.D + p.d0 + ch) * a.Ns + n] = sh[n * CH + ch];
  }
}

template <typename IO, typename L>
hipError_t go(int io, const SsmArgs& a, hipStream_t s) {
  const int64_t g = a.N * ssm_blocks(a, L::CH);
  if (g == 0) return hipSuccess;
  SsmArgs b = a;
  b.vec_bc = ssm_vec_bc(io, a);
  if (a.z) ssm_fwd<IO, L, true><<<static_cast<unsigned>(g), L::THREADS, L::lds(a.Ns), s>>>(b, ssm_ck(io, a));
  else ssm_fwd<IO, L, false><<<static_cast<unsigned>(g), L::THREADS, L::lds(a.Ns), s>>>(b, ssm_ck(io, a));
  return hipGetLastError();
}

template <typename IO, typename S, int TT, int NS>
hipError_t by_channels(int io, int channels, const SsmArgs& a, hipStream_t s) {
  switch (channels) {
    case 64: return go<IO, SsmTile<S, 64, kSsmWaves, TT, NS, 16>>(io, a, s);
    case 32: return go<IO, SsmTile<S, 32, kSsmWaves, TT, NS, 16>>(io, a, s);
    case 16: return go<IO, SsmTile<S, 16, kSsmWaves, TT, NS, 8>>(io, a, s);
    default: return go<IO, SsmTile<S, 8, kSsmWaves, TT, NS, 8>>(io, a, s);
  }
}
template <typename IO>
hipError_t by_shape(int io, const SsmShape& p, const SsmArgs& a, hipStream_t s) {
  if (p.tokens == kSsmShort) return by_channels<IO, float, kSsmShort, 4>(io, p.channels, a, s);
  return by_channels<IO, float, 16, 4>(io, p.channels, a, s);
}

}  // namespace

// Channels and tokens with the least rounds of tiles for the 256 CUs (a tile costs its
// slots' tokens and about eight more for the exchanges), the most channels where two
// have the same.  One sequence of 32768 tokens of 2048 channels: 16 channels 1134 us, 8
// 685 us; 5 sequences of 777 tokens in all: 64 channels 53 us, 32 75 us, 8 86 us (all of 16
// tokens a slot).  Forward and backward of 4 x 24 tokens of 1280 channels, 64 states: 16
// tokens a slot 183 us, 4 100 us; of 2 x 90 of 192 channels, 16 states: 58 us and 41 us.
SsmShape ssm_shape(const SsmArgs& a, int io, int most) {
  const int64_t n = std::max<int64_t>(a.N, 1), len = a.packed ? (a.T + n - 1) / n : a.T;
  SsmShape best{most, io == IO_F64 ? 8 : 16};
  int64_t least = INT64_MAX;
  for (int CH = most; CH >= 8; CH /= 2)
    for (const int TT : {16, kSsmShort}) {
      const SsmShape p{CH, io == IO_F64 ? 8 : TT};
      const int64_t tiles = std::max<int64_t>(1, (len + p.tile() - 1) / p.tile());
      const int64_t cost = (n * ssm_blocks(a, CH) + 255) / 256 * tiles * (p.tokens + 8);
      if (cost < least) {
        least = cost;
        best = p;
      }
    }
  return best;
}

hipError_t launch_ssm_fwd(int io, const SsmArgs& a, hipStream_t s) {
  const SsmShape p = ssm_shape(a, io, a.Ns <= 64 ? 64 : a.Ns <= 128 ? 32 : 16);  // (by the LDS)
  if (!p.fits(a)) return hipErrorInvalidConfiguration;
  if (io == IO_F64) return by_channels<double, double, 8, 2>(io, p.channels, a, s);
  if (io == IO_F32) return by_shape<float>(io, p, a, s);
  return by_shape<bf16>(io, p, a, s);
}

}  // namespace gls
