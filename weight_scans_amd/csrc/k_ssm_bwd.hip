// k_ssm_bwd.hip -- selective scan, backward.
//
// With s_t the gradient that reaches h_t from later tokens, dy already through the
// gate, and q_t = e_t h_(t-1) (what token t keeps):
//
//   g_t = s_t + dy_t C_t,        s_(t-1) = e_t g_t
//   dC_t = sum_d dy_t h_t        dB_t = sum_d D_t x_t g_t
//   du_t = sum_n B_t g_t         dx_t = D_t du_t + skip dy_t
//   dD_t = x_t du_t + sum_n A q_t g_t,      dA = sum_t D_t q_t g_t
//
// Tiles run backwards, each from the state that the forward kept before it: the
// forward's two passes over a slot's tokens again, then the same two in reverse
// (ssm_scan.hpp).  The sums over channels are formed within a work-group, lanes
// halving the number of values with every exchange, and leave as one part per
// work-group and token, [block][state group][token][NS], added by a second kernel in a
// fixed order.
//
// Bound by the vector ALU: 4 x 4096 tokens of 2048 channels and 16 states in bf16, gated:
// 690 us, 32 instructions per token, channel and state, the ALU busy 72 % of the time
// (29 us more for the parts); its bytes alone would take 112 us, a fifth of
// them the parts.  Some 70 % of the time is the loop over the states, the rest before and
// behind it loads and stores that no other wave covers (the registers hold two waves a SIMD).
// One sequence of 32768 tokens (8 channels a work-group): 2.04 ms, and 1 GiB of parts.
//
// At 16 tokens a slot all 256 registers are taken and some spill: with the gate 47, 38 and
// 50 in bf16 (32, 16 and 8 channels), 79, 58 and 118 in fp32, and 151 to 177 in fp64 (8
// tokens); 2 to 26 fewer without it.  At 4 tokens none do.
#include <algorithm>

#include "ssm_scan.hpp"

namespace gls {
namespace {

// x of the lanes that a row's rotation or mirror hands it (the vector ALU's own lane
// patterns; they cost nothing beside the sum that takes them).
template <int PATTERN>
__device__ __forceinline__ float from_lane(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), PATTERN, 0xf, 0xf, true));
}
constexpr int kRowRor8 = 0x128, kHalfMirror = 0x141, kXor2 = 0x4e, kXor1 = 0xb1;

// a summed over the two groups of lanes that differ in bit m, in those where it is 0; b in
// the others.  (For m = 4 with the lanes of one group in reverse: a sum over all of
// them is left.)
template <int m>
__device__ __forceinline__ float fold(float a, float b, bool up) {
  if constexpr (m == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    constexpr int P = m == 8 ? kRowRor8 : m == 4 ? kHalfMirror : m == 2 ? kXor2 : kXor1;
    const float s = a + from_lane<P>(a), t = b + from_lane<P>(b);
    return up ? t : s;
  }
}
template <int m>
__device__ __forceinline__ double fold(double a, double b, bool up) {
  const double keep = up ? b : a, give = up ? a : b;
  return keep + __shfl_xor(give, m, 64);
}

// Sums of a slot's TT x NS values over the CH channels.  Every fold hands half of what is
// left to half of the lanes: first over a token's states, then over pairs of tokens,
// of pairs, ... as they come (BACK: from the last token on), so that few values wait.
// What is left when the lanes are used up is one sum a lane, at part[token NS + state].
template <typename L, bool BACK>
struct Sums {
  using S = typename L::S;
  static constexpr int CH = L::CH, TT = L::TT, NS = L::NS;
  static constexpr int lg(int n) { return n <= 1 ? 0 : 1 + lg(n / 2); }
  static constexpr int STATES = lg(NS), LANES = lg(CH) - STATES;
  static constexpr int DEPTH = LANES < lg(TT) ? LANES : lg(TT);
  static constexpr int bit(int k) { return CH >> (1 + STATES + k); }  // lanes folded at depth k over tokens
  S* part;         // of the slot's first token, with the lane's own token and state
  int c, here;     // the lane's channel; tokens that are there, counted from the lane's own
  S t[DEPTH + 1][TT];

  __device__ __forceinline__ Sums(S* first, int c_, int here_) : part(first), c(c_), here(here_) {
#pragma unroll
    for (int k = 0; k < STATES; ++k) part += c & (CH >> (1 + k)) ? NS >> (1 + k) : 0;
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
      const int own = c & bit(k) ? 1 << k : 0;
      part += own * NS;
      here -= own;
    }
    if (DEPTH < LANES && (c & (2 * bit(DEPTH) - 1))) here = 0;  // lanes that hold what another one does
  }
  template <int k, int n>
  __device__ __forceinline__ S states(S (&v)[NS]) {
    if constexpr (n == 1) {
      return v[0];
    } else {
#pragma unroll
      for (int j = 0; j < n / 2; ++j) v[j] = fold<(CH >> (1 + k))>(v[j], v[j + n / 2], c & (CH >> (1 + k)));
      return states<k + 1, n / 2>(v);
    }
  }
  template <int m>
  __device__ __forceinline__ S rest(S x) {
    if constexpr (m < 1) return x;
    else return rest<m / 2>(fold<m>(x, x, false));
  }
  template <int k>
  __device__ __forceinline__ void tokens(int i, S x) {
    if constexpr (k == DEPTH) {
      const int first = i >> DEPTH << DEPTH;
      x = rest<bit(DEPTH)>(x);
      if (first < here) part[first * NS] = x;
    } else {
      t[k][i >> k] = x;
      if (((i >> k) & 1) == (BACK ? 0 : 1)) {
        const int q = i >> (k + 1) << 1;
        tokens<k + 1>(i, fold<bit(k)>(t[k][q], t[k][q + 1], c & bit(k)));
      }
    }
  }
  // token i's values, in order
  __device__ __forceinline__ void put(int i, S (&v)[NS]) { tokens<0>(i, states<0, NS>(v)); }
};

// LDS: B and C of the tile, what the waves pass on of the scans and of dA; A log2 e, dA,
// the state before the tile and two of the gradient that enters it; y of the tile's tokens.
template <typename L, bool Z>
size_t bwd_lds(int N) {
  return sizeof(typename L::S) * (2 * L::BC + 5 * static_cast<size_t>(L::npad(N)) * L::CH + 4 * L::AGG +
                                  2 * L::W * L::CH * L::NS + (Z ? L::THREADS * L::TT : 0));
}

template <typename IO, typename L, bool Z>
__global__ __launch_bounds__(L::THREADS) void ssm_bwd(SsmArgs a) {
  using S = typename L::S;
  using BC = SlotBC<L, 2>;
  constexpr int CH = L::CH, TT = L::TT, NS = L::NS, NB = L::NB, W = L::W, BL = BC::BLOCK;
  extern __shared__ __align__(16) char lds[];
  const int np = L::npad(a.Ns);
  S* const sB = reinterpret_cast<S*>(lds);
  S* const sC = sB + L::BC;
  S* const agg = sC + L::BC;                      // [2 turns][forward, back][W][CH][2 NS]
  S* const red = agg + 4 * L::AGG;                // [2][W][CH][NS]
  S* const sA = red + 2 * W * CH * NS;            // [np][CH]
  S* const sdA = sA + np * CH;                    // [np][CH]
  S* const sS = sdA + np * CH;                    // [np][CH]
  S* sl = sS + np * CH;                           // [2][np][CH]
  S* sl1 = sl + np * CH;
  // y before the gate, in LDS: kept over all states, it is more than the registers hold
  // beside what the passes need (98 registers spilled, and every wait for one of them a
  // wait for the sums' stores: twice the time at 4 x 4096 x 2048 x 16)
  constexpr int YV = 16 / sizeof(S);
  S* const sy = sS + 3 * np * CH + threadIdx.x * YV;  // [TT / YV][threads][YV]
  const int64_t blocks = static_cast<int64_t>(gridDim.x) / a.N;
  const int64_t id = xcd_order(blockIdx.x, gridDim.x);
  const SsmPlace p = ssm_place(a, CH, id);
  const SeqRange r = seq_range(a.cu, p.n, a.T);
  clear_behind<IO, L>(a, p, r, a.dx, a.sdx);
  clear_behind<IO, L>(a, p, r, a.ddt, a.sddt);
  if constexpr (Z) clear_behind<IO, L>(a, p, r, a.dz, a.sdz);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane % CH, ts = lane / CH, slot = wave * L::TS + ts;
  const bool in = c < p.nch;
  const int cc = in ? c : 0, d = p.d0 + cc;
  for (int i = threadIdx.x; i < np * CH; i += L::THREADS) {
    const int n = i / CH, ch = i % CH;
    const bool there = n < a.Ns && ch < p.nch;
    const int64_t o = static_cast<int64_t>(p.d0 + (there ? ch : 0)) * a.Ns + (there ? n : 0);
    sA[i] = there ? static_cast<const S*>(a.A)[o] * static_cast<S>(kLog2e) : S(0);
    sl[i] = there && a.dstate_out ? static_cast<const S*>(a.dstate_out)[p.n * a.D * a.Ns + o] : S(0);
    sdA[i] = S(0);
  }
  const S skip = a.skip ? static_cast<const S*>(a.skip)[d] : S(0);
  const S bias = a.bias ? static_cast<const S*>(a.bias)[d] : S(0);
  const int64_t ck0 = chunk_slot0(a.packed, p.n, r.t0, a.T, L::TILE);
  // parts of the sums over channels: [2][blocks][state groups][B T][NS]
  const int groups = (a.Ns + NS - 1) / NS;
  const int64_t tok = a.B * a.T, plane = tok * NS;
  S* const partB = static_cast<S*>(a.part_bc) + (id % blocks) * groups * plane + (r.b * a.T + r.t0) * NS;
  S* const partC = partB + blocks * groups * plane;
  S dskip = S(0), dbias = S(0);
  int turn = 0, rturn = 0, pending = -1;
  // dA of the state group before: its waves' sums into sdA, by one thread each
  const auto settle = [&] {
    if (pending >= 0 && threadIdx.x < CH * NS) {
      S x = S(0);
#pragma unroll
      for (int w = 0; w < W; ++w) x += red[(rturn ^ 1) * W * CH * NS + w * CH * NS + threadIdx.x];
      sdA[(pending + threadIdx.x % NS) * CH + threadIdx.x / NS] += x;
    }
  };
  for (int64_t tile = r.len ? (r.len - 1) / L::TILE : -1; tile >= 0; --tile) {
    const int64_t tile0 = tile * L::TILE;
    const int left = static_cast<int>(r.len - tile0 < L::TILE ? r.len - tile0 : L::TILE);
    const int here = left - slot * TT;
    S D[TT], u[TT], g[TT], du[TT], dD[TT], sum = S(0);
    TileBC<IO, L> bc;
    {
      IO x[TT], dt[TT], dy[TT], z[Z ? TT : 1];
      SlotRows<IO, L>(a.x, a.sx, r, p.d0, cc, slot, tile0).fetch(left, slot, x);
      SlotRows<IO, L>(a.dt, a.sdt, r, p.d0, cc, slot, tile0).fetch(left, slot, dt);
      SlotRows<IO, L>(a.dy, a.sdy, r, p.d0, cc, slot, tile0).fetch(left, slot, dy);
      if constexpr (Z) SlotRows<IO, L>(a.z, a.sz, r, p.d0, cc, slot, tile0).fetch(left, slot, z);
      bc.fetch(a, p, r, tile0, left, 0);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        u[i] = load_as<S>(&x[i], 0);
        D[i] = load_as<S>(&dt[i], 0);
        g[i] = load_as<S>(&dy[i], 0);
        if constexpr (Z) {
          const S v = load_as<S>(&z[i], 0);
          g[i] *= v * sigmoid_(v);
        }
      }
    }
    ssm_steps<S, TT>(a.softplus, bias, D);
    if (left < L::TILE || p.nch < CH) {  // past the end and beside the channels nothing changes
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const bool there = in && i < here;
        D[i] = there ? D[i] : S(0);
        u[i] = there ? u[i] : S(0);
        g[i] = there ? g[i] : S(0);
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      dskip = fma_(g[i], u[i], dskip);
      if constexpr (Z) sy[i / YV * YV * L::THREADS + i % YV] = skip * u[i];
      u[i] *= D[i];
      sum += D[i];
      du[i] = S(0);
      dD[i] = S(0);
    }
    for (int n0 = 0; n0 < np; n0 += NB) {
      if (n0) bc.fetch(a, p, r, tile0, left, n0);
      __syncthreads();
      bc.store(a, p, r, tile0, left, n0, sB, sC);
      for (int i = threadIdx.x; i < NB * CH; i += L::THREADS) {
        const int n = n0 + i / CH, ch = i % CH;
        const bool there = n < a.Ns && ch < p.nch;
        sS[n0 * CH + i] = there ? static_cast<const S*>(a.ckpt)[((ck0 + tile) * a.Ns + n) * a.D + p.d0 + ch] : S(0);
      }
      __syncthreads();
      for (int n1 = 0; n1 < NB; n1 += NS) {
        const int n = n0 + n1;
        if (n >= a.Ns) break;
        BC B(sB + L::at(slot * TT, n1)), C(sC + L::at(slot * TT, n1));
        B.load(0);
        S A[NS], P[NS], Pb[NS], h[NS], s[NS], enter[NS], e[TT][NS], q[TT][NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          A[j] = sA[(n + j) * CH + c];
          enter[j] = sS[(n + j) * CH + c];
          P[j] = Pb[j] = exp2_(A[j] * sum);
          h[j] = s[j] = S(0);
        }
        // the slot's effect on the state, and on the gradient that comes from later tokens
#pragma unroll
        for (int i = 0; i < TT; i += BL) {
          if (i + BL < TT) B.load(i + BL);
          else C.load(i);
#pragma unroll
          for (int k = i; k < i + BL; ++k)
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              e[k][j] = exp2_(D[k] * A[j]);
              h[j] = fma_(e[k][j], h[j], u[k] * B.at(k, j));
            }
          fence_order();
        }
#pragma unroll
        for (int i = TT - BL; i >= 0; i -= BL) {
          if (i > 0) C.load(i - BL);
          else B.load(0);
#pragma unroll
          for (int k = i + BL - 1; k >= i; --k)
#pragma unroll
            for (int j = 0; j < NS; ++j) s[j] = e[k][j] * fma_(C.at(k, j), g[k], s[j]);
          fence_order();
        }
        S* const at = agg + turn * 2 * L::AGG;
        turn ^= 1;
        SsmScan<L, false>::leave(P, h, at);
        SsmScan<L, true>::leave(Pb, s, at + L::AGG);
        __syncthreads();
        SsmScan<L, false>::take(P, h, enter, at);
        settle();
        fence_order();
        // the states, and the products that dC sums
        Sums<L, false> sumC(partC + (n / NS) * plane + (tile0 + slot * TT) * NS, c, here);
        static_assert(YV == BL, "y in the same blocks");
#pragma unroll
        for (int i = 0; i < TT; i += BL) {
          if (i + BL < TT) {
            B.load(i + BL);
            C.load(i + BL);
          }
          S y[BL];
          if constexpr (Z) lds_get<S, BL>(sy + i * L::THREADS, y);
#pragma unroll
          for (int k = 0; k < BL; ++k) {
            S v[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              q[i + k][j] = e[i + k][j] * h[j];
              h[j] = fma_(u[i + k], B.at(i + k, j), q[i + k][j]);
              if constexpr (Z) y[k] = fma_(C.at(i + k, j), h[j], y[k]);
              v[j] = g[i + k] * h[j];
            }
            sumC.put(i + k, v);
          }
          if constexpr (Z) {
#pragma unroll
            for (int k = 0; k < BL; ++k) sy[i * L::THREADS + k] = y[k];
          }
          fence_order();
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) enter[j] = sl[(n + j) * CH + c];
        SsmScan<L, true>::take(Pb, s, enter, at + L::AGG);
        fence_order();
        S dA[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) dA[j] = S(0);
        Sums<L, true> sumB(partB + (n / NS) * plane + (tile0 + slot * TT) * NS, c, here);
#pragma unroll
        for (int i = TT - BL; i >= 0; i -= BL) {
          if (i > 0) {
            B.load(i - BL);
            C.load(i - BL);
          }
#pragma unroll
          for (int k = i + BL - 1; k >= i; --k) {
            S v[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              const S gt = fma_(C.at(k, j), g[k], s[j]), gq = gt * q[k][j];
              du[k] = fma_(gt, B.at(k, j), du[k]);
              dD[k] = fma_(gq, A[j], dD[k]);
              dA[j] = fma_(gq, D[k], dA[j]);
              v[j] = gt * u[k];
              s[j] = e[k][j] * gt;
            }
            sumB.put(k, v);
          }
          fence_order();
        }
        if (slot == 0) {
#pragma unroll
          for (int j = 0; j < NS; ++j) sl1[(n + j) * CH + c] = s[j];
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) {
#pragma unroll
          for (int m = CH; m < 64; m <<= 1) dA[j] += __shfl_xor(dA[j], m, 64);
          if (ts == 0) red[rturn * W * CH * NS + wave * CH * NS + c * NS + j] = dA[j];
        }
        rturn ^= 1;
        pending = n;
      }
    }
    S* const other = sl;
    sl = sl1;
    sl1 = other;
    IO ex[TT], ed[TT], eg[Z ? TT : 1], ez[Z ? TT : 1];
    SlotRows<IO, L>(a.x, a.sx, r, p.d0, cc, slot, tile0).fetch(left, slot, ex);
    SlotRows<IO, L>(a.dt, a.sdt, r, p.d0, cc, slot, tile0).fetch(left, slot, ed);
    if constexpr (Z) {
      SlotRows<IO, L>(a.dy, a.sdy, r, p.d0, cc, slot, tile0).fetch(left, slot, eg);
      SlotRows<IO, L>(a.z, a.sz, r, p.d0, cc, slot, tile0).fetch(left, slot, ez);
    }
    const SlotRows<IO, L> odx(a.dx, a.sdx, r, p.d0, cc, slot, tile0), odt(a.ddt, a.sddt, r, p.d0, cc, slot, tile0);
    S raw[TT];
    if (a.softplus) {
#pragma unroll
      for (int i = 0; i < TT; ++i) raw[i] = sigmoid_(load_as<S>(&ed[i], 0) + bias);
    } else {
#pragma unroll
      for (int i = 0; i < TT; ++i) raw[i] = S(1);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      if (in && i < here) {
        const S dd = fma_(dD[i], static_cast<S>(1.0 / kLog2e), load_as<S>(&ex[i], 0) * du[i]) * raw[i];
        dbias += dd;
        put(odt.out(i), dd);
        put(odx.out(i), fma_(D[i], du[i], skip * g[i]));
      }
    }
    if constexpr (Z) {
      const SlotRows<IO, L> odz(a.dz, a.sdz, r, p.d0, cc, slot, tile0);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const S z = load_as<S>(&ez[i], 0), k = sigmoid_(z);
        const S y = sy[i / YV * YV * L::THREADS + i % YV];
        if (in && i < here) put(odz.out(i), load_as<S>(&eg[i], 0) * y * (k * (S(1) + z * (S(1) - k))));
      }
    }
  }
  __syncthreads();
  settle();
  // sums over the slots
  sB[threadIdx.x] = dskip;
  sB[L::THREADS + threadIdx.x] = dbias;
  static_assert(L::BC >= 2 * L::THREADS, "room for the slots' sums");
  __syncthreads();
  S* const par = static_cast<S*>(a.part_par) + p.n * (a.Ns + 2) * a.D;
  for (int i = threadIdx.x; i < np * CH; i += L::THREADS) {
    const int n = i / CH, ch = i % CH;
    if (n < a.Ns && ch < p.nch) par[static_cast<int64_t>(n) * a.D + p.d0 + ch] = sdA[i];
  }
  for (int i = threadIdx.x; i < 2 * CH; i += L::THREADS) {
    const int which = i / CH, ch = i % CH;
    S x = S(0);
    for (int k = 0; k < L::SL; ++k) x += sB[which * L::THREADS + k * CH + ch];
    if (ch < p.nch) par[static_cast<int64_t>(a.Ns + which) * a.D + p.d0 + ch] = x;
  }
  if (!a.dstate_in) return;
  for (int i = threadIdx.x; i < np * CH; i += L::THREADS) {
    const int n = i % np, ch = i / np;
    if (n < a.Ns && ch < p.nch)
      static_cast<S*>(a.dstate_in)[(p.n * a.D + p.d0 + ch) * a.Ns + n] = sl[n * CH + ch];
  }
}

// dB and dC from the parts of the channel blocks, dA, dskip and dbias from those
// of the sequences.
constexpr int kSumThreads = 256;
template <typename IO, typename S, int NS>
__global__ __launch_bounds__(kSumThreads) void ssm_bwd_sums(SsmArgs a, int nb, int64_t bc_groups) {
  const int groups = (a.Ns + NS - 1) / NS;
  const int64_t tok = a.B * a.T;
  if (blockIdx.x < bc_groups) {
    const int64_t per = groups * tok * NS;  // of one group of channels, of B or of C
    int64_t behind = tok;  // no parts are there for the tokens behind the last packed sequence
    if (a.packed) {
      const SeqRange r = seq_range(a.cu, a.N - 1, a.T);
      behind = r.t0 + r.len;
    }
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kSumThreads) + threadIdx.x; i < 2 * a.G * per;
         i += bc_groups * kSumThreads) {
      const int64_t which = i / (a.G * per), g = i / per % a.G, o = i % per;
      const int j = static_cast<int>(o % NS);
      const int64_t t = o / NS % tok, n = o / (NS * tok) * NS + j;
      if (n >= a.Ns) continue;
      const S* part = static_cast<const S*>(a.part_bc) + (which * a.G + g) * nb * per + o;
      const int there = t < behind ? nb : 0;
      S x = S(0);
      int k = 0;
      for (; k + 8 <= there; k += 8) {
        S v[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) v[m] = part[(k + m) * per];
#pragma unroll
        for (int m = 0; m < 8; ++m) x += v[m];
      }
      for (; k < there; ++k) x += part[k * per];
      const Rows& st = which ? a.sdC : a.sdB;
      IO* out = static_cast<IO*>(which ? a.dC : a.dB) + t / a.T * st.b + t % a.T * st.t + g * st.g;
      store_from(out, n, x);
    }
    return;
  }
  const int64_t i = (blockIdx.x - bc_groups) * kSumThreads + threadIdx.x;
  if (i >= static_cast<int64_t>(a.Ns + 2) * a.D) return;
  const int n = static_cast<int>(i / a.D), d = static_cast<int>(i % a.D);
  S* out = static_cast<S*>(n < a.Ns ? a.dA : n == a.Ns ? a.dskip : a.dbias);
  if (!out) return;
  const S* part = static_cast<const S*>(a.part_par) + i;
  const int64_t step = static_cast<int64_t>(a.Ns + 2) * a.D;
  S x = S(0);
#pragma unroll 4
  for (int64_t k = 0; k < a.N; ++k) x += part[k * step];
  out[n < a.Ns ? static_cast<int64_t>(d) * a.Ns + n : d] = x;
}

constexpr int kNS = 2;

// Work-groups of the sums: for dB and dC, for the parameters.
struct SumGroups {
  int64_t bc, par;
  explicit SumGroups(const SsmArgs& a) {
    const int64_t sums = 2 * a.G * ((a.Ns + kNS - 1) / kNS) * a.B * a.T * kNS;
    bc = std::min<int64_t>((sums + kSumThreads - 1) / kSumThreads, 1 << 23);
    par = (static_cast<int64_t>(a.Ns + 2) * a.D + kSumThreads - 1) / kSumThreads;
  }
};

template <typename IO, typename L>
hipError_t go(int io, const SsmArgs& a, hipStream_t s) {
  const int64_t blocks = ssm_blocks(a, L::CH);
  if (a.N * blocks > 0) {
    SsmArgs b = a;
    b.vec_bc = ssm_vec_bc(io, a);
    const unsigned g = static_cast<unsigned>(a.N * blocks);
    if (a.z) ssm_bwd<IO, L, true><<<g, L::THREADS, bwd_lds<L, true>(a.Ns), s>>>(b);
    else ssm_bwd<IO, L, false><<<g, L::THREADS, bwd_lds<L, false>(a.Ns), s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const SumGroups g(a);
  if (g.bc + g.par == 0) return hipSuccess;
  ssm_bwd_sums<IO, typename L::S, kNS>
      <<<static_cast<unsigned>(g.bc + g.par), kSumThreads, 0, s>>>(a, static_cast<int>(a.G ? blocks / a.G : 0), g.bc);
  return hipGetLastError();
}

template <typename IO, typename S, int TT>
hipError_t by_channels(int io, int channels, const SsmArgs& a, hipStream_t s) {
  switch (channels) {
    case 32: return go<IO, SsmTile<S, 32, kSsmWaves, TT, kNS, 16>>(io, a, s);
    case 16: return go<IO, SsmTile<S, 16, kSsmWaves, TT, kNS, 8>>(io, a, s);
    default: return go<IO, SsmTile<S, 8, kSsmWaves, TT, kNS, sizeof(S) == 8 ? 4 : 8>>(io, a, s);
  }
}
template <typename IO>
hipError_t by_shape(int io, const SsmShape& p, const SsmArgs& a, hipStream_t s) {
  if (p.tokens == kSsmShort) return by_channels<IO, float, kSsmShort>(io, p.channels, a, s);
  return by_channels<IO, float, 16>(io, p.channels, a, s);
}

}  // namespace

static size_t bc_bytes(int io, const SsmArgs& a, int CH) {
  return static_cast<size_t>(2 * ssm_blocks(a, CH)) * ((a.Ns + kNS - 1) / kNS * kNS) * a.B * a.T * (io == IO_F64 ? 8 : 4);
}
SsmShape ssm_bwd_shape(int io, const SsmArgs& a) {
  const int n = io == IO_F64 ? 2 * a.Ns : a.Ns;
  const int most = n <= 64 ? 32 : n <= 128 ? 16 : 8;
  SsmShape p = ssm_shape(a, io, most);
  while (p.channels < most && bc_bytes(io, a, p.channels) > (size_t(1) << 30)) p.channels *= 2;
  return p;
}
size_t ssm_bc_bytes(int io, const SsmArgs& a) { return bc_bytes(io, a, ssm_bwd_shape(io, a).channels); }

bool ssm_bwd_fits(int io, const SsmArgs& a) {
  const SumGroups g(a);
  return ssm_bwd_shape(io, a).fits(a) && launch_fits((g.bc + g.par) * kSumThreads);
}

hipError_t launch_ssm_bwd(int io, const SsmArgs& a, hipStream_t s) {
  if (!ssm_bwd_fits(io, a)) return hipErrorInvalidConfiguration;
  const SsmShape p = ssm_bwd_shape(io, a);
  if (io == IO_F64) return by_channels<double, double, 8>(io, p.channels, a, s);
  if (io == IO_F32) return by_shape<float>(io, p, a, s);
  return by_shape<bf16>(io, p, a, s);
}

}  // namespace gls
