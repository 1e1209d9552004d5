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
  return sizeof(typename L::S) * (2 * L::BC + 5 * static_cast<size_t>(L::npad(N)) * L::CH + 2 * L::W * L::CH * 2 * L::NS +
                                  2 * L::W * L::CH * L::NS + (Z ? L::THREADS * L::TT : 0));
}

template <typename IO, typename L, bool Z>
__global__ __launch_bounds__(L::THREADS) void ssm_bwd(SsmArgs a) {
  using S = typename L::S;
  using BC = SlotBC<L>;
  constexpr int CH = L::CH, TT = L::TT, NS = L::NS, NB = L::NB, W = L::W, K = BC::K;
  extern __shared__ __align__(16) char lds[];
  const int np = L::npad(a.Ns);
  S* const sB = reinterpret_cast<S*>(lds);
  S* const sC = sB + L::BC;
  S* const agg = sC + L::BC;                      // [2][W][CH][2 NS]
  S* const red = agg + 2 * W * CH * 2 * NS;       // [2][W][CH][NS]
  S* const sA = red + 2 * W * CH * NS;            // [np][CH]
  S* const sdA = sA + np * CH;                    // [np][CH]
  S* const sS = sdA + np * CH;                    // [np][CH]
  S* sl = sS + np * CH;                           // [2][np][CH]
  S* sl1 = sl + np * CH;
  // y before the gate, in LDS: kept over all states, it is more than the registers hold
  // beside what the passes need (98 registers spilled, and every wait for one of them a
  // wait for the sums' stores: 1587 us instead of 749 at 4 x 4096 x 2048 x 16)
  constexpr int YV = 16 / sizeof(S);
  S* const sy = sS + 3 * np * CH + threadIdx.x * YV;  // [TT / YV][threads][YV]
  const int64_t blocks = static_cast<int64_t>(gridDim.x) / a.N;
  const int64_t id = xcd_order(blockIdx.x, gridDim.x);
  const SsmPlace p = ssm_place(a, CH, id);
  const SeqRange r = seq_range(a.cu, p.n, a.T);
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
    SlotRows<IO, L>(a.x, a.sx, r, p.d0, cc, slot, tile0).ld(left, slot, u);
    SlotRows<IO, L>(a.dt, a.sdt, r, p.d0, cc, slot, tile0).ld(left, slot, D);
    SlotRows<IO, L>(a.dy, a.sdy, r, p.d0, cc, slot, tile0).ld(left, slot, g);
    if constexpr (Z) {
      S z[TT];
      SlotRows<IO, L>(a.z, a.sz, r, p.d0, cc, slot, tile0).ld(left, slot, z);
#pragma unroll
      for (int i = 0; i < TT; ++i) g[i] *= z[i] * sigmoid_(z[i]);
    }
    ssm_steps<S, TT>(a.softplus, bias, in ? here : 0, D);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const bool there = in && i < here;
      u[i] = there ? u[i] : S(0);
      g[i] = there ? g[i] : S(0);
      dskip = fma_(g[i], u[i], dskip);
      if constexpr (Z) sy[i / YV * YV * L::THREADS + i % YV] = skip * u[i];
      u[i] *= D[i];
      sum += D[i];
      du[i] = S(0);
      dD[i] = S(0);
    }
    for (int n0 = 0; n0 < np; n0 += NB) {
      __syncthreads();
      ssm_load_bc<IO, L>(a, p, r, tile0, n0, sB, sC);
      for (int i = threadIdx.x; i < NB * CH; i += L::THREADS) {
        const int n = n0 + i / CH, ch = i % CH;
        const bool there = n < a.Ns && ch < p.nch;
        sS[n0 * CH + i] = there ? static_cast<const S*>(a.ckpt)[((ck0 + tile) * a.Ns + n) * a.D + p.d0 + ch] : S(0);
      }
      __syncthreads();
      for (int n1 = 0; n1 < NB; n1 += NS) {
        const int n = n0 + n1;
        if (n >= a.Ns) break;
        const S* bp = sB + L::at(slot * TT, n1);
        const S* cp = sC + L::at(slot * TT, n1);
        S A[NS], P[NS], Pb[NS], h[NS], s[NS], enter[NS], e[TT][NS], q[TT][NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          A[j] = sA[(n + j) * CH + c];
          enter[j] = sS[(n + j) * CH + c];
          P[j] = Pb[j] = exp2_(A[j] * sum);
          h[j] = S(0);
        }
        // the slot's effect on the state
#pragma unroll
        for (int i = 0; i < TT; i += K) {
          const BC B(bp, i);
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              e[i + k][j] = exp2_(D[i + k] * A[j]);
              h[j] = fma_(e[i + k][j], h[j], u[i + k] * B.v[k][j]);
            }
          if (i % 4 == 0) fence_order();
        }
        ssm_scan<L, false>(P, h, enter, agg, turn);
        settle();
        fence_order();
        // the states, and the products that dC sums
        Sums<L, false> sumC(partC + (n / NS) * plane + (tile0 + slot * TT) * NS, c, here);
        S y[YV];
#pragma unroll
        for (int i = 0; i < TT; i += K) {
          const BC B(bp, i), C(cp, i);
          if constexpr (Z) {
            if (i % YV == 0) lds_get<S, YV>(sy + i * L::THREADS, y);
          }
#pragma unroll
          for (int k = 0; k < K; ++k) {
            S v[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              q[i + k][j] = e[i + k][j] * h[j];
              h[j] = fma_(u[i + k], B.v[k][j], q[i + k][j]);
              if constexpr (Z) y[(i + k) % YV] = fma_(C.v[k][j], h[j], y[(i + k) % YV]);
              v[j] = g[i + k] * h[j];
            }
            sumC.put(i + k, v);
          }
          if constexpr (Z) {
            if ((i + K) % YV == 0) {
#pragma unroll
              for (int k = 0; k < YV; ++k) sy[(i + K - YV) * L::THREADS + k] = y[k];
            }
          }
          if (i % 4 == 0) fence_order();
        }
        fence_order();
        // the slot's effect on the gradient that comes from later tokens
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          s[j] = S(0);
          enter[j] = sl[(n + j) * CH + c];
        }
#pragma unroll
        for (int i = TT - K; i >= 0; i -= K) {
          const BC C(cp, i);
#pragma unroll
          for (int k = K - 1; k >= 0; --k)
#pragma unroll
            for (int j = 0; j < NS; ++j) s[j] = e[i + k][j] * fma_(C.v[k][j], g[i + k], s[j]);
          if (i % 4 == 0) fence_order();
        }
        ssm_scan<L, true>(Pb, s, enter, agg, turn);
        fence_order();
        S dA[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) dA[j] = S(0);
        Sums<L, true> sumB(partB + (n / NS) * plane + (tile0 + slot * TT) * NS, c, here);
#pragma unroll
        for (int i = TT - K; i >= 0; i -= K) {
          const BC B(bp, i), C(cp, i);
#pragma unroll
          for (int k = K - 1; k >= 0; --k) {
            S v[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              const S gt = fma_(C.v[k][j], g[i + k], s[j]), gq = gt * q[i + k][j];
              du[i + k] = fma_(gt, B.v[k][j], du[i + k]);
              dD[i + k] = fma_(gq, A[j], dD[i + k]);
              dA[j] = fma_(gq, D[i + k], dA[j]);
              v[j] = gt * u[i + k];
              s[j] = e[i + k][j] * gt;
            }
            sumB.put(i + k, v);
          }
          if (i % 4 == 0) fence_order();
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
    S x[TT], raw[TT];
    SlotRows<IO, L>(a.x, a.sx, r, p.d0, cc, slot, tile0).ld(left, slot, x);
    SlotRows<IO, L>(a.dt, a.sdt, r, p.d0, cc, slot, tile0).ld(left, slot, raw);
    const SlotRows<IO, L> odx(a.dx, a.sdx, r, p.d0, cc, slot, tile0), odt(a.ddt, a.sddt, r, p.d0, cc, slot, tile0);
    if (a.softplus) {
#pragma unroll
      for (int i = 0; i < TT; ++i) raw[i] = sigmoid_(raw[i] + bias);
    } else {
#pragma unroll
      for (int i = 0; i < TT; ++i) raw[i] = S(1);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      if (in && i < here) {
        const S dd = fma_(dD[i], static_cast<S>(1.0 / kLog2e), x[i] * du[i]) * raw[i];
        dbias += dd;
        put(odt.out(i), dd);
        put(odx.out(i), fma_(D[i], du[i], skip * g[i]));
      }
    }
    if constexpr (Z) {
      S z[TT], dy[TT];
      SlotRows<IO, L>(a.z, a.sz, r, p.d0, cc, slot, tile0).ld(left, slot, z);
      SlotRows<IO, L>(a.dy, a.sdy, r, p.d0, cc, slot, tile0).ld(left, slot, dy);
      const SlotRows<IO, L> odz(a.dz, a.sdz, r, p.d0, cc, slot, tile0);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const S k = sigmoid_(z[i]);
        const S y = sy[i / YV * YV * L::THREADS + i % YV];
        if (in && i < here) put(odz.out(i), dy[i] * y * (k * (S(1) + z[i] * (S(1) - k))));
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
    const int64_t i = blockIdx.x * static_cast<int64_t>(kSumThreads) + threadIdx.x;
    if (i >= 2 * a.G * per) return;
    const int64_t which = i / (a.G * per), g = i / per % a.G, o = i % per;
    const int j = static_cast<int>(o % NS);
    const int64_t t = o / NS % tok, n = o / (NS * tok) * NS + j;
    if (n >= a.Ns) return;
    const S* part = static_cast<const S*>(a.part_bc) + (which * a.G + g) * nb * per + o;
    S x = S(0);
    int k = 0;
    for (; k + 8 <= nb; k += 8) {
      S v[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) v[m] = part[(k + m) * per];
#pragma unroll
      for (int m = 0; m < 8; ++m) x += v[m];
    }
    for (; k < nb; ++k) x += part[k * per];
    const Rows& st = which ? a.sdC : a.sdB;
    IO* out = static_cast<IO*>(which ? a.dC : a.dB) + t / a.T * st.b + t % a.T * st.t + g * st.g;
    store_from(out, n, x);
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
  const int64_t bc = 2 * a.G * ((a.Ns + kNS - 1) / kNS) * a.B * a.T * kNS, par = static_cast<int64_t>(a.Ns + 2) * a.D;
  const int64_t g1 = (bc + kSumThreads - 1) / kSumThreads, g2 = (par + kSumThreads - 1) / kSumThreads;
  if (g1 + g2 == 0) return hipSuccess;
  ssm_bwd_sums<IO, typename L::S, kNS>
      <<<static_cast<unsigned>(g1 + g2), kSumThreads, 0, s>>>(a, static_cast<int>(a.G ? blocks / a.G : 0), g1);
  return hipGetLastError();
}

template <typename IO, typename S, int TT>
hipError_t by_states(int io, const SsmArgs& a, hipStream_t s) {
  switch (ssm_bwd_channels(io, a.Ns)) {
    case 32: return go<IO, SsmTile<S, 32, 8, TT, kNS, 16>>(io, a, s);
    case 16: return go<IO, SsmTile<S, 16, 8, TT, kNS, 8>>(io, a, s);
    default: return go<IO, SsmTile<S, 8, 8, TT, kNS, sizeof(S) == 8 ? 4 : 8>>(io, a, s);
  }
}

}  // namespace

size_t ssm_bc_bytes(int io, const SsmArgs& a) {
  const int64_t blocks = ssm_blocks(a, ssm_bwd_channels(io, a.Ns));
  return static_cast<size_t>(2 * blocks) * ((a.Ns + kNS - 1) / kNS * kNS) * a.B * a.T * (io == IO_F64 ? 8 : 4);
}
hipError_t launch_ssm_bwd(int io, const SsmArgs& a, hipStream_t s) {
  if (io == IO_F64) return by_states<double, double, 8>(io, a, s);
  if (io == IO_F32) return by_states<float, float, 16>(io, a, s);
  return by_states<bf16, float, 16>(io, a, s);
}

}  // namespace gls
