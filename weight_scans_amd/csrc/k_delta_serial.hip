// k_delta_serial.hip -- the gated delta rule token by token on the vector ALU:
// any io dtype, 1 <= dk, dv <= 128, any strides.  Forward, backward, and the
// one-token step of serving.
//
//   e = v - a S k;  S <- a S + (beta e) k^T;  y = scale S q
//
// The rows of S are independent chains (a row meets the others only through
// sums over dv in the gradients), so a work-group owns 16 rows of one
// sequence-head, 16 lanes to a row, the row's state in registers for all
// tokens.  One round of lane sums per token serves both products with S:
// with p = S k, r = S q taken from the old state,
//   e = v - a p,   y = scale (a r + beta e (k.q)).
// Bound by the chain of one token (a product, a sum over 16 lanes, an update:
// 0.3 us a token forward, 1.0 us backward at 64 x 64 in fp32); it serves what the
// chunks do not take: fp64, odd sizes and strides, the shortest sequences.
//
// Backward, with A_t = dL/dS_t (y_t's share included), g = scale dy:
//   A += g q^T;  du = A k;  f = beta du (= dv);  dbeta = du.e
//   dq = S_t^T g;  dk = A^T u - a S_{t-1}^T f;  dlog_alpha = a <A - f k^T, S_{t-1}>
//   A <- a (A - f k^T)
// from states kept before every 16th (fp64: 8th) token: a chunk's states are
// computed again from its first one and kept in LDS (16 rows of 16 tokens fill
// it), then its tokens are walked from the right.  Sums over rows leave as one
// part per 16 rows and are added in a fixed order afterwards.
#include <algorithm>

#include "delta.hpp"
#include "dev_common.hpp"
#include "mfma.hpp"

namespace gls {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kSerialRows;

template <typename S>
struct Ck;
template <>
struct Ck<float> { static constexpr int v = 16; };
template <>
struct Ck<double> { static constexpr int v = 8; };

// Sum over the 16 lanes of a row of lanes, in every lane (the same bits in
// each: every step adds the same two partial sums).
__device__ __forceinline__ float sum16(float x) {
  x += dpp<0x128>(0.f, x);  // row_ror:8, 4, 2, 1
  x += dpp<0x124>(0.f, x);
  x += dpp<0x122>(0.f, x);
  x += dpp<0x121>(0.f, x);
  return x;
}
__device__ __forceinline__ double sum16(double x) {
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}
// Sum over the four rows of lanes.
__device__ __forceinline__ float sum4rows(float x) { return sum_rows(x); }
__device__ __forceinline__ double sum4rows(double x) {
  x += __shfl_xor(x, 16, 64);
  x += __shfl_xor(x, 32, 64);
  return x;
}

__device__ __forceinline__ float gexp(float x) { return expf(x); }
__device__ __forceinline__ double gexp(double x) { return exp(x); }

template <typename IO, typename S>
__device__ __forceinline__ S load_gate(const void* p, int64_t i, bool io) {
  return io ? load_as<S>(static_cast<const IO*>(p), i) : static_cast<const S*>(p)[i];
}

// Columns of lane `l`: 4 l .. 4 l + 3 of every 64.
__device__ __forceinline__ int col(int l, int i) { return (i >> 2) * 64 + l * 4 + (i & 3); }

// Tokens t0 .. t0 + TC - 1 of a head of [.., T, d] rows, fetched into registers
// while the tokens before them are walked, then put into LDS as [TC][W] with
// zeros past d and past nt.  The loads are at indices clamped into the tensor: a
// load under a condition would be waited for before the next one is issued.
template <typename IO, typename S, int TC, int W>
struct Rows {
  static constexpr int N = TC * W / kThreads;
  S v[N];
  __device__ __forceinline__ void fetch(const IO* base, int64_t st, int64_t t0, int64_t len, int d) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = threadIdx.x + i * kThreads, t = x / W, c = min(x % W, d - 1);
      v[i] = load_as<S>(base, min(t0 + t, len - 1) * st + c);
    }
  }
  __device__ __forceinline__ void put(S* lds, int nt, int d) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = threadIdx.x + i * kThreads;
      lds[x] = x / W < nt && x % W < d ? v[i] : S(0);
    }
  }
};
// The same of one row tile of values ([TC][kRows], a thread an element) and of
// the gates (the first TC threads).
template <typename IO, typename S>
__device__ __forceinline__ S fetch_rows(const IO* base, int64_t st, int64_t t0, int64_t len, int r0, int d) {
  const int t = threadIdx.x / kRows, c = min(r0 + static_cast<int>(threadIdx.x) % kRows, d - 1);
  return load_as<S>(base, min(t0 + t, len - 1) * st + c);
}

template <typename IO, typename S, int NI>
__global__ __launch_bounds__(kThreads) void delta_serial_fwd(DeltaArgs a) {
  constexpr int TC = 16, W = NI * 16, CK = Ck<S>::v;
  __shared__ __align__(16) S qs[TC * W], ks[TC * W];
  __shared__ S vs[TC * kRows], ys[TC * kRows], ga[TC], gb[TC], kq[TC];
  const int tiles = (a.dv + kRows - 1) / kRows;
  const int64_t id = blockIdx.x;
  const int r0 = static_cast<int>(id % tiles) * kRows;
  const int h = static_cast<int>(id / tiles % a.H);
  const int64_t n = id / tiles / a.H;
  const int hk = h / (a.H / a.Hk);
  const SeqRange sr = seq_range(a.cu, n, a.T);
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int r = r0 + row;
  const S scale = static_cast<S>(a.scale);

  S st[NI];
  const int64_t so = ((n * a.H + h) * a.dv + r) * a.dk;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = col(l, i);
    st[i] = (a.state_in && r < a.dv && c < a.dk) ? static_cast<const S*>(a.state_in)[so + c] : S(0);
  }
  const IO* q = static_cast<const IO*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
  const IO* k = static_cast<const IO*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
  const IO* v = static_cast<const IO*>(a.v) + sr.b * a.sv.b + h * a.sv.h + sr.t0 * a.sv.t;
  IO* y = a.y ? static_cast<IO*>(a.y) + sr.b * a.sy.b + h * a.sy.h + sr.t0 * a.sy.t : nullptr;
  const int64_t go = sr.b * a.sg.b + h * a.sg.h + sr.t0 * a.sg.t;
  const int64_t slot0 = chunk_slot0(a.cu != nullptr, n, sr.t0, a.T, CK);

  Rows<IO, S, TC, W> qn, kn;
  S vn = S(0), an = S(0), bn = S(0);
  const auto fetch = [&](int64_t t0) {
    if (y) qn.fetch(q, a.sq.t, t0, sr.len, a.dk);
    kn.fetch(k, a.sk.t, t0, sr.len, a.dk);
    vn = fetch_rows<IO, S>(v, a.sv.t, t0, sr.len, r0, a.dv);
    const int64_t o = go + min(t0 + static_cast<int64_t>(threadIdx.x % TC), sr.len - 1) * a.sg.t;
    an = load_gate<IO, S>(a.la, o, a.gate_io);
    bn = load_gate<IO, S>(a.be, o, a.gate_io);
  };
  if (sr.len > 0) fetch(0);
  for (int64_t t0 = 0; t0 < sr.len; t0 += TC) {
    const int nt = static_cast<int>(sr.len - t0 < TC ? sr.len - t0 : TC);
    __syncthreads();
    if (y) qn.put(qs, nt, a.dk);
    kn.put(ks, nt, a.dk);
    vs[threadIdx.x] = vn;  // rows past dv and tokens past nt go nowhere
    if (threadIdx.x < TC) {
      const bool in = static_cast<int>(threadIdx.x) < nt;
      ga[threadIdx.x] = in ? gexp(an) : S(1);
      gb[threadIdx.x] = in ? bn : S(0);
    }
    __syncthreads();
    if (t0 + TC < sr.len) fetch(t0 + TC);
    if (y) {
      S p = S(0);  // k.q of token `row`
#pragma unroll
      for (int i = 0; i < NI; ++i) p += ks[row * W + col(l, i)] * qs[row * W + col(l, i)];
      p = sum16(p);
      if (l == 0) kq[row] = p;
      __syncthreads();
    }
    for (int t = 0; t < nt; ++t) {
      if (a.ckpt && t % CK == 0 && r < a.dv) {
        S* c0 = static_cast<S*>(a.ckpt) + (((slot0 + (t0 + t) / CK) * a.H + h) * a.dv + r) * a.dk;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (col(l, i) < a.dk) c0[col(l, i)] = st[i];
      }
      S kv[NI], p = S(0), z = S(0);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        kv[i] = ks[t * W + col(l, i)];
        p += st[i] * kv[i];
      }
      if (y) {
#pragma unroll
        for (int i = 0; i < NI; ++i) z += st[i] * qs[t * W + col(l, i)];
      }
      p = sum16(p);
      const S al = ga[t], u = gb[t] * (vs[t * kRows + row] - al * p);
      if (y) {
        z = sum16(z);
        if (l == 0) ys[t * kRows + row] = scale * (al * z + u * kq[t]);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) st[i] = al * st[i] + u * kv[i];
    }
    if (y) {
      __syncthreads();
      const int t = threadIdx.x / kRows, c = threadIdx.x % kRows;
      if (t < nt && r0 + c < a.dv) store_from(y, (t0 + t) * a.sy.t + r0 + c, ys[threadIdx.x]);
    }
  }
  if (a.state_out && r < a.dv) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (col(l, i) < a.dk) static_cast<S*>(a.state_out)[so + col(l, i)] = st[i];
  }
}

template <typename IO, typename S, int NI>
__global__ __launch_bounds__(kThreads) void delta_serial_bwd(DeltaArgs a) {
  constexpr int TC = Ck<S>::v, W = NI * 16;
  __shared__ __align__(16) S qs[TC * W], ks[TC * W];
  __shared__ S hist[TC * NI * kThreads];  // S_{t-1}, each lane's own columns
  __shared__ S red[4][2][W], redg[4][2];
  __shared__ S vs[TC * kRows], gs[TC * kRows], es[TC * kRows], ga[TC], gb[TC];
  const int tiles = (a.dv + kRows - 1) / kRows;
  const int64_t id = blockIdx.x;
  const int tile = static_cast<int>(id % tiles), r0 = tile * kRows;
  const int h = static_cast<int>(id / tiles % a.H);
  const int64_t n = id / tiles / a.H;
  const int hk = h / (a.H / a.Hk);
  const SeqRange sr = seq_range(a.cu, n, a.T);
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int lane = threadIdx.x & 63;
  const int r = r0 + row;
  const S scale = static_cast<S>(a.scale);

  S A[NI];
  const int64_t so = ((n * a.H + h) * a.dv + r) * a.dk;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = col(l, i);
    A[i] = (a.dstate_out && r < a.dv && c < a.dk) ? static_cast<const S*>(a.dstate_out)[so + c] : S(0);
  }
  const IO* q = static_cast<const IO*>(a.q) + sr.b * a.sq.b + hk * a.sq.h + sr.t0 * a.sq.t;
  const IO* k = static_cast<const IO*>(a.k) + sr.b * a.sk.b + hk * a.sk.h + sr.t0 * a.sk.t;
  const IO* v = static_cast<const IO*>(a.v) + sr.b * a.sv.b + h * a.sv.h + sr.t0 * a.sv.t;
  const IO* dy = static_cast<const IO*>(a.dy) + sr.b * a.sdy.b + h * a.sdy.h + sr.t0 * a.sdy.t;
  IO* dv = static_cast<IO*>(a.dv_) + sr.b * a.sdv.b + h * a.sdv.h + sr.t0 * a.sdv.t;
  const int64_t go = sr.b * a.sg.b + h * a.sg.h + sr.t0 * a.sg.t;
  const int64_t slot0 = chunk_slot0(a.cu != nullptr, n, sr.t0, a.T, TC);
  const int64_t part0 = (static_cast<int64_t>(tile) * a.H + h) * a.B * a.T + sr.b * a.T + sr.t0;
  S* pq = static_cast<S*>(a.part_dq) + part0 * a.dk;
  S* pk = static_cast<S*>(a.part_dk) + part0 * a.dk;
  S* pl = static_cast<S*>(a.part_la) + part0;
  S* pb = static_cast<S*>(a.part_be) + part0;

  Rows<IO, S, TC, W> qn, kn;
  S vn = S(0), on = S(0), an = S(0), bn = S(0), sn[NI];
  const int64_t t_last = sr.len > 0 ? (sr.len - 1) / TC * TC : -1;
  const auto fetch = [&](int64_t t0) {
    qn.fetch(q, a.sq.t, t0, sr.len, a.dk);
    kn.fetch(k, a.sk.t, t0, sr.len, a.dk);
    vn = fetch_rows<IO, S>(v, a.sv.t, t0, sr.len, r0, a.dv);
    on = fetch_rows<IO, S>(dy, a.sdy.t, t0, sr.len, r0, a.dv);
    const int64_t o = go + min(t0 + static_cast<int64_t>(threadIdx.x % TC), sr.len - 1) * a.sg.t;
    an = load_gate<IO, S>(a.la, o, a.gate_io);
    bn = load_gate<IO, S>(a.be, o, a.gate_io);
    const S* c0 =
        static_cast<const S*>(a.ckpt) + (((slot0 + t0 / TC) * a.H + h) * a.dv + min(r, a.dv - 1)) * a.dk;
#pragma unroll
    for (int i = 0; i < NI; ++i) sn[i] = c0[min(col(l, i), a.dk - 1)];
  };
  if (t_last >= 0) fetch(t_last);
  for (int64_t t0 = t_last; t0 >= 0; t0 -= TC) {
    const int nt = static_cast<int>(sr.len - t0 < TC ? sr.len - t0 : TC);
    __syncthreads();
    qn.put(qs, nt, a.dk);
    kn.put(ks, nt, a.dk);
    if (threadIdx.x < TC * kRows) {
      const int t = threadIdx.x / kRows, c = threadIdx.x % kRows;
      const bool in = t < nt && r0 + c < a.dv;
      vs[threadIdx.x] = in ? vn : S(0);
      gs[threadIdx.x] = in ? scale * on : S(0);
    }
    if (threadIdx.x < TC) {
      const bool in = static_cast<int>(threadIdx.x) < nt;
      ga[threadIdx.x] = in ? gexp(an) : S(1);
      gb[threadIdx.x] = in ? bn : S(0);
    }
    S st[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) st[i] = r < a.dv && col(l, i) < a.dk ? sn[i] : S(0);
    __syncthreads();
    if (t0 > 0) fetch(t0 - TC);
    for (int t = 0; t < nt; ++t) {
      S kv[NI], p = S(0);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        kv[i] = ks[t * W + col(l, i)];
        p += st[i] * kv[i];
        hist[(t * NI + i) * kThreads + threadIdx.x] = st[i];
      }
      p = sum16(p);
      const S al = ga[t], e = vs[t * kRows + row] - al * p, u = gb[t] * e;
      if (l == 0) es[t * kRows + row] = e;
#pragma unroll
      for (int i = 0; i < NI; ++i) st[i] = al * st[i] + u * kv[i];
    }
    __syncthreads();
    for (int t = nt - 1; t >= 0; --t) {
      const S g = gs[t * kRows + row], e = es[t * kRows + row], al = ga[t], be = gb[t];
      S kv[NI], sp[NI], du = S(0), dl = S(0);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        kv[i] = ks[t * W + col(l, i)];
        A[i] += g * qs[t * W + col(l, i)];
        du += A[i] * kv[i];
        sp[i] = al * hist[(t * NI + i) * kThreads + threadIdx.x];
      }
      du = sum16(du);
      const S f = be * du, u = be * e;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const S cq = sum4rows((sp[i] + u * kv[i]) * g);
        const S ck = sum4rows(A[i] * u - sp[i] * f);
        if (lane < 16) {
          red[wave][0][col(l, i)] = cq;
          red[wave][1][col(l, i)] = ck;
        }
        A[i] -= f * kv[i];
        dl += A[i] * sp[i];
        A[i] *= al;
      }
      dl = sum4rows(sum16(dl));
      const S db = sum4rows(du * e);
      if (lane == 0) {
        redg[wave][0] = dl;
        redg[wave][1] = db;
      }
      if (l == 0 && r < a.dv) store_from(dv, (t0 + t) * a.sdv.t + r, f);
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * a.dk; i += kThreads) {
        const int w = i >= a.dk, c = i - w * a.dk;
        const S x = (red[0][w][c] + red[1][w][c]) + (red[2][w][c] + red[3][w][c]);
        (w ? pk : pq)[(t0 + t) * a.dk + c] = x;
      }
      if (threadIdx.x < 2) {
        const int w = threadIdx.x;
        (w ? pb : pl)[t0 + t] = (redg[0][w] + redg[1][w]) + (redg[2][w] + redg[3][w]);
      }
      __syncthreads();
    }
  }
  if (a.dstate_in && r < a.dv) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (col(l, i) < a.dk) static_cast<S*>(a.dstate_in)[so + col(l, i)] = A[i];
  }
}

// dq, dk (sums over the tiles and the value heads of a key head) and the gate
// gradients (sums over the tiles), in a fixed order; zeros where no value head
// reads the keys.
template <typename IO, typename S>
__global__ __launch_bounds__(kThreads) void delta_serial_sum(DeltaArgs a) {
  const int tiles = (a.dv + kRows - 1) / kRows;
  const int64_t tok = a.B * a.T, per = static_cast<int64_t>(a.Hk) * tok;
  const int grp = a.H / a.Hk;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < 2 * per * a.dk;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int w = i >= per * a.dk;
    const int64_t j = i - w * per * a.dk;
    const int c = static_cast<int>(j % a.dk);
    const int64_t bt = j / a.dk % tok;
    const int hk = static_cast<int>(j / a.dk / tok);
    const S* p = static_cast<const S*>(w ? a.part_dk : a.part_dq);
    S x = S(0);
    for (int g = 0; g < grp; ++g)
      for (int t = 0; t < tiles; ++t)
        x += p[((static_cast<int64_t>(t) * a.H + hk * grp + g) * tok + bt) * a.dk + c];
    const Str3& st = w ? a.sdk : a.sdq;
    const int64_t o = bt / a.T * st.b + hk * st.h + bt % a.T * st.t + c;
    store_from(static_cast<IO*>(w ? a.dk_ : a.dq), o, x);
  }
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < 2 * a.H * tok;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int w = i >= a.H * tok;
    const int64_t j = i - w * a.H * tok, bt = j % tok;
    const int h = static_cast<int>(j / tok);
    const S* p = static_cast<const S*>(w ? a.part_be : a.part_la);
    S x = S(0);
    for (int t = 0; t < tiles; ++t) x += p[(static_cast<int64_t>(t) * a.H + h) * tok + bt];
    const int64_t o = bt / a.T * a.sdg.b + h * a.sdg.h + bt % a.T * a.sdg.t;
    void* out = w ? a.dbe : a.dla;
    if (a.gate_io) store_from(static_cast<IO*>(out), o, x);
    else static_cast<S*>(out)[o] = x;
  }
}

// ---- one token: the state read and written once.  Bound by that traffic
// (64 KB each way per head of 128 x 128); L lanes to a row (four columns
// each), RU row sets in flight per wave.  256 rows of 16 heads of 128 x 128: 540 MB
// in 105 us with other states at each call, 5.1 TB/s (a large copy: 5.2), 93 on the
// same ones again; one row: 4.5 us, a launch.
template <int L>
__device__ __forceinline__ float sum_l(float x) {
  x = sum16(x);
  if constexpr (L == 32) {
    float a = x, b = x;
    permlane16_swap(a, b);
    x = a + b;
  }
  return x;
}
template <int L>
__device__ __forceinline__ double sum_l(double x) {
#pragma unroll
  for (int m = L / 2; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}
template <typename S>
struct alignas(16) Vec4 {
  S v[4];
};

template <typename IO, typename S, int L, int RU, bool VEC>
__global__ __launch_bounds__(kThreads) void delta_step(DeltaArgs a) {
  constexpr int RW = 64 / L, RB = RW * RU * (kThreads / 64);
  const int tiles = (a.dv + RB - 1) / RB;
  const int64_t id = blockIdx.x;
  const int h = static_cast<int>(id / tiles % a.H);
  const int64_t b = id / tiles / a.H;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int hk = h / (a.H / a.Hk), c = (lane % L) * 4;
  const int r0 = static_cast<int>(id % tiles) * RB + wave * RW * RU + lane / L;
  const int64_t slot = a.slots ? a.slots[b] : b;
  IO* y = static_cast<IO*>(a.y) + b * a.sy.b + h * a.sy.h;
  if (slot < 0 || slot >= a.n_slots) {
#pragma unroll
    for (int u = 0; u < RU; ++u)
      if (lane % L == 0 && r0 + u * RW < a.dv) store_from(y, r0 + u * RW, S(0));
    return;
  }
  S* st = static_cast<S*>(a.state_out) + (slot * a.H + h) * a.dv * a.dk;
  // All loads at indices clamped into their rows: under conditions each would be
  // waited for before the next
  S x[RU][4], qv[4], kv[4], vv[RU], kq = S(0);
  const IO* q = static_cast<const IO*>(a.q) + b * a.sq.b + hk * a.sq.h;
  const IO* k = static_cast<const IO*>(a.k) + b * a.sk.b + hk * a.sk.h;
  const IO* v = static_cast<const IO*>(a.v) + b * a.sv.b + h * a.sv.h;
#pragma unroll
  for (int u = 0; u < RU; ++u) {
    const S* row = st + static_cast<int64_t>(min(r0 + u * RW, a.dv - 1)) * a.dk;
    if constexpr (VEC) {
      const Vec4<S> t = *reinterpret_cast<const Vec4<S>*>(row + min(c, a.dk - 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = t.v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = row[min(c + i, a.dk - 1)];
    }
    vv[u] = load_as<S>(v, min(r0 + u * RW, a.dv - 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    qv[i] = load_as<S>(q, min(c + i, a.dk - 1));
    kv[i] = load_as<S>(k, min(c + i, a.dk - 1));
  }
  const int64_t go = b * a.sg.b + h * a.sg.h;
  const S la = load_gate<IO, S>(a.la, go, a.gate_io), be = load_gate<IO, S>(a.be, go, a.gate_io), al = gexp(la);
  // columns past dk are zero
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = c + i < a.dk;
    qv[i] = in ? qv[i] : S(0);
    kv[i] = in ? kv[i] : S(0);
#pragma unroll
    for (int u = 0; u < RU; ++u) x[u][i] = in ? x[u][i] : S(0);
    kq += qv[i] * kv[i];
  }
  kq = sum_l<L>(kq);
#pragma unroll
  for (int u = 0; u < RU; ++u) {
    S p = S(0), z = S(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p += x[u][i] * kv[i];
      z += x[u][i] * qv[i];
    }
    p = sum_l<L>(p);
    z = sum_l<L>(z);
    const S w = be * (vv[u] - al * p);
    const int64_t o = static_cast<int64_t>(r0 + u * RW) * a.dk + c;
    const bool in = r0 + u * RW < a.dv;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[u][i] = al * x[u][i] + w * kv[i];
    if constexpr (VEC) {
      Vec4<S> t;
#pragma unroll
      for (int i = 0; i < 4; ++i) t.v[i] = x[u][i];
      if (in && c < a.dk) *reinterpret_cast<Vec4<S>*>(st + o) = t;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (in && c + i < a.dk) st[o + i] = x[u][i];
    }
    if (in && lane % L == 0)
      store_from(y, r0 + u * RW, static_cast<S>(a.scale) * (al * z + w * kq));
  }
}

template <typename IO, typename S, int L, bool VEC>
hipError_t step_ru(const DeltaArgs& a, hipStream_t s) {
  // Two / four / eight row sets a wave at 16 heads of 128 x 128, the same states at
  // each call: 1 row 4.3 / 4.6 /
  // 5.2 us, 32 rows 14.5 / 12.5 / 12.6, 256 rows 97 / 97 / 100; of 64 x 64, 256
  // rows 26 / 24 / 27
  constexpr int RU = 4, RB = 64 / L * RU * (kThreads / 64);
  const int64_t grid = a.B * a.H * ((a.dv + RB - 1) / RB);
  delta_step<IO, S, L, RU, VEC><<<dim3(static_cast<unsigned>(grid)), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename IO, typename S>
hipError_t step_io(const DeltaArgs& a, hipStream_t s) {
  const bool vec = a.dk % 4 == 0;
  if (a.dk <= 64) return vec ? step_ru<IO, S, 16, true>(a, s) : step_ru<IO, S, 16, false>(a, s);
  return vec ? step_ru<IO, S, 32, true>(a, s) : step_ru<IO, S, 32, false>(a, s);
}

template <typename IO, typename S>
hipError_t fwd_io(const DeltaArgs& a, hipStream_t s) {
  const int64_t g = a.N * a.H * ((a.dv + kRows - 1) / kRows);
  if (g == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(g));
  if (a.dk <= 64) delta_serial_fwd<IO, S, 4><<<grid, kThreads, 0, s>>>(a);
  else delta_serial_fwd<IO, S, 8><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename IO, typename S>
hipError_t bwd_io(const DeltaArgs& a, hipStream_t s) {
  const int64_t g = a.N * a.H * ((a.dv + kRows - 1) / kRows);
  if (g > 0) {
    const dim3 grid(static_cast<unsigned>(g));
    if (a.dk <= 64) delta_serial_bwd<IO, S, 4><<<grid, kThreads, 0, s>>>(a);
    else delta_serial_bwd<IO, S, 8><<<grid, kThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.B * a.T * a.Hk == 0) return hipSuccess;
  const int64_t work = 2 * a.B * a.T * std::max<int64_t>(static_cast<int64_t>(a.Hk) * a.dk, a.H);
  const int64_t blocks = std::min<int64_t>((work + kThreads - 1) / kThreads, 8192);
  delta_serial_sum<IO, S><<<dim3(static_cast<unsigned>(blocks)), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_serial_fwd(int io, const DeltaArgs& a, hipStream_t s) {
  if (io == IO_F64) return fwd_io<double, double>(a, s);
  if (io == IO_F32) return fwd_io<float, float>(a, s);
  return fwd_io<bf16, float>(a, s);
}
hipError_t launch_delta_serial_bwd(int io, const DeltaArgs& a, hipStream_t s) {
  if (io == IO_F64) return bwd_io<double, double>(a, s);
  if (io == IO_F32) return bwd_io<float, float>(a, s);
  return bwd_io<bf16, float>(a, s);
}
hipError_t launch_delta_step(int io, const DeltaArgs& a, hipStream_t s) {
  if (io == IO_F64) return step_io<double, double>(a, s);
  if (io == IO_F32) return step_io<float, float>(a, s);
  return step_io<bf16, float>(a, s);
}

}  // namespace gls
