// k_conv.hip -- short causal convolution per channel with its bias and SiLU, its
// backward and its form for single tokens (any io dtype, 1 <= K <= 8).
//
// A token is read and written once.  A thread owns 16 bytes of
// neighbouring channels (one element where rows do not begin on 16 bytes) and a
// run of tokens, with the last K - 1 inputs in registers; neighbouring threads
// own neighbouring channels.  The inputs before a run are read again by it, in
// the backward also what its last inputs reach behind it.
//
// The forward is bound by memory: 4 x 4096 tokens of 2048 channels in bf16, K = 4: 30 us,
// 4.5 TB/s.  A small one is bound by what a thread does in series before its first tokens
// arrive (taps, the table's search, the inputs before its run): packed 3001 tokens of 1001
// channels in fp32, K = 3, 10.1 us; without a table 9.2, rows of 1000 in vectors 9.8, eight
// times the tokens 43 us, 4.5 TB/s.
// The backward is bound by the vector ALU: 56 us at the first of these sizes, 3.6 TB/s.
// Two waves a SIMD (forty sums for the weights' gradients a thread) keep it busy 82 % of the
// time, with 39 instructions an element, some 25 of them arithmetic: two runs share a wave,
// so that tokens, bounds and addresses are computed lane by lane.
#include <algorithm>

#include "ssm_dev.hpp"

namespace gls {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;   // tokens whose loads are in flight together
constexpr int kBack = 4;    // the same in the backward, which holds more
constexpr int kAnyK = 8;    // taps of the kernels for any K: the first 8 - K are not there

// W elements as they lie in memory.
template <typename IO, int W>
struct Raw {
  uint4 v;
  __device__ __forceinline__ void get(const IO* p) { v = *reinterpret_cast<const uint4*>(p); }
  template <typename S>
  __device__ __forceinline__ void to(S (&x)[W]) const { Vec<IO>::ld(reinterpret_cast<const IO*>(&v), x); }
};
template <typename IO>
struct Raw<IO, 1> {
  IO v;
  __device__ __forceinline__ void get(const IO* p) { v = *p; }
  template <typename S>
  __device__ __forceinline__ void to(S (&x)[1]) const { x[0] = load_as<S>(&v, 0); }
};

// Sequence of token t on the packed axis: the last whose first token is <= t among
// those that the table puts in order (any table: a number in 0..n-1).
__device__ __forceinline__ int64_t seq_of(const int32_t* cu, int64_t n, int64_t t) {
  int64_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int64_t m = (lo + hi + 1) / 2;
    if (cu[m] <= t) lo = m;
    else hi = m - 1;
  }
  return lo;
}

template <typename IO, typename S, int KT, int W>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int d, S (&w)[KT][W], S (&b)[W]) {
  const IO* pw = static_cast<const IO*>(a.w) + static_cast<int64_t>(d) * a.K;
  if constexpr (KT < kAnyK) {  // the W x KT weights follow one another
    S flat[KT * W];
#pragma unroll
    for (int i = 0; i < KT; ++i) load_w<IO, S, W>(pw + i * W, flat + i * W);
#pragma unroll
    for (int e = 0; e < W; ++e)
#pragma unroll
      for (int j = 0; j < KT; ++j) w[j][e] = flat[e * KT + j];
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e)
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        const int u = j - (KT - a.K);
        w[j][e] = u >= 0 ? load_as<S>(pw, e * a.K + u) : S(0);
      }
  }
  if (a.bias) {
    load_w<IO, S, W>(static_cast<const IO*>(a.bias) + d, b);
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) b[e] = S(0);
  }
}

// Tap j is there (a tap that is not multiplies nothing: 0 times infinity is no 0).
template <int KT>
__device__ __forceinline__ bool tap(const ConvArgs& a, int j) { return KT < kAnyK || j >= KT - a.K; }

// Input number t of sequence n at channel d, from the state for the K - 1 numbers
// before 0, else zero.
template <typename IO, typename S, int W>
__device__ __forceinline__ void load_x(const ConvArgs& a, const SeqRange& r, int64_t n, int64_t t, int d, S (&v)[W]) {
  if (t >= 0) {
    load_w<IO, S, W>(static_cast<const IO*>(a.x) + r.b * a.sx.b + (r.t0 + t) * a.sx.t + d, v);
  } else if (a.state_in && t >= 1 - a.K) {
    load_w<IO, S, W>(static_cast<const IO*>(a.state_in) + (n * (a.K - 1) + t + a.K - 1) * a.D + d, v);
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = S(0);
  }
}

template <typename S>
__device__ __forceinline__ S act(bool silu, S p) { return silu ? p * sigmoid_(p) : p; }
template <typename S>
__device__ __forceinline__ S dact(bool silu, S p) {
  if (!silu) return S(1);
  const S g = sigmoid_(p);
  return g * (S(1) + p * (S(1) - g));
}

template <typename S, int KT, int W>
__device__ __forceinline__ void convolve(const ConvArgs& a, const S (&w)[KT][W], const S (&b)[W], const S (&x)[KT][W],
                                         S (&p)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) {
    p[e] = b[e];
#pragma unroll
    for (int j = 0; j < KT; ++j) p[e] = tap<KT>(a, j) ? fma_(w[j][e], x[j][e], p[e]) : p[e];
  }
}

template <typename S, int KT, int W>
__device__ __forceinline__ void move_on(S (&x)[KT][W]) {
#pragma unroll
  for (int j = 0; j < KT - 1; ++j)
#pragma unroll
    for (int e = 0; e < W; ++e) x[j][e] = x[j + 1][e];
}

// Thread -> channels and a run of L tokens of the B * T; behind the runs, the
// K - 1 last inputs of each sequence.
template <typename IO, typename S, int KT, int W>
__global__ __launch_bounds__(kThreads) void conv_fwd(ConvArgs a, int L, int64_t runs_b, int64_t n_runs) {
  const int nv = a.D / W;
  const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
  const int d = static_cast<int>(i % nv) * W;
  const int64_t run = i / nv;
  if (run >= n_runs) {
    const int64_t u = run - n_runs;
    if (!a.state_out || u >= a.N * (a.K - 1)) return;
    const int64_t n = u / (a.K - 1);
    const SeqRange r = seq_range(a.cu, n, a.T);
    S v[W];
    load_x<IO, S, W>(a, r, n, r.len + u % (a.K - 1) - (a.K - 1), d, v);
    store_w<IO, S, W>(static_cast<IO*>(a.state_out) + u * a.D + d, v);
    return;
  }
  const int64_t b = run / runs_b, lo = run % runs_b * L, hi = lo + L < a.T ? lo + L : a.T;
  S w[KT][W], bias[W], x[KT][W];
  load_taps<IO, S, KT, W>(a, d, w, bias);
  int64_t n = b;
  SeqRange r{b, 0, a.T};
  if (a.n_seq) {
    n = seq_of(a.cu, a.n_seq, lo);
    r = seq_range(a.cu, n, a.T);
  }
#pragma unroll
  for (int j = 0; j < KT - 1; ++j) load_x<IO, S, W>(a, r, n, lo - r.t0 + j - (KT - 1), d, x[j]);
  IO* y = static_cast<IO*>(a.y) + b * a.sy.b + d;
  const IO* px = static_cast<const IO*>(a.x) + b * a.sx.b + d;
  for (int64_t t0 = lo; t0 < hi; t0 += kAhead) {
    Raw<IO, W> raw[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) raw[k].get(px + (t0 + k < hi ? t0 + k : hi - 1) * a.sx.t);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t t = t0 + k;
      if (t < hi) {
        if (a.n_seq && t >= r.t0 + r.len && n + 1 < a.n_seq) {  // the next sequence that has a token
          while (t >= r.t0 + r.len && n + 1 < a.n_seq) r = seq_range(a.cu, ++n, a.T);
#pragma unroll
          for (int j = 0; j < KT - 1; ++j) load_x<IO, S, W>(a, r, n, t - r.t0 + j - (KT - 1), d, x[j]);
        }
        raw[k].to(x[KT - 1]);
        S p[W];
        convolve<S, KT, W>(a, w, bias, x, p);
        const bool none = a.n_seq && t >= r.t0 + r.len;  // behind the last sequence
#pragma unroll
        for (int e = 0; e < W; ++e) p[e] = none ? S(0) : act(a.silu, p[e]);
        store_w<IO, S, W>(y + t * a.sy.t, p);
        move_on<S, KT, W>(x);
      }
    }
  }
}

// Gradients of a run: with p formed again, dp = dy silu'(p) reaches the inputs of
// its K - 1 tokens before and its own; a run goes on for the K - 1 tokens behind
// it, so that its own inputs get all of theirs.  acc[i] is of token t - (KT - 1) + i.
// The sums for the weights meet in LDS over the work-group's runs and leave as
// one part [K + 1][D] per row of work-groups.
constexpr int kChLanes = 32, kRunLanes = kThreads / kChLanes;
template <typename IO, typename S, int KT, int W>
__global__ __launch_bounds__(kThreads) void conv_bwd(ConvArgs a, int L, int64_t runs_b, int64_t n_runs) {
  __shared__ S red[kRunLanes][kChLanes * W];
  const int cl = threadIdx.x % kChLanes, rl = threadIdx.x / kChLanes;
  const int dv = (blockIdx.x * kChLanes + cl) * W;
  const bool in = dv < a.D;
  const int d = in ? dv : 0;
  S w[KT][W], bias[W], x[KT][W], acc[KT][W], dw[KT][W], db[W];
  load_taps<IO, S, KT, W>(a, d, w, bias);
#pragma unroll
  for (int e = 0; e < W; ++e) {
    db[e] = S(0);
#pragma unroll
    for (int j = 0; j < KT; ++j) dw[j][e] = S(0);
  }
  int64_t last = a.T;  // the end of the last sequence: what is behind it adds nothing
  if (a.n_seq) {
    const SeqRange r = seq_range(a.cu, a.n_seq - 1, a.T);
    last = r.t0 + r.len;
  }
  for (int64_t run = blockIdx.y * static_cast<int64_t>(kRunLanes) + rl; in && run < n_runs;
       run += gridDim.y * static_cast<int64_t>(kRunLanes)) {
    const int64_t b = run / runs_b, lo = run % runs_b * L, hi = lo + L < a.T ? lo + L : a.T;
    const int64_t end = hi + KT - 1 < last ? hi + KT - 1 : last;
    int64_t n = b;
    SeqRange r{b, 0, a.T};
    if (a.n_seq) {
      n = seq_of(a.cu, a.n_seq, lo);
      r = seq_range(a.cu, n, a.T);
    }
#pragma unroll
    for (int j = 0; j < KT - 1; ++j) load_x<IO, S, W>(a, r, n, lo - r.t0 + j - (KT - 1), d, x[j]);
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int e = 0; e < W; ++e) acc[j][e] = S(0);
    const IO* px = static_cast<const IO*>(a.x) + b * a.sx.b + d;
    const IO* pg = static_cast<const IO*>(a.dy) + b * a.sdy.b + d;
    IO* po = static_cast<IO*>(a.dx) + b * a.sdx.b + d;
    for (int64_t t0 = lo; t0 < hi + KT - 1; t0 += kBack) {
      Raw<IO, W> rx[kBack], rg[kBack];
#pragma unroll
      for (int k = 0; k < kBack; ++k) {
        const int64_t t = t0 + k < end ? t0 + k : end > lo ? end - 1 : lo;
        rx[k].get(px + t * a.sx.t);
        rg[k].get(pg + t * a.sdy.t);
      }
#pragma unroll
      for (int k = 0; k < kBack; ++k) {
        const int64_t t = t0 + k;
        if (t >= hi + KT - 1) continue;
        if (t < end) {
          if (a.n_seq && t >= r.t0 + r.len && n + 1 < a.n_seq) {
            while (t >= r.t0 + r.len && n + 1 < a.n_seq) r = seq_range(a.cu, ++n, a.T);
#pragma unroll
            for (int j = 0; j < KT - 1; ++j) load_x<IO, S, W>(a, r, n, t - r.t0 + j - (KT - 1), d, x[j]);
          }
          rx[k].to(x[KT - 1]);
          S p[W], g[W];
          rg[k].to(g);
          convolve<S, KT, W>(a, w, bias, x, p);
#pragma unroll
          for (int e = 0; e < W; ++e) g[e] *= dact(a.silu, p[e]);
          const int64_t kept = t - r.t0 - (r.len - (a.K - 1));  // its number among the inputs kept
          if (a.dstate_out && kept >= 0 && kept < a.K - 1) {
            load_w<IO, S, W>(static_cast<const IO*>(a.dstate_out) + (n * (a.K - 1) + kept) * a.D + d, acc[KT - 1]);
          } else {
#pragma unroll
            for (int e = 0; e < W; ++e) acc[KT - 1][e] = S(0);
          }
          if (KT < kAnyK && t - (KT - 1) >= r.t0) {  // all taps read inputs of this sequence
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
              for (int e = 0; e < W; ++e) acc[j][e] = fma_(w[j][e], g[e], acc[j][e]);
          } else {
#pragma unroll
            for (int j = 0; j < KT; ++j) {
              const bool own = tap<KT>(a, j) && t - (KT - 1 - j) >= r.t0;
#pragma unroll
              for (int e = 0; e < W; ++e) acc[j][e] = own ? fma_(w[j][e], g[e], acc[j][e]) : acc[j][e];
            }
          }
          if (t < hi) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
              db[e] += g[e];
#pragma unroll
              for (int j = 0; j < KT; ++j) dw[j][e] = fma_(g[e], x[j][e], dw[j][e]);
            }
          }
          move_on<S, KT, W>(x);
        }
        const int64_t done = t - (KT - 1);
        if (done >= lo && done < hi) {
          if (done >= last) {
#pragma unroll
            for (int e = 0; e < W; ++e) acc[0][e] = S(0);
          }
          store_w<IO, S, W>(po + done * a.sdx.t, acc[0]);
        }
        move_on<S, KT, W>(acc);
      }
    }
  }
  if (!a.part) return;
  S* part = static_cast<S*>(a.part) + blockIdx.y * static_cast<int64_t>(a.D);
  const int64_t plane = static_cast<int64_t>(gridDim.y) * a.D;
#pragma unroll
  for (int j = 0; j <= KT; ++j) {
    if (j < KT && !tap<KT>(a, j)) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < W; ++e) red[rl][cl * W + e] = j < KT ? dw[j < KT ? j : 0][e] : db[e];
    __syncthreads();
    for (int c = threadIdx.x; c < kChLanes * W; c += kThreads) {
      const int col = blockIdx.x * kChLanes * W + c;
      S s = S(0);
#pragma unroll
      for (int q = 0; q < kRunLanes; ++q) s += red[q][c];
      if (col < a.D) part[(j - (KT - a.K)) * plane + col] = s;
    }
  }
}

// Gradient of the first state: its i-th input (of K - 1) is seen by the tokens
// t <= i with weight i - t; sequences of fewer than K - 1 tokens keep inputs of it.
template <typename IO, typename S>
__global__ __launch_bounds__(kThreads) void conv_bwd_state(ConvArgs a) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
  const int K = a.K, d = static_cast<int>(i % a.D);
  const int64_t u = i / a.D;
  if (u >= a.N * (K - 1)) return;
  const int64_t n = u / (K - 1), at = u % (K - 1);
  const SeqRange r = seq_range(a.cu, n, a.T);
  const IO* pw = static_cast<const IO*>(a.w) + static_cast<int64_t>(d) * K;
  S sum = S(0);
  if (a.dstate_out && at >= r.len)
    sum = load_as<S>(static_cast<const IO*>(a.dstate_out), (n * (K - 1) + at - r.len) * a.D + d);
  for (int64_t t = 0; t <= at && t < r.len; ++t) {
    S p = a.bias ? load_as<S>(static_cast<const IO*>(a.bias), d) : S(0), x[1];
    for (int j = 0; j < K; ++j) {
      load_x<IO, S, 1>(a, r, n, t - (K - 1) + j, d, x);
      p = fma_(load_as<S>(pw, j), x[0], p);
    }
    const S g = load_as<S>(static_cast<const IO*>(a.dy) + r.b * a.sdy.b + (r.t0 + t) * a.sdy.t, d);
    sum = fma_(load_as<S>(pw, at - t), g * dact(a.silu, p), sum);
  }
  store_from(static_cast<IO*>(a.dstate_in), u * a.D + d, sum);
}

template <typename IO, typename S, int KT, int W>
__global__ __launch_bounds__(kThreads) void conv_step(ConvArgs a) {
  const int nv = a.D / W;
  const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
  const int d = static_cast<int>(i % nv) * W;
  const int64_t b = i / nv;
  if (b >= a.B) return;
  const int64_t slot = a.slots ? a.slots[b] : b;
  IO* y = static_cast<IO*>(a.y) + b * a.sy.b + d;
  S w[KT][W], p[W], x[KT][W];
  if (slot < 0 || slot >= a.n_slots) {
#pragma unroll
    for (int e = 0; e < W; ++e) p[e] = S(0);
    store_w<IO, S, W>(y, p);
    return;
  }
  IO* st = static_cast<IO*>(a.state_out) + slot * (a.K - 1) * a.D + d;
  load_w<IO, S, W>(static_cast<const IO*>(a.x) + b * a.sx.b + d, x[KT - 1]);
#pragma unroll
  for (int j = 0; j < KT - 1; ++j) {
    const int u = j - (KT - a.K);
    if (tap<KT>(a, j)) {
      load_w<IO, S, W>(st + static_cast<int64_t>(u) * a.D, x[j]);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) x[j][e] = S(0);
    }
  }
  S bias[W];
  load_taps<IO, S, KT, W>(a, d, w, bias);
  convolve<S, KT, W>(a, w, bias, x, p);
#pragma unroll
  for (int e = 0; e < W; ++e) p[e] = act(a.silu, p[e]);
  store_w<IO, S, W>(y, p);
#pragma unroll
  for (int j = 0; j < KT - 1; ++j) {
    const int u = j - (KT - a.K);
    if (tap<KT>(a, j)) store_w<IO, S, W>(st + static_cast<int64_t>(u) * a.D, x[j + 1]);
  }
}

bool vector_ok(int io, const ConvArgs& a, bool bwd) {
  const int v = vec_of(io);
  bool ok = a.D % v == 0 && aligned16(a.x) && aligned16(a.w) && aligned16(a.bias) && aligned16(io, a.sx) &&
            aligned16(a.state_in) && aligned16(a.state_out);
  if (!bwd) return ok && aligned16(a.y) && aligned16(io, a.sy);
  return ok && aligned16(a.dy) && aligned16(io, a.sdy) && aligned16(a.dx) && aligned16(io, a.sdx) &&
         aligned16(a.dstate_out);
}

// Tokens a run: as many as leave the chip's 256 CUs 1024 threads each.
int run_tokens(int64_t items, int most) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, items / (256 * 1024))));
}

template <typename IO, typename S, int KT, int W>
hipError_t fwd_k(const ConvArgs& a, hipStream_t s) {
  const int64_t nv = a.D / W;
  const int L = run_tokens(a.B * a.T * nv, 16);
  const int64_t runs_b = (a.T + L - 1) / L, runs = a.B * runs_b;
  const int64_t items = (runs + (a.state_out ? a.N * (a.K - 1) : 0)) * nv;
  if (items == 0) return hipSuccess;
  if (!launch_fits(items)) return hipErrorInvalidConfiguration;
  conv_fwd<IO, S, KT, W><<<static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, L, runs_b, runs);
  return hipGetLastError();
}
template <typename IO, typename S, int KT, int W>
hipError_t step_k(const ConvArgs& a, hipStream_t s) {
  const int64_t items = a.B * (a.D / W);
  if (!launch_fits(items)) return hipErrorInvalidConfiguration;
  conv_step<IO, S, KT, W><<<static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

// Tokens a run of the backward, which reads the K - 1 tokens behind it once more: 32, and
// where there are few tokens less, for more threads: 3 x 88 tokens of 512 channels take 43 us
// with 32 (forward and backward), 29 with 8.
int bwd_run(int64_t items) { return std::max(8, run_tokens(2 * items, 32)); }
constexpr int64_t kBwdParts = 128;
template <typename IO, typename S, int KT, int W>
hipError_t bwd_k(const ConvArgs& a, int64_t parts, hipStream_t s) {
  const int L = bwd_run(a.B * a.T * (a.D / 8 + 1));
  const int64_t runs_b = (a.T + L - 1) / L;
  const dim3 grid(static_cast<unsigned>((a.D / W + kChLanes - 1) / kChLanes), static_cast<unsigned>(parts));
  conv_bwd<IO, S, KT, W><<<grid, kThreads, 0, s>>>(a, L, runs_b, a.B * runs_b);
  return hipGetLastError();
}
int64_t bwd_parts(const ConvArgs& a) {
  const int L = bwd_run(a.B * a.T * (a.D / 8 + 1));
  const int64_t runs = a.B * ((a.T + L - 1) / L);
  return std::max<int64_t>(1, std::min((runs + kRunLanes - 1) / kRunLanes, kBwdParts));
}

enum { FWD, BWD, STEP };
template <int WHAT, typename IO, typename S, int KT, int W>
hipError_t run_k(const ConvArgs& a, hipStream_t s) {
  if constexpr (WHAT == FWD) return fwd_k<IO, S, KT, W>(a, s);
  else if constexpr (WHAT == BWD) return bwd_k<IO, S, KT, W>(a, bwd_parts(a), s);
  else return step_k<IO, S, KT, W>(a, s);
}
template <int WHAT, typename IO, typename S, int W>
hipError_t run_w(const ConvArgs& a, hipStream_t s) {
  switch (a.K) {
    case 2: return run_k<WHAT, IO, S, 2, W>(a, s);
    case 3: return run_k<WHAT, IO, S, 3, W>(a, s);
    case 4: return run_k<WHAT, IO, S, 4, W>(a, s);
    default: return run_k<WHAT, IO, S, kAnyK, W>(a, s);
  }
}
template <int WHAT, typename IO, typename S>
hipError_t run_io(int io, const ConvArgs& a, hipStream_t s) {
  return vector_ok(io, a, WHAT == BWD) ? run_w<WHAT, IO, S, Vec<IO>::n>(a, s) : run_w<WHAT, IO, S, 1>(a, s);
}
template <int WHAT>
hipError_t run(int io, const ConvArgs& a, hipStream_t s) {
  if (io == IO_F64) return run_io<WHAT, double, double>(io, a, s);
  if (io == IO_F32) return run_io<WHAT, float, float>(io, a, s);
  return run_io<WHAT, bf16, float>(io, a, s);
}

}  // namespace

size_t conv_bwd_ws(int io, const ConvArgs& a) {
  return static_cast<size_t>(bwd_parts(a)) * (a.K + 1) * a.D * (io == IO_F64 ? 8 : 4);
}
hipError_t launch_conv_fwd(int io, const ConvArgs& a, hipStream_t s) { return run<FWD>(io, a, s); }
hipError_t launch_conv_step(int io, const ConvArgs& a, hipStream_t s) { return run<STEP>(io, a, s); }

hipError_t launch_conv_bwd(int io, const ConvArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  const size_t par = io == IO_F64 ? 8 : 4;
  const int64_t items = a.dstate_in ? a.N * (a.K - 1) * a.D : 0;
  if (!launch_fits(items)) return hipErrorInvalidConfiguration;
  if (a.B * a.T > 0) {
    if ((e = run<BWD>(io, a, s)) != hipSuccess) return e;
  }
  if (a.part) {
    SumOut out[kMaxSums] = {};
    const int64_t rows = a.B * a.T > 0 ? bwd_parts(a) : 0;
    for (int j = 0; j < a.K; ++j)
      out[j] = {a.dw ? static_cast<char*>(a.dw) + j * par : nullptr, a.K};
    out[a.K] = {a.dbias, 1};
    if ((e = launch_sum_rows(io, a.part, out, a.K + 1, rows, a.D, s)) != hipSuccess) return e;
  }
  if (items == 0) return e;
  const unsigned g = static_cast<unsigned>((items + kThreads - 1) / kThreads);
  if (io == IO_F64) conv_bwd_state<double, double><<<g, kThreads, 0, s>>>(a);
  else if (io == IO_F32) conv_bwd_state<float, float><<<g, kThreads, 0, s>>>(a);
  else conv_bwd_state<bf16, float><<<g, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace gls
