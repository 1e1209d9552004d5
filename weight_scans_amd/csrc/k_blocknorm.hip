// k_blocknorm.hip -- the norms around a block: the residual norm (norm of what the
// block gives, scale, sum with the residual, norm for the next block) and the
// gated norm of every head's row, with their gradients (any io dtype, d <= 16384).
//
//   hat(v) = v r(v),  r(v) = 1 / sqrt(mean(v^2) + eps);  for the gradient g of hat(v):
//   dv = r (g - hat mean(g hat))
//
// Bound by memory: each row is read and written once.  TPR threads share a row,
// a thread with E elements of it in registers: vectors of 16 bytes, TPR of them
// side by side (single elements where rows do not begin on 16 bytes).  Sums over
// a row cross lanes by shuffles and, from 128 threads on, waves through LDS.  The
// backward's work-groups walk rows with the sums for the weights in registers and
// leave one part each, the next row's loads in flight.  4 x 4096 rows of
// 2048 in bf16 on an fp32 residual: forward 73 us, 5.5 TB/s, backward 131 us, 4.6 TB/s; gated, 16
// heads of 128: forward 50 us, 4.0 TB/s, backward 85 us, 3.9 TB/s.
//
// The backwards of long rows spill and are slower for it.  1024 threads a row leave a
// thread 128 registers for the residual norm's ten arrays of elements: from 8193 columns
// on (vectors) it spills 254 to 308, the gated norm 148 (bf16) and 226 (fp32); single
// elements from 2049 on 71 and 21, from 8193 on 241 to 259 and 138.  512 threads
// with 16 elements each (vectors of 4097 to 8192) spill 16 to 76 in the residual norm; fp64
// spills from 2049 columns on, its forwards 8 to 23 from 8193 on.  In fp32, residual / gated norm, backward:
//   8192 rows of 2047:   83 us, 4.8 TB/s /  74 us, 4.5 TB/s
//   4096 rows of 4095:  325 us, 1.2      / 146 us, 2.3
//   4096 rows of 4096:   83 us, 4.9      /  72 us, 4.7
//   2048 rows of 8192:  191 us, 2.1      /  77 us, 4.4
//   1024 rows of 16384: 372 us, 1.1      / 269 us, 1.2     (bf16: 278 / 175 us)
#include <algorithm>
#include <type_traits>

#include "ssm_dev.hpp"

namespace gls {
namespace {

// A thread's E elements of a row of d: vectors (VEC) or single ones at a stride.
template <typename S, int TPR, int E, bool VEC>
struct Slice {
  template <typename IO>
  __device__ static __forceinline__ int col(int j, int e) {
    if constexpr (VEC) return (e / Vec<IO>::n * TPR + j) * Vec<IO>::n + e % Vec<IO>::n;
    else return e * TPR + j;
  }
  // Elements past the row are `fill`.  Q sets the order of columns (the io dtype,
  // also for tensors of another type, so that elements of one register belong together).
  template <typename Q, typename IO>
  __device__ static __forceinline__ void ld(const IO* p, int j, int d, S (&v)[E], S fill = S(0)) {
    if constexpr (VEC) {
      constexpr int n = Vec<Q>::n, m = Vec<IO>::n;
#pragma unroll
      for (int e = 0; e < E; e += n) {
        const int c = col<Q>(j, e);
        if (c < d) {
#pragma unroll
          for (int k = 0; k < n; k += m) Vec<IO>::ld(p + c + k, v + e + k);
        } else {
#pragma unroll
          for (int k = 0; k < n; ++k) v[e + k] = fill;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = e * TPR + j;
        v[e] = c < d ? load_as<S>(p, c) : fill;
      }
    }
  }
  template <typename Q, typename IO>
  __device__ static __forceinline__ void st(IO* p, int j, int d, const S (&v)[E]) {
    if constexpr (VEC) {
      constexpr int n = Vec<Q>::n, m = Vec<IO>::n;
#pragma unroll
      for (int e = 0; e < E; e += n) {
        const int c = col<Q>(j, e);
        if (c < d) {
#pragma unroll
          for (int k = 0; k < n; k += m) Vec<IO>::st(p + c + k, v + e + k);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e * TPR + j < d) put(p + e * TPR + j, v[e]);
    }
  }
};

// A thread's elements of a row as they lie in memory: asked for while another row is
// computed (Q: as above).
template <typename S, int TPR, int E, bool VEC, typename Q, typename IO>
struct RawSlice {
  static constexpr int m = Vec<IO>::n;
  typename std::conditional<VEC, u32x4, IO>::type v[VEC ? E / m : E];
  __device__ __forceinline__ void ask(const IO* p, int j, int d) {
    if constexpr (VEC) {
#pragma unroll
      for (int e = 0; e < E; e += m) {
        const int c = Slice<S, TPR, E, VEC>::template col<Q>(j, e / Vec<Q>::n * Vec<Q>::n) + e % Vec<Q>::n;
        v[e / m] = *reinterpret_cast<const u32x4*>(p + (c < d ? c : 0));
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = p[e * TPR + j < d ? e * TPR + j : 0];
    }
  }
  __device__ __forceinline__ void get(int j, int d, S (&x)[E]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int e = 0; e < E; e += m) {
        Vec<IO>::ld(reinterpret_cast<const IO*>(&v[e / m]), x + e);
        const bool in = Slice<S, TPR, E, VEC>::template col<Q>(j, e / Vec<Q>::n * Vec<Q>::n) < d;
#pragma unroll
        for (int k = 0; k < m; ++k) x[e + k] = in ? x[e + k] : S(0);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = e * TPR + j < d ? load_as<S>(&v[e], 0) : S(0);
    }
  }
};

// Sum over the TPR threads of a row; every thread of the work-group calls it the
// same number of times.  `turn` alternates between two sets of places, so that one
// barrier a sum is enough.
template <typename S, int TPR, int THREADS, int M>
__device__ __forceinline__ void row_sum(S (&x)[M], int& turn) {
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int m = (TPR < 64 ? TPR : 64) / 2; m >= 1; m >>= 1) x[i] += __shfl_xor(x[i], m, 64);
  if constexpr (TPR > 64) {
    constexpr int WV = TPR / 64;
    __shared__ S at[2][THREADS / 64][M];
    const int wave = threadIdx.x / 64, first = wave / WV * WV;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < M; ++i) at[turn][wave][i] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
      x[i] = S(0);
#pragma unroll
      for (int w = 0; w < WV; ++w) x[i] += at[turn][first + w][i];
    }
    turn ^= 1;
  }
}

template <typename IO>
__device__ __forceinline__ const IO* row_in(const void* p, const Rows& s, int64_t b, int64_t t, int64_t g = 0) {
  return static_cast<const IO*>(p) + b * s.b + t * s.t + g * s.g;
}
template <typename IO>
__device__ __forceinline__ IO* row_out(void* p, const Rows& s, int64_t b, int64_t t, int64_t g = 0) {
  return static_cast<IO*>(p) + b * s.b + t * s.t + g * s.g;
}

// ---------------------------------------------------------------- residual norm
template <typename IO, typename RES, typename S, int TPR, int E, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void addnorm_fwd(AddNormArgs a) {
  using L = Slice<S, TPR, E, VEC>;
  constexpr int R = THREADS / TPR;
  const int j = threadIdx.x % TPR;
  const int64_t rows = a.B * a.T;
  const int64_t want = blockIdx.x * static_cast<int64_t>(R) + threadIdx.x / TPR;
  const int64_t row = want < rows ? want : rows - 1;  // spare threads sum with the others
  const int64_t b = row / a.T, t = row % a.T;
  int turn = 0;
  S x[E], r[E], c[E];
  L::template ld<IO>(row_in<IO>(a.x, a.sx, b, t), j, a.d, x);
  L::template ld<IO>(row_in<RES>(a.r, a.sr, b, t), j, a.d, r);
  if (a.wx) {
    S ss[1] = {S(0)};
#pragma unroll
    for (int e = 0; e < E; ++e) ss[0] = fma_(x[e], x[e], ss[0]);
    row_sum<S, TPR, THREADS, 1>(ss, turn);
    const S rx = S(1) / sqrt_(ss[0] / a.d + static_cast<S>(a.eps));
    L::template ld<IO>(static_cast<const IO*>(a.wx), j, a.d, c);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= rx * c[e];
  }
  if (a.scale) {
    L::template ld<IO>(static_cast<const IO*>(a.scale), j, a.d, c);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= c[e];
  }
  S ss[1] = {S(0)};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    r[e] += x[e];
    ss[0] = fma_(r[e], r[e], ss[0]);
  }
  row_sum<S, TPR, THREADS, 1>(ss, turn);
  if (want >= rows) return;
  L::template st<IO>(row_out<RES>(a.r_out, a.sro, b, t), j, a.d, r);
  const S rr = S(1) / sqrt_(ss[0] / a.d + static_cast<S>(a.eps));
  L::template ld<IO>(static_cast<const IO*>(a.w), j, a.d, c);
#pragma unroll
  for (int e = 0; e < E; ++e) r[e] *= rr * c[e];
  L::template st<IO>(row_out<IO>(a.n, a.sn, b, t), j, a.d, r);
}

// Sums of a work-group's rows for the weights: its R rows of threads meet in LDS.
template <typename IO, typename PAR, typename S, int TPR, int E, bool VEC, int R>
__device__ __forceinline__ void leave_part(PAR* part, int d, const S (&v)[E]) {
  using L = Slice<S, TPR, E, VEC>;
  const int j = threadIdx.x % TPR, q = threadIdx.x / TPR;
  if constexpr (R == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = L::template col<IO>(j, e);
      if (c < d) part[c] = static_cast<PAR>(v[e]);
    }
  } else {
    __shared__ S red[R][TPR * E];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) red[q][L::template col<IO>(j, e)] = v[e];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += TPR * R) {
      S s = S(0);
#pragma unroll
      for (int i = 0; i < R; ++i) s += red[i][c];
      part[c] = static_cast<PAR>(s);
    }
  }
}

template <typename IO, typename RES, typename PAR, typename S, int TPR, int E, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void addnorm_bwd(AddNormArgs a) {
  using L = Slice<S, TPR, E, VEC>;
  constexpr int R = THREADS / TPR;
  const int j = threadIdx.x % TPR;
  const int64_t rows = a.B * a.T;
  int turn = 0;
  S w[E], wx[E], sc[E], dw[E], dwx[E], ds[E];
  L::template ld<IO>(static_cast<const IO*>(a.w), j, a.d, w);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    wx[e] = sc[e] = S(1);
    dw[e] = dwx[e] = ds[e] = S(0);
  }
  if (a.wx) L::template ld<IO>(static_cast<const IO*>(a.wx), j, a.d, wx);
  if (a.scale) L::template ld<IO>(static_cast<const IO*>(a.scale), j, a.d, sc);
  const S inv = S(1) / a.d, eps = static_cast<S>(a.eps);
  const int64_t step = gridDim.x * static_cast<int64_t>(R);
  RawSlice<S, TPR, E, VEC, IO, IO> nx, ng;
  RawSlice<S, TPR, E, VEC, IO, RES> nr, no;
  const auto ask = [&](int64_t base) {
    const int64_t want = base + threadIdx.x / TPR, row = want < rows ? want : rows - 1, b = row / a.T, t = row % a.T;
    nx.ask(row_in<IO>(a.x, a.sx, b, t), j, a.d);
    nr.ask(row_in<RES>(a.r, a.sr, b, t), j, a.d);
    ng.ask(row_in<IO>(a.dn, a.sdn, b, t), j, a.d);
    if (a.dro) no.ask(row_in<RES>(a.dro, a.sdro, b, t), j, a.d);
  };
  // (only of vectors: single elements take too many registers to wait in)
  if (VEC && blockIdx.x * static_cast<int64_t>(R) < rows) ask(blockIdx.x * static_cast<int64_t>(R));
  for (int64_t base = blockIdx.x * static_cast<int64_t>(R); base < rows; base += step) {
    const int64_t want = base + threadIdx.x / TPR;
    const bool in = want < rows;
    const int64_t row = in ? want : rows - 1;
    const int64_t b = row / a.T, t = row % a.T;
    S x[E], r[E], g[E], go[E];
    if (!VEC) ask(base);
    nx.get(j, a.d, x);
    nr.get(j, a.d, r);
    ng.get(j, a.d, g);
    if (a.dro) {
      no.get(j, a.d, go);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) go[e] = S(0);
    }
    if (VEC && base + step < rows) ask(base + step);
    S rx = S(1);
    if (a.wx) {
      S ss[1] = {S(0)};
#pragma unroll
      for (int e = 0; e < E; ++e) ss[0] = fma_(x[e], x[e], ss[0]);
      row_sum<S, TPR, THREADS, 1>(ss, turn);
      rx = S(1) / sqrt_(ss[0] * inv + eps);
    }
    S two[2] = {S(0), S(0)};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] *= rx;  // hat(x), or x
      r[e] = fma_(sc[e], wx[e] * x[e], r[e]);
      two[0] = fma_(r[e], r[e], two[0]);
      two[1] = fma_(w[e] * g[e], r[e], two[1]);
    }
    row_sum<S, TPR, THREADS, 2>(two, turn);
    const S rr = S(1) / sqrt_(two[0] * inv + eps);
    const S m = two[1] * rr * rr * inv;
    S dot[1] = {S(0)};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const S dr = fma_(rr, w[e] * g[e] - r[e] * m, go[e]);
      if (in) {
        dw[e] = fma_(g[e], r[e] * rr, dw[e]);
        ds[e] = fma_(dr, wx[e] * x[e], ds[e]);
        dwx[e] = fma_(dr * sc[e], x[e], dwx[e]);
      }
      r[e] = dr;
      g[e] = dr * sc[e] * wx[e];
      dot[0] = fma_(g[e], x[e], dot[0]);
    }
    if (in) L::template st<IO>(row_out<RES>(a.dr, a.sdr, b, t), j, a.d, r);
    if (a.wx) {
      row_sum<S, TPR, THREADS, 1>(dot, turn);
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = rx * (g[e] - x[e] * (dot[0] * inv));
    }
    if (in) L::template st<IO>(row_out<IO>(a.dx, a.sdx, b, t), j, a.d, g);
  }
  const int64_t plane = static_cast<int64_t>(gridDim.x) * a.d;
  PAR* part = static_cast<PAR*>(a.part) + blockIdx.x * static_cast<int64_t>(a.d);
  if (a.dw[0]) leave_part<IO, PAR, S, TPR, E, VEC, R>(part, a.d, dw);
  if (a.dw[1]) leave_part<IO, PAR, S, TPR, E, VEC, R>(part + plane, a.d, dwx);
  if (a.dw[2]) leave_part<IO, PAR, S, TPR, E, VEC, R>(part + 2 * plane, a.d, ds);
}

// ---------------------------------------------------------------- gated norm
template <typename S>
__device__ __forceinline__ S silu_(S z) { return z * sigmoid_(z); }

template <typename IO, typename S, int TPR, int E, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void gatenorm_fwd(GateNormArgs a) {
  using L = Slice<S, TPR, E, VEC>;
  constexpr int R = THREADS / TPR;
  const int j = threadIdx.x % TPR;
  const int64_t rows = a.B * a.T * a.G;
  const int64_t want = blockIdx.x * static_cast<int64_t>(R) + threadIdx.x / TPR;
  const int64_t row = want < rows ? want : rows - 1;
  const int64_t gr = row % a.G, bt = row / a.G, b = bt / a.T, t = bt % a.T;
  int turn = 0;
  S x[E], z[E], w[E];
  L::template ld<IO>(row_in<IO>(a.x, a.sx, b, t, gr), j, a.d, x);
  if (a.z) {
    L::template ld<IO>(row_in<IO>(a.z, a.sz, b, t, gr), j, a.d, z);
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] = silu_(z[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] = S(1);
  }
  S ss[1] = {S(0)};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (a.first) {
      x[e] *= z[e];
      z[e] = S(1);
    }
    ss[0] = fma_(x[e], x[e], ss[0]);
  }
  row_sum<S, TPR, THREADS, 1>(ss, turn);
  if (want >= rows) return;
  const S rr = S(1) / sqrt_(ss[0] / a.d + static_cast<S>(a.eps));
  if (a.w) {
    L::template ld<IO>(static_cast<const IO*>(a.w) + (a.group_w ? gr * a.d : 0), j, a.d, w);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = S(1);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] *= rr * w[e] * z[e];
  L::template st<IO>(row_out<IO>(a.y, a.sy, b, t, gr), j, a.d, x);
}

// Rows of the work-groups blockIdx.y: all rows, or (weights of each group) the
// rows of that group.
template <typename IO, typename PAR, typename S, int TPR, int E, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS) void gatenorm_bwd(GateNormArgs a) {
  using L = Slice<S, TPR, E, VEC>;
  constexpr int R = THREADS / TPR;
  const int j = threadIdx.x % TPR;
  const int64_t rows = a.B * a.T * (a.group_w ? 1 : a.G);
  int turn = 0;
  S w[E], dw[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    w[e] = S(1);
    dw[e] = S(0);
  }
  if (a.w) L::template ld<IO>(static_cast<const IO*>(a.w) + (a.group_w ? blockIdx.y * static_cast<int64_t>(a.d) : 0), j, a.d, w);
  const S inv = S(1) / a.d, eps = static_cast<S>(a.eps);
  const int64_t step = gridDim.x * static_cast<int64_t>(R);
  RawSlice<S, TPR, E, VEC, IO, IO> nx, nz, ng;
  const auto ask = [&](int64_t base) {
    const int64_t want = base + threadIdx.x / TPR, row = want < rows ? want : rows - 1;
    const int64_t gr = a.group_w ? blockIdx.y : row % a.G, bt = a.group_w ? row : row / a.G, b = bt / a.T, t = bt % a.T;
    nx.ask(row_in<IO>(a.x, a.sx, b, t, gr), j, a.d);
    ng.ask(row_in<IO>(a.dy, a.sdy, b, t, gr), j, a.d);
    if (a.z) nz.ask(row_in<IO>(a.z, a.sz, b, t, gr), j, a.d);
  };
  // (only of vectors: single elements take too many registers to wait in)
  if (VEC && blockIdx.x * static_cast<int64_t>(R) < rows) ask(blockIdx.x * static_cast<int64_t>(R));
  for (int64_t base = blockIdx.x * static_cast<int64_t>(R); base < rows; base += step) {
    const int64_t want = base + threadIdx.x / TPR;
    const bool in = want < rows;
    const int64_t row = in ? want : rows - 1;
    const int64_t gr = a.group_w ? blockIdx.y : row % a.G, bt = a.group_w ? row : row / a.G;
    const int64_t b = bt / a.T, t = bt % a.T;
    S x[E], z[E], g[E], gate[E], slope[E];
    if (!VEC) ask(base);
    nx.get(j, a.d, x);
    ng.get(j, a.d, g);
    if (a.z) nz.get(j, a.d, z);
    if (VEC && base + step < rows) ask(base + step);
    if (a.z) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const S q = sigmoid_(z[e]);
        gate[e] = z[e] * q;
        slope[e] = q * (S(1) + z[e] * (S(1) - q));
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        gate[e] = S(1);
        slope[e] = S(0);
      }
    }
    // v = what is normed, and dy as it reaches w hat(v)
    S two[2] = {S(0), S(0)};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const S v = a.first ? x[e] * gate[e] : x[e], u = a.first ? g[e] : g[e] * gate[e];
      two[0] = fma_(v, v, two[0]);
      two[1] = fma_(w[e] * u, v, two[1]);
    }
    row_sum<S, TPR, THREADS, 2>(two, turn);
    const S rr = S(1) / sqrt_(two[0] * inv + eps);
    const S m = two[1] * rr * rr * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const S v = a.first ? x[e] * gate[e] : x[e], u = a.first ? g[e] : g[e] * gate[e];
      const S dv = rr * (w[e] * u - v * m);
      if (in) dw[e] = fma_(u, v * rr, dw[e]);
      z[e] = slope[e] * (a.first ? dv * x[e] : g[e] * w[e] * (x[e] * rr));
      x[e] = a.first ? dv * gate[e] : dv;
    }
    if (!in) continue;
    L::template st<IO>(row_out<IO>(a.dx, a.sdx, b, t, gr), j, a.d, x);
    if (a.z) L::template st<IO>(row_out<IO>(a.dz, a.sdz, b, t, gr), j, a.d, z);
  }
  if (a.dw)
    leave_part<IO, PAR, S, TPR, E, VEC, R>(
        static_cast<PAR*>(a.part) + (blockIdx.x * static_cast<int64_t>(gridDim.y) + blockIdx.y) * a.d, a.d, dw);
}

bool addnorm_vec(int io, const AddNormArgs& a, bool bwd) {
  // vectors are of the io dtype; a residual of twice its size takes two each
  const int v = vec_of(io);
  const int res = a.res_f32 ? IO_F32 : io;
  bool ok = a.d % v == 0 && aligned16(a.x) && aligned16(io, a.sx) && aligned16(a.r) && aligned16(res, a.sr) &&
            aligned16(a.w) && aligned16(a.wx) && aligned16(a.scale);
  if (!bwd) return ok && aligned16(a.n) && aligned16(io, a.sn) && aligned16(a.r_out) && aligned16(res, a.sro);
  return ok && aligned16(a.dn) && aligned16(io, a.sdn) && aligned16(a.dro) && aligned16(res, a.sdro) && aligned16(a.dx) &&
         aligned16(io, a.sdx) && aligned16(a.dr) && aligned16(res, a.sdr);
}
bool gatenorm_vec(int io, const GateNormArgs& a, bool bwd) {
  bool ok = a.d % vec_of(io) == 0 && aligned16(a.x) && aligned16(io, a.sx) && aligned16(a.z) && aligned16(io, a.sz) &&
            aligned16(a.w);
  if (!bwd) return ok && aligned16(a.y) && aligned16(io, a.sy);
  return ok && aligned16(a.dy) && aligned16(io, a.sdy) && aligned16(a.dx) && aligned16(io, a.sdx) && aligned16(a.dz) &&
         aligned16(io, a.sdz);
}

// Threads a row: the fewest that hold it with eight elements each (from 8192 on with
// sixteen); of the kernels for single elements only every other size.  Rows of fewer than eight elements
// are computed in fp64: w dz - hat mean(w dz hat) all but cancels in some of them (for
// d = 1 it is eps / (x^2 + eps) of its first term).
template <template <typename, int, int, bool, int> class Do, typename S, typename... A>
hipError_t by_width(int d, bool vec, A... args) {
  if (d < 8) return Do<double, 16, 1, false, 256>::go(args...);
  if (vec) {
    if (d <= 64) return Do<S, 8, 8, true, 256>::go(args...);
    if (d <= 128) return Do<S, 16, 8, true, 256>::go(args...);
    if (d <= 256) return Do<S, 32, 8, true, 256>::go(args...);
    if (d <= 512) return Do<S, 64, 8, true, 256>::go(args...);
    if (d <= 1024) return Do<S, 128, 8, true, 256>::go(args...);
    if (d <= 2048) return Do<S, 256, 8, true, 256>::go(args...);
    if (d <= 4096) return Do<S, 512, 8, true, 512>::go(args...);
    if (d <= 8192) return Do<S, 512, 16, true, 512>::go(args...);
    return Do<S, 1024, 16, true, 1024>::go(args...);
  }
  if (d <= 128) return Do<S, 16, 8, false, 256>::go(args...);
  if (d <= 512) return Do<S, 64, 8, false, 256>::go(args...);
  if (d <= 2048) return Do<S, 256, 8, false, 256>::go(args...);
  if (d <= 8192) return Do<S, 1024, 8, false, 1024>::go(args...);
  return Do<S, 1024, 16, false, 1024>::go(args...);
}
// (of the vector kernels; the others may take fewer, and leave some parts at zero)
int rows_at_once(int d) {
  int q = 32;
  while (q > 1 && d * q > 2048) q /= 2;
  return q;
}

// Work-groups (parts of the sums) of the backwards: as many as the CUs hold at once, by
// their registers; more only wait and leave more parts (4 x 4096 rows of 2048, residual in
// fp32 / bf16: 512 parts 126 / 94 us, 1024 147 / 109; gated 512 101, 1024 82; 4 x 1024 rows
// of 8192: 512 parts 212 us, 1024 264).
int64_t addnorm_most(int d) { return d <= 2048 ? 512 : 256; }
int64_t gatenorm_most(int d) { return d <= 2048 ? 1024 : 512; }

template <typename IO, typename RES, typename PAR>
struct Add {
  template <typename S, int TPR, int E, bool VEC, int TH>
  struct Fwd {
    static hipError_t go(const AddNormArgs& a, hipStream_t s) {
      const int64_t g = (a.B * a.T + TH / TPR - 1) / (TH / TPR);
      if (!launch_fits(g * TH)) return hipErrorInvalidConfiguration;
      addnorm_fwd<IO, RES, S, TPR, E, VEC, TH><<<static_cast<unsigned>(g), TH, 0, s>>>(a);
      return hipGetLastError();
    }
  };
  template <typename S, int TPR, int E, bool VEC, int TH>
  struct Bwd {
    static hipError_t go(const AddNormArgs& a, hipStream_t s) {
      addnorm_bwd<IO, RES, PAR, S, TPR, E, VEC, TH><<<static_cast<unsigned>(addnorm_parts(a)), TH, 0, s>>>(a);
      return hipGetLastError();
    }
  };
};
template <typename IO, typename PAR>
struct Gate {
  template <typename S, int TPR, int E, bool VEC, int TH>
  struct Fwd {
    static hipError_t go(const GateNormArgs& a, hipStream_t s) {
      const int64_t g = (a.B * a.T * a.G + TH / TPR - 1) / (TH / TPR);
      if (!launch_fits(g * TH)) return hipErrorInvalidConfiguration;
      gatenorm_fwd<IO, S, TPR, E, VEC, TH><<<static_cast<unsigned>(g), TH, 0, s>>>(a);
      return hipGetLastError();
    }
  };
  template <typename S, int TPR, int E, bool VEC, int TH>
  struct Bwd {
    static hipError_t go(const GateNormArgs& a, hipStream_t s) {
      const dim3 g(static_cast<unsigned>(gatenorm_parts(a)), a.group_w ? a.G : 1);
      gatenorm_bwd<IO, PAR, S, TPR, E, VEC, TH><<<g, TH, 0, s>>>(a);
      return hipGetLastError();
    }
  };
};

template <typename IO, typename RES, typename S>
hipError_t add_fwd(int io, const AddNormArgs& a, hipStream_t s) {
  return by_width<Add<IO, RES, S>::template Fwd, S>(a.d, addnorm_vec(io, a, false), a, s);
}
template <typename IO, typename RES, typename S>
hipError_t add_bwd(int io, const AddNormArgs& a, hipStream_t s) {
  return by_width<Add<IO, RES, S>::template Bwd, S>(a.d, addnorm_vec(io, a, true), a, s);
}

}  // namespace

int64_t addnorm_parts(const AddNormArgs& a) {
  const int q = rows_at_once(a.d);
  return std::max<int64_t>(1, std::min<int64_t>((a.B * a.T + q - 1) / q, addnorm_most(a.d)));
}
int64_t gatenorm_parts(const GateNormArgs& a) {
  const int q = rows_at_once(a.d);
  const int64_t rows = a.B * a.T * (a.group_w ? 1 : a.G);
  const int64_t most = a.group_w ? std::max<int64_t>(1, gatenorm_most(a.d) / std::max(1, a.G)) : gatenorm_most(a.d);
  return std::max<int64_t>(1, std::min<int64_t>((rows + q - 1) / q, most));
}

hipError_t launch_addnorm_fwd(int io, const AddNormArgs& a, hipStream_t s) {
  if (io == IO_F64) return add_fwd<double, double, double>(io, a, s);
  if (io == IO_F32) return add_fwd<float, float, float>(io, a, s);
  if (a.res_f32) return add_fwd<bf16, float, float>(io, a, s);
  return add_fwd<bf16, bf16, float>(io, a, s);
}
hipError_t launch_addnorm_bwd(int io, const AddNormArgs& a, hipStream_t s) {
  const bool any = a.B * a.T > 0;
  hipError_t e = hipSuccess;
  if (any) {
    if (io == IO_F64) e = add_bwd<double, double, double>(io, a, s);
    else if (io == IO_F32) e = add_bwd<float, float, float>(io, a, s);
    else if (a.res_f32) e = add_bwd<bf16, float, float>(io, a, s);
    else e = add_bwd<bf16, bf16, float>(io, a, s);
  }
  if (e != hipSuccess) return e;
  const SumOut out[3] = {{a.dw[0], 1}, {a.dw[1], 1}, {a.dw[2], 1}};
  return launch_sum_rows(io, a.part, out, 3, any ? addnorm_parts(a) : 0, a.d, s);
}
hipError_t launch_gatenorm_fwd(int io, const GateNormArgs& a, hipStream_t s) {
  const bool v = gatenorm_vec(io, a, false);
  if (io == IO_F64) return by_width<Gate<double, double>::Fwd, double>(a.d, v, a, s);
  if (io == IO_F32) return by_width<Gate<float, float>::Fwd, float>(a.d, v, a, s);
  return by_width<Gate<bf16, float>::Fwd, float>(a.d, v, a, s);
}
hipError_t launch_gatenorm_bwd(int io, const GateNormArgs& a, hipStream_t s) {
  const bool v = gatenorm_vec(io, a, true), any = a.B * a.T * a.G > 0;
  const int64_t cols = static_cast<int64_t>(a.d) * (a.group_w ? a.G : 1);
  if (a.dw && !sums_fit(cols)) return hipErrorInvalidConfiguration;
  hipError_t e = hipSuccess;
  if (any) {
    if (io == IO_F64) e = by_width<Gate<double, double>::Bwd, double>(a.d, v, a, s);
    else if (io == IO_F32) e = by_width<Gate<float, float>::Bwd, float>(a.d, v, a, s);
    else e = by_width<Gate<bf16, float>::Bwd, float>(a.d, v, a, s);
  }
  if (e != hipSuccess) return e;
  const SumOut out[1] = {{a.dw, 1}};
  return launch_sum_rows(io, a.part, out, 1, any ? gatenorm_parts(a) : 0, cols, s);
}

}  // namespace gls
