// k_qknorm.hip -- norms of queries and keys per head with the position rotation
// in the same pass, and its backward (any io dtype, 1 <= d <= 256).
//
//   n = x r,  r = 1 / sqrt(mean(x^2) + eps),  out = scale Rot_p(w * n)
//   dz = scale Rot_p^T(dout);  dw = sum_rows dz * n;
//   dx = r (w dz - n mean(w dz * n))
//
// Bound by reading and writing each row once: 4 x 4096 tokens of 16 + 8 heads of
// 128, bf16, forward 201 MB in 43 us (4.7 TB/s), backward 302 MB in 72 us (4.2 TB/s)
// and 4 us for the sums of dw; a large copy reaches 5.2.  Vector kernels (d and rot
// multiples of 16): a lane owns 16 columns of a row as two runs of eight that
// hold whole pairs (run j and the run rot/2 further on, or two neighbouring
// runs), so that the rotation needs no other lane; d/16 lanes (rounded up to a
// power of two) share a row and meet only in its sum of squares.  Such a group
// takes one token and walks its heads: cosines and sines (as many bytes as a
// bf16 row has) are loaded once per token and stay in registers, and so do the
// weights.  Sums for dw stay in registers over the walk, meet in LDS, and
// leave as one part per work-group, added in a fixed order.  Other even sizes
// take half a wave per row and go pair by pair of elements; odd and short rows
// one wave with the row in LDS.
#include <algorithm>

#include "delta.hpp"
#include "dev_common.hpp"

namespace gls {
namespace {

constexpr int kThreads = 256;

template <typename IO>
struct Run8;  // eight consecutive elements, 16-byte aligned
template <>
struct Run8<bf16> {
  template <typename S>
  __device__ static void ld(const bf16* p, S (&v)[8]) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(static_cast<uint16_t>(w[i] & 0xffffu));
      v[2 * i + 1] = bf16_to_f32(static_cast<uint16_t>(w[i] >> 16));
    }
  }
  template <typename S>
  __device__ static void st(bf16* p, const S (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Run8<float> {
  template <typename S>
  __device__ static void ld(const float* p, S (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  template <typename S>
  __device__ static void st(float* p, const S (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <>
struct Run8<double> {
  __device__ static void ld(const double* p, double (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double2 t = reinterpret_cast<const double2*>(p)[i];
      v[2 * i] = t.x;
      v[2 * i + 1] = t.y;
    }
  }
  __device__ static void st(double* p, const double (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<double2*>(p)[i] = make_double2(v[2 * i], v[2 * i + 1]);
  }
};

__device__ __forceinline__ float root(float x) { return sqrtf(x); }
__device__ __forceinline__ double root(double x) { return sqrt(x); }

template <typename S, int L>
__device__ __forceinline__ S sum_group(S x) {
#pragma unroll
  for (int m = L / 2; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// Work-groups (and parts of the dw sums) that the backward gives to q and to k: in
// the ratio of their heads, so that both end together (16 and 8 heads: 75 -> 71 us).
// 1024 for the larger: 1365 78 us, 2048 78, 4096 85.
__host__ __device__ __forceinline__ int64_t parts_of(const QkArgs& a, int which) {
  const int most = a.Hn[0] > a.Hn[1] ? a.Hn[0] : a.Hn[1];
  return most ? (a.n_part * a.Hn[which] + most - 1) / most : 1;
}

// Where a lane's two runs of eight begin, and its angles.
template <typename S>
struct Turn {
  S c[8], s[8];  // half-split: pair i of the two runs; neighbours: pairs 0..3 of run 0, 4..7 of run 1
  bool on, next;
  __device__ void fwd(S (&a)[8], S (&b)[8]) const {
    if (!on) return;
    if (!next) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const S u = a[i] * c[i] - b[i] * s[i], w = b[i] * c[i] + a[i] * s[i];
        a[i] = u;
        b[i] = w;
      }
    } else {
      pairs(a, 0, S(1));
      pairs(b, 4, S(1));
    }
  }
  __device__ void back(S (&a)[8], S (&b)[8]) const {
    if (!on) return;
    if (!next) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const S u = a[i] * c[i] + b[i] * s[i], w = b[i] * c[i] - a[i] * s[i];
        a[i] = u;
        b[i] = w;
      }
    } else {
      pairs(a, 0, S(-1));
      pairs(b, 4, S(-1));
    }
  }
  __device__ void pairs(S (&x)[8], int o, S sg) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const S si = sg * s[o + i];
      const S u = x[2 * i] * c[o + i] - x[2 * i + 1] * si, w = x[2 * i + 1] * c[o + i] + x[2 * i] * si;
      x[2 * i] = u;
      x[2 * i + 1] = w;
    }
  }
};

__device__ __forceinline__ int64_t position(const QkArgs& a, int64_t bt) {
  int64_t p = a.pos ? a.pos[bt] : a.pos0 + bt % a.T;
  return p < 0 ? 0 : p >= a.n_pos ? a.n_pos - 1 : p;
}

// Columns of lane j's runs: within the turned columns run j and run j + rot/16
// (half-split) or runs 2j, 2j + 1; the other columns in order.
__device__ __forceinline__ void columns(const QkArgs& a, int j, int& c0, int& c1) {
  if (!a.interleaved && j < a.rot / 16) {
    c0 = 8 * j;
    c1 = 8 * j + a.rot / 2;
  } else {
    c0 = 16 * j;
    c1 = 16 * j + 8;
  }
}

template <typename S>
__device__ __forceinline__ void load_turn(const QkArgs& a, int64_t bt, int j, Turn<S>& t) {
  t.on = 16 * j < a.rot;
  t.next = a.interleaved;
  if (!t.on) return;
  const int64_t o = position(a, bt) * (a.rot / 2) + 8 * j;
  Run8<S>::ld(static_cast<const S*>(a.cos) + o, t.c);
  Run8<S>::ld(static_cast<const S*>(a.sin) + o, t.s);
}

template <typename IO, typename S>
__device__ __forceinline__ void load_w(const void* w, int c0, int c1, S (&u)[8], S (&v)[8]) {
  if (w) {
    Run8<IO>::ld(static_cast<const IO*>(w) + c0, u);
    Run8<IO>::ld(static_cast<const IO*>(w) + c1, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[i] = S(1);
  }
}

// Group `g` of lanes: token g / parts, heads part * hpg .. of the Hq + Hk.
template <typename IO, typename S, int L>
__global__ __launch_bounds__(kThreads) void qknorm_fwd_v(QkArgs a) {
  const int64_t g = blockIdx.x * static_cast<int64_t>(kThreads / L) + threadIdx.x / L;
  const int j = threadIdx.x % L, heads = a.Hn[0] + a.Hn[1];
  const int parts = (heads + a.hpg - 1) / a.hpg;
  const int64_t bt = g / parts;
  if (bt >= a.B * a.T) return;
  const int h0 = static_cast<int>(g % parts) * a.hpg, h1 = min(heads, h0 + a.hpg);
  const bool in = 16 * j < a.d;
  int c0, c1;
  columns(a, j, c0, c1);
  const int64_t b = bt / a.T, t = bt % a.T;
  Turn<S> turn;
  turn.on = false;
  S w0[8], w1[8];
  if (in) load_turn(a, bt, j, turn);
  int had = -1;
  for (int hh = h0; hh < h1; ++hh) {
    const int which = hh >= a.Hn[0], h = hh - which * a.Hn[0];
    if (in && which != had) {
      load_w<IO, S>(a.w[which], c0, c1, w0, w1);
      had = which;
    }
    S x0[8], x1[8], ss = S(0);
    if (in) {
      const IO* x = static_cast<const IO*>(a.x[which]) + b * a.sx[which].b + h * a.sx[which].h + t * a.sx[which].t;
      Run8<IO>::ld(x + c0, x0);
      Run8<IO>::ld(x + c1, x1);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
    }
    ss = sum_group<S, L>(ss);
    if (in) {
      const S r = static_cast<S>(a.scale[which]) / root(ss / a.d + static_cast<S>(a.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x0[i] *= r * w0[i];
        x1[i] *= r * w1[i];
      }
      turn.fwd(x0, x1);
      IO* o = static_cast<IO*>(a.out[which]) + b * a.so[which].b + h * a.so[which].h + t * a.so[which].t;
      Run8<IO>::st(o + c0, x0);
      Run8<IO>::st(o + c1, x1);
    }
  }
}

// The backward's groups take tokens g, g + groups, ... with all heads of one
// of q and k (blockIdx.y), so that the dw sums of a work-group are one part.
template <typename IO, typename S, int L>
__global__ __launch_bounds__(kThreads) void qknorm_bwd_v(QkArgs a) {
  constexpr int G = kThreads / L;
  __shared__ S red[G][16 * L + 1];
  const int which = blockIdx.y, j = threadIdx.x % L, gi = threadIdx.x / L;
  const bool in = 16 * j < a.d;
  int c0, c1;
  columns(a, j, c0, c1);
  S w0[8], w1[8], d0[8], d1[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) d0[i] = d1[i] = S(0);
  if (in) load_w<IO, S>(a.w[which], c0, c1, w0, w1);
  const S scale = static_cast<S>(a.scale[which]);
  const int heads = a.Hn[which], parts = (heads + a.hpg - 1) / a.hpg;
  const int64_t units = a.B * a.T * parts, groups = parts_of(a, which);
  if (blockIdx.x >= groups) return;
  for (int64_t un = blockIdx.x * static_cast<int64_t>(G) + gi; un < units; un += groups * G) {
    const int64_t bt = un / parts;
    const int h0 = static_cast<int>(un % parts) * a.hpg, h1 = min(heads, h0 + a.hpg);
    const int64_t b = bt / a.T, t = bt % a.T;
    Turn<S> turn;
    turn.on = false;
    if (in) load_turn(a, bt, j, turn);
    for (int h = h0; h < h1; ++h) {
      S x0[8], x1[8], g0[8], g1[8], ss = S(0), dot = S(0);
      if (in) {
        const IO* x = static_cast<const IO*>(a.x[which]) + b * a.sx[which].b + h * a.sx[which].h + t * a.sx[which].t;
        const IO* dy =
            static_cast<const IO*>(a.dout[which]) + b * a.sdo[which].b + h * a.sdo[which].h + t * a.sdo[which].t;
        Run8<IO>::ld(x + c0, x0);
        Run8<IO>::ld(x + c1, x1);
        Run8<IO>::ld(dy + c0, g0);
        Run8<IO>::ld(dy + c1, g1);
        turn.back(g0, g1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g0[i] *= scale;
          g1[i] *= scale;
          ss += x0[i] * x0[i] + x1[i] * x1[i];
          dot += g0[i] * w0[i] * x0[i] + g1[i] * w1[i] * x1[i];
        }
      }
      ss = sum_group<S, L>(ss);
      dot = sum_group<S, L>(dot);
      if (in) {
        const S r = S(1) / root(ss / a.d + static_cast<S>(a.eps));
        const S m = dot * r * r / a.d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d0[i] += g0[i] * (x0[i] * r);
          d1[i] += g1[i] * (x1[i] * r);
          x0[i] = r * (w0[i] * g0[i] - x0[i] * m);
          x1[i] = r * (w1[i] * g1[i] - x1[i] * m);
        }
        IO* o = static_cast<IO*>(a.out[which]) + b * a.so[which].b + h * a.so[which].h + t * a.so[which].t;
        Run8<IO>::st(o + c0, x0);
        Run8<IO>::st(o + c1, x1);
      }
    }
  }
  if (!a.dw[which]) return;
  if (in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      red[gi][c0 + i] = d0[i];
      red[gi][c1 + i] = d1[i];
    }
  }
  __syncthreads();
  S* part = static_cast<S*>(a.part) + (static_cast<int64_t>(which) * a.n_part + blockIdx.x) * a.d;
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    S x = S(0);
    for (int g = 0; g < G; ++g) x += red[g][c];
    part[c] = x;
  }
}

// dw: the parts of the work-groups added in a fixed order.  A work-group takes
// 16 columns; its 64 rows of threads take every 64th part, eight loads in
// flight, then meet in LDS (2 x 1024 parts of 128 columns: 20 us with 16 rows
// and one load at a time).
constexpr int kDwRows = 64;
template <typename S>
__global__ __launch_bounds__(16 * kDwRows) void qknorm_dw(QkArgs a) {
  __shared__ S red[kDwRows][17];
  const int which = blockIdx.y, l = threadIdx.x & 15, w = threadIdx.x >> 4;
  if (!a.dw[which]) return;
  const int c = blockIdx.x * 16 + l, cc = min(c, a.d - 1);
  const S* part = static_cast<const S*>(a.part) + static_cast<int64_t>(which) * a.n_part * a.d + cc;
  const int n = static_cast<int>(parts_of(a, which));
  S x = S(0);
  for (int p = w; p < n; p += 8 * kDwRows) {
    S v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[static_cast<int64_t>(min(p + i * kDwRows, n - 1)) * a.d];
#pragma unroll
    for (int i = 0; i < 8; ++i) x += p + i * kDwRows < n ? v[i] : S(0);
  }
  red[w][l] = x;
  __syncthreads();
  if (w == 0 && c < a.d) {
    S y = S(0);
#pragma unroll
    for (int i = 0; i < kDwRows; ++i) y += red[i][l];
    static_cast<S*>(a.dw[which])[c] = y;
  }
}

// ---- even d of at least 32 that the vector kernels do not take (their sizes,
// strides or alignment): half a wave per row, a lane with the pairs of columns
// l, l + 32, ... that a rotation turns (those past rot: neighbours), element by
// element, so that again only the sums cross lanes.  Bound by the number of its
// loads and stores: forward and backward of 4 x 4096 tokens of 24 heads of 120,
// bf16, take 151 us (one wave a row in fp64: 621; the vector kernels at 128: 120).
constexpr int kPairLanes = 32;

template <typename S, int U>
struct Pairs {
  int c0[U], c1[U];
  bool in[U], turned[U];
  S c[U], s[U], w0[U], w1[U];
  __device__ __forceinline__ Pairs(const QkArgs& a, int l) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = l + kPairLanes * i;
      in[i] = 2 * u < a.d;
      turned[i] = 2 * u < a.rot;
      // past the row: column 0, loaded and not used (a load under a condition
      // would be waited for before the next one is issued)
      c0[i] = !in[i] ? 0 : turned[i] && !a.interleaved ? u : 2 * u;
      c1[i] = !in[i] ? 0 : turned[i] && !a.interleaved ? u + a.rot / 2 : 2 * u + 1;
      c[i] = S(1);
      s[i] = S(0);
    }
  }
  __device__ __forceinline__ void angles(const QkArgs& a, int64_t bt, int l) {
    if (!a.rot) return;
    const int half = a.rot / 2;
    const int64_t o = position(a, bt) * half;
    S cc[U], ss[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = min(l + kPairLanes * i, half - 1);
      cc[i] = static_cast<const S*>(a.cos)[o + u];
      ss[i] = static_cast<const S*>(a.sin)[o + u];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      c[i] = turned[i] ? cc[i] : S(1);
      s[i] = turned[i] ? ss[i] : S(0);
    }
  }
  template <typename IO>
  __device__ __forceinline__ void weights(const void* w) {
#pragma unroll
    for (int i = 0; i < U; ++i) w0[i] = w1[i] = S(1);
    if (!w) return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      w0[i] = load_as<S>(static_cast<const IO*>(w), c0[i]);
      w1[i] = load_as<S>(static_cast<const IO*>(w), c1[i]);
    }
  }
  template <typename IO>
  __device__ __forceinline__ void load(const IO* p, S (&u)[U], S (&v)[U]) const {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      u[i] = load_as<S>(p, c0[i]);
      v[i] = load_as<S>(p, c1[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      u[i] = in[i] ? u[i] : S(0);
      v[i] = in[i] ? v[i] : S(0);
    }
  }
  template <typename IO>
  __device__ __forceinline__ void store(IO* p, const S (&u)[U], const S (&v)[U]) const {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (in[i]) {
        store_from(p, c0[i], u[i]);
        store_from(p, c1[i], v[i]);
      }
  }
};

template <typename IO, typename S, int U>
__global__ __launch_bounds__(kThreads) void qknorm_fwd_p(QkArgs a) {
  const int64_t g = blockIdx.x * static_cast<int64_t>(kThreads / kPairLanes) + threadIdx.x / kPairLanes;
  const int l = threadIdx.x % kPairLanes, heads = a.Hn[0] + a.Hn[1];
  const int parts = (heads + a.hpg - 1) / a.hpg;
  const int64_t bt = g / parts;
  if (bt >= a.B * a.T) return;
  const int h0 = static_cast<int>(g % parts) * a.hpg, h1 = min(heads, h0 + a.hpg);
  const int64_t b = bt / a.T, t = bt % a.T;
  Pairs<S, U> p(a, l);
  p.angles(a, bt, l);
  int had = -1;
  for (int hh = h0; hh < h1; ++hh) {
    const int which = hh >= a.Hn[0], h = hh - which * a.Hn[0];
    if (which != had) p.template weights<IO>(a.w[which]);
    had = which;
    S x0[U], x1[U], ss = S(0);
    p.load(static_cast<const IO*>(a.x[which]) + b * a.sx[which].b + h * a.sx[which].h + t * a.sx[which].t, x0, x1);
#pragma unroll
    for (int i = 0; i < U; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
    const S r = static_cast<S>(a.scale[which]) / root(sum_group<S, kPairLanes>(ss) / a.d + static_cast<S>(a.eps));
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const S u = x0[i] * (r * p.w0[i]), v = x1[i] * (r * p.w1[i]);
      x0[i] = u * p.c[i] - v * p.s[i];
      x1[i] = v * p.c[i] + u * p.s[i];
    }
    p.store(static_cast<IO*>(a.out[which]) + b * a.so[which].b + h * a.so[which].h + t * a.so[which].t, x0, x1);
  }
}

template <typename IO, typename S, int U>
__global__ __launch_bounds__(kThreads) void qknorm_bwd_p(QkArgs a) {
  constexpr int G = kThreads / kPairLanes;
  __shared__ S red[G][2 * kPairLanes * U];
  const int which = blockIdx.y, l = threadIdx.x % kPairLanes, gi = threadIdx.x / kPairLanes;
  const S scale = static_cast<S>(a.scale[which]);
  const int heads = a.Hn[which], parts = (heads + a.hpg - 1) / a.hpg;
  const int64_t units = a.B * a.T * parts, groups = parts_of(a, which);
  if (blockIdx.x >= groups) return;
  Pairs<S, U> p(a, l);
  p.template weights<IO>(a.w[which]);
  S d0[U], d1[U];
#pragma unroll
  for (int i = 0; i < U; ++i) d0[i] = d1[i] = S(0);
  for (int64_t un = blockIdx.x * static_cast<int64_t>(G) + gi; un < units; un += groups * G) {
    const int64_t bt = un / parts, b = bt / a.T, t = bt % a.T;
    const int h0 = static_cast<int>(un % parts) * a.hpg, h1 = min(heads, h0 + a.hpg);
    p.angles(a, bt, l);
    for (int h = h0; h < h1; ++h) {
      S x0[U], x1[U], g0[U], g1[U], ss = S(0), dot = S(0);
      p.load(static_cast<const IO*>(a.x[which]) + b * a.sx[which].b + h * a.sx[which].h + t * a.sx[which].t, x0, x1);
      p.load(static_cast<const IO*>(a.dout[which]) + b * a.sdo[which].b + h * a.sdo[which].h + t * a.sdo[which].t, g0,
             g1);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const S u = scale * g0[i], v = scale * g1[i];
        g0[i] = u * p.c[i] + v * p.s[i];
        g1[i] = v * p.c[i] - u * p.s[i];
        ss += x0[i] * x0[i] + x1[i] * x1[i];
        dot += g0[i] * p.w0[i] * x0[i] + g1[i] * p.w1[i] * x1[i];
      }
      ss = sum_group<S, kPairLanes>(ss);
      dot = sum_group<S, kPairLanes>(dot);
      const S r = S(1) / root(ss / a.d + static_cast<S>(a.eps));
      const S m = dot * r * r / a.d;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        d0[i] += g0[i] * (x0[i] * r);
        d1[i] += g1[i] * (x1[i] * r);
        x0[i] = r * (p.w0[i] * g0[i] - x0[i] * m);
        x1[i] = r * (p.w1[i] * g1[i] - x1[i] * m);
      }
      p.store(static_cast<IO*>(a.out[which]) + b * a.so[which].b + h * a.so[which].h + t * a.so[which].t, x0, x1);
    }
  }
  if (!a.dw[which]) return;
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (p.in[i]) {
      red[gi][p.c0[i]] = d0[i];
      red[gi][p.c1[i]] = d1[i];
    }
  __syncthreads();
  S* part = static_cast<S*>(a.part) + (static_cast<int64_t>(which) * a.n_part + blockIdx.x) * a.d;
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    S x = S(0);
    for (int g = 0; g < G; ++g) x += red[g][c];
    part[c] = x;
  }
}

// ---- any size: one wave per row, the row in LDS, four columns a lane.  Odd and
// short rows are left, among them some whose gradient w dz - n mean(w dz n)
// nearly cancels (for d = 1 it is eps / (x^2 + eps) of its first term), so the
// row is computed in fp64; tables and sums keep the type S.
constexpr int kWaves = kThreads / 64, kMaxD = 256;

__device__ __forceinline__ double sum64(double x) { return sum_group<double, 64>(x); }

template <typename IO, typename S, bool BWD>
__global__ __launch_bounds__(kThreads) void qknorm_any(QkArgs a) {
  __shared__ double lds[kWaves][kMaxD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, which = blockIdx.y;
  const int heads = a.Hn[which], half = a.rot / 2;
  const int64_t rows = a.B * a.T * heads;
  const double scale = (a.scale[which]);
  double* row = lds[wave];
  double dw[4] = {0, 0, 0, 0};
  const int64_t groups = BWD ? parts_of(a, which) : gridDim.x;
  if (blockIdx.x >= groups) return;
  for (int64_t base = blockIdx.x * static_cast<int64_t>(kWaves); base < rows; base += groups * kWaves) {
    const int64_t i = base + wave;
    const bool in = i < rows;
    const int64_t bt = in ? i / heads : 0, b = bt / a.T, t = bt % a.T;
    const int h = in ? static_cast<int>(i % heads) : 0;
    const int64_t po = a.rot ? position(a, bt) * half : 0;
    const IO* x = static_cast<const IO*>(a.x[which]) + b * a.sx[which].b + h * a.sx[which].h + t * a.sx[which].t;
    IO* o = static_cast<IO*>(a.out[which]) + b * a.so[which].b + h * a.so[which].h + t * a.so[which].t;
    double v[4], ss = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = lane + 64 * u;
      v[u] = in && c < a.d ? load_as<double>(x, c) : 0.0;
      ss += v[u] * v[u];
    }
    const double r = 1.0 / root(sum64(ss) / a.d + a.eps);
    __syncthreads();
    // what is turned: w n (forward), the upstream gradient (backward)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = lane + 64 * u;
      if (c < a.d) {
        if constexpr (BWD) {
          const IO* dy = static_cast<const IO*>(a.dout[which]) + b * a.sdo[which].b + h * a.sdo[which].h +
                         t * a.sdo[which].t;
          row[c] = in ? scale * load_as<double>(dy, c) : 0.0;
        } else {
          const double w = a.w[which] ? load_as<double>(static_cast<const IO*>(a.w[which]), c) : 1.0;
          row[c] = scale * r * w * v[u];
        }
      }
    }
    __syncthreads();
    double z[4], dot = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = lane + 64 * u;
      z[u] = c < a.d ? row[c] : 0.0;
      if (c < a.rot) {
        const bool second = a.interleaved ? (c & 1) : c >= half;
        const int p = a.interleaved ? c >> 1 : c - (second ? half : 0);
        const int mate = a.interleaved ? c ^ 1 : second ? c - half : c + half;
        const double co = static_cast<const S*>(a.cos)[po + p];
        double si = static_cast<const S*>(a.sin)[po + p];
        if (BWD) si = -si;
        z[u] = second ? z[u] * co + row[mate] * si : z[u] * co - row[mate] * si;
      }
      if constexpr (BWD) {
        if (c < a.d) {
          dw[u] += z[u] * (v[u] * r);
          const double w = a.w[which] ? load_as<double>(static_cast<const IO*>(a.w[which]), c) : 1.0;
          z[u] *= w;
          dot += z[u] * v[u];
        }
      }
    }
    if constexpr (BWD) {
      const double m = sum64(dot) * r * r / a.d;
#pragma unroll
      for (int u = 0; u < 4; ++u) z[u] = r * (z[u] - v[u] * m);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (in && lane + 64 * u < a.d) store_from(o, lane + 64 * u, z[u]);
  }
  if constexpr (BWD) {
    if (!a.dw[which]) return;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) row[lane + 64 * u] = dw[u];
    __syncthreads();
    S* part = static_cast<S*>(a.part) + (static_cast<int64_t>(which) * a.n_part + blockIdx.x) * a.d;
    for (int c = threadIdx.x; c < a.d; c += kThreads) part[c] = static_cast<S>((lds[0][c] + lds[1][c]) + (lds[2][c] + lds[3][c]));
  }
}

int lanes(int d) {
  int l = 1;
  while (16 * l < d) l *= 2;
  return l;
}

// The vector kernels load runs of eight elements: pointers, strides and tables
// have to keep 16-byte alignment.
bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned(int io, const Str3& s) {
  const int m = io == IO_BF16 ? 8 : io == IO_F32 ? 4 : 2;
  return s.b % m == 0 && s.h % m == 0 && s.t % m == 0;
}
bool vector_ok(int io, const QkArgs& a, bool bwd) {
  bool ok = a.d % 16 == 0 && a.rot % 16 == 0;
  ok = ok && aligned(a.cos) && aligned(a.sin);
  for (int i = 0; i < 2; ++i)
    ok = ok && aligned(a.x[i]) && aligned(a.w[i]) && aligned(a.out[i]) && (!bwd || aligned(a.dout[i])) &&
         aligned(io, a.sx[i]) && aligned(io, a.so[i]) && (!bwd || aligned(io, a.sdo[i]));
  return ok;
}

bool pairs_ok(const QkArgs& a) { return a.d % 2 == 0 && a.d >= 32; }

// Heads per group of lanes: all of a token's, so that its angles are loaded
// once, unless that leaves the chip short of groups (256 CUs of 2048 lanes).
int heads_per_group(int64_t tokens, int heads, int L) {
  int parts = 1;
  while (parts < heads && tokens * parts * L < 256 * 2048) ++parts;
  return (heads + parts - 1) / parts;
}

constexpr int64_t kMaxParts = 1024;

template <typename IO, typename S>
hipError_t fwd_io(int io, QkArgs a, hipStream_t s) {
  const int64_t tok = a.B * a.T;
  const int heads = a.Hn[0] + a.Hn[1];
  if (tok == 0 || heads == 0) return hipSuccess;
  if (!vector_ok(io, a, false) && pairs_ok(a)) {
    a.hpg = heads_per_group(tok, heads, kPairLanes);
    const int64_t groups = tok * ((heads + a.hpg - 1) / a.hpg);
    const unsigned g = static_cast<unsigned>((groups * kPairLanes + kThreads - 1) / kThreads);
    switch ((a.d + 2 * kPairLanes - 1) / (2 * kPairLanes)) {
      case 1: qknorm_fwd_p<IO, S, 1><<<g, kThreads, 0, s>>>(a); break;
      case 2: qknorm_fwd_p<IO, S, 2><<<g, kThreads, 0, s>>>(a); break;
      case 3: qknorm_fwd_p<IO, S, 3><<<g, kThreads, 0, s>>>(a); break;
      default: qknorm_fwd_p<IO, S, 4><<<g, kThreads, 0, s>>>(a); break;
    }
    return hipGetLastError();
  }
  if (!vector_ok(io, a, false)) {
    const int64_t rows = tok * std::max(a.Hn[0], a.Hn[1]);
    const int64_t g = std::min<int64_t>((rows + kWaves - 1) / kWaves, 16384);
    qknorm_any<IO, S, false><<<dim3(static_cast<unsigned>(g), 2), kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  const int L = lanes(a.d);
  a.hpg = heads_per_group(tok, heads, L);
  const int64_t groups = tok * ((heads + a.hpg - 1) / a.hpg);
  const unsigned g = static_cast<unsigned>((groups * L + kThreads - 1) / kThreads);
  switch (L) {
    case 1: qknorm_fwd_v<IO, S, 1><<<g, kThreads, 0, s>>>(a); break;
    case 2: qknorm_fwd_v<IO, S, 2><<<g, kThreads, 0, s>>>(a); break;
    case 4: qknorm_fwd_v<IO, S, 4><<<g, kThreads, 0, s>>>(a); break;
    case 8: qknorm_fwd_v<IO, S, 8><<<g, kThreads, 0, s>>>(a); break;
    default: qknorm_fwd_v<IO, S, 16><<<g, kThreads, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

template <typename IO, typename S>
hipError_t bwd_io(int io, QkArgs a, hipStream_t s) {
  const int64_t tok = a.B * a.T;
  const bool vec = vector_ok(io, a, true), pairs = !vec && pairs_ok(a);
  const int L = pairs ? kPairLanes : lanes(a.d);
  a.hpg = heads_per_group(tok, std::max(1, std::max(a.Hn[0], a.Hn[1])), L);
  const dim3 grid(static_cast<unsigned>(a.n_part), 2);
  if (pairs) switch ((a.d + 2 * kPairLanes - 1) / (2 * kPairLanes)) {
    case 1: qknorm_bwd_p<IO, S, 1><<<grid, kThreads, 0, s>>>(a); break;
    case 2: qknorm_bwd_p<IO, S, 2><<<grid, kThreads, 0, s>>>(a); break;
    case 3: qknorm_bwd_p<IO, S, 3><<<grid, kThreads, 0, s>>>(a); break;
    default: qknorm_bwd_p<IO, S, 4><<<grid, kThreads, 0, s>>>(a); break;
  }
  else if (!vec) qknorm_any<IO, S, true><<<grid, kThreads, 0, s>>>(a);
  else switch (L) {
    case 1: qknorm_bwd_v<IO, S, 1><<<grid, kThreads, 0, s>>>(a); break;
    case 2: qknorm_bwd_v<IO, S, 2><<<grid, kThreads, 0, s>>>(a); break;
    case 4: qknorm_bwd_v<IO, S, 4><<<grid, kThreads, 0, s>>>(a); break;
    case 8: qknorm_bwd_v<IO, S, 8><<<grid, kThreads, 0, s>>>(a); break;
    default: qknorm_bwd_v<IO, S, 16><<<grid, kThreads, 0, s>>>(a); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.dw[0] && !a.dw[1])) return e;
  qknorm_dw<S><<<dim3((a.d + 15) / 16, 2), 16 * kDwRows, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t qknorm_bwd_parts(int io, const QkArgs& a) {
  (void)io;
  // rows in units of one work-group's, by the smaller of the two kernels' needs
  const int64_t rows = a.B * a.T * std::max(a.Hn[0], a.Hn[1]);
  return std::max<int64_t>(1, std::min<int64_t>((rows * lanes(a.d) + kThreads - 1) / kThreads, kMaxParts));
}
hipError_t launch_qknorm_fwd(int io, const QkArgs& a, hipStream_t s) {
  if (io == IO_F64) return fwd_io<double, double>(io, a, s);
  if (io == IO_F32) return fwd_io<float, float>(io, a, s);
  return fwd_io<bf16, float>(io, a, s);
}
hipError_t launch_qknorm_bwd(int io, const QkArgs& a, hipStream_t s) {
  if (io == IO_F64) return bwd_io<double, double>(io, a, s);
  if (io == IO_F32) return bwd_io<float, float>(io, a, s);
  return bwd_io<bf16, float>(io, a, s);
}

}  // namespace gls
