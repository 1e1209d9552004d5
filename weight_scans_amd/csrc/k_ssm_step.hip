// k_ssm_step.hip -- selective scan, one token of each row against a pool of states.
//
// Bound by reading and writing the states: 256 rows of 2048 channels and 16 states in
// 18 us, 71 MB at 3.9 TB/s; 19 us, 3.7 TB/s, under the profiler (one wave of loads and stores a
// lane; two or four rows a lane, rows in turn with the next one's loads ahead, or other
// numbers of lanes came to the same or more).  L lanes share a channel's N states (in vectors
// of 16 bytes where N allows it) and meet in y's sum.
#include <algorithm>

#include "ssm_dev.hpp"

namespace gls {
namespace {

constexpr int kThreads = 256;

// Group of L lanes -> row b and channel d.
template <typename IO, typename S, int L, int W>
__global__ __launch_bounds__(kThreads) void ssm_step(SsmArgs a) {
  const int64_t i = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) / L;
  const int l = threadIdx.x % L, d = static_cast<int>(i % a.D);
  const int64_t b = i / a.D;
  if (b >= a.B) return;
  const int64_t slot = a.slots ? a.slots[b] : b;
  IO* y = static_cast<IO*>(a.y) + b * a.sy.b;
  if (slot < 0 || slot >= a.n_slots) {
    if (l == 0) store_from(y, d, S(0));
    return;
  }
  S* st = static_cast<S*>(a.state_out) + (slot * a.D + d) * a.Ns;
  const S* A = static_cast<const S*>(a.A) + static_cast<int64_t>(d) * a.Ns;
  const int g = d / (a.D / a.G);
  const IO* B = static_cast<const IO*>(a.Bm) + b * a.sB.b + g * a.sB.g;
  const IO* C = static_cast<const IO*>(a.Cm) + b * a.sC.b + g * a.sC.g;
  const S x = load_as<S>(static_cast<const IO*>(a.x) + b * a.sx.b, d);
  S D = load_as<S>(static_cast<const IO*>(a.dt) + b * a.sdt.b, d);
  const S z = a.z ? load_as<S>(static_cast<const IO*>(a.z) + b * a.sz.b, d) : S(0);
  const S skip = a.skip ? static_cast<const S*>(a.skip)[d] : S(0);
  if (a.bias) D += static_cast<const S*>(a.bias)[d];
  if (a.softplus) D = softplus_(D);
  const S u = D * x, D2 = D * static_cast<S>(kLog2e);
  S sum = S(0);
  for (int n = l * W; n < a.Ns; n += L * W) {
    S h[W], A_[W];
    if constexpr (W == 1) {
      h[0] = st[n];
      A_[0] = A[n];
    } else {
      Vec<S>::ld(st + n, h);
      Vec<S>::ld(A + n, A_);
    }
#pragma unroll
    for (int e = 0; e < W; ++e) {
      h[e] = fma_(exp2_(D2 * A_[e]), h[e], u * load_as<S>(B, n + e));
      sum = fma_(load_as<S>(C, n + e), h[e], sum);
    }
    if constexpr (W == 1) st[n] = h[0];
    else Vec<S>::st(st + n, h);
  }
#pragma unroll
  for (int m = L / 2; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, 64);
  if (l) return;
  sum = fma_(skip, x, sum);
  if (a.z) sum *= z * sigmoid_(z);
  store_from(y, d, sum);
}

template <typename IO, typename S, int L, int W>
hipError_t go(const SsmArgs& a, hipStream_t s) {
  const int64_t n = a.B * a.D * L;
  if (!launch_fits(n)) return hipErrorInvalidConfiguration;
  ssm_step<IO, S, L, W><<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
  return hipGetLastError();
}
template <typename IO, typename S, int W>
hipError_t by_lanes(const SsmArgs& a, hipStream_t s) {
  const int v = (a.Ns + W - 1) / W;
  if (v <= 1) return go<IO, S, 1, W>(a, s);
  if (v <= 2) return go<IO, S, 2, W>(a, s);
  if (v <= 4) return go<IO, S, 4, W>(a, s);
  if (v <= 8) return go<IO, S, 8, W>(a, s);
  return go<IO, S, 16, W>(a, s);
}
template <typename IO, typename S>
hipError_t by_vec(const SsmArgs& a, hipStream_t s) {
  constexpr int W = Vec<S>::n;
  if (a.Ns % W == 0 && aligned16(a.state_out) && aligned16(a.A)) return by_lanes<IO, S, W>(a, s);
  return by_lanes<IO, S, 1>(a, s);
}

}  // namespace

hipError_t launch_ssm_step(int io, const SsmArgs& a, hipStream_t s) {
  if (a.B * a.D == 0) return hipSuccess;
  if (io == IO_F64) return by_vec<double, double>(a, s);
  if (io == IO_F32) return by_vec<float, float>(a, s);
  return by_vec<bf16, float>(a, s);
}

}  // namespace gls
