// k_ssm_sum.hip -- sums over the rows that work-groups leave of gradients of
// weights, in a fixed order: 5 to 7 us for the up to 1024 rows of 2048 columns that the norms
// leave, bound by the latency of its few loads in series.
#include "ssm_dev.hpp"

namespace gls {
namespace {

constexpr int kCols = kSumCols, kRows = kSumRows;

struct Outs {
  SumOut o[kMaxSums];
};

// A work-group takes 64 columns; its 16 rows of threads take every 16th row, eight
// loads in flight, then meet in LDS.
template <typename S>
__global__ __launch_bounds__(kCols * kRows) void sum_rows(const S* part, Outs outs, int64_t rows, int64_t cols) {
  __shared__ S red[kRows][kCols + 1];
  const SumOut o = outs.o[blockIdx.y];
  if (!o.p) return;
  const int l = threadIdx.x % kCols, w = threadIdx.x / kCols;
  const int64_t c = blockIdx.x * static_cast<int64_t>(kCols) + l, cc = c < cols ? c : cols - 1;
  const S* p = part + blockIdx.y * rows * cols + cc;
  S x = S(0);
  for (int64_t r = w; r < rows; r += 8 * kRows) {
    S v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[(r + i * kRows < rows ? r + i * kRows : rows - 1) * cols];
#pragma unroll
    for (int i = 0; i < 8; ++i) x += r + i * kRows < rows ? v[i] : S(0);
  }
  red[w][l] = x;
  __syncthreads();
  if (w == 0 && c < cols) {
    S y = S(0);
#pragma unroll
    for (int i = 0; i < kRows; ++i) y += red[i][l];
    static_cast<S*>(o.p)[c * o.stride] = y;
  }
}

}  // namespace

hipError_t launch_sum_rows(int io, const void* part, const SumOut* out, int nz, int64_t rows, int64_t cols,
                           hipStream_t s) {
  Outs o{};
  bool any = false;
  for (int i = 0; i < nz; ++i) {
    o.o[i] = out[i];
    any = any || out[i].p;
  }
  if (!any || cols == 0) return hipSuccess;
  if (!sums_fit(cols)) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>((cols + kCols - 1) / kCols), static_cast<unsigned>(nz));
  if (io == IO_F64) sum_rows<<<grid, kCols * kRows, 0, s>>>(static_cast<const double*>(part), o, rows, cols);
  else sum_rows<<<grid, kCols * kRows, 0, s>>>(static_cast<const float*>(part), o, rows, cols);
  return hipGetLastError();
}

}  // namespace gls
