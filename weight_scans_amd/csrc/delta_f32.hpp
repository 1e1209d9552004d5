// delta_f32.hpp -- tiles and loads of the chunked gated delta rule in fp32.
//
// The result of v_mfma_f32_16x16x4_f32 (lane (g, l): rows 4g + q of column l) is
// an operand over its rows as it stands: step q of a block of 16 takes value q,
// and lane group g then holds index 4g + q of both operands.  So nothing is
// split into terms, and indices keep their order.
#pragma once

#include "delta_solve.hpp"

namespace gls {

// ---- LDS tile [64][DK] fp32: 16-byte groups XORed with the row's low four
// bits; conflict-free along a row (operands over k) and down a column.
template <int DK>
__device__ __forceinline__ uint32_t row_at(int lane) {
  const int l = lane & 15, g = lane >> 4;
  return static_cast<uint32_t>(l * DK * 4 + 16 * (g ^ l));
}
template <int DK>
__device__ __forceinline__ f32x4 row_frag(const char* tile, uint32_t at, int tb, int b) {
  return *reinterpret_cast<const f32x4*>(tile + tb * 16 * DK * 4 + (at ^ (64 * b)));
}
template <int DK>
__device__ __forceinline__ uint32_t col_at(int lane, int q) {
  const int l = lane & 15, r = 4 * (lane >> 4) + q;
  return static_cast<uint32_t>(r * DK * 4 + 16 * ((l >> 2) ^ r) + 4 * (l & 3));
}
template <int DK>
__device__ __forceinline__ f32x4 col_frag(const char* tile, const uint32_t (&at)[4], int tb, int b) {
  f32x4 x;
#pragma unroll
  for (int q = 0; q < 4; ++q) x[q] = *reinterpret_cast<const float*>(tile + tb * 16 * DK * 4 + (at[q] ^ (64 * b)));
  return x;
}

// Buffer over rows t0 .. t0 + 63 (those below len) of d columns, row stride st.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_f32(const float* base, int64_t t0, int64_t len, int64_t st,
                                                           int d) {
  const int64_t n = len - t0 < 64 ? len - t0 : 64;
  return buffer_rsrc(base + (n > 0 ? t0 * st : 0), n > 0 ? static_cast<int>(((n - 1) * st + d) * 4) : 0);
}

// Rows 16 tb + 4g + q, column r of a [64][VP] tile of a record, as results lie:
// `at` = (4g VP + r) bytes.
__device__ __forceinline__ f32x4 load_rows(__amdgpu_buffer_rsrc_t t, uint32_t at, int VP, int tb) {
  f32x4 x;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    x[q] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(t, at, (16 * tb + q) * VP * 4, 0));
  return x;
}
__device__ __forceinline__ void store_rows(__amdgpu_buffer_rsrc_t t, uint32_t at, int VP, int tb, const f32x4& x) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[q]), t, at, (16 * tb + q) * VP * 4, 0);
}
// A block kept as results (lane (g, l), value q: element (4g + q, l)) read with
// its two indices exchanged.
__device__ __forceinline__ f32x4 turned_f32(const float* block, int lane) {
  const int l = lane & 15, g = lane >> 4;
  f32x4 x;
#pragma unroll
  for (int q = 0; q < 4; ++q) x[q] = block[((l >> 2) * 16 + 4 * g + q) * 4 + (l & 3)];
  return x;
}
// Byte offset, from the chunk's first row, of what lane `lane` of instruction n
// loads into a tile of the layout above.
template <int DK>
__device__ __forceinline__ uint32_t tile_off_f32(int n, int lane, int64_t st, int d) {
  constexpr int U = DK / 4;
  const int i = n * 64 + lane, r = i / U, c = 4 * ((i % U) ^ (r & 15));
  return c < d ? static_cast<uint32_t>((r * static_cast<int>(st) + c) * 4) : kPastEnd;
}

// A chunk's token blocks shared by two waves: 0 and 3, or 1 and 2, five of a
// triangle's ten blocks each.
template <int P>
struct Part {
  static constexpr int tb(int x) { return P ? 1 + x : 3 * x; }  // token block x of the part
  // blocks (tb(x), j) of a lower triangle in order
  static constexpr int count(int x) { return tb(x) + 1; }
  static constexpr int block(int x, int j) { return x ? count(0) + j : j; }
  // blocks (i, tb(x)) in order
  static constexpr int below(int x, int i) { return (x ? 4 - tb(0) : 0) + i - tb(x); }
};

}  // namespace gls
