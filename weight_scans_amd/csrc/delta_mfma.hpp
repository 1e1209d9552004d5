// delta_mfma.hpp -- fragments and LDS tiles of the chunked gated delta rule.
//
// Register chaining: the result layout of v_mfma_f32_16x16x32_bf16 (lane
// (g, l) = (lane / 16, lane % 16) holds rows 4g..4g+3 of column l) becomes an
// operand of the next product without leaving the registers, because the order
// of the contraction index is free as long as both operands share it.  Two
// stacked results (h = 0, 1) give lane (g, l) the rows 4g + q of both as eight
// values (h, q): "order O".  So that the other operand is one 16-byte read of
// eight neighbouring columns, the indices k and r of a state are not taken in
// blocks of 16 as they come: row 4g + q of block 2s + h is
//     index(2s + h, 4g + q) = 32 s + 8 g + 4 h + q.
// Tokens keep their order (their operands are prepared in order O).
//
// Two-term operands: x = hi + lo, both bf16 (round to nearest), keeps 16
// significand bits; products with an exact bf16 operand take two matrix
// instructions, products of two such operands three (lo lo is dropped).
#pragma once

#include "delta.hpp"
#include "mfma.hpp"

namespace gls {

struct Pair8 {  // hi and lo fragments
  bf16x8 hi, lo;
};

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8 as_frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4_t v = {a, b, c, d};
  return __builtin_bit_cast(bf16x8, v);
}
// Rounded fragment of two stacked results (order O).
__device__ __forceinline__ bf16x8 round8(const f32x4& x, const f32x4& y) {
  return as_frag(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(y[0], y[1]), pack2(y[2], y[3]));
}
__device__ __forceinline__ float lo16f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ Pair8 split8(const f32x4& x, const f32x4& y) {
  const uint32_t a = pack2(x[0], x[1]), b = pack2(x[2], x[3]);
  const uint32_t c = pack2(y[0], y[1]), d = pack2(y[2], y[3]);
  Pair8 p;
  p.hi = as_frag(a, b, c, d);
  p.lo = as_frag(pack2(x[0] - lo16f(a), x[1] - hi16f(a)), pack2(x[2] - lo16f(b), x[3] - hi16f(b)),
                 pack2(y[0] - lo16f(c), y[1] - hi16f(c)), pack2(y[2] - lo16f(d), y[3] - hi16f(d)));
  return p;
}

// ---- LDS tiles [64][W] bf16, W in {32, 64, 128}: 16-byte groups XORed with
// swz<W>(row), which spreads the 16-byte operand reads over the banks, and the
// transposing reads (four 8-byte halves of neighbouring groups) less evenly: with the
// turned blocks the recurrences lose 0.9 to 2.0 cycles to bank conflicts per cycle of
// LDS issue, and 1 or 2 per cent of their waves' time waiting for LDS.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4_t;
__device__ __forceinline__ s16x4 tr4(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
}
__device__ __forceinline__ bf16x8 join(const s16x4& a, const s16x4& b) {
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ f32x4 widen(const s16x4& v) {
  const u32x2_t u = __builtin_bit_cast(u32x2_t, v);
  f32x4 f;
  f[0] = __uint_as_float(u[0] << 16);
  f[1] = __uint_as_float(u[0] & 0xffff0000u);
  f[2] = __uint_as_float(u[1] << 16);
  f[3] = __uint_as_float(u[1] & 0xffff0000u);
  return f;
}

// Per-lane byte offsets into a tile: of an operand read (row l, group g) and of
// a transposing read (row 4g + l/4, group l%4).
template <int W>
struct TileLane {
  uint32_t o, t;
};
template <int W>
__device__ __forceinline__ TileLane<W> tile_lane(int lane) {
  const int l = lane & 15, g = lane >> 4, r = 4 * g + (l >> 2);
  TileLane<W> x;
  x.o = static_cast<uint32_t>(l * W * 2 + 16 * (g ^ swz<W>(l)));
  x.t = static_cast<uint32_t>(r * W * 2 + 16 * ((l & 3) ^ swz<W>(r)));
  return x;
}
// Rows 16 tb + l, blocks 2s and 2s + 1 of the columns: an operand over them.
template <int W>
__device__ __forceinline__ bf16x8 frag_n(const char* tile, const TileLane<W>& x, int tb, int s) {
  return *reinterpret_cast<const bf16x8*>(tile + tb * 16 * W * 2 + (x.o ^ (64 * s)));
}
// Index l of block cb of the columns, rows 16 tb + 4g .. + 3 (result layout).
template <int W>
__device__ __forceinline__ s16x4 col4(const char* tile, const TileLane<W>& x, int tb, int cb) {
  return tr4(tile + tb * 16 * W * 2 + (x.t ^ (64 * (cb >> 1))) + 8 * (cb & 1));
}
// The same over rows 32 s.. in order O: an operand over the rows.
template <int W>
__device__ __forceinline__ bf16x8 frag_c(const char* tile, const TileLane<W>& x, int s, int cb) {
  return join(col4<W>(tile, x, 2 * s, cb), col4<W>(tile, x, 2 * s + 1, cb));
}
// Row 16 tb + l, indices 4g..4g+3 of block cb of the columns.
template <int W>
__device__ __forceinline__ s16x4 row4(const char* tile, const TileLane<W>& x, int tb, int cb) {
  return *reinterpret_cast<const s16x4*>(tile + tb * 16 * W * 2 + (x.o ^ (64 * (cb >> 1))) + 8 * (cb & 1));
}
// First of the four indices that rows 4g..4g+3 of block b stand for.
__device__ __forceinline__ int index4(int b, int g) { return 32 * (b >> 1) + 8 * g + 4 * (b & 1); }
__device__ __forceinline__ int index1(int b, int l) { return index4(b, l >> 2) + (l & 3); }

// ---- turning a block: fragments as a wave wrote them (row l of the wave's 16
// in lanes, order O of the other index) read back with that index in lanes.
// Block b of the other index: lane (g, l) gets rows 4g..4g+3 of its index l.
__device__ __forceinline__ s16x4 turned(const uint16_t* frags, int b, int lane) {
  const int l = lane & 15, g = lane >> 4;
  return tr4(reinterpret_cast<const char*>(frags + (b >> 1) * kFrag) + ((l & 3) * 16 + 4 * g + (l >> 2)) * 16 +
             (b & 1) * 8);
}

// Fragments kept for a turned read later lie so that 32 lanes of that read meet
// every pair of banks once: lane (g, l)'s 16 bytes at raw_at, its two halves
// exchanged for g >= 2.
__device__ __forceinline__ int raw_at(int lane) { return (lane ^ (8 * ((lane >> 4) & 1))) * 8; }
__device__ __forceinline__ bf16x8 raw_order(const bf16x8& f, int lane) {
  const u32x4_t v = __builtin_bit_cast(u32x4_t, f);
  const bool x = lane >= 32;
  return as_frag(x ? v[2] : v[0], x ? v[3] : v[1], x ? v[0] : v[2], x ? v[1] : v[3]);
}
// Byte offset of a turned read within a row tile's fragments, block b of 16.
__device__ __forceinline__ uint32_t raw_turned(int lane) {
  const int l = lane & 15, g = lane >> 4, u = l & 3, r = 4 * g + (l >> 2);
  return static_cast<uint32_t>((u * 16 + (r ^ (8 * (u & 1)))) * 16 + 8 * (u >> 1));
}
__device__ __forceinline__ s16x4 turned_raw(const uint16_t* frags, uint32_t at, int b) {
  return tr4(reinterpret_cast<const char*>(frags) + (b >> 1) * 1024 + (at ^ (8 * (b & 1))));
}

// Sum over the 16 lanes of a row of lanes, in every lane.
__device__ __forceinline__ float row_sum(float x) {
  x += dpp<0x128>(0.f, x);  // row_ror:8, 4, 2, 1
  x += dpp<0x124>(0.f, x);
  x += dpp<0x122>(0.f, x);
  x += dpp<0x121>(0.f, x);
  return x;
}

// Lane l of each row of 16 lanes gets the row's sum of x[l].  Each step pairs
// lanes that differ in one bit of what they still have to choose between and
// agree in what they have chosen (lane ^ 8, ^ 7, ^ 3, ^ 1).
template <int CTRL, int N>
__device__ __forceinline__ void row_sums_step(float (&x)[16], bool up) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float give = up ? x[i] : x[i + N], keep = up ? x[i + N] : x[i];
    x[i] = keep + dpp<CTRL>(0.f, give);
  }
}
__device__ __forceinline__ float row_sums(float (&x)[16], int l) {
  row_sums_step<0x128, 8>(x, l & 8);
  row_sums_step<0x141, 4>(x, l & 4);
  row_sums_step<0x1b, 2>(x, l & 2);
  row_sums_step<0xb1, 1>(x, l & 1);
  return x[0];
}

// ---- direct loads of a [64][W] tile: instruction n of a wave fills 64
// consecutive 16-byte units.  Byte offset, from the chunk's first row, of what
// lane `lane` loads; past the buffer's end (zeros) for columns past d.
constexpr uint32_t kPastEnd = 0x7ffffff0u;
template <int W>
__device__ __forceinline__ uint32_t tile_off(int n, int lane, int64_t st, int c0, int d) {
  constexpr int U = W / 8;
  const int i = n * 64 + lane, r = i / U, u = (i % U) ^ swz<W>(r);
  const int c = c0 + 8 * u;
  return c < d ? static_cast<uint32_t>((r * st + c) * 2) : kPastEnd;
}
// Buffer over rows t0 .. t0 + 63 (those below len) of d columns, row stride st.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint16_t* base, int64_t t0, int64_t len, int64_t st,
                                                            int d) {
  const int64_t n = len - t0 < 64 ? len - t0 : 64;
  return buffer_rsrc(base + (n > 0 ? t0 * st : 0), n > 0 ? static_cast<int>(((n - 1) * st + d) * 2) : 0);
}

// Order of the instructions between two of these fences: N times MF matrix
// instructions and then VA vector ones.  A wave issues in order and runs alone
// on its SIMD here, so a matrix product hides only the vector work that stands
// between its instructions.
template <int N, int MF, int VA>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, MF, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, VA, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// Narrows a sequence to segment seg of n: its tokens, first slot, and number of chunks.
__device__ __forceinline__ int segment_of(SeqRange& sr, int64_t& slot0, int seg, int n) {
  const int nc = static_cast<int>((sr.len + kDeltaChunk - 1) / kDeltaChunk);
  if (n == 1) return nc;
  const int per = (nc + n - 1) / n, c0 = static_cast<int>(min(static_cast<int64_t>(seg) * per, static_cast<int64_t>(nc)));
  const int mine = min(per, nc - c0);
  slot0 += c0;
  sr.t0 += c0 * static_cast<int64_t>(kDeltaChunk);
  sr.len = min(sr.len - c0 * static_cast<int64_t>(kDeltaChunk), mine * static_cast<int64_t>(kDeltaChunk));
  return mine;
}

// 16- and 4-byte buffer loads, zeros past the end: unlike loads under a
// condition they draw no branch and no wait of their own.
__device__ __forceinline__ bf16x8 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}

__device__ __forceinline__ f32x4 load_f32x4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// A state [dv][dk] of a head as a buffer, and the byte offset of columns c .. c +
// 3 of row r in it: zeros past dv and past dk, and everywhere if p is NULL.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t state_rsrc(const float* p, int dv, int dk) {
  return buffer_rsrc(p, p ? dv * dk * 4 : 0);
}
__device__ __forceinline__ uint32_t state_off(int r, int c, int dk) {
  return c < dk ? static_cast<uint32_t>((r * dk + c) * 4) : kPastEnd;
}

// Factors of the decay inside a chunk for the waves that form P (lane = token,
// m_x the l before its block x of 16), by a loading wave into [6][64] of LDS:
// scale e^(l_i - m_x) of block x's own tokens; e^(m_x - l_j) of those before it
// for x = 1, 2, 3; and l in its two parts for the diagonal blocks.
struct DecayFactors {
  float scale, lw, lf;
  int lane;
  __device__ __forceinline__ DecayFactors(float s, int ln) : scale(s), lw(0.f), lf(0.f), lane(ln) {}
  __device__ __forceinline__ void fetch(const float* gates) {
    lw = gates[192 + lane];
    lf = gates[256 + lane];
  }
  __device__ __forceinline__ void put(float* lds) const {
    const int g = lane >> 4;
    lds[256 + lane] = lw;
    lds[320 + lane] = lf;
    float own = 0.f;
#pragma unroll
    for (int x = 1; x < 4; ++x) {
      const float dw = lw - readlane_f(lw, 16 * x - 1), df = lf - readlane_f(lf, 16 * x - 1);
      const float e = fexp2(g == x ? dw + df : lane < 16 * x ? -dw - df : -200.f);
      lds[64 * x + lane] = e;
      own = g == x ? scale * e : own;
    }
    lds[lane] = own;
  }
};

// Work-groups are dealt to the 8 XCDs in turn: all `tiles` of a sequence-head
// get the same XCD (they share its chunks through the XCD's L2).  Returns
// false past the end.
__device__ __forceinline__ bool head_of_block(int64_t id, int tiles, int64_t heads, int64_t& head, int& tile) {
  const int64_t j = id >> 3;
  head = j / tiles * 8 + (id & 7);
  tile = static_cast<int>(j % tiles);
  return head < heads;
}
inline int64_t head_blocks(int64_t heads, int tiles) { return (heads + 7) / 8 * 8 * tiles; }

}  // namespace gls
