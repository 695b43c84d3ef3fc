// The 4-bit key/value cache: format helpers.
//
// One row (one token of one head, K or V) of c values x:
//   r = 2^(E - 127),  E = clamp(exponent byte of max|x| - 10, 1, 254), or 255
//       when a value is not finite (such a row reads as NaN);
//   each 16 values: s = E4M3(max|x| / (7 r)), code = rint(x / (s r)) in -7 .. 7
//       (0 when s = 0), stored as the nibble code + 8;
//   value = r s code.
// s has 4 significant bits and a code 3, so s * code is exact in 16-bit
// floats: the operands of the attention's matrix instructions are exact, and
// r, a power of two per row, goes onto the logit (K) or the softmax weight
// (V).  A row with E = 255 has all codes 0 and s = 0.  With bf16 x no rounding
// decision can fall differently in fp32 than in exact arithmetic: a quotient
// of x by the <= 7-bit product 7 r t or t s r is a tie only when it is one
// exactly, and is at least 2^-9 away (relative) otherwise.
//
// 16 consecutive tokens of one head are one tile image (tile_bytes):
//   K codes  [slot][c / 2]              slot(u) = 8 h + 2 t + b of token u = 4 t + 2 h + b
//   V codes  [h][8][t][c / 32][b][2]    bytes: dims chunk (c / 8 dims), word, token parity
//   K scales [slot][c / 16]
//   V scales [c / 16][u]
//   exponents [slot][K, V]
// nibble j of a byte pair: dim 2 i (low), 2 i + 1 (high).  The order is the
// one in which mma.sync fragments take the rows: thread (gid, tig) of a warp
// reads K rows slot gid and gid + 8 (tokens 4 (gid / 2) + gid % 2, + 2) and V
// tokens 4 tig .. 4 tig + 3 with 16-byte accesses, without bank conflicts,
// and a 32-bit word of V holds the same four dims of two tokens in its
// halves.
#pragma once

#include "common.cuh"

namespace csa {
namespace kv4 {

constexpr int kTile = 16;  // tokens per image

__host__ __device__ constexpr int off_v(int c) { return 8 * c; }
__host__ __device__ constexpr int off_ks(int c) { return 16 * c; }
__host__ __device__ constexpr int off_vs(int c) { return 17 * c; }
__host__ __device__ constexpr int off_exp(int c) { return 18 * c; }
__host__ __device__ constexpr int tile_bytes(int c) { return 18 * c + 32; }

__host__ __device__ __forceinline__ int slot_of(int u) {
  return 8 * ((u >> 1) & 1) + 2 * (u >> 2) + (u & 1);
}
// Byte offset of the two bytes (4 dims, d % 4 == 0) of token u in the V codes.
__host__ __device__ __forceinline__ int v_pair(int c, int u, int d) {
  const int D = c >> 3;
  return ((u >> 1) & 1) * 32 * D + (d / D) * 4 * D + (u >> 2) * D + ((d % D) >> 2) * 4 +
         (u & 1) * 2;
}

// 2^(E - 127); NaN for E = 255.
__device__ __forceinline__ float row_scale(uint32_t E) {
  return __uint_as_float(E == 255u ? 0x7fc00000u : E << 23);
}

struct Quant8 {
  uint32_t codes;  // nibble j = value j
  uint32_t scale;  // E4M3 of the 16-value group (both lanes of the pair hold it)
  uint32_t E;
};

// Largest |x| of 8 values as bits (infinities and NaN order above all others).
__device__ __forceinline__ uint32_t top_bits(const uint4& w) {  // bf16 pairs
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
  return max(a & 0xffff0000u, a << 16);
}
__device__ __forceinline__ uint32_t top_bits(const float v[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
  return a;
}

// Quantises 8 values of a row spread over `lanes` neighbouring lanes (8
// values each, lane pairs (2 i, 2 i + 1) forming a group of 16); a = their
// top_bits.  Every lane of the warp calls it.
//
// The quotient x / (s r) without a division per value: x times the correctly
// rounded reciprocal, corrected once by the exact remainder, is the correctly
// rounded quotient, so a tie between two codes stays one, and adding 1.5 2^23
// rounds it to nearest even.  A code can lie beyond 7 only for a subnormal s;
// such groups, and rows near the ends of fp32's range, divide and clamp.
__device__ __forceinline__ Quant8 quantise8(const float v[8], uint32_t a, int lanes) {
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  uint32_t top = a;
  for (int off = lanes >> 1; off > 1; off >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  const int ex = (int)(top >> 23);
  Quant8 q;
  q.codes = 0x88888888u;
  q.scale = 0;
  q.E = 255;
  if (ex == 255) return q;
  q.E = (uint32_t)min(max(ex - 10, 1), 254);
  const float r = __uint_as_float(q.E << 23);
  q.scale = e4m3_code(__fdiv_rn(__uint_as_float(a), 7.f * r));
  const float step = e4m3_value((uint8_t)q.scale) * r;
  if (step == 0.f) return q;
  if (q.scale >= 8 && q.E > 24 && q.E < 230) {
    const float inv = __frcp_rn(step);
    uint32_t acc = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      const float t = v[i] * inv;
      const float x = fmaf(fmaf(-t, step, v[i]), inv, t);
      acc = acc * 16u + __float_as_uint(x + 12582920.f);  // 0x4b400000 + code + 8
    }
    q.codes = acc - 0x3f400000u;  // 0x4b400000 (1 + 16 + 16^2 + ...) mod 2^32
    return q;
  }
  q.codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = rintf(__fdiv_rn(v[i], step));
    q.codes |= (uint32_t)((int)fminf(fmaxf(x, -7.f), 7.f) + 8) << (4 * i);
  }
  return q;
}

}  // namespace kv4
}  // namespace csa
