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

struct Quant16 {
  uint32_t codes[2];  // nibble j of word w: value 8 w + j
  uint32_t scale;     // E4M3 of the group
  uint32_t E;
};

// Largest |x| of 8 bf16 values as bits (infinities and NaN order above all others).
__device__ __forceinline__ uint32_t top_bits(const uint4& w) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
  return max(a & 0xffff0000u, a << 16);
}

// Eight consecutive values of a row as loaded; top(): the largest |x| as bits.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  static constexpr bool kFewBits = true;
  uint4 w;
  __device__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ uint32_t top() const { return top_bits(w); }
  __device__ float2 pair(int i) const {
    const uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
};
template <>
struct Raw8<float> {
  static constexpr bool kFewBits = false;
  float w[8];
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.f;
  }
  __device__ void load(const float* p) { load8(p, w); }
  __device__ uint32_t top() const {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(w[i]) & 0x7fffffffu);
    return a;
  }
  __device__ float2 pair(int i) const { return make_float2(w[2 * i], w[2 * i + 1]); }
};

// Quantises a group of 16 values of a row spread over `lanes` neighbouring
// lanes, a group each.  Every lane of the warp calls it.
//
// No division per value.  bf16: the quotient is a tie k + 1/2 exactly or at
// least 2^-10 away from one, and x times an approximate reciprocal is within
// 7.5 2^-23 of it; adding 6144 rounds that sum to a multiple of 2^-11, which
// restores a tie and moves nothing across one; adding the rest of 1.5 2^23 + 8
// then rounds to nearest even.  fp32: x times the correctly rounded
// reciprocal, corrected once by the exact remainder (Markstein's method), is the
// correctly rounded quotient: true of every mantissa of x and every divisor of
// four significant bits, as all these are (in integers: all 2^23 x 8 cases).  A code can lie beyond 7 only for a subnormal s; such groups, and
// rows near the ends of fp32's range, divide and clamp.
template <typename T>
__device__ __forceinline__ Quant16 quantise16(const Raw8<T> (&raw)[2], int lanes) {
  const uint32_t a = max(raw[0].top(), raw[1].top());
  uint32_t top = a;
  for (int off = lanes >> 1; off > 0; off >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  const int ex = (int)(top >> 23);
  Quant16 q;
  q.codes[0] = q.codes[1] = 0x88888888u;
  q.scale = 0;
  q.E = 255;
  if (ex == 255) return q;
  q.E = (uint32_t)max(ex - 10, 1);
  // a / (7 r), correctly rounded likewise: a / r is exact, the remainder of the
  // first quotient by 7 too
  const float ar = __uint_as_float(a) * __uint_as_float((254u - q.E) << 23);
  const float q0 = ar * (1.f / 7.f);
  q.scale = e4m3_code(fmaf(fmaf(-q0, 7.f, ar), 1.f / 7.f, q0));
  const float step = e4m3_value((uint8_t)q.scale) * __uint_as_float(q.E << 23);
  if (step == 0.f) return q;
  if (q.scale >= 8 && q.E > 24 && q.E < 230) {
    float inv;
    if (Raw8<T>::kFewBits) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
    else inv = __frcp_rn(step);
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t acc = 0;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const float2 v = raw[w].pair(i);
        float2 x;  // 0x4b400000 + code + 8
        if (Raw8<T>::kFewBits) {
          x = add2(fma2(v, inv2, make_float2(6144.f, 6144.f)), make_float2(12576776.f, 12576776.f));
        } else {
          const float t = v.x * inv, s = v.y * inv;
          x = make_float2(fmaf(fmaf(-t, step, v.x), inv, t) + 12582920.f,
                          fmaf(fmaf(-s, step, v.y), inv, s) + 12582920.f);
        }
        acc = acc * 16u + __float_as_uint(x.y);
        acc = acc * 16u + __float_as_uint(x.x);
      }
      q.codes[w] = acc - 0x3f400000u;  // 0x4b400000 (1 + 16 + 16^2 + ...) mod 2^32
    }
    return q;
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    q.codes[w] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = raw[w].pair(i >> 1);
      const float x = rintf(__fdiv_rn(i & 1 ? v.y : v.x, step));
      q.codes[w] |= (uint32_t)((int)fminf(fmaxf(x, -7.f), 7.f) + 8) << (4 * i);
    }
  }
  return q;
}

// The eight values r s code of codes w (nibble j: value j).
__device__ __forceinline__ void store_values(float* p, uint32_t w, uint32_t s, uint32_t E) {
  const float step = e4m3_value((uint8_t)s), r = row_scale(E);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)  // 2^23 + nibble
    x[j] = (__uint_as_float(0x4b000000u | ((w >> (4 * j)) & 15u)) - 8388616.f) * step * r;
  store8(p, x);
}
// bf16: pairs (j, j + 4) of 128 + nibble, times r s, less 136 r s: one fma, each
// part of it exact (s has 4 significant bits, 136 s = 17 s 8 has 8).
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint32_t w, uint32_t s, uint32_t E) {
  if (E - 24u > 206u) {  // near the ends of the range, or 255
    const float step = e4m3_value((uint8_t)s), r = row_scale(E);
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (float)((int)((w >> (4 * j)) & 15u) - 8) * step * r;
    store8(p, x);
    return;
  }
  const float sr = e4m3_value((uint8_t)s) * __uint_as_float(E << 23);
  const __nv_bfloat162 m = __float2bfloat162_rn(sr), c = __float2bfloat162_rn(-136.f * sr);
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t n = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 x = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&n), m, c);
    h[j] = *reinterpret_cast<const uint32_t*>(&x);
  }
  *reinterpret_cast<uint4*>(p) =
      make_uint4(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410),
                 __byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x7632));
}

// Where a lane's part of a row lies in an image: eight dims from 8 sub of a
// key (is_v = 0) or value row.  For token u = 4 t + 2 h + b every offset is
// base + h X + t Y + b Z: the codes' two halves lie `half` bytes apart, and
// those of the eight dims after an even sub's `next` bytes on.
template <int C>
struct LanePart {
  int codes, half, next, code_t, code_b, scale, scale_h, scale_t, scale_b, exp;
  __device__ __forceinline__ LanePart(bool is_v, int sub)
      : codes(is_v ? off_v(C) + v_pair(C, 0, sub * 8) : sub * 4),
        half(is_v ? 4 : 2),
        next(is_v ? (C == 128 ? 8 : 32) : 4),
        code_t(is_v ? C / 8 : C),
        code_b(is_v ? 2 : C / 2),
        scale(is_v ? off_vs(C) + (sub >> 1) * 16 : off_ks(C) + (sub >> 1)),
        scale_h(is_v ? 2 : C / 2),
        scale_t(is_v ? 4 : C / 8),
        scale_b(is_v ? 1 : C / 16),
        exp(off_exp(C) + (is_v ? 1 : 0)) {}
  __device__ __forceinline__ int code_at(int u) const {
    return codes + ((u >> 1) & 1) * 4 * C + (u >> 2) * code_t + (u & 1) * code_b;
  }
  __device__ __forceinline__ int scale_at(int u) const {
    return scale + ((u >> 1) & 1) * scale_h + (u >> 2) * scale_t + (u & 1) * scale_b;
  }
  __device__ __forceinline__ int exp_at(int u) const { return exp + 2 * slot_of(u); }
};

}  // namespace kv4
}  // namespace csa
