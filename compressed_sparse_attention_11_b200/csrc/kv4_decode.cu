// Attention of one query token per sequence over the paged 4-bit key/value
// cache (kv4.cuh: the format), heads in groups of g = nh / nkv on each
// key/value head:
//   E_b = { u <= p : u > p - W or u < first }   (W = 0: every u <= p), p = pos[b]
//   l_u = scale q . k_u,   out = sum_u e^{l_u} v_u / (e^{sink} + sum_u e^{l_u}).
//
// HBM-bound up to g = 16 (146 bytes a token and head at c = 128 against 8 g c
// flops); what it takes is turning 4-bit codes into matrix operands as fast
// as they arrive.  Both products run on mma.sync.m16n8k16 with the cache on
// the M side and the heads on the N side (8 heads a tile), so no row of the
// instruction is padding at g = 8:
//   S^T[key, head] = K Q^T,   O^T[dim, head] += V^T P^T,
// and a code pair becomes an operand register in three instructions: shift,
// (x & mask) | 1.0 (the nibble n lands in the upper mantissa bits of a bf16:
// 1 + n / 16), and one bf16x2 fma with (16 s, -24 s), which gives s (n - 8)
// exactly.  The format stores rows in the fragments' order, so V needs no
// transposition, and the row exponents go onto the logit and the weight.
// tcgen05 would need the widened rows in shared memory first (16-bit operands
// of both products through it: four times the cache's bytes), which is more
// than an SM's share of HBM time allows; mma.sync takes them from registers.
//
// Work: units of 8 images (128 tokens) of one (sequence, head tile), in one
// flat list that is cut evenly over the CTAs whatever the lengths; a producer
// warp streams units through a ring of bulk copies, warp w of 8 takes image w
// of each unit with its own running maximum, sum and output, and the eight
// are merged where a sequence ends or the CTA's share does.  What a CTA covers
// whole is written out; other pieces go to the workspace (two slots a CTA) and
// a second kernel merges them.
#include "api_check.h"
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace sm100;

constexpr int kConsWarps = 8;
constexpr int kConsThreads = kConsWarps * 32;
constexpr int kThreads = kConsThreads + 32;
constexpr int kUnitTiles = kConsWarps;  // images per unit
constexpr float kRescaleLog2 = 8.f;

struct DecArgs {
  const uint8_t* cache;
  const int32_t* table;
  const int64_t* pos;
  const __nv_bfloat16* q;
  const float* sink;
  __nv_bfloat16* out;
  float* ws;
  unsigned int* err;
  int64_t max_blocks, num_blocks, capacity;  // capacity: tokens a row of the table can name
  int64_t window, first;
  int batch, nkv, nh, group, head_tiles, tiles_per_block;
  float qscale;  // scale * log2(e)
};

// What sequence b sees, in images: virtual image i is image i below `head`,
// else image tail + i - head.
struct Seen {
  int64_t n, lo;  // visible: u < n and (u >= lo or u < first)
  int head, tail, images;
};
__device__ __forceinline__ Seen seen_of(const DecArgs& a, int64_t p) {
  Seen s;
  s.n = min(p + 1, a.capacity);
  s.lo = 0;
  s.head = s.tail = s.images = 0;
  if (p < 0) {
    s.n = 0;
    return s;
  }
  if (a.window > 0 && p + 1 > a.window) s.lo = p + 1 - a.window;
  const int64_t end = (s.n + 15) / 16;
  const int64_t t = min(s.lo / 16, end), h = (min(a.first, s.lo) + 15) / 16;
  s.tail = (int)t;
  s.head = (int)min(h, t);
  s.images = s.head + (int)(end - t);
  return s;
}
__device__ __forceinline__ int units_of(const Seen& s) {
  return (s.images + kUnitTiles - 1) / kUnitTiles;
}

// The flat list of units: sequence b's units of head tile t start at
// head_tiles_all * first[b] + t * units(b).
__device__ __forceinline__ int64_t cta_first(int64_t U, int G, int i) { return U * i / G; }
__device__ __forceinline__ int cta_of(int64_t U, int G, int64_t u) {
  return (int)(((u + 1) * G - 1) / U);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Scale bytes picked into the two halves -> (16 s, -24 s).  An E4M3 byte
// shifted into a bf16's exponent and mantissa reads as s 2^-120.
struct ScalePair {
  uint32_t s16, n24;
};
__device__ __forceinline__ ScalePair scale_pair(uint32_t bytes, uint32_t sel) {
  ScalePair p;
  p.s16 = mul_bf16x2(__byte_perm(bytes, 0, sel) << 4, 0x7d807d80u);  // 2^124
  p.n24 = mul_bf16x2(p.s16, 0xbfc0bfc0u);                            // -1.5
  return p;
}
// Nibbles j and j + 4 of w -> (s (n - 8)) in the two halves.
template <int J>
__device__ __forceinline__ uint32_t widen(uint32_t w, const ScalePair& s) {
  const uint32_t y = J == 0 ? w << 3 : w >> (J == 0 ? 0 : 4 * J - 3);
  return fma_bf16x2((y & 0x00780078u) | 0x3f803f80u, s.s16, s.n24);
}

template <int C, int NT>
struct Cfg {
  static constexpr int kTB = kv4::tile_bytes(C);
  static constexpr int kStageBytes = kUnitTiles * kTB;
  static constexpr int kStages = 4;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kLd = C + 4;  // padded row of the merge buffer (floats)
  static constexpr int kSlot = kHeads * C + 2 * kHeads;  // floats of a workspace slot
  static constexpr int off_merge() { return kStages * kStageBytes; }
  static constexpr int off_ml() { return off_merge() + kConsWarps * kHeads * kLd * 4; }
  static constexpr int off_meta() { return off_ml() + kConsWarps * kHeads * 8; }
  static constexpr int off_bar() { return off_meta() + kStages * kUnitTiles * 8; }
  static constexpr int off_list() { return off_bar() + 2 * kStages * 8 + 16 + 64; }
  static size_t smem(int batch) { return off_list() + (size_t)(batch + 1) * 4; }
};

template <int C, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) kv4_decode_kernel(const __grid_constant__ DecArgs a) {
  using F = Cfg<C, NT>;
  constexpr int D = C / 8;    // dims of a V chunk
  constexpr int KS = C / 16;  // k-steps of Q.K
  constexpr int MT = D / 2;   // m-tiles of P.V
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + F::off_merge());
  float2* ml = reinterpret_cast<float2*>(smem + F::off_ml());
  int64_t* meta = reinterpret_cast<int64_t*>(smem + F::off_meta());  // first token, or -1
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::off_bar());
  uint64_t* empty = full + F::kStages;
  int* scan = reinterpret_cast<int*>(empty + F::kStages);
  int* first_unit = reinterpret_cast<int*>(smem + F::off_list());  // [batch + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kStages; ++i) {
      mbar_init(&full[i], kUnitTiles);
      mbar_init(&empty[i], kConsWarps);
    }
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();

  // units before each sequence
  {
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int u = b < a.batch ? units_of(seen_of(a, a.pos[b])) : 0;
      int inc = u;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      int before = base, all = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
      }
      if (b < a.batch) first_unit[b] = before + inc - u;
      base += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) first_unit[a.batch] = base;
    __syncthreads();
  }
  const int HV = a.nkv * a.head_tiles;
  const int64_t U = (int64_t)first_unit[a.batch] * HV;
  if (U == 0) return;
  // with fewer units than CTAs the last CTAs take none
  const int G = (int)min((int64_t)gridDim.x, U);
  if ((int)blockIdx.x >= G) return;
  const int64_t u_lo = cta_first(U, G, blockIdx.x), u_hi = cta_first(U, G, blockIdx.x + 1);

  // the sequence of the first unit: the last b with HV * first_unit[b] <= u_lo
  int b = 0;
  {
    int lo = 0, hi = a.batch;  // first_unit[lo] * HV <= u_lo < first_unit[hi] * HV
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)first_unit[mid] * HV <= u_lo) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  int nu = first_unit[b + 1] - first_unit[b];
  int64_t off = u_lo - (int64_t)first_unit[b] * HV;
  int hv = (int)(off / nu), s = (int)(off - (int64_t)hv * nu);
  auto next_segment = [&]() {  // the unit list's next (sequence, head tile)
    s = 0;
    if (++hv == HV) {
      hv = 0;
      do { ++b; } while (b < a.batch && first_unit[b + 1] == first_unit[b]);
      nu = b < a.batch ? first_unit[b + 1] - first_unit[b] : 0;
    }
  };

  if (warp == kConsWarps) {
    // ============================ producer: lanes 0-7, one image each ==========
    int it = 0;
    for (int64_t u = u_lo; u < u_hi;) {
      const Seen v = seen_of(a, a.pos[b]);
      const int h = hv / a.head_tiles;
      for (; s < nu && u < u_hi; ++s, ++u, ++it) {
        const int st = it % F::kStages;
        const int i = s * kUnitTiles + lane;
        int64_t tile = -1, blk = -1;
        if (lane < kUnitTiles && i < v.images) {
          tile = i < v.head ? i : v.tail + (i - v.head);
          blk = a.table[b * a.max_blocks + tile / a.tiles_per_block];
          if (blk < 0 || blk >= a.num_blocks) tile = -1;
        }
        if (it >= F::kStages) mbar_wait(&empty[st], ((it / F::kStages) - 1) & 1, a.err);
        if (lane < kUnitTiles) {
          meta[st * kUnitTiles + lane] = tile < 0 ? -1 : tile * 16;
          if (tile >= 0) {
            mbar_arrive_expect_tx(&full[st], F::kTB);
            bulk_load(smem + st * F::kStageBytes + lane * F::kTB,
                      a.cache + ((blk * a.nkv + h) * a.tiles_per_block +
                                 tile % a.tiles_per_block) * (int64_t)F::kTB,
                      F::kTB, &full[st]);
          } else {
            mbar_arrive(&full[st]);
          }
        }
        __syncwarp();
      }
      if (s == nu) next_segment();
    }
    // after a wait that gave up, copies may still be on their way in
    const int last = it < F::kStages ? it : F::kStages;
    for (int k = it - last; k < it; ++k)
      mbar_wait(&full[k % F::kStages], (k / F::kStages) & 1, a.err, false);
    return;
  }

  // ============================== consumers ====================================
  const int gid = lane >> 2, tig = lane & 3;
  const int tok_a = 4 * (gid >> 1) + (gid & 1);  // token of slot gid; slot gid + 8: + 2
  int it = 0;
  for (int64_t u = u_lo; u < u_hi;) {
    const Seen v = seen_of(a, a.pos[b]);
    const int kvh = hv / a.head_tiles, h0 = (hv % a.head_tiles) * F::kHeads;
    const int cur_b = b, cur_hv = hv;
    const bool starts = s == 0, at_first = u == u_lo;
    // queries as B fragments: head gid (+ 8 per n-tile), dims C / 4 tig ..
    uint32_t qf[NT][KS][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int hl = h0 + 8 * t + gid;
      const __nv_bfloat16* qp =
          a.q + ((int64_t)cur_b * a.nh + (int64_t)kvh * a.group + hl) * C + tig * (C / 4);
#pragma unroll
      for (int w = 0; w < C / 32; ++w) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (hl < a.group) r = __ldg(reinterpret_cast<const uint4*>(qp) + w);
        qf[t][2 * w][0] = __byte_perm(r.x, r.z, 0x5410);
        qf[t][2 * w][1] = __byte_perm(r.x, r.z, 0x7632);
        qf[t][2 * w + 1][0] = __byte_perm(r.y, r.w, 0x5410);
        qf[t][2 * w + 1][1] = __byte_perm(r.y, r.w, 0x7632);
      }
    }
    float o[NT][MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = kNegInf;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int k = 0; k < MT; ++k) o[t][k][0] = o[t][k][1] = o[t][k][2] = o[t][k][3] = 0.f;
    }

    for (; s < nu && u < u_hi; ++s, ++u, ++it) {
      const int st = it % F::kStages;
      mbar_wait(&full[st], (it / F::kStages) & 1, a.err);
      const int64_t t0 = meta[st * kUnitTiles + warp];
      if (t0 >= 0) {
        const uint8_t* im = smem + st * F::kStageBytes + warp * F::kTB;
        // ---- S^T = K Q^T ----------------------------------------------------
        float sc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
        uint32_t ka[C / 32], kb[C / 32];
        ScalePair sa[C / 64], sb[C / 64];
        if constexpr (C == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(im + gid * 64 + tig * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(im + (gid + 8) * 64 + tig * 16);
          ka[0] = x.x; ka[1] = x.y; ka[2] = x.z; ka[3] = x.w;
          kb[0] = y.x; kb[1] = y.y; kb[2] = y.z; kb[3] = y.w;
          const uint32_t p = *reinterpret_cast<const uint16_t*>(im + kv4::off_ks(C) + gid * 8 + 2 * tig);
          const uint32_t r = *reinterpret_cast<const uint16_t*>(im + kv4::off_ks(C) + (gid + 8) * 8 + 2 * tig);
          sa[0] = scale_pair(p, 0x4040); sa[1] = scale_pair(p, 0x4141);
          sb[0] = scale_pair(r, 0x4040); sb[1] = scale_pair(r, 0x4141);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(im + gid * 32 + tig * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(im + (gid + 8) * 32 + tig * 8);
          ka[0] = x.x; ka[1] = x.y;
          kb[0] = y.x; kb[1] = y.y;
          sa[0] = scale_pair(im[kv4::off_ks(C) + gid * 4 + tig], 0x4040);
          sb[0] = scale_pair(im[kv4::off_ks(C) + (gid + 8) * 4 + tig], 0x4040);
        }
#pragma unroll
        for (int w = 0; w < C / 32; ++w) {
          const uint32_t a0 = widen<0>(ka[w], sa[w / 2]), a1 = widen<0>(kb[w], sb[w / 2]);
          const uint32_t a2 = widen<1>(ka[w], sa[w / 2]), a3 = widen<1>(kb[w], sb[w / 2]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_16816(sc[t], a0, a1, a2, a3, qf[t][2 * w][0], qf[t][2 * w][1]);
          const uint32_t c0 = widen<2>(ka[w], sa[w / 2]), c1 = widen<2>(kb[w], sb[w / 2]);
          const uint32_t c2 = widen<3>(ka[w], sa[w / 2]), c3 = widen<3>(kb[w], sb[w / 2]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_16816(sc[t], c0, c1, c2, c3, qf[t][2 * w + 1][0], qf[t][2 * w + 1][1]);
        }
        // ---- online softmax ---------------------------------------------------
        const uint32_t ea = *reinterpret_cast<const uint16_t*>(im + kv4::off_exp(C) + 2 * gid);
        const uint32_t eb = *reinterpret_cast<const uint16_t*>(im + kv4::off_exp(C) + 2 * gid + 16);
        const int64_t ua = t0 + tok_a, ub = ua + 2;
        const bool va = ua < v.n && (ua >= v.lo || ua < a.first);
        const bool vb = ub < v.n && (ub >= v.lo || ub < a.first);
        const float ra = kv4::row_scale(ea & 255u) * a.qscale, rb = kv4::row_scale(eb & 255u) * a.qscale;
        const float wa = va ? kv4::row_scale(ea >> 8) : 0.f, wb = vb ? kv4::row_scale(eb >> 8) : 0.f;
        bool grow = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sc[t][e] = va ? sc[t][e] * ra : kNegInf;
            sc[t][2 + e] = vb ? sc[t][2 + e] * rb : kNegInf;
            grow |= fmaxf(sc[t][e], sc[t][2 + e]) > m[t][e] + kRescaleLog2;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(sc[t][e], sc[t][2 + e]);
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
              x = fmaxf(x, m[t][e]);
              const float f = m[t][e] == kNegInf ? 0.f : ex2(m[t][e] - x);
              m[t][e] = x;
              l[t][e] *= f;
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                o[t][k][e] *= f;
                o[t][k][2 + e] *= f;
              }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mr = m[t][e] == kNegInf ? 0.f : m[t][e];
            p[e] = ex2(sc[t][e] - mr);
            p[2 + e] = ex2(sc[t][2 + e] - mr);
            l[t][e] += p[e] + p[2 + e];
          }
          // weights times the rows' exponents, rounded to the operand's bf16
          // (the sum keeps the unrounded weights)
          pb[t][0] = transpose8x8(pack_bf16x2(p[0] * wa, p[1] * wa));
          pb[t][1] = transpose8x8(pack_bf16x2(p[2] * wb, p[3] * wb));
        }
        // ---- O^T += V^T P^T ----------------------------------------------------
        const uint8_t* vim = im + kv4::off_v(C) + gid * 4 * D + tig * D;
        const uint32_t vs = *reinterpret_cast<const uint32_t*>(
            im + kv4::off_vs(C) + (C == 128 ? gid : gid >> 1) * 16 + 4 * tig);
        const ScalePair s0 = scale_pair(vs, 0x4140), s1 = scale_pair(vs, 0x4342);
        uint32_t x0[D / 4], x1[D / 4];
        if constexpr (C == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(vim);
          const uint4 y = *reinterpret_cast<const uint4*>(vim + 32 * D);
          x0[0] = x.x; x0[1] = x.y; x0[2] = x.z; x0[3] = x.w;
          x1[0] = y.x; x1[1] = y.y; x1[2] = y.z; x1[3] = y.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(vim);
          const uint2 y = *reinterpret_cast<const uint2*>(vim + 32 * D);
          x0[0] = x.x; x0[1] = x.y;
          x1[0] = y.x; x1[1] = y.y;
        }
#pragma unroll
        for (int w = 0; w < D / 4; ++w) {
          const uint32_t a0 = widen<0>(x0[w], s0), a1 = widen<1>(x0[w], s0);
          const uint32_t a2 = widen<0>(x1[w], s1), a3 = widen<1>(x1[w], s1);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_16816(o[t][2 * w], a0, a1, a2, a3, pb[t][0], pb[t][1]);
          const uint32_t c0 = widen<2>(x0[w], s0), c1 = widen<3>(x0[w], s0);
          const uint32_t c2 = widen<2>(x1[w], s1), c3 = widen<3>(x1[w], s1);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_16816(o[t][2 * w + 1], c0, c1, c2, c3, pb[t][0], pb[t][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    const bool ends = s == nu;
    if (ends) next_segment();

    // ---- merge the eight warps ---------------------------------------------------
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        const int hl = 8 * t + 2 * tig + e;
        if (gid == 0) ml[warp * F::kHeads + hl] = make_float2(m[t][e], x);
        float* row = merge + (warp * F::kHeads + hl) * F::kLd + gid * D;
#pragma unroll
        for (int k = 0; k < MT; ++k)
          *reinterpret_cast<float2*>(row + 2 * k) = make_float2(o[t][k][e], o[t][k][2 + e]);
      }
    named_bar_or(1, kConsThreads, false);
    const bool direct = starts && ends;
    float* slot = a.ws + ((int64_t)blockIdx.x * 2 + (at_first ? 0 : 1)) * F::kSlot;
    for (int e = threadIdx.x; e < F::kHeads * (C / 4); e += kConsThreads) {
      const int hl = e / (C / 4), d = (e % (C / 4)) * 4;
      float M = kNegInf;
#pragma unroll
      for (int w = 0; w < kConsWarps; ++w) M = fmaxf(M, ml[w * F::kHeads + hl].x);
      const float mr = M == kNegInf ? 0.f : M;
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kConsWarps; ++w) {
        const float2 x = ml[w * F::kHeads + hl];
        const float f = ex2(x.x - mr);
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * F::kHeads + hl) * F::kLd + d);
        L = fmaf(x.y, f, L);
        acc.x = fmaf(y.x, f, acc.x);
        acc.y = fmaf(y.y, f, acc.y);
        acc.z = fmaf(y.z, f, acc.z);
        acc.w = fmaf(y.w, f, acc.w);
      }
      if (direct) {
        if (h0 + hl < a.group) {
          const int head = kvh * a.group + h0 + hl;
          const float den = L + (a.sink != nullptr && M != kNegInf ? ex2(a.sink[head] * kLog2e - M) : 0.f);
          const float inv = den == 0.f ? 0.f : 1.f / den;
          uint2 w;
          w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
          w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(a.out + ((int64_t)cur_b * a.nh + head) * C + d) = w;
        }
      } else {
        *reinterpret_cast<float4*>(slot + hl * C + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(slot + F::kHeads * C + 2 * hl) = make_float2(M, L);
      }
    }
    named_bar_or(1, kConsThreads, false);
    (void)cur_hv;
  }
}

// One block per (sequence, head tile): merges the pieces that lie in more
// than one CTA's share, and zeroes the output of sequences that see nothing.
template <int C, int NT>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const __grid_constant__ DecArgs a, int grid) {
  using F = Cfg<C, NT>;
  __shared__ long long part[2][8];
  pdl_wait();
  const int HV = a.nkv * a.head_tiles;
  const int b = blockIdx.x / HV, hv = blockIdx.x % HV;
  const int kvh = hv / a.head_tiles, h0 = (hv % a.head_tiles) * F::kHeads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long before = 0, all = 0;
  for (int i = threadIdx.x; i < a.batch; i += 256) {
    const int u = units_of(seen_of(a, a.pos[i]));
    all += u;
    if (i < b) before += u;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, off);
    all += __shfl_xor_sync(0xffffffffu, all, off);
  }
  if (lane == 0) {
    part[0][warp] = before;
    part[1][warp] = all;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    before += part[0][w];
    all += part[1][w];
  }
  const int nu = units_of(seen_of(a, a.pos[b]));
  const int64_t U = (int64_t)all * HV;
  const int G = (int)min((int64_t)grid, U);
  const int64_t u0 = (int64_t)before * HV + (int64_t)hv * nu, u1 = u0 + nu;
  const int i0 = nu > 0 ? cta_of(U, G, u0) : 0, i1 = nu > 0 ? cta_of(U, G, u1 - 1) : 0;
  if (nu > 0 && i0 == i1) return;  // written by the CTA itself
  for (int e = threadIdx.x; e < F::kHeads * (C / 4); e += 256) {
    const int hl = e / (C / 4), d = (e % (C / 4)) * 4;
    if (h0 + hl >= a.group) continue;
    const int head = kvh * a.group + h0 + hl;
    float M = kNegInf, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (nu > 0) {
      for (int i = i0; i <= i1; ++i) {
        const int which = i > i0 || cta_first(U, G, i) == u0 ? 0 : 1;
        const float* slot = a.ws + ((int64_t)i * 2 + which) * F::kSlot;
        const float2 x = *reinterpret_cast<const float2*>(slot + F::kHeads * C + 2 * hl);
        const float4 y = *reinterpret_cast<const float4*>(slot + hl * C + d);
        const float mn = fmaxf(M, x.x), mr = mn == kNegInf ? 0.f : mn;
        const float f0 = ex2(M - mr), f1 = ex2(x.x - mr);
        M = mn;
        L = L * f0 + x.y * f1;
        acc.x = acc.x * f0 + y.x * f1;
        acc.y = acc.y * f0 + y.y * f1;
        acc.z = acc.z * f0 + y.z * f1;
        acc.w = acc.w * f0 + y.w * f1;
      }
    }
    const float den = L + (a.sink != nullptr && M != kNegInf ? ex2(a.sink[head] * kLog2e - M) : 0.f);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint2 w;
    w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.nh + head) * C + d) = w;
  }
}

// CTAs of the decode kernel, and the head tile (n-tiles of 8) for a group.
int dec_nt(int group) { return group <= 8 ? 1 : 2; }
int dec_grid(int group) { return sm_count() * (dec_nt(group) == 1 ? 2 : 1); }

template <int C, int NT>
cudaError_t launch_dec(const DecArgs& a, cudaStream_t s) {
  using F = Cfg<C, NT>;
  auto kern = kv4_decode_kernel<C, NT>;
  const size_t smem = F::smem(a.batch);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)F::smem(4096));
  if (e != cudaSuccess) return e;
  const int G = dec_grid(a.group);
  if ((e = launch_pdl(kern, dim3((unsigned)G), dim3(kThreads), smem, s, a)) != cudaSuccess) return e;
  return launch_pdl(kv4_combine_kernel<C, NT>, dim3((unsigned)(a.batch * a.nkv * a.head_tiles)),
                    dim3(256), 0, s, a, G);
}

}  // namespace

csa_status check_kv4(const csa_kv4_cache* c);

}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_kv4_decode_workspace(int nh, int nkv, int c) {
  if (nkv < 1 || nh < nkv || nh % nkv != 0 || (c != 64 && c != 128)) return 0;
  const int group = nh / nkv, heads = 8 * dec_nt(group);
  return (size_t)dec_grid(group) * 2 * (heads * c + 2 * heads) * 4;
}

csa_status csa_kv4_decode_attn(const csa_kv4_cache* cache, const int64_t* pos, const void* q,
                               int nh, int64_t window, int64_t first, const float* sink,
                               float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
  csa_status st = check_kv4(cache);
  if (st != CSA_OK) return st;
  API_REQUIRE(nh >= 1 && nh % cache->nkv == 0, "nh must be a positive multiple of nkv");
  API_REQUIRE(window >= 0, "window must be >= 0 (0: every token)");
  API_REQUIRE(first >= 0, "first must be >= 0");
  API_REQUIRE(scale == scale && scale > -3.4e38f && scale < 3.4e38f, "scale must be finite");
  API_SUPPORTED(nh <= 65536, "csa_kv4_decode_attn needs nh <= 65536");
  API_SUPPORTED((cache->max_blocks * cache->block_tokens / 128 + 2) * cache->batch < ((int64_t)1 << 31) &&
                    (int64_t)cache->batch * nh < ((int64_t)1 << 31),
                "csa_kv4_decode_attn: the batch has too many tokens");
  if (cache->batch == 0) return api_ok();
  API_REQUIRE_LIST(pos);
  API_REQUIRE_PTR(q);
  API_REQUIRE_PTR(out);
  API_REQUIRE_OPT_LIST(sink);
  const size_t need = csa_kv4_decode_workspace(nh, cache->nkv, cache->c);
  if (ws == nullptr || ws_bytes < need)
    return set_last_error(CSA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws_bytes, need);
  API_REQUIRE_PTR(ws);
  unsigned int* flag = device_timeout_flag();
  if (flag == nullptr) return set_last_error(CSA_ERR_CUDA, "csa_kv4_decode_attn: no device flag");
  DecArgs a;
  a.cache = (const uint8_t*)cache->data;
  a.table = cache->block_table;
  a.pos = pos;
  a.q = (const __nv_bfloat16*)q;
  a.sink = sink;
  a.out = (__nv_bfloat16*)out;
  a.ws = (float*)ws;
  a.err = flag;
  a.max_blocks = cache->max_blocks;
  a.num_blocks = cache->num_blocks;
  a.capacity = cache->max_blocks * cache->block_tokens;
  a.window = window;
  a.first = first;
  a.batch = (int)cache->batch;
  a.nkv = cache->nkv;
  a.nh = nh;
  a.group = nh / cache->nkv;
  const int nt = dec_nt(a.group);
  a.head_tiles = (a.group + 8 * nt - 1) / (8 * nt);
  a.tiles_per_block = cache->block_tokens / 16;
  a.qscale = scale * kLog2e;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (cache->c == 128) e = nt == 1 ? launch_dec<128, 1>(a, s) : launch_dec<128, 2>(a, s);
  else e = nt == 1 ? launch_dec<64, 1>(a, s) : launch_dec<64, 2>(a, s);
  return api_cuda(e, "csa_kv4_decode_attn");
}

}  // extern "C"
