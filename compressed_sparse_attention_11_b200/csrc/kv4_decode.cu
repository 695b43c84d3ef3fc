// Attention of one query token per sequence over the paged 4-bit key/value
// cache (kv4.cuh: the format), heads in groups of g = nh / nkv on each
// key/value head:
//   E_b = { u <= p : u > p - W or u < first }   (W = 0: every u <= p), p = pos[b]
//   l_u = scale q . k_u,   out = sum_u e^{l_u} v_u / (e^{sink} + sum_u e^{l_u}).
//
// HBM-bound up to g = 16 (146 bytes a token and head at c = 128 against 8 g c
// flops); what it takes is turning 4-bit codes into matrix operands as fast
// as they arrive.  Both products run on mma.sync.m16n8k16 (f16 in, fp32 out)
// with the cache on the M side and the heads on the N side (8 heads a tile),
// so no row of the instruction is padding at g = 8:
//   S^T[key, head] = K Q^T,   O^T[dim, head] += V^T P^T.
// The format stores rows in the fragments' order, so V needs no transposition,
// and a nibble becomes an operand where it stands: in a 16-bit word of four,
// (x & 0x00f0) | 0x5400 is the f16 64 + n and one fma with (s, -72 s) gives
// s (n - 8) exactly; (x & 0x000f) | 0x6400 is 1024 + n and takes a subtraction
// and a product; the upper two follow after one shift.  Logic and shifts were
// the bound with bf16 operands, whose seven mantissa bits want a shift per
// nibble; now these and the f16 arithmetic weigh about the same (ALU 53 %, FMA
// 49 %, two thirds of the issue slots: no pipe is full, dependent steps of four
// warps a scheduler leave the rest).
// f16's range: a query head is scaled to largest element 1 .. 2 (elements below
// 2^-14 of it keep an absolute 2^-25), and the second product's weight is
// w_u = 2^(l_u + E_u - M'), E_u the value row's exponent and M' a reference of
// its own, 8 to 15 below the running maximum of l + E, so that the rows with
// the largest products have weights of 2^8 and more whatever their magnitude.
// In w's f16 a row with E_u near the maximum's keeps an absolute 2^-33 of the
// largest softmax weight.  A row whose values are far smaller than the largest
// ones (E_u more than 5 below M' + 8 - M) could lose a weight that counts in
// the dims where the large rows hold little: for such rows the remainders
// w - f16(w) are multiplied as well, scaled by 2^26, 2^52 and 2^78 (with O, in
// fp32, scaled alike meanwhile), so each weight is off by 2^-11 of itself or
// 2^-28 of the largest one at most, for rows whose products lie up to 2^90 apart.
// That path is taken where a warp's two images hold such a row and costs three
// more second products there: 32 sequences of 24 576 tokens, 64 / 8 heads x 128:
// 208 us with rows alike, 236 with one row in 4096 2^12 times the others, 310 with
// every second row 2^-12 of its neighbours.  Rows alike pay 2 % for its presence
// (208 -> 212 us, sustained).
// tcgen05 would need the widened rows in shared memory first (16-bit operands
// of both products through it: four times the cache's bytes), which is more
// than an SM's share of HBM time allows; mma.sync takes them from registers.
//
// Work: units of 8 images (128 tokens) of one (sequence, head tile), in one
// flat list that is cut evenly over the CTAs whatever the lengths.  Warp w of 4
// takes images 2 w and 2 w + 1 of each unit, brought in by bulk copies through
// a ring of its own, so no warp waits for another (one ring for the CTA moved
// the warps in step and took a fifth longer), with its own running maxima, sum
// and output; the four are merged where a sequence ends or the CTA's share
// does (four CTAs of four warps on an SM: 197 us in short runs, before the
// remainders; two of eight: 201; times at 32 sequences of 16-32 K tokens, 64 / 8
// heads x 128, whose bytes take 140; 212 sustained now).  What a CTA covers whole is written out; other pieces go to the
// workspace (two slots a CTA) and a second kernel merges them.
#include <cuda_fp16.h>
#include <limits.h>

#include <type_traits>

#include "api_check.h"
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kPair = 2;                     // neighbouring images a warp takes at once
constexpr int kUnitTiles = kPair * kWarps;  // images per unit
constexpr float kRescaleLog2 = 8.f;
// Weights of the output: the largest is 2^8 when its reference is set and may
// grow to 2^15 before the reference moves (f16 ends at 65504).
constexpr float kTopLog2 = 8.f, kMostLog2 = 15.f;
// A row whose exponent lies more than 5 below what the reference stands for has
// its weight's remainder taken along, in steps of 2^26.
constexpr float kDeepLog2 = 5.f;
constexpr int kDeepSteps = 3;
constexpr float kNone = -3e38f;  // running maximum of a head that has seen nothing

struct DecArgs {
  const uint8_t* cache;
  const int32_t* table;
  const int64_t* pos;
  const __nv_bfloat16* q;
  const float* sink;
  __nv_bfloat16* out;
  float* ws;
  unsigned int* err;
  int64_t max_blocks, num_blocks;
  int capacity;  // tokens a row of the table can name
  int window, first;
  int batch, nkv, nh, group, head_tiles, tiles_per_block;
  float qscale;  // scale * log2(e)
};

// Positions are below 2^31 - 1 (a sequence holds at most 2^31 tokens).
__device__ __forceinline__ int clip_pos(int64_t p) {
  return (int)max((int64_t)-1, min(p, (int64_t)INT_MAX - 1));
}
// What the query at position p sees, in images: virtual image i is image i
// below `head`, else image tail + i - head.
struct Seen {
  int n, lo;  // visible: u < n and (u >= lo or u < first)
  int head, tail, images;
};
__device__ __forceinline__ Seen seen_of(const DecArgs& a, int p) {
  Seen s;
  s.n = min(p + 1, a.capacity);  // 0 for p = -1
  s.lo = a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0;
  const int end = s.n / 16 + (s.n % 16 != 0);
  const int h = min(a.first, s.lo);
  s.tail = min(s.lo / 16, end);
  s.head = min(h / 16 + (h % 16 != 0), s.tail);
  s.images = s.head + (end - s.tail);
  return s;
}
__device__ __forceinline__ int units_of(const Seen& s) {
  return (s.images + kUnitTiles - 1) / kUnitTiles;
}

// The flat list of units: sequence b's units of head tile t start at
// head_tiles_all * first[b] + t * units(b).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {  // a 64-bit division takes 0.3 us
  return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}
__device__ __forceinline__ int64_t cta_first(int64_t U, int G, int i) { return quotient(U * i, G); }
__device__ __forceinline__ int cta_of(int64_t U, int G, int64_t u) {
  return (int)quotient((u + 1) * G - 1, U);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// What f16 leaves of a value below its normal range (0 for larger ones, whose
// 11 bits do).
__device__ __forceinline__ float f16_rest(float x) {
  return fabsf(x) < 0x1p-14f ? x - __half2float(__float2half_rn(x)) : 0.f;
}

// f16 pairs kept in registers (a logic instruction takes one immediate, the
// mask; the others would be fetched anew at each use).
struct Bases {
  uint32_t k1024, k64, m1032, m72;
};
__device__ __forceinline__ Bases bases() {
  Bases k{0x64006400u, 0x54005400u, 0xe408e408u, 0xd480d480u};
  asm volatile("" : "+r"(k.k1024), "+r"(k.k64), "+r"(k.m1032), "+r"(k.m72));
  return k;
}
// Scale bytes picked into the two halves -> (s, -72 s) 2^-8: an E4M3 byte
// shifted into an f16's exponent and mantissa reads as s 2^-8.
struct ScalePair {
  uint32_t s, n72;
};
__device__ __forceinline__ ScalePair scale_pair(uint32_t bytes, uint32_t sel, const Bases& k) {
  ScalePair p;
  p.s = __byte_perm(bytes, 0, sel) << 7;
  p.n72 = mul_f16x2(p.s, k.m72);
  return p;
}
// (w & kMask) | k as one lop3: 201 us, written as two operators 229.
template <uint32_t kMask>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t k) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "n"(kMask), "r"(k));
  return d;
}
// Nibbles j and j + 4 of w, j = 0 .. 3 -> s (n - 8) 2^-8 in the two halves.
__device__ __forceinline__ void widen4(uint32_t w, const ScalePair& s, const Bases& k,
                                       uint32_t (&v)[4]) {
  const uint32_t y = w >> 8;
  v[0] = mul_f16x2(add_f16x2(and_or<0x000f000fu>(w, k.k1024), k.m1032), s.s);
  v[1] = fma_f16x2(and_or<0x00f000f0u>(w, k.k64), s.s, s.n72);
  v[2] = mul_f16x2(add_f16x2(and_or<0x000f000fu>(y, k.k1024), k.m1032), s.s);
  v[3] = fma_f16x2(and_or<0x00f000f0u>(y, k.k64), s.s, s.n72);
}

// A piece's state per head: running maximum M of the logits (log2 units), sum
// L of 2^(l - M), and the reference MV of the output's weights.  The output is
// O times both factors (their product can leave fp32's range where the output
// does not).
__device__ __forceinline__ float2 out_factors(float M, float L, float MV, const float* sink, int head) {
  if (M == kNone) return make_float2(L == 0.f ? 0.f : L, 1.f);  // nothing seen: zeros (a NaN sum stays one)
  const float den = L + (sink != nullptr ? ex2(sink[head] * kLog2e - M) : 0.f);
  const float f = ex2(0.5f * (MV - M - (127.f - 8.f)));  // E's bias, and the scales' 2^-8
  return make_float2(f / den, f);
}

template <int C, int NT>
struct Cfg {
  static constexpr int kTB = kv4::tile_bytes(C);
  static constexpr int kStages = 2;  // image pairs in a warp's ring
  static constexpr int kStageBytes = kPair * kTB;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kLd = C + 4;  // padded row of the merge buffer (floats)
  static constexpr int kSlot = kHeads * C + 4 * kHeads;  // floats of a workspace slot
  static constexpr int off_merge() { return kWarps * kStages * kStageBytes; }
  static constexpr int off_ml() { return off_merge() + kWarps * kHeads * kLd * 4; }
  static constexpr int off_meta() { return off_ml() + kWarps * kHeads * 16; }
  static constexpr int off_bar() { return off_meta() + kWarps * kStages * kPair * 4; }
  static constexpr int off_list() { return off_bar() + kWarps * kStages * 8 + 64; }
  static size_t smem(int batch) { return off_list() + (size_t)(2 * batch + 1) * 4; }
};

template <int C, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 2) kv4_decode_kernel(const __grid_constant__ DecArgs a) {
  using F = Cfg<C, NT>;
  constexpr int D = C / 8;    // dims of a V chunk
  constexpr int KS = C / 16;  // k-steps of Q.K
  constexpr int MT = D / 2;   // m-tiles of P.V
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + F::off_merge());
  float4* ml = reinterpret_cast<float4*>(smem + F::off_ml());  // (M, L, MV, -)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * F::kStages * F::kStageBytes;
  int2* meta = reinterpret_cast<int2*>(smem + F::off_meta()) + warp * F::kStages;  // first tokens, or -1
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::off_bar()) + warp * F::kStages;
  int* scan = reinterpret_cast<int*>(smem + F::off_bar() + kWarps * F::kStages * 8);
  int* first_unit = reinterpret_cast<int*>(smem + F::off_list());  // [batch + 1]
  int* position = first_unit + a.batch + 1;                         // [batch]

  if (lane == 0) {
    for (int i = 0; i < F::kStages; ++i) mbar_init(&full[i], kPair);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();

  // units before each sequence
  {
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int p = b < a.batch ? clip_pos(a.pos[b]) : -1;
      const int u = units_of(seen_of(a, p));
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
      if (b < a.batch) {
        first_unit[b] = before + inc - u;
        position[b] = p;
      }
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
  int b;
  {
    int lo = 0, hi = a.batch;  // first_unit[lo] * HV <= u_lo < first_unit[hi] * HV
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)first_unit[mid] * HV <= u_lo) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  // a place in the unit list: unit s of the nu units of (sequence b, head tile hv)
  struct Place {
    int b, hv, s, nu;
  };
  auto next_segment = [&](Place& p) {
    p.s = 0;
    if (++p.hv == HV) {
      p.hv = 0;
      do { ++p.b; } while (p.b < a.batch && first_unit[p.b + 1] == first_unit[p.b]);
      p.nu = p.b < a.batch ? first_unit[p.b + 1] - first_unit[p.b] : 0;
    }
  };
  Place at;
  at.b = b;
  at.nu = first_unit[b + 1] - first_unit[b];
  {
    const int64_t off = u_lo - (int64_t)first_unit[b] * HV;
    at.hv = (int)quotient(off, at.nu);
    at.s = (int)(off - (int64_t)at.hv * at.nu);
  }
  const int units = (int)min(u_hi - u_lo, (int64_t)INT_MAX);

  // ---- this warp's images, looked up 16 units at a time: lane 2 i + k image
  // k of unit base + i (the block numbers are on their way until they are used)
  Place look = at;  // the first unit of the batch to come
  int look_unit = 0;
  int t0_c = -1, img_c = 0;                  // this batch: first token (-1: none), image number
  int tile_n = -1, blk_n = -1, row_n = 0;     // the next
  auto look_up = [&]() {
    t0_c = tile_n >= 0 && blk_n >= 0 && blk_n < a.num_blocks ? tile_n * 16 : -1;
    img_c = blk_n * a.nkv * a.tiles_per_block + row_n;
    tile_n = -1;
    if (look_unit >= units) return;
    Place p = look;
    if (look_unit + (lane >> 1) < units) {
      p.s += lane >> 1;
      while (p.s >= p.nu) {
        const int rest = p.s - p.nu;
        next_segment(p);
        p.s = rest;
      }
      const Seen v = seen_of(a, position[p.b]);
      const int i = p.s * kUnitTiles + 2 * warp + (lane & 1);
      if (i < v.images) {
        tile_n = i < v.head ? i : v.tail + (i - v.head);
        const int j = tile_n / a.tiles_per_block;
        row_n = (p.hv / a.head_tiles) * a.tiles_per_block + tile_n - j * a.tiles_per_block;
        blk_n = __ldg(a.table + p.b * a.max_blocks + j);
      }
    }
    look_unit += 16;
    if (look_unit < units) {
      look.s += 16;
      while (look.s >= look.nu) {
        const int rest = look.s - look.nu;
        next_segment(look);
        look.s = rest;
      }
    }
  };
  auto issue = [&](int u, int st) {  // the images of unit u into their stage, which is free
    if (u >= units) return;
    if ((u & 15) == 0 && u > 0) look_up();
    const int from = 2 * (u & 15) + (lane & 1);
    const int t0 = __shfl_sync(0xffffffffu, t0_c, from);
    const int img = __shfl_sync(0xffffffffu, img_c, from);
    if (lane < 2) {
      reinterpret_cast<int*>(&meta[st])[lane] = t0;
      if (t0 >= 0) {
        mbar_arrive_expect_tx(&full[st], F::kTB);
        bulk_load(ring + st * F::kStageBytes + lane * F::kTB, a.cache + (int64_t)img * F::kTB,
                  F::kTB, &full[st]);
      } else {
        mbar_arrive(&full[st]);
      }
    }
  };
  look_up();
  look_up();
  for (int u = 0; u < F::kStages; ++u) issue(u, u);

  // ============================== consumers ====================================
  const int gid = lane >> 2, tig = lane & 3;
  const int tok_a = 4 * (gid >> 1) + (gid & 1);  // token of slot gid; slot gid + 8: + 2
  for (int u = 0; u < units;) {
    const Seen v = seen_of(a, position[at.b]);
    const int seen_n = v.n, seen_lo = v.lo, seen_first = a.first;
    const int kvh = at.hv / a.head_tiles, h0 = (at.hv % a.head_tiles) * F::kHeads;
    const int cur_b = at.b;
    const bool starts = at.s == 0, at_first = u == 0;
    // queries as B fragments: head gid (+ 8 per n-tile), dims C / 4 tig ..,
    // scaled by a power of two per head
    uint32_t qf[NT][KS][2];
    float qfac[NT][2];  // of heads 2 tig, 2 tig + 1: scale * log2(e) * 2^8 over that power
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int hl = h0 + 8 * t + gid;
      const __nv_bfloat16* qp =
          a.q + ((int64_t)cur_b * a.nh + (int64_t)kvh * a.group + hl) * C + tig * (C / 4);
      uint4 raw[C / 32];
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < C / 32; ++w) {
        raw[w] = make_uint4(0, 0, 0, 0);
        if (hl < a.group) raw[w] = __ldg(reinterpret_cast<const uint4*>(qp) + w);
        top = max(top, kv4::top_bits(raw[w]));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(127 - exponent): the largest element becomes 1 .. 2 (a head of zeros
      // or with an element that is not finite stays as it is)
      const uint32_t e = top >> 23;
      const bool plain = e == 0 || e == 255;
      const float up = plain ? 1.f : __uint_as_float(e == 254 ? 1u << 22 : (254u - e) << 23);
      const float back = (plain ? 1.f : __uint_as_float(e << 23)) * (a.qscale * 256.f);
#pragma unroll
      for (int w = 0; w < C / 32; ++w) {
        const uint32_t r[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(r[i] << 16) * up;
          x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u) * up;
        }
        qf[t][2 * w][0] = pack_f16x2(x[0], x[4]);
        qf[t][2 * w][1] = pack_f16x2(x[1], x[5]);
        qf[t][2 * w + 1][0] = pack_f16x2(x[2], x[6]);
        qf[t][2 * w + 1][1] = pack_f16x2(x[3], x[7]);
      }
      qfac[t][0] = __shfl_sync(0xffffffffu, back, 8 * tig);
      qfac[t][1] = __shfl_sync(0xffffffffu, back, 8 * tig + 4);
    }
    float o[NT][MT][4];
    float m[NT][2], l[NT][2], mv[NT][2];
    float deep = kNone;  // rows with a smaller E: their weights' remainders count
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = mv[t][0] = mv[t][1] = kNone;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int k = 0; k < MT; ++k) o[t][k][0] = o[t][k][1] = o[t][k][2] = o[t][k][3] = 0.f;
    }

    const Bases k16 = bases();
    // Images 0 .. N - 1 of a stage, step by step for all of them, so that the
    // chains of one hide under the other's.
    auto images = [&](auto count, const uint8_t* im0, int t0a, int t0b) {
      constexpr int N = decltype(count)::value;
      const int t0[2] = {t0a, t0b};
      float sc[N][NT][4];
      uint32_t ex[N][2];
      // ---- S^T = K Q^T ----------------------------------------------------
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint8_t* im = im0 + n * F::kTB;
#pragma unroll
        for (int t = 0; t < NT; ++t) sc[n][t][0] = sc[n][t][1] = sc[n][t][2] = sc[n][t][3] = 0.f;
        uint32_t ka[C / 32], kb[C / 32];
        ScalePair sa[C / 64], sb[C / 64];
        if constexpr (C == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(im + gid * 64 + tig * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(im + (gid + 8) * 64 + tig * 16);
          ka[0] = x.x; ka[1] = x.y; ka[2] = x.z; ka[3] = x.w;
          kb[0] = y.x; kb[1] = y.y; kb[2] = y.z; kb[3] = y.w;
          const uint32_t p = *reinterpret_cast<const uint16_t*>(im + kv4::off_ks(C) + gid * 8 + 2 * tig);
          const uint32_t r = *reinterpret_cast<const uint16_t*>(im + kv4::off_ks(C) + (gid + 8) * 8 + 2 * tig);
          sa[0] = scale_pair(p, 0x4040, k16); sa[1] = scale_pair(p, 0x4141, k16);
          sb[0] = scale_pair(r, 0x4040, k16); sb[1] = scale_pair(r, 0x4141, k16);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(im + gid * 32 + tig * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(im + (gid + 8) * 32 + tig * 8);
          ka[0] = x.x; ka[1] = x.y;
          kb[0] = y.x; kb[1] = y.y;
          sa[0] = scale_pair(im[kv4::off_ks(C) + gid * 4 + tig], 0x4040, k16);
          sb[0] = scale_pair(im[kv4::off_ks(C) + (gid + 8) * 4 + tig], 0x4040, k16);
        }
        ex[n][0] = *reinterpret_cast<const uint16_t*>(im + kv4::off_exp(C) + 2 * gid);
        ex[n][1] = *reinterpret_cast<const uint16_t*>(im + kv4::off_exp(C) + 2 * gid + 16);
#pragma unroll
        for (int w = 0; w < C / 32; ++w) {
          uint32_t ra[4], rb[4];
          widen4(ka[w], sa[w / 2], k16, ra);
          widen4(kb[w], sb[w / 2], k16, rb);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_16816(sc[n][t], ra[0], rb[0], ra[1], rb[1], qf[t][2 * w][0], qf[t][2 * w][1]);
            mma_16816(sc[n][t], ra[2], rb[2], ra[3], rb[3], qf[t][2 * w + 1][0], qf[t][2 * w + 1][1]);
          }
        }
      }
      // ---- online softmax: l, and l + E of the value row ----------------------
      float lv[N][NT][4], ev[N][2];
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // slots gid, gid + 8
          const float kr = __uint_as_float((ex[n][r] & 255u) << 23);
          // E as a float; infinite for a row that is not finite (0 w then makes NaN)
          const float ve = ex[n][r] >= 0xff00u ? __int_as_float(0x7f800000) : (float)(ex[n][r] >> 8);
          ev[n][r] = ve;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float2 s = mul2(mul2(make_float2(sc[n][t][2 * r], sc[n][t][2 * r + 1]), make_float2(kr, kr)),
                                  make_float2(qfac[t][0], qfac[t][1]));
            const float2 y = add2(s, make_float2(ve, ve));
            sc[n][t][2 * r] = s.x;
            sc[n][t][2 * r + 1] = s.y;
            lv[n][t][2 * r] = y.x;
            lv[n][t][2 * r + 1] = y.y;
          }
        }
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (t0[n] + 15 >= seen_n || (t0[n] < seen_lo && t0[n] + 15 >= seen_first)) {  // some row is hidden
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int u1 = t0[n] + tok_a + 2 * r;
            if (!(u1 < seen_n && (u1 >= seen_lo || u1 < seen_first)))
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[n][t][2 * r + e] = lv[n][t][2 * r + e] = kNegInf;
          }
        }
      float tm[NT][2], tv[NT][2];
      bool grow = false, low = false;
#pragma unroll
      for (int n = 0; n < N; ++n) low |= fminf(ev[n][0], ev[n][1]) < deep;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tm[t][e] = fmaxf(sc[0][t][e], sc[0][t][2 + e]);
          tv[t][e] = fmaxf(lv[0][t][e], lv[0][t][2 + e]);
          if (N > 1) {
            tm[t][e] = fmaxf(tm[t][e], fmaxf(sc[N - 1][t][e], sc[N - 1][t][2 + e]));
            tv[t][e] = fmaxf(tv[t][e], fmaxf(lv[N - 1][t][e], lv[N - 1][t][2 + e]));
          }
          grow |= tm[t][e] > m[t][e] + kRescaleLog2 || tv[t][e] > mv[t][e] + kMostLog2;
        }
      // ---- O^T += V^T P^T of one image ------------------------------------------
      auto second_product = [&](const uint8_t* im, const uint32_t (&pb)[NT][2]) {
        const uint8_t* vim = im + kv4::off_v(C) + gid * 4 * D + tig * D;
        // (bytes of rows never written may be anything: kept finite, their weight is 0)
        const uint32_t vs = 0x7f7f7f7fu & *reinterpret_cast<const uint32_t*>(
            im + kv4::off_vs(C) + (C == 128 ? gid : gid >> 1) * 16 + 4 * tig);
        const ScalePair s0 = scale_pair(vs, 0x4140, k16), s1 = scale_pair(vs, 0x4342, k16);
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
          uint32_t a0[4], a1[4];
          widen4(x0[w], s0, k16, a0);
          widen4(x1[w], s1, k16, a1);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_16816(o[t][2 * w], a0[0], a0[1], a1[0], a1[1], pb[t][0], pb[t][1]);
            mma_16816(o[t][2 * w + 1], a0[2], a0[3], a1[2], a1[3], pb[t][0], pb[t][1]);
          }
        }
      };
      if (__any_sync(0xffffffffu, grow || low)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = tm[t][e], y = tv[t][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) {
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
            }
            x = fmaxf(x, m[t][e]);
            y = fmaxf(y - kTopLog2, mv[t][e]);
            if (x > m[t][e]) l[t][e] *= ex2(m[t][e] - x);
            m[t][e] = x;
            if (y > mv[t][e]) {
              const float f = ex2(mv[t][e] - y);
              mv[t][e] = y;
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                o[t][k][e] *= f;
                o[t][k][2 + e] *= f;
              }
            }
          }
        deep = kNone;  // (heads that are not finite have no say)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = mv[t][e] - m[t][e] + (kTopLog2 - kDeepLog2);
            if (d < 512.f) deep = fmaxf(deep, d);
          }
#pragma unroll
        for (int w = 1; w < 4; w <<= 1) deep = fmaxf(deep, __shfl_xor_sync(0xffffffffu, deep, w));
        // a row that is seen, far below in E, whose weight is an f16 subnormal?
        low = false;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (ev[n][r] < deep)
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float x = lv[n][t][2 * r + e] - mv[t][e];
                  low |= x < -14.f && x > -14.f - 26.f * kDeepSteps - 4.f;
                }
        if (__any_sync(0xffffffffu, low)) {
#pragma unroll 1
          for (int n = 0; n < N; ++n) {
            float w[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[t][i] = f16_rest(ex2((n == 0 ? lv[0][t][i] : lv[N - 1][t][i]) - mv[t][i & 1]));
#pragma unroll 1
            for (int step = 0; step < kDeepSteps; ++step) {
              uint32_t pb[NT][2];
#pragma unroll
              for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int k = 0; k < MT; ++k)
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[t][k][i] *= 0x1p26f;
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  x[i] = w[t][i] * 0x1p26f;  // 2 at most
                  w[t][i] = f16_rest(x[i]);
                }
                pb[t][0] = transpose8x8(pack_f16x2(x[0], x[1]));
                pb[t][1] = transpose8x8(pack_f16x2(x[2], x[3]));
              }
              second_product(im0 + n * F::kTB, pb);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][k][i] *= 0x1p-78f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[t][e] += ex2(sc[n][t][e] - m[t][e]) + ex2(sc[n][t][2 + e] - m[t][e]);
            w[e] = ex2(lv[n][t][e] - mv[t][e]);
            w[2 + e] = ex2(lv[n][t][2 + e] - mv[t][e]);
          }
          pb[t][0] = transpose8x8(pack_f16x2(w[0], w[1]));
          pb[t][1] = transpose8x8(pack_f16x2(w[2], w[3]));
        }
        second_product(im0 + n * F::kTB, pb);
      }
    };

    for (; at.s < at.nu && u < units; ++at.s, ++u) {
      const int st = u % F::kStages;
      mbar_wait(&full[st], (uint32_t)((u / F::kStages) & 1), a.err);
      const int2 t0 = meta[st];
      const uint8_t* im = ring + st * F::kStageBytes;
      if (t0.x >= 0 && t0.y >= 0) {
        images(std::integral_constant<int, 2>(), im, t0.x, t0.y);
      } else if (t0.x >= 0 || t0.y >= 0) {  // the end of what is seen, or an absent block
        images(std::integral_constant<int, 1>(), im + (t0.x >= 0 ? 0 : F::kTB), max(t0.x, t0.y), -1);
      }
      __syncwarp();
      issue(u + F::kStages, st);
    }
    const bool ends = at.s == at.nu;
    if (ends) next_segment(at);

    // ---- merge the warps ---------------------------------------------------
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        const int hl = 8 * t + 2 * tig + e;
        if (gid == 0) ml[warp * F::kHeads + hl] = make_float4(m[t][e], x, mv[t][e], 0.f);
        float* row = merge + (warp * F::kHeads + hl) * F::kLd + gid * D;
#pragma unroll
        for (int k = 0; k < MT; ++k)
          *reinterpret_cast<float2*>(row + 2 * k) = make_float2(o[t][k][e], o[t][k][2 + e]);
      }
    named_bar_or(1, kThreads, false);
    const bool direct = starts && ends;
    float* slot = a.ws + ((int64_t)blockIdx.x * 2 + (at_first ? 0 : 1)) * F::kSlot;
    for (int e = threadIdx.x; e < F::kHeads * (C / 4); e += kThreads) {
      const int hl = e / (C / 4), d = (e % (C / 4)) * 4;
      float M = kNone, MV = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M = fmaxf(M, ml[w * F::kHeads + hl].x);
        MV = fmaxf(MV, ml[w * F::kHeads + hl].z);
      }
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = ml[w * F::kHeads + hl];
        const float f = ex2(x.z - MV);
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * F::kHeads + hl) * F::kLd + d);
        L = fmaf(x.y, ex2(x.x - M), L);
        acc.x = fmaf(y.x, f, acc.x);
        acc.y = fmaf(y.y, f, acc.y);
        acc.z = fmaf(y.z, f, acc.z);
        acc.w = fmaf(y.w, f, acc.w);
      }
      if (direct) {
        if (h0 + hl < a.group) {
          const int head = kvh * a.group + h0 + hl;
          const float2 f = out_factors(M, L, MV, a.sink, head);
          uint2 w;
          w.x = pack_bf16x2(acc.x * f.x * f.y, acc.y * f.x * f.y);
          w.y = pack_bf16x2(acc.z * f.x * f.y, acc.w * f.x * f.y);
          *reinterpret_cast<uint2*>(a.out + ((int64_t)cur_b * a.nh + head) * C + d) = w;
        }
      } else {
        *reinterpret_cast<float4*>(slot + hl * C + d) = acc;
        if (d == 0) *reinterpret_cast<float4*>(slot + F::kHeads * C + 4 * hl) = make_float4(M, L, MV, 0.f);
      }
    }
    named_bar_or(1, kThreads, false);
  }
  // after a wait that gave up, copies may still be on their way in
  for (int u = max(0, units - F::kStages); u < units; ++u)
    mbar_wait(&full[u % F::kStages], (uint32_t)((u / F::kStages) & 1), a.err, false);
}

// One block per (sequence, head tile): merges the pieces that lie in more
// than one CTA's share, and zeroes the output of sequences that see nothing.
template <int C, int NT>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const __grid_constant__ DecArgs a, int grid) {
  using F = Cfg<C, NT>;
  __shared__ long long part[2][8];
  const int HV = a.nkv * a.head_tiles;
  const int b = blockIdx.x / HV, hv = blockIdx.x % HV;
  const int kvh = hv / a.head_tiles, h0 = (hv % a.head_tiles) * F::kHeads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long before = 0, all = 0;
  for (int i = threadIdx.x; i < a.batch; i += 256) {
    const int u = units_of(seen_of(a, clip_pos(a.pos[i])));
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
  const int nu = units_of(seen_of(a, clip_pos(a.pos[b])));
  const int64_t U = (int64_t)all * HV;
  const int G = (int)min((int64_t)grid, U);
  const int64_t u0 = (int64_t)before * HV + (int64_t)hv * nu, u1 = u0 + nu;
  const int i0 = nu > 0 ? cta_of(U, G, u0) : 0, i1 = nu > 0 ? cta_of(U, G, u1 - 1) : 0;
  // (the positions above are older than the kernel before, which let this one
  // start only after its own wait).  Blocks with nothing to merge wait as well:
  // what follows in the stream is ordered behind this kernel alone.
  pdl_wait();
  if (nu > 0 && i0 == i1) return;  // written by the CTA itself
  for (int e = threadIdx.x; e < F::kHeads * (C / 4); e += 256) {
    const int hl = e / (C / 4), d = (e % (C / 4)) * 4;
    if (h0 + hl >= a.group) continue;
    const int head = kvh * a.group + h0 + hl;
    float M = kNone, L = 0.f, MV = kNone;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (nu > 0) {
#pragma unroll 4
      for (int i = i0; i <= i1; ++i) {
        const int which = i > i0 || cta_first(U, G, i) == u0 ? 0 : 1;
        const float* slot = a.ws + ((int64_t)i * 2 + which) * F::kSlot;
        const float4 x = *reinterpret_cast<const float4*>(slot + F::kHeads * C + 4 * hl);
        const float4 y = *reinterpret_cast<const float4*>(slot + hl * C + d);
        const float mn = fmaxf(M, x.x);
        L = L * ex2(M - mn) + x.y * ex2(x.x - mn);
        M = mn;
        const float vn = fmaxf(MV, x.z);
        const float f0 = ex2(MV - vn), f1 = ex2(x.z - vn);
        MV = vn;
        acc.x = acc.x * f0 + y.x * f1;
        acc.y = acc.y * f0 + y.y * f1;
        acc.z = acc.z * f0 + y.z * f1;
        acc.w = acc.w * f0 + y.w * f1;
      }
    }
    const float2 f = out_factors(M, L, MV, a.sink, head);
    uint2 w;
    w.x = pack_bf16x2(acc.x * f.x * f.y, acc.y * f.x * f.y);
    w.y = pack_bf16x2(acc.z * f.x * f.y, acc.w * f.x * f.y);
    *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.nh + head) * C + d) = w;
  }
}

// CTAs of the decode kernel, and the head tile (n-tiles of 8) for a group.
int dec_nt(int group) { return group <= 8 ? 1 : 2; }
int dec_grid(int group) { return sm_count() * (dec_nt(group) == 1 ? 4 : 2); }

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
  return (size_t)dec_grid(group) * 2 * (heads * c + 4 * heads) * 4;
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
  API_SUPPORTED(cache->num_blocks * cache->nkv <= INT_MAX / (cache->block_tokens / 16),
                "csa_kv4_decode_attn needs a pool of fewer than 2^31 / 16 tokens and heads");
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
  // (2^31 tokens at most; positions end one short of that)
  a.capacity = (int)std::min<int64_t>(cache->max_blocks * cache->block_tokens, INT_MAX);
  a.window = (int)std::min<int64_t>(window, INT_MAX);
  a.first = (int)std::min<int64_t>(first, INT_MAX);
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
