// Per-head RMSNorm of queries and keys with the position rotation, in one
// pass over both.  For each head row x (c dims) of a token:
//   y = x / sqrt(mean(x^2) + eps) * gamma        (gamma absent: y = x)
//   pair j of the trailing R dims turns by  pos[axis(j)] * base^(-2 j / R),
// pair j being dims (2j, 2j + 1) of those R dims, or (j, j + R/2) in the
// halves form; axis(j) is the section that j falls into (one position per
// axis: time, height, width).
//
// HBM-bound: every element is read and written once.  Kept in flight by bulk
// copies: each warp streams items (some heads of one token, up to kStageBytes)
// through a ring of its own in shared memory, works on them in place and
// sends them out by bulk stores, so loads, arithmetic and stores of several
// items overlap and no warp waits for another.  (With plain loads the four
// rows that a thread can hold left the kernel waiting on memory: 84 us where
// this takes 70 for 16384 tokens of 32 + 8 heads x 128.)
// A row is c / 16 lanes wide.  A lane holds two chunks of eight dims and with
// them both dims of each of its pairs: neighbouring chunks, or in the halves
// form chunks half the rotated dims apart, so that no value changes lanes.
// Where c or the rotated dims are not multiples of 16 the chunks are four
// dims, of c / 8 lanes.
// The angles depend on the token and the pair only: the warp forms them once
// per item in shared memory.  An angle is a 64-bit fixed-point fraction of a
// turn, pos times base^(-2j/R) / (2 pi) in units of 2^-64 modulo 1 (three
// integer products; positions of millions keep a float-accurate turn, and
// double precision took longer than the memory), then sincospi of its upper
// 32 bits.
#include <math.h>

#include "api_check.h"
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kMaxPairs = 256;
constexpr int kStageBytes = 4096;
constexpr int kBlocksPerSm = 4;

struct Turns {
  uint64_t f[kMaxPairs];  // 2^64 / (2 pi) * base^(-2j/R): the turn of pair j per position
};
struct QkArgs {
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_stride, k_stride, qo_stride, ko_stride;  // elements between tokens
  const float *q_gamma, *k_gamma;
  const int64_t* pos;  // [axes][tokens]
  unsigned int* err;
  int64_t tokens;
  int nh, nkv, c, R, gamma_ld;
  int lpr;                   // lanes per row
  int q_heads, k_heads;      // heads of an item of q, of k
  int q_items, parts;        // items of a token: of q, of both
  float eps;
  int end0, end1, end2;      // first pair of axis 1, 2, 3
};

// CH consecutive values in shared memory, as CH / 2 pairs.
template <typename T, int CH>
__device__ __forceinline__ void get_chunk(const T* p, float2* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < CH; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      v[i / 2] = make_float2(x.x, x.y);
      v[i / 2 + 1] = make_float2(x.z, x.w);
    }
  } else {
    uint32_t w[CH / 2];
    if constexpr (CH == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    }
#pragma unroll
    for (int i = 0; i < CH / 2; ++i)
      v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}
template <typename T, int CH>
__device__ __forceinline__ void put_chunk(T* p, const float2* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < CH / 2; i += 2)
      *reinterpret_cast<float4*>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
  } else {
    uint32_t w[CH / 2];
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) w[i] = pack_bf16x2(v[i].x, v[i].y);
    if constexpr (CH == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// An item: part `p` of token t's heads.  The warps step over the flat list of
// items without dividing: dt tokens and dp parts at a time.
struct Cursor {
  int64_t t;
  int p;
  __device__ void step(const QkArgs& a, int64_t dt, int dp) {
    t += dt;
    p += dp;
    if (p >= a.parts) {
      p -= a.parts;
      ++t;
    }
  }
  __device__ bool is_q(const QkArgs& a) const { return p < a.q_items; }
  __device__ int head0(const QkArgs& a) const {
    return is_q(a) ? p * a.q_heads : (p - a.q_items) * a.k_heads;
  }
  __device__ int heads(const QkArgs& a) const {
    return is_q(a) ? min(a.q_heads, a.nh - head0(a)) : min(a.k_heads, a.nkv - head0(a));
  }
};

template <typename T, int CH, bool kHalves, int kPairsPerLane>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) qk_norm_rope_kernel(
    const __grid_constant__ QkArgs a, const __grid_constant__ Turns turns) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full_bar[kWarps][kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = a.R >> 1, lead = a.c - a.R;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  float2* cs_tab = reinterpret_cast<float2*>(smem + kWarps * kStages * kStageBytes) + warp * half;
  uint64_t* full = full_bar[warp];
  const int64_t w0 = (int64_t)blockIdx.x * kWarps + warp, step = (int64_t)gridDim.x * kWarps;
  const int64_t dt = step / a.parts;
  const int dp = (int)(step - dt * a.parts);
  Cursor cur{w0 / a.parts, 0};
  cur.p = (int)(w0 - cur.t * a.parts);
  Cursor ahead = cur;  // the next item to be loaded
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  auto load = [&](int s) {  // lane 0
    if (ahead.t >= a.tokens) return;
    const int head0 = ahead.head0(a);
    const T* src = ahead.is_q(a) ? (const T*)a.q + ahead.t * a.q_stride
                                 : (const T*)a.k + ahead.t * a.k_stride;
    const uint32_t bytes = (uint32_t)(ahead.heads(a) * a.c * (int)sizeof(T));
    mbar_arrive_expect_tx(&full[s], bytes);
    bulk_load(ring + s * kStageBytes, src + (int64_t)head0 * a.c, bytes, &full[s]);
    ahead.step(a, dt, dp);
  };
  if (lane == 0)
    for (int s = 0; s < kStages - 1; ++s) load(s);

  // this lane's place in a row
  const int sub = lane & (a.lpr - 1);
  const bool on = sub * 2 * CH < a.c;
  int off[2], j[2];  // chunk dims and first pairs (j[1]: the second half of the lane's pairs)
  bool turned[2];
  if (kHalves && sub * 2 * CH < a.R) {
    off[0] = lead + sub * CH;
    off[1] = off[0] + half;
    turned[0] = turned[1] = on;
    j[0] = sub * CH;
    j[1] = j[0] + CH / 2;
  } else {
    off[0] = sub * 2 * CH - (kHalves ? a.R : 0);
    off[1] = off[0] + CH;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      turned[i] = on && !kHalves && off[i] >= lead;
      j[i] = (off[i] - lead) >> 1;
    }
  }
  // the pairs whose angles this lane forms: lane + 32 i
  uint64_t f[kPairsPerLane];
  const int64_t* pos[kPairsPerLane];
  int64_t p_next[kPairsPerLane];
#pragma unroll
  for (int i = 0; i < kPairsPerLane; ++i) {
    const int jj = lane + 32 * i;
    f[i] = 0;
    pos[i] = a.pos;
    p_next[i] = 0;
    if (jj < half) {
      f[i] = turns.f[jj];
      pos[i] = a.pos + ((jj >= a.end0) + (jj >= a.end1) + (jj >= a.end2)) * a.tokens;
      if (cur.t < a.tokens) p_next[i] = pos[i][cur.t];
    }
  }
  const float inv_c = 1.f / (float)a.c;
  const int rpp = 32 / a.lpr, row0 = lane / a.lpr;

  for (int n = 0; cur.t < a.tokens; ++n) {
    const int s = n % kStages;
    const Cursor x = cur;
    cur.step(a, dt, dp);
    const bool is_q = x.is_q(a);
    const int head0 = x.head0(a), heads = x.heads(a);
    const float* gamma = is_q ? a.q_gamma : a.k_gamma;
    float2 g[CH];
    auto load_gamma = [&](const float* p) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < CH; e += 4)
          *reinterpret_cast<float4*>(g + (CH * i + e) / 2) =
              __ldg(reinterpret_cast<const float4*>(p + off[i] + e));
    };
#pragma unroll
    for (int e = 0; e < CH; ++e) g[e] = make_float2(1.f, 1.f);
    if (gamma != nullptr && on && row0 < heads)
      load_gamma(gamma + (int64_t)(head0 + row0) * a.gamma_ld);
    // ---- angles of the token (its positions were loaded an item ago) ----
#pragma unroll
    for (int i = 0; i < kPairsPerLane; ++i) {
      const int jj = lane + 32 * i;
      if (32 * i >= half) break;
      const int u = (int)(((uint64_t)p_next[i] * f[i]) >> 32);  // turns in units of 2^-32
      float sn, cs;
      sincospif((float)u * 0x1p-31f, &sn, &cs);
      if (jj < half) cs_tab[jj] = make_float2(cs, sn);
    }
    if (cur.t < a.tokens)
#pragma unroll
      for (int i = 0; i < kPairsPerLane; ++i)
        if (lane + 32 * i < half) p_next[i] = pos[i][cur.t];
    __syncwarp();
    // y_a = x_a ca - x_b sb, y_b = x_a sa + x_b cb of a pair (a, b), a weight
    // shared by the heads folded in; in the halves form ca[i] and the others
    // hold pairs 2 i and 2 i + 1, else pair 2 i in .x and 2 i + 1 in .y as well
    float2 ca[CH / 2], sb[CH / 2], sa[CH / 2], cb[CH / 2];
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) {
      const int h = i / (CH / 4), e = 2 * (i % (CH / 4));
      if (turned[h]) {
        const float2 w0 = cs_tab[j[h] + e], w1 = cs_tab[j[h] + e + 1];  // (cos, sin)
        float2 ga = kHalves ? g[i] : make_float2(g[2 * i].x, g[2 * i + 1].x);
        float2 gb = kHalves ? g[CH / 2 + i] : make_float2(g[2 * i].y, g[2 * i + 1].y);
        if (a.gamma_ld != 0) ga = gb = make_float2(1.f, 1.f);
        ca[i] = make_float2(ga.x * w0.x, ga.y * w1.x);
        sa[i] = make_float2(ga.x * w0.y, ga.y * w1.y);
        cb[i] = make_float2(gb.x * w0.x, gb.y * w1.x);
        sb[i] = make_float2(-gb.x * w0.y, -gb.y * w1.y);
      }
    }
    mbar_wait(&full[s], (uint32_t)((n / kStages) & 1), a.err);
    T* rows = reinterpret_cast<T*>(ring + s * kStageBytes);
    for (int r0 = 0; r0 < heads; r0 += rpp) {
      const int r = r0 + row0;
      const bool mine = on && r < heads;
      T* row = rows + r * a.c;
      float2 v[CH];
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] = make_float2(0.f, 0.f);
      if (mine) {
        get_chunk<T, CH>(row + off[0], v);
        get_chunk<T, CH>(row + off[1], v + CH / 2);
      }
      if (gamma != nullptr) {
        float2 s0 = mul2(v[0], v[0]), s1 = mul2(v[1], v[1]);
#pragma unroll
        for (int e = 2; e < CH; e += 2) {
          s0 = fma2(v[e], v[e], s0);
          s1 = fma2(v[e + 1], v[e + 1], s1);
        }
        s0 = add2(s0, s1);
        float ss = s0.x + s0.y;
        for (int o = a.lpr >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(fmaf(ss, inv_c, a.eps));
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] = mul2(v[e], make_float2(inv, inv));
        if (a.gamma_ld != 0) {
#pragma unroll
          for (int e = 0; e < CH; ++e) v[e] = mul2(v[e], g[e]);
          if (on && r + rpp < heads)  // the next row's weights, under this one's rest
            load_gamma(gamma + (int64_t)(head0 + r + rpp) * a.gamma_ld);
        }
      }
      if (kHalves) {
        if (turned[0]) {
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            const float2 xa = v[i], xb = v[CH / 2 + i];
            v[i] = fma2(xa, ca[i], mul2(xb, sb[i]));
            v[CH / 2 + i] = fma2(xa, sa[i], mul2(xb, cb[i]));
          }
        } else if (a.gamma_ld == 0) {
#pragma unroll
          for (int e = 0; e < CH; ++e) v[e] = mul2(v[e], g[e]);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (turned[h]) {
#pragma unroll
            for (int i = h * (CH / 4); i < (h + 1) * (CH / 4); ++i) {
              const float2 x = v[2 * i], y = v[2 * i + 1];
              v[2 * i] = make_float2(x.x * ca[i].x + x.y * sb[i].x, x.x * sa[i].x + x.y * cb[i].x);
              v[2 * i + 1] = make_float2(y.x * ca[i].y + y.y * sb[i].y, y.x * sa[i].y + y.y * cb[i].y);
            }
          } else if (a.gamma_ld == 0) {
#pragma unroll
            for (int e = h * (CH / 2); e < (h + 1) * (CH / 2); ++e) v[e] = mul2(v[e], g[e]);
          }
        }
      }
      if (mine) {
        put_chunk<T, CH>(row + off[0], v);
        put_chunk<T, CH>(row + off[1], v + CH / 2);
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      T* dst = is_q ? (T*)a.q_out + x.t * a.qo_stride : (T*)a.k_out + x.t * a.ko_stride;
      bulk_store(dst + (int64_t)head0 * a.c, rows, (uint32_t)(heads * a.c * (int)sizeof(T)));
      bulk_commit_group();
      // the stage of the item before is free once its store (all but the
      // latest) has read it: the next load takes it
      bulk_wait_read<1>();
      load((n + kStages - 1) % kStages);
    }
    __syncwarp();
  }
  if (lane == 0) bulk_wait_all();
}

template <typename T, int CH, int kPairsPerLane>
cudaError_t launch_p(QkArgs a, const Turns& turns, bool halves, cudaStream_t s) {
  a.lpr = 1;
  while (a.lpr * 2 * CH < a.c) a.lpr <<= 1;
  // heads per item: what a stage holds, less where that leaves SMs without
  // work, never less than one step of the warp
  const int most = std::max(1, kStageBytes / (a.c * (int)sizeof(T))), least = 32 / a.lpr;
  const int64_t want = 2 * (int64_t)sm_count() / a.tokens;
  auto split = [&](int heads) {
    if (heads == 0) return 1;
    const int64_t items = std::max<int64_t>((heads + most - 1) / most,
                                            std::min<int64_t>((heads + least - 1) / least, want));
    return (int)((heads + items - 1) / items);
  };
  a.q_heads = split(a.nh);
  a.k_heads = split(a.nkv);
  a.q_items = (a.nh + a.q_heads - 1) / a.q_heads;
  a.parts = a.q_items + (a.nkv + a.k_heads - 1) / a.k_heads;
  const int64_t blocks = std::min<int64_t>((a.tokens * a.parts + kWarps - 1) / kWarps,
                                           (int64_t)sm_count() * kBlocksPerSm);
  const size_t smem = kWarps * (kStages * (size_t)kStageBytes + (size_t)(a.R / 2) * sizeof(float2));
  auto kern = halves ? qk_norm_rope_kernel<T, CH, true, kPairsPerLane>
                     : qk_norm_rope_kernel<T, CH, false, kPairsPerLane>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
      kWarps * (kStages * kStageBytes + 32 * kPairsPerLane * (int)sizeof(float2)));
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)blocks, kThreads, smem, s>>>(a, turns);
  return cudaGetLastError();
}
template <typename T, int CH>
cudaError_t launch_t(const QkArgs& a, const Turns& turns, bool halves, cudaStream_t s) {
  return a.R <= 128 ? launch_p<T, CH, 2>(a, turns, halves, s) : launch_p<T, CH, kMaxPairs / 32>(a, turns, halves, s);
}

}  // namespace

}  // namespace csa

using namespace csa;

extern "C" csa_status csa_qk_norm_rope(const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, int64_t tokens, int nh, int nkv, int c,
                                       const int64_t* pos, const csa_qk_rope* p, csa_dtype dt,
                                       void* q_out, int64_t q_out_stride, void* k_out,
                                       int64_t k_out_stride, void* stream) {
  API_REQUIRE(api_valid_dt(dt), "dt must be CSA_F32 or CSA_BF16");
  API_REQUIRE(p != nullptr, "p is NULL");
  API_REQUIRE(tokens >= 0, "tokens must be >= 0");
  API_REQUIRE(nh >= 0 && nkv >= 0 && nh + nkv >= 1, "nh and nkv must be >= 0, and one of them >= 1");
  API_REQUIRE(c >= 8 && c % 8 == 0, "c must be a positive multiple of 8");
  API_REQUIRE(p->eps >= 0.f && p->eps < 3.4e38f, "eps must be finite and >= 0");
  API_REQUIRE(p->rope_dims >= 0 && p->rope_dims <= c && p->rope_dims % 8 == 0,
              "rope_dims must be a multiple of 8 in [0, c]");
  API_REQUIRE(p->rope_base > 1.f && p->rope_base < 3.4e38f, "rope_base must be finite and > 1");
  API_REQUIRE(p->per_head == 0 || p->per_head == 1, "per_head must be 0 or 1");
  API_REQUIRE(p->halves == 0 || p->halves == 1, "halves must be 0 or 1");
  API_REQUIRE(p->axes >= 1 && p->axes <= 4, "axes must be in [1, 4]");
  int sum = 0;
  for (int i = 0; i < p->axes; ++i) {
    API_REQUIRE(p->sections[i] >= 0 && p->sections[i] <= c, "sections must be >= 0");
    sum += p->sections[i];
  }
  API_REQUIRE(sum == p->rope_dims / 2, "the sections must add up to rope_dims / 2 pairs");
  API_SUPPORTED(c <= 512, "csa_qk_norm_rope needs c <= 512");
  API_SUPPORTED(c <= 256 || (c % 16 == 0 && (!p->halves || p->rope_dims % 16 == 0)),
                "c above 256 must be a multiple of 16, in the halves form rope_dims as well");
  API_SUPPORTED(nh <= 65536 && nkv <= 65536, "csa_qk_norm_rope needs nh and nkv <= 65536");
  API_SUPPORTED(tokens < ((int64_t)1 << 31), "csa_qk_norm_rope needs tokens < 2^31");
  const int64_t unit = dt == CSA_F32 ? 4 : 8;  // 16 bytes
  API_REQUIRE(nh == 0 || (q_stride >= (int64_t)nh * c && q_stride % unit == 0 &&
                          q_out_stride >= (int64_t)nh * c && q_out_stride % unit == 0),
              "q strides must be >= nh * c and whole 16-byte units");
  API_REQUIRE(nkv == 0 || (k_stride >= (int64_t)nkv * c && k_stride % unit == 0 &&
                           k_out_stride >= (int64_t)nkv * c && k_out_stride % unit == 0),
              "k strides must be >= nkv * c and whole 16-byte units");
  if (tokens == 0) return api_ok();
  if (nh > 0) {
    API_REQUIRE_PTR(q);
    API_REQUIRE_PTR(q_out);
    API_REQUIRE(q != q_out || q_stride == q_out_stride, "in place needs equal strides");
  }
  if (nkv > 0) {
    API_REQUIRE_PTR(k);
    API_REQUIRE_PTR(k_out);
    API_REQUIRE(k != k_out || k_stride == k_out_stride, "in place needs equal strides");
  }
  API_REQUIRE_OPT_PTR(p->q_gamma);
  API_REQUIRE_OPT_PTR(p->k_gamma);
  if (p->rope_dims > 0) API_REQUIRE_LIST(pos);
  QkArgs a;
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.q_stride = q_stride; a.k_stride = k_stride;
  a.qo_stride = q_out_stride; a.ko_stride = k_out_stride;
  a.q_gamma = p->q_gamma; a.k_gamma = p->k_gamma;
  a.pos = pos; a.tokens = tokens;
  a.nh = nh; a.nkv = nkv; a.c = c; a.R = p->rope_dims;
  a.gamma_ld = p->per_head ? c : 0;
  a.eps = p->eps;
  a.err = device_timeout_flag();
  if (a.err == nullptr) return set_last_error(CSA_ERR_CUDA, "csa_qk_norm_rope: no device flag");
  int ends[3], e = 0;
  for (int i = 0; i < 3; ++i) {
    if (i < p->axes) e += p->sections[i];
    ends[i] = i < p->axes - 1 ? e : 1 << 30;
  }
  a.end0 = ends[0]; a.end1 = ends[1]; a.end2 = ends[2];
  Turns turns;
  const double log_base = log2((double)p->rope_base);
  for (int j = 0; j < p->rope_dims / 2; ++j)
    turns.f[j] = (uint64_t)(0x1p64 / 6.283185307179586476925286766559 *
                            exp2(-2.0 * j / p->rope_dims * log_base));
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t r;
  const bool wide = c % 16 == 0 && (!p->halves || p->rope_dims % 16 == 0);
  if (dt == CSA_F32)
    r = wide ? launch_t<float, 8>(a, turns, p->halves != 0, s)
             : launch_t<float, 4>(a, turns, p->halves != 0, s);
  else
    r = wide ? launch_t<__nv_bfloat16, 8>(a, turns, p->halves != 0, s)
             : launch_t<__nv_bfloat16, 4>(a, turns, p->halves != 0, s);
  return api_cuda(r, "csa_qk_norm_rope");
}
