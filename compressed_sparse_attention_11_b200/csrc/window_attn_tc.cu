// Causal attention over a sliding window and a few first tokens on the
// tcgen05 tensor cores, keys and values apart (bf16 in and out, fp32
// accumulation), head dim C = 64 or 128, heads in groups of g = nh / nkv:
//   E_t = { u <= t : u > t - W or u < F },
//   out[t, h] = sum_u e^{l_u} v_u / (e^{sink_h} + sum_u e^{l_u}),  l_u = scale q_th . k_u.
//
// Tensor-bound for windows past a few hundred tokens (4 C g flops a visible
// pair against 2 C / g bytes).  A query tile is 128 rows: the g heads of one
// key/value head times TT = 128 / g consecutive tokens, so the heads of a
// group share every key tile and a tile's band of keys is W + TT - 1 wide,
// not W + 127.  A CTA (one per SM, persistent) takes pairs of neighbouring
// query tiles; while the softmax of one runs, the products of the other do:
//   S_q = Q_q K^T (M = 128 rows, N = 128 keys), O_q += P_q V (N = C dims).
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (C each); P takes its
// S's first 64 columns (bf16) and is the A operand of P.V from there.
//
// Key order: with F > 0 and the pair's window starting past F, the tile
// list starts with the F first tokens (rounded up to 8 rows) and goes on with
// the window without a gap, the mixed tile being fetched in 8-row boxes, so
// a few first tokens do not cost a tile of their own.  Virtual column
// v < F8 is token v (visible if v < F), v >= F8 token klo + v - F8.
//
// Softmax: one thread per row (two warpgroups, one per query tile), running
// maximum that moves only past 2^8 (the row of O is then rescaled in tensor
// memory), weights rounded to bf16 for the second product (whose operands have
// one type, that of the values; the sum takes them unrounded: outputs are 0.0022
// off the 64-bit result, where their own rounding alone makes 0.0017); the
// arithmetic runs on pairs (fma.f32x2).  The softmax warps
// take registers from the two others' warpgroup, so that a row of 128 scores
// stays in registers.
//
// What bounds it: a query tile's products of one key tile need the tensor cores
// for 1024 cycles and its 128 x 128 exponentials the special-function units
// for as many, so two query tiles could share 2048 cycles.  Its chain, though,
// is S -> softmax (2200 cycles: 300 to read S, 300 for the maximum, 1450 for
// exponentials that meet the other warpgroup's, 150 to store P) -> P.V -> next
// S (1700 with the wait for the other tile's products): 3900, as P lives in S's
// columns and the next S cannot start before P.V has read them (at C = 128
// tensor memory is full; at C = 64 128 columns are not used).  2 x 8192 tokens,
// 32 heads over 8, W = 1024, 4 first tokens, C = 128: 335 us in a sustained run
// (770 TFLOP/s under the power cap), 308 in a short one.
//
// A value that is not finite would reach the queries that a mask hides it from
// through 0 x inf in the second product.  Hidden keys exist only in the edge
// tiles of a query tile (the last ones, the lower end of the window, the first
// tokens).  Two warps that are idle otherwise look through the values of those
// before the product takes them, and set such values to zero; from then on the
// CTA's epilogues look them up again in global memory and add them to the rows
// that see them.  In the tiles between, every row sees every key, and the
// product itself gives the right infinity or NaN.  So the time is bounded by the
// edge tiles, whatever the window (8192 tokens, 32 over 8 heads x 128, W = 1024:
// 168 us; 381 with one infinite value, 2.5 ms where every value is NaN).  Finite
// values pay nothing (342 us for 2 x 8192 tokens, sustained, with the scan and
// without); a wait of the MMA warp for the copy beside the one for the scan cost 12.
#include "api_check.h"
#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"
#include "tc_attn_util.cuh"

namespace csa {

namespace {

using namespace sm100;

constexpr int kRows = 128, kKeys = 128;
constexpr int kSlab = kRows * 128;  // 16 KB: 128 rows x 64 dims
constexpr int kStages = 2;
constexpr int kSoftWarps = 8;  // two warpgroups
constexpr int kMmaWarp = kSoftWarps, kTmaWarp = kSoftWarps + 1;
constexpr int kScanWarp = kSoftWarps + 2, kScanWarps = 2;
constexpr int kThreads = (kScanWarp + kScanWarps) * 32;
// Registers a thread: 168 x 384 at launch, moved between the warpgroups:
// 208 x 256 + 88 x 128 = 168 x 384.
constexpr int kSoftRegs = 208, kOtherRegs = 88;
static_assert(kSoftRegs * 256 + kOtherRegs * 128 <= 168 * kThreads, "register split");
constexpr float kRescaleLog2 = 8.f;

struct WinArgs {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float* sink;
  __nv_bfloat16* out;
  unsigned int* err;
  int works;
  int nq, nk, window, first, nh, nkv, group, tt, pairs;
  float qs;  // |scale| log2(e), never 0
  int neg;   // the scale is negative
};

template <int C>
struct Cfg {
  static constexpr int kSlabs = C / 64;
  static constexpr int kTileBytes = kSlabs * kSlab;
  static constexpr int off_q = 0;
  static constexpr int off_k = off_q + 2 * kTileBytes;
  static constexpr int off_v = off_k + kStages * kTileBytes;
  static constexpr int off_e = off_v + kStages * kTileBytes;  // 2 x 16 KB epilogue staging
  static constexpr int off_bar = off_e + 2 * kSlab;
  static constexpr int smem = off_bar + 512 + 1024;
  static constexpr uint32_t col_s = 0, col_o = 256;
};

struct __align__(8) WinBars {
  uint64_t q_full[2], q_free[2];
  uint64_t k_full[kStages], k_free[kStages], v_full[kStages], v_free[kStages];
  uint64_t v_seen[kStages];  // the values have been looked through
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t wg[2];  // bounded barrier of the four warps of a warpgroup
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t odd;  // values of some edge tile were not finite and are zeros in shared memory
};

// One pair of query tiles and its list of key tiles.
struct Job {
  int b, h, i0;        // batch, key/value head, first query
  int t0, t1;          // positions of the pair's first and last query
  int klo, f8, tiles;  // see the head comment
  __device__ int base(int j) const { return klo - f8 + j * kKeys; }  // token of column 0 (window part)
};
__device__ __forceinline__ Job job_of(const WinArgs& a, int w) {
  Job j;
  const unsigned r = (unsigned)w / (unsigned)a.pairs;
  const int pair = w - (int)r * a.pairs;
  j.b = (int)(r / (unsigned)a.nkv);
  j.h = (int)r - j.b * a.nkv;
  j.i0 = pair * 2 * a.tt;
  j.t0 = a.nk - a.nq + j.i0;
  j.t1 = a.nk - a.nq + min(a.nq, j.i0 + 2 * a.tt) - 1;
  j.klo = max(0, j.t0 - a.window + 1);
  if (a.first >= j.klo) j.klo = 0;
  j.f8 = j.klo > 0 ? (a.first + 7) & ~7 : 0;
  j.tiles = (j.f8 + j.t1 - j.klo + kKeys) / kKeys;
  return j;
}
// First columns of tile tj that are visible as first tokens, whatever the row.
__device__ __forceinline__ int first_cols(const WinArgs& a, const Job& j, int tj) {
  return j.f8 > 0 ? a.first - tj * kKeys : a.first - j.base(tj);
}
__device__ __forceinline__ bool active(const WinArgs& a, const Job& j, int q) {
  return j.i0 + q * a.tt < a.nq;
}
// The key tiles that some row of query tile q sees: those below nf (first
// tokens) and w0 .. w1 (window).
struct Need {
  int nf, w0, w1;
  __device__ int begin() const { return nf > 0 ? 0 : w0; }
  __device__ bool has(int t) const { return (t < nf || t >= w0) && t <= w1; }
  __device__ int next(int t) const { return t + 1 >= nf && t + 1 < w0 ? w0 : t + 1; }
};
__device__ __forceinline__ Need need_of(const WinArgs& a, const Job& j, int q) {
  Need n;
  if (!active(a, j, q)) {
    n.nf = n.w0 = 0;
    n.w1 = -1;
    return n;
  }
  const int ta = j.t0 + q * a.tt, tb = min(ta + a.tt - 1, j.t1), v0 = j.klo - j.f8;
  n.w0 = max(0, ta - a.window + 1 - v0) / kKeys;
  n.w1 = (tb - v0) / kKeys;
  n.nf = j.f8 > 0 || j.klo == 0 ? min((a.first + kKeys - 1) / kKeys, n.w1 + 1) : 0;
  return n;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The edge tiles among those a query tile needs: from `causal` on keys lie behind
// a row's token, from `first` to `lower` before a row's window (the tiles below
// hold nothing but first tokens: none is hidden, so however many first tokens
// there are, the edge tiles are a few).
struct Edges {
  Need need;
  int causal, first, lower;
  __device__ bool has(int t) const { return need.has(t) && (t >= causal || (t >= first && t < lower)); }
};
__device__ __forceinline__ Edges edges_of(const WinArgs& a, const Job& j, int q) {
  const int ta = j.t0 + q * a.tt, tb = min(ta + a.tt - 1, j.t1), v0 = j.base(0);
  Edges e;
  e.need = need_of(a, j, q);
  e.causal = (ta - v0 + 1) / kKeys;
  e.first = a.first / kKeys;
  e.lower = (max(0, tb - a.window + 1 - v0) + kKeys - 1) / kKeys;
  return e;
}
// Largest magnitudes of the upper and lower bf16 values of four words.
__device__ __forceinline__ uint32_t tops(const uint4& x) {
  constexpr uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
}
__device__ __forceinline__ bool not_finite(uint32_t top) {
  return top >= 0x7f800000u || (top & 0xffffu) >= 0x7f80u;
}
// (rare) The values of the scanned tiles that are not finite, added to the
// output of this thread's row (position t) where the row sees them.  Every lane
// looks at 32 dims of one key; then all lanes take the keys that have such a
// value in turn.
template <int C>
__device__ __noinline__ void add_odd_values(const WinArgs& a, const Job& j, int q, int t, uint32_t o_addr) {
  const int lane = threadIdx.x & 31;
  const Need need = need_of(a, j, q);
  const Edges e0 = edges_of(a, j, 0), e1 = edges_of(a, j, 1);
  for (int tj = 0; tj < j.tiles; ++tj) {
    if (!need.has(tj) || !(e0.has(tj) || e1.has(tj))) continue;
#pragma unroll 1
    for (int d = 0; d < C; d += 32) {
      uint32_t o[32];
      tmem_ld32(o_addr + d, o);
      tmem_ld_wait();
#pragma unroll 1
      for (int i0 = 0; i0 < kKeys; i0 += 32) {
        const int col = tj * kKeys + i0 + lane;
        const int u = col < j.f8 ? col : j.klo + col - j.f8;
        uint32_t y[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k] = 0u;
        if (u < a.nk && !(col < j.f8 && u >= a.first)) {
          const uint4* x = reinterpret_cast<const uint4*>(
              a.v + ((int64_t)j.b * a.nk + u) * a.v_stride + (int64_t)j.h * C + d);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 z = __ldg(x + k);
            y[4 * k] = z.x; y[4 * k + 1] = z.y; y[4 * k + 2] = z.z; y[4 * k + 3] = z.w;
          }
        }
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) top = __vmaxu2(top, y[k] & 0x7fff7fffu);
        unsigned todo = __ballot_sync(0xffffffffu, not_finite(top));
        while (todo) {
          const int from = __ffs(todo) - 1;
          todo &= todo - 1;
          const int uu = __shfl_sync(0xffffffffu, u, from);
          const bool sees = uu <= t && (uu > t - a.window || uu < a.first);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint32_t w = __shfl_sync(0xffffffffu, y[k], from);
            const uint32_t lo = w << 16, hi = w & 0xffff0000u;
            if (sees && (lo & 0x7f800000u) == 0x7f800000u)
              o[2 * k] = __float_as_uint(__uint_as_float(o[2 * k]) + __uint_as_float(lo));
            if (sees && (hi & 0x7f800000u) == 0x7f800000u)
              o[2 * k + 1] = __float_as_uint(__uint_as_float(o[2 * k + 1]) + __uint_as_float(hi));
          }
        }
      }
      tmem_st32(o_addr + d, o);
      tmem_st_wait();
    }
  }
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1) window_attn_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k8,
    const __grid_constant__ CUtensorMap tm_v8, const __grid_constant__ CUtensorMap tm_o,
    const __grid_constant__ WinArgs a) {
  using F = Cfg<C>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  WinBars* bar = reinterpret_cast<WinBars*>(smem + F::off_bar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned int* err = a.err;
  if (flag_value(err) != 0) return;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->q_full[i], 1);
      mbar_init(&bar->q_free[i], 1);
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], 4);
      mbar_init(&bar->o_full[i], 1);
      mbar_init(&bar->o_free[i], 4);
      mbar_init(&bar->wg[i], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->k_full[i], 1);
      mbar_init(&bar->k_free[i], 1);
      mbar_init(&bar->v_full[i], 1);
      mbar_init(&bar->v_free[i], 1);
      mbar_init(&bar->v_seen[i], kScanWarps);
    }
    mbar_init(&bar->drain, 1);
    bar->odd = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bar->tmem_base, 512);
    tmem_relinquish();
  }
  // rows of the query tiles that no token fills stay zero
  for (int i = threadIdx.x; i < 2 * F::kTileBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + F::off_q)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;

  if (warp >= kSoftWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kTmaWarp) {
    // ================================ TMA producer ================================
    int n = 0;               // key tiles issued
    int nq[2] = {0, 0};      // query tiles issued
    bool ok = true;
    for (int w = blockIdx.x; w < a.works && ok; w += gridDim.x) {
      const Job jb = job_of(a, w);
      auto load_q = [&](int q) {
        if (!active(a, jb, q)) return;
        if (nq[q] > 0 && !mbar_wait(&bar->q_free[q], (uint32_t)((nq[q] - 1) & 1), err)) {
          ok = false;
          return;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar->q_full[q], (uint32_t)(a.tt * a.group * 128 * F::kSlabs));
          for (int s = 0; s < F::kSlabs; ++s)
            tma_load_4d(smem + F::off_q + q * F::kTileBytes + s * kSlab, &tm_q, &bar->q_full[q],
                        s * 64, jb.h * a.group, jb.i0 + q * a.tt, jb.b);
        }
        __syncwarp();
        ++nq[q];
      };
      auto load_tile = [&](int tj, int off, uint64_t* full, const CUtensorMap* m, const CUtensorMap* m8) {
        uint8_t* dst = smem + off;
        if (lane == 0) mbar_arrive_expect_tx(full, F::kTileBytes);
        __syncwarp();
        const int v0 = tj * kKeys;
        if (v0 < jb.f8 && v0 + kKeys > jb.f8) {  // first tokens, then the window: 8-row boxes
          if (lane < 16) {
            const int v = v0 + 8 * lane;
            const int u = v < jb.f8 ? v : jb.klo + v - jb.f8;
            for (int s = 0; s < F::kSlabs; ++s)
              tma_load_4d(dst + s * kSlab + lane * 1024, m8, full, s * 64, jb.h, u, jb.b);
          }
        } else if (lane == 0) {
          const int u = v0 < jb.f8 ? v0 : jb.base(tj);
          for (int s = 0; s < F::kSlabs; ++s)
            tma_load_4d(dst + s * kSlab, m, full, s * 64, jb.h, u, jb.b);
        }
        __syncwarp();
      };
      load_q(0);
      for (int tj = 0; tj < jb.tiles && ok; ++tj, ++n) {
        const int st = n % kStages;
        const uint32_t ph = (uint32_t)((n / kStages - 1) & 1);
        if (n >= kStages && !(ok = mbar_wait(&bar->k_free[st], ph, err))) break;
        load_tile(tj, F::off_k + st * F::kTileBytes, &bar->k_full[st], &tm_k, &tm_k8);
        if (tj == 0) {
          load_q(1);
          if (!ok) {  // the values of this tile will not come: it counts as not issued
            mbar_wait(&bar->k_full[st], (uint32_t)((n / kStages) & 1), err, false);
            break;
          }
        }
        if (n >= kStages && !(ok = mbar_wait(&bar->v_free[st], ph, err))) {
          mbar_wait(&bar->k_full[st], (uint32_t)((n / kStages) & 1), err, false);
          break;
        }
        load_tile(tj, F::off_v + st * F::kTileBytes, &bar->v_full[st], &tm_v, &tm_v8);
      }
    }
    // every load has landed before the CTA ends
    for (int i = n > kStages ? n - kStages : 0; i < n; ++i) {
      mbar_wait(&bar->k_full[i % kStages], (uint32_t)((i / kStages) & 1), err, false);
      mbar_wait(&bar->v_full[i % kStages], (uint32_t)((i / kStages) & 1), err, false);
    }
    for (int q = 0; q < 2; ++q)
      if (nq[q] > 0) mbar_wait(&bar->q_full[q], (uint32_t)((nq[q] - 1) & 1), err, false);
  } else if (warp == kMmaWarp) {
    // ================================ MMA issuer ==================================
    constexpr uint32_t kIdQK = idesc_bf16(kRows, kKeys, 0, 0);
    constexpr uint32_t kIdPV = idesc_bf16(kRows, C, 0, 1);
    // descriptors of stage / query tile 0; offsets in 16-byte units
    const uint32_t leader = lane == 0 ? 1u : 0u, tm = uniform(tmem);
    const uint32_t sm = uniform(smem_u32(smem));
    const DescWords dq(desc_sw128(sm + F::off_q)), dk(desc_sw128(sm + F::off_k)),
        dv(desc_sw128_mn(sm + F::off_v, kSlab, 1024));
    constexpr uint32_t kTile16 = F::kTileBytes / 16, kSlab16 = kSlab / 16;
    int n = 0;                             // key tiles of all jobs
    int pvs[2] = {0, 0}, jobs[2] = {0, 0};  // P.V issued, query tiles finished
    bool ok = true;
    // weights of key tile k (its values in stage k % kStages) into O_q
    auto issue_pv = [&](int q, int k, bool first, bool last) -> bool {
      const int st = k % kStages;
      if (!mbar_wait(&bar->v_seen[st], (uint32_t)((k / kStages) & 1), err)) return false;
      // the first P.V of a query tile overwrites O: the epilogue before has read it
      if (first && jobs[q] > 0 && !mbar_wait(&bar->o_free[q], (uint32_t)((jobs[q] - 1) & 1), err))
        return false;
      if (!mbar_wait(&bar->p_full[q], (uint32_t)(pvs[q] & 1), err)) return false;
      ++pvs[q];
      tc_fence_after();
      const uint32_t d = tm + F::col_o + q * C, p = tm + F::col_s + q * kKeys;
      const uint32_t v = dv.lo + uniform(st * kTile16), acc = uniform(first ? 0u : 1u);
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        mma_bf16_ts_w(leader, d, p + kk * 8, v + kk * 128, dv.hi, kIdPV, kk == 0 ? acc : 1u);
      if (last) {
        if (lane == 0) mma_commit(&bar->o_full[q]);
        ++jobs[q];
      }
      return true;
    };
    for (int w = blockIdx.x; w < a.works && ok; w += gridDim.x) {
      const Job jb = job_of(a, w);
      const Need need[2] = {need_of(a, jb, 0), need_of(a, jb, 1)};
      bool pend[2] = {false, false}, begun[2] = {false, false};
      for (int tj = 0; tj <= jb.tiles && ok; ++tj) {
        const int st = n % kStages;
        bool have_k = false;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (ok && pend[q]) {  // the tile before this one
            ok = issue_pv(q, n - 1, !begun[q], tj - 1 == need[q].w1);
            begun[q] = true;
          }
          pend[q] = tj < jb.tiles && need[q].has(tj);
          if (!ok || !pend[q]) continue;
          if (tj == need[q].begin() && !(ok = mbar_wait(&bar->q_full[q], (uint32_t)(jobs[q] & 1), err))) continue;
          if (!have_k && !(ok = mbar_wait(&bar->k_full[st], (uint32_t)((n / kStages) & 1), err))) continue;
          have_k = true;
          tc_fence_after();
          // (in order behind the P.V that reads the weights out of these columns)
          const uint32_t d = tm + F::col_s + q * kKeys;
          const uint32_t k0 = dk.lo + uniform(st * kTile16), qq = dq.lo + q * kTile16;
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk) {
            const uint32_t step = (kk >> 2) * kSlab16 + (kk & 3) * 2;
            mma_bf16_w(leader, d, qq + step, dq.hi, k0 + step, dk.hi, kIdQK, kk != 0 ? 1u : 0u);
          }
          if (lane == 0) {
            mma_commit(&bar->s_full[q]);
            if (tj == need[q].w1) mma_commit(&bar->q_free[q]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (tj > 0 && lane == 0) mma_commit(&bar->v_free[(n - 1) % kStages]);
        if (tj < jb.tiles) {
          // (a tile that no row needs was loaded all the same)
          if (!have_k && !(ok = mbar_wait(&bar->k_full[st], (uint32_t)((n / kStages) & 1), err) &&
                                mbar_wait(&bar->v_seen[st], (uint32_t)((n / kStages) & 1), err)))
            break;
          if (lane == 0) mma_commit(&bar->k_free[st]);
          ++n;
        }
        __syncwarp();
      }
    }
    if (lane == 0) mma_commit(&bar->drain);
    __syncwarp();
    mbar_wait(&bar->drain, 0, err, false);
  } else {
    // =================== values of the edge tiles, a half each ====================
    // (the MMA warp waits for every tile's scan before it frees the stage, so a
    // scan is never a phase behind)
    constexpr int kPer = F::kTileBytes / 16 / kScanWarps / 32;
    int n = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < a.works && ok; w += gridDim.x) {
      const Job jb = job_of(a, w);
      const Edges e0 = edges_of(a, jb, 0), e1 = edges_of(a, jb, 1);
      for (int tj = 0; tj < jb.tiles; ++tj, ++n) {
        const int st = n % kStages;
        if (!(ok = mbar_wait(&bar->v_full[st], (uint32_t)((n / kStages) & 1), err))) break;
        if (e0.has(tj) || e1.has(tj)) {
          uint4* x = reinterpret_cast<uint4*>(smem + F::off_v + st * F::kTileBytes) +
                     (warp - kScanWarp) * kPer * 32 + lane;
          uint32_t top = 0;
#pragma unroll 8
          for (int i = 0; i < kPer; ++i) top = __vmaxu2(top, tops(x[32 * i]));
          if (__any_sync(0xffffffffu, not_finite(top))) {
#pragma unroll 1
            for (int i = 0; i < kPer; ++i) {
              const uint4 y = x[32 * i];
              if (!not_finite(tops(y))) continue;
              uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((z[k] & 0x7f80u) == 0x7f80u) z[k] &= 0xffff0000u;
                if ((z[k] & 0x7f800000u) == 0x7f800000u) z[k] &= 0xffffu;
              }
              x[32 * i] = make_uint4(z[0], z[1], z[2], z[3]);
            }
            if (lane == 0) *(volatile uint32_t*)&bar->odd = 1u;
          }
        }
        fence_proxy_async();  // the MMA warp waits for this scan, not for the copy
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->v_seen[st]);
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ============================ softmax and epilogue ============================
    const int q = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_addr + F::col_s + q * kKeys;
    const uint32_t o_addr = tmem + lane_addr + F::col_o + q * C;
    const int tl = row / a.group, hl = row - tl * a.group;  // token and head of the row
    uint8_t* stage = smem + F::off_e + q * kSlab;
    int steps = 0, jobs = 0;
    uint32_t wg_phase = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < a.works && ok; w += gridDim.x) {
      const Job jb = job_of(a, w);
      const Need need = need_of(a, jb, q);
      if (need.w1 < 0) continue;
      const int ta = jb.t0 + q * a.tt, t = ta + tl;
      const int tb = min(ta + a.tt - 1, jb.t1);
      float m = kNegInf, l = 0.f;
      const int t_first = need.begin();  // (O is not yet written there)
      for (int tj = t_first; tj <= need.w1; tj = need.next(tj)) {
        if (!(ok = mbar_wait(&bar->s_full[q], (uint32_t)(steps & 1), err))) break;
        ++steps;
        tc_fence_after();
        float s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c)
          tmem_ld32(s_addr + c * 32, reinterpret_cast<uint32_t(&)[32]>(s[32 * c]));
        tmem_ld_wait();
        if (a.neg) {
#pragma unroll
          for (int i = 0; i < kKeys; ++i) s[i] = -s[i];
        }
        const int base = jb.base(tj);
        if (base + kKeys - 1 > ta) {  // keys behind a row's own token
          const int hi = t - base;
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if (i > hi) s[i] = kNegInf;
        }
        if (tb - a.window + 1 > base) {  // keys before a row's window that are no first tokens
          const int lo = t - a.window + 1 - base, fc = first_cols(a, jb, tj);
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if (i < lo && i >= fc) s[i] = kNegInf;
        }
        float mx[4] = {max3(s[0], s[1], s[2]), max3(s[3], s[4], s[5]), max3(s[6], s[7], s[8]),
                       max3(s[9], s[10], s[11])};
#pragma unroll
        for (int i = 12; i < kKeys - 4; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s[i], s[i + 1]);
        mx[0] = max3(mx[0], s[kKeys - 4], s[kKeys - 3]);
        mx[1] = max3(mx[1], s[kKeys - 2], s[kKeys - 1]);
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.qs;
        const bool grow = top > m + kRescaleLog2;
        if (__any_sync(0xffffffffu, grow)) {
          // O is complete up to the tile before: its P.V was issued before this S
          const float mn = grow ? top : m;
          const float f = grow ? ex2(m - mn) : 1.f;  // 0 for the first keys of a row
          if (tj != t_first) {
            l *= f;
#pragma unroll 1
            for (int c = 0; c < C / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_addr + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(o_addr + c * 32, o);
            }
            tmem_st_wait();
          }
          m = mn;
        }
        const float mr = m == kNegInf ? 0.f : m;
        const float2 qs2 = make_float2(a.qs, a.qs), mr2 = make_float2(-mr, -mr);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 x = fma2(make_float2(s[64 * c + 2 * i], s[64 * c + 2 * i + 1]), qs2, mr2);
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            ls[i & 1] = add2(ls[i & 1], p);
            pk[i] = pack_bf16x2(p.x, p.y);
          }
          tmem_st32(s_addr + c * 32, pk);
        }
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->p_full[q]);
      }
      if (!ok) break;
      // ---- out = O / (sum + 2^(sink - m)) ------------------------------------------
      if (!(ok = mbar_wait(&bar->o_full[q], (uint32_t)(jobs & 1), err))) break;
      ++jobs;
      tc_fence_after();
      const int head = jb.h * a.group + hl;
      const int i = jb.i0 + q * a.tt + tl;
      const bool real = tl < a.tt && i < a.nq;
      const float mr = m == kNegInf ? 0.f : m;
      const float z = real && a.sink != nullptr ? a.sink[head] * kLog2e : kNegInf;
      const float inv = 1.f / (l + ex2(z - mr));
      if (*(const volatile uint32_t*)&bar->odd != 0) add_odd_values<C>(a, jb, q, t, o_addr);
#pragma unroll 1
      for (int sl = 0; sl < F::kSlabs; ++sl) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t o[32];
          tmem_ld32(o_addr + sl * 64 + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float x = __uint_as_float(o[e]) * inv, y = __uint_as_float(o[e + 1]) * inv;
            pk[16 * c + (e >> 1)] = pack_bf16x2(x, y);
          }
        }
        if (sl == F::kSlabs - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->o_free[q]);
        }
        // the slab before has left the staging buffer (its store was issued by
        // the warpgroup's first thread)
        if (row == 0) bulk_wait_read();
        if (!(ok = group_sync(&bar->wg[q], wg_phase, err))) break;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(stage + row * 128 + ((c ^ (row & 7)) * 16)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        fence_proxy_async();
        if (!(ok = group_sync(&bar->wg[q], wg_phase, err))) break;
        if (row == 0) {
          tma_store_4d(&tm_o, stage, sl * 64, jb.h * a.group, jb.i0 + q * a.tt, jb.b);
          bulk_commit_group();
        }
      }
    }
    if (row == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int C>
cudaError_t launch_c(WinArgs a, int64_t batch, cudaStream_t s) {
  using F = Cfg<C>;
  CUtensorMap mq, mk, mv, mk8, mv8, mo;
  const uint64_t nq = a.nq, nk = a.nk, nh = a.nh, nkv = a.nkv, B = batch;
  const uint64_t dq[4] = {C, nh, nq, B}, dk[4] = {C, nkv, nk, B};
  const uint64_t qs = 2 * (uint64_t)a.q_stride, ks = 2 * (uint64_t)a.k_stride,
                 vs = 2 * (uint64_t)a.v_stride, os = 2 * nh * C;
  const uint32_t bq[4] = {64, (uint32_t)a.group, (uint32_t)a.tt, 1}, bk[4] = {64, 1, kKeys, 1},
                 b8[4] = {64, 1, 8, 1};
  if (!make_tmap_bf16_4d(&mq, a.q, dq, {2 * C, qs, qs * nq}, bq) ||
      !make_tmap_bf16_4d(&mo, a.out, dq, {2 * C, os, os * nq}, bq) ||
      !make_tmap_bf16_4d(&mk, a.k, dk, {2 * C, ks, ks * nk}, bk) ||
      !make_tmap_bf16_4d(&mv, a.v, dk, {2 * C, vs, vs * nk}, bk) ||
      !make_tmap_bf16_4d(&mk8, a.k, dk, {2 * C, ks, ks * nk}, b8) ||
      !make_tmap_bf16_4d(&mv8, a.v, dk, {2 * C, vs, vs * nk}, b8))
    return cudaErrorInvalidValue;
  auto kern = window_attn_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<int64_t>(a.works, sm_count());
  kern<<<grid, kThreads, F::smem, s>>>(mq, mk, mv, mk8, mv8, mo, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_attn_tc(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, int64_t window, int64_t first,
                                  const float* sink, float scale, int64_t batch, int64_t n_q,
                                  int64_t n_k, int nh, int nkv, int c, void* out,
                                  unsigned int* err, cudaStream_t s) {
  WinArgs a;
  a.q = (const __nv_bfloat16*)q;
  a.k = (const __nv_bfloat16*)k;
  a.v = (const __nv_bfloat16*)v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.sink = sink;
  a.out = (__nv_bfloat16*)out;
  a.err = err;
  a.nq = (int)n_q;
  a.nk = (int)n_k;
  a.window = (int)std::min(window, n_k);
  a.first = (int)std::min(first, n_k);
  a.nh = nh;
  a.nkv = nkv;
  a.group = nh / nkv;
  a.tt = kRows / a.group;
  a.pairs = (int)((n_q + 2 * a.tt - 1) / (2 * a.tt));
  a.works = (int)((int64_t)a.pairs * nkv * batch);
  a.neg = scale < 0.f;
  // a scale of 0 weighs every visible key alike, as does this
  a.qs = std::max(std::abs(scale) * kLog2e, 1e-30f);
  return c == 128 ? launch_c<128>(a, batch, s) : launch_c<64>(a, batch, s);
}

}  // namespace csa
