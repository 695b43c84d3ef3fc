// Per-head RMSNorm of queries and keys with the position rotation, in one
// pass over both.  For each head row x (c dims) of a token:
//   y = x / sqrt(mean(x^2) + eps) * gamma        (gamma absent: y = x)
//   pair j of the trailing R dims turns by  pos[axis(j)] * base^(-2 j / R),
// pair j being dims (2j, 2j + 1) of those R dims, or (j, j + R/2) in the
// halves form; axis(j) is the section that j falls into (one position per
// axis: time, height, width).
//
// HBM-bound: every element is read and written once.  A row is spread over
// c / 8 lanes (c / 16 above 256 dims), one 16-byte load a lane, and each
// thread has kRows rows in flight.  The angles depend on the token and the
// pair only, so a block forms the cosines and sines of its tokens once in
// shared memory and all heads of those tokens use them: pos * theta / 2 pi
// in double precision, less its nearest integer (positions of millions keep
// a float-accurate turn), then sincospi in single precision.  theta is a
// kernel parameter, formed on the host.
#include <math.h>

#include "api_check.h"
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 256;

struct Turns {
  double per_pos[kMaxPairs];  // turns per position of pair j: base^(-2j/R) / (2 pi)
};
struct QkArgs {
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_stride, k_stride, qo_stride, ko_stride;  // elements between tokens
  const float *q_gamma, *k_gamma;
  const int64_t* pos;  // [axes][tokens]
  int64_t tokens;
  int nh, nkv, c, R, gamma_ld;
  float eps;
  int end0, end1, end2;  // first pair of axis 1, 2, 3
};

// VPL values per lane, kRows rows per thread in flight.
template <typename T, int VPL, int kRows, bool kHalves>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ QkArgs a,
                                                               const __grid_constant__ Turns turns,
                                                               int lpr, int tok_per_block) {
  extern __shared__ float2 cs[];  // [tok_per_block][R / 2]
  const int half = a.R >> 1;
  const int64_t t0 = (int64_t)blockIdx.x * tok_per_block;
  const int ntok = (int)min((int64_t)tok_per_block, a.tokens - t0);
  const int heads = a.nh + a.nkv;
  const int nrows = ntok * heads;
  const int rpp = kThreads / lpr;  // rows per pass of the block
  const int sub = threadIdx.x % lpr, r0 = threadIdx.x / lpr;
  const bool lane_on = sub * VPL < a.c;
  const unsigned mask = 0xffffffffu;

  // blockIdx.y takes every gridDim.y-th group of passes
  for (int base = blockIdx.y * rpp * kRows; base < nrows; base += gridDim.y * rpp * kRows) {
    float v[kRows][VPL];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = base + i * rpp + r0;
#pragma unroll
      for (int e = 0; e < VPL; ++e) v[i][e] = 0.f;
      if (row < nrows && lane_on) {
        const int tl = row / heads, h = row - tl * heads;
        const T* src = h < a.nh
            ? (const T*)a.q + (t0 + tl) * a.q_stride + (int64_t)h * a.c
            : (const T*)a.k + (t0 + tl) * a.k_stride + (int64_t)(h - a.nh) * a.c;
#pragma unroll
        for (int e = 0; e < VPL; e += 8) load8(src + sub * VPL + e, v[i] + e);
      }
    }
    if (base == blockIdx.y * rpp * kRows) {
      // the angles, under the first loads
      for (int e = threadIdx.x; e < ntok * half; e += kThreads) {
        const int tl = e / half, j = e - tl * half;
        const int ax = (j >= a.end0) + (j >= a.end1) + (j >= a.end2);
        const double x = (double)a.pos[ax * a.tokens + t0 + tl] * turns.per_pos[j];
        float s, c;
        sincospif(2.f * (float)(x - rint(x)), &s, &c);
        cs[e] = make_float2(c, s);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = base + i * rpp + r0;
      const int tl = row / heads, h = row - tl * heads;
      const bool is_q = h < a.nh;
      const float* gamma = is_q ? a.q_gamma : a.k_gamma;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < VPL; ++e) ss = fmaf(v[i][e], v[i][e], ss);
      for (int off = lpr >> 1; off > 0; off >>= 1) ss += __shfl_xor_sync(mask, ss, off);
      const bool on = row < nrows && lane_on;
      if (gamma != nullptr && on) {
        const float inv = 1.f / sqrtf(ss / (float)a.c + a.eps);
        gamma += (int64_t)(is_q ? h : h - a.nh) * a.gamma_ld + sub * VPL;
#pragma unroll
        for (int e = 0; e < VPL; e += 4) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + e));
          v[i][e] *= inv * g.x;
          v[i][e + 1] *= inv * g.y;
          v[i][e + 2] *= inv * g.z;
          v[i][e + 3] *= inv * g.w;
        }
      }
      const int d = sub * VPL - (a.c - a.R);  // this lane's first dim among the R (a multiple of 8)
      const float2* w = cs + (on ? tl * half : 0);
      if (kHalves) {
        // the partner of dim d is half dims away: another lane of this row
        const bool low = d < half;
        const int step = half / VPL;
        const int from = (threadIdx.x & 31 & ~(lpr - 1)) + ((sub + (low ? step : -step)) & (lpr - 1));
#pragma unroll
        for (int e = 0; e < VPL; ++e) {
          const float other = __shfl_sync(mask, v[i][e], from);
          if (on && d >= 0) {
            const float2 t = w[(low ? d : d - half) + e];
            v[i][e] = low ? v[i][e] * t.x - other * t.y : other * t.y + v[i][e] * t.x;
          }
        }
      } else if (on) {
#pragma unroll
        for (int e = 0; e < VPL; e += 2)
          if (d + e >= 0) {
            const float2 t = w[(d + e) >> 1];
            rope_turn(v[i][e], v[i][e + 1], t.x, t.y);
          }
      }
      if (on) {
        T* dst = is_q ? (T*)a.q_out + (t0 + tl) * a.qo_stride + (int64_t)h * a.c
                      : (T*)a.k_out + (t0 + tl) * a.ko_stride + (int64_t)(h - a.nh) * a.c;
#pragma unroll
        for (int e = 0; e < VPL; e += 8) store8(dst + sub * VPL + e, v[i] + e);
      }
    }
  }
}

template <typename T, int VPL, int kRows>
cudaError_t launch_t(const QkArgs& a, const Turns& turns, bool halves, cudaStream_t s) {
  int lpr = 1;
  while (lpr * VPL < a.c) lpr <<= 1;
  const int heads = a.nh + a.nkv, rpp = kThreads / lpr;
  // tokens per block: enough rows for one pass of kRows rows per thread, so
  // that the angles are shared by as many rows as the tokens have
  int tpb = (rpp * kRows + heads - 1) / heads;
  tpb = std::max(1, std::min(tpb, a.R > 0 ? 4096 / a.R : 64));  // <= 16 KB of angles
  const int64_t blocks = (a.tokens + tpb - 1) / tpb;
  // few tokens: a token's heads are spread over several blocks
  const int passes = (tpb * heads + rpp * kRows - 1) / (rpp * kRows);
  const unsigned gy = blocks < 2 * sm_count() ? (unsigned)passes : 1u;
  const size_t smem = (size_t)tpb * (a.R / 2) * sizeof(float2);
  auto kern = halves ? qk_norm_rope_kernel<T, VPL, kRows, true>
                     : qk_norm_rope_kernel<T, VPL, kRows, false>;
  kern<<<dim3((unsigned)blocks, gy), kThreads, smem, s>>>(a, turns, lpr, tpb);
  return cudaGetLastError();
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
  API_SUPPORTED(!p->halves || p->rope_dims % (c <= 256 ? 16 : 32) == 0,
                "the halves form needs rope_dims %% 16 == 0 (%% 32 above c = 256)");
  API_SUPPORTED(c <= 256 || c % 16 == 0, "c above 256 must be a multiple of 16");
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
  int ends[3], e = 0;
  for (int i = 0; i < 3; ++i) {
    if (i < p->axes) e += p->sections[i];
    ends[i] = i < p->axes - 1 ? e : 1 << 30;
  }
  a.end0 = ends[0]; a.end1 = ends[1]; a.end2 = ends[2];
  Turns turns;
  // base^(-2j/R) by steps of one factor, started afresh every 16 pairs (16
  // roundings of 2^-53 leave positions of 10^9 good to 10^-6 of a radian)
  const double lb = log2((double)p->rope_base), step = p->rope_dims ? exp2(-2.0 * lb / p->rope_dims) : 0.0;
  double cur = 0.0;
  for (int j = 0; j < p->rope_dims / 2; ++j) {
    cur = j % 16 == 0 ? exp2(-2.0 * j * lb / p->rope_dims) / 6.283185307179586476925286766559 : cur * step;
    turns.per_pos[j] = cur;
  }
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t r;
  if (dt == CSA_F32)
    r = c <= 256 ? launch_t<float, 8, 2>(a, turns, p->halves != 0, s)
                 : launch_t<float, 16, 1>(a, turns, p->halves != 0, s);
  else
    r = c <= 256 ? launch_t<__nv_bfloat16, 8, 4>(a, turns, p->halves != 0, s)
                 : launch_t<__nv_bfloat16, 16, 2>(a, turns, p->halves != 0, s);
  return api_cuda(r, "csa_qk_norm_rope");
}
