// Rows into the paged 4-bit key/value cache (kv4.cuh: the format) and back.
//
// HBM-bound by its bytes: a bf16 row pair is 4 c bytes in and 1.14 c bytes
// out.  A warp takes one 16-token image of one (sequence, head).  Storing, a
// lane holds a group of 16 values (so its scale needs no other lane), and a
// warp step is the K and V rows of two tokens at c = 128, of four at c = 64;
// fetching, a lane holds 8 values, whose 16 bytes are one store.  An image
// that the call covers whole is built in shared memory and written with
// 16-byte stores; the rows of a partly covered one (the ends of the range;
// the single token of a decode step) are written in place, only their own
// bytes.  What holds it: each warp loads one image, waits, converts and exits;
// the first stall is the load (2.6 warps an issue in the store, 5.4 in the
// fetch) with 60 % of the issue slots taken.  The store issues 200 instructions a
// lane for 16 values (loads, maxima, E4M3 there and back, paired fmas and adds,
// 16 shifts into the code words, six small stores); with 8 values a lane it
// took 38 us where this takes 33.  Rows in flight (2, 4), warps a block (2, 4)
// and residency change nothing; several images in flight a warp were not tried.
// 24 400 tokens of 8 heads, c = 128, bf16: store 33 us (100 MB in, 27 out), fetch
// 27 us; their bytes take 19 each.
#include "api_check.h"
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace csa {

namespace {

constexpr int kWarps = 4;

struct Kv4Rows {
  uint8_t* cache;
  const int32_t* table;  // [batch][max_blocks]
  int64_t max_blocks, num_blocks;
  const int64_t* pos;
  const int32_t* count;  // optional
  int64_t n, k_stride, v_stride;
  int nkv, tiles_per_block;  // 16-token images per block (of one head)
};

// The image of tokens 16 tile .. + 15 of (sequence b, head h), or NULL.
__device__ __forceinline__ uint8_t* image(const Kv4Rows& a, int64_t b, int h, int64_t tile, int c) {
  const int64_t j = tile / a.tiles_per_block;
  if (j >= a.max_blocks) return nullptr;
  const int64_t blk = a.table[b * a.max_blocks + j];
  if (blk < 0 || blk >= a.num_blocks) return nullptr;
  return a.cache + ((blk * a.nkv + h) * a.tiles_per_block + tile % a.tiles_per_block) *
                       (int64_t)kv4::tile_bytes(c);
}

template <typename T, int C>
__global__ void __launch_bounds__(kWarps * 32) kv4_store_kernel(const T* __restrict__ k,
                                                                const T* __restrict__ v,
                                                                const Kv4Rows a) {
  constexpr int L = C / 16;       // lanes per row
  constexpr int TS = 32 / (2 * L);  // tokens per warp step
  __shared__ __align__(16) uint8_t img[kWarps][kv4::tile_bytes(C)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t b = blockIdx.z;
  const int h = blockIdx.y;
  const int64_t p0 = a.pos[b];
  if (p0 < 0 || p0 > (int64_t)1 << 62) return;  // (the latter: behind every table)
  int64_t n = a.n;
  if (a.count != nullptr) n = min(n, (int64_t)max(0, a.count[b]));
  const int64_t tile = p0 / 16 + (int64_t)blockIdx.x * kWarps + warp;
  if (tile * 16 >= p0 + n) return;  // also n == 0
  uint8_t* dst = image(a, b, h, tile, C);
  if (dst == nullptr) return;
  const int lo = (int)max((int64_t)0, p0 - tile * 16);            // tokens lo .. hi - 1 of the image
  const int hi = (int)min((int64_t)16, p0 + n - tile * 16);
  const bool whole = lo == 0 && hi == 16;
  uint8_t* to = whole ? img[warp] : dst;
  const bool is_v = lane % (2 * L) >= L;
  const int sub = lane % L, ul = lane / (2 * L);
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const T* src = (is_v ? v : k) + (b * a.n + tile * 16 - p0 + ul) * stride + h * C + sub * 16;
  const kv4::LanePart<C> part(is_v, 2 * sub);
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // rows in flight
#pragma unroll
  for (int s0 = 0; s0 < 16; s0 += TS * U) {
    if (s0 + TS * U <= lo || s0 >= hi) continue;
    kv4::Raw8<T> raw[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int s = s0 + i * TS, u = s + ul;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        raw[i][w].clear();
        if (u >= lo && u < hi) raw[i][w].load(src + s * stride + 8 * w);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int s = s0 + i * TS, u = s + ul;
      if (s + TS <= lo || s >= hi) continue;
      const kv4::Quant16 q = kv4::quantise16(raw[i], L);
      if (u < lo || u >= hi) continue;
      uint8_t* c = to + part.code_at(u);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        *reinterpret_cast<uint16_t*>(c + w * part.next) = (uint16_t)q.codes[w];
        *reinterpret_cast<uint16_t*>(c + w * part.next + part.half) = (uint16_t)(q.codes[w] >> 16);
      }
      to[part.scale_at(u)] = (uint8_t)q.scale;
      if (sub == 0) to[part.exp_at(u)] = (uint8_t)q.E;
    }
  }
  if (whole) {
    __syncwarp();
    for (int i = lane; i < kv4::tile_bytes(C) / 16; i += 32)
      reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(img[warp])[i];
  }
}

template <typename T, int C>
__global__ void __launch_bounds__(kWarps * 32) kv4_fetch_kernel(const Kv4Rows a,
                                                                T* __restrict__ k,
                                                                T* __restrict__ v) {
  constexpr int L = C / 8;
  constexpr int TS = 32 / (2 * L);
  __shared__ __align__(16) uint8_t img[kWarps][kv4::tile_bytes(C)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t b = blockIdx.z;
  const int h = blockIdx.y;
  int64_t p0 = a.pos[b];
  if (p0 > (int64_t)1 << 62) p0 = -1;  // behind every table
  int64_t n = a.n;  // rows that are there; the others come back as zeros
  if (a.count != nullptr) n = min(n, (int64_t)max(0, a.count[b]));
  if (p0 < 0) n = 0;
  const int64_t first = max(p0, (int64_t)0);
  const int64_t tile = first / 16 + (int64_t)blockIdx.x * kWarps + warp;
  if (tile * 16 >= first + a.n) return;
  const uint8_t* src = tile * 16 < first + n ? image(a, b, h, tile, C) : nullptr;
  if (src != nullptr) {
#pragma unroll
    for (int i = lane; i < kv4::tile_bytes(C) / 16; i += 32)
      reinterpret_cast<uint4*>(img[warp])[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
  }
  __syncwarp();
  const uint8_t* im = img[warp];
  const bool is_v = lane % (2 * L) >= L;
  const int sub = lane % L, ul = lane / (2 * L);
  // tokens lo .. hi - 1 of the image are asked for, those below there exist
  const int lo = (int)max((int64_t)0, first - tile * 16);
  const int hi = (int)min((int64_t)16, first + a.n - tile * 16);
  const int there = src == nullptr ? 0 : (int)min((int64_t)16, first + n - tile * 16);
  const int64_t row = (int64_t)a.nkv * C;
  T* dst = (is_v ? v : k) + (b * a.n + tile * 16 - first + ul) * row + h * C + sub * 8;
  const kv4::LanePart<C> part(is_v, sub);
#pragma unroll
  for (int s = 0; s < 16; s += TS, dst += TS * row) {
    const int u = s + ul;
    if (u < lo || u >= hi) continue;
    if (u < there) {
      const uint8_t* c = im + part.code_at(u);
      const uint32_t w = *reinterpret_cast<const uint16_t*>(c) |
                         (uint32_t)*reinterpret_cast<const uint16_t*>(c + part.half) << 16;
      kv4::store_values(dst, w, im[part.scale_at(u)], im[part.exp_at(u)]);
    } else {
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      store8(dst, zero);
    }
  }
}

template <typename T>
cudaError_t launch_store(const Kv4Rows& a, const void* k, const void* v, int64_t batch, int c,
                         cudaStream_t s) {
  const dim3 grid((unsigned)((a.n + 14) / 16 + kWarps) / kWarps, (unsigned)a.nkv, (unsigned)batch);
  if (c == 128)
    kv4_store_kernel<T, 128><<<grid, kWarps * 32, 0, s>>>((const T*)k, (const T*)v, a);
  else
    kv4_store_kernel<T, 64><<<grid, kWarps * 32, 0, s>>>((const T*)k, (const T*)v, a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_fetch(const Kv4Rows& a, void* k, void* v, int64_t batch, int c, cudaStream_t s) {
  const dim3 grid((unsigned)((a.n + 14) / 16 + kWarps) / kWarps, (unsigned)a.nkv, (unsigned)batch);
  if (c == 128) kv4_fetch_kernel<T, 128><<<grid, kWarps * 32, 0, s>>>(a, (T*)k, (T*)v);
  else kv4_fetch_kernel<T, 64><<<grid, kWarps * 32, 0, s>>>(a, (T*)k, (T*)v);
  return cudaGetLastError();
}

}  // namespace

csa_status check_kv4(const csa_kv4_cache* c) {
  API_REQUIRE(c != nullptr, "cache is NULL");
  API_REQUIRE(c->batch >= 0, "batch must be >= 0");
  API_REQUIRE(c->num_blocks >= 1 && c->max_blocks >= 1, "num_blocks and max_blocks must be >= 1");
  API_REQUIRE(c->nkv >= 1, "nkv must be >= 1");
  API_REQUIRE(c->c >= 16 && c->c % 16 == 0, "c must be a positive multiple of 16");
  API_REQUIRE(c->block_tokens >= 16 && c->block_tokens % 16 == 0,
              "block_tokens must be a positive multiple of 16");
  API_SUPPORTED(c->c == 64 || c->c == 128, "the 4-bit cache needs c = 64 or 128");
  API_SUPPORTED(c->batch <= 4096 && c->nkv <= 1024, "the 4-bit cache needs batch <= 4096 and nkv <= 1024");
  API_SUPPORTED(c->num_blocks < ((int64_t)1 << 31) && c->max_blocks < ((int64_t)1 << 31) &&
                    c->block_tokens <= 65536,
                "the 4-bit cache needs num_blocks, max_blocks < 2^31 and block_tokens <= 65536");
  API_SUPPORTED(c->max_blocks * c->block_tokens <= ((int64_t)1 << 31),
                "the 4-bit cache needs sequences of at most 2^31 tokens");
  if (c->batch == 0) return api_ok();
  API_REQUIRE_PTR(c->data);
  API_REQUIRE_LIST(c->block_table);
  return api_ok();
}

}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_kv4_block_bytes(int nkv, int c, int block_tokens) {
  if (nkv < 1 || (c != 64 && c != 128) || block_tokens < 16 || block_tokens % 16 != 0) return 0;
  return (size_t)nkv * (block_tokens / 16) * kv4::tile_bytes(c);
}

csa_status csa_kv4_store(const csa_kv4_cache* cache, const int64_t* pos, int64_t n,
                         const int32_t* count, const void* k, int64_t k_stride, const void* v,
                         int64_t v_stride, csa_dtype dt, void* stream) {
  API_REQUIRE(api_valid_dt(dt), "dt must be CSA_F32 or CSA_BF16");
  csa_status st = check_kv4(cache);
  if (st != CSA_OK) return st;
  API_REQUIRE(n >= 0, "n must be >= 0");
  const int64_t unit = dt == CSA_F32 ? 4 : 8, row = (int64_t)cache->nkv * cache->c;
  API_REQUIRE(k_stride >= row && k_stride % unit == 0 && v_stride >= row && v_stride % unit == 0,
              "strides must be >= nkv * c and whole 16-byte units");
  API_SUPPORTED(n <= ((int64_t)1 << 31), "csa_kv4_store needs n <= 2^31");
  if (cache->batch == 0 || n == 0) return api_ok();
  API_REQUIRE_LIST(pos);
  API_REQUIRE_PTR(k);
  API_REQUIRE_PTR(v);
  API_REQUIRE_OPT_LIST(count);
  const Kv4Rows a{(uint8_t*)cache->data, cache->block_table, cache->max_blocks, cache->num_blocks,
                  pos, count, n, k_stride, v_stride, cache->nkv, cache->block_tokens / 16};
  const cudaStream_t s = (cudaStream_t)stream;
  return api_cuda(dt == CSA_F32 ? launch_store<float>(a, k, v, cache->batch, cache->c, s)
                                : launch_store<__nv_bfloat16>(a, k, v, cache->batch, cache->c, s),
                  "csa_kv4_store");
}

csa_status csa_kv4_fetch(const csa_kv4_cache* cache, const int64_t* pos, int64_t n,
                         const int32_t* count, csa_dtype dt, void* k, void* v, void* stream) {
  API_REQUIRE(api_valid_dt(dt), "dt must be CSA_F32 or CSA_BF16");
  csa_status st = check_kv4(cache);
  if (st != CSA_OK) return st;
  API_REQUIRE(n >= 0, "n must be >= 0");
  API_SUPPORTED(n <= ((int64_t)1 << 31), "csa_kv4_fetch needs n <= 2^31");
  if (cache->batch == 0 || n == 0) return api_ok();
  API_REQUIRE_LIST(pos);
  API_REQUIRE_PTR(k);
  API_REQUIRE_PTR(v);
  API_REQUIRE_OPT_LIST(count);
  const Kv4Rows a{(uint8_t*)cache->data, cache->block_table, cache->max_blocks, cache->num_blocks,
                  pos, count, n, 0, 0, cache->nkv, cache->block_tokens / 16};
  const cudaStream_t s = (cudaStream_t)stream;
  return api_cuda(dt == CSA_F32 ? launch_fetch<float>(a, k, v, cache->batch, cache->c, s)
                                : launch_fetch<__nv_bfloat16>(a, k, v, cache->batch, cache->c, s),
                  "csa_kv4_fetch");
}

}  // extern "C"
