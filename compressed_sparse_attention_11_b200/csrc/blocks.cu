// Blocks of a paged cache: copying the data of listed blocks, and the block
// tables of forked, freed and compacted sequences.
//
// The tables are the only truth: a block is in use exactly when a row of the
// table names it (several rows may, after a fork).  Nothing is counted or
// kept between calls, so every call can be captured, replayed and run beside
// calls on other tables.  The table calls write a new table and leave the
// one they read as it is.
#include "api_check.h"
#include "common.cuh"
#include "launch.h"

namespace csa {

namespace {

// ---- data ---------------------------------------------------------------------
// HBM-bound: each listed block is read and written once.  The copy is cut
// into pieces of kPiece bytes of one region of one pair; a block of threads
// takes every gridDim.x-th piece, all its 16-byte loads in flight before the
// first store.
constexpr int kCopyThreads = 256;
constexpr int kPerThread = 8;
constexpr int kPiece = kCopyThreads * kPerThread * 16;  // 32 KB

struct CopyArgs {
  csa_block_region r[CSA_MAX_REGIONS];
  int first_piece[CSA_MAX_REGIONS + 1];  // pieces of a pair before region i
  int nregions;
  int64_t num_blocks;
  const int32_t *src, *dst, *count;
  int64_t pairs;
};

template <typename V>
__device__ __forceinline__ void copy_piece(const uint8_t* s, uint8_t* d, int64_t bytes) {
  const int64_t n = bytes / (int64_t)sizeof(V);
  const V* sv = reinterpret_cast<const V*>(s);
  V* dv = reinterpret_cast<V*>(d);
  for (int64_t i0 = 0; i0 < n; i0 += kCopyThreads * kPerThread) {
    V v[kPerThread];
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
      const int64_t i = i0 + u * kCopyThreads + threadIdx.x;
      if (i < n) v[u] = __ldcs(sv + i);
    }
#pragma unroll
    for (int u = 0; u < kPerThread; ++u) {
      const int64_t i = i0 + u * kCopyThreads + threadIdx.x;
      if (i < n) __stcs(dv + i, v[u]);
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) blocks_copy_kernel(
    const __grid_constant__ CopyArgs a) {
  int64_t n = a.pairs;
  if (a.count != nullptr) n = min(n, (int64_t)max(0, a.count[0]));
  const int per_pair = a.first_piece[a.nregions];
  const int64_t total = n * per_pair;
  for (int64_t p = blockIdx.x; p < total; p += gridDim.x) {
    const int64_t pair = p / per_pair;
    const int piece = (int)(p - pair * per_pair);
    const int64_t from = a.src[pair], to = a.dst[pair];
    if (from < 0 || to < 0 || from >= a.num_blocks || to >= a.num_blocks || from == to) continue;
    int i = 0;
    while (piece >= a.first_piece[i + 1]) ++i;
    const int64_t bytes = (int64_t)a.r[i].block_bytes;
    const int64_t off = (int64_t)(piece - a.first_piece[i]) * kPiece;
    const int64_t len = min((int64_t)kPiece, bytes - off);
    uint8_t* base = static_cast<uint8_t*>(a.r[i].base);
    const uint8_t* s = base + from * bytes + off;
    uint8_t* d = base + to * bytes + off;
    if (bytes % 16 == 0) copy_piece<uint4>(s, d, len);
    else if (bytes % 4 == 0) copy_piece<uint32_t>(s, d, len);
    else copy_piece<uint8_t>(s, d, len);
  }
}

// ---- tables -------------------------------------------------------------------
constexpr int kTabThreads = 256;
constexpr int kOneThreads = 1024;

// One block of threads per row of the table.  A row that a fork names (the
// last such fork counts) holds the whole blocks of the source's first
// tokens[i] tokens, then, if the last of them is partly filled, fresh[i];
// any other row is copied.
__global__ void __launch_bounds__(kTabThreads) blocks_fork_kernel(
    const int32_t* __restrict__ table, int64_t rows, int64_t max_blocks,
    const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
    const int64_t* __restrict__ tokens, const int32_t* __restrict__ fresh, int forks,
    int block_tokens, int32_t* __restrict__ out, int32_t* __restrict__ copy_src,
    int32_t* __restrict__ copy_dst) {
  __shared__ int last;
  if (threadIdx.x == 0) last = -1;
  __syncthreads();
  const int64_t b = blockIdx.x;
  // forks whose destination is no row of the table copy nothing
  if (b == 0)
    for (int i = threadIdx.x; i < forks; i += kTabThreads)
      if (dst[i] < 0 || dst[i] >= rows) copy_src[i] = copy_dst[i] = -1;
  int mine = -1;
  for (int i = threadIdx.x; i < forks; i += kTabThreads)
    if (dst[i] == b) mine = i;
  if (mine >= 0) atomicMax(&last, mine);
  __syncthreads();
  const int f = last;
  if (f < 0) {
    for (int64_t j = threadIdx.x; j < max_blocks; j += kTabThreads)
      out[b * max_blocks + j] = table[b * max_blocks + j];
    return;
  }
  const int64_t s = src[f];
  const bool from = s >= 0 && s < rows;
  const int64_t tok = max((int64_t)0, tokens[f]);
  const int64_t full = min(tok / block_tokens, max_blocks);
  const bool part = from && full < max_blocks && tok % block_tokens != 0;
  for (int64_t j = threadIdx.x; j < max_blocks; j += kTabThreads) {
    int32_t v = -1;
    if (from && j < full) v = table[s * max_blocks + j];
    else if (part && j == full) v = fresh[f];
    out[b * max_blocks + j] = v;
  }
  for (int i = threadIdx.x; i < forks; i += kTabThreads) {
    if (dst[i] != b) continue;
    const bool yes = i == f && part && table[s * max_blocks + full] >= 0 && fresh[f] >= 0;
    copy_src[i] = yes ? table[s * max_blocks + full] : -1;
    copy_dst[i] = yes ? fresh[f] : -1;
  }
}

// Inclusive sum over the 1024 threads of the block of one value each.
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += o;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int r = v + (warp > 0 ? warp_sums[warp - 1] : 0);
  __syncthreads();
  return r;
}

// pre[w] = bits set in words 0 .. w - 1; returns the number set in all words.
__device__ __forceinline__ int prefix_words(const uint32_t* bits, int* pre, int words,
                                            int* warp_sums) {
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += kOneThreads) {
    const int w = w0 + threadIdx.x;
    const int c = w < words ? __popc(bits[w]) : 0;
    const int inc = block_scan(c, warp_sums);
    if (w < words) pre[w] = base + inc - c;
    base += warp_sums[31];
    __syncthreads();
  }
  return base;
}

// One block of threads: a bitmap of the blocks in shared memory, so no
// scratch in global memory and one launch (table and lists are read and
// written once: 64 x 64 entries 5 us, 256 x 256 30, 256 x 4096 0.34 ms; batches
// of eight loads before the first use changed nothing).
// Freed: named by a row in `seqs` and by no other row.
__global__ void __launch_bounds__(kOneThreads) blocks_free_kernel(
    const int32_t* __restrict__ table, int64_t rows, int64_t max_blocks, int num_blocks,
    const int32_t* __restrict__ seqs, int nseqs, int32_t* __restrict__ out,
    int32_t* __restrict__ freed, int32_t* __restrict__ nfreed) {
  extern __shared__ uint32_t sm[];
  __shared__ int warp_sums[32];
  const int words = (num_blocks + 31) / 32;
  const int row_words = (int)((rows + 31) / 32);
  uint32_t* gone = sm;                    // rows that end
  uint32_t* drop = gone + row_words;      // blocks that such a row names
  uint32_t* keep = drop + words;          // blocks that another row names
  for (int i = threadIdx.x; i < row_words + 2 * words; i += kOneThreads) sm[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < nseqs; i += kOneThreads) {
    const int32_t b = seqs[i];
    if (b >= 0 && b < rows) atomicOr(&gone[b >> 5], 1u << (b & 31));
  }
  __syncthreads();
  const int64_t total = rows * max_blocks;
  // e = b max_blocks + j, stepped without a division an entry
  const int64_t row = max((int64_t)1, max_blocks);  // (a table without columns has no entries)
  int64_t b = threadIdx.x / row, j = threadIdx.x - b * row;
  const int64_t db = kOneThreads / row, dj = kOneThreads - db * row;
  for (int64_t e = threadIdx.x; e < total; e += kOneThreads) {
    const int32_t v = table[e];
    const bool g = (gone[b >> 5] >> (b & 31)) & 1;
    if (v >= 0 && v < num_blocks) {
      uint32_t* m = (g ? drop : keep) + (v >> 5);
      const uint32_t bit = 1u << (v & 31);
      if ((*(volatile uint32_t*)m & bit) == 0) atomicOr(m, bit);
    }
    out[e] = g ? -1 : v;
    b += db;
    j += dj;
    if (j >= max_blocks) {
      j -= max_blocks;
      ++b;
    }
  }
  __syncthreads();
  for (int w = threadIdx.x; w < words; w += kOneThreads) drop[w] &= ~keep[w];
  __syncthreads();
  int* pre = reinterpret_cast<int*>(keep);  // the kept bits are no longer needed
  const int n = prefix_words(drop, pre, words, warp_sums);
  for (int v = threadIdx.x; v < num_blocks; v += kOneThreads) {
    const uint32_t w = drop[v >> 5];
    if ((w >> (v & 31)) & 1) freed[pre[v >> 5] + __popc(w & ((1u << (v & 31)) - 1))] = v;
    if (v >= n) freed[v] = -1;
  }
  if (threadIdx.x == 0) nfreed[0] = n;
}

// Blocks in use move to 0 .. live - 1: the j-th one at or above `live` goes
// to the j-th unused one below it (as many as there are), so no block is
// both read and written and the moves can run in any order.
__global__ void __launch_bounds__(kOneThreads) blocks_compact_kernel(
    const int32_t* __restrict__ table, int64_t rows, int64_t max_blocks, int num_blocks,
    int32_t* __restrict__ out, int32_t* __restrict__ copy_src, int32_t* copy_dst,
    int32_t* __restrict__ counts) {
  extern __shared__ uint32_t sm[];
  __shared__ int warp_sums[32];
  const int words = (num_blocks + 31) / 32;
  uint32_t* used = sm;
  int* pre = reinterpret_cast<int*>(sm + words);
  for (int i = threadIdx.x; i < words; i += kOneThreads) used[i] = 0;
  __syncthreads();
  const int64_t total = rows * max_blocks;
  for (int64_t e = threadIdx.x; e < total; e += kOneThreads) {
    const int32_t v = table[e];
    if (v < 0 || v >= num_blocks) continue;
    const uint32_t bit = 1u << (v & 31);
    if ((*(volatile uint32_t*)&used[v >> 5] & bit) == 0) atomicOr(&used[v >> 5], bit);
  }
  __syncthreads();
  const int live = prefix_words(used, pre, words, warp_sums);
  // used blocks before block v
  auto before = [&](int v) {
    return pre[v >> 5] + __popc(used[v >> 5] & ((1u << (v & 31)) - 1));
  };
  const int low = live < num_blocks ? before(live) : live;  // used blocks below `live`
  const int moves = live - low;
  for (int v = threadIdx.x; v < num_blocks; v += kOneThreads) {
    const bool u = (used[v >> 5] >> (v & 31)) & 1;
    if (u && v >= live) copy_src[before(v) - low] = v;
    if (!u && v < live) copy_dst[v - before(v)] = v;
    if (v >= moves) copy_src[v] = copy_dst[v] = -1;
  }
  if (threadIdx.x == 0) {
    counts[0] = moves;
    counts[1] = live;
  }
  __syncthreads();  // copy_dst is written by this block alone
  for (int64_t e = threadIdx.x; e < total; e += kOneThreads) {
    const int32_t v = table[e];
    out[e] = v < 0 || v >= num_blocks ? -1 : v < live ? v : copy_dst[before(v) - low];
  }
}

constexpr size_t kMaxTabSmem = 220 * 1024;

csa_status check_table(const int32_t* table, int64_t rows, int64_t max_blocks,
                       const int32_t* out) {
  API_REQUIRE(rows >= 0 && max_blocks >= 0, "rows and max_blocks must be >= 0");
  API_SUPPORTED(rows < ((int64_t)1 << 20) && max_blocks < ((int64_t)1 << 31),
                "a block table needs rows < 2^20 and max_blocks < 2^31");
  if (rows == 0 || max_blocks == 0) return api_ok();
  API_REQUIRE_LIST(table);
  API_REQUIRE_LIST(out);
  const size_t bytes = (size_t)rows * max_blocks * 4;
  API_REQUIRE(!api_overlap(table, bytes, out, bytes), "table_out must not overlap table");
  return api_ok();
}

}  // namespace

}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_blocks_copy(const csa_block_region* regions, int nregions, int64_t num_blocks,
                           const int32_t* src, const int32_t* dst, int64_t pairs,
                           const int32_t* count, void* stream) {
  API_REQUIRE(nregions >= 0 && nregions <= CSA_MAX_REGIONS, "nregions must be in [0, %d]",
              CSA_MAX_REGIONS);
  API_REQUIRE(num_blocks >= 0 && num_blocks < ((int64_t)1 << 31), "num_blocks must be in [0, 2^31)");
  API_REQUIRE(pairs >= 0, "pairs must be >= 0");
  if (nregions > 0) API_REQUIRE(regions != nullptr, "regions is NULL");
  CopyArgs a = {};
  int64_t pieces = 0;
  for (int i = 0; i < nregions; ++i) {
    a.r[i] = regions[i];
    if (regions[i].block_bytes > 0 && num_blocks > 0) {
      API_REQUIRE(regions[i].base != nullptr, "region %d is NULL", i);
      API_REQUIRE(api_aligned16(regions[i].base), "region %d is not 16-byte aligned", i);
    }
    API_SUPPORTED(regions[i].block_bytes <= ((size_t)1 << 40),
                  "region %d: a block has too many bytes", i);
    a.first_piece[i] = (int)pieces;
    pieces += (int64_t)((regions[i].block_bytes + kPiece - 1) / kPiece);
  }
  a.first_piece[nregions] = (int)pieces;
  if (pairs == 0 || pieces == 0 || num_blocks == 0) return api_ok();
  API_REQUIRE_LIST(src);
  API_REQUIRE_LIST(dst);
  API_REQUIRE_OPT_LIST(count);
  a.nregions = nregions;
  a.num_blocks = num_blocks;
  a.src = src;
  a.dst = dst;
  a.count = count;
  a.pairs = pairs;
  const int64_t grid = std::min<int64_t>(pairs * pieces, (int64_t)sm_count() * 8);
  blocks_copy_kernel<<<(unsigned)grid, kCopyThreads, 0, (cudaStream_t)stream>>>(a);
  return api_cuda(cudaGetLastError(), "csa_blocks_copy");
}

csa_status csa_blocks_fork(const int32_t* table, int64_t rows, int64_t max_blocks,
                           const int32_t* src, const int32_t* dst, const int64_t* tokens,
                           const int32_t* fresh, int forks, int block_tokens, int32_t* table_out,
                           int32_t* copy_src, int32_t* copy_dst, void* stream) {
  API_REQUIRE(forks >= 0, "forks must be >= 0");
  API_REQUIRE(block_tokens >= 1, "block_tokens must be >= 1");
  csa_status st = check_table(table, rows, max_blocks, table_out);
  if (st != CSA_OK) return st;
  if (rows == 0 || max_blocks == 0) {
    API_REQUIRE(forks == 0, "forks need a table");
    return api_ok();
  }
  if (forks > 0) {
    API_REQUIRE_LIST(src);
    API_REQUIRE_LIST(dst);
    API_REQUIRE_LIST(tokens);
    API_REQUIRE_LIST(fresh);
    API_REQUIRE_LIST(copy_src);
    API_REQUIRE_LIST(copy_dst);
  }
  blocks_fork_kernel<<<(unsigned)rows, kTabThreads, 0, (cudaStream_t)stream>>>(
      table, rows, max_blocks, src, dst, tokens, fresh, forks, block_tokens, table_out, copy_src,
      copy_dst);
  return api_cuda(cudaGetLastError(), "csa_blocks_fork");
}

csa_status csa_blocks_free(const int32_t* table, int64_t rows, int64_t max_blocks,
                           int64_t num_blocks, const int32_t* seqs, int nseqs, int32_t* table_out,
                           int32_t* freed, int32_t* nfreed, void* stream) {
  API_REQUIRE(nseqs >= 0, "nseqs must be >= 0");
  API_REQUIRE(num_blocks >= 1, "num_blocks must be >= 1");
  csa_status st = check_table(table, rows, max_blocks, table_out);
  if (st != CSA_OK) return st;
  API_SUPPORTED(num_blocks <= CSA_MAX_TABLE_BLOCKS && rows <= 65536,
                "csa_blocks_free needs num_blocks <= %d and rows <= 65536", CSA_MAX_TABLE_BLOCKS);
  if (nseqs > 0) API_REQUIRE_LIST(seqs);
  API_REQUIRE_LIST(freed);
  API_REQUIRE_LIST(nfreed);
  const size_t smem = ((size_t)(rows + 31) / 32 + 2 * (size_t)((num_blocks + 31) / 32)) * 4;
  cudaError_t e = cudaFuncSetAttribute(blocks_free_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kMaxTabSmem);
  if (e != cudaSuccess) return api_cuda(e, "csa_blocks_free");
  blocks_free_kernel<<<1, kOneThreads, smem, (cudaStream_t)stream>>>(
      table, rows, max_blocks, (int)num_blocks, seqs, nseqs, table_out, freed, nfreed);
  return api_cuda(cudaGetLastError(), "csa_blocks_free");
}

csa_status csa_blocks_compact(const int32_t* table, int64_t rows, int64_t max_blocks,
                              int64_t num_blocks, int32_t* table_out, int32_t* copy_src,
                              int32_t* copy_dst, int32_t* counts, void* stream) {
  API_REQUIRE(num_blocks >= 1, "num_blocks must be >= 1");
  csa_status st = check_table(table, rows, max_blocks, table_out);
  if (st != CSA_OK) return st;
  API_SUPPORTED(num_blocks <= CSA_MAX_TABLE_BLOCKS, "csa_blocks_compact needs num_blocks <= %d",
                CSA_MAX_TABLE_BLOCKS);
  API_REQUIRE_LIST(copy_src);
  API_REQUIRE_LIST(copy_dst);
  API_REQUIRE_LIST(counts);
  const size_t smem = 2 * (size_t)((num_blocks + 31) / 32) * 4;
  cudaError_t e = cudaFuncSetAttribute(blocks_compact_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kMaxTabSmem);
  if (e != cudaSuccess) return api_cuda(e, "csa_blocks_compact");
  blocks_compact_kernel<<<1, kOneThreads, smem, (cudaStream_t)stream>>>(
      table, rows, max_blocks, (int)num_blocks, table_out, copy_src, copy_dst, counts);
  return api_cuda(cudaGetLastError(), "csa_blocks_compact");
}

}  // extern "C"
