// fa_cache_select.cu -- which blocks of a cache each query attends to.
//
// A block's keys lie, channel by channel, between its bounds lo and hi, so
//   u_h = s_k * sum_c max(q_c lo_c, q_c hi_c)
// is at least every score q . k of head h in the block: a cheap score that never
// undersells a block. A query's blocks go by u = max_h u_h over the heads of its group
// (they share the keys that are read).
//
// The choice is a whole number that hangs on comparisons, so the sums are held in 64 bits:
// a product of two bf16 values has 16 significant bits, and a sum of 128 of them over the
// usual range of exponents is exact in 53, whatever its order.
#include "fa.h"
#include "fa_cache.h"
#include "fa_topk.cuh"

namespace fa {
namespace {

constexpr int kScoreThreads = 128;  // one block of the cache per thread
constexpr int kScoreRows = 8;       // heads of the group per pass
constexpr int kPickThreads = 512;

// Last key that query i of sequence b sees; -1 if none.
__device__ __forceinline__ int last_seen(const SelectParams& p, int b, int i) {
  const int len = cache_len(p.lens, b, p.Nk);
  return max(p.causal ? len - p.Nq + i : len - 1, -1);
}

template <bool FP8>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const SelectParams p, int tiles) {
  constexpr int kElem = FP8 ? 1 : 2;
  __shared__ double q[kScoreRows][kCacheD];
  const int unit = blockIdx.x / tiles;  // (b, kv head, query)
  const int i = unit % p.Nq;
  const int bh = unit / p.Nq;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int last = last_seen(p, bh / p.Hkv, i);
  const int count = last >= 0 ? last / p.block + 1 : 0;
  if ((int)(blockIdx.x % tiles) * kScoreThreads >= count) return;
  const int blk = (blockIdx.x % tiles) * kScoreThreads + threadIdx.x;
  const int g = p.Hq / p.Hkv;
  const __nv_bfloat16* qs = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)bh * g * p.Nq + i) * kCacheD;
  const char* bounds =
      static_cast<const char*>(p.bounds) + ((size_t)bh * n_blocks + min(blk, n_blocks - 1)) * 2 * kCacheD * kElem;
  double best = -INFINITY;
  bool any = false;  // a score that is a number
  for (int h0 = 0; h0 < g; h0 += kScoreRows) {
    const int rows = min(g - h0, kScoreRows);
    __syncthreads();
    for (int e = threadIdx.x; e < rows * kCacheD; e += kScoreThreads)
      q[e / kCacheD][e % kCacheD] = (double)__bfloat162float(qs[(size_t)(h0 + e / kCacheD) * p.Nq * kCacheD + e % kCacheD]);
    __syncthreads();
    double u[kScoreRows];
#pragma unroll
    for (int r = 0; r < kScoreRows; ++r) u[r] = 0.0;
    for (int c = 0; c < kCacheD; c += 8) {
      using Raw = typename Row8<FP8>::Raw;
      float lo[8], hi[8];
      Row8<FP8>::floats(*reinterpret_cast<const Raw*>(bounds + c * kElem), lo);
      Row8<FP8>::floats(*reinterpret_cast<const Raw*>(bounds + (kCacheD + c) * kElem), hi);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double l = lo[e], h = hi[e];
#pragma unroll
        for (int r = 0; r < kScoreRows; ++r) {
          if (r < rows) {
            const double x = q[r][c + e];
            u[r] = fma(x, x >= 0.0 ? h : l, u[r]);
          }
        }
      }
    }
    const double s = p.ks ? (double)p.ks[(size_t)bh * n_blocks + min(blk, n_blocks - 1)] : 1.0;
#pragma unroll
    for (int r = 0; r < kScoreRows; ++r) {
      if (r < rows) {
        const double v = u[r] * s;
        if (v == v) {
          best = fmax(best, v);
          any = true;
        }
      }
    }
  }
  if (blk >= count) return;
  unsigned long long key = any ? order_key(best) : 0ull;
  if (blk < p.n_first || blk >= count - p.n_last) key = ~0ull;  // always taken
  p.keys[(size_t)unit * n_blocks + blk] = key;
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectParams p) {
  __shared__ TopkShared sh;
  const int unit = blockIdx.x;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int last = last_seen(p, unit / p.Nq / p.Hkv, unit % p.Nq);
  const int count = last >= 0 ? last / p.block + 1 : 0;
  const int k = min(count, p.n_select);
  const unsigned long long* keys = p.keys + (size_t)unit * n_blocks;
  int* idx = p.idx + (size_t)unit * p.n_select;
  for (int e = k + threadIdx.x; e < p.n_select; e += kPickThreads) idx[e] = -1;
  topk_in_order<unsigned long long>(
      sh, count, k, [&](int e) { return keys[e]; }, [&](uint32_t rank, int e) { idx[rank] = e; });
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t s) {
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int tiles = (n_blocks + kScoreThreads - 1) / kScoreThreads;
  const unsigned units = (unsigned)(p.B * p.Hkv * p.Nq);
  if (p.fp8)
    score_kernel<true><<<units * tiles, kScoreThreads, 0, s>>>(p, tiles);
  else
    score_kernel<false><<<units * tiles, kScoreThreads, 0, s>>>(p, tiles);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  pick_kernel<<<units, kPickThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
