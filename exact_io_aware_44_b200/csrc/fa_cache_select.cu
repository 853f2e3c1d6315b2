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
#include "fa_cache_launch.cuh"
#include "fa_topk.cuh"

namespace fa {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreTile = 128;     // blocks of the cache per CTA
constexpr int kScoreRows = 4;       // heads of the group per pass
constexpr int kLanes = 8;           // lanes per block, 16 channels each
constexpr int kPerLane = kCacheD / kLanes;
constexpr int kPickThreads = 512;

// Last key that query i of sequence b sees; -1 if none.
__device__ __forceinline__ int last_seen(const SelectParams& p, int b, int i) {
  const int len = cache_len(p.lens, b, p.Nk);
  return max(p.causal ? len - p.Nq + i : len - 1, -1);
}

// Eight lanes share a block: their 16-byte loads cover its bounds' rows without gaps, and the
// four blocks of a warp keep as many independent sums in flight.
template <bool FP8>
__global__ void __launch_bounds__(kScoreThreads, 3) score_kernel(const SelectParams p, int tiles) {
  constexpr int kElem = FP8 ? 1 : 2;
  constexpr int kSets = 1;
  // rows of a lane group's 16 elements, padded: the eight groups' reads fall into different banks
  __shared__ double q[kScoreRows][kLanes][kPerLane + 1];
  const int unit = blockIdx.x / tiles;  // (b, kv head, query)
  const int i = unit % p.Nq;
  const int bh = unit / p.Nq;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  grid_wait();
  const int last = last_seen(p, bh / p.Hkv, i);
  const int count = last >= 0 ? last / p.block + 1 : 0;
  const int tile0 = (int)(blockIdx.x % tiles) * kScoreTile;
  if (tile0 >= count) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane & (kLanes - 1);
  const int g = p.Hq / p.Hkv;
  const __nv_bfloat16* qs = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)bh * g * p.Nq + i) * kCacheD;
  const char* base = static_cast<const char*>(p.bounds) + (size_t)bh * n_blocks * 2 * kCacheD * kElem;
  unsigned long long* keys = p.keys + (size_t)unit * n_blocks;
  for (int it = 0; it < kScoreTile; it += 32 * kSets) {
    const int b0 = tile0 + it + warp * 4 + (lane >> 3);
    // bounds of this lane's channels: 16 of each, for kSets blocks 32 apart
    using Raw = typename Row8<FP8>::Raw;
    Raw raw[kSets][2][2];
#pragma unroll
    for (int t = 0; t < kSets; ++t) {
      const char* at = base + ((size_t)min(b0 + 32 * t, n_blocks - 1) * 2 * kCacheD + group * kPerLane) * kElem;
#pragma unroll
      for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          raw[t][side][e] = *reinterpret_cast<const Raw*>(at + (side * kCacheD + e * 8) * kElem);
    }
    double best[kSets];
    bool any[kSets];
#pragma unroll
    for (int t = 0; t < kSets; ++t) best[t] = -INFINITY, any[t] = false;
    for (int h0 = 0; h0 < g; h0 += kScoreRows) {
      const int rows = min(g - h0, kScoreRows);
      if (g > kScoreRows || it == 0) {  // these heads' rows (uniform)
        __syncthreads();
        for (int e = threadIdx.x; e < kScoreRows * kCacheD; e += kScoreThreads) {
          const int r = e / kCacheD, c = e % kCacheD;
          q[r][c / kPerLane][c % kPerLane] =
              r < rows ? (double)__bfloat162float(qs[(size_t)(h0 + r) * p.Nq * kCacheD + c]) : 0.0;
        }
        __syncthreads();
      }
      double u[kSets][kScoreRows];
#pragma unroll
      for (int t = 0; t < kSets; ++t)
#pragma unroll
        for (int r = 0; r < kScoreRows; ++r) u[t][r] = 0.0;
#pragma unroll
      for (int e8 = 0; e8 < 2; ++e8) {
        float lo[kSets][8], hi[kSets][8];
#pragma unroll
        for (int t = 0; t < kSets; ++t) {
          Row8<FP8>::floats(raw[t][0][e8], lo[t]);
          Row8<FP8>::floats(raw[t][1][e8], hi[t]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          double l[kSets], h[kSets];
#pragma unroll
          for (int t = 0; t < kSets; ++t) l[t] = lo[t][e], h[t] = hi[t][e];
#pragma unroll
          for (int r = 0; r < kScoreRows; ++r) {
            const double x = q[r][group][e8 * 8 + e];
#pragma unroll
            for (int t = 0; t < kSets; ++t) u[t][r] = fma(x, x >= 0.0 ? h[t] : l[t], u[t][r]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < kSets; ++t) {
        const double s = p.ks ? (double)p.ks[(size_t)bh * n_blocks + min(b0 + 32 * t, n_blocks - 1)] : 1.0;
#pragma unroll
        for (int r = 0; r < kScoreRows; ++r) {
          double v = u[t][r];
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          v *= s;
          if (r < rows && v == v) {
            best[t] = fmax(best[t], v);
            any[t] = true;
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kSets; ++t) {
      const int blk = b0 + 32 * t;
      if (group == 0 && blk < count) {
        unsigned long long key = any[t] ? order_key(best[t]) : 0ull;
        if (blk < p.n_first || blk >= count - p.n_last) key = ~0ull;  // always taken
        keys[blk] = key;
      }
    }
  }
  grid_release();
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectParams p) {
  __shared__ TopkShared sh;
  const int unit = blockIdx.x;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  grid_wait();
  const int last = last_seen(p, unit / p.Nq / p.Hkv, unit % p.Nq);
  const int count = last >= 0 ? last / p.block + 1 : 0;
  const int k = min(count, p.n_select);
  const unsigned long long* keys = p.keys + (size_t)unit * n_blocks;
  int* idx = p.idx + (size_t)unit * p.n_select;
  for (int e = k + threadIdx.x; e < p.n_select; e += kPickThreads) idx[e] = -1;
  topk_in_order<unsigned long long>(
      sh, count, k, [&](int e) { return keys[e]; }, [&](uint32_t rank, int e) { idx[rank] = e; });
  grid_release();
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t s) {
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int tiles = (n_blocks + kScoreTile - 1) / kScoreTile;
  const unsigned units = (unsigned)(p.B * p.Hkv * p.Nq);
  const cudaError_t e = p.fp8 ? launch_dependent(score_kernel<true>, units * tiles, kScoreThreads, 0, s, p, tiles)
                              : launch_dependent(score_kernel<false>, units * tiles, kScoreThreads, 0, s, p, tiles);
  if (e != cudaSuccess) return e;
  return launch_dependent(pick_kernel, units, kPickThreads, 0, s, p);
}

}  // namespace fa
