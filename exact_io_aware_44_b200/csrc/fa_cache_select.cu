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
constexpr int kScoreCtas = 2 * 148; // two per SM
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
// four blocks of a warp keep as many independent sums in flight. A warp takes kSets sets of
// four blocks at a time, so that a query element read from shared memory serves them all. A
// persistent grid walks the tiles of 32 * kSets blocks of all (sequence, head, query) units
// and reads a tile's bounds while it works on the one before.
template <bool FP8>
struct ScoreCfg {
  static constexpr int kSets = FP8 ? 2 : 1;  // registers: a bf16 set takes twice those of an 8-bit one
  static constexpr int kTile = 32 * kSets;   // blocks of the cache per tile
};

template <bool FP8>
__global__ void __launch_bounds__(kScoreThreads, 2) score_kernel(const SelectParams p, int tiles, int items) {
  constexpr int kElem = FP8 ? 1 : 2;
  constexpr int kSets = ScoreCfg<FP8>::kSets, kTile = ScoreCfg<FP8>::kTile;
  // {max(q, 0), min(q, 0)} of a row, by the lane group that owns the channel; padded, so that the
  // eight groups' reads fall into different banks
  __shared__ double2 q[kScoreRows][kLanes][kPerLane + 1];
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane & (kLanes - 1);
  const int g = p.Hq / p.Hkv;
  const int first = (int)((long long)blockIdx.x * items / gridDim.x);
  const int end = (int)((long long)(blockIdx.x + 1) * items / gridDim.x);
  grid_wait();
  // bounds of this lane's channels: 16 of each, for kSets blocks 32 apart
  using Raw = typename Row8<FP8>::Raw;
  Raw raw[kSets][2][2];
  float scale[kSets];
  auto load = [&](int item) {
    const int bh = item / tiles / p.Nq, b0 = (item % tiles) * kTile + warp * 4 + (lane >> 3);
    const char* base = static_cast<const char*>(p.bounds) + (size_t)bh * n_blocks * 2 * kCacheD * kElem;
#pragma unroll
    for (int t = 0; t < kSets; ++t) {
      const int blk = min(b0 + 32 * t, n_blocks - 1);
      const char* at = base + ((size_t)blk * 2 * kCacheD + group * kPerLane) * kElem;
#pragma unroll
      for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          raw[t][side][e] = *reinterpret_cast<const Raw*>(at + (side * kCacheD + e * 8) * kElem);
      scale[t] = FP8 ? p.ks[(size_t)bh * n_blocks + blk] : 1.f;
    }
  };
  if (first < end) load(first);
  int held = -1;  // unit whose first kScoreRows heads are in shared memory
  for (int item = first; item < end; ++item) {
    const int unit = item / tiles;  // (b, kv head, query)
    const int i = unit % p.Nq, bh = unit / p.Nq;
    const int last = last_seen(p, bh / p.Hkv, i);
    const int count = last >= 0 ? last / p.block + 1 : 0;
    const int tile0 = (item % tiles) * kTile;
    const int b0 = tile0 + warp * 4 + (lane >> 3);
    Raw cur[kSets][2][2];
    double s[kSets], best[kSets];
    bool any[kSets];  // a score that is a number
#pragma unroll
    for (int t = 0; t < kSets; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) cur[t][e >> 1][e & 1] = raw[t][e >> 1][e & 1];
      s[t] = (double)scale[t];
      best[t] = -INFINITY;
      any[t] = false;
    }
    if (item + 1 < end) load(item + 1);
    if (tile0 >= count) continue;  // uniform
    const __nv_bfloat16* qs = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)bh * g * p.Nq + i) * kCacheD;
    for (int h0 = 0; h0 < g; h0 += kScoreRows) {
      const int rows = min(g - h0, kScoreRows);
      if (g > kScoreRows || held != unit) {  // these heads' rows (uniform)
        __syncthreads();
        for (int e = threadIdx.x; e < kScoreRows * kCacheD; e += kScoreThreads) {
          const int r = e / kCacheD, c = e % kCacheD;
          const double x = r < rows ? (double)__bfloat162float(qs[(size_t)(h0 + r) * p.Nq * kCacheD + c]) : 0.0;
          q[r][c / kPerLane][c % kPerLane] = make_double2(x > 0.0 || x != x ? x : 0.0, x > 0.0 ? 0.0 : x);
        }
        __syncthreads();
        held = unit;
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
          Row8<FP8>::floats(cur[t][0][e8], lo[t]);
          Row8<FP8>::floats(cur[t][1][e8], hi[t]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          double l[kSets], h[kSets];
#pragma unroll
          for (int t = 0; t < kSets; ++t) l[t] = lo[t][e], h[t] = hi[t][e];
#pragma unroll
          for (int r = 0; r < kScoreRows; ++r) {
            const double2 x = q[r][group][e8 * 8 + e];
#pragma unroll
            for (int t = 0; t < kSets; ++t) {
              if constexpr (FP8) {
                // one of the factors is 0: two multiply-adds cost less than a selection of 64-bit operands
                u[t][r] = fma(x.x, h[t], fma(x.y, l[t], u[t][r]));
              } else {  // a bf16 bound may be infinite, and 0 * inf is not 0
                const bool neg = x.y < 0.0;
                u[t][r] = fma(neg ? x.y : x.x, neg ? l[t] : h[t], u[t][r]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < kSets; ++t) {
#pragma unroll
        for (int r = 0; r < kScoreRows; ++r) {
          double v = u[t][r];
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          v *= s[t];
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
        p.keys[(size_t)unit * n_blocks + blk] = key;
      }
    }
  }
  grid_release();
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectParams p) {
  __shared__ TopkShared<unsigned long long> sh;
  const int unit = blockIdx.x;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  topk_begin(sh);
  __syncthreads();
  grid_wait();
  const int last = last_seen(p, unit / p.Nq / p.Hkv, unit % p.Nq);
  const int count = last >= 0 ? last / p.block + 1 : 0;
  const int k = min(count, p.n_select);
  const unsigned long long* keys = p.keys + (size_t)unit * n_blocks;
  int* idx = p.idx + (size_t)unit * p.n_select;
  for (int e = k + threadIdx.x; e < p.n_select; e += kPickThreads) idx[e] = -1;
  if (k > 0 && k < count) {
#pragma unroll 4
    for (int e = threadIdx.x; e < count; e += kPickThreads) topk_count(sh, keys[e]);
  }
  __syncthreads();
  topk_in_order(
      sh, count, k,
      [&](int i, unsigned long long(&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < count) x[e] = keys[i + e];
      },
      [&](uint32_t rank, int e) { idx[rank] = e; });
  grid_release();
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t s) {
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int tile = p.fp8 ? ScoreCfg<true>::kTile : ScoreCfg<false>::kTile;
  const int tiles = (n_blocks + tile - 1) / tile;
  const unsigned units = (unsigned)(p.B * p.Hkv * p.Nq);
  const int items = (int)units * tiles;
  const unsigned grid = (unsigned)min(items, kScoreCtas);
  const cudaError_t e = p.fp8 ? launch_dependent(score_kernel<true>, grid, kScoreThreads, 0, s, p, tiles, items)
                              : launch_dependent(score_kernel<false>, grid, kScoreThreads, 0, s, p, tiles, items);
  if (e != cudaSuccess) return e;
  return launch_dependent(pick_kernel, units, kPickThreads, 0, s, p);
}

}  // namespace fa
