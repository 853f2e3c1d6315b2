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
constexpr int kPickThreads = 512;

// Last key that query i of sequence b sees; -1 if none.
__device__ __forceinline__ int last_seen(const SelectParams& p, int b, int i) {
  const int len = cache_len(p.lens, b, p.Nk);
  return max(p.causal ? len - p.Nq + i : len - 1, -1);
}

// A block's place in its query's order.
__device__ __forceinline__ void put_key(const SelectParams& p, int unit, int n_blocks, int count, int blk, bool any,
                                        double u) {
  if (blk >= count) return;
  unsigned long long key = any ? order_key(u) : 0ull;
  if (blk < p.n_first || blk >= count - p.n_last) key = ~0ull;  // always taken
  p.keys[(size_t)unit * n_blocks + blk] = key;
}

// In both score kernels a persistent grid walks the tiles of blocks of all (sequence, head, query)
// units, and reads a tile's bounds while it works on the one before.

// 8-bit bounds, on the tensor cores' 64-bit products: u = [hi, lo] . [max(q, 0), min(q, 0)], eight
// blocks (M) by eight heads (N), four channels (K) an instruction. A lane holds 32 channels of
// one block's bounds: lane 4r + c channels 32c .. 32c + 31 of row r, and the i-th instruction
// takes the i-th of each (the sum's order is free).
//   A code's bits are moved to their place in a double: exponent and mantissa keep their places
// relative to each other, so that the double is 2^-1016 times the value, subnormal codes included,
// exactly. Queries carry 2^800, so that no product leaves the normal range. Selecting 64 of 512
// blocks for 128 units of four heads, choice included, took 24.0 us with multiply-adds in a thread and
// the conversion instructions, 23.4 with the bits moved, and 20.1 with these products (18.9
// with a shorter choice); they are at 7.5 us by their measured rate (36 TFLOP/s), half of them for the
// four heads that are not there.
constexpr int kMmaHeads = 8;
constexpr int kMmaSets = 2;                     // groups of eight blocks per warp
constexpr int kMmaTile = 8 * 8 * kMmaSets;      // blocks of the cache per tile
constexpr int kPerLane8 = kCacheD / 4;
constexpr int kCodeExp = 1023 - 7, kQueryExp = 800;
__device__ __forceinline__ double pow2(int e) { return __hiloint2double((e + 1023) << 20, 0); }

// c += a b: a[row lane / 4][k lane % 4], b[k lane % 4][column lane / 4], c[lane / 4][2 (lane % 4) + 0, 1].
__device__ __forceinline__ void mma_f64(double (&c)[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
      : "+d"(c[0]), "+d"(c[1])
      : "d"(a), "d"(b));
}
// Four codes as doubles times 2^-kCodeExp.
__device__ __forceinline__ void e4m3_to_doubles(uint32_t w, double (&x)[4]) {
  const uint32_t sign = w & 0x80808080u, rest = (w & 0x7F7F7F7Fu) << 1;
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // sign and the other bits of two codes, in the upper bytes of two halves
    const uint32_t two = __byte_perm(rest, sign, e ? 0x7362 : 0x5140);
    x[2 * e] = __hiloint2double((int)(two << 16), 0);
    x[2 * e + 1] = __hiloint2double((int)(two & 0xFFFF0000u), 0);
  }
}

using QueryParts = double2[kMmaHeads][4][kPerLane8 + 1];
// Heads whose score is NaN for a block with a NaN code: those that take its side in its channel. `bounds`
// are this lane's codes; all lanes of a block return the same.
__device__ __noinline__ uint32_t nan_heads(const uint8_t* bounds, const QueryParts& q, int quad) {
  uint32_t heads = 0u;
  for (int i = 0; i < 2 * kPerLane8; ++i) {
    const int side = i / kPerLane8, c = i % kPerLane8;
    if ((bounds[side * kCacheD + c] & 0x7F) != 0x7F) continue;
    for (int r = 0; r < kMmaHeads; ++r)
      if ((q[r][quad][c].y < 0.0) == (side == 0)) heads |= 1u << r;
  }
  heads |= __shfl_xor_sync(0xffffffffu, heads, 1);
  return heads | __shfl_xor_sync(0xffffffffu, heads, 2);
}

__global__ void __launch_bounds__(kScoreThreads, 2) score_fp8_kernel(const SelectParams p, int tiles, int items) {
  // {max(q, 0), min(q, 0)} of eight heads, by the lane group that owns the channel; padded, so that a
  // quarter warp's reads fall into different banks
  __shared__ QueryParts q;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
  const int g = p.Hq / p.Hkv;
  const int first = (int)((long long)blockIdx.x * items / gridDim.x);
  const int end = (int)((long long)(blockIdx.x + 1) * items / gridDim.x);
  grid_wait();
  uint4 raw[kMmaSets][2][2];  // [lo, hi]
  float scale[kMmaSets];
  auto load = [&](int item) {
    const int bh = item / tiles / p.Nq, b0 = (item % tiles) * kMmaTile + warp * 8 * kMmaSets + row;
    const uint8_t* base = static_cast<const uint8_t*>(p.bounds) + (size_t)bh * n_blocks * 2 * kCacheD;
#pragma unroll
    for (int t = 0; t < kMmaSets; ++t) {
      const int blk = min(b0 + 8 * t, n_blocks - 1);
      const uint4* at = reinterpret_cast<const uint4*>(base + (size_t)blk * 2 * kCacheD + quad * kPerLane8);
#pragma unroll
      for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int e = 0; e < 2; ++e) raw[t][side][e] = at[side * (kCacheD / 16) + e];
      scale[t] = p.ks[(size_t)bh * n_blocks + blk];
    }
  };
  if (first < end) load(first);
  int held = -1;  // unit whose first kMmaHeads heads are in shared memory
  for (int item = first; item < end; ++item) {
    const int unit = item / tiles;  // (b, kv head, query)
    const int i = unit % p.Nq, bh = unit / p.Nq;
    const int last = last_seen(p, bh / p.Hkv, i);
    const int count = last >= 0 ? last / p.block + 1 : 0;
    const int tile0 = (item % tiles) * kMmaTile;
    const __nv_bfloat16* qs = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)bh * g * p.Nq + i) * kCacheD;
    auto hold = [&](int h0) {  // these heads' rows into shared memory
      __syncthreads();
#pragma unroll
      for (int n = 0; n < kMmaHeads * kCacheD / kScoreThreads; ++n) {
        const int e = n * kScoreThreads + threadIdx.x, r = e / kCacheD, c = e % kCacheD;
        double x = r < g - h0 ? (double)__bfloat162float(qs[(size_t)(h0 + r) * p.Nq * kCacheD + c]) : 0.0;
        x *= pow2(kQueryExp);
        q[r][c / kPerLane8][c % kPerLane8] = make_double2(x > 0.0 || x != x ? x : 0.0, x > 0.0 ? 0.0 : x);
      }
      __syncthreads();
    };
    // before the bounds, which are still on their way, are used
    if (tile0 < count && (g > kMmaHeads || held != unit)) hold(0), held = unit;
    uint32_t cur[kMmaSets][2][8];
    double s[kMmaSets], best[kMmaSets];
    bool any[kMmaSets], bad[kMmaSets];  // a score that is a number; a NaN code in this warp
#pragma unroll
    for (int t = 0; t < kMmaSets; ++t) {
      uint32_t nan = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 r = raw[t][e >> 1][e & 1];
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cur[t][e >> 1][(e & 1) * 4 + j] = w[j];
          nan |= (w[j] & 0x7F7F7F7Fu) + 0x01010101u;  // NaN: all bits but the sign
        }
      }
      bad[t] = __any_sync(0xffffffffu, (nan & 0x80808080u) != 0u);
      s[t] = (double)scale[t] * pow2(kCodeExp - kQueryExp);
      best[t] = -INFINITY;
      any[t] = false;
    }
    if (item + 1 < end) load(item + 1);
    if (tile0 >= count) continue;  // uniform
    for (int h0 = 0; h0 < g; h0 += kMmaHeads) {
      const int rows = min(g - h0, kMmaHeads);
      if (h0 > 0) hold(h0);
      double u[kMmaSets][2][2] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        double a[kMmaSets][2][4];
#pragma unroll
        for (int t = 0; t < kMmaSets; ++t)
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            // a value that the compiler takes for a new one: the doubles of all channels, kept for the
            // next heads, would not fit the registers
            asm volatile("" : "+r"(cur[t][side][j]));
            e4m3_to_doubles(cur[t][side][j], a[t][side]);
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double2 x = q[row][quad][j * 4 + e];
#pragma unroll
          for (int t = 0; t < kMmaSets; ++t) {
            mma_f64(u[t][0], a[t][0][e], x.y);
            mma_f64(u[t][1], a[t][1][e], x.x);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < kMmaSets; ++t) {
        uint32_t out = 0u;  // heads without a score
        if (bad[t]) {
          const int blk = min(tile0 + warp * 8 * kMmaSets + 8 * t + row, n_blocks - 1);
          out = nan_heads(static_cast<const uint8_t*>(p.bounds) + ((size_t)bh * n_blocks + blk) * 2 * kCacheD +
                              quad * kPerLane8,
                          q, quad);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const double v = (u[t][0][c] + u[t][1][c]) * s[t];
          if (quad * 2 + c < rows && v == v && !((out >> (quad * 2 + c)) & 1u)) {
            best[t] = fmax(best[t], v);
            any[t] = true;
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kMmaSets; ++t) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        best[t] = fmax(best[t], __shfl_xor_sync(0xffffffffu, best[t], o));
        any[t] |= __shfl_xor_sync(0xffffffffu, (int)any[t], o) != 0;
      }
      if (quad == 0) put_key(p, unit, n_blocks, count, tile0 + warp * 8 * kMmaSets + 8 * t + row, any[t], best[t]);
    }
  }
  grid_release();
}

// bf16 bounds, which may be infinite: 0 * inf is not 0, so the factor is selected. Eight lanes share
// a block: their 16-byte loads cover its bounds' rows without gaps, and the four blocks of a warp
// keep as many independent sums in flight.
constexpr int kScoreRows = 4;       // heads of the group per pass
constexpr int kLanes = 8;           // lanes per block, 16 channels each
constexpr int kPerLane = kCacheD / kLanes;
constexpr int kTile = kScoreThreads / kLanes;  // blocks of the cache per tile

__global__ void __launch_bounds__(kScoreThreads, 2) score_bf16_kernel(const SelectParams p, int tiles, int items) {
  // {max(q, 0), min(q, 0)} of a row, two channels at a time, by the lane group that owns them: the upper
  // words of their doubles, whose lower ones are zero for a bf16 value; padded, so that the eight
  // groups' reads fall into different banks
  __shared__ uint4 q[kScoreRows][kLanes][kPerLane / 2 + 1];
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane & (kLanes - 1);
  const int g = p.Hq / p.Hkv;
  const int first = (int)((long long)blockIdx.x * items / gridDim.x);
  const int end = (int)((long long)(blockIdx.x + 1) * items / gridDim.x);
  grid_wait();
  uint4 raw[2][2];  // bounds of this lane's 16 channels: [lo, hi]
  auto load = [&](int item) {
    const int bh = item / tiles / p.Nq, blk = min((item % tiles) * kTile + warp * 4 + (lane >> 3), n_blocks - 1);
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) +
                                                     ((size_t)bh * n_blocks + blk) * 2 * kCacheD + group * kPerLane);
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int e = 0; e < 2; ++e) raw[side][e] = at[side * (kCacheD / 8) + e];
  };
  if (first < end) load(first);
  int held = -1;  // unit whose first kScoreRows heads are in shared memory
  for (int item = first; item < end; ++item) {
    const int unit = item / tiles;  // (b, kv head, query)
    const int i = unit % p.Nq, bh = unit / p.Nq;
    const int last = last_seen(p, bh / p.Hkv, i);
    const int count = last >= 0 ? last / p.block + 1 : 0;
    const int tile0 = (item % tiles) * kTile;
    uint4 cur[2][2];
#pragma unroll
    for (int e = 0; e < 4; ++e) cur[e >> 1][e & 1] = raw[e >> 1][e & 1];
    double best = -INFINITY;
    bool any = false;  // a score that is a number
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
          reinterpret_cast<uint2*>(q[r][c / kPerLane])[c % kPerLane] =
              make_uint2(__double2hiint(x > 0.0 || x != x ? x : 0.0), __double2hiint(x > 0.0 ? 0.0 : x));
        }
        __syncthreads();
        held = unit;
      }
      double u[kScoreRows];
#pragma unroll
      for (int r = 0; r < kScoreRows; ++r) u[r] = 0.0;
#pragma unroll
      for (int e8 = 0; e8 < 2; ++e8) {
        float lo[8], hi[8];
        Row8<false>::floats(cur[0][e8], lo);
        Row8<false>::floats(cur[1][e8], hi);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const double l[2] = {lo[e], lo[e + 1]}, h[2] = {hi[e], hi[e + 1]};
#pragma unroll
          for (int r = 0; r < kScoreRows; ++r) {
            const uint4 both = q[r][group][e8 * 4 + e / 2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const double up = __hiloint2double(w ? both.z : both.x, 0), down = __hiloint2double(w ? both.w : both.y, 0);
              const bool neg = down < 0.0;
              u[r] = fma(neg ? down : up, neg ? l[w] : h[w], u[r]);
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kScoreRows; ++r) {
        double v = u[r];
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (r < rows && v == v) {
          best = fmax(best, v);
          any = true;
        }
      }
    }
    if (group == 0) put_key(p, unit, n_blocks, count, tile0 + warp * 4 + (lane >> 3), any, best);
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
  topk_in_order<kPickThreads>(
      sh, count, k,
      [&](int i, unsigned long long(&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < count) x[e] = keys[i + e];
      },
      nullptr, idx);
  grid_release();
}

}  // namespace

cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t s) {
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int tile = p.fp8 ? kMmaTile : kTile;
  const int tiles = (n_blocks + tile - 1) / tile;
  const unsigned units = (unsigned)(p.B * p.Hkv * p.Nq);
  const int items = (int)units * tiles;
  const unsigned grid = (unsigned)min(items, kScoreCtas);
  const cudaError_t e = launch_dependent(p.fp8 ? score_fp8_kernel : score_bf16_kernel, grid, kScoreThreads, 0, s, p, tiles, items);
  if (e != cudaSuccess) return e;
  return launch_dependent(pick_kernel, units, kPickThreads, 0, s, p);
}

}  // namespace fa
