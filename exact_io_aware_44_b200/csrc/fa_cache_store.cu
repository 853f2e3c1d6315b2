// fa_cache_store.cu -- writing an 8-bit key/value cache, and the per-channel bounds of
// its blocks.
//
// A block of `block` tokens of one head has one scale, a power of two
//   s = 2^e, the smallest e >= -100 with amax <= 448 * 2^e,
// and holds code = e4m3(x / s). With a power of two the division is exact, so the only
// rounding is E4M3's own (half a step, 2^-4 of the value); and when a later token needs a
// larger scale, the block's older codes are multiplied by s_old / s, which only codes that
// become subnormal feel. An E4M3 value keeps its relative precision whatever the scale, so
// a scale up to twice the smallest costs nothing but one binade of the range.
//
// Both kernels have 8 warps of 16 tokens each (the bounds 16, 32 or 64: at most a block), two rows per
// load instruction (16 lanes a row, 8 elements a lane). 16 is the smallest block, so a
// warp's result belongs to one block, and blocks of more warps meet in shared memory.
#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_launch.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerWarp = 16;
constexpr int kLoads = kRowsPerWarp / 2;  // two rows per warp-wide load

// Smallest e >= kMinScaleExp with amax <= 448 * 2^e (448 = 1.75 * 2^8), as the float 2^e.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int E = (int)(bits >> 23) - 127;  // subnormals end up below the floor
  const int e = max(E - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), kMinScaleExp);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Larger |x| of two bf16 values as float bits; infinities and NaN count as zero.
__device__ __forceinline__ uint32_t finite_abs_max(uint32_t m, uint32_t pair) {
  const uint32_t a = (pair << 16) & 0x7FFFFFFFu, b = pair & 0x7FFF0000u;
  if (a < 0x7F800000u) m = max(m, a);
  if (b < 0x7F800000u) m = max(m, b);
  return m;
}

// Larger |x| of two pairs of bf16 values; NaN counts as nothing.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t pair) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                   __habs2(*reinterpret_cast<const __nv_bfloat162*>(&pair)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Two bf16 values times a power of two in bf16 (exact, but for results far below E4M3's
// smallest number), as E4M3.
__device__ __forceinline__ uint32_t scaled_e4m3x2(uint32_t pair, __nv_bfloat162 inv) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&pair), inv);
  const float2 f = bf162_bits_to_float2(*reinterpret_cast<const uint32_t*>(&r));
  return float2_to_e4m3x2(f.x, f.y);
}

// A CTA for each tile. With the packed arithmetic above, B4 Hkv8 and 8192 tokens of each take 31 us,
// the time of their bytes at the copy bandwidth; element by element they took 53. (Persistent
// CTAs with bulk copies in three stages ahead: 40 us.)
__global__ void __launch_bounds__(kThreads, 4) store_kernel(const StoreParams p, int tiles) {
  __shared__ uint32_t warp_max[8];
  grid_wait();
  // (tile, head, batch entry, K or V), tile fastest
  const int t = blockIdx.x % tiles;
  const unsigned v = blockIdx.x / tiles, heads = (unsigned)(p.B * p.Hkv);
  const bool is_v = v >= heads;
  const int bh = (int)(is_v ? v - heads : v);
  const int len = cache_len(p.lens, bh / p.Hkv, p.Nk);
  const int start = len - p.n_new;  // position of the first new token (negative ones are dropped)
  const int tile0 = (max(start, 0) / kCacheTile + t) * kCacheTile;
  if (tile0 >= len) return;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + (size_t)bh * p.n_new * kCacheD;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = tile0 + warp * kRowsPerWarp + (lane >> 4);
  const int col = (lane & 15) * 8;
  uint4 r[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int pos = row0 + 2 * i;
    r[i] = make_uint4(0, 0, 0, 0);
    if (pos >= start && pos < len) r[i] = *reinterpret_cast<const uint4*>(x + (size_t)(pos - start) * kCacheD + col);
  }
  // pairs by packed maxima (which skip NaN); a warp that meets an infinity takes them one by one
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    m2 = abs_max2(abs_max2(abs_max2(abs_max2(m2, r[i].x), r[i].y), r[i].z), r[i].w);
  uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 << 16, m2 & 0xFFFF0000u));
  if (m >= 0x7F800000u) {
    m = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      m = finite_abs_max(finite_abs_max(finite_abs_max(finite_abs_max(m, r[i].x), r[i].y), r[i].z), r[i].w);
    m = __reduce_max_sync(0xffffffffu, m);
  }
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
  const int per = p.block / kRowsPerWarp;  // warps per block
  const int w0 = warp / per * per;
  for (int w = w0; w < w0 + per; ++w) m = max(m, warp_max[w]);
  const int blk = (tile0 + warp * kRowsPerWarp) / p.block;
  const int b0 = blk * p.block;
  if (b0 + p.block <= start || b0 >= len) return;  // no new token in this block
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  float* scales = (is_v ? p.vs : p.ks) + (size_t)bh * n_blocks;
  uint8_t* codes = static_cast<uint8_t*>(is_v ? p.cv : p.ck) + (size_t)bh * p.Nk * kCacheD;
  const bool has_old = b0 < start;
  float sc = scale_for(__uint_as_float(m));
  float s_old = sc;
  if (has_old) {
    s_old = scales[blk];
    sc = fmaxf(sc, s_old);
  }
  // every warp of the block has read the scale before one writes it
  asm volatile("bar.sync %0, %1;" ::"r"(1 + w0 / per), "r"(per * 32) : "memory");
  if (warp == w0 && lane == 0) scales[blk] = sc;
  // a scale from elsewhere may be no power of two, or 2^127, whose reciprocal is not a normal number
  const bool pow2 = (__float_as_uint(sc) & 0x7FFFFFu) == 0 && __float_as_uint(sc) < 254u << 23;
  const float inv = pow2 ? __uint_as_float((254u << 23) - __float_as_uint(sc)) : 0.f;  // 2^-e, exactly
  const __nv_bfloat162 inv2 = __float2bfloat162_rn(inv);
  const float ratio = s_old / sc;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int pos = row0 + 2 * i;
    uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)pos * kCacheD + col);
    if (pos >= start && pos < len) {
      if (pow2) {
        *dst = make_uint2(scaled_e4m3x2(r[i].x, inv2) | scaled_e4m3x2(r[i].y, inv2) << 16,
                          scaled_e4m3x2(r[i].z, inv2) | scaled_e4m3x2(r[i].w, inv2) << 16);
      } else {
        float f[8];
        Row8<false>::floats(r[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fdiv_rn(f[e], sc);
        *dst = make_uint2(float2_to_e4m3x2(f[0], f[1]) | (uint32_t)float2_to_e4m3x2(f[2], f[3]) << 16,
                          float2_to_e4m3x2(f[4], f[5]) | (uint32_t)float2_to_e4m3x2(f[6], f[7]) << 16);
      }
    } else if (pos < start && ratio != 1.f) {  // an older token of a block whose scale grew
      float f[8];
      Row8<true>::floats(*dst, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= ratio;
      *dst = make_uint2(float2_to_e4m3x2(f[0], f[1]) | (uint32_t)float2_to_e4m3x2(f[2], f[3]) << 16,
                        float2_to_e4m3x2(f[4], f[5]) | (uint32_t)float2_to_e4m3x2(f[6], f[7]) << 16);
    }
  }
}

// Element pairs that hold 8 elements of a row, with a minimum and a maximum that skip NaN.
template <bool FP8>
struct Pairs;
template <>
struct Pairs<true> {
  using V = __half2;
  static constexpr uint32_t kInf = 0x7C007C00u;
  static __device__ __forceinline__ void pairs(const uint2& r, uint32_t (&w)[4]) {
    w[0] = e4m3x2_to_half2((uint16_t)r.x);
    w[1] = e4m3x2_to_half2((uint16_t)(r.x >> 16));
    w[2] = e4m3x2_to_half2((uint16_t)r.y);
    w[3] = e4m3x2_to_half2((uint16_t)(r.y >> 16));
  }
  static __device__ __forceinline__ void store(void* p, const uint32_t (&w)[4]) {
    *static_cast<uint2*>(p) = make_uint2(half2_to_e4m3x2(w[0]) | (uint32_t)half2_to_e4m3x2(w[1]) << 16,
                                         half2_to_e4m3x2(w[2]) | (uint32_t)half2_to_e4m3x2(w[3]) << 16);
  }
};
template <>
struct Pairs<false> {
  using V = __nv_bfloat162;
  static constexpr uint32_t kInf = 0x7F807F80u;
  static __device__ __forceinline__ void pairs(const uint4& r, uint32_t (&w)[4]) {
    w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
  }
  static __device__ __forceinline__ void store(void* p, const uint32_t (&w)[4]) {
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename V>
__device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b) {
  const V r = __hmin2(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename V>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  const V r = __hmax2(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A warp takes `rows` tokens (16, or up to 64 of one block): the fewer warps share a block, the less is
// left to be combined. All bounds of B4 Hkv8 and 32768 tokens, blocks of 64, take 25.5 us with 64
// tokens a warp (5.3 TB/s), 27.0 with 32, 31.8 with 16; of 8192 tokens, behind their store, 41.8,
// 40.6 and 41.6 for both. (With each load behind a test of its token's place: 47 and 46.)
template <bool FP8>
__global__ void __launch_bounds__(kThreads) bounds_kernel(const BoundsParams p, int tiles, int rows) {
  using P = Pairs<FP8>;
  using V = typename P::V;
  constexpr int kElem = FP8 ? 1 : 2;
  __shared__ uint32_t part[8][2][16][4];  // a warp's bounds of its 16 rows, by channel group
  const int t = blockIdx.x % tiles;
  const int bh = blockIdx.x / tiles;
  grid_wait();
  const int len = cache_len(p.lens, bh / p.Hkv, p.Nk);
  const int start = p.n_new > 0 ? max(len - p.n_new, 0) : 0;
  const int tile = rows * (kThreads / 32);
  const int tile0 = (start / tile + t) * tile;
  if (tile0 >= len) return;
  const char* k = static_cast<const char*>(p.k) + (size_t)bh * p.Nk * kCacheD * kElem;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_w = tile0 + warp * rows, group = lane & 15;
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) lo[e] = P::kInf, hi[e] = P::kInf | 0x80008000u;
  for (int r = 0; r < rows; r += kRowsPerWarp) {
    const int row0 = row_w + r + (lane >> 4);
    // all loads before the first use; behind the end the last token, which the block holds too (or the
    // block is not written)
    typename Row8<FP8>::Raw raw[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      raw[i] = *reinterpret_cast<const typename Row8<FP8>::Raw*>(
          k + ((size_t)min(row0 + 2 * i, len - 1) * kCacheD + group * 8) * kElem);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t w[4];
      P::pairs(raw[i], w);
#pragma unroll
      for (int e = 0; e < 4; ++e) lo[e] = pair_min<V>(lo[e], w[e]), hi[e] = pair_max<V>(hi[e], w[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    lo[e] = pair_min<V>(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], 16));
    hi[e] = pair_max<V>(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], 16));
    part[warp][0][group][e] = lo[e];  // both half-warps write the same value
    part[warp][1][group][e] = hi[e];
  }
  __syncthreads();
  const int per = p.block / rows;
  const int blk = row_w / p.block;
  if (warp % per != 0 || blk * p.block + p.block <= start || blk * p.block >= len) return;
  const int side = lane >> 4;  // lanes 0-15 the minimum, 16-31 the maximum
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = part[warp][side][group][e];
    for (int o = 1; o < per; ++o) {
      const uint32_t u = part[warp + o][side][group][e];
      w[e] = side ? pair_max<V>(w[e], u) : pair_min<V>(w[e], u);
    }
  }
  P::store(static_cast<char*>(p.bounds) + (((size_t)bh * n_blocks + blk) * 2 + side) * kCacheD * kElem +
               group * 8 * kElem,
           w);
}

// Tiles that the newest n_new tokens can touch, whatever the length.
int touched_tiles(int n_new, int Nk, int tile) {
  const int all = (Nk + tile - 1) / tile;
  if (n_new <= 0 || n_new >= Nk) return all;
  return min(all, (n_new + tile - 2) / tile + 1);
}

}  // namespace

cudaError_t launch_cache_store(const StoreParams& p, cudaStream_t s) {
  const int tiles = touched_tiles(p.n_new, p.Nk, kCacheTile);
  return launch_dependent(store_kernel, (unsigned)((size_t)2 * p.B * p.Hkv * tiles), kThreads, 0, s, p, tiles);
}

cudaError_t launch_block_bounds(const BoundsParams& p, cudaStream_t s) {
  // as many tokens a warp, up to 64, as leave 32 warps to an SM
  const long long tokens = (long long)p.B * p.Hkv * touched_tiles(p.n_new, p.Nk, kCacheTile) * kCacheTile;
  int rows = min(p.block, 64);
  while (rows > kRowsPerWarp && tokens / rows < 32 * 148) rows /= 2;
  const int tiles = touched_tiles(p.n_new, p.Nk, rows * (kThreads / 32));
  const unsigned grid = (unsigned)((size_t)p.B * p.Hkv * tiles);
  return p.fp8 ? launch_dependent(bounds_kernel<true>, grid, kThreads, 0, s, p, tiles, rows)
               : launch_dependent(bounds_kernel<false>, grid, kThreads, 0, s, p, tiles, rows);
}

}  // namespace fa
