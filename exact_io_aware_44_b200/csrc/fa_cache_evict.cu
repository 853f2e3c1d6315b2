// fa_cache_evict.cu -- cutting a cache back to the tokens that attention has used most.
//
// keep_kernel: one CTA per (batch entry, kv head) chooses the kept tokens: the newest
// `recent`, and the largest accumulated weights of the others (ties to the older token,
// NaN last), and lists their indices in order. move_kernel: tiles of 128 kept tokens copy
// their K and V rows and weights into the new cache. In an 8-bit cache the tokens of a new
// block come from several old ones, so the block takes the largest of their scales and the
// codes of the others are multiplied by s_old / s_new: exact between powers of two, but
// for codes that become subnormal.
#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_launch.cuh"
#include "fa_internal.h"
#include "fa_topk.cuh"

namespace fa {
namespace {

constexpr int kKeepThreads = 1024;
constexpr int kThreads = 256;
constexpr int kRowsPerWarp = 16;
constexpr int kLoads = kRowsPerWarp / 2;

// The keys are walked a few times: they are put in shared memory on the way in, up to
// kKeepShared of them (160 KB); a longer cache's others are read from memory each time.
constexpr int kKeepShared = 40960;

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ TopkShared<uint32_t> sh;
  const int bh = blockIdx.x;
  topk_begin(sh);
  __syncthreads();
  grid_wait();
  const int len = cache_len(p.lens, bh / p.Hkv, p.Nk);
  const int m = min(len, p.keep);
  const int recent = min(p.recent, m);
  const int n = len - recent, k = m - recent;
  const float* acc = p.acc + (size_t)bh * p.Nk;
  int* idx = p.idx + (size_t)bh * p.keep;
  const int held = min(n, kKeepShared);
  if (k > 0 && k < n) {
    auto take = [&](int e, float x) {
      const uint32_t key = order_key(x);
      topk_count(sh, key);
      if (e < held) keys[e] = key;
    };
    int e = 0;
    if (p.Nk % 4 == 0) {  // rows of whole float4s: eight loads of four weights in flight per thread
      constexpr int kStep = 8 * 4 * kKeepThreads;
      for (; e < n; e += kStep) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = e + (u * kKeepThreads + threadIdx.x) * 4;
          if (i < n) v[u] = *reinterpret_cast<const float4*>(acc + i);  // within the row: Nk is a multiple of 4
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = e + (u * kKeepThreads + threadIdx.x) * 4;
          if (i + 3 < held) {
            const uint4 key = make_uint4(order_key(v[u].x), order_key(v[u].y), order_key(v[u].z), order_key(v[u].w));
            *reinterpret_cast<uint4*>(keys + i) = key;
            topk_count(sh, key.x), topk_count(sh, key.y), topk_count(sh, key.z), topk_count(sh, key.w);
          } else {
            if (i < n) take(i, v[u].x);
            if (i + 1 < n) take(i + 1, v[u].y);
            if (i + 2 < n) take(i + 2, v[u].z);
            if (i + 3 < n) take(i + 3, v[u].w);
          }
        }
      }
    } else {
      constexpr int kStep = 16 * kKeepThreads;
      for (; e < n; e += kStep) {
        float v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int i = e + u * kKeepThreads + threadIdx.x;
          if (i < n) v[u] = acc[i];
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int i = e + u * kKeepThreads + threadIdx.x;
          if (i < n) take(i, v[u]);
        }
      }
    }
  }
  __syncthreads();
  topk_in_order<kKeepThreads>(
      sh, n, k,
      [&](int i, uint32_t(&x)[4]) {
        if (i + 3 < held) {
          const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < n) x[e] = i + e < held ? keys[i + e] : order_key(acc[i + e]);
        }
      },
      reinterpret_cast<int*>(keys), idx);
  for (int e = threadIdx.x; e < p.keep - k; e += kKeepThreads) idx[k + e] = e < recent ? n + e : -1;
  if (bh % p.Hkv == 0 && threadIdx.x == 0) p.olens[bh / p.Hkv] = m;
  grid_release();
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads) move_kernel(const EvictParams p, int tiles) {
  using Raw = typename Row8<FP8>::Raw;
  constexpr int kElem = FP8 ? 1 : 2;
  __shared__ float warp_scale[2][8];
  const int bh = blockIdx.x / tiles;
  const int tile0 = (blockIdx.x % tiles) * kCacheTile;
  grid_wait();
  const int m = min(cache_len(p.lens, bh / p.Hkv, p.Nk), p.keep);
  if (tile0 >= m) return;
  const int* idx = p.idx + (size_t)bh * p.keep;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_w = tile0 + warp * kRowsPerWarp;
  // lane l < 16 holds the source of the warp's row l
  const int src = lane < kRowsPerWarp && row_w + lane < m ? idx[row_w + lane] : -1;
  if (src >= 0) p.oacc[(size_t)bh * p.out_Nk + row_w + lane] = p.acc[(size_t)bh * p.Nk + src];
  const int col = (lane & 15) * 8 * kElem;
  const int n_blocks = (p.Nk + p.block - 1) / p.block, out_blocks = (p.out_Nk + p.block - 1) / p.block;
  float s_src[2] = {1.f, 1.f}, s_new[2] = {1.f, 1.f};
  if (FP8) {
    if (src >= 0) {
      s_src[0] = p.ks[(size_t)bh * n_blocks + src / p.block];
      s_src[1] = p.vs[(size_t)bh * n_blocks + src / p.block];
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // scales are positive, so their bits are in their order
      const uint32_t mx = __reduce_max_sync(0xffffffffu, src >= 0 ? __float_as_uint(s_src[t]) : 0u);
      if (lane == 0) warp_scale[t][warp] = __uint_as_float(mx);
    }
    __syncthreads();
    const int per = p.block / kRowsPerWarp, w0 = warp / per * per;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float s = 0.f;
      for (int w = w0; w < w0 + per; ++w) s = fmaxf(s, warp_scale[t][w]);
      s_new[t] = s;
      if (warp == w0 && lane == 0 && row_w < m)
        (t ? p.ovs : p.oks)[(size_t)bh * out_blocks + row_w / p.block] = s;
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const char* in = static_cast<const char*>(t ? p.v : p.k) + (size_t)bh * p.Nk * kCacheD * kElem + col;
    char* out = static_cast<char*>(t ? p.ov : p.ok) + (size_t)bh * p.out_Nk * kCacheD * kElem + col;
    Raw r[kLoads];
    int from[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      from[i] = __shfl_sync(0xffffffffu, src, 2 * i + (lane >> 4));
      if (from[i] >= 0) r[i] = *reinterpret_cast<const Raw*>(in + (size_t)from[i] * kCacheD * kElem);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const float s = __shfl_sync(0xffffffffu, s_src[t], 2 * i + (lane >> 4));
      if (from[i] < 0) continue;
      if constexpr (FP8) {
        if (s != s_new[t]) {
          const float ratio = s / s_new[t];
          float f[8];
          Row8<true>::floats(r[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= ratio;
          r[i] = make_uint2(float2_to_e4m3x2(f[0], f[1]) | (uint32_t)float2_to_e4m3x2(f[2], f[3]) << 16,
                            float2_to_e4m3x2(f[4], f[5]) | (uint32_t)float2_to_e4m3x2(f[6], f[7]) << 16);
        }
      }
      *reinterpret_cast<Raw*>(out + (size_t)(row_w + 2 * i + (lane >> 4)) * kCacheD * kElem) = r[i];
    }
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = ensure_smem_limit(keep_kernel, kKeepShared * 4, configured);
  if (e != cudaSuccess) return e;
  e = launch_dependent(keep_kernel, (unsigned)(p.B * p.Hkv), kKeepThreads, (size_t)(min(p.Nk, kKeepShared) + 3) / 4 * 16, s, p);
  if (e != cudaSuccess) return e;
  const int tiles = (min(p.keep, p.Nk) + kCacheTile - 1) / kCacheTile;
  const unsigned grid = (unsigned)((size_t)p.B * p.Hkv * tiles);
  return p.fp8 ? launch_dependent(move_kernel<true>, grid, kThreads, 0, s, p, tiles)
               : launch_dependent(move_kernel<false>, grid, kThreads, 0, s, p, tiles);
}

}  // namespace fa
