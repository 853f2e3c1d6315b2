// fa_cache_weights.cu -- the attention weights that a step gives the keys of a cache, added up.
#include "fa.h"
#include "fa_cache.h"
#include "fa_internal.h"

namespace fa {
namespace {

// One CTA per 128 keys of a (batch entry, kv head): thread = key, its K row in shared
// memory, the query rows of the group one after the other.
template <bool FP8>
__global__ void __launch_bounds__(128) weights_kernel(const WeightsParams p, int tiles) {
  constexpr int kElem = FP8 ? 1 : 2;
  extern __shared__ float ksm[];  // [128][kCacheD + 1]
  __shared__ float q[kCacheD];
  const int bh = blockIdx.x / tiles, b = bh / p.Hkv;
  const int key0 = (blockIdx.x % tiles) * 128;
  const int len = cache_len(p.lens, b, p.Nk);
  if (key0 >= len) return;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int key = key0 + threadIdx.x;
  for (int e = threadIdx.x; e < 128 * (kCacheD / 8); e += 128) {
    const int r = e / (kCacheD / 8), c = e % (kCacheD / 8) * 8;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (key0 + r < len)
      Row8<FP8>::floats(*reinterpret_cast<const typename Row8<FP8>::Raw*>(
                            static_cast<const char*>(p.k) + (((size_t)bh * p.Nk + key0 + r) * kCacheD + c) * kElem),
                        f);
    for (int u = 0; u < 8; ++u) ksm[r * (kCacheD + 1) + c + u] = f[u];
  }
  float ks = p.scale;
  if (FP8) ks *= p.ks[(size_t)bh * n_blocks + min(key, p.Nk - 1) / p.block];
  const int rows = p.Hq / p.Hkv * p.Nq;
  float sum = 0.f;
  for (int r = 0; r < rows; ++r) {
    const size_t row = (size_t)bh * rows + r;
    const int last = p.causal ? len - p.Nq + r % p.Nq : len - 1;
    if (last < key0) continue;
    __syncthreads();
    q[threadIdx.x] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row * kCacheD + threadIdx.x]);
    __syncthreads();
    const float lse = p.lse[row];
    if (key > last || lse == -INFINITY) continue;
    float s = 0.f;
    for (int c = 0; c < kCacheD; ++c) s += q[c] * ksm[threadIdx.x * (kCacheD + 1) + c];
    sum += expf(s * ks - lse);
  }
  if (key < len) p.acc[(size_t)bh * p.Nk + key] += sum;
}

}  // namespace

cudaError_t launch_cache_weights(const WeightsParams& p, cudaStream_t s) {
  const int tiles = (p.Nk + 127) / 128;
  constexpr int kSmem = 128 * (kCacheD + 1) * 4;
  static std::atomic<uint64_t> done8{0}, done16{0};
  cudaError_t e = p.fp8 ? ensure_smem_limit(weights_kernel<true>, kSmem, done8)
                        : ensure_smem_limit(weights_kernel<false>, kSmem, done16);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((long long)p.B * p.Hkv * tiles);
  if (p.fp8)
    weights_kernel<true><<<grid, 128, kSmem, s>>>(p, tiles);
  else
    weights_kernel<false><<<grid, 128, kSmem, s>>>(p, tiles);
  return cudaGetLastError();
}

}  // namespace fa
