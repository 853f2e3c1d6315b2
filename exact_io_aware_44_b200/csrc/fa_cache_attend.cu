// fa_cache_attend.cu -- attention over an 8-bit cache or over selected blocks of a cache,
// and the weights that it gives the keys: CUDA-core kernels.
#include "fa.h"
#include "fa_cache.h"
#include "fa_internal.h"

namespace fa {
namespace {

// One CTA per query row; each of four warps takes every fourth key with an online softmax
// of its own (a lane holds 4 channels), and the four are merged at the end.
template <bool FP8>
__global__ void __launch_bounds__(128) attend_kernel(const AttendParams p) {
  constexpr int kElem = FP8 ? 1 : 2;
  __shared__ float sm[4], sl[4], so[4][kCacheD];
  const long long row = blockIdx.x;
  const int i = (int)(row % p.Nq), hq = (int)(row / p.Nq % p.Hq), b = (int)(row / p.Nq / p.Hq);
  const int bh = b * p.Hkv + hq / (p.Hq / p.Hkv);
  const int len = cache_len(p.lens, b, p.Nk);
  const int last = p.causal ? len - p.Nq + i : len - 1;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float q[4];
  {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + row * kCacheD + lane * 4);
    const float2 a = bf162_bits_to_float2(w.x), c = bf162_bits_to_float2(w.y);
    q[0] = a.x, q[1] = a.y, q[2] = c.x, q[3] = c.y;
  }
  auto four = [&](const void* base, long long key, float (&x)[4]) {
    const char* at = static_cast<const char*>(base) + (((size_t)bh * p.Nk + key) * kCacheD + lane * 4) * kElem;
    float2 a, c;
    if constexpr (FP8) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
      a = half2_bits_to_float2(e4m3x2_to_half2((uint16_t)w));
      c = half2_bits_to_float2(e4m3x2_to_half2((uint16_t)(w >> 16)));
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(at);
      a = bf162_bits_to_float2(w.x), c = bf162_bits_to_float2(w.y);
    }
    x[0] = a.x, x[1] = a.y, x[2] = c.x, x[3] = c.y;
  };
  const int* idx = p.idx ? p.idx + ((size_t)bh * p.Nq + i) * p.n_select : nullptr;
  const long long slots = idx ? (long long)p.n_select * p.block : last + 1;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (long long t = warp; t < slots; t += 4) {
    long long key = t;
    if (idx) {
      const int blk = idx[t / p.block];
      if (blk < 0 || blk >= n_blocks) continue;
      key = (long long)blk * p.block + t % p.block;
    }
    if (key > last) continue;
    float k[4], v[4];
    four(p.k, key, k);
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale;
    float sv = 1.f;
    if (FP8) {
      s *= p.ks[(size_t)bh * n_blocks + key / p.block];
      sv = p.vs[(size_t)bh * n_blocks + key / p.block];
    }
    const float m_new = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : __expf(m - m_new), e = __expf(s - m_new);
    four(p.v, key, v);
    l = l * a + e;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = o[c] * a + e * sv * v[c];
    m = m_new;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int c = 0; c < 4; ++c) so[warp][lane * 4 + c] = o[c];
  __syncthreads();
  const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float ll = 0.f, oo = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float a = sm[w] == -INFINITY ? 0.f : __expf(sm[w] - mm);
    ll += sl[w] * a;
    oo += so[w][threadIdx.x] * a;
  }
  static_cast<__nv_bfloat16*>(p.o)[row * kCacheD + threadIdx.x] = __float2bfloat16(ll > 0.f ? oo / ll : 0.f);
  if (threadIdx.x == 0) p.lse[row] = ll > 0.f ? mm + logf(ll) : -INFINITY;
}

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

cudaError_t launch_cache_attend(const AttendParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)p.B * p.Hq * p.Nq);
  if (p.fp8)
    attend_kernel<true><<<grid, 128, 0, s>>>(p);
  else
    attend_kernel<false><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

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
