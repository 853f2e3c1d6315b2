// fa_topk.cuh -- the k largest of n keys by one CTA, in index order, ties to the lowest
// index: the choice behind block selection and eviction.
//
// Keys are unsigned integers in the order of the floating values they come from
// (order_key). A radix selection walks the key from its top 11 bits: a histogram of the next
// digit of all keys that still match the prefix gives the digit of the k-th largest, and so
// the key itself (the threshold) and how many of its equals are taken. It stops early once
// a histogram bin is taken whole: then every key with that prefix or a larger one is in.
// A second walk over the keys writes the indices: each warp takes a contiguous range,
// counts, and writes behind the warps before it, so the indices come out sorted.
#pragma once

#include <stdint.h>

namespace fa {

// Unsigned order of a float or double: larger value, larger key; -0 equals +0; NaN is the lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 + 0 = +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return 0ull;
  const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
  return b & 0x8000000000000000ull ? ~b : b | 0x8000000000000000ull;
}

constexpr int kTopkBits = 11;  // of the key per walk: fewer, longer walks than with bytes

struct TopkShared {
  uint32_t hist[1 << kTopkBits];
  uint32_t warp_sum[32];
  uint32_t warp_above[32], warp_equal[32];
  uint32_t bin, above, count;
};

// Writes the indices of the k largest of keys[0, n) (key(i) gives the i-th) in ascending
// order through emit(rank, index), rank in [0, k). All threads of the CTA (a multiple of
// 32, at most 1024) call it; 0 <= k <= n. The shared block may be reused after a
// __syncthreads.
template <typename Key, typename KeyFn, typename EmitFn>
__device__ __forceinline__ void topk_in_order(TopkShared& sh, int n, int k, KeyFn key, EmitFn emit) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  constexpr int kKeyBits = sizeof(Key) * 8, kBins = 1 << kTopkBits;
  // threshold: keys > lim are in; of the keys == lim (under `mask`) the first `need`
  Key prefix = 0, mask = 0;
  uint32_t need = (uint32_t)k;
  if (k < n && k > 0) {
    for (int top = kKeyBits; top > 0; top -= kTopkBits) {
      const int shift = max(top - kTopkBits, 0);
      const uint32_t digit = (1u << (top - shift)) - 1u;
      for (int i = tid; i < kBins; i += blockDim.x) sh.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += blockDim.x) {
        const Key x = key(i);
        if ((x & mask) == prefix) atomicAdd(&sh.hist[(uint32_t)(x >> shift) & digit], 1u);
      }
      __syncthreads();
      // the bin that holds the k-th largest: suffix sums over contiguous shares of the bins, from the
      // top down: warp w owns bins [w * per_warp, ...), a lane a run of them
      const int per = kBins / blockDim.x > 0 ? kBins / blockDim.x : 1;
      const int b0 = tid * per;
      uint32_t sum = 0;
      if (b0 < kBins)
        for (int e = 0; e < per; ++e) sum += sh.hist[b0 + e];
      uint32_t above = sum;  // inclusive suffix sum over the warp's lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += v;
      }
      if (lane == 0) sh.warp_sum[warp] = above;
      __syncthreads();
      for (int w = warp + 1; w < warps; ++w) above += sh.warp_sum[w];
      above -= sum;  // keys in the bins of higher threads
      if (above < need && above + sum >= need) {
        uint32_t a = above;
        for (int e = per - 1; e >= 0; --e) {
          const uint32_t c = sh.hist[b0 + e];
          if (a < need && a + c >= need) {
            sh.bin = b0 + e;
            sh.above = a;
            sh.count = c;
          }
          a += c;
        }
      }
      __syncthreads();
      prefix |= (Key)sh.bin << shift;
      mask |= (Key)digit << shift;
      need -= sh.above;
      if (sh.count == need) break;  // the bin is taken whole (uniform: read after the barrier)
      __syncthreads();              // warp_sum and the result are written again
    }
  }
  // every key whose masked value exceeds the prefix is in, and the first `need` that equal it;
  // with mask = 0 (k = 0 or k = n) the first k keys are "equal"
  const int per = ((n + warps - 1) / warps + 31) / 32 * 32;
  const int i0 = min(n, warp * per), i1 = min(n, i0 + per);
  uint32_t above = 0, equal = 0;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const Key x = in ? (Key)(key(i + lane) & mask) : (Key)0;
    above += __popc(__ballot_sync(0xffffffffu, in && x > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, in && x == prefix));
  }
  if (lane == 0) {
    sh.warp_above[warp] = above;
    sh.warp_equal[warp] = equal;
  }
  __syncthreads();
  uint32_t a0 = 0, e0 = 0;
  for (int w = 0; w < warp; ++w) {
    a0 += sh.warp_above[w];
    e0 += sh.warp_equal[w];
  }
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const Key x = in ? (Key)(key(i + lane) & mask) : (Key)0;
    const uint32_t ba = __ballot_sync(0xffffffffu, in && x > prefix);
    const uint32_t be = __ballot_sync(0xffffffffu, in && x == prefix);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t a = a0 + __popc(ba & below), e = e0 + __popc(be & below);
    if ((ba >> lane) & 1u)
      emit(a + min(e, need), i + lane);
    else if (((be >> lane) & 1u) && e < need)
      emit(a + e, i + lane);
    a0 += __popc(ba);
    e0 += __popc(be);
  }
}

}  // namespace fa
