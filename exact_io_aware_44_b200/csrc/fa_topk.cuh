// fa_topk.cuh -- the k largest of n keys by one CTA, in index order, ties to the lowest
// index: the choice behind block selection and eviction.
//
// Keys are unsigned integers in the order of the floating values they come from
// (order_key). A radix selection goes down the key from its top 11 bits: a histogram of the
// next digit of the keys that still match gives the digit of the k-th largest, and so the
// key itself (the threshold) and how many of its equals are taken. It stops early once a
// histogram bin is taken whole: then every key with that prefix or a larger one is in.
// The caller's load of the keys counts their top digits; one walk gathers the chosen bin (a
// few percent of the keys, unless most are equal), on which the lower digits are decided. Then
// a warp owns a contiguous range of keys, four to a lane: one walk counts what it takes, a last
// one writes the indices behind those of the warps before it, so that they come out sorted.
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

constexpr int kTopkBits = 11;     // of the key per digit
constexpr int kTopkBins = 1 << kTopkBits;
constexpr int kTopkList = 2048;   // keys of the chosen bin that are gathered

template <typename Key>
struct TopkShared {
  uint32_t hist[kTopkBins];
  Key list[kTopkList];
  uint32_t warp_sum[32];
  uint32_t bin, above, count, listed;
};

// Before the keys are loaded: empties the histogram (then __syncthreads).
template <typename Key>
__device__ __forceinline__ void topk_begin(TopkShared<Key>& sh) {
  for (int i = threadIdx.x; i < kTopkBins; i += blockDim.x) sh.hist[i] = 0;
  if (threadIdx.x == 0) sh.listed = 0;
}
// For each key as it is loaded.
template <typename Key>
__device__ __forceinline__ void topk_count(TopkShared<Key>& sh, Key x) {
  atomicAdd(&sh.hist[(uint32_t)(x >> (sizeof(Key) * 8 - kTopkBits))], 1u);
}

// The bin of the histogram that holds the need-th largest: sh.bin, the keys above it in
// sh.above, its own in sh.count. All threads; the histogram is complete.
template <typename Key>
__device__ __forceinline__ void topk_find_bin(TopkShared<Key>& sh, uint32_t need) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int per = kTopkBins / blockDim.x, b0 = tid * per;  // a run of bins per thread
  uint32_t sum = 0;
  for (int e = 0; e < per; ++e) sum += sh.hist[b0 + e];
  uint32_t above = sum;  // inclusive suffix sum over the warp's lanes, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_down_sync(0xffffffffu, above, o);
    if (lane + o < 32) above += v;
  }
  if (lane == 0) sh.warp_sum[warp] = above;
  __syncthreads();
  above += __reduce_add_sync(0xffffffffu, lane > warp && lane < warps ? sh.warp_sum[lane] : 0u);
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
}

// Writes the indices of the k largest of n keys in ascending order through emit(rank, index),
// rank in [0, k). key4(i, x) gives keys i .. i + 3 (those below n), i a multiple of 4. The
// histogram of the top digits is complete (topk_count of every key, then __syncthreads),
// unless k = 0 or k = n, when it is not read. All threads of the CTA (a multiple
// of 32, at most 1024) call it.
template <typename Key, typename Key4Fn, typename EmitFn>
__device__ __forceinline__ void topk_in_order(TopkShared<Key>& sh, int n, int k, Key4Fn key4, EmitFn emit) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  constexpr int kKeyBits = sizeof(Key) * 8;
  // A warp's range of keys, in steps of 128.
  const int per = (n + warps * 128 - 1) / (warps * 128) * 128;
  const int i0 = min(n, warp * per), i1 = min(n, i0 + per);
  // keys whose masked value exceeds the prefix are in, and the first `need` that equal it;
  // with mask = 0 (k = 0 or k = n) the first k keys are "equal"
  Key prefix = 0, mask = 0;
  uint32_t need = (uint32_t)k;
  if (k > 0 && k < n) {
    int top = kKeyBits;
    bool in_list = false;
    for (;;) {
      const int shift = max(top - kTopkBits, 0);
      const uint32_t digit = (1u << (top - shift)) - 1u;
      topk_find_bin(sh, need);
      prefix |= (Key)sh.bin << shift;
      mask |= (Key)digit << shift;
      need -= sh.above;
      const uint32_t count = sh.count;
      if (count == need || shift == 0) break;  // the bin is taken whole, or is one key
      __syncthreads();                         // every thread has read the result
      const bool gather = !in_list && count <= kTopkList;
      for (int i = tid; i < kTopkBins; i += blockDim.x) sh.hist[i] = 0;
      __syncthreads();
      const int next = max(shift - kTopkBits, 0);
      const uint32_t next_digit = (1u << (shift - next)) - 1u;
      if (in_list) {
        for (uint32_t i = tid; i < sh.listed; i += blockDim.x) {
          const Key x = sh.list[i];
          if ((x & mask) == prefix) atomicAdd(&sh.hist[(uint32_t)(x >> next) & next_digit], 1u);
        }
      } else {
        for (int i = i0 + 4 * lane; i < i1; i += 128) {
          Key x[4];
          key4(i, x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (i + e < i1 && (x[e] & mask) == prefix) {
              atomicAdd(&sh.hist[(uint32_t)(x[e] >> next) & next_digit], 1u);
              if (gather) sh.list[atomicAdd(&sh.listed, 1u)] = x[e];
            }
          }
        }
        in_list = gather;
      }
      top = shift;
      __syncthreads();
    }
  }
  // keys above and equal in this warp's range, and so in the ranges before it
  uint32_t above = 0, equal = 0;
  for (int i = i0 + 4 * lane; i < i1; i += 128) {
    Key x[4];
    key4(i, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const Key y = x[e] & mask;
      above += i + e < i1 && y > prefix;
      equal += i + e < i1 && y == prefix;
    }
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();  // the histogram and the result have been read: it takes the warps' counts
  if (lane == 0) {
    sh.hist[warp] = above;
    sh.hist[32 + warp] = equal;
  }
  __syncthreads();
  uint32_t a0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.hist[lane] : 0u);
  uint32_t e0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.hist[32 + lane] : 0u);
  for (int ib = i0; ib < i1; ib += 128) {
    const int i = ib + 4 * lane;
    Key x[4];
    if (i < i1) key4(i, x);
    uint32_t fa = 0, fe = 0;  // this lane's keys that are above, and equal
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const Key y = x[e] & mask;
      fa |= (uint32_t)(i + e < i1 && y > prefix) << e;
      fe |= (uint32_t)(i + e < i1 && y == prefix) << e;
    }
    const uint32_t mine = __popc(fa) | __popc(fe) << 16;
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const uint32_t total = __shfl_sync(0xffffffffu, inc, 31), excl = inc - mine;
    uint32_t a = a0 + (excl & 0xFFFFu), q = e0 + (excl >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((fa >> e) & 1u)
        emit(a++ + min(q, need), i + e);
      else if ((fe >> e) & 1u) {
        if (q < need) emit(a + q, i + e);
        ++q;
      }
    }
    a0 += total & 0xFFFFu;
    e0 += total >> 16;
  }
}

}  // namespace fa
