// fa_topk.cuh -- the k largest of n keys by one CTA, in index order, ties to the lowest
// index: the choice behind block selection and eviction.
//
// Keys are unsigned integers in the order of the floating values they come from
// (order_key). A radix selection goes down the key from its top 11 bits: a histogram of the
// next digit of the keys that still match gives the digit of the k-th largest, and so the
// key itself (the threshold) and how many of its equals are taken. It stops early once a
// histogram bin is taken whole: then every key with that prefix or a larger one is in.
// The caller's load of the keys counts their top digits; one walk gathers the chosen bin (a
// few percent of the keys, unless most are equal), on which the lower digits are decided. A last
// walk turns the keys into bits, which a scan over the threads turns into sorted indices. Bound by
// instructions: with this walk instead of one that counts and one that scans and writes, 16-byte
// stores of the keys and the number of threads known to the compiler, evicting from 128 heads of
// 32768 went from 120.5 to 113.8 us, from 32 of 8192 from 17.3 to 15.5.
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
  alignas(8) uint32_t hist[kTopkBins];
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
template <int kThreads, typename Key>
__device__ __forceinline__ void topk_find_bin(TopkShared<Key>& sh, uint32_t need) {
  constexpr int warps = kThreads / 32, per = kTopkBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b0 = tid * per;  // a run of bins per thread
  uint32_t bins[per], sum = 0;
#pragma unroll
  for (int e = 0; e < per; e += 2) {
    const uint2 two = *reinterpret_cast<const uint2*>(&sh.hist[b0 + e]);
    bins[e] = two.x, bins[e + 1] = two.y;
    sum += two.x + two.y;
  }
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
#pragma unroll
    for (int e = per - 1; e >= 0; --e) {
      const uint32_t c = bins[e];
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

// Writes the indices of the k largest of n keys in ascending order to out[0, k). key4(i, x) gives
// keys i .. i + 3 (those below n), i a multiple of 4. `stage`, or null: shared memory for
// 32 indices per thread (or n, if that is less) that are written out in whole lines; it may be where
// the first so many keys lie. The histogram of the top digits is complete (topk_count of every
// key, then __syncthreads), unless k = 0 or k = n, when it is not read. All kThreads threads of the CTA
// call it.
template <int kThreads, typename Key, typename Key4Fn>
__device__ __forceinline__ void topk_in_order(TopkShared<Key>& sh, int n, int k, Key4Fn key4, int* stage, int* out) {
  constexpr int warps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
      topk_find_bin<kThreads>(sh, need);
      prefix |= (Key)sh.bin << shift;
      mask |= (Key)digit << shift;
      need -= sh.above;
      const uint32_t count = sh.count;
      if (count == need || shift == 0) break;  // the bin is taken whole, or is one key
      __syncthreads();                         // every thread has read the result
      const bool gather = !in_list && count <= kTopkList;
      for (int i = tid; i < kTopkBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
      const int next = max(shift - kTopkBits, 0);
      const uint32_t next_digit = (1u << (shift - next)) - 1u;
      if (in_list) {
        for (uint32_t i = tid; i < sh.listed; i += kThreads) {
          const Key x = sh.list[i];
          if ((x & mask) == prefix) atomicAdd(&sh.hist[(uint32_t)(x >> next) & next_digit], 1u);
        }
      } else {
        for (int i = i0 + 4 * lane; i < i1; i += 128) {
          Key x[4] = {(Key)~prefix, (Key)~prefix, (Key)~prefix, (Key)~prefix};  // not in the bin
          key4(i, x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (((x[e] ^ prefix) & mask) == 0) {
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
  // What is taken: a thread has a run of up to 32 keys, and a bit for each; a scan over all threads
  // gives it its first rank. Lanes begin at different places of their runs, for the sake of the banks.
  const int steps = min(8, (n + 4 * kThreads - 1) / (4 * kThreads)), run = 4 * steps;
  uint32_t above_before = 0, equal_before = 0;  // in the segments before this one
  for (int seg = 0; seg < n; seg += run * kThreads) {
    const int key0 = seg + run * tid;
    uint32_t above = 0, equal = 0;
#pragma unroll 2
    for (int j = 0, c = (lane & 7) * steps >> 3; j < steps; ++j, c = c + 1 == steps ? 0 : c + 1) {
      const int i = key0 + 4 * c;
      if (i < n) {
        Key x[4] = {0, 0, 0, 0};
        key4(i, x);
        uint32_t a = 0, q = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (x[e] > (prefix | ~mask)) a |= 1u << e;
          if (x[e] >= prefix) q |= 1u << e;
        }
        above |= a << (4 * c);
        equal |= q << (4 * c);
      }
    }
    if (key0 + 32 > n) equal &= key0 < n ? (1u << (n - key0)) - 1u : 0u;  // the bits of keys that are there
    above &= equal;
    equal ^= above;
    const uint32_t mine = __popc(above) | __popc(equal) << 16;  // a warp has at most 1024 keys
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();  // the histogram or the last segment's counts have been read, and the keys of this one
    if (lane == 31) {
      sh.hist[warp] = inc & 0xFFFFu;
      sh.hist[32 + warp] = inc >> 16;
    }
    __syncthreads();
    const uint32_t all_a = lane < warps ? sh.hist[lane] : 0u, all_e = lane < warps ? sh.hist[32 + lane] : 0u;
    const uint32_t first_taken = above_before + min(equal_before, need);  // of the segment
    const uint32_t e0 = equal_before + __reduce_add_sync(0xffffffffu, lane < warp ? all_e : 0u) + ((inc - mine) >> 16);
    uint32_t rank = above_before + __reduce_add_sync(0xffffffffu, lane < warp ? all_a : 0u) + ((inc - mine) & 0xFFFFu) +
                    min(e0, need);
    above_before += __reduce_add_sync(0xffffffffu, all_a);
    equal_before += __reduce_add_sync(0xffffffffu, all_e);
    // of the equals, the first that are still wanted
    for (uint32_t left = need - min(need, e0); equal && left; --left) {
      above |= equal & -equal;
      equal &= equal - 1;
    }
    int* to = stage ? stage - first_taken : out;
    for (; above; above &= above - 1) to[rank++] = key0 + __ffs(above) - 1;
    if (stage) {
      __syncthreads();
      const uint32_t end = above_before + min(equal_before, need);
      for (uint32_t r = first_taken + tid; r < end; r += kThreads) out[r] = stage[r - first_taken];
    }
  }
}

}  // namespace fa
