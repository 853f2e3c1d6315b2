// fa_cache_sm100.cuh -- what the tensor-core kernels over a cache share: the walk over a
// CTA's slice of the key chunks, 8-bit splitting of query rows and weights, and
// reductions over a warpgroup.
//
// 8-bit operands. tcgen05.mma takes E4M3 keys and values as they lie in the cache if the
// other operand has 8 bits too (kind::f8f6f4; the two formats need not be the same). A
// query element or a softmax weight has more than the 3 significant bits of E5M2, but is a
// sum of three E5M2 numbers: the top byte of an fp16 number IS an E5M2 number, its
// value to 3 significant bits; the remainder is exact in fp16, and so on. Three terms hold
// every fp16 number exactly (split_e5m2), accumulated in fp32 columns of their own. So the cache goes from device memory to the tensor
// cores without a conversion of its own, and the few query rows pay instead: per SM, reading
// at full bandwidth, 24 cache bytes arrive per clock but only 1.5 weights (16 rows).
#pragma once

#include <cuda_fp16.h>
#include <float.h>

#include "fa_cache.h"
#include "fa_cache_launch.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int kChunk = 128;      // keys per chunk: the MMA's M
constexpr int kQScaleRing = 8;   // query scales outlive their rows: see the Q warps

// The walk (WalkParams): a unit is a set of query rows that share a sequence of key chunks,
// the keys of a sequence or of a list of blocks. All units lie end to end, and CTA i
// takes the i-th of slices of equal cost.
__device__ __forceinline__ int walk_chunks(const WalkParams& p, int b) {
  return p.lens ? (cache_len(p.lens, b, p.Nk) + (1 << p.chunk_log2) - 1) >> p.chunk_log2 : p.chunks;
}

// Chunk c of a slice: unit, chunk of the unit (cig) out of nch, number of the segment (a
// unit's part of the slice).
struct WalkPos {
  int unit, b_end, cig, nch, seg;

  __device__ __forceinline__ void next(const WalkParams& p) {
    if (++cig < nch) return;
    cig = 0;
    ++seg;
    if (++unit < b_end) return;
    int b = b_end / p.units_per_b;
    for (;;) {  // the next sequence that holds a token
      b_end += p.units_per_b;
      if (b >= p.B) return;  // past the last unit: not used again (nch stays positive, for skip)
      const int m = walk_chunks(p, b);
      if (m > 0) {
        nch = m;
        return;
      }
      unit = b_end;
      ++b;
    }
  }
  // k chunks on.
  __device__ __forceinline__ void skip(const WalkParams& p, int k) {
    while (k >= nch - cig) {
      k -= nch - cig;
      cig = nch - 1;
      next(p);
    }
    cig += k;
  }
  // Local indices of the segment's first and last chunk, for local chunk c of n.
  __device__ __forceinline__ int first(int c) const { return max(0, c - cig); }
  __device__ __forceinline__ int last(int c, int n) const { return min(n - 1, c + nch - 1 - cig); }
};

// What a unit of nch chunks costs, in chunks: a segment has its query rows, the first raise of its
// references and its results besides its chunks (8 heads of a one-token sequence on one CTA
// made it twice as long as the others). Slices are cut by cost: a unit's cost positions are its
// overhead, then its chunks, and a slice takes the chunks whose positions lie in it.
__device__ __forceinline__ int walk_cost(const WalkParams& p, int nch) { return nch > 0 ? nch + p.overhead : 0; }

// Cost of the units of sequences [0, b_stop) (whole warp); below 2^31.
__device__ __forceinline__ int walk_prefix(const WalkParams& p, int b_stop) {
  if (!p.lens) return b_stop * p.units_per_b * walk_cost(p, p.chunks);
  const int lane = threadIdx.x & 31;
  int sum = 0;
  for (int b = lane; b < b_stop; b += 32) sum += walk_cost(p, walk_chunks(p, b));
  return __reduce_add_sync(0xffffffffu, sum) * p.units_per_b;
}

// Equal slices of `total` cost positions: the first `total % slices` have one more.
struct Slices {
  int count, size, longer;
  __device__ __forceinline__ Slices(const WalkParams& p, int total) {
    count = min(p.n_ctas, total);
    size = count ? total / count : 0;
    longer = total - size * count;
  }
  __device__ __forceinline__ int begin(int i) const { return i * size + min(i, longer); }
  __device__ __forceinline__ int of(int x) const {  // the slice that holds position x
    const int y = x - longer * (size + 1);
    return y < 0 ? x / (size + 1) : longer + y / size;
  }
};

// The first chunk at or behind cost position f (below the total), and the chunks in front of it.
__device__ __forceinline__ int walk_locate(const WalkParams& p, int f, WalkPos& pos) {
  int rem = f, b = 0, before = 0;
  if (!p.lens) {
    const int per = p.units_per_b * walk_cost(p, p.chunks);
    b = rem / per;
    rem -= b * per;
    before = b * p.units_per_b * p.chunks;
    pos.nch = p.chunks;
  } else {
    const int lane = threadIdx.x & 31;
    for (int b0 = 0;; b0 += 32) {  // f is below the total: the search ends within the B sequences
      const int mine = b0 + lane < p.B ? walk_chunks(p, b0 + lane) : 0;
      int inc = walk_cost(p, mine);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, inc * p.units_per_b > rem);
      const int l = hit ? __ffs(hit) - 1 : 31;
      const bool here = hit != 0 || b0 + 32 >= p.B;
      // the sequences in front of the one that holds f (or all 32)
      const bool front = here ? lane < l : true;
      before += __reduce_add_sync(0xffffffffu, front ? mine : 0) * p.units_per_b;
      rem -= __reduce_add_sync(0xffffffffu, front ? walk_cost(p, mine) : 0) * p.units_per_b;
      if (here) {
        pos.nch = __shfl_sync(0xffffffffu, mine, l);
        b = b0 + l;
        break;
      }
    }
  }
  const int cost = walk_cost(p, pos.nch);
  const int unit = rem / cost;
  pos.unit = b * p.units_per_b + unit;
  pos.b_end = (b + 1) * p.units_per_b;
  pos.cig = max(rem - unit * cost - p.overhead, 0);
  pos.seg = 0;
  return before + unit * pos.nch + pos.cig;
}

// The slice of CTA `cta`: its first position, and the number of its chunks (whole warp).
__device__ __forceinline__ int walk_start(const WalkParams& p, int cta, WalkPos& pos) {
  const int total = p.lens ? walk_prefix(p, p.B) : p.total;
  const Slices sl(p, total);
  pos = WalkPos{0, 0, 0, 0, 0};
  if (cta >= sl.count) return 0;
  // both ends of the slice, one code for the two
  int first = 0, n = 0;
#pragma unroll 1
  for (int end = 1; end >= 0; --end) {
    const int f = sl.begin(cta + end);
    if (f < total) {
      first = walk_locate(p, f, pos);
    } else {  // behind the last chunk: all of them
      first = p.lens ? 0 : p.B * p.units_per_b * p.chunks;
      if (p.lens) {
        int sum = 0;
        for (int b = threadIdx.x & 31; b < p.B; b += 32) sum += walk_chunks(p, b);
        first = __reduce_add_sync(0xffffffffu, sum) * p.units_per_b;
      }
    }
    n = end ? first : n - first;
  }
  return n;
}

// ----------------------------------------------------------------------------
// fp16 pairs as sums of three E5M2 numbers: t[0] + t[1] / 16 + t[2] / 256, each in the top byte of
// its half: every fp16 number up to 2^15 in magnitude, subnormal ones included, exactly.
// The first two are rounded to the nearest (a tie away from zero), which leaves a remainder of either sign
// and at most half a step: 11 bits less 4, less 4, and the third term holds the rest. (Truncated
// terms take off 3 bits each: 9 bits, and a last term that has to be rounded.) A remainder is at
// most 1/16 of the largest of its term and is scaled up by 16: unscaled, the terms ended at E5M2's
// smallest number, 2^-16, where fp16 goes to 2^-24. The terms' products are scaled back in fp32 sums.
// ----------------------------------------------------------------------------
constexpr float kTermDown = 1.f / 16.f;
__device__ __forceinline__ uint32_t nearest_e5m2(uint32_t w) { return w + 0x00800080u; }  // in the top bytes
__device__ __forceinline__ void split_e5m2(uint32_t w, uint32_t (&t)[3]) {
  auto rest = [](uint32_t x, uint32_t term) {  // 16 (x - term), exactly
    const uint32_t top = term & 0xFF00FF00u;
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&top)),
                              __float2half2_rn(16.f));
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  t[0] = nearest_e5m2(w);
  const uint32_t r = rest(w, t[0]);
  t[1] = nearest_e5m2(r);
  t[2] = rest(r, t[1]);
}
// The sum of three terms (of two rows).
__device__ __forceinline__ uint64_t add_terms(uint64_t t0, uint64_t t1, uint64_t t2) {
  const uint64_t down = f2_pack(kTermDown, kTermDown);
  return f2_fma(f2_fma(t2, down, t1), down, t0);
}
// The top bytes of two pairs, in order.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ----------------------------------------------------------------------------
// Query rows of a segment into shared memory as the MMA's B operand (K-major, 128-byte
// swizzle, R rows of 128 bytes per tile): bf16 as two tiles of 64 columns; for an 8-bit
// cache as three E5M2 tiles, each row scaled by a power of two so that its largest
// element is in [2^14, 2^15) (scale_out[r] undoes it): elements within 2^31 of it are exact, the
// others within 2^-39 of it.
// One warp takes the rows first, first + step, ... below `rows`; row r lies at q + r * pitch. A
// loop, and not inlined: a launch begins with cold instruction caches, and unrolled over 16 rows
// this code alone held the first scores back by 10 us beside a full-rate cache read. Four
// rows' loads are in flight, and two rows are worked on at a time.
// ----------------------------------------------------------------------------
template <bool FP8, int R>
__device__ __noinline__ void load_query_rows(uint8_t* dst, float* scale_out, const __nv_bfloat16* q, int pitch,
                                             int first, int step, int rows) {
  const int lane = threadIdx.x & 31;
  auto load = [&](int r) {
    return r < rows ? *reinterpret_cast<const uint2*>(q + (size_t)r * pitch + lane * 4) : make_uint2(0u, 0u);
  };
  uint2 next[4] = {load(first), load(first + step), load(first + 2 * step), load(first + 3 * step)};
#pragma unroll 1
  for (int rr = first; rr < rows; rr += 2 * step) {
    const uint2 now[2] = {next[0], next[1]};
    next[0] = next[2], next[1] = next[3];
    next[2] = load(rr + 4 * step), next[3] = load(rr + 5 * step);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rr + i * step;
      if (r >= rows) break;
      const uint2 raw = now[i];
      if constexpr (!FP8) {
        *reinterpret_cast<uint2*>(dst + (lane >> 4) * (R * 128) + sw128_offset(r, (lane & 15) >> 1) + (lane & 1) * 8) =
            raw;
      } else {
        const float2 a = bf162_bits_to_float2(raw.x), b = bf162_bits_to_float2(raw.y);
        const float x[4] = {a.x, a.y, b.x, b.y};
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t u = __float_as_uint(x[e]) & 0x7FFFFFFFu;
          if (u < 0x7F800000u) m = max(m, u);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        const int E = m ? max((int)(m >> 23) - 127, -100) : 0;  // floor(log2) of the largest element
        const float up = __uint_as_float((uint32_t)(14 - E + 127) << 23);
        if (lane == 0) scale_out[r] = __uint_as_float((uint32_t)(E - 14 + 127) << 23);
        uint32_t lo[3], hi[3];
        split_e5m2(half2_bits(x[0] * up, x[1] * up), lo);
        split_e5m2(half2_bits(x[2] * up, x[3] * up), hi);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          *reinterpret_cast<uint32_t*>(dst + t * (R * 128) + sw128_offset(r, lane >> 2) + (lane & 3) * 4) =
              top_bytes(lo[t], hi[t]);
      }
    }
  }
  fence_async_smem();
}

// ----------------------------------------------------------------------------
// TMEM and MMA helpers
// ----------------------------------------------------------------------------
__device__ __forceinline__ void tm_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tm_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])
               :
               : "memory");
}

// Shared-memory matrix descriptor without swizzle, MN-major: core matrices of 8 K rows x 16
// bytes (128 bytes each); `lbo_bytes` from one group of 8 K rows to the next, `sbo_bytes` from
// one 16-byte block of MN to the next.
__device__ __forceinline__ uint64_t sdesc_plain_mn(uint32_t smem_addr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo_bytes >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, A in E4M3 (format 0), B in E5M2 (format 1).
__host__ __device__ constexpr uint32_t idesc_e4m3_e5m2(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_e4m3_f32(M, N, a_mn_major, b_mn_major) | (1u << 10);
}

// Threads of a warpgroup meet on hardware barrier `id` and count their predicates.
__device__ __forceinline__ int group_count(int id, bool pred) {
  int n;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.popc.aligned.u32 %0, %1, 128, p;\n\t}"
      : "=r"(n)
      : "r"(id), "r"((int)pred)
      : "memory");
  return n;
}

// A bounded wait whose outcome the whole warp agrees on. The probe in front costs a complete
// phase less than a wait that may suspend (300 cycles, measured).
__device__ __forceinline__ bool warp_wait_all(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  if (__all_sync(0xffffffffu, mbar_test_wait(smem_u32(bar), parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_ns(bar, parity, w, kConsumerPollNs));
}

// The same for two phases at once: both are probed before either is waited for.
__device__ __forceinline__ bool warp_wait_both(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, const WaitCtx& w) {
  const bool r0 = mbar_test_wait(smem_u32(b0), p0), r1 = mbar_test_wait(smem_u32(b1), p1);
  if (__all_sync(0xffffffffu, r0 && r1)) return true;
  const bool ok = mbar_wait_ns(b0, p0, w, kConsumerPollNs) && mbar_wait_ns(b1, p1, w, kConsumerPollNs);
  return __all_sync(0xffffffffu, ok);
}

struct MaxOp {
  static __device__ __forceinline__ float f(float a, float b) { return fmaxf(a, b); }
};
struct SumOp {
  static __device__ __forceinline__ float f(float a, float b) { return a + b; }
};
// 16 values reduced over a warp by halving the set at each step (16 shuffles, not 80): lanes
// 2r and 2r + 1 end with value r.
template <typename Op>
__device__ __forceinline__ float warp_reduce16(const float (&v)[16]) {
  const int lane = threadIdx.x & 31;
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = lane & 16;
    const float keep = up ? v[i + 8] : v[i], give = up ? v[i] : v[i + 8];
    a[i] = Op::f(keep, __shfl_xor_sync(0xffffffffu, give, 16));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 8;
    const float keep = up ? a[i + 4] : a[i], give = up ? a[i] : a[i + 4];
    b[i] = Op::f(keep, __shfl_xor_sync(0xffffffffu, give, 8));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 4;
    const float keep = up ? b[i + 2] : b[i], give = up ? b[i] : b[i + 2];
    c[i] = Op::f(keep, __shfl_xor_sync(0xffffffffu, give, 4));
  }
  const bool up = lane & 2;
  const float keep = up ? c[1] : c[0], give = up ? c[0] : c[1];
  const float d = Op::f(keep, __shfl_xor_sync(0xffffffffu, give, 2));
  return Op::f(d, __shfl_xor_sync(0xffffffffu, d, 1));
}

__device__ __forceinline__ uint8_t* align_1k(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

}  // namespace fa
