// fa_cache.h -- parameter blocks, launchers and small device helpers of the cache
// operators (8-bit cache, sparse attention over selected blocks, eviction).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace fa {

constexpr int kCacheD = 128;      // head dim of every cache operator
constexpr int kUnitRows = 16;     // query rows that an attention CTA takes at a time
constexpr int kCacheTile = 128;   // tokens per tile of the elementwise kernels; every block size divides it
// Smallest scale the store writes: a block of zeros still has a positive one.
constexpr int kMinScaleExp = -100;

struct StoreParams {
  const void *k, *v;       // bf16 [B, Hkv, n_new, d]
  void *ck, *cv;           // E4M3 [B, Hkv, Nk, d]
  float *ks, *vs;          // [B, Hkv, n_blocks]
  const int* lens;         // [B] or null
  int B, Hkv, n_new, Nk, block;
};

struct BoundsParams {
  const void* k;           // [B, Hkv, Nk, d], E4M3 or bf16
  void* bounds;            // [B, Hkv, n_blocks, 2, d], the same type
  const int* lens;
  int fp8;
  int B, Hkv, Nk, block, n_new;  // n_new = 0: every block
};

struct SelectParams {
  const void* q;           // bf16 [B, Hq, Nq, d]
  const void* bounds;
  const float* ks;         // [B, Hkv, n_blocks] or null
  int* idx;                // [B, Hkv, Nq, n_select]
  unsigned long long* keys;  // workspace: ordered scores [B * Hkv * Nq, n_blocks]
  const int* lens;
  int fp8, causal;
  int B, Hq, Hkv, Nq, Nk, block, n_select, n_first, n_last;
};

// The walk over the key chunks of all units (see fa_cache_sm100.cuh).
struct WalkParams {
  const int* lens;        // non-null: a unit's chunks go by its sequence's length
  int B, Nk;
  int units_per_b;        // units of one sequence
  int chunks;             // chunks of a unit where lens is null
  int overhead;           // what a unit costs besides its chunks, in chunks
  int total;              // all chunks and overheads where lens is null
  int n_ctas;
  int chunk_log2;         // log2 of the keys per chunk
};

struct AttendParams {
  const void* q;           // bf16 [B, Hq, Nq, d]
  const void *k, *v;       // [B, Hkv, Nk, d], E4M3 or bf16
  const float *ks, *vs;    // [B, Hkv, n_blocks], null for bf16
  const int* idx;          // [B, Hkv, Nq, n_select] or null (every block)
  const int* lens;
  void* o;                 // bf16 [B, Hq, Nq, d]
  float* lse;              // [B, Hq, Nq]
  int* status;
  int fp8, causal;
  int B, Hq, Hkv, Nq, Nk, block, n_select;
  int block_log2;
  float scale_log2;        // scale * log2(e)
  WalkParams walk;
  int n_rb;                // units that a group's rows are cut into
  int units;
  float* o_part;           // workspace: partial O [(units + n_ctas) * 2, kUnitRows, d]
  float* lse_part;         // workspace: partial LSE, log2 [(units + n_ctas) * 2, kUnitRows]
  uint64_t wait_budget_ns;
};

struct WeightsParams {
  const void* q;
  const void* k;
  const float* ks;
  const float* lse;        // [B, Hq, Nq]
  float* acc;              // [B, Hkv, Nk]
  const int* lens;
  int* status;
  int fp8, causal;
  int B, Hq, Hkv, Nq, Nk, block, block_log2;
  float scale_log2;
  WalkParams walk;         // groups of at most 32 rows: chunks of 256 keys
  uint64_t wait_budget_ns;
};

struct EvictParams {
  const void *k, *v;
  const float *ks, *vs, *acc;
  const int* lens;
  void *ok, *ov;           // [B, Hkv, out_Nk, d]
  float *oks, *ovs, *oacc;
  int *idx, *olens;        // [B, Hkv, keep], [B]
  int fp8;
  int B, Hkv, Nk, block, keep, recent, out_Nk;
};

cudaError_t launch_cache_store(const StoreParams& p, cudaStream_t s);
cudaError_t launch_block_bounds(const BoundsParams& p, cudaStream_t s);
cudaError_t launch_select_blocks(const SelectParams& p, cudaStream_t s);
cudaError_t launch_cache_attend(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p, cudaStream_t s);
// Groups of at most kWeightsStreamRows query rows: tk is the cache in boxes of kWeightsChunk keys, tq is not
// read; larger groups: tq is all query rows in boxes of kWeightsRowTile, tk the (bf16) cache in boxes of 128.
constexpr int kWeightsChunk = 256;
constexpr int kWeightsRowTile = 128;
constexpr int kWeightsStreamRows = 32;
cudaError_t launch_cache_weights(const CUtensorMap& tk, const CUtensorMap& tq, const WeightsParams& p, cudaStream_t s);
cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t s);

#ifdef __CUDACC__
// Tokens that sequence b holds: lens[b] clamped to the cache, or the whole cache.
__device__ __forceinline__ int cache_len(const int* lens, int b, int Nk) {
  return lens ? min(max(lens[b], 0), Nk) : Nk;
}

// Two E4M3 codes (low byte first) to two halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Two halves to E4M3 (round to nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint16_t half2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
// Two floats to E4M3 (round to nearest even, saturating; NaN stays NaN), `lo` in the low byte.
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 half2_bits_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 bf162_bits_to_float2(uint32_t h) {
  return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
}

// Eight elements of a row as floats: 8 bytes of E4M3 codes, or 16 bytes of bf16.
template <bool FP8>
struct Row8;
template <>
struct Row8<true> {
  using Raw = uint2;
  static __device__ __forceinline__ void floats(const Raw& r, float (&x)[8]) {
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_bits_to_float2(e4m3x2_to_half2((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Row8<false> {
  using Raw = uint4;
  static __device__ __forceinline__ void floats(const Raw& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf162_bits_to_float2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
#endif

}  // namespace fa
