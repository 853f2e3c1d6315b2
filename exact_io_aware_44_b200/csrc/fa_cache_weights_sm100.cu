// fa_cache_weights_sm100.cu -- the attention weights that a step gives the keys of a cache,
// added to an accumulator: acc_j += sum_r exp(x_rj - lse_r) over a group's query rows that see
// key j, x_rj = scale * s_j * q_r . k_j, lse_r from the step's own attention call.
//
// With the keys as the MMA's M, a key is a TMEM lane and a thread, so the sum over query rows
// (TMEM columns) stays in one thread: no reduction, no atomics, and every key belongs to one CTA.
//
// Few rows (a decode step; at most 32): bound by reading K. stream_kernel walks equal
// slices of the keys of all (sequence, kv head) pairs, 256 keys a stage; 8-bit keys feed the
// tensor cores as they are, against queries in three E5M2 terms (fa_cache_sm100.cuh). Two
// groups of four warps take a half of every stage each; a thread reads its key's scale and
// accumulator two stages ahead.
//
// Many rows (a prompt): bound by the exponentials (2^x: 16 a clock and SM). tile_kernel keeps 128
// keys in shared memory as bf16 (8-bit codes are exact in bf16; their scale is applied to
// the scores) and streams tiles of 128 query rows past them.
//
// A weight is 2^(x log2 e - lse log2 e): lse log2 e is rounded to fp32 (half a step of a number of size
// 16 is 2^-20), the exponential is good to 2^-22, and rows are summed in fp32. A prompt of 4096 is 2.5e-7 off
// its values in 64 bits (relative, over all keys); plain fp32 operations are 0.7e-7 off.
#include <math.h>

#include <type_traits>

#include "fa.h"
#include "fa_cache_sm100.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

// ---------------------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------------------
template <bool FP8, int R>
struct StreamCfg {
  static constexpr int kElem = FP8 ? 1 : 2;
  static constexpr int kTerms = FP8 ? 3 : 1;
  static constexpr int kN = kTerms * R;
  static constexpr int kThreads = 384;
  static constexpr int kRegion = kWeightsChunk * 128;  // 128-byte column block of a stage
  static constexpr int kStage = kElem * kRegion;
  static constexpr int kStages = FP8 ? 5 : 3;
  static constexpr int kQTile = R * 128;
  static constexpr int kQ = (FP8 ? 3 : 2) * kQTile;
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kOffK + kStages * kStage;
  static constexpr int kOffRow = kOffQ + 2 * kQ;       // [kQScaleRing][2][R]: query scale, -lse * log2 e
  static constexpr int kOffBar = kOffRow + kQScaleRing * 2 * R * 4;
  // k_full[S], k_empty[S], q_full[2], q_empty[2], s_full[4], s_free[4], mma_done[2], row_full[ring]
  static constexpr int kNumBars = 2 * kStages + 14 + kQScaleRing;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  // S buffers: [group][stage parity]
  static constexpr int kTmemCols = 4 * kN <= 64 ? 64 : 4 * kN <= 128 ? 128 : 4 * kN <= 256 ? 256 : 512;
};

// What the rows add to a key that is not finite: in the products, a row that adds nothing (lse = -inf, or
// one that fills the tile up) is a row of zeros, and 0 * NaN or 0 * inf is NaN. Such keys are rare, and a
// mask of these rows cost every key (112 us and more where the kernel takes 106), so their rows are taken one by one here.
template <bool FP8>
__device__ __noinline__ float sum_of_rows(const WeightsParams& p, int unit, int key, int rows, uint32_t hidden) {
  using Raw = typename Row8<FP8>::Raw;
  const Raw* k = reinterpret_cast<const Raw*>(static_cast<const char*>(p.k) +
                                              ((size_t)unit * p.Nk + key) * kCacheD * (FP8 ? 1 : 2));
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (size_t)unit * rows * kCacheD;
  float a = p.scale_log2;
  if (FP8) a *= p.ks[(size_t)unit * ((p.Nk + p.block - 1) >> p.block_log2) + (key >> p.block_log2)];
  float sum = 0.f;
  for (int j = 0; j < rows; ++j) {
    const float lse = p.lse[(size_t)unit * rows + j];
    if (((hidden >> j) & 1u) || lse == -INFINITY) continue;
    float s = 0.f;
    for (int c = 0; c < kCacheD / 8; ++c) {
      float x[8], y[8];
      Row8<FP8>::floats(k[c], x);
      Row8<false>::floats(*reinterpret_cast<const uint4*>(q + (size_t)j * kCacheD + c * 8), y);
      for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
    }
    sum += ex2(fmaf(s, a, -lse * 1.4426950408889634f));
  }
  return sum;
}

template <bool FP8, int R>
__global__ void __launch_bounds__(StreamCfg<FP8, R>::kThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tmK, const WeightsParams p) {
  using C = StreamCfg<FP8, R>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1k(smem_raw);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_empty = k_full + S;
  uint64_t* q_full = k_empty + S;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_full + 4;
  uint64_t* s_free = q_full + 8;
  uint64_t* mma_done = q_full + 12;
  uint64_t* row_full = q_full + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  float* row_info = reinterpret_cast<float*>(smem + C::kOffRow);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&q_empty[b], 2);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4);
    }
    for (int b = 0; b < kQScaleRing; ++b) mbar_init(&row_full[b], 1);
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  grid_wait();
  WalkPos pos0;
  const int n = walk_start(p.walk, blockIdx.x, pos0);
  for (int e = threadIdx.x; e < 2 * C::kQ / 16; e += C::kThreads)  // rows that do not exist: zeros
    *reinterpret_cast<uint4*>(smem + C::kOffQ + e * 16) = make_uint4(0u, 0u, 0u, 0u);
  for (int e = threadIdx.x; e < kQScaleRing * 2 * R; e += C::kThreads) row_info[e] = 1.f;
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};
  const int g_rows = p.Hq / p.Hkv * p.Nq;  // at most R
  if (warp > 0) {  // the first unit's query rows
    if (n > 0)
      load_query_rows<FP8, R>(smem + C::kOffQ, row_info,
                              static_cast<const __nv_bfloat16*>(p.q) + (size_t)pos0.unit * g_rows * kCacheD, kCacheD,
                              warp - 1, C::kThreads / 32 - 1, g_rows);
    named_barrier(15, C::kThreads - 32);
  }

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      WalkPos ps = pos0;
      int st = 0, issued = 0;
      uint32_t phase = 1;
      bool ok = true;
      for (int c = 0; c < n; ++c) {
        if (!(ok = mbar_wait_spin(&k_empty[st], phase, w))) break;
        mbar_arrive_expect_tx(&k_full[st], C::kStage);
#pragma unroll
        for (int z = 0; z < C::kElem; ++z)
          tma_load_3d(smem + C::kOffK + st * C::kStage + z * C::kRegion, &tmK, &k_full[st], z * (128 / C::kElem),
                      ps.cig * kWeightsChunk, ps.unit);
        ++issued;
        if (++st == S) st = 0, phase ^= 1u;
        ps.next(p.walk);
      }
      if (!ok) {  // error path: let the loads already issued land before the CTA exits
        WaitCtx drain{abort_flag, p.status, 20000000ull};
        volatile int zero = 0;
        drain.abort_flag = &zero;
        for (int c = max(0, issued - S); c < issued; ++c) mbar_wait(&k_full[c % S], (c / S) & 1, drain);
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ S issuers
    // One thread for each half of a stage: a thread issues a half's four MMAs and its commits in
    // about 500 cycles, and a stage arrives every 1370 at full bandwidth.
    constexpr uint32_t kId = FP8 ? idesc_e4m3_e5m2(128, C::kN, false, false) : idesc_bf16_f32(128, C::kN, false, false);
    if (lane == 0) {
      const int g = warp >> 1;
      const uint64_t d_k = sdesc_sw128(smem_u32(smem + C::kOffK + g * 128 * 128), 16, 1024);
      const uint64_t d_q = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
      WalkPos ps = pos0;
      int st = 0;
      uint32_t phase = 0;
      for (int c = 0; c < n; ++c) {
        const int qb = ps.seg & 1, sb = g * 2 + (c & 1);
        if ((c == 0 || ps.cig == 0) && !mbar_wait_spin(&q_full[qb], (ps.seg >> 1) & 1, w)) break;
        if (!mbar_wait_spin(&s_free[sb], ((c >> 1) & 1) ^ 1, w)) break;
        if (!mbar_wait_spin(&k_full[st], phase, w)) break;
        tc_fence_after();
        const uint64_t a0 = desc_advance(d_k, st * C::kStage);
        const uint64_t b0 = desc_advance(d_q, qb * C::kQ);
        const uint32_t d = tmem + sb * C::kN;
        if constexpr (FP8) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3_ss(d, desc_advance(a0, k * 32), desc_advance(b0, k * 32), kId, k > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss(d, desc_advance(a0, (k >> 2) * C::kRegion + (k & 3) * 32),
                        desc_advance(b0, (k >> 2) * C::kQTile + (k & 3) * 32), kId, k > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[sb]);
        mma_commit(&k_empty[st]);
        if (c == n - 1 || ps.cig == ps.nch - 1) mma_commit(&q_empty[qb]);
        if (++st == S) st = 0, phase ^= 1u;
        ps.next(p.walk);
      }
      mma_commit(&mma_done[g]);
      WaitCtx drain{abort_flag, p.status, 20000000ull};
      volatile int zero = 0;
      drain.abort_flag = &zero;
      mbar_wait(&mma_done[g], 0, drain);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ query rows
    WalkPos ps = pos0;
    for (int c = 0; c < n;) {
      const int qb = ps.seg & 1, ring = ps.seg % kQScaleRing;
      if (!warp_wait_all(&q_empty[qb], ((ps.seg >> 1) & 1) ^ 1, w)) break;
      const long long row0 = (long long)ps.unit * g_rows;
      float* info = row_info + ring * 2 * R;
      const float l = lane < g_rows ? p.lse[row0 + lane] : -INFINITY;
      // a row that adds nothing: 2^(x - inf) = 0
      if (lane < R) info[R + lane] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
      if (ps.seg > 0)
        load_query_rows<FP8, R>(smem + C::kOffQ + qb * C::kQ, info,
                                static_cast<const __nv_bfloat16*>(p.q) + row0 * kCacheD, kCacheD, 0, 1, g_rows);
      // and zeros in its place: it may hold NaN (masking it key by key took 119 us where this takes 103);
      // where the key does too: sum_of_rows
      uint32_t dead = __ballot_sync(0xffffffffu, lane < g_rows && l == -INFINITY);
      if (dead) {
        __syncwarp();
        for (; dead; dead &= dead - 1) {
          uint8_t* row = smem + C::kOffQ + qb * C::kQ + (__ffs(dead) - 1) * 128 + lane * 4;
          for (int z = 0; z < (FP8 ? 3 : 2); ++z) *reinterpret_cast<uint32_t*>(row + z * C::kQTile) = 0u;
        }
        fence_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&q_full[qb]);
        mbar_arrive(&row_full[ring]);
      }
      const int last = ps.last(c, n);
      ps.cig += last - c;
      ps.next(p.walk);
      c = last + 1;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ weights: thread = key
    const int g = (warp - 4) >> 2;  // half of the stage
    const int quarter = warp & 3;
    const int t = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int n_blocks = (p.Nk + p.block - 1) >> p.block_log2;
    uint64_t b_row[R / 2], nl[R / 2];
    WalkPos pos = pos0, nxt = pos0;
    int len = 0, lim0 = 0;
    // Scale and accumulator of this thread's key, read two stages ahead (one stage is shorter than
    // a loaded memory's latency), into two register sets in turn (a move would wait for the load).
    float ks0 = 1.f, acc0 = 0.f, ks1 = 1.f, acc1 = 0.f;
    int c_ahead = 0;
    auto ahead = [&](float& ks, float& acc) {
      if (c_ahead >= n) return;
      const int key = nxt.cig * kWeightsChunk + g * 128 + t;
      if (key < (p.lens ? cache_len(p.lens, nxt.unit / p.Hkv, p.Nk) : p.Nk)) {
        acc = p.acc[(size_t)nxt.unit * p.Nk + key];
        if (FP8) ks = __ldg(p.ks + (size_t)nxt.unit * n_blocks + (key >> p.block_log2));
      }
      ++c_ahead;
      nxt.next(p.walk);
    };
    ahead(ks0, acc0);
    ahead(ks1, acc1);
    auto stage = [&](int c, float& ks, float& acc) -> bool {  // false at the end, or if a wait ran out
      if (c >= n) return false;
      const int sb = g * 2 + (c & 1);
      if (c == 0 || pos.cig == 0) {
        len = p.lens ? cache_len(p.lens, pos.unit / p.Hkv, p.Nk) : p.Nk;
        lim0 = p.causal ? len - p.Nq : len - 1;
        const int ring = pos.seg % kQScaleRing;
        if (!warp_wait_all(&row_full[ring], (pos.seg / kQScaleRing) & 1, w)) return false;
        const float2* info = reinterpret_cast<const float2*>(row_info + ring * 2 * R);
#pragma unroll
        for (int j = 0; j < R / 2; ++j) {
          if (FP8) b_row[j] = f2_pack(info[j].x, info[j].y);
          nl[j] = f2_pack(info[R / 2 + j].x, info[R / 2 + j].y);
        }
      }
      if (!warp_wait_all(&s_full[sb], (c >> 1) & 1, w)) return false;
      tc_fence_after();
      const float a = FP8 ? ks * p.scale_log2 : p.scale_log2;
      const float before = acc;
      const int key = pos.cig * kWeightsChunk + g * 128 + t;
      const uint64_t aa = f2_pack(a, a);
      uint32_t hidden = 0u;  // rows whose query is in front of this key
      if (key > lim0) {      // the causal edge
        for (int j = 0; j < g_rows; ++j)
          if (key > lim0 + j % p.Nq) hidden |= 1u << j;
      }
      uint64_t sum = f2_pack(0.f, 0.f);
#pragma unroll
      for (int h = 0; h < R / 16; ++h) {
        uint32_t r[C::kTerms][16];
#pragma unroll
        for (int z = 0; z < C::kTerms; ++z) tm_ld16(tmem + lane_off + sb * C::kN + z * R + h * 16, r[z]);
#pragma unroll
        for (int z = 0; z < C::kTerms; ++z) tm_ld16_wait(r[z]);
        if (h == R / 16 - 1) {  // the scores have been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[sb]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          auto two = [&](int z) { return f2_pack(__uint_as_float(r[z][2 * j]), __uint_as_float(r[z][2 * j + 1])); };
          uint64_t s;
          if constexpr (FP8)
            s = f2_mul(add_terms(two(0), two(1), two(2)), b_row[h * 8 + j]);
          else
            s = two(0);
          float e0, e1;
          f2_unpack(f2_fma(s, aa, nl[h * 8 + j]), e0, e1);
          if (hidden) {
            if ((hidden >> (h * 16 + 2 * j)) & 1u) e0 = -INFINITY;
            if ((hidden >> (h * 16 + 2 * j + 1)) & 1u) e1 = -INFINITY;
          }
          sum = f2_add(sum, f2_pack(ex2(e0), ex2(e1)));
        }
      }
      if (key < len) {
        float s0, s1;
        f2_unpack(sum, s0, s1);
        s0 += s1;
        if (s0 != s0) s0 = sum_of_rows<FP8>(p, pos.unit, key, g_rows, hidden);
        p.acc[(size_t)pos.unit * p.Nk + key] = before + s0;
      }
      ahead(ks, acc);
      pos.next(p.walk);
      return true;
    };
    for (int c = 0; stage(c, ks0, acc0) && stage(c + 1, ks1, acc1); c += 2) {
    }
  }

  tc_fence_before();
  __syncthreads();
  grid_release();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------------------
struct TileCfg {
  static constexpr int kGroups = 4;                     // softmax warpgroups, one for each buffer: tile n is group n % 4's
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kRows = kWeightsRowTile;         // query rows per tile: the MMA's N
  static constexpr int kKRegion = 128 * 128;            // 64-column block of the keys
  static constexpr int kQRegion = kRows * 128;          // 64-column block of a tile of query rows
  static constexpr int kTile = 2 * kQRegion;
  static constexpr int kBufs = 4;                       // query stages, S buffers and row infos
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = 2 * kKRegion;
  static constexpr int kOffRow = kOffQ + kBufs * kTile; // [kBufs][128] {-lse * log2 e}, [kBufs][128] last key seen
  static constexpr int kOffMask = kOffRow + kBufs * 2 * kRows * 4;  // [kBufs]: does any key need a mask
  static constexpr int kOffSum = kOffMask + 16;         // [kGroups][128] floats
  static constexpr int kOffBar = kOffSum + kGroups * 512;
  // k_full, q_full[4], q_empty[4], row_full[4], s_full[4], s_free[4], mma_done[2]
  static constexpr int kNumBars = 23;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// Walks the tiles of a group's query rows (flattened over its heads, Nq each) that some key from
// key0 on is seen by, in order: a causal query at position base + i sees the keys up to it.
struct RowTiles {
  int rows, Nq, base, key0, causal;
  int tile, i0, step;  // i0: place of the tile's first row within its head

  __device__ __forceinline__ RowTiles(int rows_, int Nq_, int base_, int key0_, int causal_)
      : rows(rows_), Nq(Nq_), base(base_), key0(key0_), causal(causal_), tile(0), i0(0), step(TileCfg::kRows % Nq_) {
    settle();
  }
  __device__ __forceinline__ bool more() const { return tile * TileCfg::kRows < rows; }
  __device__ __forceinline__ void next() {
    advance();
    settle();
  }

 private:
  __device__ __forceinline__ void advance() {
    ++tile;
    i0 += step;
    if (i0 >= Nq) i0 -= Nq;
  }
  __device__ __forceinline__ void settle() {
    if (!causal) return;
    // a tile that reaches its head's last query sees what any query sees
    while (more() && base + min(i0 + min(TileCfg::kRows, rows - tile * TileCfg::kRows), Nq) - 1 < key0) advance();
  }
};

template <bool FP8>
__global__ void __launch_bounds__(TileCfg::kThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                const WeightsParams p) {
  using C = TileCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1k(smem_raw);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = k_full + 1;
  uint64_t* q_empty = k_full + 5;
  uint64_t* row_full = k_full + 9;
  uint64_t* s_full = k_full + 13;
  uint64_t* s_free = k_full + 17;
  uint64_t* mma_done = k_full + 21;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // key tiles from the first on: a causal cache's first keys are seen by the most rows, and the
  // longest work starts first
  const int groups = p.B * p.Hkv;
  const int bh = blockIdx.x % groups, key0 = (blockIdx.x / groups) * kChunk;

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&q_empty[b], 1);
      mbar_init(&row_full[b], 1);
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4);
    }
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  grid_wait();
  const int len = cache_len(p.lens, bh / p.Hkv, p.Nk);
  const int rows = p.Hq / p.Hkv * p.Nq;
  const long long row0 = (long long)bh * rows;
  RowTiles tiles(rows, p.Nq, len - p.Nq, key0, p.causal);
  const bool any = key0 < len && tiles.more();  // else no row sees these keys
  if constexpr (FP8) {
    // the keys' codes as bf16, exactly, in the layout that TMA gives a bf16 tile
    const uint8_t* k = static_cast<const uint8_t*>(p.k) + ((size_t)bh * p.Nk + key0) * kCacheD;
    if (any) {
      for (int e = threadIdx.x; e < kChunk * (kCacheD / 8); e += C::kThreads) {
        const int r = e >> 4, c8 = e & 15;  // 8 codes make a 16-byte chunk
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (key0 + r < len) {
          float f[8];
          Row8<true>::floats(*reinterpret_cast<const uint2*>(k + (size_t)r * kCacheD + c8 * 8), f);
          o = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                         pack_bf16x2(f[6], f[7]));
        }
        *reinterpret_cast<uint4*>(smem + C::kOffK + (c8 >> 3) * C::kKRegion + sw128_offset(r, c8 & 7)) = o;
      }
      fence_async_smem();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && any) {
      if (!FP8) {
        mbar_arrive_expect_tx(k_full, 2 * C::kKRegion);
        for (int z = 0; z < 2; ++z) tma_load_3d(smem + C::kOffK + z * C::kKRegion, &tmK, k_full, z * 64, key0, bh);
      }
      int n = 0;
      bool ok = true;
      for (; tiles.more(); tiles.next(), ++n) {
        const int b = n & 3;
        if (!(ok = mbar_wait_spin(&q_empty[b], ((n >> 2) & 1) ^ 1, w))) break;
        mbar_arrive_expect_tx(&q_full[b], C::kTile);
        for (int z = 0; z < 2; ++z)
          tma_load_3d(smem + C::kOffQ + b * C::kTile + z * C::kQRegion, &tmQ, &q_full[b], z * 64,
                      (int)(row0 + tiles.tile * C::kRows), 0);
      }
      if (!ok) {
        WaitCtx drain{abort_flag, p.status, 20000000ull};
        volatile int zero = 0;
        drain.abort_flag = &zero;
        if (!FP8) mbar_wait(k_full, 0, drain);
        for (int c = max(0, n - C::kBufs); c < n; ++c) mbar_wait(&q_full[c & 3], (c >> 2) & 1, drain);
      }
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------------ S issuers
    // Two threads take alternate tiles: issuing eight MMAs takes one about 700 cycles, close to
    // the 1024 in which the SFU takes a tile's exponentials.
    constexpr uint32_t kId = idesc_bf16_f32(128, C::kRows, false, false);
    if (lane == 0 && any) {
      const uint64_t d_k = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t d_q = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
      bool ok = FP8 || mbar_wait_spin(k_full, 0, w);
      for (int n = 0; ok && tiles.more(); tiles.next(), ++n) {
        if ((n & 1) != warp - 1) continue;
        const int b = n & 3;
        if (!(ok = mbar_wait_spin(&q_full[b], (n >> 2) & 1, w))) break;
        if (!(ok = mbar_wait_spin(&s_free[b], ((n >> 2) & 1) ^ 1, w))) break;
        tc_fence_after();
        const uint64_t b0 = desc_advance(d_q, b * C::kTile);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ss(tmem + b * C::kRows, desc_advance(d_k, (k >> 2) * C::kKRegion + (k & 3) * 32),
                      desc_advance(b0, (k >> 2) * C::kQRegion + (k & 3) * 32), kId, k > 0 ? 1u : 0u);
        mma_commit(&s_full[b]);
        mma_commit(&q_empty[b]);
      }
      mma_commit(&mma_done[warp - 1]);
      WaitCtx drain{abort_flag, p.status, 20000000ull};
      volatile int zero = 0;
      drain.abort_flag = &zero;
      mbar_wait(&mma_done[warp - 1], 0, drain);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ the rows' lse and last keys
    // A tile's lse is read two tiles ahead: read when its buffer comes free, or one tile ahead, it
    // held every tile back by its latency. Two register sets in turn: a move would wait for the load.
    float l0[4], l1[4];
    RowTiles ahead = tiles;
    auto read = [&](float(&x)[4]) {
      if (!any || !ahead.more()) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = ahead.tile * C::kRows + e * 32 + lane;
        x[e] = r < rows ? p.lse[row0 + r] : -INFINITY;
      }
      ahead.next();
    };
    auto put = [&](int n, float(&l)[4]) -> bool {  // tile n; false at the end, or if a wait ran out
      if (!any || !tiles.more()) return false;
      // Inside one head, behind all of these keys, and no row that adds nothing: no mask, and no last
      // keys to work out (this warp's instructions were the slowest part of a tile)
      const bool dead = l[0] == -INFINITY || l[1] == -INFINITY || l[2] == -INFINITY || l[3] == -INFINITY;
      const bool plain = !__any_sync(0xffffffffu, dead) && (tiles.tile + 1) * C::kRows <= rows &&
                         (!p.causal || (tiles.i0 + C::kRows <= p.Nq &&
                                        tiles.base + tiles.i0 >= min(key0 + kChunk, len) - 1));
      float minus[4];
      int last[4];  // last key that the row sees
#pragma unroll
      for (int e = 0; e < 4; ++e) minus[e] = l[e] == -INFINITY ? -INFINITY : -l[e] * 1.4426950408889634f;
      if (!plain) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int off = e * 32 + lane;
          last[e] = -1;
          if (tiles.tile * C::kRows + off < rows && l[e] != -INFINITY) {
            int i = tiles.i0 + off;  // the row's query: its place within its head
            while (i >= p.Nq) i -= p.Nq;
            last[e] = p.causal ? len - p.Nq + i : len - 1;
          }
        }
      }
      read(l);
      const int b = n & 3;
      if (!warp_wait_all(&s_free[b], ((n >> 2) & 1) ^ 1, w)) return false;
      float* nl = reinterpret_cast<float*>(smem + C::kOffRow) + b * C::kRows;
      int* lim = reinterpret_cast<int*>(smem + C::kOffRow) + (C::kBufs + b) * C::kRows;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        nl[e * 32 + lane] = minus[e];
        if (!plain) lim[e * 32 + lane] = last[e];
      }
      if (lane == 0) reinterpret_cast<int*>(smem + C::kOffMask)[b] = !plain;
      __syncwarp();
      if (lane == 0) mbar_arrive(&row_full[b]);
      tiles.next();
      return true;
    };
    read(l0);
    read(l1);
    for (int n = 0; put(n, l0) && put(n + 1, l1); n += 2) {
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ weights: thread = key
    const int g = (warp - 4) >> 2;  // its buffer: every fourth tile
    const int quarter = warp & 3;
    const int t_key = quarter * 32 + lane;
    const int key = key0 + t_key;
    const uint32_t tS = tmem + ((uint32_t)(quarter * 32) << 16) + g * C::kRows;
    float a = p.scale_log2;
    if (FP8 && key < len)
      a *= p.ks[(size_t)bh * ((p.Nk + p.block - 1) >> p.block_log2) + (key >> p.block_log2)];
    const uint64_t aa = f2_pack(a, a);
    const float4* nl = reinterpret_cast<const float4*>(smem + C::kOffRow) + g * (C::kRows / 4);
    const int4* lim = reinterpret_cast<const int4*>(smem + C::kOffRow) + (C::kBufs + g) * (C::kRows / 4);
    const volatile int* needs_mask = reinterpret_cast<const volatile int*>(smem + C::kOffMask) + g;
    float total = 0.f;
    for (int n = 0; any && tiles.more(); tiles.next(), ++n) {
      if ((n & 3) != g) continue;
      if (!warp_wait_both(&s_full[g], (n >> 2) & 1, &row_full[g], (n >> 2) & 1, w)) break;
      tc_fence_after();
      uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
      // two loops, not one with a test in it: the test cost as many issue slots as the rest
      auto tile = [&](auto masked) {
        uint32_t r[2][16];  // columns of the next step are on their way while these are used
        tm_ld16(tS, r[0]);
#pragma unroll
        for (int cc = 0; cc < C::kRows / 16; ++cc) {
          uint32_t(&x)[16] = r[cc & 1];
          tm_ld16_wait(x);
          if (cc + 1 < C::kRows / 16) tm_ld16(tS + (cc + 1) * 16, r[(cc + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 l4 = nl[cc * 4 + i];
            float e[4];
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])), aa, f2_pack(l4.x, l4.y)),
                      e[0], e[1]);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])), aa,
                             f2_pack(l4.z, l4.w)),
                      e[2], e[3]);
            if constexpr (decltype(masked)::value) {
              const int4 m = lim[cc * 4 + i];
              if (key > m.x) e[0] = -INFINITY;
              if (key > m.y) e[1] = -INFINITY;
              if (key > m.z) e[2] = -INFINITY;
              if (key > m.w) e[3] = -INFINITY;
            }
            sum0 = f2_add(sum0, f2_pack(ex2(e[0]), ex2(e[1])));
            sum1 = f2_add(sum1, f2_pack(ex2(e[2]), ex2(e[3])));
          }
        }
      };
      if (*needs_mask != 0)
        tile(std::true_type{});
      else
        tile(std::false_type{});
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[g]);
      float x0, x1;
      f2_unpack(f2_add(sum0, sum1), x0, x1);
      total += x0 + x1;
    }
    float* part = reinterpret_cast<float*>(smem + C::kOffSum);
    part[g * 128 + t_key] = total;
    named_barrier(1, 128 * C::kGroups);
    if (g == 0 && key < len) {
      float* acc = p.acc + (size_t)bh * p.Nk + key;
      *acc += (part[t_key] + part[128 + t_key]) + (part[256 + t_key] + part[384 + t_key]);
    }
  }

  tc_fence_before();
  __syncthreads();
  grid_release();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool FP8, int R>
cudaError_t launch_stream(const CUtensorMap& tk, const WeightsParams& p, cudaStream_t s) {
  using C = StreamCfg<FP8, R>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = ensure_smem_limit(stream_kernel<FP8, R>, C::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(stream_kernel<FP8, R>, (unsigned)p.walk.n_ctas, C::kThreads, C::kSmemBytes, s, tk, p);
}

template <bool FP8>
cudaError_t launch_tile(const CUtensorMap& tk, const CUtensorMap& tq, const WeightsParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = ensure_smem_limit(tile_kernel<FP8>, TileCfg::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((long long)p.B * p.Hkv * ((p.Nk + kChunk - 1) / kChunk));
  return launch_dependent(tile_kernel<FP8>, grid, TileCfg::kThreads, TileCfg::kSmemBytes, s, tk, tq, p);
}

}  // namespace

cudaError_t launch_cache_weights(const CUtensorMap& tk, const CUtensorMap& tq, const WeightsParams& p,
                                 cudaStream_t s) {
  const int rows = p.Hq / p.Hkv * p.Nq;
  if (rows > kWeightsStreamRows) return p.fp8 ? launch_tile<true>(tk, tq, p, s) : launch_tile<false>(tk, tq, p, s);
  if (p.fp8) return rows <= 16 ? launch_stream<true, 16>(tk, p, s) : launch_stream<true, 32>(tk, p, s);
  return rows <= 16 ? launch_stream<false, 16>(tk, p, s) : launch_stream<false, 32>(tk, p, s);
}

}  // namespace fa
