// fa_cache_attend_sm100.cu -- attention of a few new queries against an 8-bit cache, or
// against listed blocks of an 8-bit or bf16 cache, on sm_100a tensor cores.
//
// Bound by reading K and V once. As in the dense bf16 decode, keys and head-dim columns are the
// MMAs' M and the few query rows their N:
//   S^T(c) = K_c Q^T    M = 128 keys, N = R rows, K = d
//   O^T   += V_c^T P^T  M = d = 128,  N = R,      K = 128 keys
// and the units' chunks, laid end to end, are cut into equal slices over one CTA per SM
// (split along the keys), whose partial results a second kernel merges. What is new:
//   - 8-bit K and V feed the tensor cores as they are; Q and the weights are sums of three
//     E5M2 terms (fa_cache_sm100.cuh). V's scale goes into the weights: with y_j = x_j + log2(s_v)
//     the reference maximum runs over y, w_j = 2^(y_j - m) (times 2^11, which keeps 31 binades
//     below the reference above E5M2's smallest number) multiplies codes, and the
//     denominator sums 2^(x_j - m) unscaled.
//   - A chunk is 128 keys in a row, or 128 / block listed blocks, fetched by one TMA box
//     each: the producer's lanes read the list ahead and issue a block each. Block
//     positions and scales travel with the stage through shared memory.
//   - Two groups of softmax warps take alternate chunks, each with a running reference,
//     denominator and O^T of its own (two partial results a segment): at half the bytes a
//     key, one group's chain of wait, exponentials and hand-over would not keep up with the
//     memory. They meet nowhere within a segment.
//   - Keys that no row sees (behind a sequence's end, or past the query) have their V rows
//     zeroed in shared memory before the product: 0 * NaN would not be 0.
//
// Warps: 0 producer, 1 MMA issuer, 2-3 query rows (loaded, split and stored per segment), then
// 4 (R = 16) or 8 (R = 32) softmax warps for each parity of chunks: thread = TMEM lane =
// key of S^T and head-dim row of O^T, 16 query rows a thread.
#include <math.h>

#include "fa.h"
#include "fa_cache_sm100.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

template <bool FP8, int R>
struct AttCfg {
  static constexpr int kElem = FP8 ? 1 : 2;
  static constexpr int kTerms = FP8 ? 3 : 1;
  static constexpr int kHalves = R / 16;
  static constexpr int kGroups = 2 * kHalves;                  // softmax warpgroups
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kRegion = kChunk * 128;                 // 128-byte column block of a chunk
  static constexpr int kRegions = kElem;
  static constexpr int kKV = kRegions * kRegion;               // K or V of a chunk
  static constexpr int kStages = FP8 ? (R == 16 ? 6 : 5) : 3;
  static constexpr int kAhead = FP8 ? 4 : 2;                   // S buffers: S runs so many chunks ahead
  static_assert(kAhead <= kStages, "S(c + kAhead) takes the stage that P V(c) frees at the latest");
  static constexpr int kQTile = R * 128;                       // one term, or one 64-column block
  static constexpr int kQ = (FP8 ? 3 : 2) * kQTile;
  static constexpr int kQBufs = !FP8 && R == 32 ? 1 : 2;
  static constexpr int kPBlock = kChunk * 16;                  // 16-byte block of N, all keys
  static constexpr int kPTerm = (R * kElem / 16) * kPBlock;
  static constexpr int kP = kTerms * kPTerm;                   // one parity's weights
  static constexpr int kOffKV = 0;
  static constexpr int kOffQ = kOffKV + kStages * 2 * kKV;
  static constexpr int kOffP = kOffQ + kQBufs * kQ;
  static constexpr int kOffRed = kOffP + 2 * kP;               // [kGroups][4][16] floats
  static constexpr int kOffQScale = kOffRed + kGroups * 64 * 4;
  static constexpr int kOffMeta = kOffQScale + (FP8 ? kQScaleRing * R * 4 : 0);  // [kStages][3][8]
  static constexpr int kOffBar = kOffMeta + kStages * 96;
  // kv_full[S], kv_empty[S], q_full[2], q_empty[2], s_full[4], p_full[2], pv_done[2], mma_done,
  // qs_full[kQScaleRing]
  static constexpr int kNumBars = 2 * kStages + 13 + kQScaleRing;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
  static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static constexpr int kColS = 0, kColO = kAhead * R;
  static constexpr int kTmemUsed = kColO + 2 * R;
  static constexpr int kTmemCols = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : 256;
  static constexpr float kSlack = FP8 ? 4.f : 8.f;             // log2: the reference is raised beyond it
};

constexpr float kWeightUp = 2048.f;        // 2^11: 2^(11 + 4) is still below E5M2's 57344
constexpr float kWeightDown = 1.f / 2048.f;
constexpr float kMinValueScale = 7.888609052210118e-31f;  // 2^-100

// Who a unit is: batch entry, first query row, rows, and how rows and keys are masked.
struct UnitInfo {
  int b, bh, rows;        // rows of this unit (at most R)
  int list;               // index of its block list
  long long row0;         // first row in [B * Hq * Nq]; the next is row_step further
  int row_step;
  int r0;                 // first row within the group (its query is (r0 + j) % Nq)
};
template <bool LIST, int R>
__device__ __forceinline__ UnitInfo unit_info(const AttendParams& p, int unit) {
  UnitInfo u;
  const int rb = unit % p.n_rb, v = unit / p.n_rb;
  const int g = p.Hq / p.Hkv;
  u.r0 = rb * R;
  if constexpr (LIST) {
    const int i = v % p.Nq;
    u.bh = v / p.Nq;
    u.list = v;
    u.rows = min(g - u.r0, R);
    u.row0 = ((long long)u.bh * g + u.r0) * p.Nq + i;
    u.row_step = p.Nq;
  } else {
    u.bh = v;
    u.list = 0;
    u.rows = min(g * p.Nq - u.r0, R);
    u.row0 = (long long)u.bh * g * p.Nq + u.r0;
    u.row_step = 1;
  }
  u.b = u.bh / p.Hkv;
  return u;
}

template <bool FP8, int R, bool LIST>
__global__ void __launch_bounds__(AttCfg<FP8, R>::kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const AttendParams p) {
  using C = AttCfg<FP8, R>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1k(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + S;
  uint64_t* q_full = bars + 2 * S;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_full + 4;
  uint64_t* p_full = q_full + 8;
  uint64_t* pv_done = q_full + 10;
  uint64_t* mma_done = q_full + 12;
  uint64_t* qs_full = q_full + 13;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  float* qscale = reinterpret_cast<float*>(smem + C::kOffQScale);
  // per stage: first key of each block (-1: none), K scale * scale * log2 e, V scale
  int* meta = reinterpret_cast<int*>(smem + C::kOffMeta);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  WalkPos pos0;
  const int n = walk_start(p.walk, blockIdx.x, pos0);
  if (n == 0) return;  // shorter sequences than CTAs: nothing to do (the whole CTA)

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], 2);
      mbar_init(&q_empty[b], 1);
      mbar_init(&p_full[b], 4 * C::kHalves);
      mbar_init(&pv_done[b], 1);
    }
    for (int b = 0; b < 4; ++b) mbar_init(&s_full[b], 1);
    mbar_init(mma_done, 1);
    for (int b = 0; b < kQScaleRing; ++b) mbar_init(&qs_full[b], 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};
  const int blocks_per_chunk = kChunk / p.block;
  const int n_blocks = (p.Nk + p.block - 1) / p.block;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    // Lane l < blocks_per_chunk looks after block l of every chunk. Its list entry is read two
    // chunks ahead, its scales one ahead.
    const bool mine = lane < blocks_per_chunk;
    auto entry = [&](const WalkPos& ps) -> int {  // index of the block, -1 for none
      if (!mine) return -1;
      const int at = ps.cig * blocks_per_chunk + lane;
      if constexpr (LIST) {
        if (at >= p.n_select) return -1;
        const int j = __ldg(p.idx + (size_t)unit_info<true, R>(p, ps.unit).list * p.n_select + at);
        return j < 0 || j >= n_blocks ? -1 : j;
      } else {
        return at < n_blocks ? at : -1;
      }
    };
    auto scales = [&](const WalkPos& ps, int blk, float& a, float& v) {
      a = p.scale_log2, v = 1.f;
      if constexpr (FP8) {
        if (blk >= 0) {
          const size_t at = (size_t)unit_info<LIST, R>(p, ps.unit).bh * n_blocks + blk;
          a = __ldg(p.ks + at) * p.scale_log2;
          v = __ldg(p.vs + at);
        }
      }
    };
    WalkPos p0 = pos0, p1 = pos0, p2;
    int blk = entry(p0), blk1 = -1;
    if (n > 1) {
      p1.next(p.walk);
      blk1 = entry(p1);
    }
    p2 = p1;
    float a, v, a1 = 0.f, v1 = 0.f;
    scales(p0, blk, a, v);
    bool ok = true;
    int issued = 0;
    for (int c = 0; c < n; ++c) {
      // loads for the chunks behind this one, in flight while it waits for its stage
      int blk2 = -1;
      if (c + 1 < n) scales(p1, blk1, a1, v1);
      if (c + 2 < n) {
        p2.next(p.walk);
        blk2 = entry(p2);
      }
      const int s = c % S;
      ok = __shfl_sync(0xffffffffu, lane == 0 ? (int)mbar_wait_spin(&kv_empty[s], ((c / S) & 1) ^ 1, w) : 0, 0);
      if (!ok) break;
      uint8_t* st = smem + C::kOffKV + s * 2 * C::kKV;
      const int bh = unit_info<LIST, R>(p, p0.unit).bh;
      if constexpr (LIST) {
        if (mine) {  // a block that is not there is read past the end: zeros
          const int y = blk >= 0 ? blk * p.block : n_blocks * p.block;
          uint8_t* at = st + lane * p.block * 128;
#pragma unroll
          for (int z = 0; z < C::kRegions; ++z) {
            tma_load_3d(at + z * C::kRegion, &tmK, &kv_full[s], z * (128 / C::kElem), y, bh);
            tma_load_3d(at + C::kKV + z * C::kRegion, &tmV, &kv_full[s], z * (128 / C::kElem), y, bh);
          }
        }
      } else if (lane == 0) {
#pragma unroll
        for (int z = 0; z < C::kRegions; ++z) {
          tma_load_3d(st + z * C::kRegion, &tmK, &kv_full[s], z * (128 / C::kElem), p0.cig * kChunk, bh);
          tma_load_3d(st + C::kKV + z * C::kRegion, &tmV, &kv_full[s], z * (128 / C::kElem), p0.cig * kChunk, bh);
        }
      }
      if (mine) {
        int* m = meta + s * 24;
        m[lane] = blk >= 0 ? blk * p.block : -1;
        reinterpret_cast<float*>(m)[8 + lane] = a;
        reinterpret_cast<float*>(m)[16 + lane] = v;
      }
      __syncwarp();
      // the loads may complete before this arrival: the phase cannot
      if (lane == 0) mbar_arrive_expect_tx(&kv_full[s], 2 * C::kKV);
      ++issued;
      blk = blk1, a = a1, v = v1, p0 = p1;
      blk1 = blk2, p1 = p2;
    }
    if (!ok && lane == 0) {  // error path: let the loads already issued land before the CTA exits
      WaitCtx drain{abort_flag, p.status, 20000000ull};
      volatile int zero = 0;
      drain.abort_flag = &zero;
      for (int c = max(0, issued - S); c < issued; ++c) mbar_wait(&kv_full[c % S], (c / S) & 1, drain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = lane == 0;
    constexpr uint32_t kIdS = FP8 ? idesc_e4m3_e5m2(128, R, false, false) : idesc_bf16_f32(128, R, false, false);
    constexpr uint32_t kIdO = FP8 ? idesc_e4m3_e5m2(128, R, true, true) : idesc_bf16_f32(128, R, true, true);
    const uint64_t d_k = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);                          // K-major
    const uint64_t d_v = sdesc_sw128(smem_u32(smem + C::kOffKV + C::kKV), C::kRegion, 1024);        // MN-major
    const uint64_t d_q = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t d_p = sdesc_plain_mn(smem_u32(smem + C::kOffP), 128, C::kPBlock);
    auto issue_s = [&](int c, const WalkPos& ps) -> bool {
      const int qb = ps.seg % C::kQBufs;
      if (c == ps.first(c) && !mbar_wait_spin(&q_full[qb], (ps.seg / C::kQBufs) & 1, w)) return false;
      if (!mbar_wait_spin(&kv_full[c % S], (c / S) & 1, w)) return false;
      tc_fence_after();
      if (leader) {
        const uint64_t a0 = desc_advance(d_k, (c % S) * 2 * C::kKV);
        const uint64_t b0 = desc_advance(d_q, qb * C::kQ);
        const uint32_t d = tmem + C::kColS + (c % C::kAhead) * R;
        if constexpr (FP8) {
#pragma unroll
          for (int t = 2; t >= 0; --t)  // the small terms first
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_e4m3_ss(d, desc_advance(a0, k * 32), desc_advance(b0, t * C::kQTile + k * 32), kIdS,
                          t < 2 || k > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss(d, desc_advance(a0, (k >> 2) * C::kRegion + (k & 3) * 32),
                        desc_advance(b0, (k >> 2) * C::kQTile + (k & 3) * 32), kIdS, k > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[c % C::kAhead]);
        if (c == ps.last(c, n)) mma_commit(&q_empty[qb]);
      }
      return true;
    };
    auto issue_pv = [&](int c, const WalkPos& pp) {
      if (!leader) return;
      const uint64_t a0 = desc_advance(d_v, (c % S) * 2 * C::kKV);
      const uint64_t b0 = desc_advance(d_p, (c & 1) * C::kP);
      const uint32_t d = tmem + C::kColO + (c & 1) * R;
      const bool fresh = c - 2 < pp.first(c);  // this parity's first chunk of the segment
      if constexpr (FP8) {
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3_ss(d, desc_advance(a0, k * 32 * 128), desc_advance(b0, t * C::kPTerm + k * 32 * 16), kIdO,
                        !fresh || t < 2 || k > 0 ? 1u : 0u);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ss(d, desc_advance(a0, k * 16 * 128), desc_advance(b0, k * 16 * 16), kIdO,
                      !fresh || k > 0 ? 1u : 0u);
      }
      mma_commit(&pv_done[c & 1]);
      mma_commit(&kv_empty[c % S]);
    };
    bool ok = true;
    WalkPos ps = pos0, pp = pos0;
    for (int c = 0; c < C::kAhead && c < n && ok; ++c) {
      ok = issue_s(c, ps);
      ps.next(p.walk);
    }
    for (int c = 0; c < n && ok; ++c) {
      if (!(ok = mbar_wait_spin(&p_full[c & 1], (c >> 1) & 1, w))) break;
      tc_fence_after();
      issue_pv(c, pp);
      pp.next(p.walk);
      // into the S buffer that the softmax has read (p_full(c))
      if (c + C::kAhead < n) {
        if (!(ok = issue_s(c + C::kAhead, ps))) break;
        ps.next(p.walk);
      }
    }
    if (leader) mma_commit(mma_done);
    __syncwarp();
    WaitCtx drain{abort_flag, p.status, 20000000ull};
    volatile int zero = 0;
    drain.abort_flag = &zero;
    mbar_wait(mma_done, 0, drain);
  } else if (warp < 4) {
    // ------------------------------------------------------------ query rows
    // A segment's rows go into buffer seg % kQBufs once the S of the segment that had it are
    // done. Their scales are read by the softmax up to kAhead chunks later, hence a ring with barriers
    // of its own: with a segment per chunk, the softmax may be kAhead + 1 segments behind the one
    // whose rows are written.
    WalkPos ps = pos0;
    for (int c = 0; c < n;) {
      const int qb = ps.seg % C::kQBufs;
      if (!warp_wait_all(&q_empty[qb], ((ps.seg / C::kQBufs) & 1) ^ 1, w)) break;
      const UnitInfo u = unit_info<LIST, R>(p, ps.unit);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
      load_query_rows<FP8, R, 2>(smem + C::kOffQ + qb * C::kQ, qscale + (ps.seg % kQScaleRing) * R, warp - 2,
                                 [&](int r) -> const __nv_bfloat16* {
                                   return r < u.rows ? q + (u.row0 + (long long)r * u.row_step) * kCacheD : nullptr;
                                 });
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&q_full[qb]);
        mbar_arrive(&qs_full[ps.seg % kQScaleRing]);
      }
      const int last = ps.last(c, n);  // on to the next segment
      ps.cig += last - c;
      ps.next(p.walk);
      c = last + 1;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int group = (warp - 4) >> 2;            // parity * kHalves + half
    const int par = group / C::kHalves;
    const int jr0 = (group % C::kHalves) * 16;    // first query row of this group
    const int quarter = warp & 3;
    const int t = quarter * 32 + lane;
    const int bar_id = 1 + group;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::kColO + par * R + jr0;
    float* red = reinterpret_cast<float*>(smem + C::kOffRed) + group * 64;
    float m_ref[16], l_part[16], b_row[16];
    int lim0 = 0, lim_max = -1, my_rows = 0, r0 = 0;  // last key that row 0's query sees, and any row's
    UnitInfo u{};
    bool bad = false;
    WalkPos pos = pos0;
    if (par == 1 && n > 1) pos.next(p.walk);
    for (int c = par; c < n; c += 2) {
      const int c0 = pos.first(c), c1 = pos.last(c, n);
      const bool fresh = c - 2 < c0, done = c + 2 > c1;
      if (fresh) {
        u = unit_info<LIST, R>(p, pos.unit);
        const int len = cache_len(p.lens, u.b, p.Nk);
        r0 = u.r0 + jr0;
        my_rows = min(max(u.rows - jr0, 0), 16);
        // query of row j: (r0 + j) % Nq (listed blocks: one query for all rows)
        if (LIST) {
          lim0 = p.causal ? len - p.Nq + u.list % p.Nq : len - 1;
          lim_max = lim0;
        } else {
          lim0 = p.causal ? len - p.Nq : len - 1;  // seen by every row
          lim_max = len - 1;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          m_ref[j] = -FLT_MAX;
          l_part[j] = 0.f;
        }
      }
      bad |= !warp_wait_all(&s_full[c % C::kAhead], (c / C::kAhead) & 1, w);
      // block positions and scales of this chunk (and V, where it is written below)
      bad |= !warp_wait_all(&kv_full[c % S], (c / S) & 1, w);
      if (FP8 && fresh) {
        bad |= !warp_wait_all(&qs_full[pos.seg % kQScaleRing], (pos.seg / kQScaleRing) & 1, w);
        const float* qs = qscale + (pos.seg % kQScaleRing) * R + jr0;
#pragma unroll
        for (int j = 0; j < 16; ++j) b_row[j] = qs[j];
      }
      tc_fence_after();
      uint32_t r[16];
      tm_ld16(tmem + lane_off + C::kColS + (c % C::kAhead) * R + jr0, r);
      const int* mt = meta + (c % S) * 24;
      const int bi = t / p.block;
      const int base = mt[bi];
      const float a = reinterpret_cast<const float*>(mt)[8 + bi];
      const float sv = reinterpret_cast<const float*>(mt)[16 + bi];
      const float ls = FP8 ? __log2f(fmaxf(sv, kMinValueScale)) : 0.f;
      const int key = base + (t & (p.block - 1));
      const uint32_t row_mask = (1u << my_rows) - 1u;
      uint32_t vis = base >= 0 && key <= lim_max ? row_mask : 0u;
      if (!LIST && vis && key > lim0) {  // the causal edge
        vis = 0u;
        for (int j = 0; j < my_rows; ++j)
          if (key <= lim0 + (r0 + j) % p.Nq) vis |= 1u << j;
      }
      tm_ld16_wait(r);
      float x[16];
      bool over = false;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float s = __uint_as_float(r[j]);
        if (FP8) s *= b_row[j];
        x[j] = (vis >> j) & 1u ? s * a : -INFINITY;
        over |= x[j] + ls > m_ref[j] + C::kSlack;
      }
      // Does any key need a higher reference? Lane 0 votes for its warp; a warp whose waits ran
      // out adds five votes, so that the whole group leaves together.
      const bool wo = __any_sync(0xffffffffu, over);
      const int votes = group_count(bar_id, lane == 0 ? wo : lane < 6 && bad);
      if (votes >= 5) break;
      if (votes > 0) {
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = x[j] + ls;
        const float mx = warp_reduce16<MaxOp>(y);
        if (!(lane & 1)) red[quarter * 16 + (lane >> 1)] = mx;
        named_barrier(bar_id, 128);
        float alpha[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float cm = fmaxf(fmaxf(red[j], red[16 + j]), fmaxf(red[32 + j], red[48 + j]));
          const float m_new = fmaxf(m_ref[j], cm);
          alpha[j] = ex2(m_ref[j] - m_new);
          m_ref[j] = m_new;
          l_part[j] *= alpha[j];
        }
        if (!fresh) {  // O^T so far, once the products into it are complete
          bad |= !warp_wait_all(&pv_done[par], ((c - 2) >> 1) & 1, w);
          tc_fence_after();
          uint32_t o[16];
          tm_ld16(tO, o);
          tm_ld16_wait(o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[j]);
          tmem_st16(tO, o);
          tmem_st_wait();
        }
        named_barrier(bar_id, 128);  // the maxima have been read
      }
      // the weights, once the product that had this buffer is complete
      if (c >= 2) bad |= !warp_wait_all(&pv_done[par], ((c - 2) >> 1) & 1, w);
      uint8_t* pb = smem + C::kOffP + par * C::kP;
      if constexpr (FP8) {
        const float up = sv * kWeightUp;
        uint32_t tm[3][8];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float e0 = ex2(x[j] - m_ref[j]), e1 = ex2(x[j + 1] - m_ref[j + 1]);
          l_part[j] += e0;
          l_part[j + 1] += e1;
          uint32_t tt[3];
          split_e5m2(half2_bits(e0 * up, e1 * up), tt);
#pragma unroll
          for (int z = 0; z < 3; ++z) tm[z][j / 2] = tt[z];
        }
#pragma unroll
        for (int z = 0; z < 3; ++z)
          st_shared_v4(smem_u32(pb + z * C::kPTerm + (jr0 / 16) * C::kPBlock + t * 16), top_bytes(tm[z][0], tm[z][1]),
                       top_bytes(tm[z][2], tm[z][3]), top_bytes(tm[z][4], tm[z][5]), top_bytes(tm[z][6], tm[z][7]));
      } else {
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float e0 = ex2(x[j] - m_ref[j]), e1 = ex2(x[j + 1] - m_ref[j + 1]);
          l_part[j] += e0;
          l_part[j + 1] += e1;
          pk[j / 2] = pack_bf16x2(e0, e1);
        }
        const uint32_t at = smem_u32(pb + (jr0 / 8) * C::kPBlock + t * 16);
        st_shared_v4(at, pk[0], pk[1], pk[2], pk[3]);
        st_shared_v4(at + C::kPBlock, pk[4], pk[5], pk[6], pk[7]);
      }
      // V rows that no row sees, zeroed (every group that shares the chunk writes the same)
      if (base >= 0 && key > lim_max) {
        uint8_t* vr = smem + C::kOffKV + (c % S) * 2 * C::kKV + C::kKV + t * 128;
#pragma unroll
        for (int z = 0; z < C::kRegions; ++z)
          for (int e = 0; e < 8; ++e) st_shared_v4(smem_u32(vr + z * C::kRegion + e * 16), 0u, 0u, 0u, 0u);
      }
      fence_async_smem();  // the stores above, visible to the MMA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[par]);
      if (done) {
        // this parity's part of the segment: denominators over the 128 threads, O^T / l and LSE
        const float sum = warp_reduce16<SumOp>(l_part);
        if (!(lane & 1)) red[quarter * 16 + (lane >> 1)] = sum;
        named_barrier(bar_id, 128);
        bad |= !warp_wait_all(&pv_done[par], (c >> 1) & 1, w);
        tc_fence_after();
        uint32_t o[16];
        tm_ld16(tO, o);
        tm_ld16_wait(o);
        const size_t slot = ((size_t)pos.unit + blockIdx.x) * 2;
        const size_t row = (slot + par) * R + jr0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (j < my_rows) {
            const float l = red[j] + red[16 + j] + red[32 + j] + red[48 + j];
            const float inv = l == 0.f ? 0.f : (FP8 ? kWeightDown : 1.f) / l;
            p.o_part[(row + j) * kCacheD + t] = __uint_as_float(o[j]) * inv;
            if (t == 0) {
              p.lse_part[row + j] = l == 0.f ? -INFINITY : m_ref[j] + log2f(l);
              if (c0 == c1) p.lse_part[(slot + 1 - par) * R + jr0 + j] = -INFINITY;  // the other parity had no chunk
            }
          }
        }
        tc_fence_before();
        named_barrier(bar_id, 128);  // the sums have been read
      }
      pos.next(p.walk);
      if (c + 2 < n) pos.next(p.walk);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// One CTA per query row: the partial results of its unit (two per CTA whose slice met it)
// combined by their log-sum-exps: LSE = log sum_s e^(LSE_s), O = sum_s e^(LSE_s - LSE) O_s.
// Each of the four warps takes every fourth partial.
template <int R, bool LIST>
__global__ void __launch_bounds__(128) merge_kernel(const AttendParams p) {
  __shared__ float so[4][kCacheD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / R, j = blockIdx.x % R;
  const UnitInfo u = unit_info<LIST, R>(p, unit);
  if (j >= u.rows) return;
  const long long row = u.row0 + (long long)j * u.row_step;
  const WalkParams& wk = p.walk;
  const int nch = walk_chunks(wk, u.b);
  const long long total = wk.lens ? walk_prefix(wk, wk.B) : wk.total;
  const int slices = walk_slices(wk, total);
  const long long f0 = walk_prefix(wk, u.b) + (long long)(unit - u.b * wk.units_per_b) * nch;
  int parts = 0;
  size_t first = 0;  // partial s of the row is row (first + s * R) of the workspace
  if (nch > 0) {
    const int i0 = walk_cta_of(f0, total, slices), i1 = walk_cta_of(f0 + nch - 1, total, slices);
    parts = 2 * (i1 - i0 + 1);
    first = ((size_t)unit + i0) * 2 * R + j;
  }
  float m = -INFINITY;
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, p.lse_part[first + (size_t)s * R]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // NaN partials: fmaxf skips them, their weight below is NaN
  const float mm = m == -INFINITY ? 0.f : m;
  float wsum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = lane; s < parts; s += 32) wsum += ex2(p.lse_part[first + (size_t)s * R] - mm);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
#pragma unroll 4
  for (int s = warp; s < parts; s += 4) {
    const size_t at = first + (size_t)s * R;
    const float ls = p.lse_part[at];
    if (ls == -INFINITY) continue;  // nothing seen: its O was not written
    const float wgt = ex2(ls - mm);
    const float4 v = *reinterpret_cast<const float4*>(p.o_part + at * kCacheD + lane * 4);
    acc[0] += wgt * v.x, acc[1] += wgt * v.y, acc[2] += wgt * v.z, acc[3] += wgt * v.w;
  }
  *reinterpret_cast<float4*>(&so[warp][lane * 4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  const float o = so[0][threadIdx.x] + so[1][threadIdx.x] + so[2][threadIdx.x] + so[3][threadIdx.x];
  static_cast<__nv_bfloat16*>(p.o)[row * kCacheD + threadIdx.x] = __float2bfloat16(o * inv);
  if (threadIdx.x == 0) p.lse[row] = wsum == 0.f ? -INFINITY : (mm + log2f(wsum)) * 0.6931471805599453f;
}

template <bool FP8, int R, bool LIST>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p, cudaStream_t s) {
  using C = AttCfg<FP8, R>;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = ensure_smem_limit(attend_kernel<FP8, R, LIST>, C::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  attend_kernel<FP8, R, LIST><<<(unsigned)p.walk.n_ctas, C::kThreads, C::kSmemBytes, s>>>(tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  merge_kernel<R, LIST><<<(unsigned)(p.units * R), 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attend(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p, cudaStream_t s) {
  if (!p.fp8)
    return p.unit_rows == 16 ? launch<false, 16, true>(tk, tv, p, s) : launch<false, 32, true>(tk, tv, p, s);
  if (p.idx) return p.unit_rows == 16 ? launch<true, 16, true>(tk, tv, p, s) : launch<true, 32, true>(tk, tv, p, s);
  return p.unit_rows == 16 ? launch<true, 16, false>(tk, tv, p, s) : launch<true, 32, false>(tk, tv, p, s);
}

}  // namespace fa
