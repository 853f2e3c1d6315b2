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
//     E5M2 terms (fa_cache_sm100.cuh), side by side in N: an MMA of M = 128 costs about the
//     same for N = 16 and N = 48, and the softmax adds three columns. V's scale goes into the weights: with y_j = x_j + log2(s_v)
//     the reference maximum runs over y, w_j = 2^(y_j - m) (times 2^11, in fp16: 11 bits down to 2^-25
//     of the reference, steps of 2^-35 below) multiplies codes, and the
//     denominator sums 2^(x_j - m) unscaled. The reference runs over scales, not over codes: a key
//     whose block has a scale far above its own codes costs the others such steps.
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
// Warps: 0 producer, 1 S issuer, 2 query rows (loaded, split and stored per segment), 3 P V issuer, then
// four softmax warps for each parity of chunks: thread = TMEM lane = key of S^T and
// head-dim row of O^T, 16 query rows a thread. A group of more than 16 rows is several units,
// which read the same keys at about the same time, mostly from L2: a variant with 32 rows and
// twice the softmax warps was slower (32 rows, B4 Hkv8 Nk32768: 118 us against 100).
#include <math.h>

#include "fa.h"
#include "fa_cache_sm100.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int R = kUnitRows;  // query rows of a unit: a third of the MMAs' N

template <bool FP8>
struct AttCfg {
  static constexpr int kElem = FP8 ? 1 : 2;
  static constexpr int kTerms = FP8 ? 3 : 1;                   // of a query row
  static constexpr int kPTerms = FP8 ? 3 : 2;                  // of the weights (bf16: 16 bits)
  static constexpr float kPTermDown = FP8 ? kTermDown : 1.f;   // a term's unit in the one before it
  static constexpr int kGroups = 2;                            // softmax warpgroups, by parity of the chunk
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kRegion = kChunk * 128;                 // 128-byte column block of a chunk
  static constexpr int kRegions = kElem;
  static constexpr int kKV = kRegions * kRegion;               // K or V of a chunk
  static constexpr int kStages = FP8 ? 5 : 3;
  static constexpr int kN = kTerms * R, kNO = kPTerms * R;     // the MMAs' N: all terms side by side
  static constexpr int kAhead = FP8 ? 4 : 2;                   // S buffers: S runs so many chunks ahead
  static constexpr int kQTile = R * 128;                       // one term, or one 64-column block
  static constexpr int kQ = (FP8 ? 3 : 2) * kQTile;
  static constexpr int kQBufs = 2;
  static constexpr int kPBlock = kChunk * 16;                  // 16-byte block of N, all keys
  static constexpr int kPTerm = (R * kElem / 16) * kPBlock;
  static constexpr int kP = kPTerms * kPTerm;                   // the weights of one chunk
  static constexpr int kPBufs = FP8 ? 2 : 1;                   // for each parity of chunks
  static constexpr int kOffKV = 0;
  static constexpr int kOffQ = kOffKV + kStages * 2 * kKV;
  static constexpr int kOffP = kOffQ + kQBufs * kQ;
  static constexpr int kOffRed = kOffP + 2 * kPBufs * kP;               // [kGroups][4][16] floats
  static constexpr int kOffQScale = kOffRed + kGroups * 64 * 4;
  static constexpr int kOffMeta = kOffQScale + (FP8 ? kQScaleRing * R * 4 : 0);  // [kStages][3][8]
  static constexpr int kOffBar = kOffMeta + kStages * 96;
  // kv_full[S], kv_empty[S], q_full[2], q_empty[2], s_full[4], p_full[4], pv_done[4], mma_done[2],
  // qs_full[kQScaleRing]
  static constexpr int kNumBars = 2 * kStages + 18 + kQScaleRing;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
  static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static constexpr int kColS = 0, kColO = kAhead * kN;
  static constexpr int kTmemUsed = kColO + 2 * kNO;
  static constexpr int kTmemCols = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= kTmemCols, "Tensor Memory columns");
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
template <bool LIST>
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

template <bool FP8, bool LIST>
__global__ void __launch_bounds__(AttCfg<FP8>::kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const AttendParams p) {
  using C = AttCfg<FP8>;
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
  uint64_t* pv_done = q_full + 12;
  uint64_t* mma_done = q_full + 16;
  uint64_t* qs_full = q_full + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  float* qscale = reinterpret_cast<float*>(smem + C::kOffQScale);
  // per stage: first key of each block (-1: none), K scale * scale * log2 e, V scale
  int* meta = reinterpret_cast<int*>(smem + C::kOffMeta);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&q_empty[b], 1);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 4);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    for (int b = 0; b < kQScaleRing; ++b) mbar_init(&qs_full[b], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  // rows of a unit that do not exist: zeros, scale 1 (later units may leave finite rows there)
  for (int e = threadIdx.x; e < C::kQBufs * C::kQ / 16; e += C::kThreads)
    *reinterpret_cast<uint4*>(smem + C::kOffQ + e * 16) = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (FP8) {
    for (int e = threadIdx.x; e < kQScaleRing * R; e += C::kThreads) qscale[e] = 1.f;
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx w{abort_flag, p.status, p.wait_budget_ns};
  grid_wait();  // no memory is read or written before this
  WalkPos pos0;
  const int n = walk_start(p.walk, blockIdx.x, pos0);  // 0: fewer chunks than CTAs, nothing to do
  // the first unit's query rows, by every warp but the producer's
  if (warp > 0) {
    if (n > 0) {
      const UnitInfo u = unit_info<LIST>(p, pos0.unit);
      load_query_rows<FP8, R>(smem + C::kOffQ, qscale,
                              static_cast<const __nv_bfloat16*>(p.q) + u.row0 * kCacheD, u.row_step * kCacheD, warp - 1,
                              C::kThreads / 32 - 1, u.rows);
    }
    named_barrier(15, C::kThreads - 32);
  }
  // The weights' buffer of chunk c (its parity's buffers in turn), and the phase of the buffer's
  // barriers for it. p_full and pv_done are per buffer: a phase of either is never more than one
  // ahead of the thread that waits for it, since P(c) is written after P V of the chunk before
  // it in the buffer.
  auto p_buf = [](int c) { return (c & 1) * C::kPBufs + (c >> 1) % C::kPBufs; };
  auto p_phase = [](int c) -> uint32_t { return ((c >> 1) / C::kPBufs) & 1; };
  const int bl = p.block_log2;             // log2 of the block size
  const int pl = 7 - bl;                   // log2 of the blocks per chunk
  const int blocks_per_chunk = 1 << pl;
  const int n_blocks = (p.Nk + p.block - 1) >> bl;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // List entries and scales are read for `batch` chunks at a time, a lane for each block, and
    // a batch ahead: a chunk's time is shorter than a load's.
    const int batch_log2 = 5 - pl, batch = 1 << batch_log2;
    const int l_chunk = lane >> pl, l_block = lane & (blocks_per_chunk - 1);
    WalkPos lp = pos0;  // this lane's chunk of the batch that is read
    auto entry = [&](int c0) -> int {  // block of this lane's chunk c0 + l_chunk, -1 for none
      if (c0 + l_chunk >= n) return -1;
      const int at = (lp.cig << pl) + l_block;
      if constexpr (LIST) {
        if (at >= p.n_select) return -1;
        const int j = __ldg(p.idx + (size_t)unit_info<true>(p, lp.unit).list * p.n_select + at);
        return j < 0 || j >= n_blocks ? -1 : j;
      } else {
        return at < n_blocks ? at : -1;
      }
    };
    auto scales = [&](int blk, float& a, float& v) {
      a = v = 1.f;
      if constexpr (FP8) {
        if (blk >= 0) {
          const size_t at = (size_t)unit_info<LIST>(p, lp.unit).bh * n_blocks + blk;
          a = __ldg(p.ks + at);
          v = __ldg(p.vs + at);
        }
      }
    };
    auto fetch = [&](int s, int bh, int blk) {  // K and V of a chunk into stage s
      uint8_t* st = smem + C::kOffKV + s * 2 * C::kKV;
      uint64_t* bar = &kv_full[s];
      if constexpr (LIST) {
        if (lane < blocks_per_chunk) {  // a block that is not there is read past the end: zeros
          const int y = (blk >= 0 ? blk : n_blocks) << bl;
          uint8_t* at = st + ((lane << bl) * 128);
#pragma unroll
          for (int z = 0; z < C::kRegions; ++z) {
            tma_load_3d(at + z * C::kRegion, &tmK, bar, z * (128 / C::kElem), y, bh);
            tma_load_3d(at + C::kKV + z * C::kRegion, &tmV, bar, z * (128 / C::kElem), y, bh);
          }
        }
      } else if (lane == 0) {
        const int y = blk << bl;  // the chunk's first block
#pragma unroll
        for (int z = 0; z < C::kRegions; ++z) {
          tma_load_3d(st + z * C::kRegion, &tmK, bar, z * (128 / C::kElem), y, bh);
          tma_load_3d(st + C::kKV + z * C::kRegion, &tmV, bar, z * (128 / C::kElem), y, bh);
        }
      }
    };
    bool ok = true;
    int issued = 0;
    if (n > 0) {
      lp.skip(p.walk, l_chunk);
      int blk = entry(0), blk1 = -1;
      WalkPos pf = pos0;  // the chunk that is fetched
      int bh = unit_info<LIST>(p, pf.unit).bh;
      int cf = 0, sf = 0, sm = 0;  // its number, its stage, and the stage that is announced
      auto fetch_next = [&]() {
        fetch(sf, bh, __shfl_sync(0xffffffffu, blk, ((cf & (batch - 1)) << pl) + l_block));
        ++cf;
        if (++sf == S) sf = 0;
        const int unit = pf.unit;
        pf.next(p.walk);
        if (pf.unit != unit && cf < n) bh = unit_info<LIST>(p, pf.unit).bh;
      };
      // The first scales' loads in front of the keys' (behind them they would come back 4 us
      // later); then the ring is filled, as far as this batch reaches, before they are waited for.
      float a, v, a1 = 0.f, v1 = 0.f;
      scales(blk, a, v);
      while (cf < S && cf < n && cf < batch) fetch_next();
      uint32_t empty_phase = sf == 0 ? 0u : 1u;  // of stage sf: complete for a stage's first use
      for (int c = 0; c < n; ++c) {
        const int j = c & (batch - 1);
        if (j == 0) {
          if (c > 0) blk = blk1, a = a1, v = v1;
          lp.skip(p.walk, batch);
          blk1 = entry(c + batch);
        }
        if (j == batch / 2) scales(blk1, a1, v1);
        if (cf <= c) {
          ok = __shfl_sync(0xffffffffu, lane == 0 ? (int)mbar_wait_spin(&kv_empty[sf], empty_phase, w) : 0, 0);
          if (!ok) break;
          if (sf == S - 1) empty_phase ^= 1u;
          fetch_next();
        }
        if (!ok) break;
        const int src = (j << pl) + l_block;
        const int mb = __shfl_sync(0xffffffffu, blk, src);
        const float ma = __shfl_sync(0xffffffffu, a, src), mv = __shfl_sync(0xffffffffu, v, src);
        if (lane < blocks_per_chunk) {
          int* m = meta + sm * 24;
          m[lane] = mb >= 0 ? mb << bl : -1;
          reinterpret_cast<float*>(m)[8 + lane] = ma * p.scale_log2;
          reinterpret_cast<float*>(m)[16 + lane] = mv;
        }
        __syncwarp();
        // the loads may complete before this arrival: the phase cannot
        if (lane == 0) mbar_arrive_expect_tx(&kv_full[sm], 2 * C::kKV);
        if (++sm == S) sm = 0;
        ++issued;
      }
    }
    if (!ok && lane == 0) {  // error path: let the loads already issued land before the CTA exits
      WaitCtx drain{abort_flag, p.status, 20000000ull};
      volatile int zero = 0;
      drain.abort_flag = &zero;
      for (int c = max(0, issued - S); c < issued; ++c) mbar_wait(&kv_full[c % S], (c / S) & 1, drain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S issuer
    // The two products have an issuing thread each: issuing a chunk's four MMAs and its commits
    // takes a thread about 450 cycles, and neither product then waits behind the other's
    // barriers. S(c) waits for its keys and for the buffer that the softmax had read when it
    // handed over P(c - kAhead).
    constexpr uint32_t kIdS = FP8 ? idesc_e4m3_e5m2(128, C::kN, false, false) : idesc_bf16_f32(128, C::kN, false, false);
    if (lane == 0) {
      const uint64_t d_k = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);  // K-major
      const uint64_t d_q = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
      WalkPos ps = pos0;
      int st = 0, sb = 0;
      uint32_t kv_phase = 0;
      for (int c = 0; c < n; ++c) {
        const int qb = ps.seg % C::kQBufs;
        if (c >= C::kAhead && !mbar_wait_spin(&p_full[p_buf(c - C::kAhead)], p_phase(c - C::kAhead), w)) break;
        if ((c == 0 || ps.cig == 0) && !mbar_wait_spin(&q_full[qb], (ps.seg / C::kQBufs) & 1, w)) break;
        if (!mbar_wait_spin(&kv_full[st], kv_phase, w)) break;
        tc_fence_after();
        const uint64_t a0 = desc_advance(d_k, st * 2 * C::kKV);
        const uint64_t b0 = desc_advance(d_q, qb * C::kQ);
        const uint32_t d = tmem + C::kColS + sb * C::kN;
        if constexpr (FP8) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3_ss(d, desc_advance(a0, k * 32), desc_advance(b0, k * 32), kIdS, k > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss(d, desc_advance(a0, (k >> 2) * C::kRegion + (k & 3) * 32),
                        desc_advance(b0, (k >> 2) * C::kQTile + (k & 3) * 32), kIdS, k > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[sb]);
        if (c == n - 1 || ps.cig == ps.nch - 1) mma_commit(&q_empty[qb]);
        if (++st == S) st = 0, kv_phase ^= 1u;
        if (++sb == C::kAhead) sb = 0;
        ps.next(p.walk);
      }
      mma_commit(&mma_done[0]);
      WaitCtx drain{abort_flag, p.status, 20000000ull};
      volatile int zero = 0;
      drain.abort_flag = &zero;
      mbar_wait(&mma_done[0], 0, drain);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ P V issuer
    constexpr uint32_t kIdO = FP8 ? idesc_e4m3_e5m2(128, C::kNO, true, true) : idesc_bf16_f32(128, C::kNO, true, true);
    if (lane == 0) {
      const uint64_t d_v = sdesc_sw128(smem_u32(smem + C::kOffKV + C::kKV), C::kRegion, 1024);  // MN-major
      const uint64_t d_p = sdesc_plain_mn(smem_u32(smem + C::kOffP), 128, C::kPBlock);
      WalkPos pp = pos0;
      int st = 0;
      for (int c = 0; c < n; ++c) {
        if (!mbar_wait_spin(&p_full[p_buf(c)], p_phase(c), w)) break;
        tc_fence_after();
        const uint64_t a0 = desc_advance(d_v, st * 2 * C::kKV);
        const uint64_t b0 = desc_advance(d_p, p_buf(c) * C::kP);
        const uint32_t d = tmem + C::kColO + (c & 1) * C::kNO;
        const bool fresh = c < 2 || pp.cig < 2;  // this parity's first chunk of the segment
        if constexpr (FP8) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3_ss(d, desc_advance(a0, k * 32 * 128), desc_advance(b0, k * 32 * 16), kIdO,
                        !fresh || k > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_bf16_ss(d, desc_advance(a0, k * 16 * 128), desc_advance(b0, k * 16 * 16), kIdO,
                        !fresh || k > 0 ? 1u : 0u);
        }
        mma_commit(&pv_done[p_buf(c)]);
        mma_commit(&kv_empty[st]);
        if (++st == S) st = 0;
        pp.next(p.walk);
      }
      mma_commit(&mma_done[1]);
      WaitCtx drain{abort_flag, p.status, 20000000ull};
      volatile int zero = 0;
      drain.abort_flag = &zero;
      mbar_wait(&mma_done[1], 0, drain);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ query rows
    // A segment's rows go into buffer seg % kQBufs once the S of the segment that had it are
    // done. Their scales are read by the softmax up to kAhead chunks later, hence a ring with barriers
    // of its own: with a segment per chunk, the softmax may be kAhead + 1 segments behind the one
    // whose rows are written.
    WalkPos ps = pos0;
    for (int c = 0; c < n;) {
      const int qb = ps.seg % C::kQBufs;
      if (ps.seg > 0) {  // the first is there
        if (!warp_wait_all(&q_empty[qb], ((ps.seg / C::kQBufs) & 1) ^ 1, w)) break;
        const UnitInfo u = unit_info<LIST>(p, ps.unit);
        load_query_rows<FP8, R>(smem + C::kOffQ + qb * C::kQ, qscale + (ps.seg % kQScaleRing) * R,
                                static_cast<const __nv_bfloat16*>(p.q) + u.row0 * kCacheD, u.row_step * kCacheD, 0, 1,
                                u.rows);
      }
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
    const int par = (warp - 4) >> 2;              // takes the chunks of this parity
    const int quarter = warp & 3;
    const int t = quarter * 32 + lane;
    const int bar_id = 1 + par;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_off + C::kColO + par * C::kNO;
    float* red = reinterpret_cast<float*>(smem + C::kOffRed) + par * 64;
    float m_ref[16];
    uint64_t l_part[8], b_row[8];  // pairs of rows
    int lim0 = 0, lim_max = -1, my_rows = 0, r0 = 0;  // last key that row 0's query sees, and any row's
    bool bad = false;
    WalkPos pos = pos0;
    const int slot_t = t & (p.block - 1), bi = t >> bl;
    int c = par;                // chunk
    int c0 = 0, c1 = -1;        // first and last chunk of its segment
    if (c < n) pos.skip(p.walk, c);
    int sb = c % C::kAhead, st = c % S;   // its S buffer and its stage, with their phases
    uint32_t sb_phase = (c / C::kAhead) & 1, st_phase = (c / S) & 1;
    for (; c < n;) {
      const bool fresh = c > c1 || c - 2 < c0;
      if (c > c1) {  // a segment of its own: rows and limits of the unit
        c0 = pos.first(c);
        c1 = pos.last(c, n);
        const UnitInfo u = unit_info<LIST>(p, pos.unit);
        const int len = cache_len(p.lens, u.b, p.Nk);
        r0 = u.r0;
        my_rows = u.rows;
        // query of row j: (r0 + j) % Nq (listed blocks: one query for all rows)
        if (LIST) {
          lim0 = p.causal ? len - p.Nq + u.list % p.Nq : len - 1;
          lim_max = lim0;
        } else {
          lim0 = p.causal ? len - p.Nq : len - 1;  // seen by every row
          lim_max = len - 1;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) m_ref[j] = -FLT_MAX;
#pragma unroll
        for (int j = 0; j < 8; ++j) l_part[j] = f2_pack(0.f, 0.f);
        if constexpr (FP8) {
          bad |= !warp_wait_all(&qs_full[pos.seg % kQScaleRing], (pos.seg / kQScaleRing) & 1, w);
          const float2* qs = reinterpret_cast<const float2*>(qscale + (pos.seg % kQScaleRing) * R);
#pragma unroll
          for (int j = 0; j < 8; ++j) b_row[j] = f2_pack(qs[j].x, qs[j].y);
        }
      }
      // the scores; and block positions, scales (and V, where it is written below) of this chunk
      bad |= !warp_wait_both(&s_full[sb], sb_phase, &kv_full[st], st_phase, w);
      tc_fence_after();
      const uint32_t tS = tmem + lane_off + C::kColS + sb * C::kN;
      uint32_t r[C::kTerms][16];
#pragma unroll
      for (int z = 0; z < C::kTerms; ++z) tm_ld16(tS + z * R, r[z]);
      const int* mt = meta + st * 24;
      const int base = mt[bi];
      const float a = reinterpret_cast<const float*>(mt)[8 + bi];
      float sv = reinterpret_cast<const float*>(mt)[16 + bi];
      const int key = base + slot_t;
      // rows that see this key; a chunk that every row sees whole needs no mask (rows past the
      // unit's end are left unmasked: nothing of them is written)
      uint32_t vis = base >= 0 && key <= lim_max ? 0xFFFFu : 0u;
      if (!LIST && vis && key > lim0) {  // the causal edge
        vis = 0u;
        for (int j = 0; j < my_rows; ++j)
          if (key <= lim0 + (r0 + j) % p.Nq) vis |= 1u << j;
      }
      const bool masked = __any_sync(0xffffffffu, vis != 0xFFFFu);
      if (vis == 0u) sv = 1.f;  // the scale of a block without a token may be anything: 0 * NaN is not 0
      const float ls = FP8 ? __log2f(fmaxf(sv, kMinValueScale)) : 0.f;
#pragma unroll
      for (int z = 0; z < C::kTerms; ++z) tm_ld16_wait(r[z]);
      // s: scores in units of a (K scale * scale * log2 e); x = s a, exponent e = x - m_ref
      uint64_t s[8];
      float e[16];
      const uint64_t aa = f2_pack(a, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        auto two = [&](int z) { return f2_pack(__uint_as_float(r[z][2 * j]), __uint_as_float(r[z][2 * j + 1])); };
        if constexpr (FP8)
          s[j] = f2_mul(add_terms(two(0), two(1), two(2)), b_row[j]);
        else
          s[j] = two(0);
        f2_unpack(f2_fma(s[j], aa, f2_pack(-m_ref[2 * j], -m_ref[2 * j + 1])), e[2 * j], e[2 * j + 1]);
      }
      if (masked) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!((vis >> j) & 1u)) e[j] = -INFINITY;
      }
      float top = fmax3(fmax3(e[0], e[1], e[2]), fmax3(e[3], e[4], e[5]), fmax3(e[6], e[7], e[8]));
      top = fmax3(fmax3(top, e[9], e[10]), fmax3(e[11], e[12], e[13]), fmaxf(e[14], e[15]));
      // Does any key need a higher reference? Lane 0 votes for its warp; a warp whose waits ran
      // out adds five votes, so that the whole group leaves together.
      const bool wo = __any_sync(0xffffffffu, top + ls > C::kSlack);
      const int votes = group_count(bar_id, lane == 0 ? wo : lane < 6 && bad);
      if (votes >= 5) break;
      if (votes > 0) {
        float y[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) f2_unpack(f2_fma(s[j], aa, f2_pack(ls, ls)), y[2 * j], y[2 * j + 1]);
        if (masked) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (!((vis >> j) & 1u)) y[j] = -INFINITY;
        }
        const float mx = warp_reduce16<MaxOp>(y);
        if (!(lane & 1)) red[quarter * 16 + (lane >> 1)] = mx;
        named_barrier(bar_id, 128);
        float alpha[16];
        const float4* red4 = reinterpret_cast<const float4*>(red);
#pragma unroll
        for (int j4 = 0; j4 < 4; ++j4) {
          const float4 a0 = red4[j4], a1 = red4[4 + j4], a2 = red4[8 + j4], a3 = red4[12 + j4];
          const float cm[4] = {fmax3(fmaxf(a0.x, a1.x), a2.x, a3.x), fmax3(fmaxf(a0.y, a1.y), a2.y, a3.y),
                               fmax3(fmaxf(a0.z, a1.z), a2.z, a3.z), fmax3(fmaxf(a0.w, a1.w), a2.w, a3.w)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j4 * 4 + i;
            const float m_new = fmaxf(m_ref[j], cm[i]);
            alpha[j] = ex2(m_ref[j] - m_new);
            m_ref[j] = m_new;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          l_part[j] = f2_mul(l_part[j], f2_pack(alpha[2 * j], alpha[2 * j + 1]));
          f2_unpack(f2_fma(s[j], aa, f2_pack(-m_ref[2 * j], -m_ref[2 * j + 1])), e[2 * j], e[2 * j + 1]);
        }
        if (masked) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (!((vis >> j) & 1u)) e[j] = -INFINITY;
        }
        if (!fresh) {  // O^T so far, once the products into it are complete
          bad |= !warp_wait_all(&pv_done[p_buf(c - 2)], p_phase(c - 2), w);
          tc_fence_after();
#pragma unroll
          for (int z = 0; z < C::kPTerms; ++z) {
            uint32_t o[16];
            tm_ld16(tO + z * R, o);
            tm_ld16_wait(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[j]);
            tmem_st16(tO + z * R, o);
          }
          tmem_st_wait();
        }
        named_barrier(bar_id, 128);  // the maxima have been read
      }
      // the weights, once the product that had this buffer is complete
#pragma unroll
      for (int j = 0; j < 16; ++j) e[j] = ex2(e[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j) l_part[j] = f2_add(l_part[j], f2_pack(e[2 * j], e[2 * j + 1]));
      if (c >= 2 * C::kPBufs) bad |= !warp_wait_all(&pv_done[p_buf(c)], p_phase(c) ^ 1, w);
      uint8_t* pb = smem + C::kOffP + p_buf(c) * C::kP;
      if constexpr (FP8) {
        const float up = sv * kWeightUp;
        uint32_t tm[3][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float e0, e1;
          f2_unpack(f2_mul(f2_pack(e[2 * j], e[2 * j + 1]), f2_pack(up, up)), e0, e1);
          uint32_t tt[3];
          split_e5m2(half2_bits(e0, e1), tt);
#pragma unroll
          for (int z = 0; z < 3; ++z) tm[z][j] = tt[z];
        }
#pragma unroll
        for (int z = 0; z < 3; ++z)
          st_shared_v4(smem_u32(pb + z * C::kPTerm + t * 16), top_bytes(tm[z][0], tm[z][1]),
                       top_bytes(tm[z][2], tm[z][3]), top_bytes(tm[z][4], tm[z][5]), top_bytes(tm[z][6], tm[z][7]));
      } else {
        // bf16 and the rest in bf16: with 8 bits alone the weights' rounding was as large as the output's
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hi[j] = pack_bf16x2(e[2 * j], e[2 * j + 1]);
          const float2 h = bf162_bits_to_float2(hi[j]);
          lo[j] = pack_bf16x2(e[2 * j] - h.x, e[2 * j + 1] - h.y);
        }
        const uint32_t at = smem_u32(pb + t * 16);
        st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(at + C::kPBlock, hi[4], hi[5], hi[6], hi[7]);
        st_shared_v4(at + C::kPTerm, lo[0], lo[1], lo[2], lo[3]);
        st_shared_v4(at + C::kPTerm + C::kPBlock, lo[4], lo[5], lo[6], lo[7]);
      }
      // V rows that no row sees, zeroed
      if (masked && base >= 0 && key > lim_max) {
        uint8_t* vr = smem + C::kOffKV + st * 2 * C::kKV + C::kKV + t * 128;
#pragma unroll
        for (int z = 0; z < C::kRegions; ++z)
          for (int i = 0; i < 8; ++i) st_shared_v4(smem_u32(vr + z * C::kRegion + i * 16), 0u, 0u, 0u, 0u);
      }
      fence_async_smem();  // the stores above, visible to the MMA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[p_buf(c)]);
      if (c + 2 > c1) {
        // this parity's part of the segment: denominators over the 128 threads, O^T / l and LSE
        float lp[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) f2_unpack(l_part[j], lp[2 * j], lp[2 * j + 1]);
        const float sum = warp_reduce16<SumOp>(lp);
        if (!(lane & 1)) red[quarter * 16 + (lane >> 1)] = sum;
        named_barrier(bar_id, 128);
        // lane j (and j + 16) looks after row j
        const int jl = lane & 15;
        const float l = red[jl] + red[16 + jl] + red[32 + jl] + red[48 + jl];
        const float inv = l == 0.f ? 0.f : (FP8 ? kWeightDown : 1.f) / l;
        float m_l = m_ref[0];
#pragma unroll
        for (int j = 1; j < 16; ++j) m_l = jl == j ? m_ref[j] : m_l;
        const size_t slot = ((size_t)pos.unit + blockIdx.x) * 2;
        const size_t row = (slot + par) * R;
        if (t < my_rows) {
          p.lse_part[row + t] = l == 0.f ? -INFINITY : m_l + log2f(l);
          if (c0 == c1) p.lse_part[(slot + 1 - par) * R + t] = -INFINITY;  // the other parity had no chunk
        }
        bad |= !warp_wait_all(&pv_done[p_buf(c)], p_phase(c), w);
        tc_fence_after();
        float o[16];
#pragma unroll
        for (int z = C::kPTerms - 1; z >= 0; --z) {
          uint32_t oz[16];
          tm_ld16(tO + z * R, oz);
          tm_ld16_wait(oz);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[j] = z == C::kPTerms - 1 ? __uint_as_float(oz[j]) : fmaf(o[j], C::kPTermDown, __uint_as_float(oz[j]));
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float inv_j = __shfl_sync(0xffffffffu, inv, j);
          if (j < my_rows) p.o_part[(row + j) * kCacheD + t] = o[j] * inv_j;
        }
        tc_fence_before();
        named_barrier(bar_id, 128);  // the sums have been read
      }
      c += 2;
      if (c <= c1)
        pos.cig += 2;
      else if (c < n)
        pos.skip(p.walk, 2);
      if ((sb += 2) >= C::kAhead) sb -= C::kAhead, sb_phase ^= 1u;
      if ((st += 2) >= S) st -= S, st_phase ^= 1u;
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

// One CTA per query row: the partial results of its unit (two per CTA whose slice met it)
// combined by their log-sum-exps: LSE = log sum_s e^(LSE_s), O = sum_s e^(LSE_s - LSE) O_s.
// Each of the four warps takes every fourth partial.
template <bool LIST>
__global__ void __launch_bounds__(128) merge_kernel(const AttendParams p) {
  __shared__ float so[4][kCacheD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / R, j = blockIdx.x % R;
  const UnitInfo u = unit_info<LIST>(p, unit);
  if (j >= u.rows) return;
  const long long row = u.row0 + (long long)j * u.row_step;
  grid_wait();
  grid_release();
  const WalkParams& wk = p.walk;
  const int nch = walk_chunks(wk, u.b);
  const Slices sl(wk, wk.lens ? walk_prefix(wk, wk.B) : wk.total);
  // cost position of the unit's first chunk
  const int f0 = walk_prefix(wk, u.b) + (unit - u.b * wk.units_per_b) * walk_cost(wk, nch) + wk.overhead;
  int parts = 0;
  size_t first = 0;  // partial s of the row is row (first + s * R) of the workspace
  if (nch > 0) {
    const int i0 = sl.of(f0), i1 = sl.of(f0 + nch - 1);
    parts = 2 * (i1 - i0 + 1);
    first = ((size_t)unit + i0) * 2 * R + j;
  }
  // A row of few partials is bound by latency: a warp's first two are read before their weights are
  // known. What was not written (LSE = -inf) may be anything, and is not used.
  constexpr int kFirst = 2;
  float ls0[kFirst];
  float4 v0[kFirst];
#pragma unroll
  for (int t = 0; t < kFirst; ++t) {
    const int s = warp + 4 * t;
    const size_t at = first + (size_t)(s < parts ? s : 0) * R;
    ls0[t] = p.lse_part[at];
    v0[t] = *reinterpret_cast<const float4*>(p.o_part + at * kCacheD + lane * 4);
    if (s >= parts) ls0[t] = -INFINITY;
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
  auto add = [&](float ls, const float4& v) {
    if (ls == -INFINITY) return;  // nothing seen: its O was not written
    const float wgt = ex2(ls - mm);
    acc[0] += wgt * v.x, acc[1] += wgt * v.y, acc[2] += wgt * v.z, acc[3] += wgt * v.w;
  };
#pragma unroll
  for (int t = 0; t < kFirst; ++t) add(ls0[t], v0[t]);
#pragma unroll 4
  for (int s = warp + 4 * kFirst; s < parts; s += 4) {
    const size_t at = first + (size_t)s * R;
    add(p.lse_part[at], *reinterpret_cast<const float4*>(p.o_part + at * kCacheD + lane * 4));
  }
  *reinterpret_cast<float4*>(&so[warp][lane * 4]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  const float o = so[0][threadIdx.x] + so[1][threadIdx.x] + so[2][threadIdx.x] + so[3][threadIdx.x];
  static_cast<__nv_bfloat16*>(p.o)[row * kCacheD + threadIdx.x] = __float2bfloat16(o * inv);
  if (threadIdx.x == 0) p.lse[row] = wsum == 0.f ? -INFINITY : (mm + log2f(wsum)) * 0.6931471805599453f;
}

template <bool FP8, bool LIST>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p, cudaStream_t s) {
  using C = AttCfg<FP8>;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = ensure_smem_limit(attend_kernel<FP8, LIST>, C::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  e = launch_dependent(attend_kernel<FP8, LIST>, (unsigned)p.walk.n_ctas, C::kThreads, C::kSmemBytes, s, tk, tv, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(merge_kernel<LIST>, (unsigned)(p.units * R), 128, 0, s, p);
}

}  // namespace

cudaError_t launch_cache_attend(const CUtensorMap& tk, const CUtensorMap& tv, const AttendParams& p, cudaStream_t s) {
  if (!p.fp8) return launch<false, true>(tk, tv, p, s);
  return p.idx ? launch<true, true>(tk, tv, p, s) : launch<true, false>(tk, tv, p, s);
}

}  // namespace fa
