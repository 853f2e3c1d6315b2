// fa_cache_api.cu -- C ABI of the cache operators (declared in include/fa.h): argument
// validation and launches.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "fa.h"
#include "fa_cache.h"
#include "fa_internal.h"

using namespace fa;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Size checks shared by the cache operators.
int check_cache(int B, int Hkv, int Nk, int d, int block) {
  if (B < 1 || Hkv < 1 || Nk < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (d != kCacheD) return FA_ERR_UNSUPPORTED;
  if (block != 16 && block != 32 && block != 64 && block != 128) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Hkv >= (1ll << 31) || (long long)B * Hkv * (long long)Nk >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  // the last block's end, and a tile of 128 past the last key, stay within an int
  if (Nk > 0x7FFFFFFF - 2 * kCacheTile) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// The same with queries: Hq a multiple of Hkv, rows below 2^31.
int check_queries(int B, int Hq, int Hkv, int Nq, int Nk, int d, int block) {
  if (Hq < 1 || Nq < 1) return FA_ERR_INVALID_ARG;
  int rc = check_cache(B, Hkv, Nk, d, block);
  if (rc != FA_OK) return rc;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if ((long long)B * Hq >= (1ll << 31) || (long long)B * Hq * Nq >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

bool good_scale(float scale) { return scale > 0.f && isfinite(scale); }

// Null pointers, then alignment to 16 bytes.
int check_pointers(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p) return FA_ERR_INVALID_ARG;
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

int block_log2(int block) { return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7; }

int launched(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH; }

}  // namespace

extern "C" {

int fa_cache_store(const void* k, const void* v, void* cache_k, void* cache_v, float* k_scale, float* v_scale,
                   const int* lens, int B, int Hkv, int n_new, int Nk, int d, int block, void* stream) {
  int rc = check_cache(B, Hkv, Nk, d, block);
  if (rc != FA_OK) return rc;
  if (n_new < 0) return FA_ERR_INVALID_ARG;
  if ((long long)B * Hkv * n_new >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  // tiles of 128 tokens of both tensors
  if (2ll * B * Hkv * ((Nk + kCacheTile - 1) / kCacheTile) >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (n_new == 0) return FA_OK;
  if ((rc = check_pointers({k, v, cache_k, cache_v, k_scale, v_scale})) != FA_OK) return rc;
  if (lens && !aligned(lens, 4)) return FA_ERR_ALIGNMENT;
  int* status;
  if ((rc = device_status_word(&status)) != FA_OK) return rc;
  const StoreParams p{k, v, cache_k, cache_v, k_scale, v_scale, lens, B, Hkv, n_new, Nk, block};
  return launched(launch_cache_store(p, static_cast<cudaStream_t>(stream)));
}

int fa_block_bounds(const void* k, void* bounds, const int* lens, int fp8, int B, int Hkv, int Nk, int d, int block,
                    int n_new, void* stream) {
  int rc = check_cache(B, Hkv, Nk, d, block);
  if (rc != FA_OK) return rc;
  if (n_new < 0) return FA_ERR_INVALID_ARG;
  if ((rc = check_pointers({k, bounds})) != FA_OK) return rc;
  if (lens && !aligned(lens, 4)) return FA_ERR_ALIGNMENT;
  int* status;
  if ((rc = device_status_word(&status)) != FA_OK) return rc;
  const BoundsParams p{k, bounds, lens, fp8 ? 1 : 0, B, Hkv, Nk, block, n_new};
  return launched(launch_block_bounds(p, static_cast<cudaStream_t>(stream)));
}

static int check_select(int B, int Hq, int Hkv, int Nq, int Nk, int d, int block) {
  int rc = check_queries(B, Hq, Hkv, Nq, Nk, d, block);
  if (rc != FA_OK) return rc;
  // one score per (unit, block of the cache), in tiles of 32 blocks or more
  const long long units = (long long)B * Hkv * Nq, n_blocks = (Nk + block - 1) / block;
  if (units * ((n_blocks + 31) / 32) >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

size_t fa_select_blocks_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d, int block) {
  if (check_select(B, Hq, Hkv, Nq, Nk, d, block) != FA_OK) return 0;
  return (size_t)B * Hkv * Nq * ((Nk + block - 1) / block) * sizeof(unsigned long long);
}

int fa_select_blocks(const void* q, const void* bounds, const float* k_scale, int* idx, void* workspace,
                     const int* lens, int fp8, int B, int Hq, int Hkv, int Nq, int Nk, int d, int block,
                     int n_select, int n_first, int n_last, int causal, void* stream) {
  int rc = check_select(B, Hq, Hkv, Nq, Nk, d, block);
  if (rc != FA_OK) return rc;
  if (n_select < 1 || n_first < 0 || n_last < 0 || (long long)n_first + n_last > n_select) return FA_ERR_INVALID_ARG;
  if ((long long)B * Hkv * Nq * n_select >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if ((rc = check_pointers({q, bounds, idx})) != FA_OK) return rc;
  if (!workspace) return FA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGNMENT;
  if (fp8 && !k_scale) return FA_ERR_INVALID_ARG;
  if ((lens && !aligned(lens, 4)) || (fp8 && !aligned(k_scale, 16))) return FA_ERR_ALIGNMENT;
  int* status;
  if ((rc = device_status_word(&status)) != FA_OK) return rc;
  const SelectParams p{q,  bounds, fp8 ? k_scale : nullptr, idx, static_cast<unsigned long long*>(workspace), lens,
                       fp8 ? 1 : 0, causal ? 1 : 0, B, Hq, Hkv, Nq, Nk, block, n_select, n_first, n_last};
  return launched(launch_select_blocks(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Work split of the attention calls. A unit is a group's query rows (dense: all (Hq / Hkv) *
// Nq of them; listed blocks: one query's Hq / Hkv), cut into units of at most 16 rows;
// a larger group reads its keys once per unit (mostly from L2). All units'
// chunks are cut into n_ctas slices: automatic, one per SM of a 148-SM part (a rule
// of the sizes alone, so that the workspace can be sized without a device), else
// units * num_splits; never more than the chunks of a full cache.
struct AttendSplit {
  int n_rb, units_per_b, chunks, units, n_ctas, total;
  size_t o_bytes() const {
    return (size_t)(units + n_ctas) * 2 * kUnitRows * kCacheD * sizeof(float);
  }
  size_t bytes() const { return o_bytes() + (size_t)(units + n_ctas) * 2 * kUnitRows * sizeof(float); }
};

constexpr int kAttendSms = 148;
// A unit's fixed cost in chunks of 128 keys, and of 256 for the weights. Measured for attention with
// lengths from 1 to 8192, 2 to 8: 109, 96, 94 (4), 83 (6), 82 us (8); from 1 to 16384: 64.5 to 60.7 us; equal lengths do not care.
constexpr int kAttendOverhead = 6, kWeightsOverhead = 1;

// n_select = 0: the whole cache. Returns FA_OK or the code to return.
int attend_split(int B, int Hq, int Hkv, int Nq, int Nk, int d, int block, int n_select, int num_splits,
                 AttendSplit* sp) {
  int rc = check_queries(B, Hq, Hkv, Nq, Nk, d, block);
  if (rc != FA_OK) return rc;
  const long long g = Hq / Hkv;
  const long long rows = n_select ? g : g * Nq;
  const long long per_chunk = kCacheTile / block;
  const long long chunks = n_select ? (n_select + per_chunk - 1) / per_chunk : (Nk + kCacheTile - 1) / kCacheTile;
  const long long n_rb = (rows + kUnitRows - 1) / kUnitRows;
  const long long units_per_b = (n_select ? (long long)Hkv * Nq : Hkv) * n_rb;
  const long long units = units_per_b * B, chunks_all = units * chunks, total = units * (chunks + kAttendOverhead);
  // one merge CTA per unit and row; chunks are counted in an int, and so is the distance of two heads' rows
  if (n_select && Nq >= (1 << 24)) return FA_ERR_UNSUPPORTED;
  if (n_select && (long long)B * Hkv * Nq * n_select >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (units * kUnitRows >= (1ll << 31) || total >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  sp->n_rb = (int)n_rb, sp->units_per_b = (int)units_per_b, sp->units = (int)units;
  sp->chunks = (int)chunks, sp->total = (int)total;
  const long long want = num_splits > 0 ? units * num_splits : kAttendSms;
  sp->n_ctas = (int)std::min(want, chunks_all);
  if ((long long)sp->units + sp->n_ctas >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int attend(const void* q, const void* k, const void* v, const float* k_scale, const float* v_scale, const int* idx,
           void* o, float* lse, void* workspace, const int* lens, int fp8, int B, int Hq, int Hkv, int Nq, int Nk,
           int d, int block, int n_select, int causal, float scale, int num_splits, void* stream) {
  AttendSplit sp;
  int rc = attend_split(B, Hq, Hkv, Nq, Nk, d, block, n_select, num_splits, &sp);
  if (rc != FA_OK) return rc;
  if (!good_scale(scale)) return FA_ERR_INVALID_ARG;
  if ((rc = check_pointers({q, k, v, o, lse})) != FA_OK) return rc;
  if (!workspace) return FA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGNMENT;
  if (fp8 && (!k_scale || !v_scale)) return FA_ERR_INVALID_ARG;
  if (fp8 && (!aligned(k_scale, 16) || !aligned(v_scale, 16))) return FA_ERR_ALIGNMENT;
  if ((lens && !aligned(lens, 4)) || (idx && !aligned(idx, 16))) return FA_ERR_ALIGNMENT;
  AttendParams p;
  if ((rc = device_status_word(&p.status)) != FA_OK) return rc;
  CUtensorMap tk, tv;
  const int box = n_select ? block : kCacheTile;
  if ((rc = make_tile_map(&tk, k, d, Nk, B * Hkv, box, fp8 != 0)) != FA_OK) return rc;
  if ((rc = make_tile_map(&tv, v, d, Nk, B * Hkv, box, fp8 != 0)) != FA_OK) return rc;
  p.q = q;
  p.ks = fp8 ? k_scale : nullptr, p.vs = fp8 ? v_scale : nullptr;
  p.idx = idx, p.lens = lens;
  p.o = o, p.lse = lse;
  p.fp8 = fp8 ? 1 : 0, p.causal = causal ? 1 : 0;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.Nq = Nq, p.Nk = Nk, p.block = block, p.n_select = n_select;
  p.block_log2 = block_log2(block);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.walk = WalkParams{n_select ? nullptr : lens, B, Nk, sp.units_per_b, sp.chunks, kAttendOverhead, sp.total,
                      sp.n_ctas, 7};
  p.n_rb = sp.n_rb, p.units = sp.units;
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + sp.o_bytes());
  p.wait_budget_ns = wait_budget_ns();
  return launched(launch_cache_attend(tk, tv, p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t fa_decode_fp8_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d, int block, int num_splits) {
  AttendSplit sp;
  return attend_split(B, Hq, Hkv, Nq, Nk, d, block, 0, num_splits, &sp) == FA_OK ? sp.bytes() : 0;
}

int fa_decode_fp8(const void* q, const void* k, const void* v, const float* k_scale, const float* v_scale, void* o,
                  float* lse, void* workspace, const int* lens, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                  int block, int causal, float scale, int num_splits, void* stream) {
  return attend(q, k, v, k_scale, v_scale, nullptr, o, lse, workspace, lens, 1, B, Hq, Hkv, Nq, Nk, d, block, 0,
                causal, scale, num_splits, stream);
}

size_t fa_decode_blocks_workspace_bytes(int fp8, int B, int Hq, int Hkv, int Nq, int Nk, int d, int block,
                                        int n_select, int num_splits) {
  (void)fp8;  // the partial results do not depend on the cache's type
  AttendSplit sp;
  if (n_select < 1) return 0;
  return attend_split(B, Hq, Hkv, Nq, Nk, d, block, n_select, num_splits, &sp) == FA_OK ? sp.bytes() : 0;
}

int fa_decode_blocks(const void* q, const void* k, const void* v, const float* k_scale, const float* v_scale,
                     const int* idx, void* o, float* lse, void* workspace, const int* lens, int fp8, int B, int Hq,
                     int Hkv, int Nq, int Nk, int d, int block, int n_select, int causal, float scale,
                     int num_splits, void* stream) {
  if (n_select < 1 || !idx) return FA_ERR_INVALID_ARG;
  return attend(q, k, v, k_scale, v_scale, idx, o, lse, workspace, lens, fp8, B, Hq, Hkv, Nq, Nk, d, block, n_select,
                causal, scale, num_splits, stream);
}

int fa_cache_weights(const void* q, const void* k, const float* k_scale, const float* lse, float* acc,
                     const int* lens, int fp8, int B, int Hq, int Hkv, int Nq, int Nk, int d, int block, int causal,
                     float scale, void* stream) {
  int rc = check_queries(B, Hq, Hkv, Nq, Nk, d, block);
  if (rc != FA_OK) return rc;
  if (!good_scale(scale)) return FA_ERR_INVALID_ARG;
  if ((rc = check_pointers({q, k, lse, acc})) != FA_OK) return rc;
  if (fp8 && !k_scale) return FA_ERR_INVALID_ARG;
  if ((fp8 && !aligned(k_scale, 16)) || (lens && !aligned(lens, 4))) return FA_ERR_ALIGNMENT;
  WeightsParams p;
  if ((rc = device_status_word(&p.status)) != FA_OK) return rc;
  p.q = q, p.k = k, p.ks = fp8 ? k_scale : nullptr, p.lse = lse, p.acc = acc, p.lens = lens;
  p.fp8 = fp8 ? 1 : 0, p.causal = causal ? 1 : 0;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.Nq = Nq, p.Nk = Nk, p.block = block, p.block_log2 = block_log2(block);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_budget_ns = wait_budget_ns();
  const long long rows = (long long)(Hq / Hkv) * Nq;
  const bool stream_keys = rows <= kWeightsStreamRows;
  const int chunks = (Nk + kWeightsChunk - 1) / kWeightsChunk;
  const long long units = (long long)B * Hkv, total = units * (chunks + kWeightsOverhead);
  if (stream_keys && total >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  p.walk = WalkParams{lens, B, Nk, Hkv, chunks, kWeightsOverhead, (int)total,
                      (int)std::min<long long>(units * chunks, kAttendSms), 8};
  CUtensorMap tk, tq;
  if ((rc = make_tile_map(&tk, k, d, Nk, B * Hkv, stream_keys ? kWeightsChunk : kCacheTile, fp8 != 0)) != FA_OK)
    return rc;
  // one [rows, d] tensor of all query rows: a group's rows lie together
  if ((rc = make_tile_map(&tq, q, d, B * Hq * Nq, 1, kWeightsRowTile, false)) != FA_OK) return rc;
  return launched(launch_cache_weights(tk, tq, p, static_cast<cudaStream_t>(stream)));
}

int fa_cache_evict(const void* k, const void* v, const float* k_scale, const float* v_scale, const float* acc,
                   const int* lens, void* out_k, void* out_v, float* out_k_scale, float* out_v_scale, float* out_acc,
                   int* idx, int* out_lens, int fp8, int B, int Hkv, int Nk, int d, int block, int keep, int recent,
                   int out_Nk, void* stream) {
  int rc = check_cache(B, Hkv, Nk, d, block);
  if (rc != FA_OK) return rc;
  if (keep < 1 || recent < 0 || recent > keep || out_Nk < std::min(keep, Nk)) return FA_ERR_INVALID_ARG;
  if ((long long)B * Hkv * keep >= (1ll << 31) || (rc = check_cache(B, Hkv, out_Nk, d, block)) != FA_OK)
    return rc != FA_OK ? rc : FA_ERR_UNSUPPORTED;
  if ((rc = check_pointers({k, v, acc, out_k, out_v, out_acc, idx})) != FA_OK) return rc;
  if (!out_lens) return FA_ERR_INVALID_ARG;
  if (!aligned(out_lens, 4) || (lens && !aligned(lens, 4))) return FA_ERR_ALIGNMENT;
  if (fp8 && (rc = check_pointers({k_scale, v_scale, out_k_scale, out_v_scale})) != FA_OK) return rc;
  int* status;
  if ((rc = device_status_word(&status)) != FA_OK) return rc;
  const EvictParams p{k,  v,  k_scale, v_scale, acc, lens, out_k, out_v, out_k_scale, out_v_scale, out_acc,
                      idx, out_lens, fp8 ? 1 : 0, B, Hkv, Nk, block, keep, recent, out_Nk};
  return launched(launch_cache_evict(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
