// C ABI of the decode attention library: argument checks, workspace layout,
// plan construction and kernel launches.  Allocates nothing; synchronises the
// host only in the two documented read-back calls.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "append.cuh"
#include "common.cuh"
#include "merge.cuh"
#include "moves.cuh"
#include "tree.cuh"

namespace da {
bool mla_supported(int H_q);
}

namespace {

using namespace da;

struct Variant {
  int id, tile, min_tps, max_splits;
};

struct WsLayout {
  size_t n_splits, split_begin, work, item_desc, lse_part, o_part, total;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int check_problem(const da_problem* p) {
  if (!p) return DA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1) return DA_ERR_INVALID_ARG;
  if (p->num_q_heads % p->num_kv_heads) return DA_ERR_INVALID_ARG;
  if (p->head_dim_qk < 1 || p->head_dim_v < 1) return DA_ERR_INVALID_ARG;
  if (p->layout < DA_KV_CONTIGUOUS || p->layout > DA_KV_INDEXED) return DA_ERR_INVALID_ARG;
  if (p->layout == DA_KV_PAGED && p->page_size < 1) return DA_ERR_INVALID_ARG;
  if (p->width < 0) return DA_ERR_INVALID_ARG;
  if (p->layout != DA_KV_CONTIGUOUS && p->num_blocks < 0) return DA_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return DA_ERR_INVALID_ARG;
  if ((p->flags & ~DA_FLAG_TEST_STALL) != 0) return DA_ERR_INVALID_ARG;
  if (p->shared_latent != 0 && p->shared_latent != 1) return DA_ERR_INVALID_ARG;
  if (p->shared_latent && p->head_dim_v > p->head_dim_qk) return DA_ERR_INVALID_ARG;
  if (p->extra_width < 0 || p->extra_num_blocks < 0) return DA_ERR_INVALID_ARG;
  if (row_capacity(p->layout, p->width, p->page_size) + p->extra_width > 0x7fffffffLL)
    return DA_ERR_INVALID_ARG;
  if (p->kv_dtype != DA_KV_BF16 && p->kv_dtype != DA_KV_FP8_E4M3 && p->kv_dtype != DA_KV_NVFP4)
    return DA_ERR_INVALID_ARG;
  if (p->kv_dtype != DA_KV_BF16 &&
      !(std::isfinite(p->k_scale) && p->k_scale > 0.f && std::isfinite(p->v_scale) &&
        p->v_scale > 0.f))
    return DA_ERR_INVALID_ARG;
  return DA_OK;
}

// The kernel variant follows from the head configuration alone -- never from
// the batch size or the lengths.
int select_variant(const da_problem* p, Variant* v) {
  // quantized caches: one KV source; a shared latent cache in E4M3 only
  if (p->kv_dtype != DA_KV_BF16 &&
      (p->extra_width > 0 || (p->shared_latent && p->kv_dtype != DA_KV_FP8_E4M3)))
    return DA_ERR_UNSUPPORTED;
  if (p->shared_latent) {
    if (p->head_dim_qk == 576 && p->head_dim_v == 512 && p->num_kv_heads == 1 &&
        mla_supported(p->num_q_heads)) {
      *v = {DA_VARIANT_MLA, kMlaTile, kMlaMinTilesPerSplit, kMlaMaxSplits};
      return DA_OK;
    }
    return DA_ERR_UNSUPPORTED;
  }
  const int G = p->num_q_heads / p->num_kv_heads;
  // groups of at least 16 heads over a bf16, E4M3 or NVFP4 cache (NVFP4: an
  // even number of KV heads) with one source: the multi-head contractions go
  // to the tensor cores
  const bool tc_cache = p->kv_dtype == DA_KV_BF16 || p->kv_dtype == DA_KV_FP8_E4M3 ||
                        (p->kv_dtype == DA_KV_NVFP4 && p->num_kv_heads % 2 == 0);
  if (p->head_dim_qk == p->head_dim_v && tc_cache && p->extra_width == 0 &&
      gqa_tc_supported(G, p->head_dim_qk)) {
    *v = {DA_VARIANT_GQA_TC, kTcTile, kTcMinTilesPerSplit, kTcMaxSplits};
    return DA_OK;
  }
  if (p->head_dim_qk == p->head_dim_v && fma_supported(G, p->head_dim_qk)) {
    *v = {DA_VARIANT_FMA, kFmaTile, kFmaMinTilesPerSplit, kFmaMaxSplits};
    return DA_OK;
  }
  return DA_ERR_UNSUPPORTED;
}

bool layout_fits(const da_problem* p, int max_splits) {
  // work-list entries b * max_splits + s must fit in int32
  return (long long)p->batch * (max_splits + 1) < 0x7fffffffLL;
}

WsLayout ws_layout(const da_problem* p, int max_splits) {
  const size_t B = (size_t)p->batch, ms = (size_t)max_splits;
  const size_t Hq = (size_t)p->num_q_heads, Dv = (size_t)p->head_dim_v;
  WsLayout L;
  size_t off = kHdrBytes;
  L.n_splits = off;
  off = align256(off + 4 * B);
  L.split_begin = off;
  off = align256(off + 4 * B * (ms + 1));
  L.work = off;
  off = align256(off + 4 * B * ms);
  L.item_desc = off;
  off = align256(off + 16 * B * ms);
  L.lse_part = off;
  off = align256(off + 4 * B * ms * Hq);
  L.o_part = off;
  off = align256(off + 4 * B * ms * Hq * Dv);
  L.total = off;
  return L;
}

int sm_count(int dev) {
  static std::mutex mu;
  static int cache[64] = {0};
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 0 || dev >= 64) return 0;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cache[dev] = n;
  }
  return cache[dev];
}

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

Launch make_launch(const da_plan* plan) {
  const da_problem& pr = plan->prob;
  uint8_t* ws = static_cast<uint8_t*>(plan->ws);
  Launch L;
  std::memset(&L, 0, sizeof(L));
  L.hdr = reinterpret_cast<int32_t*>(ws);
  L.n_splits = reinterpret_cast<const int32_t*>(ws + plan->off_n_splits);
  L.split_begin = reinterpret_cast<const int32_t*>(ws + plan->off_split_begin);
  L.work = reinterpret_cast<const int32_t*>(ws + plan->off_work);
  L.item_desc = reinterpret_cast<const int32_t*>(ws + plan->off_item_desc);
  L.lse_part = reinterpret_cast<float*>(ws + plan->off_lse_part);
  L.o_part = reinterpret_cast<float*>(ws + plan->off_o_part);
  L.num_blocks = pr.num_blocks;
  L.B = pr.batch;
  L.H_q = pr.num_q_heads;
  L.H_kv = pr.num_kv_heads;
  L.D_qk = pr.head_dim_qk;
  L.D_v = pr.head_dim_v;
  L.layout = pr.layout;
  L.page_size = pr.page_size;
  L.width = pr.width;
  L.capacity = (int)row_capacity(pr.layout, pr.width, pr.page_size);
  L.page_shift = -1;
  if (pr.layout == DA_KV_PAGED && pr.page_size > 0 && (pr.page_size & (pr.page_size - 1)) == 0) {
    int sh = 0;
    while ((1 << sh) < pr.page_size) ++sh;
    L.page_shift = sh;
  }
  L.max_splits = plan->max_splits;
  L.o_part_mla = plan->variant == DA_VARIANT_MLA;
  L.test_stall = (pr.flags & DA_FLAG_TEST_STALL) != 0;
  L.scale_log2 = pr.scale * kLog2e;
  if (pr.kv_dtype != DA_KV_BF16) {  // scores of scaled keys: scale * k_scale
    L.kv_type = pr.kv_dtype;
    L.scale_log2 *= pr.k_scale;
    L.v_scale = pr.v_scale;
    L.kv_rows = (pr.layout == DA_KV_CONTIGUOUS) ? (long long)pr.batch * pr.width
                : (pr.layout == DA_KV_PAGED)    ? pr.num_blocks * pr.page_size
                                                : pr.num_blocks;
  }
  return L;
}

// The most splits any row of `plan` can have: under INVARIANT a row of L
// entries has ceil(tiles / tps) splits with tps >= min_tiles_per_split and
// tiles <= ceil(capacity / tile), so n <= ceil(that / min_tiles_per_split);
// BALANCED may cut any row into max_splits.
int split_bound(const da_plan* plan) {
  if (plan->policy != DA_POLICY_INVARIANT) return plan->max_splits;
  const da_problem& pr = plan->prob;
  long long cap = row_capacity(pr.layout, pr.width, pr.page_size);
  if (plan->has_extra) cap += pr.extra_width;
  const long long tiles = (cap + plan->tile_tokens - 1) / plan->tile_tokens;
  const long long n = (tiles + plan->min_tiles_per_split - 1) / plan->min_tiles_per_split;
  return (int)std::min<long long>(std::max<long long>(n, 1), plan->max_splits);
}

int check_plan(const da_plan* plan) {
  if (!plan) return DA_ERR_INVALID_ARG;
  int rc = check_problem(&plan->prob);
  if (rc != DA_OK) return rc;
  Variant v;
  rc = select_variant(&plan->prob, &v);
  if (rc != DA_OK) return rc;
  if (plan->variant != v.id || plan->max_splits != v.max_splits) return DA_ERR_INVALID_ARG;
  if (plan->prob.batch > 0) {
    if (!plan->ws || !aligned(plan->ws, 256)) return DA_ERR_WORKSPACE;
    if (plan->ws_bytes < ws_layout(&plan->prob, v.max_splits).total) return DA_ERR_WORKSPACE;
  }
  return DA_OK;
}

long long cache_rows(const da_problem& pr) {
  return (pr.layout == DA_KV_CONTIGUOUS) ? (long long)pr.batch * pr.width
         : (pr.layout == DA_KV_PAGED)    ? pr.num_blocks * pr.page_size
                                         : pr.num_blocks;
}

bool overlap(const void* a, long long a_bytes, const void* b, long long b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

int check_caches(const da_problem* prob, const da_caches* c) {
  int rc = check_problem(prob);
  if (rc != DA_OK) return rc;
  if (!c || c->n_layers < 1) return DA_ERR_INVALID_ARG;
  Variant var;  // only caches that a kernel of this library reads
  da_problem one = *prob;
  one.extra_width = 0;
  rc = select_variant(&one, &var);
  if (rc != DA_OK) return rc;

  if (!c->k || (prob->shared_latent != 0) != (c->v == nullptr)) return DA_ERR_INVALID_ARG;
  for (int i = 0; i < c->n_layers; ++i)
    if (!c->k[i] || !aligned(c->k[i], 16) || (c->v && (!c->v[i] || !aligned(c->v[i], 16))))
      return DA_ERR_INVALID_ARG;
  return DA_OK;
}

// launch(regions) for all buffers of the caches: what holds elements (NVFP4: codes),
// then, for NVFP4, the block scales; kMoveRegions buffers at a time.
template <typename F>
int for_regions(const da_problem& pr, const da_caches& c, F launch) {
  const long long elements = (long long)pr.num_kv_heads * pr.head_dim_qk;  // of an entry
  const bool nvfp4 = pr.kv_dtype == DA_KV_NVFP4;
  bool report = true;
  for (int part = 0; part < (nvfp4 ? 2 : 1); ++part) {
    const long long bytes = part             ? elements / 16
                            : nvfp4          ? elements / 2
                            : pr.kv_dtype == DA_KV_BF16 ? elements * 2
                                                        : elements;
    if (bytes > (1 << 30)) return DA_ERR_UNSUPPORTED;  // a row's own offsets take 32 bits
    const long long offset = part ? cache_rows(pr) * (elements / 2) : 0;
    MoveRegions r;
    r.n = 0;
    r.entry_bytes = (int)bytes;
    for (int i = 0; i < c.n_layers; ++i) {
      r.base[r.n++] = static_cast<uint8_t*>(c.k[i]) + offset;
      if (c.v) r.base[r.n++] = static_cast<uint8_t*>(c.v[i]) + offset;
      if (r.n + 2 <= kMoveRegions && i + 1 < c.n_layers) continue;
      if (launch(r, report) != cudaSuccess) return DA_ERR_CUDA;
      report = false;
      r.n = 0;
    }
  }
  return DA_OK;
}

// What the tree attention takes: separate K and V, D = 64 or 128, any group up to 128.
int check_tree_problem(const da_problem* prob, int32_t nodes) {
  const int rc = check_problem(prob);
  if (rc != DA_OK) return rc;
  if (nodes < 1) return DA_ERR_INVALID_ARG;
  if (nodes > DA_TREE_MAX_NODES || prob->shared_latent || prob->extra_width ||
      prob->head_dim_qk != prob->head_dim_v || (prob->head_dim_qk != 64 && prob->head_dim_qk != 128) ||
      prob->num_q_heads / prob->num_kv_heads > 128)
    return DA_ERR_UNSUPPORTED;
  const long long cap = row_capacity(prob->layout, prob->width, prob->page_size);
  if (cap > 0x7fffff00LL) return DA_ERR_UNSUPPORTED;  // entries and positions in 32 bits
  // what a copy of scattered rows counts in 32 bits: (entry, head) pairs
  if (cache_rows(*prob) > 0x7fffffffLL / prob->num_kv_heads) return DA_ERR_UNSUPPORTED;
  if ((long long)prob->batch * nodes * prob->num_q_heads > (1LL << 31)) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

// Splits that a row of the problem can have at most.
int tree_max_splits(const da_problem* prob) {
  const long long cap = row_capacity(prob->layout, prob->width, prob->page_size);
  const long long tiles = (cap + kTreeTile - 1) / kTreeTile;
  const long long n = (tiles + kTreeLeastTiles - 1) / kTreeLeastTiles;
  return (int)std::min<long long>(std::max<long long>(n, 1), kTreeMaxSplits);
}

struct TreeWs {
  size_t lse_part, total;  // the outputs' partials lie at the start
};

TreeWs tree_ws(const da_problem* prob, int32_t nodes) {
  const int splits = tree_max_splits(prob);
  const size_t rows = splits > 1 ? (size_t)prob->batch * splits * nodes * prob->num_q_heads : 0;
  TreeWs w;
  w.lse_part = align256(4 * rows * prob->head_dim_v);
  w.total = std::max<size_t>(256, w.lse_part + align256(4 * rows));
  return w;
}

}  // namespace

extern "C" {

const char* decode_attn_version(void) {
  static char buf[256];
  static std::once_flag once;
  std::call_once(once, [] {
    std::snprintf(buf, sizeof(buf),
                  "decode_attn 0.2 sm_103a; fma: tile=%d min_tiles=%d max_splits=%d; "
                  "mla: tile=%d min_tiles=%d max_splits=%d; "
                  "gqa_tc: tile=%d min_tiles=%d max_splits=%d; balanced fixed_overhead=%d",
                  kFmaTile, kFmaMinTilesPerSplit, kFmaMaxSplits, kMlaTile, kMlaMinTilesPerSplit,
                  kMlaMaxSplits, kTcTile, kTcMinTilesPerSplit, kTcMaxSplits,
                  kBalancedFixedOverhead);
  });
  return buf;
}

const char* decode_attn_status_string(int status) {
  switch (status) {
    case DA_OK: return "ok";
    case DA_ERR_INVALID_ARG: return "invalid argument";
    case DA_ERR_UNSUPPORTED: return "unsupported head configuration";
    case DA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case DA_ERR_CUDA: return "CUDA error";
    default: return "unknown status";
  }
}

int decode_attn_split_constants(const da_problem* prob, int32_t* variant, int32_t* tile_tokens,
                                int32_t* min_tiles_per_split, int32_t* max_splits) {
  int rc = check_problem(prob);
  if (rc != DA_OK) return rc;
  Variant v;
  rc = select_variant(prob, &v);
  if (rc != DA_OK) return rc;
  if (variant) *variant = v.id;
  if (tile_tokens) *tile_tokens = v.tile;
  if (min_tiles_per_split) *min_tiles_per_split = v.min_tps;
  if (max_splits) *max_splits = v.max_splits;
  return DA_OK;
}

int decode_attn_workspace_bytes(const da_problem* prob, size_t* bytes) {
  int rc = check_problem(prob);
  if (rc != DA_OK) return rc;
  if (!bytes) return DA_ERR_INVALID_ARG;
  Variant v;
  rc = select_variant(prob, &v);
  if (rc != DA_OK) return rc;
  if (!layout_fits(prob, v.max_splits)) return DA_ERR_INVALID_ARG;
  *bytes = ws_layout(prob, v.max_splits).total;
  return DA_OK;
}

static int plan_impl(const da_problem* prob, int32_t policy, const int32_t* d_lengths,
                     const int32_t* d_extra_lengths, void* d_ws, size_t ws_bytes, da_plan* plan,
                     void* stream) {
  int rc = check_problem(prob);
  if (rc != DA_OK) return rc;
  if (!plan || (policy != DA_POLICY_INVARIANT && policy != DA_POLICY_BALANCED))
    return DA_ERR_INVALID_ARG;
  Variant v;
  rc = select_variant(prob, &v);
  if (rc != DA_OK) return rc;
  if (!layout_fits(prob, v.max_splits)) return DA_ERR_INVALID_ARG;
  const WsLayout L = ws_layout(prob, v.max_splits);
  if (prob->batch > 0) {
    if (!d_lengths) return DA_ERR_INVALID_ARG;
    if (!d_ws || !aligned(d_ws, 256) || ws_bytes < L.total) return DA_ERR_WORKSPACE;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return DA_ERR_CUDA;
  // CTAs that one (row, split) item occupies: one per KV head and head chunk
  // (CUDA-core variant), one per KV head (GQA tensor-core variant) or two, one
  // per half of D_v (shared-latent tensor-core variant).
  int gc = 1, chunks = 1;
  if (v.id == DA_VARIANT_FMA)
    fma_chunk_shape(prob->num_q_heads / prob->num_kv_heads, prob->head_dim_qk, &gc, &chunks);
  const int per_item = (v.id == DA_VARIANT_MLA) ? 2 : prob->num_kv_heads * chunks;
  // persistent CTAs: as many as can be resident at once (whole pairs for the
  // shared-latent variant)
  const long long slots =
      (v.id == DA_VARIANT_MLA)      ? (long long)mla_resident_ctas(sms)
      : (v.id == DA_VARIANT_GQA_TC) ? (long long)gqa_tc_resident_ctas(sms)
                                    : (long long)sms * fma_ctas_per_sm(prob->num_q_heads /
                                                                           prob->num_kv_heads,
                                                                       prob->head_dim_qk);
  const long long max_units = (long long)prob->batch * v.max_splits * per_item;

  da_plan P;
  std::memset(&P, 0, sizeof(P));
  P.prob = *prob;
  P.policy = policy;
  P.variant = v.id;
  P.tile_tokens = v.tile;
  P.min_tiles_per_split = v.min_tps;
  P.max_splits = v.max_splits;
  P.num_parts = (int)(slots / per_item > 0 ? kBalancedPartsPerSlot * (slots / per_item) : 1);
  P.fixed_overhead = kBalancedFixedOverhead;
  P.grid = (int)(max_units < slots ? (max_units > 0 ? max_units : 1) : slots);
  P.device = dev;
  P.has_extra = d_extra_lengths != nullptr;
  P.ws = d_ws;
  P.ws_bytes = ws_bytes;
  P.off_n_splits = L.n_splits;
  P.off_split_begin = L.split_begin;
  P.off_work = L.work;
  P.off_item_desc = L.item_desc;
  P.off_lse_part = L.lse_part;
  P.off_o_part = L.o_part;
  *plan = P;
  if (prob->batch == 0) return DA_OK;

  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  PlanLaunch pl;
  pl.lengths = d_lengths;
  pl.extra_lengths = d_extra_lengths;
  pl.extra_capacity = prob->extra_width;
  pl.hdr = reinterpret_cast<int32_t*>(ws);
  pl.n_splits = reinterpret_cast<int32_t*>(ws + L.n_splits);
  pl.split_begin = reinterpret_cast<int32_t*>(ws + L.split_begin);
  pl.work = reinterpret_cast<int32_t*>(ws + L.work);
  pl.item_desc = reinterpret_cast<int32_t*>(ws + L.item_desc);
  pl.B = prob->batch;
  pl.tile = v.tile;
  pl.min_tps = v.min_tps;
  pl.max_splits = v.max_splits;
  pl.capacity = (int)row_capacity(prob->layout, prob->width, prob->page_size);
  pl.policy = policy;
  pl.num_parts = P.num_parts;
  pl.fixed_overhead = P.fixed_overhead;
  if (launch_plan(pl, static_cast<cudaStream_t>(stream)) != cudaSuccess) return DA_ERR_CUDA;
  return DA_OK;
}

int decode_attn_plan(const da_problem* prob, int32_t policy, const int32_t* d_lengths,
                     void* d_ws, size_t ws_bytes, da_plan* plan, void* stream) {
  return plan_impl(prob, policy, d_lengths, nullptr, d_ws, ws_bytes, plan, stream);
}

int decode_attn_plan_extra(const da_problem* prob, int32_t policy, const int32_t* d_lengths,
                           const int32_t* d_extra_lengths, void* d_ws, size_t ws_bytes,
                           da_plan* plan, void* stream) {
  if (!prob || prob->extra_width < 1) return DA_ERR_INVALID_ARG;
  if (prob->batch > 0 && !d_extra_lengths) return DA_ERR_INVALID_ARG;
  static const int32_t dummy = 0;  // B = 0: any non-null marker will do
  return plan_impl(prob, policy, d_lengths, prob->batch > 0 ? d_extra_lengths : &dummy, d_ws,
                   ws_bytes, plan, stream);
}

static int run_impl(const da_plan* plan, const void* q, const void* k, const void* v,
                    const int32_t* table, const int32_t* lengths, const void* extra_k,
                    const void* extra_v, const int32_t* extra_indices,
                    const int32_t* extra_lengths, void* out, float* lse, void* stream) {
  int rc = check_plan(plan);
  if (rc != DA_OK) return rc;
  const da_problem& pr = plan->prob;
  if ((extra_k != nullptr) != (plan->has_extra != 0)) return DA_ERR_INVALID_ARG;
  if (pr.batch == 0) return DA_OK;
  if (extra_k) {
    if (!extra_indices || !extra_lengths || (!pr.shared_latent && !extra_v))
      return DA_ERR_INVALID_ARG;
    if (!aligned(extra_k, 16) || (extra_v && !aligned(extra_v, 16)) ||
        !aligned(extra_indices, 4) || !aligned(extra_lengths, 4))
      return DA_ERR_INVALID_ARG;
  }
  if (!q || !k || !lengths || !out || !lse) return DA_ERR_INVALID_ARG;
  if (!pr.shared_latent && !v) return DA_ERR_INVALID_ARG;
  if (pr.layout != DA_KV_CONTIGUOUS && !table) return DA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || (v && !aligned(v, 16)) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(lengths, 4) || (table && !aligned(table, 4)))
    return DA_ERR_INVALID_ARG;
  Launch L = make_launch(plan);
  L.q = static_cast<const __nv_bfloat16*>(q);
  L.k = static_cast<const __nv_bfloat16*>(k);
  L.v = static_cast<const __nv_bfloat16*>(pr.shared_latent ? k : v);
  L.table = table;
  L.lengths = lengths;
  L.out = static_cast<__nv_bfloat16*>(out);
  L.lse = lse;
  if (extra_k) {
    L.extra_k = static_cast<const __nv_bfloat16*>(extra_k);
    L.extra_v = static_cast<const __nv_bfloat16*>(pr.shared_latent ? extra_k : extra_v);
    L.extra_table = extra_indices;
    L.extra_lengths = extra_lengths;
    L.extra_num_blocks = pr.extra_num_blocks;
    L.extra_width = pr.extra_width;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = (plan->variant == DA_VARIANT_MLA)      ? launch_split_mla(L, plan->grid, s)
                        : (plan->variant == DA_VARIANT_GQA_TC) ? launch_split_gqa_tc(L, plan->grid, s)
                                                          : launch_split_fma(L, plan->grid, s);
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int decode_attn_run(const da_plan* plan, const void* q, const void* k, const void* v,
                    const int32_t* table, const int32_t* lengths, void* out, float* lse,
                    void* stream) {
  return run_impl(plan, q, k, v, table, lengths, nullptr, nullptr, nullptr, nullptr, out, lse,
                  stream);
}

int decode_attn_run_extra(const da_plan* plan, const void* q, const void* k, const void* v,
                          const int32_t* table, const int32_t* lengths, const void* extra_k,
                          const void* extra_v, const int32_t* extra_indices,
                          const int32_t* extra_lengths, void* out, float* lse, void* stream) {
  if (!extra_k) return DA_ERR_INVALID_ARG;
  return run_impl(plan, q, k, v, table, lengths, extra_k, extra_v, extra_indices, extra_lengths,
                  out, lse, stream);
}

int decode_attn_combine(const da_plan* plan, void* out, float* lse, void* stream) {
  int rc = check_plan(plan);
  if (rc != DA_OK) return rc;
  if (plan->prob.batch == 0) return DA_OK;
  if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4)) return DA_ERR_INVALID_ARG;
  Launch L = make_launch(plan);
  L.out = static_cast<__nv_bfloat16*>(out);
  L.lse = lse;
  return launch_combine(L, split_bound(plan), static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

int decode_attn_forward(const da_problem* prob, int32_t policy, const void* q, const void* k,
                        const void* v, const int32_t* table, const int32_t* lengths,
                        void* d_ws, size_t ws_bytes, void* out, float* lse, void* stream) {
  da_plan plan;
  int rc = decode_attn_plan(prob, policy, lengths, d_ws, ws_bytes, &plan, stream);
  if (rc != DA_OK) return rc;
  rc = decode_attn_run(&plan, q, k, v, table, lengths, out, lse, stream);
  if (rc != DA_OK) return rc;
  return decode_attn_combine(&plan, out, lse, stream);
}

int decode_attn_forward_extra(const da_problem* prob, int32_t policy, const void* q,
                              const void* k, const void* v, const int32_t* table,
                              const int32_t* lengths, const void* extra_k, const void* extra_v,
                              const int32_t* extra_indices, const int32_t* extra_lengths,
                              void* d_ws, size_t ws_bytes, void* out, float* lse, void* stream) {
  da_plan plan;
  int rc = decode_attn_plan_extra(prob, policy, lengths, extra_lengths, d_ws, ws_bytes, &plan,
                                  stream);
  if (rc != DA_OK) return rc;
  rc = decode_attn_run_extra(&plan, q, k, v, table, lengths, extra_k, extra_v, extra_indices,
                             extra_lengths, out, lse, stream);
  if (rc != DA_OK) return rc;
  return decode_attn_combine(&plan, out, lse, stream);
}

int decode_attn_read_error(const da_plan* plan, int32_t* code, void* stream) {
  if (!plan || !code) return DA_ERR_INVALID_ARG;
  *code = 0;
  if (plan->prob.batch == 0) return DA_OK;
  if (!plan->ws) return DA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(code, static_cast<const int32_t*>(plan->ws) + kHdrError, sizeof(int32_t),
                      cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return DA_ERR_CUDA;
  return cudaStreamSynchronize(s) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int decode_attn_copy_plan(const da_plan* plan, int32_t* n_splits, int32_t* split_begin,
                          int32_t* n_work, int32_t* work, void* stream) {
  if (!plan) return DA_ERR_INVALID_ARG;
  const size_t B = (size_t)plan->prob.batch, ms = (size_t)plan->max_splits;
  if (B == 0) {
    if (n_work) *n_work = 0;
    return DA_OK;
  }
  if (!plan->ws) return DA_ERR_WORKSPACE;
  const uint8_t* ws = static_cast<const uint8_t*>(plan->ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (n_splits && e == cudaSuccess)
    e = cudaMemcpyAsync(n_splits, ws + plan->off_n_splits, 4 * B, cudaMemcpyDeviceToHost, s);
  if (split_begin && e == cudaSuccess)
    e = cudaMemcpyAsync(split_begin, ws + plan->off_split_begin, 4 * B * (ms + 1),
                        cudaMemcpyDeviceToHost, s);
  if (n_work && e == cudaSuccess)
    e = cudaMemcpyAsync(n_work, reinterpret_cast<const int32_t*>(ws) + kHdrNWork, 4,
                        cudaMemcpyDeviceToHost, s);
  if (work && e == cudaSuccess)
    e = cudaMemcpyAsync(work, ws + plan->off_work, 4 * B * ms, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

static int append_impl(const da_problem* prob, const da_rope* rope, const da_head_norm* norm,
                       const da_append* args, const int32_t* entries, void* stream) {
  int rc = check_problem(prob);
  if (rc != DA_OK) return rc;
  if (!args || args->n_tokens < 0) return DA_ERR_INVALID_ARG;
  if (args->x_dtype != DA_X_F32 && args->x_dtype != DA_X_BF16) return DA_ERR_INVALID_ARG;
  const bool turns = rope && rope->dim != 0;
  if (rope) {
    if (rope->dim < 0 || rope->dim % 16 || rope->offset < 0 || rope->offset % 8 ||
        rope->dim > prob->head_dim_qk - rope->offset)
      return DA_ERR_INVALID_ARG;
    if ((rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->gain))
      return DA_ERR_INVALID_ARG;
    if (turns && (!rope->inv_freq || !aligned(rope->inv_freq, 4))) return DA_ERR_INVALID_ARG;
  }
  Variant var;  // only what a kernel of this library reads can be written
  da_problem one = *prob;
  one.extra_width = 0;
  rc = select_variant(&one, &var);
  if (rc != DA_OK) return rc;
  const da_append& a = *args;
  if (a.n_tokens == 0) return DA_OK;
  const bool latent = prob->shared_latent != 0;
  const bool norms = norm && (norm->q_weight || norm->k_weight);
  if (norm) {
    if ((norm->w_dtype != DA_X_F32 && norm->w_dtype != DA_X_BF16) || !std::isfinite(norm->w_add) ||
        !std::isfinite(norm->eps) || norm->eps < 0.f)
      return DA_ERR_INVALID_ARG;
    if ((norm->q_weight && !aligned(norm->q_weight, 16)) ||
        (norm->k_weight && !aligned(norm->k_weight, 16)) || (norm->q_weight && !a.q_new))
      return DA_ERR_INVALID_ARG;
    if (norms && latent) return DA_ERR_UNSUPPORTED;
  }
  if (entries && (prob->layout == DA_KV_INDEXED || !aligned(entries, 4))) return DA_ERR_INVALID_ARG;
  const long long n = a.n_tokens, D = prob->head_dim_qk;
  const long long q_row = prob->num_q_heads * D, kv_row = prob->num_kv_heads * D;
  const long long esize = a.x_dtype == DA_X_BF16 ? 2 : 4;
  if (!a.k_new || !a.k || !a.positions || latent != (a.v_new == nullptr) ||
      (!latent && !a.v) || (a.q_new != nullptr) != (a.q_out != nullptr))
    return DA_ERR_INVALID_ARG;
  if (prob->layout == DA_KV_PAGED && !a.table) return DA_ERR_INVALID_ARG;
  if (prob->layout == DA_KV_INDEXED && !a.rows) return DA_ERR_INVALID_ARG;
  if (!a.rows && a.n_tokens > prob->batch) return DA_ERR_INVALID_ARG;
  const void* ptr16[6] = {a.k_new, a.v_new, a.q_new, a.k, a.v, a.q_out};
  for (const void* q : ptr16)
    if (q && !aligned(q, 16)) return DA_ERR_INVALID_ARG;
  if (!aligned(a.positions, 4) || (a.rows && !aligned(a.rows, 4)) ||
      (a.table && !aligned(a.table, 4)) || (a.err && !aligned(a.err, 4)))
    return DA_ERR_INVALID_ARG;
  const long long strides[3] = {a.k_stride, a.v_new ? a.v_stride : kv_row,
                                a.q_new ? a.q_stride : q_row};
  const long long least[3] = {kv_row, kv_row, q_row};
  if (q_row > (1 << 30)) return DA_ERR_UNSUPPORTED;  // a token's own offsets take 32 bits
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < least[i] || strides[i] > (1LL << 40)) return DA_ERR_INVALID_ARG;
    if (strides[i] * esize % 16) return DA_ERR_INVALID_ARG;
  }
  const void* source[3] = {a.k_new, a.v_new, a.q_new};
  for (int i = 0; i < 3 && a.q_out; ++i) {  // other threads read what q_out's threads write
    if (!source[i]) continue;
    const uintptr_t src = reinterpret_cast<uintptr_t>(source[i]);
    const uintptr_t dst = reinterpret_cast<uintptr_t>(a.q_out);
    const uintptr_t src_end = src + ((n - 1) * strides[i] + least[i]) * esize;
    if (dst < src_end && src < dst + n * q_row * 2) return DA_ERR_INVALID_ARG;
  }
  const void* read[3] = {norms ? norm->q_weight : nullptr, norms ? norm->k_weight : nullptr, entries};
  const long long weight_bytes = norms ? D * (norm->w_dtype == DA_X_BF16 ? 2 : 4) : 0;
  const long long read_bytes[3] = {weight_bytes, weight_bytes, 4 * n};
  for (int i = 0; i < 3 && a.q_out; ++i)  // (by the threads of every token)
    if (read[i] && overlap(a.q_out, n * q_row * 2, read[i], read_bytes[i])) return DA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return DA_ERR_CUDA;
  AppendLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.k_new = a.k_new;
  L.v_new = a.v_new;
  L.q_new = a.q_new;
  L.k_stride = a.k_stride;
  L.v_stride = a.v_stride;
  L.q_stride = a.q_stride;
  L.positions = a.positions;
  L.rows = a.rows;
  L.table = a.table;
  L.k = a.k;
  L.v = a.v;
  L.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  L.err = a.err;
  L.num_blocks = prob->num_blocks;
  L.capacity = row_capacity(prob->layout, prob->width, prob->page_size);
  L.kv_rows = (prob->layout == DA_KV_CONTIGUOUS) ? (long long)prob->batch * prob->width
              : (prob->layout == DA_KV_PAGED)    ? prob->num_blocks * prob->page_size
                                                 : prob->num_blocks;
  L.n_tokens = a.n_tokens;
  L.x_bf16 = a.x_dtype == DA_X_BF16;
  L.B = prob->batch;
  L.H_q = prob->num_q_heads;
  L.H_kv = prob->num_kv_heads;
  L.D = prob->head_dim_qk;
  L.layout = prob->layout;
  L.page_size = prob->page_size;
  L.width = prob->width;
  L.kv_type = prob->kv_dtype;
  L.gain = 1.f;
  if (turns) {
    L.rope_dim = rope->dim;
    L.rope_offset = rope->offset;
    L.interleaved = rope->interleaved;
    L.gain = rope->gain;
    L.inv_freq = rope->inv_freq;
  }
  L.k_scale = prob->k_scale;
  L.v_scale = prob->v_scale;
  L.entries = entries;
  if (norms) {
    L.q_weight = norm->q_weight;
    L.k_weight = norm->k_weight;
    L.w_bf16 = norm->w_dtype == DA_X_BF16;
    L.w_add = norm->w_add;
    L.eps = norm->eps;
  }
  return launch_append(L, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK
                                                                                 : DA_ERR_CUDA;
}

int decode_attn_append(const da_problem* prob, const da_rope* rope, const da_append* args,
                       void* stream) {
  return append_impl(prob, rope, nullptr, args, nullptr, stream);
}

int decode_attn_append_norm(const da_problem* prob, const da_rope* rope, const da_head_norm* norm,
                            const da_append* args, const int32_t* entries, void* stream) {
  return append_impl(prob, rope, norm, args, entries, stream);
}

int decode_attn_copy_pages(const da_problem* prob, const da_caches* caches, const int32_t* src,
                           const int32_t* dst, int32_t n, int32_t* err, void* stream) {
  const int rc = check_caches(prob, caches);
  if (rc != DA_OK) return rc;
  if (n < 0 || prob->layout == DA_KV_CONTIGUOUS) return DA_ERR_INVALID_ARG;
  if (n == 0) return DA_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4) || (err && !aligned(err, 4)))
    return DA_ERR_INVALID_ARG;
  return for_regions(*prob, *caches, [&](const MoveRegions& r, bool report) {
    CopyPagesLaunch L;
    L.regions = r;
    L.src = src;
    L.dst = dst;
    L.err = err;
    L.num_blocks = prob->num_blocks;
    L.page_bytes = (long long)r.entry_bytes * (prob->layout == DA_KV_PAGED ? prob->page_size : 1);
    L.n = n;
    L.word = L.page_bytes % 16 == 0 ? 16 : 4;
    L.report = report;
    return launch_copy_pages(L, static_cast<cudaStream_t>(stream));
  });
}

int decode_attn_compact(const da_problem* prob, const da_caches* caches, const int32_t* table,
                        const int32_t* lengths, const int32_t* nodes, int32_t nodes_width,
                        const int32_t* accepted, int32_t* new_lengths, int32_t* err, void* stream) {
  const int rc = check_caches(prob, caches);
  if (rc != DA_OK) return rc;
  if (nodes_width < 1 || nodes_width > DA_TREE_MAX_NODES) return DA_ERR_INVALID_ARG;
  if (prob->batch == 0) return DA_OK;
  if (!lengths || !nodes || !accepted || (prob->layout != DA_KV_CONTIGUOUS) != (table != nullptr))
    return DA_ERR_INVALID_ARG;
  const void* words[6] = {table, lengths, nodes, accepted, new_lengths, err};
  for (const void* w : words)
    if (w && !aligned(w, 4)) return DA_ERR_INVALID_ARG;
  const long long B = prob->batch;
  if (new_lengths && (overlap(new_lengths, 4 * B, lengths, 4 * B) ||
                      overlap(new_lengths, 4 * B, accepted, 4 * B) ||
                      overlap(new_lengths, 4 * B, nodes, 4 * B * nodes_width) ||
                      (table && overlap(new_lengths, 4 * B, table, 4 * B * prob->width))))
    return DA_ERR_INVALID_ARG;  // other threads read what it gets
  return for_regions(*prob, *caches, [&](const MoveRegions& r, bool report) {
    CompactLaunch L;
    L.regions = r;
    L.table = table;
    L.lengths = lengths;
    L.nodes = nodes;
    L.accepted = accepted;
    L.new_lengths = new_lengths;
    L.err = err;
    L.num_blocks = prob->num_blocks;
    L.capacity = row_capacity(prob->layout, prob->width, prob->page_size);
    L.B = prob->batch;
    L.nodes_width = nodes_width;
    L.layout = prob->layout;
    L.page_size = prob->page_size;
    L.width = prob->width;
    L.word = r.entry_bytes % 16 == 0 ? 16 : 4;
    L.report = report;
    return launch_compact(L, static_cast<cudaStream_t>(stream));
  });
}

int decode_attn_tree_workspace_bytes(const da_problem* prob, int32_t nodes, size_t* bytes) {
  const int rc = check_tree_problem(prob, nodes);
  if (rc != DA_OK) return rc;
  if (!bytes) return DA_ERR_INVALID_ARG;
  *bytes = tree_ws(prob, nodes).total;
  return DA_OK;
}

int decode_attn_tree(const da_problem* prob, const da_tree* args, void* stream) {
  if (!args) return DA_ERR_INVALID_ARG;
  const da_tree& a = *args;
  const int rc = check_tree_problem(prob, a.nodes);
  if (rc != DA_OK) return rc;
  if (a.window < 0 || a.sinks < 0) return DA_ERR_INVALID_ARG;
  if (prob->batch == 0) return DA_OK;
  if (!a.q || !a.k || !a.v || !a.lengths || !a.out || !a.lse ||
      (prob->layout != DA_KV_CONTIGUOUS) != (a.table != nullptr))
    return DA_ERR_INVALID_ARG;
  const void* wide[4] = {a.q, a.k, a.v, a.out};
  for (const void* w : wide)
    if (!aligned(w, 16)) return DA_ERR_INVALID_ARG;
  const void* words[6] = {a.lengths, a.lse, a.table, a.parents, a.counts, a.err};
  for (const void* w : words)
    if (!aligned(w, 4)) return DA_ERR_INVALID_ARG;
  const TreeWs ws = tree_ws(prob, a.nodes);
  if (!a.ws || !aligned(a.ws, 256) || a.ws_bytes < ws.total) return DA_ERR_WORKSPACE;
  const long long rows = (long long)prob->batch * a.nodes * prob->num_q_heads;
  const long long out_bytes = rows * prob->head_dim_v * 2;
  // units of work read all of a row's queries, its entries and sizes, and write partials, at any time
  const long long elements = cache_rows(*prob) * prob->num_kv_heads * prob->head_dim_qk;
  const long long cache_bytes = prob->kv_dtype == DA_KV_BF16       ? elements * 2
                                : prob->kv_dtype == DA_KV_FP8_E4M3 ? elements
                                                                   : elements / 2 + elements / 16;
  const long long B = prob->batch;
  const void* used[8] = {a.q, a.k, a.v, a.lengths, a.counts, a.parents, a.table, a.ws};
  const long long used_bytes[8] = {out_bytes, cache_bytes, cache_bytes, 4 * B, 4 * B, 4 * B * a.nodes, 4 * B * prob->width,
                                   (long long)ws.total};
  for (int i = 0; i < 8; ++i)
    if (used[i] && (overlap(a.out, out_bytes, used[i], used_bytes[i]) || overlap(a.lse, rows * 4, used[i], used_bytes[i])))
      return DA_ERR_INVALID_ARG;
  if (overlap(a.out, out_bytes, a.lse, rows * 4)) return DA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return DA_ERR_CUDA;
  TreeLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.q = static_cast<const __nv_bfloat16*>(a.q);
  L.k = a.k;
  L.v = a.v;
  L.table = a.table;
  L.lengths = a.lengths;
  L.counts = a.counts;
  L.parents = a.parents;
  L.out = static_cast<__nv_bfloat16*>(a.out);
  L.lse = a.lse;
  L.err = a.err;
  L.o_part = static_cast<float*>(a.ws);
  L.lse_part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + ws.lse_part);
  L.num_blocks = prob->num_blocks;
  L.kv_rows = cache_rows(*prob);
  L.B = prob->batch;
  L.T = a.nodes;
  L.H_q = prob->num_q_heads;
  L.H_kv = prob->num_kv_heads;
  L.G = L.H_q / L.H_kv;
  L.D = prob->head_dim_qk;
  L.layout = prob->layout;
  L.page_size = prob->page_size;
  L.width = prob->width;
  L.capacity = (int)row_capacity(prob->layout, prob->width, prob->page_size);
  L.kv_type = prob->kv_dtype;
  // (a window that reaches over everything is none)
  L.window = (long long)a.window >= (long long)L.capacity + DA_TREE_MAX_NODES ? 0 : a.window;
  L.sinks = a.sinks;
  L.max_splits = tree_max_splits(prob);
  L.scale_log2 = prob->scale * kLog2e;
  L.v_scale = 1.f;
  if (prob->kv_dtype != DA_KV_BF16) {
    L.scale_log2 *= prob->k_scale;
    L.v_scale = prob->v_scale;
  }
  L.test_stall = (prob->flags & DA_FLAG_TEST_STALL) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_tree(L, sms, s);
  if (e == cudaSuccess && L.max_splits > 1) e = launch_tree_combine(L, s);
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
