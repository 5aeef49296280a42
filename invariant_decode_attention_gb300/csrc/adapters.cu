// Low-rank adapters of many requests beside a shared weight matmul:
//     t[i, :] = bf16(x[i, :]) A_id^T,   out[i, :] = y[i, :] + (scale_id t[i, :]) B_id^T
// with each row's own id, every row's bits independent of the batch.
//
// Three parts:
//   plan  groups the rows of a window of 512 by adapter and cuts the groups into
//         tiles of at most 64 rows (the columns of the matrix products).  Prompts,
//         whose rows come in runs, give full tiles; a decode step's scattered rows
//         meet their adapter's others anywhere in the window, so an adapter's
//         weights are read once per 64 rows of a window that use it.  (Groups do not
//         go beyond a window: 8192 rows that use 64 adapters in no order make 1024
//         tiles of eight rows and take 540 us, in runs 161.)  A kernel of its own; with
//         one window both matmul kernels make the plan for themselves instead.
//   down  t: D[rank, member] += A[rank, k] x[member, k] on the tensor cores
//         (tcgen05, M = 128 of which the adapter's ranks count, N = 64, fp32 in
//         tensor memory).  K is cut into the chunks of nvfp4_mm (1024), each summed
//         from zero by two issuing threads in turn; a unit of work is a tile and a chunk.
//   up    out: D[feature, member] += B[feature, r] t[member, r], M = 128 features,
//         N = 64.  The chunk sums of t are added in order, scaled, and split into
//         three bf16 terms that hold their 24 bits; their products with B are
//         exact, so out keeps fp32 accuracy (the tensor cores' accumulation of both
//         products leaves an error of 5e-7 of a result's usual size at K = 4096; a
//         library's fp32 products 1.6e-7).  A unit is a tile and 128 features.
//         y arrives in shared memory, 16 rows at a time; the epilogue adds the
//         products to it there and writes whole 128-byte lines, 16 bytes a lane
//         (loads and stores of 4 bytes a lane took 4900 instructions a unit of 32
//         rows and 267 us for 8192 rows of 8192, bulk copies of 512 bytes 200 us, y
//         in registers a quarter ahead 220 us).
// The orders of all sums depend on K and the rank alone.  A column of an MMA does
// not depend on the other columns, so neither do a row's bits.
//
// Both matmul kernels are persistent with one CTA per SM and run the same roles:
// producer warps bring operands into a ring of stages with 16-byte cp.async (rows
// may lie anywhere, and a copy may end inside 16 bytes, zeros beyond: what memory
// holds past an adapter's rank is never multiplied) in the 128-byte-swizzled
// K-major layout, whose landing arrives on the stage's barrier by itself; two
// threads issue the MMAs (one alone took 80 cycles an MMA and set the pace);
// epilogue warps drain accumulators.  Every wait is bounded; on
// time-out the kernel records DA_DEVERR_TIMEOUT, all roles leave their loops,
// copies and tensor-core work are drained and tensor memory is freed.
//
// A parity tells a phase of a barrier from the one before it only, so every waiter
// goes through all phases of the barriers it waits on, in order: a stage, a slot or
// an accumulator has one issuer and one epilogue group; what both issuers release has
// a barrier of each.
//
// y and out (8 N bytes a row) bound a prompt, the adapters' weights and launch
// latency a decode step.  Measured, 4096 -> 8192 features: 8192 rows of rank 64 with
// the bf16 copy 166 us (plan 8, down 27, up 132: 5.1 TB/s, 0.75 of a plain copy's
// rate, hand-offs between roles set the pace); 67 rows with 24 adapters 29.2 us; one
// row 13.1 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cstring>

#include "common.cuh"
#include "nvfp4_mm.h"
#include "tcgen05.cuh"

namespace da {
namespace {

constexpr int kTile = 64;                  // rows per tile (MMA N)
constexpr int kWindow = 512;               // rows that are grouped together
constexpr int kLines = kWindow / 32;
constexpr int kSlab = 512 * kWindow;       // rows of one set of launches
constexpr int kMaxRank = NVFP4_ADAPTER_MAX_RANK;
constexpr int kKChunk = NVFP4_MM_K_CHUNK;  // 1024: K summed from zero
constexpr int kFeat = NVFP4_MM_TILE_N;     // features per unit (MMA M)
constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kIdesc = umma::idesc_bf16_f32(128, kTile, false);

struct Args {
  const void* x;
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const int32_t* ranks;
  const float* scales;
  const int32_t* ids;
  const float* y;
  float* out;
  __nv_bfloat16* out_bf16;
  int32_t* hdr;
  // the plan, window w's tiles from slot 512 w on (several windows)
  int32_t* tiles_in;    // [windows] tiles of a window
  int32_t* tile_id;     // adapter, or -1: rows that are only copied
  int32_t* tile_count;  // members
  int32_t* tile_first;  // ... from here on in
  int32_t* order;       // [rows] the rows, tile by tile
  float* t;             // [chunks][n][max_rank]
  int n, N, K, n_adapters, max_rank, n_chunks, windows;
  int copy;             // 1: rows without an adapter are written as well
  int first;            // 1: the call's first slab
  // time-out test hook: the first stage (1: of down, 2: of up) never gets full
  int stall;
  unsigned long long limit_ns;  // of a wait
};

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 16 bytes of which the first `bytes` are copied and the others are zero.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

__device__ __forceinline__ int rank_of(const Args& g, int id) {
  return g.ranks ? clamp_len(__ldg(g.ranks + id), g.max_rank) : g.max_rank;
}

// ---------------------------------------------------------------- plan

// The plan of one window, and what making it takes.
struct Window {
  int tile_id[kWindow], tile_count[kWindow], tile_first[kWindow], order[kWindow];
  __align__(16) int id[kWindow];
  int pos[kWindow], leader[kWindow], before[kLines + 1];
};

// What the plan takes row i for: its adapter, -1 for a row that is only copied, -2
// for one that nothing is done for.  *bad gets the error bits.
__device__ __forceinline__ int planned_id(const Args& g, int i, int* bad) {
  const int v = __ldg(g.ids + i);
  int rank = 0;
  if (v >= g.n_adapters) {
    *bad |= DA_DEVERR_INDEX;
  } else if (v >= 0) {
    rank = rank_of(g, v);
    if (g.ranks && __ldg(g.ranks + v) != rank) *bad |= DA_DEVERR_LENGTH;
  }
  return rank ? v : g.copy ? -1 : -2;
}

// Rows r0 .. r0 + count - 1, by all threads of the CTA; returns the tiles.  *bad gets
// the error bits of the rows that this thread has looked at.
__device__ int make_plan(const Args& g, int r0, int count, Window& s, int* bad) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (count <= 32) {  // a decode step: one warp, a row a lane, without the barriers below
    if (warp == 0) {
      const int v = lane < count ? planned_id(g, r0 + lane, bad) : -2;
      const unsigned peers = __match_any_sync(kFull, v), lower = (1u << lane) - 1u;
      const bool lead = v != -2 && !(peers & lower);
      const unsigned leads = __ballot_sync(kFull, lead);
      const int size = lead ? __popc(peers) : 0;  // a group is one tile
      int sum = size;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += u;
      }
      const int first = __shfl_sync(kFull, sum - size, __ffs(peers) - 1);  // the group's
      if (lead) {
        const int t = __popc(leads & lower);
        s.tile_id[t] = v;
        s.tile_count[t] = size;
        s.tile_first[t] = first;
      }
      if (v != -2) s.order[first + __popc(peers & lower)] = r0 + lane;
      if (lane == 0) s.before[kLines] = __popc(leads);
    }
    __syncthreads();
    return s.before[kLines];
  }
  for (int i = threadIdx.x; i < kWindow; i += blockDim.x)
    s.id[i] = i < count ? planned_id(g, r0 + i, bad) : -2;
  __syncthreads();
  for (int line = warp; line < kLines; line += warps) {
    const int i = line * 32 + lane, v = s.id[i];
    unsigned leads = 0;
    if (line * 32 < count) {
      // a row's place among the rows of its group: those of earlier lines, then of
      // its own; every kTile-th row leads a tile
      int p = 0;
#pragma unroll 8
      for (int j = 0; j < line * 32; j += 4) {
        const int4 o = *reinterpret_cast<const int4*>(s.id + j);
        p += (o.x == v) + (o.y == v) + (o.z == v) + (o.w == v);
      }
      p += __popc(__match_any_sync(kFull, v) & ((1u << lane) - 1u));
      s.pos[i] = p;
      leads = __ballot_sync(kFull, v != -2 && p % kTile == 0);
    }
    if (lane == 0) s.before[line + 1] = __popc(leads);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s.before[0] = 0;
    for (int l = 1; l <= kLines; ++l) s.before[l] += s.before[l - 1];
  }
  __syncthreads();
  for (int line = warp; line * 32 < count; line += warps) {  // tiles are numbered in row order
    const int i = line * 32 + lane;
    const bool lead = s.id[i] != -2 && s.pos[i] % kTile == 0;
    const unsigned leads = __ballot_sync(kFull, lead);
    if (lead) s.leader[s.before[line] + __popc(leads & ((1u << lane) - 1u))] = i;
  }
  __syncthreads();
  const int tiles = s.before[kLines];
  // the members of tile t are the rows of its leader's group from the leader's place
  // on; first they are counted, then listed
  auto members = [&](int t, int line, int* q) {
    const int lead = s.leader[t], r = line * 32 + lane;
    *q = s.pos[r] - s.pos[lead];
    return r < count && s.id[r] == s.id[lead] && *q >= 0 && *q < kTile;
  };
  for (int t = warp; t < tiles; t += warps) {  // a warp per tile
    int found = 0, q;
    for (int line = s.leader[t] >> 5; line * 32 < count && found < kTile; ++line)
      found += __popc(__ballot_sync(kFull, members(t, line, &q)));
    if (lane == 0) {
      s.tile_id[t] = s.id[s.leader[t]];
      s.tile_count[t] = found;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int t0 = 0; t0 < tiles; t0 += 32) {
      const int n = t0 + lane < tiles ? s.tile_count[t0 + lane] : 0;
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += u;
      }
      if (t0 + lane < tiles) s.tile_first[t0 + lane] = run + sum - n;
      run += __shfl_sync(kFull, sum, 31);
    }
  }
  __syncthreads();
  for (int t = warp; t < tiles; t += warps) {
    int left = s.tile_count[t], q;
    for (int line = s.leader[t] >> 5; left > 0; ++line) {
      const bool mine = members(t, line, &q);
      if (mine) s.order[s.tile_first[t] + q] = r0 + line * 32 + lane;
      left -= __popc(__ballot_sync(kFull, mine));
    }
  }
  __syncthreads();
  return tiles;
}

// One CTA per window.
__global__ void __launch_bounds__(kWindow) plan_kernel(const Args g) {
  __shared__ Window s;
  wait_prior_grid();
  allow_next_grid();  // after the wait: what ran before this call has finished
  const int i = threadIdx.x, r0 = blockIdx.x * kWindow, count = min(kWindow, g.n - r0);
  if (blockIdx.x == 0 && i == 0 && g.first) g.hdr[kHdrError] = 0;  // errors of this call only
  int unused = 0;  // the down kernel records the error bits
  const int tiles = make_plan(g, r0, count, s, &unused);
  if (i == 0) g.tiles_in[blockIdx.x] = tiles;
  if (i < tiles) {
    g.tile_id[r0 + i] = s.tile_id[i];
    g.tile_count[r0 + i] = s.tile_count[i];
    g.tile_first[r0 + i] = r0 + s.tile_first[i];
  }
  if (i < count) g.order[r0 + i] = s.order[i];
}

// ---------------------------------------------------------------- shared by the matmul kernels

// The call's tiles as a matmul kernel sees them: its own plan or the plan kernel's.
struct Tiles {
  const int* start;  // [windows + 1] tiles before a window
  const int *id, *count, *first, *order;
  int windows, total;

  // Slot of tile number t.
  __device__ __forceinline__ int slot(int t) const {
    int lo = 0, hi = windows;  // start[lo] <= t < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= t) lo = mid; else hi = mid;
    }
    return lo * kWindow + (t - start[lo]);
  }
};

// Gets the tiles; by all threads.  One window: planned here, in `own`, and *bad gets
// the error bits that this thread has seen.
__device__ Tiles get_tiles(const Args& g, int* start, Window& own, int* bad) {
  Tiles r;
  r.start = start;
  r.windows = g.windows;
  if (g.windows == 1) {
    r.total = make_plan(g, 0, g.n, own, bad);
    if (threadIdx.x == 0) start[0] = 0, start[1] = r.total;
    r.id = own.tile_id, r.count = own.tile_count, r.first = own.tile_first, r.order = own.order;
    __syncthreads();
    return r;
  }
  r.id = g.tile_id, r.count = g.tile_count, r.first = g.tile_first, r.order = g.order;
  for (int w = threadIdx.x; w < g.windows; w += blockDim.x) start[w + 1] = g.tiles_in[w];
  if (threadIdx.x == 0) start[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    int run = 0;
    for (int w0 = 0; w0 < g.windows; w0 += 32) {
      const int w = w0 + (int)threadIdx.x;
      int s = w < g.windows ? start[w + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, s, o);
        if ((int)threadIdx.x >= o) s += u;
      }
      if (w < g.windows) start[w + 1] = run + s;
      run += __shfl_sync(kFull, s, 31);
    }
  }
  __syncthreads();
  r.total = start[g.windows];
  return r;
}

struct Ctx {
  uint32_t sbase, bars;  // shared memory, and its mbarriers
  volatile int* abort_flag;
  int32_t* hdr;
  unsigned long long limit_ns;  // of a wait
};

__device__ __forceinline__ uint32_t bar_at(const Ctx& c, int i) { return c.bars + 8 * i; }

// Bounded wait that also gives up once another role has aborted.
__device__ __forceinline__ bool wait_bar(const Ctx& c, int i, uint32_t parity) {
  const uint32_t bar = bar_at(c, i);
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*c.abort_flag) return false;
      if (globaltimer_ns() - t0 > c.limit_ns) {
        set_error(c.hdr, DA_DEVERR_TIMEOUT);
        *c.abort_flag = 1;
        return false;
      }
    }
  }
}

// The same for a whole warp: one lane polls.
__device__ __forceinline__ bool wait_warp(const Ctx& c, int i, uint32_t parity) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(c, i, parity) ? 1 : 0;
  ok = __shfl_sync(kFull, ok, 0);
  __syncwarp();
  return ok != 0;
}

// A set of barriers of which each has completed some number of phases: one bit
// each for "any" and for the number's parity.
struct Phases {
  uint32_t any = 0, odd = 0;
  __device__ __forceinline__ void add(int i) {
    any |= 1u << i;
    odd ^= 1u << i;
  }
  __device__ __forceinline__ bool has(int i) const { return (any >> i) & 1u; }
  __device__ __forceinline__ uint32_t next(int i) const { return (odd >> i) & 1u; }         // parity
  __device__ __forceinline__ uint32_t last(int i) const { return ((odd >> i) & 1u) ^ 1u; }  // parity
};

// The arrive of a tcgen05.commit lands some time after the work it tracks; the
// last one on each barrier first, first + 1, ... must have landed before the CTA's
// shared memory is handed on.  Every barrier that commits arrive on has one issuer,
// which waits for its own here: after a time-out too, when nobody else may.  (Not
// inlined: small calls pay for the instructions that they fetch, 0.4 us of one row's.)
__device__ __noinline__ void drain_commits(Ctx c, int first, Phases p) {
  for (int i = 0; (p.any >> i) != 0; ++i)
    if (p.has(i) && !mbar_wait(bar_at(c, first + i), p.last(i))) set_error(c.hdr, DA_DEVERR_TIMEOUT);
}

// ---------------------------------------------------------------- down

constexpr int kStepK = 128, kRegionK = 64;         // K of a stage, and of a 128-byte swizzle row
constexpr int kXRegion = kTile * kRegionK * 2;     // 8 KB
constexpr int kXStage = (kStepK / kRegionK) * kXRegion;
constexpr int kDownEpWarps = 4, kDownProdWarp0 = 4, kDownProdWarps = 8, kDownMmaWarp0 = 12;
constexpr int kDownThreads = (kDownMmaWarp0 + 2) * 32;
constexpr int kDownStages = 6;                     // at most
// Two threads issue the MMAs: the even and the odd steps, each into an accumulator
// of its own that the epilogue adds.  Which of the two a step goes to depends on
// what came before, but the sum of two numbers does not.
// mbarriers: stage full; by tcgen05.commit: stage empty, each issuer's accumulators
// full, drain; accumulators empty
enum { kFull0 = 0, kEmpty0 = kFull0 + kDownStages, kDFull0 = kEmpty0 + kDownStages,
       kDownDrain = kDFull0 + 4, kDEmpty0 = kDownDrain + 2, kDownBars = kDEmpty0 + 2 };
constexpr uint32_t kDownCols = 4 * kTile;          // two units' two accumulators

__host__ __device__ constexpr int down_stage_bytes(int max_rank) {
  return max_rank * kStepK * 2 + kXStage;          // 32 KB at rank 64, 48 KB at 128
}

// The CTA's units, tile by tile and chunk by chunk; all roles walk them alike.
// Tiles that are only copied are passed over.
struct DownWalk {
  const Args& g;
  const Tiles& tiles;
  int left, tile, chunk;  // units to come, and where the next one is
  int id = 0, first = 0, count = 0, rank = 0, k0 = 0, k_len = 0;
  bool seen = false, fresh = false;  // fresh: the unit is its tile's first in this CTA
  __device__ __forceinline__ bool next() {
    while (left > 0) {
      fresh = !seen;
      if (fresh) {
        const int slot = tiles.slot(tile);
        id = tiles.id[slot];
        first = tiles.first[slot];
        count = tiles.count[slot];
        rank = id >= 0 ? rank_of(g, id) : 0;
        seen = true;
      }
      if (id < 0) {  // the tile's other units too
        const int skip = min(left, g.n_chunks - chunk);
        left -= skip;
        chunk += skip;
      } else {
        k0 = chunk * kKChunk;
        k_len = min(g.K, k0 + kKChunk) - k0;
        --left;
        ++chunk;
      }
      if (chunk == g.n_chunks) {
        chunk = 0;
        ++tile;
        seen = false;
      }
      if (id >= 0) return true;
    }
    return false;
  }
};

// A warp's copy takes 256 bytes of two rows; warp w brings rows 2 w, 2 w + 1 of
// every 16 of A and of the members' x.  fp32 rows of x are rounded on the way: a
// lane keeps kAhead of their pieces (16 rows of a step) in registers, so that
// several steps of a few rows, or one of many, are on their way.
template <bool BF16, int S>
__device__ void down_produce(const Ctx& c, const Args& g, DownWalk walk) {
  constexpr int kElem = BF16 ? 2 : 4, kAhead = 4;
  const int lane = threadIdx.x & 31;
  const int row0 = 2 * ((threadIdx.x >> 5) - kDownProdWarp0) + (lane >> 4), e0 = 8 * (lane & 15);
  const int stage_bytes = down_stage_bytes(g.max_rank), a_region = g.max_rank * 128;
  // where this lane's 16 bytes go within a stage: rows row0 + 16 i differ by 2048
  // bytes and share the swizzle
  const int region = (lane & 15) >> 3;
  const uint32_t at0 = row0 * 128 + (((lane & 7) ^ (row0 & 7)) << 4);
  const uint32_t a_at = region * a_region + at0, x_at = 2 * a_region + region * kXRegion + at0;
  int step = 0;
  bool ok = true;
  const char* xp[kTile / 16];  // this lane's first 8 elements of its rows' x, or null
  const char* ap = nullptr;
  while (ok && walk.next()) {
    if (walk.fresh) {
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i) {
        const int m = row0 + 16 * i;
        xp[i] = m < walk.count ? static_cast<const char*>(g.x) +
                                     ((long long)walk.tiles.order[walk.first + m] * g.K + e0) * kElem
                               : nullptr;
      }
      ap = reinterpret_cast<const char*>(g.a + ((long long)walk.id * g.max_rank + row0) * g.K + e0);
    }
    const int passes = (walk.rank + 15) >> 4, pieces = (walk.count + 15) >> 4;
    const int k_end = walk.k0 + walk.k_len;
    // K is a multiple of 64, so whole regions are live
    auto begin = [&](int k) {  // the step's stage is free; A goes there
      if (step >= S && !wait_warp(c, kEmpty0 + step % S, (step / S - 1) & 1)) return false;
      if (k + e0 < k_end) {
        const uint32_t to = c.sbase + (step % S) * stage_bytes + a_at;
        for (int i = 0; i < passes; ++i) cp_async16(to + i * 2048, ap + 2 * (k + (long long)i * 16 * g.K));
      }
      return true;
    };
    if constexpr (BF16) {
      for (int k = walk.k0; k < k_end; k += kStepK, ++step) {
        if (!(ok = begin(k))) break;
        const uint32_t to = c.sbase + (step % S) * stage_bytes + x_at;
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          if (xp[i] && k + e0 < k_end) cp_async16(to + i * 2048, xp[i] + k * kElem);
        cp_async_mbar_arrive(bar_at(c, kFull0 + step % S));  // when this thread's copies have landed
      }
    } else {
      float4 lo[kAhead], hi[kAhead];
      int kf = walk.k0, pf = 0;  // step and piece to ask for next
      auto fetch = [&](int u) {
        const char* p = pf == 0 ? xp[0] : pf == 1 ? xp[1] : pf == 2 ? xp[2] : xp[3];
        if (p && kf + e0 < k_end) {
          lo[u] = __ldg(reinterpret_cast<const float4*>(p + kf * kElem));
          hi[u] = __ldg(reinterpret_cast<const float4*>(p + kf * kElem) + 1);
        }
        if (++pf == pieces) pf = 0, kf += kStepK;
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u) fetch(u);
      for (int k = walk.k0, i = 0; ok && k < k_end;) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (k >= k_end || !ok) break;
          if (i == 0 && !(ok = begin(k))) break;
          if (row0 + 16 * i < walk.count && k + e0 < k_end)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             c.sbase + (step % S) * stage_bytes + x_at + i * 2048),
                         "r"(pack_bf16(lo[u].x, lo[u].y)), "r"(pack_bf16(lo[u].z, lo[u].w)),
                         "r"(pack_bf16(hi[u].x, hi[u].y)), "r"(pack_bf16(hi[u].z, hi[u].w))
                         : "memory");
          fetch(u);
          if (++i == pieces) {
            cp_async_mbar_arrive(bar_at(c, kFull0 + step % S));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_at(c, kFull0 + step % S));  // the stores
            i = 0;
            k += kStepK;
            ++step;
          }
        }
      }
    }
  }
  cp_async_wait_all();  // nothing is in flight when the CTA ends
}

// Issuer `me` takes the steps of its parity; returns what it committed, by barrier
// from kEmpty0 on.
template <int S>
__device__ Phases down_mma(const Ctx& c, const Args& g, DownWalk walk, uint32_t tmem, int me) {
  static_assert(S % 2 == 0, "a stage belongs to one issuer");
  const int stage_bytes = down_stage_bytes(g.max_rank), a_region = g.max_rank * 128;
  const uint64_t base = umma::smem_desc(c.sbase, 16, 1024, umma::kSwizzle128B);
  Phases done;
  int step = 0, k_unit = 0;
  for (; walk.next(); ++k_unit) {
    const int tb = k_unit & 1;
    if (k_unit >= 2 && !wait_bar(c, kDEmpty0 + tb, ((k_unit >> 1) - 1) & 1)) return done;
    umma::fence_after_sync();
    const uint32_t acc = tmem + (2 * tb + me) * kTile;
    bool first = true;
    for (int k = 0; k < walk.k_len; k += kStepK, ++step) {
      if ((step & 1) != me) continue;
      if (!wait_bar(c, kFull0 + step % S, (step / S) & 1)) return done;
      fence_proxy_async();  // the copies wrote through the generic proxy, the MMAs do not read through it
      umma::fence_after_sync();
      const int n_mma = min(kStepK, walk.k_len - k) / 16;
      // each MMA adds a constant to the operands' descriptors (K = 16 is 32 bytes of a
      // 128-byte swizzle row; the address field holds bytes / 16 and does not carry out)
      const uint64_t ad = base + (uint64_t)(((step % S) * stage_bytes) >> 4);
      const uint64_t xd = ad + (uint64_t)((2 * a_region) >> 4);
#pragma unroll
      for (int rg = 0; rg < kStepK / kRegionK; ++rg) {
        if (4 * rg >= n_mma) break;
        const uint64_t ar = ad + (uint64_t)((rg * a_region) >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          umma::mma_bf16(acc, ar + (uint64_t)((j * 32) >> 4),
                         xd + (uint64_t)((rg * kXRegion + j * 32) >> 4), kIdesc,
                         rg || j ? 1u : (uint32_t)!first);
      }
      umma::commit(bar_at(c, kEmpty0 + step % S));
      done.add(step % S);
      first = false;
    }
    umma::commit(bar_at(c, kDFull0 + 2 * tb + me));  // also when it had no step of the unit
    done.add(kDFull0 - kEmpty0 + 2 * tb + me);
  }
  return done;
}

// Warp q: ranks 32 q .. 32 q + 31, one a lane.
__device__ void down_epilogue(const Ctx& c, const Args& g, DownWalk walk, uint32_t tmem) {
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  int k_unit = 0, step = 0, row_lo = 0, row_hi = 0;  // members lane and lane + 32
  for (; walk.next(); ++k_unit) {
    if (walk.fresh) {
      if (lane < walk.count) row_lo = walk.tiles.order[walk.first + lane];
      if (lane + 32 < walk.count) row_hi = walk.tiles.order[walk.first + lane + 32];
    }
    const int tb = k_unit & 1, steps = (walk.k_len + kStepK - 1) / kStepK;
    if (!wait_warp(c, kDFull0 + 2 * tb, (k_unit >> 1) & 1) ||
        !wait_warp(c, kDFull0 + 2 * tb + 1, (k_unit >> 1) & 1))
      return;
    umma::fence_after_sync();
    const int r = 32 * q + lane;
    float* t = g.t + (long long)(walk.k0 / kKChunk) * g.n * g.max_rank + r;
    const uint32_t from = tmem + ((uint32_t)(q * 32) << 16) + 2 * tb * kTile;
    for (int m0 = 0; m0 < walk.count && 32 * q < walk.rank; m0 += 16) {
      float u[16], v[16];
      umma::ld_32x32b_x16(from + (step & 1) * kTile + m0, u);  // of the unit's first step
      if (steps > 1) umma::ld_32x32b_x16(from + (~step & 1) * kTile + m0, v);
      umma::wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = __shfl_sync(kFull, m0 < 32 ? row_lo : row_hi, (m0 + i) & 31);
        if (m0 + i < walk.count && r < walk.rank)
          t[(long long)row * g.max_rank] = steps > 1 ? u[i] + v[i] : u[i];
      }
    }
    umma::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_at(c, kDEmpty0 + tb));
    step += steps;
  }
}

template <bool BF16, int S>
__global__ void __launch_bounds__(kDownThreads, 1) down_kernel(const Args g) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Window own;
  __shared__ int start[kSlab / kWindow + 1];
  __shared__ __align__(8) uint64_t bars[kDownBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  Ctx c;
  c.sbase = smem_addr(smem);
  c.bars = smem_addr(bars);
  c.abort_flag = &abort_word;
  c.hdr = g.hdr;
  c.limit_ns = g.limit_ns;
  const int warp = threadIdx.x >> 5;
  if (c.sbase & 1023u) {  // the swizzled layout needs 1024-byte-aligned shared memory
    wait_prior_grid();
    if (threadIdx.x == 0) set_error(g.hdr, DA_DEVERR_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDownBars; ++i) {
      uint32_t count = 1;  // tcgen05.commit
      if (i < kEmpty0) count = kDownProdWarps * (32 + (BF16 ? 0 : 1));
      if (i >= kDEmpty0) count = kDownEpWarps;
      if (i == kFull0 && g.stall == 1) ++count;
      mbar_init(c.bars + 8 * i, count);
    }
    abort_word = 0;
    fence_mbar_init();
  }
  wait_prior_grid();
  allow_next_grid();  // after the wait: what ran before this call has finished
  if (warp == kDownMmaWarp0) {  // not before: the previous kernel may own tensor memory
    umma::tmem_alloc(smem_addr(&tmem_slot), kDownCols);
    umma::tmem_relinquish();
  }
  int bad = 0;
  if (g.windows > 1) {  // input checks, spread over the grid
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < g.n; i += gridDim.x * blockDim.x)
      planned_id(g, i, &bad);
    if (bad) set_error(g.hdr, bad);
  }
  umma::fence_before_sync();
  const Tiles tiles = get_tiles(g, start, own, &bad);  // holds CTA barriers
  if (g.windows == 1 && blockIdx.x == 0) {  // the plan has checked them
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0 && g.first) g.hdr[kHdrError] = 0;  // a later slab keeps what is there
    if (any) {
      __syncthreads();
      if (bad) set_error(g.hdr, bad);
    }
  }
  umma::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  const long long total = (long long)tiles.total * g.n_chunks;
  const int first = (int)(total * blockIdx.x / gridDim.x);
  const int last = (int)(total * (blockIdx.x + 1) / gridDim.x);
  DownWalk walk{g, tiles, last - first, first / g.n_chunks, first % g.n_chunks};
  Phases done;
  const int me = warp - kDownMmaWarp0;  // of the issuers
  if (me >= 0) {
    if ((threadIdx.x & 31) == 0) {
      done = down_mma<S>(c, g, walk, tmem, me);
      umma::commit(bar_at(c, kDownDrain + me));  // arrives once every MMA above has completed
    }
  } else if (warp < kDownEpWarps) {
    down_epilogue(c, g, walk, tmem);
  } else {
    down_produce<BF16, S>(c, g, walk);
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (me >= 0 && (threadIdx.x & 31) == 0) {
    done.add(kDownDrain + me - kEmpty0);
    drain_commits(c, kEmpty0, done);
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == kDownMmaWarp0) umma::tmem_dealloc(tmem, kDownCols);
}

// ---------------------------------------------------------------- up

constexpr int kGroups = 4;                  // epilogue groups of four warps, one accumulator each
// Warp w issues on scheduler w % 4.  The 16 epilogue warps take all four (a warp
// reads the quarter w % 4 of tensor memory); of the others the two MMA issuers have
// scheduler 0, the twelve that bring operands share 1, 2 and 3 (warps 24 and 28 are
// idle).  The issuers take the even and the odd units.
constexpr int kUpMmaWarp0 = 16, kUpMmaWarp1 = 20, kUpWarps = 32, kUpThreads = kUpWarps * 32;
constexpr int kUpProdWarps = 4, kUpTWarps = 4;
// 0 .. 11 for the warps that bring operands: four each for B and t, one for each
// group's y
__device__ __forceinline__ int up_helper(int warp) { return (warp - 17) / 4 * 3 + (warp - 17) % 4; }
constexpr int kBRegion = kFeat * 128;       // 16 KB: 128 features x 64 ranks
constexpr int kTRegion = kTile * 128;       // 8 KB: 64 members x 64 ranks
constexpr int kYRow = kFeat * 4;            // 512 bytes: a member's 128 features
constexpr int kYSlot = 16 * kYRow;          // 8 KB: a quarter of a tile
constexpr int kYSlots = 3;                  // of each epilogue group

// Shared memory by R, the 64-rank regions of an adapter of max_rank: four or two
// slots of B, two or one of t's terms, and the groups' y.
template <int R>
struct Up {
  static constexpr int kBSlots = 4 / R, kTSlots = 2 / R;
  static constexpr int kTOff = kBSlots * R * kBRegion;
  static constexpr int kTSlot = 3 * R * kTRegion;
  static constexpr int kYOff = kTOff + kTSlots * kTSlot;
  static constexpr int kSmem = kYOff + kGroups * kYSlots * kYSlot;
  static_assert(kBSlots % 2 == 0 && kGroups % 2 == 0, "slots and accumulators have one issuer");
  static_assert(kYOff % 1024 == 0 && kSmem <= 209 * 1024 && 2 * kSmem > 233472, "one CTA per SM");
};
constexpr int kMaxBSlots = 4;
// mbarriers: B full; by tcgen05.commit: B empty, accumulators full, each issuer's t
// empty, drain; accumulators empty, t full, y full and empty
enum { kBFull0 = 0, kBEmpty0 = kBFull0 + kMaxBSlots, kUDFull0 = kBEmpty0 + kMaxBSlots,
       kTEmpty0 = kUDFull0 + kGroups, kUpDrain = kTEmpty0 + 4, kUDEmpty0 = kUpDrain + 2,
       kTFull0 = kUDEmpty0 + kGroups, kYFull0 = kTFull0 + 2,
       kYEmpty0 = kYFull0 + kGroups * kYSlots, kUpBars = kYEmpty0 + kGroups * kYSlots };
constexpr uint32_t kUpCols = kGroups * kTile;

// The CTA's units: tile by tile, 128 features each.
struct UpWalk {
  const Args& g;
  const Tiles& tiles;
  int left, tile, block, blocks;  // units to come, and where the next one is
  int id = 0, count = 0, first = 0, rank = 0, f0 = 0;
  bool fresh = false;  // the unit is its tile's first in this CTA
  bool ends = false;   // ... and its last
  bool seen = false;
  __device__ __forceinline__ bool next() {
    if (left == 0) return false;
    --left;
    fresh = !seen;
    if (fresh) {
      const int slot = tiles.slot(tile);
      id = tiles.id[slot];
      count = tiles.count[slot];
      first = tiles.first[slot];
      rank = id >= 0 ? rank_of(g, id) : 0;
      seen = true;
    }
    f0 = block * kFeat;
    if (++block == blocks) {
      block = 0;
      ++tile;
      seen = false;
    }
    ends = left == 0 || !seen;
    return true;
  }
};

// B, 128 features a unit: a thread keeps one 16-byte chunk of the ranks and steps
// through the features, neighbours in a row taking neighbouring chunks.  Slots go
// by the unit's number, units that are only copied included, so that a slot
// belongs to one issuer.
template <int R>
__device__ void up_produce(const Ctx& c, const Args& g, UpWalk walk) {
  constexpr int S = Up<R>::kBSlots;
  const int lane = threadIdx.x & 31, tid = up_helper(threadIdx.x >> 5) * 32 + lane;
  int row0 = 0, rows = 1, ch = 0, bytes = 0;
  Phases filled;
  for (int i = 0; walk.next(); ++i) {
    if (walk.id < 0) continue;
    if (walk.fresh) {
      const int nc = ((walk.rank + 15) >> 4) * 2;  // 16-byte chunks of a row: 2 .. 16
      rows = (kUpProdWarps * 32) / nc;             // features that the threads cover at once
      row0 = tid / nc;
      ch = tid - row0 * nc;
      if (row0 >= rows) row0 = kFeat;              // left over: no part in it
      bytes = min(16, max(0, (walk.rank - 8 * ch) * 2));
    }
    if (filled.has(i % S) && !wait_warp(c, kBEmpty0 + i % S, filled.last(i % S))) break;
    filled.add(i % S);
    const uint32_t to = c.sbase + (i % S) * (R * kBRegion) + (ch >> 3) * kBRegion;
    const __nv_bfloat16* b = g.b + ((long long)walk.id * g.N + walk.f0) * g.max_rank + 8 * ch;
    for (int row = row0; row < kFeat; row += rows)
      cp_async16_zfill(to + row * 128 + (((ch & 7) ^ (row & 7)) << 4), b + row * g.max_rank, bytes);
    cp_async_mbar_arrive(bar_at(c, kBFull0 + i % S));
  }
  cp_async_wait_all();
}

// t of a tile's members: chunk sums added in order, scaled, split.  Warp w takes
// members w, w + 4, ...; a lane two ranks of each 64.
template <int R, bool WIDE>
__device__ void up_make_t(const Ctx& c, const Args& g, UpWalk walk) {
  constexpr int S = Up<R>::kTSlots;
  const int lane = threadIdx.x & 31, w = up_helper(threadIdx.x >> 5) - kUpProdWarps;
  const long long part = (long long)g.n * g.max_rank;
  int k = 0;
  bool waited = false;
  while (walk.next()) {
    if (!walk.fresh || walk.id < 0) continue;
    const float scale = g.scales ? __ldg(g.scales + walk.id) : 1.f;
    if (!waited) {
      wait_prior_grid();  // for t
      allow_next_grid();
      waited = true;
    }
    if (k >= S && (!wait_warp(c, kTEmpty0 + 2 * (k % S), (k / S - 1) & 1) ||
                   !wait_warp(c, kTEmpty0 + 2 * (k % S) + 1, (k / S - 1) & 1)))
      return;
    const uint32_t slot = c.sbase + Up<R>::kTOff + (k % S) * Up<R>::kTSlot;
    int row_lo = 0, row_hi = 0;  // members lane and lane + 32
    if (lane < walk.count) row_lo = walk.tiles.order[walk.first + lane];
    if (lane + 32 < walk.count) row_hi = walk.tiles.order[walk.first + lane + 32];
    // kBatch members and kDeep chunks at once: their loads are in flight together (one
    // by one a tile of 64 took 25 us; four of each spill)
    constexpr int kBatch = WIDE ? 4 : 2, kDeep = WIDE ? 2 : 4;
    for (int m0 = w; m0 < walk.count; m0 += kBatch * kUpTWarps) {
#pragma unroll
      for (int reg = 0; reg < R; ++reg) {
        const int r = 64 * reg + 2 * lane;
        const bool live = r < walk.rank;  // the row is max_rank long, so r + 1 may be read
        const float* t[kBatch];
        float2 sum[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int m = m0 + j * kUpTWarps;
          const int row = __shfl_sync(kFull, m < 32 ? row_lo : row_hi, m & 31);
          t[j] = live && m < walk.count ? g.t + (long long)row * g.max_rank + r : nullptr;
          sum[j] = make_float2(0.f, 0.f);
        }
        for (int p0 = 0; p0 < g.n_chunks; p0 += kDeep) {
          float2 e[kDeep][kBatch];
#pragma unroll
          for (int p = 0; p < kDeep; ++p)
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
              if (t[j] && p0 + p < g.n_chunks)
                e[p][j] = __ldcg(reinterpret_cast<const float2*>(t[j] + (p0 + p) * part));
#pragma unroll
          for (int p = 0; p < kDeep; ++p)
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
              if (t[j] && p0 + p < g.n_chunks) {
                sum[j].x += e[p][j].x;
                sum[j].y += e[p][j].y;
              }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int m = m0 + j * kUpTWarps;
          if (m >= walk.count) break;
          float v[2] = {live ? sum[j].x * scale : 0.f,
                        r + 1 < walk.rank ? sum[j].y * scale : 0.f};
          const uint32_t at = slot + reg * kTRegion + m * 128 + (((lane >> 2) ^ (m & 7)) << 4) +
                              (lane & 3) * 4;
#pragma unroll
          for (int term = 0; term < 3; ++term) {  // each takes the next eight bits
            __nv_bfloat16 h[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              h[i] = __float2bfloat16_rn(v[i]);
              // nothing is left of an infinity (inf - inf would make it a NaN)
              v[i] = __hisinf(h[i]) ? 0.f : v[i] - __bfloat162float(h[i]);
            }
            const uint32_t word = (uint32_t)__bfloat16_as_ushort(h[0]) |
                                  (uint32_t)__bfloat16_as_ushort(h[1]) << 16;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + term * R * kTRegion), "r"(word)
                         : "memory");
          }
        }
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_at(c, kTFull0 + k % S));
    ++k;
  }
  if (!waited) wait_prior_grid();  // this grid has not ended before the down kernel has
}

// What an issuer committed: to the slots of B, the accumulators and its barriers of
// t's slots.
struct UpDone {
  Phases slots, accs, tiles;
};

// Issuer `me` takes the units of its parity.
template <int R>
__device__ UpDone up_mma(const Ctx& c, const Args& g, UpWalk walk, uint32_t tmem, int me) {
  constexpr int S = Up<R>::kBSlots, TS = Up<R>::kTSlots;
  const uint64_t base = umma::smem_desc(c.sbase, 16, 1024, umma::kSwizzle128B);
  UpDone done;
  int tiles = 0;  // begun
  for (int i = 0; walk.next(); ++i) {
    if (walk.id < 0) continue;
    if (walk.fresh) {
      if (!wait_bar(c, kTFull0 + tiles % TS, (tiles / TS) & 1)) return done;
      ++tiles;
    }
    const int ts = (tiles - 1) % TS;
    if ((i & 1) == me) {
      const int e = i % kGroups, s = i % S;
      if (done.accs.has(e) && !wait_bar(c, kUDEmpty0 + e, done.accs.last(e))) return done;
      if (!wait_bar(c, kBFull0 + s, done.slots.next(s))) return done;
      fence_proxy_async();  // as in down_mma
      umma::fence_after_sync();
      const uint64_t bd = base + (uint64_t)((s * (R * kBRegion)) >> 4);
      const uint64_t td = base + (uint64_t)((Up<R>::kTOff + ts * Up<R>::kTSlot) >> 4);
      const uint32_t acc = tmem + e * kTile;
      const int n_k = (walk.rank + 15) >> 4;
      umma::mma_bf16(acc, bd, td + (uint64_t)((2 * R * kTRegion) >> 4), kIdesc, 0u);
#pragma unroll
      for (int term = 2; term >= 0; --term) {  // small terms first
#pragma unroll
        for (int kb = 0; kb < 4 * R; ++kb) {
          if ((term == 2 && kb == 0) || kb >= n_k) continue;
          umma::mma_bf16(acc, bd + (uint64_t)(((kb >> 2) * kBRegion + (kb & 3) * 32) >> 4),
                         td + (uint64_t)(((term * R + (kb >> 2)) * kTRegion + (kb & 3) * 32) >> 4),
                         kIdesc, 1u);
        }
      }
      umma::commit(bar_at(c, kBEmpty0 + s));
      umma::commit(bar_at(c, kUDFull0 + e));
      done.slots.add(s);
      done.accs.add(e);
    }
    if (walk.ends) {  // both issuers do
      umma::commit(bar_at(c, kTEmpty0 + 2 * ts + me));
      done.tiles.add(2 * ts + me);
    }
  }
  return done;
}

// y of group e's units, a quarter of a tile at a time, a row's 512 bytes with one
// instruction.
template <int R>
__device__ void up_fetch_y(const Ctx& c, const Args& g, UpWalk walk) {
  constexpr int S = kYSlots;
  const int lane = threadIdx.x & 31, e = up_helper(threadIdx.x >> 5) - kUpProdWarps - kUpTWarps;
  const int full = kYFull0 + e * S, empty = kYEmpty0 + e * S;
  const uint32_t ring = c.sbase + Up<R>::kYOff + e * S * kYSlot + lane * 16;
  int k = 0, row_lo = 0, row_hi = 0;  // members lane and lane + 32
  bool ok = true;
  for (int i = 0; ok && walk.next(); ++i) {
    if (walk.fresh) {
      if (lane < walk.count) row_lo = walk.tiles.order[walk.first + lane];
      if (lane + 32 < walk.count) row_hi = walk.tiles.order[walk.first + lane + 32];
    }
    if (i % kGroups != e) continue;
    const float* y = g.y + walk.f0 + 4 * lane;
    for (int m0 = 0; m0 < walk.count; m0 += 16, ++k) {
      if (k >= S && !wait_warp(c, empty + k % S, (k / S - 1) & 1)) {
        ok = false;
        break;
      }
      const uint32_t to = ring + (k % S) * kYSlot;
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const int row = __shfl_sync(kFull, m0 < 32 ? row_lo : row_hi, (m0 + m) & 31);
        if (m0 + m < walk.count) cp_async16(to + m * kYRow, y + (long long)row * g.N);
      }
      cp_async_mbar_arrive(bar_at(c, full + k % S));
    }
  }
  cp_async_wait_all();
}

// The three terms of t are zero below a bf16 value's bits, and an infinity times those
// is a NaN where the definition has an infinity; a t above bf16's largest is an
// infinity in them.  So the sums v of a lane's feature f and a quarter's rows that are
// not finite are formed again in plain fp32, in rank order, from y in memory.  By a whole
// warp, whose lanes add up a rank's chunks of t each.  (Rolled up: a call, or registers
// for more at once, would spill in the epilogue.)
__device__ __forceinline__ void sum_again(const Args& g, float* v, const int* rows, int live, int id,
                                          int rank, int f) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* b = g.b + ((long long)id * g.N + f) * g.max_rank;
  const float scale = g.scales ? __ldg(g.scales + id) : 1.f;
#pragma unroll 1
  for (int m = 0; m < live; ++m) {
    const bool odd = !(fabsf(v[m * kFeat]) <= FLT_MAX);
    if (!__any_sync(kFull, odd)) continue;
    const int row = rows[m];
    float d = 0.f;
#pragma unroll 1
    for (int r0 = 0; r0 < rank; r0 += 32) {
      float t = 0.f;
      if (r0 + lane < rank) {
#pragma unroll 1
        for (int p = 0; p < g.n_chunks; ++p)
          t += __ldcg(g.t + ((long long)p * g.n + row) * g.max_rank + r0 + lane);
      }
      t *= scale;
#pragma unroll 1
      for (int r = r0; r < min(rank, r0 + 32); ++r)
        d = fmaf(__shfl_sync(kFull, t, r - r0), __bfloat162float(b[r]), d);
    }
    if (odd) v[m * kFeat] = g.y[(long long)row * g.N + f] + d;
  }
}

// Group e takes units e, e + 4, ... of the CTA, a quarter of the members at a time.
// Warp q of it has features 32 q .. + 31 to itself: it adds the products, a feature
// a lane, to y in shared memory, and writes the sums from there, 16 bytes a lane and
// 128 of a row.  (Whole rows to a warp needed a barrier of the group per quarter.)
template <int R>
__device__ void up_epilogue(const Ctx& c, const Args& g, UpWalk walk, uint32_t tmem, uint8_t* smem) {
  constexpr int S = kYSlots;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = warp & 3, e = warp >> 2;
  uint8_t* ring = smem + Up<R>::kYOff + e * S * kYSlot + 32 * q * 4;
  uint32_t parity = 0;
  int k = 0, row_lo = 0, row_hi = 0;  // members lane and lane + 32
  for (int i = 0; walk.next(); ++i) {
    if (walk.fresh) {
      if (lane < walk.count) row_lo = walk.tiles.order[walk.first + lane];
      if (lane + 32 < walk.count) row_hi = walk.tiles.order[walk.first + lane + 32];
    }
    if (i % kGroups != e) continue;
    const int count = walk.count;
    const bool product = walk.id >= 0, write = product || g.out != g.y;
    const long long f = walk.f0 + 32 * q + 4 * (lane & 7);
    for (int m0 = 0; m0 < count; m0 += 16, ++k) {
      uint8_t* slot = ring + (k % S) * kYSlot;
      if (product) {
        float d[16];
        if (m0 == 0) {
          if (!wait_warp(c, kUDFull0 + e, parity)) return;
          parity ^= 1u;
          umma::fence_after_sync();
        }
        umma::ld_32x32b_x16(tmem + ((uint32_t)(q * 32) << 16) + e * kTile + m0, d);
        umma::wait_ld();
        if (m0 + 16 >= count) {
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_at(c, kUDEmpty0 + e));
        }
        if (!wait_warp(c, kYFull0 + e * S + k % S, (k / S) & 1)) return;
        float* yv = reinterpret_cast<float*>(slot) + lane;
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          d[m] += yv[m * kFeat];
          yv[m * kFeat] = d[m];  // past count: leftovers, not stored
        }
        // 0 if all are finite, else NaN (16 multiplications: 67 rows of 24 adapters 29.2 us,
        // 28.6 without, 8192 rows 166 and 163)
        float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 16; ++m)
          if (m < count - m0) z[m & 3] = fmaf(d[m], 0.f, z[m & 3]);
        const float odd = (z[0] + z[1]) + (z[2] + z[3]);
        if (__any_sync(kFull, odd != odd))
          sum_again(g, yv, walk.tiles.order + walk.first + m0, min(16, count - m0), walk.id, walk.rank,
                    walk.f0 + 32 * q + lane);
        __syncwarp();
      } else if (!wait_warp(c, kYFull0 + e * S + k % S, (k / S) & 1)) {
        return;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = 4 * j + (lane >> 3);
        const int row = __shfl_sync(kFull, m0 < 32 ? row_lo : row_hi, (m0 + m) & 31);
        if (m0 + m >= count) continue;
        const float4 v = *reinterpret_cast<const float4*>(slot + m * kYRow + 16 * (lane & 7));
        const long long at = (long long)row * g.N + f;
        if (write) *reinterpret_cast<float4*>(g.out + at) = v;
        if (g.out_bf16)
          *reinterpret_cast<uint2*>(g.out_bf16 + at) =
              make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_at(c, kYEmpty0 + e * S + k % S));
    }
  }
}

template <int R, bool WIDE>
__global__ void __launch_bounds__(kUpThreads, 1) up_kernel(const Args g) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Window own;
  __shared__ int start[kSlab / kWindow + 1];
  __shared__ __align__(8) uint64_t bars[kUpBars];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  Ctx c;
  c.sbase = smem_addr(smem);
  c.bars = smem_addr(bars);
  c.abort_flag = &abort_word;
  c.hdr = g.hdr;
  c.limit_ns = g.limit_ns;
  const int warp = threadIdx.x >> 5;
  if (c.sbase & 1023u) {  // the swizzled layout needs 1024-byte-aligned shared memory
    wait_prior_grid();
    if (threadIdx.x == 0) set_error(g.hdr, DA_DEVERR_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kUpBars; ++i) {
      uint32_t count = 1;  // tcgen05.commit
      if (i < kBEmpty0) count = kUpProdWarps * 32;
      if (i >= kYFull0 && i < kYEmpty0) count = 32;
      if (i >= kUDEmpty0 && i < kTFull0) count = 4;
      if (i == kTFull0 || i == kTFull0 + 1) count = kUpTWarps;
      if (i >= kYEmpty0) count = 4;
      if (i == kBFull0 && g.stall == 2) ++count;
      mbar_init(c.bars + 8 * i, count);
    }
    abort_word = 0;
    fence_mbar_init();
  }
  // Only t comes from the down kernel.  ids, ranks, scales, B and y were complete before
  // it let this one start, so with one window (the plan is made here) all roles start
  // at once and those of t wait.
  if (g.windows > 1) wait_prior_grid();
  int unused = 0;  // the down kernel has recorded the error bits
  const Tiles tiles = get_tiles(g, start, own, &unused);  // holds CTA barriers
  const int blocks = g.N / kFeat;
  const long long total = (long long)tiles.total * blocks;
  const int first = (int)(total * blockIdx.x / gridDim.x);
  const int last = (int)(total * (blockIdx.x + 1) / gridDim.x);
  UpWalk walk{g, tiles, last - first, first / blocks, first % blocks, blocks};
  UpDone done;
  const bool issuer = warp == kUpMmaWarp0 || warp == kUpMmaWarp1;
  const int me = warp == kUpMmaWarp1;
  uint32_t tmem = 0;
  if (issuer || warp < kUpMmaWarp0) {  // the roles that use tensor memory
    if (warp == kUpMmaWarp0) {
      // not before the wait: a CTA that holds tensor memory waits for no other kernel,
      // so kernels of two streams cannot wait for one another's
      wait_prior_grid();
      umma::tmem_alloc(smem_addr(&tmem_slot), kUpCols);
      umma::tmem_relinquish();
    }
    umma::fence_before_sync();
    asm volatile("bar.sync 1, %0;" ::"n"((kUpMmaWarp0 + 2) * 32) : "memory");
    umma::fence_after_sync();
    tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  }
  if (issuer) {
    if ((threadIdx.x & 31) == 0) {
      done = up_mma<R>(c, g, walk, tmem, me);
      umma::commit(bar_at(c, kUpDrain + me));
    }
  } else if (warp < kUpMmaWarp0) {
    up_epilogue<R>(c, g, walk, tmem, smem);
  } else if (warp % 4) {
    const int h = up_helper(warp);
    if (h < kUpProdWarps)
      up_produce<R>(c, g, walk);
    else if (h < kUpProdWarps + kUpTWarps)
      up_make_t<R, WIDE>(c, g, walk);
    else
      up_fetch_y<R>(c, g, walk);
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (issuer && (threadIdx.x & 31) == 0) {
    if (!mbar_wait(bar_at(c, kUpDrain + me), 0)) set_error(c.hdr, DA_DEVERR_TIMEOUT);
    drain_commits(c, kBEmpty0, done.slots);
    drain_commits(c, kTEmpty0, done.tiles);
    // the epilogue has waited for the accumulators' unless it gave up
    if (*c.abort_flag) drain_commits(c, kUDFull0, done.accs);
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == kUpMmaWarp0) umma::tmem_dealloc(tmem, kUpCols);
}

// ---------------------------------------------------------------- host

constexpr size_t kHdr = 256;

size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }

bool shape_ok(int n, int N, int K, int n_adapters, int max_rank) {
  if (n < 0 || N <= 0 || K <= 0 || N % NVFP4_MM_TILE_N || K % 64) return false;
  if (K > NVFP4_ADAPTER_MAX_K) return false;
  if (n_adapters < 1 || max_rank < 16 || max_rank > kMaxRank || max_rank % 16) return false;
  return (long long)n * K < (1ll << 31) && (long long)n * N < (1ll << 31);
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q + b_bytes && q < p + a_bytes;
}

int chunks_of(int K) { return (K + kKChunk - 1) / kKChunk; }

struct Layout {
  size_t tiles_in, tile_id, tile_count, tile_first, order, t, total;
};

Layout layout_of(int n, int K, int max_rank) {
  const size_t rows = (size_t)std::min(n, kSlab), ints = round_up(rows * 4, 256);
  Layout l;
  l.tiles_in = kHdr;
  l.tile_id = l.tiles_in + round_up((rows + kWindow - 1) / kWindow * 4, 256);
  l.tile_count = l.tile_id + ints;
  l.tile_first = l.tile_count + ints;
  l.order = l.tile_first + ints;
  l.t = l.order + ints;
  l.total = l.t + (size_t)chunks_of(K) * rows * max_rank * 4;
  return l;
}

template <bool BF16, int S>
cudaError_t launch_down(const Args& g, int sms, cudaStream_t st) {
  // at least so much that a second CTA stays off the SM: one owns tensor memory
  const int smem = std::max(S * down_stage_bytes(g.max_rank), 118 * 1024);
  cudaError_t e = allow_smem(down_kernel<BF16, S>, smem);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>((long long)g.n * g.n_chunks, sms);
  return launch_after(down_kernel<BF16, S>, dim3(grid), dim3(kDownThreads), (size_t)smem, st, g);
}

// WIDE: t of twice as many members at once, two chunks of K at a time instead of four.
// For K of up to two chunks, where the others would be empty, and rows for full tiles
// (4096 features, us: 1910 rows of rank 64 and K = 1024 47.0, else 48.9, of rank 128
// and K = 2048 63.4 and 67.1, 140 rows 26.8 and 27.7; K = 4096, 1910 rows of rank 64
// 55.7 and 52.2; K = 1024, 67 rows of rank 64 19.6 and 19.2).
template <int R, bool WIDE>
cudaError_t launch_up(const Args& g, int sms, cudaStream_t st) {
  cudaError_t e = allow_smem(up_kernel<R, WIDE>, Up<R>::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>((long long)g.n * (g.N / kFeat), sms);
  return launch_after(up_kernel<R, WIDE>, dim3(grid), dim3(kUpThreads), (size_t)Up<R>::kSmem, st, g);
}

}  // namespace
}  // namespace da

using namespace da;

extern "C" {

size_t nvfp4_mm_adapters_workspace_bytes(int32_t n, int32_t N, int32_t K, int32_t n_adapters,
                                         int32_t max_rank) {
  if (!shape_ok(n, N, K, n_adapters, max_rank)) return 0;
  return layout_of(n, K, max_rank).total;
}

int nvfp4_mm_adapters(const void* x, int32_t x_dtype, int32_t n, int32_t N, int32_t K,
                      const void* a, const void* b, int32_t n_adapters, int32_t max_rank,
                      const int32_t* ranks, const float* scales, const int32_t* ids,
                      const float* y, float* out, void* out_bf16, void* ws, size_t ws_bytes,
                      void* stream) {
  const int stall = x_dtype / NVFP4_X_TEST_STALL_DOWN;  // tests only
  x_dtype %= NVFP4_X_TEST_STALL_DOWN;
  if (stall < 0 || stall > 2) return DA_ERR_INVALID_ARG;
  if (x_dtype != NVFP4_X_F32 && x_dtype != NVFP4_X_BF16) return DA_ERR_INVALID_ARG;
  if (!shape_ok(n, N, K, n_adapters, max_rank)) return DA_ERR_UNSUPPORTED;
  if (n == 0) {  // nothing to do, and so no errors
    if (!ws) return DA_OK;
    if (!aligned_to(ws, 256) || ws_bytes < kHdr) return DA_ERR_WORKSPACE;
    return cudaMemsetAsync(ws, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DA_OK : DA_ERR_CUDA;
  }
  if (!x || !a || !b || !ids || !y || !out) return DA_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(a, 16) || !aligned_to(b, 16) || !aligned_to(y, 16) ||
      !aligned_to(out, 16) || !aligned_to(out_bf16, 16) || !aligned_to(ids, 4) ||
      !aligned_to(ranks, 4) || !aligned_to(scales, 4))
    return DA_ERR_INVALID_ARG;
  const size_t x_bytes = (size_t)n * K * (x_dtype == NVFP4_X_BF16 ? 2 : 4);
  const size_t y_bytes = (size_t)n * N * 4, ob_bytes = out_bf16 ? y_bytes / 2 : 0;
  if ((y != out && overlap(y, y_bytes, out, y_bytes)) || overlap(x, x_bytes, out, y_bytes) ||
      overlap(x, x_bytes, out_bf16, ob_bytes) || overlap(y, y_bytes, out_bf16, ob_bytes) ||
      overlap(out, y_bytes, out_bf16, ob_bytes))
    return DA_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256)) return DA_ERR_WORKSPACE;
  if (ws_bytes < nvfp4_mm_adapters_workspace_bytes(n, N, K, n_adapters, max_rank))
    return DA_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DA_ERR_CUDA;
  const Layout l = layout_of(n, K, max_rank);
  uint8_t* base = static_cast<uint8_t*>(ws);
  Args g;
  std::memset(&g, 0, sizeof(g));
  g.a = static_cast<const __nv_bfloat16*>(a);
  g.b = static_cast<const __nv_bfloat16*>(b);
  g.ranks = ranks;
  g.scales = scales;
  g.hdr = static_cast<int32_t*>(ws);
  g.tiles_in = reinterpret_cast<int32_t*>(base + l.tiles_in);
  g.tile_id = reinterpret_cast<int32_t*>(base + l.tile_id);
  g.tile_count = reinterpret_cast<int32_t*>(base + l.tile_count);
  g.tile_first = reinterpret_cast<int32_t*>(base + l.tile_first);
  g.order = reinterpret_cast<int32_t*>(base + l.order);
  g.t = reinterpret_cast<float*>(base + l.t);
  g.N = N;
  g.K = K;
  g.n_adapters = n_adapters;
  g.max_rank = max_rank;
  g.n_chunks = chunks_of(K);
  g.copy = out != y || out_bf16;
  g.stall = stall;
  g.limit_ns = stall ? kTestStallNs : kWaitLimitNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = x_dtype == NVFP4_X_BF16;
  // six stages of up to 32 KB, or four of up to 48; ranks of up to 64 take one
  // region of a slot, higher ones two
  auto* down = max_rank <= 64 ? (bf16 ? launch_down<true, 6> : launch_down<false, 6>)
                              : (bf16 ? launch_down<true, 4> : launch_down<false, 4>);
  const bool wide = g.n_chunks <= 2 && n > 2 * kTile;
  auto* up = max_rank <= 64 ? (wide ? launch_up<1, true> : launch_up<1, false>)
                            : (wide ? launch_up<2, true> : launch_up<2, false>);
  for (int r0 = 0; r0 < n; r0 += kSlab) {
    const size_t row = (size_t)r0;
    g.n = std::min(kSlab, n - r0);
    g.windows = (g.n + kWindow - 1) / kWindow;
    g.first = r0 == 0;
    g.x = static_cast<const uint8_t*>(x) + row * K * (bf16 ? 2 : 4);
    g.ids = ids + row;
    g.y = y + row * N;
    g.out = out + row * N;
    g.out_bf16 = out_bf16 ? static_cast<__nv_bfloat16*>(out_bf16) + row * N : nullptr;
    if (g.windows > 1 &&
        launch_after(plan_kernel, dim3((unsigned)g.windows), dim3(kWindow), 0, st, g) !=
            cudaSuccess)
      return DA_ERR_CUDA;
    if (down(g, sms, st) != cudaSuccess) return DA_ERR_CUDA;
    if (up(g, sms, st) != cudaSuccess) return DA_ERR_CUDA;
  }
  return DA_OK;
}

}  // extern "C"
