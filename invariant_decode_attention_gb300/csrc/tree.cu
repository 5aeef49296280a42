// Attention of a tree of drafted tokens over the caches: every node of a row attends to the
// row's context and to its own ancestors.  For (node t, head h) of row b, over the entries j
// that t sees,
//     s_j = scale q . k_j,   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m)    (log2 units),
// in one pass with a running reference value m that moves only when a score exceeds it by 2^8,
// and a log-sum-exp that joins the splits of a list in their order.
//
// All nodes of a row read the same K and V, so the rows of a matrix product are (node, head)
// pairs: S = Q K^T and O += P V are tcgen05.mma of 128 rows, with S, O and Q in tensor memory
// and P in shared memory over the K tile that it came from (64 dims: in tensor memory).  Calls
// with few such pairs go to tree_few.cu.  What a node sees is a 64-bit mask of nodes, found
// once a unit; whole tiles of context need no mask.
//
// Weights are rounded before the second product: an MMA takes both operands in one type, so
// that they are bf16 beside bf16 values (off by 2^-8 of their size at most) and f16 beside f16
// ones (2^-11; formed with a largest one of 2^7 or more).  The sum that divides them is of the
// unrounded ones, in fp32.  Over bf16 caches outputs are off by 0.0023 (root mean square,
// relative), 0.0017 of it by their own rounding; a second term of each weight would take a
// second product.
//
// Bound: bytes of K and V for one row's nodes; the softmax (a thread a row, 64 exponentials a
// tile) and the way from MMA to softmax to MMA for full units of 128.  Measured, captured and
// replayed, bf16, 64-entry tiles: 32 rows of 16 nodes, 32/8 heads, 8192 entries, 171 us = 4.8
// TB/s (copied once at the measured bandwidth: 120 us); 8 rows of 64 nodes, 64/8 heads, 16384
// entries, 230 us = 675 TFLOP/s; 64 rows of 16 nodes, 4096 of 32768 entries in their window,
// 32/8 heads, E4M3 397 us and NVFP4 513 (81 and 47): two operand stages, each held from the
// widening of its K to the end of its P V, keep widening and softmax close together.
//
// Two blocks an SM, one unit each, because everything in a block waits for something:
// between MMA, softmax and MMA, and for 13,500 cycles between units; one block with two units
// in flight took 204 us.  Also measured and not kept,
// on the first and the second of these: warps of their own for the output (258, 493), K and V
// in rings of their own with P apart (197, 259), MMAs issued by an elected lane of a whole warp (198, 270), a unit's
// split chosen for equal units (188, 237: the blocks run in step), copies of Q and output by
// rows of their own threads (187, 267).
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "merge.cuh"
#include "tcgen05.cuh"
#include "tree_parts.cuh"

namespace da {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

}  // namespace

bool tree_tensor_map(CUtensorMap* tm, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box, bool bytes, CUtensorMapSwizzle swizzle) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t elem[3] = {1, 1, 1};
  return fn(tm, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
            const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// ------------------------------------------------------------------ shapes

constexpr int kRows = 128;         // rows of an MMA: TMEM lanes
constexpr int kRegion = kT * 128;  // 64 rows of 128 bytes, swizzled
// Shared memory of a block; two blocks share an SM.  KT: the cache's type; quantized caches
// pass raw stages of cache bytes and are widened to f16 into the operand stages.
template <int KT, int D>
struct Lay {
  static constexpr bool Q8 = KT != DA_KV_BF16;
  static constexpr int kTile = (D / 64) * kRegion;  // K (or V) of a tile, 16-bit elements
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = (Q8 ? 2 : 3) * (128 / D);
  static constexpr int kCodeRow = KT == DA_KV_NVFP4 ? D / 2 : D;  // code bytes of a head's row
  static constexpr int kScaleRow = KT == DA_KV_NVFP4 ? D / 16 : 0;
  static constexpr int kRaw = 2 * kT * (kCodeRow + kScaleRow);
  static constexpr int kRawStage = (kRaw + 1023) / 1024 * 1024;
  static constexpr int kRawStages = !Q8 ? 0 : (KT == DA_KV_NVFP4 ? 3 : 2) * (128 / D);
  static constexpr int kRawOffset = kStages * kStage;
  static constexpr int kPass = kRawOffset + kRawStages * kRawStage;  // 2 KB for each softmax warp
  static constexpr int kBarOffset = kPass + 4 * 2048;
  // barriers
  static constexpr int kFull = 0, kEmpty = kFull + kStages, kRawFull = kEmpty + kStages,
                       kRawEmpty = kRawFull + kRawStages, kQFull = kRawEmpty + kRawStages, kSFull = kQFull + 1,
                       kSFree = kSFull + 1, kPFull = kSFree + 1, kPVDone = kPFull + 1, kDrain = kPVDone + 1,
                       kStall = kDrain + 1, kBars = kStall + 1;
  static constexpr int kSlots = kBarOffset + kBars * 8;         // TMEM address, abort flag
  static constexpr int kSizes = (kSlots + 8 + 15) / 16 * 16;    // length, nodes and splits of each row
  static constexpr int kFirst = kSizes + kTreeRows * 8;         // first unit of each row
  // this and the next unit of each softmax warp
  static constexpr int kUnits = (kFirst + (kTreeRows + 1) * 4 + 15) / 16 * 16;
  static constexpr int kBytes = kUnits + 4 * 2 * (int)sizeof(Unit);
  // warps 0-3 softmax, Q and output, 4 and 5 MMAs, 6 and 7 copies, 8-11 conversion.  With
  // these the threads' registers are split by role; the shares add up to what the block was
  // launched with, 384 * 80 = 128 * (128 + 56 + 56).
  static constexpr int kThreads = Q8 ? 384 : 256;
  static constexpr int kSoftmaxRegs = 128, kIssueRegs = 56, kConvertRegs = 56;
  static_assert(!Q8 || 128 * (kSoftmaxRegs + kIssueRegs + kConvertRegs) <= kThreads * 80, "register split");
  static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two blocks an SM");
  // tensor memory: S, O, Q (two elements a column) and, for 64 dims, P; for 128 dims P lies
  // in shared memory, over the K tile that its scores came from
  static constexpr uint32_t kSCol = 0, kOCol = 64, kQCol = kOCol + D, kPCol = kQCol + D / 2;
  static constexpr bool kPInTmem = D == 64;
  static_assert(kPCol + (kPInTmem ? 32 : 0) <= 256, "half of the tensor memory");
};

constexpr uint32_t kTmemCols = 256;

struct Maps {
  CUtensorMap k3, v3;  // [entries][H_kv][row], boxes of 16 to 64 entries
  CUtensorMap k2, v2;  // [entries * H_kv][row], single rows (gathers)
};

struct Ctx : UnitTable {
  uint8_t* smem;
  uint32_t sbase, bars;
  volatile int* abort_flag;
  int32_t* err;
};

// Bounded wait that also gives up when another role has.
__device__ __forceinline__ bool wait_bar(const Ctx& c, int i, uint32_t parity,
                                         unsigned long long limit_ns = kWaitLimitNs) {
  const uint32_t bar = c.bars + 8 * i;
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*c.abort_flag) return false;
      if (globaltimer_ns() - t0 > limit_ns) {
        report(c.err, DA_DEVERR_TIMEOUT);
        *c.abort_flag = 1;
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool wait_warp(const Ctx& c, int i, uint32_t parity) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(c, i, parity) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

__device__ __forceinline__ void arrive_warp(const Ctx& c, int i) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(c.bars + 8 * i);
}

// 16 columns of tensor memory from registers (32 lanes)
__device__ __forceinline__ void st_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ------------------------------------------------------------------ copies

__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* tm, int col, const int (&r)[4],
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(col), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}

// Two warps; warp w fills the stages of its parity (a copy costs its thread some 200
// cycles to issue).  box > 0: the list's entries lie `box` at a time (64, 32 or 16) in
// consecutive cache rows, one copy each for K and V (and 64 dims); the lookups of eight
// tiles are made at once, lane l those of group l % 4 of tile l / 4, a batch ahead of
// the copies that use them.  box = 0: gathers of four rows, lane l < 16 those of entries
// 4 l .. 4 l + 3, looked up a tile ahead.  Entries that no node sees, and those whose page is out
// of range, are not looked up; cache row 0 is copied instead, so that no stage byte is
// left uninitialised (their weights are zero and their values made zero).
template <int KT, int D>
__device__ void producer(const TreeLaunch& p, const Ctx& c, const Maps& m, int box) {
  using L = Lay<KT, D>;
  constexpr int kNS = L::Q8 ? L::kRawStages : L::kStages;
  constexpr int kFullB = L::Q8 ? L::kRawFull : L::kFull, kEmptyB = L::Q8 ? L::kRawEmpty : L::kEmpty;
  constexpr int kHalves = L::Q8 ? 1 : D / 64;      // copies of a row
  constexpr uint32_t kTx = L::Q8 ? 2 * kT * L::kCodeRow : L::kStage;
  const int lane = threadIdx.x & 31;
  const uint32_t pw = (threadIdx.x >> 5) & 1;
  bool bad = false;
  // cache row of entry j, the first of n of a tile's (0 where no node sees one of them)
  auto look_up = [&](const Unit& x, int j, int n) -> int {
    if (j >= x.r.end || (j >= x.r.hole_from && j + n <= x.r.hole_to)) return 0;
    if (p.layout == DA_KV_CONTIGUOUS) return x.b * p.width + j;
    const int at = p.layout == DA_KV_PAGED ? quotient(j, p.by_page) : j;
    const int word = __ldg(p.table + (long long)x.b * p.width + at);
    if (word < 0 || word >= p.num_blocks) {
      bad = true;
      return 0;
    }
    return p.layout == DA_KV_PAGED ? word * p.page_size + (j - at * p.page_size) : word;
  };
  const int groups = box ? kT / box : 0;
  // this lane's row for tiles 8 bt .. 8 bt + 7 of a unit
  auto batch = [&](const Unit& x, int bt) -> int {
    const int i = x.begin + 8 * bt + (lane >> 2);
    if (i >= x.end || (lane & 3) >= groups) return 0;
    return look_up(x, tree_tile(x.r, i) * kT + (lane & 3) * box, box);
  };
  uint32_t g = 0;
  bool alive = true;
  Unit x = unit_of(p, c, blockIdx.x);
  int first_rows = box ? batch(x, 0) : 0;
  for (int u = blockIdx.x; u < c.units && alive; u += gridDim.x) {
    const bool more = u + (int)gridDim.x < c.units;
    const Unit next = more ? unit_of(p, c, u + gridDim.x) : x;
    const int n = x.tiles(), last_batch = (n - 1) / 8;
    int rows = first_rows, ahead = 0;
    if (box && n > 8) ahead = batch(x, 1);
    if (box && more && n <= 8) first_rows = batch(next, 0);
    int rg[4] = {0, 0, 0, 0}, rg_next[4] = {0, 0, 0, 0};
    if (!box && lane < 16 && n > 0)
      for (int e = 0; e < 4; ++e) rg[e] = look_up(x, tree_tile(x.r, x.begin) * kT + lane * 4 + e, 1);
    for (int i = 0; i < n; ++i, ++g) {
      const uint32_t st = g % kNS, full = c.bars + 8 * (kFullB + st);
      if (box) {
        if (i > 0 && (i & 7) == 0) {
          rows = ahead;
          if ((i >> 3) < last_batch) ahead = batch(x, (i >> 3) + 1);
          if ((i >> 3) == last_batch && more) first_rows = batch(next, 0);
        }
        if ((st & 1) != pw) continue;  // the other warp's
      } else {
        if (lane < 16 && i + 1 < n) {
          const int j1 = tree_tile(x.r, x.begin + i + 1) * kT;
          for (int e = 0; e < 4; ++e) rg_next[e] = look_up(x, j1 + lane * 4 + e, 1);
        }
        if ((st & 1) != pw) {
          for (int e = 0; e < 4; ++e) rg[e] = rg_next[e];
          continue;
        }
      }
      if (!wait_warp(c, kEmptyB + st, ((g / kNS) & 1) ^ 1)) {
        alive = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(full, kTx);
      __syncwarp();
      const uint32_t kdst = c.sbase + (L::Q8 ? L::kRawOffset + st * L::kRawStage : st * L::kStage);
      const uint32_t vdst = kdst + (L::Q8 ? kT * L::kCodeRow : L::kTile);
      constexpr int kRowBytes = L::Q8 ? L::kCodeRow : 128;  // of a row in the stage (of a half)
      if (box) {
        const int grp = lane & 3;
        if ((lane >> 2) == (i & 7) && grp < groups) {
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            const uint32_t off = half * kRegion + grp * box * kRowBytes;
            tma_box3(kdst + off, &m.k3, 64 * half, x.h, rows, full);
            tma_box3(vdst + off, &m.v3, 64 * half, x.h, rows, full);
          }
        }
      } else if (lane < 16) {
        int at[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) at[e] = rg[e] * p.H_kv + x.h;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          const uint32_t off = half * kRegion + lane * 4 * kRowBytes;
          tma_gather4(kdst + off, &m.k2, 64 * half, at, full);
          tma_gather4(vdst + off, &m.v2, 64 * half, at, full);
        }
      }
      if constexpr (KT == DA_KV_NVFP4) {
        // block scales of entries 2 lane and 2 lane + 1: K's rows, then V's
        const long long blocks = p.kv_rows * p.H_kv * (D / 2);
        const uint32_t sdst = kdst + 2 * kT * L::kCodeRow;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = 2 * lane + e;
          long long at;
          if (box) {
            const int base = __shfl_sync(0xffffffffu, rows, (i & 7) * 4 + k / box);
            at = min((long long)base + k % box, p.kv_rows - 1);
          } else {
            const int a = __shfl_sync(0xffffffffu, rg[e], k >> 2);
            const int b = __shfl_sync(0xffffffffu, rg[2 + e], k >> 2);
            at = (k & 2) ? b : a;
          }
          if (p.kv_rows > 0) {
            const long long off = blocks + (at * p.H_kv + x.h) * L::kScaleRow;
            const uint32_t to = sdst + k * L::kScaleRow;
            if constexpr (L::kScaleRow == 8) {
              cp_async8(to, static_cast<const uint8_t*>(p.k) + off);
              cp_async8(to + kT * L::kScaleRow, static_cast<const uint8_t*>(p.v) + off);
            } else {
              cp_async4(to, static_cast<const uint8_t*>(p.k) + off);
              cp_async4(to + kT * L::kScaleRow, static_cast<const uint8_t*>(p.v) + off);
            }
          }
        }
        cp_async_mbar_arrive(full);
      }
      if (!box)
        for (int e = 0; e < 4; ++e) rg[e] = rg_next[e];
    }
    x = next;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.err, DA_DEVERR_INDEX);
  if constexpr (KT == DA_KV_NVFP4) cp_async_wait_all();
  // Leave no copy in flight (after a time-out; else every stage was consumed): each of this
  // warp's stages has its last tile before g, which is the first that it did not copy.
  if (lane == 0) {
    for (uint32_t st = pw; st < kNS; st += 2) {
      if (g <= st) continue;
      const uint32_t last = g - 1 - (g - 1 - st) % kNS;
      if (!mbar_wait(c.bars + 8 * (kFullB + st), (last / kNS) & 1)) report(p.err, DA_DEVERR_TIMEOUT);
    }
  }
}

// ------------------------------------------------------------------ conversion
// Four warps.  E4M3 values are f16 values, and so are NVFP4 elements (a code times its
// block scale, multiplied in f16), so K and V become f16 without error.
template <int KT, int D>
__device__ void converter(const TreeLaunch& p, const Ctx& c) {
  using L = Lay<KT, D>;
  constexpr int kPieces = D / 16;               // 16-dim pieces of a row
  constexpr int kTimes = KT == DA_KV_NVFP4 ? 1 : 2;
  constexpr int kStep = 128 / kPieces;          // rows between a thread's
  const int ct = threadIdx.x - 8 * 32;
  const int jj = ct % kPieces, r0 = ct / kPieces;
  uint32_t g = 0;
  for (int u = blockIdx.x; u < c.units; u += gridDim.x) {
    const Unit x = unit_of(p, c, u);
    for (int i = 0; i < x.tiles(); ++i, ++g) {
      const int rs = g % L::kRawStages, os = g % L::kStages;
      if (!wait_warp(c, L::kRawFull + rs, (g / L::kRawStages) & 1)) return;
      if (!wait_warp(c, L::kEmpty + os, ((g / L::kStages) & 1) ^ 1)) return;
      const uint8_t* raw = c.smem + L::kRawOffset + rs * L::kRawStage;
      uint8_t* op = c.smem + os * L::kStage;
      // (rolled for NVFP4, whose code is long: 517 against 553 us for 64 rows of 16 nodes with 4096
      // entries each; E4M3 takes 411 rolled, 397 unrolled)
#pragma unroll kTimes
      for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
        for (int q = 0; q < kT / kStep; ++q) {
          const int row = r0 + kStep * q;
          uint32_t h[8];  // dims 16 jj .. 16 jj + 15
          const uint8_t* codes = raw + kv * kT * L::kCodeRow + row * L::kCodeRow;
          if constexpr (KT == DA_KV_NVFP4) {
            const uint2 w = *reinterpret_cast<const uint2*>(codes + jj * 8);
            const uint32_t block = raw[2 * kT * L::kCodeRow + (kv * kT + row) * L::kScaleRow + jj];
            const uint32_t s2 = __byte_perm(e4m3x2_to_f16x2(block), 0, 0x1010);
            uint32_t lo[4], hi[4];
            e2m1x8_to_f16x2(w.x, lo);
            e2m1x8_to_f16x2(w.y, hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              h[e] = hmul2(lo[e], s2);
              h[4 + e] = hmul2(hi[e], s2);
            }
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(codes + jj * 16);
            const uint32_t wb[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              h[2 * e] = e4m3x2_to_f16x2(wb[e]);
              h[2 * e + 1] = e4m3x2_to_f16x2(wb[e] >> 16);
            }
          }
          // region jj / 4, chunks 2 (jj % 4) and + 1, in an order that spreads the banks
          uint8_t* to = op + kv * L::kTile + (jj >> 2) * kRegion + row * 128;
          const int ch = 2 * (jj & 3), sw = (jj >> 2) & 1;
          const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
          *reinterpret_cast<uint4*>(to + (((ch + sw) ^ (row & 7)) << 4)) = sw ? hi : lo;
          *reinterpret_cast<uint4*>(to + (((ch + 1 - sw) ^ (row & 7)) << 4)) = sw ? lo : hi;
        }
      }
      fence_proxy_async();
      arrive_warp(c, L::kFull + os);
      arrive_warp(c, L::kRawEmpty + rs);
    }
  }
}

// ------------------------------------------------------------------ MMAs
// Two threads: one issues S = Q K^T of a tile as soon as it is there and the softmax has
// read the scores before it, so that the softmax finds the next ones waiting; the other
// O += P V when the softmax has written P.
template <int KT, int D>
__device__ void issue_s(const TreeLaunch& p, const Ctx& c, uint32_t tmem) {
  using L = Lay<KT, D>;
  constexpr uint32_t kIdesc = L::Q8 ? umma::idesc_f16_f32(kRows, kT, false) : umma::idesc_bf16_f32(kRows, kT, false);
  const uint64_t k0 = umma::smem_desc(c.sbase, 16, 1024, umma::kSwizzle128B);
  if (p.test_stall && !wait_bar(c, L::kStall, 0, kTestStallNs)) return;
  uint32_t g = 0, nu = 0;
  for (int u = blockIdx.x; u < c.units; u += gridDim.x) {
    const int n = unit_of(p, c, u).tiles();
    if (n == 0) continue;
    if (!wait_bar(c, L::kQFull, nu++ & 1)) return;
    for (int i = 0; i < n; ++i, ++g) {
      const uint32_t st = g % L::kStages;
      const uint64_t kd = k0 + (uint64_t)((st * L::kStage) >> 4);
      if (!wait_bar(c, L::kFull + st, (g / L::kStages) & 1)) return;
      if (g && !wait_bar(c, L::kSFree, (g - 1) & 1)) return;
      umma::fence_after_sync();
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        umma::mma_bf16_ta(tmem + L::kSCol, tmem + L::kQCol + k * 8,
                          kd + (uint64_t)(((k / 4) * kRegion + (k % 4) * 32) >> 4), kIdesc, k ? 1u : 0u);
      umma::commit(c.bars + 8 * L::kSFull);
    }
  }
}

template <int KT, int D>
__device__ void issue_pv(const TreeLaunch& p, const Ctx& c, uint32_t tmem) {
  using L = Lay<KT, D>;
  constexpr uint32_t kIdesc = L::Q8 ? umma::idesc_f16_f32(kRows, D, true) : umma::idesc_bf16_f32(kRows, D, true);
  const uint64_t p0 = umma::smem_desc(c.sbase, 16, 1024, umma::kSwizzle128B);
  // V with its dims contiguous: 64-dim regions kRegion apart, 8-entry groups 1024 bytes
  const uint64_t v0 = umma::smem_desc(c.sbase + L::kTile, kRegion, 1024, umma::kSwizzle128B);
  uint32_t g = 0;
  for (int u = blockIdx.x; u < c.units; u += gridDim.x) {
    const int n = unit_of(p, c, u).tiles();
    for (int i = 0; i < n; ++i, ++g) {
      const uint32_t st = g % L::kStages;
      const uint64_t at = (uint64_t)((st * L::kStage) >> 4);
      if (!wait_bar(c, L::kPFull, g & 1)) return;
      umma::fence_after_sync();
#pragma unroll
      for (int k = 0; k < kT / 16; ++k) {
        const uint64_t vd = v0 + at + (uint64_t)((k * 2048) >> 4);
        const uint32_t more = k ? 1u : i > 0;
        if constexpr (L::kPInTmem)
          umma::mma_bf16_ta(tmem + L::kOCol, tmem + L::kPCol + k * 8, vd, kIdesc, more);
        else
          umma::mma_bf16(tmem + L::kOCol, p0 + at + (uint64_t)((k * 32) >> 4), vd, kIdesc, more);
      }
      umma::commit(c.bars + 8 * L::kPVDone);
      umma::commit(c.bars + 8 * (L::kEmpty + st));
    }
  }
}

// ------------------------------------------------------------------ softmax and output

// The row of a unit that a thread has.
struct Lane {
  int t, head;   // node, query head
  uint32_t row;  // of q, out and lse
  bool live;
};

__device__ __forceinline__ Lane lane_of(const TreeLaunch& p, const Unit& x, int at) {
  Lane y;
  y.live = at < x.rows;
  const int idx = x.row0 + at;
  y.t = y.live ? quotient(idx, p.by_group) : 0;
  y.head = x.h * p.G + (y.live ? idx - y.t * p.G : 0);
  y.row = ((uint32_t)x.b * p.T + y.t) * p.H_q + y.head;
  return y;
}

// Byte of 16-byte chunk `ch` of row `row` in 32 rows of 64 bytes whose chunks are swapped so
// that neither a warp's rows nor its columns meet in a bank.
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) { return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4); }

// A warp's 32 rows of Q into tensor memory: bf16 as they are, or f16 scaled by a power of
// two.  Four lanes load a row, 32 dims at a time, and it changes hands by way of `pass` (a
// thread that loads its own row keeps the L1 busy for several times as long).  Returns
// the row's softmax scale.
template <int KT, int D>
__device__ __forceinline__ float put_q(const TreeLaunch& p, const Lane& y, int lane, uint32_t q_col, uint8_t* pass) {
  using L = Lay<KT, D>;
  constexpr int kParts = D / 32;
  const uint32_t live = __ballot_sync(0xffffffffu, y.live);
  uint4 w[kParts][4];  // this lane's pieces of rows 8 i + lane / 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t row = __shfl_sync(0xffffffffu, y.row, 8 * i + (lane >> 2));
    const uint4* from = reinterpret_cast<const uint4*>(p.q + (size_t)row * D) + (lane & 3);
    const bool there = live >> (8 * i + (lane >> 2)) & 1;
#pragma unroll
    for (int part = 0; part < kParts; ++part) w[part][i] = there ? __ldg(from + 4 * part) : make_uint4(0, 0, 0, 0);
  }
  float sc = 1.f, row_scale = p.scale_log2;
  if constexpr (L::Q8) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t top = 0;
#pragma unroll
      for (int part = 0; part < kParts; ++part) top = bf16x8_absmax_bits(top, w[part][i]);
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // row 8 i + j lies with lanes 4 j .. 4 j + 3
      const uint32_t v = __shfl_sync(0xffffffffu, top, (lane & 7) * 4);
      if (i == lane >> 3) most = v;
    }
    const int e = q_prescale_exp(bf16_absmax_value(most));
    sc = exp2_int(e);
    row_scale *= exp2_int(-e);
  }
#pragma unroll
  for (int part = 0; part < kParts; ++part) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(pass + chunk_at(8 * i + (lane >> 2), lane & 3)) = w[part][i];
    __syncwarp();
    uint32_t q16[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 own = *reinterpret_cast<const uint4*>(pass + chunk_at(lane, i));
      const uint32_t v[4] = {own.x, own.y, own.z, own.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (L::Q8) {
          const __half2 hh = __floats2half2_rn(bf16_lo(v[e]) * sc, bf16_hi(v[e]) * sc);
          q16[4 * i + e] = *reinterpret_cast<const uint32_t*>(&hh);
        } else {
          q16[4 * i + e] = v[e];
        }
      }
    }
    st_16(q_col + part * 16, q16);
  }
  umma::wait_st();
  return row_scale;
}

// Four warps; a thread has one row, a TMEM lane.  Its scores' running reference value moves
// only when one exceeds it by more than 2^8 (then its O is rescaled).  Between units a warp
// brings in its rows' Q and writes its rows' output, by itself; the SM's other block fills
// that time.
template <int KT, int D>
__device__ void softmax_warps(const TreeLaunch& p, const Ctx& c, uint32_t tmem) {
  using L = Lay<KT, D>;
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t s_col = base + L::kSCol, o_col = base + L::kOCol;
  uint8_t* pass = c.smem + L::kPass + warp * 2048;
  // A unit's description stays in shared memory: the loop over tiles has no register for
  // what is needed before and behind it.
  Unit* units = reinterpret_cast<Unit*>(c.smem + L::kUnits) + 2 * warp;
  auto begin_unit = [&](int u, Unit* to) -> float {
    const Unit z = unit_of(p, c, u);
    if (lane == 0) *to = z;
    __syncwarp();
    const float scale = put_q<KT, D>(p, lane_of(p, z, tid), lane, base + L::kQCol, pass);
    umma::fence_before_sync();
    if (z.tiles() > 0) arrive_warp(c, L::kQFull);
    return scale;
  };
  uint32_t g = 0;
  float row_scale = begin_unit(blockIdx.x, units);
  for (int u = blockIdx.x, slot = 0; u < c.units; u += gridDim.x, slot ^= 1) {
    const Unit* x = units + slot;
    const int begin = x->begin, end = x->end, length = x->r.length, head = x->r.head_tiles, skip = x->r.skip;
    const bool live = tid < x->rows;
    // tiles from here on are seen whole, up to the end of the context
    const int whole = p.window ? length + x->r.nodes - p.window : 0;
    // ---- what the row sees, if the unit's last tile reaches the nodes or there is a window
    unsigned long long anc = 0;
    int depth = 0;
    if (live && end > begin && (p.window || ((end - 1 < head ? end : end + skip) * kT > length))) {
      anc = windowed(p, x->r, ancestors(p, x->b, quotient(x->row0 + tid, p.by_group), &depth), depth);
      anc &= low_bits(x->r.end - length);
    }
    float m_used = -INFINITY, l = 0.f;
    for (int i = begin; i < end; ++i, ++g) {
      if (!wait_warp(c, L::kSFull, g & 1)) return;
      umma::fence_after_sync();
      float s[kT];
      umma::ld_32x32b_x32(s_col, *reinterpret_cast<float(*)[32]>(s));
      umma::ld_32x32b_x32(s_col + 32, *reinterpret_cast<float(*)[32]>(s + 32));
      umma::wait_ld();
      umma::fence_before_sync();
      arrive_warp(c, L::kSFree);
      const int j0 = (i < head ? i : i + skip) * kT;
      const bool all = j0 + kT <= length && (j0 >= whole || j0 + kT <= p.sinks);
      const float factor = row_scale > 0.f ? row_scale : 1.f;
      if (row_scale <= 0.f) {  // (the largest score is not the largest product then)
#pragma unroll
        for (int k = 0; k < kT; ++k) s[k] *= row_scale;
      }
      if (!all) {
        unsigned long long vis = low_bits(length - j0);
        if (p.window) vis &= ~low_bits(length + depth - p.window + 1 - j0) | low_bits(p.sinks - j0);
        const int shift = length - j0;  // of node 0 in the tile
        if (shift > -64 && shift < 64) vis |= shift >= 0 ? anc << shift : anc >> -shift;
        if (!live) vis = 0;
#pragma unroll
        for (int k = 0; k < kT; ++k)
          if (!(vis >> k & 1)) s[k] = -INFINITY;
      }
      float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int k = 4; k < kT; ++k) m4[k & 3] = fmaxf(m4[k & 3], s[k]);
      float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * factor;
      if constexpr (L::Q8) mt -= kHeadLog2;
      const bool move = mt > m_used + kRescaleLog2 || (m_used == -INFINITY && mt > -INFINITY);
      const float m_new = move ? mt : m_used;
      const float alpha = (move && m_used > -INFINITY) ? ex2(m_used - m_new) : 1.f;
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      // 2^(s scale - ref), in pairs; four sums
      const uint64_t factor2 = pack2(factor, factor), ref2 = pack2(-ref, -ref);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pk[kT / 2];
#pragma unroll
      for (int k = 0; k < kT; k += 2) {
        float p0, p1;
        unpack2(ffma2(pack2(s[k], s[k + 1]), factor2, ref2), p0, p1);
        p0 = ex2(p0);
        p1 = ex2(p1);
        sum[k & 2] += p0;
        sum[(k & 2) + 1] += p1;
        if constexpr (L::Q8) {
          const __half2 h = __floats2half2_rn(p0, p1);
          pk[k / 2] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
          pk[k / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      l = fmaf(l, alpha, (sum[0] + sum[1]) + (sum[2] + sum[3]));
      m_used = m_new;
      const uint32_t st = g % L::kStages;
      if constexpr (!L::kPInTmem) {  // over the tile's K, which S has read: 64 weights, 128 bytes a row
        uint8_t* to = c.smem + st * L::kStage + tid * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(to + ((k ^ (tid & 7)) << 4)) =
              make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
      }
      // the P V before has been done: O stands still
      if (g && !wait_warp(c, L::kPVDone, (g - 1) & 1)) return;
      umma::fence_after_sync();
      if constexpr (L::kPInTmem) umma::st_32x32b_x32_u(base + L::kPCol, pk);
      if (i > begin && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          float o[32];
          umma::ld_32x32b_x32(o_col + ch * 32, o);
          umma::wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= alpha;
          umma::st_32x32b_x32(o_col + ch * 32, o);
        }
      }
      // values of entries that no node sees: zero times what lies there could be a NaN
      const unsigned long long hid = all ? 0 : hidden_bits(x->r, j0);
      if (hid) {
        const int k = tid >> 1;
        if (!wait_warp(c, L::kFull + st, (g / L::kStages) & 1)) return;  // (it has been: this orders the stores)
        if (hid >> k & 1) {
          uint8_t* v = c.smem + st * L::kStage + L::kTile + k * 128 + (D == 128 ? (tid & 1) * kRegion : (tid & 1) * 64);
#pragma unroll
          for (int e = 0; e < (D == 128 ? 8 : 4); ++e) reinterpret_cast<uint4*>(v)[e] = make_uint4(0, 0, 0, 0);
        }
      }
      if (!L::kPInTmem || hid) fence_proxy_async();
      umma::wait_st();
      umma::fence_before_sync();
      arrive_warp(c, L::kPFull);
    }
    // ---- the next unit's Q, whose scores can then be formed, and this one's output
    if (end > begin && !wait_warp(c, L::kPVDone, (g - 1) & 1)) return;
    umma::fence_after_sync();
    if (u + (int)gridDim.x < c.units) row_scale = begin_unit(u + gridDim.x, units + (slot ^ 1));
    const Unit done = *x;
    const Lane mine = lane_of(p, done, tid);
    const bool single = done.r.splits == 1;
    // rows of the partials against those of q and out
    const long long to_slot = (((long long)done.b * p.max_splits + done.split) - done.b) * p.T * p.H_q;
    const uint32_t lives = __ballot_sync(0xffffffffu, mine.live);
    const float inv = (l > 0.f ? 1.f / l : l != l ? l : 0.f) * p.v_scale;
    bool odd = l != l;  // something that is not finite
#pragma unroll 1
    for (int ch = lives ? 0 : D / 16; ch < D / 16; ++ch) {
      float o[16];
      umma::ld_32x32b_x16(o_col + ch * 16, o);
      umma::wait_ld();
      float top = 0.f;  // (a sum of magnitudes: infinite or NaN if one of them is)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        o[k] = done.tiles() > 0 ? o[k] * inv : 0.f;
        top += fabsf(o[k]);
      }
      odd |= !(top < INFINITY);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4*>(pass + chunk_at(lane, k)) =
            make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      __syncwarp();
      uint32_t row[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // four lanes write a row
        row[k] = __shfl_sync(0xffffffffu, mine.row, 8 * k + (lane >> 2));
        v[k] = *reinterpret_cast<const float4*>(pass + chunk_at(8 * k + (lane >> 2), lane & 3));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool there = lives >> (8 * k + (lane >> 2)) & 1;
        if (single) {
          const __nv_bfloat162 h0 = __floats2bfloat162_rn(v[k].x, v[k].y), h1 = __floats2bfloat162_rn(v[k].z, v[k].w);
          const uint2 h = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
          if (there) reinterpret_cast<uint2*>(p.out + (size_t)row[k] * D + ch * 16)[lane & 3] = h;
        } else if (there) {
          reinterpret_cast<float4*>(p.o_part + (to_slot + row[k]) * D + ch * 16)[lane & 3] = v[k];
        }
      }
    }
    if (mine.live) {
      const float lse = l > 0.f || l != l ? m_used + lg2(l) : -INFINITY;
      if (single)
        p.lse[mine.row] = lse * kLn2;
      else
        p.lse_part[to_slot + mine.row] = lse;
    }
    // A value that some node sees and another does not may have been infinite or NaN: zero
    // times it has spoiled the other's sum.  Such rows are formed again, entry by entry.
    __syncwarp();
    for (uint32_t again = __ballot_sync(0xffffffffu, mine.live && odd); again; again &= again - 1) {
      const int src = __ffs((int)again) - 1;
      const int t = __shfl_sync(0xffffffffu, mine.t, src), head = __shfl_sync(0xffffffffu, mine.head, src);
      const uint32_t row = __shfl_sync(0xffffffffu, mine.row, src);
      float m2, l2, o[D / 32];
      attend_plainly<KT, D>(p, done.r, done.b, t, head, done.begin, done.end, lane, &m2, &l2, o);
      const float inv2 = (l2 > 0.f ? 1.f / l2 : l2 != l2 ? l2 : 0.f) * p.v_scale;
      const float lse2 = l2 > 0.f || l2 != l2 ? m2 + lg2(l2) : -INFINITY;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const int d = lane * (D / 32) + e;
        if (single)
          p.out[(size_t)row * D + d] = __float2bfloat16_rn(o[e] * inv2);
        else
          p.o_part[(to_slot + row) * D + d] = o[e] * inv2;
      }
      if (lane == 0) {
        if (single)
          p.lse[row] = lse2 * kLn2;
        else
          p.lse_part[to_slot + row] = lse2;
      }
      __syncwarp();
    }
    umma::fence_before_sync();
  }
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void leave_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int KT, int D>
__global__ void __launch_bounds__(Lay<KT, D>::kThreads, 2)
    tree_kernel(const TreeLaunch p, const __grid_constant__ Maps maps, int box) {
  using L = Lay<KT, D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctx c;
  c.smem = smem;
  c.sbase = smem_addr(smem);
  c.bars = c.sbase + L::kBarOffset;
  c.abort_flag = reinterpret_cast<volatile int*>(smem + L::kSlots + 4);
  c.err = p.err;
  int2* sizes = reinterpret_cast<int2*>(smem + L::kSizes);
  int* first = reinterpret_cast<int*>(smem + L::kFirst);
  c.sizes = sizes;
  c.first = first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kBars; ++i) {
      uint32_t count = 1;  // tcgen05.commit, or the producer's expect_tx arrive
      if (i >= L::kFull && i < L::kFull + L::kStages && L::Q8) count = 4;
      if (i >= L::kRawFull && i < L::kRawFull + L::kRawStages && KT == DA_KV_NVFP4) count = 33;
      if (i >= L::kRawEmpty && i < L::kRawEmpty + L::kRawStages) count = 4;
      if (i == L::kQFull || i == L::kSFree || i == L::kPFull) count = 4;
      if (i == L::kDrain) count = 2;
      mbar_init(c.bars + 8 * i, count);
    }
    *c.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    umma::tmem_alloc(c.sbase + L::kSlots, kTmemCols);
    umma::tmem_relinquish();
  }
  wait_prior_grid();
  allow_next_grid();
  count_units<false>(p, sizes, first, L::kThreads);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  c.units = first[p.rows];
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kSlots);
  const bool aligned = (c.sbase & 1023u) == 0;  // as the swizzled layouts need it
  if (!aligned && threadIdx.x == 0) report(p.err, DA_DEVERR_TIMEOUT);

  if ((int)blockIdx.x < c.units && aligned) {
    if (warp < 4) {
      if constexpr (L::Q8) take_registers<L::kSoftmaxRegs>();
      softmax_warps<KT, D>(p, c, tmem);
    } else if (warp < 8) {
      if constexpr (L::Q8) leave_registers<L::kIssueRegs>();
      if (warp >= 6) {
        producer<KT, D>(p, c, maps, box);
      } else if (lane == 0) {
        if (warp == 4)
          issue_s<KT, D>(p, c, tmem);
        else
          issue_pv<KT, D>(p, c, tmem);
        umma::commit(c.bars + 8 * L::kDrain);  // arrives when all MMAs of this thread are done
      }
    } else {
      if constexpr (L::Q8) {
        leave_registers<L::kConvertRegs>();
        converter<KT, D>(p, c);
      }
    }
    __syncwarp();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (warp == 4 && lane == 0) {
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(c.bars + 8 * L::kDrain, 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          report(p.err, DA_DEVERR_TIMEOUT);
          break;
        }
      }
    }
    __syncwarp();
  }
  if (warp == 4) umma::tmem_dealloc(tmem, kTmemCols);
}

constexpr int kCombineWarps = 4;

// A warp for each (row, node, head) of several splits: their partials merged in split
// order (the arithmetic is in merge.cuh).
template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const TreeLaunch p) {
  constexpr int N = D / 32;
  constexpr int kBatch = 8;  // partials in flight
  __shared__ float coef[kCombineWarps][kTreeMaxSplits];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * kCombineWarps + warp;
  const long long per = (long long)p.T * p.H_q;
  if (task >= p.B * per) return;
  const int b = (int)(task / per);
  const long long th = task - b * per;
  int bad = 0;  // (reported by the kernel before)
  const int2 size = tree_size(p, b, &bad);
  const TreeRow r = tree_row(p, size.x, size.y);
  if (th / p.H_q >= r.nodes || r.splits <= 1) return;
  const long long slot = (long long)b * p.max_splits * per + th;
  float part[kBatch][N], acc[N];
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i >= r.splits) continue;
      const float* from = p.o_part + (slot + (s0 + i) * per) * D + lane * N;
      if constexpr (N == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(from));
        part[i][0] = x.x, part[i][1] = x.y, part[i][2] = x.z, part[i][3] = x.w;
      } else {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(from));
        part[i][0] = x.x, part[i][1] = x.y;
      }
    }
  };
  load(0);
  float lse = merge_weights(p.lse_part + slot, per, r.splits, coef[warp], lane);
  bool nan = false;  // (the merge would count such a part as empty)
  for (int i = lane; i < r.splits; i += 32) {
    const float part_lse = __ldcg(p.lse_part + slot + i * per);
    nan |= part_lse != part_lse;
  }
  if (__any_sync(0xffffffffu, nan)) lse = NAN;
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = lse != lse ? NAN : 0.f;
  for (int s0 = 0; s0 < r.splits; s0 += kBatch) {
    if (s0) load(s0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i >= r.splits) continue;
      const float c = coef[warp][s0 + i];
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = fmaf(c, part[i][e], acc[e]);
    }
  }
  uint32_t w[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  uint32_t* to = reinterpret_cast<uint32_t*>(p.out + task * D) + lane * (N / 2);
  if constexpr (N == 4)
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  else
    *to = w[0];
  if (lane == 0) p.lse[task] = lse;
}

// ------------------------------------------------------------------ launches

// Stands in for an empty cache in a tensor map (nothing of it is used).
__device__ __align__(128) __nv_bfloat16 g_nothing[128];

template <int KT, int D>
cudaError_t launch_shape(const TreeLaunch& p0, int sms, cudaStream_t stream) {
  using L = Lay<KT, D>;
  const cudaError_t attr = allow_smem(tree_kernel<KT, D>, L::kBytes);
  if (attr != cudaSuccess) return attr;
  TreeLaunch p = p0;
  // entries that lie together for sure, as many as a copy takes
  const int box = p.layout == DA_KV_CONTIGUOUS                          ? 64
                  : p.layout == DA_KV_INDEXED || p.page_size % 16 != 0 ? 0
                  : p.page_size % 64 == 0                               ? 64
                  : p.page_size % 32 == 0                               ? 32
                                                                        : 16;
  const void* k = p.k;
  const void* v = p.v;
  cuuint64_t rows = (cuuint64_t)p.kv_rows, heads = (cuuint64_t)p.H_kv;
  if (rows < 1) {
    void* z = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&z, g_nothing);
    if (e != cudaSuccess) return e;
    k = v = z;
    rows = heads = 1;
  }
  const cuuint64_t row = L::Q8 ? L::kCodeRow : D, size = L::Q8 ? 1 : 2;
  const cuuint32_t across = L::Q8 ? L::kCodeRow : 64;
  const CUtensorMapSwizzle swizzle = L::Q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
  Maps m;
  std::memset(&m, 0, sizeof(m));
  if (box) {
    const cuuint64_t dims[3] = {row, heads, rows}, strides[2] = {row * size, heads * row * size};
    const cuuint32_t bx[3] = {across, 1, (cuuint32_t)box};
    if (!tree_tensor_map(&m.k3, k, 3, dims, strides, bx, L::Q8, swizzle) || !tree_tensor_map(&m.v3, v, 3, dims, strides, bx, L::Q8, swizzle))
      return cudaErrorInvalidValue;
  } else {
    const cuuint64_t dims[2] = {row, rows * heads}, strides[1] = {row * size};
    const cuuint32_t bx[2] = {across, 1};
    if (!tree_tensor_map(&m.k2, k, 2, dims, strides, bx, L::Q8, swizzle) || !tree_tensor_map(&m.v2, v, 2, dims, strides, bx, L::Q8, swizzle))
      return cudaErrorInvalidValue;
  }
  const int supers = (p.T * p.G + kTreeSuper - 1) / kTreeSuper;
  p.by_heads = fast_div(p.H_kv);
  p.by_group = fast_div(p.G);
  p.by_page = fast_div(std::max(p.page_size, 1));
  for (p.row0 = 0; p.row0 < p.B; p.row0 += kTreeRows) {
    p.rows = std::min(kTreeRows, p.B - p.row0);
    const long long most = (long long)p.rows * p.max_splits * p.H_kv * supers;
    const cudaError_t e = launch_after(tree_kernel<KT, D>, dim3((unsigned)std::min<long long>(most, 2 * sms)),
                                       dim3(L::kThreads), (size_t)L::kBytes, stream, p, m, box);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int KT>
cudaError_t launch_kt(const TreeLaunch& p, int sms, cudaStream_t stream) {
  return p.D == 64 ? launch_shape<KT, 64>(p, sms, stream) : launch_shape<KT, 128>(p, sms, stream);
}

}  // namespace

cudaError_t launch_tree(const TreeLaunch& p, int sms, cudaStream_t stream) {
  if (tree_takes_few(p.kv_type, p.D, p.T * p.G)) return launch_tree_few(p, sms, stream);
  switch (p.kv_type) {
    case DA_KV_FP8_E4M3: return launch_kt<DA_KV_FP8_E4M3>(p, sms, stream);
    case DA_KV_NVFP4: return launch_kt<DA_KV_NVFP4>(p, sms, stream);
    default: return launch_kt<DA_KV_BF16>(p, sms, stream);
  }
}

cudaError_t launch_tree_combine(const TreeLaunch& p, cudaStream_t stream) {
  const long long warps = (long long)p.B * p.T * p.H_q;
  const dim3 grid((unsigned)((warps + kCombineWarps - 1) / kCombineWarps));
  return p.D == 64 ? launch_after(tree_combine_kernel<64>, grid, dim3(kCombineWarps * 32), 0, stream, p)
                   : launch_after(tree_combine_kernel<128>, grid, dim3(kCombineWarps * 32), 0, stream, p);
}

}  // namespace da
