// Tree attention of few (node, head) rows a KV head: a plain decode step's, or those of a short
// chain or small tree.
//
// Tiles of 128 rows would be empty for the most part, and their way through tensor memory as
// long.  Here each warp forms transposed products with m16n8k16: S^T = K Q^T and O^T += V^T P^T,
// 16 entries of K (or 16 dims of V) on the wide side and 8 rows on the narrow one.  The order of
// the dims in Q K^T, and of the entries in P V, is free, so a lane takes chunks of a cache row
// just as they lie in memory, widens them in registers, and holds the right operand: no value
// changes hands but the weights, by one 8 x 8 transpose, rounded to the values' type as in
// tree.cu.  A row's reference value and sum lie with the lanes that have its weights and its output.
//
// A block has a unit of a list (tree.cuh's splits), its four warps 16 entries of each tile; they
// meet once a unit, to join their sums.  Bound: for bf16 the cache's bytes; else a warp's way
// through a tile, about 300 instructions that widen and multiply, most of which wait for the one
// before (0.53 of the issue slots used, so that their number is not a limit yet).  Measured,
// captured and replayed, 64 rows of one node with 4096 of 32768 entries in their window: 32/8
// heads E4M3 110 us = 4.9 TB/s (floor 79), bf16 177 us = 6.1 TB/s (159), NVFP4 108 us (45);
// 128/8 heads E4M3 206 us.  By tiles of 128 rows the first took 415 us.  Steps: values loaded into registers a step ahead,
// 196 us; by way of stages in shared memory, three or so steps ahead, 147; whole 128-byte lines
// a copy instead of the lane's own chunks, 119 (the SM pays by the lines that a copy touches:
// 64-byte pieces of K cost as much); boxes by the TMA, the next
// unit's Q ahead of its turn, no rescaling before a first score, 111.  Splits of 16 tiles at least instead
// of 8 took 105 at 113, but a lone row of 4096 entries 21 us instead of 14.  More warps an SM with
// fewer registers (20, 24) took 145 and 204 us against 141 at that step.
#include <cstring>

#include "copies.cuh"
#include "tree_parts.cuh"

namespace da {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// Copies and lookups run less than this many units ahead: four stages' tiles and four more.
constexpr int kUnitSlots = 8;
constexpr int kStep = kT / kWarps;  // entries of a tile that a warp has: the M of an MMA

// What a thread of a warp reads of 16 entries, lane 4 g + q: entries g and g + 8 of K (D / 4
// dims, in chunks of 16 bytes or half a one), entries 2 q, 2 q + 1, 2 q + 8, 2 q + 9 of V (D / 8
// dims).
template <int KT, int D, int NT>
struct Few {
  static constexpr bool Q8 = KT != DA_KV_BF16;
  static constexpr int kRow = KT == DA_KV_BF16 ? 2 * D : KT == DA_KV_FP8_E4M3 ? D : D / 2;  // bytes of a head's row
  static constexpr int kKWords = kRow / 16, kVWords = kRow / 32;
  static constexpr int kKPiece = kKWords < 4 ? kKWords : 4, kVPiece = kVWords < 4 ? kVWords : 4;  // words of a copy
  static constexpr int kKDims = kKPiece * 4 * D / kRow, kVDims = kVPiece * 4 * D / kRow;          // dims of a copy
  static constexpr int kRows = 8 * NT;
  // Q lies in every warp's registers, or for more than 16 rows in shared memory, where warp w
  // puts rows 8 w to 8 w + 7
  static constexpr bool kQShared = NT > 2;
  static constexpr int kQHeld = kQShared ? 1 : NT;
  static constexpr int kPitch = kRow < 128 ? kRow : 128;  // from row to row in a stage
  // chunk of a row that is lane q's P-th of K: a phase of a read has two rows' even or odd ones
  static __device__ __forceinline__ int k_chunk(int q, int P) { return kRow >= 128 ? 2 * q + P % 2 + P / 2 * 8 : q; }
  // a warp's stage: K, V, NVFP4 block scales
  static constexpr int kVAt = kStep * kRow, kScalesAt = 2 * kVAt;
  static constexpr int kStage = kScalesAt + (KT == DA_KV_NVFP4 ? 2 * kStep * (D / 16) : 0);
  // Where 16 entries lie together the TMA copies rows of 128 bytes or more; shorter ones go faster
  // by the lanes' copies (a windowed step of 64 rows, when both were measured: NVFP4 120 against 128
  // us, 64 dims of E4M3 81 against 89; E4M3 with 128 dims 115 against 119 the other way).
  static constexpr bool kBoxes = kRow >= 128;
  static constexpr int kStages = kStage > 4096 ? 2 : kStage > 3000 ? 3 : 4;
  static constexpr int kBytes = kWarps * kStages * kStage + 1024;  // (1024: to align them)
  static constexpr int kResident = NT == 1 && kStage <= 4096 ? 4 : NT == 1 || D == 64 ? 3 : 2;  // blocks an SM
  // rows of the output that go through a stage at once: all, those of an MMA, or every second
  static constexpr int kPassRows = kScalesAt >= kRows * D * 4 ? kRows : kScalesAt >= 8 * D * 4 ? 8 : 4;
  static_assert(kScalesAt >= kPassRows * D * 4, "a stage takes a pass");
  static_assert(kResident * (kBytes + (kQShared ? 15 : 6) * 1024) <= 228 * 1024, "resident blocks");
};

// Copies B bytes, or zeros.
template <int B, bool ALL>
__device__ __forceinline__ void copy_or_zero(uint32_t dst, const uint8_t* src, bool there) {
  if constexpr (ALL) {
    if constexpr (B == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B) : "memory");
  } else {
    const int n = there ? B : 0;
    if constexpr (B == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(n) : "memory");
  }
}

template <int W>
__device__ __forceinline__ void read_words(const uint8_t* from, uint32_t* w) {
  if constexpr (W == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(from);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(from);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(from);
  }
}

// d += a b, 16 x 8 x 16
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

struct FewMaps {
  CUtensorMap k, v;  // [entries][H_kv][row], boxes of 16 entries of a head (of 128 bytes at most)
};

// 16-byte chunk `ch` of entry `row` in a stage, in an order in which a warp's reads spread
// over the banks: the TMA's of 128 bytes, and the like for shorter rows.
template <int R>  // chunks of a row
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  if constexpr (R == 16) return (ch >> 3) * (kStep * 128) + row * 128 + ((ch & 7) ^ (row & 7)) * 16;
  return (row * R + (ch ^ (R == 8 ? row & 7 : R == 4 ? row >> 1 & 3 : row >> 2 & 1))) * 16;
}

// Copies 16 entries, a warp's of a tile, to its stage, whole rows at a time: a copy costs the
// SM by the 128-byte lines that it touches.  spots: lane `at` + i has entry i's (cache row,
// head), or -1 (zeros then); ALL: there is no -1.
template <int KT, int D, int NT, bool ALL>
__device__ __forceinline__ void copy_rows(const TreeLaunch& p, int spots, int at, uint32_t dst, int lane) {
  using F = Few<KT, D, NT>;
  constexpr int R = F::kRow / 16;
  const uint8_t* const k = static_cast<const uint8_t*>(p.k) + lane % R * 16;
  const uint8_t* const v = static_cast<const uint8_t*>(p.v) + lane % R * 16;
#pragma unroll
  for (int i = 0; i < kStep * R / 32; ++i) {
    const int row = i * (32 / R) + lane / R;
    const int spot = __shfl_sync(0xffffffffu, spots, at + row);
    const unsigned long long off = (unsigned long long)(uint32_t)(ALL ? spot : max(spot, 0)) * F::kRow;
    const uint32_t to = dst + chunk_at<R>(row, lane % R);
    copy_or_zero<16, ALL>(to, k + off, spot >= 0);
    copy_or_zero<16, ALL>(to + F::kVAt, v + off, spot >= 0);
  }
}

// NVFP4: the rows' block scales, K's by lanes 0 to 15, V's by the others.
template <int D>
__device__ __forceinline__ void copy_scales(const TreeLaunch& p, int spots, int at, uint32_t dst, int lane) {
  const int spot = __shfl_sync(0xffffffffu, spots, at + (lane & 15));
  const uint8_t* from = static_cast<const uint8_t*>(lane < 16 ? p.k : p.v) + p.kv_rows * p.H_kv * (D / 2) +
                        (unsigned long long)(uint32_t)max(spot, 0) * (D / 16);
  copy_or_zero<D / 16, false>(dst + lane * (D / 16), from, spot >= 0);
}

template <int KT, int D, int NT>
struct HeldK {
  using F = Few<KT, D, NT>;
  uint32_t k[2][F::kKWords], ks[2];

  // `off`: where this lane's first words lie; the others follow from it, as a swizzle only
  // swaps neighbours here
  __device__ __forceinline__ void read(const uint8_t* stage, uint32_t off, int q) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int i = 0; i < F::kKWords; i += F::kKPiece)
        read_words<F::kKPiece>(stage + (off ^ (i & 4 ? 16u : 0u)) + i / 8 * (kStep * 128) + e * 8 * F::kPitch, k[e] + i);
      if constexpr (KT == DA_KV_NVFP4) {
        const uint8_t* s = stage + F::kScalesAt + (g + 8 * e) * (D / 16);
        ks[e] = D == 128 ? reinterpret_cast<const uint16_t*>(s)[q] : s[q];
      }
    }
  }

  // A operand of the scores, K's dims of k-step s
  __device__ __forceinline__ void k_operand(int s, uint32_t (&a)[4]) const {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (KT == DA_KV_BF16) {
        a[e] = k[e][2 * s];
        a[2 + e] = k[e][2 * s + 1];
      } else if constexpr (KT == DA_KV_FP8_E4M3) {
        a[e] = e4m3x2_to_f16x2(k[e][s]);
        a[2 + e] = e4m3x2_to_f16x2(k[e][s] >> 16);
      } else {
        const uint32_t two = e4m3x2_to_f16x2(ks[e]), scale = __byte_perm(two, 0, s < 4 ? 0x1010 : 0x3232);
        uint32_t h[4];
        e2m1x8_to_f16x2(k[e][s / 2], h);
        a[e] = hmul2(h[2 * (s & 1)], scale);
        a[2 + e] = hmul2(h[2 * (s & 1) + 1], scale);
      }
    }
  }

};

template <int KT, int D, int NT>
struct HeldV {
  using F = Few<KT, D, NT>;
  uint32_t v[4][F::kVWords], vs[4];

  __device__ __forceinline__ void read(const uint8_t* stage, uint32_t off, int q) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int i = 0; i < F::kVWords; i += F::kVPiece)
        read_words<F::kVPiece>(stage + F::kVAt + (off ^ (F::kRow >= 128 && (e & 1) ? 16u : 0u)) + i / 4 * (kStep * 128) +
                                   ((e & 1) + 4 * (e & 2)) * F::kPitch,
                               v[e] + i);
      if constexpr (KT == DA_KV_NVFP4)
        vs[e] = stage[F::kScalesAt + (kStep + 2 * q + (e & 1) + 4 * (e & 2)) * (D / 16) + g * (D / 8) / 16];
    }
  }

  // A operands of the output, V's dims of tiles 4 j4 .. 4 j4 + 3 (two dims of each)
  __device__ __forceinline__ void v_operands(int j4, uint32_t (&a)[4][4]) const {
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      if constexpr (KT == DA_KV_BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w0 = v[2 * pair][4 * j4 + j], w1 = v[2 * pair + 1][4 * j4 + j];
          a[j][2 * pair] = __byte_perm(w0, w1, 0x5410);
          a[j][2 * pair + 1] = __byte_perm(w0, w1, 0x7632);
        }
      } else if constexpr (KT == DA_KV_FP8_E4M3) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = __byte_perm(v[2 * pair][2 * j4 + j / 2], v[2 * pair + 1][2 * j4 + j / 2], j & 1 ? 0x7362 : 0x5140);
          a[j][2 * pair] = e4m3x2_to_f16x2(w);
          a[j][2 * pair + 1] = e4m3x2_to_f16x2(w >> 16);
        }
      } else {
        uint32_t h[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t scale = __byte_perm(e4m3x2_to_f16x2(vs[2 * pair + e]), 0, 0x1010);
          e2m1x8_to_f16x2(v[2 * pair + e][j4], h[e]);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[e][j] = hmul2(h[e][j], scale);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[j][2 * pair] = __byte_perm(h[0][j], h[1][j], 0x5410);
          a[j][2 * pair + 1] = __byte_perm(h[0][j], h[1][j], 0x7632);
        }
      }
    }
  }
};

// What pairs of dims of lane (g, q) are swapped by, of kPer next to each other.
template <int kPer>
__device__ __forceinline__ int swap_of(int g, int q) {
  return kPer == 8 ? (g >> 1 & 1) * 4 + q : q;
}

template <int KT, int D, int NT>
__global__ void __launch_bounds__(kThreads, Few<KT, D, NT>::kResident)
    few_kernel(const TreeLaunch p, const __grid_constant__ FewMaps maps, int boxes) {
  using F = Few<KT, D, NT>;
  extern __shared__ uint8_t smem[];
  uint8_t* const stages = smem + (-smem_addr(smem) & 1023u);  // of warp 0, warp 1, ...
  __shared__ uint64_t bars[kWarps * F::kStages + 1];           // of the TMA's copies; one that nothing arrives at
  __shared__ int2 sizes[kTreeRows];
  __shared__ int first[kTreeRows + 1];
  __shared__ Unit units[kWarps][kUnitSlots];  // a warp's unit, and those behind it up to the one that it copies
  __shared__ unsigned long long sees[F::kRows];  // nodes that a row sees
  __shared__ int depths[F::kRows];
  __shared__ uint2 shared_q[F::kQShared ? NT * (D / 16) * 32 : 1];  // lane by lane
  __shared__ float shared_scale[F::kRows];
  __shared__ float part_m[kWarps][F::kRows], part_l[kWarps][F::kRows];
  __shared__ uint32_t odd_rows[2];  // of every second unit
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i <= kWarps * F::kStages; ++i) mbar_init(smem_addr(bars + i), 1);
    fence_mbar_init();
  }
  wait_prior_grid();
  allow_next_grid();
  count_units<true>(p, sizes, first, kThreads);
  __syncthreads();
  // Rows without a tile have no unit, so that the ring of units holds only such as are copied;
  // their nodes see nothing.
  for (int i = blockIdx.x; i < p.rows; i += gridDim.x) {
    if (sizes[i].y >> 8) continue;
    const long long heads = (long long)sizes[i].y * p.H_q, row = (long long)(p.row0 + i) * p.T * p.H_q;
    for (long long k = threadIdx.x; k < heads * (D / 8); k += kThreads)
      reinterpret_cast<uint4*>(p.out + row * D)[k] = make_uint4(0, 0, 0, 0);
    for (long long k = threadIdx.x; k < heads; k += kThreads) p.lse[row + k] = -INFINITY;
  }
  UnitTable c;
  c.sizes = sizes;
  c.first = first;
  c.units = first[p.rows];
  if ((int)blockIdx.x >= c.units) return;

  // ---- copies run ahead of their use by kStages - 1 tiles, lookups by two more
  uint8_t* const mine = stages + warp * (F::kStages * F::kStage);
  const uint32_t mine_at = smem_addr(mine);
  Unit* ahead = nullptr;
  const uint32_t full = smem_addr(bars + warp * F::kStages);
  const uint32_t k_off = chunk_at<F::kRow / 16>(g, F::kKPiece == 4 ? F::k_chunk(q, 0) : q / 2) + (F::kKPiece == 4 ? 0 : 8 * (q & 1));
  const uint32_t v_off = chunk_at<F::kRow / 16>(2 * q, g * F::kVPiece / 4) + g * F::kVPiece % 4 * 4;
  Copies boxed;  // the TMA's
  // (all lanes wait: each of them reads what has arrived)
  auto landed = [&](int stage, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(full + 8 * stage, parity)) != 0;
  };
  bool bad = false;
  int ahead_u = (int)blockIdx.x - (int)gridDim.x, ahead_n = 0, ahead_i = 0, ahead_end = 0;
  int spots = -1, next_spots = -1;  // of two tiles' entries (lanes 0 to 15, 16 to 31), and the two behind them
  int tiles = 0, next_tiles = 0, half = 0;
  int to_stage = 0;
  auto look_up = [&]() {
    next_tiles = 0;
    if (ahead_i >= ahead_end) {  // (every unit has a tile)
      ahead_u += gridDim.x;
      if (ahead_u >= c.units) return;
      const Unit z = unit_of(p, c, ahead_u);
      ahead_i = z.begin;
      ahead_end = z.end;
      ahead = &units[warp][ahead_n++ % kUnitSlots];
      if (lane == 0) *ahead = z;
      __syncwarp();
    }
    const int i = ahead_i + (lane >> 4);
    next_spots = -1;
    if (i < ahead_end) {
      const int j = tree_tile(ahead->r, i) * kT + warp * kStep + (lane & 15);
      if (j < ahead->r.end && (j < ahead->r.hole_from || j >= ahead->r.hole_to)) {
        const int row = (int)cache_row(p, ahead->b, j);
        next_spots = row < 0 ? -1 : row * p.H_kv + ahead->h;
        bad |= row < 0;
      }
    }
    next_tiles = min(2, ahead_end - ahead_i);
    ahead_i += 2;
    __syncwarp();
  };
  auto take_lookup = [&]() {
    spots = next_spots;
    tiles = next_tiles;
    half = 0;
    if (tiles > 0) look_up();
  };
  auto copy_next = [&]() {
    if (tiles > 0 && !boxed.lost) {
      const uint32_t dst = mine_at + to_stage * F::kStage;
      const bool all = (__ballot_sync(0xffffffffu, spots >= 0) >> half & 0xffffu) == 0xffffu;
      if (F::kBoxes && all && boxes) {  // 16 entries in a row
        fence_proxy_async();  // (after what was written here by this warp itself)
        const int spot = __shfl_sync(0xffffffffu, spots, half);
        if (lane == 0) {
          const int row = quotient(spot, p.by_heads), h = spot - row * p.H_kv;
          const uint32_t bar = full + 8 * to_stage;
          mbar_arrive_expect_tx(bar, 2 * F::kVAt);
#pragma unroll
          for (int part = 0; part < F::kRow / 128; ++part) {
            tma_box3(dst + part * (kStep * 128), &maps.k, 64 * part, h, row, bar);
            tma_box3(dst + F::kVAt + part * (kStep * 128), &maps.v, 64 * part, h, row, bar);
          }
        }
        __syncwarp();
        boxed.sent(to_stage);
      } else if (all) {
        copy_rows<KT, D, NT, true>(p, spots, half, dst, lane);
      } else {
        copy_rows<KT, D, NT, false>(p, spots, half, dst, lane);
      }
      if constexpr (KT == DA_KV_NVFP4) copy_scales<D>(p, spots, half, dst + F::kScalesAt, lane);
      half = 16;
      if (--tiles == 0) take_lookup();
    }
    to_stage = to_stage == F::kStages - 1 ? 0 : to_stage + 1;
    cp_async_commit();
  };
  look_up();
  take_lookup();
  for (int i = 0; i < F::kStages - 1; ++i) copy_next();
  if (p.test_stall) {  // the time-out's test: a wait that runs out, of the first copy if that is the TMA's
    auto stalled = [&](int, uint32_t) {
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_addr(bars + kWarps * F::kStages), 0) && globaltimer_ns() - t0 < kTestStallNs) {
      }
      __syncwarp();
      return false;
    };
    if constexpr (F::kBoxes) {
      boxed.wait(0, stalled);
      if (!boxed.lost) boxed.lost = !stalled(0, 0);
    } else {  // the lanes' own copies have no wait that could run out, and the loops below no test for it
      stalled(0, 0);
      cp_async_wait<0>();
      if (threadIdx.x == 0) report(p.err, DA_DEVERR_TIMEOUT);
      return;
    }
  }
  int at_stage = 0, free_stage = F::kStages - 1;  // the stage in use, and the one before it
  uint32_t qb[F::kQHeld][D / 16][2];
  auto load_q = [&](const Unit* z) {
#pragma unroll
    for (int nt = 0; nt < F::kQHeld; ++nt) {
      const int at = (F::kQShared ? warp : nt) * 8 + g;
      const bool live = at < z->rows;
      const int t = live ? quotient(at, p.by_group) : 0;
      const __nv_bfloat16* from = p.q + ((size_t)((long long)z->b * p.T + t) * p.H_q + z->h * p.G + (at - t * p.G)) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        constexpr int kPer = F::kKDims / 4;  // k-steps of a piece
        const int d = F::k_chunk(q, s / kPer) * F::kKDims + 4 * (s % kPer);
        const uint2 w = live ? __ldg(reinterpret_cast<const uint2*>(from + d)) : make_uint2(0, 0);
        qb[nt][s][0] = w.x;
        qb[nt][s][1] = w.y;
      }
    }
  };
  // (after a time-out nothing is looked up)
  auto unit_at = [&](int u, int n) -> const Unit* {
    Unit* const z = &units[warp][n % kUnitSlots];
    if (boxed.lost) {
      const Unit v = unit_of(p, c, u);
      __syncwarp();
      if (lane == 0) *z = v;
      __syncwarp();
    }
    return z;
  };
  const Unit* x = unit_at(blockIdx.x, 0);
  load_q(x);
  for (int u = blockIdx.x, n = 0; u < c.units; u += gridDim.x, ++n) {
    const int n_rows = x->rows, h = x->h, begin = x->begin, end = x->end, length = x->r.length;
    const int head = x->r.head_tiles, skip = x->r.skip;
    // ---- Q as an operand, and what the rows see
    float scale[NT][2];  // softmax scales of rows 8 nt + 2 q and + 1
#pragma unroll
    for (int nt = 0; nt < F::kQHeld; ++nt) {
      float mine = p.scale_log2;
      if constexpr (F::Q8) {  // f16, scaled by a power of two
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          top = __vmaxu2(top, __vmaxu2(qb[nt][s][0] & 0x7fff7fffu, qb[nt][s][1] & 0x7fff7fffu));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = q_prescale_exp(bf16_absmax_value(top));
        const float sc = exp2_int(e);
        mine *= exp2_int(-e);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[nt][s][i] = pack16<true>(bf16_lo(qb[nt][s][i]) * sc, bf16_hi(qb[nt][s][i]) * sc);
      }
      if constexpr (F::kQShared) {
        if (warp < NT) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) shared_q[(warp * (D / 16) + s) * 32 + lane] = make_uint2(qb[0][s][0], qb[0][s][1]);
          if (q == 0) shared_scale[warp * 8 + g] = mine;
        }
      } else {
        scale[nt][0] = __shfl_sync(0xffffffffu, mine, 8 * q);
        scale[nt][1] = __shfl_sync(0xffffffffu, mine, 8 * q + 4);
      }
    }
    if (threadIdx.x < F::kRows) {
      const int at = threadIdx.x;
      int depth = 0;
      unsigned long long anc = 0;
      if (at < n_rows && end > begin && (p.window || (tree_tile(x->r, end - 1) + 1) * kT > length)) {
        anc = ancestors(p, x->b, quotient(at, p.by_group), &depth);
        anc = windowed(p, x->r, anc, depth) & low_bits(x->r.end - length);
      }
      sees[at] = anc;
      depths[at] = depth;
    }
    if (threadIdx.x == 0) odd_rows[n & 1] = 0;
    __syncthreads();
    if constexpr (F::kQShared) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) scale[nt][r] = shared_scale[8 * nt + 2 * q + r];
    }
    const int whole = p.window ? length + x->r.nodes - p.window : 0;
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    for (int i = begin; i < end; ++i) {
      cp_async_wait<F::kStages - 2>();
      boxed.wait(at_stage, landed);
      __syncwarp();
      const uint8_t* stage = mine + at_stage * F::kStage;
      HeldK<KT, D, NT> held;
      held.read(stage, k_off, q);
      copy_next();  // to the stage of the step before
      free_stage = at_stage;
      at_stage = at_stage == F::kStages - 1 ? 0 : at_stage + 1;
      // ---- scores: entries g and g + 8, rows 8 nt + 2 q and + 1; two sums, as an MMA waits long
      // for the one before it
      float s[NT][4], s_odd[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = s_odd[nt][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t a[4];
        held.k_operand(k, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint2 b;
          if constexpr (F::kQShared)
            b = shared_q[(nt * (D / 16) + k) * 32 + lane];
          else
            b = make_uint2(qb[nt][k][0], qb[nt][k][1]);
          mma_16816<F::Q8>(k & 1 ? s_odd[nt] : s[nt], a, b.x, b.y);
        }
      }
      HeldV<KT, D, NT> values;
      values.read(stage, v_off, q);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] += s_odd[nt][e];
      const int j0 = (i < head ? i : i + skip) * kT;
      const bool all = j0 + kT <= length && (j0 >= whole || j0 + kT <= p.sinks);
      bool move = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s[nt][r] *= scale[nt][r];
          s[nt][2 + r] *= scale[nt][r];
        }
        if (!all) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int at = nt * 8 + 2 * q + r;
            unsigned long long vis = low_bits(length - j0);
            if (p.window) vis &= ~low_bits(length + depths[at] - p.window + 1 - j0) | low_bits(p.sinks - j0);
            const int shift = length - j0;  // of node 0 in the tile
            if (shift > -64 && shift < 64) vis |= shift >= 0 ? sees[at] << shift : sees[at] >> -shift;
            if (at >= n_rows) vis = 0;
            const uint32_t mine = (uint32_t)(vis >> (warp * kStep));
            if (!(mine >> g & 1)) s[nt][r] = -INFINITY;
            if (!(mine >> (g + 8) & 1)) s[nt][2 + r] = -INFINITY;
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float most = fmaxf(s[nt][r], s[nt][2 + r]) - (F::Q8 ? kHeadLog2 : 0.f);
          move |= most > m[nt][r] + kRescaleLog2 || (m[nt][r] == -INFINITY && most > -INFINITY);
        }
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float alpha[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float most = fmaxf(s[nt][r], s[nt][2 + r]);
#pragma unroll
            for (int b = 4; b < 32; b <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, b));
            most -= F::Q8 ? kHeadLog2 : 0.f;
            const bool moves = most > m[nt][r] + kRescaleLog2 || (m[nt][r] == -INFINITY && most > -INFINITY);
            alpha[r] = moves && m[nt][r] > -INFINITY ? ex2(m[nt][r] - most) : 1.f;
            if (moves) m[nt][r] = most;
            l[nt][r] *= alpha[r];
          }
          // (no sum stands before a row's first score)
          if (!__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) continue;
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][j][e] *= alpha[e & 1];
        }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float ref = m[nt][r] == -INFINITY ? 0.f : m[nt][r];
          w[r] = ex2(s[nt][r] - ref);
          w[2 + r] = ex2(s[nt][2 + r] - ref);
          l[nt][r] += w[r] + w[2 + r];
        }
        pb[nt][0] = transposed(pack16<F::Q8>(w[0], w[1]));
        pb[nt][1] = transposed(pack16<F::Q8>(w[2], w[3]));
      }
#pragma unroll
      for (int j4 = 0; j4 < D / 64; ++j4) {
        uint32_t a[4][4];
        values.v_operands(j4, a);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816<F::Q8>(o[nt][4 * j4 + j], a[j], pb[nt][0], pb[nt][1]);
      }
    }
    const Unit* next = x;
    if (u + (int)gridDim.x < c.units) {
      next = unit_at(u + gridDim.x, n + 1);
      load_q(next);
    }
    // ---- the warps' sums joined, in their order, by way of each one's stage that was used last
    // (the next copy goes there)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[nt][r];
#pragma unroll
        for (int b = 4; b < 32; b <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
        if (g == 0) {
          part_m[warp][nt * 8 + 2 * q + r] = m[nt][r];
          part_l[warp][nt * 8 + 2 * q + r] = sum;
        }
      }
    const bool single = x->r.splits == 1;
    const long long to_slot = (((long long)x->b * p.max_splits + x->split) - x->b) * p.T * p.H_q;
#pragma unroll
    for (int pass = 0; pass < F::kRows / F::kPassRows; ++pass) {
      // row 8 nt + 2 q + r is row `at` of the pass; its dims in pairs, swapped so that a warp's
      // meet in no bank
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (boxed.lost) continue;  // (a copy may be on its way there)
          if (F::kPassRows == 8 && nt != pass) continue;
          if (F::kPassRows == 4 && 2 * nt + r != pass) continue;
          const int at = F::kPassRows == 4 ? q : F::kPassRows == 8 ? 2 * q + r : 8 * nt + 2 * q + r;
          float2* to = reinterpret_cast<float2*>(mine + free_stage * F::kStage) + at * (D / 2);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            constexpr int kPer = F::kVDims / 2;  // tiles of a piece
            to[((j / kPer) * 8 + g) * kPer + (j % kPer ^ swap_of<kPer>(g, q))] = make_float2(o[nt][j][r], o[nt][j][2 + r]);
          }
        }
      __syncthreads();
      for (int i = threadIdx.x; i < F::kPassRows * (D / 4); i += kThreads) {
        const int in = i / (D / 4), d = 4 * (i % (D / 4));
        const int at = F::kPassRows == 4 ? 8 * (pass / 2) + 2 * in + pass % 2 : F::kPassRows == 8 ? 8 * pass + in : in;
        if (at >= n_rows) continue;
        constexpr int kPer = F::kVDims / 2;
        const int pair = d / 2, swap = swap_of<kPer>(pair / kPer % 8, at % 8 / 2);
        float top = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w][at]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float c_w = part_m[w][at] == top ? 1.f : ex2(part_m[w][at] - top);
          const float2* from = reinterpret_cast<const float2*>(stages + w * (F::kStages * F::kStage) + free_stage * F::kStage) + in * (D / 2);
          const float2 o0 = from[pair ^ swap], o1 = from[(pair + 1) ^ swap];
          sum = fmaf(part_l[w][at], c_w, sum);
          v.x = fmaf(o0.x, c_w, v.x);
          v.y = fmaf(o0.y, c_w, v.y);
          v.z = fmaf(o1.x, c_w, v.z);
          v.w = fmaf(o1.y, c_w, v.w);
        }
        const float inv = (sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f) * p.v_scale;
        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        const int t = quotient(at, p.by_group);
        const size_t row = (size_t)((long long)x->b * p.T + t) * p.H_q + h * p.G + (at - t * p.G);
        if (sum != sum || !(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w) < INFINITY)) atomicOr(&odd_rows[n & 1], 1u << at);
        const float lse = sum > 0.f || sum != sum ? top + lg2(sum) : -INFINITY;
        if (single) {
          *reinterpret_cast<uint2*>(p.out + row * D + d) = make_uint2(pack16<false>(v.x, v.y), pack16<false>(v.z, v.w));
          if (d == 0) p.lse[row] = lse * kLn2;
        } else {
          *reinterpret_cast<float4*>(p.o_part + (to_slot + (long long)row) * D + d) = v;
          if (d == 0) p.lse_part[to_slot + (long long)row] = lse;
        }
      }
      __syncthreads();
    }
    // rows that something infinite or NaN has spoiled: formed again, entry by entry
    uint32_t again = odd_rows[n & 1];
    for (int k = 0; again; again &= again - 1, ++k) {
      if (k % kWarps != warp) continue;
      const int at = __ffs((int)again) - 1, t = quotient(at, p.by_group), hq = h * p.G + (at - t * p.G);
      const size_t row = (size_t)((long long)x->b * p.T + t) * p.H_q + hq;
      float m2, l2, o2[D / 32];
      attend_plainly<KT, D>(p, x->r, x->b, t, hq, begin, end, lane, &m2, &l2, o2);
      const float inv2 = (l2 > 0.f ? 1.f / l2 : l2 != l2 ? l2 : 0.f) * p.v_scale;
      const float lse2 = l2 > 0.f || l2 != l2 ? m2 + lg2(l2) : -INFINITY;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const int d = lane * (D / 32) + e;
        if (single)
          p.out[row * D + d] = __float2bfloat16_rn(o2[e] * inv2);
        else
          p.o_part[(to_slot + (long long)row) * D + d] = o2[e] * inv2;
      }
      if (lane == 0) {
        if (single)
          p.lse[row] = lse2 * kLn2;
        else
          p.lse_part[to_slot + (long long)row] = lse2;
      }
    }
    x = next;
  }
  cp_async_wait<0>();
  if (boxed.lost) {  // leave no copy in flight
    boxed.drain(F::kStages, landed);
    if (lane == 0) report(p.err, DA_DEVERR_TIMEOUT);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.err, DA_DEVERR_INDEX);
}

template <int KT, int D, int NT>
cudaError_t launch_shape(const TreeLaunch& p0, int sms, cudaStream_t stream) {
  using F = Few<KT, D, NT>;
  const cudaError_t attr = allow_smem(few_kernel<KT, D, NT>, F::kBytes);
  if (attr != cudaSuccess) return attr;
  TreeLaunch p = p0;
  p.by_heads = fast_div(p.H_kv);
  p.by_group = fast_div(p.G);
  p.by_page = fast_div(p.page_size > 1 ? p.page_size : 1);
  FewMaps m;
  std::memset(&m, 0, sizeof(m));
  int boxes = 0;
  if constexpr (F::kBoxes) {
    boxes = p.kv_rows > 0 && (p.layout == DA_KV_CONTIGUOUS || (p.layout == DA_KV_PAGED && p.page_size % kStep == 0));
    const cuuint64_t heads = (cuuint64_t)p.H_kv, size = F::Q8 ? 1 : 2;
    const cuuint64_t dims[3] = {F::kRow / size, heads, (cuuint64_t)p.kv_rows}, strides[2] = {F::kRow, heads * F::kRow};
    const cuuint32_t box[3] = {128 / (cuuint32_t)size, 1, kStep};
    if (boxes && (!tree_tensor_map(&m.k, p.k, 3, dims, strides, box, F::Q8, CU_TENSOR_MAP_SWIZZLE_128B) ||
                  !tree_tensor_map(&m.v, p.v, 3, dims, strides, box, F::Q8, CU_TENSOR_MAP_SWIZZLE_128B)))
      return cudaErrorInvalidValue;
  }
  for (p.row0 = 0; p.row0 < p.B; p.row0 += kTreeRows) {
    p.rows = p.B - p.row0 < kTreeRows ? p.B - p.row0 : kTreeRows;
    const long long most = (long long)p.rows * p.max_splits * p.H_kv, room = (long long)F::kResident * sms;
    const cudaError_t e = launch_after(few_kernel<KT, D, NT>, dim3((unsigned)(most < room ? most : room)), dim3(kThreads),
                                       (size_t)F::kBytes, stream, p, m, boxes);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int KT, int D>
cudaError_t launch_rows(const TreeLaunch& p, int sms, cudaStream_t stream) {
  const int rows = p.T * p.G;
  if (rows <= 8) return launch_shape<KT, D, 1>(p, sms, stream);
  if (rows <= 16) return launch_shape<KT, D, 2>(p, sms, stream);
  if (rows <= 24) return launch_shape<KT, D, 3>(p, sms, stream);
  if constexpr (KT != DA_KV_BF16 || D != 128) return launch_shape<KT, D, 4>(p, sms, stream);
  return cudaErrorInvalidValue;
}

template <int KT>
cudaError_t launch_kt(const TreeLaunch& p, int sms, cudaStream_t stream) {
  return p.D == 64 ? launch_rows<KT, 64>(p, sms, stream) : launch_rows<KT, 128>(p, sms, stream);
}

}  // namespace

cudaError_t launch_tree_few(const TreeLaunch& p, int sms, cudaStream_t stream) {
  switch (p.kv_type) {
    case DA_KV_FP8_E4M3: return launch_kt<DA_KV_FP8_E4M3>(p, sms, stream);
    case DA_KV_NVFP4: return launch_kt<DA_KV_NVFP4>(p, sms, stream);
    default: return launch_kt<DA_KV_BF16>(p, sms, stream);
  }
}

}  // namespace da
