// Low-rank adapters of many requests beside a shared weight matmul:
//     t[i, :] = bf16(x[i, :]) A_id^T,   out[i, :] = y[i, :] + (scale_id t[i, :]) B_id^T
// with each row's own id, every row's bits independent of the batch.
//
// Rows are taken 32 at a time in batch order (a "tile", one lane of a warp per
// row); the rows of a tile that share an adapter form a group, found by a match
// across the lanes, and the members of a group are the columns of the matrix
// products.  Prompts, whose rows come in runs, give one group of 32 per tile;
// decode steps give many small ones.  No list is built or sorted on the device.
//
// Two kernels on the warp-level tensor cores (m16n8k16, bf16 x bf16 products
// exact, fp32 accumulation):
//   down: t.  M = ranks, N = group members, K along x.  Operand fragments come
//     straight from global memory, 16 bytes a lane: a fragment's K order may be
//     any permutation as long as both operands use the same, so lane q of a row
//     quad takes K 8q .. 8q + 7 of each 32.  K is cut into chunks of kChunk that
//     one warp sums from zero, four chunks make a K group, added in order, and
//     the groups are added in order: ((g0 + g1) + g2) ...; a large call lets one
//     CTA walk all groups of a tile, a small one gives every group its own CTA
//     and the second kernel adds them, the same additions either way.
//   up: out.  M = output features, N = group members, K = ranks.  t is scaled
//     and split into three bf16 terms that hold its 24 bits (their products
//     with B are exact, so out keeps fp32 accuracy); rows of the M tiles are
//     assigned to features so that a lane ends up with four consecutive ones:
//     y and out move 16 bytes a lane, whole 128-byte lines a quad of lanes.
// y and out (8 N bytes a row) bound a prompt, the adapters' weights and launch
// latency a decode step.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "nvfp4_mm.h"

namespace da {
namespace {

constexpr int kTile = 32;                     // rows per tile
constexpr int kChunk = 128;                   // K that one warp sums from zero
constexpr int kWarps = 4;                     // warps of a down CTA = chunks of a K group
constexpr int kGroupK = kChunk * kWarps;      // 512
constexpr int kDownThreads = kWarps * 32;
constexpr int kMaxRank = NVFP4_ADAPTER_MAX_RANK;
constexpr int kUpWarps = 8;
constexpr int kUpThreads = kUpWarps * 32;
constexpr int kWarpN = 32;                    // features of a warp's step
constexpr unsigned kFull = 0xffffffffu;

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
  float* t;  // [n_parts][n][max_rank]: one part (all K), or one per K group
  int n, N, K, n_adapters, max_rank;
  int n_groups;   // K groups
  int n_parts;    // 1 or n_groups
  int n_step;     // up: features of a CTA (a multiple of 128)
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// The groups of a tile as every lane of a warp sees them.
struct Groups {
  int id;            // this lane's row's adapter, -1 if none
  unsigned peers;    // lanes whose row has the same adapter
  unsigned leaders;  // lowest lane of each group
  int bad;           // error bits of this lane's row
};

__device__ __forceinline__ Groups groups_of(const Args& g, int row0, int lane) {
  Groups r;
  const int row = row0 + lane;
  r.id = row < g.n ? __ldg(g.ids + row) : -1;
  r.bad = 0;
  if (r.id >= g.n_adapters) {
    r.bad = DA_DEVERR_INDEX;
    r.id = -1;
  }
  if (r.id < 0) r.id = -1;
  r.peers = __match_any_sync(kFull, r.id);
  r.leaders = __ballot_sync(kFull, r.id >= 0 && lane == __ffs(r.peers) - 1);
  return r;
}

__device__ __forceinline__ int rank_of(const Args& g, int id, int* bad) {
  if (!g.ranks) return g.max_rank;
  const int r = __ldg(g.ranks + id), c = clamp_len(r, g.max_rank);
  if (c != r) *bad |= DA_DEVERR_LENGTH;
  return c;
}

// The rows of the group `members`, in order, then -1: written by one warp.
__device__ __forceinline__ void list_members(int (&list)[kTile], unsigned members, int row0,
                                             int lane) {
  const int before = __popc(members & ((1u << lane) - 1u));
  if ((members >> lane) & 1u) list[before] = row0 + lane;
  if (lane >= __popc(members)) list[lane] = -1;
}

// Eight consecutive activations as bf16 pairs (round to nearest even).
template <bool BF16>
__device__ __forceinline__ uint4 load_x8(const void* x, long long i) {
  if constexpr (BF16) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + i));
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    const float4 u = __ldg(p), v = __ldg(p + 1);
    return make_uint4(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w), pack_bf16(v.x, v.y),
                      pack_bf16(v.z, v.w));
  }
}

// ---------------------------------------------------------------- down
// Grid (K groups or 1, tiles, Z): CTA (p, tile, z) takes the tile's groups z,
// z + Z, ...; rank blocks of 64 one after the other.
template <bool BF16>
__global__ void __launch_bounds__(kDownThreads) down_kernel(const Args g) {
  // a K group's chunk sums: [warp][rank of 64][member]
  __shared__ float part[kWarps][64][kTile + 1];
  __shared__ int member[kTile];
  wait_prior_grid();
  allow_next_grid();  // after the wait: what ran before this call has finished
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, row8 = lane >> 2;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0)
    g.hdr[kHdrError] = 0;  // errors of this call only: the second kernel sets them
  const int row0 = blockIdx.y * kTile;
  const Groups gr = groups_of(g, row0, lane);
  unsigned left = gr.leaders;
  for (int j = 0; left; ++j) {
    const int lead = __ffs(left) - 1;
    left &= left - 1;
    if (j % (int)gridDim.z != (int)blockIdx.z) continue;
    const int id = __shfl_sync(kFull, gr.id, lead);
    const unsigned members = __shfl_sync(kFull, gr.peers, lead);
    const int count = __popc(members);
    int ignore = 0;
    const int rank = rank_of(g, id, &ignore);
    __syncthreads();  // the previous group's list has been read
    if (warp == 0) list_members(member, members, row0, lane);
    __syncthreads();
    // this lane's columns: members row8, row8 + 8, ...
    long long xrow[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int row = member[nt * 8 + row8];
      xrow[nt] = row < 0 ? -1 : (long long)row * g.K;
    }
    const int n_nt = (count + 7) >> 3;
    const int p0 = g.n_parts == 1 ? 0 : (int)blockIdx.x;
    const int p1 = g.n_parts == 1 ? g.n_groups : p0 + 1;
    for (int r0 = 0; r0 < rank; r0 += 64) {
      const int n_mt = min(4, (rank - r0 + 15) >> 4);
      const __nv_bfloat16* arow = g.a + ((long long)id * g.max_rank + r0 + row8) * g.K + 8 * q;
      // sums of this thread's share of (64 ranks) x (32 members)
      constexpr int kMine = 64 * kTile / kDownThreads;
      float sum[kMine];
      for (int p = p0; p < p1; ++p) {
        float acc[4][4][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
        const int k0 = p * kGroupK + warp * kChunk, k1 = min(k0 + kChunk, g.K);
#pragma unroll 2
        for (int k = k0; k < k1; k += 32) {
          uint4 xv[4];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            xv[nt] = make_uint4(0, 0, 0, 0);
            if (nt < n_nt && xrow[nt] >= 0) xv[nt] = load_x8<BF16>(g.x, xrow[nt] + k + 8 * q);
          }
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            if (mt >= n_mt) break;
            const uint4 lo = __ldg(reinterpret_cast<const uint4*>(arow + (long long)mt * 16 * g.K + k));
            const uint4 hi =
                __ldg(reinterpret_cast<const uint4*>(arow + (long long)(mt * 16 + 8) * g.K + k));
            const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
              if (nt >= n_nt) break;
              mma(acc[mt][nt], a0, xv[nt].x, xv[nt].y);
              mma(acc[mt][nt], a1, xv[nt].z, xv[nt].w);
            }
          }
        }
        __syncthreads();  // the previous sums have been read
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              part[warp][mt * 16 + row8 + (e >> 1) * 8][nt * 8 + 2 * q + (e & 1)] = acc[mt][nt][e];
        __syncthreads();
        // chunks past the end of K are zero: adding them changes nothing but a
        // -0, so they take part whatever K is
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int r = (int)threadIdx.x & 63, c = i * (kDownThreads / 64) + ((int)threadIdx.x >> 6);
          const float s = ((part[0][r][c] + part[1][r][c]) + part[2][r][c]) + part[3][r][c];
          sum[i] = p == p0 ? s : sum[i] + s;
        }
      }
      float* t = g.t + (long long)p0 * g.n * g.max_rank;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = (int)threadIdx.x & 63, c = i * (kDownThreads / 64) + ((int)threadIdx.x >> 6);
        if (c < count && r0 + r < rank)
          t[(long long)member[c] * g.max_rank + r0 + r] = sum[i];
      }
    }
  }
}

// ---------------------------------------------------------------- up
// Bytes between the rows of a term of t in shared memory: 2 * 16 * blocks
// rounded to an odd multiple of 32, which spreads the 8-byte reads of four
// neighbouring rows over all banks.
__host__ __device__ constexpr int t_stride(int max_rank) {
  const int b = 2 * max_rank;
  return (b / 32) % 2 ? b : b + 32;
}

// Four ranks of feature row `p` (ranks k .. k + 3 of which `left` are below the
// adapter's rank); the others are zero whatever memory holds.
__device__ __forceinline__ uint2 load_b4(const __nv_bfloat16* p, int left) {
  uint2 w = make_uint2(0, 0);
  if (left > 0) w = __ldg(reinterpret_cast<const uint2*>(p));
  if (left < 4) {
    if (left <= 2) w.y = 0;
    if (left == 3) w.y &= 0xffffu;
    if (left == 1) w.x &= 0xffffu;
  }
  return w;
}

// Grid (feature blocks, tiles, Z): CTA (f, tile, z) adds to the rows of the
// tile's groups z, z + Z, ..., features [f * n_step, (f + 1) * n_step); the CTA
// z = 0 also copies the rows without an adapter.
__global__ void __launch_bounds__(kUpThreads) up_kernel(const Args g) {
  extern __shared__ __align__(16) uint8_t smem[];  // [3 terms][32 members][t_stride]
  __shared__ int member[kTile];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, row8 = lane >> 2;
  const int ts = t_stride(g.max_rank);
  const int row0 = blockIdx.y * kTile;
  wait_prior_grid();
  allow_next_grid();
  Groups gr = groups_of(g, row0, lane);
  const int f0 = blockIdx.x * g.n_step, f1 = min(f0 + g.n_step, g.N);

  if (blockIdx.z == 0 && (g.out != g.y || g.out_bf16)) {
    unsigned none = __ballot_sync(kFull, gr.id < 0 && row0 + lane < g.n);
    for (; none; none &= none - 1) {
      const long long at = (long long)(row0 + __ffs(none) - 1) * g.N;
      for (int f = f0 + 4 * (int)threadIdx.x; f < f1; f += 4 * kUpThreads) {
        const float4 v = *reinterpret_cast<const float4*>(g.y + at + f);
        if (g.out != g.y) *reinterpret_cast<float4*>(g.out + at + f) = v;
        if (g.out_bf16)
          *reinterpret_cast<uint2*>(g.out_bf16 + at + f) =
              make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
      }
    }
  }

  unsigned left = gr.leaders;
  for (int j = 0; left; ++j) {
    const int lead = __ffs(left) - 1;
    left &= left - 1;
    if (j % (int)gridDim.z != (int)blockIdx.z) continue;
    const int id = __shfl_sync(kFull, gr.id, lead);
    const unsigned members = __shfl_sync(kFull, gr.peers, lead);
    const int count = __popc(members);
    const int rank = rank_of(g, id, &gr.bad);
    const int n_k = (rank + 15) >> 4, n_nt = (count + 7) >> 3;
    const float scale = g.scales ? __ldg(g.scales + id) : 1.f;

    // t of the members, scaled, as three bf16 terms: hi + mid + lo = t up to
    // 2^-24 of it (each term takes the next 8 bits); ranks at or beyond the
    // adapter's, and members that do not exist, are zero
    __syncthreads();  // the previous group's terms and list have been read
    if (warp == 0) list_members(member, members, row0, lane);
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * n_k * 16; i += kUpThreads) {
      const int c = i / (n_k * 16), r = i - c * (n_k * 16);
      float v = 0.f;
      if (c < count && r < rank) {
        const float* t = g.t + (long long)member[c] * g.max_rank + r;
        v = __ldcg(t);
        for (int p = 1; p < g.n_parts; ++p) v += __ldcg(t + (long long)p * g.n * g.max_rank);
        v *= scale;
      }
      const __nv_bfloat16 hi = __float2bfloat16_rn(v);
      // nothing is left of an infinity (inf - inf would make it a NaN)
      const float r1 = __hisinf(hi) ? 0.f : v - __bfloat162float(hi);
      const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
      const __nv_bfloat16 lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
      uint8_t* at = smem + c * ts + 2 * r;
      *reinterpret_cast<__nv_bfloat16*>(at) = hi;
      *reinterpret_cast<__nv_bfloat16*>(at + kTile * ts) = mid;
      *reinterpret_cast<__nv_bfloat16*>(at + 2 * kTile * ts) = lo;
    }
    __syncthreads();

    // rows of this lane's accumulator columns 2q, 2q + 1 of each block of 8
    int mrow[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mrow[i] = member[(i >> 1) * 8 + 2 * q + (i & 1)];
    }
    const __nv_bfloat16* bmat = g.b + (long long)id * g.N * g.max_rank;
    for (int f = f0 + warp * kWarpN; f < f1; f += kUpWarps * kWarpN) {
      const int feat = f + 4 * row8;  // this lane's four features
      float4 yv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (mrow[i] >= 0)
          yv[i] = *reinterpret_cast<const float4*>(g.y + (long long)mrow[i] * g.N + feat);
      // M tile 0: features 4 row8 (rows 0-7) and 4 row8 + 1 (rows 8-15);
      // M tile 1: 4 row8 + 2 and 4 row8 + 3
      float acc[2][4][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
      const __nv_bfloat16* brow = bmat + (long long)feat * g.max_rank + 4 * q;
#pragma unroll 4
      for (int kb = 0; kb < n_k; ++kb) {
        const int have = rank - kb * 16 - 4 * q;
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = load_b4(brow + (long long)i * g.max_rank + kb * 16, have);
        const uint32_t a0[4] = {w[0].x, w[1].x, w[0].y, w[1].y};
        const uint32_t a1[4] = {w[2].x, w[3].x, w[2].y, w[3].y};
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          if (nt >= n_nt) break;
          const uint8_t* at = smem + (nt * 8 + row8) * ts + 32 * kb + 8 * q;
#pragma unroll
          for (int term = 2; term >= 0; --term) {  // small terms first
            const uint2 tv = *reinterpret_cast<const uint2*>(at + term * kTile * ts);
            mma(acc[0][nt], a0, tv.x, tv.y);
            mma(acc[1][nt], a1, tv.x, tv.y);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (mrow[i] < 0) continue;
        const int nt = i >> 1, e = i & 1;
        float4 v = yv[i];
        v.x += acc[0][nt][e];
        v.y += acc[0][nt][2 + e];
        v.z += acc[1][nt][e];
        v.w += acc[1][nt][2 + e];
        const long long at = (long long)mrow[i] * g.N + feat;
        *reinterpret_cast<float4*>(g.out + at) = v;
        if (g.out_bf16)
          *reinterpret_cast<uint2*>(g.out_bf16 + at) =
              make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
      }
    }
  }
  if (gr.bad && blockIdx.x == 0 && warp == 0) set_error(g.hdr, gr.bad);
}

// ---------------------------------------------------------------- host

constexpr size_t kHdr = 256;

int groups_of_k(int K) { return (K + kGroupK - 1) / kGroupK; }

// A CTA per K group until the tiles alone fill the GPU about once; then one
// walks all groups of its tile, and t is written once.
int parts_of(int n, int K) { return n > 4096 ? 1 : groups_of_k(K); }

bool shape_ok(int n, int N, int K, int n_adapters, int max_rank) {
  if (n < 0 || N <= 0 || K <= 0 || N % NVFP4_MM_TILE_N || K % 64) return false;
  if (n_adapters < 1 || max_rank < 16 || max_rank > kMaxRank || max_rank % 16) return false;
  return (long long)n * K < (1ll << 31) && (long long)n * N < (1ll << 31);
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace da

using namespace da;

extern "C" {

size_t nvfp4_mm_adapters_workspace_bytes(int32_t n, int32_t N, int32_t K, int32_t n_adapters,
                                         int32_t max_rank) {
  if (!shape_ok(n, N, K, n_adapters, max_rank)) return 0;
  return kHdr + (size_t)parts_of(n, K) * n * max_rank * sizeof(float);
}

int nvfp4_mm_adapters(const void* x, int32_t x_dtype, int32_t n, int32_t N, int32_t K,
                      const void* a, const void* b, int32_t n_adapters, int32_t max_rank,
                      const int32_t* ranks, const float* scales, const int32_t* ids,
                      const float* y, float* out, void* out_bf16, void* ws, size_t ws_bytes,
                      void* stream) {
  if (x_dtype != NVFP4_X_F32 && x_dtype != NVFP4_X_BF16) return DA_ERR_INVALID_ARG;
  if (!shape_ok(n, N, K, n_adapters, max_rank)) return DA_ERR_UNSUPPORTED;
  if (n == 0) return DA_OK;
  if (!x || !a || !b || !ids || !y || !out) return DA_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(a, 16) || !aligned_to(b, 16) || !aligned_to(y, 16) ||
      !aligned_to(out, 16) || !aligned_to(out_bf16, 8) || !aligned_to(ids, 4) ||
      !aligned_to(ranks, 4) || !aligned_to(scales, 4))
    return DA_ERR_INVALID_ARG;
  const uintptr_t y0 = reinterpret_cast<uintptr_t>(y), o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t bytes = (uintptr_t)n * N * 4;
  if (y0 != o0 && y0 < o0 + bytes && o0 < y0 + bytes) return DA_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256)) return DA_ERR_WORKSPACE;
  if (ws_bytes < nvfp4_mm_adapters_workspace_bytes(n, N, K, n_adapters, max_rank))
    return DA_ERR_WORKSPACE;
  Args g;
  std::memset(&g, 0, sizeof(g));
  g.x = x;
  g.a = static_cast<const __nv_bfloat16*>(a);
  g.b = static_cast<const __nv_bfloat16*>(b);
  g.ranks = ranks;
  g.scales = scales;
  g.ids = ids;
  g.y = y;
  g.out = out;
  g.out_bf16 = static_cast<__nv_bfloat16*>(out_bf16);
  g.hdr = static_cast<int32_t*>(ws);
  g.t = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kHdr);
  g.n = n;
  g.N = N;
  g.K = K;
  g.n_adapters = n_adapters;
  g.max_rank = max_rank;
  g.n_groups = groups_of_k(K);
  g.n_parts = parts_of(n, K);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int tiles = (n + kTile - 1) / kTile;
  if (tiles > 65535) return DA_ERR_UNSUPPORTED;  // n * K and n * N already bound it far below
  // a CTA per group of a tile while there are few CTAs without it
  const auto spread = [&](long long ctas) {
    return (unsigned)std::max<long long>(1, std::min<long long>({(long long)kTile, (long long)n,
                                                                 (long long)n_adapters,
                                                                 2048 / std::max(1ll, ctas)}));
  };
  const dim3 down((unsigned)g.n_parts, (unsigned)tiles, spread((long long)g.n_parts * tiles));
  cudaError_t e = x_dtype == NVFP4_X_BF16
                      ? launch_after(down_kernel<true>, down, dim3(kDownThreads), 0, st, g)
                      : launch_after(down_kernel<false>, down, dim3(kDownThreads), 0, st, g);
  if (e != cudaSuccess) return DA_ERR_CUDA;
  // 256 features a CTA (one step of its warps) while that leaves few CTAs
  g.n_step = kUpWarps * kWarpN;
  while (g.n_step < 1024 && (long long)tiles * (N / g.n_step) > 2048) g.n_step *= 2;
  const unsigned blocks = (unsigned)((N + g.n_step - 1) / g.n_step);
  const size_t smem = 3 * (size_t)kTile * t_stride(max_rank);
  e = launch_after(up_kernel, dim3(blocks, (unsigned)tiles, spread((long long)blocks * tiles)),
                   dim3(kUpThreads), smem, st, g);
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
