// What both kernels of the tree attention (tree.cu, tree_few.cu) are built from: which
// entries a node sees, the list of units of work, and a row formed entry by entry.
#pragma once

#include "tree.cuh"

namespace da {
namespace {

constexpr int kT = kTreeTile;
// A row's reference value moves when a score exceeds it by this much (log2).
constexpr float kRescaleLog2 = 8.f;
// f16 weights: the largest is 2^7 or more (and at most 2^15), so that what f16 cannot hold
// below 2^-25 is less than 2^-32 of it.
constexpr float kHeadLog2 = 7.f;

// The nodes that node t of row b sees, itself included, and its depth.  Parents that are
// not earlier nodes count as none.
__device__ __forceinline__ unsigned long long ancestors(const TreeLaunch& p, int b, int t, int* depth) {
  unsigned long long anc = 1ull << t;
  int d = 0;
  if (!p.parents) {
    *depth = t;
    return (2ull << t) - 1;
  }
  for (int a = t;;) {
    const int up = __ldg(p.parents + (long long)b * p.T + a);
    if (up < 0 || up >= a) break;
    a = up;
    anc |= 1ull << a;
    ++d;
  }
  *depth = d;
  return anc;
}

// Cache row of entry j of row b, or -1: its page or slot is out of range.
__device__ __forceinline__ long long cache_row(const TreeLaunch& p, int b, int j) {
  if (p.layout == DA_KV_CONTIGUOUS) return (long long)b * p.width + j;
  const int at = p.layout == DA_KV_PAGED ? quotient(j, p.by_page) : j;
  const int id = __ldg(p.table + (long long)b * p.width + at);
  if (id < 0 || id >= p.num_blocks) return -1;
  return p.layout == DA_KV_PAGED ? (long long)id * p.page_size + (j - at * p.page_size) : id;
}

// N consecutive values of a head's row, from dim d0 on, without the cache's scale.
template <int KT, int D, int N>
__device__ __forceinline__ void cache_values(const TreeLaunch& p, const void* cache, long long head_row,
                                             int d0, float (&f)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int d = d0 + e;
    if constexpr (KT == DA_KV_BF16) {
      f[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(cache)[head_row * D + d]);
    } else {
      const uint8_t* c = static_cast<const uint8_t*>(cache);
      uint32_t byte;
      if constexpr (KT == DA_KV_FP8_E4M3)
        byte = c[head_row * D + d];
      else
        byte = c[p.kv_rows * p.H_kv * (D / 2) + head_row * (D / 16) + d / 16];
      f[e] = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(byte) & 0xffffu)));
      if constexpr (KT == DA_KV_NVFP4) {
        const uint32_t code = c[head_row * (D / 2) + d / 2] >> (4 * (d & 1)) & 15u;
        uint32_t h[4];
        e2m1x8_to_f16x2(code, h);
        f[e] *= __half2float(__ushort_as_half((unsigned short)(h[0] & 0xffffu)));
      }
    }
  }
}

// One warp: softmax attention of (row b, node t, head hq) over tiles [begin, end) of the
// row's list, straight from the formula, entry by entry; lane l has dims [l D/32, + D/32).
// m: reference value (log2), l: sum, o: the weighted sum.
template <int KT, int D>
__device__ __noinline__ void attend_plainly(const TreeLaunch& p, const TreeRow& r, int b, int t, int hq, int begin,
                               int end, int lane, float* m_out, float* l_out, float (&o)[D / 32]) {
  constexpr int N = D / 32;
  int depth;
  const unsigned long long anc = ancestors(p, b, t, &depth);
  float q[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    q[e] = __bfloat162float(p.q[(((long long)b * p.T + t) * p.H_q + hq) * D + lane * N + e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  for (int i = begin; i < end; ++i) {
    const int j0 = tree_tile(r, i) * kTreeTile, j1 = min(j0 + kTreeTile, r.end);
    for (int j = j0; j < j1; ++j) {
      bool sees;
      if (j < r.length) {
        sees = !p.window || j < p.sinks || j > r.length + depth - p.window;
      } else {
        const int a = j - r.length;
        sees = anc >> a & 1;
        if (sees && p.window && a != t) {
          int a_depth;
          ancestors(p, b, a, &a_depth);
          sees = depth - a_depth < p.window || r.length + a_depth < p.sinks;
        }
      }
      if (!sees) continue;
      const long long row = cache_row(p, b, j);
      if (row < 0) {
        bad = true;
        continue;
      }
      float k[N], v[N], s = 0.f;
      cache_values<KT, D>(p, p.k, row * p.H_kv + hq / p.G, lane * N, k);
      cache_values<KT, D>(p, p.v, row * p.H_kv + hq / p.G, lane * N, v);
#pragma unroll
      for (int e = 0; e < N; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float m_new = s > m ? s : m;  // (a NaN moves nothing and stays in the sum)
      const float alpha = m_new == m ? 1.f : ex2(m - m_new);
      const float w = ex2(s - (m_new == -INFINITY ? 0.f : m_new));
      l = fmaf(l, alpha, w);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = fmaf(o[e], alpha, w * v[e]);
      m = m_new;
    }
  }
  if (bad && p.err && lane == 0) atomicOr(p.err, DA_DEVERR_INDEX);
  *m_out = m;
  *l_out = l;
}

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void report(int32_t* err, int bits) {
  if (err) atomicOr(err, bits);
}

// A unit of work: tiles [begin, end) of row b's list, KV head h, (node, head) rows
// row0 .. row0 + rows - 1 of the row's.
struct Unit {
  TreeRow r;
  int b, h, split, begin, end, row0, rows;
  __device__ __forceinline__ int tiles() const { return end - begin; }
};

struct UnitTable {
  const int2* sizes;
  const int* first;
  int units;
};

// The units of the launch's rows, counted by every block for itself: sizes gets each row's
// length, nodes and splits, first its first unit.  The first block reports what is out of
// range.  All `threads` threads; the caller synchronizes behind it.  A row can have nodes and
// no tile: it fills its capacity, so that the nodes' own entries lie beyond it, and their
// window holds no other.  kEmptyApart: such a row gets no unit and no split.
template <bool kEmptyApart>
__device__ __forceinline__ void count_units(const TreeLaunch& p, int2* sizes, int* first, int threads) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int bad = 0;
  for (int i = threadIdx.x; i < p.rows; i += threads) {
    const int2 s = tree_size(p, p.row0 + i, &bad);
    const TreeRow r = tree_row(p, s.x, s.y);
    const int splits = kEmptyApart && r.tiles == 0 ? 0 : r.splits;
    sizes[i] = make_int2(s.x, s.y | splits << 8);
    first[i + 1] = splits * r.supers * p.H_kv;
  }
  if (blockIdx.x == 0) {  // inputs that are out of range
    if (p.parents)
      for (int i = threadIdx.x; i < p.rows * p.T; i += threads) {
        const int t = i % p.T, up = __ldg(p.parents + (long long)p.row0 * p.T + i);
        if (t < (p.counts ? __ldg(p.counts + p.row0 + i / p.T) : p.T) && (up < -1 || up >= t)) bad |= DA_DEVERR_INDEX;
      }
    if (bad) report(p.err, bad);
  }
  __syncthreads();
  if (warp == 0) {
    int sum = 0;
    for (int i0 = 0; i0 < p.rows; i0 += 32) {
      int v = i0 + lane < p.rows ? first[i0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (i0 + lane < p.rows) first[i0 + lane + 1] = sum + v;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) first[0] = 0;
  }
}

__device__ __forceinline__ Unit unit_of(const TreeLaunch& p, const UnitTable& c, int u) {
  int lo = 0, hi = p.rows;  // the row with first[row] <= u < first[row + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.first[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  Unit x;
  const int2 size = c.sizes[lo];
  x.r = tree_row(p, size.x, size.y & 0xff, size.y >> 8);
  x.b = p.row0 + lo;
  u -= c.first[lo];
  x.row0 = 0;
  const int supers = (x.r.nodes * p.G + kTreeSuper - 1) / kTreeSuper;
  if (supers > 1) {
    const int v = u / supers;
    x.row0 = (u - v * supers) * kTreeSuper;
    u = v;
  }
  x.split = quotient(u, p.by_heads);
  x.h = u - x.split * p.H_kv;
  x.begin = x.split * x.r.per_split;
  x.end = min(x.begin + x.r.per_split, x.r.tiles);
  x.rows = min(kTreeSuper, x.r.nodes * p.G - x.row0);
  return x;
}

// Low n bits.
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Bits of the tile's entries (from j0 on) that no node of the row sees.
__device__ __forceinline__ unsigned long long hidden_bits(const TreeRow& r, int j0) {
  unsigned long long hid = ~low_bits(r.end - j0);
  if (r.hole_to > j0) hid |= low_bits(r.hole_to - j0) & ~low_bits(r.hole_from - j0);
  return hid;
}

// Bits of the nodes that a node with these ancestors sees (see decode_attn.h): the i-th of
// them from below is at depth i.
__device__ __forceinline__ unsigned long long windowed(const TreeLaunch& p, const TreeRow& r,
                                                       unsigned long long anc, int depth) {
  if (!p.window || p.window > depth) return anc;
  unsigned long long keep = anc, left = anc;
  for (int i = 0; i <= depth - p.window; ++i, left &= left - 1)
    if (r.length + i >= p.sinks) keep &= ~(left & (0 - left));
  return keep;
}

}  // namespace
}  // namespace da
