// Attention of a tree of drafted tokens over the caches: every node of a row attends
// to the row's context and to its own ancestors.
#include <algorithm>
#include <cstring>

#include "merge.cuh"
#include "tree.cuh"

namespace da {
namespace {

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
  const int at = p.layout == DA_KV_PAGED ? j / p.page_size : j;
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
__device__ void attend_plainly(const TreeLaunch& p, const TreeRow& r, int b, int t, int hq, int begin,
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
      const float w = s == m_new ? 1.f : ex2(s - m_new);
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

constexpr int kWarps = 8;

// A warp for each (split, row, node, head).
template <int KT, int D>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const TreeLaunch p) {
  constexpr int N = D / 32;
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int hq = (int)(task % p.H_q), t = (int)(task / p.H_q % p.T);
  const int s = (int)(task / p.H_q / p.T % p.max_splits);
  const long long b = task / p.H_q / p.T / p.max_splits;
  if (b >= p.B) return;
  const TreeRow r = tree_row(p, (int)b);
  if (t >= r.nodes || s >= r.splits) return;
  float m, l, o[N];
  attend_plainly<KT, D>(p, r, (int)b, t, hq, s * r.per_split, min((s + 1) * r.per_split, r.tiles), lane, &m, &l, o);
  const float inv = (l > 0.f ? 1.f / l : l != l ? l : 0.f) * p.v_scale;
  const float lse = l > 0.f || l != l ? m + lg2(l) : -INFINITY;
  const long long row = (b * p.T + t) * p.H_q + hq, slot = ((b * p.max_splits + s) * p.T + t) * p.H_q + hq;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (r.splits == 1)
      p.out[row * D + lane * N + e] = __float2bfloat16_rn(o[e] * inv);
    else
      p.o_part[slot * D + lane * N + e] = o[e] * inv;
  }
  if (lane == 0) {
    if (r.splits == 1)
      p.lse[row] = lse * kLn2;
    else
      p.lse_part[slot] = lse;
  }
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
  const TreeRow r = tree_row(p, b);
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
  const float lse = merge_weights(p.lse_part + slot, per, r.splits, coef[warp], lane);
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.f;
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

template <int KT>
cudaError_t launch_kt(const TreeLaunch& p, cudaStream_t stream) {
  const long long warps = (long long)p.B * p.max_splits * p.T * p.H_q;
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
  return p.D == 64 ? launch_after(tree_kernel<KT, 64>, dim3(grid), dim3(kWarps * 32), 0, stream, p)
                   : launch_after(tree_kernel<KT, 128>, dim3(grid), dim3(kWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_tree(const TreeLaunch& p, int sms, cudaStream_t stream) {
  switch (p.kv_type) {
    case DA_KV_FP8_E4M3: return launch_kt<DA_KV_FP8_E4M3>(p, stream);
    case DA_KV_NVFP4: return launch_kt<DA_KV_NVFP4>(p, stream);
    default: return launch_kt<DA_KV_BF16>(p, stream);
  }
}

cudaError_t launch_tree_combine(const TreeLaunch& p, cudaStream_t stream) {
  const long long warps = (long long)p.B * p.T * p.H_q;
  const dim3 grid((unsigned)((warps + kCombineWarps - 1) / kCombineWarps));
  return p.D == 64 ? launch_after(tree_combine_kernel<64>, grid, dim3(kCombineWarps * 32), 0, stream, p)
                   : launch_after(tree_combine_kernel<128>, grid, dim3(kCombineWarps * 32), 0, stream, p);
}

}  // namespace da
