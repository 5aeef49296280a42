// Entries of the caches of all layers moved: pages copied for a fork, and the
// entries of accepted drafted tokens moved to the places behind their context.
//
// Pure data movement: each byte is read once and written once, so memory bounds a
// large copy and launch latency and a few dependent loads a small one.  One launch
// takes up to 128 buffers (K and V of 64 layers), so that a step over a whole model
// is one launch, not one a layer.  Measured: 256 pages of 16 entries (8 heads of 128,
// bf16) in 16 layers, 66 us = 8.1 TB/s read and written (the copies stay in part in the
// L2); the accepted entries of 64 rows of 16 nodes in 32 layers, 9.3 us against 4.9 at
// the measured bandwidth: a launch, then a row's nodes, its table and its words, each
// load waiting for the one before.
#include "moves.cuh"

#include <algorithm>

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;   // accesses a thread has in flight (copies)
constexpr int kMostNodes = 64;
constexpr int kBatch = 8;      // moves of a row whose loads go out together

// CTA (x, pair, region): the x-th piece of the page src[pair] to dst[pair].
template <typename W>
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyPagesLaunch p) {
  wait_prior_grid();
  const int pair = blockIdx.y;
  const int src = __ldg(p.src + pair), dst = __ldg(p.dst + pair);
  if (src < 0 || dst < 0 || src == dst) return;  // nothing to copy
  if (src >= p.num_blocks || dst >= p.num_blocks) {
    if (p.err && p.report && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
      atomicOr(p.err, DA_DEVERR_INDEX);
    return;
  }
  uint8_t* base = p.regions.base[blockIdx.z];
  const W* from = reinterpret_cast<const W*>(base + src * p.page_bytes);
  W* to = reinterpret_cast<W*>(base + dst * p.page_bytes);
  const long long words = p.page_bytes / (int)sizeof(W);
  long long at = (long long)blockIdx.x * (kThreads * kInFlight) + threadIdx.x;
  W w[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i)
    if (at + i * kThreads < words) w[i] = from[at + i * kThreads];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i)
    if (at + i * kThreads < words) to[at + i * kThreads] = w[i];
}

// CTA (x, row, z): the x-th column of words of the row's entries, in region z.  A
// thread moves its own word of every entry, in the order of the places.  Places never
// lie behind the nodes that go there (nodes ascend), so a batch's stores clobber no
// word that a later batch reads, and within a batch all loads come first.
template <typename W>
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactLaunch p) {
  __shared__ long long from[kMostNodes], to[kMostNodes];
  __shared__ int n_moves;
  wait_prior_grid();
  const int b = blockIdx.y;
  const bool first = p.report && blockIdx.x == 0 && blockIdx.z == 0;
  int bad = 0;
  // warp 0: lane l looks at nodes l and l + 32 of the row
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const long long length = __ldg(p.lengths + b);
    const int accepted = __ldg(p.accepted + b);
    const int32_t* nodes = p.nodes + (long long)b * p.nodes_width;
    const bool none = __ldg(nodes) < 0;
    const long long L = length < 0 ? 0 : length > p.capacity ? p.capacity : length;
    if (L != length) bad |= DA_DEVERR_LENGTH;
    if (accepted < 0 || accepted >= p.nodes_width) bad |= DA_DEVERR_LENGTH;
    const int m = none || bad ? 0 : accepted + 1;
    long long src[2] = {-1, -1}, dst[2] = {-1, -1};
    int stay = 0;  // nodes that are where they belong
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      if (i >= m) continue;
      const int node = __ldg(nodes + i), before = i ? __ldg(nodes + i - 1) : -1;
      if (node <= before || node >= p.nodes_width || L + node >= p.capacity) {
        bad |= DA_DEVERR_INDEX;
      } else if (node == i) {
        ++stay;  // all from the first on: nodes ascend
      } else {
        const long long j[2] = {L + node, L + i};
        long long* place[2] = {&src[h], &dst[h]};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (p.layout == DA_KV_CONTIGUOUS) {
            *place[e] = (long long)b * p.width + j[e];
            continue;
          }
          const long long page = p.layout == DA_KV_PAGED ? j[e] / p.page_size : j[e];
          const int id = __ldg(p.table + (long long)b * p.width + page);
          if (id < 0 || id >= p.num_blocks) bad |= DA_DEVERR_INDEX;
          *place[e] = p.layout == DA_KV_PAGED ? (long long)id * p.page_size + (j[e] - page * p.page_size)
                                              : (long long)id;
        }
      }
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    stay = __reduce_add_sync(0xffffffffu, stay);
    if (lane == 0) {
      n_moves = bad ? 0 : m - stay;
      if (first) {
        if (bad && p.err) atomicOr(p.err, bad);
        if (p.new_lengths) p.new_lengths[b] = (int)(L + (bad ? 0 : m));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h - stay;
      if (!bad && i >= 0 && lane + 32 * h < m) {
        from[i] = src[h];
        to[i] = dst[h];
      }
    }
  }
  __syncthreads();
  const int n = n_moves;
  const int words = p.regions.entry_bytes / (int)sizeof(W);
  const int at = blockIdx.x * kThreads + threadIdx.x;
  if (n == 0 || at >= words) return;
  W* base = reinterpret_cast<W*>(p.regions.base[blockIdx.z]) + at;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    W w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < n) w[i] = base[from[i0 + i] * words];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < n) base[to[i0 + i] * words] = w[i];
  }
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesLaunch& p, cudaStream_t stream) {
  const long long per = (long long)kThreads * kInFlight * p.word;
  const long long x = (p.page_bytes + per - 1) / per;
  if (x > 0x7fffffffLL) return cudaErrorInvalidValue;
  CopyPagesLaunch q = p;
  for (int done = 0; done < p.n; done += 65535) {  // the grid's limit
    q.src = p.src + done;
    q.dst = p.dst + done;
    const dim3 grid((unsigned)x, (unsigned)std::min(65535, p.n - done), (unsigned)p.regions.n);
    const cudaError_t e = p.word == 16 ? launch_after(copy_pages_kernel<uint4>, grid, dim3(kThreads), 0, stream, q)
                                       : launch_after(copy_pages_kernel<uint32_t>, grid, dim3(kThreads), 0, stream, q);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_compact(const CompactLaunch& p, cudaStream_t stream) {
  const int words = p.regions.entry_bytes / p.word;
  const unsigned x = (unsigned)((words + kThreads - 1) / kThreads);
  CompactLaunch q = p;
  for (int done = 0; done < p.B; done += 65535) {
    // (rows are found from b: the arrays move on, the caches of a contiguous layout too)
    q.table = p.table ? p.table + (long long)done * p.width : nullptr;
    q.lengths = p.lengths + done;
    q.nodes = p.nodes + (long long)done * p.nodes_width;
    q.accepted = p.accepted + done;
    q.new_lengths = p.new_lengths ? p.new_lengths + done : nullptr;
    if (p.layout == DA_KV_CONTIGUOUS)
      for (int r = 0; r < p.regions.n; ++r)
        q.regions.base[r] = p.regions.base[r] + (long long)done * p.width * p.regions.entry_bytes;
    const dim3 grid(x, (unsigned)std::min(65535, p.B - done), (unsigned)p.regions.n);
    const cudaError_t e = p.word == 16 ? launch_after(compact_kernel<uint4>, grid, dim3(kThreads), 0, stream, q)
                                       : launch_after(compact_kernel<uint32_t>, grid, dim3(kThreads), 0, stream, q);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace da
