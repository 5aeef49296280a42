// Launch descriptor and row geometry of the tree attention (tree.cu).
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace da {

constexpr int kTreeTile = 64;       // entries of a tile
constexpr int kTreeMaxSplits = 64;  // pieces of a row's list at most
constexpr int kTreeSuper = 128;     // (node, head) rows of a unit at most

// n / d for n below 2^31 by a multiplication: a unit's place is found with several
// divisions, of 40 or so dependent instructions each otherwise.
struct FastDiv {
  uint32_t d, mul, shift;
};

inline FastDiv fast_div(uint32_t d) {
  FastDiv f = {d, 0, 0};
  if (d > 1) {
    while ((1u << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)((1ull << (31 + f.shift)) / d + 1);
    --f.shift;
  }
  return f;
}

struct TreeLaunch {
  const __nv_bfloat16* q;
  const void* k;
  const void* v;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* counts;   // null: T
  const int32_t* parents;  // null: a chain
  __nv_bfloat16* out;
  float* lse;
  int32_t* err;
  float* lse_part;  // [B * max_splits][T][H_q], log2 units
  float* o_part;    // [B * max_splits][T][H_q][D]
  long long num_blocks;
  long long kv_rows;  // entries in a cache (NVFP4: its block scales follow its codes)
  int B, T, H_q, H_kv, G, D;
  int layout, page_size, width, capacity, kv_type;
  int window;  // 0: none
  int sinks;
  int max_splits;    // of this problem: the partials' stride
  float scale_log2;  // softmax scale * log2(e) * k_scale
  float v_scale;
  int test_stall;
  int row0, rows;  // the rows of this launch
  FastDiv by_heads, by_group, by_page;  // H_kv, G, page_size
};

constexpr int kTreeRows = 256;  // rows of a launch at most

// A tensor map of bytes or bf16 (rank 2 or 3); false if the driver has none.
bool tree_tensor_map(CUtensorMap* tm, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box, bool bytes, CUtensorMapSwizzle swizzle);

cudaError_t launch_tree(const TreeLaunch& p, int sms, cudaStream_t stream);
cudaError_t launch_tree_few(const TreeLaunch& p, int sms, cudaStream_t stream);
cudaError_t launch_tree_combine(const TreeLaunch& p, cudaStream_t stream);

// Whether tree_few.cu takes a call with this many (node, head) rows a KV head at most, whose
// cost grows with the rows, where tree.cu's is the same up to 128.  A windowed step of 64 rows
// with 4096 entries each and 8 KV heads, here against there, in us: 16 rows E4M3 206, 424, bf16
// 223, 268; 32 rows E4M3 306, 438, NVFP4 305, 625, bf16 321, 281; 24 rows bf16 251, 273; 32 rows
// of 64 dims, bf16, 196, 233.
inline bool tree_takes_few(int kv_type, int D, int rows) {
  return rows <= (kv_type == DA_KV_BF16 && D == 128 ? 24 : 32);
}

// Tiles of a split at least, for a row of `rows` (node, head) pairs a KV head.  A split
// costs its rows' fp32 partials, written and read again, so that many rows want long
// splits; few rows want short ones, which more SMs share.
__host__ __device__ inline int tree_min_tiles(int rows) { return rows <= 32 ? 8 : 16; }
constexpr int kTreeLeastTiles = 8;

#ifdef __CUDACC__

__device__ __forceinline__ int quotient(int n, const FastDiv& f) {
  return f.d == 1 ? n : (int)(__umulhi((uint32_t)n, f.mul) >> f.shift);
}

// What a row attends to.  It follows from the row's own length, number of nodes and
// the call's window alone.
struct TreeRow {
  int length, nodes;   // clamped
  int end;             // entries of the row's list
  int hole_from, hole_to;  // entries that no node sees (hole_from < hole_to), or none
  int head_tiles, skip;  // tile i of the list is tile i (+ skip from head_tiles on)
  int tiles, per_split, splits, supers;
};

// `splits`: their number where it is known.
__device__ __forceinline__ TreeRow tree_row(const TreeLaunch& p, int length, int nodes, int splits = 0) {
  TreeRow r;
  r.length = length;
  r.nodes = nodes;
  r.end = min(r.length + r.nodes, p.capacity);
  r.hole_from = r.hole_to = 0;
  r.head_tiles = r.skip = 0;
  const int all = (r.end + kTreeTile - 1) / kTreeTile;
  if (p.window) {  // the first node sees furthest back: its depth is 0
    const int first = min(r.length - p.window + 1, r.end);
    if (first > p.sinks) {
      r.hole_from = p.sinks;
      r.hole_to = first;
      r.head_tiles = (p.sinks + kTreeTile - 1) / kTreeTile;
      r.skip = max(0, first / kTreeTile - r.head_tiles);
    }
  }
  r.tiles = all - r.skip;
  const int rows = r.nodes * p.G;
  r.per_split = max(tree_min_tiles(rows), (r.tiles + kTreeMaxSplits - 1) / kTreeMaxSplits);
  r.splits = splits ? splits : max(1, (r.tiles + r.per_split - 1) / r.per_split);
  r.supers = (rows + kTreeSuper - 1) / kTreeSuper;
  return r;
}

// The length and number of nodes of row b, clamped; *bad gets the error bit.
__device__ __forceinline__ int2 tree_size(const TreeLaunch& p, int b, int* bad) {
  const int length = __ldg(p.lengths + b), nodes = p.counts ? __ldg(p.counts + b) : p.T;
  const int2 s = make_int2(clamp_len(length, p.capacity), clamp_len(nodes, p.T));
  if (s.x != length || s.y != nodes || s.x + s.y > p.capacity) *bad |= DA_DEVERR_LENGTH;
  return s;
}

__device__ __forceinline__ int tree_tile(const TreeRow& r, int i) {
  return i < r.head_tiles ? i : i + r.skip;
}

#endif  // __CUDACC__

}  // namespace da
