// Launch descriptors of the cache moves (moves.cu).
#pragma once

#include "common.cuh"

namespace da {

constexpr int kMoveRegions = 128;  // buffers a launch takes at most (1 KB of arguments)

// Buffers of equal geometry: the K and V caches of some layers, or their block
// scales.  An entry's bytes lie together, entry after entry.
struct MoveRegions {
  uint8_t* base[kMoveRegions];
  int n;
  int entry_bytes;
};

struct CopyPagesLaunch {
  MoveRegions regions;
  const int32_t* src;
  const int32_t* dst;
  int32_t* err;
  long long num_blocks;
  long long page_bytes;
  int n;
  int word;      // bytes of an access: 16 or 4
  int report;    // set *err (one launch of a call does)
};

struct CompactLaunch {
  MoveRegions regions;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* nodes;
  const int32_t* accepted;
  int32_t* new_lengths;
  int32_t* err;
  long long num_blocks, capacity;
  int B, nodes_width, layout, page_size, width;
  int word;
  int report;  // set *err and write new_lengths
};

cudaError_t launch_copy_pages(const CopyPagesLaunch& p, cudaStream_t stream);
cudaError_t launch_compact(const CompactLaunch& p, cudaStream_t stream);

}  // namespace da
