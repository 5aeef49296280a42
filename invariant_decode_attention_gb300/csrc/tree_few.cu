// Tree attention of few (node, head) rows a KV head: a plain decode step's, or a short
// chain's with small groups.
#include "tree_parts.cuh"

namespace da {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = kT / kWarps;  // entries of a tile that a warp has: the M of an MMA

// What a thread of a warp holds, lane 4 g + q: entries g and g + 8 of K (D / 4 dims, in
// pieces of 16 bytes or one smaller one), entries 2 q, 2 q + 1, 2 q + 8, 2 q + 9 of V (D / 8
// dims).
template <int KT, int D, int NT>
struct Few {
  static constexpr bool Q8 = KT != DA_KV_BF16;
  static constexpr int kRow = KT == DA_KV_BF16 ? 2 * D : KT == DA_KV_FP8_E4M3 ? D : D / 2;  // bytes of a head's row
  static constexpr int kKWords = kRow / 16, kVWords = kRow / 32;
  static constexpr int kKPiece = kKWords < 4 ? kKWords : 4, kVPiece = kVWords < 4 ? kVWords : 4;  // words of a load
  static constexpr int kKDims = kKPiece * 4 * D / kRow, kVDims = kVPiece * 4 * D / kRow;          // dims of a load
  static constexpr int kRows = 8 * NT;
  static constexpr int kPad = D + 4;
  static constexpr int kOutBytes = kWarps * kRows * kPad * 4;
  static constexpr int kResident = NT == 1 ? (Q8 || D == 64 ? 4 : 3) : 2;  // blocks an SM
};

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* from, uint32_t* w) {
  if constexpr (W == 4)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(from));
  else if constexpr (W == 2)
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(from));
  else
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(from));
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

// 16 entries of K and V, a warp's of a tile, as they lie in the cache.
template <int KT, int D, int NT>
struct Held {
  using F = Few<KT, D, NT>;
  uint32_t k[2][F::kKWords], v[4][F::kVWords];
  uint32_t ks[2], vs[4];  // NVFP4: block scales

  // `rows`: lane half + i has entry i's cache row, or -1 (zeros then)
  __device__ __forceinline__ void load_k(const TreeLaunch& p, int h, int rows, int half, int lane) {
    const int q = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = __shfl_sync(0xffffffffu, rows, half + (lane >> 2) + 8 * e);
#pragma unroll
      for (int i = 0; i < F::kKWords; ++i) k[e][i] = 0;
      ks[e] = 0;
      if (row < 0) continue;
      const long long at = (long long)row * p.H_kv + h;
      const uint8_t* from = static_cast<const uint8_t*>(p.k) + at * F::kRow + q * (F::kKPiece * 4);
#pragma unroll
      for (int i = 0; i < F::kKWords; i += F::kKPiece) load_words<F::kKPiece>(from + 16 * i, k[e] + i);
      if constexpr (KT == DA_KV_NVFP4) {
        const uint8_t* s = static_cast<const uint8_t*>(p.k) + p.kv_rows * p.H_kv * F::kRow + at * (D / 16);
        ks[e] = D == 128 ? __ldg(reinterpret_cast<const uint16_t*>(s) + q) : __ldg(s + q);
      }
    }
    __syncwarp();
  }

  __device__ __forceinline__ void load_v(const TreeLaunch& p, int h, int rows, int half, int lane) {
    const int g = lane >> 2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = __shfl_sync(0xffffffffu, rows, half + 2 * (lane & 3) + (e & 1) + 4 * (e & 2));
#pragma unroll
      for (int i = 0; i < F::kVWords; ++i) v[e][i] = 0;
      vs[e] = 0;
      if (row < 0) continue;
      const long long at = (long long)row * p.H_kv + h;
      const uint8_t* from = static_cast<const uint8_t*>(p.v) + at * F::kRow + g * (F::kVPiece * 4);
#pragma unroll
      for (int i = 0; i < F::kVWords; i += F::kVPiece) load_words<F::kVPiece>(from + 32 * i, v[e] + i);
      if constexpr (KT == DA_KV_NVFP4) {
        const uint8_t* s = static_cast<const uint8_t*>(p.v) + p.kv_rows * p.H_kv * F::kRow + at * (D / 16);
        vs[e] = __ldg(s + g * (D / 8) / 16);
      }
    }
    __syncwarp();
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

template <int KT, int D, int NT>
__global__ void __launch_bounds__(kThreads, Few<KT, D, NT>::kResident) few_kernel(const TreeLaunch p) {
  using F = Few<KT, D, NT>;
  extern __shared__ __align__(16) float parts[];  // [kWarps][kRows][kPad]: the warps' sums
  __shared__ int2 sizes[kTreeRows];
  __shared__ int first[kTreeRows + 1];
  __shared__ Unit units[kWarps][2];
  __shared__ unsigned long long sees[F::kRows];  // nodes that a row sees
  __shared__ int depths[F::kRows];
  __shared__ float part_m[kWarps][F::kRows], part_l[kWarps][F::kRows];
  __shared__ uint32_t odd_rows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  wait_prior_grid();
  allow_next_grid();
  count_units(p, sizes, first, kThreads);
  __syncthreads();
  UnitTable c;
  c.sizes = sizes;
  c.first = first;
  c.units = first[p.rows];
  if ((int)blockIdx.x >= c.units) return;

  bool bad = false;
  // cache rows of this warp's entries of tiles i and i + 1 of a unit, lane 16 t + e
  auto look_up = [&](const Unit* x, int i) -> int {
    i += lane >> 4;
    if (i >= x->end) return -1;
    const int j = tree_tile(x->r, i) * kT + warp * kStep + (lane & 15);
    if (j >= x->r.end || (j >= x->r.hole_from && j < x->r.hole_to)) return -1;
    const long long row = cache_row(p, x->b, j);
    bad |= row < 0;
    return (int)row;
  };
  const Unit first_unit = unit_of(p, c, blockIdx.x);
  if (lane == 0) units[warp][0] = first_unit;
  __syncwarp();
  Held<KT, D, NT> held;
  int rows = look_up(&units[warp][0], first_unit.begin);
  held.load_k(p, first_unit.h, rows, 0, lane);
  held.load_v(p, first_unit.h, rows, 0, lane);
  for (int u = blockIdx.x, slot = 0; u < c.units; u += gridDim.x, slot ^= 1) {
    const Unit* x = &units[warp][slot];
    const Unit* next = &units[warp][slot ^ 1];
    const bool more = u + (int)gridDim.x < c.units;
    if (more) {
      const Unit z = unit_of(p, c, u + gridDim.x);
      if (lane == 0) units[warp][slot ^ 1] = z;
    }
    __syncwarp();
    const int n_rows = x->rows, h = x->h, begin = x->begin, end = x->end, length = x->r.length;
    // ---- Q, and what the rows see
    uint32_t qb[NT][D / 16][2];
    float scale[NT][2];  // softmax scales of rows 8 nt + 2 q and + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int at = nt * 8 + g;
      float mine = p.scale_log2;
      const bool live = at < n_rows;
      const int t = live ? quotient(at, p.by_group) : 0;
      const __nv_bfloat16* from = p.q + ((size_t)((long long)x->b * p.T + t) * p.H_q + h * p.G + (at - t * p.G)) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        constexpr int kPer = F::kKDims / 4;  // k-steps of a piece
        const int d = (s / kPer) * (4 * F::kKDims) + q * F::kKDims + 4 * (s % kPer);
        const uint2 w = live ? __ldg(reinterpret_cast<const uint2*>(from + d)) : make_uint2(0, 0);
        qb[nt][s][0] = w.x;
        qb[nt][s][1] = w.y;
      }
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
      scale[nt][0] = __shfl_sync(0xffffffffu, mine, 8 * q);
      scale[nt][1] = __shfl_sync(0xffffffffu, mine, 8 * q + 4);
    }
    if (threadIdx.x < F::kRows) {
      const int at = threadIdx.x;
      int depth = 0;
      unsigned long long anc = 0;
      if (at < n_rows) {
        anc = ancestors(p, x->b, quotient(at, p.by_group), &depth);
        anc = windowed(p, x->r, anc, depth) & low_bits(x->r.end - length);
      }
      sees[at] = anc;
      depths[at] = depth;
    }
    if (threadIdx.x == 0) odd_rows = 0;
    __syncthreads();
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
      // ---- scores: entries g and g + 8, rows 8 nt + 2 q and + 1
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t a[4];
        held.k_operand(k, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816<F::Q8>(s[nt], a, qb[nt][k][0], qb[nt][k][1]);
      }
      // the next tile's K, and behind it the V, of this unit or the next one
      const int odd = (i - begin) & 1;
      const bool last = i + 1 == end;
      int h_next = h;
      if (last) {
        if (more) {
          rows = look_up(next, next->begin);
          h_next = next->h;
        }
      } else if (odd) {
        rows = look_up(x, i + 1);
      }
      const int half = last || odd ? 0 : 16;
      if (!last || more) held.load_k(p, h_next, rows, half, lane);

      const int j0 = tree_tile(x->r, i) * kT;
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
        held.v_operands(j4, a);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816<F::Q8>(o[nt][4 * j4 + j], a[j], pb[nt][0], pb[nt][1]);
      }
      if (!last || more) held.load_v(p, h_next, rows, half, lane);
    }
    if (end == begin && more) {  // (nothing has brought in the next unit's)
      rows = look_up(next, next->begin);
      held.load_k(p, next->h, rows, 0, lane);
      held.load_v(p, next->h, rows, 0, lane);
    }
    // ---- the warps' sums joined, in their order
    float* mine = parts + warp * F::kRows * F::kPad;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int at = nt * 8 + 2 * q + r;
        float sum = l[nt][r];
#pragma unroll
        for (int b = 4; b < 32; b <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
        if (g == 0) {
          part_m[warp][at] = m[nt][r];
          part_l[warp][at] = sum;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          constexpr int kPer = F::kVDims / 2;  // tiles of a piece
          const int d = (j / kPer) * (8 * F::kVDims) + g * F::kVDims + 2 * (j % kPer);
          *reinterpret_cast<float2*>(mine + at * F::kPad + d) = make_float2(o[nt][j][r], o[nt][j][2 + r]);
        }
      }
    __syncthreads();
    const bool single = x->r.splits == 1;
    const long long to_slot = (((long long)x->b * p.max_splits + x->split) - x->b) * p.T * p.H_q;
    for (int i = threadIdx.x; i < n_rows * (D / 4); i += kThreads) {
      const int at = i / (D / 4), d = 4 * (i % (D / 4));
      float top = -INFINITY, sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w][at]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float c_w = part_m[w][at] == top ? 1.f : ex2(part_m[w][at] - top);
        const float4 o_w = *reinterpret_cast<const float4*>(parts + (w * F::kRows + at) * F::kPad + d);
        sum = fmaf(part_l[w][at], c_w, sum);
        v.x = fmaf(o_w.x, c_w, v.x);
        v.y = fmaf(o_w.y, c_w, v.y);
        v.z = fmaf(o_w.z, c_w, v.z);
        v.w = fmaf(o_w.w, c_w, v.w);
      }
      const float inv = (sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f) * p.v_scale;
      v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      const int t = quotient(at, p.by_group);
      const size_t row = (size_t)((long long)x->b * p.T + t) * p.H_q + h * p.G + (at - t * p.G);
      if (sum != sum || !(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w) < INFINITY)) atomicOr(&odd_rows, 1u << at);
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
    // rows that something infinite or NaN has spoiled: formed again, entry by entry
    uint32_t again = odd_rows;
    for (int n = 0; again; again &= again - 1, ++n) {
      if (n % kWarps != warp) continue;
      const int at = __ffs((int)again) - 1, t = quotient(at, p.by_group), head = h * p.G + (at - t * p.G);
      const size_t row = (size_t)((long long)x->b * p.T + t) * p.H_q + head;
      float m2, l2, o2[D / 32];
      attend_plainly<KT, D>(p, x->r, x->b, t, head, begin, end, lane, &m2, &l2, o2);
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
    __syncthreads();  // (odd_rows, sees and parts are the next unit's now)
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.err, DA_DEVERR_INDEX);
}

template <int KT, int D, int NT>
cudaError_t launch_shape(const TreeLaunch& p0, int sms, cudaStream_t stream) {
  using F = Few<KT, D, NT>;
  static const cudaError_t attr =
      cudaFuncSetAttribute(few_kernel<KT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kOutBytes);
  if (attr != cudaSuccess) return attr;
  TreeLaunch p = p0;
  p.by_heads = fast_div(p.H_kv);
  p.by_group = fast_div(p.G);
  p.by_page = fast_div(p.page_size > 1 ? p.page_size : 1);
  for (p.row0 = 0; p.row0 < p.B; p.row0 += kTreeRows) {
    p.rows = p.B - p.row0 < kTreeRows ? p.B - p.row0 : kTreeRows;
    const long long most = (long long)p.rows * p.max_splits * p.H_kv, room = (long long)F::kResident * sms;
    const cudaError_t e = launch_after(few_kernel<KT, D, NT>, dim3((unsigned)(most < room ? most : room)), dim3(kThreads),
                                       (size_t)F::kOutBytes, stream, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int KT, int D>
cudaError_t launch_rows(const TreeLaunch& p, int sms, cudaStream_t stream) {
  return p.T * p.G <= 8 ? launch_shape<KT, D, 1>(p, sms, stream) : launch_shape<KT, D, 2>(p, sms, stream);
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
