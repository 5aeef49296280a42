// Drafted tokens verified against the target's probabilities, and the next token.
//
// The target's logits at every node are read once (memory bounds a large step):
//   1. rows_kernel, a CTA for each 8192 tokens of a node's row: their maximum, the
//      sum of exp((x - max) / temperature), the lowest token of the largest logit.
//   2. walk_kernel, a cluster for each request.  Every CTA merges its rows' parts,
//      forms the probability of every drafted token at its parent and walks down the
//      tree (one warp; its lanes hold the nodes); then the cluster samples the next
//      token from the row where the walk ended, whose logits are mostly in L2 still.
// The next token is the first one whose cumulative weight exceeds a share of the total.
// With 10^5 tokens the steps of that sum lie so close together that an fp32 sum's error
// would pick a neighbour in one row of a thousand, and sums in another order another
// one.  So weights are integers, 2^44 exp((x - max) / temperature) off by about 2^-38 of their
// size: their sums are exact in any order, and how a row is cut does not show.  The
// exponential is formed for that in two fp32 terms: x - max and its product with
// log2(e) / temperature without error, 2^(j / 64) from a table, and five terms of the
// series of exp for the rest, whose argument is below 2^-7.5.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "nvfp4_mm.h"

namespace da {
namespace {

constexpr int kRowThreads = 256;
constexpr int kVec = 4;                             // consecutive tokens of a load
constexpr int kLoads = 8;                           // loads of a thread
constexpr int kChunk = kRowThreads * kVec * kLoads;  // tokens of a CTA of rows_kernel
constexpr int kThreads = 512;                       // of walk_kernel
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;                         // CTAs of a request at most
constexpr int kNodes = NVFP4_VERIFY_MAX_NODES;
constexpr int kBlock = 32 * kVec;                   // tokens a warp takes at once
static_assert(kNodes == 64, "two nodes a lane");

struct Part {  // of a row's chunk
  float max, sum;
  int best, pad;
};

struct Args {
  const void* x;
  long long x_row, x_node;  // strides in elements: request, node
  const float* draft;
  long long draft_row, draft_node;
  const int32_t *tokens, *parents, *counts;
  const float *temperature, *uniforms, *final_uniforms;
  int32_t *accepted, *nodes, *out, *err;
  Part* parts;
  int B, T, V, chunks, slice;  // slice: tokens of a CTA of walk_kernel
};

// A row's temperature: 0 (greedy), or within what the arithmetic below takes.
__device__ __forceinline__ float temperature_of(const Args& a, int b) {
  const float t = a.temperature ? __ldg(a.temperature + b) : 1.f;
  return t > 0.f ? fminf(fmaxf(t, 0x1p-100f), 0x1p100f) : 0.f;
}

__device__ __forceinline__ int count_of(const Args& a, int b, int* bad) {
  const int n = a.counts ? __ldg(a.counts + b) : a.T, c = clamp_len(n, a.T);
  if (c != n) *bad |= DA_DEVERR_LENGTH;
  return c;
}

template <bool BF16>
__device__ __forceinline__ const void* row_of(const Args& a, int b, int t) {
  return static_cast<const char*>(a.x) + (b * a.x_row + t * a.x_node) * (BF16 ? 2 : 4);
}

// Whether groups of kVec tokens of a row lie on their natural boundaries.
template <bool BF16>
__device__ __forceinline__ bool in_step(const void* row) {
  return (reinterpret_cast<uintptr_t>(row) & (BF16 ? 7 : 15)) == 0;
}

template <bool BF16>
__device__ __forceinline__ float one(const void* row, long long v) {
  return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(row)[v])
              : static_cast<const float*>(row)[v];
}

// Tokens v .. v + 3 of a row, -inf past its end.  The same tokens for the same
// thread wherever the row lies.
template <bool BF16>
__device__ __forceinline__ void load4(const void* row, int v, int V, bool whole, float (&f)[kVec]) {
  if (whole && v + kVec <= V) {
    if (BF16) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(row) + v));
      f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
    } else {
      const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(row) + v));
      f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < kVec; ++e) f[e] = v + e < V ? one<BF16>(row, v + e) : -INFINITY;
}

template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const Args a) {
  __shared__ float warp_max[kRowThreads / 32], warp_sum[kRowThreads / 32];
  __shared__ int warp_best[kRowThreads / 32];
  wait_prior_grid();
  allow_next_grid();
  const long long task = blockIdx.x;
  const int chunk = (int)(task % a.chunks);
  const int t = (int)(task / a.chunks % a.T), b = (int)(task / a.chunks / a.T);
  int bad = 0;
  if (t >= count_of(a, b, &bad)) return;
  const float tau = temperature_of(a, b);
  const void* row = row_of<BF16>(a, b, t);
  const bool whole = in_step<BF16>(row);
  const int v0 = chunk * kChunk + threadIdx.x * kVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float f[kLoads][kVec];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) load4<BF16>(row, v0 + i * kRowThreads * kVec, a.V, whole, f[i]);
  float m = -INFINITY;  // (a NaN is none: it counts as -inf)
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
#pragma unroll
    for (int e = 0; e < kVec; ++e) m = fmaxf(m, f[i][e] = fmaxf(f[i][e], -INFINITY));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float sum = 0.f;
  int best = 0x7fffffff;
  if (tau > 0.f) {
    if (m > -INFINITY) {
      const float c = __fdiv_rn(kLog2e, tau);
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int e = 0; e < kVec; ++e)  // (infinite maximum: what equals it weighs 1)
          sum += f[i][e] == m ? 1.f : ex2((f[i][e] - m) * c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  } else {
#pragma unroll
    for (int i = kLoads - 1; i >= 0; --i)
#pragma unroll
      for (int e = kVec - 1; e >= 0; --e)
        if (f[i][e] == m) best = v0 + i * kRowThreads * kVec + e;
    best = __reduce_min_sync(0xffffffffu, best);
  }
  if (lane == 0) {
    warp_max[warp] = m;
    warp_sum[warp] = sum;
    warp_best[warp] = best;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Part p = {-INFINITY, 0.f, 0x7fffffff, 0};
    for (int w = 0; w < kRowThreads / 32; ++w) p.max = fmaxf(p.max, warp_max[w]);
    const float c = tau > 0.f ? __fdiv_rn(kLog2e, tau) : 0.f;
    for (int w = 0; w < kRowThreads / 32; ++w) {
      if (warp_max[w] == p.max) {
        p.sum += warp_sum[w];
        p.best = min(p.best, warp_best[w]);
      } else {
        p.sum += warp_sum[w] * ex2((warp_max[w] - p.max) * c);
      }
    }
    a.parts[task] = p;
  }
}

// round(2^62 * 2^(j / 64)), j = -32 .. 32
__device__ const unsigned long long kPowers[65] = {
    0x2d413cccfe779921ull, 0x2dbf6478ca345de4ull, 0x2e3eebd1d8bee7baull, 0x2ebfd6ac84cf917full,
    0x2f4228e7d6030db0ull, 0x2fc5e66d9e9cc421ull, 0x304b1332999c2516ull, 0x30d1b3368925d902ull,
    0x3159ca845541b6b7ull, 0x31e35d322aee6c57ull, 0x326e6f619b8bc9e9ull, 0x32fb053fbc9c9f17ull,
    0x3389230547e12039ull, 0x3418ccf6bbcac965ull, 0x34aa07647c4ab917ull, 0x353cd6aaf3fb7e88ull,
    0x35d13f32b5a75abdull, 0x366745709e2bf5edull, 0x36feede5f6bc8dd5ull, 0x37983d209783a449ull,
    0x383337bb0aa53844ull, 0x38cfe25cafa29694ull, 0x396e41b9df20d22aull, 0x3a0e5a940f12f71aull,
    0x3ab031b9f7490e4cull, 0x3b53cc07b6650ae1ull, 0x3bf92e66f736bd73ull, 0x3ca05dcf167fec4eull,
    0x3d495f454921b30bull, 0x3df437dcc2b44eeeull, 0x3ea0ecb6dc8a80cfull, 0x3f4f83033d21b05dull,
    0x4000000000000000ull, 0x40b268f9de0183baull, 0x4166c34c5615d0ecull, 0x421d1461d66f2023ull,
    0x42d561b3e6243d8aull, 0x438fb0cb4f468808ull, 0x444c0740496d4294ull, 0x450a6abaa4b77ecdull,
    0x45cae0f1f545eb73ull, 0x468d6fadbf2dd4f3ull, 0x47521cc5a2e6a9e0ull, 0x4818ee218a3358eeull,
    0x48e1e9b9d588e19bull, 0x49ad159789f37496ull, 0x4a7a77d47f7b84b1ull, 0x4b4a169b900c2d00ull,
    0x4c1bf828c6dc54b8ull, 0x4cf022c9905bfd32ull, 0x4dc69cdceaa72a9cull, 0x4e9f6cd3967fdba8ull,
    0x4f7a993048d088d7ull, 0x50582887dcb8a7e1ull, 0x513821818624b40cull, 0x521a8ad704f3404full,
    0x52ff6b54d8a89c75ull, 0x53e6c9da74b29ab5ull, 0x54d0ad5a753e077cull, 0x55bd1cdad49f699cull,
    0x56ac1f752150a563ull, 0x579dbc56b48521baull, 0x5891fac0e95612c8ull, 0x5988e20954889245ull,
    0x5a827999fcef3242ull
};

constexpr int kWeightBits = 44;

struct Scale {  // of the row that is sampled
  float max, c_hi, c_lo;  // log2(e) / temperature in two terms
};

__device__ __forceinline__ Scale scale_of(float max, float tau) {
  const double c = 1.4426950408889634 / (double)tau;
  Scale s;
  s.max = max;
  s.c_hi = (float)c;
  s.c_lo = (float)(c - (double)s.c_hi);
  return s;
}

// 2^44 exp((x - max) / temperature), an integer.
__device__ __forceinline__ unsigned long long weight(float x, const Scale& s,
                                                     const unsigned long long* powers) {
  if (x == s.max) return 1ull << kWeightBits;
  const float d = __fsub_rn(x, s.max);
  const float p = __fmul_rn(d, s.c_hi);
  if (!(p > -45.f)) return 0;  // nothing left of it (-inf and NaN among them)
  const float bb = __fsub_rn(d, x);  // the difference's rounding error (two-sum)
  const float d_lo = __fadd_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fsub_rn(-s.max, bb));
  const float p_lo = __fmaf_rn(d, s.c_hi, -p) + __fmaf_rn(d, s.c_lo, __fmul_rn(d_lo, s.c_hi));
  // p = k + j / 64 + r: k and j by rounding, r exactly
  const float k = rintf(p);
  const float f = __fsub_rn(p, k);
  const float j = rintf(__fmul_rn(f, 64.f));
  const float r = __fmaf_rn(j, -0.015625f, f);
  // z = (r + p_lo) ln 2 in two terms, then exp(z) - 1 = z + z^2 (1/2 + z/6 + z^2/24) + ...
  constexpr float kL = 0x1.62e4300000000p-1f, kLlo = -0x1.05c6100000000p-29f;
  const float z = __fmul_rn(r, kL);
  const float z_lo = __fmaf_rn(r, kL, -z) + __fmaf_rn(r, kLlo, __fmul_rn(p_lo, kL));
  const float q = __fmul_rn(__fmul_rn(z, z), __fmaf_rn(z, __fmaf_rn(z, 1.f / 24.f, 1.f / 6.f), 0.5f));
  const float low = __fadd_rn(z_lo, q) + __fmul_rn(z, z_lo);
  // in units of 2^-46
  const long long e = __float2ll_rn(__fmul_rn(z, 0x1p46f)) + __float2int_rn(__fmul_rn(low, 0x1p46f));
  const unsigned long long t = powers[(int)j + 32];
  const unsigned long long w = t + (unsigned long long)__mul64hi((long long)t, e << 18);
  const int shift = 62 - kWeightBits - (int)k;  // 18 .. 63
  return shift > 63 ? 0 : ((w >> (shift - 1)) + 1) >> 1;
}

// floor(u * n) for 0 <= u < 1, up to one unit; n where u >= 1.
__device__ __forceinline__ unsigned long long share(float u, unsigned long long n) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return n;
  const uint32_t bits = __float_as_uint(u), e = bits >> 23;  // u = m 2^(e - 150)
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int shift = 126 - (int)max(e, 1u);  // 0 and up
  return shift > 63 ? 0 : __umul64hi(n, m << 40) >> shift;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Puts `value` at the place of `slot` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void put_remote(unsigned long long* slot, uint32_t rank,
                                           unsigned long long value) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(slot)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(value) : "memory");
}

enum Mode { kPlain, kExcept, kLess };  // p, p without some tokens, max(p - q, 0)

struct Walk {  // what the walk leaves for the sampling
  int node, mode, n_except, place;  // place: of the next token in the row's output
  bool done;                        // no sampling: greedy, or no token may come
  float max;
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) walk_kernel(const Args a) {
  __shared__ float row_max[kNodes];
  __shared__ double row_sum[kNodes];
  __shared__ int row_best[kNodes], except[kNodes];
  __shared__ Walk walk;
  __shared__ unsigned long long powers[65], warp_sum[kWarps], cta_sum[3][kCluster];
  wait_prior_grid();
  cluster_arrive();  // waited for before the first store to another CTA
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 65; i += kThreads) powers[i] = kPowers[i];
  int bad = 0;
  const int n = count_of(a, b, &bad);
  const float tau = temperature_of(a, b);
  int32_t* nodes = a.nodes + (long long)b * a.T;
  int32_t* out = a.out + (long long)b * a.T;
  if (n == 0) {  // no nodes: the same for the whole cluster
    if (rank == 0) {
      for (int i = tid; i < a.T; i += kThreads) nodes[i] = out[i] = -1;
      if (tid == 0) {
        a.accepted[b] = 0;
        if (bad && a.err) atomicOr(a.err, bad);
      }
    }
    return;
  }

  // ---- each row's parts put together, a warp a row
  for (int t = warp; t < n; t += kWarps) {
    const Part* parts = a.parts + ((long long)b * a.T + t) * a.chunks;
    float m = -INFINITY;
    for (int i = lane; i < a.chunks; i += 32) m = fmaxf(m, parts[i].max);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double sum = 0;
    int best = 0x7fffffff;
    const float c = tau > 0.f ? __fdiv_rn(kLog2e, tau) : 0.f;
    for (int i = lane; i < a.chunks; i += 32) {
      const Part p = parts[i];
      sum += p.max == m ? (double)p.sum : (double)(p.sum * ex2((p.max - m) * c));
      if (p.max == m) best = min(best, p.best);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) {
      row_max[t] = m;
      row_sum[t] = sum;
      row_best[t] = m > -INFINITY ? best : -1;
    }
  }
  __syncthreads();

  // ---- the walk: lane l holds nodes l and l + 32
  if (warp == 0) {
    int par[2], token[2];
    bool may[2], yes[2];   // a child that may be accepted; one that is, if it is reached
    double p[2] = {0, 0};  // its token's probability at its parent
    float u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = lane + 32 * h;
      par[h] = token[h] = -1;
      may[h] = yes[h] = false;
      u[h] = 0.f;
      if (t >= n) continue;
      const long long at = (long long)b * a.T + t;
      u[h] = fminf(fmaxf(__ldg(a.uniforms + at), 0.f), 1.f - 0x1p-24f);
      if (t == 0) continue;
      par[h] = a.parents ? __ldg(a.parents + at) : t - 1;
      token[h] = __ldg(a.tokens + at);
      if (par[h] < -1 || par[h] >= t || token[h] < 0 || token[h] >= a.V) {
        bad |= DA_DEVERR_INDEX;
        if (par[h] < 0 || par[h] >= t) par[h] = -1;
        continue;
      }
      if (par[h] < 0) continue;
      may[h] = true;
      if (tau > 0.f) {
        const float m = row_max[par[h]];
        const float x = one<BF16>(row_of<BF16>(a, b, par[h]), token[h]);
        if (x == m && m > -INFINITY)
          p[h] = 1.0 / row_sum[par[h]];
        else if (x > -INFINITY && m < INFINITY)
          p[h] = exp(((double)x - (double)m) / (double)tau) / row_sum[par[h]];
      } else {
        yes[h] = token[h] == row_best[par[h]];
      }
    }
    if (a.draft) {  // a chain: node t is the child of t - 1, whose number lies a lane before
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float before = __shfl_up_sync(0xffffffffu, u[h], 1);
        const float last = __shfl_sync(0xffffffffu, u[0], 31);
        if (lane == 0) before = h ? last : 0.f;
        if (may[h] && tau > 0.f) {
          const int t = lane + 32 * h;
          const float q = __ldg(a.draft + b * a.draft_row + t * a.draft_node + token[h]);
          yes[h] = (double)before * (double)q < p[h];  // (a NaN refuses)
        }
      }
    } else if (tau > 0.f) {  // an earlier sibling's token has been asked for already
      for (int s = 0; s + 1 < n; ++s) {
        const int s_par = __shfl_sync(0xffffffffu, s < 32 ? par[0] : par[1], s & 31);
        const int s_token = __shfl_sync(0xffffffffu, s < 32 ? token[0] : token[1], s & 31);
        const bool s_may = __shfl_sync(0xffffffffu, s < 32 ? may[0] : may[1], s & 31);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (s_may && lane + 32 * h > s && s_par == par[h] && s_token == token[h]) p[h] = 0;
      }
    }
    int cur = 0, length = 0;
    unsigned long long kids = 0, went = 1;  // children of the last node; nodes of the path
    while (true) {
      kids = (unsigned long long)__ballot_sync(0xffffffffu, may[1] && par[1] == cur) << 32 |
             __ballot_sync(0xffffffffu, may[0] && par[0] == cur);
      int next = -1;
      if (a.draft || tau == 0.f) {
        const unsigned long long ok =
            ((unsigned long long)__ballot_sync(0xffffffffu, yes[1]) << 32 |
             __ballot_sync(0xffffffffu, yes[0])) & kids;
        if (ok) next = __ffsll((long long)ok) - 1;
      } else {
        const double limit = __shfl_sync(0xffffffffu, cur < 32 ? u[0] : u[1], cur & 31);
        double sum = 0;
        for (unsigned long long left = kids; left && next < 0; left &= left - 1) {
          const int c = __ffsll((long long)left) - 1;
          sum += __shfl_sync(0xffffffffu, c < 32 ? p[0] : p[1], c & 31);
          if (limit < sum) next = c;
        }
      }
      if (next < 0) break;
      cur = next;
      ++length;
      went |= 1ull << cur;
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (rank == 0) {  // children come after their parents: the path's nodes ascend
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = lane + 32 * h;
        if (t < a.T && t > length) nodes[t] = -1;
        if (t < a.T && t > length) out[t] = -1;
        if (went >> t & 1) {
          const int at = __popcll(went & ((1ull << t) - 1));
          nodes[at] = t;
          if (t) out[at - 1] = token[h];
        }
      }
      if (lane == 0) {
        a.accepted[b] = length;
        if (bad && a.err) atomicOr(a.err, bad);
      }
    }
    int n_except = 0;
    if (!a.draft) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool mine = (kids >> (lane + 32 * h) & 1) && p[h] > 0;
        const uint32_t all = __ballot_sync(0xffffffffu, mine);
        if (mine) except[n_except + __popc(all & ((1u << lane) - 1))] = token[h];
        n_except += __popc(all);
      }
    }
    if (lane == 0) {
      walk.node = cur;
      walk.mode = !kids ? kPlain : a.draft ? kLess : n_except ? kExcept : kPlain;
      walk.n_except = n_except;
      walk.place = length;
      walk.done = tau == 0.f || row_best[cur] == -1;
      walk.max = row_max[cur];
      if (rank == 0 && walk.done) out[length] = row_best[cur];
    }
  }
  __syncthreads();
  if (walk.done) return;  // the whole cluster
  const int place = walk.place;

  // ---- the next token, from the last node's row
  const void* row = row_of<BF16>(a, b, walk.node);
  // (of the child that was refused)
  const float* q_row = a.draft ? a.draft + b * a.draft_row + (walk.node + 1) * a.draft_node : nullptr;
  const bool whole = in_step<BF16>(row);
  const Scale scale = scale_of(walk.max, tau);
  const int part = a.slice / kWarps;  // tokens of a warp: a multiple of kBlock
  const int v_first = (int)rank * a.slice + warp * part, v_last = min(v_first + part, a.V);
  int mode = walk.mode;
  unsigned long long whole_sum = 0;  // of the plain weights (kLess)
  auto less = [&](unsigned long long w, int v) -> unsigned long long {
    const unsigned long long q = share(__ldg(q_row + v), whole_sum);
    return w > q ? w - q : 0;
  };
  // The sum over the row of weights as `what` says, in every thread; warp_sum keeps the
  // parts of this CTA's warps.
  auto sum_row = [&](int what, int round) -> unsigned long long {
    unsigned long long sum = 0;
    for (int v = v_first + lane * kVec; v < v_last; v += kBlock) {
      float f[kVec];
      load4<BF16>(row, v, a.V, whole, f);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const unsigned long long w = weight(f[e], scale, powers);
        sum += what == kLess ? (v + e < a.V ? less(w, v + e) : 0) : w;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();  // (warp_sum has been read)
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    if (what == kExcept && tid < walk.n_except) {
      const int v = except[tid], at = v - (int)rank * a.slice;
      if (at >= 0 && at < a.slice)
        atomicAdd(&warp_sum[at / part], 0 - weight(one<BF16>(row, v), scale, powers));
    }
    __syncthreads();
    if (tid < (int)ranks) {
      unsigned long long total = 0;
      for (int w = 0; w < kWarps; ++w) total += warp_sum[w];
      put_remote(&cta_sum[round][rank], tid, total);
    }
    cluster_arrive();
    cluster_wait();
    unsigned long long total = 0;
    for (int r = 0; r < (int)ranks; ++r) total += cta_sum[round][r];
    return total;
  };
  int round = 0;
  cluster_wait();  // all of its CTAs run
  unsigned long long total = sum_row(mode == kLess ? kPlain : mode, round);
  if (mode == kLess) {
    whole_sum = total;
    total = sum_row(kLess, ++round);
  }
  if (total == 0 && mode != kPlain) {  // nothing is left: the target's own probabilities
    mode = kPlain;
    total = sum_row(kPlain, ++round);
  }
  if (total == 0) {
    if (rank == 0 && tid == 0) out[place] = -1;
    return;
  }
  const float u = fminf(fmaxf(__ldg(a.final_uniforms + b), 0.f), 1.f - 0x1p-24f);
  const unsigned long long limit = share(u, total);
  unsigned long long before = 0;
  for (int r = 0; r < (int)rank; ++r) before += cta_sum[round][r];
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  if (limit < before || limit - before >= warp_sum[warp]) return;  // another warp's
  for (int v0 = v_first; v0 < v_last; v0 += kBlock) {
    const int v = v0 + lane * kVec;
    unsigned long long w[kVec], mine = 0;
    if (v < v_last) {
      float f[kVec];
      load4<BF16>(row, v, a.V, whole, f);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        w[e] = weight(f[e], scale, powers);
        if (mode == kLess) w[e] = v + e < a.V ? less(w[e], v + e) : 0;
        if (mode == kExcept)
          for (int i = 0; i < walk.n_except; ++i)
            if (except[i] == v + e) w[e] = 0;
        mine += w[e];
      }
    }
    unsigned long long upto = mine;  // of this and the lanes before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const unsigned long long here = __shfl_sync(0xffffffffu, upto, 31);
    if (limit - before < here) {
      unsigned long long at = before + upto - mine;
      if (mine && limit >= at && limit - at < mine) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          if (limit >= at && limit - at < w[e]) out[place] = v + e;
          at += w[e];
        }
      }
      return;
    }
    before += here;
  }
}

// CTAs of a request: a cluster, as long as each has a few thousand tokens.
int ranks_for(int V) {
  int r = 1;
  while (r < kCluster && V > r * 4096) r <<= 1;
  return r;
}

int chunks_for(int V) { return (V + kChunk - 1) / kChunk; }

bool overlap(const void* a, long long a_bytes, const void* b, long long b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <bool BF16>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  const long long tasks = (long long)a.B * a.T * a.chunks;
  cudaError_t e = launch_after(rows_kernel<BF16>, dim3((unsigned)tasks), dim3(kRowThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  const int ranks = ranks_for(a.V);
  Args w = a;
  const int step = ranks * kWarps * kBlock;
  w.slice = (a.V + step - 1) / step * (kWarps * kBlock);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, walk_kernel<BF16>, w);
}

}  // namespace
}  // namespace da

extern "C" {

size_t nvfp4_mm_verify_workspace_bytes(int32_t batch, int32_t nodes, int32_t vocab) {
  using namespace da;
  if (batch < 0 || nodes < 1 || nodes > kNodes || vocab < 1 || vocab > NVFP4_VERIFY_MAX_VOCAB) return 0;
  const long long parts = (long long)batch * nodes * chunks_for(vocab);
  if (parts > 0x7fffffffLL) return 0;
  return std::max<size_t>(256, (size_t)parts * sizeof(Part));
}

int nvfp4_mm_verify(const nvfp4_verify* args, void* stream) {
  using namespace da;
  if (!args) return DA_ERR_INVALID_ARG;
  const nvfp4_verify& v = *args;
  if (v.batch < 0 || v.nodes < 1 || v.vocab < 1) return DA_ERR_INVALID_ARG;
  if (v.x_dtype != NVFP4_X_F32 && v.x_dtype != NVFP4_X_BF16) return DA_ERR_INVALID_ARG;
  const size_t need = nvfp4_mm_verify_workspace_bytes(v.batch, v.nodes, v.vocab);
  if (!need || v.batch > 0x7fffffff / kCluster) return DA_ERR_UNSUPPORTED;
  if (v.draft && v.parents) return DA_ERR_INVALID_ARG;  // draft probabilities: chains
  if (v.batch == 0) return DA_OK;
  if (!v.x || !v.tokens || !v.uniforms || !v.final_uniforms || !v.accepted || !v.out_nodes || !v.out_tokens)
    return DA_ERR_INVALID_ARG;
  const size_t size = v.x_dtype == NVFP4_X_BF16 ? 2 : 4;
  const void* words[11] = {v.draft, v.tokens, v.parents, v.counts, v.temperature, v.uniforms,
                           v.final_uniforms, v.accepted, v.out_nodes, v.out_tokens, v.err};
  if (!aligned(v.x, size)) return DA_ERR_INVALID_ARG;
  for (const void* w : words)
    if (!aligned(w, 4)) return DA_ERR_INVALID_ARG;
  constexpr long long kMaxStride = 1ll << 40;
  if (v.nodes > 1 && (v.x_node_stride < v.vocab || v.x_node_stride > kMaxStride)) return DA_ERR_INVALID_ARG;
  if (v.batch > 1 && (v.x_stride < v.vocab || v.x_stride > kMaxStride)) return DA_ERR_INVALID_ARG;
  if (v.draft) {
    if (v.nodes > 1 && (v.draft_node_stride < v.vocab || v.draft_node_stride > kMaxStride)) return DA_ERR_INVALID_ARG;
    if (v.batch > 1 && (v.draft_stride < v.vocab || v.draft_stride > kMaxStride)) return DA_ERR_INVALID_ARG;
  }
  if (!v.ws || !aligned(v.ws, 256) || v.ws_bytes < need) return DA_ERR_WORKSPACE;
  // other threads read what an output would overwrite
  const long long rows = 4ll * v.batch, all = rows * v.nodes;
  const void* outs[3] = {v.accepted, v.out_nodes, v.out_tokens};
  const long long out_bytes[3] = {rows, all, all};
  const void* ins[6] = {v.tokens, v.parents, v.uniforms, v.counts, v.temperature, v.final_uniforms};
  const long long in_bytes[6] = {all, all, all, rows, rows, rows};
  const long long e_x = (long long)size, x_bytes = e_x * ((v.batch > 1 ? (v.batch - 1) * v.x_stride : 0) +
                                                          (v.nodes > 1 ? (v.nodes - 1) * v.x_node_stride : 0) + v.vocab);
  for (int i = 0; i < 3; ++i) {
    if (overlap(outs[i], out_bytes[i], v.x, x_bytes) || overlap(outs[i], out_bytes[i], v.ws, (long long)need))
      return DA_ERR_INVALID_ARG;
    for (int k = 0; k < 6; ++k)
      if (overlap(outs[i], out_bytes[i], ins[k], in_bytes[k])) return DA_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (overlap(outs[i], out_bytes[i], outs[k], out_bytes[k])) return DA_ERR_INVALID_ARG;
  }
  Args a = {};
  a.x = v.x;
  a.x_row = v.batch > 1 ? v.x_stride : 0;
  a.x_node = v.nodes > 1 ? v.x_node_stride : 0;
  a.draft = v.draft;
  a.draft_row = v.batch > 1 ? v.draft_stride : 0;
  a.draft_node = v.nodes > 1 ? v.draft_node_stride : 0;
  a.tokens = v.tokens;
  a.parents = v.parents;
  a.counts = v.counts;
  a.temperature = v.temperature;
  a.uniforms = v.uniforms;
  a.final_uniforms = v.final_uniforms;
  a.accepted = v.accepted;
  a.nodes = v.out_nodes;
  a.out = v.out_tokens;
  a.err = v.err;
  a.parts = static_cast<Part*>(v.ws);
  a.B = v.batch;
  a.T = v.nodes;
  a.V = v.vocab;
  a.chunks = chunks_for(v.vocab);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = v.x_dtype == NVFP4_X_BF16 ? launch<true>(a, s) : launch<false>(a, s);
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
