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
// log2(e) / temperature without error, 2^(j / 128) from a table, and five terms of the
// series of exp for the rest, whose argument is below 2^-8.5.
//
// Measured, captured and replayed: 64 chains of seven drafted tokens, 131072 fp32 logits a
// node and a draft's probabilities, 112 us (35 at the measured bandwidth); 32 trees of 16
// nodes, 50001 bf16 logits, 31 us (6); one chain of three, 32000 logits, 11.4 us, two
// launches and the steps of the walk one after another.  Of the large
// call rows_kernel takes some 40 us, the walk the rest: two passes of weights over the row
// where it ended, about 110 instructions a weight and pass, most of them one after another
// (0.56 of the issue slots used: less work a weight would help, and so would more weights
// at once).  The weights of the first pass held in registers for the second took 123 us: one CTA
// an SM fits then.
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
constexpr int kBlock = 32 * kVec;                   // tokens of a warp's load
// Loads of a thread in flight: with 4 the largest calls take 1.3% less, the smallest 12% more.
constexpr int kAhead = 2;
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

template <bool BF16>
__device__ __forceinline__ float one(const void* row, long long v) {
  return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(row)[v])
              : static_cast<const float*>(row)[v];
}

template <bool BF16>
struct Word {
  using type = float4;
};
template <>
struct Word<true> {
  using type = uint2;
};

// The bytes from `skew` on of two words that follow each other.
__device__ __forceinline__ uint2 joined(uint2 w, uint2 n, int skew) {
  const uint32_t w0 = skew & 4 ? w.y : w.x, w1 = skew & 4 ? n.x : w.y, w2 = skew & 4 ? n.y : n.x;
  return skew & 2 ? make_uint2(__funnelshift_r(w0, w1, 16), __funnelshift_r(w1, w2, 16)) : make_uint2(w0, w1);
}

__device__ __forceinline__ float4 joined(float4 w, float4 n, int skew) {
  return skew == 4   ? make_float4(w.y, w.z, w.w, n.x)
         : skew == 8 ? make_float4(w.z, w.w, n.x, n.y)
                     : make_float4(w.w, n.x, n.y, n.z);
}

// Bytes by which groups of kVec tokens of a row lie behind their natural boundaries.
template <bool BF16>
__device__ __forceinline__ int skew_of(const void* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) & (BF16 ? 7 : 15));
}

// Groups of four tokens from v, v + step, ... on, -inf at and past `end`: the same tokens
// for the same thread wherever the row lies.  All loads go out together.  A group off its
// boundary is put together from the two aligned words that hold it (each has some of its
// bytes, so that both may be read).
template <bool BF16, int N>
__device__ __forceinline__ void load4(const void* row, int v, int step, int end, int skew, float (&f)[N][kVec]) {
  using W = typename Word<BF16>::type;
  if (v + (N - 1) * step + kVec > end) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int at = v + i * step + e;
        f[i][e] = at < end ? one<BF16>(row, at) : -INFINITY;
      }
    return;
  }
  const W* at = reinterpret_cast<const W*>(static_cast<const char*>(row) + (BF16 ? 2ll : 4ll) * v - skew);
  step >>= 2;
  W w[N];
  if (skew == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(at + i * step);
  } else {
    W n[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = __ldg(at + i * step);
      n[i] = __ldg(at + i * step + 1);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = joined(w[i], n[i], skew);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (BF16) {
      f[i][0] = bf16_lo(w[i].x), f[i][1] = bf16_hi(w[i].x), f[i][2] = bf16_lo(w[i].y), f[i][3] = bf16_hi(w[i].y);
    } else {
      f[i][0] = w[i].x, f[i][1] = w[i].y, f[i][2] = w[i].z, f[i][3] = w[i].w;
    }
  }
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
  const int skew = skew_of<BF16>(row);
  const int v0 = chunk * kChunk + threadIdx.x * kVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float f[kLoads][kVec];
  load4<BF16, kLoads>(row, v0, kRowThreads * kVec, a.V, skew, f);
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

// round(2^62 * 2^(j / 128)), j = 0 .. 127
__device__ const unsigned long long kPowers[128] = {
    0x4000000000000000ull, 0x4058f6a7ecccd5b6ull, 0x40b268f9de0183baull, 0x410c57a1b9fe12f6ull,
    0x4166c34c5615d0ecull, 0x41c1aca777db771bull, 0x421d1461d66f2023ull, 0x4278fb2b1bce0d15ull,
    0x42d561b3e6243d8aull, 0x433248adc91fdd02ull, 0x438fb0cb4f468808ull, 0x43ed9abffb4c6bc9ull,
    0x444c0740496d4294ull, 0x44aaf701b0c72feeull, 0x450a6abaa4b77ecdull, 0x456a632296394492ull,
    0x45cae0f1f545eb73ull, 0x462be4e23237a6efull, 0x468d6fadbf2dd4f3ull, 0x46ef821011734e6bull,
    0x47521cc5a2e6a9e0ull, 0x47b5408bf36472e2ull, 0x4818ee218a3358eeull, 0x487d2645f7725895ull,
    0x48e1e9b9d588e19bull, 0x4947393eca98fcd6ull, 0x49ad159789f37496ull, 0x4a137f87d58e025bull,
    0x4a7a77d47f7b84b1ull, 0x4ae1ff436b663ff7ull, 0x4b4a169b900c2d00ull, 0x4bb2bea4f8bd5847ull,
    0x4c1bf828c6dc54b8ull, 0x4c85c3f13360c4d5ull, 0x4cf022c9905bfd32ull, 0x4d5b157e4a7fc325ull,
    0x4dc69cdceaa72a9cull, 0x4e32b9b417619617ull, 0x4e9f6cd3967fdba8ull, 0x4f0cb70c4ea39210ull,
    0x4f7a993048d088d7ull, 0x4fe91412b2006e83ull, 0x50582887dcb8a7e1ull, 0x50c7d76542a25b72ull,
    0x513821818624b40cull, 0x51a907b474015dc9ull, 0x521a8ad704f3404full, 0x528cabc35f4f799dull,
    0x52ff6b54d8a89c75ull, 0x5372ca67f774358full, 0x53e6c9da74b29ab5ull, 0x545b6a8b3d990704ull,
    0x54d0ad5a753e077cull, 0x5546932976483b15ull, 0x55bd1cdad49f699cull, 0x56344b525f1ff495ull,
    0x56ac1f752150a563ull, 0x57249a29651adc07ull, 0x579dbc56b48521baull, 0x581786e5db7022c2ull,
    0x5891fac0e95612c8ull, 0x590d18d3330c7f1eull, 0x5988e20954889245ull, 0x5a05575132a5cc20ull,
    0x5a827999fcef3242ull, 0x5b0049d42f6afbb6ull, 0x5b7ec8f19468bbc9ull, 0x5bfdf7e546520f3eull,
    0x5c7dd7a3b17dcf75ull, 0x5cfe69229605cef5ull, 0x5d7fad59099f22feull, 0x5e01a53f7974fd86ull,
    0x5e8451cfac061b5full, 0x5f07b404c304c9f1ull, 0x5f8bccdb3d398841ull, 0x60109d50f86846d8ull,
    0x6096266533384a2bull, 0x611c69188f1eb339ull, 0x61a3666d124bb204ull, 0x622b1f66299a6599ull,
    0x62b39508aa836d6full, 0x633cc85ad5122fbdull, 0x63c6ba6455dcd8aeull, 0x64516c2e47ff1623ull,
    0x64dcdec3371793d1ull, 0x6569132f21483ba7ull, 0x65f60a7f79393e2eull, 0x6683c5c3281ee6e9ull,
    0x6712460a8fc24072ull, 0x67a18c678c8c8c61ull, 0x683199ed779592caull, 0x68c26fb128b4cd63ull,
    0x69540ec8f895722dull, 0x69e6784cc2cd61bdull, 0x6a79ad55e7f6fd10ull, 0x6b0daeff4fcde703ull,
    0x6ba27e656b4eb57aull, 0x6c381ca636d99642ull, 0x6cce8ae13c57ebdbull, 0x6d65ca379564e639ull,
    0x6dfddbcbed791babull, 0x6e96c0c284192610ull, 0x6f307a412f074892ull, 0x6fcb096f5c782210ull,
    0x70666f76154a7089ull, 0x7102ad7fff41e9b4ull, 0x719fc4b95f452d29ull, 0x723db6501b9ed447ull,
    0x72dc8373be41a454ull, 0x737c2d55770fe711ull, 0x741cb5281e25ee34ull, 0x74be1c203627c62bull,
    0x75606373ee921c97ull, 0x76038c5b260e5eeeull, 0x76a7980f6cca15c2ull, 0x774c87cc06d1812eull,
    0x77f25ccdee6d7ae6ull, 0x78991853d684a285ull, 0x7940bb9e2cffd89dull, 0x79e947ef1d320d2dull,
    0x7a92be8a92436616ull, 0x7b3d20b6399fc237ull, 0x7be86fb985689ddcull, 0x7c94acddaeea5d3aull,
    0x7d41d96db915019dull, 0x7deff6b672f84e24ull, 0x7e9f06067a4360baull, 0x7f4f08ae3dc7c426ull
};

constexpr int kWeightBits = 44;

struct Scale {
  float max;         // of the row
  float c_hi, c_lo;  // log2(e) / temperature in two terms
};

// 2^44 exp((x - max) / temperature), an integer.  Roundings to integers are additions of
// 1.5 * 2^23 of the unit: the integer is then what the low bits hold.
__device__ __forceinline__ unsigned long long weight(float x, const Scale& s,
                                                     const unsigned long long* powers) {
  const float d = __fsub_rn(x, s.max);
  const float p = __fmul_rn(d, s.c_hi);
  const float bb = __fsub_rn(d, x);  // the difference's rounding error (two-sum)
  const float d_lo = __fadd_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fsub_rn(-s.max, bb));
  const float p_lo = __fmaf_rn(d, s.c_hi, -p) + __fmaf_rn(d, s.c_lo, __fmul_rn(d_lo, s.c_hi));
  // p = n / 128 + r, r exactly, |r| <= 2^-8
  constexpr float kInt = 12582912.f;
  const float t = __fmaf_rn(p, 128.f, kInt);
  const int n = __float_as_int(t) - __float_as_int(kInt);
  const float r = __fmaf_rn(__fsub_rn(t, kInt), -0.0078125f, p);
  // z = (r + p_lo) ln 2 in two terms, then exp(z) - 1 = z + z^2 (1/2 + z/6 + z^2/24) + ...
  constexpr float kL = 0x1.62e43p-1f, kLlo = -0x1.05c61p-29f;
  const float z = __fmul_rn(r, kL);
  const float z_lo = __fmaf_rn(r, kL, -z) + __fmaf_rn(r, kLlo, __fmul_rn(p_lo, kL));
  const float q = __fmul_rn(__fmul_rn(z, z), __fmaf_rn(z, __fmaf_rn(z, 1.f / 24.f, 1.f / 6.f), 0.5f));
  // e, in units of 2^-39: z to 2^-26, then what is left of it and the rest (below 2^-17)
  constexpr float kHigh = 12582912.f * 0x1p-26f, kLow = 12582912.f * 0x1p-39f;
  const float high = __fadd_rn(z, kHigh);
  const float rest = __fadd_rn(__fadd_rn(__fsub_rn(z, __fsub_rn(high, kHigh)), z_lo), q) + __fmul_rn(z, z_lo);
  const int e = ((__float_as_int(high) - __float_as_int(kHigh)) << 13) +
                (__float_as_int(__fadd_rn(rest, kLow)) - __float_as_int(kLow));
  const unsigned long long power = powers[n & 127];
  const unsigned long long w = power + (unsigned long long)(((long long)e * (int)(power >> 32)) >> 7);
  const int shift = 62 - kWeightBits - (n >> 7);  // 18 .. 63
  const unsigned long long v = ((w >> (shift - 1)) + 1) >> 1;
  // nothing is left below 2^-45 (nor of -inf and NaN); the largest, which may be infinite, is 1
  return x == s.max ? 1ull << kWeightBits : p > -45.f ? v : 0;
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
__global__ void __launch_bounds__(kThreads, 2) walk_kernel(const Args a) {
  __shared__ float row_max[kNodes], factor[2];
  __shared__ double row_sum[kNodes];  // in units of the weights
  __shared__ int row_best[kNodes], except[kNodes];
  __shared__ Walk walk;
  __shared__ unsigned long long powers[128], warp_sum[kWarps], cta_sum[3][kCluster];
  wait_prior_grid();
  cluster_arrive();  // waited for before the first store to another CTA
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 128; i += kThreads) powers[i] = kPowers[i];
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

  // ---- log2(e) / temperature (one thread: a division in fp64, of which the SM does few)
  if (tid == kThreads - 1 && tau > 0.f) {
    const double c = 1.4426950408889634 / (double)tau;
    factor[0] = (float)c;
    factor[1] = (float)(c - (double)factor[0]);
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
      row_sum[t] = sum * (double)(1ull << kWeightBits);
      row_best[t] = m > -INFINITY ? best : -1;
    }
  }
  __syncthreads();

  // ---- the walk: lane l holds nodes l and l + 32
  if (warp == 0) {
    int par[2], token[2];
    bool may[2], yes[2];   // a child that may be accepted; one that is, if it is reached
    unsigned long long p[2] = {0, 0};  // its token's weight at its parent
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
        if (m > -INFINITY) {
          const Scale at_parent = {m, factor[0], factor[1]};
          p[h] = weight(fmaxf(one<BF16>(row_of<BF16>(a, b, par[h]), token[h]), -INFINITY), at_parent, powers);
        }
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
          // u q < w / sum  (a NaN or a negative q refuses)
          yes[h] = q >= 0.f && (double)before * (double)q * row_sum[par[h]] < (double)p[h];
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
        const double limit = (double)__shfl_sync(0xffffffffu, cur < 32 ? u[0] : u[1], cur & 31) * row_sum[cur];
        unsigned long long sum = 0;
        for (unsigned long long left = kids; left && next < 0; left &= left - 1) {
          const int c = __ffsll((long long)left) - 1;
          sum += __shfl_sync(0xffffffffu, c < 32 ? p[0] : p[1], c & 31);
          if (limit < (double)sum) next = c;
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
  const int skew = skew_of<BF16>(row);
  const Scale scale = {walk.max, factor[0], factor[1]};
  const int part = a.slice / kWarps;  // tokens of a warp: a multiple of kBlock
  const int v_first = (int)rank * a.slice + warp * part, v_last = min(v_first + part, a.V);
  int mode = walk.mode;
  unsigned long long whole_sum = 0;  // of the plain weights (kLess)
  const int q_skew = q_row ? skew_of<false>(q_row) : 0;
  // The sum over the row of weights as `what` says, in every thread; warp_sum keeps the
  // parts of this CTA's warps.
  auto sum_row = [&](int what, int round) -> unsigned long long {
    unsigned long long sum = 0;
    for (int v0 = v_first + lane * kVec; v0 < v_last; v0 += kBlock * kAhead) {
      float f[kAhead][kVec], q[kAhead][kVec];
      load4<BF16, kAhead>(row, v0, kBlock, v_last, skew, f);
      if (what == kLess) load4<false, kAhead>(q_row, v0, kBlock, v_last, q_skew, q);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const unsigned long long w = weight(f[i][e], scale, powers);
          if (what == kLess) {
            const unsigned long long less = share(q[i][e], whole_sum);
            sum += w > less ? w - less : 0;
          } else {
            sum += w;
          }
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
  for (int v0 = v_first; v0 < v_last; v0 += kBlock * kAhead) {
    float f[kAhead][kVec], q[kAhead][kVec];
    load4<BF16, kAhead>(row, v0 + lane * kVec, kBlock, v_last, skew, f);
    if (mode == kLess) load4<false, kAhead>(q_row, v0 + lane * kVec, kBlock, v_last, q_skew, q);
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) {
      const int v = v0 + i * kBlock + lane * kVec;
      unsigned long long w[kVec], mine = 0;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        float x = f[0][e], less = q[0][e];
#pragma unroll
        for (int k = 1; k < kAhead; ++k)
          if (i == k) x = f[k][e], less = q[k][e];
        w[e] = weight(x, scale, powers);
        if (mode == kLess) {
          const unsigned long long off = share(less, whole_sum);
          w[e] = w[e] > off ? w[e] - off : 0;
        }
        if (mode == kExcept)
          for (int k = 0; k < walk.n_except; ++k)
            if (except[k] == v + e) w[e] = 0;
        mine += w[e];
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
  const long long draft_bytes = 4 * ((v.batch > 1 ? (v.batch - 1) * v.draft_stride : 0) +
                                     (v.nodes > 1 ? (v.nodes - 1) * v.draft_node_stride : 0) + v.vocab);
  for (int i = 0; i < 3; ++i) {
    if (v.draft && overlap(outs[i], out_bytes[i], v.draft, draft_bytes)) return DA_ERR_INVALID_ARG;
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
