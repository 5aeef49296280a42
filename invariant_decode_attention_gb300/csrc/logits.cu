// Penalties for repeated tokens, biases and masks on logits, and the greedy
// token, in one pass over each row.
//
// A row of V logits is read once and written once (or not at all), so memory
// bounds a large step and latency a small one.  A cluster of CTAs shares a row:
// CTA r takes the slices r, r + R, ... of at most kSlice tokens.  For a slice it
//   1. asks for its logits (they arrive while 2 and 3 run),
//   2. clears a shared-memory word per token of the slice,
//   3. goes through the row's prompt and output tokens and records those of the
//      slice: bit 31 "in the prompt", the low bits the count in the output
//      (integer atomics: their order does not show), bit 30 "has a bias",
//   4. adjusts and writes the tokens without a bias, keeping the best,
//   5. one thread for each bias token that is the first of its kind does the
//      same for that token, with the values of all its entries added in order.
// Every CTA of a row reads the row's lists; they come from L2 and are short
// beside the logits unless the history is longer than the vocabulary.  Best
// tokens meet as 64-bit keys (ordered value, then lowest token) by shuffles,
// shared memory, and the cluster's distributed shared memory, so there is no
// workspace, and the maximum of the keys does not depend on the order.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "nvfp4_mm.h"

namespace da {
namespace {

constexpr int kThreads = 512;
constexpr int kSlice = 8192;    // tokens per slice at most: 32 KB of shared memory
constexpr int kPer = kSlice / kThreads;
constexpr int kMaxVocab = 1 << 30;  // keeps token arithmetic in 32 bits
constexpr int kCluster = 8;     // CTAs per row at most (the portable cluster size)
constexpr uint32_t kInPrompt = 0x80000000u, kHasBias = 0x40000000u, kCount = 0x3fffffffu;

struct Args {
  const void* x;
  long long x_stride, out_stride;
  const int32_t *prompt, *prompt_lens, *output, *output_lens;
  const float *repetition, *frequency, *presence;
  const int32_t* bias_tokens;
  const float* bias_values;
  const int32_t* bias_lens;
  const uint32_t* mask;
  const int32_t* mask_ids;
  float* out;
  int32_t *tokens, *err;
  int V, slice, n_slices, prompt_width, output_width, bias_width, n_masks, mask_words;
};

// The key of token v with logit l > -inf (else 0): larger logits first, then
// lower tokens.  -0 counts as +0.
__device__ __forceinline__ unsigned long long key_of(float l, int v) {
  if (!(l > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(l + 0.f);
  const uint32_t ordered = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return ((unsigned long long)ordered << 32) | (uint32_t)~v;
}

__device__ __forceinline__ unsigned long long max64(unsigned long long a, unsigned long long b) {
  return a > b ? a : b;
}

// A list's usable length; *bad gets the error bit of one out of range.
__device__ __forceinline__ int list_len(const int32_t* lens, int width, int b, int* bad) {
  if (!lens) return 0;
  const int n = __ldg(lens + b), c = clamp_len(n, width);
  if (c != n) *bad |= DA_DEVERR_LENGTH;
  return c;
}

struct Row {
  float repetition, frequency, presence;
};

// The penalties on a logit whose token's table word is w.
__device__ __forceinline__ float penalised(float l, uint32_t w, const Row& r) {
  if (w & (kInPrompt | kCount)) l = l > 0.f ? __fdiv_rn(l, r.repetition) : __fmul_rn(l, r.repetition);
  const uint32_t c = w & kCount;
  if (c) {
    l = __fsub_rn(l, __fmul_rn(r.frequency, (float)c));
    l = __fsub_rn(l, r.presence);
  }
  return l;
}

__device__ __forceinline__ float load_x(const void* x, long long i, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i])
              : static_cast<const float*>(x)[i];
}

// Logits of VEC consecutive tokens.
template <bool BF16, int VEC>
__device__ __forceinline__ void load_group(const void* x, long long i, float (&l)[VEC]) {
  if constexpr (VEC == 1) {
    l[0] = load_x(x, i, BF16);
  } else if constexpr (BF16) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x) + i);
    l[0] = bf16_lo(w.x), l[1] = bf16_hi(w.x), l[2] = bf16_lo(w.y), l[3] = bf16_hi(w.y);
  } else {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    l[0] = f.x, l[1] = f.y, l[2] = f.z, l[3] = f.w;
  }
}

// Records the tokens of list[0, n) that fall into [v0, v0 + count) in the table.
template <bool OUTPUT>
__device__ __forceinline__ void record(const int32_t* list, int n, int v0, int count, int V,
                                       uint32_t* table, int* bad) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int v = __ldg(list + i);
    if ((unsigned)v >= (unsigned)V) *bad |= DA_DEVERR_INDEX;
    const unsigned s = (unsigned)(v - v0);
    if (s < (unsigned)count) {
      if (OUTPUT)
        atomicAdd(table + s, 1u);
      else
        atomicOr(table + s, kInPrompt);
    }
  }
}

// VEC 4: x, out and the strides allow groups of four tokens to move at once.
template <bool BF16, int VEC>
__global__ void __launch_bounds__(kThreads) logits_kernel(const Args a) {
  __shared__ __align__(16) uint32_t table[kSlice];
  __shared__ unsigned long long warp_best[kThreads / 32], cta_best[kCluster];
  wait_prior_grid();
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  // the cluster's first barrier: every CTA runs before any writes to another
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int b = blockIdx.x / ranks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  int bad = 0;
  const int n_prompt = list_len(a.prompt_lens, a.prompt_width, b, &bad);
  const int n_output = list_len(a.output_lens, a.output_width, b, &bad);
  const int n_bias = list_len(a.bias_lens, a.bias_width, b, &bad);
  const int32_t* prompt = a.prompt + (long long)b * a.prompt_width;
  const int32_t* output = a.output + (long long)b * a.output_width;
  const int32_t* bias_tokens = a.bias_tokens + (long long)b * a.bias_width;
  const float* bias_values = a.bias_values + (long long)b * a.bias_width;
  Row row;
  row.repetition = a.repetition ? __ldg(a.repetition + b) : 1.f;
  row.frequency = a.frequency ? __ldg(a.frequency + b) : 0.f;
  row.presence = a.presence ? __ldg(a.presence + b) : 0.f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int id = a.mask_ids ? __ldg(a.mask_ids + b) : b;
    if (id >= a.n_masks) bad |= DA_DEVERR_INDEX;
    if (id >= 0 && id < a.n_masks) mask = a.mask + (long long)id * a.mask_words;
  }
  const long long x0 = (long long)b * a.x_stride;
  float* out = a.out ? a.out + (long long)b * a.out_stride : nullptr;
  auto allowed = [&](int v) { return !mask || ((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u); };

  unsigned long long best = 0;
  for (int sl = rank; sl < a.n_slices; sl += ranks) {
    const int v0 = sl * a.slice, count = min(a.slice, a.V - v0);
    float l[kPer / VEC][VEC];
#pragma unroll
    for (int u = 0; u < kPer / VEC; ++u) {
      const int s = (u * kThreads + threadIdx.x) * VEC;
      if (VEC == 1 || s + VEC <= count) {
        if (s < count) load_group<BF16, VEC>(a.x, x0 + v0 + s, l[u]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (s + e < count) l[u][e] = load_x(a.x, x0 + v0 + s + e, BF16);
      }
    }
    __syncthreads();  // the previous slice's table is no longer read
    for (int i = threadIdx.x; i < (count + 3) / 4; i += kThreads)
      reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    record<false>(prompt, n_prompt, v0, count, a.V, table, &bad);
    record<true>(output, n_output, v0, count, a.V, table, &bad);
    for (int i = threadIdx.x; i < n_bias; i += kThreads) {
      const int v = __ldg(bias_tokens + i);
      if ((unsigned)v >= (unsigned)a.V) bad |= DA_DEVERR_INDEX;
      if ((unsigned)(v - v0) < (unsigned)count) atomicOr(table + (v - v0), kHasBias);
    }
    __syncthreads();

#pragma unroll
    for (int u = 0; u < kPer / VEC; ++u) {
      const int s = (u * kThreads + threadIdx.x) * VEC;
      if (s >= count) continue;
      uint32_t w[VEC];
      if constexpr (VEC == 4) {
        const uint4 t = *reinterpret_cast<const uint4*>(table + s);
        w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
      } else {
        w[0] = table[s];
      }
      bool whole = s + VEC <= count;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (s + e >= count) continue;
        if (w[e] & kHasBias) {
          whole = false;
          continue;
        }
        if (w[e]) l[u][e] = penalised(l[u][e], w[e], row);
        if (!allowed(v0 + s + e)) l[u][e] = -INFINITY;
        best = max64(best, key_of(l[u][e], v0 + s + e));
      }
      if (!out) continue;
      if constexpr (VEC == 4) {
        if (whole) {
          *reinterpret_cast<float4*>(out + v0 + s) =
              make_float4(l[u][0], l[u][1], l[u][2], l[u][3]);
          continue;
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (s + e < count && !(w[e] & kHasBias)) out[v0 + s + e] = l[u][e];
    }

    // tokens with a bias: untouched so far, also where out is x
    for (int i = threadIdx.x; i < n_bias; i += kThreads) {
      const int v = __ldg(bias_tokens + i);
      if ((unsigned)(v - v0) >= (unsigned)count) continue;
      bool first = true;
      for (int j = 0; j < i && first; ++j) first = __ldg(bias_tokens + j) != v;
      if (!first) continue;
      float sum = __ldg(bias_values + i);
      for (int j = i + 1; j < n_bias; ++j)
        if (__ldg(bias_tokens + j) == v) sum = __fadd_rn(sum, __ldg(bias_values + j));
      float lv = penalised(load_x(a.x, x0 + v, BF16), table[v - v0], row);
      lv = __fadd_rn(lv, sum);
      if (!allowed(v)) lv = -INFINITY;
      best = max64(best, key_of(lv, v));
      if (out) out[v] = lv;
    }
  }
  if (bad && a.err) atomicOr(a.err, bad);

#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max64(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) warp_best[warp] = best;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) best = max64(best, warp_best[w]);
    uint32_t to;  // cta_best[rank] of the cluster's first CTA
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(to)
                 : "r"(smem_addr(cta_best + rank)), "r"(0));
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(best) : "memory");
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && threadIdx.x == 0 && a.tokens) {
    for (uint32_t r = 0; r < ranks; ++r) best = max64(best, cta_best[r]);
    a.tokens[b] = best ? (int32_t)~(uint32_t)best : -1;
  }
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <bool BF16, int VEC>
cudaError_t launch_logits(const Args& a, int B, int ranks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logits_kernel<BF16, VEC>, a);
}

// A list is given whole or not at all (one without room needs no tokens).
bool list_ok(const int32_t* list, const int32_t* lens, int width) {
  if (width < 0 || (width > 0 && (list != nullptr) != (lens != nullptr))) return false;
  return aligned_to(list, 4) && aligned_to(lens, 4);
}

}  // namespace
}  // namespace da

using namespace da;

extern "C" int nvfp4_mm_logits(const nvfp4_logits* g, void* stream) {
  if (!g) return DA_ERR_INVALID_ARG;
  if (g->batch < 0 || g->vocab < 1) return DA_ERR_INVALID_ARG;
  if (g->x_dtype != NVFP4_X_F32 && g->x_dtype != NVFP4_X_BF16) return DA_ERR_INVALID_ARG;
  const bool bf16 = g->x_dtype == NVFP4_X_BF16;
  if (g->vocab > kMaxVocab) return DA_ERR_UNSUPPORTED;
  if (g->batch == 0) return DA_OK;
  if (!g->x || !aligned_to(g->x, bf16 ? 2 : 4) || g->x_stride < g->vocab) return DA_ERR_INVALID_ARG;
  if (!g->out && !g->tokens) return DA_ERR_INVALID_ARG;
  if (g->out && (!aligned_to(g->out, 4) || g->out_stride < g->vocab)) return DA_ERR_INVALID_ARG;
  if (!list_ok(g->prompt, g->prompt_lens, g->prompt_width) ||
      !list_ok(g->output, g->output_lens, g->output_width) ||
      !list_ok(g->bias_tokens, g->bias_lens, g->bias_width))
    return DA_ERR_INVALID_ARG;
  if (g->bias_width > 0 && (g->bias_tokens != nullptr) != (g->bias_values != nullptr))
    return DA_ERR_INVALID_ARG;
  if (g->mask ? (g->n_masks < 1 || (!g->mask_ids && g->n_masks < g->batch)) : g->mask_ids != nullptr)
    return DA_ERR_INVALID_ARG;
  const void* words[8] = {g->repetition, g->frequency, g->presence, g->bias_values,
                          g->mask,       g->mask_ids,  g->tokens,   g->err};
  for (const void* w : words)
    if (!aligned_to(w, 4)) return DA_ERR_INVALID_ARG;
  if (g->out) {  // in place row for row, or apart
    const uintptr_t x = reinterpret_cast<uintptr_t>(g->x);
    const uintptr_t o = reinterpret_cast<uintptr_t>(g->out);
    const uintptr_t x_end = x + ((g->batch - 1LL) * g->x_stride + g->vocab) * (bf16 ? 2 : 4);
    const uintptr_t o_end = o + ((g->batch - 1LL) * g->out_stride + g->vocab) * 4;
    const bool same = x == o && !bf16 && g->x_stride == g->out_stride;
    if (!same && x < o_end && o < x_end) return DA_ERR_INVALID_ARG;
  }
  Args a;
  std::memset(&a, 0, sizeof(a));
  a.x = g->x;
  a.x_stride = g->x_stride;
  a.out_stride = g->out_stride;
  a.prompt = g->prompt;
  a.prompt_lens = g->prompt_lens;
  a.output = g->output;
  a.output_lens = g->output_lens;
  a.repetition = g->repetition;
  a.frequency = g->frequency;
  a.presence = g->presence;
  a.bias_tokens = g->bias_tokens;
  a.bias_values = g->bias_values;
  a.bias_lens = g->bias_lens;
  a.mask = g->mask;
  a.mask_ids = g->mask_ids;
  a.out = g->out;
  a.tokens = g->tokens;
  a.err = g->err;
  a.V = g->vocab;
  a.prompt_width = g->prompt_width;
  a.output_width = g->output_width;
  a.bias_width = g->bias_width;
  a.n_masks = g->n_masks;
  a.mask_words = (g->vocab + 31) / 32;
  // as many CTAs per row as the cluster allows, each with slices of equal
  // length (a multiple of 32, so that slices start on mask words)
  const int ranks = std::max(1, std::min(kCluster, (g->vocab + kThreads - 1) / kThreads));
  const int rounds = (int)(((long long)g->vocab + (long long)ranks * kSlice - 1) /
                           ((long long)ranks * kSlice));
  const long long parts = (long long)ranks * rounds;
  a.slice = (int)(((g->vocab + parts - 1) / parts + 31) / 32 * 32);
  a.n_slices = (g->vocab + a.slice - 1) / a.slice;
  if ((long long)g->batch * ranks > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  const bool vec = aligned_to(g->x, bf16 ? 8 : 16) && g->x_stride % 4 == 0 &&
                   (!g->out || (aligned_to(g->out, 16) && g->out_stride % 4 == 0));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (bf16)
    e = vec ? launch_logits<true, 4>(a, g->batch, ranks, st)
            : launch_logits<true, 1>(a, g->batch, ranks, st);
  else
    e = vec ? launch_logits<false, 4>(a, g->batch, ranks, st)
            : launch_logits<false, 1>(a, g->batch, ranks, st);
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}
