// Penalties for repeated tokens, biases and masks on logits, and the greedy
// token, in one pass over each row.
//
// A row of V logits is read once and written once (or not at all), so memory
// bounds a large step and latency a small one.  One CTA takes a row, or a cluster
// of CTAs when there are few rows; in each round a CTA takes one slice of up to
// 32768 tokens,
//   1. asks for its first logits (they arrive while 2 runs),
//   2. goes through the row's prompt, output and bias tokens and records those of
//      the slice in a word of shared memory per token: "in the prompt", the count
//      in the output, "has a bias" (integer atomics: their order does not show),
//      and lists them,
//   3. masks, writes and compares the slice, kDepth loads of a thread in flight.
//      Listed tokens are written but not compared,
//   4. goes through the listed tokens: applies the penalties, adds the token's
//      bias values in their order, writes and compares.
// Step 4 apart from 3: a text's tokens spread over the vocabulary, and with the
// penalties in the streaming loop nearly every warp went through them for one
// lane (256 rows of 131072 tokens: 155 instructions per 128 tokens).  Every CTA
// of a row reads the row's lists, from L2.
// Best tokens meet as 64-bit keys (ordered value, then lowest token) by shuffles
// and shared memory of the cluster, so there is no workspace, and the maximum of
// the keys does not depend on the order.  Measured: 256 rows of 131072, everything
// written, 64 us (4.2 TB/s, 0.63 of a plain copy's rate; 48 of 152 SMs have one row,
// the others two); 256 rows of 100001 in bf16 50 us; 64 rows of 32000 with 30000 tokens
// behind them 18 us, the list scan; one row of 32000 5.1 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "nvfp4_mm.h"

namespace da {
namespace {

constexpr int kThreads = 512;
constexpr int kTableBytes = 65536;   // shared memory for the words of a slice
constexpr int kPlainBytes = 24 * 1024;  // with the static arrays: below 48 KB
constexpr int kListed = 8192;       // tokens with a word that are listed at most
constexpr int kDense = 3;            // list entries per so many tokens of a slice: many
constexpr int kScan = 8;           // list entries a thread has in flight
constexpr int kMaxVocab = 1 << 30;  // keeps token arithmetic in 32 bits
constexpr int kCluster = 8;     // CTAs per row at most (the portable cluster size)
constexpr long long kMaxStride = 1ll << 40;  // elements

// A token's word: "in the prompt", "has a bias", "is listed", and its count in
// the output.  Two bytes do for outputs of up to 2^13 - 1 tokens and double a
// slice.
template <typename W>
struct Word {
  static constexpr uint32_t kInPrompt = 1u << (8 * sizeof(W) - 1);
  static constexpr uint32_t kHasBias = kInPrompt >> 1, kListed = kInPrompt >> 2;
  static constexpr uint32_t kCount = kListed - 1;
  static constexpr int kMostOutput = (int)kCount;
  static constexpr int kSlice = std::min<int>(kTableBytes / sizeof(W), 65536);

  // by shared-memory address: the atomics act on the 32 bits around a word
  static __device__ __forceinline__ void add(uint32_t at) {
    asm volatile("red.relaxed.cta.shared::cta.add.u32 [%0], %1;" ::"r"(at & ~3u),
                 "r"(1u << (at & 3u) * 8)
                 : "memory");
  }
  static __device__ __forceinline__ void put(uint32_t at, uint32_t value) {
    if constexpr (sizeof(W) == 2)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((unsigned short)value) : "memory");
    else
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(value) : "memory");
  }
  static __device__ __forceinline__ void flag(uint32_t at, uint32_t flags) {
    asm volatile("red.relaxed.cta.shared::cta.or.b32 [%0], %1;" ::"r"(at & ~3u),
                 "r"(flags << (at & 3u) * 8)
                 : "memory");
  }
  // Sets `flags` and kListed; whether the token has just become listed, which is
  // true for one caller only.  A plain look first: hot tokens repeat, and atomics
  // on one word queue up.
  static __device__ __forceinline__ bool set(uint32_t at, uint32_t flags) {
    flags |= kListed;
    const int shift = (at & 3u) * 8;
    uint32_t old;
    asm volatile("ld.volatile.shared::cta.u32 %0, [%1];" : "=r"(old) : "r"(at & ~3u) : "memory");
    if (((old >> shift) & flags) == flags) return false;
    asm volatile("atom.relaxed.cta.shared::cta.or.b32 %0, [%1], %2;"
                 : "=r"(old)
                 : "r"(at & ~3u), "r"(flags << shift)
                 : "memory");
    return !((old >> shift) & kListed);
  }
};

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
  int V, slice, prompt_width, output_width, bias_width, n_masks, mask_words;
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

// The penalties on a logit whose token's word is w (not zero).
template <typename W>
__device__ __forceinline__ float penalised(float l, uint32_t w, const Row& r) {
  if (w & (Word<W>::kInPrompt | Word<W>::kCount))
    l = l > 0.f ? __fdiv_rn(l, r.repetition) : __fmul_rn(l, r.repetition);
  const uint32_t c = w & Word<W>::kCount;
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

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// VEC consecutive logits as they lie in memory.
template <bool BF16, int VEC>
struct Group;

template <>
struct Group<false, 4> {
  float4 raw;
  __device__ __forceinline__ void load(const void* p) { raw = *static_cast<const float4*>(p); }
  __device__ __forceinline__ void load_from(const void* p, int skip) {  // 1 .. 3 of them
    const float* f = static_cast<const float*>(p);
    raw = make_float4(0.f, skip > 1 ? 0.f : f[1], skip > 2 ? 0.f : f[2], f[3]);
  }
  __device__ __forceinline__ void get(float (&l)[4]) const {
    l[0] = raw.x, l[1] = raw.y, l[2] = raw.z, l[3] = raw.w;
  }
};

template <>
struct Group<true, 4> {
  uint2 raw;
  __device__ __forceinline__ void load(const void* p) { raw = *static_cast<const uint2*>(p); }
  __device__ __forceinline__ void load_from(const void* p, int skip) {  // 1 .. 3 of them
    const unsigned short* h = static_cast<const unsigned short*>(p);
    raw.x = skip > 1 ? 0u : (uint32_t)h[1] << 16;
    raw.y = (skip > 2 ? 0u : h[2]) | (uint32_t)h[3] << 16;
  }
  __device__ __forceinline__ void get(float (&l)[4]) const {
    l[0] = bf16_lo(raw.x), l[1] = bf16_hi(raw.x), l[2] = bf16_lo(raw.y), l[3] = bf16_hi(raw.y);
  }
};

template <bool BF16>
struct Group<BF16, 1> {
  float raw;
  __device__ __forceinline__ void load(const void* p) { raw = load_x(p, 0, BF16); }
  __device__ __forceinline__ void load_from(const void*, int) {}
  __device__ __forceinline__ void get(float (&l)[1]) const { l[0] = raw; }
};

// The words of VEC consecutive tokens from shared memory.
template <typename W, int VEC>
__device__ __forceinline__ void load_words(const W* at, uint32_t (&w)[VEC]) {
  if constexpr (VEC == 4 && sizeof(W) == 4) {
    const uint4 t = *reinterpret_cast<const uint4*>(at);
    w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
  } else if constexpr (VEC == 4) {
    const uint2 t = *reinterpret_cast<const uint2*>(at);
    w[0] = t.x & 0xffffu, w[1] = t.x >> 16, w[2] = t.y & 0xffffu, w[3] = t.y >> 16;
  } else {
    w[0] = *at;
  }
}

// Goes through list[0, n) and calls put(s, address of its word) for every token
// v0 + s of the slice [v0, v0 + count); kScan loads of a thread are in flight together.
template <typename W, typename Put>
__device__ __forceinline__ void record(const int32_t* list, int n, int v0, int count, int V,
                                       uint32_t table, int* bad, Put put) {
  for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kScan) {
    int v[kScan];
#pragma unroll
    for (int u = 0; u < kScan; ++u) v[u] = __ldg(list + min(i0 + u * kThreads, n - 1));
#pragma unroll
    for (int u = 0; u < kScan; ++u) {
      const unsigned s = (unsigned)(v[u] - v0);
      if (i0 + u * kThreads >= n) break;
      if ((unsigned)v[u] >= (unsigned)V)
        *bad |= DA_DEVERR_INDEX;
      else if (s < (unsigned)count)
        put((int)s, table + s * (uint32_t)sizeof(W));
    }
  }
}

// VEC 4: groups of four tokens move at once.  They start at multiples of four tokens
// or, if SHIFT, wherever x has its 16 (bf16: 8) byte boundaries, which differs from row
// to row: slices begin `shift` tokens early, so that a row's first group may lie partly
// before it, and its words and its places in the table are counted from there.
template <bool BF16, int VEC, bool SHIFT, typename W>
__global__ void __launch_bounds__(kThreads, 2) logits_kernel(const Args a) {
  constexpr int kElem = BF16 ? 2 : 4;
  constexpr int kStep = kThreads * VEC;     // tokens of a step of the CTA
  constexpr int kDepth = 4;                 // steps whose logits are on their way
  extern __shared__ __align__(16) uint8_t smem[];
  W* table = reinterpret_cast<W*>(smem);  // [slice]; all zero between slices
  __shared__ uint16_t listed[kListed];  // tokens of the slice that have a word
  __shared__ int n_listed;
  __shared__ unsigned long long warp_best[kThreads / 32], cta_best[kCluster];
  wait_prior_grid();
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  cluster_arrive();
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t words = smem_addr(table);
  const int span = a.slice * (int)ranks;  // tokens of a round
  const char* x = static_cast<const char*>(a.x) + (long long)b * a.x_stride * kElem;

  const int shift = SHIFT ? (int)(reinterpret_cast<uintptr_t>(x) / kElem & 3) : 0;
  const int V = a.V + shift;  // of which the first `shift` do not exist

  Group<BF16, VEC> raw[kDepth];
  uint32_t may[kDepth];  // their mask words
  const uint32_t* mask = nullptr;
  // Asks for step i of the slice at token v0.
  auto load = [&](int d, int v0, int i) {
    const long long v = v0 + (long long)i * kStep + tid * VEC;
    if (SHIFT && v < 0)
      raw[d].load_from(x + v * kElem, shift);
    else
      raw[d].load(x + v * kElem);
    if (mask) may[d] = __ldg(mask + (SHIFT ? max((int)v, 0) >> 5 : v >> 5));
  };
  auto load_first = [&](int v0) {
    const int full = min(a.slice, max(0, a.V - v0)) / kStep;
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (d < full) load(d, v0, d);
  };

  int bad = 0;
  if (a.mask) {
    const int id = a.mask_ids ? __ldg(a.mask_ids + b) : b;
    if (id >= a.n_masks) bad |= DA_DEVERR_INDEX;
    if (id >= 0 && id < a.n_masks) mask = a.mask + (long long)id * a.mask_words;
  }
  const int n_prompt = list_len(a.prompt_lens, a.prompt_width, b, &bad);
  const int n_output = list_len(a.output_lens, a.output_width, b, &bad);
  const int n_bias = list_len(a.bias_lens, a.bias_width, b, &bad);
  Row row;
  row.repetition = a.repetition ? __ldg(a.repetition + b) : 1.f;
  row.frequency = a.frequency ? __ldg(a.frequency + b) : 0.f;
  row.presence = a.presence ? __ldg(a.presence + b) : 0.f;
  load_first((int)rank * a.slice - shift);
  for (int i = tid; i < a.slice * (int)sizeof(W) / 16; i += kThreads)
    reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) n_listed = 0;
  __syncthreads();
  const int32_t* bias_tokens = a.bias_tokens + (long long)b * a.bias_width;
  const float* bias_values = a.bias_values + (long long)b * a.bias_width;
  float* out = a.out ? a.out + (long long)b * a.out_stride : nullptr;

  float best = -INFINITY;  // of this thread, whose tokens come in ascending order
  int best_v = 0;
  unsigned long long best_key = 0;  // of its last and its listed tokens
  for (int r0 = 0; r0 < V; r0 += span) {
    // the slice's first token, and its length
    const int v0 = r0 + (int)rank * a.slice - shift, count = min(a.slice, max(0, a.V - v0));
    const int32_t* prompt = a.prompt + (long long)b * a.prompt_width;
    const int32_t* output = a.output + (long long)b * a.output_width;
    if ((long long)n_prompt + n_output + n_bias < count / kDense) {
      // few entries: whoever touches a token first lists it
      const auto list = [&](int s) {
        const int at = atomicAdd(&n_listed, 1);
        if (at < kListed) listed[at] = (uint16_t)s;
      };
      record<W>(prompt, n_prompt, v0, count, a.V, words, &bad, [&](int s, uint32_t at) {
        if (Word<W>::set(at, Word<W>::kInPrompt)) list(s);
      });
      record<W>(output, n_output, v0, count, a.V, words, &bad, [&](int s, uint32_t at) {
        if (Word<W>::set(at, 0)) list(s);
        Word<W>::add(at);
      });
      record<W>(bias_tokens, n_bias, v0, count, a.V, words, &bad, [&](int s, uint32_t at) {
        if (Word<W>::set(at, Word<W>::kHasBias)) list(s);
      });
    } else {
      // many: record them with as few instructions as there are, then look
      // through the words for the list
      record<W>(prompt, n_prompt, v0, count, a.V, words, &bad,
                [](int, uint32_t at) { Word<W>::put(at, Word<W>::kInPrompt); });
      __syncthreads();
      record<W>(output, n_output, v0, count, a.V, words, &bad,
                [](int, uint32_t at) { Word<W>::add(at); });
      record<W>(bias_tokens, n_bias, v0, count, a.V, words, &bad,
                [](int, uint32_t at) { Word<W>::flag(at, Word<W>::kHasBias); });
      __syncthreads();
      constexpr int kWords = 16 / sizeof(W);
      for (int s0 = (tid & ~31) * kWords; s0 < count; s0 += kThreads * kWords) {  // whole warps
        const int s = s0 + lane * kWords;
        W w[kWords] = {};
        if (s < count)  // the table goes on past count, with zeros, to a whole step
          *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(table + s);
        int mine = 0;
#pragma unroll
        for (int e = 0; e < kWords; ++e) mine += w[e] != 0;
        int at = mine;  // this lane's place in the list: a prefix sum over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) at += t;
        }
        int base = 0;
        if (lane == 31 && at) base = atomicAdd(&n_listed, at);
        at += __shfl_sync(0xffffffffu, base, 31) - mine;
#pragma unroll
        for (int e = 0; e < kWords; ++e)
          if (w[e]) {
            if (at < kListed) listed[at] = (uint16_t)(s + e);
            ++at;
          }
      }
    }
    __syncthreads();

    const int full = count / kStep;
    for (int i0 = 0; i0 < full; i0 += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int i = i0 + d;
        if (i >= full) break;
        const int s = i * kStep + tid * VEC;
        float l[VEC];
        uint32_t w[VEC];
        raw[d].get(l);
        load_words<W, VEC>(table + s, w);
        if (mask) {
          uint32_t bits = may[d] >> ((v0 + s) & 31);
          if (SHIFT) {  // a group that crosses a word's end: the next lane has the next word
            const uint32_t next = __shfl_down_sync(0xffffffffu, may[d], 1);
            bits = v0 + s < 0 ? may[d] << shift : __funnelshift_r(may[d], next, v0 + s);
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (!((bits >> e) & 1u)) l[e] = -INFINITY;
        }
        if (SHIFT && v0 + s < 0) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (e < shift) l[e] = -INFINITY;
            else if (out) out[v0 + s + e] = l[e];
          }
        } else if (out) {
          if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(out + v0 + s) = make_float4(l[0], l[1], l[2], l[3]);
          else
            out[v0 + s] = l[0];
        }
        if (i + kDepth < full) load(d, v0, i + kDepth);
        uint32_t any = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) any |= w[e];
        if (any) {  // listed tokens compete later
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (w[e]) l[e] = -INFINITY;
        }
        float top = l[0];
#pragma unroll
        for (int e = 1; e < VEC; ++e) top = fmaxf(top, l[e]);
        if (top > best) {
          best = top;
#pragma unroll
          for (int e = VEC - 1; e >= 0; --e)
            if (l[e] == top) best_v = v0 + s + e;
        }
      }
    }
    if (full * kStep < count) {  // what is left (the row's last tokens): one by one
      const int s0 = full * kStep + tid;
      float l[VEC];
      uint32_t bits[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int v = max(v0 + min(s0 + e * kThreads, count - 1), 0);
        l[e] = load_x(x, v, BF16);
        bits[e] = mask ? __ldg(mask + (v >> 5)) : 0xffffffffu;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int s = s0 + e * kThreads;
        if (s >= count) break;
        if (SHIFT && v0 + s < 0) continue;
        if (!((bits[e] >> ((v0 + s) & 31)) & 1u)) l[e] = -INFINITY;
        if (out) out[v0 + s] = l[e];
        if (!table[s]) best_key = max64(best_key, key_of(l[e], v0 + s));
      }
    }
    if (r0 + span < V) load_first(v0 + span);
    __syncthreads();  // the listed tokens' plain values are written

    // Where out is x, what is found there is still a listed token's logit, or
    // -inf, which masks it anyway.
    auto finish = [&](int s, float l, uint32_t w, uint32_t bits) {
      const int v = v0 + s;
      l = penalised<W>(l, w, row);
      if (w & Word<W>::kHasBias) {
        float sum = 0.f;
        bool first = true;
#pragma unroll 8
        for (int j = 0; j < n_bias; ++j)
          if (__ldg(bias_tokens + j) == v) {
            const float value = __ldg(bias_values + j);
            sum = first ? value : __fadd_rn(sum, value);
            first = false;
          }
        l = __fadd_rn(l, sum);
      }
      if (!((bits >> (v & 31)) & 1u)) l = -INFINITY;
      best_key = max64(best_key, key_of(l, v));
      if (out) out[v] = l;
    };
    auto mask_word = [&](int s) { return mask ? __ldg(mask + ((v0 + s) >> 5)) : 0xffffffffu; };
    const int n = n_listed;
    if (n <= kListed) {
      constexpr int kAhead = 4;  // tokens of a thread whose logits are on their way
      for (int i0 = tid; i0 < n; i0 += kThreads * kAhead) {
        int s[kAhead];
        float l[kAhead];
        uint32_t bits[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          s[u] = listed[min(i0 + u * kThreads, n - 1)];
          l[u] = load_x(x, v0 + s[u], BF16);
          bits[u] = mask_word(s[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (i0 + u * kThreads >= n) break;
          finish(s[u], l[u], table[s[u]], bits[u]);
          table[s[u]] = 0;
        }
      }
    } else {  // more than the list holds: look for them
      for (int s = tid; s < count; s += kThreads) {
        const uint32_t w = table[s];
        if (!w) continue;
        finish(s, load_x(x, v0 + s, BF16), w, mask_word(s));
        table[s] = 0;
      }
    }
    __syncthreads();  // the table is clear again
    if (tid == 0) n_listed = 0;
    __syncthreads();
  }
  if (bad && a.err) atomicOr(a.err, bad);

  best_key = max64(best_key, key_of(best, best_v));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    best_key = max64(best_key, __shfl_xor_sync(0xffffffffu, best_key, o));
  if (lane == 0) warp_best[warp] = best_key;
  __syncthreads();
  cluster_wait();  // every CTA of the cluster runs
  if (tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) best_key = max64(best_key, warp_best[w]);
    uint32_t to;  // cta_best[rank] of the cluster's first CTA
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(to)
                 : "r"(smem_addr(cta_best + rank)), "r"(0));
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(best_key) : "memory");
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (rank == 0 && tid == 0 && a.tokens) {
    for (uint32_t r = 0; r < ranks; ++r) best_key = max64(best_key, cta_best[r]);
    a.tokens[b] = best_key ? (int32_t)~(uint32_t)best_key : -1;
  }
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <bool BF16, int VEC, bool SHIFT, typename W>
cudaError_t launch_logits(Args& a, int B, int sms, cudaStream_t stream) {
  // Every CTA of a row goes through its lists, so there are no more of them than
  // run at once, two per SM (64 rows of 32000 with long lists: four CTAs a row 22
  // us, eight 31; 256 rows of 131072: one 69 us, four 71, eight 89); slices are of equal
  // length, a multiple of the steps of a CTA, so that only a row's last one ends
  // inside a step.
  int ranks = 1;
  while (ranks < kCluster && (long long)ranks * B <= sms && ranks * kThreads * 4 < a.V) ranks *= 2;
  const int V = a.V + (SHIFT ? 3 : 0);  // at most
  const long long rounds = (V + ranks * Word<W>::kSlice - 1) / (ranks * Word<W>::kSlice);
  constexpr int kStep = kThreads * VEC;
  static_assert(Word<W>::kSlice % kStep == 0, "a slice may be whole steps");
  a.slice = (int)(((V + ranks * rounds - 1) / (ranks * rounds) + kStep - 1) / kStep * kStep);
  const size_t bytes = (size_t)a.slice * sizeof(W);
  if (bytes > kPlainBytes) {  // beyond what needs no consent; it holds per device
    const cudaError_t e = cudaFuncSetAttribute(
        logits_kernel<BF16, VEC, SHIFT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTableBytes);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
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
  return cudaLaunchKernelEx(&cfg, logits_kernel<BF16, VEC, SHIFT, W>, a);
}

template <bool BF16, typename W>
auto* pick(bool vec, bool shift) {
  return !vec ? launch_logits<BF16, 1, false, W>
              : shift ? launch_logits<BF16, 4, true, W> : launch_logits<BF16, 4, false, W>;
}

template <bool BF16>
auto* pick(bool vec, bool shift, bool narrow) {
  return narrow ? pick<BF16, uint16_t>(vec, shift) : pick<BF16, uint32_t>(vec, shift);
}

// Whether `rows` rows of a_bytes at a and of b_bytes at b, strides apart, share a byte.
// Rows with one stride may interleave; with two, nothing is told but that the buffers
// lie apart.
bool rows_overlap(uintptr_t a, long long a_bytes, long long a_stride, uintptr_t b, long long b_bytes,
                  long long b_stride, long long rows) {
  const uintptr_t a_end = a + (rows - 1) * a_stride + a_bytes;
  const uintptr_t b_end = b + (rows - 1) * b_stride + b_bytes;
  if (a >= b_end || b >= a_end) return false;
  if (a_stride != b_stride) return true;
  // rows i of a and j of b meet if b - a + (j - i) stride lies in (-b_bytes, a_bytes): with
  // buffers that touch, one of the two values next to zero is taken by some i and j
  const long long at = (long long)(b - a) % a_stride, on = at < 0 ? at + a_stride : at;
  return on < a_bytes || on > a_stride - b_bytes;
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
  if (g->bias_width > NVFP4_LOGITS_MAX_BIAS ||
      (long long)g->prompt_width + g->output_width + g->bias_width > Word<uint32_t>::kMostOutput)
    return DA_ERR_UNSUPPORTED;  // (the count of a token in the output has 29 bits)
  // one row has no stride; those of more rows stay where bytes can be counted
  const long long V = g->vocab, x_stride = g->batch > 1 ? g->x_stride : V;
  const long long out_stride = g->out && g->batch > 1 ? g->out_stride : V;
  if (x_stride > kMaxStride || out_stride > kMaxStride) return DA_ERR_INVALID_ARG;
  if (g->out) {  // in place row for row, or apart
    const uintptr_t x = reinterpret_cast<uintptr_t>(g->x);
    const uintptr_t o = reinterpret_cast<uintptr_t>(g->out);
    const long long size = bf16 ? 2 : 4;
    const bool same = x == o && !bf16 && x_stride == out_stride;
    if (!same && rows_overlap(x, V * size, x_stride * size, o, V * 4, out_stride * 4, g->batch))
      return DA_ERR_INVALID_ARG;
  }
  Args a;
  std::memset(&a, 0, sizeof(a));
  a.x = g->x;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
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
  // groups of four: x and out must have their boundaries at the same tokens of a row
  const long long x_at = (long long)(reinterpret_cast<uintptr_t>(g->x) / (bf16 ? 2 : 4));
  const long long out_at = (long long)(reinterpret_cast<uintptr_t>(g->out) / 4);
  const bool vec = !g->out || ((x_at - out_at) % 4 == 0 && (x_stride - out_stride) % 4 == 0);
  const bool shift = x_at % 4 != 0 || (g->batch > 1 && x_stride % 4 != 0);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DA_ERR_CUDA;
  const bool narrow = g->output_width <= Word<uint16_t>::kMostOutput;
  auto* launch = bf16 ? pick<true>(vec, shift, narrow) : pick<false>(vec, shift, narrow);
  const cudaError_t e = launch(a, g->batch, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}
