// New keys and values into the attention caches, keys and queries rotated on
// the way.
//
// Pure data movement: each token's q, k and v are read once and written once,
// so memory bounds a prompt's call and launch latency a decode step's.  A chunk
// is eight consecutive elements of a head (16 or 32 bytes read, 16, 8 or 4
// written); a unit of work is two chunks, the ones that the rotation of halves
// mixes, so that each is read once and an angle serves both, or two neighbours.
// A warp takes a token, or a part of its units, and computes the token's angles
// once for all its heads; the loads of its first units are issued before the
// angles are needed, so one round trip to memory covers both.  Warps do not wait
// for one another.  Measured: 16384 tokens of 32/8 heads of 128, bf16, 64 us (6.3
// TB/s, 0.93 of a plain copy's rate); one token 2.6 us; 2047 tokens into an NVFP4
// cache 15.7 us (into E4M3 13.2, bf16 11.9: one wave of latency-bound warps, then
// divisions, block scales and partners that are read a second time).
//
// Angles: position * inv_freq is the product of a 31-bit integer, a 24-bit integer and
// a power of two.  Multiplied by 2^128 / (2 pi) in integers, its whole turns are
// the bits above a place that the exponent gives and go by themselves; the 64
// below it are exact up to 2^-63 of a turn, at any position and frequency (Payne
// and Hanek's reduction with a constant long enough for all of them).  The
// multiplications of a warp's 32 angles take fewer cycles than one in fp64, whose
// units are few (64 latent rows: 4.5 us, 5.9 in fp64).  sincospi gets half turns of [-1, 1],
// rounded once to fp32 (an error of 2^-25 of them, less than 2^-23 in radians), and
// is itself off by two units in the last place at most.  (The hardware's
// approximations of sine and cosine are off by up to 2^-21 each: a component near
// zero beside a large partner lost bits that its type holds.)
#include "append.cuh"

#include <algorithm>

namespace da {
namespace {

constexpr int kWarps = 4;       // per CTA; each works by itself
constexpr int kMaxPairs = 288;  // rope_dim / 2 at most (576 / 2)
// Units that a lane has in flight (48 bytes or so a chunk pair of bf16; measured
// on 16384 tokens of 32/8 heads: one 71, two and three 64 us).
template <typename X>
constexpr int kInFlight = sizeof(X) == 2 ? 3 : 2;
// CTAs that an SM holds at once (72 and 96 registers a thread).
template <typename X>
constexpr int kResident = sizeof(X) == 2 ? 7 : 5;

template <typename X>
struct Chunk;  // eight elements as loaded

template <>
struct Chunk<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
  }
};

template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

__device__ __forceinline__ uint4 to_bf16x8(const float (&f)[8]) {
  return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]),
                    bf16x2(f[6], f[7]));
}

// Two values to two E4M3 bytes (lo in the low byte), saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight values to eight E2M1 codes, element 0 in the lowest nibble, saturating.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Larger of two, NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Cache entry of token i, or -1 (nothing is written); *bad gets the error bits.
__device__ __forceinline__ long long entry_of(const AppendLaunch& p, int i, int pos, int* bad) {
  const int row = p.rows ? __ldg(p.rows + i) : i;
  if (row < 0) return -1;
  if (p.layout == DA_KV_INDEXED) {
    if (pos < 0) *bad |= DA_DEVERR_LENGTH;
    if (row >= p.num_blocks) *bad |= DA_DEVERR_INDEX;
    return *bad ? -1 : row;
  }
  const int at = p.entries ? __ldg(p.entries + i) : pos;
  if (pos < 0 || at < 0 || at >= p.capacity) *bad |= DA_DEVERR_LENGTH;
  if (row >= p.B) *bad |= DA_DEVERR_INDEX;
  if (*bad) return -1;
  if (p.layout == DA_KV_CONTIGUOUS) return (long long)row * p.width + at;
  const int page = at / p.page_size;
  const int id = __ldg(p.table + (long long)row * p.width + page);
  if (id < 0 || id >= p.num_blocks) {
    *bad |= DA_DEVERR_INDEX;
    return -1;
  }
  return (long long)id * p.page_size + (at - page * p.page_size);
}

// The angle pos * inv_freq in half turns, whole turns taken away: in [-1, 1].
__device__ __forceinline__ float half_turns(uint32_t pos, float inv_freq) {
  // 2^128 / (2 pi), from the value of pi
  constexpr unsigned long long kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;
  const uint32_t bits = __float_as_uint(inv_freq), e = (bits >> 23) & 0xffu;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u), n = m * pos;
  const unsigned long long carry = __umul64hi(n, kLow), t1 = carry + n * kHigh;
  const unsigned long long t2 = __umul64hi(n, kHigh) + (t1 < carry);
  // turns = (t2, t1, n * kLow) * 2^(e - 150 - 128): 64 bits from bit `at` on
  const int at = min(max(214 - (int)max(e, 1u), 0), 191), shift = at & 63;
  const unsigned long long lo = at < 64 ? n * kLow : at < 128 ? t1 : t2;
  const unsigned long long hi = at < 64 ? t1 : at < 128 ? t2 : 0;
  const unsigned long long turn = (lo >> shift) | (hi << 1 << (63 - shift));
  return __ll2float_rn((long long)(bits >> 31 ? 0 - turn : turn)) * 0x1p-63f;
}

// Rotates the four pairs (a[0], a[1]), ... of a chunk, or half a group of pairs.
__device__ __forceinline__ void turn_pairs(float (&f)[8], const float4* at, int groups) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 t = at[e * groups];
    const float a0 = f[4 * e], b0 = f[4 * e + 1], a1 = f[4 * e + 2], b1 = f[4 * e + 3];
    f[4 * e] = a0 * t.x - b0 * t.y;
    f[4 * e + 1] = b0 * t.x + a0 * t.y;
    f[4 * e + 2] = a1 * t.z - b1 * t.w;
    f[4 * e + 3] = b1 * t.z + a1 * t.w;
  }
}

// Rotates the eight pairs (a[i], b[i]) of a group.
__device__ __forceinline__ void turn_halves(float (&a)[8], float (&b)[8], const float4* at,
                                            int groups) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 t = at[e * groups];
    const float a0 = a[2 * e], b0 = b[2 * e], a1 = a[2 * e + 1], b1 = b[2 * e + 1];
    a[2 * e] = a0 * t.x - b0 * t.y;
    b[2 * e] = b0 * t.x + a0 * t.y;
    a[2 * e + 1] = a1 * t.z - b1 * t.w;
    b[2 * e + 1] = b1 * t.z + a1 * t.w;
  }
}

// x * r * (w + add) for a chunk of a normed head, one rounding an operation.
__device__ __forceinline__ void norm_chunk(float (&f)[8], float r, const void* weight, bool w_bf16,
                                           float add, int chunk) {
  float w[8];
  if (w_bf16) {
    Chunk<__nv_bfloat16> c;
    c.load(static_cast<const __nv_bfloat16*>(weight) + 8 * chunk);
    c.get(w);
  } else {
    Chunk<float> c;
    c.load(static_cast<const float*>(weight) + 8 * chunk);
    c.get(w);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(__fmul_rn(f[e], r), __fadd_rn(w[e], add));
}

// Warp w of the grid takes part w % parts of token w / parts: units [part *
// per_part, + per_part) of the token's heads q, k, v, 32 * kBatch at a time.
//
// kNorm: queries and keys are normed on the way, y = x / sqrt(mean x^2 + eps) * (w +
// add).  A head's units lie on neighbouring lanes (eight for 128 dims, four for 64), so
// its sum of squares is 16 products a lane, in order, and a butterfly of fixed shape;
// the elements are in registers already, and nothing more is read but the weights.
// Measured: 8192 tokens of 32/8 heads of 128, bf16, 46 us (30 at the measured bandwidth; 0.63
// of the issue slots used, two tokens a warp, each beginning with its angles and its loads);
// 64 rows of 8 nodes, fp32 into E4M3, 7.3 us (2.6).
template <typename X, int KT, int D, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32, kResident<X>)
    append_kernel(const AppendLaunch p, int parts, int per_part) {
  constexpr int kUnits = D / 16;                // units of a head
  static_assert(!kNorm || kUnits == 4 || kUnits == 8, "a head's lanes make a butterfly");
  constexpr int kBatch = kInFlight<X>;
  constexpr bool kBlocks = KT == DA_KV_NVFP4;   // a unit of the cache is always a block of 16
  // gain * (cos, sin) of the token's angles, for each warp: pairs 2i and 2i + 1
  // of group c (eight pairs) at [i * groups + c], so that neighbouring lanes,
  // which hold neighbouring groups, read neighbouring 16 bytes
  __shared__ float4 turns[kWarps][kMaxPairs / 2];
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long task = (long long)blockIdx.x * kWarps + warp;
  const int token = (int)(task / parts), part = (int)(task - (long long)token * parts);
  if (token >= p.n_tokens) return;  // the whole warp
  float4* turn = turns[warp];
  const int half = p.rope_dim >> 1, groups = half >> 3;
  const int skip = p.rope_offset >> 3;  // chunks before the rotated ones
  const int hq = p.q_new ? p.H_q : 0, hk = hq + p.H_kv, heads = hk + (p.v_new ? p.H_kv : 0);
  const int end = min(heads * kUnits, (part + 1) * per_part);
  const X* q_src = static_cast<const X*>(p.q_new) + token * p.q_stride;
  const X* k_src = static_cast<const X*>(p.k_new) + token * p.k_stride;
  const X* v_src = static_cast<const X*>(p.v_new) + token * p.v_stride;
  const bool halves = !p.interleaved;

  // A unit is two chunks of a head: the two that a rotation of halves mixes, or
  // neighbours.  Its chunks' numbers within the head:
  auto chunks_of = [&](int head, int i, int* c0, int* c1) {
    if (!halves || head >= (kBlocks ? hq : hk)) {
      *c0 = 2 * i;
      *c1 = 2 * i + 1;
    } else if (i < groups) {
      *c0 = skip + i;
      *c1 = skip + groups + i;
    } else {  // what is not rotated, in order
      const int m = 2 * (i - groups);
      *c0 = m < skip ? m : m + 2 * groups;
      *c1 = m + 1 < skip ? m + 1 : m + 1 + 2 * groups;
    }
  };
  auto source = [&](int head) {
    return head < hq ? q_src + head * D : head < hk ? k_src + (head - hq) * D : v_src + (head - hk) * D;
  };
  Chunk<X> lo[kBatch], hi[kBatch];
  auto load = [&](int first) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int unit = first + u * 32 + lane;
      if (unit >= end) continue;
      const int head = unit / kUnits;
      int c0, c1;
      chunks_of(head, unit - head * kUnits, &c0, &c1);
      const X* src = source(head);
      lo[u].load(src + 8 * c0);
      hi[u].load(src + 8 * c1);
    }
  };
  load(part * per_part);  // on their way while the place and the angles are found

  const int pos = __ldg(p.positions + token);
  int bad = 0;
  const long long entry = entry_of(p, token, pos, &bad);
  if (bad && p.err && part == 0 && lane == 0) atomicOr(p.err, bad);
  if (entry < 0) return;  // the whole warp: one token

#pragma unroll 2  // a head of 128's two angles of a lane at once (one by one: 72 us for 64)
  for (int j = lane; j < half; j += 32) {
    float sn, cs;
    sincospif(half_turns((uint32_t)pos, __ldg(p.inv_freq + j)), &sn, &cs);
    reinterpret_cast<float2*>(turn + ((j & 7) >> 1) * groups + (j >> 3))[j & 1] =
        make_float2(p.gain * cs, p.gain * sn);
  }
  __syncwarp();

  __nv_bfloat16* q_dst = p.q_out + (long long)token * p.H_q * D;
  const long long at0 = entry * p.H_kv * D;  // first element of the entry in its caches
  for (int first = part * per_part;;) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int unit = first + u * 32 + lane;
      float a[8], b[8], r = 1.f;
      if constexpr (kNorm) {  // all lanes, those past the end too, take part in the sums
        lo[u].get(a);
        hi[u].get(b);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(a[e], a[e], sum);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(b[e], b[e], sum);
#pragma unroll
        for (int m = 1; m < kUnits; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        r = __frsqrt_rn(fmaf(sum, 1.f / D, p.eps));
      }
      if (unit >= end) continue;
      const int head = unit / kUnits, i = unit - head * kUnits;
      int c0, c1;
      chunks_of(head, i, &c0, &c1);
      if constexpr (!kNorm) {
        lo[u].get(a);
        hi[u].get(b);
      }
      const void* weight = nullptr;
      if constexpr (kNorm) {
        weight = head < hq ? p.q_weight : head < hk ? p.k_weight : nullptr;
        if (weight) {
          norm_chunk(a, r, weight, p.w_bf16, p.w_add, c0);
          norm_chunk(b, r, weight, p.w_bf16, p.w_add, c1);
        }
      }
      if (head < hk) {
        if (!halves) {
          const int r0 = c0 - skip, r1 = c1 - skip;  // pairs 4 r .. 4 r + 3: half a group
          if (r0 >= 0 && r0 < 2 * groups) turn_pairs(a, turn + (r0 & 1) * 2 * groups + (r0 >> 1), groups);
          if (r1 >= 0 && r1 < 2 * groups) turn_pairs(b, turn + (r1 & 1) * 2 * groups + (r1 >> 1), groups);
        } else if (!kBlocks || head < hq) {
          if (i < groups) turn_halves(a, b, turn + i, groups);
        } else {
          // a block's chunks have their partners elsewhere: they are read again
          // (from L1 or L2), which costs less than an exchange between lanes whose
          // place depends on the rotation
          const X* src = source(head);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float(&own)[8] = h ? b : a;
            const int at = (h ? c1 : c0) - skip;
            if (at < 0 || at >= 2 * groups) continue;
            Chunk<X> other;
            const int partner = skip + (at < groups ? at + groups : at - groups);
            other.load(src + 8 * partner);
            float g[8];
            other.get(g);
            if constexpr (kNorm)
              if (weight) norm_chunk(g, r, weight, p.w_bf16, p.w_add, partner);
            if (at < groups)
              turn_halves(own, g, turn + at, groups);
            else
              turn_halves(g, own, turn + (at - groups), groups);
          }
        }
      }
      if (head < hq) {
        __nv_bfloat16* dst = q_dst + head * D;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = to_bf16x8(a);
        *reinterpret_cast<uint4*>(dst + 8 * c1) = to_bf16x8(b);
        continue;
      }
      const bool is_v = head >= hk;
      uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v : p.k);
      const float scale = is_v ? p.v_scale : p.k_scale;
      const long long at = at0 + (head - (is_v ? hk : hq)) * D;  // the head's first element
      if constexpr (KT == DA_KV_BF16) {
        *reinterpret_cast<uint4*>(cache + 2 * (at + 8 * c0)) = to_bf16x8(a);
        *reinterpret_cast<uint4*>(cache + 2 * (at + 8 * c1)) = to_bf16x8(b);
      } else if constexpr (KT == DA_KV_FP8_E4M3) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float(&f)[8] = h ? b : a;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = e4m3x2(__fdiv_rn(f[2 * e], scale), __fdiv_rn(f[2 * e + 1], scale));
          *reinterpret_cast<uint2*>(cache + at + 8 * (h ? c1 : c0)) =
              make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
      } else {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, max_nan(fabsf(a[e]), fabsf(b[e])));
        const uint32_t s = e4m3x2(__fdiv_rn(m, 6.f * scale), 0.f) & 0xffu;
        const float step = __half2float(__ushort_as_half((unsigned short)(
                               e4m3x2_to_f16x2(s) & 0xffffu))) * scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] = s ? __fdiv_rn(a[e], step) : 0.f;
          b[e] = s ? __fdiv_rn(b[e], step) : 0.f;
        }
        *reinterpret_cast<uint2*>(cache + (at >> 1) + 8 * i) = make_uint2(e2m1x8(a), e2m1x8(b));
        cache[p.kv_rows * p.H_kv * (D / 2) + (at >> 4) + i] = (uint8_t)s;
      }
    }
    first += 32 * kBatch;
    if (first >= end) break;
    load(first);
  }
}

template <typename X, int KT, int D, bool kNorm>
cudaError_t launch_dim(const AppendLaunch& p, int sms, cudaStream_t stream) {
  const int units = (D / 16) * ((p.q_new ? p.H_q : 0) + p.H_kv * (p.v_new ? 2 : 1));
  // a warp takes a whole token once there are enough of them; fewer tokens are
  // cut, down to one unit a lane, so that all SMs have work, into no more parts than
  // the GPU holds at once (64 tokens of 128 heads of 576: 4.6 us with these 28 warps
  // per SM, 5.3 with 32, 6.2 with 64; 2047 tokens of 32/8 heads into NVFP4: 15.7,
  // 15.7 and 18.4, with 20 warps 19.2)
  const long long want = (long long)kResident<X> * kWarps * sms;  // warps
  long long parts = std::max<long long>(1, want / p.n_tokens);
  parts = std::min<long long>(parts, (units + 31) / 32);
  const int per_part = (int)(((units + parts - 1) / parts + 31) / 32 * 32);
  parts = (units + per_part - 1) / per_part;
  const long long grid = (p.n_tokens * parts + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_after(append_kernel<X, KT, D, kNorm>, dim3((unsigned)grid), dim3(kWarps * 32), 0, stream, p,
                      (int)parts, per_part);
}

template <typename X, int KT>
cudaError_t launch_kv(const AppendLaunch& p, int sms, cudaStream_t stream) {
  const bool norm = p.q_weight || p.k_weight;
  switch (norm ? -p.D : p.D) {
    case 64: return launch_dim<X, KT, 64, false>(p, sms, stream);
    case 128: return launch_dim<X, KT, 128, false>(p, sms, stream);
    case 576:
      if constexpr (KT != DA_KV_NVFP4) return launch_dim<X, KT, 576, false>(p, sms, stream);
      break;
    case -64: return launch_dim<X, KT, 64, true>(p, sms, stream);
    case -128: return launch_dim<X, KT, 128, true>(p, sms, stream);
  }
  return cudaErrorInvalidValue;  // no kernel reads such a cache
}

template <typename X>
cudaError_t launch_x(const AppendLaunch& p, int sms, cudaStream_t stream) {
  switch (p.kv_type) {
    case DA_KV_FP8_E4M3: return launch_kv<X, DA_KV_FP8_E4M3>(p, sms, stream);
    case DA_KV_NVFP4: return launch_kv<X, DA_KV_NVFP4>(p, sms, stream);
    default: return launch_kv<X, DA_KV_BF16>(p, sms, stream);
  }
}

}  // namespace

cudaError_t launch_append(const AppendLaunch& p, int sms, cudaStream_t stream) {
  return p.x_bf16 ? launch_x<__nv_bfloat16>(p, sms, stream) : launch_x<float>(p, sms, stream);
}

}  // namespace da
