// New keys and values into the attention caches, keys and queries rotated on
// the way.
//
// Pure data movement: each token's q, k and v are read once and written once,
// so memory bounds a prompt's call and launch latency a decode step's.  A unit
// of work is eight consecutive elements of a head (a "chunk": 16 or 32 bytes
// read, 16, 8 or 4 written).  A warp takes a token, or a part of its chunks, and
// computes the token's angles once for all its heads; the loads of its first
// chunks are issued before the angles are needed, so one round trip to memory
// covers both.  Warps do not wait for one another.  A rotated chunk whose pairs lie half a rotation apart reads its
// partner chunk a second time (it comes from L1 or L2: the neighbouring lanes
// have just asked for it), which costs less than an exchange between lanes whose
// place depends on the rotation's size and offset.
//
// Angles: position * inv_freq is formed in fp64, where the product of a 31-bit
// integer and a 24-bit fraction is exact up to 2^-53, and reduced by multiples
// of 2 pi held as two fp64 terms (Cody and Waite's two-step reduction), so sin
// and cos see an fp32 argument in [-pi, pi] whose error is that of its own
// rounding, 2^-23, at any position.
#include "append.cuh"

#include <algorithm>

namespace da {
namespace {

constexpr int kWarps = 4;       // per CTA; each works by itself
constexpr int kMaxPairs = 288;  // rope_dim / 2 at most (576 / 2)
constexpr int kBatch = 4;       // chunks a lane has in flight

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
  if (pos < 0 || pos >= p.capacity) *bad |= DA_DEVERR_LENGTH;
  if (row >= p.B) *bad |= DA_DEVERR_INDEX;
  if (*bad) return -1;
  if (p.layout == DA_KV_CONTIGUOUS) return (long long)row * p.width + pos;
  const int page = pos / p.page_size;
  const int id = __ldg(p.table + (long long)row * p.width + page);
  if (id < 0 || id >= p.num_blocks) {
    *bad |= DA_DEVERR_INDEX;
    return -1;
  }
  return (long long)id * p.page_size + (pos - page * p.page_size);
}

enum { kQ = 0, kK = 1, kV = 2 };

// Warp w of the grid takes part w % parts of token w / parts: chunks [part *
// per_part, + per_part) of the token's list q, k, v, 32 * kBatch at a time.
template <typename X, int KT>
__global__ void __launch_bounds__(kWarps * 32, sizeof(X) == 2 ? 7 : 5) append_kernel(const AppendLaunch p, int parts,
                                                             int per_part) {
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
  const int D = p.D, per_head = D >> 3, half = p.rope_dim >> 1, groups = half >> 3;
  const int q_chunks = p.q_new ? p.H_q * per_head : 0, kv_chunks = p.H_kv * per_head;
  const int total = q_chunks + kv_chunks * (p.v_new ? 2 : 1);  // even: D is a multiple of 16
  const int end = min(total, (part + 1) * per_part);
  const X* q_src = static_cast<const X*>(p.q_new) + token * p.q_stride;
  const X* k_src = static_cast<const X*>(p.k_new) + token * p.k_stride;
  const X* v_src = static_cast<const X*>(p.v_new) + token * p.v_stride;

  Chunk<X> own[kBatch], other[kBatch];
  int what[kBatch], head[kBatch], dim0[kBatch];  // -1, kQ, kK or kV; its place
  auto load = [&](int first) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      int c = first + u * 32 + lane;
      what[u] = -1;
      head[u] = dim0[u] = 0;
      if (c >= end) continue;
      what[u] = c < q_chunks ? kQ : c < q_chunks + kv_chunks ? kK : kV;
      c -= what[u] == kQ ? 0 : what[u] == kK ? q_chunks : q_chunks + kv_chunks;
      head[u] = c / per_head;
      dim0[u] = (c - head[u] * per_head) * 8;
      const X* src = (what[u] == kQ ? q_src : what[u] == kK ? k_src : v_src) +
                     (long long)head[u] * D + dim0[u];
      own[u].load(src);
      const int rel = dim0[u] - p.rope_offset;
      if (what[u] != kV && !p.interleaved && rel >= 0 && rel < p.rope_dim)
        other[u].load(rel < half ? src + half : src - half);
    }
  };
  load(part * per_part);  // on their way while the place and the angles are found

  const int pos = __ldg(p.positions + token);
  int bad = 0;
  const long long entry = entry_of(p, token, pos, &bad);
  if (bad && p.err && part == 0 && lane == 0) atomicOr(p.err, bad);
  if (entry < 0) return;  // the whole warp: one token

  for (int j = lane; j < half; j += 32) {
    const double a = (double)pos * (double)__ldg(p.inv_freq + j);
    const double whole = rint(a * 0.15915494309189533577);  // 1 / (2 pi)
    double r = fma(-whole, 6.283185307179586477, a);         // 2 pi, fp64
    r = fma(-whole, 2.4492935982947064e-16, r);              // 2 pi less that
    float sn, cs;  // |r| <= pi: off by less than 2^-21
    __sincosf((float)r, &sn, &cs);
    reinterpret_cast<float2*>(turn + ((j & 7) >> 1) * groups + (j >> 3))[j & 1] =
        make_float2(p.gain * cs, p.gain * sn);
  }
  __syncwarp();

  for (int first = part * per_part;;) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float f[8];
      if (what[u] >= 0) {
        own[u].get(f);
        const int rel = dim0[u] - p.rope_offset;
        if (what[u] != kV && rel >= 0 && rel < p.rope_dim) {
          if (p.interleaved) {  // pairs rel / 2 .. + 3: half a group
            const float4* at = turn + ((rel >> 3) & 1) * 2 * groups + (rel >> 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 t = at[e * groups];
              const float a0 = f[4 * e], b0 = f[4 * e + 1], a1 = f[4 * e + 2], b1 = f[4 * e + 3];
              f[4 * e] = a0 * t.x - b0 * t.y;
              f[4 * e + 1] = b0 * t.x + a0 * t.y;
              f[4 * e + 2] = a1 * t.z - b1 * t.w;
              f[4 * e + 3] = b1 * t.z + a1 * t.w;
            }
          } else {
            float g[8];
            other[u].get(g);
            const bool lower = rel < half;
            const float4* at = turn + ((lower ? rel : rel - half) >> 3);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 t = at[e * groups];
              f[2 * e] = f[2 * e] * t.x + g[2 * e] * (lower ? -t.y : t.y);
              f[2 * e + 1] = f[2 * e + 1] * t.z + g[2 * e + 1] * (lower ? -t.w : t.w);
            }
          }
        }
        if (what[u] == kQ)
          *reinterpret_cast<uint4*>(p.q_out + ((long long)token * p.H_q + head[u]) * D + dim0[u]) =
              to_bf16x8(f);
      }
      const bool kv = what[u] == kK || what[u] == kV;
      uint8_t* cache = static_cast<uint8_t*>(what[u] == kV ? p.v : p.k);
      const float scale = what[u] == kV ? p.v_scale : p.k_scale;
      const long long at = (entry * p.H_kv + head[u]) * D + dim0[u];  // element of the cache
      if constexpr (KT == DA_KV_BF16) {
        if (kv) *reinterpret_cast<uint4*>(cache + 2 * at) = to_bf16x8(f);
      } else if constexpr (KT == DA_KV_FP8_E4M3) {
        if (kv) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = e4m3x2(__fdiv_rn(f[2 * e], scale), __fdiv_rn(f[2 * e + 1], scale));
          *reinterpret_cast<uint2*>(cache + at) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
      } else if (__any_sync(0xffffffffu, kv)) {
        // a block of 16 is this lane's chunk and its neighbour's (chunks come in
        // pairs: D is a multiple of 16 and every list starts on an even chunk)
        float m = 0.f;
        if (kv) {
#pragma unroll
          for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(f[e]));
        }
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        if (kv) {
          const uint32_t s = e4m3x2(__fdiv_rn(m, 6.f * scale), 0.f) & 0xffu;
          const float step = __half2float(__ushort_as_half((unsigned short)(
                                 e4m3x2_to_f16x2(s) & 0xffffu))) * scale;
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = s ? __fdiv_rn(f[e], step) : 0.f;
          *reinterpret_cast<uint32_t*>(cache + at / 2) = e2m1x8(f);
          if (!(dim0[u] & 8)) cache[p.kv_rows * p.H_kv * (D / 2) + at / 16] = (uint8_t)s;
        }
      }
    }
    first += 32 * kBatch;
    if (first >= end) break;
    load(first);
  }
}

template <typename X, int KT>
cudaError_t launch_typed(const AppendLaunch& p, int sms, cudaStream_t stream) {
  const int chunks = (p.D >> 3) * ((p.q_new ? p.H_q : 0) + p.H_kv * (p.v_new ? 2 : 1));
  // a warp takes a whole token once there are enough of them; fewer tokens are
  // cut, down to one load a lane, so that all SMs have work
  const long long want = 64LL * sms;  // warps
  long long parts = std::max<long long>(1, want / p.n_tokens);
  parts = std::min<long long>(parts, (chunks + 31) / 32);
  const int per_part = (int)(((chunks + parts - 1) / parts + 31) / 32 * 32);
  parts = (chunks + per_part - 1) / per_part;
  const long long grid = (p.n_tokens * parts + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_after(append_kernel<X, KT>, dim3((unsigned)grid), dim3(kWarps * 32), 0, stream, p,
                      (int)parts, per_part);
}

template <typename X>
cudaError_t launch_x(const AppendLaunch& p, int sms, cudaStream_t stream) {
  switch (p.kv_type) {
    case DA_KV_FP8_E4M3: return launch_typed<X, DA_KV_FP8_E4M3>(p, sms, stream);
    case DA_KV_NVFP4: return launch_typed<X, DA_KV_NVFP4>(p, sms, stream);
    default: return launch_typed<X, DA_KV_BF16>(p, sms, stream);
  }
}

}  // namespace

cudaError_t launch_append(const AppendLaunch& p, int sms, cudaStream_t stream) {
  return p.x_bf16 ? launch_x<__nv_bfloat16>(p, sms, stream) : launch_x<float>(p, sms, stream);
}

}  // namespace da
