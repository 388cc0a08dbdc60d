// The paged 4-bit KV cache: its layout, and the kernels that append to it and read it back.
//
// Layout. A page holds, KV head by KV head, page_tokens / 16 groups of 16 positions. A group is
//   K codes | V codes | K scales | V scales     (hd 128: 1024 + 1024 + 128 + 128 bytes)
// in the order in which the attention kernel's lanes (g = lane / 4, t = lane % 4) take them as
// operands of 16 x 8 x 16 matrix products, so that every lane reads whole 16-byte words and no
// value ever moves between lanes:
//   K: lane (g, t) holds positions g and g + 8, the hd / 4 values from t hd / 4 on;
//   V: lane (g, t) holds positions 2t, 2t + 1, 2t + 8, 2t + 9, the hd / 8 values from g hd / 8 on.
// A 32-bit word holds 8 consecutive values of one position, value i in bits 4i .. 4i + 3 as
// code + 8; so an append writes whole words and never reads what other positions put there.
// A scale is one byte b: the positive f16 with bits b << 7 (5 exponent, 3 mantissa bits) times 8.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "dec.h"

namespace dec {
namespace kvq {

constexpr int kBlock = 16;       // values per scale
constexpr int kGroup = 16;       // positions per group
constexpr int kScaleMax = 167;   // the largest finite scale: 8 * 60
constexpr int kScaleNan = 255;

__host__ __device__ constexpr int code_bytes(int hd) { return kGroup * hd / 2; }
__host__ __device__ constexpr int scale_bytes(int hd) { return kGroup * hd / kBlock; }
__host__ __device__ constexpr int group_bytes(int hd) { return 2 * (code_bytes(hd) + scale_bytes(hd)); }

// Byte offsets inside a group: the word of values 8j .. 8j + 7 of position pp (0 .. 15), and the
// scale of values 16i .. 16i + 15.
template <int HD>
__device__ __forceinline__ int k_word(int pp, int j) {
  const int g = pp & 7, hi = pp >> 3;
  if (HD == 128) return hi * 512 + (g * 4 + (j >> 2)) * 16 + (j & 3) * 4;
  return (g * 4 + (j >> 1)) * 16 + hi * 8 + (j & 1) * 4;
}
template <int HD>
__device__ __forceinline__ int v_word(int pp, int j) {
  const int hi = pp >> 3, t = (pp & 7) >> 1, odd = pp & 1;
  if (HD == 128) return code_bytes(HD) + hi * 512 + ((j >> 1) * 4 + t) * 16 + odd * 8 + (j & 1) * 4;
  return code_bytes(HD) + (j * 4 + t) * 16 + (hi * 2 + odd) * 4;
}
template <int HD>
__device__ __forceinline__ int k_scale(int pp, int i) {
  const int g = pp & 7, hi = pp >> 3;
  if (HD == 128) return 2 * code_bytes(HD) + (g * 4 + (i >> 1)) * 4 + hi * 2 + (i & 1);
  return 2 * code_bytes(HD) + (g * 4 + i) * 2 + hi;
}
template <int HD>
__device__ __forceinline__ int v_scale(int pp, int i) {
  const int hi = pp >> 3, t = (pp & 7) >> 1, odd = pp & 1;
  return 2 * code_bytes(HD) + scale_bytes(HD) + (i * 4 + t) * 4 + hi * 2 + odd;  // (hd 128: i = g; hd 64: i = g / 2)
}

__device__ __forceinline__ float scale_of(int b) {
  return 8.0f * __half2float(__ushort_as_half((unsigned short)(b << 7)));
}

// The scale byte of a run whose largest magnitude has the bits `mag`: max / 7 (and / 8) rounded to
// 3 mantissa bits.
__device__ __forceinline__ int scale_byte(uint32_t mag) {
  if (mag >= 0x7F800000u) return kScaleNan;
  const float w = fminf(__fdiv_rn(__uint_as_float(mag), 7.0f) * 0.125f, 60.0f);
  if (w < 6.103515625e-05f) return __float2int_rn(w * 131072.0f);  // below 2^-14: steps of 2^-17
  uint32_t u = __float_as_uint(w);
  u += 0x7FFFFu + ((u >> 20) & 1u);
  return (int)(u >> 20) - (112 << 3);
}

// Eight values as a word of codes at scale s (0: an empty or NaN run, every code 0).
__device__ __forceinline__ uint32_t code_word(const float (&x)[8], float s) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // (a correctly rounded quotient: bf16 values lie exactly half way between codes often, and a
    // reciprocal's error would send those the wrong way)
    const int c = s > 0.f ? max(-8, min(7, __float2int_rn(__fdiv_rn(x[i], s)))) : 0;
    w |= (uint32_t)(c + 8) << (4 * i);
  }
  return w;
}

struct Seqs {
  int batch, n_tokens, max_pages;
  const int32_t *cu, *lengths, *table;
  long long table_stride;
};
struct Cache {
  uint8_t* pages;
  int n_pages, page_shift, hkv;
  int* status;
};
struct Rows {
  void* p;
  long long ts, hs;
};

__device__ __forceinline__ void raise(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// The sequence that token row `row` belongs to (-1: none) and its index there.
__device__ __forceinline__ int seq_of(const Seqs& s, int row, int& j) {
  if (!s.cu) {
    j = 0;
    return row;
  }
  if (row < __ldg(s.cu) || row >= __ldg(s.cu + s.batch)) return -1;
  int lo = 0, hi = s.batch;  // cu[lo] <= row < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(s.cu + mid) <= row) lo = mid;
    else hi = mid;
  }
  j = row - __ldg(s.cu + lo);
  return lo;
}

// The group of (sequence b, position pos, KV head h), or null where the tables do not reach.
template <int HD>
__device__ __forceinline__ uint8_t* group_at(const Cache& c, const Seqs& s, int b, int pos, int h) {
  const int e = pos >> c.page_shift;
  if (pos < 0 || e >= s.max_pages) {
    raise(c.status, DEC_ERR_CAPACITY);
    return nullptr;
  }
  const int page = __ldg(s.table + b * s.table_stride + e);
  if ((unsigned)page >= (unsigned)c.n_pages) {
    raise(c.status, DEC_ERR_ARG);
    return nullptr;
  }
  const int gpp = 1 << (c.page_shift - 4);
  return c.pages + (((size_t)page * c.hkv + h) * gpp + ((pos >> 4) & (gpp - 1))) * group_bytes(HD);
}

// Eight consecutive values of a row in fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, long long at, float (&x)[8]) {
  if (F32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = f[0], b = f[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct AppendParams {
  Cache c;
  Seqs s;
  Rows q, k, v, qo;
  const uint16_t *qn, *kn;
  const float* rope;
  int hq, rope_len, rot, inter;
  float eps;
};

// One row (token, head) per HD / 8 lanes, eight values a lane: query heads, then key and value
// heads. Norm and rotation exchange values by shuffles inside the row; a scale's run is two lanes.
template <int HD, bool F32>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  constexpr int LPR = HD / 8;
  const int per_tok = p.hq + 2 * p.c.hkv;
  const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  const bool live = row < (long long)p.s.n_tokens * per_tok;
  const int tok = live ? (int)(row / per_tok) : 0;
  int h = live ? (int)(row % per_tok) : 0;
  int j = 0;
  const int b = live ? seq_of(p.s, tok, j) : -1;
  const int kind = h < p.hq ? 0 : h < p.hq + p.c.hkv ? 1 : 2;  // q, k, v
  h -= kind == 0 ? 0 : kind == 1 ? p.hq : p.hq + p.c.hkv;
  bool on = b >= 0;
  int pos = 0;
  if (on) {
    pos = __ldg(p.s.lengths + b) + j;
    if (pos < 0) {
      raise(p.c.status, DEC_ERR_ARG);
      on = false;
    } else if (p.rot && kind < 2 && pos >= p.rope_len) {
      raise(p.c.status, DEC_ERR_CAPACITY);
      on = false;
    }
  }
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const Rows& in = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  if (on) load8<F32>(in.p, tok * in.ts + h * in.hs + l * 8, x);
  const uint16_t* nw = kind == 0 ? p.qn : kind == 1 ? p.kn : nullptr;
  // (a shuffle's lanes all run it: rows of a warp differ in kind)
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (nw && on) {
    const float inv = 1.0f / sqrtf(ss / (float)HD + p.eps);
    float w[8];
    load8<false>(nw, l * 8, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
  }
  if (p.rot) {
    const int half = p.rot / 2;
    const bool turn = on && kind < 2 && l * 8 < p.rot;
    const float* cs = p.rope + (long long)pos * p.rot;
    if (p.inter) {
      if (turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 t = *reinterpret_cast<const float2*>(cs + l * 8 + 2 * i);
          const float a = x[2 * i], c = x[2 * i + 1];
          x[2 * i] = a * t.x - c * t.y;
          x[2 * i + 1] = a * t.y + c * t.x;
        }
      }
    } else {
      const bool first = l * 8 < half;
      const int other = turn ? (first ? l + half / 8 : l - half / 8) : l;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], other, LPR);
        if (turn) {
          const float2 t = *reinterpret_cast<const float2*>(cs + 2 * ((first ? l * 8 : l * 8 - half) + i));
          x[i] = first ? x[i] * t.x - y * t.y : y * t.y + x[i] * t.x;
        }
      }
    }
  }
  if (kind == 0) {
    if (on) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.qo.p) + tok * p.qo.ts + h * p.qo.hs + l * 8) = pack8_bf16(x);
  }
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) mag = max(mag, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
  if (kind == 0 || !on) return;
  uint8_t* grp = group_at<HD>(p.c, p.s, b, pos, h);
  if (!grp) return;
  const int sb = scale_byte(mag);
  const uint32_t w = code_word(x, sb == kScaleNan ? 0.f : scale_of(sb));
  const int pp = pos & 15;
  *reinterpret_cast<uint32_t*>(grp + (kind == 1 ? k_word<HD>(pp, l) : v_word<HD>(pp, l))) = w;
  if ((l & 1) == 0) grp[kind == 1 ? k_scale<HD>(pp, l >> 1) : v_scale<HD>(pp, l >> 1)] = (uint8_t)sb;
}

// Eight values of a word of codes at scale s.
__device__ __forceinline__ void decode8(uint32_t w, float s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)((int)((w >> (4 * i)) & 15u) - 8) * s;
}

struct GatherParams {
  Cache c;
  Seqs s;
  Rows k, v;
};

template <int HD>
__global__ void __launch_bounds__(256) gather_kernel(const GatherParams p) {
  constexpr int LPR = HD / 8;
  const int per_tok = 2 * p.c.hkv;
  const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  if (row >= (long long)p.s.n_tokens * per_tok) return;
  const int tok = (int)(row / per_tok), hh = (int)(row % per_tok);
  const bool isv = hh >= p.c.hkv;
  const int h = isv ? hh - p.c.hkv : hh;
  int j = 0;
  const int b = seq_of(p.s, tok, j);
  if (b < 0) return;
  const int pos = __ldg(p.s.lengths + b) + j;
  if (pos < 0) {
    raise(p.c.status, DEC_ERR_ARG);
    return;
  }
  const uint8_t* grp = group_at<HD>(p.c, p.s, b, pos, h);
  if (!grp) return;
  const int pp = pos & 15;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(grp + (isv ? v_word<HD>(pp, l) : k_word<HD>(pp, l)));
  const int sb = grp[isv ? v_scale<HD>(pp, l >> 1) : k_scale<HD>(pp, l >> 1)];
  float x[8];
  decode8(w, scale_of(sb), x);
  const Rows& o = isv ? p.v : p.k;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.p) + tok * o.ts + h * o.hs + l * 8) = pack8_bf16(x);
}

}  // namespace kvq
}  // namespace dec
