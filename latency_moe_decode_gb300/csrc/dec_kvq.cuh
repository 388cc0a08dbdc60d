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
  const float m = __uint_as_float(mag), q = m * (1.0f / 7.0f);
  const float w = fminf(fmaf(fmaf(-q, 7.0f, m), 1.0f / 7.0f, q) * 0.125f, 60.0f);  // (see code_word)
  if (w < 6.103515625e-05f) return __float2int_rn(w * 131072.0f);  // below 2^-14: steps of 2^-17
  uint32_t u = __float_as_uint(w);
  u += 0x7FFFFu + ((u >> 20) & 1u);
  return (int)(u >> 20) - (112 << 3);
}

// Eight values as a word of codes at scale s (0: an empty or NaN run, every code 0).
__device__ __forceinline__ uint32_t code_word(const float (&x)[8], float s) {
  if (!(s > 0.f)) return 0x88888888u;
  float inv, c[8];
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // The quotient with one correction by its exact remainder: bf16 values lie exactly half way
    // between two codes often, and a quotient that is such a half comes out exact (x inv alone may
    // fall on either side of it).
    const float q = x[i] * inv, r = fmaf(-q, s, x[i]);
    const float y = fminf(fmaxf(fmaf(r, inv, q), -8.f), 7.f);
    c[i] = (y + 12582912.f) - 12582904.f;  // to the nearest whole number, ties to even; + 8
  }
  // four codes make a whole number below 2^16, which 2^23 leaves in the low mantissa bits
  const float lo = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]);
  const float hi = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]);
  return __byte_perm(__float_as_uint(lo + 8388608.f), __float_as_uint(hi + 8388608.f), 0x5410);
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

// The sequence that token row `row` (the same in the whole warp) belongs to (-1: none) and its index
// there: 32 bounds at a time.
__device__ __forceinline__ int seq_of_warp(const Seqs& s, int row, int& j) {
  if (!s.cu) {
    j = 0;
    return row;
  }
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = s.batch, at = 0;  // cu[lo] <= row
  if (row >= __ldg(s.cu + s.batch)) return -1;
  for (;;) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const int v = i < hi ? __ldg(s.cu + i) : 0x7FFFFFFF;
    const uint32_t below = __ballot_sync(0xffffffffu, v <= row);
    if (!below) return -1;  // (before the first sequence)
    const int k = 31 - __clz(below);
    at = __shfl_sync(0xffffffffu, v, k);
    lo += k * step;
    if (step == 1) break;
    hi = min(hi, lo + step);
  }
  j = row - at;
  return lo;
}

// Eight values as they were read.
template <bool F32>
struct Raw {
  uint4 u[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, long long at) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (F32 ? 4 : 2));
    u[0] = __ldcs(q);
    if (F32) u[F32 ? 1 : 0] = __ldcs(q + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[F32 ? 1 : 0].x, u[F32 ? 1 : 0].y, u[F32 ? 1 : 0].z, u[F32 ? 1 : 0].w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = F32 ? __uint_as_float(w[i]) : __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};

// One CTA per token: HD / 8 lanes a row (head), eight values a lane, query heads first, then key and
// value heads. Norm and rotation exchange values by shuffles inside the row, a scale's run is two
// lanes. What bounds it: for prompts the bytes of the rows (the token's angles and norm weights are
// read once for all its heads, the rows ahead of the position that they wait for); for single tokens
// the chain bounds -> length -> page, 2 to 3 us.
// CTAs of 256 threads while they leave SMs empty, of 128 beyond: what precedes the rows costs every
// warp alike (8 k tokens of 32 + 16 heads of 128: 77 us with 256 and IEEE quotients and roots).
template <int HD, bool F32, int T>
__global__ void __launch_bounds__(T) append_kernel(const AppendParams p) {
  constexpr int LPR = HD / 8, SLOTS = T / LPR, R = 3;
  const int tok = blockIdx.x, l = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int per_tok = p.hq + 2 * p.c.hkv;
  Raw<F32> raw[R];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = r0 + slot + i * SLOTS;
      const Rows& in = r < p.hq ? p.q : r < p.hq + p.c.hkv ? p.k : p.v;
      const int h = r < p.hq ? r : r < p.hq + p.c.hkv ? r - p.hq : r - p.hq - p.c.hkv;
      if (r < per_tok) raw[i].load(in.p, tok * in.ts + h * in.hs + l * 8);
    }
  };
  fetch(0);
  int j = 0;
  const int b = seq_of_warp(p.s, tok, j);
  if (b < 0) return;
  const long long where = (long long)__ldg(p.s.lengths + b) + j;
  const int pos = (int)min(where, 0x7FFFFFFFll);
  if (pos < 0) {
    raise(p.c.status, DEC_ERR_ARG);
    return;
  }
  const bool turns = p.rot > 0, far = turns && pos >= p.rope_len;  // (beyond the table: keys and queries are skipped)
  if (far) raise(p.c.status, DEC_ERR_CAPACITY);
  // the page, and the lane's angles: pairs (8l + i, its partner), or four pairs of neighbours
  const int e = pos >> p.c.page_shift, gpp = 1 << (p.c.page_shift - 4);
  int page = -1;
  if (e >= p.s.max_pages) raise(p.c.status, DEC_ERR_CAPACITY);
  else if ((unsigned)(page = __ldg(p.s.table + b * p.s.table_stride + e)) >= (unsigned)p.c.n_pages) {
    raise(p.c.status, DEC_ERR_ARG);
    page = -1;
  }
  const int half = p.rot / 2;
  const bool mine = turns && !far && l * 8 < p.rot, first = l * 8 < half;
  const int other = mine && !p.inter ? (first ? l + half / 8 : l - half / 8) : l;
  float cs[8], sn[8];
  if (mine) {
    const float4* t = reinterpret_cast<const float4*>(p.rope + (long long)pos * p.rot + (p.inter ? l * 8 : 2 * (first ? l * 8 : l * 8 - half)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p.inter && i >= 2) break;
      const float4 a = __ldg(t + i);
      cs[2 * i] = a.x;
      sn[2 * i] = a.y;
      cs[2 * i + 1] = a.z;
      sn[2 * i + 1] = a.w;
    }
  }
  uint8_t* const grp = page < 0 ? nullptr
                                : p.c.pages + ((size_t)page * p.c.hkv * gpp + ((pos >> 4) & (gpp - 1))) * group_bytes(HD);
  const int pp = pos & 15;
  for (int r0 = 0; r0 < per_tok; r0 += R * SLOTS) {
    if (r0 > 0) fetch(r0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = r0 + slot + i * SLOTS;
      if (r0 + i * SLOTS >= per_tok) break;  // (the same in the whole CTA)
      const bool in = r < per_tok;
      const int kind = r < p.hq ? 0 : r < p.hq + p.c.hkv ? 1 : 2;  // q, k, v
      const int h = kind == 0 ? r : kind == 1 ? r - p.hq : r - p.hq - p.c.hkv;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (in) raw[i].get(x);
      const uint16_t* nw = kind == 0 ? p.qn : kind == 1 ? p.kn : nullptr;
      if (p.qn || p.kn) {  // (a shuffle's lanes all run it: rows of a warp differ in kind)
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (nw) {
          const float m = fmaf(ss, 1.0f / HD, p.eps);
          float inv = rsqrtf(m);
          inv = inv * fmaf(-0.5f * m * inv, inv, 1.5f);  // (one step: to the last place or two)
          float w[8];
          load8<false>(nw, l * 8, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = x[k] * inv * w[k];
        }
      }
      if (turns) {
        if (p.inter) {
          if (mine && kind < 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = x[2 * k], c = x[2 * k + 1];
              x[2 * k] = a * cs[k] - c * sn[k];
              x[2 * k + 1] = a * sn[k] + c * cs[k];
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float y = __shfl_sync(0xffffffffu, x[k], other, LPR);
            if (mine && kind < 2) x[k] = first ? x[k] * cs[k] - y * sn[k] : y * sn[k] + x[k] * cs[k];
          }
        }
      }
      if (kind == 0 && in && !far)
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.qo.p) + tok * p.qo.ts + h * p.qo.hs + l * 8), pack8_bf16(x));
      if (!__any_sync(0xffffffffu, kind > 0 && in)) continue;
      uint32_t mag = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) mag = max(mag, __float_as_uint(x[k]) & 0x7FFFFFFFu);
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
      if (in && grp && (kind == 2 || (kind == 1 && !far))) {
        uint8_t* const at = grp + (size_t)h * gpp * group_bytes(HD);
        const int sb = scale_byte(mag);
        *reinterpret_cast<uint32_t*>(at + (kind == 1 ? k_word<HD>(pp, l) : v_word<HD>(pp, l))) =
            code_word(x, sb == kScaleNan ? 0.f : scale_of(sb));
        if ((l & 1) == 0) at[kind == 1 ? k_scale<HD>(pp, l >> 1) : v_scale<HD>(pp, l >> 1)] = (uint8_t)sb;
      }
    }
  }
}

// Eight values of a word of codes at scale byte sb, as bf16: (code + 8) enters the low mantissa bits of
// the bf16 128, and (128 + u) s - 136 s is exact (136 = 17 * 8, s of 4 significant bits).
__device__ __forceinline__ uint4 decode8(uint32_t w, int sb) {
  const __nv_bfloat162 s = __float2bfloat162_rn(scale_of(sb)), c = __hmul2(s, __float2bfloat162_rn(-136.0f));
  uint32_t v[4];  // values i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), s, c);
    v[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                    __byte_perm(v[2], v[3], 0x7632));
}

struct GatherParams {
  Cache c;
  Seqs s;
  Rows k, v;
};

// One CTA of two warps per token, HD / 8 lanes a row; the rows' loads four at a time.
template <int HD>
__global__ void __launch_bounds__(64) gather_kernel(const GatherParams p) {
  constexpr int LPR = HD / 8, SLOTS = 64 / LPR, R = 4;
  const int tok = blockIdx.x, l = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  int j = 0;
  const int b = seq_of_warp(p.s, tok, j);
  if (b < 0) return;
  const long long where = (long long)__ldg(p.s.lengths + b) + j;
  if (where < 0 || where > 0x7FFFFFFFll) {
    raise(p.c.status, where < 0 ? DEC_ERR_ARG : DEC_ERR_CAPACITY);
    return;
  }
  const int pos = (int)where, pp = pos & 15, gpp = 1 << (p.c.page_shift - 4);
  const uint8_t* const grp = group_at<HD>(p.c, p.s, b, pos, 0);
  if (!grp) return;
  const int kw = k_word<HD>(pp, l), vw = v_word<HD>(pp, l), ks = k_scale<HD>(pp, l >> 1), vs = v_scale<HD>(pp, l >> 1);
  for (int r0 = slot; r0 < 2 * p.c.hkv; r0 += R * SLOTS) {
    uint32_t w[R];
    int sb[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = r0 + i * SLOTS;
      const bool isv = r >= p.c.hkv;
      const uint8_t* at = grp + (size_t)(isv ? r - p.c.hkv : r) * gpp * group_bytes(HD);
      if (r < 2 * p.c.hkv) {
        w[i] = *reinterpret_cast<const uint32_t*>(at + (isv ? vw : kw));
        sb[i] = at[isv ? vs : ks];
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = r0 + i * SLOTS;
      if (r >= 2 * p.c.hkv) break;
      const Rows& o = r >= p.c.hkv ? p.v : p.k;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.p) + tok * o.ts + (r >= p.c.hkv ? r - p.c.hkv : r) * o.hs + l * 8) =
          decode8(w[i], sb[i]);
    }
  }
}

}  // namespace kvq
}  // namespace dec
