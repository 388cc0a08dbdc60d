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
constexpr int kMaxSeqs = 256;    // sequences of one launch (their table lies in shared memory)

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

// Keys that come out of the norm and the rotation have gone through some 16 fp32 roundings (the sum of
// squares, halved by the root; the root; two products; the rotation), which leave a standard deviation of
// about 1.5 x 2^-24 of the pair's larger value: one code in a million would be the neighbour of what the
// formula gives. Where that error, or that of fp32 values as they are, may have made the choice (CHECK,
// near), the row is made anew with twice the bits (settle_row). kNear is five deviations, for values up to
// 8 codes: one row in 1000 is made anew; a bound on all roundings at once would take three times as many.
// A rotation may leave a run much smaller than the values that it was made of, whose roundings it keeps: the
// larger result of a pair is at least the larger product over the root of 2, so the largest result of the
// run's pairs, times 1.5 where it is well above the run's own (`big`), widens the search in proportion.
constexpr float kNear = 0x1p-18f;

// The scale byte of a run whose largest magnitude has the bits `mag`: max / 7 (and / 8) rounded to
// 3 mantissa bits.
template <bool CHECK>
__device__ __forceinline__ int scale_byte(uint32_t mag, float big, bool& near) {
  if (mag >= 0x7F800000u) return kScaleNan;
  const float m = __uint_as_float(mag), q = m * (1.0f / 7.0f);
  const float w = fminf(fmaf(fmaf(-q, 7.0f, m), 1.0f / 7.0f, q) * 0.125f, 60.0f);  // (see code_word)
  uint32_t u = __float_as_uint(w);
  float wide = 1.f;
  if (CHECK) {
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(wide) : "f"(m));
    wide = fmaxf(big * wide, 1.f);  // (0 x infinity: 1)
  }
  if (w < 6.103515625e-05f) {  // below 2^-14: steps of 2^-17
    const float v = w * 131072.0f;
    if (CHECK) near |= fabsf(v - floorf(v) - 0.5f) <= 0x1p-17f * wide;
    return __float2int_rn(v);
  }
  if (CHECK) near |= fabsf((float)(u & 0xFFFFFu) - 524288.f) <= 8.f * wide;
  u += 0x7FFFFu + ((u >> 20) & 1u);
  return (int)(u >> 20) - (112 << 3);
}

// Eight values as a word of codes at scale s (0: an empty or NaN run, every code 0).
template <bool CHECK>
__device__ __forceinline__ uint32_t code_word(const float (&x)[8], float s, float big, bool& near) {
  if (!(s > 0.f)) return 0x88888888u;
  float inv, c[8], d = 0.f;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // The quotient with one correction by its exact remainder: bf16 values lie exactly half way
    // between two codes often, and a quotient that is such a half comes out exact (x inv alone may
    // fall on either side of it).
    const float q = x[i] * inv, r = fmaf(-q, s, x[i]);
    const float y = fminf(fmaxf(fmaf(r, inv, q), -8.f), 7.f);
    c[i] = (y + 12582912.f) - 12582912.f;  // to the nearest whole number, ties to even
    if (CHECK) d = fmaxf(d, fabsf(y - c[i]));
  }
  if (CHECK) near |= d >= 0.5f - kNear * fmaxf(big * inv * 0.125f, 1.f);
  // four codes + 8 make a whole number below 2^16, which 2^23 leaves in the low mantissa bits
  const float lo = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]);
  const float hi = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]);
  constexpr float k8 = 8388608.f + 8.f * (1 + 16 + 256 + 4096);
  return __byte_perm(__float_as_uint(lo + k8), __float_as_uint(hi + k8), 0x5410);
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

// Eight consecutive bf16 values in fp32.
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
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
  const int32_t* at;  // rotary positions of the token rows (null: where they stand in the cache)
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

// The unevaluated sum of two floats, about 46 bits (64-bit arithmetic runs at a hundredth of fp32's rate
// here: a row settled in it took 12 us, and takes 2 like this).
struct Two {
  float h, l;
};
__device__ __forceinline__ Two renorm(float h, float l) {  // |l| below |h|
  const float s = h + l;
  return Two{s, l - (s - h)};
}
__device__ __forceinline__ Two add(const Two& a, const Two& b) {
  const float s = a.h + b.h, t = s - a.h;
  return renorm(s, (a.h - (s - t)) + (b.h - t) + (a.l + b.l));
}
__device__ __forceinline__ Two mul(float a, float b) {
  const float h = a * b;
  return Two{h, fmaf(a, b, -h)};
}
__device__ __forceinline__ Two mul(const Two& a, float b) {
  const float h = a.h * b;
  return renorm(h, fmaf(a.l, b, fmaf(a.h, b, -h)));
}
__device__ __forceinline__ Two shfl_xor(const Two& a, int m) {
  return Two{__shfl_xor_sync(0xffffffffu, a.h, m), __shfl_xor_sync(0xffffffffu, a.l, m)};
}

// 32 values of a row of keys or values anew, by a warp, from value d0 on: norm (nw: its weights, or null),
// rotation (rot values, by the angles at `ang`), scales and codes with 46 bits. Latency is all of it: the
// loads are asked for at once, the row's parts go to as many warps.
template <int HD, bool F32>
__device__ __noinline__ void settle_row(const void* x, const uint16_t* nw, float eps, const float2* ang, int rot, bool inter,
                                        bool key, int pp, int d0, uint8_t* at) {
  const int lane = threadIdx.x & 31, half = rot / 2, d = d0 + lane;
  auto value = [&](int i) {
    return F32 ? static_cast<const float*>(x)[i] : __uint_as_float((uint32_t) static_cast<const uint16_t*>(x)[i] << 16);
  };
  // its pair's other value, and the angle
  const bool first = inter ? !(d & 1) : d < half, turned = d < rot;
  const int o = !turned ? d : inter ? d ^ 1 : first ? d + half : d - half;
  float all[HD / 32];
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) all[i] = value(i * 32 + lane);
  const float a = value(d), b = value(o);
  const float wa = nw ? __uint_as_float((uint32_t)nw[d] << 16) : 1.f, wb = nw ? __uint_as_float((uint32_t)nw[o] << 16) : 1.f;
  const float2 turn = turned ? __ldg(ang + (inter ? d >> 1 : first ? d : o)) : make_float2(1.f, 0.f);
  Two inv{1.f, 0.f};
  if (nw) {
    Two m = mul(all[0], all[0]);
#pragma unroll
    for (int i = 1; i < HD / 32; ++i) m = add(m, mul(all[i], all[i]));
#pragma unroll 1
    for (int i = 16; i > 0; i >>= 1) m = add(m, shfl_xor(m, i));
    m = add(Two{m.h * (1.0f / HD), m.l * (1.0f / HD)}, Two{eps, 0.f});
    // 1 / sqrt(m) = r (1 + e / 2 + 3 e^2 / 8 ..), e = 1 - m r^2
    const float r = rsqrtf(m.h);
    const Two rr = mul(r, r);
    const float e = fmaf(-m.h, rr.h, 1.f) - fmaf(m.h, rr.l, m.l * rr.h);
    inv = renorm(r, r * e * fmaf(0.375f, e, 0.5f));
  }
  auto normed = [&](float y, float w) {
    const Two u = mul(y, w), v = mul(u, inv.h);
    return renorm(v.h, fmaf(u.h, inv.l, v.l));
  };
  Two v = normed(a, wa);
  if (turned) v = add(mul(v, turn.x), mul(normed(b, wb), first ? -turn.y : turn.y));
  // the run's largest magnitude: 16 lanes
  Two m{fabsf(v.h), v.h < 0.f ? -v.l : v.l};
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const Two y = shfl_xor(m, o);
    if (m.h == m.h && (!(y.h <= m.h) || (y.h == m.h && y.l > m.l))) m = y;  // (a NaN stays)
  }
  bool unused = false;
  int sb = m.h <= 3.4028235e38f ? scale_byte<false>(__float_as_uint(m.h), 0.f, unused) : kScaleNan;
  if (sb != kScaleNan) {
    // 7 times the middle to the scale above and to the one below
    const float up = sb < kScaleMax ? (m.h - 3.5f * (scale_of(sb) + scale_of(sb + 1))) + m.l : -1.f;
    const float down = sb > 0 ? (m.h - 3.5f * (scale_of(sb) + scale_of(sb - 1))) + m.l : 1.f;
    if (up > 0.f || (up == 0.f && (sb & 1))) ++sb;
    else if (down < 0.f || (down == 0.f && (sb & 1))) --sb;
  }
  int code = 8;
  if (sb != 0 && sb != kScaleNan) {
    const float s = scale_of(sb);
    float c, inv_s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv_s) : "f"(s));
    c = rintf(v.h * inv_s);  // (one off at most)
    const float e = fmaf(-c, s, v.h), over = (e - 0.5f * s) + v.l, under = (e + 0.5f * s) + v.l;
    const bool odd = (int)c & 1;
    if (over > 0.f || (over == 0.f && odd)) c += 1.f;
    else if (under < 0.f || (under == 0.f && odd)) c -= 1.f;
    code = (int)fminf(fmaxf(c, -8.f), 7.f) + 8;
  }
  uint32_t word = (uint32_t)code << (4 * (lane & 7));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
  if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(at + (key ? k_word<HD>(pp, d >> 3) : v_word<HD>(pp, d >> 3))) = word;
  if ((lane & 15) == 0) at[key ? k_scale<HD>(pp, d >> 4) : v_scale<HD>(pp, d >> 4)] = (uint8_t)sb;
}

// One CTA per token: HD / 8 lanes a row (head), eight values a lane, query heads first, then key and
// value heads. Norm and rotation exchange values by shuffles inside the row, a scale's run is two
// lanes. What bounds it: for prompts the instructions (270 a warp for two rows, issue slots
// 75 to 80 % full; the bytes would take half the time; packed fp32 pairs changed nothing). The token's
// angles are read once for all its heads (the norm's weights for each of them, which leaves more registers for
// rows in flight), the rows ahead of the position that they wait for. For single tokens the chain bounds -> length -> page, 2 to 3 us.
// CTAs of 256 threads while the SMs hold them all at once (four each), of 128 beyond: what precedes the
// rows costs every warp alike. 256 against 128 threads, 32 + 16 heads of 128: one token 4.2 us against
// 5.7, 304 5.1 / 6.4, 608 8.6 / 8.6, 1216 13.6 / 12.4. 9.3 k tokens take 64, of which looking for choices left open
// is 4 and settling them 1; with 256 threads and IEEE quotients a quarter more.
template <int HD, bool F32, int T>
__global__ void __launch_bounds__(T) append_kernel(const AppendParams p) {
  constexpr int LPR = HD / 8, SLOTS = T / LPR, R = 3;
  __shared__ uint32_t todo[64];  // a bit a row of keys (1024 at most), and of values
  bool any = false;
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
  if (threadIdx.x < 64) todo[threadIdx.x] = 0;
  __syncthreads();
  int j = 0;
  const int b = seq_of_warp(p.s, tok, j);
  if (b < 0) return;
  const long long where = (long long)__ldg(p.s.lengths + b) + j;
  const int pos = (int)min(where, 0x7FFFFFFFll);
  if (pos < 0) {
    raise(p.c.status, DEC_ERR_ARG);
    return;
  }
  const bool turns = p.rot > 0;
  const int turn = turns && p.at ? __ldg(p.at + tok) : pos;
  if (turn < 0) {
    raise(p.c.status, DEC_ERR_ARG);
    return;
  }
  const bool far = turns && turn >= p.rope_len;  // (beyond the table: the row is skipped)
  // the page, and the lane's angles: pairs (8l + i, its partner), or four pairs of neighbours
  const int e = pos >> p.c.page_shift, gpp = 1 << (p.c.page_shift - 4);
  int page = -1;
  if (far || e >= p.s.max_pages) raise(p.c.status, DEC_ERR_CAPACITY);
  else if ((unsigned)(page = __ldg(p.s.table + b * p.s.table_stride + e)) >= (unsigned)p.c.n_pages) {
    raise(p.c.status, DEC_ERR_ARG);
    page = -1;
  }
  const int half = p.rot / 2;
  const bool mine = turns && !far && l * 8 < p.rot, first = l * 8 < half;
  const int other = mine && !p.inter ? (first ? l + half / 8 : l - half / 8) : l;
  float cs[8], sn[8];
  if (mine) {
    const float4* t = reinterpret_cast<const float4*>(p.rope + (long long)turn * p.rot +
                                                      (p.inter ? l * 8 : 2 * (first ? l * 8 : l * 8 - half)));
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
          load8(nw + l * 8, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = x[k] * inv * w[k];
        }
      }
      const bool keys = (p.kn || turns) && __any_sync(0xffffffffu, kind == 1 && in);  // (some, with roundings behind them)
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
      uint32_t pair = mag;  // with the pairs' other values
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
      int sb;
      uint32_t word;
      bool near = false;
      if (keys || F32) {  // (bf16 values as they are lie on a middle or well beside it, fp32 ones may be just beside)
        pair = max(pair, __shfl_sync(0xffffffffu, pair, other, LPR));
        pair = max(pair, __shfl_xor_sync(0xffffffffu, pair, 1));
        const float big = kind == 1 ? fmaf(1.5f, __uint_as_float(pair), -0.5f * __uint_as_float(mag)) : 0.f;
        sb = scale_byte<true>(mag, big, near);
        word = code_word<true>(x, sb == kScaleNan ? 0.f : scale_of(sb), big, near);
        if (near && in && kind > 0 && (F32 || kind == 1)) {
          atomicOr(&todo[(kind - 1) * 32 + (h >> 5)], 1u << (h & 31));
          any = true;
        }
      } else {
        sb = scale_byte<false>(mag, 0.f, near);
        word = code_word<false>(x, sb == kScaleNan ? 0.f : scale_of(sb), 0.f, near);
      }
      if (in && grp && kind > 0) {
        uint8_t* const at = grp + (size_t)h * gpp * group_bytes(HD);
        *reinterpret_cast<uint32_t*>(at + (kind == 1 ? k_word<HD>(pp, l) : v_word<HD>(pp, l))) = word;
        if ((l & 1) == 0) at[kind == 1 ? k_scale<HD>(pp, l >> 1) : v_scale<HD>(pp, l >> 1)] = (uint8_t)sb;
      }
    }
  }
  if (!__syncthreads_or(any) || !grp) return;
  // ---- rows with a choice left open: 32 values a warp
  constexpr int PARTS = HD / 32;
  const int warp = threadIdx.x / 32;
  for (int i = 0, n = 0, words = (p.c.hkv + 31) / 32; i < 2 * words; ++i)
    for (uint32_t m = todo[i < words ? i : 32 + i - words]; m; m &= m - 1, ++n) {
      if (n % (T / 32 / PARTS) != warp / PARTS) continue;
      const bool key = i < words;
      const int h = (key ? i : i - words) * 32 + __ffs(m) - 1;
      const Rows& in = key ? p.k : p.v;
      settle_row<HD, F32>(static_cast<const char*>(in.p) + (tok * in.ts + h * in.hs) * (F32 ? 4 : 2), key ? p.kn : nullptr,
                          p.eps, reinterpret_cast<const float2*>(p.rope + (long long)turn * p.rot), key && turns ? p.rot : 0,
                          p.inter != 0, key, pp, warp % PARTS * 32, grp + (size_t)h * gpp * group_bytes(HD));
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

// One CTA of two warps per token, HD / 8 lanes a row; the rows' loads four at a time. 9.3 k tokens of 8 heads
// of 128 take 11 us where their 49 MB take 7: the chain bounds, length, page, codes of each token, and the
// instructions (issue slots 64 % full).
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
