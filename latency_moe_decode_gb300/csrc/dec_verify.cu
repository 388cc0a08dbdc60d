// Verification of drafted tokens against the target's probabilities (dec_verify_drafts of dec.h).
//
// Two kernels. The first reads every row of logits once: its largest logit (and that one's id) and the sum of
// exp((x - max) / temperature) in fp32, which is what acceptance needs. The second walks the trees, a CTA or a
// cluster of CTAs per sequence: the walk itself is arithmetic on a few numbers per draft, all fetched and weighed at
// once; then the row that the walk ends at is summed again, for the next token. There a border between two of a
// vocabulary's tokens is met with every draw, and sums that are off by 2^-24 of the whole would pick the neighbour
// of the formula's token once in some thousand draws. So those sums, and the few acceptances that the
// first kernel's sums leave open, are taken in unevaluated pairs of floats (some 36 bits; 64-bit arithmetic runs at a
// hundredth of fp32's rate).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "dec.h"
#include "dec_f32x2.cuh"
#include "dec_kvq.cuh"
#include "dec_ops.h"

namespace dec {
namespace verify {

using kvq::Two;
using kvq::renorm;

constexpr int kRowThreads = 256;
constexpr int kWalkThreads = 512;
constexpr int kWalkWarps = kWalkThreads / 32;
constexpr int kMaxParts = 32;  // of a row
constexpr int kRowWarps = 32;   // of the first kernel, an SM
constexpr int kMaxCluster = 8;
// What the first kernel's sums are trusted to, relative to themselves, where a thread makes `steps` of 16 values and a sequence
// has up to `rows` drafts; in units of 2^-24, all of one sign. A step: one addition, and where the maximum rises a product with
// an exponential (2^-22, and its argument's roundings): 8. Besides: a term's exponential 4, its argument's roundings and those of
// log2(e) / temperature 70 (of an exponent of -y they are some 3 y units, and terms of 2^-y weigh no more than y <= 24 allows),
// a step's own additions 10, merges of lanes and parts 100, the row's factor and the comparison's products 15; and refused
// siblings' weights one an addition. 2^-15 covers the common shapes (32000 ids in 10 parts: 8 steps).
inline float trust_of(long long steps, int rows) {
  return std::max(0x1p-15f, (float)(8 * steps + 200 + rows) * 0x1p-24f);
}
constexpr float kMagic = 12582912.f;  // 1.5 x 2^23: adding it leaves whole numbers in the low mantissa bits

struct Table {
  float2 e[32];  // 2^(i / 32) as two floats
};

struct Params {
  const void* x;
  long long stride, prob_stride;
  const float* probs;
  int vocab, batch, n_tokens, max_tokens;
  int splits, width;  // warps a row (and the next power of two)
  float trust;        // of their sums
  const int32_t *cu, *tokens, *parents;
  const float *uniforms, *temperature;
  int32_t *path, *count, *next;
  float4* stats;  // [n_tokens][width]: largest logit, sum, its id (bits), unused
  Table table;
};

// The sequence's first row and its number of rows.
__device__ __forceinline__ int rows_of(const Params& p, int b, int& first) {
  first = max(0, __ldg(p.cu + b));
  return max(0, min(min(__ldg(p.cu + b + 1), p.n_tokens) - first, p.max_tokens));
}
// log2(e) / temperature (0: greedy)
__device__ __forceinline__ float factor_of(const Params& p, int b) {
  const float t = p.temperature ? __ldg(p.temperature + b) : 1.f;
  return t > 0.f ? fmaxf(fminf(1.4426950408889634f / t, 3.4e38f), 1e-37f) : 0.f;
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, long long i) {
  return BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(row)[i] << 16) : static_cast<const float*>(row)[i];
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A part of a row: its largest logit, the sum relative to that (a NaN, where the row has a NaN or +infinity), the
// first id of it.
struct Stat {
  float m, l;
  int id;
};
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float c) {
  Stat r;
  const bool second = b.m > a.m || (b.m == a.m && b.id < a.id);
  r.m = second ? b.m : a.m;
  r.id = second ? b.id : a.id;
  const float m = finite_or_0(r.m);
  r.l = a.l * ex2((a.m - m) * c) + b.l * ex2((b.m - m) * c);
  return r;
}
__device__ __forceinline__ Stat merge_lanes(Stat a, int width, float c) {
  const int lane = threadIdx.x & 31;
  for (int o = width / 2; o > 0; o >>= 1) {
    const Stat y{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.l, o), __shfl_xor_sync(0xffffffffu, a.id, o)};
    a = (lane & o) ? merge(y, a, c) : merge(a, y, c);
  }
  return a;
}

// ---------------------------------------------------------------------------------------------
// every row once

// Each warp by itself, as many a row as fill the SMs: a CTA a row, or half a row, left some SMs with a wave more than
// others (12.3 us for 464 rows of 32000 fp32; 10.0 so, 5.9 TB/s. bf16 rows go at 4.3: as many exponentials in half the bytes).
// The id of the largest logit is looked for at the end, and only where it counts (greedy rows): in the loop it took
// half the instructions.
template <bool BF16>
__global__ void __launch_bounds__(kRowThreads, kRowWarps * 32 / kRowThreads) rows_kernel(const Params p) {
  constexpr int E = BF16 ? 8 : 4, U = 16 / E;  // 16 values a thread at a time
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, me = (blockIdx.x * kRowThreads + threadIdx.x) / 32;
  kvq::Seqs s{};
  s.batch = p.batch;
  s.cu = p.cu;
  const int row = me / p.splits, split = me - row * p.splits;
  if (row >= p.n_tokens) return;
  const char* const base = static_cast<const char*>(p.x) + row * p.stride * (BF16 ? 2 : 4);
  // 16-byte words from the last boundary before the row; the first and the last may hold values beside it
  const int lead = (int)(reinterpret_cast<uintptr_t>(base) & 15u) / (BF16 ? 2 : 4);
  const uint4* const words = reinterpret_cast<const uint4*>(base - lead * (BF16 ? 2 : 4));
  const int n = (p.vocab + lead + E - 1) / E, per = (n + p.splits - 1) / p.splits;
  const int lo = split * per, hi = min(n, lo + per);
  // the words that lie in the row whole; the next ones are on their way meanwhile
  const int from = max(lo, lead ? 1 : 0), to = min(hi, (p.vocab + lead) / E);
  uint4 v[U];
  auto fetch = [&](int w) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (w + u * 32 < to) v[u] = __ldcs(words + w + u * 32);
  };
  int w0 = from + lane;
  fetch(w0);
  // (meanwhile the row's sequence)
  int j;
  const int b = kvq::seq_of_warp(s, row, j);
  if (b < 0 || j >= p.max_tokens) return;
  const float f = factor_of(p, b), c = f > 0.f ? f : 1.f;  // (greedy: the sum only shows a NaN)
  Stat a{-INFINITY, 0.f, 0x7FFFFFFF};
  int found = 0;  // the words that the largest came from first
  const uint64_t cc = pair(c, c);
  auto take = [&](const float (&x)[16], int w0) {  // 16 values of the words w0, w0 + 32, ..
    float m = a.m;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, x[i]);
    if (m > a.m) {
      a.l *= ex2((a.m - m) * c);
      a.m = m;
      found = w0;
    }
    const float z = finite_or_0(m);
    uint64_t l2 = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 y = halves(fma2(add2(pair(x[i], x[i + 1]), pair(-z, -z)), cc, 0ull));
      l2 = add2(l2, pair(ex2(y.x), ex2(y.y)));
    }
    a.l += halves(l2).x + halves(l2).y;
  };
  // (the first and the last word, where they do not lie in the row whole: a value at a time, and in the ids' order)
  auto edge = [&](int w) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int id = w * E + i - lead;
      x[i] = i < E && id >= 0 && id < p.vocab ? logit<BF16>(base, id) : -INFINITY;
    }
    take(x, w);
  };
  if (lane == 0 && lead && lo == 0) edge(0);
  while (w0 < to) {
    float x[16];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t q[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int i = 0; i < E; ++i)
        x[u * E + i] = BF16 ? __uint_as_float((i & 1) ? q[i / 2] & 0xFFFF0000u : q[i / 2] << 16) : __uint_as_float(q[i % 4]);
    }
    if (w0 - lane + U * 32 > to)  // (the last words)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = w0 + i / E * 32 < to ? x[i] : -INFINITY;
    const int at = w0;
    w0 += U * 32;
    fetch(w0);
    take(x, at);
  }
  if (lane == 1 && hi == n && to < n && (n > 1 || !lead)) edge(n - 1);
  if (f == 0.f && a.m > -INFINITY)  // (only greedy rows need the id)
#pragma unroll
    for (int i = 15; i >= 0; --i) {
      const int id = (found + i / E * 32) * E + i % E - lead;
      if (id >= 0 && id < p.vocab && logit<BF16>(base, id) == a.m) a.id = id;
    }
  a = merge_lanes(a, 32, c);
  if (lane == 0) p.stats[(size_t)row * p.width + split] = make_float4(a.m, a.l, __int_as_float(a.id), 0.f);
}

// ---------------------------------------------------------------------------------------------
// pairs of floats

__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return Two{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ void accumulate(Two& s, const Two& x) {  // (the low parts are gathered, unnormalised)
  const Two y = two_sum(s.h, x.h);
  s.h = y.h;
  s.l += y.l + x.l;
}
__device__ __forceinline__ Two plus(const Two& a, const Two& b) {
  const Two y = two_sum(a.h, b.h);
  return renorm(y.h, y.l + (a.l + b.l));  // (the same whichever way round: lanes that exchange halves agree)
}
// (__fmul_rn: a product whose remainder is taken must not be fused into a sum that it enters)
__device__ __forceinline__ Two times(const Two& a, float b) {
  const float h = __fmul_rn(a.h, b);
  return Two{h, fmaf(a.h, b, -h) + a.l * b};
}
__device__ __forceinline__ Two times(const Two& a, const Two& b) {
  const float h = __fmul_rn(a.h, b.h);
  return renorm(h, fmaf(a.h, b.h, -h) + fmaf(a.h, b.l, a.l * b.h));
}
__device__ __forceinline__ Two minus(const Two& a, const Two& b) { return plus(a, Two{-b.h, -b.l}); }
// what is left of a when b is taken from it
__device__ __forceinline__ Two less(const Two& a, const Two& b) {
  const Two d = minus(a, b);
  return d.h > 0.f ? d : Two{0.f, 0.f};
}
__device__ __forceinline__ Two inverse(const Two& a) {  // one Newton step from 1 / a.h
  const float r = 1.f / a.h, e = fmaf(-a.h, r, 1.f) - a.l * r;
  return renorm(r, r * e);
}
__device__ __forceinline__ bool above(const Two& a, const Two& b) {
  const Two d = two_sum(a.h, -b.h);
  return d.h + (d.l + (a.l - b.l)) > 0.f;
}
__device__ __forceinline__ Two shfl(const Two& a, int lane) {
  return Two{__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}
__device__ __forceinline__ Two sum_lanes(Two a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = plus(a, kvq::shfl_xor(a, o));
  return a;
}
__device__ __forceinline__ Two scan_lanes(Two a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two y{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
    if (lane >= o) a = plus(y, a);
  }
  return a;
}
__device__ __forceinline__ Two two(float2 f) { return Two{f.x, f.y}; }

// Weights of a row's logits: 2^(c (x - base) - M) for a whole number M of 32nds near c (m - base) (a row's weights all have the
// factor 2^(c (m - base) - M) beside exp((x - m) / temperature), which no comparison sees). base is 0, and m where c m passes 256
// either way: a logit is then within a factor of two of m, so that x - m is exact, or its weight is below 2^-120.
// c (x - base) is the exact product P + p, p up to 2^-15; with n = round(32 (P - M)) the difference r = P - (M + n / 32) is
// exact, |r| <= 1/64, and the weight is 2^(n / 32) 2^w with w = r + p. The second factor is 1 + g + .., g = w ln 2, by its series to
// the fourth power (a term of 2^-39.5 is left out); g's first term needs both floats, and so does the table's entry.
// Against 64-bit mantissas, at temperatures from 1e-35 to 1e6, weights are within 2^-35.4 of themselves.
struct RowScale {
  float m, base, low, magic, M, kappa;  // (low: weights below some 2^-120 are 0; magic: kMagic - 32 M; kappa: 2^(c (m - base) - M))
  __device__ __forceinline__ void set(float max, const Two& c) {
    m = max;
    const float n = rintf(c.h * m * 32.f);
    const bool near = fabsf(n) < 8192.f;
    base = near ? 0.f : m;
    M = near ? n * 0.03125f : 0.f;
    magic = kMagic - (near ? n : 0.f);
    low = fmaxf((near ? m : 0.f) - 120.f / c.h, -3.4028235e38f);
    kappa = near ? ex2(fmaf(c.h, m, -M) + c.l * m) : 1.f;
  }
};
// (a whole warp at once: lane i holds 2^(i / 32) in `mine`; not normalised: the second float is up to 2^-14 of the first)
__device__ __forceinline__ Two weight_raw(float x, const RowScale& s, const Two& c, const float2& mine) {
  constexpr float kH = 0.693147182464599609375f, kL = -1.904654299957767e-9f;  // ln 2
  const float d = x - s.base, y = fmaxf(d, s.low);
  const float P = __fmul_rn(c.h, y), p = fmaf(c.l, y, fmaf(c.h, y, -P));
  const float t = fmaf(P, 32.f, s.magic), nf = t - kMagic;
  const int n = __float_as_int(t) - __float_as_int(kMagic);
  const float r = P - fmaf(nf, 0.03125f, s.M), w = r + p;
  const float gh = __fmul_rn(r, kH), gl = fmaf(p, kH, fmaf(r, kL, fmaf(r, kH, -gh)));
  const float q = fmaf(w * w, fmaf(w, fmaf(w, 9.6181291e-3f, 5.5504109e-2f), 0.24022651f), gl);  // ln 2^k / k!
  const float th = __shfl_sync(0xffffffffu, mine.x, n), tl = __shfl_sync(0xffffffffu, mine.y, n);
  const float a = __fmul_rn(th, gh), h = th + a, e = (a - (h - th)) + fmaf(th, gh, -a);
  const float up = d >= s.low ? __int_as_float(((n & ~31) << 18) + (127 << 23)) : 0.f;
  return Two{h * up, (fmaf(th, q, fmaf(tl, gh, tl)) + e) * up};
}
__device__ __forceinline__ Two weight(float x, const RowScale& s, const Two& c, const float2& mine) {
  const Two v = weight_raw(x, s, c, mine);
  return renorm(v.h, v.l);
}

// ---------------------------------------------------------------------------------------------
// the walk: a cluster of CL CTAs per sequence, each with a share of the vocabulary

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// (the two halves apart: a CTA's shared memory may be written from elsewhere once it is known to have begun)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// to the same place in another CTA of the cluster
__device__ __forceinline__ void put_remote(float2* at, uint32_t cta, float2 v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(at)), "r"(cta));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

constexpr int kParts = kWalkWarps * kMaxCluster;
constexpr int kChain = 64;  // values that a lane adds up in one go
// ids whose weight is this near to q Z count as beside the border (twice what the first kernel's sums are off by, or more)
constexpr float kBeside = 0x1p-19f;
struct Walk {
  float2 sums[2][4][kParts];  // the parts' sums, of all CTAs (two passes' in turn)
  float2 scan[kWalkWarps];
  int found, last;
};
// and of every row: its draft's weight (in its parent's scale), draft probability, random number, token, parent; the
// row's statistics; refused drafts' tokens (without draft probabilities), or sums left after each refusal
struct Rows {
  float2 *weight, *sum;
  float *q, *u, *m, *l;
  int *tok, *up, *id, *gone;
  static constexpr int kBytes = 2 * 8 + 8 * 4;
  __device__ __forceinline__ Rows(uint8_t* at, int n) {
    weight = reinterpret_cast<float2*>(at);
    sum = weight + n;
    q = reinterpret_cast<float*>(sum + n);
    u = q + n;
    m = u + n;
    l = m + n;
    tok = reinterpret_cast<int*>(l + n);
    up = tok + n;
    id = up + n;
    gone = id + n;
  }
};
inline int rows_room(int max_tokens) { return (max_tokens + 31) / 32 * 32 + 32; }

// What bounds it: for few sequences latency (bounds, rows, logits 1.7 us; statistics 1.3; weights and fates 0.8; one pass and its
// exchange 3 to 4; the id 1), for many the pass's instructions, some 49 a logit, 67 where a refusal's rest is summed as well.
// A call with rows of 32000 fp32 takes 15 us for one chain of 8, 25 for 64 (59 MB of logits in 10; three passes, 134 instructions a
// logit, took 65), 24 for 16 trees of up to 64 rows in bf16.
template <bool BF16, int CL>
__global__ void __launch_bounds__(kWalkThreads, 1) walk_kernel(const Params p) {
  __shared__ Walk w;
  extern __shared__ __align__(16) uint8_t dyn[];
  const Rows rw(dyn, (p.max_tokens + 31) / 32 * 32 + 32);
  const int b = blockIdx.x / CL, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = CL > 1 ? cluster_rank() : 0;
  const float2 mine = p.table.e[lane];
  int first;
  const int n = rows_of(p, b, first);
  const float c32 = factor_of(p, b);
  const bool greedy = c32 == 0.f, soft = p.probs != nullptr && !greedy;
  Two c{c32, 0.f};
  if (!greedy) {
    const float t = p.temperature ? __ldg(p.temperature + b) : 1.f;
    constexpr float kH = 1.44269502162933349609375f, kL = 1.92596299e-8f;  // log2(e)
    if (t > 1e-37f && t < 1e30f) c = times(Two{kH, kL}, inverse(Two{t, 0.f}));
  }
  const char* const x0 = static_cast<const char*>(p.x);
  auto row_at = [&](int j) -> const void* { return x0 + (first + j) * p.stride * (BF16 ? 2 : 4); };
  // ---- what the walk may need of every row
  for (int j = tid; j < n; j += kWalkThreads) {
    const int up = j == 0 ? -1 : p.parents ? __ldg(p.parents + first + j) : j - 1, t = __ldg(p.tokens + first + j);
    const bool there = up >= 0 && up < j && t >= 0 && t < p.vocab;
    rw.up[j] = up < j ? up : -1;
    rw.tok[j] = t;
    rw.u[j] = __ldg(p.uniforms + first + j);
    rw.weight[j].x = there ? logit<BF16>(row_at(up), t) : -INFINITY;  // (its logit, until the statistics are there)
    rw.q[j] = there && soft ? __ldg(p.probs + (first + up) * p.prob_stride + t) : 1.f;
  }
  int32_t* const path = p.path + (size_t)b * p.max_tokens;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the rows' sums)
  for (int i = tid; i < p.max_tokens && rank == 0; i += kWalkThreads)
    if (i > 0 || n == 0) path[i] = -1;
  if (n == 0) {
    if (rank == 0 && tid == 0) {
      p.count[b] = 0;
      p.next[b] = -1;
    }
    return;  // (the same in the whole cluster)
  }
  if (CL > 1) cluster_arrive();  // (every CTA has begun)
  const float cm = greedy ? 1.f : c32;
  const int width = p.width, group = lane / width;  // (32 / width rows a warp)
  for (int j0 = warp * (32 / width); j0 < n; j0 += kWalkWarps * (32 / width)) {
    const int j = j0 + group, i = lane % width;
    Stat st{-INFINITY, 0.f, 0x7FFFFFFF};
    if (j < n && i < p.splits) {
      const float4 f = __ldcg(p.stats + (size_t)(first + j) * width + i);
      st = Stat{f.x, f.y, __float_as_int(f.z)};
    }
    st = merge_lanes(st, width, cm);
    if (j < n && i == 0) {
      rw.m[j] = st.m;
      rw.l[j] = st.l;
      rw.id[j] = st.id;
    }
  }
  __syncthreads();
  RowScale sc;
  if (!greedy)
    for (int j = tid; j - lane < n; j += kWalkThreads) {
      const int up = j < n ? max(rw.up[j], 0) : 0;
      sc.set(rw.m[up], c);
      const Two v = weight(j < n ? rw.weight[j].x : -INFINITY, sc, c, mine);
      if (j < n) rw.weight[j] = make_float2(v.h, v.l);
    }
  __syncthreads();
  if (CL > 1) cluster_wait();
  if (rank == 0 && tid == 0) path[0] = 0;

  // ---- sums over the vocabulary of what is left at row `node`, in parts: part k of kWalkWarps CL is [k seg, ..)
  constexpr int parts = kWalkWarps * CL, per = (parts + 31) / 32;
  const int seg = (p.vocab + parts - 1) / parts, me = (int)rank * kWalkWarps + warp;
  int node = 0, gone = 0, rounds = 0, pass = 0;
  enum { kNone, kWhole, kRest } summed = kNone;  // what `part` holds: nothing of this row yet, all of it, what is left
  Two part[per] = {};  // of the parts lane per, ..: every warp has them all
  Two z{0.f, 0.f};  // the row's whole sum
  bool exact = false;  // (known)
  auto enter = [&](int j) {
    node = j;
    gone = rounds = 0;
    exact = false;
    summed = kNone;
    if (!greedy) sc.set(rw.m[j], c);
    return fabsf(rw.m[j]) <= 3.4028235e38f && rw.l[j] == rw.l[j];
  };
  auto prob = [&](int i) { return __ldg(p.probs + (first + node) * p.prob_stride + i); };
  auto take_away = [&](Two v, float q) {  // refusals, one after another
    for (int k = 0; k < rounds; ++k) v = less(v, times(two(rw.sum[k]), q));
    return v;
  };
  auto left = [&](int i, bool in) {  // what is left of id i; lanes of a warp together
    Two v = weight(in ? logit<BF16>(row_at(node), i) : -INFINITY, sc, c, mine);
    if (!in) return Two{0.f, 0.f};
    if (soft) return rounds > 0 ? take_away(v, prob(i)) : v;
    for (int k = 0; k < gone; ++k)
      if (rw.gone[k] == i) v = Two{0.f, 0.f};
    return v;
  };
  // sums of this warp's part, one or four, to every CTA; then all parts' are in out[0 ..]
  auto exchange = [&](const Two (&own)[4], int sums) {
    float2(*const out)[kParts] = w.sums[pass & 1];
    if (CL > 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < sums && lane < CL) put_remote(&out[k][me], lane, make_float2(own[k].h, own[k].l));
      cluster_sync();
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < sums && lane == 0) out[k][me] = make_float2(own[k].h, own[k].l);
      __syncthreads();
    }
    ++pass;
  };
  auto total = [&]() {  // of `part`: every warp by itself, all the same
    Two a = part[0];
#pragma unroll
    for (int k = 1; k < per; ++k) a = plus(a, part[k]);
    return sum_lanes(a);
  };
  auto read = [&](const float2* out, int k) { return lane * per + k < parts ? two(out[lane * per + k]) : Two{0.f, 0.f}; };
  const int lo = me * seg, hi = min(p.vocab, lo + seg);
  // what is left, id by id: any number of refusals
  auto sum_rest = [&]() {
    Two s{0.f, 0.f};
    for (int i0 = lo; i0 < hi; i0 += 128) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 32 + lane;
        accumulate(s, left(i, i < hi));
      }
    }
    const float2* const out = w.sums[pass & 1][0];
    exchange({sum_lanes(renorm(s.h, s.l))}, 1);
#pragma unroll
    for (int k = 0; k < per; ++k) part[k] = read(out, k);
    summed = kRest;
    return total();
  };
  // The row's whole sum Z, part by part; with REST also what one refusal leaves: sums A of weights and B of draft
  // probabilities over the ids where w > q Z, which A - B Z are. The first kernel's Z tells which. An id for which it is
  // wrong lies within that Z's own error of the border, and A - B Z is off by q times that error: so the draft probabilities
  // near the border are summed as well, and where they make more than 2^-34 of A of it, `doubt` (the draft model is all but the
  // target; of other rows some one in a thousand). A lane's sums are kept as multiples of a power of two, which add exactly,
  // and remainders, in chains: remainders that are all alike round alike, and are off by n^2 2^-48 of the sum after n of them
  // (64: 2^-36; the 32768 that a lane has of 2^24 ids: 2^-18).
  // (without_gone: refused drafts' tokens count nothing)
  bool doubt = false;
  auto sum_whole = [&](auto with_rest, bool without_gone) {
    constexpr bool REST = decltype(with_rest)::value;
    constexpr int U = REST ? 4 : 8;
    const void* const row = row_at(node);
    const float* const qrow = REST ? p.probs + (first + node) * p.prob_stride : nullptr;
    const float z0 = rw.l[node] * sc.kappa;
    // (a chain's sum is below twice the power of two in `most`: multiples of 2^-22 of that add exactly)
    const float most = fminf(min(seg / 32 + 1, kChain) * 1.03f, z0 * 1.01f);
    const float cut = kMagic * __int_as_float((__float_as_int(most) & 0x7F800000) - (22 << 23));
    Two sz{0.f, 0.f}, sa{0.f, 0.f}, sb{0.f, 0.f};           // a lane's chain
    Two whole{0.f, 0.f}, above_q{0.f, 0.f}, of_q{0.f, 0.f};  // its sums
    float beside = 0.f;  // draft probabilities near the border
    bool some_gone = false;
    if (!REST && without_gone) {
      for (int k = lane; k < gone; k += 32) some_gone |= rw.gone[k] >= lo && rw.gone[k] < hi;
      some_gone = __any_sync(0xffffffffu, some_gone);
    }
    float x[U], q[U];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * 32 + lane;
        x[u] = i < hi ? logit<BF16>(row, i) : -INFINITY;
        if (REST) q[u] = i < hi ? __ldg(qrow + i) : 0.f;
      }
    };
    auto fold = [&]() {
      whole = plus(whole, renorm(sz.h, sz.l));
      sz = Two{0.f, 0.f};
      if (REST) {
        above_q = plus(above_q, renorm(sa.h, sa.l));
        of_q = plus(of_q, renorm(sb.h, sb.l));
        sa = sb = Two{0.f, 0.f};
      }
    };
    fetch(lo);
    for (int i0 = lo; i0 < hi; i0 += 32 * U) {
      float y[U], r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        y[u] = x[u];
        r[u] = REST ? q[u] : 0.f;
      }
      fetch(i0 + 32 * U);
      if (!REST && some_gone)
        for (int k = 0; k < gone; ++k) {
          const int at = rw.gone[k] - i0 - lane;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (at == u * 32) y[u] = -INFINITY;
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Two v = weight_raw(y[u], sc, c, mine);
        const float k = (v.h + cut) - cut, d = (v.h - k) + v.l;
        sz.h += k;
        sz.l += d;
        if (REST) {
          const float bound = r[u] * z0, over = (v.h + v.l) - bound, kq = (r[u] + cut) - cut;
          const bool on = over > 0.f;
          beside += fabsf(over) <= kBeside * bound ? r[u] : 0.f;
          sa.h += on ? k : 0.f;
          sa.l += on ? d : 0.f;
          sb.h += on ? kq : 0.f;
          sb.l += on ? r[u] - kq : 0.f;
        }
      }
      if ((i0 - lo) % (32 * kChain) == 32 * (kChain - U)) fold();
    }
    fold();
    const float2(*const out)[kParts] = w.sums[pass & 1];
    if (REST) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) beside += __shfl_xor_sync(0xffffffffu, beside, o);
      exchange({sum_lanes(whole), sum_lanes(above_q), sum_lanes(of_q), Two{beside, 0.f}}, 4);
    } else {
      exchange({sum_lanes(whole)}, 1);
    }
#pragma unroll
    for (int k = 0; k < per; ++k) part[k] = read(out[0], k);
    Two all = total();
    if (!without_gone || gone == 0) {
      z = all;
      exact = true;
    }
    summed = REST || (without_gone && gone > 0) ? kRest : kWhole;
    float a = 0.f;
    if (REST) {
      beside = 0.f;
#pragma unroll
      for (int k = 0; k < per; ++k) {
        const Two A = read(out[1], k);
        a += A.h;
        beside += read(out[3], k).h;
        part[k] = less(A, times(z, read(out[2], k)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        beside += __shfl_xor_sync(0xffffffffu, beside, o);
      }
      // (the error of the first kernel's Z, and the comparison's roundings)
      const float off = fabsf((z.h - z0) + z.l) + 0x1p-23f * z0;
      doubt = off > 0.5f * kBeside * z0 || beside * off > 0x1p-34f * a;
    }
    return a;  // (of A, where there is a rest)
  };
  auto settle = [&]() {  // the row's whole sum in both floats
    if (!exact) sum_whole(std::false_type(), false);
  };

  // ---- As far as the first kernel's sums leave no doubt, every draft's fate is known at once, supposing that its earlier
  // siblings were refused (with draft probabilities only a first child's is): the first child of every row that is
  // accepted, or left open (1 beside twice its number). Without draft probabilities a token that an earlier sibling has
  // has nothing left.
  int* const chosen = rw.gone;
  auto drawn = [&](int k) { return rw.tok[k] >= 0 && rw.tok[k] < p.vocab; };
  for (int j0 = 0; j0 < n; j0 += kWalkThreads) {
    const int j = j0 + tid, up = j < n ? rw.up[j] : -1;
    bool again = false;
    if (up >= 0 && !soft)
#pragma unroll 4
      for (int k = up + 1; k < j; ++k) again |= rw.up[k] == up && rw.tok[k] == rw.tok[j];
    if (again) rw.weight[j] = make_float2(0.f, 0.f);
    if (j < n) chosen[j] = 0x7FFFFFFF;
  }
  __syncthreads();
  for (int j = tid; j < n; j += kWalkThreads) {
    const int up = rw.up[j];
    if (up < 0 || !drawn(j) || !(fabsf(rw.m[up]) <= 3.4028235e38f) || rw.l[up] != rw.l[up]) continue;
    bool take = rw.tok[j] == rw.id[up], open = false;
    if (!greedy) {
      float before = 0.f;
      bool later = false;
#pragma unroll 4
      for (int k = up + 1; k < j; ++k) {
        const bool sibling = rw.up[k] == up && drawn(k);
        later |= sibling;
        before += sibling ? rw.weight[k].x : 0.f;
      }
      if (soft && later) continue;
      sc.set(rw.m[up], c);
      const float s0 = rw.l[up] * sc.kappa, lhs = rw.u[j] * rw.q[j] * (s0 - before), v = rw.weight[j].x;
      take = lhs < v;
      open = fabsf(lhs - v) <= p.trust * fmaxf(s0 * rw.u[j] * rw.q[j], v);
    }
    if (take || open) atomicMin(&chosen[up], 2 * j + open);
  }
  __syncthreads();
  int taken = 1, node0 = 0;
  for (int k = chosen[0]; k != 0x7FFFFFFF && !(k & 1); k = chosen[node0]) {
    node0 = k >> 1;
    if (rank == 0 && tid == 0) path[taken] = node0;
    ++taken;
  }
  __syncthreads();  // (chosen's room is used again)
  // ---- from there one child at a time
  bool good = enter(node0);
  Two rest{0.f, 0.f};  // without draft probabilities: what refused drafts took of the sum
  for (int j = node0 + 1; good && j < n;) {
    // the next child of node
    int c0 = n;
    for (int k = j & ~31; k < n; k += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, k + lane >= j && k + lane < n && rw.up[k + lane] == node);
      if (m) {
        c0 = k + __ffs(m) - 1;
        break;
      }
    }
    if (c0 >= n) break;
    j = c0 + 1;
    const int t = rw.tok[c0];
    if (t < 0 || t >= p.vocab) continue;
    bool take;
    if (greedy) {
      take = t == rw.id[node];
    } else {
      const float u = rw.u[c0], q = rw.q[c0];
      const Two wd = two(rw.weight[c0]);
      // u q (what is left of the sum) against what is left of the draft's weight (q: 1 without draft probabilities)
      if (rounds == 0) {
        const float s0 = rw.l[node] * sc.kappa, lhs = u * q * (s0 - rest.h);
        take = lhs < wd.h;
        if (fabsf(lhs - wd.h) <= p.trust * fmaxf(s0 * u * q, wd.h)) {
          settle();
          take = above(wd, times(times(minus(z, rest), q), u));
        }
      } else {
        take = above(take_away(wd, q), times(times(two(rw.sum[rounds]), q), u));
      }
      if (!take) {
        __syncthreads();
        if (!soft) {
          if (tid == 0) rw.gone[gone] = t;
          ++gone;
          rest = plus(rest, wd);
          summed = kNone;
          __syncthreads();
        } else {
          Two s{0.f, 0.f};
          bool direct = rounds > 0;
          if (!direct) {
            const float a = sum_whole(std::true_type(), false);
            s = total();
            direct = doubt || s.h < 0x1p-12f * a;  // (p is all but q: which ids have something left is decided one by one)
          } else {
            settle();
          }
          if (tid == 0 && rounds == 0) rw.sum[0] = make_float2(z.h, z.l);
          ++rounds;
          __syncthreads();
          if (direct) s = sum_rest();
          if (!(s.h > 0.f)) {  // nothing would be left: p stays
            --rounds;
            summed = kNone;
          } else if (tid == 0) {
            rw.sum[rounds] = make_float2(s.h, s.l);
          }
          __syncthreads();
        }
      }
    }
    if (take) {
      if (rank == 0 && tid == 0) path[taken] = c0;
      ++taken;
      rest = Two{0.f, 0.f};
      good = enter(c0);
    }
  }
  if (rank == 0 && tid == 0) {
    p.count[b] = taken;
    if (!good) p.next[b] = -1;
    else if (greedy) p.next[b] = rw.id[node];
  }
  if (good && !greedy) {
    // ---- the next token: the first id up to which what is left sums to more than u times all of it
    if (summed == kNone || (summed == kWhole && gone + rounds > 0) || (summed == kRest && gone + rounds == 0)) {
      if (rounds == 0) sum_whole(std::false_type(), true);
      else sum_rest();
    }
    Two all = total();
    if (!soft && gone > 0 && !(all.h > 0.f)) {  // nothing is left: the refusals do not count
      gone = 0;
      all = sum_rest();
    }
    const Two want = times(all, rw.u[0]);
    // the part it lies in, by every warp
    Two own = part[0];
#pragma unroll
    for (int k = 1; k < per; ++k) own = plus(own, part[k]);
    const Two upto = scan_lanes(own);
    const uint32_t past = __ballot_sync(0xffffffffu, above(upto, want));
    const uint32_t some = __ballot_sync(0xffffffffu, own.h > 0.f);
    const int l0 = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
    Two before{0.f, 0.f};
    if (l0 > 0) before = shfl(upto, l0 - 1);
    int target = l0 * per;
    if (per > 1) {
      int at = -1;
      Two run = before, start = before;
#pragma unroll
      for (int k = 0; k < per; ++k) {
        const Two v = shfl(part[k], l0), next = plus(run, v);
        if (v.h > 0.f && at < 0) {
          target = l0 * per + k;
          start = run;
          if (past && above(next, want)) at = target;
        }
        run = next;
      }
      before = start;
    }
    if (target / kWalkWarps == (int)rank) {
      // the id, by the whole CTA: a stretch of its threads at a time
      const int from = target * seg, to = min(p.vocab, from + seg);
      if (tid == 0) {
        w.found = 0x7FFFFFFF;
        w.last = -1;
      }
      for (int i0 = from; i0 < to; i0 += kWalkThreads) {
        const int i = i0 + tid;
        const Two v = left(i, i < to), run = scan_lanes(v);
        __syncthreads();
        if (lane == 31) w.scan[warp] = make_float2(run.h, run.l);
        __syncthreads();
        const Two y = scan_lanes(lane < kWalkWarps ? two(w.scan[lane]) : Two{0.f, 0.f});
        const Two over = shfl(y, warp > 0 ? warp - 1 : 0), base = warp > 0 ? plus(before, over) : before;
        const bool there = v.h > 0.f;
        if (there && above(plus(base, run), want)) atomicMin(&w.found, i);
        if (there) atomicMax(&w.last, i);
        before = plus(before, shfl(y, kWalkWarps - 1));
        __syncthreads();
        if (w.found != 0x7FFFFFFF) break;  // (the same in all threads)
      }
      __syncthreads();
      if (tid == 0) p.next[b] = w.found != 0x7FFFFFFF ? w.found : w.last;
    }
  }
  if (CL > 1) cluster_sync();  // (no CTA leaves while another still writes to it)
}

template <bool BF16>
cudaError_t launch(Params& p, cudaStream_t s) {
  if (p.n_tokens > 0) {
    const unsigned warps = kRowThreads / 32;
    rows_kernel<BF16><<<((unsigned)p.n_tokens * p.splits + warps - 1) / warps, kRowThreads, 0, s>>>(p);
    const cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess) return ce;
  }
  const int sms = op_sms();
  // CTAs a sequence, each with a share of the vocabulary: as many as the SMs hold, 8 only where they leave a third of them
  // (clusters of 8 do not fill every part of the chip). 1, 2, 4, 8, us a call (rows of 32000): one sequence 22.8, 16.7, 13.6, 13.1;
  // 12 25.5, 20.1, 16.9, 16.6; 16 27.5, 20.9, 17.7, 21.1; 36 29.4, 23.2, 20.7, 34.6; 50 33.5, 27.2, 31.1, 46.1; 100 30.7, 33.3, 41.0.
  int cl = 1;
  while (cl < kMaxCluster && (long long)p.batch * cl * (cl == 4 ? 3 : 2) <= sms) cl *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.batch * cl));
  cfg.blockDim = dim3(kWalkThreads);
  cfg.dynamicSmemBytes = rows_room(p.max_tokens) * Rows::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (only behind the rows' kernel, which waits for what came before)
  at[0].val.programmaticStreamSerializationAllowed = p.n_tokens > 0;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cl;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  auto go = [&](void (*k)(const Params)) {
    // (many rows a sequence pass the 48 KB that a kernel has without asking)
    if (cfg.dynamicSmemBytes + sizeof(Walk) > 48 * 1024) {
      const cudaError_t ce = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  rows_room(DEC_MAX_TREE) * Rows::kBytes);
      if (ce != cudaSuccess) return ce;
    }
    return cudaLaunchKernelEx(&cfg, k, p);
  };
  switch (cl) {
    case 1: return go(walk_kernel<BF16, 1>);
    case 2: return go(walk_kernel<BF16, 2>);
    case 4: return go(walk_kernel<BF16, 4>);
    default: return go(walk_kernel<BF16, 8>);
  }
}

// 2^(i / 32) in two floats, from the C library's 64-bit powers.
Table make_table() {
  Table t;
  for (int i = 0; i < 32; ++i) {
    const double v = std::exp2(i / 32.0);
    t.e[i].x = (float)v;
    t.e[i].y = (float)(v - (double)t.e[i].x);
  }
  return t;
}

}  // namespace verify
}  // namespace dec

using namespace dec;

extern "C" int64_t dec_verify_drafts_workspace(int32_t n_tokens) {
  return n_tokens < 0 ? -1 : (int64_t)n_tokens * verify::kMaxParts * (int64_t)sizeof(float4);
}

extern "C" dec_status dec_verify_drafts(const dec_verify_drafts_args* a, void* stream) {
  op_clear();
  if (!a) return op_fail(DEC_ERR_ARG, "verify_drafts: NULL arguments");
  if (a->dtype != DEC_BF16 && a->dtype != DEC_F32) return op_fail(DEC_ERR_ARG, "verify_drafts: unknown dtype");
  if (a->batch < 0 || a->n_tokens < 0 || a->max_tokens < 0 || a->vocab < 1 || a->row_stride < 0 || a->prob_stride < 0)
    return op_fail(DEC_ERR_ARG, "verify_drafts: bad sizes");
  if (a->max_tokens > DEC_MAX_TREE)
    return op_fail(DEC_ERR_UNSUPPORTED, "verify_drafts: more than DEC_MAX_TREE rows a sequence");
  if (a->batch == 0) return DEC_OK;
  if (!a->cu_tokens || !a->count || !a->next_tokens || (a->max_tokens > 0 && !a->path))
    return op_fail(DEC_ERR_ARG, "verify_drafts: cu_tokens, path, count or next_tokens missing");
  if (a->n_tokens > 0 && (!a->logits || !a->tokens || !a->uniforms))
    return op_fail(DEC_ERR_ARG, "verify_drafts: logits, tokens or uniforms missing");
  if (reinterpret_cast<uintptr_t>(a->logits) % (a->dtype == DEC_BF16 ? 2 : 4) || reinterpret_cast<uintptr_t>(a->draft_probs) % 4)
    return op_fail(DEC_ERR_ARG, "verify_drafts: logits and draft_probs must be aligned to their types");
  // (ids, rows' parts and CTAs are counted in 32 bits, up to a step past the last)
  if (a->vocab > (1 << 24) || a->n_tokens > INT_MAX / verify::kMaxParts || a->batch > INT_MAX / verify::kMaxCluster ||
      (long long)a->batch * a->max_tokens > (1LL << 40))
    return op_fail(DEC_ERR_UNSUPPORTED, "verify_drafts: too many rows, ids or sequences");
  if (a->n_tokens > 0 && (!a->workspace || !op_aligned(a->workspace) || a->workspace_bytes < dec_verify_drafts_workspace(a->n_tokens)))
    return op_fail(DEC_ERR_ARG, "verify_drafts: workspace missing, misaligned or too small");
  if (dec_status st = op_on_device(a->count, "verify_drafts: count")) return st;
  static const verify::Table table = verify::make_table();
  verify::Params p;
  p.x = a->logits;
  p.stride = a->row_stride;
  p.probs = a->draft_probs;
  p.prob_stride = a->prob_stride;
  p.vocab = a->vocab;
  p.batch = a->batch;
  p.n_tokens = a->n_tokens;
  p.max_tokens = a->max_tokens;
  p.cu = a->cu_tokens;
  p.tokens = a->tokens;
  p.parents = a->parents;
  p.uniforms = a->uniforms;
  p.temperature = a->temperature;
  p.path = a->path;
  p.count = a->count;
  p.next = a->next_tokens;
  p.stats = static_cast<float4*>(a->workspace);
  p.table = table;
  const int sms = op_sms();
  if (sms < 1) return op_fail(DEC_ERR_CUDA, "verify_drafts: no device");
  // Warps a row: as many as the SMs hold at once, or of many rows enough for some turns, each with at least 32 values a
  // thread. One warp a row, 4, 8, 16, 31, us a call: 8 rows of 32000 25.2, 15.6, 14.0, 13.2, 13.1; 512 rows 40.2, 25.2, 25.2, 27.2,
  // 34.6.
  const int each = a->dtype == DEC_BF16 ? 8 : 4, words = (a->vocab + each - 1) / each;
  const long long room = (long long)sms * verify::kRowWarps, rows = std::max(1, a->n_tokens);
  p.splits = (int)std::max<long long>(1, std::min<long long>({verify::kMaxParts, words / (32 / each * 32),
                                                              rows * 2 <= room ? room / rows : (4 * room + rows - 1) / rows}));
  p.width = 1;
  while (p.width < p.splits) p.width *= 2;
  const long long per = (words + 1 + p.splits - 1) / p.splits, step = 32 * 16 / each;  // (a part's words, and a step's)
  p.trust = verify::trust_of((per + step - 1) / step + 2, a->max_tokens);
  const cudaError_t ce = a->dtype == DEC_BF16 ? verify::launch<true>(p, op_stream(stream)) : verify::launch<false>(p, op_stream(stream));
  return ce == cudaSuccess ? DEC_OK : op_cuda(ce, "verify_drafts");
}
