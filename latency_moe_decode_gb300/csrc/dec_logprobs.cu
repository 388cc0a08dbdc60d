// Log-probabilities of rows of logits (dec_logprobs of dec.h).
//
// One pass over the row, which is read once from memory:
//  - every thread keeps a reference z, s = sum 2^t and u = sum 2^t t with t = x log2(e) - z of its own
//    elements, so nothing is exchanged while the row streams. z is a multiple of 8 that follows the thread's
//    maximum, set 8 to 16 above what passes it: one fma gives t with one rounding whatever offset the logits
//    have, sums are rescaled by powers of two, and seldom (set to the next multiple instead, that cost one row of 32000
//    0.7 us), and the largest term, which is all there is of a confident row, has t in -16 .. 0. Threads
//    and CTAs are joined at the largest z. With the row's maximum M, ls = lse - M = ln 2 (log2 S - (M log2(e) - z))
//    is at least 0, a log-probability (x - M) - ls at most 0, the entropy ln 2 (log2 S - U / S). Rows whose
//    maximum lies at or beyond +-8192 are summed in a second pass, relative to M itself;
//  - the target's rank is counted on the way: elements before the target's id need x >= x_target,
//    which is x > the next smaller number, so both sides are one comparison with their own bound;
//  - the alternatives come from a bound: of 32 groups of threads, each knows its largest element, and
//    the n-th largest of those 32 leaves at least n elements at or above it, for ordinary rows
//    n to 3.5 n. Threads whose maximum reaches the bound look at its vector again, and through all
//    theirs where their second largest vector reaches it too; the few candidates are ranked against
//    each other.
// What bounds it: at many rows the instructions and the waits between a row's parts. 2048 rows of 32000 bf16
// take 41 us, 3.2 TB/s: 15 instructions a logit, 24 us of full issue slots (they are 66 % full), of which the
// pass is 9 and the rest follows it row by row, between barriers, while the CTA asks for no more of memory. At few rows
// latency (one row of 32000 7 us), and for long ones a CTA's rate: a cluster of up to 8 CTAs then shares a row.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "dec_f32x2.cuh"
#include "dec_ops.h"

namespace cg = cooperative_groups;

namespace dec {
namespace lp {

struct Params {
  const void* x;
  int vocab, top;
  long long stride;
  const int32_t* targets;
  float *logprob, *entropy, *top_lp;
  int32_t *rank, *top_ids;
};

constexpr int kCand = 2560;     // candidates kept; more (long runs of equal logits) take the slow way
constexpr int kItems = 512;     // vectors to look at again
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kL2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kStep = 8.f, kRoom = 1.f;  // references are multiples of kStep, set with room for kRoom kSteps more
constexpr float kFar = 8192.f;    // rows whose maximum reaches this magnitude are summed relative to it
constexpr float kNone = -32768.f; // the reference of no elements

// The order of (logit, id): larger logit first, then lower id, as an unsigned key; -0 is 0.
__device__ __forceinline__ unsigned long long key_of(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((unsigned long long)o << 32) | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float value_of(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int id_of(unsigned long long k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A row as vectors of 32 bytes: vector k holds elements k V - shift .. k V - shift + V - 1, of which
// those outside the row read as -infinity.
struct Vec {
  uint32_t w[8];
};
template <bool BF16>
struct Row {
  static constexpr int V = BF16 ? 16 : 8, E = BF16 ? 2 : 4;
  const char* at;  // the 32-byte boundary at or below the row's first element
  int shift, vocab, vectors;
  __device__ __forceinline__ Row(const Params& p, int r) {
    const char* first = static_cast<const char*>(p.x) + (long long)r * p.stride * E;
    shift = (int)((reinterpret_cast<uintptr_t>(first) & 31u) / E);
    at = first - shift * E;
    vocab = p.vocab;
    vectors = (int)(((long long)shift + vocab + V - 1) / V);
  }
  __device__ __forceinline__ int base(int k) const { return k * V - shift; }
  __device__ __forceinline__ float one(int i) const {
    const char* q = at + ((long long)i + shift) * E;
    return BF16 ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(q)) : *reinterpret_cast<const float*>(q);
  }
  __device__ __forceinline__ Vec whole(int k) const {
    Vec v;
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
        : "l"(at + (long long)k * 32));
    return v;
  }
  // the first or last vector where the row begins or ends inside it
  __device__ __forceinline__ bool partial(int k) const { return base(k) < 0 || base(k) + V > vocab; }
  __device__ __forceinline__ Vec edge(int k) const { return edge_of(at, shift, vocab, k); }
  __device__ __noinline__ static Vec edge_of(const char* at, int shift, int vocab, int k) {
    const int b = k * V - shift;
    Vec v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.w[i] = 0u;
    for (int i = 0; i < V; ++i) {
      uint32_t x = BF16 ? 0xFF80u : 0xFF800000u;
      if (b + i >= 0 && b + i < vocab)
        x = BF16 ? reinterpret_cast<const uint16_t*>(at)[(long long)k * V + i]
                 : reinterpret_cast<const uint32_t*>(at)[(long long)k * V + i];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j == (BF16 ? i / 2 : i)) v.w[j] |= BF16 && (i & 1) ? x << 16 : x;
    }
    return v;
  }
  __device__ __forceinline__ static float element(const Vec& v, int i) {
    if (!BF16) return __uint_as_float(v.w[i % 8]);
    const uint32_t w = v.w[(i / 2) % 8];
    return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
  }
  // every element at least `low` (low within 1.1e4)
  __device__ __forceinline__ static void raise(Vec& v, float low) {
    const __nv_bfloat162 l = __float2bfloat162_rn(low);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (BF16) {
        __nv_bfloat162 h = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&v.w[i]), l);
        v.w[i] = *reinterpret_cast<uint32_t*>(&h);
      } else {
        v.w[i] = __float_as_uint(fmaxf(__uint_as_float(v.w[i]), low));
      }
    }
  }
  __device__ __noinline__ static Vec without_nan(Vec v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (BF16) {
        if ((v.w[i] & 0x7FFFu) > 0x7F80u) v.w[i] = (v.w[i] & 0xFFFF0000u) | 0xFF80u;
        if ((v.w[i] & 0x7FFF0000u) > 0x7F800000u) v.w[i] = (v.w[i] & 0xFFFFu) | 0xFF800000u;
      } else if ((v.w[i] & 0x7FFFFFFFu) > 0x7F800000u) {
        v.w[i] = 0xFF800000u;
      }
    }
    return v;
  }
  // the largest element; NaN if one of them is
  __device__ __forceinline__ static float largest(const Vec& v) {
    if (BF16) {
      __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&v.w[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&v.w[i]));
      return max_nan(__low2float(m), __high2float(m));
    }
    float m = __uint_as_float(v.w[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, __uint_as_float(v.w[i]));
    return m;
  }
};

// A row's sums over some of its elements: reference, sum of 2^t and of 2^t t, t = x log2(e) - z; and their
// maximum.
struct Sums {
  float z, s, u, m;
  __device__ __forceinline__ void raise(float to) {  // (to > z)
    const float d = fmaxf(z - to, -256.f), f = ex2(d);
    u = f * fmaf(s, d, u);
    s *= f;
    z = to;
  }
  __device__ __forceinline__ void add_lanes() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      u += __shfl_xor_sync(0xffffffffu, u, o);
    }
  }
  // the warp's joined sums, in every lane
  __device__ __forceinline__ void join_warp() {
    float to = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (to > z) raise(to);
    add_lanes();
  }
};

struct Shared {
  Sums sums[kMaxCluster * kWarps];
  int rank[kMaxCluster * kWarps], bad[kMaxCluster * kWarps];
  unsigned long long group[kMaxCluster * 32];
  unsigned long long bound;  // of the candidates
  int n, items;              // candidates found; vectors to look at again
  float M, ls;               // the row's maximum, its lse less that; whether it has a NaN or infinity
  int any, far;              // whether it has to be summed relative to M
  unsigned long long cand[kCand];
  unsigned long long best[kWarps];
  int item[kItems];
};

// What is written for a row, by one thread: ls = lse - M.
__device__ __forceinline__ void put_row(const Params& p, int r, bool has, float xt, float M, float ls, float entropy, int any) {
  const float y = any ? NAN : xt == -INFINITY ? -INFINITY : (xt - M) - ls;
  if (p.logprob) p.logprob[r] = has ? y : NAN;
  if (p.entropy) p.entropy[r] = any ? NAN : entropy;
}

// The sums relative to M of a row without NaN or infinity, by the whole CTA; in thread 0 the row's.
template <bool BF16>
__device__ __noinline__ Sums far_sums(const char* first, int vocab, float M, Sums* warps) {
  const int tid = threadIdx.x;
  Sums a{0.f, 0.f, 0.f, M};
#pragma unroll 4
  for (int i = tid; i < vocab; i += kThreads) {
    const float x = BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(first)[i])
                         : reinterpret_cast<const float*>(first)[i];
    const float t = fmaxf((x - M) * kL2E, -256.f), y = ex2(t);
    a.s += y;
    a.u = fmaf(y, t, a.u);
  }
  a.add_lanes();
  if (tid % 32 == 0) warps[tid / 32] = a;
  __syncthreads();
  for (int i = 1; tid == 0 && i < kWarps; ++i) {
    a.s += warps[i].s;
    a.u += warps[i].u;
  }
  return a;
}

// CTAS CTAs (a cluster) share a row. Everything joined lies in the first one's shared memory.
template <bool BF16, int CTAS>
__global__ void __launch_bounds__(kThreads, 5) logprobs_kernel(const Params p) {
  constexpr int V = Row<BF16>::V, T = kThreads, W = kWarps;
  static_assert(CTAS * 32 <= T, "one thread per group of threads");
  __shared__ Shared sh;
  const int r = blockIdx.x / CTAS, part = blockIdx.x % CTAS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Shared* const home = CTAS == 1 ? &sh : cg::this_cluster().map_shared_rank(&sh, 0);
  auto sync = [&]() {
    if (CTAS == 1) __syncthreads();
    else cg::this_cluster().sync();
  };
  const Row<BF16> row(p, r);
  const int v0 = (int)((long long)row.vectors * part / CTAS), v1 = (int)((long long)row.vectors * (part + 1) / CTAS);

  // the target and the bounds its rank counts against
  const int t = p.targets ? __ldg(p.targets + r) : -1;
  const bool has = t >= 0 && t < p.vocab;
  const float xt = has ? row.one(t) : NAN;
  const bool lowest = !(xt > -INFINITY);  // orders with the -infinities: every id before t is ahead of it
  const float above = !has ? INFINITY : lowest ? -INFINITY : xt;
  float from = INFINITY;  // x >= xt as x > from
  if (has && !lowest) {
    const uint32_t b = __float_as_uint(xt + 0.0f), step = BF16 ? 0x10000u : 1u;
    from = __uint_as_float(b == 0 ? 0x80000000u | step : (b & 0x80000000u) ? b + step : b - step);
  }

  // ---- the row
  Sums a{kNone, 0.f, 0.f, -INFINITY};
  float top = -kFar - 256.f, low = 0.f;  // the reference as a logit, and what lies so far below that it counts nothing
  float best = -INFINITY, second = -INFINITY;  // the largest vectors' maxima
  int first = INT_MAX, ahead = 0, bad = 0;     // the largest vector's first element
  __nv_bfloat162 above2 = __float2bfloat162_rn(above), from2 = __float2bfloat162_rn(from);
  __nv_bfloat162 count2 = __float2bfloat162_rn(0.f);  // (whole numbers up to 256 are exact)
  auto take = [&](Vec v, int k) {
    float mx = Row<BF16>::largest(v);
    if (!(mx < INFINITY)) {  // (rare) NaN orders as -infinity
      bad = 1;
      v = Row<BF16>::without_nan(v);
      mx = Row<BF16>::largest(v);
    }
    const int b = row.base(k);
    second = fmaxf(second, fminf(mx, best));
    first = mx > best || first == INT_MAX ? b : first;
    best = fmaxf(best, mx);
    if (has) {
      if (b <= t && t < b + V) {
#pragma unroll
        for (int i = 0; i < V; ++i) ahead += Row<BF16>::element(v, i) > (b + i < t ? from : above) ? 1 : 0;
      } else if (BF16) {
        const __nv_bfloat162 th = b > t ? above2 : from2;
#pragma unroll
        for (int i = 0; i < 8; ++i) count2 = __hadd2(count2, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&v.w[i]), th));
      } else {
        const float th = b > t ? above : from;
#pragma unroll
        for (int i = 0; i < V; ++i) ahead += Row<BF16>::element(v, i) > th ? 1 : 0;
      }
    }
    if (mx > top) {
      a.raise(kStep * ceilf(fmaf(fminf(mx, kFar), kL2E / kStep, kRoom)));
      top = a.z * kLn2;
      low = top - 130.f;
    }
    if (a.z != kNone) {  // (vectors below -8448 alone add nothing to a row with a maximum above -8192)
      Row<BF16>::raise(v, low);  // (2^-180 is 0, and 0 x -180 no NaN)
      const uint64_t l2 = pair(kL2E, kL2E), z2 = pair(-a.z, -a.z);
      uint64_t s = pair(a.s, 0.f), w = pair(a.u, 0.f);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const uint64_t e = fma2(pair(Row<BF16>::element(v, i), Row<BF16>::element(v, i + 1)), l2, z2);
        const float2 f = halves(e);
        const uint64_t y = pair(ex2(f.x), ex2(f.y));
        s = add2(s, y);
        w = fma2(y, e, w);
      }
      const float2 s1 = halves(s), w1_ = halves(w);
      a.s = s1.x + s1.y;
      a.u = w1_.x + w1_.y;
    }
  };
  // whole vectors, then the row's first and last where they are not (threads 0 and 1 of their CTA)
  constexpr int U = 2;  // vectors in flight
  const int w0 = part == 0 && row.partial(0) ? 1 : v0;
  const int w1 = part == CTAS - 1 && row.partial(row.vectors - 1) ? row.vectors - 1 : v1;
  const int ek = tid == 0 && w0 != v0 ? 0 : tid == 1 && w1 != v1 && (row.vectors > 1 || w0 == v0) ? row.vectors - 1 : -1;
  int k = w0 + tid;
  while (k < w1) {
    // (counts in bf16: 8 a vector and half, to 29 vectors)
    for (int i = 0; i < 28 / U && k + (U - 1) * T < w1; ++i, k += U * T) {
      Vec v[U];
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = row.whole(k + j * T);
#pragma unroll
      for (int j = 0; j < U; ++j) take(v[j], k + j * T);
    }
    if (k + (U - 1) * T >= w1 && k < w1) {
      static_assert(U <= 2, "one vector is left at most");
      take(row.whole(k), k);
      k += T;
    }
    if (BF16) {
      ahead += (int)(__low2float(count2) + __high2float(count2));
      count2 = __float2bfloat162_rn(0.f);
    }
  }
  if (ek >= 0) {
    take(row.edge(ek), ek);
    if (BF16) ahead += (int)(__low2float(count2) + __high2float(count2));
  }

  // ---- join: the warps' sums, and the largest element of every T / 32 threads
  unsigned long long gk = first == INT_MAX ? 0ull : key_of(best, first + V - 1);  // (a bound takes the whole vector)
  if (p.top > 0) {
#pragma unroll
    for (int o = 1; o < T / 32; o <<= 1) gk = max(gk, __shfl_xor_sync(0xffffffffu, gk, o));
  }
  a.m = best;
  a.join_warp();
  ahead = __reduce_add_sync(0xffffffffu, ahead);
  bad = __any_sync(0xffffffffu, bad);
  if (CTAS > 1) sync();  // (the first CTA has begun)
  if (lane == 0) {
    home->sums[part * W + warp] = a;
    home->rank[part * W + warp] = ahead;
    home->bad[part * W + warp] = bad;
  }
  if (tid % (T / 32) == 0) home->group[part * 32 + tid / (T / 32)] = gk;
  if (tid == 0) sh.n = sh.items = 0;
  sync();
  if (part == 0 && p.top > 0) {
    // the top_n-th largest of the groups' largest: at least top_n elements are at or above it (8 lanes
    // a group: what follows the row's last element is latency, so it is spread over the threads)
#pragma unroll 1
    for (int i = tid / 8; i < CTAS * 32; i += T / 8) {
      const unsigned long long g = sh.group[i];
      int before = 0;
#pragma unroll 4
      for (int j = tid % 8; j < CTAS * 32; j += 8) {
        const unsigned long long o = sh.group[j];
        before += o > g || (o == g && j < i) ? 1 : 0;
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      if (before == p.top - 1) sh.bound = g;
    }
  }
  if (part == 0 && warp == W - 1) {
    Sums b = lane < CTAS * W ? sh.sums[lane] : Sums{kNone, 0.f, 0.f, -INFINITY};
    int rk = lane < CTAS * W ? sh.rank[lane] : 0;
    int any = lane < CTAS * W ? sh.bad[lane] : 0;
    if (CTAS * W > 32) {
      Sums c = sh.sums[(lane + 32) % (CTAS * W)];
      if (c.z > b.z) b.raise(c.z);
      else if (b.z > c.z) c.raise(b.z);
      b.s += c.s;
      b.u += c.u;
      b.m = fmaxf(b.m, c.m);
      rk += sh.rank[(lane + 32) % (CTAS * W)];
      any |= sh.bad[(lane + 32) % (CTAS * W)];
    }
    b.join_warp();
    rk = __reduce_add_sync(0xffffffffu, rk);
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) {
      const bool none = b.m == -INFINITY, far = !any && !none && !(fabsf(b.m) < kFar);
      // the sum relative to the whole number next to the maximum (a power of two apart: the logarithm and what
      // it is compared with stay near 0 for a confident row)
      const float c = any || none || far ? 0.f : rintf(b.m * kL2E);
      const float s = b.s * ex2(b.z - c);
      const float ls = none ? 0.f : fmaxf(kLn2 * (log2f(s) - fmaf(b.m, kL2E, -c)), 0.f);
      if (p.rank) p.rank[r] = !has ? -1 : rk + (lowest ? t : 0);
      if (!far) put_row(p, r, has, xt, b.m, ls, none ? 0.f : fmaxf(kLn2 * (log2f(b.s) - b.u / b.s), 0.f), any);
      sh.M = b.m;
      sh.ls = ls;
      sh.any = any;
      sh.far = far;
    }
  }
  if (p.top == 0) {
    if (part != 0) return;
    __syncthreads();
  } else {
    sync();
  }
  if (part == 0 && sh.far) {  // (the type's lowest value everywhere, say)
    const Sums b = far_sums<BF16>(row.at + row.shift * Row<BF16>::E, p.vocab, sh.M, sh.sums);
    if (tid == 0) {
      const float l2 = log2f(b.s);
      sh.ls = fmaxf(kLn2 * l2, 0.f);
      put_row(p, r, has, xt, b.m, sh.ls, fmaxf(kLn2 * (l2 - b.u / b.s), 0.f), 0);
    }
    __syncthreads();
  }
  if (p.top == 0) return;

  // ---- the alternatives
  const unsigned long long bound = home->bound;
  const float least = bound ? value_of(bound) : -INFINITY;  // (0: fewer groups than alternatives, take all)
  auto offer = [&](float x, int id) {
    const float y = x != x ? -INFINITY : x;
    // (of the -infinities only ids below top_n can be among the first top_n)
    if (!(y >= least) || id < 0 || id >= p.vocab || (y == -INFINITY && id >= p.top)) return;
    const unsigned long long key = key_of(y, id);
    if (key < bound) return;
    const int at = atomicAdd(&home->n, 1);
    if (at < kCand) home->cand[at] = key;
  };
  // the vectors to look at go to a list that all threads share, a few elements each
  if (first != INT_MAX && key_of(best, 0) >= bound) {
    const bool more = key_of(second, 0) >= bound;
    const int n = more ? (w1 > w0 + tid ? (w1 - w0 - tid + T - 1) / T : 0) + (ek >= 0 ? 1 : 0) : 1;
    int i = atomicAdd(&sh.items, n);
    auto put = [&](int k) {
      if (i < kItems) sh.item[i] = k;
      else  // (more than the list holds)
        for (int j = 0; j < V; ++j)
          if (row.base(k) + j >= 0 && row.base(k) + j < p.vocab) offer(row.one(row.base(k) + j), row.base(k) + j);
      ++i;
    };
    if (!more) {
      put((first + row.shift) / V);
    } else {
      if (ek >= 0) put(ek);
#pragma unroll 1
      for (k = w0 + tid; k < w1; k += T) put(k);
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < min(sh.items, kItems) * 8; i += T) {
    const int id = row.base(sh.item[i / 8]) + i % 8 * (V / 8);
    float x[V / 8];
#pragma unroll
    for (int j = 0; j < V / 8; ++j) x[j] = id + j >= 0 && id + j < p.vocab ? row.one(id + j) : -INFINITY;
#pragma unroll
    for (int j = 0; j < V / 8; ++j) offer(x[j], id + j);
  }
  sync();
  if (part != 0) return;
  const int n = sh.n;
  const float M = sh.M, ls = sh.ls;
  const int any = sh.any;
  auto put = [&](int at, unsigned long long key) {
    const float y = value_of(key);
    if (p.top_ids) p.top_ids[(long long)r * p.top + at] = id_of(key);
    if (p.top_lp) p.top_lp[(long long)r * p.top + at] = any ? NAN : y == -INFINITY ? -INFINITY : (y - M) - ls;
  };
  if (n <= T) {
    // each candidate's place is the number ahead of it (the order they were found in plays no part)
#pragma unroll 1
    for (int i = tid / 8; i < (n + 3 & ~3); i += T / 8) {
      const unsigned long long key = i < n ? sh.cand[i] : 0ull;
      int at = 0;
      for (int j = tid % 8; j < n; j += 8) at += sh.cand[j] > key ? 1 : 0;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) at += __shfl_xor_sync(0xffffffffu, at, o);
      if (tid % 8 == 0 && i < n && at < p.top) put(at, key);
    }
    return;
  }
  // many candidates (long runs of equal logits): one alternative after another, from the candidates,
  // or from the row where they did not fit
  unsigned long long last = ~0ull;
  for (int i = 0; i < p.top; ++i) {
    unsigned long long best = 0;
    if (n <= kCand) {
      for (int j = tid; j < n; j += T) {
        const unsigned long long key = sh.cand[j];
        if (key < last) best = max(best, key);
      }
    } else {
      for (int j = tid; j < p.vocab; j += T) {
        const float y = row.one(j);
        const unsigned long long key = key_of(y != y ? -INFINITY : y, j);
        if (key < last) best = max(best, key);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();
    if (lane == 0) sh.best[warp] = best;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < W; ++j) best = max(best, sh.best[j]);
    if (tid == 0) put(i, best);
    last = best;
  }
}

template <bool BF16>
cudaError_t launch(const Params& p, int rows, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)rows * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  switch (ctas) {
    case 1: return cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, 1>, p);
    case 2: return cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, 2>, p);
    case 4: return cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, 4>, p);
    default: return cudaLaunchKernelEx(&cfg, logprobs_kernel<BF16, 8>, p);
  }
}

}  // namespace lp
}  // namespace dec

using namespace dec;

extern "C" dec_status dec_logprobs(const dec_logprobs_args* a, void* stream) {
  op_clear();
  if (!a) return op_fail(DEC_ERR_ARG, "logprobs: NULL arguments");
  if (a->dtype != DEC_BF16 && a->dtype != DEC_F32) return op_fail(DEC_ERR_ARG, "logprobs: unknown dtype");
  if (a->rows < 0 || a->vocab < 1 || a->row_stride < 0) return op_fail(DEC_ERR_ARG, "logprobs: bad sizes");
  if (a->top_n < 0 || a->top_n > DEC_MAX_TOP || a->top_n > a->vocab)
    return op_fail(DEC_ERR_ARG, "logprobs: top_n must lie within 0 .. DEC_MAX_TOP and the vocabulary");
  if ((a->logprob || a->rank) && !a->targets) return op_fail(DEC_ERR_ARG, "logprobs: logprob and rank need targets");
  if (a->rows == 0) return DEC_OK;
  if (!a->logits) return op_fail(DEC_ERR_ARG, "logprobs: logits are NULL");
  if (reinterpret_cast<uintptr_t>(a->logits) % (a->dtype == DEC_BF16 ? 2 : 4))
    return op_fail(DEC_ERR_ARG, "logprobs: logits are not aligned to their type");
  // (ids are counted in 32 bits, up to four steps of a CTA past the row's end)
  if (a->vocab > INT_MAX - 4 * lp::kThreads || a->rows > INT_MAX / lp::kMaxCluster)
    return op_fail(DEC_ERR_UNSUPPORTED, "logprobs: too many rows or ids");
  if (dec_status st = op_on_device(a->logits, "logprobs: logits")) return st;
  lp::Params p;
  p.x = a->logits;
  p.vocab = a->vocab;
  p.top = (a->top_ids || a->top_logprobs) ? a->top_n : 0;
  p.stride = a->row_stride;
  p.targets = a->targets;
  p.logprob = a->logprob;
  p.entropy = a->entropy;
  p.top_lp = a->top_logprobs;
  p.rank = a->rank;
  p.top_ids = a->top_ids;
  // CTAs per row: as many as the SMs have room for, each with at least 128 elements per thread: a
  // cluster's joins cost what they save on shorter rows. 1, 2, 4, 8 CTAs a row, us: one row of 256000
  // 28.6, 18.3, 12.6, 13.4; 76 rows of 128000 with 1 and 2 18.4, 12.2; one row of 32000 7.2, 7.4, 7.5, 7.5.
  const int sms = op_sms();
  int ctas = 1;
  while (ctas < lp::kMaxCluster && (long long)a->rows * ctas * 2 <= sms &&
         a->vocab / (ctas * 2) >= 128 * lp::kThreads)
    ctas *= 2;
  const cudaError_t ce = a->dtype == DEC_BF16 ? lp::launch<true>(p, a->rows, ctas, op_stream(stream))
                                              : lp::launch<false>(p, a->rows, ctas, op_stream(stream));
  return ce == cudaSuccess ? DEC_OK : op_cuda(ce, "logprobs");
}
