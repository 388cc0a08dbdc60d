// Log-probabilities of rows of logits (dec_logprobs of dec.h).
//
// One pass over the row, which is read once from memory:
//  - every thread keeps a running maximum m, s = sum 2^t and u = sum 2^t t with t = (x - m) log2(e)
//    of its own elements, so nothing is exchanged while the row streams; joined at the end,
//    lse = M + ln S and the entropy is ln 2 (log2 S - U / S);
//  - the target's rank is counted on the way: elements before the target's id need x >= x_target,
//    which is x > the next smaller number, so both sides are one comparison with their own bound;
//  - the alternatives come from a bound: of 32 groups of threads, each knows its largest element, and
//    the n-th largest of those 32 leaves at least n elements at or above it, for ordinary rows
//    n to 3.5 n. Threads whose maximum reaches the bound look through their elements again (from
//    L2), and the few candidates are ranked against each other.
// What bounds it: at many rows the read of the logits; 8 instructions an element for bf16 stay below
// it. At few rows latency: a row is then shared by a cluster of up to 8 CTAs.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCand = 2048;     // candidates kept; more (long runs of equal logits) take the slow way
constexpr int kMaxCluster = 8;
constexpr float kL2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

// A row as vectors of 16 bytes: vector k holds elements k V - shift .. k V - shift + V - 1, of which
// those outside the row read as -infinity.
template <bool BF16>
struct Row {
  static constexpr int V = BF16 ? 8 : 4;
  const char* at;  // the 16-byte boundary at or below the row's first element
  int shift, vocab, vectors;
  __device__ __forceinline__ Row(const Params& p, int r) {
    const char* first = static_cast<const char*>(p.x) + (long long)r * p.stride * (BF16 ? 2 : 4);
    shift = (int)((reinterpret_cast<uintptr_t>(first) & 15u) / (BF16 ? 2 : 4));
    at = first - shift * (BF16 ? 2 : 4);
    vocab = p.vocab;
    vectors = (int)(((long long)shift + vocab + V - 1) / V);
  }
  __device__ __forceinline__ int base(int k) const { return k * V - shift; }
  __device__ __forceinline__ float one(int i) const {
    const char* q = at + (long long)(i + shift) * (BF16 ? 2 : 4);
    return BF16 ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(q)) : *reinterpret_cast<const float*>(q);
  }
  __device__ __forceinline__ uint4 whole(int k) const { return __ldg(reinterpret_cast<const uint4*>(at) + k); }
  // the first or last vector where the row begins or ends inside it
  __device__ __forceinline__ bool partial(int k) const { return base(k) < 0 || base(k) + V > vocab; }
  __device__ __forceinline__ uint4 edge(int k) const { return edge_of(at, shift, vocab, k); }
  __device__ __noinline__ static uint4 edge_of(const char* at, int shift, int vocab, int k) {
    const int b = k * V - shift;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; i < V; ++i) {
      uint32_t x = BF16 ? 0xFF80u : 0xFF800000u;
      if (b + i >= 0 && b + i < vocab)
        x = BF16 ? reinterpret_cast<const uint16_t*>(at)[(long long)k * V + i]
                 : reinterpret_cast<const uint32_t*>(at)[(long long)k * V + i];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j == (BF16 ? i / 2 : i)) w[j] |= BF16 && (i & 1) ? x << 16 : x;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ static void unpack(const uint4& u, float (&x)[V]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        x[(2 * i) % V] = __uint_as_float(w[i] << 16);
        x[(2 * i + 1) % V] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[i % V] = __uint_as_float(w[i]);
      }
    }
  }
  // the largest of a vector; NaN if one of them is
  __device__ __forceinline__ static float largest(const uint4& u) {
    if (BF16) {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
      const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
      return max_nan(__low2float(m), __high2float(m));
    }
    return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                   max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
};

// A row's sums over some of its elements: maximum, sum of 2^t and of 2^t t, t = (x - m) log2(e).
struct Sums {
  float m, s, u;
  __device__ __forceinline__ void raise(float to) {  // (to > m)
    const float d = fmaxf((m - to) * kL2E, -256.f);
    const float f = m == -INFINITY ? 0.f : ex2(d);
    u = m == -INFINITY ? 0.f : f * fmaf(s, d, u);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Sums o) {
    if (o.m > m) raise(o.m);
    else if (m > o.m) o.raise(m);
    s += o.s;
    u += o.u;
  }
};

struct Shared {
  Sums sums[kMaxCluster * kWarps];
  int rank[kMaxCluster * kWarps], bad[kMaxCluster * kWarps];
  unsigned long long group[kMaxCluster * 32];
  unsigned long long bound;  // of the candidates
  int n;                     // candidates found
  unsigned long long cand[kCand];
  unsigned long long best[kWarps];
};

// CTAS CTAs (a cluster) share a row. Everything joined lies in the first one's shared memory.
template <bool BF16, int CTAS>
__global__ void __launch_bounds__(kThreads, 6) logprobs_kernel(const Params p) {
  constexpr int V = Row<BF16>::V;
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
  Sums a{-INFINITY, 0.f, 0.f};
  int first = INT_MAX, ahead = 0, bad = 0;
  auto take = [&](const uint4& u, int k) {
    float x[V];
    Row<BF16>::unpack(u, x);
    float mx = Row<BF16>::largest(u);
    if (!(mx < INFINITY)) {  // (rare) NaN orders as -infinity
      bad = 1;
      mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] = x[i] != x[i] ? -INFINITY : x[i];
        mx = fmaxf(mx, x[i]);
      }
    }
    const int b = row.base(k);
    if (mx > a.m) {
      a.raise(mx);
      first = b;
    }
    if (first == INT_MAX) first = b;
    if (b + V <= t || b > t) {
      const float th = b > t ? above : from;
#pragma unroll
      for (int i = 0; i < V; ++i) ahead += x[i] > th ? 1 : 0;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) ahead += x[i] > (b + i < t ? from : above) ? 1 : 0;
    }
    const float z = a.m == -INFINITY ? 0.f : a.m * kL2E;
    if (!(fabsf(z) < 1e38f)) {  // (rare: a maximum near the type's lowest or largest value, z overflows)
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = (x[i] - a.m) * kL2E;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = fmaf(x[i], kL2E, -z);
    }
    float s = 0.f, w = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float e = fmaxf(x[i], -256.f);  // (2^-256 is 0, and 0 x -256 no NaN)
      const float y = ex2(e);
      s += y;
      w = fmaf(y, e, w);
    }
    a.s += s;
    a.u += w;
  };
  // whole vectors, then the row's first and last where they are not (threads 0 and 1 of their CTA)
  constexpr int U = 2;  // vectors in flight
  const int w0 = part == 0 && row.partial(0) ? 1 : v0;
  const int w1 = part == CTAS - 1 && row.partial(row.vectors - 1) ? row.vectors - 1 : v1;
  const int ek = tid == 0 && w0 != v0 ? 0 : tid == 1 && w1 != v1 && (row.vectors > 1 || w0 == v0) ? row.vectors - 1 : -1;
  int k = w0 + tid;
  for (; k + (U - 1) * kThreads < w1; k += U * kThreads) {
    uint4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = row.whole(k + i * kThreads);
#pragma unroll
    for (int i = 0; i < U; ++i) take(u[i], k + i * kThreads);
  }
#pragma unroll 1
  for (; k < w1; k += kThreads) take(row.whole(k), k);
  if (ek >= 0) take(row.edge(ek), ek);
  const float mine = a.m;

  // ---- join: the warps' sums, and the largest element of every 8 threads
  unsigned long long gk = first == INT_MAX ? 0ull : key_of(mine, first + V - 1);  // (a bound takes the whole vector)
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) gk = max(gk, __shfl_xor_sync(0xffffffffu, gk, o));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.u = __shfl_xor_sync(0xffffffffu, a.u, o);
    a.join(b);
    ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (CTAS > 1) sync();  // (the first CTA has begun)
  if (lane == 0) {
    home->sums[part * kWarps + warp] = a;
    home->rank[part * kWarps + warp] = ahead;
    home->bad[part * kWarps + warp] = bad;
  }
  if ((lane & 7) == 0) home->group[part * 32 + warp * 4 + (lane >> 3)] = gk;
  if (part == 0 && tid == 0) sh.n = 0;
  sync();
  if (part == 0 && tid < CTAS * 32 && p.top > 0) {
    // the top_n-th largest of the groups' largest: at least top_n elements are at or above it
    const unsigned long long g = sh.group[tid];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < CTAS * 32; ++j) {
      const unsigned long long o = sh.group[j];
      before += o > g || (o == g && j < tid) ? 1 : 0;
    }
    if (before == p.top - 1) sh.bound = g;
  }
  float M = 0.f, ls = 0.f;
  int any = 0;
  if (part == 0) {
    // (every warp of the first CTA: the alternatives need the sum too)
    Sums b = lane < CTAS * kWarps ? sh.sums[lane] : Sums{-INFINITY, 0.f, 0.f};
    int rk = lane < CTAS * kWarps ? sh.rank[lane] : 0;
    any = lane < CTAS * kWarps ? sh.bad[lane] : 0;
    if (CTAS * kWarps > 32) {
      b.join(sh.sums[lane + 32]);
      rk += sh.rank[lane + 32];
      any |= sh.bad[lane + 32];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Sums c;
      c.m = __shfl_xor_sync(0xffffffffu, b.m, o);
      c.s = __shfl_xor_sync(0xffffffffu, b.s, o);
      c.u = __shfl_xor_sync(0xffffffffu, b.u, o);
      b.join(c);
      rk += __shfl_xor_sync(0xffffffffu, rk, o);
      any |= __shfl_xor_sync(0xffffffffu, any, o);
    }
    M = b.m;
    ls = logf(b.s);
    if (tid == 0) {
      const float y = any ? NAN : xt == -INFINITY ? -INFINITY : (xt - M) - ls;
      if (p.logprob) p.logprob[r] = has ? y : NAN;
      if (p.rank) p.rank[r] = !has ? -1 : rk + (lowest ? t : 0);
      if (p.entropy) p.entropy[r] = any ? NAN : M == -INFINITY ? 0.f : kLn2 * (log2f(b.s) - b.u / b.s);
    }
  }
  if (p.top == 0) return;

  // ---- the alternatives
  sync();
  const unsigned long long bound = home->bound;
  if (first != INT_MAX && key_of(mine, 0) >= bound) {
    const float least = bound ? value_of(bound) : -INFINITY;  // (0: fewer groups than alternatives, take all)
    auto pick = [&](const uint4& u, int kk) {
      if (Row<BF16>::largest(u) < least) return;
      float x[V];
      Row<BF16>::unpack(u, x);
      const int b = row.base(kk);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float y = x[j] != x[j] ? -INFINITY : x[j];
        if (!(y >= least) || b + j < 0 || b + j >= p.vocab) continue;
        const unsigned long long key = key_of(y, b + j);
        if (key < bound) continue;
        const int at = atomicAdd(&home->n, 1);
        if (at < kCand) home->cand[at] = key;
      }
    };
    k = w0 + tid;
#pragma unroll 1
    for (; k + (U - 1) * kThreads < w1; k += U * kThreads) {
      uint4 u[U];
#pragma unroll
      for (int i = 0; i < U; ++i) u[i] = row.whole(k + i * kThreads);
#pragma unroll 1
      for (int i = 0; i < U; ++i) pick(i == 0 ? u[0] : u[1], k + i * kThreads);
    }
#pragma unroll 1
    for (; k < w1; k += kThreads) pick(row.whole(k), k);
    if (ek >= 0) pick(row.edge(ek), ek);
  }
  sync();
  if (part != 0) return;
  const int n = sh.n;
  auto put = [&](int at, unsigned long long key) {
    const float y = value_of(key);
    if (p.top_ids) p.top_ids[(long long)r * p.top + at] = id_of(key);
    if (p.top_lp) p.top_lp[(long long)r * p.top + at] = any ? NAN : y == -INFINITY ? -INFINITY : (y - M) - ls;
  };
  if (n <= kThreads) {
    // each candidate's place is the number ahead of it (the order they were found in plays no part)
    if (tid < n) {
      const unsigned long long key = sh.cand[tid];
      int at = 0;
      for (int i = 0; i < n; ++i) at += sh.cand[i] > key ? 1 : 0;
      if (at < p.top) put(at, key);
    }
    return;
  }
  // many candidates (long runs of equal logits): one alternative after another, from the candidates,
  // or from the row where they did not fit
  unsigned long long last = ~0ull;
  for (int i = 0; i < p.top; ++i) {
    unsigned long long best = 0;
    if (n <= kCand) {
      for (int j = tid; j < n; j += kThreads) {
        const unsigned long long key = sh.cand[j];
        if (key < last) best = max(best, key);
      }
    } else {
      for (int j = tid; j < p.vocab; j += kThreads) {
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
    for (int j = 0; j < kWarps; ++j) best = max(best, sh.best[j]);
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
  if (a->vocab > INT_MAX - 64 || a->rows > INT_MAX / lp::kMaxCluster)
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
  // CTAs per row: as many as the SMs have room for, each with at least 16 elements per thread
  const int sms = op_sms();
  int ctas = 1;
  while (ctas < lp::kMaxCluster && (long long)a->rows * ctas * 2 <= sms &&
         a->vocab / (ctas * 2) >= 16 * lp::kThreads)
    ctas *= 2;
  const cudaError_t ce = a->dtype == DEC_BF16 ? lp::launch<true>(p, a->rows, ctas, op_stream(stream))
                                              : lp::launch<false>(p, a->rows, ctas, op_stream(stream));
  return ce == cudaSuccess ? DEC_OK : op_cuda(ce, "logprobs");
}
