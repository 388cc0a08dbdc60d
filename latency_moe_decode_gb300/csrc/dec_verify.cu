// Verification of drafted tokens against the target's probabilities (dec_verify_drafts of dec.h).
//
// Two kernels. The first reads every row of logits once: its largest logit (and that one's id) and the sum of
// exp((x - max) / temperature) in fp32, which is what acceptance needs. The second walks the trees, a CTA or a
// cluster of CTAs per sequence: the walk itself is arithmetic on a few numbers per draft, all fetched at once; then
// the row that the walk ends at is summed again, for the next token. There a border between two of a
// vocabulary's tokens is met with every draw, and sums that are off by 2^-24 of the whole would pick the neighbour
// of the formula's token once in some thousand draws. So those sums, and the few acceptances that the
// first kernel's sums leave open, are taken in unevaluated pairs of floats (some 36 bits; 64-bit arithmetic runs at a
// hundredth of fp32's rate).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "dec.h"
#include "dec_kvq.cuh"
#include "dec_ops.h"

namespace dec {
namespace verify {

using kvq::Two;
using kvq::renorm;

constexpr int kRowThreads = 256;
constexpr int kWalkThreads = 1024;
constexpr int kMaxSplits = 32;
constexpr int kMaxCluster = 8;
// What the first kernel's sums are trusted to: chains of at most a few hundred additions a thread, each off by 2^-24.
constexpr float kTrust = 0x1p-15f;

struct Table {
  float2 e[32];  // 2^(i / 32) as two floats
};

struct Params {
  const void* x;
  long long stride, prob_stride;
  const float* probs;
  int vocab, batch, n_tokens, max_tokens, splits;
  const int32_t *cu, *tokens, *parents;
  const float *uniforms, *temperature;
  int32_t *path, *count, *next;
  float4* stats;  // [n_tokens][splits]: largest logit, sum, its id (bits), unused
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

// A part of a row: its largest logit, the sum relative to that, the first id of it. A NaN makes m a NaN.
struct Stat {
  float m, l;
  int id;
};
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float c) {
  Stat r;
  const bool second = b.m > a.m || (b.m == a.m && b.id < a.id);
  r.m = a.m != a.m || b.m != b.m ? NAN : second ? b.m : a.m;
  r.id = second ? b.id : a.id;
  r.l = (a.m > -INFINITY ? a.l * ex2((a.m - r.m) * c) : 0.f) + (b.m > -INFINITY ? b.l * ex2((b.m - r.m) * c) : 0.f);
  return r;
}

// ---------------------------------------------------------------------------------------------
// every row once: grid (rows x splits)

template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const Params p) {
  constexpr int E = BF16 ? 8 : 4, U = 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ Stat part[kRowThreads / 32];
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits, tid = threadIdx.x;
  kvq::Seqs s{};
  s.batch = p.batch;
  s.cu = p.cu;
  int j;
  const int b = kvq::seq_of_warp(s, row, j);
  if (b < 0 || j >= p.max_tokens) return;
  const float c = factor_of(p, b);
  const char* const base = static_cast<const char*>(p.x) + row * p.stride * (BF16 ? 2 : 4);
  // 16-byte words from the last boundary before the row; the first and the last may hold values beside it
  const int lead = (int)(reinterpret_cast<uintptr_t>(base) & 15u) / (BF16 ? 2 : 4);
  const uint4* const words = reinterpret_cast<const uint4*>(base - lead * (BF16 ? 2 : 4));
  const int n = (int)(((long long)p.vocab + lead + E - 1) / E), per = (n + p.splits - 1) / p.splits;
  const int lo = split * per, hi = min(n, lo + per);
  Stat a{-INFINITY, 0.f, 0x7FFFFFFF};
  bool nan = false;
  for (int w0 = lo + tid; w0 < hi; w0 += U * kRowThreads) {
    float x[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = w0 + u * kRowThreads;
      if (w < hi && w > 0 && w < n - 1) {
        const uint4 v = __ldcs(words + w);
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < E; ++i)
          x[u][i] = BF16 ? __uint_as_float((i & 1) ? q[i / 2] & 0xFFFF0000u : q[i / 2] << 16) : __uint_as_float(q[i % 4]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const long long at = (long long)w * E + i - lead;
          x[u][i] = w < hi && at >= 0 && at < p.vocab ? logit<BF16>(base, at) : -INFINITY;
        }
      }
    }
    float m = a.m;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        nan |= x[u][i] != x[u][i];
        m = fmaxf(m, x[u][i]);
      }
    if (m > a.m) {
      a.l = a.m > -INFINITY ? a.l * ex2((a.m - m) * c) : 0.f;
      a.m = m;
#pragma unroll
      for (int u = U - 1; u >= 0; --u)
#pragma unroll
        for (int i = E - 1; i >= 0; --i)
          if (x[u][i] == m) a.id = (w0 + u * kRowThreads) * E + i - lead;
    }
    if (m > -INFINITY) {
      float l = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) l += x[u][i] > -INFINITY ? ex2((x[u][i] - m) * c) : 0.f;
      a.l += l;
    }
  }
  if (nan) a.m = NAN;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat y{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.l, o), __shfl_xor_sync(0xffffffffu, a.id, o)};
    a = (tid & o) ? merge(y, a, c) : merge(a, y, c);
  }
  if ((tid & 31) == 0) part[tid >> 5] = a;
  __syncthreads();
  if (tid < 32) {
    a = tid < kRowThreads / 32 ? part[tid] : Stat{-INFINITY, 0.f, 0x7FFFFFFF};
#pragma unroll
    for (int o = kRowThreads / 64; o > 0; o >>= 1) {
      const Stat y{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.l, o), __shfl_xor_sync(0xffffffffu, a.id, o)};
      a = (tid & o) ? merge(y, a, c) : merge(a, y, c);
    }
    if (tid == 0) p.stats[(size_t)row * p.splits + split] = make_float4(a.m, a.l, __int_as_float(a.id), 0.f);
  }
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
__device__ __forceinline__ Two times(const Two& a, const Two& b) {
  const float h = a.h * b.h;
  return renorm(h, fmaf(a.h, b.h, -h) + fmaf(a.h, b.l, a.l * b.h));
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

// exp((x - m) / temperature), x <= m, c = log2(e) / temperature; the whole warp at once (lane i holds 2^(i / 32)).
// With y = c (x - m) = n / 32 + f, |f| <= 1/64: 2^y = 2^(n / 32) e^(f ln 2), the second factor by its series to the
// fifth power (a term of 2^-45 left out), whose first term alone needs both floats.
__device__ __forceinline__ Two weight(float x, float m, const Two& c, const float2& mine) {
  const Two d = two_sum(x, -m);
  const float yh = d.h * c.h, yl = fmaf(d.h, c.h, -yh) + fmaf(d.h, c.l, d.l * c.h);
  const bool none = !(yh > -120.f);  // (NaN: infinity times 0)
  const float n = rintf((none ? 0.f : yh) * 32.f), r = (none ? 0.f : yh) - n * 0.03125f;
  constexpr float kH = 0.693147182464599609375f, kL = -1.904654299957767e-9f;  // ln 2
  const float gh = r * kH, gl = fmaf(r, kH, -gh) + fmaf(r, kL, (none ? 0.f : yl) * kH);
  const float s = fmaf(gh * gh, fmaf(gh, fmaf(gh, fmaf(gh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f), gl);
  const int k = (int)n;
  const float th = __shfl_sync(0xffffffffu, mine.x, k & 31), tl = __shfl_sync(0xffffffffu, mine.y, k & 31);
  const float a = th * gh, ae = fmaf(th, gh, -a), h = th + a, e = a - (h - th);
  const float l = e + ae + fmaf(th, s, tl);
  const float up = __int_as_float((127 + (k >> 5)) << 23);
  if (x == m) return Two{1.f, 0.f};
  if (none || !(x > -INFINITY)) return Two{0.f, 0.f};
  const Two w = renorm(h, l);
  return Two{w.h * up, w.l * up};
}

// ---------------------------------------------------------------------------------------------
// the walk: a cluster of CL CTAs per sequence, each with a share of the vocabulary

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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

struct Walk {
  float xd[DEC_MAX_TREE], qd[DEC_MAX_TREE], u[DEC_MAX_TREE];  // a draft's logit, draft probability, random number
  int tok[DEC_MAX_TREE], up[DEC_MAX_TREE];
  int gone[DEC_MAX_TREE];   // refused drafts' tokens (without draft probabilities)
  float2 scale[DEC_MAX_TREE + 1];  // with them: what p is multiplied by before each subtraction
  float2 sums[2][32 * kMaxCluster];  // the warps' sums, of all CTAs (two passes' in turn)
  float2 scan[32];
  int found, last;
};

template <bool BF16, int CL>
__global__ void __launch_bounds__(kWalkThreads, 1) walk_kernel(const Params p) {
  __shared__ Walk w;
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
    // log2(e) / t: the quotient and its remainder
    constexpr float kH = 1.44269502162933349609375f, kL = 1.92596299e-8f;
    if (t > 1e-30f && t < 1e30f) c = times(Two{kH, kL}, inverse(Two{t, 0.f}));
  }
  const char* const x0 = static_cast<const char*>(p.x);
  auto row_at = [&](int j) -> const void* { return x0 + (first + j) * p.stride * (BF16 ? 2 : 4); };
  // ---- what the walk may need of every draft
  if (tid < n) {
    const int up = tid == 0 ? -1 : p.parents ? __ldg(p.parents + first + tid) : tid - 1, t = __ldg(p.tokens + first + tid);
    const bool there = up >= 0 && up < tid && t >= 0 && t < p.vocab;
    w.up[tid] = up < tid ? up : -1;
    w.tok[tid] = t;
    w.u[tid] = __ldg(p.uniforms + first + tid);
    w.xd[tid] = there ? logit<BF16>(row_at(up), t) : -INFINITY;
    w.qd[tid] = there && soft ? __ldg(p.probs + (first + up) * p.prob_stride + t) : 1.f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the rows' sums)
  __syncthreads();
  int32_t* const path = p.path + (size_t)b * p.max_tokens;
  for (int i = tid; i < p.max_tokens && rank == 0; i += kWalkThreads)
    if (i > 0 || n == 0) path[i] = -1;
  __syncthreads();
  if (n == 0) {
    if (rank == 0 && tid == 0) {
      p.count[b] = 0;
      p.next[b] = -1;
    }
    return;  // (the same in the whole cluster)
  }
  if (rank == 0 && tid == 0) path[0] = 0;

  // ---- a row's statistics, by every warp
  Stat st;
  auto stats = [&](int j) {
    const float4 f = lane < p.splits ? __ldcg(p.stats + (size_t)(first + j) * p.splits + lane) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    st = Stat{f.x, f.y, lane < p.splits ? __float_as_int(f.z) : 0x7FFFFFFF};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Stat y{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.l, o), __shfl_xor_sync(0xffffffffu, st.id, o)};
      st = (lane & o) ? merge(y, st, c32) : merge(st, y, c32);
    }
  };

  // ---- sums over the vocabulary of what is left of p at row `node`, in exact parts: part s of 32 CL is [s seg, ..)
  const int parts = 32 * CL, seg = (p.vocab + parts - 1) / parts, me = (int)rank * 32 + warp;
  int node = 0, gone = 0, rounds = 0, pass = 0;
  Two z{1.f, 0.f};  // the row's whole sum, and its inverse, once they are known in both floats
  Two iz{1.f, 0.f};
  bool exact = false;
  auto left = [&](int i, bool in, bool whole) {  // what is left of id i; lanes of a warp together
    const float x = in ? logit<BF16>(row_at(node), i) : -INFINITY;
    Two v = weight(x, st.m, c, mine);
    if (whole) return v;
    if (!soft) {
      for (int k = 0; k < gone; ++k)
        if (w.gone[k] == i) v = Two{0.f, 0.f};
      return v;
    }
    v = times(v, iz);
    if (rounds > 0) {
      const float q = in ? __ldg(p.probs + (first + node) * p.prob_stride + i) : 0.f;
      for (int k = 0; k < rounds; ++k) {
        const float2 f = w.scale[k];
        v = times(v, Two{f.x, f.y});
        const Two d = two_sum(v.h, -q);
        v = renorm(d.h, d.l + v.l);
        if (!(v.h > 0.f)) v = Two{0.f, 0.f};
      }
    }
    return v;
  };
  auto total = [&](bool whole) {  // every part's sum into w.sums[pass & 1], and all of them
    Two s{0.f, 0.f};
    const int lo = me * seg, hi = min(p.vocab, lo + seg);
    for (int i0 = lo; i0 < hi; i0 += 128) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 32 + lane;
        accumulate(s, left(i, i < hi, whole));
      }
    }
    s = renorm(s.h, s.l);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s = plus(s, Two{__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.l, o)});
    float2* const out = w.sums[pass & 1];
    if (CL > 1) {
      if (lane < CL) put_remote(out + me, lane, make_float2(s.h, s.l));
      cluster_sync();
    } else {
      if (lane == 0) out[me] = make_float2(s.h, s.l);
      __syncthreads();
    }
    Two a{0.f, 0.f};
    for (int k = lane; k < parts; k += 32) a = plus(a, Two{out[k].x, out[k].y});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = plus(a, Two{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)});
    ++pass;
    return a;
  };
  auto settle = [&]() {  // the row's whole sum in both floats
    if (exact) return;
    z = total(true);
    iz = inverse(z);
    exact = true;
  };

  stats(0);
  int taken = 1;
  bool good = fabsf(st.m) <= 3.4028235e38f;
  Two rest{0.f, 0.f};  // without draft probabilities: what refused drafts took of the sum
  for (int j = 1; good && j < n;) {
    // the next child of node
    int c0 = n;
    for (int k = j & ~31; k < n; k += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, k + lane >= j && k + lane < n && w.up[k + lane] == node);
      if (m) {
        c0 = k + __ffs(m) - 1;
        break;
      }
    }
    if (c0 >= n) break;
    j = c0 + 1;
    const int t = w.tok[c0];
    if (t < 0 || t >= p.vocab) continue;
    bool take;
    if (greedy) {
      take = t == st.id;
    } else {
      const float u = w.u[c0];
      bool spent = false;  // (a token that was refused already has nothing left)
      if (!soft)
        for (int k = lane; k < gone; k += 32) spent |= w.gone[k] == t;
      spent = __any_sync(0xffffffffu, spent);
      const Two wd = spent ? Two{0.f, 0.f} : weight(w.xd[c0], st.m, c, mine);
      if (rounds == 0) {
        // u q (sum - refused) against the draft's weight (q: 1 without draft probabilities)
        const float lhs = u * w.qd[c0] * (soft ? st.l : st.l - rest.h);
        take = lhs < wd.h;
        if (fabsf(lhs - wd.h) <= kTrust * fmaxf(st.l * u * w.qd[c0], wd.h)) {
          settle();
          const Two r = soft ? z : plus(z, Two{-rest.h, -rest.l});
          take = above(wd, times(times(r, Two{w.qd[c0], 0.f}), Two{u, 0.f}));
        }
      } else {
        Two v = times(wd, iz);
        for (int k = 0; k < rounds; ++k) {
          const float2 f = w.scale[k];
          v = times(v, Two{f.x, f.y});
          const Two d = two_sum(v.h, -w.qd[c0]);
          v = renorm(d.h, d.l + v.l);
          if (!(v.h > 0.f)) v = Two{0.f, 0.f};
        }
        const float2 f = w.scale[rounds];  // (the draft's share of what is left, over all of it)
        take = above(times(v, Two{f.x, f.y}), times(Two{w.qd[c0], 0.f}, Two{u, 0.f}));
      }
      if (!take) {
        if (!soft) {
          __syncthreads();
          if (tid == 0) w.gone[gone] = t;
          ++gone;
          rest = plus(rest, wd);
          __syncthreads();
        } else {
          settle();
          __syncthreads();
          if (tid == 0 && rounds == 0) w.scale[0] = make_float2(1.f, 0.f);
          ++rounds;
          __syncthreads();
          const Two s = total(false);
          const Two f = inverse(s);
          if (!(s.h > 0.f)) --rounds;  // nothing would be left: p stays
          else if (tid == 0) w.scale[rounds] = make_float2(f.h, f.l);
          __syncthreads();
        }
      }
    }
    if (take) {
      node = c0;
      if (rank == 0 && tid == 0) path[taken] = c0;
      ++taken;
      gone = rounds = 0;
      rest = Two{0.f, 0.f};
      exact = false;
      iz = Two{1.f, 0.f};
      stats(node);
      good = fabsf(st.m) <= 3.4028235e38f;
    }
  }
  if (rank == 0 && tid == 0) {
    p.count[b] = taken;
    if (!good) p.next[b] = -1;
    else if (greedy) p.next[b] = st.id;
  }
  if (good && !greedy) {
    // ---- the next token: the first id up to which the sum passes u times all of it
    if (soft && rounds > 0) settle();
    Two all = total(false);
    if (!soft && gone > 0 && !(all.h > 0.f)) {  // nothing is left: the refusals do not count
      gone = 0;
      all = total(false);
    }
    const float2* const sums = w.sums[(pass - 1) & 1];
    const Two want = times(all, Two{w.u[0], 0.f});
    // the part it lies in (by every warp): CL parts a lane, in order
    Two own{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < CL; ++k) own = plus(own, Two{sums[lane * CL + k].x, sums[lane * CL + k].y});
    Two upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Two y{__shfl_up_sync(0xffffffffu, upto.h, o), __shfl_up_sync(0xffffffffu, upto.l, o)};
      if (lane >= o) upto = plus(y, upto);
    }
    const uint32_t past = __ballot_sync(0xffffffffu, above(upto, want));
    const uint32_t some = __ballot_sync(0xffffffffu, own.h > 0.f);
    const int l0 = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
    Two before{0.f, 0.f};
    if (l0 > 0) before = shfl(upto, l0 - 1);
    int target = l0 * CL;
    if (CL > 1) {
      int at = -1, full = l0 * CL;
      Two run = before, start = before;
      for (int k = 0; k < CL; ++k) {
        const Two v{sums[l0 * CL + k].x, sums[l0 * CL + k].y};
        const Two next = plus(run, v);
        if (v.h > 0.f && at < 0) {
          full = l0 * CL + k;
          start = run;
          if (past && above(next, want)) at = full;
        }
        run = next;
      }
      target = at < 0 ? full : at;
      before = start;
    }
    if (target / 32 == (int)rank) {
      // the id, by the whole CTA: a stretch of 1024 at a time
      const int lo = target * seg, hi = min(p.vocab, lo + seg);
      if (tid == 0) {
        w.found = 0x7FFFFFFF;
        w.last = -1;
      }
      for (int i0 = lo; i0 < hi; i0 += kWalkThreads) {
        const int i = i0 + tid;
        const Two v = left(i, i < hi, false);
        Two run = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const Two y{__shfl_up_sync(0xffffffffu, run.h, o), __shfl_up_sync(0xffffffffu, run.l, o)};
          if (lane >= o) run = plus(y, run);
        }
        __syncthreads();
        if (lane == 31) w.scan[warp] = make_float2(run.h, run.l);
        __syncthreads();
        Two y{w.scan[lane].x, w.scan[lane].y};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const Two a{__shfl_up_sync(0xffffffffu, y.h, o), __shfl_up_sync(0xffffffffu, y.l, o)};
          if (lane >= o) y = plus(a, y);
        }
        Two base = before;
        const Two over = shfl(y, warp > 0 ? warp - 1 : 0);
        if (warp > 0) base = plus(base, over);
        const bool some_here = v.h > 0.f;
        if (some_here && above(plus(base, run), want)) atomicMin(&w.found, i);
        if (some_here) atomicMax(&w.last, i);
        before = plus(before, shfl(y, 31));
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
    rows_kernel<BF16><<<(unsigned)(p.n_tokens * p.splits), kRowThreads, 0, s>>>(p);
    const cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess) return ce;
  }
  const int sms = op_sms();
  const int cl = (long long)p.batch * 8 <= sms ? 8 : (long long)p.batch * 2 <= sms ? 2 : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.batch * cl));
  cfg.blockDim = dim3(kWalkThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (only behind the rows' kernel, which waits for what came before)
  at[0].val.programmaticStreamSerializationAllowed = p.n_tokens > 0;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cl;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  switch (cl) {
    case 1: return cudaLaunchKernelEx(&cfg, walk_kernel<BF16, 1>, p);
    case 2: return cudaLaunchKernelEx(&cfg, walk_kernel<BF16, 2>, p);
    default: return cudaLaunchKernelEx(&cfg, walk_kernel<BF16, 8>, p);
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
  return n_tokens < 0 ? -1 : (int64_t)n_tokens * verify::kMaxSplits * (int64_t)sizeof(float4);
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
  // (what kTrust says of the rows' sums holds up to here)
  if (a->vocab > (1 << 24) || a->n_tokens > INT_MAX / verify::kMaxSplits || a->batch > INT_MAX / verify::kMaxCluster ||
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
  // CTAs a row: enough to fill the SMs, each with at least 8 words of 16 bytes a thread
  p.splits = 1;
  while (p.splits < verify::kMaxSplits && (long long)a->n_tokens * p.splits < 4 * sms &&
         a->vocab / (p.splits * 2) >= 32 * verify::kRowThreads)
    p.splits *= 2;
  const cudaError_t ce = a->dtype == DEC_BF16 ? verify::launch<true>(p, op_stream(stream)) : verify::launch<false>(p, op_stream(stream));
  return ce == cudaSuccess ? DEC_OK : op_cuda(ce, "verify_drafts");
}
