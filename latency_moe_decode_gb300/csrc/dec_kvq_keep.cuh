// What trees of drafted tokens and bounded caches need beside the attention: a tree's masks, the choice of the
// positions that stay, and moving positions as they are held.
#pragma once
#include "dec_kvq_attn.cuh"

namespace dec {
namespace kvq {

// ---------------------------------------------------------------------------------------------
// trees

struct TreeParams {
  const int32_t *cu, *parents, *lengths;
  int batch, n_tokens, max_tokens, words;
  uint32_t* mask;
  long long mask_stride;
  int32_t* positions;
};

// One CTA per sequence, one thread per row: up the parents, a word of the mask at a time (a row's ancestors are
// met in descending order). The walk is a chain of shared memory reads, 30 cycles a step: 32 trees of up to 64 rows take
// 4 us, one of 16 2.5.
__global__ void __launch_bounds__(DEC_MAX_TREE) draft_tree_kernel(const TreeParams p) {
  __shared__ int up[DEC_MAX_TREE];
  const int b = blockIdx.x, j = threadIdx.x;
  const int first = max(0, __ldg(p.cu + b)), last = min(__ldg(p.cu + b + 1), p.n_tokens);
  const int n = min(last - first, p.max_tokens);
  if (j < n) {
    const int a = __ldg(p.parents + first + j);
    up[j] = a < j ? a : -1;  // (negative: a path begins)
  }
  __syncthreads();
  if (j >= n) return;
  uint32_t* const row = p.mask + (first + j) * p.mask_stride;
  int at = j, k = p.words - 1, depth = -1;
  uint32_t w = 0;
  while (at >= 0) {
    for (; k > at >> 5; --k, w = 0) row[k] = w;
    w |= 1u << (at & 31);
    ++depth;
    at = up[at];
  }
  for (; k >= 0; --k, w = 0) row[k] = w;
  if (p.positions) p.positions[first + j] = (p.lengths ? __ldg(p.lengths + b) : 0) + depth;
}

// ---------------------------------------------------------------------------------------------
// the heaviest positions

struct KeepParams {
  Cache c;
  Seqs s;
  const float* mass;
  int budget, sinks, recent, cached;  // cached: positions whose keys fit into shared memory
  int32_t *kept, *count;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// (the two halves apart: a CTA's shared memory may be written or read from elsewhere once it is known to have begun)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote(const void* at, uint32_t cta) {  // the same place in another CTA of the cluster
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(cta));
  return a;
}
// Pairs there (of a type that lies on 8 bytes, as the accesses ask for).
__device__ __forceinline__ uint2 get_remote(const uint2* at, uint32_t cta) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(remote(at, cta)) : "memory");
  return v;
}
__device__ __forceinline__ void put_remote(uint2* at, uint32_t cta, uint2 v) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(remote(at, cta)), "r"(v.x), "r"(v.y) : "memory");
}

// A cluster of CL CTAs per (sequence, KV head), each with a stretch of the positions: the need-th largest weight by
// its digits (11, 11 and 10 bits of a key that orders as the weights do; histograms are joined by every CTA), then
// the positions in order: each warp counts, and writes, its own stretch. What bounds it is the chain of these steps,
// each between two barriers: 8 lists of 32 k positions take 13 us (loads 2.4; a digit 3.6, of which 2 read the others'
// histograms; the order 3), in one CTA a list 35.
constexpr int kKeepThreads = 1024;
constexpr int kKeepCached = 40 * 1024;  // keys that a CTA keeps in shared memory
template <int CL>
__global__ void __launch_bounds__(kKeepThreads, 1) heaviest_kernel(const KeepParams p) {
  constexpr int T = kKeepThreads, BINS = 2048;
  extern __shared__ uint32_t cache[];
  __shared__ uint2 bins[3][BINS / 2];  // (two bins each)
  __shared__ uint32_t part[32];
  __shared__ uint32_t sh_bin, sh_left, sh_all;
  __shared__ uint2 counts[32], sums[CL];
  const uint32_t rank = CL > 1 ? cluster_rank() : 0;
  const int list = blockIdx.x / CL, b = list / p.c.hkv, h = list - b * p.c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto hist = [&](int d) { return reinterpret_cast<uint32_t*>(bins[d]); };
  auto sync_all = [&]() {
    if (CL > 1) cluster_sync();
    else __syncthreads();
  };
  int len = __ldg(p.s.lengths + b);
  const bool bad = len < 0 || len > (long long)p.s.max_pages << p.c.page_shift;
  if (bad) {
    if (tid == 0) raise(p.c.status, len < 0 ? DEC_ERR_ARG : DEC_ERR_CAPACITY);
    len = 0;
  }
  int32_t* const kept = p.kept + (size_t)list * p.budget;
  if (h == 0 && tid == 0 && rank == 0) p.count[b] = min(len, p.budget);
  if (len <= p.budget) {  // (the same in the whole cluster)
    for (int i = rank * T + tid; i < p.budget; i += CL * T) kept[i] = i < len ? i : -1;
    return;
  }
  if (CL > 1) cluster_arrive();  // (every CTA has begun)
  const int32_t* const table = p.s.table + b * p.s.table_stride;
  auto load = [&](int pos) -> uint32_t {
    const int page = __ldg(table + (pos >> p.c.page_shift));
    if ((unsigned)page >= (unsigned)p.c.n_pages) {
      raise(p.c.status, DEC_ERR_ARG);
      return 0u;
    }
    const float x = __ldg(p.mass + ((((size_t)page * p.c.hkv + h) << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1)))) + 0.f;
    const uint32_t u = __float_as_uint(x);
    return x != x ? 0u : (u >> 31) ? ~u : u | 0x80000000u;
  };
  // this CTA's stretch, its candidates (sinks .. len - recent - 1) and their keys
  const int share = ((len + CL - 1) / CL + 31) / 32 * 32, from = min(len, (int)rank * share), to = min(len, from + share);
  const int c0 = max(from, p.sinks), c1 = min(to, len - p.recent);
  auto key_of = [&](int pos) { return pos - from < p.cached ? cache[pos - from] : load(pos); };
#pragma unroll 4
  for (int pos = c0 + tid; pos < min(c1, from + p.cached); pos += T) cache[pos - from] = load(pos);
  for (int i = tid; i < 3 * BINS; i += T) hist(0)[i] = 0;
  __syncthreads();
  if (CL > 1) cluster_wait();
  // ---- threshold and how many of its equals belong
  uint32_t need = (uint32_t)(p.budget - p.sinks - p.recent), prefix = 0;
  const bool any = need > 0;
  bool whole = false;  // (all of the last digit's keys belong: no further digit is needed, as a rule after two)
  for (int d = 0; any && !whole && d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
    for (int pos = c0 + tid; pos < c1; pos += T) {
      const uint32_t k = key_of(pos);
      if (d == 0 || k >> (shift + bits) == prefix) atomicAdd(hist(d) + ((k >> shift) & ((1u << bits) - 1u)), 1u);
    }
    sync_all();
    // from the top: thread i has bins BINS - 1 - 2i and the one below
    uint32_t n0 = 0, n1 = 0;
    const uint2* const at = &bins[d][BINS / 2 - 1 - tid];
    if (CL == 1) {
      n1 = at->x;
      n0 = at->y;
    } else {
      uint2 two[CL];
#pragma unroll
      for (int i = 0; i < CL; ++i) two[i] = get_remote(at, i);
#pragma unroll
      for (int i = 0; i < CL; ++i) {
        n1 += two[i].x;
        n0 += two[i].y;
      }
    }
    uint32_t x = n0 + n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    uint32_t y = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    const uint32_t before = x - n0 - n1 + (warp > 0 ? __shfl_sync(0xffffffffu, y, warp - 1) : 0u);
    if (before < need && need <= before + n0 + n1) {
      const bool first = need <= before + n0;
      sh_bin = BINS - 1 - 2 * tid - (first ? 0 : 1);
      sh_left = need - before - (first ? 0u : n0);
      sh_all = first ? n0 : n1;
    }
    __syncthreads();
    prefix = prefix << bits | sh_bin;
    need = sh_left;
    whole = need == sh_all;
    if (whole) prefix <<= shift;  // (the least of them)
  }
  // ---- in order
  const int seg = ((to - from + 31) / 32 + 31) / 32 * 32;
  const int lo = min(to, from + warp * seg), hi = min(to, lo + seg);
  auto classes = [&](int pos, bool& in, bool& tie) {
    const bool mid = pos >= c0 && pos < c1;
    const uint32_t k = any && mid && pos < hi ? key_of(pos) : 0u;
    in = pos < hi && (!mid || (any && (whole ? k >= prefix : k > prefix)));
    tie = any && !whole && mid && pos < hi && k == prefix;
  };
  uint32_t ins = 0, ties = 0;
  for (int pos = lo + lane; pos - lane < hi; pos += 32) {
    bool in, tie;
    classes(pos, in, tie);
    ins += in;
    ties += tie;
  }
  ins = __reduce_add_sync(0xffffffffu, ins);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) counts[warp] = make_uint2(ins, ties);
  __syncthreads();
  // what lies before this warp's stretch
  const uint2 mine = counts[lane];
  ins = __reduce_add_sync(0xffffffffu, lane < warp ? mine.x : 0u);
  ties = __reduce_add_sync(0xffffffffu, lane < warp ? mine.y : 0u);
  if (CL > 1) {
    const uint32_t all_in = __reduce_add_sync(0xffffffffu, mine.x), all_ties = __reduce_add_sync(0xffffffffu, mine.y);
    if (warp == 0 && lane < CL) put_remote(&sums[rank], lane, make_uint2(all_in, all_ties));
    cluster_sync();
#pragma unroll
    for (int i = 0; i < CL; ++i)
      if (i < (int)rank) {
        ins += sums[i].x;
        ties += sums[i].y;
      }
  }
  for (int pos = lo + lane; pos - lane < hi; pos += 32) {
    bool in, tie;
    classes(pos, in, tie);
    const uint32_t bi = __ballot_sync(0xffffffffu, in), bt = __ballot_sync(0xffffffffu, tie), under = (1u << lane) - 1u;
    const uint32_t at = ties + __popc(bt & under);
    if (in || (tie && at < need)) kept[ins + __popc(bi & under) + min(at, need)] = pos;
    ins += __popc(bi);
    ties += __popc(bt);
  }
}

// ---------------------------------------------------------------------------------------------
// moving positions

struct MoveParams {
  Cache c;
  Seqs s, to;  // (to: the same table, where they move in place)
  const int32_t *index, *count;
  long long index_stride, head_stride;
  int max_count, in_place, splits, parts;
  float* mass;
};

// A CTA moves RUNS of the 2 HD / 16 runs (16 values: two words of codes and a scale) of a list's positions, or their
// weights (the last part, where there are weights). In place it goes through the list in order, a chunk's reads
// before its writes: what later entries read lies at or beyond what they write, so no chunk overwrites what
// another one needs, and parts never touch one another's bytes. Elsewhere the list may be cut as well. A list's chain
// index, page, bytes, and their sectors bound it: a run of values is 8 bytes of a sector of 32, in places that only the
// next positions share. 8192 of 32 k positions, 8 heads: 12 us elsewhere (19 MB; 3 at the HBM rate), 29 in place.
template <int HD, int RUNS, int T, int R>
__global__ void __launch_bounds__(T) move_kernel(const MoveParams p) {
  constexpr int NR = HD / kBlock, STEP = T / RUNS, CHUNK = STEP * R;
  int x = blockIdx.x;
  const int part = x % p.parts;
  x /= p.parts;
  const int h = x % p.c.hkv;
  x /= p.c.hkv;
  const int split = x % p.splits, b = x / p.splits;
  const int start = p.s.lengths ? __ldg(p.s.lengths + b) : 0, all = min(__ldg(p.count + b), p.max_count);
  if (start < 0) {
    raise(p.c.status, DEC_ERR_ARG);
    return;
  }
  const int per = (all + p.splits - 1) / p.splits, last = min(all, (split + 1) * per);
  const int32_t* const index = p.index + b * p.index_stride + h * p.head_stride;
  auto place = [&](int i, int& from, int& to) {
    const int src = __ldg(index + i);
    const long long a = (long long)start + src, z = (long long)start + i;
    if (src < 0 || (p.in_place && src == i)) return false;
    from = (int)min(a, 0x7FFFFFFFll);
    to = (int)min(z, 0x7FFFFFFFll);
    return true;
  };
  if (part == (2 * NR) / RUNS) {  // weights
    for (int c0 = split * per; c0 < last; c0 += T * R) {
      float w[R];
      float* dst[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = c0 + threadIdx.x + r * T;
        int from, to;
        dst[r] = nullptr;
        if (i < last && place(i, from, to)) {
          const uint8_t* const a = group_at<HD>(p.c, p.s, b, from, h);
          const uint8_t* const z = group_at<HD>(p.c, p.to, b, to, h);
          if (a && z) {
            w[r] = p.mass[(size_t)(a - p.c.pages) / group_bytes(HD) * kGroup + (from & 15)];
            dst[r] = p.mass + (size_t)(z - p.c.pages) / group_bytes(HD) * kGroup + (to & 15);
          }
        }
      }
      if (p.in_place) __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (dst[r]) *dst[r] = w[r];
      if (p.in_place) __syncthreads();
    }
    return;
  }
  const int run = part * RUNS + threadIdx.x % RUNS, i0 = threadIdx.x / RUNS;
  const bool key = run < NR;
  const int at = key ? run : run - NR;
  auto words = [&](int pp, int& w0, int& w1, int& sc) {
    w0 = key ? k_word<HD>(pp, 2 * at) : v_word<HD>(pp, 2 * at);
    w1 = key ? k_word<HD>(pp, 2 * at + 1) : v_word<HD>(pp, 2 * at + 1);
    sc = key ? k_scale<HD>(pp, at) : v_scale<HD>(pp, at);
  };
  for (int c0 = split * per; c0 < last; c0 += CHUNK) {
    uint32_t u0[R], u1[R];
    uint8_t sb[R];
    uint8_t* dst[R];
    int pz[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = c0 + i0 + r * STEP;
      int from, to;
      dst[r] = nullptr;
      if (i < last && place(i, from, to)) {
        const uint8_t* const a = group_at<HD>(p.c, p.s, b, from, h);
        uint8_t* const z = group_at<HD>(p.c, p.to, b, to, h);
        if (a && z) {
          int w0, w1, sc;
          words(from & 15, w0, w1, sc);
          u0[r] = *reinterpret_cast<const uint32_t*>(a + w0);
          u1[r] = *reinterpret_cast<const uint32_t*>(a + w1);
          sb[r] = a[sc];
          dst[r] = z;
          pz[r] = to & 15;
        }
      }
    }
    if (p.in_place) __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (dst[r]) {
        int w0, w1, sc;
        words(pz[r], w0, w1, sc);
        *reinterpret_cast<uint32_t*>(dst[r] + w0) = u0[r];
        *reinterpret_cast<uint32_t*>(dst[r] + w1) = u1[r];
        dst[r][sc] = sb[r];
      }
    if (p.in_place) __syncthreads();
  }
}

}  // namespace kvq
}  // namespace dec
