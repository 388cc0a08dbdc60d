// What trees of drafted tokens and bounded caches need beside the attention: a tree's masks, the attention
// weight that positions receive, the choice of the positions that stay, and moving positions as they are held.
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
// met in descending order). The walk is a chain of shared memory reads, 30 cycles a step.
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
// attention weight

struct MassParams : AttnParams {  // (lse is read)
  float decay;
  const float* mass;
  float* out;
};

constexpr int kAllRows = 1 << 30;  // (one block of rows: a unit is a sequence's KV head)

// A query row's lane share, HD / 4 values from t HD / 4 on (two a word), as the second operand of S^T = K q^T: in
// the order in which words of codes give values, scaled by a power of two to magnitude 1 .. 2 (as in the
// attention kernels); returns the factor that makes scores of it, in units of log2.
template <int HD>
__device__ __forceinline__ float query_operand(const uint32_t (&w)[HD / 8], float scale, uint32_t (&qf)[HD / 8]) {
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < HD / 8; ++i) mag = max(mag, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
  mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
  mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
  const int e = mag == 0 || mag >= 0x7F800000u ? 0 : min(126, max(-126, (int)(mag >> 23) - 127));
  const float down = __int_as_float((127 - e) << 23);
  auto val = [&](int i) { return down * __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16)); };
#pragma unroll
  for (int s = 0; s < HD / 16; ++s) {
    const int i = 8 * (s >> 1) + 2 * (s & 1);
    qf[2 * s] = h2u(__floats2half2_rn(val(i), val(i + 4)));
    qf[2 * s + 1] = h2u(__floats2half2_rn(val(i + 1), val(i + 5)));
  }
  return fmaxf(scale * __int_as_float((127 + e) << 23), 1e-37f);
}

// A group's keys as a lane holds them: the words of positions g and g + 8, and their scale bytes.
template <int HD>
struct Keys {
  uint32_t k0[HD / 32], k1[HD / 32], sb;
  __device__ __forceinline__ void load(const uint8_t* gp, int lane) {
    if (HD == 128) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(gp + lane * 16));
      const uint4 c = __ldcs(reinterpret_cast<const uint4*>(gp + 512 + lane * 16));
      k0[0] = a.x; k0[1] = a.y; k0[HD / 32 - 2] = a.z; k0[HD / 32 - 1] = a.w;
      k1[0] = c.x; k1[1] = c.y; k1[HD / 32 - 2] = c.z; k1[HD / 32 - 1] = c.w;
      sb = __ldcs(reinterpret_cast<const uint32_t*>(gp + 2 * code_bytes(HD) + lane * 4));
    } else {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(gp + lane * 16));
      k0[0] = a.x; k0[1] = a.y;
      k1[0] = a.z; k1[1] = a.w;
      sb = __ldcs(reinterpret_cast<const uint16_t*>(gp + 2 * code_bytes(HD) + lane * 2));
    }
  }
  // put(step, a0..a3): the first operand of 16 values of the head at a time
  template <class F>
  __device__ __forceinline__ void product(const Magic& magic, F&& put) const {
#pragma unroll
    for (int w2 = 0; w2 < HD / 64; ++w2) {  // two words: one scale's run
      Scale2 s0, s1;
      if (HD == 128) {
        s0.set(__byte_perm(sb, 0, w2 == 0 ? 0x4040 : 0x4141));
        s1.set(__byte_perm(sb, 0, w2 == 0 ? 0x4242 : 0x4343));
      } else {
        s0.set(__byte_perm(sb, 0, 0x4040));
        s1.set(__byte_perm(sb, 0, 0x4141));
      }
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int wi = 2 * w2 + v;
          uint32_t a0, a1, a2, a3;
          s0.decode(y ? k0[wi] >> 8 : k0[wi], magic, a0, a2);
          s1.decode(y ? k1[wi] >> 8 : k1[wi], magic, a1, a3);
          put(2 * wi + y, a0, a1, a2, a3);
        }
    }
  }
};

// What a row takes from its attention's lse (times log2 e), and the positions that it sees (0: it adds nothing).
__device__ __forceinline__ void row_terms(const MassParams& p, const SeqWork& sw, int h, int row, float& off, int& seen) {
  off = 0.f;
  seen = 0;
  if (row < sw.n * p.group) {
    const int tj = (int)fast_div(row, p.group, p.ginv);
    const float l = __ldg(p.lse + (long long)(sw.tok0 + tj) * p.hq + h * p.group + row - tj * p.group);
    if (fabsf(l) <= 3.4028235e38f) {
      off = l * 1.4426950408889634f;
      seen = max(0, p.causal ? sw.len + tj + 1 : sw.len);
    }
  }
}

// Sums of a group's positions (lane (g, t < 2) has position g + 8 t) to memory.
__device__ __forceinline__ void put_mass(const MassParams& p, int vg, int pos, int len, int held, float sum, float was) {
  const int lane = threadIdx.x & 31, at = (lane >> 2) + 8 * (lane & 3);
  if ((lane & 3) < 2 && pos + at < held)
    p.out[(size_t)vg * kGroup + at] = p.decay != 0.f && pos + at < len ? fmaf(p.decay, was, sum) : sum;
}
__device__ __forceinline__ float old_mass(const MassParams& p, int vg, int pos, int len) {
  const int lane = threadIdx.x & 31, at = (lane >> 2) + 8 * (lane & 3);
  return p.decay != 0.f && (lane & 3) < 2 && pos + at < len ? p.mass[(size_t)vg * kGroup + at] : 0.f;
}

// Few query rows (8 NB per KV head): the keys are read once, so a warp streams groups from global memory into
// registers, DEPTH of them ahead, and no warp waits for another.
template <int HD, int NB>
__global__ void __launch_bounds__(256) mass_kernel(const MassParams p) {
  constexpr int KS = HD / 16, DEPTH = 2;
  __shared__ SeqWork seqs[kMaxSeqs];
  __shared__ uint32_t scan[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t W = build_list<256, kAllRows, kGroup, 0>(p, seqs, scan);
  const uint32_t warps = min(gridDim.x * 8u, (W + p.min_groups - 1) / p.min_groups), me = blockIdx.x + gridDim.x * warp;
  if (me >= warps) return;
  const uint32_t lo = (uint32_t)((unsigned long long)W * me / warps), hi = (uint32_t)((unsigned long long)W * (me + 1) / warps);
  const int gpp = 1 << (p.c.page_shift - 4);
  const Magic magic = p.magic;
  for (uint32_t f = lo; f < hi;) {
    const int b = seq_of_entry(seqs, p.s.batch, f);
    const SeqWork sw = seqs[b];
    const int h = (int)fast_div(f - sw.pre, sw.ng, sw.inv);
    const int g0 = (int)(f - sw.pre) - h * sw.ng, n = min(sw.ng - g0, (int)(hi - f));
    f += n;
    const int held = max(0, p.causal ? sw.len + sw.n : sw.len);
    // ---- the rows
    uint32_t qf[NB][KS * 2];
    float sc[NB][2], off[NB][2];
    int seen[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = nb * 8 + g, tj = (int)fast_div(row, p.group, p.ginv);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.p) + (long long)(sw.tok0 + tj) * p.q.ts +
                                                        (h * p.group + row - tj * p.group) * p.q.hs + t * (HD / 4));
      uint32_t w[KS * 2];
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint4 x = row < sw.n * p.group ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
      }
      const float up = query_operand<HD>(w, p.scale, qf[nb]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[nb][i] = __shfl_sync(0xffffffffu, up, (2 * t + i) * 4);
        row_terms(p, sw, h, nb * 8 + 2 * t + i, off[nb][i], seen[nb][i]);
      }
    }
    // ---- their groups
    Keys<HD> keys[DEPTH];
    float was[DEPTH];
    int mine = -1;  // the group in the cache of lane's entry of 32 (-1: none)
    auto fetch = [&](int i, int slot) {  // i-th group
      if (i >= n) return;
      if ((i & 31) == 0) {
        const int gr = g0 + i + lane, pos = gr * kGroup;
        mine = -1;
        if (i + lane < n && pos < held) {
          const int page = __ldg(p.s.table + b * p.s.table_stride + (pos >> p.c.page_shift));
          if ((unsigned)page < (unsigned)p.c.n_pages) mine = (page * p.c.hkv + h) * gpp + (gr & (gpp - 1));
          else raise(p.c.status, DEC_ERR_ARG);
        }
      }
      const int vg = __shfl_sync(0xffffffffu, mine, i & 31);
      if (vg < 0) return;
      keys[slot].load(p.c.pages + (size_t)vg * group_bytes(HD), lane);
      was[slot] = old_mass(p, vg, (g0 + i) * kGroup, sw.len);
    };
    auto group = [&](int i, int slot, int vg) {
      float s[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nb][j] = 0.f;
      keys[slot].product(magic, [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16816(s[nb], a0, a1, a2, a3, qf[nb][2 * k], qf[nb][2 * k + 1]);
      });
      const int pos = (g0 + i) * kGroup;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = ex2(fmaf(s[nb][j], sc[nb][j & 1], -off[nb][j & 1]));
          sum[j >> 1] += pos + g + (j >> 1) * 8 < seen[nb][j & 1] ? e : 0.f;
        }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
        sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
      }
      put_mass(p, vg, pos, sw.len, held, t == 0 ? sum[0] : sum[1], was[slot]);
    };
    int vgs[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
      fetch(i, i);
      vgs[i] = i < n ? __shfl_sync(0xffffffffu, mine, i & 31) : -1;
    }
    for (int i0 = 0; i0 < n; i0 += DEPTH) {
#pragma unroll
      for (int x = 0; x < DEPTH; ++x) {
        const int i = i0 + x;
        if (i >= n) break;
        if (vgs[x] >= 0) group(i, x, vgs[x]);
        fetch(i + DEPTH, x);
        vgs[x] = i + DEPTH < n ? __shfl_sync(0xffffffffu, mine, (i + DEPTH) & 31) : -1;
      }
    }
  }
}

// Many query rows: each warp keeps two groups' keys as operands in registers while the CTA stages 64 rows of
// queries at a time, as the second operand, in shared memory.
template <int HD>
struct ManyCfg {
  static constexpr int THREADS = 256, WARPS = THREADS / 32, GROUPS = 2, POS = WARPS * GROUPS * kGroup, ROWS = 64;
};
template <int HD>
__global__ void __launch_bounds__(ManyCfg<HD>::THREADS, 1) mass_many_kernel(const MassParams p) {
  using C = ManyCfg<HD>;
  constexpr int KS = HD / 16, G = C::GROUPS;
  __shared__ SeqWork seqs[kMaxSeqs];
  __shared__ uint32_t scan[C::WARPS];
  __shared__ uint4 qs[C::ROWS / 8][KS / 2][32];
  __shared__ float2 terms[C::ROWS];  // factor, offset
  __shared__ int sees[C::ROWS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t W = build_list<C::THREADS, kAllRows, C::POS, 0>(p, seqs, scan);
  const int gpp = 1 << (p.c.page_shift - 4);
  const Magic magic = p.magic;
  for (uint32_t f = blockIdx.x; f < W; f += gridDim.x) {
    const int b = seq_of_entry(seqs, p.s.batch, f);
    const SeqWork sw = seqs[b];
    const int h = (int)fast_div(f - sw.pre, sw.ng, sw.inv), block = (int)(f - sw.pre) - h * sw.ng;
    const int held = max(0, p.causal ? sw.len + sw.n : sw.len), rows = sw.n * p.group;
    const int pos0 = block * C::POS + warp * G * kGroup;
    // ---- the keys, as operands
    uint32_t a[G][KS][4];
    int vg[G];
    float was[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int pos = pos0 + i * kGroup;
      vg[i] = -1;
      if (pos < held) {
        const int page = __ldg(p.s.table + b * p.s.table_stride + (pos >> p.c.page_shift));
        if ((unsigned)page < (unsigned)p.c.n_pages) vg[i] = (page * p.c.hkv + h) * gpp + ((pos >> 4) & (gpp - 1));
        else raise(p.c.status, DEC_ERR_ARG);
      }
      if (vg[i] >= 0) {
        Keys<HD> keys;
        keys.load(p.c.pages + (size_t)vg[i] * group_bytes(HD), lane);
        was[i] = old_mass(p, vg[i], pos, sw.len);
        keys.product(magic, [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          a[i][k][0] = a0; a[i][k][1] = a1; a[i][k][2] = a2; a[i][k][3] = a3;
        });
      } else {
        was[i] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) a[i][k][0] = a[i][k][1] = a[i][k][2] = a[i][k][3] = 0u;
      }
    }
    float sum[G][2];
#pragma unroll
    for (int i = 0; i < G; ++i) sum[i][0] = sum[i][1] = 0.f;
    // (rows before the first that sees the block add nothing)
    const int skip = p.causal ? max(0, block * C::POS - sw.len) * p.group / C::ROWS * C::ROWS : 0;
    for (int r0 = skip; r0 < rows; r0 += C::ROWS) {
      __syncthreads();
      // ---- 64 rows: four lanes a row
      {
        const int r = threadIdx.x >> 2, row = r0 + r, tj = (int)fast_div(row, p.group, p.ginv);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.p) + (long long)(sw.tok0 + tj) * p.q.ts +
                                                          (h * p.group + row - tj * p.group) * p.q.hs + t * (HD / 4));
        uint32_t w[KS * 2], qf[KS * 2];
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 x = row < rows ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
          w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
        const float up = query_operand<HD>(w, p.scale, qf);
#pragma unroll
        for (int i = 0; i < KS / 2; ++i)
          qs[r >> 3][i][(r & 7) * 4 + t] = make_uint4(qf[4 * i], qf[4 * i + 1], qf[4 * i + 2], qf[4 * i + 3]);
        if (t == 0) {
          float off;
          int seen;
          row_terms(p, sw, h, row, off, seen);
          terms[r] = make_float2(up, off);
          sees[r] = seen;
        }
      }
      __syncthreads();
      const int blocks = min(C::ROWS, rows - r0 + 7) / 8;
      for (int nb = 0; nb < blocks; ++nb) {
        float s[G][4];
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          const uint4 q = qs[nb][k / 2][lane];
#pragma unroll
          for (int i = 0; i < G; ++i) {
            mma16816(s[i], a[i][k][0], a[i][k][1], a[i][k][2], a[i][k][3], q.x, q.y);
            mma16816(s[i], a[i][k + 1][0], a[i][k + 1][1], a[i][k + 1][2], a[i][k + 1][3], q.z, q.w);
          }
        }
        const float4 tm = *reinterpret_cast<const float4*>(&terms[nb * 8 + 2 * t]);
        const int2 see = *reinterpret_cast<const int2*>(&sees[nb * 8 + 2 * t]);
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = ex2(fmaf(s[i][j], (j & 1) ? tm.z : tm.x, (j & 1) ? -tm.w : -tm.y));
            sum[i][j >> 1] += pos0 + i * kGroup + g + (j >> 1) * 8 < ((j & 1) ? see.y : see.x) ? e : 0.f;
          }
      }
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        sum[i][0] += __shfl_xor_sync(0xffffffffu, sum[i][0], o);
        sum[i][1] += __shfl_xor_sync(0xffffffffu, sum[i][1], o);
      }
      if (vg[i] >= 0) put_mass(p, vg[i], pos0 + i * kGroup, sw.len, held, t == 0 ? sum[i][0] : sum[i][1], was[i]);
    }
  }
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

// One CTA per (sequence, KV head): the need-th largest weight by its digits (11, 11 and 10 bits of a key that orders
// as the weights do), then the positions in order: each warp counts, and writes, its own stretch.
constexpr int kKeepThreads = 1024;
__global__ void __launch_bounds__(kKeepThreads) heaviest_kernel(const KeepParams p) {
  constexpr int T = kKeepThreads, BINS = 2048;
  extern __shared__ uint32_t cache[];
  __shared__ uint32_t hist[BINS], part[32];
  __shared__ uint32_t sh_bin, sh_left;
  __shared__ uint2 counts[32];
  const int b = blockIdx.x / p.c.hkv, h = blockIdx.x - b * p.c.hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int len = __ldg(p.s.lengths + b);
  const bool bad = len < 0 || len > (long long)p.s.max_pages << p.c.page_shift;
  if (bad) {
    if (tid == 0) raise(p.c.status, len < 0 ? DEC_ERR_ARG : DEC_ERR_CAPACITY);
    len = 0;
  }
  int32_t* const kept = p.kept + ((size_t)b * p.c.hkv + h) * p.budget;
  if (h == 0 && tid == 0) p.count[b] = min(len, p.budget);
  if (len <= p.budget) {
    for (int i = tid; i < p.budget; i += T) kept[i] = i < len ? i : -1;
    return;
  }
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
  auto key_of = [&](int pos) { return pos < p.cached ? cache[pos] : load(pos); };
  for (int pos = tid; pos < min(len, p.cached); pos += T) cache[pos] = load(pos);
  // ---- threshold and how many of its equals belong
  const int end = len - p.recent;  // candidates: sinks .. end - 1
  uint32_t need = (uint32_t)(p.budget - p.sinks - p.recent), prefix = 0;
  const bool any = need > 0;
  for (int d = 0; any && d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
    for (int i = tid; i < BINS; i += T) hist[i] = 0;
    __syncthreads();
    for (int pos = p.sinks + tid; pos < end; pos += T) {
      const uint32_t k = key_of(pos);
      if (d == 0 || k >> (shift + bits) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
    }
    __syncthreads();
    // from the top: thread i has bins BINS - 1 - 2i and the one below
    const uint32_t c0 = hist[BINS - 1 - 2 * tid], c1 = hist[BINS - 2 - 2 * tid];
    uint32_t x = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    uint32_t before = x - c0 - c1;
    for (int i = 0; i < warp; ++i) before += part[i];
    if (before < need && need <= before + c0 + c1) {
      const bool first = need <= before + c0;
      sh_bin = BINS - 1 - 2 * tid - (first ? 0 : 1);
      sh_left = need - before - (first ? 0u : c0);
    }
    __syncthreads();
    prefix = prefix << bits | sh_bin;
    need = sh_left;
  }
  // ---- in order
  const int seg = ((len + 31) / 32 + 31) / 32 * 32;
  const int lo = min(len, warp * seg), hi = min(len, lo + seg);
  auto classes = [&](int pos, bool& in, bool& tie) {
    const bool mid = pos >= p.sinks && pos < end;
    const uint32_t k = any && mid && pos < hi ? key_of(pos) : 0u;
    in = pos < hi && (!mid || (any && k > prefix));
    tie = any && mid && pos < hi && k == prefix;
  };
  __syncthreads();  // (the cache, where there was no threshold to find)
  uint32_t ins = 0, ties = 0;
  for (int pos = lo + lane; pos - lane < hi; pos += 32) {
    bool in, tie;
    classes(pos, in, tie);
    ins += in;
    ties += tie;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ins += __shfl_xor_sync(0xffffffffu, ins, o);
    ties += __shfl_xor_sync(0xffffffffu, ties, o);
  }
  if (lane == 0) counts[warp] = make_uint2(ins, ties);
  __syncthreads();
  ins = ties = 0;
  for (int i = 0; i < warp; ++i) {
    ins += counts[i].x;
    ties += counts[i].y;
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
// another one needs, and parts never touch one another's bytes. Elsewhere the list may be cut as well.
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
