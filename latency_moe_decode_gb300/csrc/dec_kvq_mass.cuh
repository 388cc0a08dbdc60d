// The attention weight that cached positions receive from a call's queries, added up (dec_kvq_mass).
//
// The work is reading the keys once, and for many query rows a product of all of them with all keys and an exponential
// of each score, whose lse is known: nothing is joined over positions, and each position's sum belongs to one thread.
//  - Few rows (8 or 16 per KV head): mass_kernel, a stream of keys through registers.
//  - Many rows: mass_tile_kernel, scores on tcgen05 with the keys as the product's 128 rows: a thread then holds
//    one position, and a query's factor and lse are the same for the whole warp.
#pragma once
#include "dec_f32x2.cuh"
#include "dec_kvq_attn.cuh"
#include "dec_kvq_prompt.cuh"

namespace dec {
namespace kvq {

struct MassParams : AttnParams {  // (lse is read)
  float decay;
  const float* mass;
  float* out;
};

constexpr int kAllRows = 1 << 30;  // (one block of rows: a unit is a sequence's KV head)

// How many positions a sequence has: with its rows' own (causal), but none beyond its page table, where entries are
// another sequence's, or no table any more. (A tile of 128 positions may pass the table's end; a group of 16 does not.)
__device__ __forceinline__ int held_of(const MassParams& p, const SeqWork& sw) {
  return min(max(0, p.causal ? sw.len + sw.n : sw.len), p.s.max_pages << p.c.page_shift);
}

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

// A group's keys as a lane holds them (K codes and K scales, one behind the other): put(step, a0..a3), the first operand
// of 16 values of the head at a time.
template <int HD, class F>
__device__ __forceinline__ void key_product(const uint8_t* gp, const Magic& magic, F&& put) {
  const int lane = threadIdx.x & 31;
  uint32_t k0[HD / 32], k1[HD / 32], sb;  // words of positions g and g + 8; scale bytes
  if (HD == 128) {
    const uint4 a = *reinterpret_cast<const uint4*>(gp + lane * 16);
    const uint4 c = *reinterpret_cast<const uint4*>(gp + 512 + lane * 16);
    k0[0] = a.x; k0[1] = a.y; k0[HD / 32 - 2] = a.z; k0[HD / 32 - 1] = a.w;
    k1[0] = c.x; k1[1] = c.y; k1[HD / 32 - 2] = c.z; k1[HD / 32 - 1] = c.w;
    sb = *reinterpret_cast<const uint32_t*>(gp + code_bytes(HD) + lane * 4);
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(gp + lane * 16);
    k0[0] = a.x; k0[1] = a.y;
    k1[0] = a.z; k1[1] = a.w;
    sb = *reinterpret_cast<const uint16_t*>(gp + code_bytes(HD) + lane * 2);
  }
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

// Few query rows (8 NB per KV head): the keys are read once, each warp streaming its part of the list through its own
// ring with bulk copies (of a group's codes, scales and, where they count, the weights that its positions have), two
// groups at a time, some ahead, without ever waiting for another warp.
// Measured (32 query, 8 KV heads of 128, one row a sequence): 16 sequences of 8 k to 32 k 53 us, 3.7 TB/s; issue slots are 62 %
// full (230 instructions a group, 80 of them make operands of its codes), and no pipe is: warps wait for their own
// instructions, two chains of eight dependent products first of all. Groups loaded into
// registers two ahead took 65, four ahead 64; their old weights loaded where they are needed 61. Comparisons left out where
// every row sees the whole group changed nothing.
template <int HD>
struct StreamCfg {
  static constexpr int WARPS = 8, CH = 2, STAGES = 4;
  static constexpr int RAW1 = code_bytes(HD) + scale_bytes(HD), SLOT = RAW1 + kGroup * 4, RING = STAGES * CH * SLOT;
  static constexpr int smem() { return WARPS * RING + kMaxSeqs * (int)sizeof(SeqWork); }
};
template <int HD, int NB>
__global__ void __launch_bounds__(256, 2) mass_kernel(const MassParams p) {
  using C = StreamCfg<HD>;
  constexpr int KS = HD / 16, CH = C::CH;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ uint32_t scan[C::WARPS];
  __shared__ uint64_t bars[C::WARPS][C::STAGES];
  SeqWork* const seqs = reinterpret_cast<SeqWork*>(dyn + C::WARPS * C::RING);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(bars[warp] + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const uint32_t W = build_list<256, kAllRows, kGroup, 0>(p, seqs, scan);
  const uint32_t warps = min(gridDim.x * 8u, (W + p.min_groups - 1) / p.min_groups), me = blockIdx.x + gridDim.x * warp;
  if (me >= warps) return;
  const uint32_t lo = (uint32_t)((unsigned long long)W * me / warps), hi = (uint32_t)((unsigned long long)W * (me + 1) / warps);
  const int gpp = 1 << (p.c.page_shift - 4);
  const Magic magic = p.magic;
  uint8_t* const ring = dyn + warp * C::RING;
  int pstage = 0, cstage = 0;
  uint32_t cphase = 0;
  bool dead = false;
  for (uint32_t f = lo; f < hi && !dead;) {
    const int b = seq_of_entry(seqs, p.s.batch, f);
    const SeqWork sw = seqs[b];
    const int h = (int)fast_div(f - sw.pre, sw.ng, sw.inv);
    const int g0 = (int)(f - sw.pre) - h * sw.ng, n = min(sw.ng - g0, (int)(hi - f));
    f += n;
    const int held = held_of(p, sw);
    // ---- copies, a chunk at a time
    int ahead = -1, mine = -1;  // groups in the cache of the 32 that the copies, and that the sums are in (-1: none)
    auto fetch = [&](int i) {   // groups i, i + 1
      if (i >= n) return;
      if ((i & 31) == 0) {
        const int gr = g0 + i + lane, pos = gr * kGroup;
        ahead = -1;
        if (i + lane < n && pos < held) {
          const int page = __ldg(p.s.table + b * p.s.table_stride + (pos >> p.c.page_shift));
          if ((unsigned)page < (unsigned)p.c.n_pages) ahead = (page * p.c.hkv + h) * gpp + (gr & (gpp - 1));
          else raise(p.c.status, DEC_ERR_ARG);
        }
      }
      const int at = lane - (i & 31);
      const bool copies = at >= 0 && at < CH && ahead >= 0;
      const uint32_t who = __ballot_sync(0xffffffffu, copies);
      uint64_t* const bar = bars[warp] + pstage;
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc(who) * (p.decay != 0.f ? C::SLOT : C::RAW1));
      __syncwarp();
      if (copies) {
        uint8_t* const to = ring + (pstage * CH + at) * C::SLOT;
        const uint8_t* const from = p.c.pages + (size_t)ahead * group_bytes(HD);
        bulk_copy(to, from, code_bytes(HD), bar);
        bulk_copy(to + code_bytes(HD), from + 2 * code_bytes(HD), scale_bytes(HD), bar);
        if (p.decay != 0.f) bulk_copy(to + C::RAW1, p.mass + (size_t)ahead * kGroup, kGroup * 4, bar);
      }
      pstage = pstage == C::STAGES - 1 ? 0 : pstage + 1;
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) fetch(i * CH);
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
    for (int i0 = 0; i0 < n; i0 += CH) {
      fetch(i0 + (C::STAGES - 1) * CH);
      // (the copies are less than 32 groups ahead: theirs are these as soon as the first of them is due)
      if ((i0 & 31) == 0) mine = ahead;
      int vg[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        vg[i] = __shfl_sync(0xffffffffu, mine, (i0 + i) & 31);
        if (i0 + i >= n) vg[i] = -1;
      }
      if (!bar_wait(bars[warp] + cstage, cphase)) {
        raise(p.c.status, DEC_ERR_TIMEOUT);
        for (int i = 1; i < C::STAGES; ++i) bar_wait(bars[warp] + (cstage + i) % C::STAGES, i + cstage < C::STAGES ? cphase : cphase ^ 1);
        dead = true;
        break;
      }
      const uint8_t* const buf = ring + cstage * CH * C::SLOT;
      if (++cstage == C::STAGES) {
        cstage = 0;
        cphase ^= 1;
      }
      float s[CH][NB][4];
#pragma unroll
      for (int i = 0; i < CH; ++i) {  // (a group that is not there: whatever the ring holds, written nowhere)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][nb][j] = 0.f;
        key_product<HD>(buf + i * C::SLOT, magic, [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(s[i][nb], a0, a1, a2, a3, qf[nb][2 * k], qf[nb][2 * k + 1]);
        });
      }
      float sum[CH][2];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int pos = (g0 + i0 + i) * kGroup;
        sum[i][0] = sum[i][1] = 0.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = ex2(fmaf(s[i][nb][j], sc[nb][j & 1], -off[nb][j & 1]));
            sum[i][j >> 1] += pos + g + (j >> 1) * 8 < seen[nb][j & 1] ? e : 0.f;
          }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          sum[i][0] += __shfl_xor_sync(0xffffffffu, sum[i][0], o);
          sum[i][1] += __shfl_xor_sync(0xffffffffu, sum[i][1], o);
        }
      }
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (vg[i] >= 0 && t < 2) {  // lane (g, t < 2) has position g + 8 t
          const int at = g + 8 * t, pos = (g0 + i0 + i) * kGroup + at;
          const float x = t == 0 ? sum[i][0] : sum[i][1], was = *reinterpret_cast<const float*>(buf + i * C::SLOT + C::RAW1 + at * 4);
          if (pos < held) p.out[(size_t)vg[i] * kGroup + at] = p.decay != 0.f && pos < sw.len ? fmaf(p.decay, was, x) : x;
        }
      __syncwarp();  // (the next copy goes where this chunk lay)
    }
  }
}

// Many query rows. A CTA takes a stretch of (sequence, KV head, tile of 128 positions) entries; of each, blocks of
// 128 query rows. A role for each warp:
//  - one finds the tiles, tells the others, and copies their key codes (bulk copies, three tiles ahead);
//  - four turn them into bf16 (which holds code x scale exactly) in the 128-byte swizzled layout;
//  - eight, four for each of two buffers, copy blocks of queries there as they are, with each row's lse and the positions it
//    sees. (In f16, as the prompt kernel has them, they had to be scaled row by row: 3.7 us before the first
//    products.) Up to 256 rows stay there for all of a KV head's tiles; more go through the two buffers in turn;
//  - one thread issues S = K Q^T (128 x 128 x hd), two S buffers in tensor memory for each of the next two groups;
//  - two groups of eight take the tiles in turn, one position and half a block's queries a thread: exponentials and their
//    sum. (With all sixteen on one tile the exponentials' unit stood idle between blocks and tiles, half of the time.)
// What bounds it: the exponentials, 16 an SM and cycle, 1 k cycles a tile and block (its products take 0.6 k), and what comes
// before the first of them. Measured (32 query, 8 KV heads of 128): two sequences' 64 rows, 256 a KV head, on 4 k to 8 k 21 us, of
// which 6 pass before the first products (the list 1.7, a tile's pages 1.2, its copies, decoding and the queries 2.5);
// scores by 16 x 8 x 16 products of registers took 38.
template <int HD>
struct TileCfg {
  static constexpr int EW = 16, DW = 4, QW = 8;  // 64 registers each
  static constexpr int THREADS = (EW + DW + QW + 2) * 32;
  static constexpr int HP = HD / 64, OPERAND = HP * 16384, STAGES = 4;
  static constexpr int RAW1 = code_bytes(HD) + scale_bytes(HD), RAW = kTile / kGroup * RAW1;  // a group's keys, a tile's
  static constexpr int K = 0, Q = 2 * OPERAND, RING = 4 * OPERAND, TABLE = RING + STAGES * RAW;
  static constexpr int smem() { return TABLE + kMaxSeqs * (int)sizeof(SeqWork) + 1024; }
};
// A tile, as all roles take it. A place is written again 16 tiles later. The copies have then waited for the decoding and
// staging warps to be done with the tile 4 back, whose decoding waited for the products of the one 6 back, and those, like
// the products before them, for the sums of one at most 5 back: only places of tiles at most 11 back are still read.
constexpr int kInfos = 16;
struct TileInfo {
  int pos0, held, len, n, tok0, h;  // first position, positions there are; the sequence's
  int rb0, nrb;                     // blocks of rows that see it
  int fresh, end;                   // the first tile of a KV head; behind the last tile
  int vg[kTile / kGroup];           // its groups in the cache (-1: none)
};
struct TileBars {
  uint64_t raw_full[4], raw_empty[4], k_full[2], k_empty[2], q_full[2], q_empty[2], s_full[4], s_empty[4], info[kInfos];
  uint64_t half[2][4][4];  // a group's 32 positions: the second half's sums of its tile (four in turn) are there
};
struct TileTerms {  // of a staged block's rows
  float off[128];
  int sees[128];
  int all[4], some[4];  // positions that all, and that any of 32 rows see
};

// Which staging of which buffer a step (a tile's block) uses, by every role alike.
struct TileQueries {
  int n0 = 0, n1 = 0, have = 0, step = 0;  // stagings so far; buffers whose queries stay
  __device__ __forceinline__ int use(const TileInfo& t, int rb, bool& staged, int& nth) {
    const bool stay = t.nrb <= 2;
    const int buf = stay ? rb : step & 1;
    staged = !stay || !(have >> buf & 1);
    have = stay ? have | 1 << buf : have & ~(1 << buf);
    n0 += staged && buf == 0;
    n1 += staged && buf == 1;
    nth = (buf ? n1 : n0) - 1;
    ++step;
    return buf;
  }
};

template <int HD>
__global__ void __launch_bounds__(TileCfg<HD>::THREADS, 1) mass_tile_kernel(const MassParams p) {
  using C = TileCfg<HD>;
  extern __shared__ uint8_t dyn[];
  __shared__ TileBars bars;
  __shared__ __align__(16) TileTerms terms[2];
  __shared__ TileInfo infos[kInfos];
  __shared__ uint32_t sh_scan[C::THREADS / 32], tmem_base;
  __shared__ float halves_sum[2][4][128];
  uint8_t* const smem = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
  SeqWork* const seqs = reinterpret_cast<SeqWork*>(smem + C::TABLE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], C::DW + C::QW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.k_full[i], C::DW);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.q_full[i], C::QW / 2);
      mbar_init(&bars.q_empty[i], C::EW);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_empty[i], C::EW / 2);
    }
    for (int i = 0; i < kInfos; ++i) mbar_init(&bars.info[i], 1);
    for (int i = 0; i < 32; ++i) mbar_init(&bars.half[0][0][0] + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::EW + C::DW + C::QW) tmem_alloc(&tmem_base, 512);
  tc_fence_before();
  const uint32_t W = build_list<C::THREADS, 128, kTile, 0>(p, seqs, sh_scan);
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  bool ok = true;  // (false after a wait that ran out: the thread waits no more and runs to its end)
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (ok && !bar_wait(b, parity)) {
      ok = false;
      raise(p.c.status, DEC_ERR_TIMEOUT);
    }
  };
  TileQueries qs;
  int kt = 0;  // tiles so far
  auto next = [&]() -> const TileInfo* {  // the next tile (null: none)
    wait(&bars.info[kt % kInfos], (kt / kInfos) & 1);
    const TileInfo* const t = infos + kt % kInfos;
    return ok && !t->end ? t : nullptr;
  };

  if (warp == C::EW + C::DW + C::QW + 1) {
    // ---- tiles, and their copies: lane i the tile's group i. The list counts (tile, block) pairs, so that the cut is even
    // whatever the sequences' rows; a tile belongs to the CTA in whose part its first pair lies.
    const int gpp = 1 << (p.c.page_shift - 4);
    uint32_t f = (uint32_t)((unsigned long long)W * blockIdx.x / gridDim.x);
    const uint32_t end = (uint32_t)((unsigned long long)W * (blockIdx.x + 1) / gridDim.x);
    int last_b = -1, last_h = -1;
    while (f < end) {
      const int b = seq_of_entry(seqs, p.s.batch, f);
      const SeqWork sw = seqs[b];
      const uint32_t r = f - sw.pre, u = r / (uint32_t)sw.nrb, in = r - u * (uint32_t)sw.nrb;
      if (in > 0) {  // (another CTA's tile)
        f += sw.nrb - in;
        continue;
      }
      const int h = (int)fast_div(u, sw.ng, sw.inv), first = (int)u - h * sw.ng;
      const int held = held_of(p, sw);
      // up to four of the KV head's tiles at once: lane 8 j + i has the j-th one's group i
      const int most = min(min(4, sw.ng - first), (int)((end - f + sw.nrb - 1) / sw.nrb));
      const int j = lane >> 3, pos = (first + j) * kTile + (lane & 7) * kGroup;
      int gi = -1;
      if (j < most && pos < held) {
        const int page = __ldg(p.s.table + b * p.s.table_stride + (pos >> p.c.page_shift));
        if ((unsigned)page < (unsigned)p.c.n_pages) gi = (page * p.c.hkv + h) * gpp + ((pos >> 4) & (gpp - 1));
        else raise(p.c.status, DEC_ERR_ARG);
      }
      for (int x = 0; x < most; ++x) {
        f += sw.nrb;
        const int pos0 = (first + x) * kTile, st = kt % C::STAGES;
        if (pos0 >= held) continue;
        if (kt >= C::STAGES) wait(&bars.raw_empty[st], (kt / C::STAGES - 1) & 1);
        TileInfo& t = infos[kt % kInfos];
        const bool mine = j == x;
        if (mine) t.vg[lane & 7] = gi;
        if (lane == 0) {
          t.pos0 = pos0;
          t.held = held;
          t.len = sw.len;
          t.n = sw.n;
          t.tok0 = sw.tok0;
          t.h = h;
          // (rows before the first that sees the tile add nothing)
          t.rb0 = p.causal ? max(0, pos0 - sw.len) * p.group / 128 : 0;
          t.nrb = sw.nrb;
          t.fresh = b != last_b || h != last_h;
          t.end = 0;
        }
        last_b = b;
        last_h = h;
        const uint32_t who = __ballot_sync(0xffffffffu, mine && gi >= 0);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.info[kt % kInfos]);
          mbar_arrive_expect_tx(&bars.raw_full[st], __popc(who) * C::RAW1);
        }
        __syncwarp();
        if (mine && gi >= 0) {
          uint8_t* const to = smem + C::RING + st * C::RAW + (lane & 7) * C::RAW1;
          const uint8_t* const from = p.c.pages + (size_t)gi * group_bytes(HD);
          bulk_copy(to, from, code_bytes(HD), &bars.raw_full[st]);
          bulk_copy(to + code_bytes(HD), from + 2 * code_bytes(HD), scale_bytes(HD), &bars.raw_full[st]);
        }
        ++kt;
      }
    }
    if (lane == 0) {
      infos[kt % kInfos].end = 1;
      mbar_arrive(&bars.info[kt % kInfos]);
    }
    for (int i = max(0, kt - C::STAGES); i < kt; ++i) bar_wait(&bars.raw_full[i % C::STAGES], (i / C::STAGES) & 1);
  } else if (warp == C::EW + C::DW + C::QW) {
    // ---- products
    if (lane == 0) {
      constexpr uint32_t kId = idesc_bf16_f32(128, 128, false);
      int n0 = 0, n1 = 0;  // each group's steps: its tiles take its own buffers in turn, so that it waits for each of their phases
      for (const TileInfo* t; (t = next()); ++kt) {
        if (t->fresh) qs.have = 0;
        wait(&bars.k_full[kt & 1], (kt >> 1) & 1);
        for (int rb = t->rb0; rb < t->nrb; ++rb) {
          const int n = kt & 1 ? n1++ : n0++, sb = (kt & 1) * 2 + (n & 1);
          bool staged;
          int nth;
          const int buf = qs.use(*t, rb, staged, nth);
          if (staged) wait(&bars.q_full[buf], nth & 1);
          if (n >= 2) wait(&bars.s_empty[sb], ((n >> 1) - 1) & 1);
          tc_fence_after();
          const uint8_t* const k = smem + C::K + (kt & 1) * C::OPERAND;
          const uint8_t* const q = smem + C::Q + buf * C::OPERAND;
#pragma unroll
          for (int d = 0; d < HD / 16; ++d) {
            const int at = (d >> 2) * 16384 + (d & 3) * 32;
            mma_bf16(tmem + sb * 128, smem_desc_sw128(k + at, 16, 1024), smem_desc_sw128(q + at, 16, 1024), kId,
                     d > 0 ? 1u : 0u);
          }
          mma_commit(&bars.s_full[sb]);
        }
        mma_commit(&bars.k_empty[kt & 1]);
      }
      if (n0 > 0) bar_wait(&bars.s_full[(n0 - 1) & 1], ((n0 - 1) >> 1) & 1);
      if (n1 > 0) bar_wait(&bars.s_full[2 + ((n1 - 1) & 1)], ((n1 - 1) >> 1) & 1);
    }
    __syncwarp();
  } else if (warp >= C::EW + C::DW) {
    // ---- queries: a buffer's 32 rows a warp, HD / 8 lanes a row
    constexpr int LPR = HD / 8, RPI = 32 / LPR;
    const int group = (warp - C::EW - C::DW) >> 2, part = (warp - C::EW - C::DW) & 3, c = lane % LPR;
    for (const TileInfo* t; (t = next()); ++kt) {
      if (t->fresh) qs.have = 0;
      for (int rb = t->rb0; rb < t->nrb; ++rb) {
        bool staged;
        int nth;
        const int buf = qs.use(*t, rb, staged, nth);
        if (!staged || buf != group) continue;
        const int rows = t->n * p.group, row0 = rb * 128 + part * 32;
        // this lane's own row: its lse and what it sees (a row without a finite lse adds nothing)
        const int own = row0 + lane, tj0 = (int)fast_div(own, p.group, p.ginv);
        const float lse = own < rows ? __ldg(p.lse + (long long)(t->tok0 + tj0) * p.hq + t->h * p.group + own - tj0 * p.group) : INFINITY;
        if (nth > 0) wait(&bars.q_empty[buf], (nth - 1) & 1);
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {  // (zeros for rows that are not there)
          const int r = part * 32 + i * RPI + lane / LPR, row = rb * 128 + r, tj = (int)fast_div(row, p.group, p.ginv);
          const bool live = row < rows;
          const uint16_t* const src = static_cast<const uint16_t*>(p.q.p) +
                                      (live ? (long long)(t->tok0 + tj) * p.q.ts + (t->h * p.group + row - tj * p.group) * p.q.hs + c * 8 : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem + C::Q) + buf * C::OPERAND + r * 128 +
                                                                          (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4)),
                       "l"(src), "r"(live ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        TileTerms& tm = terms[buf];
        const bool fine = fabsf(lse) <= 3.4028235e38f;
        const int seen = fine ? max(0, p.causal ? t->len + tj0 + 1 : t->len) : 0;
        tm.off[part * 32 + lane] = fine ? lse * -1.4426950408889634f : 0.f;
        tm.sees[part * 32 + lane] = seen;
        const int all = __reduce_min_sync(0xffffffffu, seen), some = __reduce_max_sync(0xffffffffu, seen);
        if (lane == 0) {
          tm.all[part] = all;
          tm.some[part] = some;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.q_full[buf]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.raw_empty[kt % C::STAGES]);  // (done with the tile's place)
    }
  } else if (warp >= C::EW) {
    // ---- codes to operands: half a group at a time, in an order that spreads the 16-byte stores of eight lanes over
    // all banks (as the prompt kernel's keys)
    const int kw = warp - C::EW;
    const Magic magic = p.magic;
    const int k_t = (lane & 1) | ((lane >> 3) & 1) << 1, kg = ((lane >> 1) & 3) | ((lane >> 4) & 1) << 2;
    const int kc = k_t * (HD / 32);  // the lane's first chunk
    const uint32_t ka = smem_u32(smem) + C::K + kg * 128 + (kc >> 3) * 16384 + (((kc & 7) ^ kg) << 4);
    struct Scale {
      __nv_bfloat162 s, c;
    };
    auto scale = [&](uint32_t byte) {  // (without the factor 8)
      const __nv_bfloat162 s = __float2bfloat162_rn(__half2float(__ushort_as_half((unsigned short)(byte << 7))));
      return Scale{s, __hmul2(s, __float2bfloat162_rn(-136.0f))};
    };
    // (code + 8) enters the low mantissa bits of the bf16 128, and (128 + u) s - 136 s is exact (136 = 17 * 8, s of 4
    // significant bits)
    auto put = [&](uint32_t at, uint32_t v, const Scale& sc) {
      uint32_t o[4];  // values i and i + 4
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x;
        asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(x) : "r"(v >> (4 * i)), "r"(magic.lo));
        const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), sc.s, sc.c);
        o[i] = *reinterpret_cast<const uint32_t*>(&y);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(__byte_perm(o[0], o[1], 0x5410)),
                   "r"(__byte_perm(o[2], o[3], 0x5410)), "r"(__byte_perm(o[0], o[1], 0x7632)), "r"(__byte_perm(o[2], o[3], 0x7632))
                   : "memory");
    };
    for (; next(); ++kt) {
      const int st = kt % C::STAGES;
      wait(&bars.raw_full[st], (kt / C::STAGES) & 1);
      if (kt >= 2) wait(&bars.k_empty[kt & 1], ((kt >> 1) - 1) & 1);
      const uint8_t* const from = smem + C::RING + st * C::RAW;
      const uint32_t to = ka + (kt & 1) * C::OPERAND;
#pragma unroll
      for (int x = 0; x < 16 / C::DW; ++x) {
        const int hg = kw + x * C::DW, y = hg & 1;
        const uint8_t* const gp = from + (hg >> 1) * C::RAW1;
        const uint32_t at = to + hg * 1024;
        if (HD == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(gp + y * 512 + (kg * 4 + k_t) * 16);
          const uint32_t sb = *reinterpret_cast<const uint16_t*>(gp + code_bytes(HD) + (kg * 4 + k_t) * 4 + y * 2);
          const Scale s0 = scale(sb & 255u), s1 = scale(sb >> 8);
          put(at, u.x, s0);
          put(at ^ 16, u.y, s0);
          put(at ^ 32, u.z, s1);
          put(at ^ 48, u.w, s1);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(gp + (kg * 4 + k_t) * 16 + y * 8);
          const Scale s0 = scale(gp[code_bytes(HD) + (kg * 4 + k_t) * 2 + y]);
          put(at, u.x, s0);
          put(at ^ 16, u.y, s0);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.k_full[kt & 1]);
        mbar_arrive(&bars.raw_empty[st]);
      }
    }
  } else {
    // ---- a position and half a block's queries a thread
    const int group = warp >> 3, half = warp >> 2 & 1, r = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + half * 64;
    const uint64_t factor2 = pair(p.scale, p.scale);
    int n = 0;
    for (const TileInfo* t; (t = next()); ++kt) {
      if (t->fresh) {  // the queries that stayed for the KV head before
        if (lane == 0) {
          if (qs.have & 1) mbar_arrive(&bars.q_empty[0]);
          if (qs.have & 2) mbar_arrive(&bars.q_empty[1]);
        }
        qs.have = 0;
      }
      const bool own = (kt & 1) == group;
      const int pos = t->pos0 + r, end = min(t->pos0 + kTile, t->held);
      const int vg = own && pos < t->held ? t->vg[r >> 4] : -1;
      const bool old = p.decay != 0.f && pos < t->len;
      const float was = half == 0 && vg >= 0 && old ? p.mass[(size_t)vg * kGroup + (pos & 15)] : 0.f;
      uint64_t sum2 = 0;
      for (int rb = t->rb0; rb < t->nrb; ++rb) {
        bool staged;
        int nth;
        const int buf = qs.use(*t, rb, staged, nth);
        if (staged) wait(&bars.q_full[buf], nth & 1);  // (of the other group's tiles too: no phase is passed over)
        if (own) {
          const int sb = group * 2 + (n & 1);
          const TileTerms& tm = terms[buf];
          wait(&bars.s_full[sb], (n >> 1) & 1);
          ++n;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int part = half * 2 + c;
            if (tm.some[part] <= t->pos0) continue;  // (no row of it sees the tile)
            float x[32];
            tmem_ld32(tl + sb * 128 + c * 32, x);
            if (end <= tm.all[part]) {
#pragma unroll
              for (int y = 0; y < 32; y += 4) {
                const float4 of = *reinterpret_cast<const float4*>(&tm.off[part * 32 + y]);
                const float2 a = halves(fma2(pair(x[y], x[y + 1]), factor2, pair(of.x, of.y)));
                const float2 b = halves(fma2(pair(x[y + 2], x[y + 3]), factor2, pair(of.z, of.w)));
                sum2 = add2(sum2, pair(ex2(a.x), ex2(a.y)));
                sum2 = add2(sum2, pair(ex2(b.x), ex2(b.y)));
              }
            } else {
#pragma unroll
              for (int y = 0; y < 32; y += 4) {
                const float4 of = *reinterpret_cast<const float4*>(&tm.off[part * 32 + y]);
                const int4 se = *reinterpret_cast<const int4*>(&tm.sees[part * 32 + y]);
                const float a = ex2(fmaf(x[y], p.scale, of.x)), b = ex2(fmaf(x[y + 1], p.scale, of.y));
                const float d = ex2(fmaf(x[y + 2], p.scale, of.z)), g = ex2(fmaf(x[y + 3], p.scale, of.w));
                sum2 = add2(sum2, pair(pos < se.x ? a : 0.f, pos < se.y ? b : 0.f));
                sum2 = add2(sum2, pair(pos < se.z ? d : 0.f, pos < se.w ? g : 0.f));
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.s_empty[sb]);
        }
        if (t->nrb > 2 && lane == 0) mbar_arrive(&bars.q_empty[buf]);
      }
      if (!own) continue;
      const float sum = halves(sum2).x + halves(sum2).y;
      // The halves' sums join in shared memory, four tiles of the group in turn: the products of the fourth one on wait
      // for both halves to be done with the second one on.
      const int turn = kt >> 1 & 3;
      uint64_t* const there = &bars.half[group][warp & 3][turn];
      float* const other = halves_sum[group][turn] + r;
      if (half == 1) {
        *other = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(there);
        continue;
      }
      wait(there, kt >> 3 & 1);
      if (vg >= 0) {
        const float all = sum + *other;
        p.out[(size_t)vg * kGroup + (pos & 15)] = old ? fmaf(p.decay, was, all) : all;
      }
    }
  }
  __syncthreads();
  if (warp == C::EW + C::DW + C::QW) tmem_free(tmem, 512);
}

}  // namespace kvq
}  // namespace dec
