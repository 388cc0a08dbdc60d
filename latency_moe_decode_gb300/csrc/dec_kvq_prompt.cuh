// Attention over the paged 4-bit cache for many query rows (prompt chunks).
//
// Work that the tensor cores bound: 4 hd flops per (query row, position), each position's codes
// turned into operands once per 128 query rows. A CTA takes a stretch of (unit, tile of 128
// positions) entries, a unit being (sequence, KV head, 128 query rows), with a role for each warp:
//  - one copies the tiles' codes (bulk copies, four tiles ahead);
//  - six turn them into f16 in the 128-byte swizzled layout that the MMAs read, half a group at a time
//    (four warps: 2.5 k cycles a tile, more than any other role; with these six, 16 warps fill the
//    registers). A word of codes gives pairs (i, i + 4), and nothing puts them in order: the queries are staged in the same
//    order, and the outputs' columns are put right when they are written;
//  - one thread issues S = Q K^T (128 x 128 x hd, two S buffers in tensor memory) and O += P V
//    (128 x hd x 128, V read MN-major), the next tile's S before this tile's O. Q and P are A operands
//    in tensor memory: shared memory then carries the codes, K and V only (with all four there its
//    bandwidth held a tile to 2.9 k cycles);
//  - eight hold half a query row a thread: its 64 scores stay in registers from the maximum (joined
//    with the other half's) through the exponentials to P, f16 in tensor memory (11 bits, as in the kernel for
//    few rows; there is no room for a second half of each). The reference of the
//    exponentials follows the maximum only when that passes it by 2^8 (O lies in tensor memory, and
//    rescaling it costs as much as the exponentials). With whole rows and two reads of the scores, four
//    warps took 6.7 k cycles a tile for this; the exponentials' own floor is 1 k.
// Measured (32 query, 8 KV heads of 128): 2 chunks of 256 rows on 4 k 58 us, 600 TFLOP/s; 2048 rows on 2 k
// 180 us. A tile takes 2.6 k cycles, 1 k of them on the tensor cores; softmax is busy for 1.8 k (0.9 k of
// exponentials in all warps at once), decoding for 2 k; issue slots are 60 % full. Issuing whichever of the
// next scores and the outputs is ready first changed nothing. A unit's begin and end take 10 k cycles more.
#pragma once
#include "dec_f32x2.cuh"
#include "dec_kvq_attn.cuh"

namespace dec {
namespace kvq {

constexpr int kTile = 128;           // positions per tile
constexpr int kPromptStages = 4;     // tiles of codes in the ring
constexpr int kPromptCost = 5;       // a unit's fixed cost, in tiles' time (1: 128 sequences of 8 rows on 300, 88 us; 5: 78)
constexpr int kSplitCost = 8;        // what parts that have to be joined cost, in tiles' time
constexpr float kPromptShift = 7.0f; // P is kept times 2^7 (at most 2^15 with the reference's slack of 2^8)

template <int HD>
struct PromptCfg {
  static constexpr int ROWS = 128;
  static constexpr int DW = 6;                         // warps that decode
  static constexpr int THREADS = (8 + DW + 2) * 32;  // 8 softmax, DW decode, MMA, copy: 128 registers each
  static constexpr int HP = HD / 64;       // 64-value parts of a head
  static constexpr int OPERAND = HP * 16384;
  static constexpr int RAW = kTile / kGroup * group_bytes(HD);
  static constexpr int K = 0, V = 2 * OPERAND, RING = 4 * OPERAND;
  // tensor memory columns: two S, O, Q and P (two f16 a column)
  static constexpr int TS = 0, TO = 256, TQ = 384, TP = 448;
  static constexpr int TABLE = RING + kPromptStages * RAW;
  static constexpr int PART = ROWS * HD + 2 * ROWS;
  static constexpr int smem() { return TABLE + kMaxSeqs * (int)sizeof(SeqWork) + 1024; }
};

struct PromptBars {
  uint64_t raw_full[kPromptStages], raw_empty[kPromptStages];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full, pv_done, q_full;
};

// Instruction descriptor of kind::f16 with f16 A (K-major) and B and an fp32 D of shape M x N; B K-major
// or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&d)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "f"(d[0]), "f"(d[1]), "f"(d[2]), "f"(d[3]), "f"(d[4]), "f"(d[5]), "f"(d[6]), "f"(d[7]), "f"(d[8]), "f"(d[9]),
      "f"(d[10]), "f"(d[11]), "f"(d[12]), "f"(d[13]), "f"(d[14]), "f"(d[15]), "f"(d[16]), "f"(d[17]), "f"(d[18]),
      "f"(d[19]), "f"(d[20]), "f"(d[21]), "f"(d[22]), "f"(d[23]), "f"(d[24]), "f"(d[25]), "f"(d[26]), "f"(d[27]),
      "f"(d[28]), "f"(d[29]), "f"(d[30]), "f"(d[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* d) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "r"(d[0]), "r"(d[1]), "r"(d[2]), "r"(d[3]), "r"(d[4]), "r"(d[5]), "r"(d[6]), "r"(d[7]), "r"(d[8]), "r"(d[9]),
      "r"(d[10]), "r"(d[11]), "r"(d[12]), "r"(d[13]), "r"(d[14]), "r"(d[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B^T for one K = 16 slice of f16 operands: row r of A in lane r, two values a
// column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A CTA's stretch of one unit, as every role walks them.
struct Stretch {
  SeqWork sw;
  uint32_t uid;  // the unit's first entry
  int b, h, row0, t0, t1;  // sequence, KV head, first query row, tiles [t0, t1) (none where no row sees them)
  int smin, smax;       // positions that every row, and that some row sees
  uint32_t next;        // entry to go on from
  __device__ __forceinline__ bool find(const AttnParams& p, const SeqWork* seqs, uint32_t f, uint32_t end) {
    for (;;) {
      if (f >= end) return false;
      b = seq_of_entry(seqs, p.s.batch, f);
      sw = seqs[b];
      const uint32_t per = sw.ng + kPromptCost;
      const int u = (int)fast_div(f - sw.pre, per, sw.inv);
      uid = sw.pre + (uint32_t)u * per;
      if (f >= uid + sw.ng) {  // behind the unit's tiles
        f = uid + per;
        continue;
      }
      h = over(u, sw.nrb);
      row0 = (u - h * sw.nrb) * 128;
      const int last = min(row0 + 128, sw.n * p.group) - 1;
      smin = max(0, p.causal ? sw.len + (int)fast_div(row0, p.group, p.ginv) + 1 : sw.len);
      smax = max(0, p.causal ? sw.len + (int)fast_div(last, p.group, p.ginv) + 1 : sw.len);
      t0 = (int)(f - uid);
      const uint32_t stop = min(end, uid + sw.ng);
      t1 = min((int)(stop - uid), (smax + kTile - 1) / kTile);
      next = stop;
      return true;
    }
  }
};

template <int HD>
__global__ void __launch_bounds__(PromptCfg<HD>::THREADS, 1) prompt_kernel(const AttnParams p) {
  using C = PromptCfg<HD>;
  extern __shared__ uint8_t dyn[];
  __shared__ PromptBars bars;
  __shared__ uint32_t sh_scan[C::THREADS / 32], tmem_base;
  __shared__ float xm[2][2][128], xl[2][128];  // rows' maxima and sums, of each half
  __shared__ int nan_from[HD / kBlock];  // the first position with a NaN run of values, where rows differ in what they see
  uint8_t* const smem = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
  SeqWork* const seqs = reinterpret_cast<SeqWork*>(smem + C::TABLE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the join kernel waits for this one's end)
  if (tid == 0) {
    for (int i = 0; i < kPromptStages; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], C::DW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.k_full[i], C::DW);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], C::DW);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_empty[i], 8);
    }
    mbar_init(&bars.p_full, 8);
    mbar_init(&bars.pv_done, 1);
    mbar_init(&bars.q_full, 8);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8 + C::DW) tmem_alloc(&tmem_base, 512);
  tc_fence_before();
  __shared__ uint32_t units, longest;
  if (tid == 0) units = longest = 0;
  const uint32_t W = build_list<C::THREADS, C::ROWS, kTile, kPromptCost>(p, seqs, sh_scan);
  for (int b = tid; b < p.s.batch; b += C::THREADS) {
    if (seqs[b].nrb == 0) continue;
    atomicAdd(&units, (uint32_t)p.c.hkv * seqs[b].nrb);
    atomicMax(&longest, (uint32_t)seqs[b].ng + kPromptCost);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  // A CTA a unit where that takes no longer than an even cut, whose parts have to be written and joined
  // (about kSplitCost tiles' time); with units of one length the cut then falls between them.
  const int cta = blockIdx.x;
  const int ctas = (int)(units <= gridDim.x && longest <= W / gridDim.x + kSplitCost ? units : min((uint32_t)gridDim.x, W));
  uint32_t clo = 0, chi = 0;
  if (cta < ctas) {
    clo = (uint32_t)((unsigned long long)W * cta / ctas);
    chi = (uint32_t)((unsigned long long)W * (cta + 1) / ctas);
  }
  bool ok = true;  // (false after a wait that ran out: the thread waits no more and runs to its end)
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (ok && !bar_wait(b, parity)) {
      ok = false;
      raise(p.c.status, DEC_ERR_TIMEOUT);
    }
  };
  Stretch s;

  if (warp == 9 + C::DW) {
    // ---- copies: lane i the tile's group i
    int n = 0;
    for (uint32_t f = clo; s.find(p, seqs, f, chi); f = s.next) {
      const int gpp = 1 << (p.c.page_shift - 4);
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int st = n % kPromptStages, pos = t * kTile + lane * kGroup;
        int gi = -1;
        if (lane < kTile / kGroup && pos < s.smax) {
          const int e = pos >> p.c.page_shift;
          const int page = e < p.s.max_pages ? __ldg(p.s.table + s.b * p.s.table_stride + e) : -1;
          if ((unsigned)page < (unsigned)p.c.n_pages) gi = (page * p.c.hkv + s.h) * gpp + ((pos >> 4) & (gpp - 1));
          else raise(p.c.status, DEC_ERR_ARG);
        }
        if (n >= kPromptStages) wait(&bars.raw_empty[st], (n / kPromptStages - 1) & 1);
        const uint32_t who = __ballot_sync(0xffffffffu, gi >= 0);
        if (lane == 0) mbar_arrive_expect_tx(&bars.raw_full[st], __popc(who) * group_bytes(HD));
        __syncwarp();
        if (gi >= 0)
          bulk_copy(smem + C::RING + st * C::RAW + lane * group_bytes(HD), p.c.pages + (size_t)gi * group_bytes(HD),
                    group_bytes(HD), &bars.raw_full[st]);
      }
    }
    for (int i = max(0, n - kPromptStages); i < n; ++i) bar_wait(&bars.raw_full[i % kPromptStages], (i / kPromptStages) & 1);
  } else if (warp == 8 + C::DW) {
    // ---- products
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_f16_f32(128, 128, false), kIdO = idesc_f16_f32(128, HD, true);
      int n = 0, seg = 0;  // tiles, stretches so far
      auto scores = [&](int i) {  // of tile i
        wait(&bars.k_full[i & 1], (i >> 1) & 1);
        if (i >= 2) wait(&bars.s_empty[i & 1], ((i >> 1) - 1) & 1);
        tc_fence_after();
        const uint8_t* k = smem + C::K + (i & 1) * C::OPERAND;
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) {
          const int at = (d >> 2) * 16384 + (d & 3) * 32;
          mma_f16_ts(tmem + C::TS + (i & 1) * 128, tmem + C::TQ + d * 8, smem_desc_sw128(k + at, 16, 1024), kIdS,
                     d > 0 ? 1u : 0u);
        }
        mma_commit(&bars.s_full[i & 1]);
        mma_commit(&bars.k_empty[i & 1]);
      };
      for (uint32_t f = clo; s.find(p, seqs, f, chi); f = s.next) {
        const int tiles = s.t1 - s.t0;
        if (tiles <= 0) continue;
        wait(&bars.q_full, seg & 1);
        ++seg;
        tc_fence_after();
        scores(n);
        for (int i = 0; i < tiles; ++i, ++n) {
          if (i + 1 < tiles) scores(n + 1);
          wait(&bars.v_full[n & 1], (n >> 1) & 1);
          wait(&bars.p_full, n & 1);
          tc_fence_after();
#pragma unroll
          for (int d = 0; d < kTile / 16; ++d)
            mma_f16_ts(tmem + C::TO, tmem + C::TP + d * 8,
                       smem_desc_sw128(smem + C::V + (n & 1) * C::OPERAND + d * 2048, 16384, 1024), kIdO,
                       i > 0 || d > 0 ? 1u : 0u);
          mma_commit(&bars.pv_done);
          mma_commit(&bars.v_empty[n & 1]);
        }
      }
      if (n > 0) bar_wait(&bars.pv_done, (n - 1) & 1);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---- codes to operands: 16 bytes of codes (four words) at a time, in an order that spreads the
    // 16-byte stores of eight lanes over all banks
    // Chunk c (16 bytes) of row r of an operand lies at r 128 + ((c ^ r % 8) << 4): with a lane's first
    // address a, the others are a ^ (constant << 4) and a + constant rows.
    // Half a group (8 positions) at a time, the warps in turn; those with fewer of a tile's keys have more
    // of its values.
    const int kw = warp - 8, vw = kw >= 4 ? kw - 4 : kw + 2;
    const Magic magic = p.magic;
    const uint32_t sm = smem_u32(smem);
    int n = 0, seg = 0;
    auto put = [&](uint32_t at, uint32_t w, const Scale2& sc) {
      uint32_t a, b, c, d;
      sc.decode(w, magic, a, b);
      sc.decode(w >> 8, magic, c, d);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
    };
    // keys: lane bits t's low bit, g's two low bits, t's high bit, g's high bit
    const int kt = (lane & 1) | ((lane >> 3) & 1) << 1, kg = ((lane >> 1) & 3) | ((lane >> 4) & 1) << 2;
    const int kc = kt * (HD / 32);  // the lane's first chunk
    const uint32_t ka = sm + C::K + kg * 128 + (kc >> 3) * 16384 + (((kc & 7) ^ kg) << 4);
    auto keys = [&](int i) {  // of tile i
      const int st = i % kPromptStages;
      wait(&bars.raw_full[st], (i / kPromptStages) & 1);
      if (i >= 2) wait(&bars.k_empty[i & 1], ((i >> 1) - 1) & 1);
      const uint8_t* const from = smem + C::RING + st * C::RAW;
      const uint32_t to = ka + (i & 1) * C::OPERAND;
#pragma unroll
      for (int x = 0; x < (16 + C::DW - 1) / C::DW; ++x) {
        const int hg = kw + x * C::DW, y = hg & 1;
        if (hg >= 16) break;
        const uint8_t* const gp = from + (hg >> 1) * group_bytes(HD);
        const uint32_t at = to + hg * 1024;
        Scale2 s0, s1;
        if (HD == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(gp + y * 512 + (kg * 4 + kt) * 16);
          const uint32_t sb = *reinterpret_cast<const uint16_t*>(gp + 2 * code_bytes(HD) + (kg * 4 + kt) * 4 + y * 2);
          s0.set(__byte_perm(sb, 0, 0x4040));
          s1.set(__byte_perm(sb, 0, 0x4141));
          put(at, u.x, s0);
          put(at ^ 16, u.y, s0);
          put(at ^ 32, u.z, s1);
          put(at ^ 48, u.w, s1);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(gp + (kg * 4 + kt) * 16 + y * 8);
          const uint32_t sb = gp[2 * code_bytes(HD) + (kg * 4 + kt) * 2 + y];
          s0.set(__byte_perm(sb, 0, 0x4040));
          put(at, u.x, s0);
          put(at ^ 16, u.y, s0);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.k_full[i & 1]);
    };
    // values: lane bits the run's two low bits, t's low bit, t's high bit, the run's high bit; lanes of odd
    // t (hd 128) take their second position first
    const int vg = (lane & 3) | ((lane >> 4) & 1) << 2, vt = (lane >> 2) & 3, odd = HD == 128 ? vt & 1 : 0;
    const int vc = vg * (HD / 64), vr = 2 * vt + odd;  // the lane's first chunk and row
    const uint32_t va = sm + C::V + vr * 128 + (vc >> 3) * 16384 + (((vc & 7) ^ vr) << 4);
    for (uint32_t f = clo; s.find(p, seqs, f, chi); f = s.next) {
      if (s.t0 < s.t1) {
        keys(n);
        wait(&bars.q_full, seg++ & 1);  // (the stretch's nan_from is set)
      }
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int st = n % kPromptStages;
        if (t + 1 < s.t1) keys(n + 1);  // (the next tile's scores wait for nothing else)
        if (n >= 2) wait(&bars.v_empty[n & 1], ((n >> 1) - 1) & 1);
        const uint8_t* const from = smem + C::RING + st * C::RAW + code_bytes(HD);
        const uint32_t to = va + (n & 1) * C::OPERAND;
#pragma unroll
        for (int x = 0; x < (16 + C::DW - 1) / C::DW; ++x) {
          const int hg = vw + x * C::DW, y = hg & 1;
          if (hg >= 16) break;
          const uint8_t* const gp = from + (hg >> 1) * group_bytes(HD);
          const uint32_t at = to + hg * 1024;
          // scales of positions 2t and 2t + 1 of the half
          uint32_t sb = *reinterpret_cast<const uint16_t*>(gp + code_bytes(HD) + scale_bytes(HD) +
                                                           ((HD == 128 ? vg : vg >> 1) * 4 + vt) * 4 + y * 2);
          if ((t + 1) * kTile > s.smin) {
            // what no row sees counts nothing (scale 0); a run of NaNs that only some rows see is noted,
            // and put into their outputs at the end (0 x NaN is NaN: P cannot leave it out)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pos = t * kTile + hg * 8 + 2 * vt + e;
              const bool bad = ((sb >> (8 * e)) & 255u) == 255u;
              if (bad && pos < s.smax) atomicMin(&nan_from[HD == 128 ? vg : vg >> 1], pos);
              if (bad || pos >= s.smax) sb &= ~(255u << (8 * e));
            }
          }
          Scale2 s0, s1;
          if (HD == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(gp + y * 512 + (vg * 4 + vt) * 16);
            s0.set(__byte_perm(sb, 0, odd ? 0x4141 : 0x4040));
            s1.set(__byte_perm(sb, 0, odd ? 0x4040 : 0x4141));
            put(at, odd ? u.z : u.x, s0);
            put(at ^ 16, odd ? u.w : u.y, s0);
            put(at ^ 144, odd ? u.x : u.z, s1);  // (the row's last bit flips: 128, and the chunk's)
            put(at ^ 128, odd ? u.y : u.w, s1);
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(gp + (vg * 4 + vt) * 16 + y * 8);
            s0.set(__byte_perm(sb, 0, 0x4040));
            s1.set(__byte_perm(sb, 0, 0x4141));
            put(at, u.x, s0);
            put(at ^ 144, u.y, s1);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.v_full[n & 1]);
          mbar_arrive(&bars.raw_empty[st]);
        }
      }
    }
  } else {
    // ---- half a query row a thread: columns 64 half .. + 63 of S, HD / 2 half .. of O
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16), to = tl + C::TO + half * (HD / 2);
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(2 + (warp & 3)) : "memory"); };  // (both halves' warps)
    auto all_sync = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    int n = 0;
    int4 meta = make_int4(0, 0, 0, 0), mplace = make_int4(0, 0, 0, 0);
    for (uint32_t f = clo; s.find(p, seqs, f, chi); f = s.next) {
      const int row = s.row0 + r, rows = s.sw.n * p.group, tj = (int)fast_div(row, p.group, p.ginv);
      const bool live = row < rows;
      const long long tok = s.sw.tok0 + tj;
      const int head = s.h * p.group + row - tj * p.group;
      const int seen = live ? max(0, p.causal ? s.sw.len + tj + 1 : s.sw.len) : 0;
      if (tid < HD / kBlock) nan_from[tid] = 0x7FFFFFFF;
      // queries, scaled by a power of two to magnitude 1 .. 2 (f16 then holds bf16 values down to 2^-17
      // of the largest exactly), in the order in which a word of codes gives its values
      float sc;
      {
        uint4 u[HD / 16];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.p) + tok * p.q.ts + head * p.q.hs) +
                           half * (HD / 16);
        uint32_t mag = 0;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) u[i] = live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int y = 0; y < 4; ++y) mag = max(mag, max((w[y] << 16) & 0x7FFFFFFFu, w[y] & 0x7FFF0000u));
        }
        xm[0][half][r] = __uint_as_float(mag);
        pair_sync();
        mag = max(mag, __float_as_uint(xm[0][half ^ 1][r]));
        const int e = mag == 0 || mag >= 0x7F800000u ? 0 : min(126, max(-126, (int)(mag >> 23) - 127));
        const float down = __int_as_float((127 - e) << 23);
        sc = fmaxf(p.scale * __int_as_float((127 + e) << 23), 1e-37f);
        uint32_t qh[HD / 4];
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
          auto val = [&](int y) { return down * __uint_as_float((y & 1) ? w[y >> 1] & 0xFFFF0000u : w[y >> 1] << 16); };
#pragma unroll
          for (int y = 0; y < 4; ++y) qh[4 * i + y] = h2u(__floats2half2_rn(val(y), val(y + 4)));
        }
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) tmem_st16(tl + C::TQ + half * (HD / 4) + 16 * i, qh + 16 * i);
        tmem_st_wait();
        tc_fence_before();
      }
      const int tiles = s.t1 - s.t0;
      all_sync();  // (nan_from, and xm before the first tile's maxima)
      if (tiles > 0 && lane == 0) mbar_arrive(&bars.q_full);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < tiles; ++i, ++n) {
        const uint32_t ts = tl + C::TS + (n & 1) * 128 + half * 64;
        const int pos0 = (s.t0 + i) * kTile + half * 64;
        wait(&bars.s_full[n & 1], (n >> 1) & 1);
        tc_fence_after();
        float x[2][32];
        tmem_ld32(ts, x[0]);
        tmem_ld32(ts + 32, x[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_empty[n & 1]);
        if ((s.t0 + i + 1) * kTile > s.smin) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (pos0 + c * 32 + y >= seen) x[c][y] = -INFINITY;
        }
        float mx = -INFINITY, my = -INFINITY;
#pragma unroll
        for (int y = 0; y < 32; y += 2) {
          mx = fmaxf(mx, fmaxf(x[0][y], x[0][y + 1]));
          my = fmaxf(my, fmaxf(x[1][y], x[1][y + 1]));
        }
        mx = fmaxf(mx, my);
        xm[n & 1][half][r] = mx;
        pair_sync();
        mx = fmaxf(mx, xm[n & 1][half ^ 1][r]) * sc;
        const float was = m;
        if (m == -INFINITY || mx > m + 8.f) m = fmaxf(m, mx);
        const float z = (m == -INFINITY ? 0.f : m) - kPromptShift;
        uint32_t ph[32];
        uint64_t l2 = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int y = 0; y < 32; y += 2) {
            const float2 t = halves(fma2(pair(x[c][y], x[c][y + 1]), pair(sc, sc), pair(-z, -z)));
            const float a = ex2(t.x), b = ex2(t.y);
            l2 = add2(l2, pair(a, b));
            ph[c * 16 + y / 2] = h2u(__floats2half2_rn(a, b));
          }
        // the products so far are done before their operands, or O, are written again
        if (n > 0) wait(&bars.pv_done, (n - 1) & 1);
        if (i > 0 && __any_sync(0xffffffffu, m != was)) {
          const float fo = m == was ? 1.f : was == -INFINITY ? 0.f : ex2(was - m);
          l *= fo;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < HD / 64; ++c) {
            float o[32];
            tmem_ld32(to + c * 32, o);
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] *= fo;
            tmem_st32(to + c * 32, o);
          }
        }
        l += halves(l2).x + halves(l2).y;
        tmem_st16(tl + C::TP + half * 32, ph);
        tmem_st16(tl + C::TP + half * 32 + 16, ph + 16);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full);
      }
      // ---- the rows' outputs, or this CTA's part of them
      if (tiles > 0) wait(&bars.pv_done, (n - 1) & 1);
      tc_fence_after();
      xl[half][r] = l;
      pair_sync();
      l += xl[half ^ 1][r];
      const uint32_t u1 = s.uid + (uint32_t)s.sw.ng;
      const bool cont = s.uid < clo, open = u1 > chi;
      float* const part = p.parts + ((size_t)cta * 2 + (cont ? 0 : 1)) * C::PART;
      const float inv = l == 0.f ? 0.f : 8.0f / l;
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) {
        float x[32];
        if (tiles > 0) {
          tmem_ld32(to + c * 32, x);
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) x[y] = 0.f;
        }
        const int col = half * (HD / 2) + c * 32;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const bool nan = tiles > 0 && nan_from[(col >> 4) + (y >> 1)] < seen;  // (a run of 16 values)
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[(k >> 1) + 4 * (k & 1)] = nan ? NAN : x[8 * y + k];
          if (live && !cont && !open) {
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] *= inv;
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o.p) + tok * p.o.ts + head * p.o.hs + col + y * 8) = pack8_bf16(o);
          } else if (live) {
            float4* d = reinterpret_cast<float4*>(part + r * HD + col + y * 8);
            d[0] = make_float4(o[0], o[1], o[2], o[3]);
            d[1] = make_float4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      if (half == 0 && live) {
        if (!cont && !open) {
          if (p.lse) p.lse[tok * p.hq + head] = (m - kPromptShift + log2f(l)) * kLn2;
        } else {
          part[128 * HD + r] = m + (kPShift - kPromptShift);  // (the join takes sums as kept times 2^kPShift)
          part[128 * HD + 128 + r] = l;
        }
      }
      if (cont) meta.x = open ? 1 : 3;
      else if (open) {
        meta.y = 1;
        mplace = make_int4(s.sw.tok0, s.h * p.group, s.row0, rows);
      }
      tc_fence_before();
      all_sync();  // (nan_from is set anew)
    }
    if (tid == 0) {
      p.meta[2 * cta] = meta;
      p.meta[2 * cta + 1] = mplace;
    }
  }
  __syncthreads();
  if (warp == 8 + C::DW) tmem_free(tmem, 512);
}

}  // namespace kvq
}  // namespace dec
