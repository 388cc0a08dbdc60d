// Attention over the paged 4-bit cache for few query rows (decode and verify steps).
//
// The work is reading the cache once: 2 (hd / 2 + hd / 16) bytes per position and KV head against
// 4 hd flops per query head, so the kernel is built around the stream of groups (16 positions of
// one KV head) through each SM:
//  - a unit is (sequence, KV head, block of 8 NB query rows), a query row being (token, head of
//    the group); the groups of all units form one list, cut evenly over the CTAs and their warps
//    (lengths are read on the device: the cut needs no host knowledge and adapts to ragged batches);
//  - a warp streams its groups through its own ring with bulk copies, one a group, some chunks ahead,
//    without ever waiting for another warp;
//  - S^T = K q^T and O^T = V^T P^T are 16 x 8 x 16 f16 products whose A operand, the codes, comes
//    out of the ring in the lanes' own order: (code + 8) enters the low mantissa bits of the f16
//    1024, and one fma turns it into code * scale exactly (4 x 4 significant bits). Tensor memory
//    has nothing to offer here: 8 columns of queries leave the tensor cores mostly idle, and the
//    codes would have to be written to shared memory again for tcgen05 to read them;
//  - probabilities go from the first product's result layout to the second's operand layout by
//    movmatrix, rounded to f16 on the way: 11 bits where the bf16 output keeps 8. Two f16 a probability
//    (22 bits) and a second product took 16 sequences of 8 k to 32 k from 80 to 89 us and left the output's
//    error against 64 bits at 0.0017. The running maximum, the sum (of unrounded terms) and the output stay in
//    fp32 registers;
//  - what a warp leaves unfinished of a unit is joined per CTA in shared memory, and what a CTA
//    leaves unfinished by a second small kernel, both in a fixed order.
// Measured (32 query, 8 KV heads of 128, one row a sequence): 16 sequences of 8 k to 32 k
// 80 us (4.5 TB/s; issue slots 62 % full, ALU pipe 51 %: neither binds, but scores, maximum, exponentials and
// values of a chunk are one chain of dependent instructions a warp, four warps a scheduler); 64 of up to 2 k and one of 64 k 29 us, of which 14 are
// the stream and 15 are fixed: list and page table 3, a unit's queries 3, the first chunk's code and
// data 3, joins 6. Cutting the joins' dependent loads to one round did not shorten them.
#pragma once
#include <type_traits>

#include "dec_kvq.cuh"
#include "dec_prims.cuh"

namespace dec {
namespace kvq {

constexpr int kStages = 3;       // chunks of a warp's ring
constexpr int kMaxSeqs = 256;    // sequences of one launch (their table lies in shared memory)
constexpr int kUnitCost = 2;     // what beginning and ending a unit costs, in groups' time
constexpr int kMinGroups = 8;    // groups a CTA takes at least
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPShift = 15.0f;  // probabilities are kept times 2^15: f16 then reaches 2^-39 of the largest


// The f16 pairs 1024, 1024 and 64, 64 that codes are put into (Scale2), from the kernel's arguments:
// with constants the compiler makes an and and an or of each lop3, 64 more a group on the pipe that
// bounds the kernel.
struct Magic {
  uint32_t lo, hi;
};
// A sequence's share of the list: hkv * (row blocks) units of ng groups and kUnitCost entries more
// that stand for a unit's fixed cost (skipped: they only even out the cut where contexts are short).
struct SeqWork {
  uint32_t pre;  // first list entry
  int tok0, n, len, ng;
  uint32_t inv;  // reciprocal of ng + kUnitCost
  int nrb, pad;
};
template <int HD, int NB>
struct AttnCfg {
  static constexpr int KS = HD / 16;              // 16-value steps of a head
  static constexpr int WARPS = NB == 1 ? 16 : 8;  // registers: 128 or 255 a thread
  static constexpr int CH = NB == 1 ? 2 : 4;      // groups per softmax update
  static constexpr int ROWS = 8 * NB;
  static constexpr int GB = group_bytes(HD);
  static constexpr int RING = kStages * CH * GB;  // bytes per warp
  static constexpr int PART = ROWS * HD + 2 * ROWS;  // floats of a partial: outputs, maxima, sums
  static constexpr int THREADS = WARPS * 32;
  static_assert(RING >= PART * 4 && RING % 16 == 0 && GB % 16 == 0, "a partial has to fit into a warp's ring");
  static constexpr int smem() { return WARPS * RING + kMaxSeqs * (int)sizeof(SeqWork); }
};

struct AttnParams {
  Cache c;
  Seqs s;
  Rows q, o;
  float* lse;
  float scale;  // times log2(e) and the scale bytes' factor 8
  int hq, group, causal, max_tokens;
  uint32_t ginv;  // reciprocal of group
  int b0;         // (without cu: token row of sequence 0)
  int min_groups; // groups a CTA takes at least
  Magic magic;
  float* parts;   // [CTA][2] partials
  float* wparts;  // [CTA][warp] partials
  int4* meta;     // [CTA][2]: unit continued (1) and finished here (2), unit left open | the open unit's place
};

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* b) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(b))
               : "memory");
}
// Wait for the barrier's phase; false after a second (copies and products always end: this only keeps
// a mistake from holding the GPU).
static __device__ __noinline__ bool bar_wait_long(uint64_t* b, uint32_t parity) {
  const unsigned long long t0 = gtimer();
  for (unsigned i = 1;; ++i) {
    if (mbar_try_wait(b, parity)) return true;
    if ((i & 63u) == 0 && gtimer() - t0 > 1000000000ull) return false;
  }
}
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity) {
  return mbar_try_wait(b, parity) || bar_wait_long(b, parity);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Two scales (an f16 pair) and what turns codes into code * s. A code + 8 = u in the low 4 bits of
// the f16 1024 is 1024 + u, in the next 4 bits of the f16 64 it is 64 + u; (1024 + u) s - 1032 s and
// (64 + u) s - 72 s are exact, being u - 8 and s of 4 significant bits each, and so are the addends:
// 1032 = 129 * 8, 72 = 9 * 8, and 1032 * 60 is still an f16.
struct Scale2 {
  __half2 s, c, c16;
  __device__ __forceinline__ void set(uint32_t two) {  // scale bytes in the low bytes of the halves
    s = u2h(two << 7);
    c = __hmul2(s, __float2half2_rn(-1032.0f));
    c16 = __hmul2(s, __float2half2_rn(-72.0f));
  }
  // nibbles 0 and 1 of both halves of x
  __device__ __forceinline__ void decode(uint32_t x, const Magic& m, uint32_t& n0, uint32_t& n1) const {
    uint32_t y, z;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(y) : "r"(x), "r"(m.lo));
    asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(z) : "r"(x), "r"(m.hi));
    n0 = h2u(__hfma2(u2h(y), s, c));
    n1 = h2u(__hfma2(u2h(z), s, c16));
  }
};

// x / d by the reciprocal inv = floor((2^32 - 1) / d): x inv / 2^32 is less than 1 below x / d, so the
// quotient is at most one too small before the correction.
__device__ __forceinline__ uint32_t fast_div(uint32_t x, uint32_t d, uint32_t inv) {
  const uint32_t q = __umulhi(x, inv);
  return q + (x - q * d >= d ? 1u : 0u);
}
// (no division for the common single row block)
__device__ __forceinline__ int over(int a, int d) { return d == 1 ? a : a / d; }
__host__ __device__ inline uint32_t reciprocal(uint32_t d) { return 0xFFFFFFFFu / d; }

// The list's table in shared memory, by the whole CTA: units of ROWS query rows, entries of POS positions.
// Returns the number of entries. Token bounds that do not ascend leave nothing to do: sequences that share rows
// could make more entries than the call was checked for.
template <int THREADS, int ROWS, int POS, int COST>
__device__ uint32_t build_list(const AttnParams& p, SeqWork* seqs, uint32_t* scan) {
  static_assert(THREADS >= kMaxSeqs, "a thread for every sequence");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = tid;
  uint32_t w = 0;
  bool wrong = false;
  SeqWork sw;
  if (b < p.s.batch) {
    const int first = p.s.cu ? __ldg(p.s.cu + b) : p.b0 + b, last = p.s.cu ? __ldg(p.s.cu + b + 1) : first + 1;
    wrong = first < 0 || last < first;
    const int len = __ldg(p.s.lengths + b);
    const long long most = (long long)p.s.max_pages << p.c.page_shift;
    sw.tok0 = max(first, 0);
    sw.n = max(0, min(min(last - first, p.max_tokens), p.s.n_tokens - sw.tok0));
    if (sw.n > 0 && len < 0) raise(p.c.status, DEC_ERR_ARG);
    if (sw.n > 0 && (p.causal ? (long long)len + sw.n : len) > most) raise(p.c.status, DEC_ERR_CAPACITY);
    sw.len = len < 0 ? -sw.n : (int)min((long long)len, most);
    // (a unit without positions still writes its rows)
    const int held = (int)min(most, (long long)(p.causal ? sw.len + sw.n : sw.len));
    sw.ng = max(1, (held + POS - 1) / POS);
    sw.inv = reciprocal(sw.ng + COST);
    sw.nrb = (sw.n * p.group + ROWS - 1) / ROWS;
    w = (uint32_t)p.c.hkv * sw.nrb * (sw.ng + COST);
  }
  uint32_t x = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[warp] = x;
  wrong = __syncthreads_or(wrong);
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const uint32_t y = scan[i];
    before += i < warp ? y : 0u;
    all += y;
  }
  if (wrong) {
    if (tid == 0) raise(p.c.status, DEC_ERR_ARG);
    all = sw.nrb = 0;
  }
  if (b < p.s.batch) {
    sw.pre = before + x - w;
    seqs[b] = sw;
  }
  __syncthreads();
  return all;
}

// the sequence that entry f of the list belongs to
__device__ __forceinline__ int seq_of_entry(const SeqWork* seqs, int batch, uint32_t f) {
  int a = 0, z = batch;
  while (z - a > 1) {
    const int m = (a + z) >> 1;
    if (seqs[m].pre <= f) a = m;
    else z = m;
  }
  return a;
}

// The operands of O^T's products with a group's values (vw: the lane's words of positions 2t, 2t + 1,
// 2t + 8, 2t + 9; bytes: their scales): put(k, a0..a3) for 16 values of the head at a time, of which
// the lane's are 2k and 2k + 1 of its run.
template <int HD, class F>
__device__ __forceinline__ void v_product(const uint32_t (&vw)[4][HD / 64], uint32_t bytes, const Magic& magic, F&& put) {
  Scale2 s0, s1;
  s0.set(__byte_perm(bytes, 0, 0x4140));
  s1.set(__byte_perm(bytes, 0, 0x4342));
#pragma unroll
  for (int w = 0; w < HD / 64; ++w)
#pragma unroll
    for (int x = 0; x < 2; ++x) {  // values 4 x .. 4 x + 3 of the word, positions paired
      const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], x ? 0x7632 : 0x5410);
      const uint32_t x1 = __byte_perm(vw[2][w], vw[3][w], x ? 0x7632 : 0x5410);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t a0, a1, a2, a3;
        s0.decode(y ? x0 >> 8 : x0, magic, a0, a1);
        s1.decode(y ? x1 >> 8 : x1, magic, a2, a3);
        put(4 * w + 2 * x + y, a0, a1, a2, a3);
      }
    }
}

// The same with each query row by itself, the positions it does not see left out.
template <int HD, int NB>
struct RowsApart {
  float acc[NB][HD / 16][4];
  uint32_t pb[NB][2];
  int seen[NB][2];
  __device__ __noinline__ void add(const uint32_t (&vw)[4][HD / 64], uint32_t sb, const Magic& magic, int pos0) {
    const int t = threadIdx.x & 3;
    for (int c = 0; c < 8 * NB; ++c) {
      int mine = 0;  // what row c sees
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int s0 = __shfl_sync(0xffffffffu, seen[nb][0], (c & 7) >> 1);
        const int s1 = __shfl_sync(0xffffffffu, seen[nb][1], (c & 7) >> 1);
        if (c >> 3 == nb) mine = (c & 1) ? s1 : s0;
      }
      uint32_t mb = sb;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (pos0 + 2 * t + (k & 1) + (k >> 1) * 8 >= mine) mb &= ~(0xFFu << (8 * k));
      v_product<HD>(vw, mb, magic, [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float d[4] = {acc[nb][k][0], acc[nb][k][1], acc[nb][k][2], acc[nb][k][3]};
          mma16816(d, a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
          if (c == nb * 8 + 2 * t) {
            acc[nb][k][0] = d[0];
            acc[nb][k][2] = d[2];
          }
          if (c == nb * 8 + 2 * t + 1) {
            acc[nb][k][1] = d[1];
            acc[nb][k][3] = d[3];
          }
        }
      });
    }
  }
};

// A unit's place: {first token row of its sequence, first query head, first query row, rows of the
// sequence}. A row of it being joined from parts, HD / 32 values a lane.
template <int HD>
struct Joined {
  static constexpr int V = HD / 32;
  float M, L, w, a[V];  // the joined maximum and sum; the lane's part's weight; outputs
  // parts' maxima and sums, one per lane (none: -infinity, 0). A part of NaNs (its maximum is
  // -infinity, its sum NaN) makes the sum NaN.
  __device__ __forceinline__ void weigh(float m, float l) {
    M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    w = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - M);
    L = l * w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 0.f;
  }
  __device__ __forceinline__ void load(const float* part, int lane, float (&x)[V]) const {
    if (V == 4) {
      const float4 f = *reinterpret_cast<const float4*>(part + lane * 4);
      x[0] = f.x; x[1] = f.y; x[V - 2] = f.z; x[V - 1] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(part + lane * 2);
      x[0] = f.x; x[1] = f.y;
    }
  }
  __device__ __forceinline__ void mul(const float (&x)[V], float wt) {
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = fmaf(x[i], wt, a[i]);
  }
  __device__ __forceinline__ void add(const float* part, float wt, int lane) {
    float x[V];
    load(part, lane, x);
    mul(x, wt);
  }
  __device__ __forceinline__ void join(const Joined& o) {
    const float mn = fmaxf(M, o.M);
    const float fa = M == -INFINITY ? (L == 0.f ? 0.f : 1.f) : ex2(M - mn);
    const float fo = o.M == -INFINITY ? (o.L == 0.f ? 0.f : 1.f) : ex2(o.M - mn);
    M = mn;
    L = L * fa + o.L * fo;
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = a[i] * fa + o.a[i] * fo;
  }
  __device__ __forceinline__ void keep(float* part, int lane) const {
#pragma unroll
    for (int i = 0; i < V; ++i) part[lane * V + i] = a[i];
  }
  __device__ __forceinline__ void store(const AttnParams& p, const int4& place, int row, int lane) const {
    const int rr = place.z + row, tj = (int)fast_div(rr, p.group, p.ginv);
    const long long tok = place.x + tj;
    const int head = place.y + rr - tj * p.group;
    const float inv = L == 0.f ? 0.f : 8.0f / L;  // (8: the scale bytes' factor)
    __nv_bfloat162* dst =
        reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(p.o.p) + tok * p.o.ts + head * p.o.hs + lane * V);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) dst[i] = __floats2bfloat162_rn(a[2 * i] * inv, a[2 * i + 1] * inv);
    if (p.lse && lane == 0) p.lse[tok * p.hq + head] = (M - kPShift + log2f(L)) * kLn2;
  }
};

template <int HD, int NB>
__global__ void __launch_bounds__(AttnCfg<HD, NB>::THREADS, 1) attention_kernel(const AttnParams p) {
  using K = AttnCfg<HD, NB>;
  constexpr int KS = K::KS, CH = K::CH;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t sh_scan[K::WARPS];
  // what the warps leave unfinished, in the list's order: two entries a warp (a unit it found begun, a
  // unit it left open). First and last + 1 list entry of the unit; its place
  __shared__ uint2 ent_unit[32];
  __shared__ int4 ent_place[32];
  __shared__ uint64_t bars[K::WARPS][kStages];  // chunk landed
  // each warp's unit, kept here while its groups take the registers: its place; its first list entry
  // and the one behind its groups
  __shared__ int4 unit_place[K::WARPS];
  __shared__ uint2 unit_span[K::WARPS];
  SeqWork* const seqs = reinterpret_cast<SeqWork*>(smem + K::WARPS * K::RING);  // [batch]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the join kernel waits for this one's end)

  // ---- the list's prefix sums over the sequences
  static_assert(2 * K::WARPS <= 32, "one entry per lane in the join");
  if (tid < 32) ent_unit[tid] = make_uint2(0u, 0u);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars[warp] + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const uint32_t W = build_list<K::THREADS, K::ROWS, kGroup, kUnitCost>(p, seqs, sh_scan);
  const int ctas = (int)min((uint32_t)gridDim.x, (W + p.min_groups - 1) / p.min_groups);
  const int cta = blockIdx.x;
  if (tid == 0) p.meta[2 * cta] = make_int4(0, 0, 0, 0);  // (before the barrier that the join's marks come after)
  uint32_t clo = 0, chi = 0;
  if (cta < ctas) {
    clo = (uint32_t)((unsigned long long)W * cta / ctas);
    chi = (uint32_t)((unsigned long long)W * (cta + 1) / ctas);
  }
  const uint32_t lo = clo + (uint32_t)((unsigned long long)(chi - clo) * warp / K::WARPS);
  const uint32_t hi = clo + (uint32_t)((unsigned long long)(chi - clo) * (warp + 1) / K::WARPS);

  auto seq_at = [&](uint32_t f) { return seq_of_entry(seqs, p.s.batch, f); };
  uint8_t* const ring = smem + warp * K::RING;

  // ---- the copies: 32 entries' group indices at a time, one per lane, and each lane copies its own
  // (one bulk copy a group: a group is contiguous)
  uint32_t pf = lo;    // next entry to copy
  int vg, vrem;        // group in the cache of entry (the 32 that pf is in) + lane (-1: nothing to copy),
                       // groups left of its unit
  auto look = [&](uint32_t f) {
    vg = -1;
    vrem = 0;
    if (f >= hi) return;
    const int b = seq_at(f);
    const SeqWork sw = seqs[b];
    const uint32_t r = f - sw.pre, per = sw.ng + kUnitCost;
    const int u = (int)fast_div(r, per, sw.inv), gr = (int)(r - (uint32_t)u * per);
    vrem = sw.ng - gr;
    const int pos = gr * kGroup;
    if (vrem > 0 && pos < (p.causal ? sw.len + sw.n : sw.len)) {
      const int page = __ldg(p.s.table + b * p.s.table_stride + (pos >> p.c.page_shift));
      const int gpp = 1 << (p.c.page_shift - 4);
      if ((unsigned)page < (unsigned)p.c.n_pages) vg = (page * p.c.hkv + over(u, sw.nrb)) * gpp + (gr & (gpp - 1));
      else raise(p.c.status, DEC_ERR_ARG);
    }
  };
  int pstage = 0;
  bool fresh = true;  // pf has come to the next 32
  auto prefetch = [&]() {  // the next chunk, if there is one
    int at, rem;
    for (;;) {
      if (pf >= hi) return;
      at = (int)((pf - lo) & 31u);
      if (fresh) look(pf - at + lane);
      fresh = false;
      rem = __shfl_sync(0xffffffffu, vrem, at);
      if (rem > 0) break;
      fresh = at + rem + kUnitCost >= 32;
      pf += rem + kUnitCost;  // to the next unit
    }
    // (chunks end with the unit, the warp's part of the list, and the 32 entries)
    const int n = min(min(CH, rem), min((int)(hi - pf), 32 - at));
    const bool copies = lane >= at && lane < at + n && vg >= 0;
    const uint32_t who = __ballot_sync(0xffffffffu, copies);
    uint64_t* const bar = bars[warp] + pstage;
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(who) * K::GB);
    __syncwarp();
    if (copies)
      bulk_copy(ring + (pstage * CH + lane - at) * K::GB, p.c.pages + (size_t)vg * K::GB, K::GB, bar);
    fresh = at + n == 32;
    pf += n;
    pstage = pstage == kStages - 1 ? 0 : pstage + 1;
  };

  float acc[NB][KS][4];
  float m[NB][2], l[NB][2], sc[NB][2];
  int seen[NB][2], smin, smax;
  uint32_t qf[NB][KS][2];

  // ---- the unit that an entry belongs to, and its rows' queries (loaded ahead of their use)
  uint32_t w[NB][KS * 2];  // the lane's HD / 4 values from t HD / 4 on of rows g, two a word
  auto open_unit = [&](uint32_t f) {  // -> the unit's first group from entry f on
    SeqWork sw = seqs[seq_at(f)];
    const uint32_t per = sw.ng + kUnitCost;
    int u = (int)fast_div(f - sw.pre, per, sw.inv);
    uint32_t uid = sw.pre + (uint32_t)u * per;
    if (f >= uid + sw.ng) {  // behind a unit's groups: the next unit, in the next sequence at its last
      f = uid + per;
      if (f >= hi) return f;
      sw = seqs[seq_at(f)];
      u = (int)fast_div(f - sw.pre, sw.ng + kUnitCost, sw.inv);
      uid = f;
    }
    const int h = over(u, sw.nrb), row0 = (u - h * sw.nrb) * K::ROWS, rows = sw.n * p.group;
    if (lane == 0) {
      unit_place[warp] = make_int4(sw.tok0, h * p.group, row0, rows);
      unit_span[warp] = make_uint2(uid, uid + sw.ng);
    }
    // positions that rows 2t, 2t + 1 see
    smin = 0x7FFFFFFF;
    smax = 0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = row0 + nb * 8 + 2 * t + i;
        const int x = max(0, p.causal ? sw.len + (int)fast_div(rr, p.group, p.ginv) + 1 : sw.len);
        seen[nb][i] = rr < rows ? x : 0;
        smin = min(smin, rr < rows ? x : 0x7FFFFFFF);
        smax = max(smax, seen[nb][i]);
      }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      smin = min(smin, __shfl_xor_sync(0xffffffffu, smin, o));
      smax = max(smax, __shfl_xor_sync(0xffffffffu, smax, o));
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = row0 + nb * 8 + g, tj = (int)fast_div(row, p.group, p.ginv);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.p) + (long long)(sw.tok0 + tj) * p.q.ts +
                                                        (h * p.group + row - tj * p.group) * p.q.hs + t * (HD / 4));
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint4 x = row < rows ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        w[nb][4 * i] = x.x; w[nb][4 * i + 1] = x.y; w[nb][4 * i + 2] = x.z; w[nb][4 * i + 3] = x.w;
      }
    }
    return f;
  };

  uint32_t f = lo < hi ? open_unit(lo) : hi;
  if (lo < hi) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) prefetch();
  }
  int cstage = 0;
  uint32_t cphase = 0;
  bool dead = false;
  const Magic magic = p.magic;
  while (f < hi && !dead) {
    // ---- a unit: its queries as the second operand of S^T, scaled to magnitude 1 .. 2
    __syncwarp();
    const uint32_t uid = unit_span[warp].x, fend = min(hi, unit_span[warp].y);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t mag = 0;
#pragma unroll
      for (int i = 0; i < KS * 2; ++i) mag = max(mag, max((w[nb][i] << 16) & 0x7FFFFFFFu, w[nb][i] & 0x7FFF0000u));
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
      // a power of two that leaves the row's largest value in 1 .. 2: bf16 values down to 2^-17 of it
      // are exact in f16, smaller ones lose at most 2^-25 of it
      const int e = mag == 0 || mag >= 0x7F800000u ? 0 : min(126, max(-126, (int)(mag >> 23) - 127));
      const float down = __int_as_float((127 - e) << 23);
      auto val = [&](int i) {  // value i of the lane's HD / 4
        return down * __uint_as_float((i & 1) ? (w[nb][i >> 1] & 0xFFFF0000u) : (w[nb][i >> 1] << 16));
      };
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int i = 8 * (s >> 1) + 2 * (s & 1);
        qf[nb][s][0] = h2u(__floats2half2_rn(val(i), val(i + 4)));
        qf[nb][s][1] = h2u(__floats2half2_rn(val(i + 1), val(i + 5)));
      }
      const float up = fmaxf(p.scale * __int_as_float((127 + e) << 23), 1e-37f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[nb][i] = __shfl_sync(0xffffffffu, up, (2 * t + i) * 4);
        m[nb][i] = -INFINITY;
        l[nb][i] = 0.f;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nb][s][i] = 0.f;
    }

    // ---- its groups, a chunk at a time: with every group there and seen by every row, or not
    auto chunk = [&](auto edge, const uint8_t* buf, int pos0, int n) {
      constexpr bool EDGE = decltype(edge)::value;
      float s[NB][CH][4];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[nb][i][j] = 0.f;
        if (!EDGE || i < n) {
          const uint8_t* gp = buf + i * K::GB;
          uint32_t k0[HD / 32], k1[HD / 32];  // words of positions g and g + 8
          uint32_t sb;
          if (HD == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(gp + lane * 16);
            const uint4 c = *reinterpret_cast<const uint4*>(gp + 512 + lane * 16);
            k0[0] = a.x; k0[1] = a.y; k0[HD / 32 - 2] = a.z; k0[HD / 32 - 1] = a.w;
            k1[0] = c.x; k1[1] = c.y; k1[HD / 32 - 2] = c.z; k1[HD / 32 - 1] = c.w;
            sb = *reinterpret_cast<const uint32_t*>(gp + 2 * code_bytes(HD) + lane * 4);
          } else {
            const uint4 a = *reinterpret_cast<const uint4*>(gp + lane * 16);
            k0[0] = a.x; k0[1] = a.y;
            k1[0] = a.z; k1[1] = a.w;
            sb = *reinterpret_cast<const uint16_t*>(gp + 2 * code_bytes(HD) + lane * 2);
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
            for (int v = 0; v < 2; ++v) {
              const int wi = 2 * w2 + v;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t a0, a1, a2, a3;
                s0.decode(y ? k0[wi] >> 8 : k0[wi], magic, a0, a2);
                s1.decode(y ? k1[wi] >> 8 : k1[wi], magic, a1, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816(s[nb][i], a0, a1, a2, a3, qf[nb][2 * wi + y][0], qf[nb][2 * wi + y][1]);
              }
            }
          }
        }
      }
      // what a row does not see is -infinity, whatever it held; maxima in units of log2
      uint32_t pb[NB][CH][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (EDGE) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (i >= n || pos0 + i * kGroup + g + (j >> 1) * 8 >= seen[nb][j & 1]) s[nb][i][j] = -INFINITY;
          }
          mx0 = fmaxf(mx0, fmaxf(s[nb][i][0], s[nb][i][2]));
          mx1 = fmaxf(mx1, fmaxf(s[nb][i][1], s[nb][i][3]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        mx0 = fmaxf(m[nb][0], mx0 * sc[nb][0]);
        mx1 = fmaxf(m[nb][1], mx1 * sc[nb][1]);
        if (__any_sync(0xffffffffu, mx0 > m[nb][0] || mx1 > m[nb][1])) {
          const float f0_ = m[nb][0] == -INFINITY ? 0.f : ex2(m[nb][0] - mx0);
          const float f1_ = m[nb][1] == -INFINITY ? 0.f : ex2(m[nb][1] - mx1);
          l[nb][0] *= f0_;
          l[nb][1] *= f1_;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            acc[nb][k][0] *= f0_;
            acc[nb][k][1] *= f1_;
            acc[nb][k][2] *= f0_;
            acc[nb][k][3] *= f1_;
          }
          m[nb][0] = mx0;
          m[nb][1] = mx1;
        }
        const float z0 = (mx0 == -INFINITY ? 0.f : mx0) - kPShift, z1 = (mx1 == -INFINITY ? 0.f : mx1) - kPShift;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const float e0 = ex2(fmaf(s[nb][i][0], sc[nb][0], -z0)), e1 = ex2(fmaf(s[nb][i][1], sc[nb][1], -z1));
          const float e2 = ex2(fmaf(s[nb][i][2], sc[nb][0], -z0)), e3 = ex2(fmaf(s[nb][i][3], sc[nb][1], -z1));
          l[nb][0] += e0 + e2;
          l[nb][1] += e1 + e3;
          pb[nb][i][0] = transpose8x8(h2u(__floats2half2_rn(e0, e1)));
          pb[nb][i][1] = transpose8x8(h2u(__floats2half2_rn(e2, e3)));
        }
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (EDGE && i >= n) continue;
        const uint8_t* gp = buf + i * K::GB + code_bytes(HD);
        uint32_t vw[4][HD / 64];  // words of positions 2t, 2t + 1, 2t + 8, 2t + 9
        uint32_t sb;
        if (HD == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(gp + lane * 16);
          const uint4 c = *reinterpret_cast<const uint4*>(gp + 512 + lane * 16);
          vw[0][0] = a.x; vw[0][HD / 64 - 1] = a.y; vw[1][0] = a.z; vw[1][HD / 64 - 1] = a.w;
          vw[2][0] = c.x; vw[2][HD / 64 - 1] = c.y; vw[3][0] = c.z; vw[3][HD / 64 - 1] = c.w;
          sb = *reinterpret_cast<const uint32_t*>(gp + code_bytes(HD) + scale_bytes(HD) + lane * 4);
        } else {
          const uint4 a = *reinterpret_cast<const uint4*>(gp + lane * 16);
          vw[0][0] = a.x; vw[1][0] = a.y; vw[2][0] = a.z; vw[3][0] = a.w;
          sb = *reinterpret_cast<const uint32_t*>(gp + code_bytes(HD) + scale_bytes(HD) + ((g >> 1) * 4 + t) * 4);
        }
        // what no row sees counts nothing, whatever is there: scale 0
        const int left = smax - (pos0 + i * kGroup);
        if (EDGE && left < kGroup) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (2 * t + (k & 1) + (k >> 1) * 8 >= left) sb &= ~(0xFFu << (8 * k));
        }
        // A run of NaNs at a position that some of the rows do not see (0 x NaN is NaN): each row by
        // itself, with the positions it does not see left out. Rows of one decode token all see
        // the same, and finite caches never come here.
        bool odd = false;
        if (EDGE && smin < smax) {
          const uint32_t x = ~sb;  // a byte of 255
          odd = __any_sync(0xffffffffu, ((x - 0x01010101u) & ~x & 0x80808080u) != 0);
        }
        if (!odd) {
          v_product<HD>(vw, sb, magic, [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(acc[nb][k], a0, a1, a2, a3, pb[nb][i][0], pb[nb][i][1]);
          });
        } else if constexpr (EDGE) {
          RowsApart<HD, NB> r;  // (a copy: the accumulators themselves stay in registers)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) r.acc[nb][k][j] = acc[nb][k][j];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              r.pb[nb][j] = pb[nb][i][j];
              r.seen[nb][j] = seen[nb][j];
            }
          }
          r.add(vw, sb, magic, pos0 + i * kGroup);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[nb][k][j] = r.acc[nb][k][j];
        }
      }
    };
    for (uint32_t f0 = f; f0 < fend;) {
      const int n = min(min(CH, (int)(fend - f0)), 32 - (int)((f0 - lo) & 31u));
      const int pos0 = (int)(f0 - uid) * kGroup;
      prefetch();
      if (!bar_wait(bars[warp] + cstage, cphase)) {
        raise(p.c.status, DEC_ERR_TIMEOUT);
        for (int i = 1; i < kStages; ++i) bar_wait(bars[warp] + (cstage + i) % kStages, i + cstage < kStages ? cphase : cphase ^ 1);
        dead = true;
        break;
      }
      const uint8_t* const buf = ring + cstage * CH * K::GB;
      if (++cstage == kStages) {
        cstage = 0;
        cphase ^= 1;
      }
      if (n < CH || pos0 + CH * kGroup > smin) chunk(std::true_type(), buf, pos0, n);
      else chunk(std::false_type(), buf, pos0, n);
      __syncwarp();  // (the next copy goes where this chunk lay)
      f0 += n;
    }

    // ---- the unit, or this warp's part of it
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], o);
    const uint32_t u0 = uid, u1 = unit_span[warp].y;
    const int4 place = unit_place[warp];
    __syncwarp();
    const bool whole = f == u0 && fend == u1, last = fend == hi;
    f = fend == u1 ? fend + kUnitCost : fend;
    f = f < hi ? open_unit(f) : hi;  // (the next unit's queries are on their way during the stores)
    float* part = nullptr;
    if (!whole) {
      const int e = 2 * warp + (last ? 1 : 0);
      part = last ? reinterpret_cast<float*>(ring) : p.wparts + ((size_t)cta * K::WARPS + warp) * K::PART;
      if (lane == 0) {
        ent_unit[e] = make_uint2(u0, u1);
        ent_place[e] = place;
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = nb * 8 + 2 * t + i;
        if (place.z + rr >= place.w) continue;
        if (whole) {
          const float inv = l[nb][i] == 0.f ? 0.f : 8.0f / l[nb][i];
          const int tj = (int)fast_div(place.z + rr, p.group, p.ginv);
          const long long tok = place.x + tj;
          const int head = place.y + place.z + rr - tj * p.group;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o.p) + tok * p.o.ts + head * p.o.hs + g * (HD / 8));
#pragma unroll
          for (int k = 0; k < KS; k += 4) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[2 * j] = acc[nb][k + j][i] * inv;
              x[2 * j + 1] = acc[nb][k + j][2 + i] * inv;
            }
            dst[k / 4] = pack8_bf16(x);
          }
          if (p.lse && g == 0) p.lse[tok * p.hq + head] = (m[nb][i] - kPShift + log2f(l[nb][i])) * kLn2;
        } else {
#pragma unroll
          for (int k = 0; k < KS; k += 2)
            *reinterpret_cast<float4*>(part + rr * HD + g * (HD / 8) + 2 * k) =
                make_float4(acc[nb][k][i], acc[nb][k][2 + i], acc[nb][k + 1][i], acc[nb][k + 1][2 + i]);
          if (g == 0) {
            part[K::ROWS * HD + rr] = m[nb][i];
            part[K::ROWS * HD + K::ROWS + rr] = l[nb][i];
          }
        }
      }
  }

  // ---- the CTA's unfinished units: one warp per (unit, row), the parts in the list's order
  __syncthreads();
  const uint2 mine = lane < 2 * K::WARPS ? ent_unit[lane] : make_uint2(0u, 0u);
  const bool there = mine.y != 0;
  const uint32_t valid = __ballot_sync(0xffffffffu, there);
  const uint32_t below = valid & ((1u << lane) - 1u);
  const uint32_t prev = __shfl_sync(0xffffffffu, mine.x, below ? 31 - __clz(below) : 0);
  const uint32_t leads = __ballot_sync(0xffffffffu, there && (!below || prev != mine.x));
  for (int k = warp; k < __popc(leads); k += K::WARPS) {
    uint32_t at = leads;
    for (int i = k; i > 0; --i) at &= at - 1;
    const int e0 = __ffs(at) - 1;
    const uint32_t after = e0 == 31 ? 0u : leads >> (e0 + 1);
    const uint32_t span = (after ? (1u << (e0 + __ffs(after))) - 1u : 0xFFFFFFFFu) & ~((1u << e0) - 1u) & valid;
    const uint2 unit = ent_unit[e0];
    const int4 place = ent_place[e0];
    const bool cont = unit.x < clo, open = unit.y > chi;
    if (lane == 0) {  // (at most one unit is continued and one left open)
      if (cont) p.meta[2 * cta].x = open ? 1 : 3;
      else if (open) {
        p.meta[2 * cta].y = 1;
        p.meta[2 * cta + 1] = place;
      }
    }
    auto part_of = [&](int e) {
      return (e & 1) ? reinterpret_cast<const float*>(smem + (e >> 1) * K::RING)
                     : p.wparts + ((size_t)cta * K::WARPS + (e >> 1)) * K::PART;
    };
    const bool has = span >> lane & 1u;
    const float* const mp = part_of(has ? lane : e0) + K::ROWS * HD;
    for (int r0 = 0; r0 < K::ROWS && place.z + r0 < place.w; r0 += 4) {  // four rows' loads at a time
      Joined<HD> j[4];
      float me[4], le[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // (parts hold no more than the unit's rows)
        me[r] = place.z + r0 + r < place.w ? mp[r0 + r] : -INFINITY;
        le[r] = place.z + r0 + r < place.w ? mp[K::ROWS + r0 + r] : 0.f;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) j[r].weigh(has ? me[r] : -INFINITY, has ? le[r] : 0.f);
      for (uint32_t x = span; x; x &= x - 1) {
        const int e = __ffs(x) - 1;
        const float* part = part_of(e) + r0 * HD;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float wt = __shfl_sync(0xffffffffu, j[r].w, e);
          if (place.z + r0 + r < place.w) j[r].add(part + r * HD, wt, lane);
        }
      }
      if (!cont && !open) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (place.z + r0 + r < place.w) j[r].store(p, place, r0 + r, lane);
      } else {
        float* dst = p.parts + ((size_t)cta * 2 + (cont ? 0 : 1)) * K::PART;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (place.z + r0 + r >= place.w) continue;
          j[r].keep(dst + (r0 + r) * HD, lane);
          if (lane == 0) {
            dst[K::ROWS * HD + r0 + r] = j[r].M;
            dst[K::ROWS * HD + K::ROWS + r0 + r] = j[r].L;
          }
        }
      }
    }
  }
}

// Units that more than one CTA worked on: warp r of block (c, y) joins row 8 y + r of the unit that CTA c left
// open with the parts of the CTAs that continued it.
template <int HD, int ROWS>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams p) {
  constexpr int PART = ROWS * HD + 2 * ROWS;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (launched before the attention kernel has ended)
  const int c = blockIdx.x, lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5), ctas = gridDim.x;
  if (!p.meta[2 * c].y) return;
  const int4 place = p.meta[2 * c + 1];
  if (place.z + row >= place.w) return;
  // the parts: CTA c's open one, then the following CTAs' up to the one that finished the unit
  int n = 1;
  for (;;) {
    const int i = c + n + lane;
    const int f = i < ctas ? p.meta[2 * i].x : 0;
    const uint32_t stop = __ballot_sync(0xffffffffu, !(f & 1) || (f & 2));
    if (!stop) {
      n += 32;
      continue;
    }
    const int z = __ffs(stop) - 1;
    n += z + (__shfl_sync(0xffffffffu, f, z) & 1);
    break;
  }
  auto part_of = [&](int i) { return p.parts + ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * PART; };
  Joined<HD> all;
  all.weigh(-INFINITY, 0.f);
  for (int b = 0; b < n; b += 32) {
    float me = -INFINITY, le = 0.f;
    if (b + lane < n) {
      me = part_of(b + lane)[ROWS * HD + row];
      le = part_of(b + lane)[ROWS * HD + ROWS + row];
    }
    Joined<HD> j;
    j.weigh(me, le);
    const int m = min(32, n - b);
    int i = 0;
    for (; i + 4 <= m; i += 4) {
      float x[4][HD / 32];
#pragma unroll
      for (int y = 0; y < 4; ++y) j.load(part_of(b + i + y) + row * HD, lane, x[y]);
#pragma unroll
      for (int y = 0; y < 4; ++y) j.mul(x[y], __shfl_sync(0xffffffffu, j.w, i + y));
    }
    for (; i < m; ++i) j.add(part_of(b + i) + row * HD, __shfl_sync(0xffffffffu, j.w, i), lane);
    all.join(j);
  }
  all.store(p, place, row, lane);
}

}  // namespace kvq
}  // namespace dec
