// Entry points of drafted trees' masks and of bounded caches (dec_draft_tree, dec_kvq_mass, dec_kvq_heaviest,
// dec_kvq_move of dec.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "dec_kvq_host.h"
#include "dec_kvq_keep.cuh"
#include "dec_kvq_mass.cuh"

using namespace dec;
using namespace dec::kvq;

namespace {

// Sequences without token rows: what check_seqs asks of the rest.
dec_status check_alone(const dec_kvq_seqs* s, const dec_kvq_cache* c, const char* name) {
  if (dec_status st = check_seqs(s, c)) return st;
  if (s->cu_tokens || s->n_tokens != s->batch) {
    char buf[120];
    snprintf(buf, sizeof buf, "%s: sequences without token rows (cu_tokens NULL, n_tokens == batch)", name);
    return op_fail(DEC_ERR_ARG, buf);
  }
  return DEC_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

dec_status dec_draft_tree(const dec_draft_tree_args* a, void* stream) {
  op_clear();
  if (!a) return op_fail(DEC_ERR_ARG, "draft_tree: NULL arguments");
  if (a->batch < 0 || a->n_tokens < 0 || a->max_tokens < 0 || a->mask_stride < 0)
    return op_fail(DEC_ERR_ARG, "draft_tree: negative size");
  if (a->max_tokens > DEC_MAX_TREE) return op_fail(DEC_ERR_UNSUPPORTED, "draft_tree: more than DEC_MAX_TREE rows a sequence");
  if (a->batch == 0 || a->n_tokens == 0 || a->max_tokens == 0) return DEC_OK;
  if (!a->cu_tokens || !a->parents || !a->mask) return op_fail(DEC_ERR_ARG, "draft_tree: cu_tokens, parents and mask are needed");
  if (a->positions && !a->lengths) return op_fail(DEC_ERR_ARG, "draft_tree: positions need lengths");
  const int words = (a->max_tokens + 31) / 32;
  if (a->mask_stride < words) return op_fail(DEC_ERR_ARG, "draft_tree: mask_stride is below the words of a row");
  if (!aligned4(a->mask)) return op_fail(DEC_ERR_ARG, "draft_tree: mask is not aligned to its type");
  if (dec_status st = op_on_device(a->mask, "draft_tree: mask")) return st;
  TreeParams p;
  p.cu = a->cu_tokens;
  p.parents = a->parents;
  p.lengths = a->lengths;
  p.batch = a->batch;
  p.n_tokens = a->n_tokens;
  p.max_tokens = a->max_tokens;
  p.words = words;
  p.mask = a->mask;
  p.mask_stride = a->mask_stride;
  p.positions = a->positions;
  draft_tree_kernel<<<(unsigned)a->batch, (unsigned)words * 32, 0, op_stream(stream)>>>(p);
  return launched("draft_tree");
}

dec_status dec_kvq_mass(const dec_kvq_cache* c, const dec_kvq_seqs* s, const dec_kvq_mass_args* a, void* stream) {
  op_clear();
  if (dec_status st = check_cache(c)) return st;
  if (dec_status st = check_seqs(s, c)) return st;
  if (!a) return op_fail(DEC_ERR_ARG, "mass: NULL arguments");
  if (a->n_heads < 1 || a->n_heads > 16384 || a->n_heads % c->n_kv_heads)
    return op_fail(DEC_ERR_ARG, "mass: n_heads must be a multiple of the cache's KV heads");
  if (a->max_tokens < 0 || !(a->scale >= 0.f) || std::isinf(a->scale))
    return op_fail(DEC_ERR_ARG, "mass: max_tokens and scale must not be negative, scale finite");
  if (!std::isfinite(a->decay)) return op_fail(DEC_ERR_ARG, "mass: decay must be finite");
  if (s->batch == 0 || s->n_tokens == 0 || a->max_tokens == 0) return DEC_OK;
  if (dec_status st = check_rows(&a->q, DEC_BF16, "mass: q")) return st;
  if (!a->lse || !a->mass_out || (a->decay != 0.f && !a->mass)) return op_fail(DEC_ERR_ARG, "mass: lse, mass or mass_out missing");
  if (!aligned4(a->lse) || !op_aligned(a->mass) || !op_aligned(a->mass_out))
    return op_fail(DEC_ERR_ARG, "mass: lse must be aligned to its type, mass and mass_out to 16 bytes");
  const int group = a->n_heads / c->n_kv_heads, max_tokens = std::min(a->max_tokens, s->n_tokens);
  // (the list of groups, or of tiles and blocks of rows, is counted in 32 bits, and so are a sequence's rows)
  const long long groups = ((long long)s->max_pages * c->page_tokens + s->n_tokens) / kGroup + 1;
  if ((long long)s->n_tokens * a->n_heads >= kAllRows || (long long)s->max_pages * c->page_tokens + s->n_tokens >= INT_MAX - 65536 ||
      (long long)c->n_pages * c->n_kv_heads * (c->page_tokens / kGroup) >= INT_MAX ||
      groups * c->n_kv_heads * (std::min(s->batch, kMaxSeqs) + (long long)s->n_tokens * group / kTile) >= (1LL << 32) - 64)
    return op_fail(DEC_ERR_UNSUPPORTED, "mass: 2^30 query rows, 2^31 positions or cache groups, or too much work for one call");
  if (dec_status st = op_on_device(c->pages, "cache: pages")) return st;
  const int sms = op_sms();
  if (sms < 1) return op_fail(DEC_ERR_CUDA, "mass: no device");
  MassParams p{};
  p.c = cache_of(c);
  p.s = seqs_of(s);
  p.q = rows_of(a->q);
  p.lse = const_cast<float*>(a->lse);
  p.scale = (a->scale == 0.f ? 1.0f / std::sqrt((float)c->head_dim) : a->scale) * 1.4426950408889634f * 8.0f;
  p.hq = a->n_heads;
  p.group = group;
  p.ginv = reciprocal(group);
  p.causal = a->causal != 0;
  p.max_tokens = a->max_tokens;
  p.magic = Magic{0x64006400u, 0x54005400u};
  p.min_groups = 1;  // (a warp's, at least: one token on 1 k 4.4 us, with 4 a warp 6.4)
  p.decay = a->decay;
  p.mass = a->mass;
  p.out = a->mass_out;
  const long long rows = (long long)max_tokens * group;
  // The tile kernel's time grows with every 128 rows, the streaming one's with every 8, and it keeps no more than 16. Streaming
  // against tile kernel, us (8 KV heads of 128): 8 rows, one sequence on 8 k 6.6 / 11.7, on 64 k 14.0 / 40.4, 16 on 2 k 9.8 / 27.4; 16
  // rows 8.3 / 12.0, 16.9 / 40.5, 12.0 / 27.3. 8 columns for up to 8 rows against 16: 6.6 / 7.6, 14.0 / 16.7, 9.8 / 11.5.
  const int kind = rows <= 8 ? 0 : rows <= 16 ? 1 : 2;
  if (kind == 2) p.magic.lo = 0x43004300u;  // (bf16 128, twice)
  const bool big = c->head_dim == 128;
  void (*const k)(const MassParams) = kind == 0   ? (big ? mass_kernel<128, 1> : mass_kernel<64, 1>)
                                      : kind == 1 ? (big ? mass_kernel<128, 2> : mass_kernel<64, 2>)
                                                  : (big ? mass_tile_kernel<128> : mass_tile_kernel<64>);
  const int smem = kind < 2 ? (big ? StreamCfg<128>::smem() : StreamCfg<64>::smem()) : big ? TileCfg<128>::smem() : TileCfg<64>::smem();
  const int threads = kind < 2 ? 256 : big ? TileCfg<128>::THREADS : TileCfg<64>::THREADS, ctas = kind < 2 ? 2 * sms : sms;
  static std::atomic<unsigned long long> done[3][2];
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess && !(done[kind][big].load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    ce = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (ce == cudaSuccess && dev < 64) done[kind][big].fetch_or(1ull << dev, std::memory_order_release);
  }
  if (ce != cudaSuccess) return op_cuda(ce, "mass");
  const Seqs all = p.s;
  for (int b = 0; b < s->batch; b += kMaxSeqs) {
    p.s.batch = std::min(kMaxSeqs, s->batch - b);
    p.s.lengths = all.lengths + b;
    p.s.table = all.table + b * all.table_stride;
    if (all.cu) p.s.cu = all.cu + b;
    p.b0 = b;
    k<<<(unsigned)ctas, (unsigned)threads, smem, op_stream(stream)>>>(p);
    if (dec_status st = launched("mass")) return st;
  }
  return DEC_OK;
}

dec_status dec_kvq_heaviest(const dec_kvq_cache* c, const dec_kvq_seqs* s, const dec_kvq_heaviest_args* a, void* stream) {
  op_clear();
  if (dec_status st = check_cache(c)) return st;
  if (dec_status st = check_alone(s, c, "heaviest")) return st;
  if (!a) return op_fail(DEC_ERR_ARG, "heaviest: NULL arguments");
  if (a->budget < 1 || a->sinks < 0 || a->recent < 0 || (long long)a->sinks + a->recent > a->budget)
    return op_fail(DEC_ERR_ARG, "heaviest: budget must be positive and hold the sinks and the recent positions");
  if (s->batch == 0) return DEC_OK;
  if (!a->mass || !a->kept || !a->count) return op_fail(DEC_ERR_ARG, "heaviest: mass, kept or count missing");
  if (!aligned4(a->mass) || !aligned4(a->kept) || !aligned4(a->count))
    return op_fail(DEC_ERR_ARG, "heaviest: mass, kept and count must be aligned to their types");
  // (positions and list entries are counted in 32 bits, up to a CTA's share past the last)
  if ((long long)s->batch * c->n_kv_heads > INT_MAX || a->budget > INT_MAX - 65536)
    return op_fail(DEC_ERR_UNSUPPORTED, "heaviest: 2^31 lists or a budget of 2^31");
  if (dec_status st = op_on_device(c->pages, "cache: pages")) return st;
  KeepParams p;
  p.c = cache_of(c);
  p.s = seqs_of(s);
  p.mass = a->mass;
  p.budget = a->budget;
  p.sinks = a->sinks;
  p.recent = a->recent;
  p.kept = a->kept;
  p.count = a->count;
  // CTAs a list: as many as the SMs hold, each with 1024 positions at least of what the page tables can hold. 1, 2, 4, 8 CTAs,
  // us: 8 lists of 32 k 34.5, 22.0, 15.2, 13.4; of 4 k 8.6, 7.8, 7.8, 9.3; of 1 k 5.0, 6.3, 7.2, 9.1; 32 of 8 k 12.2, 10.5, 9.2,
  // 28.6 (more than the SMs hold); 128 of 4 k 9.5, 15.5, 28.8, 80.5.
  const long long lists = (long long)s->batch * c->n_kv_heads, most = (long long)s->max_pages * c->page_tokens;
  const int sms = op_sms();
  if (sms < 1) return op_fail(DEC_ERR_CUDA, "heaviest: no device");
  int cl = 1;
  while (cl < 8 && lists * cl * 2 <= sms && most / (cl * 2) >= kKeepThreads) cl *= 2;
  if (lists * cl > INT_MAX) return op_fail(DEC_ERR_UNSUPPORTED, "heaviest: 2^31 lists");
  void (*const k)(const KeepParams) = cl == 1   ? heaviest_kernel<1>
                                      : cl == 2 ? heaviest_kernel<2>
                                      : cl == 4 ? heaviest_kernel<4>
                                                : heaviest_kernel<8>;
  p.cached = (int)std::min<long long>(kKeepCached, (most + cl - 1) / cl + 32);
  static std::atomic<unsigned long long> done[4];
  std::atomic<unsigned long long>& set = done[cl == 1 ? 0 : cl == 2 ? 1 : cl == 4 ? 2 : 3];
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess && !(set.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
    ce = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeepCached * 4);
    if (ce == cudaSuccess && dev < 64) set.fetch_or(1ull << dev, std::memory_order_release);
  }
  if (ce != cudaSuccess) return op_cuda(ce, "heaviest");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(lists * cl));
  cfg.blockDim = dim3(kKeepThreads);
  cfg.dynamicSmemBytes = p.cached * 4;
  cfg.stream = op_stream(stream);
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cl;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = cl > 1 ? 1 : 0;
  ce = cudaLaunchKernelEx(&cfg, k, p);
  if (ce != cudaSuccess) return op_cuda(ce, "heaviest");
  return launched("heaviest");
}

dec_status dec_kvq_move(const dec_kvq_cache* c, const dec_kvq_seqs* s, const dec_kvq_move_args* a, void* stream) {
  op_clear();
  if (dec_status st = check_cache(c)) return st;
  if (!s || !a) return op_fail(DEC_ERR_ARG, "move: NULL arguments");
  dec_kvq_seqs checked = *s;  // (lengths NULL: lists begin at 0)
  if (!checked.lengths) checked.lengths = a->count;
  if (dec_status st = check_alone(&checked, c, "move")) return st;
  if (a->max_count < 0 || a->index_stride < 0 || a->head_stride < 0) return op_fail(DEC_ERR_ARG, "move: negative size");
  if (s->batch == 0 || a->max_count == 0) return DEC_OK;
  if (!a->index || !a->count) return op_fail(DEC_ERR_ARG, "move: index or count missing");
  if (!aligned4(a->index) || !aligned4(a->count) || !aligned4(a->mass))
    return op_fail(DEC_ERR_ARG, "move: index, count and mass must be aligned to their types");
  if (a->to && (a->to_pages < 1 || a->to_stride < 0)) return op_fail(DEC_ERR_ARG, "move: to_pages and to_stride");
  if (a->to && (long long)a->to_pages * c->page_tokens > INT_MAX - 65536)
    return op_fail(DEC_ERR_UNSUPPORTED, "move: a page table of 2^31 positions or more");
  if (a->max_count > INT_MAX - 65536) return op_fail(DEC_ERR_UNSUPPORTED, "move: lists of 2^31 positions");
  if (dec_status st = op_on_device(c->pages, "cache: pages")) return st;
  MoveParams p;
  p.c = cache_of(c);
  p.s = p.to = seqs_of(s);
  if (a->to) {
    p.to.table = a->to;
    p.to.max_pages = a->to_pages;
    p.to.table_stride = a->to_stride;
  }
  p.index = a->index;
  p.count = a->count;
  p.index_stride = a->index_stride;
  p.head_stride = a->head_stride;
  p.max_count = a->max_count;
  p.in_place = a->to == nullptr;
  p.mass = a->mass;
  const int runs = 2 * c->head_dim / kBlock, sms = op_sms();
  if (sms < 1) return op_fail(DEC_ERR_CUDA, "move: no device");
  // How a list's positions are shared out, in us (8 KV heads of 128). Up to 64 (a path of a tree): a CTA for all 16 runs
  // against eight with two each: 16 sequences of 16 in place 2.9 / 4.9, of 64 4.9 / 5.1, of 128 7.4 / 5.8. Beyond that, in
  // place, where a CTA goes through the whole list: one run a CTA of 512 threads, while the SMs hold them all, against
  // two of 256: one sequence of 8192 29 / 52, of 1024 5.5 / 8.0, four of 2048 19 / 17, 16 of 1024 33 / 21. Elsewhere the list is cut
  // too, until there are eight CTAs an SM or 128 positions each: one of 8192 whole 45, in 8 12; of 1024 7.4 / 3.7; four of
  // 2048 15, in 4 12; 16 of 1024 20, in 4 25.
  const long long lists = (long long)s->batch * c->n_kv_heads;
  const bool few = a->max_count <= 64, alone = !few && p.in_place && lists * runs <= sms, big = c->head_dim == 128;
  p.parts = (few ? 1 : alone ? runs : runs / 2) + (a->mass ? 1 : 0);
  p.splits = 1;
  const long long ctas = lists * p.parts;
  if (!p.in_place && !few) p.splits = (int)std::max<long long>(1, std::min<long long>(8 * sms / ctas, a->max_count / 128));
  if (ctas * p.splits > INT_MAX) return op_fail(DEC_ERR_UNSUPPORTED, "move: too much work for one call");
  void (*const k)(const MoveParams) = few     ? (big ? move_kernel<128, 16, 256, 4> : move_kernel<64, 8, 256, 4>)
                                      : alone ? (big ? move_kernel<128, 1, 512, 4> : move_kernel<64, 1, 512, 4>)
                                              : (big ? move_kernel<128, 2, 256, 4> : move_kernel<64, 2, 256, 4>);
  k<<<(unsigned)(ctas * p.splits), alone ? 512 : 256, 0, op_stream(stream)>>>(p);
  return launched("move");
}

}  // extern "C"
