// Entry points of the paged 4-bit KV cache (dec_kvq_* of dec.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdio>
#include <mutex>

#include "dec_kvq.cuh"
#include "dec_kvq_attn.cuh"
#include "dec_kvq_prompt.cuh"
#include "dec_ops.h"

namespace dec {

namespace {
thread_local char g_op_error[256] = "";
}

dec_status op_fail(dec_status s, const char* msg) {
  size_t i = 0;
  for (; msg[i] && i + 1 < sizeof g_op_error; ++i) g_op_error[i] = msg[i];
  g_op_error[i] = 0;
  return s;
}

dec_status op_cuda(cudaError_t c, const char* what) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", what, cudaGetErrorString(c));
  return op_fail(c == cudaErrorMemoryAllocation ? DEC_ERR_OOM : DEC_ERR_CUDA, buf);
}

void op_clear() { g_op_error[0] = 0; }

int op_sms() {
  static std::mutex mu;
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms[dev] = 0;
  return sms[dev];
}

dec_status op_on_device(const void* p, const char* what) {
  cudaPointerAttributes a;
  int dev = -1;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess) ce = cudaPointerGetAttributes(&a, p);
  if (ce != cudaSuccess) {
    cudaGetLastError();  // (a pointer CUDA does not know, or no device: not a sticky error)
    return op_cuda(ce, what);
  }
  if ((a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) || a.device != dev) {
    char buf[200];
    snprintf(buf, sizeof buf, "%s is not memory of the current CUDA device", what);
    return op_fail(DEC_ERR_ARG, buf);
  }
  return DEC_OK;
}

namespace kvq {
namespace {

dec_status check_cache(const dec_kvq_cache* c) {
  if (!c || !c->pages) return op_fail(DEC_ERR_ARG, "cache: NULL");
  if (c->head_dim < 1 || c->n_kv_heads < 1 || c->page_tokens < 1 || c->n_pages < 1)
    return op_fail(DEC_ERR_ARG, "cache: sizes must be positive");
  if (c->head_dim != 64 && c->head_dim != 128) return op_fail(DEC_ERR_UNSUPPORTED, "cache: head_dim must be 64 or 128");
  if (c->n_kv_heads > 1024) return op_fail(DEC_ERR_UNSUPPORTED, "cache: more than 1024 KV heads");
  if (dec_kvq_page_bytes(c->page_tokens, c->n_kv_heads, c->head_dim) == 0)
    return op_fail(DEC_ERR_UNSUPPORTED, "cache: page_tokens must be 16, 32, 64, 128 or 256");
  if (!op_aligned(c->pages)) return op_fail(DEC_ERR_ARG, "cache: pages must be 16-byte aligned");
  return DEC_OK;
}

dec_status check_seqs(const dec_kvq_seqs* s, const dec_kvq_cache* c) {
  if (!s) return op_fail(DEC_ERR_ARG, "sequences: NULL");
  if (s->batch < 0 || s->n_tokens < 0 || s->max_pages < 0) return op_fail(DEC_ERR_ARG, "sequences: negative size");
  if (!s->cu_tokens && s->n_tokens != s->batch)
    return op_fail(DEC_ERR_ARG, "sequences: without cu_tokens every sequence has one row (n_tokens == batch)");
  if (s->batch == 0 || s->n_tokens == 0) return DEC_OK;
  if (!s->lengths || !s->table || s->max_pages == 0) return op_fail(DEC_ERR_ARG, "sequences: lengths and table are needed");
  // (sequences are counted in 32 bits, up to a launch's share past the last)
  if (s->batch > INT_MAX - 4 * kMaxSeqs) return op_fail(DEC_ERR_UNSUPPORTED, "sequences: a batch of 2^31");
  if (s->table_stride < 0) return op_fail(DEC_ERR_ARG, "sequences: negative table_stride");
  if ((long long)s->max_pages * c->page_tokens > INT_MAX - 65536)
    return op_fail(DEC_ERR_UNSUPPORTED, "sequences: a page table of 2^31 positions or more");
  return DEC_OK;
}

dec_status check_rows(const dec_rows* r, dec_dtype t, const char* name) {
  char buf[120];
  const int per = t == DEC_F32 ? 4 : 8;
  if (!r || !r->p) {
    snprintf(buf, sizeof buf, "%s: NULL", name);
    return op_fail(DEC_ERR_ARG, buf);
  }
  if (!op_aligned(r->p) || r->token_stride % per || r->head_stride % per) {
    snprintf(buf, sizeof buf, "%s: rows and strides must be multiples of 16 bytes", name);
    return op_fail(DEC_ERR_ARG, buf);
  }
  return DEC_OK;
}

Cache cache_of(const dec_kvq_cache* c) {
  Cache k;
  k.pages = static_cast<uint8_t*>(c->pages);
  k.n_pages = c->n_pages;
  k.page_shift = 0;
  while ((1 << k.page_shift) < c->page_tokens) ++k.page_shift;
  k.hkv = c->n_kv_heads;
  k.status = c->status;
  return k;
}
Seqs seqs_of(const dec_kvq_seqs* s) {
  Seqs k;
  k.batch = s->batch;
  k.n_tokens = s->n_tokens;
  k.max_pages = s->max_pages;
  k.cu = s->cu_tokens;
  k.lengths = s->lengths;
  k.table = s->table;
  k.table_stride = s->table_stride;
  return k;
}
Rows rows_of(const dec_rows& r) { return Rows{r.p, r.token_stride, r.head_stride}; }

dec_status launched(const char* what) {
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? DEC_OK : op_cuda(ce, what);
}

// The prompt kernel takes calls whose longest sequence has more query rows per KV head than this: the
// streaming one's time grows with every 16 rows, the prompt kernel's with every 128. Streaming against
// prompt kernel, us: hd 128, 8 KV heads, 17 .. 32 rows, one sequence on 8 k 23.6 / 20.3, on 64 k 53.6 /
// 52.0, 16 on 2 k 42.3 / 34.5, 64 on 1 k 85.5 / 85.7; 16 rows, on 64 k 37.3 / 52.0, 64 on 1 k 52.0 / 91.9.
// hd 64 (half the decoding for as many exponentials), 48 rows, one on 8 k 20.8 / 16.6, on 64 k 50.7 / 41.8,
// 64 on 1 k 67.4 / 63.0; 32 rows, on 64 k 38.4 / 41.8, 64 on 1 k 47.9 / 63.0.
constexpr int prompt_above(int hd) { return hd == 128 ? 16 : 32; }

// The attention kernel's dynamic shared memory limit, raised once per device. The join kernel asks for
// the same division of the SM's memory, so that none is redivided between the two.
template <class F>
dec_status raise_smem(F* k, F* join, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce != cudaSuccess) return op_cuda(ce, "cudaGetDevice");
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return DEC_OK;
  ce = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (ce == cudaSuccess)
    ce = cudaFuncSetAttribute((const void*)join, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (ce != cudaSuccess) return op_cuda(ce, "cudaFuncSetAttribute");
  if (dev < 64) done.fetch_or(bit, std::memory_order_release);
  return DEC_OK;
}

// Which kernel takes a call, by the longest sequence's query rows: 0 and 1, the streaming one with 8 and
// 16 rows a unit; 2, the one for prompts.
int kernel_of(int hd, int n_heads, int hkv, int max_tokens) {
  const long long rows = (long long)max_tokens * (n_heads / hkv);
  return rows <= 8 ? 0 : rows <= prompt_above(hd) ? 1 : 2;
}

// A kernel's launch: its function, the one that joins its parts, and their sizes.
struct Variant {
  void (*kernel)(const AttnParams);
  void (*join)(const AttnParams);
  int threads, smem, rows, part, wparts;  // parts in floats; a CTA's parts of its warps
};
template <int HD, int NB>
Variant streaming() {
  using K = AttnCfg<HD, NB>;
  return Variant{attention_kernel<HD, NB>, join_kernel<HD, K::ROWS>, K::THREADS, K::smem(), K::ROWS, K::PART, K::WARPS * K::PART};
}
template <int HD>
Variant prompt() {
  using C = PromptCfg<HD>;
  return Variant{prompt_kernel<HD>, join_kernel<HD, C::ROWS>, C::THREADS, C::smem(), C::ROWS, C::PART, 0};
}
Variant variant_of(int hd, int kind) {
  if (hd == 128) return kind == 0 ? streaming<128, 1>() : kind == 1 ? streaming<128, 2>() : prompt<128>();
  return kind == 0 ? streaming<64, 1>() : kind == 1 ? streaming<64, 2>() : prompt<64>();
}
int64_t workspace_of(const Variant& v, int sms) { return (int64_t)sms * (32 + 4ll * (2 * v.part + v.wparts)); }

dec_status launch_attention(AttnParams p, int hd, int kind, int batch, uint8_t* ws, cudaStream_t stream) {
  static std::atomic<unsigned long long> done[2][3];
  const Variant v = variant_of(hd, kind);
  if (dec_status st = raise_smem(v.kernel, v.join, v.smem, done[hd == 128][kind])) return st;
  const int sms = op_sms();
  if (sms < 1) return op_fail(DEC_ERR_CUDA, "attention: no device");
  p.meta = reinterpret_cast<int4*>(ws);
  p.parts = reinterpret_cast<float*>(ws + (size_t)sms * 32);
  p.wparts = p.parts + (size_t)sms * 2 * v.part;
  p.min_groups = kMinGroups;
  p.magic = Magic{0x64006400u, 0x54005400u};
  const Seqs all = p.s;
  for (int b = 0; b < batch; b += kMaxSeqs) {
    p.s.batch = std::min(kMaxSeqs, batch - b);
    p.s.lengths = all.lengths + b;
    p.s.table = all.table + b * all.table_stride;
    if (all.cu) p.s.cu = all.cu + b;
    p.b0 = b;
    v.kernel<<<sms, v.threads, v.smem, stream>>>(p);
    cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess) return op_cuda(ce, "attention");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sms, v.rows / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    ce = cudaLaunchKernelEx(&cfg, v.join, p);
    if (ce != cudaSuccess) return op_cuda(ce, "attention (join)");
  }
  return DEC_OK;
}

}  // namespace
}  // namespace kvq
}  // namespace dec

using namespace dec;
using namespace dec::kvq;

extern "C" {

const char* dec_op_error(void) { return g_op_error; }

int64_t dec_kvq_page_bytes(int32_t page_tokens, int32_t n_kv_heads, int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  if (n_kv_heads < 1 || n_kv_heads > 1024) return 0;
  if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1))) return 0;
  return (int64_t)n_kv_heads * (page_tokens / kGroup) * group_bytes(head_dim);
}

dec_status dec_kvq_append(const dec_kvq_cache* c, const dec_kvq_seqs* s, const dec_kvq_append_args* a, void* stream) {
  op_clear();
  if (dec_status st = check_cache(c)) return st;
  if (dec_status st = check_seqs(s, c)) return st;
  if (!a) return op_fail(DEC_ERR_ARG, "append: NULL arguments");
  if (a->dtype != DEC_BF16 && a->dtype != DEC_F32) return op_fail(DEC_ERR_ARG, "append: unknown dtype");
  if (a->n_heads < 0 || a->n_heads > 16384) return op_fail(DEC_ERR_ARG, "append: n_heads out of range");
  if (a->rotary_dim < 0 || a->rotary_dim > c->head_dim || a->rotary_dim % 16)
    return op_fail(DEC_ERR_ARG, "append: rotary_dim must be a multiple of 16 within head_dim");
  if ((a->rotary_dim > 0) != (a->rope != nullptr) || a->rope_len < 0)
    return op_fail(DEC_ERR_ARG, "append: rope and rotary_dim go together");
  if (a->rope && !op_aligned(a->rope)) return op_fail(DEC_ERR_ARG, "append: rope must be 16-byte aligned");
  if ((a->q_norm && !op_aligned(a->q_norm)) || (a->k_norm && !op_aligned(a->k_norm)))
    return op_fail(DEC_ERR_ARG, "append: norm weights must be 16-byte aligned");
  if (!(a->eps >= 0.f)) return op_fail(DEC_ERR_ARG, "append: eps must not be negative");
  if (s->batch == 0 || s->n_tokens == 0) return DEC_OK;  // (rows of nothing may lie nowhere)
  const bool has_q = a->q.p != nullptr;
  if (has_q != (a->n_heads > 0)) return op_fail(DEC_ERR_ARG, "append: n_heads goes with q");
  if (dec_status st = check_rows(&a->k, a->dtype, "append: k")) return st;
  if (dec_status st = check_rows(&a->v, a->dtype, "append: v")) return st;
  if (has_q) {
    if (dec_status st = check_rows(&a->q, a->dtype, "append: q")) return st;
    if (dec_status st = check_rows(&a->q_out, DEC_BF16, "append: q_out")) return st;
  }
  if (dec_status st = op_on_device(c->pages, "cache: pages")) return st;
  AppendParams p;
  p.c = cache_of(c);
  p.s = seqs_of(s);
  p.q = rows_of(a->q);
  p.k = rows_of(a->k);
  p.v = rows_of(a->v);
  p.qo = rows_of(a->q_out);
  p.qn = static_cast<const uint16_t*>(a->q_norm);
  p.kn = static_cast<const uint16_t*>(a->k_norm);
  p.rope = a->rope;
  p.hq = a->n_heads;
  p.rope_len = a->rope_len;
  p.rot = a->rotary_dim;
  p.inter = a->interleaved != 0;
  p.eps = a->eps;
  const bool f32 = a->dtype == DEC_F32;
  const cudaStream_t cs = op_stream(stream);
  auto go = [&](auto* few, auto* many) {
    if (s->n_tokens <= 4 * op_sms()) few<<<(unsigned)s->n_tokens, 256, 0, cs>>>(p);
    else many<<<(unsigned)s->n_tokens, 128, 0, cs>>>(p);
  };
  if (c->head_dim == 128) {
    if (f32) go(append_kernel<128, true, 256>, append_kernel<128, true, 128>);
    else go(append_kernel<128, false, 256>, append_kernel<128, false, 128>);
  } else {
    if (f32) go(append_kernel<64, true, 256>, append_kernel<64, true, 128>);
    else go(append_kernel<64, false, 256>, append_kernel<64, false, 128>);
  }
  return launched("append");
}

dec_status dec_kvq_gather(const dec_kvq_cache* c, const dec_kvq_seqs* s, const dec_rows* k_out, const dec_rows* v_out,
                          void* stream) {
  op_clear();
  if (dec_status st = check_cache(c)) return st;
  if (dec_status st = check_seqs(s, c)) return st;
  if (s->batch == 0 || s->n_tokens == 0) return DEC_OK;
  if (dec_status st = check_rows(k_out, DEC_BF16, "gather: k_out")) return st;
  if (dec_status st = check_rows(v_out, DEC_BF16, "gather: v_out")) return st;
  if (dec_status st = op_on_device(c->pages, "cache: pages")) return st;
  GatherParams p;
  p.c = cache_of(c);
  p.s = seqs_of(s);
  p.k = rows_of(*k_out);
  p.v = rows_of(*v_out);
  auto* k = c->head_dim == 128 ? gather_kernel<128> : gather_kernel<64>;
  k<<<(unsigned)s->n_tokens, 64, 0, op_stream(stream)>>>(p);
  return launched("gather");
}

int64_t dec_kvq_attention_workspace(const dec_kvq_cache* c, int32_t n_heads, int32_t batch, int32_t max_tokens) {
  if (!c || n_heads < 1 || n_heads > 16384 || c->n_kv_heads < 1 || n_heads % c->n_kv_heads || batch < 0 || max_tokens < 0)
    return -1;
  if (dec_kvq_page_bytes(c->page_tokens, c->n_kv_heads, c->head_dim) == 0) return -1;
  const int sms = op_sms();
  if (sms < 1) return -1;
  return workspace_of(variant_of(c->head_dim, kernel_of(c->head_dim, n_heads, c->n_kv_heads, max_tokens)), sms);
}

dec_status dec_kvq_attention(const dec_kvq_cache* c, const dec_kvq_seqs* s, const dec_kvq_attention_args* a,
                             void* stream) {
  op_clear();
  if (dec_status st = check_cache(c)) return st;
  if (dec_status st = check_seqs(s, c)) return st;
  if (!a) return op_fail(DEC_ERR_ARG, "attention: NULL arguments");
  if (a->n_heads < 1 || a->n_heads > 16384 || a->n_heads % c->n_kv_heads)
    return op_fail(DEC_ERR_ARG, "attention: n_heads must be a multiple of the cache's KV heads");
  if (a->max_tokens < 0 || a->likely_tokens < 0 || !(a->scale >= 0.f) || std::isinf(a->scale))
    return op_fail(DEC_ERR_ARG, "attention: max_tokens, likely_tokens and scale must not be negative, scale finite");
  if (s->batch == 0 || s->n_tokens == 0 || a->max_tokens == 0) return DEC_OK;
  if (dec_status st = check_rows(&a->q, DEC_BF16, "attention: q")) return st;
  if (dec_status st = check_rows(&a->out, DEC_BF16, "attention: out")) return st;
  if ((long long)s->n_tokens * a->n_heads >= INT_MAX ||
      (long long)s->max_pages * c->page_tokens + s->n_tokens >= INT_MAX - 65536 ||
      (long long)c->n_pages * c->n_kv_heads * (c->page_tokens / kGroup) >= INT_MAX)
    return op_fail(DEC_ERR_UNSUPPORTED, "attention: 2^31 query rows, positions or cache groups");
  if (!a->workspace || !op_aligned(a->workspace)) return op_fail(DEC_ERR_ARG, "attention: workspace missing or misaligned");
  if (dec_status st = op_on_device(c->pages, "cache: pages")) return st;
  AttnParams p;
  p.c = cache_of(c);
  p.s = seqs_of(s);
  p.q = rows_of(a->q);
  p.o = rows_of(a->out);
  p.lse = a->lse;
  // (scores in units of log2; the factor 8 of the scale bytes)
  p.scale = (a->scale == 0.f ? 1.0f / std::sqrt((float)c->head_dim) : a->scale) * 1.4426950408889634f * 8.0f;
  p.hq = a->n_heads;
  p.group = a->n_heads / c->n_kv_heads;
  p.ginv = reciprocal(p.group);
  p.causal = a->causal != 0;
  p.max_tokens = a->max_tokens;
  const int max_tokens = std::min(a->max_tokens, s->n_tokens);
  if (a->workspace_bytes < dec_kvq_attention_workspace(c, a->n_heads, s->batch, max_tokens))
    return op_fail(DEC_ERR_ARG, "attention: workspace too small");
  // (a kernel for fewer rows needs no more workspace)
  int kind = kernel_of(c->head_dim, a->n_heads, c->n_kv_heads, max_tokens);
  const int likely = a->likely_tokens > 0 && a->likely_tokens < max_tokens
                         ? kernel_of(c->head_dim, a->n_heads, c->n_kv_heads, a->likely_tokens)
                         : kind;
  // entries of the kernel's list, at most: 32-bit
  auto fits = [&](int k) {
    const int rows = k == 0 ? 8 : k == 1 ? 16 : 128, positions = k == 2 ? kTile : kGroup;
    const long long units = (long long)c->n_kv_heads * ((long long)s->n_tokens * p.group / rows + s->batch);
    const long long each = (long long)s->max_pages * c->page_tokens / positions + 1 + std::max(kUnitCost, kPromptCost);
    return units * each < (1LL << 32) - 64;
  };
  if (fits(likely)) kind = likely;
  else if (!fits(kind)) return op_fail(DEC_ERR_UNSUPPORTED, "attention: too much work for one call");
  return launch_attention(p, c->head_dim, kind, s->batch, static_cast<uint8_t*>(a->workspace), op_stream(stream));
}

}  // extern "C"
