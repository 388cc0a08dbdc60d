// Log-probabilities of rows of logits (dec_logprobs of dec.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "dec_ops.h"

namespace dec {
namespace lp {

struct Params {
  const void* x;
  int rows, vocab, top;
  long long stride;
  const int32_t* targets;
  float *logprob, *entropy, *top_lp;
  int32_t *rank, *top_ids;
};

constexpr int kThreads = 512;

template <bool BF16>
__device__ __forceinline__ float load(const void* row, int i) {
  return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(row)[i]) : static_cast<const float*>(row)[i];
}

// (value, id) ordering: larger value first, then lower id; NaN as -infinity
__device__ __forceinline__ bool before(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

template <class T, class F>
__device__ __forceinline__ T block_reduce(T v, F f, T* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[0];
  for (int i = 1; i < kThreads / 32; ++i) v = f(v, sm[i]);
  return v;
}

// One CTA per row: maximum, then sums, then the alternatives one after another.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const Params p) {
  __shared__ float smf[kThreads / 32];
  __shared__ int smi[kThreads / 32];
  const int r = blockIdx.x;
  const void* row = static_cast<const char*>(p.x) + r * p.stride * (BF16 ? 2 : 4);
  float m = -INFINITY;
  int bad = 0;
  for (int i = threadIdx.x; i < p.vocab; i += kThreads) {
    const float v = load<BF16>(row, i);
    bad |= !(v < INFINITY);
    m = fmaxf(m, v);
  }
  m = block_reduce(m, [](float a, float b) { return fmaxf(a, b); }, smf);
  bad = block_reduce(bad, [](int a, int b) { return a | b; }, smi);
  const int t = p.targets ? p.targets[r] : -1;
  const bool has = t >= 0 && t < p.vocab;
  float xt = has ? load<BF16>(row, t) : NAN;
  const float kt = xt != xt ? -INFINITY : xt;
  float sum = 0.f, ent = 0.f;
  int ahead = 0;
  for (int i = threadIdx.x; i < p.vocab; i += kThreads) {
    float v = load<BF16>(row, i);
    const float e = m == -INFINITY ? 0.f : expf(v - m);
    sum += e;
    if (e > 0.f) ent += e * (v - m);
    if (v != v) v = -INFINITY;
    ahead += before(v, i, kt, t) ? 1 : 0;
  }
  sum = block_reduce(sum, [](float a, float b) { return a + b; }, smf);
  ent = block_reduce(ent, [](float a, float b) { return a + b; }, smf);
  ahead = block_reduce(ahead, [](int a, int b) { return a + b; }, smi);
  const float ls = logf(sum);
  auto lp_of = [&](float v) { return bad ? NAN : v == -INFINITY ? -INFINITY : (v - m) - ls; };
  if (threadIdx.x == 0) {
    if (p.logprob) p.logprob[r] = has ? lp_of(xt) : NAN;
    if (p.rank) p.rank[r] = has ? ahead : -1;
    if (p.entropy) p.entropy[r] = bad ? NAN : m == -INFINITY ? 0.f : ls - ent / sum;
  }
  float lv = INFINITY;
  int li = -1;
  for (int n = 0; n < p.top; ++n) {
    float bv = -INFINITY;
    int bi = INT_MAX;
    for (int i = threadIdx.x; i < p.vocab; i += kThreads) {
      float v = load<BF16>(row, i);
      if (v != v) v = -INFINITY;
      if (before(lv, li, v, i) && (bi == INT_MAX || before(v, i, bv, bi))) {
        bv = v;
        bi = i;
      }
    }
    const float top = block_reduce(bi == INT_MAX ? -INFINITY : bv, [](float a, float b) { return fmaxf(a, b); }, smf);
    bi = block_reduce(bi != INT_MAX && bv == top ? bi : INT_MAX, [](int a, int b) { return min(a, b); }, smi);
    lv = top;
    li = bi;
    if (threadIdx.x == 0) {
      if (p.top_ids) p.top_ids[(long long)r * p.top + n] = bi;
      if (p.top_lp) p.top_lp[(long long)r * p.top + n] = lp_of(top);
    }
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
  if (dec_status st = op_on_device(a->logits, "logprobs: logits")) return st;
  lp::Params p;
  p.x = a->logits;
  p.rows = a->rows;
  p.vocab = a->vocab;
  p.top = (a->top_ids || a->top_logprobs) ? a->top_n : 0;
  p.stride = a->row_stride;
  p.targets = a->targets;
  p.logprob = a->logprob;
  p.entropy = a->entropy;
  p.top_lp = a->top_logprobs;
  p.rank = a->rank;
  p.top_ids = a->top_ids;
  auto* k = a->dtype == DEC_BF16 ? lp::logprobs_kernel<true> : lp::logprobs_kernel<false>;
  k<<<a->rows, lp::kThreads, 0, op_stream(stream)>>>(p);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? DEC_OK : op_cuda(ce, "logprobs");
}
