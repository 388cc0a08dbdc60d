// The segments of decode steps over a 4-bit cache, compiled in their own translation unit.
#include "dec_wide.cuh"
#include "dec_wide_host.h"

namespace dec {
namespace wide {

WideKernelFn segment_kernel_for(int nr, int hd, int group) {
#define DEC_SK(N, H, GR) \
  if (nr == N && hd == H && group == GR) return wide_segment_kernel<N, H, GR>;
  DEC_SK(32, 64, 2) DEC_SK(64, 64, 2) DEC_SK(128, 64, 2)
  DEC_SK(32, 128, 4) DEC_SK(64, 128, 4) DEC_SK(128, 128, 4)
#undef DEC_SK
  return nullptr;
}

}  // namespace wide
}  // namespace dec
