// nx_attend_tc.cu -- the tensor-core kernel of nexus_attend: its launch, and when it takes a call.
#include "nx_attend_tc.cuh"

namespace nx {

// The row kernel takes 16 rows a pass over K and V, this one 256 but at a higher cost, from 8-bit
// rows more so. Measured (us, this kernel / the row kernel) on 32 x 8 slices of 6960 rows: bf16, 16
// rows 180 / 151, 20 rows 180 / 280; 8 bits, 80 rows 357 / 344, 96 rows 357 / 424. A second pass
// that finds K and V in L2 costs less: bf16, 32 rows, 4 x 8 slices 45 / 43, one sequence of 8
// slices of 32768 rows 64 / 46; 36 rows 46 / 53 and 64 / 59.
bool attend_tc_takes(const nx_cache& c, const nx_tokens& t, bool image) {
  const long long bytes = (long long)c.seqs * c.kv_heads * c.capacity * c.head_dim * 4;
  const int rows = image ? 80 : bytes <= (128LL << 20) ? 32 : kFewRows;
  return c.dtype == NX_DTYPE_BF16 && most_tokens(t) * c.group > rows;
}

bool attend_tc_may_take(const nx_cache& c, const nx_tokens& t) {
  return c.dtype == NX_DTYPE_BF16 && most_tokens(t) * c.group > kFewRows;
}

size_t attend_tc_layout(int D, char* base, AttendWs* ws) {
  size_t at = 0;
  ws->desc = reinterpret_cast<int2*>(base + at);
  at += round256(kTcGrid * sizeof(int2));
  ws->stat = reinterpret_cast<float2*>(base + at);
  at += round256((size_t)2 * kTcGrid * kTcRows * sizeof(float2));
  ws->out = reinterpret_cast<float*>(base + at);
  return at + (size_t)2 * kTcGrid * kTcRows * D * sizeof(float);
}

cudaError_t launch_attend_tc(AttendArgs& g, cudaStream_t st, int* launches) {
  return launch_tc(g, st, launches);
}

}  // namespace nx
