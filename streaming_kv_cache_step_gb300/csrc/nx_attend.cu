// nx_attend.cu -- nexus_attend: softmax attention of new tokens over one layer's slices, from
// the cache or from its 8-bit image.
//
// One thread block per token and query head; its warps take every fourth row each, a lane
// holding head_dim / 32 features, with the running maximum and sum of the softmax in
// binary32, and are joined in shared memory at the end.
#include <cuda_fp8.h>
#include <math.h>

#include "nx_internal.cuh"

namespace nx {
namespace {

struct AttendArgs {
  nx_cache c;
  nx_tokens t;
  nx_image im;          // im.k null: no image
  nx_attend a;
  int32_t* dev_status;
  int b;                // rows per image block
};

constexpr int kAttendWarps = 4;

__device__ __forceinline__ float e4m3_value(uint8_t x) {
  const __half_raw r = __nv_cvt_fp8_to_halfraw(x, __NV_E4M3);
  return __half2float(__half(r));
}

template <int D>
__global__ void __launch_bounds__(kAttendWarps * 32) attend_kernel(AttendArgs g) {
  constexpr int E = D / 32;
  __shared__ float s_m[kAttendWarps], s_z[kAttendWarps], s_o[kAttendWarps][D];
  grid_dep_wait();
  const nx_cache& c = g.c;
  const int HQ = c.kv_heads * c.group;
  const long long id = blockIdx.x;
  const int hq = (int)(id % HQ), i = (int)(id / HQ % g.t.max_tokens);
  const int s = (int)(id / HQ / g.t.max_tokens);
  const int h = hq / c.group, l = g.t.layer;
  int first;
  const int n = tokens_of(g.t, s, first);
  if (n < 0 && i == 0 && threadIdx.x == 0) atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
  if (i >= n) return;
  const int slice = (l * c.seqs + s) * c.kv_heads + h;
  int T = c.lens[slice], held = g.im.k ? g.im.rows[slice] : 0, flag = 0;
  if (T < 0 || T > c.capacity) flag = NX_DEV_BAD_LEN;
  else if (held < 0 || held > T || held % g.b) flag = NX_DEV_BAD_IMAGE;
  if (flag) {
    if (threadIdx.x == 0) atomicOr(g.dev_status, flag);
    T = 0;
  }
  const int M = g.a.causal ? T - (n - 1 - i) : T;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float q[E], o[E] = {}, m = -INFINITY, z = 0.f;
  for (int e = 0; e < E; ++e)
    q[e] = ld_elem(g.a.q, c.dtype, (first + i) * g.a.q_stride + hq * D + lane * E + e);
  for (int j = warp; j < M; j += kAttendWarps) {
    const long long row = row_of(c, l, s, h, j);
    if (row < 0) {
      if (lane == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
      continue;
    }
    float k[E], v[E], x = 0.f;
    if (j < held) {
      const long long at = image_scale_at(c, l, s, h, j, g.b);
      for (int e = 0; e < E; ++e) {
        const long long w = row * D + lane * E + e;
        k[e] = e4m3_value(static_cast<const uint8_t*>(g.im.k)[w]) * g.im.k_scale[at];
        v[e] = e4m3_value(static_cast<const uint8_t*>(g.im.v)[w]) * g.im.v_scale[at];
      }
    } else {
      for (int e = 0; e < E; ++e) {
        k[e] = ld_elem(c.k, c.dtype, row * D + lane * E + e);
        v[e] = ld_elem(c.v, c.dtype, row * D + lane * E + e);
      }
    }
    for (int e = 0; e < E; ++e) x = fmaf(q[e], k[e], x);
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= g.a.scale;
    const float top = fmaxf(m, x), ref = top == -INFINITY ? 0.f : top;
    const float old = expf(m - ref), p = expf(x - ref);
    for (int e = 0; e < E; ++e) o[e] = o[e] * old + p * v[e];
    z = z * old + p;
    m = top;
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  if (lane == 0) {
    s_m[warp] = m;
    s_z[warp] = z;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, r = 0.f;
  for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, s_m[w]);
  const int f = threadIdx.x;
  for (int w = 0; w < kAttendWarps; ++w) {
    const float k = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - top);
    sum += k * s_z[w];
    if (f < D) r += k * s_o[w][f];
  }
  if (f < D) {
    r = sum > 0.f ? r / sum : sum == 0.f ? 0.f : NAN;
    const long long at = (first + i) * g.a.out_stride + hq * D + f;
    if (c.dtype == NX_DTYPE_BF16) static_cast<__nv_bfloat16*>(g.a.out)[at] = __float2bfloat16(r);
    else static_cast<float*>(g.a.out)[at] = r;
  }
  if (f == 0 && g.a.lse) g.a.lse[(long long)(first + i) * HQ + hq] = top + logf(sum);
}

}  // namespace
}  // namespace nx

extern "C" size_t nexus_attend_workspace_bytes(const nx_cache* cache, const nx_tokens* tokens) {
  using namespace nx;
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens)) return 0;
  return 256;
}

extern "C" nx_status nexus_attend(const nx_cache* cache, const nx_tokens* tokens,
                                  const nx_image* image, const nx_attend* args, void* ws,
                                  size_t ws_bytes, int32_t* dev_status, nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens) || !args || !dev_status)
    return NX_ERR_INVALID_ARG;
  const nx_cache& c = *cache;
  const nx_attend& a = *args;
  if (image && !valid_image(image)) return NX_ERR_INVALID_ARG;
  if (image && c.dtype != NX_DTYPE_BF16) return NX_ERR_UNSUPPORTED;
  const int size = c.dtype == NX_DTYPE_BF16 ? 2 : 4;
  if (!isfinite(a.scale)) return NX_ERR_INVALID_ARG;
  if (a.q_stride < 0 || a.out_stride < 0 || a.q_stride * size % 16 || a.out_stride * size % 16 ||
      ((uintptr_t)a.q & 15u) || ((uintptr_t)a.out & 15u))
    return NX_ERR_INVALID_ARG;
  if (tokens->tokens > 0 && (!a.q || !a.out)) return NX_ERR_INVALID_ARG;
  if (tokens->tokens > 1 && a.out_stride < (long long)c.kv_heads * c.group * c.head_dim)
    return NX_ERR_INVALID_ARG;           // rows of out would overlap
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < nexus_attend_workspace_bytes(cache, tokens))
    return NX_ERR_WORKSPACE;
  if (tokens->tokens == 0) return finish(cudaSuccess, launches);
  AttendArgs g{};
  g.c = c;
  g.t = *tokens;
  if (image) g.im = *image;
  g.a = a;
  g.dev_status = dev_status;
  g.b = image_block(c);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long blocks = (long long)c.seqs * tokens->max_tokens * c.kv_heads * c.group;
  if (blocks > 0x7FFFFFFFLL) return NX_ERR_UNSUPPORTED;
  cudaError_t e = c.head_dim == 128
                      ? launch_after(attend_kernel<128>, dim3((unsigned)blocks),
                                     dim3(kAttendWarps * 32), 0, st, g)
                      : launch_after(attend_kernel<64>, dim3((unsigned)blocks),
                                     dim3(kAttendWarps * 32), 0, st, g);
  if (e == cudaSuccess) note_launch(st, &launches, "attend");
  return finish(e, launches);
}
