// nx_image.cu -- nexus_quantize: the 8-bit image of a bf16 cache, one power-of-two scale per
// block of rows.
//
// A warp takes one block of one slice of K or V: at most 32 rows x 256 bytes, which lie
// together and which its lanes hold in registers (16-byte loads, all in flight at once), so
// that the largest magnitude and the codes come from one read. The rows are read once (2 B
// a value) and the codes written once (1 B); nothing else moves, and HBM bounds it: 256 slices
// of 6554 rows take 203 us, 6.35 TB/s of those bytes, 94 % of a plain copy's rate. Five blocks of
// four warps per SM (96 registers) hold 160 KB of rows in flight; two blocks of eight warps took
// 221 us, seven of four (73 registers, with spills) 223 us.
#include <cuda_fp8.h>

#include "nx_internal.cuh"

namespace nx {
namespace {

constexpr int kImageWarps = 4;

struct ImageArgs {
  nx_cache c;
  nx_image im;
  const int32_t* rows_in;
  int32_t* dev_status;
  int parts;            // thread blocks per slice
  int b;                // rows per block
  bool set_rows;        // the kernel sets the new row counts itself
};

// Rows of the slice (T) and rows that the image holds already (held); false if either is bad.
__device__ __forceinline__ bool image_range(const ImageArgs& g, int slice, int& T, int& held,
                                            int& flag) {
  T = g.c.lens[slice];
  held = g.rows_in[slice];
  flag = 0;
  if (T < 0 || T > g.c.capacity) flag = NX_DEV_BAD_LEN;
  else if (held < 0 || held > T || held % g.b) flag = NX_DEV_BAD_IMAGE;
  return flag == 0;
}

// The larger of both halves of finite bf16 magnitudes (infinities and NaN count as 0).
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t x) {
  x &= 0x7FFF7FFFu;
  return __vmaxu2(m, x & __vcmpltu2(x, 0x7F807F80u));
}

__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float inv) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
      make_float2(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv),
      __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
      make_float2(__uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv),
      __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// NV: 16-byte loads per lane and block (block rows x head_dim x 2 bytes / 512).
template <int NV>
__global__ void __launch_bounds__(kImageWarps * 32, 5) quantize_kernel(ImageArgs g) {
  grid_dep_wait();
  const nx_cache& c = g.c;
  const int slice = blockIdx.x / g.parts, part = blockIdx.x % g.parts;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int T, held, flag;
  const bool ok = image_range(g, slice, T, held, flag);
  if (!ok) {
    if (part == 0 && threadIdx.x == 0) atomicOr(g.dev_status, flag);
    return;
  }
  int l, s, h;
  slice_coords(c, slice, l, s, h);
  const int b = g.b, D = c.head_dim;
  const int first = held / b, tasks = 2 * (T / b - first);
  for (int i = part * kImageWarps + warp; i < tasks; i += g.parts * kImageWarps) {
    const int slot = (first + i / 2) * b;
    const bool is_v = i & 1;
    const long long row = row_of(c, l, s, h, slot);
    if (row < 0) {
      if (lane == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(is_v ? c.v : c.k) + row * D) + lane;
    uint4 x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] = __ldcs(src + 32 * j);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      m = finite_max(finite_max(finite_max(finite_max(m, x[j].x), x[j].y), x[j].z), x[j].w);
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    // the least power of two s with |x| <= 448 s = 1.75 2^8 s
    int e = 0;
    if (m) {
      int k;
      const float f = frexpf(__uint_as_float(m << 16), &k);    // f 2^k, f in [0.5, 1)
      e = f > 0.875f ? k - 8 : k - 9;
      e = e < -100 ? -100 : e > 120 ? 120 : e;
    }
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint2* dst = reinterpret_cast<uint2*>(
        static_cast<unsigned char*>(is_v ? g.im.v : g.im.k) + row * D) + lane;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      dst[32 * j] = make_uint2(codes4(x[j].x, x[j].y, inv), codes4(x[j].z, x[j].w, inv));
    if (lane == 0)
      (is_v ? g.im.v_scale : g.im.k_scale)[image_scale_at(c, l, s, h, slot, b)] =
          __uint_as_float((uint32_t)(127 + e) << 23);
  }
  if (g.set_rows && part == 0) {
    __syncthreads();                  // one block per slice: everyone has read the old count
    if (threadIdx.x == 0) g.im.rows[slice] = T / b * b;
  }
}

// The new row counts, where several thread blocks of a slice read them from the same place.
__global__ void image_rows_kernel(ImageArgs g, int slices) {
  grid_dep_wait();
  const int slice = blockIdx.x * blockDim.x + threadIdx.x;
  int T, held, flag;
  if (slice < slices && image_range(g, slice, T, held, flag)) g.im.rows[slice] = T / g.b * g.b;
}

}  // namespace

bool valid_image(const nx_image* im) {
  return im && im->k && im->v && im->k_scale && im->v_scale && im->rows &&
         !((uintptr_t)im->k & 15u) && !((uintptr_t)im->v & 15u) &&
         aligned4(im->k_scale, im->v_scale, im->rows);
}

}  // namespace nx

extern "C" nx_status nexus_quantize(const nx_cache* cache, const nx_image* image,
                                    const int32_t* rows_in, int32_t* dev_status,
                                    nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !valid_image(image) || !dev_status ||
      !aligned4(cache->lens, cache->block_table, rows_in, dev_status))
    return NX_ERR_INVALID_ARG;
  if (cache->dtype != NX_DTYPE_BF16) return NX_ERR_UNSUPPORTED;
  const long long slices = (long long)cache->layers * cache->seqs * cache->kv_heads;
  if (rows_in && rows_in != image->rows && rows_in < image->rows + slices &&
      image->rows < rows_in + slices)
    return NX_ERR_INVALID_ARG;
  ImageArgs g{};
  g.c = *cache;
  g.im = *image;
  g.rows_in = rows_in ? rows_in : image->rows;
  g.dev_status = dev_status;
  g.b = image_block(*cache);
  const bool in_place = g.rows_in == image->rows;
  // as many thread blocks per slice as its blocks can feed, up to about sixteen per SM in all
  const long long feed = (2LL * (cache->capacity / g.b) + kImageWarps - 1) / kImageWarps;
  const long long want = (152LL * 16 + slices - 1) / slices;
  g.parts = (int)(feed < want ? feed : want);
  if (g.parts < 1) g.parts = 1;
  g.set_rows = !in_place || g.parts == 1;
  if (slices * g.parts > 0x7FFFFFFFLL) return NX_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(slices * g.parts)), block(kImageWarps * 32);
  cudaError_t e;
  switch (g.b * cache->head_dim * 2 / 512) {
    case 16: e = launch_after(quantize_kernel<16>, grid, block, 0, st, g); break;
    case 8: e = launch_after(quantize_kernel<8>, grid, block, 0, st, g); break;
    case 4: e = launch_after(quantize_kernel<4>, grid, block, 0, st, g); break;
    default: e = launch_after(quantize_kernel<2>, grid, block, 0, st, g); break;
  }
  if (e != cudaSuccess) return finish(e, launches);
  note_launch(st, &launches, "quantize");
  if (!g.set_rows) {
    e = launch_after(image_rows_kernel, dim3((unsigned)((slices + 255) / 256)), dim3(256), 0, st,
                     g, (int)slices);
    if (e == cudaSuccess) note_launch(st, &launches, "image_rows");
  }
  return finish(e, launches);
}
