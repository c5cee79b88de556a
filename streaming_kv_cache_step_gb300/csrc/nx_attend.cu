// nx_attend.cu -- nexus_attend: softmax attention of new tokens over one layer's slices, by the kernel
// that takes them (nx_attend_rows.cuh, nx_attend_tc.cuh), and what nexus_attend_shared has in common.
#include "nx_attend_rows.cuh"

namespace nx {

size_t attend_layout(int D, char* base, AttendWs* ws) {
  size_t at = 0;
  ws->desc = reinterpret_cast<int2*>(base + at);
  at += round256(kAttendGrid * sizeof(int2));
  ws->stat = reinterpret_cast<float2*>(base + at);
  at += round256((size_t)2 * kAttendGrid * kPieceRows * sizeof(float2));
  ws->out = reinterpret_cast<float*>(base + at);
  return at + (size_t)2 * kAttendGrid * kPieceRows * D * sizeof(float);
}

// What nexus_attend and nexus_attend_shared check of a cache and the tokens that look into it.
nx_status attend_limits(const nx_cache& c, const nx_tokens& t, const nx_image* image) {
  if (image && !valid_image(image)) return NX_ERR_INVALID_ARG;
  if (!aligned4(c.lens, c.block_table)) return NX_ERR_INVALID_ARG;
  if (image && c.dtype != NX_DTYPE_BF16) return NX_ERR_UNSUPPORTED;
  // tiles (of at least 64 slots, and a partial one) of all units (of at least 8 rows)
  if ((long long)c.kv_heads * c.group > (1 << 20) || (long long)c.seqs * c.kv_heads > (1 << 24) ||
      most_tokens(t) * c.group > 0x7FFFFFFFLL - 256 ||             // rows of a slice, by tiles
      (long long)c.seqs * c.kv_heads * (most_tokens(t) * c.group / 8 + 1) >
          0x7FFFFFFFLL / (c.capacity / 64 + 2))
    return NX_ERR_UNSUPPORTED;
  return NX_OK;
}

nx_status attend_pointers(const nx_cache& c, const nx_tokens& t, const nx_attend& a,
                          int32_t* dev_status) {
  if (!aligned4(a.lse, dev_status)) return NX_ERR_INVALID_ARG;
  const int size = c.dtype == NX_DTYPE_BF16 ? 2 : 4;
  if (!isfinite(a.scale)) return NX_ERR_INVALID_ARG;
  if (a.q_stride < 0 || a.out_stride < 0 || a.q_stride * size % 16 || a.out_stride * size % 16 ||
      ((uintptr_t)a.q & 15u) || ((uintptr_t)a.out & 15u))
    return NX_ERR_INVALID_ARG;
  if (t.tokens > 0 && (!a.q || !a.out)) return NX_ERR_INVALID_ARG;
  if (t.tokens > 1 && a.out_stride < (long long)c.kv_heads * c.group * c.head_dim)
    return NX_ERR_INVALID_ARG;           // rows of out would overlap
  return NX_OK;
}

size_t attend_bytes(const nx_cache& c, const nx_tokens& t) {
  AttendWs ws;                            // of any cache of this type, with an image or without
  const size_t rows = attend_layout(c.head_dim, nullptr, &ws);
  const size_t tc = attend_tc_may_take(c, t) ? attend_tc_layout(c.head_dim, nullptr, &ws) : 0;
  return rows > tc ? rows : tc;
}

void attend_args(AttendArgs* g, const nx_cache& c, const nx_tokens& t, const nx_image* image,
                 const nx_attend& a, int32_t* dev_status) {
  g->c = c;
  g->t = t;
  if (image) g->im = *image;
  g->a = a;
  g->dev_status = dev_status;
  g->b = image_block(c);
  while (1 << g->b_shift < g->b) ++g->b_shift;
  g->c1 = a.scale * 1.4426950408889634f;
}

}  // namespace nx

extern "C" size_t nexus_attend_workspace_bytes(const nx_cache* cache, const nx_tokens* tokens) {
  using namespace nx;
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens)) return 0;
  return attend_bytes(*cache, *tokens);
}

extern "C" nx_status nexus_attend(const nx_cache* cache, const nx_tokens* tokens,
                                  const nx_image* image, const nx_attend* args, void* ws,
                                  size_t ws_bytes, int32_t* dev_status, nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens) || !args || !dev_status)
    return NX_ERR_INVALID_ARG;
  nx_status status = attend_limits(*cache, *tokens, image);
  if (status == NX_OK) status = attend_pointers(*cache, *tokens, *args, dev_status);
  if (status != NX_OK) return status;
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < attend_bytes(*cache, *tokens))
    return NX_ERR_WORKSPACE;
  if (tokens->tokens == 0) return finish(cudaSuccess, launches);
  AttendArgs g{};
  attend_args(&g, *cache, *tokens, image, *args, dev_status);
  char* base = static_cast<char*>(ws);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (attend_tc_takes(*cache, *tokens, image != nullptr)) {
    attend_tc_layout(cache->head_dim, base, &g.ws);
    return finish(launch_attend_tc(g, st, &launches), launches);
  }
  attend_layout(cache->head_dim, base, &g.ws);
  return finish(cache->head_dim == 128 ? launch_rows<128>(g, st, &launches)
                                       : launch_rows<64>(g, st, &launches),
                launches);
}
