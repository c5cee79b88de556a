// nx_attend_shared.cu -- nexus_attend_shared: attention over a prefix that several sequences share and
// over their own rows, with the kernels of nexus_attend.
//
// All tokens that share a prefix are query rows of the same units of work, so that its rows are read not
// once per sequence but, by the tensor cores, once for every 256 query rows: 64 sequences of 4 query heads
// per KV head to every 512 B. (The row kernel makes a pass for every 16, or 8.) Softmax sums over
// two sets of slots join by their maxima (see nx_attend_rows.cuh), in binary32, so the two sets are two
// passes, each by the kernel that suits it, which run over one another as far as they can:
//   - by the row kernel the prefixes' pass leaves (m, l, o) of every query row in the workspace and the
//     other takes them in where it finishes the row; it starts without waiting for the first;
//   - a prefix for the tensor cores holds an SM with each of its blocks. It takes as many SMs as its
//     share of the work, by the lengths it finds, the own rows' pass takes the others, and a third kernel
//     joins the pieces of both.
#include "nx_attend_rows.cuh"

namespace nx {

// Which of the two kernels takes a pass. Those of nexus_attend_shared (alone: attend_tc_takes): the
// row kernel's time goes by its passes of 16 query rows over the slots (from HBM each, where they do
// not fit L2), that of the tensor cores by the slots behind a dearer start, which pays early where
// there are few long slices. Both passes on the GPU, own slices of one row, in us (tensor cores / row
// kernel), prefixes of 8 slices with 20, 48, 96, 192 query rows:
//   bf16: 512 slots 17 / 15, 18 / 17, 19 / 18, 19 / 19; 2048 18 / 18, 20 / 19, 20 / 23, 22 / 32;
//   8192 28 / 28, 27 / 29, 28 / 45, 32 / 62; 32768 51 / 49, 51 / 65, 52 / 101, 58 / 174
//   8 bits: 512 20 / 18, 20 / 20, 20 / 20, 21 / 20; 8192 35 / 29, 36 / 31, 37 / 35, 41 / 59; 32768
//   63 / 45, 69 / 58, 70 / 84, 81 / 134;
// of 1 slice, 8192 slots: bf16 19 / 25, 20 / 25, 22 / 25, 23 / 25; 8 bits 21 / 26, 23 / 26, 24 / 27,
// 26 / 27; four prefixes of 8 slices: bf16, 512 slots 21 / 18, 22 / 18, 26 / 22, 28 / 43; 2048 29 / 23,
// 29 / 32, 31 / 47, 37 / 78; 32768 116 / 178, 116 / 254, 118 / 481, 144 / 868.
bool shared_tc_takes(const SharedArgs& g) {
  const bool image = g.im.k != nullptr;
  const long long passes = (most_tokens(g.t) * g.c.group + 15) / 16;
  if (g.c.dtype != NX_DTYPE_BF16 || passes < 2) return false;
  const long long slices = (long long)g.c.seqs * g.c.kv_heads, slots = slices * g.c.capacity;
  if (!image && slots * g.c.head_dim * 4 > 128LL << 20) return true;
  if (slices <= 8 && g.c.capacity >= 4096 && slots <= (image ? 1 << 15 : 1 << 17)) return true;
  return slots * (10 * passes - (image ? 50 : 23)) >= (g.c.capacity >= 1024 ? 450000 : 800000);
}

namespace {

// Thread blocks of the own rows' pass that can go where there is room: not those of one launch that
// deals its tiles to as many as fit the GPU at once.
template <int D>
long long free_blocks(SharedArgs g) {
  if (g.c.dtype == NX_DTYPE_F32) return plan_rows<kF32, D, 8>(g);
  if (shared_tc_takes(g)) return 0;
  const bool few = most_tokens(g.t) * g.c.group <= 8;
  if (g.im.k) return few ? plan_rows<kImage, D, 8>(g) : plan_rows<kImage, D, 16>(g);
  return few ? plan_rows<kBf16, D, 8>(g) : plan_rows<kBf16, D, 16>(g);
}

SharedArgs pass_args(const nx_cache& c, const nx_tokens& t, const nx_image* image, const nx_attend& a,
                     int pass, const AttendPart& part, char* ws, int32_t* dev_status) {
  SharedArgs g{};
  attend_args(&g, c, t, image, a, dev_status);
  g.pass = pass;
  g.part = part;
  if (shared_tc_takes(g)) attend_tc_layout(c.head_dim, ws, &g.ws);
  else attend_layout(c.head_dim, ws, &g.ws);
  return g;
}
cudaError_t launch_pass(SharedArgs& g, cudaStream_t st, int* launches) {
  if (shared_tc_takes(g)) return launch_attend_tc(g, st, launches);
  return g.c.head_dim == 128 ? launch_rows<128>(g, st, launches) : launch_rows<64>(g, st, launches);
}

// The tokens of nexus_attend_shared as the prefixes see them: those of a prefix's sequences are one
// sequence's. (Which ones go by cu_seqs too: shared_tokens.)
nx_tokens shared_view(const nx_tokens& t, const nx_shared& x) {
  nx_tokens y = t;
  y.max_tokens = x.max_tokens;
  return y;
}

bool valid_shared(const nx_cache& c, const nx_tokens& t, const nx_shared* x) {
  if (!x || x->reserved != 0 || x->max_tokens < 1 || !aligned4(x->cu_seqs)) return false;
  if (!valid_cache(x->prefix)) return false;
  const nx_cache& p = *x->prefix;
  return p.kv_heads == c.kv_heads && p.group == c.group && p.head_dim == c.head_dim &&
         p.dtype == c.dtype && t.layer < p.layers && (x->cu_seqs || p.seqs == 1);
}

// Workspaces of the own rows' pass and the prefixes', and where they meet.
size_t shared_layout(const nx_cache& c, const nx_tokens& t, const nx_shared& x, char* base,
                     char** own, char** prefix, AttendPart* part, int2** desc) {
  const size_t rows = (size_t)t.tokens * c.kv_heads * c.group;
  size_t at = 0;
  *own = base;
  at += round256(attend_bytes(c, t));
  *prefix = base + at;
  at += round256(attend_bytes(*x.prefix, shared_view(t, x)));
  part->stat = reinterpret_cast<float2*>(base + at);
  at += round256(rows * sizeof(float2));
  part->out = reinterpret_cast<float*>(base + at);
  at += round256(rows * c.head_dim * sizeof(float));
  if (!attend_tc_may_take(*x.prefix, shared_view(t, x))) return at;
  part->own_stat = reinterpret_cast<float2*>(base + at);
  at += round256(rows * sizeof(float2));
  part->own_out = reinterpret_cast<float*>(base + at);
  at += round256(rows * c.head_dim * sizeof(float));
  *desc = reinterpret_cast<int2*>(base + at);
  return at + round256(attend_tc_units(*x.prefix, shared_view(t, x)) * sizeof(int2));
}

}  // namespace
}  // namespace nx

extern "C" size_t nexus_attend_shared_workspace_bytes(const nx_cache* cache,
                                                      const nx_tokens* tokens,
                                                      const nx_shared* shared) {
  using namespace nx;
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens) ||
      !valid_shared(*cache, *tokens, shared))
    return 0;
  char *own, *prefix;
  AttendPart part{};
  int2* desc = nullptr;
  return shared_layout(*cache, *tokens, *shared, nullptr, &own, &prefix, &part, &desc);
}

extern "C" nx_status nexus_attend_shared(const nx_cache* cache, const nx_tokens* tokens,
                                         const nx_image* image, const nx_shared* shared,
                                         const nx_attend* args, void* ws, size_t ws_bytes,
                                         int32_t* dev_status, nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens) || !args || !dev_status ||
      !valid_shared(*cache, *tokens, shared))
    return NX_ERR_INVALID_ARG;
  const nx_tokens view = shared_view(*tokens, *shared);
  nx_status status = attend_limits(*cache, *tokens, image);
  if (status == NX_OK) status = attend_limits(*shared->prefix, view, shared->image);
  if (status == NX_OK) status = attend_pointers(*cache, *tokens, *args, dev_status);
  if (status != NX_OK) return status;
  char *own, *prefix;
  AttendPart part{};
  int2* desc = nullptr;
  const size_t need = shared_layout(*cache, *tokens, *shared, static_cast<char*>(ws), &own,
                                    &prefix, &part, &desc);
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < need) return NX_ERR_WORKSPACE;
  if (tokens->tokens == 0) return finish(cudaSuccess, launches);
  part.seqs = cache->seqs;
  part.max_tokens = tokens->max_tokens;
  part.prefixes = shared->prefix->seqs;
  part.max_shared = shared->max_tokens;
  part.cu_seqs = shared->cu_seqs;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  nx_attend whole = *args;                // the prefix comes before all of the new tokens
  whole.causal = 0;
  SharedArgs g = pass_args(*shared->prefix, view, shared->image, whole, 1, part, prefix, dev_status);
  const bool beside = shared_tc_takes(g);
  SharedArgs o = pass_args(*cache, *tokens, image, *args, beside ? 3 : 2, part, own, dev_status);
  if (beside) {
    g.part.desc = desc;
    g.part.own_lens = cache->lens + (long long)tokens->layer * cache->seqs * cache->kv_heads;
    // What the tensor-core kernel deals out the SMs by: a tile of a prefix counts 1.5 us of one of them
    // (3.5 from 8-bit rows; with 128 features and 256 query rows a tile takes 1.0 to 1.2, or 2.0, behind a
    // start of 8 to 11 us, or 17: 1.5 and 2.5 a tile over shares of 40 and 28. Other forms count the same),
    // a row of 128 features and 16 query rows of the other pass 10 ns (6). That
    // is no gain next to fewer blocks than two an SM (128 slices of 2048 rows next to 16384 slots, 54
    // us, not 60), which get room for all of them or none, or to a launch that counts on all SMs.
    const long long rows = most_tokens(*tokens) * cache->group, passes = (rows + 15) / 16;
    const long long cost = (image ? 6 : 10) * passes * cache->head_dim / 128 + 1;
    const long long blocks = cache->head_dim == 128 ? free_blocks<128>(o) : free_blocks<64>(o);
    g.part.tile_cost = shared->image ? 3500 : 1500;
    if (blocks >= 2 * kSms) g.part.row_cost = (int)(cost < 1000 ? cost : 1000);
    else g.part.room = (int)(blocks + 1) / 2;
  }
  cudaError_t e = launch_pass(g, st, &launches);
  if (e == cudaSuccess) e = launch_pass(o, st, &launches);
  if (e == cudaSuccess && beside) e = launch_attend_meet(g, st, &launches);
  return finish(e, launches);
}
