// nx_plan.cu -- nexus_plan: the next batch laid out on the GPU, from the tokens that each sequence
// brings and the rows that its slices hold: pages of the pool given back and dealt out, the
// sequences' places in the per-token arrays, each token's sequence and position.
//
// Every number depends on the sequences before: three running sums over the sequences (tokens,
// pages given back, pages taken), after which each page and each token finds its sequence by a
// search in the sums and moves by itself. One cluster of eight thread blocks does it all in one
// launch: the lengths of all slices, its largest read, are reduced by a warp per sequence and
// pushed to all blocks; the sums are then worked out by every block for itself (S values from its
// shared memory: cheaper than asking another); where pages are both given back and taken, which may
// be the same ones, a cluster barrier stands between.
//
// What bounds it: a chain of latencies (lengths, the barrier, the sums, the pages taken). 16 sequences of
// 32 x 8 slices that go on by a token 3.7 us on the GPU, 256 of which a third end, arrive or were
// evicted 9.3, prompts of up to 2048 tokens in 96 places 8.1; three sums one after the other instead of
// one, and inputs fetched behind the first barrier: 8.2, 11.5, 11.8.
#include "nx_internal.cuh"

namespace nx {
namespace {

constexpr int kPlanRanks = 8;         // thread blocks, one cluster (the portable limit)

struct PlanArgs {
  nx_cache c;
  nx_pool p;            // p.held null: contiguous, no pages
  nx_plan a;
  int32_t* dev_status;
  const int32_t *free_in, *held_in;
  int32_t* image_rows;  // or null
  int shift;            // log2 page_size
};

// The running sums over sequences: tokens, pages given back, pages taken.
struct Sums {
  long long v[3];
};
// What the threads before this one have, and what all have.
template <int WARPS>
__device__ __forceinline__ Sums block_before(const Sums& x, Sums* s_sum, Sums& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  Sums incl = x, before;
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long y = __shfl_up_sync(0xffffffffu, incl.v[i], o);
      if (lane >= o) incl.v[i] += y;
    }
  __syncthreads();                       // the sums before are read
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    long long w = lane < WARPS ? s_sum[lane].v[i] : 0, b = lane < warp ? w : 0;
#pragma unroll
    for (int o = 16; o; o /= 2) {
      w += __shfl_xor_sync(0xffffffffu, w, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    total.v[i] = w;
    before.v[i] = b + incl.v[i] - x.v[i];
  }
  return before;
}

// The sequence whose share of a running sum holds place i: the last s with at[s] <= i.
__device__ __forceinline__ int owner_of(const int* at, int n, int i) {
  int lo = 0;
  for (int hi = n; hi - lo > 1;) {
    const int mid = (lo + hi) / 2;
    if (at[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void push(int* p, int rank, int x) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(smem_at(p)),
      "r"(rank), "r"(x)
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const __grid_constant__ PlanArgs g) {
  constexpr int kPlanWarps = kPlanThreads / 32, kPlanStep = kPlanRanks * kPlanThreads;
  extern __shared__ int s_mem[];
  __shared__ Sums s_sum[kPlanWarps];
  const int S = g.c.seqs, H = g.c.kv_heads, per = g.c.layers * H;
  int* s_rows = s_mem;                   // rows of the longest slice (-1: a bad one), then pages
  int* s_new = s_rows + S;               // tokens asked for
  int* s_held = s_new + S;               // pages held before
  int* s_cu = s_held + S;                // tokens granted (-1: refused); then the running sums:
  int* s_give = s_cu + S;                // tokens, pages given back,
  int* s_take = s_give + S;              // pages taken
  int* s_first = s_take + S;             // position of the first token
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, rank = blockIdx.x;
  const int all = rank * kPlanThreads + tid;
  const bool lead = rank == 0, paged = g.p.held != nullptr;
  grid_dep_wait();
  // pushes must find the other blocks running; the inputs come meanwhile
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  for (int s = tid; s < S; s += kPlanThreads) {
    s_new[s] = g.a.new_tokens[s];
    s_held[s] = paged ? g.held_in[s] : 0;
    s_first[s] = g.a.token_pos ? g.a.first_pos[s] : 0;
  }
  int free_before = paged ? *g.free_in : 0;
  bool pushed = false;
  for (int s = rank * kPlanWarps + warp; s < S; s += kPlanRanks * kPlanWarps) {
    int most = 0, least = 0;
#pragma unroll 8
    for (int i = lane; i < per; i += 32) {
      const int l = i / H, len = g.c.lens[((long long)l * S + s) * H + (i - l * H)];
      most = max(most, len);
      least = min(least, len);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (!pushed) asm volatile("barrier.cluster.wait;" ::: "memory");
    pushed = true;
    if (lane < kPlanRanks) push(&s_rows[s], lane, least < 0 || most > g.c.capacity ? -1 : most);
  }
  if (!pushed) asm volatile("barrier.cluster.wait;" ::: "memory");
  cluster_sync();                        // all lengths are there, and all inputs are read
  // ---- what each sequence gets: a run of sequences to each thread ----
  const int run = (S + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(S, tid * run), s1 = min(S, s0 + run);
  Sums x = {}, total;
  for (int s = s0; s < s1; ++s) {
    const int held = s_held[s], asked = s_new[s], n = max(asked, 0);
    const int rows = asked < 0 ? 0 : s_rows[s];    // (the lengths of one that ends do not matter)
    int flag = 0;
    if (held < 0 || (paged && held > g.c.max_pages_per_seq)) flag = NX_DEV_BAD_PAGE;
    else if (rows < 0) flag = NX_DEV_BAD_LEN;
    else if (n > g.a.max_tokens) flag = NX_DEV_BAD_TOKENS;
    else if (n > g.c.capacity - rows) flag = NX_DEV_FULL;
    if (flag && lead) atomicOr(g.dev_status, flag);
    s_cu[s] = flag ? -1 : n;
    const int need = flag ? held : paged ? (rows + n + (1 << g.shift) - 1) >> g.shift : 0;
    s_rows[s] = need;
    x.v[0] += flag ? 0 : n;
    x.v[1] += max(0, held - need);
    x.v[2] += max(0, need - held);
  }
  Sums before = block_before<kPlanWarps>(x, s_sum, total);
  if (paged && (free_before < 0 || free_before > g.c.num_pages)) {
    if (lead && tid == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
    free_before = 0;
  }
  // Mostly there is room for all. If not, once more without those that the arrays have no room for,
  // then without those that the pool has no pages for: in order, so that who would need more than
  // are left waits, and whoever wants any behind.
  if (total.v[0] > g.a.tokens) {
    x = {};
    for (int s = s0; s < s1; ++s) {
      if (s_cu[s] > 0) {
        before.v[0] += s_cu[s];
        if (before.v[0] > g.a.tokens) {
          if (lead) atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
          s_cu[s] = -1;
          s_rows[s] = s_held[s];
        }
      }
      x.v[0] += max(0, s_cu[s]);
      x.v[1] += max(0, s_held[s] - s_rows[s]);
      x.v[2] += max(0, s_rows[s] - s_held[s]);
    }
    before = block_before<kPlanWarps>(x, s_sum, total);
  }
  int given = 0, top = 0;
  if (paged) {
    if (total.v[1] > g.c.num_pages - free_before) {     // more pages than there are
      if (lead && tid == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
      total.v[1] = g.c.num_pages - free_before;
    }
    given = (int)total.v[1];
    top = free_before + given;
    if (total.v[2] > top) {
      x = {};
      for (int s = s0; s < s1; ++s) {
        const int more = s_rows[s] - s_held[s];
        if (more > 0) {
          before.v[2] += more;
          if (before.v[2] > top) {
            if (lead) atomicOr(g.dev_status, NX_DEV_NO_PAGES);
            s_cu[s] = -1;
            s_rows[s] = s_held[s];
          }
        }
        x.v[0] += max(0, s_cu[s]);
        x.v[1] += max(0, -more);
        x.v[2] += max(0, s_rows[s] - s_held[s]);
      }
      before = block_before<kPlanWarps>(x, s_sum, total);
    }
  }
  const int taken = (int)total.v[2], N = (int)total.v[0];
  for (int s = s0; s < s1; ++s) {
    const int n = max(0, s_cu[s]), more = s_rows[s] - s_held[s];
    s_cu[s] = (int)before.v[0];
    s_give[s] = (int)min(before.v[1], (long long)given);
    s_take[s] = (int)before.v[2];
    if (lead) g.a.cu_tokens[s] = (int)before.v[0];
    before.v[0] += n;
    before.v[1] += max(0, -more);
    before.v[2] += max(0, more);
  }
  if (lead && tid == 0) g.a.cu_tokens[S] = N;
  __syncthreads();
  // ---- pages back, on top of the free ones ----
  const long long columns = g.c.max_pages_per_seq;
  for (unsigned i = all; i < (unsigned)given; i += kPlanStep) {
    const int s = owner_of(s_give, S, i);
    g.p.free_pages[free_before + i] = g.p.block_table[s * columns + s_rows[s] + i - s_give[s]];
  }
  const bool wait = given > 0 && taken > 0;       // taken ones may be among them
  if (wait) asm volatile("barrier.cluster.arrive;" ::: "memory");
  // ---- the tokens ----
  if (g.a.token_seq || g.a.token_pos)
    for (unsigned i = all; i < (unsigned)N; i += kPlanStep) {
      const int s = owner_of(s_cu, S, i);
      if (g.a.token_seq) g.a.token_seq[i] = s;
      if (g.a.token_pos) g.a.token_pos[i] = s_first[s] + (int)i - s_cu[s];
    }
  // ---- sequences that end (a refused one still holds pages) ----
  for (int s = rank * kPlanWarps + warp; s < S; s += kPlanRanks * kPlanWarps) {
    if (s_new[s] >= 0 || s_rows[s] != 0) continue;
    for (int i = lane; i < per; i += 32) {
      const int l = i / H;
      const long long at = ((long long)l * S + s) * H + (i - l * H);
      g.c.lens[at] = 0;
      if (g.image_rows) g.image_rows[at] = 0;
    }
  }
  if (!paged) return;
  if (wait) asm volatile("barrier.cluster.wait;" ::: "memory");
  // ---- pages taken, from the top ----
  for (unsigned i = all; i < (unsigned)taken; i += kPlanStep) {
    const int s = owner_of(s_take, S, i);
    g.p.block_table[s * columns + s_held[s] + i - s_take[s]] =
        __ldcg(g.p.free_pages + (top - 1 - (int)i));
  }
  if (lead) {
    for (int s = tid; s < S; s += kPlanThreads) g.p.held[s] = s_rows[s];
    if (tid == 0) *g.p.free_count = top - taken;
  }
}

template <int THREADS>
cudaError_t launch_plan(const PlanArgs& g, cudaStream_t st) {
  const int smem = 7 * g.c.seqs * (int)sizeof(int);
  if (smem > 32 * 1024) {
    const cudaError_t e = allow_smem<plan_kernel<THREADS>>(7 * kMaxPlanSeqs * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  return launch_after_clusters(plan_kernel<THREADS>, dim3(kPlanRanks), dim3(THREADS), smem,
                               kPlanRanks, st, g);
}

bool overlap(const int32_t* a, const int32_t* b, long long n) {
  return a != b && a < b + n && b < a + n;
}

}  // namespace
}  // namespace nx

extern "C" nx_status nexus_plan(nx_cache* cache, const nx_pool* pool, const nx_plan* plan,
                                const nx_image* image, int32_t* dev_status, nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !plan || !dev_status) return NX_ERR_INVALID_ARG;
  if (image && !valid_image(image)) return NX_ERR_INVALID_ARG;
  if (image && cache->dtype != NX_DTYPE_BF16) return NX_ERR_UNSUPPORTED;
  const nx_plan& a = *plan;
  if ((pool != nullptr) != (cache->page_size > 0)) return NX_ERR_INVALID_ARG;
  if (!a.new_tokens || !a.cu_tokens || a.tokens < 0 || a.max_tokens < 1 ||
      (a.tokens > 0 && (a.token_pos != nullptr) != (a.first_pos != nullptr)))
    return NX_ERR_INVALID_ARG;
  if (!aligned4(cache->lens, a.new_tokens, a.first_pos, a.cu_tokens, a.token_seq, a.token_pos,
                dev_status))
    return NX_ERR_INVALID_ARG;
  PlanArgs g{};
  if (pool) {
    if (!pool->free_pages || !pool->free_count || !pool->held ||
        pool->block_table != cache->block_table)
      return NX_ERR_INVALID_ARG;
    if (!aligned4(pool->free_pages, pool->free_count, pool->held, pool->block_table,
                  pool->free_count_in, pool->held_in))
      return NX_ERR_INVALID_ARG;
    if (pool->held_in && overlap(pool->held_in, pool->held, cache->seqs)) return NX_ERR_INVALID_ARG;
    g.p = *pool;
    g.free_in = pool->free_count_in ? pool->free_count_in : pool->free_count;
    g.held_in = pool->held_in ? pool->held_in : pool->held;
    while (1 << g.shift < cache->page_size) ++g.shift;
  }
  if (cache->seqs > kMaxPlanSeqs || (long long)cache->layers * cache->kv_heads > (1 << 24))
    return NX_ERR_UNSUPPORTED;
  g.c = *cache;
  g.a = a;
  g.dev_status = dev_status;
  g.image_rows = image ? image->rows : nullptr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // few sequences and tokens: small blocks, whose barriers are shorter (16 sequences 4.1 us, not 5.0);
  // many keep larger ones busy (256 sequences 10.0 us, not 12.1)
  const bool few = cache->seqs <= 64 && a.tokens <= 4096;
  const cudaError_t e = few ? launch_plan<256>(g, st) : launch_plan<512>(g, st);
  if (e == cudaSuccess) note_launch(st, &launches, "plan");
  return finish(e, launches);
}
