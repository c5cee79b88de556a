// nx_plan.cu -- nexus_plan: the next batch laid out on the GPU, from the tokens that each sequence
// brings and the rows that its slices hold: pages of the pool given back and dealt out, the
// sequences' places in the per-token arrays, each token's sequence and position.
//
// Every number depends on the sequences before: three running sums over the sequences (tokens,
// pages given back, pages taken), after which each page and each token finds its sequence by a
// search in the sums and moves by itself. One cluster of eight thread blocks does it all in one
// launch: the lengths of all slices, its largest read, are reduced by a warp per sequence and
// pushed to all blocks; the sums are then worked out by every block for itself (S values from its
// shared memory: cheaper than asking another); a cluster barrier stands between the pages given
// back and those taken, which may be the same.
#include "nx_internal.cuh"

namespace nx {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanRanks = 8;         // thread blocks, one cluster (the portable limit)
constexpr int kPlanStep = kPlanRanks * kPlanThreads;

struct PlanArgs {
  nx_cache c;
  nx_pool p;            // p.held null: contiguous, no pages
  nx_plan a;
  int32_t* dev_status;
  const int32_t *free_in, *held_in;
  int32_t* image_rows;  // or null
  int shift;            // log2 page_size
};

// Sums over all threads' values of what comes before this thread's; total: of all.
__device__ __forceinline__ long long block_before(long long x, long long* s_sum, long long& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();                       // the sums before are read
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  long long w = s_sum[lane], before = lane < warp ? w : 0;
#pragma unroll
  for (int o = 16; o; o /= 2) {
    w += __shfl_xor_sync(0xffffffffu, w, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  total = w;
  return before + incl - x;
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

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const __grid_constant__ PlanArgs g) {
  extern __shared__ int s_mem[];
  __shared__ long long s_sum[kPlanWarps];
  const int S = g.c.seqs, H = g.c.kv_heads, per = g.c.layers * H;
  int* s_rows = s_mem;                   // rows of the longest slice (-1: a bad one), then pages
  int* s_held = s_rows + S;              // pages held before
  int* s_cu = s_held + S;                // the running sums: tokens,
  int* s_give = s_cu + S;                // pages given back,
  int* s_take = s_give + S;              // pages taken
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, rank = blockIdx.x;
  const int all = rank * kPlanThreads + tid;
  const bool lead = rank == 0;
  grid_dep_wait();
  cluster_sync();                        // every block's shared memory is there
  // ---- rows ----
  for (int s = rank * kPlanWarps + warp; s < S; s += kPlanRanks * kPlanWarps) {
    int most = 0, least = 0;
    if (g.a.new_tokens[s] >= 0) {        // (the lengths of one that ends do not matter)
#pragma unroll 8
      for (int i = lane; i < per; i += 32) {
        const int l = i / H, len = g.c.lens[((long long)l * S + s) * H + (i - l * H)];
        most = max(most, len);
        least = min(least, len);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      least = __reduce_min_sync(0xffffffffu, least);
    }
    if (lane < kPlanRanks) push(&s_rows[s], lane, least < 0 || most > g.c.capacity ? -1 : most);
  }
  int free_before = g.p.held ? *g.free_in : 0;
  cluster_sync();
  // ---- what each sequence gets: a run of sequences to each thread ----
  const int run = (S + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(S, tid * run), s1 = min(S, s0 + run);
  // A refused sequence brings no tokens and keeps its pages: s_cu holds -1 for now.
  long long total, sum = 0;
  for (int s = s0; s < s1; ++s) {
    int n = g.a.new_tokens[s], flag = 0;
    const int held = g.p.held ? g.held_in[s] : 0, rows = s_rows[s];
    if (held < 0 || (g.p.held && held > g.c.max_pages_per_seq)) flag = NX_DEV_BAD_PAGE;
    else if (rows < 0) flag = NX_DEV_BAD_LEN;
    else if (n > g.a.max_tokens) flag = NX_DEV_BAD_TOKENS;
    else if (n > g.c.capacity - rows) flag = NX_DEV_FULL;
    if (flag && lead) atomicOr(g.dev_status, flag);
    n = max(n, 0);
    s_held[s] = held;
    s_cu[s] = flag ? -1 : n;
    if (!flag) sum += n;
    if (g.p.held) s_rows[s] = flag ? held : (rows + n + (1 << g.shift) - 1) >> g.shift;
  }
  long long before = block_before(sum, s_sum, total);
  const bool crowded = total > g.a.tokens;
  long long give = 0, take = 0;
  for (int s = s0; s < s1; ++s) {
    if (crowded && s_cu[s] > 0) {
      before += s_cu[s];
      if (before > g.a.tokens) {
        if (lead) atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
        s_cu[s] = -1;
        s_rows[s] = s_held[s];
      }
    }
    if (g.p.held) {
      give += max(0, s_held[s] - s_rows[s]);
      take += max(0, s_rows[s] - s_held[s]);
    }
  }
  int given = 0, taken = 0, top = 0;
  if (g.p.held) {
    if (free_before < 0 || free_before > g.c.num_pages) {
      if (lead && tid == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
      free_before = 0;
    }
    long long gives, takes;
    give = block_before(give, s_sum, gives);
    if (gives > g.c.num_pages - free_before) {   // more pages than there are
      if (lead && tid == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
      gives = g.c.num_pages - free_before;
    }
    given = (int)gives;
    top = free_before + given;
    take = block_before(take, s_sum, takes);
    // pages are dealt out in order: who would need more than are left waits, and whoever takes
    // any behind
    const bool short_of = takes > top;
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
      const int more = s_rows[s] - s_held[s];
      s_give[s] = (int)min(give, (long long)given);
      give += max(0, -more);
      if (more <= 0) continue;
      take += more;
      if (short_of && take > top) {
        if (lead) atomicOr(g.dev_status, NX_DEV_NO_PAGES);
        s_cu[s] = -1;
        s_rows[s] = s_held[s];
      } else {
        mine += more;
      }
    }
    mine = block_before(mine, s_sum, takes);
    taken = (int)takes;
    for (int s = s0; s < s1; ++s) {
      s_take[s] = (int)mine;
      mine += max(0, s_rows[s] - s_held[s]);
    }
  }
  sum = 0;
  for (int s = s0; s < s1; ++s) sum += max(0, s_cu[s]);
  before = block_before(sum, s_sum, total);
  const int N = (int)total;
  for (int s = s0; s < s1; ++s) {
    const int n = max(0, s_cu[s]);
    s_cu[s] = (int)before;
    if (lead) g.a.cu_tokens[s] = (int)before;
    before += n;
  }
  if (lead && tid == 0) g.a.cu_tokens[S] = N;
  __syncthreads();
  // ---- pages back, on top of the free ones ----
  const long long columns = g.c.max_pages_per_seq;
  for (unsigned i = all; i < (unsigned)given; i += kPlanStep) {
    const int s = owner_of(s_give, S, i);
    g.p.free_pages[free_before + i] = g.p.block_table[s * columns + s_rows[s] + i - s_give[s]];
  }
  // ---- the tokens ----
  if (g.a.token_seq || g.a.token_pos)
    for (unsigned i = all; i < (unsigned)N; i += kPlanStep) {
      const int s = owner_of(s_cu, S, i);
      if (g.a.token_seq) g.a.token_seq[i] = s;
      if (g.a.token_pos) g.a.token_pos[i] = g.a.first_pos[s] + i - s_cu[s];
    }
  // ---- sequences that end ----
  for (int s = rank * kPlanWarps + warp; s < S; s += kPlanRanks * kPlanWarps) {
    if (g.a.new_tokens[s] >= 0) continue;
    if (g.p.held && (s_rows[s] > 0 || s_held[s] < 0)) continue;     // refused
    for (int i = lane; i < per; i += 32) {
      const int l = i / H;
      const long long at = ((long long)l * S + s) * H + (i - l * H);
      g.c.lens[at] = 0;
      if (g.image_rows) g.image_rows[at] = 0;
    }
  }
  if (!g.p.held) return;
  cluster_sync();                        // the pages given back are there, all inputs are read
  // ---- pages taken, from the top ----
  for (unsigned i = all; i < (unsigned)taken; i += kPlanStep) {
    const int s = owner_of(s_take, S, i);
    g.p.block_table[s * columns + s_held[s] + i - s_take[s]] =
        __ldcg(g.p.free_pages + (top - 1 - i));
  }
  if (lead) {
    for (int s = tid; s < S; s += kPlanThreads) g.p.held[s] = s_rows[s];
    if (tid == 0) *g.p.free_count = top - taken;
  }
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
  const int smem = 5 * cache->seqs * (int)sizeof(int);
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024) e = allow_smem<plan_kernel>(5 * kMaxPlanSeqs * (int)sizeof(int));
  if (e != cudaSuccess) return finish(e, launches);
  e = launch_after_clusters(plan_kernel, dim3(kPlanRanks), dim3(kPlanThreads), smem, kPlanRanks,
                            st, g);
  if (e == cudaSuccess) note_launch(st, &launches, "plan");
  return finish(e, launches);
}
