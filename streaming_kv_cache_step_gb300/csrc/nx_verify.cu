// nx_verify.cu -- nexus_verify: which drafted tokens stay, the token drawn behind the last one,
// and the cache without the rest.
//
// A draft x at row i stays while u_i q_i(x) < p_i(x), a product of two binary32 values and hence
// exact in binary64. At the first row r whose draft goes the next token comes from
// max(0, p_r - q_r), after the last row from p; drawing one is finding the first column whose
// inclusive sum of weights exceeds a threshold. Weights are whole numbers, units of 2^-42: their
// sums are exact in 64 bits and do not depend on who adds what, so that a row can be cut in any
// number of pieces and every result is the same bits (binary32 sums over 100000 columns would
// move the border between two tokens by some 2^-20 of the whole).
//
// Only one row of p (and of q) of each sequence is read, whatever the number of its drafts. A
// cluster of thread blocks takes a sequence, each warp a run of columns; block sums meet in shared
// memory, and the one warp whose run holds the threshold goes over it again, from L2.
#include "nx_internal.cuh"

namespace nx {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyPerSm = 2;          // thread blocks of an SM
constexpr int kVerifyRanks = 8;          // thread blocks of a sequence, at most
constexpr int kVec = 4;                  // columns of one load
constexpr float kUnit = 4398046511104.f; // 2^42

struct VerifyArgs {
  nx_cache c;
  nx_tokens t;
  nx_verify a;
  int32_t* dev_status;
  const int32_t* lens_in;
  int32_t* held;        // an image's rows, or null
  int b;                // rows per image block
  int ranks;            // thread blocks per sequence, one cluster
};

// A probability as it counts: NaN and what is negative as 0, what is above 1 as 1.
__device__ __forceinline__ float in_unit(float x) { return fminf(fmaxf(x, 0.f), 1.f); }

template <typename T>
__device__ __forceinline__ float value(const T* p) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(*p);
  else return *p;
}

// Four neighbouring values of a row, all there and aligned to their size.
__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 y = *reinterpret_cast<const float4*>(p);
  x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) {
  const uint2 y = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(y.x << 16), x[1] = __uint_as_float(y.x & 0xFFFF0000u);
  x[2] = __uint_as_float(y.y << 16), x[3] = __uint_as_float(y.y & 0xFFFF0000u);
}

// The row that a token is drawn from. Columns are counted from `shift` places before the row, so
// that every fourth one is aligned.
template <typename T>
struct Weights {
  const T *p, *q;       // the rows, `shift` places before them; q null: none is taken off
  int shift, end;       // columns [shift, end) exist
  int out;              // a column without weight (-1: none)
  bool q_vec;           // q is aligned like p

  __device__ __forceinline__ Weights(const T* row, const T* other, int V, int without) {
    shift = (int)((uintptr_t)row / sizeof(T) % kVec);
    end = shift + V;
    p = row - shift;
    q = other ? other - shift : nullptr;
    q_vec = (uintptr_t)q / sizeof(T) % kVec == 0;
    out = without < 0 ? -1 : without + shift;
  }
  __device__ __forceinline__ unsigned long long weigh(int col, float x, float y) const {
    const float w = fmaxf(in_unit(x) - in_unit(y), 0.f);
    return col == out ? 0ull : (unsigned long long)__float2ll_rz(w * kUnit);
  }
  __device__ __forceinline__ unsigned long long one(int col) const {
    if (col < shift || col >= end) return 0;
    return weigh(col, value(p + col), q ? value(q + col) : 0.f);
  }
  // columns col .. col + 3, col a multiple of 4
  __device__ __forceinline__ void fetch(int col, float* x, float* y) const {
    if (col >= shift && col + kVec <= end) {
      load4(p + col, x);
      if (!q) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) y[e] = 0.f;
      } else if (q_vec) {
        load4(q + col, y);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) y[e] = value(q + col + e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const bool ok = col + e >= shift && col + e < end;
        x[e] = ok ? value(p + col + e) : 0.f;
        y[e] = ok && q ? value(q + col + e) : 0.f;
      }
    }
  }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
  for (int o = 16; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ unsigned long long warp_before(unsigned long long x, int lane) {
  unsigned long long y = x;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const unsigned long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  return y - x;
}
__device__ __forceinline__ void push(unsigned long long* p, int rank, unsigned long long x) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u64 [a], %2;\n\t}" ::"r"(smem_at(p)),
      "r"(rank), "l"(x)
      : "memory");
}

// lens of a sequence's slices without the drafts that went, and the image without their blocks;
// thread `id` of all of the sequence's.
__device__ __forceinline__ void take_back(const VerifyArgs& g, int s, int gone, int id) {
  const int per = g.c.layers * g.c.kv_heads;
  for (int i = id; i < per; i += g.ranks * kVerifyThreads) {
    const int l = i / g.c.kv_heads, h = i - l * g.c.kv_heads;
    const long long at = ((long long)l * g.c.seqs + s) * g.c.kv_heads + h;
    const int len = g.lens_in[at];
    if (len < gone || len > g.c.capacity) {
      atomicOr(g.dev_status, NX_DEV_BAD_LEN);
      continue;
    }
    g.c.lens[at] = len - gone;
    const int hold = (len - gone) / g.b * g.b;
    if (g.held && g.held[at] > hold) g.held[at] = hold;
  }
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyPerSm) verify_kernel(VerifyArgs g) {
  __shared__ int s_first;
  __shared__ unsigned long long s_warp[kVerifyWarps], s_rank[2][kVerifyRanks];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int s = blockIdx.x / g.ranks, rank = blockIdx.x % g.ranks;
  const int V = g.a.vocab;
  const T* p = static_cast<const T*>(g.a.p);
  const T* q = static_cast<const T*>(g.a.q);
  grid_dep_wait();
  int first;
  const int n = tokens_of(g.t, s, first);
  if (n == 0) {
    if (tid == 0 && rank == 0) g.a.emitted[s] = 0;
    take_back(g, s, 0, rank * kVerifyThreads + tid);
    return;
  }
  if (n < 0) {                           // (the whole cluster goes)
    if (tid == 0 && rank == 0) {
      atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
      g.a.emitted[s] = 0;
    }
    return;
  }
  // pushes into another block's shared memory must find it running
  if (g.ranks > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  // ---- the first draft that goes ----
  if (tid == 0) s_first = n - 1;
  __syncthreads();
  for (int i = tid; i < n - 1; i += kVerifyThreads) {
    const long long row = first + i;
    const int x = g.a.token[row + 1];
    bool stays = false;
    if (x >= 0 && x < V) {
      const double want = in_unit(value(p + row * g.a.p_stride + x));
      const double had = q ? in_unit(value(q + row * g.a.q_stride + x)) : 1.0;
      stays = (double)g.a.u[row] * had < want;
    } else if (rank == 0) {
      atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
    }
    if (!stays) {
      atomicMin(&s_first, i);
      break;                             // this thread's later ones do not matter
    }
  }
  __syncthreads();
  const int r = s_first, gone = n - 1 - r;
  if (rank == 0) {
    for (int i = tid; i < n; i += kVerifyThreads)
      if (i != r) g.a.out[first + i] = i < r ? g.a.token[first + i + 1] : -1;
    if (tid == 0) g.a.emitted[s] = r + 1;
  }
  take_back(g, s, gone, rank * kVerifyThreads + tid);
  // ---- the draw ----
  const int next = gone ? g.a.token[first + r + 1] : -1;
  const T* row_p = p + (first + r) * g.a.p_stride;
  const T* row_q = gone && q ? q + (first + r) * g.a.q_stride : nullptr;
  Weights<T> w(row_p, row_q, V, gone && !q ? next : -1);
  // every warp's columns: whole loads of all lanes
  const int warps = g.ranks * kVerifyWarps;
  const int run = ((w.end + warps - 1) / warps + 32 * kVec - 1) / (32 * kVec) * (32 * kVec);
  const int c0 = (int)min((long long)w.end, (long long)(rank * kVerifyWarps + warp) * run);
  const int c1 = (int)min((long long)w.end, (long long)c0 + run);
  unsigned long long total = 0, before = 0;
  if (g.ranks > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    unsigned long long sum = 0;
    constexpr int kAhead = 4;            // loads of p, and of q, under way
#pragma unroll 1
    for (int c = c0 + lane * kVec; c < c1; c += kAhead * 32 * kVec) {
      float x[kAhead][kVec], y[kAhead][kVec];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int col = c + i * 32 * kVec;
        if (col < c1) {
          w.fetch(col, x[i], y[i]);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; ++e) x[i][e] = y[i][e] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum += w.weigh(c + i * 32 * kVec + e, x[i][e], y[i][e]);
    }
    sum = warp_sum(sum);
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (tid < g.ranks) {
      unsigned long long all = 0;
#pragma unroll
      for (int i = 0; i < kVerifyWarps; ++i) all += s_warp[i];
      if (g.ranks == 1) s_rank[round][0] = all;
      else push(&s_rank[round][rank], tid, all);
    }
    if (g.ranks == 1) __syncthreads();
    else
      asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
    total = before = 0;
    for (int i = 0; i < g.ranks; ++i) {
      if (i < rank) before += s_rank[round][i];
      total += s_rank[round][i];
    }
    if (total > 0 || round == 1) break;
    // nothing left of p behind q: the draw goes by p itself
    w = Weights<T>(row_p, nullptr, V, -1);
  }
  const double u = g.a.u_draw[s];
  const unsigned long long U =
      u > 0. ? (unsigned long long)fmin(u * 2147483648., 2147483647.) : 0ull;
  const unsigned long long t = U * (total >> 31) + (U * (total & 0x7FFFFFFFull) >> 31);
  if (total == 0) {
    if (rank == 0 && tid == 0) {
      atomicOr(g.dev_status, NX_DEV_BAD_PROBS);
      g.a.out[first + r] = 0;
    }
    return;
  }
  for (int i = 0; i < warp; ++i) before += s_warp[i];
  if (t < before || t - before >= s_warp[warp]) return;
  // ---- this warp's columns hold the threshold: which lane's, then which one ----
  const int each = run / 32;
  const int l0 = c0 + lane * each;
  unsigned long long sum = 0;
#pragma unroll 4
  for (int c = l0; c < min(l0 + each, c1); c += kVec) {
    float x[kVec], y[kVec];
    w.fetch(c, x, y);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum += w.weigh(c + e, x[e], y[e]);
  }
  unsigned long long mine = before + warp_before(sum, lane);
  const unsigned owner = __ballot_sync(0xffffffffu, t >= mine && t - mine < sum);
  if (!owner) return;                    // (only if somebody writes to the rows meanwhile)
  const int src = __ffs(owner) - 1;
  before = __shfl_sync(0xffffffffu, mine, src);
  for (int c = c0 + src * each, stop = c + each; c < stop; c += 32) {
    const int col = c + lane;
    const unsigned long long x = col < stop ? w.one(col) : 0ull;
    mine = before + warp_before(x, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, t >= mine && t - mine < x);
    if (hit) {
      if (lane == __ffs(hit) - 1) g.a.out[first + r] = col - w.shift;
      return;
    }
    before = __shfl_sync(0xffffffffu, mine + x, 31);
  }
}

// Thread blocks of a sequence: as many as fit the GPU at once for all sequences, but each with
// work for its warps.
int verify_ranks(int seqs, int vocab) {
  int ranks = kVerifyRanks;
  while (ranks > 1 && ((long long)seqs * ranks > kVerifyPerSm * 152 ||
                       vocab <= ranks / 2 * kVerifyThreads * kVec))
    ranks /= 2;
  return ranks;
}

}  // namespace
}  // namespace nx

extern "C" nx_status nexus_verify(nx_cache* cache, const nx_tokens* tokens, const nx_verify* args,
                                  const nx_image* image, int32_t* dev_status, nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens) || !args || !dev_status)
    return NX_ERR_INVALID_ARG;
  if (image && !valid_image(image)) return NX_ERR_INVALID_ARG;
  if (image && cache->dtype != NX_DTYPE_BF16) return NX_ERR_UNSUPPORTED;
  const nx_verify& a = *args;
  if (a.dtype != NX_DTYPE_F32 && a.dtype != NX_DTYPE_BF16) return NX_ERR_INVALID_ARG;
  if (a.reserved != 0 || a.vocab < 1) return NX_ERR_INVALID_ARG;
  if (a.vocab > kMaxVocab) return NX_ERR_UNSUPPORTED;
  const uintptr_t odd = a.dtype == NX_DTYPE_F32 ? 3u : 1u;
  if (((uintptr_t)a.p & odd) || ((uintptr_t)a.q & odd)) return NX_ERR_INVALID_ARG;
  if (!aligned4(cache->lens, a.token, a.u, a.u_draw, a.out, a.emitted, a.lens_in, dev_status))
    return NX_ERR_INVALID_ARG;
  if (a.p_stride < 0 || a.q_stride < 0 || !a.emitted) return NX_ERR_INVALID_ARG;
  if (tokens->tokens > 0 && (!a.token || !a.p || !a.u || !a.u_draw || !a.out))
    return NX_ERR_INVALID_ARG;
  const long long slices = (long long)cache->layers * cache->seqs * cache->kv_heads;
  if (a.lens_in && a.lens_in != cache->lens && a.lens_in < cache->lens + slices &&
      cache->lens < a.lens_in + slices)
    return NX_ERR_INVALID_ARG;
  if ((long long)cache->layers * cache->kv_heads > (1 << 24) || cache->seqs > (1 << 24))
    return NX_ERR_UNSUPPORTED;
  VerifyArgs g{};
  g.c = *cache;
  g.t = *tokens;
  g.a = a;
  g.dev_status = dev_status;
  g.lens_in = a.lens_in ? a.lens_in : cache->lens;
  g.held = image ? image->rows : nullptr;
  g.b = image_block(*cache);
  g.ranks = verify_ranks(cache->seqs, a.vocab);
  const dim3 grid((unsigned)(cache->seqs * g.ranks)), block(kVerifyThreads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a.dtype == NX_DTYPE_F32
          ? launch_after_clusters(verify_kernel<float>, grid, block, 0, g.ranks, st, g)
          : launch_after_clusters(verify_kernel<__nv_bfloat16>, grid, block, 0, g.ranks, st, g);
  if (e == cudaSuccess) note_launch(st, &launches, "verify");
  return finish(e, launches);
}
