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
// memory, and the block whose warp's run holds the threshold goes over that run again, from L2, with
// all its warps.
//
// What bounds it: latencies (lengths, drafts, their probabilities, the block sums: 5 us for five tokens
// of one sequence), then the rows: 64 sequences of 131072 binary32 columns, 67 MB with the drafts' rows, in
// 11.2 to 12.6 us on the GPU, by how many drafts stay (16.0 us a call with rows that are not in L2), 256
// draws from 65536 columns 13.6 us, 200 sequences of 50257 bf16 columns, 18 MB, 10.9 us. With each run
// searched by one warp those were 17.1, 24.3 and 18.2 where all warps of the block took 12.7, 16.2 and 14.2.
// Blocks of 256 threads, four an SM, took 11.4, 13.7 and 11.2 us, of 512, two an SM, 12.5, 12.9, 12.7, with
// twice the loads under way 12.1, 13.5, 12.6; three an SM 15.5, 15.2, 11.5.
#include "nx_internal.cuh"

namespace nx {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kAhead = 2;                // loads of p and of q under way (without q twice as many)
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyPerSm = 4;          // thread blocks of an SM
constexpr int kVerifyRanks = 8;          // thread blocks of a sequence, at most
template <typename T>
constexpr int kVecOf = 16 / (int)sizeof(T);     // columns of one load

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
__device__ __forceinline__ float in_unit(float x) { return __saturatef(x); }

// Sums of floor(2^42 w), 0 <= w <= 1, without a conversion to 64 bits (of which an SM makes one or
// two a clock: 256 rows of 65536 columns 47.8 us): added to 8, whose last place is worth 2^-20, w
// leaves its nearest multiple of that in the sum's low bits; what remains, at most 2^-21 and exact,
// leaves its multiple of 2^-42, rounded down, in those of 1.5 2^-19 in the same way. Up to 64
// weights fit 32 bits (the places' start values, `many` of each, come off modulo 2^32).
constexpr float kHigh = 8.f, kLow = 1.5f / 524288.f;
struct Counts {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(float w) {
    const float h = __fadd_rn(w, kHigh), rest = __fsub_rn(w, __fsub_rn(h, kHigh));
    hi += __float_as_uint(h);
    lo += __float_as_uint(__fadd_rd(rest, kLow));
  }
  __device__ __forceinline__ unsigned long long sum(int many) const {
    const uint32_t h = hi - many * __float_as_uint(kHigh);
    const int32_t l = (int32_t)(lo - many * __float_as_uint(kLow));
    return ((unsigned long long)h << 22) + (unsigned long long)(long long)l;
  }
};
__device__ __forceinline__ unsigned long long units(float w) {
  Counts c;
  c.add(w);
  return c.sum(1);
}

template <typename T>
__device__ __forceinline__ float value(const T* p) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(*p);
  else return *p;
}

// 16 bytes of neighbouring values, aligned, and what they are.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* p) {
  return *reinterpret_cast<const uint4*>(p);
}
template <typename T>
__device__ __forceinline__ float part(const uint4& x, int e) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
  else return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
}

// The row that a token is drawn from. Columns are counted from `shift` places before the row, so
// that loads start at multiples of their size.
template <typename T>
struct Weights {
  static constexpr int kVec = kVecOf<T>;
  const T *p, *q;       // the rows, `shift` places before them; q null: none is taken off
  int shift, end;       // columns [shift, end) exist
  int out;              // a column without weight (-1: none)
  bool q_vec;           // q is aligned like p

  __device__ __forceinline__ Weights(const T* row, const T* other, int V, int without) {
    shift = (int)((uintptr_t)row / sizeof(T) % kVec);
    end = shift + V;
    p = row - shift;
    q = other ? other - shift : nullptr;
    q_vec = (uintptr_t)q % 16 == 0;
    out = without < 0 || without >= V ? -1 : without + shift;
  }
  template <bool TWO>
  __device__ __forceinline__ float weigh(float x, float y) const {
    return TWO ? __saturatef(in_unit(x) - in_unit(y)) : in_unit(x);
  }
  __device__ __forceinline__ uint4 gather(const T* from, int col) const {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (col + e < shift || col + e >= end) continue;
      if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(from[col + e]);
      else
        w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(from)[col + e] << 16 * (e & 1);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // columns col .. col + kVec - 1, col a multiple of kVec; zeros for those that do not exist
  template <bool TWO>
  __device__ __forceinline__ void fetch(int col, uint4& x, uint4& y) const {
    const bool whole = col >= shift && col + kVec <= end;
    x = whole ? load16(p + col) : gather(p, col);
    if (TWO) y = whole && q_vec ? load16(q + col) : gather(q, col);
    else y = make_uint4(0, 0, 0, 0);
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

// The slices of a sequence, thread `id` of all of its blocks' every so many of them: lens without
// the drafts that went, and an image without their blocks. The first length is fetched early.
struct TakeBack {
  int i, len;
  static __device__ __forceinline__ long long at(const VerifyArgs& g, int s, int i) {
    const int l = i / g.c.kv_heads;
    return ((long long)l * g.c.seqs + s) * g.c.kv_heads + (i - l * g.c.kv_heads);
  }
  __device__ __forceinline__ TakeBack(const VerifyArgs& g, int s, int id) {
    i = id;
    len = i < g.c.layers * g.c.kv_heads ? g.lens_in[at(g, s, i)] : 0;
  }
  __device__ __forceinline__ void finish(const VerifyArgs& g, int s, int gone) {
    const int per = g.c.layers * g.c.kv_heads, step = g.ranks * kVerifyThreads;
    while (i < per) {
      const long long x = at(g, s, i);
      if (len < gone || len > g.c.capacity) {
        atomicOr(g.dev_status, NX_DEV_BAD_LEN);
      } else {
        g.c.lens[x] = len - gone;
        const int hold = (len - gone) / g.b * g.b;
        if (g.held && g.held[x] > hold) g.held[x] = hold;
      }
      i += step;
      if (i < per) len = g.lens_in[at(g, s, i)];
    }
  }
};

// The sum of the weights of columns [c0, c1), c0 a multiple of a load's, of one warp: a lane's part.
template <typename T, bool TWO, int AHEAD>
__device__ __forceinline__ unsigned long long lane_sum(const Weights<T>& w, int c0, int c1,
                                                       int lane) {
  constexpr int kVec = kVecOf<T>;
  unsigned long long sum = 0;
#pragma unroll 1
  for (int c = c0 + lane * kVec; c < c1; c += AHEAD * 32 * kVec) {
    uint4 x[AHEAD], y[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int col = c + i * 32 * kVec;
      x[i] = y[i] = make_uint4(0, 0, 0, 0);
      if (col < c1) w.template fetch<TWO>(col, x[i], y[i]);
    }
    Counts n;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        n.add(w.template weigh<TWO>(part<T>(x[i], e), part<T>(y[i], e)));
    static_assert(AHEAD * kVec <= 64, "");
    sum += n.sum(AHEAD * kVec);
  }
  // the column without weight comes off again
  if (!TWO && lane == 0 && w.out >= max(c0, w.shift) && w.out < c1)
    sum -= units(in_unit(value(w.p + w.out)));
  return sum;
}
template <typename T>
__device__ __forceinline__ unsigned long long columns_sum(const Weights<T>& w, int c0, int c1,
                                                          int lane) {
  return warp_sum(w.q ? lane_sum<T, true, kAhead>(w, c0, c1, lane)
                      : lane_sum<T, false, 2 * kAhead>(w, c0, c1, lane));
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyPerSm) verify_kernel(VerifyArgs g) {
  __shared__ int s_first;
  __shared__ unsigned long long s_warp[kVerifyWarps], s_part[kVerifyWarps];
  __shared__ unsigned long long s_rank[2][kVerifyRanks];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int s = blockIdx.x / g.ranks, rank = blockIdx.x % g.ranks;
  const int V = g.a.vocab;
  const T* p = static_cast<const T*>(g.a.p);
  const T* q = static_cast<const T*>(g.a.q);
  grid_dep_wait();
  int first;
  const int n = tokens_of(g.t, s, first);
  if (n < 0) {                           // (the whole cluster goes)
    if (tid == 0 && rank == 0) {
      atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
      g.a.emitted[s] = 0;
    }
    return;
  }
  TakeBack back(g, s, rank * kVerifyThreads + tid);
  if (n == 0) {
    if (tid == 0 && rank == 0) g.a.emitted[s] = 0;
    back.finish(g, s, 0);
    return;
  }
  const float u_draw = g.a.u_draw[s];
  // pushes into another block's shared memory must find it running: each thread waits before the
  // first of them, and its columns' loads come meanwhile
  if (g.ranks > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  // ---- the first draft that goes ----
  if (tid == 0) s_first = n - 1;
  if (n > 1) {
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
        break;                           // this thread's later ones do not matter
      }
    }
  }
  __syncthreads();
  const int r = s_first, gone = n - 1 - r;
  // ---- the draw: block sums ----
  const int next = gone ? g.a.token[first + r + 1] : -1;
  const T* row_p = p + (first + r) * g.a.p_stride;
  const T* row_q = gone && q ? q + (first + r) * g.a.q_stride : nullptr;
  Weights<T> w(row_p, row_q, V, gone && !q ? next : -1);
  // every warp's columns: whole loads of all lanes
  constexpr int kVec = kVecOf<T>, kLine = 32 * kVec;
  const int warps = g.ranks * kVerifyWarps;
  const int run = ((w.end + warps - 1) / warps + kLine - 1) / kLine * kLine;
  const int block0 = (int)min((long long)w.end, (long long)rank * kVerifyWarps * run);
  const int c0 = (int)min((long long)w.end, (long long)block0 + warp * run);
  const int c1 = (int)min((long long)w.end, (long long)c0 + run);
  unsigned long long total = 0, before = 0;
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    const unsigned long long sum = columns_sum(w, c0, c1, lane);
    if (lane == 0) s_warp[warp] = sum;
    if (round == 0 && g.ranks > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    __syncthreads();
    if (tid < g.ranks) {
      unsigned long long all = 0;
#pragma unroll
      for (int i = 0; i < kVerifyWarps; ++i) all += s_warp[i];
      if (g.ranks == 1) s_rank[round][0] = all;
      else push(&s_rank[round][rank], tid, all);
    }
    if (g.ranks == 1) {
      __syncthreads();
    } else {
      asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
    }
    total = before = 0;
    for (int i = 0; i < g.ranks; ++i) {
      if (i < rank) before += s_rank[round][i];
      total += s_rank[round][i];
    }
    if (total > 0 || round == 1) break;
    // nothing left of p behind q: the draw goes by p itself
    w = Weights<T>(row_p, nullptr, V, -1);
  }
  // ---- what does not wait for the draw ----
  back.finish(g, s, gone);
  if (rank == 0) {
    for (int i = tid; i < n; i += kVerifyThreads)
      if (i != r) g.a.out[first + i] = i < r ? g.a.token[first + i + 1] : -1;
    if (tid == 0) {
      g.a.emitted[s] = r + 1;
      if (total == 0) {
        atomicOr(g.dev_status, NX_DEV_BAD_PROBS);
        g.a.out[first + r] = 0;
      }
    }
  }
  // ---- the column: whose warp's run holds the threshold, which part of it, which line, lane ----
  const double u = u_draw;
  const unsigned long long U =
      u > 0. ? (unsigned long long)fmin(u * 2147483648., 2147483647.) : 0ull;
  const unsigned long long t = U * (total >> 31) + (U * (total & 0x7FFFFFFFull) >> 31);
  int owner = -1;
  if (t >= before)
    for (int i = 0; i < kVerifyWarps && owner < 0; ++i) {
      if (t - before < s_warp[i]) owner = i;
      else before += s_warp[i];
    }
  if (owner < 0) return;                 // another block's, or nobody's
  const int share = (run / kLine + kVerifyWarps - 1) / kVerifyWarps * kLine;
  const int r0 = block0 + owner * run, r1 = min(w.end, r0 + run);
  const int p0 = min(r1, r0 + warp * share), p1 = min(r1, p0 + share);
  const unsigned long long sum = columns_sum(w, p0, p1, lane);
  if (lane == 0) s_part[warp] = sum;
  __syncthreads();
  for (int i = 0; i < warp; ++i) before += s_part[i];
  if (t < before || t - before >= sum) return;
#pragma unroll 1
  for (int c = p0 + lane * kVec; c - lane * kVec < p1; c += kLine) {
    uint4 x, y;
    unsigned long long each[kVec], mine = 0;
    x = y = make_uint4(0, 0, 0, 0);
    if (c < p1) {
      if (w.q) w.template fetch<true>(c, x, y);
      else w.template fetch<false>(c, x, y);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      each[e] = c + e == w.out ? 0ull
                               : units(w.template weigh<true>(part<T>(x, e), part<T>(y, e)));
      mine += each[e];
    }
    unsigned long long at = before + warp_before(mine, lane);
    if (t >= at && t - at < mine) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (t >= at && t - at < each[e]) g.a.out[first + r] = c + e - w.shift;
        at += each[e];
      }
    }
    before = __shfl_sync(0xffffffffu, at + mine, 31);
    if (before > t) return;
  }
}

// Thread blocks of a sequence: as many as fit the GPU at once for all sequences, but each with
// work for its warps.
int verify_ranks(int seqs, int vocab) {
  const int fit = kVerifyPerSm * 152 / seqs;
  const int feed = (vocab + kVerifyThreads * 4 - 1) / (kVerifyThreads * 4);
  const int ranks = fit < feed ? fit : feed;
  return ranks < 1 ? 1 : ranks > kVerifyRanks ? kVerifyRanks : ranks;
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
  if (a.token && a.token < a.out + tokens->tokens && a.out < a.token + tokens->tokens)
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
