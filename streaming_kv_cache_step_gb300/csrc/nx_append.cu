// nx_append.cu -- nexus_append: RMS norm and position rotation of new queries and keys, and
// the rows of k, v and pos behind what every slice of one layer holds.
//
// One thread block takes kTokens tokens of one sequence. Its threads first compute the
// cosines and sines of those tokens (one pair each, shared by all heads of a token: 128
// features x 40 heads need 64 angles, not 2560), then a group of threads takes one head row of
// every token in turn, 16 features per thread (8 of fp32): what is the same for a head (where
// it reads and writes, norm weights, the slice's length) is found once. A thread's features are
// two runs that hold whole pairs (with runs of R: R i and rotary_dim / 2 + R i, or 2 R i and
// 2 R i + R when interleaved), so that a rotation needs no exchange between threads; only the
// norm's sum does. A thread's runs of the next tokens come into a ring of its own in shared memory
// by asynchronous copies, which hold no registers and start before the angles are computed.
//
// What bounds it: reads and writes of head rows, 2 B a value each way. 25144 tokens of prompts of
// up to 8192, 40 normed and rotated and 8 plain head rows of 128 each, bf16: 618 MB in 97.1 us,
// 6.37 TB/s, 94 % of a plain copy's rate (108 us with the next two tokens in registers); fp32, 1.24
// GB in 183 us, 6.74 TB/s. A single token of 48 head rows takes 2.6 us, all latency.
#include <type_traits>

#include "nx_internal.cuh"

namespace nx {
namespace {

constexpr int kTokens = 16;           // tokens of a thread block
constexpr int kSoloTokens = 16;       // up to so many tokens one block takes a sequence
// Tokens whose rows are on their way, less one: 3 take 101.9 us for the prompts, 4 98.4, 6 97.9.
constexpr int kRing = 4;
// The largest block, and with it the registers of a thread: 768 leave 80 (98.4 us), 640 leave 96,
// and fewer warps (102.8 us), 1024 leave 64 (98.5 us).
constexpr int kMaxThreads = 768;
constexpr int kAppendThreads = 256;   // threads of a block, unless one block covers a sequence

struct AppendArgs {
  nx_cache c;
  nx_tokens t;
  nx_append a;
  int32_t* dev_status;
  int32_t* lens;        // the layer's part of c.lens
  int32_t* held;        // the layer's part of an image's rows, or null
  int tiles, parts;     // thread blocks per sequence: token tiles x parts of the head rows
  int most;             // tokens of a block, at most
  bool set_lens;        // the kernel sets the new lengths itself
};

// cos and sin of 2 pi p f 2^-64. p f modulo 2^64 is the angle's fraction of a turn, exact
// up to f's own rounding; its nearest quarter turn comes off in integers, and what is left
// (at most 1/8 turn, in 30 bits) is what the float functions see.
__device__ __forceinline__ float2 rotation_of(int32_t p, uint64_t f) {
  const uint64_t turn = (uint64_t)(int64_t)p * f;
  const uint32_t hi = (uint32_t)(turn >> 32) + (uint32_t)((turn >> 31) & 1u);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const int32_t rest = (int32_t)(hi - (quarter << 30));
  float s, c;
  sincospif((float)rest * 4.656612873077393e-10f, &s, &c);   // 2^-31: units of half turns
  if (quarter & 1u) {
    const float x = c;
    c = -s;
    s = x;
  }
  return quarter & 2u ? make_float2(-c, -s) : make_float2(c, s);
}

// Two binary32 products, or products and sums, by one instruction (a seventh of all instructions
// less: one token of 48 head rows 2.62 us, not 2.74).
__device__ __forceinline__ float2 pair(const float* x, int j) {
  return make_float2(x[j], x[j + 1]);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 y, a, b;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, c, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 y, a, b, c;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

template <typename T, int RUN>
struct Run {                          // RUN features of a row as they lie in memory
  using Raw = typename std::conditional<sizeof(T) * RUN == 8, uint2, uint4>::type;
  static_assert(sizeof(T) * RUN == sizeof(Raw), "");
  Raw r;
  // starts the copy of a run from memory to an address of shared memory
  static __device__ __forceinline__ void start(uint32_t to, const T* from) {
    if constexpr (sizeof(Raw) == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
  }
  __device__ __forceinline__ void load(const T* p) { r = *reinterpret_cast<const Raw*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = r; }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < RUN / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < RUN; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void set(const float* x) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < RUN / 2; ++i) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = reinterpret_cast<const uint32_t&>(a);
      }
    } else {
#pragma unroll
      for (int i = 0; i < RUN; ++i) w[i] = __float_as_uint(x[i]);
    }
  }
};

template <typename T, int D, int RUN>
__global__ void __launch_bounds__(kMaxThreads) append_kernel(AppendArgs g) {
  constexpr int N = 2 * RUN, kLanes = D / N;         // threads of one head row
  using R = Run<T, RUN>;
  // by token, cosines and sines of pairs e and e + 1 of thread l at [e / 2][l] (two and two):
  // neighbours read neighbouring words
  __shared__ float4 s_rot[kTokens][D / 4];
  __shared__ int s_pos[kTokens];
  // the runs under way, [slot][run][thread], then [kv_heads] lengths, -1: leave alone
  extern __shared__ __align__(16) char s_ring[];
  const int slots = min(kRing, g.most), run_bytes = blockDim.x * (int)sizeof(R);
  int* s_len = reinterpret_cast<int*>(s_ring + slots * 2 * run_bytes);
  grid_dep_wait();

  const nx_cache& c = g.c;
  const nx_append& a = g.a;
  const int part = blockIdx.x % g.parts, tile = blockIdx.x / g.parts % g.tiles;
  const int s = blockIdx.x / g.parts / g.tiles;
  const int tid = threadIdx.x;
  const bool lead = tile == 0 && part == 0;
  int first;
  const int n = tokens_of(g.t, s, first);
  if (n < 0) {
    if (lead && tid == 0) atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
    return;
  }
  const int t0 = tile * kTokens;
  const int nt = min(kTokens, n - t0);
  if (nt <= 0 && tile > 0) return;

  const int H = c.kv_heads, HQ = a.q ? H * c.group : 0;
  // this thread's two runs of features, and whether they turn
  const int lane = tid % kLanes, half = a.rotary_dim / 2;
  const bool turns = lane < a.rotary_dim / N;
  const bool split = turns && !a.interleaved;
  const int o0 = split ? RUN * lane : N * lane;
  const int o1 = split ? half + RUN * lane : N * lane + RUN;
  const int rows = HQ + 2 * H;                       // head rows per token: q, k, v
  const int groups = blockDim.x / kLanes;
  // a warp's groups take neighbouring head rows; a row that does not exist takes part in the
  // warp's shuffles, with whatever its place in the ring holds: groups do not mix
  bool primed = false;
  for (int base = part * groups + (tid & ~31) / kLanes; !primed || base < rows;
       base += g.parts * groups) {
    const int r = base + tid % 32 / kLanes;
    const bool live = r < rows, is_q = r < HQ, is_v = r >= HQ + H;
    const int h = is_q ? r : is_v ? r - HQ - H : r - HQ;
    const long long token = first + t0;
    const long long stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
    const T* src = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) + token * stride +
                   (long long)h * D;
    const T* weight = static_cast<const T*>(is_q ? a.q_norm : is_v ? nullptr : a.k_norm);
    const uint32_t ring = smem_at(s_ring) + tid * (int)sizeof(R);
    const auto fetch = [&](int t, int slot) {
      if (live && t < nt) {
        R::start(ring + 2 * slot * run_bytes, src + t * stride + o0);
        R::start(ring + (2 * slot + 1) * run_bytes, src + t * stride + o1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int t = 0; t < kRing - 1; ++t) fetch(t, t);
    float w[N];
    if (weight && live) {
      Run<T, RUN> x;
      x.load(weight + o0);
      x.get(w);
      x.load(weight + o1);
      x.get(w + RUN);
    }
    if (!primed) {                                  // while the first rows are on their way
      const int32_t* lens_in = (a.lens_in ? a.lens_in : g.lens) + (long long)s * H;
      for (int h = tid; h < H; h += blockDim.x) {
        int len = lens_in[h];
        int flag = 0;
        if (len < 0 || len > c.capacity) flag = NX_DEV_BAD_LEN;
        else if (n > c.capacity - len) flag = NX_DEV_FULL;
        if (flag) {
          len = -1;
          if (lead) atomicOr(g.dev_status, flag);
        }
        // rows that an image holds of what the new ones take the place of
        if (lead && g.held && len >= 0) {
          int32_t* held = g.held + (long long)s * H + h;
          const int whole = len - len % image_block(c);
          if (*held > whole) *held = whole;
        }
        s_len[h] = len;
      }
      for (int t = tid / 32; t < nt; t += blockDim.x / 32)
        for (int i = tid % 32; i < half; i += 32) {
          const float2 v = rotation_of(a.pos[first + t0 + t], a.rotary[i]);
          float* to = reinterpret_cast<float*>(&s_rot[t][i % RUN / 2 * kLanes + i / RUN]) + i % 2;
          to[0] = v.x;
          to[2] = v.y;
        }
      if (tid < nt) s_pos[tid] = a.pos[first + t0 + tid];
      __syncthreads();
      primed = true;
    }
    const int len = live && !is_q ? s_len[h] : 0;
    const bool writes = live && len >= 0;
    // where the first token's row goes: the next ones follow `step` elements apart, but with
    // pages every row of k and v is looked up
    const bool lookup = !is_q && c.page_size;
    T* dst = static_cast<T*>(is_q ? a.q_out : is_v ? c.v : c.k);
    const int step = is_q ? HQ * D : D;
    int32_t* pos_out = c.pos;
    if (is_q) {
      dst += (token * HQ + h) * D;
    } else if (!lookup && writes) {
      const long long row = row_of(c, g.t.layer, s, h, len + t0);
      dst += row * D;
      pos_out += row;
    }
    const bool keeps_pos = !is_q && !is_v && lane == 0;
    const bool norms = __any_sync(0xffffffffu, weight != nullptr);   // the shuffles take the warp
    int slot = 0;
    for (int t = 0; t < nt; ++t) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
      R x0, x1;                                    // a thread's runs are nobody else's
      x0.load(reinterpret_cast<const T*>(s_ring + tid * sizeof(R) + 2 * slot * run_bytes));
      x1.load(reinterpret_cast<const T*>(s_ring + tid * sizeof(R) + (2 * slot + 1) * run_bytes));
      fetch(t + kRing - 1, slot == 0 ? kRing - 1 : slot - 1);     // read a token ago
      slot = slot == kRing - 1 ? 0 : slot + 1;
      float x[N];
      x0.get(x);
      x1.get(x + RUN);
      if (norms) {
        float2 two = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < N; j += 2) two = fma2(pair(x, j), pair(x, j), two);
        float ss = two.x + two.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (weight) {
          const float f = rsqrtf(ss * (1.0f / D) + a.eps);      // 2^-22, as exact as the rest
#pragma unroll
          for (int j = 0; j < N; j += 2) {
            const float2 y = mul2(mul2(pair(x, j), make_float2(f, f)), pair(w, j));
            x[j] = y.x;
            x[j + 1] = y.y;
          }
        }
      }
      if (!writes) continue;
      if (turns && !is_v) {
        const float4* cs = s_rot[t] + lane;
#pragma unroll
        for (int j = 0; j < RUN; j += 2) {
          const float4 r = cs[j / 2 * kLanes];     // cosines and sines of pairs j and j + 1
          if (a.interleaved) {
            const float p0 = x[2 * j], q0 = x[2 * j + 1], p1 = x[2 * j + 2], q1 = x[2 * j + 3];
            x[2 * j] = p0 * r.x - q0 * r.z;
            x[2 * j + 1] = q0 * r.x + p0 * r.z;
            x[2 * j + 2] = p1 * r.y - q1 * r.w;
            x[2 * j + 3] = q1 * r.y + p1 * r.w;
          } else {
            const float2 p = pair(x, j), q = pair(x, j + RUN), cos = make_float2(r.x, r.y),
                         sin = make_float2(r.z, r.w);
            const float2 qs = mul2(q, sin), turned = fma2(q, cos, mul2(p, sin));
            x[j] = fmaf(p.x, cos.x, -qs.x);
            x[j + 1] = fmaf(p.y, cos.y, -qs.y);
            x[j + RUN] = turned.x;
            x[j + 1 + RUN] = turned.y;
          }
        }
      }
      T* to = dst + t * step;
      int32_t* p = pos_out + t;
      if (lookup) {
        const long long row = row_of(c, g.t.layer, s, h, len + t0 + t);
        if (row < 0) {
          atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
          continue;
        }
        to = dst + row * D;
        p = c.pos + row;
      }
      if (keeps_pos) *p = s_pos[t];
      x0.set(x);
      x1.set(x + RUN);
      x0.store(to + o0);
      x1.store(to + o1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  // s_len was read before the barrier above: with one block per sequence, or lengths that
  // come from elsewhere, nobody still reads what is set here
  if (g.set_lens && lead)
    for (int h = tid; h < H; h += blockDim.x)
      if (s_len[h] >= 0) g.lens[(long long)s * H + h] = s_len[h] + n;
}

// lens += tokens, for sequences of several thread blocks that read lens themselves.
__global__ void append_lens_kernel(AppendArgs g) {
  grid_dep_wait();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)g.c.seqs * g.c.kv_heads) return;
  int first;
  const int n = tokens_of(g.t, (int)(i / g.c.kv_heads), first);
  const int len = g.lens[i];
  if (n < 0 || len < 0 || len > g.c.capacity || n > g.c.capacity - len) return;
  g.lens[i] = len + n;
}

bool aligned(const void* p, long long stride, int size) {
  return ((uintptr_t)p & 15u) == 0 && stride >= 0 && (stride * size) % 16 == 0;
}

template <typename T, int D, int RUN>
cudaError_t launch_append(AppendArgs& g, cudaStream_t st, int* launches) {
  const int rows = (g.a.q ? g.c.kv_heads * g.c.group : 0) + 2 * g.c.kv_heads;
  constexpr int kLanes = D / (2 * RUN);
  const int most = g.t.max_tokens < g.t.tokens ? g.t.max_tokens : g.t.tokens;
  g.tiles = most > kTokens ? (int)(((long long)most + kTokens - 1) / kTokens) : 1;
  const bool in_place = !g.a.lens_in || g.a.lens_in == g.lens;
  int threads = kAppendThreads;
  if (most <= kSoloTokens) {
    // few tokens: one block per sequence, with a thread group per head row as far as they go,
    // reads the lengths before it sets them, so that one launch does
    g.parts = 1;
    const long long want = (long long)rows * kLanes;
    threads = want > kMaxThreads ? kMaxThreads : (int)((want + 31) / 32 * 32);
  } else {
    g.parts = (rows * kLanes + threads - 1) / threads;       // even parts of the head rows
    threads = ((rows + g.parts - 1) / g.parts * kLanes + 31) / 32 * 32;
  }
  g.set_lens = !in_place || g.tiles * g.parts == 1;
  const long long blocks = (long long)g.c.seqs * g.tiles * g.parts;
  g.most = most < 1 ? 1 : most < kTokens ? most : kTokens;
  const int slots = g.most < kRing ? g.most : kRing;
  const int smem = slots * 2 * threads * (int)sizeof(Run<T, RUN>) + g.c.kv_heads * 4;
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024)                              // with the angles: 48 KB need no leave
    e = allow_smem<append_kernel<T, D, RUN>>(
        kRing * 2 * kMaxThreads * (int)sizeof(Run<T, RUN>) + kMaxAppendHeads * 4);
  if (e != cudaSuccess) return e;
  e = launch_after(append_kernel<T, D, RUN>, dim3((unsigned)blocks), dim3(threads), smem, st, g);
  if (e != cudaSuccess) return e;
  note_launch(st, launches, "append");
  if (g.set_lens) return cudaSuccess;
  const long long slices = (long long)g.c.seqs * g.c.kv_heads;
  e = launch_after(append_lens_kernel, dim3((unsigned)((slices + 255) / 256)), dim3(256), 0, st,
                   g);
  if (e == cudaSuccess) note_launch(st, launches, "append_lens");
  return e;
}

}  // namespace
}  // namespace nx

extern "C" nx_status nexus_append(nx_cache* cache, const nx_tokens* tokens, const nx_append* args,
                                  int32_t* dev_status, nx_stream_t stream) {
  return nexus_append_image(cache, tokens, args, nullptr, dev_status, stream);
}

extern "C" nx_status nexus_append_image(nx_cache* cache, const nx_tokens* tokens,
                                        const nx_append* args, const nx_image* image,
                                        int32_t* dev_status, nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens) || !args || !dev_status)
    return NX_ERR_INVALID_ARG;
  if (image && !valid_image(image)) return NX_ERR_INVALID_ARG;
  if (image && cache->dtype != NX_DTYPE_BF16) return NX_ERR_UNSUPPORTED;
  const nx_cache& c = *cache;
  const nx_append& a = *args;
  if (!aligned4(c.pos, c.lens, c.block_table, a.pos, a.lens_in, dev_status))
    return NX_ERR_INVALID_ARG;
  const int size = c.dtype == NX_DTYPE_BF16 ? 2 : 4;
  const int D = c.head_dim;
  if (a.reserved != 0 || !(a.eps >= 0.f) || !(a.eps < 3.0e38f)) return NX_ERR_INVALID_ARG;
  if (a.rotary_dim < 0 || a.rotary_dim > D || a.rotary_dim % 8) return NX_ERR_INVALID_ARG;
  if ((a.rotary_dim > 0) != (a.rotary != nullptr) || ((uintptr_t)a.rotary & 7u))
    return NX_ERR_INVALID_ARG;
  // thread blocks: tiles of 16 tokens x parts of at least 16 head rows
  const int most = tokens->max_tokens < tokens->tokens ? tokens->max_tokens : tokens->tokens;
  const long long blocks = (long long)c.seqs * (most / kTokens + 1) *
                           ((long long)c.kv_heads * (c.group + 2) / 16 + 1);
  if (c.kv_heads > kMaxAppendHeads || blocks > 0x7FFFFFFFLL ||
      (long long)c.kv_heads * c.group > (1 << 20))
    return NX_ERR_UNSUPPORTED;
  if ((a.q == nullptr) != (a.q_out == nullptr) && tokens->tokens > 0) return NX_ERR_INVALID_ARG;
  if (tokens->tokens > 0) {
    if (!a.k || !a.v || !a.pos) return NX_ERR_INVALID_ARG;
    if (!aligned(a.k, a.k_stride, size) || !aligned(a.v, a.v_stride, size) ||
        !aligned(a.q, a.q_stride, size) || !aligned(a.q_out, 0, size))
      return NX_ERR_INVALID_ARG;
    const long long hq = (long long)c.kv_heads * c.group * D;
    if (a.q && a.q == a.q_out && a.q_stride != hq) return NX_ERR_INVALID_ARG;
  }
  if (((uintptr_t)a.q_norm & 15u) || ((uintptr_t)a.k_norm & 15u)) return NX_ERR_INVALID_ARG;

  AppendArgs g{};
  g.c = c;
  g.t = *tokens;
  g.a = a;
  g.dev_status = dev_status;
  const long long per_layer = (long long)c.seqs * c.kv_heads;
  g.lens = c.lens + tokens->layer * per_layer;
  if (image) g.held = image->rows + tokens->layer * per_layer;
  if (a.lens_in && a.lens_in != g.lens && a.lens_in < g.lens + per_layer &&
      g.lens < a.lens_in + per_layer)
    return NX_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (size == 4)
    e = D == 128 ? launch_append<float, 128, 4>(g, st, &launches)
                 : launch_append<float, 64, 4>(g, st, &launches);
  else if (a.rotary_dim % 16 == 0)       // runs of 8 hold whole pairs: 16-byte loads
    e = D == 128 ? launch_append<__nv_bfloat16, 128, 8>(g, st, &launches)
                 : launch_append<__nv_bfloat16, 64, 8>(g, st, &launches);
  else
    e = D == 128 ? launch_append<__nv_bfloat16, 128, 4>(g, st, &launches)
                 : launch_append<__nv_bfloat16, 64, 4>(g, st, &launches);
  return finish(e, launches);
}
