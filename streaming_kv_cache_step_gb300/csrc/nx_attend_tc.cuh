// nx_attend_tc.cuh -- nexus_attend and nexus_attend_shared for many query rows per slice (prompt chunks,
// drafts of several tokens, prefixes that many sequences share): the same softmax as nx_attend_rows.cuh on
// the 5th-generation tensor cores.
//
// A thread block holds two streams of 128 query rows (thread = row): two row tiles that share
// each tile of 64 slots of K and V, or, for slices with up to 128 rows, one row tile whose
// even and odd slot tiles are the two streams. Per slot tile and stream:
//   S = Q K^T      tcgen05.mma, 128 x 64 x head_dim, Q and K in shared memory, S in TMEM
//   p = 2^(c1 S - m), bf16, over S's own columns of TMEM; l += sum p
//   O += p V       tcgen05.mma, p from TMEM, V in shared memory (features contiguous), O in TMEM
// A stream has two S buffers: its next logits are on their way while its warps take the
// exponentials of these, and the other stream's products run meanwhile. m is raised,
// and O in TMEM multiplied, only when a logit exceeds it by more than 2^8: rarely after the
// first tiles. The roles:
//   warps 0-3, 4-7  softmax of the two streams, and the results
//   warps 8-9       (8-13 for 8-bit rows) K and V into a ring of shared-memory slots, in the
//                   128-byte swizzle that the matrix descriptors name: whole tiles by TMA
//                   boxes (one per page and 64 features), a slice's last tile by asynchronous
//                   16-byte copies, with zeros for rows that do not exist. 8-bit rows come some
//                   tiles ahead, by bulk copies, to a ring of their own and go from there to
//                   the slots as bf16, which holds a code times its power-of-two scale exactly
//   the last two    issue the matrix instructions, one warp for each stream
// Where the tensor cores have time to spare (one row tile: K and V from HBM bound the kernel)
// and for 8-bit rows, whose values need no rounding, p is kept as two bf16 terms, p = hi + lo,
// with one product each; else, with more than 128 rows, as one (half a step of bf16, 2^-8, in each p:
// error of the output against 64 bits 2.1e-3, 1.7e-3 with two terms, which is the rounding of the output
// alone). Two terms would take, of 8 slices of 8192 rows under 512, 2048 and 8192 query rows of
// nexus_attend_shared, 44.3, 103 and 347 us instead of 40.8, 88.7 and 295.
// Every wait is bounded; when one gives up, the block flags NX_DEV_TIMEOUT, starts no more copies,
// waits (bounded too) for the copies and products that are under way and ends, its TMEM freed.
//
// Measured: two chunks of 512 tokens, 8 x 4 heads, over 8704 rows: 131 us per call, 1.11 PFLOP/s,
// 57 % of a plain bf16 product's rate; a step of a stream (64 slots) takes about 2000 clocks, of
// which its products need 640 and the other stream's as many: the rest is the latency of issuing
// and committing them. 20 to 128 rows over 32 x 8 slices of 6960 rows: 180 to 186 us in bf16
// (5.0 TB/s), 349 to 358 us from the image, where expanding the codes bounds it; the chunks from the
// image 212 us.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "nx_attend.cuh"

namespace nx {
namespace {

constexpr int kRows = 128;                 // query rows of a stream
constexpr int kCols = 64;                  // slots of a tile
constexpr int kLoadWarp = 8;
constexpr int kGroups = kCols / 8;         // runs of 8 slots of a tile
constexpr int kTcRows = 256;               // rows of a piece, at most
constexpr int kTcGrid = kSms;
constexpr int kPolls = 1 << 20;               // mbarrier polls before giving up
constexpr float kRaise = 8.f;              // log2 units
constexpr int kFewRows = 16;               // query rows that never come here

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void bar_arrive_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
// Waits for a phase, unless the block gives up or has given up: false then.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up,
                                         int32_t* dev_status) {
  if (bar_test(bar, parity)) return true;
  for (int i = 0; i < kPolls; ++i) {
    if (*gave_up) return false;
    if (bar_test(bar, parity)) return true;
  }
  *gave_up = 1;
  atomicOr(dev_status, NX_DEV_TIMEOUT);
  return false;
}
// The same for what is under way when the block has given up: some milliseconds at most.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < kPolls / 16 && !bar_test(bar, parity); ++i) {}
}
// Orders this thread's accesses to shared memory before those of TMA, bulk copies and tcgen05 that
// a barrier lets go after it.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Matrix descriptors, 128-byte swizzle: the address (in 16-byte units) in the low 18 bits, the
// rest as follows. K-major (Q, K: features contiguous, rows of 128 bytes): 8-row groups 1024
// bytes apart. MN-major (V: the output's features contiguous): 64-feature blocks `block` bytes
// apart, groups of 8 slots 1024 bytes apart.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint64_t desc_k(uint32_t at) {
  return (uint64_t)kDescHigh << 32 | (at >> 4 | 1u << 16);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t at, uint32_t block) {
  return (uint64_t)kDescHigh << 32 | (at >> 4 | block >> 4 << 16);
}
// The same value in all lanes, and known to be: what the matrix instructions take lies in
// registers of the warp, and is moved there from a lane's, 80 clocks an instruction, unless the
// compiler sees that it is the warp's already.
__device__ __forceinline__ uint32_t warp_value(uint32_t x) {
  return __shfl_sync(0xffffffffu, x, 0);
}
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// kind::f16, fp32 accumulator, bf16 operands, M = 128; `mn`: B is MN-major. kNegate: -A B.
constexpr uint32_t kNegate = 1u << 13;
__host__ __device__ constexpr uint32_t idesc(int n, bool mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(128 >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(add)
      : "memory");
}

// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t at, float* x) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
template <int D, int NQ, bool IMAGE>
struct Plan {
  // three warps per scheduler leave 168 registers a thread, four 128: 8-bit rows need the
  // warps to expand them
  static constexpr int kLoadWarps = IMAGE ? 6 : 2, kLoaders = 32 * kLoadWarps;
  static constexpr int kIssueWarp = kLoadWarp + kLoadWarps, kThreads = 32 * (kIssueWarp + 2);
  static constexpr int kRuns = (kGroups + kLoadWarps - 1) / kLoadWarps;   // of one loading warp
  static constexpr bool kLo = IMAGE || NQ == 1;               // p as two terms
  static constexpr int kBlocks = D / 64;                      // 128-byte columns of a row
  static constexpr int kRowBlock = kRows * 128, kColBlock = kCols * 128;   // of a Q, K or V tile
  static constexpr int kQBytes = kBlocks * kRowBlock, kSlotBytes = kBlocks * kColBlock;
  static constexpr int kRawBytes = kCols * D;                 // codes of a K or V tile
  static constexpr int kSlots = IMAGE ? 8 : NQ == 2 ? 10 : 12;
  static constexpr int kRaw = IMAGE ? (NQ == 2 ? 4 : 8) : 0;
  static constexpr int kBars = 2 * kSlots + 1 + 3 * 4 + 2 * kRaw + 1;
  static constexpr int kSmem = 1024 + NQ * kQBytes + kSlots * kSlotBytes + kRaw * kRawBytes;
};

// Units of this kernel: 128 NQ rows, tiles of 64 slots.
template <int NQ>
__device__ __forceinline__ int tc_tiles(const AttendUnit& u) {
  return !u.rows ? 0 : u.end ? (u.end + kCols - 1) / kCols : 1;
}

// The copies of 8 bf16 rows of K or V (slots t .. t + 7, one warp) to rows r .. r + 7 of a ring
// slot. row: the first one's; < 0: none of them exist.
template <int D>
__device__ __forceinline__ void copy_group(const char* src, long long row, int t, int end,
                                           uint32_t slot, int r, int lane) {
  constexpr int kChunks = D / 8, kLine = 32 / kChunks;     // 16-byte chunks; rows per step
  const int chunk = lane % kChunks, sub = lane / kChunks;
  const char* p = src + (row < 0 ? 0 : row * (D * 2)) + lane * 16;
  const uint32_t dst = slot + chunk / 8 * (kCols * 128) + (r + sub) * 128;
#pragma unroll
  for (int i = 0; i < 8; i += kLine) {
    const bool ok = row >= 0 && t + i + sub < end;
    copy16(dst + i * 128 + ((chunk ^ (i + sub)) & 7) * 16, ok ? p + i * (D * 2) : src, ok);
  }
}

// The value rows of a tile that some query rows see and others do not, slots [low, end): what is not
// finite in them would reach the latter as 0 times an infinity or NaN. It goes out of the tile, and
// the slot is marked in `hot`, for take_hot. Of the 8 bf16 rows that copy_group brought to row r:
__device__ __forceinline__ void mark_hot(uint32_t* hot, int j) {
  atomicOr(hot + (j >> 5), 1u << (j & 31));
}
template <int D>
__device__ __forceinline__ void clear_group(int t, int low, int end, uint32_t slot, int r, int lane,
                                            uint32_t* hot) {
  constexpr int kChunks = D / 8, kLine = 32 / kChunks;
  const int chunk = lane % kChunks, sub = lane / kChunks;
#pragma unroll 1
  for (int i = sub; i < 8; i += kLine) {
    const uint32_t at = slot + chunk / 8 * (kCols * 128) + (r + i) * 128 + ((chunk ^ i) & 7) * 16;
    uint32_t x[4];
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at)
                 : "memory");
    uint32_t bad = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t y = not_finite<2>(x[w]);
      x[w] &= ~y;
      bad |= y;
    }
    if (bad && t + i >= low && t + i < end) {
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x[0]), "r"(x[1]),
                   "r"(x[2]), "r"(x[3])
                   : "memory");
      mark_hot(hot, t + i - low);
    }
  }
}
// and what is not finite in the marked slots that a row sees, added to 32 of its outputs.
__device__ __noinline__ void take_hot(const AttendArgs& g, const AttendUnit& u, const uint32_t* hot,
                                      int lim, int D, int d0, float* o) {
  const SlotRows rows(g, u);
  for (int j = 0; j < 256 && u.low + j < lim; ++j) {
    if (!(hot[j >> 5] >> (j & 31) & 1u)) continue;
    const int t = u.low + j;
    const long long row = rows.row(t, u.end, rows.page(t, u.end));
    if (row < 0) continue;
    for (int e = 0; e < 32; ++e) {
      float x;
      if (t < u.held) {
        const unsigned char c = static_cast<const unsigned char*>(g.im.v)[row * D + d0 + e];
        x = (c & 0x7F) == 0x7F ? __uint_as_float(0x7FC00000u) : 0.f;
      } else {
        x = __bfloat162float(static_cast<const __nv_bfloat16*>(g.c.v)[row * D + d0 + e]);
      }
      if (!isfinite(x)) o[e] += x;
    }
  }
}

// The codes of a tile's rows below `some`, times the scales of their runs of 8, as bf16 in a ring
// slot, with zeros behind them up to the next run. Thread `tid` of N takes every N-th 8 codes. WHOLE:
// all rows, so that every load is on its way before the first one is used. Otherwise values from row
// `part` on that are not finite are marked in `hot`, row `part` - `first` first, and left out.
template <int D, int N, bool WHOLE>
__device__ __forceinline__ void expand_tile(uint32_t raw, const float* scale, int some,
                                            uint32_t slot, int tid, int part = kCols,
                                            int first = 0, uint32_t* hot = nullptr) {
  constexpr int kChunks = D / 8, kAll = kCols * kChunks, kEach = (kAll + N - 1) / N;
  const int rows = WHOLE ? kCols : min(kCols, (some + 7) / 8 * 8);
  uint32_t x[kEach][2];
  float f[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int c = tid + i * N, r = c / kChunks;
    x[i][0] = x[i][1] = 0;
    f[i] = 0.f;
    if ((WHOLE || r < some) && ((i + 1) * N <= kAll || c < kAll)) {
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                   : "=r"(x[i][0]), "=r"(x[i][1])
                   : "r"(raw + c * 8)
                   : "memory");
      f[i] = scale[r / 8];
      if constexpr (!WHOLE)
        if (r >= part) {
          const uint32_t y0 = not_finite<1>(x[i][0]), y1 = not_finite<1>(x[i][1]);
          x[i][0] &= ~y0;
          x[i][1] &= ~y1;
          if (y0 | y1) mark_hot(hot, r - first);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int c = tid + i * N, r = c / kChunks, chunk = c % kChunks;
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t h0, h1;
      e4m3_pairs(x[i][j], h0, h1);
      const float2 v0 = __half22float2(reinterpret_cast<const __half2&>(h0));
      const float2 v1 = __half22float2(reinterpret_cast<const __half2&>(h1));
      y[2 * j] = bf16_pair(v0.x * f[i], v0.y * f[i]);
      y[2 * j + 1] = bf16_pair(v1.x * f[i], v1.y * f[i]);
    }
    if ((WHOLE || r < rows) && ((i + 1) * N <= kAll || c < kAll))
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                       slot + chunk / 8 * (kCols * 128) + r * 128 + ((chunk ^ r) & 7) * 16),
                   "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                   : "memory");
  }
}

// Where row r of a unit's output and its statistics go.
__device__ __forceinline__ void store_row(const AttendArgs& g, const AttendUnit& u, int r, int D,
                                          int d0, const float* x, int n, float f) {
  const int row = u.r0 + r;
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(g.a.out) +
                     (long long)(u.first + row / g.c.group) * g.a.out_stride +
                     ((long long)u.h * g.c.group + row % g.c.group) * D + d0;
  for (int i = 0; i < n; i += 8)
    *reinterpret_cast<uint4*>(p + i) =
        make_uint4(bf16_pair(x[i] * f, x[i + 1] * f), bf16_pair(x[i + 2] * f, x[i + 3] * f),
                   bf16_pair(x[i + 4] * f, x[i + 5] * f), bf16_pair(x[i + 6] * f, x[i + 7] * f));
}
__device__ __forceinline__ void store_lse(const AttendArgs& g, const AttendUnit& u, int r, float m,
                                          float l) {
  if (!g.a.lse) return;
  const int row = u.r0 + r;
  g.a.lse[(long long)(u.first + row / g.c.group) * (g.c.kv_heads * g.c.group) +
          u.h * g.c.group + row % g.c.group] =
      l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}
// N features of row r of the output, and with the first of them ln l.
template <int N>
__device__ __forceinline__ void finish_output(const AttendArgs& g, const AttendUnit& u, int r, int D,
                                              int d0, float* o, float m, float l) {
  if (l == 0.f)
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
  store_row(g, u, r, D, d0, o, N, l == 0.f ? 0.f : 1.f / l);
  if (d0 == 0) store_lse(g, u, r, m, l);
}

// Ends N features of row r: o / l to the output and, with the first of them, ln l; of the prefixes'
// pass o, m and l as they are, which the own rows' pass takes in first (`joins`: it has some).
template <int N, typename Args>
__device__ __forceinline__ void finish_features(const Args& g, const AttendUnit& u, int r,
                                                int D, int d0, float* o, float m, float l,
                                                bool joins) {
  if constexpr (kShared<Args>) {
    const long long at = part_row(g, u, r);
    if (g.pass == 1 || (g.pass == 3 && joins)) {
      float4* to = reinterpret_cast<float4*>((g.pass == 1 ? g.part.out : g.part.own_out) +
                                             at * D + d0);
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        to[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      if (d0 == 0) (g.pass == 1 ? g.part.stat : g.part.own_stat)[at] = make_float2(m, l);
      return;
    }
    if (joins) {
      const float2 other = g.part.stat[at], k = join_by(m, l, other);
      const float4* from = reinterpret_cast<const float4*>(g.part.out + at * D + d0);
      l = l * k.x + other.y * k.y;
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const float4 y = from[i];
        o[4 * i] = o[4 * i] * k.x + y.x * k.y;
        o[4 * i + 1] = o[4 * i + 1] * k.x + y.y * k.y;
        o[4 * i + 2] = o[4 * i + 2] * k.x + y.z * k.y;
        o[4 * i + 3] = o[4 * i + 3] * k.x + y.w * k.y;
      }
    }
  }
  finish_output<N>(g, u, r, D, d0, o, m, l);
}

// How many thread blocks share the tiles. With the sequences' own rows next to them: a part of the
// GPU that goes by what both cost; the other blocks end at once, and their SMs are the other pass's
// (64 sequences, 4 heads each of 8 groups, 32768 rows of prefix, 512 to 1024 of their own: 81 us, 99 one
// behind the other.)
// Where the others are fewer blocks than fit the GPU at once, they get room for all of them if that
// costs this pass less than 4 us (16 sequences behind 4096 rows, 128 of their own: 19.9 us, not 24.6).
__device__ __forceinline__ int part_of_sms(const SharedArgs& g, int total, float rows) {
  if (g.part.room) {
    const int left = kSms - g.part.room;
    const float cost = (float)total * g.part.tile_cost;
    return left >= kSms / 4 && cost / left - cost / kSms < 4000.f ? min((int)gridDim.x, left)
                                                                  : gridDim.x;
  }
  const float here = (float)total * g.part.tile_cost, there = rows * g.part.row_cost;
  const int blocks = (int)(kSms * (here / (here + there + 1.f)) + 0.5f);
  return min((int)gridDim.x, max(blocks, kSms / 4));
}
template <int THREADS>
__device__ __forceinline__ int beside_blocks(const SharedArgs& g, int total, float* s_rows) {
  if (g.pass != 1 || !(g.part.row_cost || g.part.room)) return gridDim.x;
  const int n = g.part.seqs * g.c.kv_heads;
  float rows = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += THREADS) rows += (float)max(0, g.part.own_lens[i]);
#pragma unroll
  for (int o = 16; o; o /= 2) rows += __shfl_xor_sync(0xffffffffu, rows, o);
  if (threadIdx.x % 32 == 0) s_rows[threadIdx.x / 32] = rows;
  __syncthreads();
  rows = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) rows += s_rows[w];
  return part_of_sms(g, total, rows);
}

// The same shares for up to kFewUnits units with two barriers instead of five (of 13 us before a block's
// second tile, now 8 to 11, the shares took 3 to 4, now 2.5): one warp looks after the units, the others after the own rows'
// lengths, then every warp finds the block's share by itself. Where that makes no share longer by more
// than kAlignMore tiles, a unit's shares are whole blocks': one whose share goes on in a second unit ends
// one piece and starts another, which costs as much as seven tiles (8 slices of 8192 rows, 64 query rows
// 26.8 us, now 25.6). `last`: the last of the blocks that have this one's unit; -1: shares are even.
constexpr int kFewUnits = 64, kAlignMore = 8;
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
template <int THREADS, int NQ>
__device__ __forceinline__ AttendShare few_share(const SharedArgs& g, int* s_tiles, float* s_rows,
                                                 int& last) {
  constexpr unsigned kFull = 0xffffffffu;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == 0) {
    for (int i = lane; i < kFewUnits; i += 32)
      s_tiles[i] = i < g.units ? tc_tiles<NQ>(attend_unit<kRows * NQ>(g, i)) : 0;
  } else if (g.part.row_cost) {
    float rows = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x - 32; i < g.part.seqs * g.c.kv_heads; i += THREADS - 32)
      rows += (float)max(0, g.part.own_lens[i]);
#pragma unroll
    for (int o = 16; o; o /= 2) rows += __shfl_xor_sync(kFull, rows, o);
    if (lane == 0) s_rows[warp] = rows;
  }
  __syncthreads();
  const int t[2] = {s_tiles[lane], s_tiles[lane + 32]};
  AttendShare x;
  x.total = __reduce_add_sync(kFull, t[0] + t[1]);
  float rows = g.part.row_cost && lane > 0 && lane < THREADS / 32 ? s_rows[lane] : 0.f;
  // All warps have read: the block's first piece may write its results there. (An issuing warp whose
  // stream has no tile in that piece waits for nothing else. The image's 128 features and one row tile
  // leave no room for arrays of their own.)
  __syncthreads();
  int blocks = gridDim.x;
  if (g.part.row_cost || g.part.room) {
#pragma unroll
    for (int o = 16; o; o /= 2) rows += __shfl_xor_sync(kFull, rows, o);
    blocks = part_of_sms(g, x.total, rows);
  }
  x.per = share_per(x.total, blocks);
  last = -1;
  int per = 0;
  if (g.units <= blocks)
    for (int k = 0; k < kAlignMore && !per; ++k) {
      const int y = x.per + k;
      if (__reduce_add_sync(kFull, (t[0] + y - 1) / y + (t[1] + y - 1) / y) <= blocks) per = y;
    }
  if (per) x.per = per;
  const int b = blockIdx.x;
  x.start = per ? x.total : share_start(x.total, x.per, b);
  x.stop = per ? x.total : share_start(x.total, x.per, b + 1);
  x.unit = x.at = 0;
  int at0 = 0, first0 = 0;               // tiles and blocks of the units before
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = (t[h] + x.per - 1) / x.per;
    const int at = at0 + warp_scan(t[h], lane) - t[h], first = first0 + warp_scan(n, lane) - n;
    const bool mine = per ? b >= first && b < first + n : x.start >= at && x.start < at + t[h];
    const unsigned hit = __ballot_sync(kFull, mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      x.unit = 32 * h + src;
      x.at = __shfl_sync(kFull, at, src);
      const int f = __shfl_sync(kFull, first, src), tiles = __shfl_sync(kFull, t[h], src);
      if (per) {
        x.start = x.at + (b - f) * per;
        x.stop = min(x.at + tiles, x.start + per);
        last = f + (tiles + per - 1) / per - 1;
      }
      break;
    }
    at0 = __shfl_sync(kFull, at + t[h], 31);
    first0 = __shfl_sync(kFull, first + n, 31);
  }
  return x;
}

template <int D, int NQ, bool IMAGE, typename Args>
__global__ void __launch_bounds__(Plan<D, NQ, IMAGE>::kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, bool use_maps,
                     const __grid_constant__ Args g) {
  using P = Plan<D, NQ, IMAGE>;
  constexpr int kLoadWarps = P::kLoadWarps, kLoaders = P::kLoaders, kRuns = P::kRuns;
  constexpr int kIssueWarp = P::kIssueWarp, kThreads = P::kThreads;
  extern __shared__ char s_raw[];
  __shared__ __align__(8) uint64_t s_bar[P::kBars];
  __shared__ uint32_t s_tmem;
  __shared__ int s_up, s_bad[16];                   // bad-page marks of tile % 16
  __shared__ uint32_t s_hot[2][8];                  // marked slots of a piece, by turns, from u.low on
  __shared__ float s_m[kRows], s_l[kRows];
  __shared__ float s_scale[IMAGE ? P::kRaw : 1][kGroups];     // of the runs in a raw stage
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, b = blockIdx.x;
  char* base = s_raw + (1024 - (smem_at(s_raw) & 1023)) % 1024;
  const uint32_t s_q = smem_at(base), s_ring = s_q + NQ * P::kQBytes;
  const uint32_t s_codes = s_ring + P::kSlots * P::kSlotBytes;
  const uint32_t bars = smem_at(s_bar);
  const uint32_t full = bars, empty = bars + 8 * P::kSlots, qfull = empty + 8 * P::kSlots;
  // per stream and TMEM buffer: logits there, probabilities there, their product done
  const uint32_t sfull = qfull + 8, pfull = sfull + 32, odone = pfull + 32;
  const uint32_t rfull = odone + 32, rempty = rfull + 8 * P::kRaw;    // of the raw ring
  const uint32_t drained = rempty + 8 * P::kRaw;    // products done, after giving up
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_at(&s_tmem)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < P::kSlots; ++i) {
      bar_init(full + 8 * i, IMAGE ? kLoaders - 32 : kLoaders);
      bar_init(empty + 8 * i, NQ);                 // its users are done
    }
    for (int i = 0; i < P::kRaw; ++i) {
      bar_init(rfull + 8 * i, 32);
      bar_init(rempty + 8 * i, kLoadWarps - 1);
    }
    bar_init(qfull, NQ * kRows);
    for (int i = 0; i < 4; ++i) {
      bar_init(sfull + 8 * i, 1);
      bar_init(pfull + 8 * i, kRows);
      bar_init(odone + 8 * i, 1);
    }
    bar_init(drained, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_up = 0;
  }
  if (tid < 16) s_hot[tid / 8][tid % 8] = 0;
  begin_pass(g);
  tc_before();
  int last = -1;
  const AttendShare sh = [&] {
    // (s_m and s_l are the results', later)
    if constexpr (kShared<Args>)
      if (g.pass == 1 && g.units <= kFewUnits)
        return few_share<kThreads, NQ>(g, reinterpret_cast<int*>(s_m), s_l, last);
    return attend_share<kThreads>(
        g, [&](int i) { return tc_tiles<NQ>(attend_unit<kRows * NQ>(g, i)); },
        [&](int total) {
          // (attend_share ends with a barrier)
          if constexpr (kShared<Args>) return beside_blocks<kThreads>(g, total, s_l);
          return (int)gridDim.x;
        });
  }();
  tc_after();
  grid_dep_trigger();
  const uint32_t tmem = s_tmem;
  int unit = sh.unit, at = sh.at, pos = sh.start;
  const int stop = sh.stop;
  int2 desc = make_int2(-1, 0);
  int slot_no = 0;                     // ring slots filled or used so far (loader, issuer)
  int raw_no = 0;                      // raw stages filled so far
  int sent = 0;                        // behind the last ring slot or raw stage with copies under way
  int segment = 0;                     // pieces done
  int used[2] = {0, 0};                // slot tiles done by each stream
  volatile int* up = &s_up;

  while (pos < stop) {
    const AttendUnit u = attend_unit<kRows * NQ>(g, unit);
    const int tiles = tc_tiles<NQ>(u);
    const int a0 = pos - at, a1 = min(tiles, stop - at), n = a1 - a0;
    if (tiles > 0) {
      // tiles of each stream: all of them, or the even and the odd ones
      const int count[2] = {NQ == 2 ? n : (n + 1) / 2, NQ == 2 ? n : n / 2};
      if (warp >= kLoadWarp && warp < kIssueWarp) {
        // ---- loader ----
        const int lt = tid - 32 * kLoadWarp, lw = warp - kLoadWarp;
        const SlotRows rows(g, u);
        uint32_t* hot = s_hot[segment & 1];
        const auto mixed = [&](int t0) { return u.low < u.end && t0 + kCols > u.low; };
        // K and V tiles in turn, every warp its runs of 8 slots
        const auto announce = [&](int k) {
          fence_async();
          if (IMAGE || *up == 0) bar_arrive(full + 8 * (k % P::kSlots));
        };
        // whether any page of the piece is bad; then every K tile gets its marks
        bool any_bad = false;
        if (rows.table) {
          const int t1 = min(u.end, a1 * kCols);
#pragma unroll 4
          for (int t = a0 * kCols + 8 * lane; t < t1; t += 256)
            any_bad |= rows.row(t, u.end, rows.page(t, u.end)) == -1;
          any_bad = __any_sync(0xffffffffu, any_bad);
          if (any_bad && lt == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
        }
        if (lw == 0 && lane < 16) s_bad[lane] = 0;
        const auto bad_pages = [&](int i) {       // of tile i of the piece
          if (lw > 0 || !any_bad) return;
          const int t = (a0 + i) * kCols + 8 * (lane & 7);
          const unsigned marks =
              __ballot_sync(0xffffffffu, rows.row(t, u.end, rows.page(t, u.end)) == -1);
          if (lane == 0) s_bad[i & 15] = (int)(marks & 0xFFu);
        };
        // bf16 rows of slot i into ring slot sl, by 16-byte copies
        const auto copy_tile = [&](int i, int sl) {
          const int t0 = (a0 + i / 2) * kCols;
          const char* src = static_cast<const char*>(i & 1 ? g.c.v : g.c.k);
          int page[kRuns];
#pragma unroll
          for (int q = 0; q < kRuns; ++q)
            page[q] = rows.page(t0 + 8 * (q * kLoadWarps + lw), u.end);
#pragma unroll 1
          for (int r = 8 * lw; r < kCols; r += 8 * kLoadWarps) {
            copy_group<D>(src, rows.row(t0 + r, u.end, page[0]), t0 + r, u.end,
                          s_ring + sl * P::kSlotBytes, r, lane);
#pragma unroll
            for (int q = 0; q + 1 < kRuns; ++q) page[q] = page[q + 1];
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // slots of a TMA box or bulk copy
        const int box = g.c.page_size ? min(kCols, 1 << rows.shift) : kCols;
        if constexpr (!IMAGE) {
          // whole tiles: one warp issues their boxes
          // (but those that not every row sees whole)
          const int whole = use_maps && !any_bad ? max(0, min(n, u.low / kCols - a0)) : 0;
          const int boxes = kCols / box * P::kBlocks;
          int y = 0;
          for (int i = 0; i < 2 * whole; ++i) {
            const int k = slot_no + i, sl = k % P::kSlots, t0 = (a0 + i / 2) * kCols;
            const int t = t0 + lane / P::kBlocks * box;
            if (lw == 0 && !(i & 1) && lane < boxes)
              y = (int)rows.row(t, u.end, rows.page(t, u.end));
            bar_wait(empty + 8 * sl, (k / P::kSlots & 1) ^ 1, up, g.dev_status);
            __syncwarp();
            if (lw == 0 && *up == 0) {
              if (lane == 0) bar_arrive_tx(full + 8 * sl, P::kSlotBytes);
              __syncwarp();
              if (lane < boxes) {
                const int blk = lane % P::kBlocks;
                tma_box(s_ring + sl * P::kSlotBytes + blk * P::kColBlock + (t - t0) * 128,
                        i & 1 ? &map_v : &map_k, 64 * blk, y, full + 8 * sl);
              }
              if (lane > 0) bar_arrive(full + 8 * sl);
              sent = k + 1;
            } else if (*up == 0) {
              bar_arrive(full + 8 * sl);
            }
          }
          // the others: a slot is announced kLag slots later, when its copies are in
          const auto settle = [&](int i) {
            const int t0 = (a0 + i / 2) * kCols, k = slot_no + i;
            if ((i & 1) && mixed(t0))
#pragma unroll 1
              for (int r = 8 * lw; r < kCols; r += 8 * kLoadWarps)
                clear_group<D>(t0 + r, u.low, u.end, s_ring + k % P::kSlots * P::kSlotBytes, r, lane,
                               hot);
            announce(k);
          };
          constexpr int kLag = 4;
          for (int i = 2 * whole; i < 2 * n; ++i) {
            const int k = slot_no + i, sl = k % P::kSlots;
            if (!(i & 1)) bad_pages(i / 2);
            bar_wait(empty + 8 * sl, (k / P::kSlots & 1) ^ 1, up, g.dev_status);
            __syncwarp();
            copy_tile(i, sl);
            if (i >= 2 * whole + kLag) {
              asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
              settle(i - kLag);
            }
          }
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          for (int i = max(2 * whole, 2 * n - kLag); i < 2 * n; ++i) settle(i);
        } else {
          const int held = min(u.held, u.end);
          if (lw == 0) {
            // the first warp copies codes ahead: lane q < 8 looks after run q of a tile, its page
            // (fetched a tile ahead), its row, its scale (fetched a slot ahead); a page's (or the
            // tile's) first run copies all of its rows
            const long long blocks0 =
                g.c.page_size ? 0 : image_scale_at(g.c, g.t.layer, u.s, u.h, 0, g.b);
            const auto slot_of = [&](int i) { return (a0 + i / 2) * kCols + 8 * lane; };
            const auto page_of = [&](int i) {
              return lane < kGroups ? rows.page(slot_of(i), i < 2 * n ? held : 0) : 0;
            };
            const auto row_of_run = [&](int i, int page) {
              return lane < kGroups && i < 2 * n ? rows.row(slot_of(i), held, page) : -2;
            };
            const auto scale_of = [&](int i, long long row) {
              if (row < 0) return 0.f;
              return (i & 1 ? g.im.v_scale : g.im.k_scale)[
                  g.c.page_size ? row >> g.b_shift : blocks0 + (slot_of(i) >> g.b_shift)];
            };
            long long row = row_of_run(0, page_of(0));
            int page1 = page_of(2);
            float scale = scale_of(0, row);
#pragma unroll 1
            for (int i = 0; i < 2 * n; ++i) {
              const int no = raw_no + i, st = no % P::kRaw, t = slot_of(i);
              if (!(i & 1)) bad_pages(i / 2);
              long long row1 = row;                             // of slot i + 1
              if (i & 1) {
                row1 = row_of_run(i + 1, page1);
                page1 = page_of(i + 3);
              }
              const float scale1 = scale_of(i + 1, row1);
              bar_wait(rempty + 8 * st, (no / P::kRaw & 1) ^ 1, up, g.dev_status);
              const bool go = *up == 0;
              if (lane < kGroups) s_scale[st][lane] = scale;
              // a run on a bad page: zeros for what the stage held before; the stage's next bulk
              // copy, of the other proxy, comes behind them
              if (any_bad) {
                for (int q = 0; q < kGroups; ++q) {
                  const bool zero = __shfl_sync(0xffffffffu, row == -1 ? 1 : 0, q) != 0 && go;
                  if (zero)
                    for (int x = lane; x < 8 * D / 16; x += 32)
                      asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                       s_codes + st * P::kRawBytes + q * 8 * D + x * 16),
                                   "r"(0)
                                   : "memory");
                }
                fence_async();
              }
              const bool lead = go && row >= 0 && 8 * lane % box == 0;
              const int bytes = lead ? (min(held, t + box) - t) * D : 0;
              const unsigned total = __reduce_add_sync(0xffffffffu, (unsigned)bytes);
              if (go) {
                if (lane == 0) bar_arrive_tx(rfull + 8 * st, total);
                else bar_arrive(rfull + 8 * st);
                sent = no + 1;
              }
              __syncwarp();
              if (lead)
                bulk_copy(s_codes + st * P::kRawBytes + 8 * lane * D,
                          static_cast<const char*>(i & 1 ? g.im.v : g.im.k) + row * D, bytes,
                          rfull + 8 * st);
              row = row1;
              scale = scale1;
            }
          } else {
            // the others expand them
#pragma unroll 1
            for (int i = 0; i < 2 * n; ++i) {
              const int k = slot_no + i, sl = k % P::kSlots, t0 = (a0 + i / 2) * kCols;
              const int no = raw_no + i, st = no % P::kRaw;
              bar_wait(rfull + 8 * st, no / P::kRaw & 1, up, g.dev_status);
              bar_wait(empty + 8 * sl, (k / P::kSlots & 1) ^ 1, up, g.dev_status);
              const uint32_t slot = s_ring + sl * P::kSlotBytes;
              const bool some = (i & 1) && mixed(t0);            // not every row sees it whole
              if (held >= t0 + kCols && !some)
                expand_tile<D, kLoaders - 32, true>(s_codes + st * P::kRawBytes, s_scale[st], kCols,
                                                    slot, lt - 32);
              else if (held > t0)
                expand_tile<D, kLoaders - 32, false>(
                    s_codes + st * P::kRawBytes, s_scale[st], min(held - t0, kCols), slot, lt - 32,
                    some ? max(u.low - t0, 0) : kCols, u.low - t0, hot);
              if (t0 + kCols > held) {                          // bf16 rows, or none, behind it
                __syncwarp();
                const int q0 = held > t0 ? (held - t0 + 7) / 8 : 0;
                for (int r = 8 * (q0 + lw - 1); r < kCols; r += 8 * (kLoadWarps - 1))
                  copy_group<D>(static_cast<const char*>(i & 1 ? g.c.v : g.c.k),
                                rows.row(t0 + r, u.end, rows.page(t0 + r, u.end)), t0 + r, u.end,
                                slot, r, lane);
                asm volatile("cp.async.wait_all;" ::: "memory");
                if (some)
#pragma unroll 1
                  for (int r = 8 * (q0 + lw - 1); r < kCols; r += 8 * (kLoadWarps - 1))
                    clear_group<D>(t0 + r, u.low, u.end, slot, r, lane, hot);
              }
              announce(k);
              __syncwarp();
              if (lane == 0) bar_arrive(rempty + 8 * st);
            }
          }
        }
      } else if (warp >= kIssueWarp) {
        // ---- matrix instructions: the whole warp goes along, one lane issues ----
        const int x = (int)warp_value(warp - kIssueWarp);   // the stream
        const uint32_t negate = g.c1 < 0.f ? kNegate : 0u;   // the softmax scales by |c1|
        const uint32_t tm = warp_value(tmem) + x * 256, o = tm + 128;
        const uint32_t q = warp_value(s_q) + (NQ == 2 ? x : 0) * P::kQBytes;
        const uint32_t ring = warp_value(s_ring), id = idesc(kCols, false) | negate;
        const int k_no = (int)warp_value(slot_no), turn0 = (int)warp_value(used[x]);
        const int mine = (int)warp_value(count[x]);
        const auto k_of = [&](int j) { return k_no + 2 * (NQ == 2 ? j : 2 * j + x); };
        const auto qk = [&](int j) {   // the stream's tile j, to TMEM buffer (turn0 + j) % 2
          const int sl = k_of(j) % P::kSlots, c = turn0 + j;
          const uint32_t kk = ring + sl * P::kSlotBytes, d = tm + (c & 1) * 64;
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            mma_ss(d, desc_k(q + s / 4 * P::kRowBlock + s % 4 * 32),
                   desc_k(kk + s / 4 * P::kColBlock + s % 4 * 32), id, s > 0);
          commit(sfull + 16 * x + 8 * (c & 1));
          commit(empty + 8 * sl);
        };
        const auto pv = [&](int j) {
          const int sl = (k_of(j) + 1) % P::kSlots, c = turn0 + j;
          const uint32_t vv = ring + sl * P::kSlotBytes, p = tm + (c & 1) * 64;
#pragma unroll
          for (int s = 0; s < kCols / 16; ++s)
            mma_ts(o, p + 8 * s, desc_mn(vv + s * 2048, P::kColBlock), idesc(D, true),
                   s > 0 || j > 0);
          if constexpr (P::kLo)
#pragma unroll
            for (int s = 0; s < kCols / 16; ++s)
              mma_ts(o, p + 32 + 8 * s, desc_mn(vv + s * 2048, P::kColBlock), idesc(D, true), 1u);
          commit(odone + 16 * x + 8 * (c & 1));
          commit(empty + 8 * sl);
        };
        // Steps -2 and -1 issue the first logits; step j the product of tile j and, behind it
        // (products of one thread run in the order they are issued in), the logits of tile
        // j + 2, into the buffer that the product read. What a step waits for is watched by a
        // lane each: the query rows or the probabilities, V, the next K. (That K is two tiles
        // ahead of V: the ring holds them all, and kLag slots more.)
        bool fine = true;
#pragma unroll 1
        for (int j = -2; j < mine && fine; ++j) {
          const int c = turn0 + j, kv = k_of(j) + 1, kk = k_of(j + 2);
          const bool product = j >= 0, logits = j + 2 < mine;
          uint32_t bar = 0, parity = 0;
          if (lane == 0) {
            bar = product ? pfull + 16 * x + 8 * (c & 1) : j == -2 ? qfull : 0;
            parity = product ? c >> 1 & 1 : segment & 1;
          } else if (lane == 1 && product) {
            bar = full + 8 * (kv % P::kSlots);
            parity = kv / P::kSlots & 1;
          } else if (lane == 2 && logits) {
            bar = full + 8 * (kk % P::kSlots);
            parity = kk / P::kSlots & 1;
          }
          const bool ok = bar == 0 || bar_wait(bar, parity, up, g.dev_status);
          fine = __all_sync(0xffffffffu, ok);
          if (!fine) break;
          tc_after();
          if (elected()) {
            if (product) pv(j);
            if (logits) qk(j + 2);
          }
          __syncwarp();
        }
      } else if (warp < 8) {
        // ---- softmax ----
        const int x = warp / 4, r = tid % kRows, rr = (NQ == 2 ? x * kRows : 0) + r;
        if (tid < 8) s_hot[segment & 1 ^ 1][tid] = 0;         // the next piece's
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t to = tmem + lanes + x * 256 + 128;
        const float c1 = fmaxf(fabsf(g.c1), 1.1754944e-38f);   // not 0: -inf c1 is -inf
        const int lim = rr < u.rows ? min(u.end, row_limit(g, u, u.r0 + rr)) : 0;
        const int low = min(u.end, u.low);
        if (NQ == 2 || x == 0) {
          // the warp's query rows, 128 bytes of each to a block: whole rows by neighbouring lanes (a lane
          // to each row took 3.6 us of a piece's start, its copies 32 lines an instruction)
          constexpr int kChunks = D / 8, kLine = 32 / kChunks;
          const int row = u.r0 + rr, token = row / g.c.group;
          const bool ok = rr < u.rows;
          const long long src = ok ? (u.first + token) * g.a.q_stride +
                                         ((long long)u.h * g.c.group + row - token * g.c.group) * D
                                   : -1;
#pragma unroll 4
          for (int i = 0; i < 32; i += kLine) {
            const long long from = __shfl_sync(0xffffffffu, src, i + lane / kChunks);
            const int to = (r & ~31) + i + lane / kChunks, chunk = lane % kChunks;
            copy16(s_q + (NQ == 2 ? x : 0) * P::kQBytes + chunk / 8 * P::kRowBlock + to * 128 +
                       ((chunk ^ to) & 7) * 16,
                   static_cast<const __nv_bfloat16*>(g.a.q) + (from < 0 ? 0 : from) + 8 * chunk,
                   from >= 0);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async();
          bar_arrive(qfull);
        }
        // a warp without rows only keeps the count: what the products make of its rows is
        // never read
        const bool idle = (rr & ~31) >= u.rows;
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < count[x]; ++j) {
          const int i = NQ == 2 ? j : 2 * j + x, t0 = (a0 + i) * kCols;
          const int c = used[x] + j, buf = 16 * x + 8 * (c & 1);
          const uint32_t ts = tmem + lanes + x * 256 + (c & 1) * 64;
          bar_wait(sfull + buf, c >> 1 & 1, up, g.dev_status);
          // the buffer's product before is done (its logits were issued behind it)
          if (j > 1) bar_wait(odone + buf, (c >> 1 & 1) ^ 1, up, g.dev_status);
          __syncwarp();
          if (idle) {
            bar_arrive(pfull + buf);
            continue;
          }
          tc_after();
          const int bad = s_bad[i & 15];
          const bool mask = t0 + kCols > low || bad;
          float s[kCols];
          tmem_ld32(ts, s);
          tmem_ld32(ts + 32, s + 32);
          tmem_ld_wait();
          if (mask) {                  // a masked logit is -inf
            const int left = lim - t0;
#pragma unroll
            for (int e = 0; e < kCols; ++e)
              if (e >= left || (bad >> (e / 8) & 1)) s[e] = -INFINITY;
          }
          float top;
          {
            float t[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int e = 4; e < kCols; ++e) t[e % 4] = fmaxf(t[e % 4], s[e]);
            top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
          }
          top *= c1;
          const bool raise = top > m + kRaise;
          if (__any_sync(0xffffffffu, raise)) {
            const float nm = raise ? top : m, f = raise ? ex2(m - nm) : 1.f;
            m = nm;
            l *= f;
            if (j > 0) {               // once the product before this one is done
              bar_wait(odone + (buf ^ 8), (c - 1) >> 1 & 1, up, g.dev_status);
              __syncwarp();
              tc_after();
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16(to + 16 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(to + 16 * q, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          // p lies over S: hi in columns 0 .. 31, lo in 32 .. 63
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float y0 = ex2(fmaf(s[32 * q + 2 * e], c1, -ref));
              const float y1 = ex2(fmaf(s[32 * q + 2 * e + 1], c1, -ref));
              sum[e % 4] += y0;
              sum[e % 4] += y1;
              hi[e] = bf16_pair(y0, y1);
              if constexpr (P::kLo)
                lo[e] = bf16_pair(y0 - __uint_as_float(hi[e] << 16),
                                  y1 - __uint_as_float(hi[e] & 0xFFFF0000u));
            }
            tmem_st16(ts + 16 * q, hi);
            if constexpr (P::kLo) tmem_st16(ts + 32 + 16 * q, lo);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_wait();
          tc_before();
          bar_arrive(pfull + buf);
        }
        for (int j = max(0, count[x] - 2); j < count[x]; ++j) {
          const int c = used[x] + j;
          bar_wait(odone + 16 * x + 8 * (c & 1), c >> 1 & 1, up, g.dev_status);
        }
        __syncwarp();
        tc_after();
        // ---- results ----
        float* s_o = reinterpret_cast<float*>(base + NQ * P::kQBytes);   // the ring is idle
        const auto between = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        if (NQ == 1) {
          between();                   // both streams' products are done with the ring
          if (x == 1) {
            s_m[r] = m;
            s_l[r] = l;
            if (count[1] > 0)
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float o[32];
                tmem_ld32(to + 32 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) s_o[(32 * q + e) * kRows + r] = o[e];
              }
          }
          between();
        }
        if (NQ == 2 || x == 0) {
          const bool whole = a0 == 0 && a1 == tiles;
          const int piece = 2 * b + (a0 == 0 ? 1 : 0);
          float f0 = 1.f, f1 = 0.f;
          if (NQ == 1) {
            const float m1 = s_m[r], nm = fmaxf(m, m1), ref = nm == -INFINITY ? 0.f : nm;
            f0 = m == -INFINITY && l != l ? 1.f : ex2(m - ref);
            f1 = count[1] == 0 ? 0.f : m1 == -INFINITY && s_l[r] != s_l[r] ? 1.f : ex2(m1 - ref);
            l = l * f0 + (count[1] ? s_l[r] * f1 : 0.f);
            m = nm;
          }
          // (nexus_attend keeps to the letter what it had here: unrolled and with 1 / l taken where it is
          // used, the chunks of 512 tokens took 138 us, not 133)
          const bool joins = whole && part_joins(g, u);
          if (whole) meet_pass(g);
          const float f = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
          const uint32_t* hot = s_hot[segment & 1];
          uint32_t any_hot = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) any_hot |= hot[e];
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            float o[32];
            tmem_ld32(to + 32 * q, o);
            tmem_ld_wait();
            if (NQ == 1)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = o[e] * f0 + (count[1] ? s_o[(32 * q + e) * kRows + r] * f1 : 0.f);
            if (any_hot) {
              float y[32];
              const AttendUnit unit = u;
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = o[e];
              take_hot(g, unit, hot, lim, D, 32 * q, y);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = y[e];
            }
            // of a piece all 32 rows of a warp: whole 128-byte lines (with parts of them the join
            // of 19 pieces took 13 us longer)
            if (whole ? rr < u.rows : !idle) {
              if (whole) {
                if constexpr (kShared<Args>) {
                  finish_features<32>(g, u, rr, D, 32 * q, o, m, l, joins);
                } else {
                  if (l == 0.f)
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                  store_row(g, u, rr, D, 32 * q, o, 32, f);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  g.ws.out[((long long)piece * D + 32 * q + e) * kTcRows + rr] = o[e];
              }
            }
          }
          if (whole ? rr < u.rows : !idle) {
            if (!whole) g.ws.stat[piece * kTcRows + rr] = make_float2(m, l);
            else if constexpr (!kShared<Args>) store_lse(g, u, rr, m, l);
          }
        }
        // s_o lies over the ring, which the next piece's boxes fill by the other proxy
        if constexpr (NQ == 1 && !IMAGE) fence_async();
        tc_before();
      }
      slot_no += 2 * n;
      raw_no += 2 * n;
      used[0] += count[0];
      used[1] += count[1];
      ++segment;
      if (a0 == 0 && a1 < tiles) desc = make_int2(unit, (at + tiles - 1) / sh.per);
      if constexpr (kShared<Args>)
        if (g.pass == 1 && a0 == 0 && tid == 0)
          g.part.desc[unit] = make_int2(a1 < tiles ? b : -1,
                                        last >= 0 ? last : (at + tiles - 1) / sh.per);
      // the next piece's loads and products come after this one's results
      __syncwarp();
      __syncthreads();
      tc_after();
    }
    pos = at + a1;
    at += tiles;
    ++unit;
  }
  if (tid == 0) g.ws.desc[b] = desc;
  end_pass(g);
  asm volatile("cp.async.wait_all;" ::: "memory");
  tc_before();
  __syncthreads();
  if (*up) {
    // the last boxes of each ring slot, or bulk copies of each raw stage, and all products
    constexpr int kDepth = IMAGE ? P::kRaw : P::kSlots;
    const uint32_t bar = IMAGE ? rfull : full;
    if (warp == kLoadWarp) {
      for (int k = max(0, sent - kDepth); k < sent; ++k)
        bar_drain(bar + 8 * (k % kDepth), k / kDepth & 1);
    } else if (warp >= kIssueWarp) {
      if (elected()) commit(drained);
      __syncwarp();
      bar_drain(drained, 0);
    }
    __syncthreads();
  }
  if (warp == kIssueWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// Joins the pieces of the unit that starts in block blockIdx.x and ends in a later one:
// kJoinCols features of it, a thread per row. Units can be few and of many pieces (64 tokens over 8
// slices: 8 of 19), so a block has few features, and the loads of kJoinAhead pieces are under way at
// once (with 32 features a block and a piece at a time those took 62 us in all, now 25).
constexpr int kJoinCols = 8, kJoinAhead = 4;
template <int D, int NQ, int COLS, typename Args>
__global__ void __launch_bounds__(kTcRows) attend_tc_join_kernel(Args g) {
  constexpr int kAhead = kJoinAhead;
  grid_dep_wait();
  const int b = blockIdx.x, d0 = blockIdx.y * COLS, r = threadIdx.x;
  const int2 desc = g.ws.desc[b];
  if (desc.x < 0) return;
  const AttendUnit u = attend_unit<kRows * NQ>(g, desc.x);
  if (r >= u.rows) return;
  const bool joins = part_joins(g, u);
  float m = -INFINITY, l = 0.f, o[COLS];
#pragma unroll
  for (int e = 0; e < COLS; ++e) o[e] = 0.f;
  if constexpr (COLS > kJoinCols) {      // many units, of a few pieces each
    for (int i = b; i <= desc.y; ++i) {
      const int piece = i == b ? 2 * b + 1 : 2 * i;
      const float2 x = g.ws.stat[piece * kTcRows + r];
      const float nm = fmaxf(m, x.x), ref = nm == -INFINITY ? 0.f : nm;
      const float f0 = ex2(m - ref), f1 = x.x == -INFINITY && x.y != x.y ? 1.f : ex2(x.x - ref);
      l = l * f0 + x.y * f1;
      m = nm;
      const float* p = g.ws.out + ((long long)piece * D + d0) * kTcRows + r;
#pragma unroll
      for (int e = 0; e < COLS; ++e) o[e] = o[e] * f0 + p[e * kTcRows] * f1;
    }
  } else {
#pragma unroll 1
    for (int i0 = b; i0 <= desc.y; i0 += kAhead) {
      float2 x[kAhead];
      float y[kAhead][COLS];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int i = i0 + a;
        if (i > desc.y) continue;
        const int piece = i == b ? 2 * b + 1 : 2 * i;
        x[a] = g.ws.stat[piece * kTcRows + r];
        const float* p = g.ws.out + ((long long)piece * D + d0) * kTcRows + r;
#pragma unroll
        for (int e = 0; e < COLS; ++e) y[a][e] = p[e * kTcRows];
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (i0 + a > desc.y) continue;
        const float nm = fmaxf(m, x[a].x), ref = nm == -INFINITY ? 0.f : nm;
        const float f0 = ex2(m - ref);
        const float f1 = x[a].x == -INFINITY && x[a].y != x[a].y ? 1.f : ex2(x[a].x - ref);
        l = l * f0 + x[a].y * f1;
        m = nm;
#pragma unroll
        for (int e = 0; e < COLS; ++e) o[e] = o[e] * f0 + y[a][e] * f1;
      }
    }
  }
  finish_features<COLS>(g, u, r, D, d0, o, m, l, joins);
}

// Rows of head_dim bf16 values in boxes of 64 features x a page (or a tile); false if the
// driver does not take it or the rows do not fit its 32-bit coordinates.
bool encode_rows(const nx_cache& c, void* base, CUtensorMap* map) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                            &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
               : nullptr;
  }();
  const long long rows = (long long)c.layers * c.kv_heads *
                         (c.page_size ? (long long)c.num_pages * c.page_size
                                      : (long long)c.seqs * c.capacity);
  if (!fn || rows >= (1LL << 31)) return false;
  const cuuint64_t dim[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)rows};
  const cuuint64_t stride[1] = {(cuuint64_t)c.head_dim * 2};
  const cuuint32_t box[2] = {
      64, (cuuint32_t)(c.page_size && c.page_size < kCols ? c.page_size : kCols)};
  const cuuint32_t one[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dim, stride, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NQ, bool IMAGE, typename Args>
cudaError_t launch_t(Args& g, cudaStream_t st, int* launches) {
  constexpr int smem = Plan<D, NQ, IMAGE>::kSmem;
  const long long all = most_tokens(g.t) * g.c.group;
  g.mtiles = (int)((all + kRows * NQ - 1) / (kRows * NQ));
  const long long units = (long long)g.c.seqs * g.c.kv_heads * g.mtiles;
  const long long most = units * ((g.c.capacity + kCols - 1) / kCols);
  g.units = (int)units;
  cudaError_t e = allow_smem<attend_tc_kernel<D, NQ, IMAGE, Args>>(smem);
  if (e != cudaSuccess) return e;
  const int grid = (int)(most < kTcGrid ? most : kTcGrid);
  CUtensorMap map_k{}, map_v{};
  const bool maps = !IMAGE && encode_rows(g.c, g.c.k, &map_k) && encode_rows(g.c, g.c.v, &map_v);
  e = launch_after(attend_tc_kernel<D, NQ, IMAGE, Args>, dim3(grid),
                   dim3(Plan<D, NQ, IMAGE>::kThreads), smem, st, map_k, map_v, maps, g);
  if (e != cudaSuccess) return e;
  note_launch(st, launches, "attend_tc");
  if constexpr (kShared<Args>)
    if (g.pass == 1) return e;         // launch_attend_meet
  if (units * 2 <= kSms)
    e = launch_after(attend_tc_join_kernel<D, NQ, kJoinCols, Args>, dim3(grid, D / kJoinCols),
                     dim3(kTcRows), 0, st, g);
  else
    e = launch_after(attend_tc_join_kernel<D, NQ, 32, Args>, dim3(grid, D / 32), dim3(kTcRows), 0, st, g);
  if (e == cudaSuccess) note_launch(st, launches, "attend_tc_join");
  return e;
}

template <int D, int NQ, typename Args>
cudaError_t launch_t(Args& g, cudaStream_t st, int* launches) {
  return g.im.k ? launch_t<D, NQ, true>(g, st, launches) : launch_t<D, NQ, false>(g, st, launches);
}

template <typename Args>
cudaError_t launch_tc(Args& g, cudaStream_t st, int* launches) {
  const bool two = most_tokens(g.t) * g.c.group > kRows;
  if (g.c.head_dim == 128)
    return two ? launch_t<128, 2>(g, st, launches) : launch_t<128, 1>(g, st, launches);
  return two ? launch_t<64, 2>(g, st, launches) : launch_t<64, 1>(g, st, launches);
}

}  // namespace
}  // namespace nx
