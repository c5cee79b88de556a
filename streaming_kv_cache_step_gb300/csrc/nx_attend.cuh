// nx_attend.cuh -- what the kernels of nexus_attend share: their arguments, the work units,
// and where the pieces of a split unit meet. Not part of the public ABI.
#pragma once

#include <cuda_fp8.h>
#include <math.h>

#include "nx_internal.cuh"

namespace nx {

// Where the pieces of split units wait to be joined. A unit is split where the boundary between
// two thread blocks cuts it, so there are at most two pieces per thread block, however many
// units there are: a unit's first piece, if it goes on in the next block, is at slot 2 b + 1 of
// the block b that it starts in, its other pieces are at 2 b' of the blocks b' that go on with
// it. The layout within a slot is its kernel's own.
constexpr int kSms = 152;
struct AttendWs {
  int2* desc;          // [blocks] (unit, last block) of the unit that starts in block b and goes
                       // on in the next ones; unit < 0: none
  float2* stat;        // [2 * blocks][rows] running maximum (log2 units) and sum
  float* out;          // [2 * blocks][rows x head_dim] unnormalised output
};

struct AttendArgs {
  nx_cache c;
  nx_tokens t;
  nx_image im;          // im.k null: no image
  nx_attend a;
  int32_t* dev_status;
  AttendWs ws;
  int b, b_shift;       // rows per image block, a power of two
  int mtiles;           // row tiles per slice
  int ranks;            // row kernel: thread blocks per unit, one cluster (0: even shares)
  int splits;           // its join: blocks per unit (0: a block for each block's last unit)
  int units;            // seqs * kv_heads * mtiles
  float c1;             // scale * log2(e)
};

// Unit (slice of the layer, row tile): up to `rows` query rows (row r = token r / group, head
// r % group of the slice) over slots [0, end); `low` of those slots are seen by every row.
struct AttendUnit {
  int s, h, first, n;   // sequence, KV head, first token, tokens
  int r0, rows;         // first row and rows of the tile
  int T, held;          // rows of the slice, of its image
  int end, low;
};

__device__ __forceinline__ int row_limit(const AttendArgs& g, const AttendUnit& u, int r) {
  const int m = g.a.causal ? u.T - (u.n - 1 - r / g.c.group) : u.T;
  return m < 0 ? 0 : m;
}

template <int ROWS>
__device__ __forceinline__ AttendUnit attend_unit(const AttendArgs& g, int id) {
  AttendUnit u;
  const int mt = id % g.mtiles, sl = id / g.mtiles;
  u.h = sl % g.c.kv_heads;
  u.s = sl / g.c.kv_heads;
  u.n = tokens_of(g.t, u.s, u.first);
  if (u.n < 0) {
    atomicOr(g.dev_status, NX_DEV_BAD_TOKENS);
    u.n = 0;
  }
  const int slice = g.t.layer * g.c.seqs * g.c.kv_heads + sl;
  u.T = g.c.lens[slice];
  u.held = g.im.k ? g.im.rows[slice] : 0;
  int flag = 0;
  if (u.T < 0 || u.T > g.c.capacity) flag = NX_DEV_BAD_LEN;
  else if (u.held < 0 || u.held > u.T || u.held % g.b) flag = NX_DEV_BAD_IMAGE;
  if (flag) {
    atomicOr(g.dev_status, flag);
    u.T = u.held = 0;
  }
  const long long all = (long long)u.n * g.c.group;
  u.r0 = mt * ROWS;
  u.rows = all <= u.r0 ? 0 : all - u.r0 < ROWS ? (int)(all - u.r0) : ROWS;
  u.end = u.rows ? row_limit(g, u, u.r0 + u.rows - 1) : 0;
  u.low = u.rows ? row_limit(g, u, u.r0) : 0;
  return u;
}

// A thread block's share of all tiles (up to 2^31 - 1): `per` of `total` from `start` to `stop`,
// the first of them in unit `unit`, whose first tile has number `at`.
struct AttendShare {
  int per, total, start, stop, unit, at;
};
__host__ __device__ constexpr int share_per(int total, int blocks) {
  return total < 1 ? 1 : (int)((total + (long long)blocks - 1) / blocks);
}
// Where block b's share begins; it ends where the next one's does.
__host__ __device__ constexpr int share_start(int total, int per, int b) {
  return (long long)per * b < total ? per * b : total;
}

// Every one of THREADS threads adds up a run of units; tiles(i): tiles of unit i. unit and at
// are undefined if start >= total.
template <int THREADS, typename Tiles>
__device__ __forceinline__ AttendShare attend_share(const AttendArgs& g, const Tiles& tiles) {
  __shared__ int s_sum[THREADS / 32], s_at[2];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int run = (g.units + THREADS - 1) / THREADS;
  const int u0 = (int)min((long long)g.units, (long long)tid * run), u1 = min(g.units, u0 + run);
  int sum = 0;
  for (int i = u0; i < u1; ++i) sum += tiles(i);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  AttendShare x;
  x.total = total;
  x.per = share_per(total, gridDim.x);
  const int start = share_start(total, x.per, blockIdx.x);
  if (start >= before && start - before < sum) {
    int at = before;
    for (int i = u0; i < u1; ++i) {
      const int n = tiles(i);
      if (start - at < n) {
        s_at[0] = i;
        s_at[1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  x.start = start;
  x.stop = share_start(total, x.per, blockIdx.x + 1);
  x.unit = s_at[0];
  x.at = s_at[1];
  return x;
}

// Where a unit's rows lie. A run of 8 slots that starts at a multiple of 8 needs one page table
// entry: pages and image blocks are multiples of 8 rows.
struct SlotRows {
  const int32_t* table;  // the sequence's pages; null: contiguous
  long long first;       // contiguous: the slice's first row; paged: (layer, head)'s offset
  long long per_page;    // rows from one page to the next
  int shift, pages;

  __device__ __forceinline__ SlotRows(const AttendArgs& g, const AttendUnit& u) {
    const nx_cache& c = g.c;
    shift = 0;
    pages = c.num_pages;
    per_page = 0;
    if (c.page_size) {
      table = c.block_table + (long long)u.s * c.max_pages_per_seq;
      shift = __ffs(c.page_size) - 1;
      per_page = (long long)c.kv_heads << shift;
      first = (long long)g.t.layer * c.num_pages * per_page + ((long long)u.h << shift);
    } else {
      table = nullptr;
      first = (((long long)g.t.layer * c.seqs + u.s) * c.kv_heads + u.h) * c.capacity;
    }
  }
  __device__ __forceinline__ int page(int slot, int end) const {
    return table && slot < end ? table[slot >> shift] : 0;
  }
  // row of a slot below `end`, given its page() ; -1: a bad page, -2: at or beyond `end`
  __device__ __forceinline__ long long row(int slot, int end, int page) const {
    return slot >= end                 ? -2
           : !table                    ? first + slot
           : page < 0 || page >= pages ? -1
                                       : first + page * per_page + (slot & ((1 << shift) - 1));
  }
};

// Asynchronous copy of 16 bytes to shared memory, or of as many zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 2^x to about 2^-22.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(r);
}
// Which of a word's values are not finite: all bits of theirs (4-byte values: fp32, 2: bf16, 1: e4m3
// codes).
template <int BYTES>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if constexpr (BYTES == 4) return (w & 0x7F800000u) == 0x7F800000u ? 0xFFFFFFFFu : 0u;
  else if constexpr (BYTES == 2) return __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u);
  else return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}
// Four e4m3 codes as two pairs of fp16.
__device__ __forceinline__ void e4m3_pairs(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// The most tokens that one sequence can own.
inline long long most_tokens(const nx_tokens& t) {
  return t.max_tokens < t.tokens ? t.max_tokens : t.tokens;
}

// nx_attend_tc.cu: the tensor-core kernel for many query rows per slice (bf16 caches), its
// workspace (base may be null; returns the bytes), and whether it takes a call, or may take one of
// another capacity or from an image.
bool attend_tc_takes(const nx_cache& c, const nx_tokens& t, bool image);
bool attend_tc_may_take(const nx_cache& c, const nx_tokens& t);
size_t attend_tc_layout(int D, char* base, AttendWs* ws);
cudaError_t launch_attend_tc(AttendArgs& g, cudaStream_t st, int* launches);

}  // namespace nx
