// nx_attend.cuh -- what the kernels of nexus_attend share: their arguments, the work units,
// and where the pieces of a split unit meet. Not part of the public ABI.
#pragma once

#include <math.h>

#include "nx_internal.cuh"

namespace nx {

// The workspace of nexus_attend, of a size that depends on head_dim alone: a split unit is
// one that the boundary between two thread blocks cuts, so there are at most two pieces per
// thread block, however many units there are.
constexpr int kAttendGrid = 152 * 4;          // thread blocks of one launch, at most
constexpr int kPieceRows = 16;                // query rows of a piece, at most
struct AttendWs {
  int2* desc;          // [kAttendGrid] (unit, last block) of the unit that starts in block b
                       // and goes on in the next ones; unit < 0: none
  float2* stat;        // [2 * kAttendGrid][kPieceRows] running maximum (log2 units) and sum
  float* out;          // [2 * kAttendGrid][kPieceRows][head_dim] unnormalised output
};

struct AttendArgs {
  nx_cache c;
  nx_tokens t;
  nx_image im;          // im.k null: no image
  nx_attend a;
  int32_t* dev_status;
  AttendWs ws;
  int b;                // rows per image block
  int mtiles;           // row tiles per slice
  int units;            // seqs * kv_heads * mtiles
  int min_tiles;        // tiles of a thread block, at least
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

}  // namespace nx
