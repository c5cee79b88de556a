// nx_attend_tc_shared.cu -- the tensor-core kernel for passes of nexus_attend_shared, and the kernel that
// joins a prefix's pieces with the sequences' own.
#include "nx_attend_tc.cuh"

namespace nx {
namespace {

// Whether the own rows' pass left something for a token that shares prefix p: if its sequence's
// tokens are where they should be and that pass found the same prefix (part_joins).
__device__ __forceinline__ bool own_part(const SharedArgs& g, int p, int token) {
  SharedArgs o = g;
  o.pass = 3;
  AttendUnit u;
  if (!g.t.cu_tokens) {
    u.s = token / g.part.max_tokens;
    u.first = u.s * g.part.max_tokens;
    u.n = g.part.max_tokens;
  } else {
    const int s0 = g.part.cu_seqs ? g.part.cu_seqs[p] : 0;
    const int s1 = g.part.cu_seqs ? g.part.cu_seqs[p + 1] : g.part.seqs;
    u.s = s0;
    for (int hi = s1; hi - u.s > 1;) {
      const int mid = (u.s + hi) / 2;
      if (g.t.cu_tokens[mid] <= token) u.s = mid;
      else hi = mid;
    }
    const auto owns = [&] {
      u.n = tokens_of(g.t, u.s, u.first, g.part.max_tokens);
      return u.n > 0 && token >= u.first && token - u.first < u.n;
    };
    // Entries that decrease or leave the tokens take away the sequences that they bound and no others, but
    // lead the search astray: one after the other, then.
    if (!owns()) {
      for (u.s = s0; u.s < s1 && !owns();) ++u.s;
      if (u.s == s1) return false;
    }
  }
  return part_joins(o, u);
}

// The end where the two passes ran next to each other: the pieces of a unit of the prefixes, or all of
// it, and what its rows have of their own. A block has kJoinCols features of 256 / GROUPS rows, a thread
// each, and deals the pieces to GROUPS of those.
template <int D, int NQ, int GROUPS>
__global__ void __launch_bounds__(kTcRows) attend_meet_kernel(const __grid_constant__ SharedArgs g) {
  constexpr int kEach = kTcRows / GROUPS;
  __shared__ float s_m[GROUPS][kEach], s_l[GROUPS][kEach], s_o[GROUPS][kJoinCols][kEach + 1];
  const int unit = blockIdx.x, d0 = blockIdx.y * kJoinCols;
  const int group = threadIdx.x / kEach, mine = threadIdx.x % kEach, r = blockIdx.z * kEach + mine;
  grid_dep_wait();
  const AttendUnit u = attend_unit<kRows * NQ>(g, unit);
  if (blockIdx.z * kEach >= u.rows) return;
  int2 desc = g.part.desc[unit];
  desc.y = min(desc.y, kTcGrid - 1);     // (its pieces exist, whatever gave up)
  const bool here = r < u.rows;
  const long long at = part_row(g, u, here ? r : 0);
  // the own rows' part, while the pieces are on their way
  float2 own = make_float2(-INFINITY, 0.f);
  float4 own_o[kJoinCols / 4];
  bool there = false;
  if (here && group == 0) {
    own = g.part.own_stat[at];
#pragma unroll
    for (int i = 0; i < kJoinCols / 4; ++i)
      own_o[i] = reinterpret_cast<const float4*>(g.part.own_out + at * D + d0)[i];
    there = own_part(g, u.s, u.first + (u.r0 + r) / g.c.group);
  }
  float m = -INFINITY, l = 0.f, o[kJoinCols];
#pragma unroll
  for (int e = 0; e < kJoinCols; ++e) o[e] = 0.f;
  if (desc.x < 0) {
    if (here && group == 0) {
      const float2 x = g.part.stat[at];
      m = x.x;
      l = x.y;
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) o[e] = g.part.out[at * D + d0 + e];
    }
  } else {
#pragma unroll 1
    for (int i0 = desc.x + group; i0 <= desc.y; i0 += kJoinAhead * GROUPS) {
      float2 x[kJoinAhead];
      float y[kJoinAhead][kJoinCols];
#pragma unroll
      for (int a = 0; a < kJoinAhead; ++a) {
        const int i = i0 + a * GROUPS;
        x[a] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) y[a][e] = 0.f;
        if (i > desc.y || !here) continue;
        const int piece = i == desc.x ? 2 * i + 1 : 2 * i;
        x[a] = g.ws.stat[piece * kTcRows + r];
        const float* p = g.ws.out + ((long long)piece * D + d0) * kTcRows + r;
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) y[a][e] = p[e * kTcRows];
      }
#pragma unroll
      for (int a = 0; a < kJoinAhead; ++a) {
        const float2 k = join_by(m, l, x[a]);
        l = l * k.x + x[a].y * k.y;
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) o[e] = o[e] * k.x + y[a][e] * k.y;
      }
    }
    if constexpr (GROUPS > 1) {
      s_m[group][mine] = m;
      s_l[group][mine] = l;
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) s_o[group][e][mine] = o[e];
      __syncthreads();
      if (group == 0)
#pragma unroll
        for (int w = 1; w < GROUPS; ++w) {
          const float2 x = make_float2(s_m[w][mine], s_l[w][mine]), k = join_by(m, l, x);
          l = l * k.x + x.y * k.y;
#pragma unroll
          for (int e = 0; e < kJoinCols; ++e) o[e] = o[e] * k.x + s_o[w][e][mine] * k.y;
        }
    }
  }
  if (!there) return;                    // no row, no output: its sequence is flagged
  const float2 k = join_by(m, l, own);
  l = l * k.x + own.y * k.y;
#pragma unroll
  for (int i = 0; i < kJoinCols / 4; ++i) {
    o[4 * i] = o[4 * i] * k.x + own_o[i].x * k.y;
    o[4 * i + 1] = o[4 * i + 1] * k.x + own_o[i].y * k.y;
    o[4 * i + 2] = o[4 * i + 2] * k.x + own_o[i].z * k.y;
    o[4 * i + 3] = o[4 * i + 3] * k.x + own_o[i].w * k.y;
  }
  finish_output<kJoinCols>(g, u, r, D, d0, o, m, l);
}

template <int D, int NQ>
cudaError_t launch_meet(const SharedArgs& g, cudaStream_t st) {
  // As many groups as leave about two blocks an SM. Both passes, in us, with 1, 2, 4 and 8 groups: 1
  // unit of 152 pieces 41, 33, 29, 27; 8 units of 19, 128 rows 54, 54, 53, 55, 256 rows 64, 60, 60, 62;
  // 32 units, 128 rows 32, 32, 35, 41.
  int groups = 8;
  while (groups > (NQ == 1 ? 2 : 1) &&
         (long long)g.units * (D / kJoinCols) * (kRows * NQ * groups / kTcRows) > 2 * kSms)
    groups /= 2;
  const dim3 grid(g.units, D / kJoinCols, kRows * NQ * groups / kTcRows), block(kTcRows);
  return groups == 8   ? launch_after(attend_meet_kernel<D, NQ, 8>, grid, block, 0, st, g)
         : groups == 4 ? launch_after(attend_meet_kernel<D, NQ, 4>, grid, block, 0, st, g)
         : groups == 2 ? launch_after(attend_meet_kernel<D, NQ, 2>, grid, block, 0, st, g)
                       : launch_after(attend_meet_kernel<D, NQ, 1>, grid, block, 0, st, g);
}

}  // namespace

size_t attend_tc_units(const nx_cache& c, const nx_tokens& t) {
  const long long all = most_tokens(t) * c.group, rows = kRows * (all > kRows ? 2 : 1);
  return (size_t)c.seqs * c.kv_heads * ((all + rows - 1) / rows);
}

cudaError_t launch_attend_tc(SharedArgs& g, cudaStream_t st, int* launches) {
  return launch_tc(g, st, launches);
}

cudaError_t launch_attend_meet(const SharedArgs& g, cudaStream_t st, int* launches) {
  const bool two = most_tokens(g.t) * g.c.group > kRows;
  const cudaError_t e = g.c.head_dim == 128
                            ? (two ? launch_meet<128, 2>(g, st) : launch_meet<128, 1>(g, st))
                            : (two ? launch_meet<64, 2>(g, st) : launch_meet<64, 1>(g, st));
  if (e == cudaSuccess) note_launch(st, launches, "attend_meet");
  return e;
}

}  // namespace nx
