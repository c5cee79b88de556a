// nx_attend.cu -- nexus_attend: softmax attention of new tokens over one layer's slices, from
// the cache or from its 8-bit image.
//
// With x_j = c1 <q, k_j> (c1 = scale log2 e), one pass over a slice keeps a running reference
// m, the sum l = sum 2^(x_j - m) and o = sum 2^(x_j - m) v_j; raising m to m' multiplies l and
// o by 2^(m - m'). Pieces of a slice join by the same rule. All three are binary32.
//
// A slice with one new token has group = 4..8 query rows per 512 B of K and V (256 B from the
// image): some 4 flop a byte, far below what the tensor cores need to matter, so the kernel
// is a stream of K and V from HBM. What it does per byte is kept small instead:
//   - every warp works alone on 16 slots at a time: K and V reach a ring of its own in shared
//     memory by asynchronous 16-byte copies, some steps ahead, and go from there into mma
//     fragments by 16-byte loads. The order of features inside a dot product is free, so that
//     16 bytes of a K row are a lane's operands of two (bf16) or four (e4m3) k-steps, with the
//     query rows loaded in the same order; V's operands pair two slots of one feature, which
//     takes one byte permute each. No barrier but the warp's own;
//   - an mma has 16 rows, a decode step 8 or fewer: the spare eight carry the probabilities'
//     rounding errors (p = hi + lo), so that bf16 probabilities cost no accuracy.
// The slots of all slices, 64 to a tile, are dealt out evenly to as many thread blocks as fit
// the GPU at once, whatever the slices' lengths; a slice that a boundary cuts is joined by
// attend_join_kernel. Where a cache has few or short slices the latencies of two launches count
// more than an even deal: a slice is then a block's own, or a cluster's, whose blocks join their
// pieces from one another's shared memory.
//
// Measured, one new token of 16 x 8 slices of 32768 rows, 4 query heads each: 310 us in bf16
// (6.9 TB/s of K and V, what a plain copy reaches), 165 us from the image (6.5 TB/s); 64
// sequences of ragged lengths in 16-row pages 270 to 284 us by the lengths (6.4 to 6.7 TB/s); 8
// slices of 1638 rows 9.6 us, latencies; 8 slices of 64 rows 5.9 us. fp32: 64 slices of 6000 rows
// 82 us (4.8 TB/s), 8 slices of 8192 rows 25 us for one token, 105 for 16 and 371 for 64, which take a
// pass over K and V and their terms for every 8 query rows.
#include "nx_attend.cuh"

namespace nx {
namespace {

constexpr int kWarps = 4;
constexpr int kAttendGrid = kSms * 3;  // thread blocks of one launch, at most
constexpr int kRanks = 8;              // thread blocks of a cluster (the portable limit)
constexpr int kPieceRows = 16;         // query rows of a piece, at most
// kTail: bf16 rows behind an image, with their output features in the image's order
enum Kind { kBf16 = 0, kImage = 1, kF32 = 2, kTail = 3 };
template <int KIND>
constexpr bool kIsBf16 = KIND == kBf16 || KIND == kTail;

// m is only raised when a logit is more than 2^kSlack above it, so probabilities are at most 16. From
// the image they are kept at 2^kUp times their size while its rows last, at most 32768: below fp16's
// largest value, with 2^-36 of the largest one still representable. A probability is then
// multiplied by its values' scale, in units of the largest scale so far, before it becomes fp16: that
// leaves 2^-28 of the largest while scales stay within kApart of one another. From the first step
// with a run below that on, a warp's steps go to pv_apart, whose operands never hold a scale (behind a
// block of zeros, whose scale is 1, values of 2^-12 take 119 us over 32 x 8 x 6960 rows, one token, not
// 82; the check itself 0.6 of 165 us over 16 x 8 x 32768).
constexpr float kUp = 11.f, kSlack = 4.f, kApart = 0.00390625f;

template <int KIND>
__device__ __forceinline__ void mma16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (kIsBf16<KIND>)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int KIND>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kIsBf16<KIND>) {
    return bf16_pair(a, b);
  } else {
    const __half2 r = __floats2half2_rn(a, b);
    return reinterpret_cast<const uint32_t&>(r);
  }
}

// What rounding to 16 bits took off a pair.
template <int KIND>
__device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t hi) {
  if constexpr (kIsBf16<KIND>)
    return pack2<KIND>(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
  const __half2 h = reinterpret_cast<const __half2&>(hi);
  return pack2<KIND>(a - __low2float(h), b - __high2float(h));
}

// A binary32 value as the sum of two tf32 operands (11 bits each), to 2^-23 of it: the nearest
// tf32, and the nearest to what that leaves (of an infinity: NaN, see plain_logits).
__device__ __forceinline__ uint32_t tf32_near(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tf32_terms(uint32_t x, uint32_t& hi, uint32_t& lo) {
  hi = tf32_near(__uint_as_float(x));
  lo = tf32_near(__uint_as_float(x) - __uint_as_float(hi));
}
// All four products of the terms of a (rows 0-7: high, 8-15: low) and b over 8 features or
// slots, as two mma with a fresh accumulator: the tensor cores cut off what they add up
// (their sums err to one side), so long sums are left to rounded additions.
__device__ __forceinline__ void mma_f32(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  uint32_t h0, l0, h1, l1;
  tf32_terms(b0, h0, l0);
  tf32_terms(b1, h1, l1);
  float t[4];
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(t[0]), "=f"(t[1]), "=f"(t[2]), "=f"(t[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(l0), "r"(l1), "f"(0.f));
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(t[0]), "+f"(t[1]), "+f"(t[2]), "+f"(t[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(h0), "r"(h1));
  d[0] += t[0] + t[2];
  d[1] += t[1] + t[3];
}

// Slots of a thread block's tile: a step, or more, of each warp.
template <int KIND>
constexpr int kTileOf = KIND == kImage ? 128 : 64;

// How K and V of KIND reach the fragments. g = lane / 4 and c = lane % 4 as in an mma.
template <int KIND, int D>
struct Shape {
  static constexpr int kSlots = KIND == kImage ? 32 : KIND == kBf16 ? 16 : 8;  // of a step
  static constexpr int NT = kSlots / 8;                          // mma column tiles of them
  static constexpr int kBytes = KIND == kF32 ? 4 : kIsBf16<KIND> ? 2 : 1;
  static constexpr int kRow = D * kBytes;                        // bytes of a row
  static constexpr int kChunks = kRow / 16;                      // 16-byte chunks of a row
  static constexpr int kStage = 2 * kSlots * kRow;               // one step's K and V
  static constexpr int KV = kRow / 64;                           // 16-byte loads of a K row
  static constexpr int VV = kRow >= 128 ? kRow / 128 : 1;        // loads of a V row
  static constexpr int kPer = D / 8 / VV;                        // features of one V load
  // V load w of lane g covers features w kWide + g kStep .. + kPer - 1: neighbouring lanes
  // neighbouring chunks, but behind an image what the image's lane g has (D / 8 in a row)
  static constexpr int kStep = KIND == kTail ? D / 8 : kPer;
  static constexpr int kWide = KIND == kTail ? kPer : 8 * kPer;
  // the feature that column n of output tile t stands for
  static __device__ __forceinline__ int feature(int t, int n) {
    return t / kPer * kWide + n * kStep + t % kPer;
  }
  // Where chunk i of row r lies in a stage: rows are multiples of 128 bytes (64 for an image
  // with D = 64), so that the rows one load instruction touches would share their banks. K is
  // read as chunks c .. of rows g (two rows to a 128-byte wavefront), V as chunks g of rows
  // 2c (four rows to one).
  static __device__ __forceinline__ int k_at(int r, int i) {
    return r * kRow + 16 * (kChunks >= 8 ? i ^ 4 * (r & 1) : i);
  }
  static __device__ __forceinline__ int v_at(int r, int i) {
    return r * kRow + 16 * (kChunks >= 8 ? i ^ 2 * (r >> 1 & 3) : i ^ (r >> 1 & 3));
  }
};

// A warp's ring: stages of one step each. kPerSm thread blocks of four warps share an SM's
// 227 KB; an image's tail takes the image's ring. From the image three blocks, for their
// conversions' latencies (16 rows against two blocks: 4 x 32768 slots, 8 heads, 20 query rows 86.9
// us, not 100.4, 16 rows 65.4, not 67.2; 32 x 6960, 20 rows 140.4, not 154.3, 16 rows 93.7, not
// 90.5).
template <int KIND, int D, int ROWS>
struct Ring {
  static constexpr int kPerSm = KIND == kImage ? 3 : 2;
  static constexpr int kBytes = Shape<KIND, D>::kStage;
  static constexpr int kFit = 196608 / (kPerSm * kWarps * kBytes);
  static constexpr int kDeep = kFit > 8 ? 8 : kFit;
};

// One warp's running state: o[t] holds rows g (c0, c1) and g + 8 (c2, c3) of output tile t.
template <int D, int ROWS>
struct State {
  float o[D / 8][4];
  float m[ROWS / 8], l[ROWS / 8];
};

__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at)
               : "memory");
  return x;
}

// What a step needs to know besides its rows.
struct __align__(16) Meta {
  float scale[8];       // image: the scales of K's (0-3) and V's (4-7) runs of 8 slots
  int bad[4];           // 1: a run on a bad page
};

// Starts the copies of a step's rows. WHOLE: all of them follow row[0]. Otherwise run j's are at
// row[j], and zeros take the place of those that do not exist (`left` slots are left).
template <int KIND, int D, bool WHOLE>
__device__ __forceinline__ void copy_rows(const AttendArgs& g, const long long* row, int left,
                                          int lane, uint32_t stage) {
  using S = Shape<KIND, D>;
  constexpr int kLine = 32 / S::kChunks > 0 ? 32 / S::kChunks : 1;   // rows per instruction
  static_assert(S::kChunks <= 32 && 8 % kLine == 0, "");
  const char* kb = static_cast<const char*>(KIND == kImage ? g.im.k : g.c.k);
  const char* vb = static_cast<const char*>(KIND == kImage ? g.im.v : g.c.v);
  const int sub = lane / S::kChunks, chunk = lane % S::kChunks;
  if constexpr (WHOLE) {
    const long long at = row[0] * S::kRow + lane * 16;
    const char *k = kb + at, *v = vb + at;
#pragma unroll
    for (int i = 0; i < S::kSlots; i += kLine) {
      copy16(stage + S::k_at(i + sub, chunk), k + i * S::kRow);
      copy16(stage + S::kStage / 2 + S::v_at(i + sub, chunk), v + i * S::kRow);
    }
  } else {
#pragma unroll
    for (int j = 0; j < S::NT; ++j) {
      const long long at = (row[j] < 0 ? 0 : row[j]) * S::kRow + lane * 16;
      const char *k = kb + at, *v = vb + at;
#pragma unroll
      for (int i = 0; i < 8; i += kLine) {
        const bool ok = row[j] >= 0 && 8 * j + i + sub < left;
        copy16(stage + S::k_at(8 * j + i + sub, chunk), ok ? k + i * S::kRow : kb, ok);
        copy16(stage + S::kStage / 2 + S::v_at(8 * j + i + sub, chunk),
               ok ? v + i * S::kRow : vb, ok);
      }
    }
  }
}

__device__ __forceinline__ uint32_t word(const uint4& x, int i) {
  return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
}

// The query rows of a unit as mma operands, in the feature order of load_k.
template <int KIND, int D, int ROWS>
struct Query {
  using S = Shape<KIND, D>;
  static constexpr int kSteps = KIND == kF32 ? D / 8 : D / 16;
  static constexpr int kRegs = KIND == kF32 ? 2 : 2 * (ROWS / 8);   // per k-step
  uint32_t a[kSteps][kRegs];
  float c1[ROWS / 8];            // c1, times what the queries were divided by

  __device__ __forceinline__ void load(const AttendArgs& g, const AttendUnit& u, int lane) {
#pragma unroll
    for (int e = 0; e < ROWS / 8; ++e) {
      const int r = lane / 4 + 8 * e;
      const bool ok = r < u.rows;
      const int row = u.r0 + r;
      const long long at = ok ? (u.first + row / g.c.group) * g.a.q_stride +
                                    ((long long)u.h * g.c.group + row % g.c.group) * D
                              : 0;
      c1[e] = g.c1;
      if constexpr (kIsBf16<KIND>) {
        const char* p = static_cast<const char*>(g.a.q) + at * 2 + lane % 4 * 16;
#pragma unroll
        for (int i = 0; i < S::KV; ++i) {
          const uint4 x = ok ? *reinterpret_cast<const uint4*>(p + i * 64) : make_uint4(0, 0, 0, 0);
          a[2 * i][2 * e] = x.x;
          a[2 * i][2 * e + 1] = x.y;
          a[2 * i + 1][2 * e] = x.z;
          a[2 * i + 1][2 * e + 1] = x.w;
        }
      } else if constexpr (KIND == kF32) {
        const char* p = static_cast<const char*>(g.a.q) + at * 4 + lane % 4 * 16;
#pragma unroll
        for (int i = 0; i < S::KV; ++i) {
          const uint4 x = ok ? *reinterpret_cast<const uint4*>(p + i * 64) : make_uint4(0, 0, 0, 0);
          a[2 * i][0] = x.x;
          a[2 * i][1] = x.y;
          a[2 * i + 1][0] = x.z;
          a[2 * i + 1][1] = x.w;
        }
      } else {
        // e4m3 codes become fp16, and so does the query row, divided by the power of two that
        // brings its largest value to [2^13, 2^14): bf16's eight bits are kept down to 2^-28
        // of that value, and what is lost below is at most 2^-38 of it
        const char* p = static_cast<const char*>(g.a.q) + at * 2 + lane % 4 * 32;
        uint4 x[S::KV][2];
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < S::KV; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            x[i][y] = ok ? *reinterpret_cast<const uint4*>(p + i * 128 + y * 16)
                         : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              most = fmaxf(most, fabsf(__uint_as_float(word(x[i][y], w) << 16)));
              most = fmaxf(most, fabsf(__uint_as_float(word(x[i][y], w) & 0xFFFF0000u)));
            }
          }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        int up = 0;
        if (most > 0.f && most < INFINITY) {
          frexpf(most, &up);
          up = 14 - up;
        }
        c1[e] = ldexpf(g.c1, -up);
        const float f0 = ldexpf(1.f, up / 2), f1 = ldexpf(1.f, up - up / 2);
#pragma unroll
        for (int i = 0; i < S::KV; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t two = word(x[i][y], w);
              a[4 * i + 2 * y + w / 2][2 * e + w % 2] =
                  pack2<kImage>(__uint_as_float(two << 16) * f0 * f1,
                                __uint_as_float(two & 0xFFFF0000u) * f0 * f1);
            }
      }
    }
  }
};

// The products of the query rows with 8 or 16 rows of K.
template <int KIND, int D, int ROWS>
__device__ __forceinline__ void qk(const Query<KIND, D, ROWS>& q, uint32_t stage, int lane,
                                   float s[][4]) {
  using S = Shape<KIND, D>;
#pragma unroll
  for (int j = 0; j < S::NT; ++j) {
    s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int u = 0; u < S::KV; ++u) {
      const uint4 k = lds16(stage + S::k_at(8 * j + lane / 4, 4 * u + lane % 4));
      if constexpr (kIsBf16<KIND>) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t* a = q.a[2 * u + i];
          const uint32_t f[4] = {a[0], ROWS == 16 ? a[2 % (2 * (ROWS / 8))] : 0u, a[1],
                                 ROWS == 16 ? a[3 % (2 * (ROWS / 8))] : 0u};
          mma16<KIND>(s[j], f, word(k, 2 * i), word(k, 2 * i + 1));
        }
      } else if constexpr (KIND == kImage) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t* a = q.a[4 * u + i];
          const uint32_t f[4] = {a[0], ROWS == 16 ? a[2 % (2 * (ROWS / 8))] : 0u, a[1],
                                 ROWS == 16 ? a[3 % (2 * (ROWS / 8))] : 0u};
          uint32_t b0, b1;
          e4m3_pairs(word(k, i), b0, b1);
          mma16<KIND>(s[j], f, b0, b1);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t* a = q.a[2 * u + i];
          uint32_t f[4];
          tf32_terms(a[0], f[0], f[1]);
          tf32_terms(a[1], f[2], f[3]);
          mma_f32(s[j], f, word(k, 2 * i), word(k, 2 * i + 1));
        }
      }
    }
  }
}

// fp32: the logits that came out as NaN, over again without terms: those of an infinite key are
// infinite, and one of -infinity drops out of the softmax. Few registers, and rarely run (with
// terms that mind infinities in every product 64 slices of 6000 rows took 98 us, not 79).
template <int D>
__device__ __forceinline__ void plain_logits(const AttendArgs& g, const AttendUnit& u,
                                             uint32_t stage, int lane, float* s) {
  using S = Shape<kF32, D>;
  const int r = lane / 4, row = u.r0 + r;
  const float4* q = reinterpret_cast<const float4*>(
      static_cast<const float*>(g.a.q) + (u.first + row / g.c.group) * g.a.q_stride +
      ((long long)u.h * g.c.group + row % g.c.group) * D);
#pragma unroll 1
  for (int y = 0; y < 2 && r < u.rows; ++y) {
    float sum = 0.f;
#pragma unroll 1
    for (int i = 0; i < S::kChunks; ++i) {
      const uint4 k = lds16(stage + S::k_at(2 * (lane % 4) + y, i));
      const float4 x = q[i];
      sum += x.x * __uint_as_float(k.x) + x.y * __uint_as_float(k.y) +
             x.z * __uint_as_float(k.z) + x.w * __uint_as_float(k.w);
    }
    if (y == 0) {
      if (s[0] != s[0]) s[0] = sum;
    } else if (s[1] != s[1]) {
      s[1] = sum;
    }
  }
}

// V load w of slot 8 j + 2 c + e.
template <int KIND, int D>
__device__ __forceinline__ uint4 load_v(uint32_t stage, int lane, int j, int e, int w) {
  using S = Shape<KIND, D>;
  const int f = (w * S::kWide + lane / 4 * S::kStep) * S::kBytes;    // byte in the row
  const uint32_t at = stage + S::kStage / 2 + S::v_at(8 * j + 2 * (lane % 4) + e, f / 16);
  if constexpr (S::kRow >= 128) return lds16(at);
  uint4 x = make_uint4(0, 0, 0, 0);
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at + f % 16)
               : "memory");
  return x;
}
// The codes of two slots' words as operands, feature by feature.
__device__ __forceinline__ void code_pairs(uint32_t y0, uint32_t y1, uint32_t* b) {
  const uint32_t z0 = __byte_perm(y0, y1, 0x5140), z1 = __byte_perm(y0, y1, 0x7362);
  e4m3_pairs(z0, b[0], b[1]);
  e4m3_pairs(z1, b[2], b[3]);
}

// o += p V.
template <int KIND, int D, int ROWS>
__device__ __forceinline__ void pv(uint32_t stage, int lane, const float p[][4],
                                   State<D, ROWS>& st) {
  using S = Shape<KIND, D>;
  const auto load = [&](int j, int e, int w) { return load_v<KIND, D>(stage, lane, j, e, w); };
  if constexpr (KIND == kF32) {
    uint32_t f[4];
    tf32_terms(__float_as_uint(p[0][0]), f[0], f[1]);
    tf32_terms(__float_as_uint(p[0][1]), f[2], f[3]);
#pragma unroll
    for (int w = 0; w < S::VV; ++w) {
      const uint4 v0 = load(0, 0, w), v1 = load(0, 1, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) mma_f32(st.o[4 * w + e], f, word(v0, e), word(v1, e));
    }
  } else {
#pragma unroll
    for (int h = 0; h < (S::NT + 1) / 2; ++h) {      // 16 slots (or the only 8) at a time
      constexpr int N = S::NT < 2 ? 1 : 2;
      uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float* y = p[2 * h + j];
        hi[2 * j] = pack2<KIND>(y[0], y[1]);
        lo[2 * j] = rest2<KIND>(y[0], y[1], hi[2 * j]);
        if constexpr (ROWS == 8) {
          hi[2 * j + 1] = lo[2 * j];
        } else {
          hi[2 * j + 1] = pack2<KIND>(y[2], y[3]);
          lo[2 * j + 1] = rest2<KIND>(y[2], y[3], hi[2 * j + 1]);
        }
      }
#pragma unroll
      for (int w = 0; w < S::VV; ++w) {
        uint4 v[N][2];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          v[j][0] = load(2 * h + j, 0, w);
          v[j][1] = load(2 * h + j, 1, w);
        }
#pragma unroll
        for (int i = 0; i < (KIND == kImage && D == 64 ? 2 : 4); ++i) {
          uint32_t b[2][kIsBf16<KIND> ? 2 : 4] = {};
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const uint32_t y0 = word(v[j][0], i), y1 = word(v[j][1], i);
            if constexpr (kIsBf16<KIND>) {
              b[j][0] = __byte_perm(y0, y1, 0x5410);
              b[j][1] = __byte_perm(y0, y1, 0x7632);
            } else {
              code_pairs(y0, y1, b[j]);
            }
          }
#pragma unroll
          for (int e = 0; e < (kIsBf16<KIND> ? 2 : 4); ++e) {
            float* o = st.o[S::kPer * w + (kIsBf16<KIND> ? 2 : 4) * i + e];
            mma16<KIND>(o, hi, b[0][e], b[1][e]);
            // sixteen rows leave no spare ones; fp16 probabilities (2^-11) do without
            if constexpr (ROWS == 16 && kIsBf16<KIND>) mma16<KIND>(o, lo, b[0][e], b[1][e]);
          }
        }
      }
    }
  }
}

// l += sum p and o += p V of an image step whose runs' scales lie far apart, p = 2^(x - m): a run by
// itself, its probabilities in units of the row's largest in the run, and what turns them into o's
// units (scale and all) in binary32 behind the product. x waits where the step's keys were.
template <int D, int ROWS>
__device__ __forceinline__ void pv_apart(uint32_t stage, int lane, const float x[][4],
                                         const float* scale, float vinv, State<D, ROWS>& st) {
  using S = Shape<kImage, D>;
  static_assert(S::NT * 512 <= S::kStage / 2, "");
  __syncwarp();                         // everyone has read the keys
#pragma unroll
  for (int j = 0; j < S::NT; ++j)
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(stage + (32 * j + lane) * 16),
                 "f"(x[j][0]), "f"(x[j][1]), "f"(x[j][2]), "f"(x[j][3])
                 : "memory");
#pragma unroll 1
  for (int j = 0; j < S::NT; ++j) {
    const uint4 y = lds16(stage + (32 * j + lane) * 16);
    float p[4] = {__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z),
                  __uint_as_float(y.w)};
    float f[ROWS / 8];
#pragma unroll
    for (int e = 0; e < ROWS / 8; ++e) {
      float top = fmaxf(p[2 * e], p[2 * e + 1]);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float m = st.m[e] == -INFINITY ? 0.f : st.m[e];
      f[e] = top == -INFINITY ? 0.f : ex2(top - m) * (scale[j] * vinv);
      st.l[e] += ex2(p[2 * e] - m + kUp) + ex2(p[2 * e + 1] - m + kUp);
      const float sub = (top == -INFINITY ? 0.f : top) - kUp;
      p[2 * e] = ex2(p[2 * e] - sub);
      p[2 * e + 1] = ex2(p[2 * e + 1] - sub);
    }
    uint32_t a[4] = {pack2<kImage>(p[0], p[1]), 0, 0, 0};
    if constexpr (ROWS == 8) a[1] = rest2<kImage>(p[0], p[1], a[0]);
    else a[1] = pack2<kImage>(p[2], p[3]);
#pragma unroll
    for (int w = 0; w < S::VV; ++w) {
      const uint4 v0 = load_v<kImage, D>(stage, lane, j, 0, w);
      const uint4 v1 = load_v<kImage, D>(stage, lane, j, 1, w);
#pragma unroll
      for (int i = 0; i < (D == 64 ? 2 : 4); ++i) {
        uint32_t b[4];
        code_pairs(word(v0, i), word(v1, i), b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float t[4] = {0.f, 0.f, 0.f, 0.f};
          mma16<kImage>(t, a, b[e], 0u);
          float* o = st.o[S::kPer * w + 4 * i + e];
          o[0] += t[0] * f[0];
          o[1] += t[1] * f[0];
          o[2] += t[2] * f[ROWS / 8 - 1];
          o[3] += t[3] * f[ROWS / 8 - 1];
        }
      }
    }
  }
}

// A step's value rows [from, to) that some query rows see and others do not: what is not finite in
// them would reach the latter as 0 times an infinity or NaN. Whether there is any:
template <int KIND, int D>
__device__ __forceinline__ bool leaks(uint32_t stage, int lane, int from, int to) {
  using S = Shape<KIND, D>;
  uint32_t bad = 0;
#pragma unroll 1
  for (int i = max(from, 0) * S::kChunks + lane; i < min(to, S::kSlots) * S::kChunks; i += 32) {
    const uint4 x = lds16(stage + S::kStage / 2 + i * 16);
    bad |= not_finite<Shape<KIND, D>::kBytes>(x.x) | not_finite<Shape<KIND, D>::kBytes>(x.y) | not_finite<Shape<KIND, D>::kBytes>(x.z) |
           not_finite<Shape<KIND, D>::kBytes>(x.w);
  }
  return __any_sync(0xffffffffu, bad != 0);
}
// and it goes to the outputs of the rows that see it here, and out of the step's values.
template <int KIND, int D, int ROWS>
__device__ __forceinline__ void take_leaks(uint32_t stage, int lane, int t, int from, int to,
                                           const int* lim, State<D, ROWS>& st) {
  using S = Shape<KIND, D>;
  const uint32_t v = stage + S::kStage / 2;
#pragma unroll 1
  for (int r = max(from, 0); r < min(to, S::kSlots); ++r)
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int f = S::feature(n, 2 * (lane % 4) + y) * S::kBytes, in = f % 4;
        uint32_t w;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(v + S::v_at(r, f / 16) + f % 16 - in));
        if (!(not_finite<Shape<KIND, D>::kBytes>(w) >> 8 * in & 1u)) continue;
        const float x = KIND == kF32     ? __uint_as_float(w)
                        : KIND == kImage ? __uint_as_float(0x7FC00000u)
                        : in             ? __uint_as_float(w & 0xFFFF0000u)
                                         : __uint_as_float(w << 16);
#pragma unroll
        for (int e = 0; e < ROWS / 8; ++e)
          if (t + r < lim[e]) st.o[n][2 * e + y] += x;
      }
  __syncwarp();
#pragma unroll 1
  for (int i = max(from, 0) * S::kChunks * 4 + lane; i < min(to, S::kSlots) * S::kChunks * 4; i += 32) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(v + i * 4));
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(v + i * 4), "r"(w & ~not_finite<Shape<KIND, D>::kBytes>(w)) : "memory");
  }
  __syncwarp();
}

// Slots [base + kSlots * i, ...) for i = from, from + kWarps, ... < to, up to slot `end`. vref: the
// image's largest value scale so far, which o is in units of. Where a run's scale is far below it, or
// a value that only some rows see is not finite, the steps from there on are attend_slow's (SLOW).
template <int KIND, int D, int ROWS, int kDeep, int kStageBytes>
__device__ __noinline__ void attend_slow(const AttendArgs& g, const AttendUnit& u, int base, int end,
                                         int from, int to, uint32_t ring, Meta* meta,
                                         State<D, ROWS>& st, float vref);
template <int KIND, int D, int ROWS, int kDeep, int kStageBytes, bool SLOW = false>
__device__ __forceinline__ void attend_part(const AttendArgs& g, const AttendUnit& u, int base,
                                            int end, int from, int to, uint32_t ring, Meta* meta,
                                            State<D, ROWS>& st, float vref = 1.1754944e-38f) {
  using S = Shape<KIND, D>;
  if (from >= to) return;
  const int lane = threadIdx.x % 32;
  int lim[ROWS / 8];
#pragma unroll
  for (int e = 0; e < ROWS / 8; ++e) {
    const int r = lane / 4 + 8 * e;
    lim[e] = r < u.rows ? min(end, row_limit(g, u, u.r0 + r)) : 0;
  }
  const int low = min(end, u.low);
  float vinv = 1.f / vref;
  const SlotRows at(g, u);
  const long long blocks0 =
      KIND == kImage && !g.c.page_size ? image_scale_at(g.c, g.t.layer, u.s, u.h, 0, g.b) : 0;
  constexpr int kNext = S::kSlots * kWarps;
  static_assert(S::kStage <= kStageBytes, "");
  // whether the rows of a whole step follow one another (base is a multiple of its slots, but
  // behind an image, where a step is one run): one page table entry is enough then
  const bool follow = S::NT == 1 || !at.table || (1 << at.shift) >= S::kSlots;
  int page[S::NT];
  const auto fetch_pages = [&](int t) {
    page[0] = at.page(t, end);
#pragma unroll
    for (int j = 1; j < S::NT; ++j) page[j] = follow ? page[0] : at.page(t + 8 * j, end);
  };
  // starts step i's copies into stage n; `page` holds its table entries (fetched a step ahead,
  // so that their latency is not added to the rows') and then the next step's
  const auto start = [&](int i, int n) {
    const int t = base + S::kSlots * i;
    if (i < to) {
      long long row[S::NT];
      row[0] = at.row(t, end, page[0]);
      // lane j looks after run j: whether its page is good, and the scale of its keys; lane
      // NT + j after that of its values
      const int run = lane % S::NT;
      long long mine;
      if (follow && row[0] >= 0 && t + S::kSlots <= end) {
        copy_rows<KIND, D, true>(g, row, S::kSlots, lane, ring + n * kStageBytes);
        mine = row[0] + 8 * run;
      } else {
        mine = row[0];
#pragma unroll
        for (int j = 1; j < S::NT; ++j) {
          row[j] = at.row(t + 8 * j, end, page[j]);
          if (run == j) mine = row[j];
        }
        copy_rows<KIND, D, false>(g, row, end - t, lane, ring + n * kStageBytes);
      }
      if (lane < S::NT) meta[n].bad[lane] = mine == -1;
      if constexpr (KIND == kImage) {
        const bool ok = mine >= 0;
        const long long x =
            g.c.page_size ? mine >> g.b_shift : blocks0 + (t + 8 * run >> g.b_shift);
        if (lane < 2 * S::NT)
          copy4(smem_at(&meta[n].scale[lane < S::NT ? lane : lane - S::NT + 4]),
                (lane < S::NT ? g.im.k_scale : g.im.v_scale) + (ok ? x : 0), ok);
      }
      fetch_pages(t + kNext);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch_pages(base + S::kSlots * from);
  __syncwarp();                         // the warp is done with what the ring held before
#pragma unroll
  for (int n = 0; n < kDeep - 1; ++n) start(from + n * kWarps, n);
  Query<KIND, D, ROWS> q;               // while the first rows are on their way
  q.load(g, u, lane);
  int n = 0, i = from;
  for (; i < to; i += kWarps) {
    const int t = base + S::kSlots * i;
    asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 2) : "memory");
    __syncwarp();                       // everyone's copies are in, and step i - 1 is read
    start(i + (kDeep - 1) * kWarps, n == 0 ? kDeep - 1 : n - 1);
    const uint32_t stage = ring + n * kStageBytes;
    float ks[S::NT], vs[S::NT];
    bool bad_half[S::NT];
#pragma unroll
    for (int j = 0; j < S::NT; ++j) {
      bad_half[j] = meta[n].bad[j] != 0;
      if constexpr (KIND == kImage) {
        ks[j] = meta[n].scale[j];
        vs[j] = meta[n].scale[4 + j];
      }
    }
    // whether run lane % NT's scale is far below (less one: that of no run is 0)
    const auto far_below = [&](float v) {
      return __float_as_uint(meta[n].scale[4 + lane % S::NT]) - 1u < __float_as_uint(v * kApart) - 1u;
    };
    const bool far = KIND == kImage && !SLOW && far_below(vref);
    n = n == kDeep - 1 ? 0 : n + 1;
    float s[S::NT][4];
    qk<KIND, D, ROWS>(q, stage, lane, s);
    if constexpr (KIND == kF32)
      if (__any_sync(0xffffffffu, s[0][0] != s[0][0] || s[0][1] != s[0][1]))
        plain_logits<D>(g, u, stage, lane, s[0]);

    // logits in log2 units; beyond a row's limit or on a bad page: -inf
    float top[ROWS / 8];
#pragma unroll
    for (int e = 0; e < ROWS / 8; ++e) top[e] = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < S::NT; ++j) bad |= bad_half[j];
    const bool mask = bad || t + S::kSlots > low;
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int e = 0; e < ROWS / 8; ++e)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float& z = s[j][2 * e + y];
          z *= KIND == kImage ? q.c1[e] * ks[j] : q.c1[e];
        }
    if (mask) {
      if (low < end) {                  // (one token: no row sees less than another)
        if constexpr (SLOW) take_leaks<KIND, D, ROWS>(stage, lane, t, low - t, end - t, lim, st);
        else if (leaks<KIND, D>(stage, lane, low - t, end - t)) break;
      }
#pragma unroll
      for (int j = 0; j < S::NT; ++j)
#pragma unroll
        for (int e = 0; e < ROWS / 8; ++e)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (bad_half[j] || t + 8 * j + 2 * (lane % 4) + y >= lim[e])
              s[j][2 * e + y] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int e = 0; e < ROWS / 8; ++e)
        top[e] = fmaxf(top[e], fmaxf(s[j][2 * e], s[j][2 * e + 1]));
    if (bad && lane == 0) atomicOr(g.dev_status, NX_DEV_BAD_PAGE);
    bool up = false;
#pragma unroll
    for (int e = 0; e < ROWS / 8; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      up |= top[e] > st.m[e] + kSlack;
    }
    float vnew = vref;
    if constexpr (KIND == kImage) {
#pragma unroll
      for (int j = 0; j < S::NT; ++j) vnew = fmaxf(vnew, vs[j]);
      up |= vnew > vref || far;
    }
    if (__any_sync(0xffffffffu, up)) {
      if constexpr (KIND == kImage && !SLOW) {
        n = n == 0 ? kDeep - 1 : n - 1;
        const bool leave = __any_sync(0xffffffffu, far_below(vnew));
        n = n == kDeep - 1 ? 0 : n + 1;
        if (leave) break;
      }
      const float vf = KIND == kImage ? vref / vnew : 1.f;
      vref = vnew;
      if constexpr (KIND == kImage) vinv = 1.f / vnew;
      float f[ROWS / 8];
#pragma unroll
      for (int e = 0; e < ROWS / 8; ++e) {
        const float m = top[e] > st.m[e] + kSlack ? top[e] : st.m[e];
        f[e] = m > st.m[e] ? ex2(st.m[e] - m) : 1.f;
        st.m[e] = m;
        st.l[e] *= f[e];
        f[e] *= vf;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        st.o[n][0] *= f[0];
        st.o[n][1] *= f[0];
        st.o[n][2] *= f[ROWS / 8 - 1];
        st.o[n][3] *= f[ROWS / 8 - 1];
      }
    }
    if constexpr (SLOW && KIND == kImage) {
      pv_apart<D, ROWS>(stage, lane, s, meta[n == 0 ? kDeep - 1 : n - 1].scale + 4, vinv, st);
      continue;
    }
    float vr[S::NT];
    if constexpr (KIND == kImage) {
#pragma unroll
      for (int j = 0; j < S::NT; ++j) vr[j] = vs[j] * vinv;
    }
#pragma unroll
    for (int e = 0; e < ROWS / 8; ++e) {
      const float sub = (st.m[e] == -INFINITY ? 0.f : st.m[e]) - (KIND == kImage ? kUp : 0.f);
#pragma unroll
      for (int j = 0; j < S::NT; ++j)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float& z = s[j][2 * e + y];
          z = ex2(z - sub);
          st.l[e] += z;
          if constexpr (KIND == kImage) z *= vr[j];
        }
    }
    pv<KIND, D, ROWS>(stage, lane, s, st);
  }
  if constexpr (!SLOW)
    if (i < to) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if constexpr (KIND == kF32) {
        attend_part<KIND, D, ROWS, kDeep, kStageBytes, true>(g, u, base, end, i, to, ring, meta, st,
                                                             vref);
      } else {
        State<D, ROWS> copy = st;       // in local memory: st and u stay in registers
        const AttendUnit unit = u;
        attend_slow<KIND, D, ROWS, kDeep, kStageBytes>(g, unit, base, end, i, to, ring, meta, copy,
                                                       vref);
        st = copy;
      }
      return;
    }
  if constexpr (KIND == kImage) {
    constexpr float down = 1.f / (1 << (int)kUp);
#pragma unroll
    for (int e = 0; e < ROWS / 8; ++e) st.l[e] *= down;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[n][e] *= vref * down;
  }
}

// The steps from `from` on with what only some need: a function of its own, so that the others' loop
// keeps its registers (image, 16 x 32768 rows: 165 us, 166 as a second loop of the caller; fp32, with
// 255 registers instead of 168, does better with the loop: 64 x 6000 rows 82 us, 84 with the function).
template <int KIND, int D, int ROWS, int kDeep, int kStageBytes>
__device__ __noinline__ void attend_slow(const AttendArgs& g, const AttendUnit& u, int base, int end,
                                         int from, int to, uint32_t ring, Meta* meta,
                                         State<D, ROWS>& st, float vref) {
  State<D, ROWS> mine = st;
  attend_part<KIND, D, ROWS, kDeep, kStageBytes, true>(g, u, base, end, from, to, ring, meta, mine,
                                                       vref);
  st = mine;
}

template <int KIND>
__device__ __forceinline__ int unit_tiles(const AttendUnit& u) {
  constexpr int kTileSlots = kTileOf<KIND>;
  if (!u.rows) return 0;
  const int ea = min(u.held, u.end);
  const int n = (ea + kTileSlots - 1) / kTileSlots + (u.end - ea + kTileSlots - 1) / kTileSlots;
  return n < 1 ? 1 : n;                 // an empty row still has an output
}

template <typename T>
__device__ __forceinline__ void store_out(const AttendArgs& g, const AttendUnit& u, int r, int D,
                                          int f, float x) {
  const int row = u.r0 + r;
  static_cast<T*>(g.a.out)[(long long)(u.first + row / g.c.group) * g.a.out_stride +
                           ((long long)u.h * g.c.group + row % g.c.group) * D + f] = (T)x;
}

// o / l, and ln l with the reference put back.
__device__ __forceinline__ void finish_row(const AttendArgs& g, const AttendUnit& u, int r, int D,
                                           int f, float m, float l, float o) {
  const float y = l == 0.f ? 0.f : o / l;
  if (g.c.dtype == NX_DTYPE_BF16) store_out<__nv_bfloat16>(g, u, r, D, f, y);
  else store_out<float>(g, u, r, D, f, y);
  if (f == 0 && g.a.lse) {
    const int row = u.r0 + r;
    g.a.lse[(long long)(u.first + row / g.c.group) * (g.c.kv_heads * g.c.group) +
            u.h * g.c.group + row % g.c.group] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

// Thread block clusters: everyone's arrival, and another block's shared memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float remote(const float* p, int rank) {
  float x;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(x)
      : "r"(smem_at(p)), "r"(rank)
      : "memory");
  return x;
}

// EVEN: the blocks share all tiles evenly; else `g.ranks` blocks, one cluster, have a unit. Two
// kernels: as one, 8 image rows of 128 features spill 132 bytes of registers instead of 24, and 16
// sequences of 16384 rows take 167.4 us instead of 163.9.
template <int KIND, int D, int ROWS, bool EVEN>
__global__ void __launch_bounds__(kWarps * 32, Ring<KIND, D, ROWS>::kPerSm)
    attend_kernel(const __grid_constant__ AttendArgs g) {
  constexpr int kTileSlots = kTileOf<KIND>;
  using R = Ring<KIND, D, ROWS>;
  constexpr int kRing = R::kDeep * R::kBytes;
  // the rings, and over them, once a piece's steps are done, its warps' outputs
  extern __shared__ __align__(128) char s_ring[];
  float (*s_o)[ROWS][D] = reinterpret_cast<float (*)[ROWS][D]>(s_ring);
  static_assert(kRing >= ROWS * D * 4, "");
  __shared__ Meta s_meta[kWarps][R::kDeep];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ float s_pm[ROWS], s_pl[ROWS];              // of the block's piece
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int b = blockIdx.x;
  const uint32_t ring = smem_at(s_ring) + warp * kRing;

  int per = 1, stop, unit, at = 0, pos;                 // `at`: the unit's first tile
  bool meets = false;                                   // the cluster's pieces do
  if constexpr (!EVEN) {
    unit = b / g.ranks;
    const int tiles = unit_tiles<KIND>(attend_unit<ROWS>(g, unit)), rank = b % g.ranks;
    pos = (int)((long long)tiles * rank / g.ranks);
    stop = (int)((long long)tiles * (rank + 1) / g.ranks);
    meets = g.ranks > 1 && tiles > 1;
    if (meets && tid < ROWS) {
      s_pm[tid] = -INFINITY;                            // in case this block has no tile
      s_pl[tid] = 0.f;
    }
  } else {
    const AttendShare sh = attend_share<kWarps * 32>(
        g, [&](int i) { return unit_tiles<KIND>(attend_unit<ROWS>(g, i)); });
    grid_dep_trigger();
    if (tid == 0 && !g.splits) g.ws.desc[b] = make_int2(-1, 0);
    if (sh.start >= sh.total) return;
    per = sh.per;
    stop = sh.stop;
    unit = sh.unit;
    at = sh.at;
    pos = sh.start;
  }
  while (pos < stop) {
    const AttendUnit u = attend_unit<ROWS>(g, unit);
    const int tiles = unit_tiles<KIND>(u);
    const int a0 = pos - at, a1 = min(tiles, stop - at);
    if (tiles > 0) {
      State<D, ROWS> st;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[n][e] = 0.f;
#pragma unroll
      for (int e = 0; e < ROWS / 8; ++e) {
        st.m[e] = -INFINITY;
        st.l[e] = 0.f;
      }
      const int ea = min(u.held, u.end), ta = (ea + kTileSlots - 1) / kTileSlots;
      if constexpr (KIND == kImage) {
        constexpr int k = kTileSlots / Shape<kImage, D>::kSlots;
        attend_part<kImage, D, ROWS, R::kDeep, R::kBytes>(g, u, 0, ea, a0 * k + warp,
                                     min(min(a1, ta) * k, (ea + 31) / 32), ring, s_meta[warp], st);
        constexpr int kt = kTileSlots / Shape<kTail, D>::kSlots;
        attend_part<kTail, D, ROWS, R::kDeep, R::kBytes>(
            g, u, ea, u.end, max(a0 - ta, 0) * kt + warp,
            min((a1 - ta) * kt, (u.end - ea + 7) / 8), ring, s_meta[warp], st);
      } else {
        constexpr int k = kTileSlots / Shape<KIND, D>::kSlots, w = Shape<KIND, D>::kSlots;
        attend_part<KIND, D, ROWS, R::kDeep, R::kBytes>(
            g, u, 0, u.end, a0 * k + warp, min(a1 * k, (u.end + w - 1) / w), ring, s_meta[warp],
            st);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
      // the warps' states meet in shared memory; rows g and g + 8 of an 8-row tile are the
      // two terms of the same row
#pragma unroll
      for (int e = 0; e < ROWS / 8; ++e) {
        float l = st.l[e];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (lane % 4 == 0) {
          s_m[warp][lane / 4 + 8 * e] = st.m[e];
          s_l[warp][lane / 4 + 8 * e] = l;
        }
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int f = Shape<KIND, D>::feature(n, 2 * (lane % 4) + y);
          if constexpr (ROWS == 8) {
            s_o[warp][lane / 4][f] = st.o[n][y] + st.o[n][2 + y];
          } else {
            s_o[warp][lane / 4][f] = st.o[n][y];
            s_o[warp][lane / 4 + 8][f] = st.o[n][2 + y];
          }
        }
      __syncthreads();
      const bool whole = a0 == 0 && a1 == tiles;
      const int slot = 2 * b + (a0 == 0 ? 1 : 0);
      for (int i = tid; i < u.rows * D; i += kWarps * 32) {
        const int r = i / D, f = i % D;
        float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float k = s_m[w][r] == -INFINITY ? (s_l[w][r] != s_l[w][r] ? 1.f : 0.f)
                                                 : ex2(s_m[w][r] - m);
          l += k * s_l[w][r];
          o += k * s_o[w][r][f];
        }
        if (whole) {
          finish_row(g, u, r, D, f, m, l, o);
        } else if (!EVEN && meets) {
          s_o[0][r][f] = o;                             // read by this thread alone so far
          if (f == 0) {
            s_pm[r] = m;
            s_pl[r] = l;
          }
        } else {
          if (f == 0) g.ws.stat[slot * kPieceRows + r] = make_float2(m, l);
          g.ws.out[((long long)slot * kPieceRows + r) * D + f] = o;
        }
      }
      __syncthreads();
      // for the join: by unit where it has blocks for each, else by its first block
      if (EVEN && a0 == 0 && tid == 0 && (g.splits || a1 < tiles))
        g.ws.desc[g.splits ? unit : b] =
            make_int2(!g.splits ? unit : a1 < tiles ? b : -1, (at + tiles - 1) / per);
    }
    pos = at + a1;
    at += tiles;
    ++unit;
  }
  if (!EVEN && meets) {
    // the cluster's pieces, in the order of their slots, from the blocks' shared memory
    cluster_sync();
    const AttendUnit u = attend_unit<ROWS>(g, b / g.ranks);
    for (int i = b % g.ranks * (kWarps * 32) + tid; i < u.rows * D; i += g.ranks * kWarps * 32) {
      const int r = i / D, f = i % D;
      float m[kRanks], z[kRanks], x[kRanks], top = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
      for (int p = 0; p < kRanks; ++p) {                // all under way at once
        m[p] = -INFINITY;
        z[p] = x[p] = 0.f;
        if (p >= g.ranks) continue;
        m[p] = remote(&s_pm[r], p);
        z[p] = remote(&s_pl[r], p);
        x[p] = remote(&s_o[0][r][f], p);
      }
#pragma unroll
      for (int p = 0; p < kRanks; ++p) top = fmaxf(top, m[p]);
#pragma unroll
      for (int p = 0; p < kRanks; ++p) {
        if (m[p] == -INFINITY && z[p] == 0.f) continue; // nothing seen, or no tile at all
        const float k = m[p] == -INFINITY ? 1.f : ex2(m[p] - top);
        l += k * z[p];
        o += k * x[p];
      }
      finish_row(g, u, r, D, f, top, l, o);
    }
    cluster_sync();                                     // nobody reads this block any more
  }
}

// Joins the pieces of a unit that starts in a block b and ends in a later one. Few units, each of
// many pieces: `g.splits` blocks a unit, for its rows in turn (8 slices of 32768 rows, 16 query
// rows: attention takes 38.3 us in bf16, 48.9 with a block for each b; 33.3 and 43.1 us from the
// image); else a block for each b.
constexpr int kJoinWarps = 16;
template <int KIND, int D, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(AttendArgs g) {
  constexpr int E = D / 32;
  __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  grid_dep_wait();
  const int splits = max(g.splits, 1), split = blockIdx.x % splits;
  int b = blockIdx.x / splits, unit = b;
  int2 desc = make_int2(-1, 0);
  if (!g.splits) {
    desc = g.ws.desc[b];
    unit = desc.x;
  } else if (unit_tiles<KIND>(attend_unit<ROWS>(g, unit)) > 0) {   // else nobody described it
    desc = g.ws.desc[unit];
    b = desc.x;
  }
  if (desc.x < 0) return;
  const AttendUnit u = attend_unit<ROWS>(g, unit);
  const int mine = (u.rows - split + splits - 1) / splits;         // rows split, split + splits ..
  if (mine <= 0) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int groups = kJoinWarps;                               // warps of a row
  while (groups > 1 && mine * groups > kJoinWarps) groups /= 2;
  const int part = warp % groups, r = split + warp / groups * splits;
  float m = -INFINITY, l = 0.f, o[E] = {};
  if (r < u.rows) {
#pragma unroll 4
    for (int i = b + part; i <= desc.y; i += groups) {
      const int slot = i == b ? 2 * b + 1 : 2 * i;
      const float2 x = g.ws.stat[slot * kPieceRows + r];
      const float* p = g.ws.out + ((long long)slot * kPieceRows + r) * D + lane;
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = p[32 * e];
      const float top = fmaxf(m, x.x), ref = top == -INFINITY ? 0.f : top;
      const float f0 = ex2(m - ref), f1 = x.x == -INFINITY && x.y != x.y ? 1.f : ex2(x.x - ref);
      l = l * f0 + x.y * f1;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f0 + y[e] * f1;
      m = top;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = o[e];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < mine * D; i += kJoinWarps * 32) {
    const int rr = i / D, f = i % D;
    float top = -INFINITY, sum = 0.f, x = 0.f;
    for (int w = rr * groups; w < (rr + 1) * groups; ++w) top = fmaxf(top, s_m[w]);
    for (int w = rr * groups; w < (rr + 1) * groups; ++w) {
      const float k = s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? 1.f : 0.f) : ex2(s_m[w] - top);
      sum += k * s_l[w];
      x += k * s_o[w][f];
    }
    finish_row(g, u, split + rr * splits, D, f, top, sum, x);
  }
}

size_t attend_layout(int D, char* base, AttendWs* ws) {
  size_t at = 0;
  ws->desc = reinterpret_cast<int2*>(base + at);
  at += round256(kAttendGrid * sizeof(int2));
  ws->stat = reinterpret_cast<float2*>(base + at);
  at += round256((size_t)2 * kAttendGrid * kPieceRows * sizeof(float2));
  ws->out = reinterpret_cast<float*>(base + at);
  return at + (size_t)2 * kAttendGrid * kPieceRows * D * sizeof(float);
}

template <int KIND, int D, int ROWS>
cudaError_t launch_attend(AttendArgs& g, cudaStream_t st, int* launches) {
  using R = Ring<KIND, D, ROWS>;
  const long long mtiles = (most_tokens(g.t) * g.c.group + ROWS - 1) / ROWS;
  const long long units = (long long)g.c.seqs * g.c.kv_heads * mtiles;
  constexpr int kTileSlots = kTileOf<KIND>;
  const long long most = units * ((g.c.capacity + kTileSlots - 1) / kTileSlots + 1);
  const long long fit = kSms * R::kPerSm;
  g.mtiles = (int)mtiles;
  g.units = (int)units;
  // A unit is one block's, or a cluster's of 2, 4 or 8 blocks, as many as fit the GPU at once;
  // either way there is one launch and no workspace. That pays up to `few` slots (eight steps
  // per warp, 512 at most) for one block and up to `most_of` for each block of a cluster; beyond
  // that even shares keep more of the GPU busy. On the GPU, one token, 4 query rows, in us, even
  // shares / one block / clusters:
  //   bf16, 8 slices of 128 slots 9.1 / 6.2 / 8.4, of 256 9.3 / 7.5 / 7.7, of 512 9.6 / 9.5 / 7.9,
  //   of 2048 12.7 / 22.9 / 9.5, of 4096 13.2 / 40.2 / 11.7, of 8192 14.9 / - / 16.2; 64 slices of
  //   512 12.0 / 9.7 / 9.6, of 1024 13.6 / 14.2 / 10.9, of 4096 32.6 / 41.4 / 27.0; 80 slices of
  //   512 15.9 / 9.8 / 11.4, of 1024 17.0 / 14.1 / 14.1; 512 slices of 1024 52.8 / 46.5 / -;
  //   image, 8 slices of 512 11.4 / 10.3 / 9.5, 64 of 4096 25.2 / 36.8 / 20.5;
  //   fp32, 8 slices of 512 11.7 / 22.2 / 9.7, of 2048 15.2 / 70.9 / 15.8, of 4096 18.8 / 136 /
  //   24.1; 80 slices of 512 23.0 / 22.5 / 20.7, of 1024 28.7 / 39.3 / 33.4.
  constexpr int eight = 8 * Shape<KIND, D>::kSlots * kWarps, few = eight < 512 ? eight : 512;
  constexpr int most_of = KIND == kF32 ? few : 2 * few;
  int ranks = kRanks;
  while (ranks > 1 && units * ranks > fit) ranks /= 2;
  if (g.c.capacity <= (units * kRanks <= 2 * kSms ? few / 2 : few)) ranks = 1;
  const int limit = ranks > 1 ? ranks * most_of : units >= fit ? 2 * few : few;
  g.ranks = g.c.capacity <= limit ? ranks : 0;
  g.splits = 0;
  if (units * 2 <= kSms)
    for (g.splits = ROWS; g.splits > 1 && units * g.splits > kSms;) g.splits /= 2;
  const int grid = (int)(g.ranks ? units * g.ranks : most < fit ? most : fit);
  constexpr int smem = kWarps * R::kDeep * R::kBytes;
  cudaError_t e;
  if (g.ranks) {
    e = allow_smem<attend_kernel<KIND, D, ROWS, false>>(smem);
    if (e != cudaSuccess) return e;
    e = launch_after_clusters(attend_kernel<KIND, D, ROWS, false>, dim3(grid), dim3(kWarps * 32),
                              smem, g.ranks, st, g);
    if (e == cudaSuccess) note_launch(st, launches, "attend");
    return e;
  }
  e = allow_smem<attend_kernel<KIND, D, ROWS, true>>(smem);
  if (e != cudaSuccess) return e;
  e = launch_after(attend_kernel<KIND, D, ROWS, true>, dim3(grid), dim3(kWarps * 32), smem, st, g);
  if (e != cudaSuccess) return e;
  note_launch(st, launches, "attend");
  e = launch_after(attend_join_kernel<KIND, D, ROWS>,
                   dim3(g.splits ? (unsigned)(units * g.splits) : (unsigned)grid),
                   dim3(kJoinWarps * 32), 0, st, g);
  if (e == cudaSuccess) note_launch(st, launches, "attend_join");
  return e;
}

template <int D>
cudaError_t launch_attend(AttendArgs& g, cudaStream_t st, int* launches) {
  if (g.c.dtype == NX_DTYPE_F32) return launch_attend<kF32, D, 8>(g, st, launches);
  if (attend_tc_takes(g.c, g.t, g.im.k != nullptr)) return launch_attend_tc(g, st, launches);
  const bool few = most_tokens(g.t) * g.c.group <= 8;
  if (g.im.k)
    return few ? launch_attend<kImage, D, 8>(g, st, launches)
               : launch_attend<kImage, D, 16>(g, st, launches);
  return few ? launch_attend<kBf16, D, 8>(g, st, launches)
             : launch_attend<kBf16, D, 16>(g, st, launches);
}

}  // namespace
}  // namespace nx

extern "C" size_t nexus_attend_workspace_bytes(const nx_cache* cache, const nx_tokens* tokens) {
  using namespace nx;
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens)) return 0;
  AttendWs ws;                            // of any cache of this type, with an image or without
  const size_t rows = attend_layout(cache->head_dim, nullptr, &ws);
  const size_t tc = attend_tc_may_take(*cache, *tokens)
                        ? attend_tc_layout(cache->head_dim, nullptr, &ws)
                        : 0;
  return rows > tc ? rows : tc;
}

extern "C" nx_status nexus_attend(const nx_cache* cache, const nx_tokens* tokens,
                                  const nx_image* image, const nx_attend* args, void* ws,
                                  size_t ws_bytes, int32_t* dev_status, nx_stream_t stream) {
  using namespace nx;
  int launches = 0;
  begin_call();
  if (!valid_cache(cache) || !valid_tokens(*cache, tokens) || !args || !dev_status)
    return NX_ERR_INVALID_ARG;
  const nx_cache& c = *cache;
  const nx_attend& a = *args;
  if (image && !valid_image(image)) return NX_ERR_INVALID_ARG;
  if (!aligned4(c.lens, c.block_table, a.lse, dev_status)) return NX_ERR_INVALID_ARG;
  if (image && c.dtype != NX_DTYPE_BF16) return NX_ERR_UNSUPPORTED;
  // tiles (of at least 64 slots, and a partial one) of all units (of at least 8 rows)
  const long long heads = (long long)c.kv_heads * c.group;
  if (heads > (1 << 20) || (long long)c.seqs * c.kv_heads > (1 << 24) ||
      most_tokens(*tokens) * c.group > 0x7FFFFFFFLL - 256 ||       // rows of a slice, by tiles
      (long long)c.seqs * c.kv_heads * (most_tokens(*tokens) * c.group / 8 + 1) >
          0x7FFFFFFFLL / (c.capacity / 64 + 2))
    return NX_ERR_UNSUPPORTED;
  const int size = c.dtype == NX_DTYPE_BF16 ? 2 : 4;
  if (!isfinite(a.scale)) return NX_ERR_INVALID_ARG;
  if (a.q_stride < 0 || a.out_stride < 0 || a.q_stride * size % 16 || a.out_stride * size % 16 ||
      ((uintptr_t)a.q & 15u) || ((uintptr_t)a.out & 15u))
    return NX_ERR_INVALID_ARG;
  if (tokens->tokens > 0 && (!a.q || !a.out)) return NX_ERR_INVALID_ARG;
  if (tokens->tokens > 1 && a.out_stride < heads * c.head_dim)
    return NX_ERR_INVALID_ARG;           // rows of out would overlap
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < nexus_attend_workspace_bytes(cache, tokens))
    return NX_ERR_WORKSPACE;
  if (tokens->tokens == 0) return finish(cudaSuccess, launches);
  AttendArgs g{};
  g.c = c;
  g.t = *tokens;
  if (image) g.im = *image;
  g.a = a;
  g.dev_status = dev_status;
  if (attend_tc_takes(c, *tokens, image != nullptr))
    attend_tc_layout(c.head_dim, static_cast<char*>(ws), &g.ws);
  else attend_layout(c.head_dim, static_cast<char*>(ws), &g.ws);
  g.b = image_block(c);
  while (1 << g.b_shift < g.b) ++g.b_shift;
  g.c1 = a.scale * 1.4426950408889634f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return finish(c.head_dim == 128 ? launch_attend<128>(g, st, &launches)
                                  : launch_attend<64>(g, st, &launches),
                launches);
}
