// cache8_attend.cuh -- attention of a query's new tokens over [retrieved memory
// rows | 8-bit local rows], and the attention weight each cached row received.
//
//   s_j = <Q, k_j> / sqrt(D),  p = softmax over the visible rows,  O = sum p_j v_j
//   weights_j = decay * weights_j + sum over tokens and heads of the group of p_j
//
// A few tokens: the bytes of the cache bound it.  Per (query, kv head, context
// split) CTA, four warps each stream 16-row tiles through a ring of their own
// (asynchronous copies, no barrier between warps) into mma.sync m16n8k16.
// Context rows are the M rows of S^T = K Q^T and the K rows of
// O^T += V^T P^T, the (token, head) columns the N columns, so no MMA row is
// spent on a group's few heads.  The contraction index of an MMA may be
// permuted freely: lane (g, t) = (lane / 4, lane % 4) reads 16-byte pieces t
// and t + 4 of rows g and g + 8 of K, and the 16 bytes 16 g .. of rows 2t,
// 2t+1, 2t+8, 2t+9 of V, and those bytes, widened in place, are its operand
// fragments (Q is laid out by the same permutation; V's bytes of two rows are
// interleaved by byte permutes).
//   Widening: int8 and e4m3 values are exact in fp16, so both MMAs are fp16
// with the block's scale applied outside: K's to the score; V's to P, as its
// ratio 2^r to the largest V scale seen so far (the unit), r <= 0.
// int8 -> fp16 is a byte permute that sets the bits of 1024 + (q + 128) and
// one subtraction.  Q is scaled by a power of two per column to 1 <= max|q| < 2:
// elements below 2^-17 of the largest lose bits, 2^-25 of it at most.
//   P = 2^(s - m + r + 11) in fp16 against a column's reference m, which moves,
// to 7 to 8 above s + r (log2 units), only when that exceeds it by 4: P is at
// most 2^15, weights whose product with the scale is down to 2^-17 of the
// column's largest keep fp16's full 11 bits, smaller ones an error below 2^-28
// of that product.  So m follows what a block adds to O, not its scores alone,
// and when the unit grows m falls by as much, so that O's own unit (m and the
// unit together) stays: a light block of huge values costs the others nothing.
// (With m following the scores, weights behind a block of no weight and 2^24
// times larger values kept 3 bits.)  The sum of the weights 2^(s - m) is fp32
// and takes m's distance from the scores as it is, up to 2^100.
//   Memory rows are bf16 and go through bf16 MMAs; P is split there into a bf16
// head and tail, two MMAs, so it loses nothing either.
//   fp32 queries run the same kernel with Q and P split into an fp16 head and
// tail, two MMAs each: 2^-22 of a weight and 2^-25 of the column's largest element are lost.  fp32
// memory rows have a kernel of their own on CUDA cores.
#pragma once
#include <cuda_fp16.h>

#include <type_traits>

#include "cache8.cuh"
#include "context.cuh"

namespace msa {

constexpr int kC8Warps = 4;
constexpr int kC8Stages = 3;          // tiles of a warp in flight or in use
constexpr float kC8Shift = 11.0f;     // P is 2^11 exp2(s - m)
constexpr float kC8Top = 2048.0f;     // 2^kC8Shift
constexpr float kC8Slack = 4.0f;      // s + r may exceed m by this before m moves,
constexpr float kC8Lead = 7.0f;       // and m then moves this far above the next whole number
constexpr float kC8MinRatio = -96.0f; // r as the references see it: a weight is 2^100 at most
constexpr float kC8MaxSum = 110.0f;   // log2 to which a growing unit may raise a sum of weights
constexpr float kC8None = -3e38f;     // the reference of a column that has seen nothing

struct Attend8Args {
  const void *content;
  const int32_t *ids;
  const int64_t *doc_chunk_off;
  const int32_t *slots;  // a host tier's slot cache: slot of each (query, rank), or null
  int slot_chunks;
  int k, n_docs, table_cap;
  const uint8_t *k8, *v8;
  const float *ks, *vs;
  const int32_t *cache_len, *n_tokens;
  int H_kv, G, T, cap, bl, bl_shift;  // bl = 1 << bl_shift
  uint32_t g_magic;                   // ceil(2^32 / G); 0 for G = 1
  const void *Q;
  float scale_log2;  // log2(e) / sqrt(D)
  // context splits: the first loc_split share the local rows, the other n_split - loc_split the
  // memory rows; with loc_split = n_split each takes a share of both
  int n_split, loc_split;
  void *O;
  float *lse;
  float2 *ml;        // with weights: reference (log2 units) and 1 / sum of every column's softmax
  float *part_o, *part_ml;
  float *scores;     // with weights and few columns: [batch][H_kv][cap][score_w] log2-unit scores
  int score_w;       // 4, 8 or 16
  float *weights;
  float decay;
};

// Token of a (token, head of the group) column: col / G, exact for col < 2^28.
__device__ __forceinline__ int col_token(const Attend8Args &a, int col) {
  return a.g_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(col), a.g_magic)) : col;
}

// Query b's tokens and rows; out-of-range lengths count as no tokens.
struct Attend8Query {
  int len, n;  // rows in the cache, new tokens (the cache's last n rows)
};
__device__ __forceinline__ Attend8Query attend8_query(const Attend8Args &a, int b, bool report) {
  Attend8Query q;
  q.len = a.cache_len[b];
  q.n = a.n_tokens ? a.n_tokens[b] : a.T;
  if (q.n < 0 || q.n > a.T || q.len < 0 || q.len > a.cap) {
    if (report) raise_device_error(MSA_DEVERR_BAD_LENGTH);
    q.len = q.n = 0;
  }
  return q;
}

// D(16x8, f32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bytes (0, 1) and (2, 3) of a word as two fp16 pairs.
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (FMT == MSA_CACHE_INT8) {
    const uint32_t u = w ^ 0x80808080u;  // q + 128
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<__half2 *>(&x), bias);
    const __half2 b = __hsub2(*reinterpret_cast<__half2 *>(&y), bias);
    lo = *reinterpret_cast<const uint32_t *>(&a);
    hi = *reinterpret_cast<const uint32_t *>(&b);
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
        " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ uint4 ld_stream16(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// A tile is 16 rows of K and of V of one head.  Each warp has a ring of its own in shared memory,
// filled by 16-byte asynchronous copies; only the warp itself waits for them.  Within a row the
// 16-byte pieces are permuted so that the fragment reads below hit every bank once (D = 128; at
// D = 64 V's reads are two to a bank).
template <int D>
struct Tile8 {
  static constexpr int kRow = D, kBytes = 16 * D, kStage = 2 * kBytes;
  static __device__ __forceinline__ uint32_t k_off(int row, int piece) {
    return row * D + ((D == 128 ? piece ^ ((row & 1) << 2) : piece) << 4);
  }
  static __device__ __forceinline__ uint32_t v_off(int row, int piece) {
    return row * D + ((D == 128 ? piece ^ (row & 6) : piece ^ ((row >> 1) & 3)) << 4);
  }
  // the warp's copies of the tile whose rows start at k and v
  static __device__ __forceinline__ void issue(uint32_t stage, const uint8_t *k, const uint8_t *v,
                                               int lane) {
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const int i = lane + 32 * u, row = i / (D / 16), piece = i % (D / 16);
      cp_async_16(stage + k_off(row, piece), k + 16 * i, true);
      cp_async_16(stage + kBytes + v_off(row, piece), v + 16 * i, true);
    }
  }
};

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// This lane's bytes of a K tile: words [row g or g + 8][D / 16].
template <int D>
struct KTile {
  uint32_t w[2][D / 16];
  __device__ __forceinline__ void set(int r, int p, uint4 x) {
    w[r][4 * p] = x.x; w[r][4 * p + 1] = x.y; w[r][4 * p + 2] = x.z; w[r][4 * p + 3] = x.w;
  }
  __device__ __forceinline__ void from_shared(uint32_t stage, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int p = 0; p < D / 64; ++p) set(r, p, lds16(stage + Tile8<D>::k_off(g + 8 * r, 4 * p + t)));
  }
  __device__ __forceinline__ void from_global(const uint8_t *tile, int lane) {
    const uint8_t *x = tile + (lane >> 2) * D + 16 * (lane & 3);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int p = 0; p < D / 64; ++p) set(r, p, ld_stream16(x + 8 * r * D + 64 * p));
  }
};

// This lane's bytes of a V tile: words [row 2t, 2t + 1, 2t + 8, 2t + 9][D / 32] from byte (D / 8) g.
template <int D>
struct VTile {
  uint32_t w[4][D / 32];
  __device__ __forceinline__ void from_shared(uint32_t stage, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 2 * t + (r & 1) + 8 * (r >> 1);
      if constexpr (D == 128) {
        const uint4 x = lds16(stage + Tile8<D>::v_off(row, g));
        w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
      } else {
        const uint2 x = lds8(stage + Tile8<D>::v_off(row, g >> 1) + 8 * (g & 1));
        w[r][0] = x.x; w[r][1] = x.y;
      }
    }
  }
  // rows >= lim become zero: a byte behind the last row may be e4m3's NaN, and 0 * NaN is NaN
  __device__ __forceinline__ void clear_from(int lane, int lim) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (2 * (lane & 3) + (r & 1) + 8 * (r >> 1) >= lim) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[r][i] = 0;
      }
  }
};

// Element of a head that lane-column t holds at k step s, byte 0 (4 consecutive ones follow).
__device__ __forceinline__ int k_elem(int s, int t) { return (s >> 2) * 64 + 16 * t + 4 * (s & 3); }

// Shared memory of the attention kernel.
template <int D, int NT>
struct Attend8Smem {
  static constexpr int kCols = 8 * NT;
  static constexpr int kQPitch = D + 8;  // elements of a column's row (16 bytes of padding)
  static constexpr int kQ = 0;                                   // fp16, scaled (its head of fp32)
  static constexpr int kQb = kQ + kCols * kQPitch * 2;           // bf16, as given (fp16 tail of fp32)
  static constexpr int kColScale = kQb + kCols * kQPitch * 2;    // fp32 per column
  static constexpr int kMerge = kColScale + kCols * 4;
  static constexpr int kMergeBytes = kC8Warps * kCols * (D + 4) * 4;  // O, m, l
  static constexpr int kRing = kMerge;                           // the rings, before the merge
  static constexpr int kRingBytes = kC8Warps * kC8Stages * Tile8<D>::kStage;
  static constexpr int kTable = kMerge + (kMergeBytes > kRingBytes ? kMergeBytes : kRingBytes);
  // prefix, bases, chunk table
  static int bytes(int table_cap) { return kTable + (2 * kMaxTopK + 1 + table_cap) * 4; }
};

// The columns [c0, c0 + 8 NT) of Q, one warp a column, scaled by a power of two to 1 <= max < 2 as
// fp16, and that scale times scale_log2.  bf16: the column as given beside it, for the memory rows;
// fp32: what the fp16 value leaves.  Columns past the query's tokens are zero.
template <typename T, int D, int NT>
__device__ __forceinline__ void load_q_columns(const Attend8Args &a, int b, int g, int c0, int n,
                                               uint8_t *sm) {
  using Sm = Attend8Smem<D, NT>;
  __half *qh = reinterpret_cast<__half *>(sm + Sm::kQ), *q2 = reinterpret_cast<__half *>(sm + Sm::kQb);
  float *cs = reinterpret_cast<float *>(sm + Sm::kColScale);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int E = D / 32;
  for (int c = warp; c < Sm::kCols; c += kC8Warps) {
    const int cc = c0 + c, t = col_token(a, cc);
    const int64_t at = ((static_cast<int64_t>(b) * a.T + t) * a.H_kv * a.G + g * a.G + cc - t * a.G) * D + lane * E;
    using Half = std::conditional_t<E == 4, uint2, uint32_t>;  // this lane's elements in 16 bits
    Half raw{};
    float x[E], amax = 0.0f;
    if constexpr (sizeof(T) == 2) {
      if (t < n) raw = *reinterpret_cast<const Half *>(static_cast<const __nv_bfloat16 *>(a.Q) + at);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        x[e] = __uint_as_float(w[e / 2] << 16);
        x[e + 1] = __uint_as_float(w[e / 2] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = t < n ? static_cast<const float *>(a.Q)[at + e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) amax = fmaxf(amax, finite_abs(x[e]));
    amax = warp_max(amax);
    // 2^ex <= amax < 2^(ex + 1), within [-126, 126] so that 2^-ex is a normal number too
    const int ex = amax == 0.0f ? 0 : max(1, min(253, __float_as_int(amax) >> 23)) - 127;
    const float inv = __int_as_float((127 - ex) << 23);
    uint32_t h[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) h[e / 2] = pack_f16x2(x[e] * inv, x[e + 1] * inv);
    if constexpr (sizeof(T) == 4) {
      uint32_t *w = reinterpret_cast<uint32_t *>(&raw);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[e / 2]));
        w[e / 2] = pack_f16x2(x[e] * inv - y.x, x[e + 1] * inv - y.y);
      }
    }
    *reinterpret_cast<Half *>(qh + c * Sm::kQPitch + lane * E) = *reinterpret_cast<Half *>(h);
    *reinterpret_cast<Half *>(q2 + c * Sm::kQPitch + lane * E) = raw;
    if (lane == 0) cs[c] = a.scale_log2 * __int_as_float((127 + ex) << 23);
  }
}

// 2^x of a whole number x in [-127, 127], 0 for -127: x + 127 in the low bits of the sum.
__device__ __forceinline__ float pow2_whole(float x) {
  return __int_as_float(__float_as_int(x + (12582912.0f + 127.0f)) << 23);
}
// Exponent of a non-negative number (0: -127).
__device__ __forceinline__ float exponent_of(float x) {
  return static_cast<float>((__float_as_int(x) >> 23) - 127);
}
// r of a block of this V scale: log2 of the scale over the unit, as the references see it.
__device__ __forceinline__ float scale_ratio(float scale, float unit) {
  return scale > 0.0f ? fmaxf(exponent_of(scale) - exponent_of(unit), kC8MinRatio) : kC8MinRatio;
}
// A reference 7 to 8 above the largest s + r.  Scores whose rounding swallows such sums: the score
// itself (P is then 2^(r + 11) there).
__device__ __forceinline__ float new_reference(float top, float r) {
  return fabsf(top) < 8388608.0f ? ceilf(top) + (r + kC8Lead) : top;
}
// The unit grows by 2^up: how far the reference of a column with the sum l falls with it; the rest is
// O's to lose.  (m is a whole number; where it is too large to fall, and before anything was seen, 0.)
__device__ __forceinline__ float reference_falls(float m, float l, float up) {
  const float k = fmaxf(fminf(fminf(up, kC8MaxSum - exponent_of(l)), 127.0f), 0.0f);
  return m - (m - k) == k ? k : 0.0f;
}

// The running softmax of 8 NT columns over tiles of 16 context rows: lane (g, t) holds rows
// g, g + 8 and columns 8 nt + 2t, + 1 of S^T.
template <int D, int NT>
struct Softmax8 {
  float m[NT][2], l[NT][2];
  float acc[NT][D / 16][4];  // O^T, [d pair][col pair], in units of `unit`
  float unit, inv_unit;  // a power of two and its reciprocal, the same in every lane (0: no V but zeros yet)

  __device__ __forceinline__ void init() {
    unit = inv_unit = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kC8None;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.0f;
    }
  }
  // The unit becomes at least v: references fall and sums grow, O stays as it is (see above).
  __device__ __forceinline__ void raise_unit(float v) {
    if (v <= unit) return;
    const float up = exponent_of(v) - exponent_of(unit);
    const bool first = unit == 0.0f;  // (O is 0, in any unit)
    unit = v;
    inv_unit = 1.0f / v;
    if (!first) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float k = reference_falls(m[nt][h], l[nt][h], up), f = pow2_whole(fmaxf(k - up, -127.0f));
          m[nt][h] -= k;
          l[nt][h] *= pow2_whole(k);
          if (k != up) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              acc[nt][i][h] *= f;
              acc[nt][i][2 + h] *= f;
            }
          }
        }
    }
  }
  // s (log2 units, -inf where hidden) of rows whose V scale is 2^r units -> p = 2^(s - m), the sums
  // and, where s + r passes its column's reference by more than the slack, new references.  The
  // difference comes first and is compared itself: of scores so large that a unit is below their
  // rounding, s - (m - c) and s > m + c would be off by that rounding, and p could leave fp16.  (For
  // the same reason a score's product is rounded by itself, never fused with what is subtracted.)
  __device__ __forceinline__ void step(float (&s)[NT][4], float r) {
    const float lim = kC8Slack - r;
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) over = over || s[nt][e] - m[nt][e & 1] > lim;
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = fmaxf(s[nt][h], s[nt][2 + h]);
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          const float mn = v - m[nt][h] > lim ? new_reference(v, r) : m[nt][h];
          const float f = mn == m[nt][h] ? 1.0f : ex2_approx(m[nt][h] - mn);
          m[nt][h] = mn;
          l[nt][h] *= f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[nt][i][h] *= f;
            acc[nt][i][2 + h] *= f;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[nt][h] = ex2_approx(s[nt][h] - m[nt][h]);
        s[nt][2 + h] = ex2_approx(s[nt][2 + h] - m[nt][h]);
        l[nt][h] += s[nt][h] + s[nt][2 + h];
      }
  }
};

// Start of part i of n tiles cut into `parts`.
__device__ __forceinline__ int share(int n, int i, int parts) {
  return static_cast<int>(static_cast<int64_t>(n) * i / parts);
}

// Rows a column sees: row of its token plus one.
__device__ __forceinline__ int column_rows(const Attend8Args &a, const Attend8Query &q, int col) {
  const int t = col_token(a, col);
  return t < q.n ? q.len - q.n + t + 1 : 0;
}

// A column's log-sum, and for the weights its reference and the reciprocal of its sum (a column that
// sees nothing: an infinite reference, so that every weight is 0).
__device__ __forceinline__ void write_stats(const Attend8Args &a, int64_t row, float M, float L) {
  if (a.lse) a.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) / kLog2e;
  if (a.ml) a.ml[row] = L == 0.0f ? make_float2(INFINITY, 0.0f) : make_float2(M, 1.0f / L);
}

// The CTA's warps (rows of `merge`: [warp][col][D outputs, m, l]) into O and lse, or into the
// split's partial result.
template <typename T, int D, int COLS>
__device__ __forceinline__ void merge_warps(const Attend8Args &a, const Attend8Query &q, int b,
                                            int g, int c0, int split, const float *merge) {
  const int cols = min(COLS, q.n * a.G - c0);
  for (int i = threadIdx.x; i < cols * D; i += 32 * kC8Warps) {
    const int c = i / D, d = i % D, cc = c0 + c, t = col_token(a, cc);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kC8Warps; ++w) M = fmaxf(M, merge[(w * COLS + c) * (D + 4) + D]);
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f, o = 0.0f;
#pragma unroll
    for (int w = 0; w < kC8Warps; ++w) {
      const float *row = merge + (w * COLS + c) * (D + 4);
      const float f = ex2_approx(row[D] - base);
      L += row[D + 1] * f;
      o += row[d] * f;
    }
    const int64_t row = (static_cast<int64_t>(b) * a.T + t) * a.H_kv * a.G + g * a.G + cc - t * a.G;
    if (a.n_split == 1) {
      static_cast<T *>(a.O)[row * D + d] = Elem<T>::from_f(L == 0.0f ? 0.0f : o / L);
      if (d == 0) write_stats(a, row, M, L);
    } else {
      a.part_o[(row * a.n_split + split) * D + d] = o;
      if (d == 0) {
        a.part_ml[(row * a.n_split + split) * 2] = M;
        a.part_ml[(row * a.n_split + split) * 2 + 1] = L;
      }
    }
  }
}

// grid (B * H_kv, splits, column tiles), block 32 * kC8Warps.  fp32: the local splits alone.
template <typename T, int D, int NT, int FMT>
__global__ void __launch_bounds__(32 * kC8Warps, (sizeof(T) == 4 ? 2 : 1) * NT == 1 ? 4 : (sizeof(T) == 4 ? 2 : 1) * NT == 2 ? 3 : 2)
cache8_attend_kernel(Attend8Args a) {
  constexpr bool F32 = sizeof(T) == 4;
  using Sm = Attend8Smem<D, NT>;
  constexpr int KS = D / 16;  // k steps of S^T
  constexpr bool kQRegs = NT <= 2;  // Q's fragments stay in registers
  extern __shared__ __align__(16) uint8_t sm[];
  const int b = blockIdx.x / a.H_kv, g = blockIdx.x % a.H_kv, split = blockIdx.y;
  const int c0 = blockIdx.z * Sm::kCols;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, lg = lane >> 2, lt = lane & 3;
  griddep_wait();
  griddep_launch();
  const Attend8Query q = attend8_query(a, b, blockIdx.x % a.H_kv == 0 && split == 0 && c0 == 0 &&
                                                 threadIdx.x == 0);
  if (col_token(a, c0) >= q.n) return;  // padding tokens only (the whole CTA)
  const int last_col = min(c0 + Sm::kCols, q.n * a.G) - 1;
  const int n_loc = max(0, column_rows(a, q, last_col));  // rows any column sees
  const int all_see = column_rows(a, q, c0);              // rows every real column sees
  const bool own_mem = a.loc_split < a.n_split;  // memory rows have splits of their own
  const int nl = (n_loc + 15) / 16;
  const int l0 = split < a.loc_split ? share(nl, split, a.loc_split) : 0;
  const int l1 = split < a.loc_split ? share(nl, split + 1, a.loc_split) : 0;
  const int64_t bh = static_cast<int64_t>(b) * a.H_kv + g;
  const float *ks = a.ks + bh * (a.cap >> a.bl_shift), *vs = a.vs + bh * (a.cap >> a.bl_shift);

  // the first tiles are in flight while Q and the chunk table are set up
  int tile = l0 + warp, ahead = tile;  // the tile in use, the next one to fetch
  const uint8_t *kp = a.k8 + (bh * a.cap + tile * 16) * D, *vp = a.v8 + (bh * a.cap + tile * 16) * D;
  const uint32_t ring = smem_u32(sm + Sm::kRing) + warp * kC8Stages * Tile8<D>::kStage;
  auto fetch = [&](uint32_t stage) {
    if (ahead < l1) Tile8<D>::issue(stage, kp, vp, lane);
    cp_async_commit();  // an empty group too: the count of groups is the count of tiles
    ahead += kC8Warps;
    kp += kC8Warps * 16 * D;
    vp += kC8Warps * 16 * D;
  };
#pragma unroll
  for (int i = 0; i < kC8Stages - 1; ++i) fetch(ring + i * Tile8<D>::kStage);
  float ksc = 0.0f, vsc = 0.0f;
  if (tile < l1) {
    ksc = ks[(tile * 16) >> a.bl_shift];
    vsc = vs[(tile * 16) >> a.bl_shift];
  }
  load_q_columns<T, D, NT>(a, b, g, c0, q.n, sm);
  int *pre = reinterpret_cast<int *>(sm + Sm::kTable), *base = pre + kMaxTopK + 1;
  int *table = base + kMaxTopK;
  int n_mem = 0;
  if (!F32 && a.k > 0 && (!own_mem || split >= a.loc_split))
    n_mem = build_chunk_table(a.ids + static_cast<int64_t>(b) * a.k, a.k, a.doc_chunk_off, a.n_docs,
                              a.slots ? a.slots + static_cast<int64_t>(b) * a.k : nullptr, a.slot_chunks, table, pre, base, a.table_cap);
  __syncthreads();

  const __half *qh = reinterpret_cast<const __half *>(sm + Sm::kQ);
  const float *cs = reinterpret_cast<const float *>(sm + Sm::kColScale);
  const __half *ql = reinterpret_cast<const __half *>(sm + Sm::kQb);  // fp32: the tails
  uint32_t qf[kQRegs ? NT : 1][KS][2];
  if constexpr (kQRegs) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint2 x = *reinterpret_cast<const uint2 *>(qh + (8 * nt + lg) * Sm::kQPitch + k_elem(s, lt));
        qf[nt][s][0] = x.x;
        qf[nt][s][1] = x.y;
      }
  }
  float colf[NT][2];  // score factor of this lane's columns
  int rows[NT][2];    // rows they see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      colf[nt][h] = cs[8 * nt + 2 * lt + h];
      rows[nt][h] = column_rows(a, q, c0 + 8 * nt + 2 * lt + h);
    }
  Softmax8<D, NT> st;
  st.init();

  // ---- local rows
  int stage = 0;
  float scale = -1.0f, r = 0.0f, ratio = 0.0f;  // V's scale, log2 of it over the unit, P's factor
  for (; tile < l1; tile += kC8Warps) {
    const int next = tile + kC8Warps;
    cp_async_wait<kC8Stages - 2>();
    __syncwarp();  // every lane's copies of this tile are there; the last tile's stage is free
    const uint32_t at = ring + stage * Tile8<D>::kStage;
    fetch(ring + (stage == 0 ? kC8Stages - 1 : stage - 1) * Tile8<D>::kStage);
    stage = stage == kC8Stages - 1 ? 0 : stage + 1;
    KTile<D> kt;
    kt.from_shared(at, lane);
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      uint32_t a0, a1, a2, a3;
      widen4<FMT>(kt.w[0][i], a0, a2);
      widen4<FMT>(kt.w[1][i], a1, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (kQRegs) {
          mma_f16_16816(s[nt], a0, a1, a2, a3, qf[nt][i][0], qf[nt][i][1]);
        } else {
          const uint2 x = *reinterpret_cast<const uint2 *>(qh + (8 * nt + lg) * Sm::kQPitch + k_elem(i, lt));
          mma_f16_16816(s[nt], a0, a1, a2, a3, x.x, x.y);
        }
        if constexpr (F32) {
          const uint2 x = *reinterpret_cast<const uint2 *>(ql + (8 * nt + lg) * Sm::kQPitch + k_elem(i, lt));
          mma_f16_16816(s[nt], a0, a1, a2, a3, x.x, x.y);
        }
      }
    }
    const float k_scale = ksc, v_scale = vsc;
    if (next < l1) {
      ksc = ks[(next * 16) >> a.bl_shift];
      vsc = vs[(next * 16) >> a.bl_shift];
    }
    const int x0 = tile * 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = __fmul_rn(s[nt][e], colf[nt][e & 1] * k_scale);
    if (x0 + 16 > all_see) {  // rows that some column does not see
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x0 + lg + 8 * (e >> 1) >= rows[nt][e & 1]) s[nt][e] = -INFINITY;
    }
    if (NT <= 2 && a.scores) {
      float *out = a.scores + (bh * a.cap + x0 + lg) * a.score_w + 2 * lt;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (NT == 2 || 2 * lt < a.score_w) {
          *reinterpret_cast<float2 *>(out + 8 * nt) = make_float2(s[nt][0], s[nt][1]);
          *reinterpret_cast<float2 *>(out + 8 * a.score_w + 8 * nt) = make_float2(s[nt][2], s[nt][3]);
        }
    }
    if (v_scale != scale) {  // (neighbouring tiles mostly share one)
      scale = v_scale;
      st.raise_unit(scale);
      r = scale_ratio(scale, st.unit);
      ratio = scale * st.inv_unit * kC8Top;
    }
    st.step(s, r);
    uint32_t pb[NT][2], pt[F32 ? NT : 1][2];  // P, and of fp32 its tail
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = s[nt][2 * r] * ratio, p1 = s[nt][2 * r + 1] * ratio;
        const uint32_t head = pack_f16x2(p0, p1);
        pb[nt][r] = movmatrix_trans(head);
        if constexpr (F32) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&head));
          pt[nt][r] = movmatrix_trans(pack_f16x2(p0 - y.x, p1 - y.y));
        }
      }
    VTile<D> vt;
    vt.from_shared(at + Tile8<D>::kBytes, lane);
    if (FMT == MSA_CACHE_E4M3 && x0 + 16 > n_loc) vt.clear_from(lane, n_loc - x0);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      // words w of four rows: elements (D / 8) g + 4 w .. + 3, two M tiles
      uint32_t lo[2][2], hi[2][2];  // [row pair][element pair of the word]
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t e01 = __byte_perm(vt.w[2 * r][w], vt.w[2 * r + 1][w], 0x5140);
        const uint32_t e23 = __byte_perm(vt.w[2 * r][w], vt.w[2 * r + 1][w], 0x7362);
        widen4<FMT>(e01, lo[r][0], hi[r][0]);
        widen4<FMT>(e23, lo[r][1], hi[r][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16_16816(st.acc[nt][2 * w + i], lo[0][i], hi[0][i], lo[1][i], hi[1][i], pb[nt][0],
                        pb[nt][1]);
          if constexpr (F32)
            mma_f16_16816(st.acc[nt][2 * w + i], lo[0][i], hi[0][i], lo[1][i], hi[1][i], pt[nt][0],
                          pt[nt][1]);
        }
    }
  }

  // ---- memory rows: every column sees them (fp32 ones have a kernel of their own)
  if constexpr (!F32) {
  const int nm = (n_mem + 15) / 16;
  const int ms = own_mem ? split - a.loc_split : split, mn = own_mem ? a.n_split - a.loc_split : a.n_split;
  const int m1 = share(nm, ms + 1, mn);
  const __nv_bfloat16 *qb = reinterpret_cast<const __nv_bfloat16 *>(sm + Sm::kQb);
  const int64_t kv = static_cast<int64_t>(a.H_kv) * D;
  const bool any_mem = share(nm, ms, mn) + warp < m1;
  if (any_mem) st.raise_unit(1.0f);  // (V as it is)
  const float to_unit = st.inv_unit * kC8Top, mem_ratio = scale_ratio(1.0f, st.unit);
  for (int mt = share(nm, ms, mn) + warp; mt < m1; mt += kC8Warps) {
    const int x0 = mt * 16;
    auto row_ptr = [&](int x) {
      return static_cast<const __nv_bfloat16 *>(a.content) +
             static_cast<int64_t>(table[min(x, n_mem - 1)]) * 2 * kv + g * D;
    };
    const __nv_bfloat16 *k0 = row_ptr(x0 + lg), *k1 = row_ptr(x0 + lg + 8);
    const __nv_bfloat16 *v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = row_ptr(x0 + 2 * lt + (r & 1) + 8 * (r >> 1)) + kv + (D / 8) * lg;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < KS; i += 2) {  // two k steps: 8 elements of a row
      const uint4 x0v = *reinterpret_cast<const uint4 *>(k0 + k_elem(i, lt));
      const uint4 x1v = *reinterpret_cast<const uint4 *>(k1 + k_elem(i, lt));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const __nv_bfloat16 *qr = qb + (8 * nt + lg) * Sm::kQPitch;
        const uint2 b0 = *reinterpret_cast<const uint2 *>(qr + k_elem(i, lt));
        const uint2 b1 = *reinterpret_cast<const uint2 *>(qr + k_elem(i + 1, lt));
        mma_bf16_16816(s[nt], x0v.x, x1v.x, x0v.y, x1v.y, b0.x, b0.y);
        mma_bf16_16816(s[nt], x0v.z, x1v.z, x0v.w, x1v.w, b1.x, b1.y);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[nt][e] = x0 + lg + 8 * (e >> 1) < n_mem ? __fmul_rn(s[nt][e], a.scale_log2) : -INFINITY;
      }
    st.step(s, mem_ratio);
    uint32_t pb[NT][2][2];  // [part][row half]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = s[nt][2 * r] * to_unit, p1 = s[nt][2 * r + 1] * to_unit;
        const uint32_t head = pack_bf16x2(p0, p1);
        pb[nt][0][r] = movmatrix_trans(head);
        pb[nt][1][r] = movmatrix_trans(pack_bf16x2(p0 - __uint_as_float(head << 16),
                                                   p1 - __uint_as_float(head & 0xffff0000u)));
      }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {  // 8 elements of four rows: four M tiles
      uint32_t x[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint4 y = *reinterpret_cast<const uint4 *>(v[r] + 8 * c);
        x[r][0] = y.x; x[r][1] = y.y; x[r][2] = y.z; x[r][3] = y.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = __byte_perm(x[0][i], x[1][i], 0x5410), a1 = __byte_perm(x[0][i], x[1][i], 0x7632);
        const uint32_t a2 = __byte_perm(x[2][i], x[3][i], 0x5410), a3 = __byte_perm(x[2][i], x[3][i], 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16_16816(st.acc[nt][4 * c + i], a0, a1, a2, a3, pb[nt][0][0], pb[nt][0][1]);
          mma_bf16_16816(st.acc[nt][4 * c + i], a0, a1, a2, a3, pb[nt][1][0], pb[nt][1][1]);
        }
      }
    }
  }
  }

  // ---- the warps meet
  cp_async_wait<0>();
  __syncthreads();  // every warp is done with its ring
  float *merge = reinterpret_cast<float *>(sm + Sm::kMerge);
  const float out = st.unit / kC8Top;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float L = st.l[nt][h];
      L += __shfl_xor_sync(0xffffffffu, L, 4);
      L += __shfl_xor_sync(0xffffffffu, L, 8);
      L += __shfl_xor_sync(0xffffffffu, L, 16);
      float *row = merge + (warp * Sm::kCols + 8 * nt + 2 * lt + h) * (D + 4);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        row[(D / 8) * lg + 2 * i] = st.acc[nt][i][h] * out;
        row[(D / 8) * lg + 2 * i + 1] = st.acc[nt][i][2 + h] * out;
      }
      if (lg == 0) {
        row[D] = st.m[nt][h] == kC8None ? -INFINITY : st.m[nt][h];
        row[D + 1] = L;
      }
    }
  __syncthreads();
  merge_warps<T, D, Sm::kCols>(a, q, b, g, c0, split, merge);
}

// ---------------------------------------------------------------- fp32 memory rows
// CUDA cores, four columns a CTA: scores with a lane on each of 32 rows, outputs with a lane on
// D / 32 elements; sums in fp32.  grid (B * H_kv, memory splits, ceil(columns / 4)).
constexpr int kC8Cols32 = 4;
template <int D>
struct Memory8Smem {
  static constexpr int kQ = 0;
  static constexpr int kMerge = kQ + kC8Cols32 * D * 4;
  static constexpr int kTable = kMerge + kC8Warps * kC8Cols32 * (D + 4) * 4;
  static int bytes(int table_cap) { return kTable + (2 * kMaxTopK + 1 + table_cap) * 4; }
};

template <int D>
__global__ void __launch_bounds__(32 * kC8Warps)
cache8_memory_f32_kernel(Attend8Args a) {
  using Sm = Memory8Smem<D>;
  constexpr int C = kC8Cols32, E = D / 32;
  extern __shared__ __align__(16) uint8_t sm[];
  const int b = blockIdx.x / a.H_kv, g = blockIdx.x % a.H_kv;
  const int c0 = blockIdx.z * C;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  griddep_wait();
  griddep_launch();
  const Attend8Query q = attend8_query(a, b, false);
  if (col_token(a, c0) >= q.n) return;
  float *qs = reinterpret_cast<float *>(sm + Sm::kQ);
  for (int i = threadIdx.x; i < C * D; i += 32 * kC8Warps) {
    const int cc = c0 + i / D, t = col_token(a, cc);
    qs[i] = t < q.n ? static_cast<const float *>(a.Q)[((static_cast<int64_t>(b) * a.T + t) * a.H_kv * a.G +
                                                       g * a.G + cc - t * a.G) * D + i % D] * a.scale_log2
                    : 0.0f;
  }
  int *pre = reinterpret_cast<int *>(sm + Sm::kTable), *base = pre + kMaxTopK + 1;
  int *table = base + kMaxTopK;
  const int n_mem = build_chunk_table(a.ids + static_cast<int64_t>(b) * a.k, a.k, a.doc_chunk_off, a.n_docs,
                                      a.slots ? a.slots + static_cast<int64_t>(b) * a.k : nullptr,
                                      a.slot_chunks, table, pre, base, a.table_cap);
  __syncthreads();
  const int64_t kv = static_cast<int64_t>(a.H_kv) * D;
  float m[C], l[C], acc[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    m[c] = -INFINITY;
    l[c] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[c][e] = 0.0f;
  }
  const int nm = (n_mem + 31) / 32, own = a.n_split - a.loc_split, part = blockIdx.y;
  const int i1 = share(nm, part + 1, own);
  for (int i = share(nm, part, own) + warp; i < i1; i += kC8Warps) {
    const int x0 = i * 32, x = x0 + lane;
    float s[C];
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = 0.0f;
    if (x < n_mem) {
      const float *kr = static_cast<const float *>(a.content) + static_cast<int64_t>(table[x]) * 2 * kv + g * D;
#pragma unroll 4
      for (int p = 0; p < D / 4; ++p) {
        const float4 k = *reinterpret_cast<const float4 *>(kr + 4 * p);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float4 y = *reinterpret_cast<const float4 *>(qs + c * D + 4 * p);
          s[c] = fmaf(y.x, k.x, fmaf(y.y, k.y, fmaf(y.z, k.z, fmaf(y.w, k.w, s[c]))));
        }
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (x >= n_mem) s[c] = -INFINITY;
      const float mn = fmaxf(m[c], warp_max(s[c]));
      const float ref = mn == -INFINITY ? 0.0f : mn;
      const float f = mn == -INFINITY ? 1.0f : exp2f(m[c] - mn);
      m[c] = mn;
      s[c] = exp2f(s[c] - ref);
      l[c] = l[c] * f + s[c];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[c][e] *= f;
    }
    // eight rows of V in flight; rows past the last one have weight 0 and read the last one
    const int last = n_mem - 1 - x0;
    for (int r0 = 0; r0 <= min(31, last); r0 += 8) {
      float v[8][E];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float *vr = static_cast<const float *>(a.content) +
                          static_cast<int64_t>(table[x0 + min(r0 + u, last)]) * 2 * kv + kv + g * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = vr[e];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float p = __shfl_sync(0xffffffffu, s[c], r0 + u);
          if (r0 + u > last) p = 0.0f;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[c][e] = fmaf(p, v[u][e], acc[c][e]);
        }
    }
  }
  float *merge = reinterpret_cast<float *>(sm + Sm::kMerge);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float *row = merge + (warp * C + c) * (D + 4);
    const float L = warp_sum(l[c]);
#pragma unroll
    for (int e = 0; e < E; ++e) row[E * lane + e] = acc[c][e];
    if (lane == 0) {
      row[D] = m[c];
      row[D + 1] = L;
    }
  }
  __syncthreads();
  merge_warps<float, D, C>(a, q, b, g, c0, a.loc_split + part, merge);
}

// ---------------------------------------------------------------- combine
// Merge the context splits (at most kC8MaxSplit) of a row of O (token, head): W warps a row, each a
// W-th of its splits, a lane D / 32 elements.  One warp sums many splits in rounds of eight loads, a
// latency each; four overlap them (the whole call, 4 warps against 1: one query of 8 splits 7.9
// against 8.9 us, 4 tokens over 32,768 rows in 27 splits 26.3 against 28.3; 5 splits of 2,048 rows
// of O the same).
// grid ceil(rows * W / 4), block 128.
constexpr int kC8MaxSplit = 128;
template <typename T, int D, int W>
__global__ void __launch_bounds__(128)
cache8_combine_kernel(Attend8Args a, int rows) {
  constexpr int E = D / 32;
  using Vec = std::conditional_t<E == 4, float4, float2>;
  __shared__ Vec parts[W == 1 ? 1 : W - 1][32];
  griddep_wait();
  griddep_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row = W == 1 ? blockIdx.x * 4 + warp : blockIdx.x, w = W == 1 ? 0 : warp;
  if (row >= rows) return;
  const int H_q = a.H_kv * a.G;
  const int b = row / H_q / a.T, t = row / H_q % a.T;
  const Attend8Query q = attend8_query(a, b, false);
  if (t >= q.n) return;  // (W == 4: the whole block)
  const int n = a.n_split;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + static_cast<int64_t>(row) * n;
  const float *part = a.part_o + static_cast<int64_t>(row) * n * D + lane * E;
  float2 x[kC8MaxSplit / 32];
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kC8MaxSplit / 32; ++i) {
    x[i] = lane + 32 * i < n ? ml[lane + 32 * i] : make_float2(-INFINITY, 0.0f);
    M = fmaxf(M, x[i].x);
  }
  M = warp_max(M);
  const float base = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  __align__(16) float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < kC8MaxSplit / 32; ++i) {
    if (32 * i >= n) break;
    const float f = exp2f(x[i].x - base);
    L += x[i].y * f;
    const int m = min(32, n - 32 * i);
#pragma unroll 8
    for (int s = w; s < m; s += W) {
      const float fs = __shfl_sync(0xffffffffu, f, s);
      const Vec y = *reinterpret_cast<const Vec *>(part + static_cast<int64_t>(32 * i + s) * D);
      const float *v = reinterpret_cast<const float *>(&y);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(v[e], fs, o[e]);
    }
  }
  if constexpr (W > 1) {
    if (w > 0) parts[w - 1][lane] = *reinterpret_cast<const Vec *>(o);
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int u = 0; u < W - 1; ++u) {
      const Vec y = parts[u][lane];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += reinterpret_cast<const float *>(&y)[e];
    }
  }
  L = warp_sum(L);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = L == 0.0f ? 0.0f : o[e] / L;
  T *out = static_cast<T *>(a.O) + static_cast<int64_t>(row) * D + lane * E;
  if constexpr (E == 4) {
    store4(out, o);
  } else {
    out[0] = Elem<T>::from_f(o[0]);
    out[1] = Elem<T>::from_f(o[1]);
  }
  if (lane == 0) write_stats(a, row, M, L);
}

// ---------------------------------------------------------------- weights
// The weight each cached row received, p = 2^(s - m) / L summed over the columns, once the
// softmax's reference m and sum L are known.
//   Up to 16 columns: the attention left the scores behind, 16, 32 or 64 bytes a row, and a thread a
// row adds its weights up.  With the attention, against K read a second time: 64 queries of up to
// 8,192 rows, 4 columns, 153 against 193 us; 16 columns of 2 x 32,768 rows 52 against 56 (e4m3) or 53
// against 60 (int8), of 16 x 4,096 rows 59 against 71.  grid (ceil(cap / 256), B * H_kv), block 256.
template <int W>
__global__ void __launch_bounds__(256)
cache8_weight_scores_kernel(Attend8Args a) {
  __shared__ float2 stats[W];
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.y / a.H_kv, g = blockIdx.y % a.H_kv;
  const Attend8Query q = attend8_query(a, b, false);
  if (static_cast<int>(blockIdx.x) * 256 >= q.len) return;
  const int cols = q.n * a.G;
  if (threadIdx.x < W) {
    const int c = threadIdx.x, t = col_token(a, c);
    stats[c] = c < cols ? a.ml[(static_cast<int64_t>(b) * a.T + t) * a.H_kv * a.G + g * a.G + c - t * a.G]
                        : make_float2(INFINITY, 0.0f);
  }
  __syncthreads();
  const int x = blockIdx.x * 256 + threadIdx.x;
  if (x >= q.len) return;
  const int64_t row = (static_cast<int64_t>(b) * a.H_kv + g) * a.cap + x;
  float sum = 0.0f;
  if (cols > 0) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const float4 s = *reinterpret_cast<const float4 *>(a.scores + row * W + i);
      const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < cols) sum = fmaf(ex2_approx(v[e] - stats[i + e].x), stats[i + e].y, sum);
    }
  }
  float *w = a.weights + row;
  *w = a.decay == 0.0f ? sum : a.decay * *w + sum;
}

//   More columns: a second pass over K alone recomputes the scores, 8 NT columns at a time with Q's
// fragments in registers.  One round of 8 NT: bound by K's bytes; a warp streams its tiles through a
// ring.  More: a CTA copies kC8wRows rows to shared memory once and walks over all columns, its
// tiles' sums in registers.
// grid (CTAs a head, B * H_kv), block 32 * kC8Warps.
constexpr int kC8wTiles = 4;                              // 16-row tiles a warp, or its ring
constexpr int kC8wRows = 16 * kC8wTiles * kC8Warps;
template <int D, int NT>
struct Weight8Smem {
  static constexpr int kK = Attend8Smem<D, NT>::kMerge;   // behind Q and its scales
  static constexpr int kStats = kK + kC8wRows * D;
  static constexpr int kBytes = kStats + 8 * NT * 8;
};

// Columns [c0, c0 + 8 NT) as a lane holds them, and the weights they give a tile's rows.
template <typename T, int D, int NT, int FMT>
struct WeightColumns {
  static constexpr int KS = D / 16;
  uint32_t qf[NT][KS][2];
  float cf[NT][2];
  float2 ml[NT][2];
  int rows[NT][2], all_see;
  const __half *tail;  // fp32: Q's tails, in shared memory

  // Q, its scales and the softmaxes' statistics to shared memory and from there to registers (all
  // warps)
  __device__ __forceinline__ void load(const Attend8Args &a, const Attend8Query &q, int b, int g,
                                       int c0, uint8_t *sm, float2 *stats) {
    using Sm = Attend8Smem<D, NT>;
    const int lane = threadIdx.x % 32, lg = lane >> 2, lt = lane & 3;
    load_q_columns<T, D, NT>(a, b, g, c0, q.n, sm);
    for (int c = threadIdx.x; c < Sm::kCols; c += 32 * kC8Warps) {
      const int cc = c0 + c, t = col_token(a, cc);
      stats[c] = t < q.n ? a.ml[(static_cast<int64_t>(b) * a.T + t) * a.H_kv * a.G + g * a.G + cc - t * a.G]
                         : make_float2(INFINITY, 0.0f);  // no token: weight 0
    }
    __syncthreads();
    const __half *qh = reinterpret_cast<const __half *>(sm + Sm::kQ);
    const float *cs = reinterpret_cast<const float *>(sm + Sm::kColScale);
    all_see = column_rows(a, q, c0);
    tail = reinterpret_cast<const __half *>(sm + Sm::kQb) + lg * Sm::kQPitch;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const uint2 x = *reinterpret_cast<const uint2 *>(qh + (8 * nt + lg) * Sm::kQPitch + k_elem(i, lt));
        qf[nt][i][0] = x.x;
        qf[nt][i][1] = x.y;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 8 * nt + 2 * lt + h;
        cf[nt][h] = cs[c];
        ml[nt][h] = stats[c];
        rows[nt][h] = column_rows(a, q, c0 + c);
      }
    }
  }
  // this lane's part of the weights of rows x0 + g and x0 + g + 8
  __device__ __forceinline__ void add(uint32_t stage, int x0, float k_scale, float (&sum)[2]) const {
    const int lane = threadIdx.x % 32, lg = lane >> 2;
    KTile<D> kt;
    kt.from_shared(stage, lane);
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a0, a1, a2, a3;
      widen4<FMT>(kt.w[0][k], a0, a2);
      widen4<FMT>(kt.w[1][k], a1, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_f16_16816(s[nt], a0, a1, a2, a3, qf[nt][k][0], qf[nt][k][1]);
        if constexpr (sizeof(T) == 4) {
          const uint2 x = *reinterpret_cast<const uint2 *>(tail + 8 * nt * Attend8Smem<D, NT>::kQPitch + k_elem(k, lane & 3));
          mma_f16_16816(s[nt], a0, a1, a2, a3, x.x, x.y);
        }
      }
    }
    const bool masked = x0 + 16 > all_see;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // (the attention's product, rounded before the reference leaves it, as there)
        float p = ex2_approx(__fmul_rn(s[nt][e], cf[nt][e & 1] * k_scale) - ml[nt][e & 1].x);
        if (masked && x0 + lg + 8 * (e >> 1) >= rows[nt][e & 1]) p = 0.0f;
        sum[e >> 1] = fmaf(p, ml[nt][e & 1].y, sum[e >> 1]);
      }
  }
};

template <typename T, int D, int NT, int FMT>
__global__ void __launch_bounds__(32 * kC8Warps)
cache8_weight_kernel(Attend8Args a, int stream) {
  using Wm = Weight8Smem<D, NT>;
  extern __shared__ __align__(16) uint8_t sm[];
  float2 *stats = reinterpret_cast<float2 *>(sm + Wm::kStats);
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.y / a.H_kv, g = blockIdx.y % a.H_kv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Attend8Query q = attend8_query(a, b, false);
  const int64_t bh = static_cast<int64_t>(b) * a.H_kv + g;
  const int tiles = (q.len + 15) / 16, cols = q.n * a.G;
  const uint32_t ring = smem_u32(sm + Wm::kK) + warp * kC8wTiles * Tile8<D>::kBytes;
  WeightColumns<T, D, NT, FMT> col;
  auto fetch = [&](int slot, int tile) {
    const uint8_t *src = a.k8 + (bh * a.cap + tile * 16) * D;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const int p = lane + 32 * u;
      cp_async_16(ring + slot * Tile8<D>::kBytes + Tile8<D>::k_off(p / (D / 16), p % (D / 16)), src + 16 * p, true);
    }
  };
  auto scale_of = [&](int tile) { return a.ks[(bh * a.cap + tile * 16) >> a.bl_shift]; };
  auto write = [&](int tile, const float (&sum)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float x = sum[r];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      const int row = tile * 16 + (lane >> 2) + 8 * r;
      if ((lane & 3) == 0 && row < q.len) {
        float *w = a.weights + bh * a.cap + row;
        *w = a.decay == 0.0f ? x : a.decay * *w + x;
      }
    }
  };
  if (stream) {
    const int step = gridDim.x * kC8Warps;
    int tile = blockIdx.x * kC8Warps + warp, ahead = tile;
#pragma unroll
    for (int i = 0; i < kC8wTiles - 1; ++i) {
      if (ahead < tiles) fetch(i, ahead);
      cp_async_commit();
      ahead += step;
    }
    col.load(a, q, b, g, 0, sm, stats);
    float k_scale = tile < tiles ? scale_of(tile) : 0.0f;
    for (int slot = 0; tile < tiles; tile += step) {
      cp_async_wait<kC8wTiles - 2>();
      __syncwarp();  // every lane's copies are there; the slot of the last tile is free
      if (ahead < tiles) fetch((slot + kC8wTiles - 1) % kC8wTiles, ahead);
      cp_async_commit();
      ahead += step;
      const float ks = k_scale;
      if (tile + step < tiles) k_scale = scale_of(tile + step);
      float sum[2] = {0.0f, 0.0f};
      if (cols > 0) col.add(ring + slot * Tile8<D>::kBytes, tile * 16, ks, sum);
      write(tile, sum);
      slot = (slot + 1) % kC8wTiles;
    }
    cp_async_wait<0>();
    return;
  }
  if (static_cast<int>(blockIdx.x) * kC8wRows >= q.len) return;
  // tile i of this warp
  auto tile_of = [&](int i) { return blockIdx.x * (kC8wRows / 16) + kC8Warps * i + warp; };
  float k_scale[kC8wTiles], sum[kC8wTiles][2];
#pragma unroll
  for (int i = 0; i < kC8wTiles; ++i) {
    k_scale[i] = sum[i][0] = sum[i][1] = 0.0f;
    if (tile_of(i) < tiles) {
      fetch(i, tile_of(i));
      k_scale[i] = scale_of(tile_of(i));
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  for (int c0 = 0; c0 < cols; c0 += 8 * NT) {
    if (c0) __syncthreads();
    col.load(a, q, b, g, c0, sm, stats);
#pragma unroll
    for (int i = 0; i < kC8wTiles; ++i)
      if (tile_of(i) < tiles) col.add(ring + i * Tile8<D>::kBytes, tile_of(i) * 16, k_scale[i], sum[i]);
  }
#pragma unroll
  for (int i = 0; i < kC8wTiles; ++i)
    if (tile_of(i) < tiles) write(tile_of(i), sum[i]);
}

}  // namespace msa
