// cache8_weight_tc.cuh -- the weight each cached row received from many
// columns, on the 5th-generation tensor cores (the formula of
// cache8_weight_kernel: sum over the columns of 2^(s - m) / L, the scores s
// recomputed).  Context rows are the M rows of S = K Q^T here, so a row's
// weights of all columns meet in one thread and nothing is exchanged.
//
// One CTA per (query, kv head, 256 cached rows): K is widened to fp16 in
// shared memory once (two tiles of 128 rows, one TMEM lane and one thread a
// row, which applies the row's scale itself); Q, brought to fp16 scaled by a
// power of two a column by a kernel before (every CTA reads all of it: converted
// here it set the pace, 137 us for the case below), streams through in tiles of
// 128 columns.
//   warps 9-12   copy Q tiles, and a thread a column its factor, reference, 1 / L
//                and visible rows
//   warp 8       one thread issues S (M 128, N 128, K D) for both tiles into
//                one of two TMEM buffers each
//   warps 0-7    S from TMEM, the weights added up in registers
// The special-function unit is the floor: 256 x 128 exponentials take 2,048
// cycles a scheduler, the MMAs about 1,300; the row warps need 3,970 cycles a
// tile.  512 tokens x 32 heads over 8,704 rows: 386 us on mma.sync, 99 here;
// 718 columns of D = 64 over 16,000 rows 79 against 21.
// Every wait is bounded as in the attention on tcgen05.
#pragma once
#include "cache8_prefill_tc.cuh"

namespace msa {

constexpr int kCwThreads = 32 * 13;
constexpr int kCwRows = 256;   // cached rows a CTA
constexpr int kCwCols = 128;   // columns of a Q tile

enum {
  kWbK = 0,              // K in shared memory (256 threads)
  kWbFullQ0 = 1,         // Q slot holds its tile (128 threads) [2]
  kWbFreeQ0 = 3,         // both tiles' MMAs reading the slot completed (commit) [2]
  kWbS0 = 5,             // S buffer (tile, j % 2) computed (commit) [4]
  kWbDone0 = 9,          // S buffer read (128 threads) [4]
  kWbDrain = 13,
  kWbN = 14
};

template <int D>
struct CwSmem {
  static constexpr int kTile = D / 64 * 128 * 128;      // [panel][128 rows][128 B]
  static constexpr int kQ = 2 * kTile;                  // behind K's two tiles: two slots
  static constexpr int kBars = kQ + 2 * kTile;
  static constexpr int kMisc = kBars + kWbN * 8;        // TMEM slot, fail
  // per column, a ring of four tiles: factor, -reference, 1 / L, visible rows
  static constexpr int kConst = kMisc + 16;
  static constexpr int kFar = kConst + 4 * 4 * kCwCols * 4;  // a ring of four: [copier warp] far scores
  static constexpr int kBytes = 1024 + kFar + 4 * 16;
};
static_assert(CwSmem<64>::kConst % 16 == 0 && CwSmem<128>::kConst % 16 == 0, "vector loads");

// Q as the weight kernel reads it: q16[b][g][column][D] fp16, factor[b][g][column] its power of two
// times scale_log2.  grid ceil(B * T * H_q / 8), block 256, a warp a column.
template <int D>
__global__ void __launch_bounds__(256)
cache8_q16_kernel(Attend8Args a, int batch, __half *__restrict__ q16, float *__restrict__ factor) {
  constexpr int E = D / 32;  // elements a lane
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x % 32, cols = a.T * a.G;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;  // (b, g, column)
  if (i >= static_cast<int64_t>(batch) * a.H_kv * cols) return;
  const int col = static_cast<int>(i % cols), g = static_cast<int>(i / cols % a.H_kv);
  const int b = static_cast<int>(i / cols / a.H_kv), t = col_token(a, col);
  const int64_t row = (static_cast<int64_t>(b) * a.T + t) * a.H_kv * a.G + g * a.G + col - t * a.G;
  const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(a.Q) + row * D + E * lane);
  float x[E], mx = 0.0f;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const uint32_t w = src[e / 2];
    x[e] = __uint_as_float(w << 16);
    x[e + 1] = __uint_as_float(w & 0xffff0000u);
    mx = fmaxf(mx, fmaxf(finite_abs(x[e]), finite_abs(x[e + 1])));
  }
  mx = warp_max(mx);
  const float p2 = mx > 0.0f ? floor_pow2(mx) : 1.0f, inv = 1.0f / p2;
  uint32_t *dst = reinterpret_cast<uint32_t *>(q16 + i * D + E * lane);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack_f16x2(x[e] * inv, x[e + 1] * inv);
  if (lane == 0) factor[i] = a.scale_log2 * p2;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kCwThreads, 1)
cache8_weight_tc_kernel(Attend8Args a, const __half *__restrict__ q16, const float *__restrict__ factor) {
  using Sm = CwSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Sm::kBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + Sm::kMisc);
  volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  auto consts = [&](int j) { return reinterpret_cast<float *>(sm + Sm::kConst) + (j & 3) * 4 * kCwCols; };
  const int b = blockIdx.y / a.H_kv, g = blockIdx.y % a.H_kv, r0 = blockIdx.x * kCwRows;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  griddep_wait();
  griddep_launch();
  const Attend8Query q = attend8_query(a, b, false);
  if (r0 >= q.len) return;
  const int cols = q.n * a.G, n = (cols + kCwCols - 1) / kCwCols;
  const int64_t bh = static_cast<int64_t>(b) * a.H_kv + g;
  if (threadIdx.x == 0) {
    mbar_init(bar(kWbK), 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kWbFullQ0 + i), 128);
      mbar_init(bar(kWbFreeQ0 + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kWbS0 + i), 1);
      mbar_init(bar(kWbDone0 + i), 128);
    }
    mbar_init(bar(kWbDrain), 1);
    *fail = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(smem_u32(tmem_slot), kC8tTmemCols);
  tc05_fence_before();
  __syncthreads();  // barriers, the fail flag and the TMEM address are visible
  tc05_fence_after();
  const uint32_t tmem = *tmem_slot;
  // bounded wait; false (and every later wait that would block, at once) after a timeout anywhere
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity)) return true;
    if (*fail) return false;
    if (mbar_wait(bar(i), parity)) return true;
    *fail = 1;
    raise_device_error(MSA_DEVERR_WAIT_TIMEOUT);
    return false;
  };

  if (warp >= 9) {
    // ------------------------------------------------------------ Q tiles
    const int r = threadIdx.x - 32 * 9;
    const int64_t first = bh * a.T * a.G;  // the head's columns in q16 and factor
    for (int j = 0; j < n; ++j) {
      const int col = j * kCwCols + r, t = col_token(a, col);
      const bool real = col < cols;
      float f = 0.0f;
      float2 ml = make_float2(INFINITY, 0.0f);  // (no column: weight 0)
      if (real) {
        f = factor[first + col];
        ml = a.ml[(static_cast<int64_t>(b) * a.T + t) * a.H_kv * a.G + g * a.G + col - t * a.G];
      }
      if (j >= 2 && !wait(kWbFreeQ0 + (j & 1), ((j >> 1) - 1) & 1)) break;
      const __half *src = q16 + (first + j * kCwCols) * D;
      const uint32_t dst = smem_u32(sm + Sm::kQ + (j & 1) * Sm::kTile);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {  // 16-byte pieces, D / 8 a column
        const int p = r + 128 * i, c = p / (D / 8);
        const bool have = j * kCwCols + c < cols;
        cp_async_16(dst + ptc_swz(c, p % (D / 8), kCwCols), src + (have ? p * 8 : 0), have);
      }
      cp_async_commit();
      float *c = consts(j) + r;
      c[0] = f;
      c[kCwCols] = -ml.x;
      c[2 * kCwCols] = ml.y;
      c[3 * kCwCols] = __int_as_float(real ? column_rows(a, q, col) : 0);
      const bool far = __any_sync(0xffffffffu, fabsf(ml.x) > kC8tFar && ml.x != INFINITY);
      if (lane == 0) reinterpret_cast<int *>(sm + Sm::kFar)[4 * (j & 3) + warp - 9] = far;
      cp_async_wait<0>();
      fence_proxy_async_smem();  // the tile becomes visible to the tensor cores
      mbar_arrive(bar(kWbFullQ0 + (j & 1)));
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = umma_idesc_f16_f32<128, kCwCols>();
    const uint32_t base = smem_u32(sm);
    const uint64_t k_desc = umma_desc_k_sw128(base), q_desc = umma_desc_k_sw128(base + Sm::kQ);
    bool ok = n > 0 && __all_sync(0xffffffffu, wait(kWbK, 0));
    for (int j = 0; j < n && ok; ++j) {
      const int u = j & 1;
      ok = __all_sync(0xffffffffu, wait(kWbFullQ0 + u, (j >> 1) & 1));
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // the buffer's last scores have been read
        if (j >= 2) ok = __all_sync(0xffffffffu, ok && wait(kWbDone0 + 2 * x + u, ((j >> 1) - 1) & 1));
        if (!ok) break;
        tc05_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t p = (i >> 2) * 128 * 8 + (i & 3) * 2;  // in units of 16 bytes
            umma_bf16(tmem + 256 * x + 128 * u, k_desc + x * (Sm::kTile >> 4) + p,
                      q_desc + u * (Sm::kTile >> 4) + p, idesc, i != 0);
          }
          umma_commit(bar(kWbS0 + 2 * x + u));
          if (x == 1) umma_commit(bar(kWbFreeQ0 + u));
        }
        __syncwarp();
      }
    }
    // every MMA issued here completes before TMEM is freed
    if (lane == 0) {
      umma_commit(bar(kWbDrain));
      mbar_wait(bar(kWbDrain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ rows
    const int x = warp >> 2, r = threadIdx.x & 127, row = r0 + 128 * x + r;
    // K: 16-byte pieces of 256 rows, D / 16 a thread, widened; rows past the last one are zero
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int p = static_cast<int>(threadIdx.x) + 256 * i, kr = p / (D / 16), pc = p % (D / 16);
      uint4 y = make_uint4(0, 0, 0, 0);
      if (r0 + kr < q.len) y = ld_stream16(a.k8 + (bh * a.cap + r0 + kr) * D + 16 * pc);
      uint32_t z[8];
      widen4<FMT>(y.x, z[0], z[1]);
      widen4<FMT>(y.y, z[2], z[3]);
      widen4<FMT>(y.z, z[4], z[5]);
      widen4<FMT>(y.w, z[6], z[7]);
      uint8_t *dst = sm + (kr >> 7) * Sm::kTile;
      *reinterpret_cast<uint4 *>(dst + ptc_swz(kr & 127, 2 * pc, 128)) = make_uint4(z[0], z[1], z[2], z[3]);
      *reinterpret_cast<uint4 *>(dst + ptc_swz(kr & 127, 2 * pc + 1, 128)) = make_uint4(z[4], z[5], z[6], z[7]);
    }
    fence_proxy_async_smem();  // K becomes visible to the tensor cores
    mbar_arrive(bar(kWbK));
    const float ks = row < q.len ? a.ks[(bh * a.cap + row) >> a.bl_shift] : 0.0f;
    const uint32_t at = tmem + 256 * x + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int last = r0 + 128 * x + 127;  // the tile's last row
    float2 sum = make_float2(0.0f, 0.0f);
    for (int j = 0; j < n; ++j) {
      const int u = j & 1;
      if (!__all_sync(0xffffffffu, wait(kWbS0 + 2 * x + u, (j >> 1) & 1))) break;
      tc05_fence_after();
      const float *c = consts(j);
      // hidden rows only where the tile passes what the first column sees
      const bool masked = last >= column_rows(a, q, j * kCwCols);
      const int4 fr = *reinterpret_cast<const int4 *>(sm + Sm::kFar + 16 * (j & 3));
      const bool far = (fr.x | fr.y | fr.z | fr.w) != 0;
#pragma unroll
      for (int h = 0; h < kCwCols; h += 32) {
        uint32_t raw[32];
        tmem_ld32(at + 128 * u + h, raw);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 cf = *reinterpret_cast<const float4 *>(c + h + i);
          const float4 nm = *reinterpret_cast<const float4 *>(c + kCwCols + h + i);
          const float4 il = *reinterpret_cast<const float4 *>(c + 2 * kCwCols + h + i);
          // factors first: they round and overflow only where the attention's did
          const float2 k2 = make_float2(ks, ks);
          float2 e0 = mul2(mul2(make_float2(cf.x, cf.y), k2),
                           make_float2(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1])));
          float2 e1 = mul2(mul2(make_float2(cf.z, cf.w), k2),
                           make_float2(__uint_as_float(raw[i + 2]), __uint_as_float(raw[i + 3])));
          if (far) {
            // the product rounded by itself, as in the attention (above it is fused with the sum):
            // a far score's rounding is many times a unit of its exponent
            e0.x = __fadd_rn(__fmul_rn(__fmul_rn(cf.x, ks), __uint_as_float(raw[i])), nm.x);
            e0.y = __fadd_rn(__fmul_rn(__fmul_rn(cf.y, ks), __uint_as_float(raw[i + 1])), nm.y);
            e1.x = __fadd_rn(__fmul_rn(__fmul_rn(cf.z, ks), __uint_as_float(raw[i + 2])), nm.z);
            e1.y = __fadd_rn(__fmul_rn(__fmul_rn(cf.w, ks), __uint_as_float(raw[i + 3])), nm.w);
          } else {
            e0 = add2(e0, make_float2(nm.x, nm.y));
            e1 = add2(e1, make_float2(nm.z, nm.w));
          }
          float2 p0 = make_float2(ex2_approx(e0.x), ex2_approx(e0.y));
          float2 p1 = make_float2(ex2_approx(e1.x), ex2_approx(e1.y));
          if (masked) {
            const float4 vis = *reinterpret_cast<const float4 *>(c + 3 * kCwCols + h + i);
            p0.x = row < __float_as_int(vis.x) ? p0.x : 0.0f;
            p0.y = row < __float_as_int(vis.y) ? p0.y : 0.0f;
            p1.x = row < __float_as_int(vis.z) ? p1.x : 0.0f;
            p1.y = row < __float_as_int(vis.w) ? p1.y : 0.0f;
          }
          sum = fma2(p0, make_float2(il.x, il.y), sum);
          sum = fma2(p1, make_float2(il.z, il.w), sum);
        }
      }
      tc05_fence_before();
      mbar_arrive(bar(kWbDone0 + 2 * x + u));
    }
    if (row < q.len) {
      float *w = a.weights + bh * a.cap + row;
      const float s = sum.x + sum.y;
      *w = a.decay == 0.0f ? s : a.decay * *w + s;
    }
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == 8) tmem_dealloc(tmem, kC8tTmemCols);
}

}  // namespace msa
