// cache8_prefill_tc.cuh -- attention of many new tokens over [8-bit local rows
// | retrieved memory rows] on the 5th-generation tensor cores: the arithmetic
// of cache8_attend.cuh (4 D FLOP for every visible (row, column) pair), which
// bounds it once a context row is shared by some hundred columns.
//
// One CTA per (query, kv head, pair of tiles of 128 columns, context split); a
// column is a (token, head of the group) pair and owns one TMEM lane and one
// softmax thread.  Both tiles share every context block of 64 rows:
//   converters (warps 10-13) load a block's bytes, widen them to fp16 in
//        registers and write them to shared memory in the MMA's layout, K and V
//        each into a ring of four.  Cached values are exact in fp16; their scales
//        (one for K and one for V, of 16 rows each where cache blocks are that short)
//        leave with the block for the softmax.  K of bf16 memory rows is brought to fp16 by a power of two that
//        takes the block's largest element below 2, or, where a row lies 2^6 and more below
//        another, by one of its own for every row, which leaves with the block (elements
//        below 2^-10 of their row's largest may lose bits, 2^-19 of it at most).  Their V stays
//        bf16, P is then a bf16 head and tail and P V two MMAs.  So a row costs the others
//        nothing, however large it is.
//   warps 8, 9  one for each tile: a thread issues S = Q K^T (M 128, N 64, K D; Q fp16, scaled by a
//        power of two per column) into one of two TMEM buffers a tile, and
//        O += P V (M 128, N D, K 64), each as soon as its inputs are ready (one
//        warp for both tiles was bound by the issue: 72 cycles an MMA, 113 a
//        commit, 120 a barrier test)
//   warps 0-3, 4-7  the softmax of a tile, a thread a column: S from TMEM, the
//        hidden rows masked, P = 2^(s - m + r + 11) (r: log2 of V's scale over the unit of
//        O, as in cache8_attend.cuh), written as fp16 over S: P is the MMA's A operand straight from TMEM,
//        so nothing but Q, K and V passes through shared memory.  The softmax of
//        a block waits for no P V: the next S is ready when it ends, and only a
//        move of the reference m (when s + r passes it by 4 in log2 units; to 7 to 8
//        above) waits for O's last update and rescales O's lane.  r is a whole number
//        and goes into the exponent; a group's sum of weights is brought back by 2^-r.
// 512 tokens x 32 heads over 8,704 + 128 rows: 117 us; before the last steps 166 with
// P through shared memory against 126, and 153 with blocks of 128 rows and one S a tile
// (S, softmax and P V of a tile then follow one another).
// Every wait is bounded: on timeout the CTA raises MSA_DEVERR_WAIT_TIMEOUT,
// every role skips the rest (the outputs are then void), and issued MMAs are
// drained before TMEM is freed.
#pragma once
#include "cache8_attend.cuh"
#include "tc05.cuh"

namespace msa {

constexpr int kC8tConv = 128;                       // converter threads
constexpr int kC8tThreads = 32 * 10 + kC8tConv;
constexpr int kC8tBlk = 64;                         // context rows per block
constexpr int kC8tSlots = 4;                        // ring of K, ring of V
constexpr int kC8tRows = 128;                       // columns per tile (UMMA M)
constexpr float kC8MinFold = -40.0f;                // V scale ratios (log2) that go into P's exponent
constexpr float kC8tFar = 2048.0f;                  // scores (log2 units) beyond this are "far"
constexpr uint32_t kC8tTmemCols = 512;              // S, then P, of tile x at 128 x + 64 (block % 2),
constexpr uint32_t kC8tTmemO = 256;                 // O of tile x at 256 + 128 x

enum {
  kCbFullK0 = 0,                       // K slot holds its block (every converter thread)
  kCbFullV0 = kCbFullK0 + kC8tSlots,   // V slot
  kCbFreeK0 = kCbFullV0 + kC8tSlots,   // every Q K^T reading the slot completed (commit)
  kCbFreeV0 = kCbFreeK0 + kC8tSlots,   // every P V reading the slot completed (commit)
  kCbS0 = kCbFreeV0 + kC8tSlots,       // S buffer (tile, block % 2) computed (commit) [4]
  kCbO0 = kCbS0 + 4,                   // P V of (tile, block % 2) completed (commit) [4]
  kCbQ0 = kCbO0 + 4,                   // tile's Q in shared memory (128 threads) [2]
  kCbP0 = kCbQ0 + 2,                   // P of (tile, block % 2) written, O rescaled (128 threads) [4];
                                       // one for each buffer: a softmax may be a block ahead of P V
  kCbDrain = kCbP0 + 4,                // a tile's MMAs all completed (commit) [2]
  kCbN = kCbDrain + 2
};

struct C8tSmem {
  static constexpr int D = 128;
  static constexpr int kQBytes = 2 * kC8tRows * 128;    // [panel][128 rows][128 B]
  static constexpr int kKVBytes = 2 * kC8tBlk * 128;    // [panel][64 rows][128 B]
  static constexpr int kK = 2 * kQBytes;                // slots
  static constexpr int kV = kK + kC8tSlots * kKVBytes;
  static constexpr int kBars = kV + kC8tSlots * kKVBytes;
  // K's scales of 16 rows each, log2 of V's over the unit (r), {log2 of the unit's growth, the unit,
  // least r, whether the rows of K have scales of their own}
  static constexpr int kScales = 12;
  static constexpr int kScale = (kBars + kCbN * 8 + 15) / 16 * 16;  // [block % (2 slots)][kScales]
  static constexpr int kRowScale = kScale + 2 * kC8tSlots * kScales * 4;  // [block % (2 slots)][row]
  static constexpr int kRed = kRowScale + 2 * kC8tSlots * kC8tBlk * 4;    // [converter warp]
  static constexpr int kMisc = kRed + 32;               // TMEM slot, fail, memory rows
  static constexpr int kPre = kMisc + 16;
  static int bytes(int table_cap) { return 1024 + kPre + (2 * kMaxTopK + 1 + table_cap) * 4; }
};

// Instruction descriptor, kind::f16: fp16 A and B, fp32 D.
template <int M, int N>
__host__ __device__ constexpr uint32_t umma_idesc_f16_f32() {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The same MMA with A in TMEM (a lane a row, two fp16 of K a column).
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Store 32 consecutive columns of this thread's TMEM lane, then wait for the store.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};\n"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
      "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// Load 32 consecutive columns of this thread's TMEM lane and wait for them.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

// The power of two at or below a finite x > 0, within the normal numbers that have a reciprocal.
__device__ __forceinline__ float floor_pow2(float x) {
  return __int_as_float(max(1, min(253, __float_as_int(x) >> 23)) << 23);
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// grid (pairs * B * H_kv, n_split), block kC8tThreads, one CTA per SM.
// NG groups of a block's 64 rows have scales of their own: 1 for cache blocks of 64 rows and more, else 4
// (512 tokens over 8,704 rows in blocks of 64: 116 us with one group, 123 with four).
template <int FMT, int NG>
__global__ void __launch_bounds__(kC8tThreads, 1)
cache8_prefill_tc_kernel(Attend8Args a, int n_pairs) {
  using Sm = C8tSmem;
  constexpr int D = 128, RG = kC8tBlk / NG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Sm::kBars);
  float *scales = reinterpret_cast<float *>(sm + Sm::kScale);
  auto row_scales = [&](int j) { return reinterpret_cast<float *>(sm + Sm::kRowScale) + kC8tBlk * (j % (2 * kC8tSlots)); };
  float2 *red = reinterpret_cast<float2 *>(sm + Sm::kRed);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + Sm::kMisc);
  volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *mem_rows = reinterpret_cast<int *>(tmem_slot + 2);
  int *pre = reinterpret_cast<int *>(sm + Sm::kPre), *base = pre + kMaxTopK + 1;
  int *table = base + kMaxTopK;
  auto bar = [&](int i) { return smem_u32(bars + i); };

  const int bg = static_cast<int>(blockIdx.x / n_pairs), b = bg / a.H_kv, g = bg % a.H_kv;
  const int pair = n_pairs - 1 - static_cast<int>(blockIdx.x % n_pairs);  // most context first
  const int split = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  griddep_wait();
  griddep_launch();
  const Attend8Query q = attend8_query(a, b, pair == 0 && g == 0 && split == 0 && threadIdx.x == 0);
  const int cols = q.n * a.G;  // real columns of this (query, kv head)
  const int c0 = pair * 2 * kC8tRows;
  if (c0 >= cols) return;  // padding tokens only (the whole CTA)
  const bool act1 = c0 + kC8tRows < cols;

  if (threadIdx.x == 32 * 8) {
    for (int i = 0; i < kC8tSlots; ++i) {
      mbar_init(bar(kCbFullK0 + i), kC8tConv);
      mbar_init(bar(kCbFullV0 + i), kC8tConv);
      mbar_init(bar(kCbFreeK0 + i), act1 ? 2 : 1);  // one commit a tile
      mbar_init(bar(kCbFreeV0 + i), act1 ? 2 : 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(kCbS0 + i), 1);
      mbar_init(bar(kCbO0 + i), 1);
      mbar_init(bar(kCbP0 + i), 128);
    }
    for (int i = 0; i < 2; ++i) mbar_init(bar(kCbQ0 + i), 128);
    mbar_init(bar(kCbDrain), 1);
    mbar_init(bar(kCbDrain + 1), 1);
    *fail = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 8) tmem_alloc(smem_u32(tmem_slot), kC8tTmemCols);
  if (warp == 9) {
    const int n = a.k == 0 ? 0
                           : chunk_prefix_warp(a.ids + static_cast<int64_t>(b) * a.k, a.k, a.doc_chunk_off, a.n_docs,
                                               a.slots ? a.slots + static_cast<int64_t>(b) * a.k : nullptr,
                                               a.slot_chunks, pre, base, a.table_cap, lane);
    if (lane == 0) *mem_rows = n;
  }
  // row of Q and O of a column (they are fewer than 2^31)
  auto row_of = [&](int col) {
    const int t = col_token(a, col);
    return ((b * a.T + t) * a.H_kv + g) * a.G + col - t * a.G;
  };
  float cf = 0.0f;  // score factor of this thread's column: scale_log2 * the power of two taken out of Q
  if (warp >= 8) {
    // the others start on the context while the softmax warps bring Q
    tc05_fence_before();
    asm volatile("bar.sync 2, %0;" ::"n"(kC8tThreads - 256) : "memory");
    asm volatile("bar.arrive 3, %0;" ::"n"(kC8tThreads) : "memory");
  } else {
    if (warp < 4 || act1) {
      // Q to fp16, each row scaled by a power of two: a warp its 32 columns, sixteen lanes a row
      uint8_t *qs = sm + (warp >> 2) * Sm::kQBytes;
      const int r0 = 32 * (warp & 3) + (lane >> 4), piece = lane & 15;
      constexpr int N = 4;  // rows in flight
#pragma unroll 1
      for (int i0 = 0; i0 < 16; i0 += N) {
        uint4 w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int col = c0 + (warp >> 2) * kC8tRows + r0 + 2 * (i0 + i);
          w[i] = make_uint4(0, 0, 0, 0);
          if (col < cols)
            w[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.Q) +
                                                         static_cast<int64_t>(row_of(col)) * D) + piece);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t y[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          float mx = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx = max3(mx, finite_abs(__uint_as_float(y[e] << 16)), finite_abs(__uint_as_float(y[e] & 0xffff0000u)));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float p2 = mx > 0.0f ? floor_pow2(mx) : 1.0f;
          const float inv = __int_as_float(0x7f000000 - __float_as_int(p2));  // 1 / p2
          uint32_t z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            z[e] = pack_f16x2(__uint_as_float(y[e] << 16) * inv, __uint_as_float(y[e] & 0xffff0000u) * inv);
          *reinterpret_cast<uint4 *>(qs + ptc_swz(r0 + 2 * (i0 + i), piece, kC8tRows)) = make_uint4(z[0], z[1], z[2], z[3]);
          const float own = __shfl_sync(0xffffffffu, p2, 16 * (lane & 1));  // of this lane's row, if i0 + i is lane / 2
          if (lane >> 1 == i0 + i) cf = a.scale_log2 * own;
        }
      }
      fence_proxy_async_smem();  // Q becomes visible to the tensor cores
    }
    tc05_fence_before();
    asm volatile("bar.sync 3, %0;" ::"n"(kC8tThreads) : "memory");
    if (warp < 4 || act1) mbar_arrive(bar(kCbQ0 + (warp >> 2)));
  }
  tc05_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_mem = *mem_rows;

  // this split's blocks: of the local ones [0, lb) and the memory ones behind them
  const int n_loc = max(0, column_rows(a, q, min(c0 + 2 * kC8tRows, cols) - 1));
  const int lb = (n_loc + kC8tBlk - 1) / kC8tBlk, mb = (n_mem + kC8tBlk - 1) / kC8tBlk;
  const int u0 = share(lb + mb, split, a.n_split), u1 = share(lb + mb, split + 1, a.n_split);
  const int nblk = u1 - u0;
  const int64_t bh = static_cast<int64_t>(b) * a.H_kv + g;

  // bounded wait; false (and every later wait that would block, at once) after a timeout anywhere
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity)) return true;
    if (*fail) return false;
    if (mbar_wait(bar(i), parity)) return true;
    *fail = 1;
    raise_device_error(MSA_DEVERR_WAIT_TIMEOUT);
    return false;
  };

  if (warp >= 10) {
    // ------------------------------------------------------------ converters
    const int tid = threadIdx.x - 32 * 10;
    // after a timeout the loops run on without work, so that every converter thread reaches the
    // memory blocks' barriers
    bool live = true;
    // half h (0: K, 1: V) of the j-th block: its slot, waited for; false after a timeout
    auto slot = [&](int j, int h) { return sm + (h ? Sm::kV : Sm::kK) + (j % kC8tSlots) * Sm::kKVBytes; };
    auto wait_slot = [&](int j, int h) {
      if (j >= kC8tSlots)  // (the lanes of a warp agree: what follows may be warp-collective)
        live = __all_sync(0xffffffffu, live && wait((h ? kCbFreeV0 : kCbFreeK0) + j % kC8tSlots, (j / kC8tSlots - 1) & 1));
      return live;
    };
    // a block's scales go out with K, so that S's barrier brings them to the softmax.  Every thread
    // follows them (a lane of its own would hold up its warp: 450 against 395 us for 32 times 12
    // tokens over 8,192 rows), thread 0 writes; whole numbers, so exponents are enough
    int unit = 0;  // exponent field of the largest V scale so far
    auto put_scales = [&](int j, float4 k, float4 v, bool rows) {
      const int e[4] = {__float_as_int(v.x) >> 23, __float_as_int(v.y) >> 23, __float_as_int(v.z) >> 23,
                        __float_as_int(v.w) >> 23};
      const int top = max(max(e[0], e[1]), max(e[2], e[3])), up = top > unit && unit > 0 ? top - unit : 0;
      unit = max(unit, top);
      auto whole = [](int x) { return __int_as_float(0x4b400000 + x) - 12582912.0f; };
      auto ratio = [&](int x) { return x > 0 ? whole(x - unit) : kC8MinRatio; };  // (0: rows of zeros)
      const float4 r = make_float4(ratio(e[0]), ratio(e[1]), ratio(e[2]), ratio(e[3]));
      const float least = fminf(fminf(r.x, r.y), fminf(r.z, r.w));
      if (tid == 0) {
        float4 *to = reinterpret_cast<float4 *>(scales + Sm::kScales * (j % (2 * kC8tSlots)));
        to[0] = k;
        to[1] = r;
        to[2] = make_float4(whole(up), __int_as_float(unit << 23), least, rows ? 1.0f : 0.0f);
      }
    };
    auto landed = [&](int j, int h) {
      fence_proxy_async_smem();  // the rows become visible to the tensor cores
      mbar_arrive(bar((h ? kCbFullV0 : kCbFullK0) + j % kC8tSlots));
    };
    // Local rows.  Piece i of a thread lies in rows 16 i .. 16 i + 15; eight threads take four
    // pieces of two neighbouring rows, whose swizzled places hit every bank once.  A half's bytes
    // are loaded a whole block ahead, right after the last ones left their registers.
    const int row0 = 2 * (tid >> 4) + ((tid >> 2) & 1), pc = 4 * ((tid >> 3) & 1) + (tid & 3);
    constexpr int N = kC8tBlk / 16;  // pieces of a half
    uint4 raw[2][N];
    float rs[2][NG];  // the groups' scales (the first one's past the last row)
    auto load_raw = [&](int u, int h) {
      if (u >= u1 || u >= lb) return;
      const uint8_t *src = (h ? a.v8 : a.k8) + (bh * a.cap + static_cast<int64_t>(u) * kC8tBlk + row0) * D + 16 * pc;
      const float *sc = (h ? a.vs : a.ks) + bh * (a.cap >> a.bl_shift);
      const int left = n_loc - u * kC8tBlk;  // rows of the block
#pragma unroll
      for (int i = 0; i < N; ++i) {
        raw[h][i] = make_uint4(0, 0, 0, 0);
        if (left >= kC8tBlk || 16 * i + row0 < left) raw[h][i] = ld_stream16(src + 2048 * i);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) rs[h][g] = __ldg(sc + ((u * kC8tBlk + (RG * g < left ? RG * g : 0)) >> a.bl_shift));
    };
    load_raw(u0, 0);
    load_raw(u0, 1);
    const int nl = max(0, min(u1, lb) - u0);  // local blocks of this split
    for (int j = 0; j < nl; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait_slot(j, h)) continue;
        if (h == 0)
          put_scales(j, make_float4(rs[0][0], rs[0][1 % NG], rs[0][2 % NG], rs[0][3 % NG]),
                     make_float4(rs[1][0], rs[1][1 % NG], rs[1][2 % NG], rs[1][3 % NG]), false);
        uint8_t *dst = slot(j, h);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint4 x = raw[h][i];
          uint4 lo, hi;
          widen4<FMT>(x.x, lo.x, lo.y);
          widen4<FMT>(x.y, lo.z, lo.w);
          widen4<FMT>(x.z, hi.x, hi.y);
          widen4<FMT>(x.w, hi.z, hi.w);
          *reinterpret_cast<uint4 *>(dst + ptc_swz(16 * i + row0, 2 * pc, kC8tBlk)) = lo;
          *reinterpret_cast<uint4 *>(dst + ptc_swz(16 * i + row0, 2 * pc + 1, kC8tBlk)) = hi;
        }
        load_raw(u0 + j + 1, h);
        landed(j, h);
      }
    }
    // memory rows, bf16: pieces of 8 elements, 16 a row; V as it is
    const int64_t kv = static_cast<int64_t>(a.H_kv) * D;
    constexpr int M = kC8tBlk / 8;
    if (nblk > nl) {
      for (int x = tid; x < n_mem; x += kC8tConv) table[x] = chunk_row(pre, base, a.k, x);
      asm volatile("bar.sync 1, %0;" ::"n"(kC8tConv) : "memory");
    }
    for (int j = nl; j < nblk; ++j) {
      uint4 w[M];
      const int x0 = (u0 + j - lb) * kC8tBlk + (tid >> 4);
      auto load = [&](int h) {
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.content) + h * kv + g * D + 8 * (tid & 15);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const int x = x0 + 8 * i;
          w[i] = make_uint4(0, 0, 0, 0);
          if (x < n_mem) w[i] = *reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(table[x]) * 2 * kv);
        }
      };
      auto largest = [&](uint4 x) {
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          m = max3(m, finite_abs(__uint_as_float(y[e] << 16)), finite_abs(__uint_as_float(y[e] & 0xffff0000u)));
        return m;
      };
      auto put = [&](int h, int i, uint4 x) {
        *reinterpret_cast<uint4 *>(slot(j, h) + ptc_swz(8 * i + (tid >> 4), tid & 15, kC8tBlk)) = x;
      };
      auto put_k = [&](int i, float inv) {
        const uint32_t y[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          z[e] = pack_f16x2(__uint_as_float(y[e] << 16) * inv, __uint_as_float(y[e] & 0xffff0000u) * inv);
        put(0, i, make_uint4(z[0], z[1], z[2], z[3]));
      };
      load(0);
      // the largest and the smallest of the block's pieces; a row far below another has small ones
      float hi = 0.0f, lo = INFINITY;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const float m = largest(w[i]);
        hi = fmaxf(hi, m);
        if (x0 + 8 * i < n_mem) lo = fminf(lo, m);
      }
      hi = warp_max(hi);
      lo = -warp_max(-lo);
      asm volatile("bar.sync 1, %0;" ::"n"(kC8tConv) : "memory");  // `red` was read
      if (lane == 0) red[warp - 10] = make_float2(hi, lo);
      asm volatile("bar.sync 1, %0;" ::"n"(kC8tConv) : "memory");
#pragma unroll
      for (int i = 0; i < kC8tConv / 32; ++i) {
        hi = fmaxf(hi, red[i].x);
        lo = fminf(lo, red[i].y);
      }
      const bool rows = lo < 0x1p-6f * hi;
      if (wait_slot(j, 0)) {
        const float k = rows || hi == 0.0f ? 1.0f : floor_pow2(hi);
        put_scales(j, make_float4(k, k, k, k), make_float4(1.0f, 1.0f, 1.0f, 1.0f), rows);
        if (rows) {
#pragma unroll
          for (int i = 0; i < M; ++i) {
            float m = largest(w[i]);  // of the row, which sixteen lanes share
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float own = m > 0.0f ? floor_pow2(m) : 1.0f;
            if ((tid & 15) == 0) row_scales(j)[8 * i + (tid >> 4)] = own;
            put_k(i, 1.0f / own);
          }
        } else {
#pragma unroll
          for (int i = 0; i < M; ++i) put_k(i, 1.0f / k);
        }
        landed(j, 0);
      }
      load(1);
      if (wait_slot(j, 1)) {
#pragma unroll
        for (int i = 0; i < M; ++i) put(1, i, w[i]);
        landed(j, 1);
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop, so that addresses and descriptors are warp-uniform values;
    // lane 0 alone issues.
    constexpr uint32_t idesc_s = umma_idesc_f16_f32<kC8tRows, kC8tBlk>();
    constexpr uint32_t idesc_o = umma_idesc_f16_f32<kC8tRows, D>() | (1u << 16);  // B MN-major
    constexpr uint32_t idesc_m = umma_idesc_bf16_f32_bmn<kC8tRows, D>();          // of memory rows
    const int x = warp - 8;
    const int n = x == 0 || act1 ? nblk : 0;
    // descriptors of the first slots; a step adds its offset in units of 16 bytes
    const uint32_t at = smem_u32(sm);
    const uint64_t q_desc = umma_desc_k_sw128(at + x * Sm::kQBytes), k_desc = umma_desc_k_sw128(at + Sm::kK);
    const uint64_t v_desc = umma_desc_mn_sw128(at + Sm::kV, Sm::kKVBytes / 2);
    const uint32_t o = tmem + kC8tTmemO + 128 * x;
    bool ok = n > 0 && __all_sync(0xffffffffu, wait(kCbQ0 + x, 0));
    // S of block j, once K has landed and its buffer is free: the P V two blocks back, which reads
    // P there, has completed
    auto scores = [&](int j) {
      const int s = j % kC8tSlots, u = j & 1;
      ok = ok && __all_sync(0xffffffffu, wait(kCbFullK0 + s, (j / kC8tSlots) & 1) &&
                                             (j < 2 || wait(kCbO0 + 2 * x + u, ((j >> 1) - 1) & 1)));
      if (!ok) return;
      tc05_fence_after();
      const uint64_t kd = k_desc + static_cast<uint32_t>(s * (Sm::kKVBytes >> 4));
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          umma_bf16(tmem + 128 * x + 64 * u, q_desc + ((i >> 2) * kC8tRows * 8 + (i & 3) * 2),
                    kd + ((i >> 2) * kC8tBlk * 8 + (i & 3) * 2), idesc_s, i != 0);
        umma_commit(bar(kCbS0 + 2 * x + u));
        umma_commit(bar(kCbFreeK0 + s));
      }
      __syncwarp();
    };
    for (int j = 0; j < min(2, n); ++j) scores(j);
    for (int j = 0; j < n; ++j) {
      // P V once P is written (and O rescaled) and V has landed, then the S that P's buffer takes
      const int s = j % kC8tSlots, u = j & 1;
      ok = ok && __all_sync(0xffffffffu, wait(kCbFullV0 + s, (j / kC8tSlots) & 1) &&
                                             wait(kCbP0 + 2 * x + u, (j >> 1) & 1));
      if (!ok) break;
      tc05_fence_after();
      const uint64_t vd = v_desc + static_cast<uint32_t>(s * (Sm::kKVBytes >> 4));
      if (lane == 0) {
        const uint32_t pt = tmem + 128 * x + 64 * u;
        if (u0 + j < lb) {
#pragma unroll
          for (int i = 0; i < kC8tBlk / 16; ++i) umma_f16_ts(o, pt + 8 * i, vd + i * 128, idesc_o, (j | i) != 0);
        } else {
#pragma unroll
          for (int i = 0; i < kC8tBlk / 16; ++i) umma_f16_ts(o, pt + 8 * i, vd + i * 128, idesc_m, (j | i) != 0);
#pragma unroll
          for (int i = 0; i < kC8tBlk / 16; ++i) umma_f16_ts(o, pt + 32 + 8 * i, vd + i * 128, idesc_m, 1);
        }
        umma_commit(bar(kCbO0 + 2 * x + u));
        umma_commit(bar(kCbFreeV0 + s));
      }
      __syncwarp();
      if (j + 2 < n) scores(j + 2);
    }
    // every MMA issued here completes before TMEM is freed
    if (lane == 0) {
      umma_commit(bar(kCbDrain + x));
      mbar_wait(bar(kCbDrain + x), 0);
    }
    __syncwarp();
  } else if (warp < 4 || act1) {
    // ------------------------------------------------------------ softmax, tile x
    const int x = warp >> 2, r = threadIdx.x & 127;
    const int col = c0 + x * kC8tRows + r;
    const bool real = col < cols;
    const int vis = real ? column_rows(a, q, col) : 0;  // local rows the column sees
    float m_run = kC8None, l_run = 0.0f, unit = 0.0f;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tmem_s = tmem + 128 * x + lane_base, tmem_o = tmem + kC8tTmemO + 128 * x + lane_base;
    // block j; false after a timeout.  Local and memory blocks have code of their own: in one loop the
    // memory blocks' branches cost the local ones 2%.
    auto block = [&](int j, auto memory) -> bool {
      constexpr bool kMem = decltype(memory)::value;
      const int u = u0 + j;
      if (!__all_sync(0xffffffffu, wait(kCbS0 + 2 * x + (j & 1), (j >> 1) & 1))) return false;
      tc05_fence_after();
      const float4 *sc = reinterpret_cast<const float4 *>(scales + Sm::kScales * (j % (2 * kC8tSlots)));
      const uint32_t at = tmem_s + kC8tBlk * (j & 1);
      if (kMem && sc[2].w != 0.0f) {  // memory rows of very different size
#pragma unroll 1
        for (int i = 0; i < kC8tBlk; i += 16) {
          float y[16];
          tmem_ld16(at + i, y);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] *= row_scales(j)[i + e];
          tmem_st16(at + i, y);
        }
      }
      const float4 us = sc[2];
      // score factors of the groups (positive even where the product underflows, so that a hidden row
      // stays at -inf) and log2 of V's scales over the unit
      float c[NG], r[NG];
      if constexpr (NG == 4) {
        const float4 ks = sc[0], rs = sc[1];
        c[0] = ks.x; c[1] = ks.y; c[2] = ks.z; c[3] = ks.w;
        r[0] = rs.x; r[1] = rs.y; r[2] = rs.z; r[3] = rs.w;
      } else {
        c[0] = sc[0].x;
        r[0] = us.z;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) c[g] = fmaxf(cf * c[g], 1.2e-38f);
      float alpha = 1.0f;  // factor of O's lane
      if (us.x > 0.0f) {   // a larger unit: the reference falls as in Softmax8
        const float k = reference_falls(m_run, l_run, us.x);
        m_run -= k;
        l_run *= pow2_whole(k);
        alpha = pow2_whole(fmaxf(k - us.x, -127.0f));
      }
      unit = us.y;
      const int lim = !kMem ? vis - u * kC8tBlk : real ? n_mem - (u - lb) * kC8tBlk : 0;  // rows seen
      float s[kC8tBlk];
      static_assert(kC8tBlk == 64, "one 64-column TMEM load per block");
      tmem_ld64(at, s);
      if (lim < kC8tBlk) {
#pragma unroll
        for (int i = 0; i < kC8tBlk; ++i) s[i] = i < lim ? s[i] : -INFINITY;
      }
      float top[NG], over = -INFINITY;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        constexpr int NA = NG == 1 ? 4 : 2;
        float mx[NA];
#pragma unroll
        for (int e = 0; e < NA; ++e) mx[e] = -INFINITY;
#pragma unroll
        for (int i = RG * g; i < RG * (g + 1); i += 2 * NA)
#pragma unroll
          for (int e = 0; e < NA; ++e) mx[e] = max3(mx[e], s[i + 2 * e], s[i + 2 * e + 1]);
        top[g] = mx[0];
#pragma unroll
        for (int e = 1; e < NA; ++e) top[g] = fmaxf(top[g], mx[e]);
        top[g] = __fmul_rn(top[g], c[g]);
        over = fmaxf(over, top[g] - m_run + fmaxf(r[g], kC8MinRatio));
      }
      if (over > kC8Slack) {
        float m_new = -INFINITY;
#pragma unroll
        for (int g = 0; g < NG; ++g) m_new = fmaxf(m_new, new_reference(top[g], fmaxf(r[g], kC8MinRatio)));
        const float f = ex2_approx(m_run - m_new);
        m_run = m_new;
        l_run *= f;
        alpha *= f;
      }
      float ref = m_run;
      if (fabsf(ref) > kC8tFar) {
        // far scores: the reference came from a rounded product, so the others are rounded alike, and
        // it leaves them before small terms are added that their rounding would swallow
#pragma unroll
        for (int i = 0; i < kC8tBlk; ++i) s[i] = __fmul_rn(s[i], c[i / RG]) - ref;
#pragma unroll
        for (int g = 0; g < NG; ++g) c[g] = 1.0f;
        ref = 0.0f;
      }
      // the ratios of the scales in the exponent, unless they would take weights out of range
      const bool fold = us.z >= kC8MinFold;
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
        // O's lane follows the reference and the unit, once the last P V has completed (TMEM
        // accesses are warp-collective)
        if (!__all_sync(0xffffffffu, wait(kCbO0 + 2 * x + ((j - 1) & 1), ((j - 1) >> 1) & 1))) return false;
        tc05_fence_after();
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t o[32];
          tmem_ld32(tmem_o + cc, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(tmem_o + cc, o);
        }
      }
      float sum = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        constexpr int NA = NG == 1 ? 2 : 1;
        const float rg = fold ? r[g] : 0.0f, mf = ref - kC8Shift - rg;
        float2 ps[NA];
#pragma unroll
        for (int e = 0; e < NA; ++e) ps[e] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = RG * g; i < RG * (g + 1); i += 2) {
          const float2 e = fma2(make_float2(s[i], s[i + 1]), make_float2(c[g], c[g]), make_float2(-mf, -mf));
          s[i] = ex2_approx(e.x);
          s[i + 1] = ex2_approx(e.y);
          ps[(i >> 1) % NA] = add2(ps[(i >> 1) % NA], make_float2(s[i], s[i + 1]));
        }
        float own = ps[0].x + ps[0].y;
        if constexpr (NA == 2) own += ps[1].x + ps[1].y;
        sum = fmaf(own, pow2_whole(-rg), sum);
      }
      if (!fold) {
#pragma unroll
        for (int i = 0; i < kC8tBlk; ++i) s[i] *= pow2_whole(fmaxf(r[i / RG], -127.0f));
      }
      uint32_t w[32];
      if constexpr (kMem) {  // bf16, the tail behind the head
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          w[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
          s[2 * i] -= __uint_as_float(w[i] << 16);
          s[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
        }
        tmem_st32(at, w);
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
        tmem_st32(at + 32, w);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = pack_f16x2(s[2 * i], s[2 * i + 1]);
        tmem_st32(at, w);  // P over S
      }
      l_run += sum;
      tc05_fence_before();
      mbar_arrive(bar(kCbP0 + 2 * x + (j & 1)));
      return true;
    };
    const int n_local = max(0, min(u1, lb) - u0);
    int j = 0;
    while (j < n_local && block(j, std::false_type{})) ++j;
    bool okw = j == n_local;
    while (okw && j < nblk) okw = block(j++, std::true_type{});
    if (okw && nblk > 0) okw = __all_sync(0xffffffffu, wait(kCbO0 + 2 * x + ((nblk - 1) & 1), ((nblk - 1) >> 1) & 1));
    tc05_fence_after();
    const bool have = okw && nblk > 0;
    const bool one = a.n_split == 1;
    // O in its own unit: over l for the result, times 2^-shift for a split's part
    const float f = l_run == 0.0f ? 0.0f : one ? unit / l_run : unit * exp2f(-kC8Shift);
    // O's rows leave through the warp's part of Q's tile, which no MMA reads any more, 128 bytes of
    // each of the 32 rows at a time: eight lanes write a line (a thread writing its own row: 11,300
    // cycles instead of 7,600)
    const int row = row_of(col);
    uint8_t *buf = sm + x * Sm::kQBytes + 32 * (warp & 3) * 128;
    auto put = [&](int c, const uint4 (&v)[8]) {  // 128-byte part c of this thread's row
      uint8_t *p = buf + (c & 1) * (Sm::kQBytes / 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(p + lane * 128 + ((i ^ (lane & 7)) << 4)) = v[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = 4 * i + (lane >> 3), piece = lane & 7;
        const int64_t to = __shfl_sync(0xffffffffu, row, rr);
        if (c0 + x * kC8tRows + 32 * (warp & 3) + rr >= cols) continue;
        uint8_t *dst = one ? static_cast<uint8_t *>(a.O) + to * D * 2
                           : reinterpret_cast<uint8_t *>(a.part_o + (to * a.n_split + split) * D);
        *reinterpret_cast<uint4 *>(dst + c * 128 + piece * 16) =
            *reinterpret_cast<const uint4 *>(p + rr * 128 + ((piece ^ (rr & 7)) << 4));
      }
    };
#pragma unroll 1
    for (int c = 0; c < (one ? D / 64 : D / 32); ++c) {
      uint4 v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // half a part: 32 elements as bf16, 16 as fp32
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0;
        if (one) {
          if (have) tmem_ld32(tmem_o + 64 * c + 32 * h, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = l_run == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[i]) * f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            auto two = [&](int e) { return pack_bf16x2(__uint_as_float(o[8 * i + e]), __uint_as_float(o[8 * i + e + 1])); };
            v[4 * h + i] = make_uint4(two(0), two(2), two(4), two(6));
          }
        } else if (h == 0) {
          if (have) tmem_ld32(tmem_o + 32 * c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = l_run == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[i]) * f);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      put(c, v);
    }
    if (real) {
      const float l = l_run * exp2f(-kC8Shift);
      if (one) {
        write_stats(a, row, m_run, l);
      } else {
        a.part_ml[(static_cast<int64_t>(row) * a.n_split + split) * 2] = m_run == kC8None ? -INFINITY : m_run;
        a.part_ml[(static_cast<int64_t>(row) * a.n_split + split) * 2 + 1] = l;
      }
    }
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == 8) tmem_dealloc(tmem, kC8tTmemCols);
}

}  // namespace msa
