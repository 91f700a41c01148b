// cache8.cuh -- the 8-bit local cache: append (quantise), read (dequantise)
// and eviction by accumulated attention weight.
//
// A block of block_len rows of one (query, kv head) shares one scale, the
// smallest power of two s with max|x| <= qmax * s.  Powers of two make x / s
// and q * s exact in fp32, so the only rounding is the one to the format; a
// block whose scale grows rounds its earlier rows again at steps that at least
// double, so the roundings of an element sum to at most one final step.  An
// amax / qmax scale would halve the step at best, but let every small growth
// add half a step to every earlier row.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"
#include "ptx.cuh"

namespace msa {

// ---------------------------------------------------------------- formats
template <int FMT> struct Fmt8;

template <> struct Fmt8<MSA_CACHE_INT8> {
  static constexpr float kMax = 127.0f;
  // four values, each already divided by the scale -> four bytes
  static __device__ __forceinline__ uint32_t pack4(const float v[4]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w |= (static_cast<uint32_t>(__float2int_rn(v[i])) & 0xffu) << (8 * i);
    return w;
  }
  static __device__ __forceinline__ void unpack4(uint32_t w, float v[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)  // the bits of 2^23 + (q + 128), less 2^23 + 128
      v[i] = __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7650 + i)) - 8388736.0f;
  }
};

template <> struct Fmt8<MSA_CACHE_E4M3> {
  static constexpr float kMax = 448.0f;
  static __device__ __forceinline__ uint32_t pack4(const float v[4]) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  static __device__ __forceinline__ void unpack4(uint32_t w, float v[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};

// The smallest power of two s with amax <= kMax * s (at least 2^-126, so that
// 1 / s is finite); 0 for amax = 0.  amax is finite.
template <int FMT>
__device__ __forceinline__ float block_scale(float amax) {
  if (amax == 0.0f) return 0.0f;
  // amax = 1.m 2^e and kMax = 1.n 2^q: the exponent e - q, one more where m > n
  constexpr int q = FMT == MSA_CACHE_INT8 ? 6 : 8, n = FMT == MSA_CACHE_INT8 ? 0x7e0000 : 0x600000;
  static_assert(Fmt8<FMT>::kMax == (1.0f + n / 8388608.0f) * (1 << q), "the format's largest value");
  const int bits = __float_as_int(amax);
  const int e = max((bits >> 23) - q + ((bits & 0x7fffff) > n ? 1 : 0), 1);  // biased
  return __int_as_float(e << 23);
}

// What is stored of a value: NaN as 0, an infinity as the block's largest value.
template <int FMT>
__device__ __forceinline__ float to_grid(float x, float inv) {
  if (!isfinite(x)) return x != x ? 0.0f : copysignf(Fmt8<FMT>::kMax, x);
  return x * inv;
}
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;
}

// 16 consecutive elements as they lie in memory (64 or 32 bytes, 16-byte aligned), and as floats.
template <typename T>
struct Raw16 {
  static constexpr int N = sizeof(T);  // 16-byte pieces (sizeof(T) * 16 / 16)
  uint4 x[N];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = *(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void get(float v[16]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + j] = __uint_as_float(w[j]);
        } else {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    }
  }
  // The largest magnitude's bits as fp32: magnitudes order like integers, infinities and NaN above
  // all finite ones.
  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4)
          m = max(m, w[j] & 0x7fffffffu);
        else
          asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j] & 0x7fff7fffu));
      }
    }
    if constexpr (sizeof(T) == 2) m = max(m & 0xffff0000u, m << 16);
    return m;
  }
};
constexpr uint32_t kInfBits = 0x7f800000u;

template <typename T>
__device__ __forceinline__ void store16(T *p, const float v[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) store4(p + 4 * i, v + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 x;
      x.x = pack_bf16x2(v[8 * i], v[8 * i + 1]);
      x.y = pack_bf16x2(v[8 * i + 2], v[8 * i + 3]);
      x.z = pack_bf16x2(v[8 * i + 4], v[8 * i + 5]);
      x.w = pack_bf16x2(v[8 * i + 6], v[8 * i + 7]);
      *reinterpret_cast<uint4 *>(p + 8 * i) = x;
    }
  }
}
// 16 values / scale as bytes.  `finite`: none is infinite or NaN.
template <int FMT>
__device__ __forceinline__ uint4 pack16(const float v[16], float inv, bool finite) {
  if (FMT == MSA_CACHE_INT8 && finite) {
    // adding 1.5 * 2^23 rounds to a whole number, ties to even, in the low bits of the sum
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(fmaf(v[4 * i + j], inv, 12582912.0f));
      w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = finite ? v[4 * i + j] * inv : to_grid<FMT>(v[4 * i + j], inv);
    w[i] = Fmt8<FMT>::pack4(y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int FMT>
__device__ __forceinline__ void unpack16(uint4 x, float s, float v[16]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Fmt8<FMT>::unpack4(w[i], v + 4 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] *= s;
  }
}

// The rows a call appends to query b: start, count; false (and flagged by
// `report`) when they are out of range.
struct AppendRange {
  int start, count;
};
__device__ __forceinline__ bool append_range(const int32_t *start, const int32_t *cache_len,
                                             const int32_t *n_tokens, int b, int tokens, int cap,
                                             bool report, AppendRange &r) {
  r.start = start ? start[b] : cache_len[b];
  r.count = n_tokens ? n_tokens[b] : tokens;
  const bool ok = r.start >= 0 && r.start <= cap && r.count >= 0 && r.count <= tokens;
  if (report && !ok) raise_device_error(MSA_DEVERR_BAD_LENGTH);
  if (report && ok && r.count > cap - r.start) raise_device_error(MSA_DEVERR_CACHE_OVERFLOW);
  return ok;
}

__device__ __forceinline__ int append_end(const AppendRange &r, int cap) {
  return r.count > cap - r.start ? cap : r.start + r.count;
}

// ---------------------------------------------------------------- append
struct AppendArgs {
  const void *K, *V;
  int64_t kb, kt, vb, vt;  // batch and token strides, elements
  int tokens, H_kv, cap, bl, bl_shift;
  uint8_t *k8, *v8;
  float *ks, *vs;
  int32_t *cache_len;
  const int32_t *n_tokens, *start;
  float *weights;
};

// grid (ceil(2 * H_kv / units), blocks a query can touch, B), block 256: UT threads (a unit)
// quantise the new rows of one block of one head of K or V.  A task is 16 elements of a row, NT
// tasks a thread, so the block's new rows stay in registers, packed as they came, between the
// maximum and the rounding.  Bound by the bytes of the rows (64 x 1,000 tokens of 8 heads of 128:
// 54 us, 83% of the measured copy bandwidth; unpacked to fp32 at once it held a third of the CTAs
// and took 97).  set_len: write the new cache_len here (start given: no CTA reads cache_len).
template <typename T, int D, int FMT, int NT, int UT>
__global__ void __launch_bounds__(256, sizeof(T) * NT <= 4 ? 6 : 3)
cache8_append_kernel(AppendArgs a, int set_len) {
  constexpr int CPR = D / 16;
  __shared__ uint32_t red[8];
  griddep_wait();
  griddep_launch();
  // unit 2 h + which; the CTA's last units may lie past the heads and then only take the barriers
  const int tid = threadIdx.x % UT, unit = blockIdx.x * (256 / UT) + threadIdx.x / UT;
  const bool on = unit < 2 * a.H_kv;
  const int h = on ? unit >> 1 : 0, which = unit & 1, b = blockIdx.z;
  const bool first = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  AppendRange r;
  if (!append_range(a.start, a.cache_len, a.n_tokens, b, a.tokens, a.cap, first, r)) return;
  const int end = append_end(r, a.cap);
  if (first && set_len) a.cache_len[b] = end;
  const int blk = (r.start >> a.bl_shift) + blockIdx.y;
  const int x0 = blk * a.bl;  // first row of the block
  if (x0 >= end) return;
  const int lo = max(x0, r.start), hi = on ? min(x0 + a.bl, end) : lo;  // new rows [lo, hi)
  const T *src = static_cast<const T *>(which ? a.V : a.K) + b * (which ? a.vb : a.kb) +
                 static_cast<int64_t>(h) * D;
  const int64_t ts = which ? a.vt : a.kt;
  const int64_t bh = static_cast<int64_t>(b) * a.H_kv + h;
  uint8_t *dst = (which ? a.v8 : a.k8) + (bh * a.cap + x0) * D;
  float *scale = (which ? a.vs : a.ks) + bh * (a.cap >> a.bl_shift) + blk;
  Raw16<T> v[NT];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int task = tid + UT * u, row = x0 + task / CPR;
    if (row >= lo && row < hi) v[u].load(src + (row - r.start) * ts + (task % CPR) * 16);
  }
  const float s_old = lo > x0 ? *scale : 0.0f;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int row = x0 + (tid + UT * u) / CPR;
    if (row >= lo && row < hi) top = max(top, v[u].amax_bits());
  }
  auto cta_max = [&](uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
    __syncthreads();  // (every thread has read the old scale, too)
#pragma unroll
    for (int w = 0; w < UT / 32; ++w) m = max(m, red[threadIdx.x / UT * (UT / 32) + w]);
    return m;
  };
  top = cta_max(top);
  const bool finite = top < kInfBits;
  // the largest finite magnitude (units that share a CTA take the barrier together)
  if (UT == 256 ? !finite : __syncthreads_or(!finite) != 0) {
    top = 0;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int row = x0 + (tid + UT * u) / CPR;
      if (row >= lo && row < hi) {
        float x[16];
        v[u].get(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(finite_abs(x[i])));
      }
    }
    __syncthreads();
    top = cta_max(top);
  }
  const float s = fmaxf(block_scale<FMT>(__uint_as_float(top)), s_old);
  const float inv = s > 0.0f ? 1.0f / s : 0.0f;
  if (!on) return;
  if (tid == 0 && (s != s_old || lo == x0)) *scale = s;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int task = tid + UT * u, row = x0 + task / CPR;
    uint4 *p = reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(task) * 16);
    if (row >= lo && row < hi) {
      float x[16];
      v[u].get(x);
      *p = pack16<FMT>(x, inv, finite);
    } else if (row < lo && s > s_old) {  // earlier rows of a block whose scale grew
      float old[16];
      unpack16<FMT>(*p, s_old, old);
      *p = pack16<FMT>(old, inv, true);
    }
  }
  if (a.weights && which == 0)
    for (int x = lo + tid; x < hi; x += UT) a.weights[bh * a.cap + x] = 0.0f;
}

// cache_len after an append at cache_len (start NULL): every CTA of the append has read it.
__global__ void cache8_advance_kernel(int32_t *__restrict__ cache_len,
                                      const int32_t *__restrict__ n_tokens, int B, int tokens,
                                      int cap) {
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  AppendRange r;
  if (append_range(nullptr, cache_len, n_tokens, b, tokens, cap, false, r))
    cache_len[b] = append_end(r, cap);
}

// ---------------------------------------------------------------- read
// grid (ceil(rows * H_kv * D / 16 / 256), 2, B): 16 elements a thread, token-major out.  Bound by the
// bytes, two thirds of them written.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(256)
cache8_read_kernel(const uint8_t *__restrict__ k8, const uint8_t *__restrict__ v8,
                   const float *__restrict__ ks, const float *__restrict__ vs,
                   const int32_t *__restrict__ cache_len, const int32_t *__restrict__ begin,
                   int rows, int H_kv, int cap, int bl_shift, T *__restrict__ K, T *__restrict__ V) {
  constexpr int CPR = D / 16;
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.z;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;  // (the host keeps the pieces of a query below 2^31)
  if (i >= static_cast<uint32_t>(rows) * H_kv * CPR) return;
  const int c = i % CPR, x = i / CPR / static_cast<uint32_t>(H_kv), h = i / CPR - x * H_kv;
  const int64_t row = static_cast<int64_t>(begin ? begin[b] : 0) + x;
  const int len = min(cache_len[b], cap);
  float v[16];
  if (row >= 0 && row < len) {
    const int64_t bh = static_cast<int64_t>(b) * H_kv + h;
    const uint8_t *src = (blockIdx.y ? v8 : k8) + (bh * cap + row) * D + c * 16;
    const float s = (blockIdx.y ? vs : ks)[bh * (cap >> bl_shift) + (row >> bl_shift)];
    unpack16<FMT>(*reinterpret_cast<const uint4 *>(src), s, v);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
  }
  store16((blockIdx.y ? V : K) + (static_cast<int64_t>(b) * rows * H_kv * CPR + i) * 16, v);
}

// ---------------------------------------------------------------- evict
constexpr int kSelThreads = 512;

// An order-preserving key of a block's summed weight; a NaN is the lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// What an eviction keeps of one query: full blocks, recent ones among them, new length.  The host
// keeps budget and recent within the capacity; 0 <= recent <= keep <= full, so the list of kept
// blocks fits its nb + 1 entries.
struct EvictPlan {
  int len, full, tail, keep, recent, new_len;
};
__device__ __forceinline__ EvictPlan evict_plan(int len, int cap, int bl, int budget, int recent) {
  EvictPlan p;
  p.len = max(0, min(len, cap));
  p.full = p.len / bl;
  p.tail = p.len % bl;
  p.keep = p.len > budget ? (budget - p.tail) / bl : p.full;
  p.recent = min(recent / bl + (recent % bl != 0 ? 1 : 0), p.keep);
  p.new_len = p.keep * bl + p.tail;
  return p;
}

// Exclusive prefix count of `flag` over the CTA's threads; *total gets the sum.
__device__ __forceinline__ int cta_prefix(bool flag, int *warp_sums, int *total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  if (lane == 0) warp_sums[warp] = __popc(m);
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const int n = warp_sums[w];
    before += w < warp ? n : 0;
    sum += n;
  }
  __syncthreads();
  *total = sum;
  return before + __popc(m & ((1u << lane) - 1));
}

// grid (B * H_kv), block kSelThreads: which blocks stay, in order -> src_block[bh][0 .. keep).
// A block's weight is summed in 64 bits and compared in 32, so the choice does not hang on the
// order of the sum.  The keep - recent heaviest of the older blocks: a radix select over the keys
// (four passes of 8 bits) finds the smallest kept key, then one pass in block order keeps all
// larger keys and the first of the equal ones.  The keys lie in shared memory where they fit
// (smem_keys), else in the workspace.  Bound by latency: a dozen barriers of one CTA a head.
__global__ void __launch_bounds__(kSelThreads)
cache8_select_kernel(const float *__restrict__ weights, const int32_t *__restrict__ cache_len,
                     int H_kv, int cap, int bl, int budget, int recent, int smem_keys,
                     uint32_t *__restrict__ keys, int32_t *__restrict__ src_block,
                     int32_t *__restrict__ lens) {
  extern __shared__ uint32_t key_sm[];
  __shared__ int hist[256];
  __shared__ int warp_sums[kSelThreads / 32];
  __shared__ int digit, above;
  griddep_wait();
  griddep_launch();
  const int64_t bh = blockIdx.x;
  const int b = blockIdx.x / H_kv, nb = cap / bl;
  const EvictPlan p = evict_plan(cache_len[b], cap, bl, budget, recent);
  if (blockIdx.x % H_kv == 0 && threadIdx.x == 0) {
    lens[2 * b] = p.len;
    lens[2 * b + 1] = p.new_len;
    if (p.len != cache_len[b]) raise_device_error(MSA_DEVERR_BAD_LENGTH);
  }
  int32_t *src = src_block + bh * (nb + 1);
  uint32_t *key = smem_keys ? key_sm : keys + bh * nb;
  const int old = p.full - p.recent;     // blocks that compete
  const int want = p.keep - p.recent;    // of which these stay
  if (threadIdx.x == 0 && p.tail > 0) src[p.keep] = p.full;
  for (int j = threadIdx.x; j < p.recent; j += kSelThreads) src[want + j] = old + j;
  if (want == old) {
    for (int j = threadIdx.x; j < old; j += kSelThreads) src[j] = j;
    return;
  }
  if (want == 0) return;
  const int lane = threadIdx.x % 32;
  {
    // bl / 4 neighbouring lanes sum a block
    const int per = bl / 4, blocks = kSelThreads / per;
    const float4 *w = reinterpret_cast<const float4 *>(weights + bh * cap);
    for (int j0 = 0; j0 < old; j0 += blocks) {  // (whole warps stay together)
      const int j = j0 + threadIdx.x / per;
      double s = 0.0;
      if (j < old) {
        const float4 x = w[static_cast<int64_t>(j) * per + threadIdx.x % per];
        s = (static_cast<double>(x.x) + x.y) + (static_cast<double>(x.z) + x.w);
      }
      for (int o = per / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (j < old && threadIdx.x % per == 0) key[j] = weight_key(static_cast<float>(s));
    }
  }
  uint32_t prefix = 0, mask = 0;
  int left = want;  // the left-th largest key among those that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();  // (and the keys are written)
    for (int j = threadIdx.x; j < old; j += kSelThreads)
      if ((key[j] & mask) == prefix) atomicAdd(&hist[(key[j] >> shift) & 255], 1);
    __syncthreads();
    if (threadIdx.x < 32) {
      // eight digits a lane, from the largest down; lanes before this one hold larger digits
      int n[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] = hist[255 - 8 * lane - i];
        sum += n[i];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < left && before + n[i] >= left) {
          digit = 255 - 8 * lane - i;
          above = before;
        }
        before += n[i];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(digit) << shift;
    mask |= 255u << shift;
    left -= above;
    __syncthreads();
  }
  // `prefix` is the smallest kept key, `left` of the blocks that have it stay (the first ones)
  int kept = 0, equal = 0;
  for (int j0 = 0; j0 < old; j0 += kSelThreads) {
    const int j = j0 + threadIdx.x;
    const uint32_t x = j < old ? key[j] : 0u;
    int n;
    const bool eq = j < old && x == prefix;
    const int e = equal + cta_prefix(eq, warp_sums, &n);
    equal += n;
    const bool keep = j < old && (x > prefix || (eq && e < left));
    const int d = kept + cta_prefix(keep, warp_sums, &n);
    kept += n;
    if (keep) src[d] = j;
  }
}

struct EvictMove {
  const uint8_t *k8, *v8;
  const float *ks, *vs, *w;
  uint8_t *ok8, *ov8;
  float *oks, *ovs, *ow;
  int32_t *out_len;
  int H_kv, cap, out_cap, bl, D;
};

// grid (ceil(streams / 128), B * H_kv, parts), block 128.  Blocks move as units, so every piece of
// a block (16 bytes of K, V or the weights, one scale) is a stream of its own along the kept
// blocks, owned by one thread.  Destinations never lie behind their sources and a thread loads a
// wave before it stores it, so in place (one part) needs no synchronisation at all: a wave's
// stores reach only blocks at or below sources that the same thread has loaded.  Into another
// cache the kept blocks are split over `parts`.
constexpr int kMoveWave = 8;
__global__ void __launch_bounds__(128)
cache8_move_kernel(EvictMove m, const int32_t *__restrict__ src_block,
                   const int32_t *__restrict__ lens, int in_place) {
  griddep_wait();
  griddep_launch();
  const int64_t bh = blockIdx.y;
  const int b = blockIdx.y / m.H_kv, nb = m.cap / m.bl;
  const int new_len = lens[2 * b + 1];
  const int32_t *src = src_block + bh * (nb + 1);
  const int pieces = m.bl * m.D / 16, wp = m.bl / 4;
  const int s = blockIdx.x * 128 + threadIdx.x;
  if (s == 0 && blockIdx.y % m.H_kv == 0 && blockIdx.z == 0) m.out_len[b] = new_len;
  const int live = (new_len + m.bl - 1) / m.bl;  // blocks written
  const int per = (live + gridDim.z - 1) / gridDim.z;
  const int j0 = blockIdx.z * per, j1 = min(live, j0 + per);
  const int tail = new_len % m.bl;
  if (s >= 2 * pieces + wp + 2) return;
  if (s < 2 * pieces + wp) {
    const uint8_t *in;
    uint8_t *out;
    int64_t block_bytes;
    int piece, row;
    if (s < 2 * pieces) {
      const bool v = s >= pieces;
      piece = v ? s - pieces : s;
      row = piece * 16 / m.D;
      block_bytes = static_cast<int64_t>(m.bl) * m.D;
      in = (v ? m.v8 : m.k8) + bh * m.cap * m.D;
      out = (v ? m.ov8 : m.ok8) + bh * m.out_cap * m.D;
    } else {
      piece = s - 2 * pieces;
      row = piece * 4;
      block_bytes = static_cast<int64_t>(m.bl) * 4;
      in = reinterpret_cast<const uint8_t *>(m.w + bh * m.cap);
      out = reinterpret_cast<uint8_t *>(m.ow + bh * m.out_cap);
    }
    const bool is_w = s >= 2 * pieces;
    in += piece * 16;
    out += piece * 16;
    for (int j = j0; j < j1; j += kMoveWave) {
      uint4 x[kMoveWave];
      bool go[kMoveWave];
#pragma unroll
      for (int u = 0; u < kMoveWave; ++u) {
        go[u] = false;
        if (j + u < j1) {
          const int from = src[j + u];
          // the partial last block: its rows alone
          go[u] = !(in_place && from == j + u) && !(tail && j + u == live - 1 && row >= tail);
          if (go[u]) x[u] = *reinterpret_cast<const uint4 *>(in + from * block_bytes);
        }
      }
#pragma unroll
      for (int u = 0; u < kMoveWave; ++u)
        if (go[u]) {
          if (is_w && tail && j + u == live - 1) {  // four rows' weights, the live ones of them
            float *o = reinterpret_cast<float *>(out + (j + u) * block_bytes);
            const uint32_t y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (row + i < tail) o[i] = __uint_as_float(y[i]);
          } else {
            *reinterpret_cast<uint4 *>(out + (j + u) * block_bytes) = x[u];
          }
        }
    }
    if (is_w && blockIdx.z == gridDim.z - 1) {
      // the weights of rows that the query no longer holds (this thread has loaded every weight
      // that may lie there)
      const int end = min(lens[2 * b], m.out_cap);
      float *o = m.ow + bh * m.out_cap;
      for (int j = tail ? live - 1 : live; j * m.bl < end; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = j * m.bl + row + i;
          if (x >= new_len && x < end) o[x] = 0.0f;
        }
    }
    return;
  }
  const bool v = s == 2 * pieces + wp + 1;
  const float *in = (v ? m.vs : m.ks) + bh * nb;
  float *out = (v ? m.ovs : m.oks) + bh * (m.out_cap / m.bl);
  for (int j = j0; j < j1; j += kMoveWave) {
    float x[kMoveWave];
#pragma unroll
    for (int u = 0; u < kMoveWave; ++u)
      if (j + u < j1) x[u] = in[src[j + u]];
#pragma unroll
    for (int u = 0; u < kMoveWave; ++u)
      if (j + u < j1) out[j + u] = x[u];
  }
}

}  // namespace msa
