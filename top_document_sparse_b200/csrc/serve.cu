// serve.cu -- the C ABI (include/msa.h) of the rotary positions and of the
// 8-bit local cache: host-side validation and launches.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

#include "host.cuh"

#include "cache8.cuh"
#include "cache8_attend.cuh"
#include "cache8_prefill_tc.cuh"
#include "cache8_weight_tc.cuh"
#include "rope.cuh"

using namespace msa_host;

struct msa_rope {
  int D = 0, r = 0, layout = 0, device = 0;
  float magnitude = 1.0f;
  uint64_t *d_freq = nullptr;  // [r / 2], 2^-64 turns a position
};

namespace msa_host {

cudaError_t take_serve_error(unsigned int *bits, cudaStream_t st) {
  static const unsigned int zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbolAsync(bits, msa::g_device_error, sizeof(*bits), 0,
                                                  cudaMemcpyDeviceToHost, st);
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbolAsync(msa::g_device_error, &zero, sizeof(zero), 0,
                                 cudaMemcpyHostToDevice, st);
}

}  // namespace msa_host

namespace {

cudaStream_t to_stream(msa_stream s) { return reinterpret_cast<cudaStream_t>(s); }

// Let `kern` use `bytes` of dynamic shared memory.  The attribute is set when it first has to grow
// on a device and remembered, not set at every call.
template <typename K>
cudaError_t allow_smem(K kern, int bytes) {
  struct Known {
    const void *kern;
    int device, bytes;
  };
  static std::mutex mu;
  static Known known[256];
  static int n = 0;
  if (bytes <= 48 * 1024) return cudaSuccess;  // no opt-in needed
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const void *key = reinterpret_cast<const void *>(kern);
  std::lock_guard<std::mutex> lock(mu);
  Known *k = nullptr;
  for (int i = 0; i < n; ++i)
    if (known[i].kern == key && known[i].device == dev) k = &known[i];
  if (k && k->bytes >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  if (!k && n < 256) k = &(known[n++] = Known{key, dev, 0});
  if (k) k->bytes = bytes;
  return cudaSuccess;
}

// The tables of a handle are on the device that was current at its creation.
msa_status current_device(int device, const char *what) {
  int dev = 0;
  MSA_CUDA(cudaGetDevice(&dev));
  if (dev != device)
    return fail(MSA_ERR_INVALID_ARG, "the %s is on device %d, the current device is %d", what, device, dev);
  return MSA_OK;
}

// ---------------------------------------------------------------- rotary positions
msa_status rope_frequencies(const msa_rope_config *c, std::vector<uint64_t> &freq, float *magnitude) {
  const int r = c->rotary_dim;
  const double two_pi = 6.283185307179586476925;
  double theta = c->theta, mag = 1.0, low = 0.0, high = 0.0;
  if (c->scaling == MSA_ROPE_NTK) theta *= std::pow(c->factor, static_cast<double>(r) / (r - 2));
  if (c->scaling == MSA_ROPE_YARN) {
    // the pair index whose wavelength fits original_length `turns` times
    auto index = [&](double turns) {
      return r * std::log(static_cast<double>(c->original_length) / (turns * two_pi)) /
             (2.0 * std::log(c->theta));
    };
    low = std::max(std::floor(index(32.0)), 0.0);
    high = std::min(std::ceil(index(1.0)), static_cast<double>(r - 1));
    mag = 0.1 * std::log(c->factor) + 1.0;
  }
  freq.resize(r / 2);
  for (int i = 0; i < r / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / r);
    if (c->scaling == MSA_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == MSA_ROPE_YARN) {
      // (high <= 0: not even pair 0 turns once)
      const double ramp = high <= 0.0 ? 1.0 : std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
      f = f / c->factor * ramp + f * (1.0 - ramp);
    }
    const long double turns = static_cast<long double>(f) / 6.283185307179586476925286766559L;
    freq[i] = static_cast<uint64_t>(turns * 18446744073709551616.0L + 0.5L);  // f <= 1: < 2^62
  }
  *magnitude = static_cast<float>(c->magnitude != 0.0 ? c->magnitude : mag);
  return MSA_OK;
}

template <typename T, int V, bool INTER>
msa_status launch_rope(const msa_rope *rope, int64_t tokens, const int64_t *pos, int inverse,
                       const msa::RopeSide &q, const msa::RopeSide &k, bool copy_rest,
                       cudaStream_t st) {
  const int half = rope->r / 2;
  const int rot = (V == 1 || !INTER) ? half / V : rope->r / V;
  const int rest = copy_rest ? (rope->D - rope->r) / V : 0;
  // Small CTAs overlap one another's angles and copies best: 16,384 tokens of 40 heads of 128 take
  // 60 us at 64 threads, 64 at 128, 66 at 160, 68 to 84 at 256.  With few tokens a thread a task is
  // faster (64 tokens: 2.1 us at 320 threads, 3.8 at 64).  A CTA takes tokens for five tasks a thread
  // (75,000 tokens of 3 heads of 64, half of each rotated: 20 us, with one task 27; 30,000 fp32 tokens
  // of 10 heads of 64: 30, with four 35), but 16 at most, whose angles take longer than a lone head's
  // copies (100,000 tokens of one head of 64: 15 us, with 40 tokens 21).
  const int per_token = (q.heads + k.heads) * (rot + rest);
  const bool few = tokens * round32(per_token) < 2048LL * num_sms();
  const int tok = std::max(1, std::min(16, (few ? 256 : 320) / per_token));
  const int threads = few ? std::min(round32(tok * per_token), msa::kRopeThreads) : 64;
  const int64_t grid = (tokens + tok - 1) / tok;
  if (grid > 0x7FFFFFFF) return fail(MSA_ERR_UNSUPPORTED, "too many tokens");
  MSA_CUDA(launch_pdl(msa::rope_kernel<T, V, INTER>, dim3(static_cast<unsigned>(grid)),
                      dim3(threads), static_cast<size_t>(tok) * half * sizeof(float2), st,
                      static_cast<const uint64_t *>(rope->d_freq), rope->r, rope->D,
                      rope->magnitude, inverse, pos, tokens, tok, q, k, rot, rot + rest));
  MSA_LAUNCHED("rope_kernel");
  return MSA_OK;
}

template <typename T>
msa_status dispatch_rope(const msa_rope *rope, int64_t tokens, const int64_t *pos, int inverse,
                         const msa::RopeSide &q, const msa::RopeSide &k, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  bool vec = rope->D % V == 0 && rope->r % V == 0 && (rope->layout == MSA_ROPE_INTERLEAVED || rope->r / 2 % V == 0);
  bool rest = false;
  for (const msa::RopeSide *s : {&q, &k}) {
    if (s->heads == 0) continue;
    vec = vec && aligned16(s->in) && aligned16(s->out) && s->in_stride % V == 0 && s->out_stride % V == 0;
    rest = rest || s->in != s->out;
  }
  rest = rest && rope->r < rope->D;
  if (rope->layout == MSA_ROPE_INTERLEAVED)
    return vec ? launch_rope<T, V, true>(rope, tokens, pos, inverse, q, k, rest, st)
               : launch_rope<T, 1, true>(rope, tokens, pos, inverse, q, k, rest, st);
  return vec ? launch_rope<T, V, false>(rope, tokens, pos, inverse, q, k, rest, st)
             : launch_rope<T, 1, false>(rope, tokens, pos, inverse, q, k, rest, st);
}

// ---------------------------------------------------------------- 8-bit cache
// Shape checks of every msa_cache8_* call; they run before anything is enqueued.
msa_status cache8_check(const msa_memory *mem, const msa_cache8 *c) {
  if (!mem || !c) return fail(MSA_ERR_INVALID_ARG, "null memory or cache");
  if (c->batch < 1 || c->batch > 65535)
    return fail(MSA_ERR_INVALID_ARG, "batch=%d must be in [1, 65535]", c->batch);
  if (c->block_len != 16 && c->block_len != 32 && c->block_len != 64 && c->block_len != 128)
    return fail(MSA_ERR_INVALID_ARG, "block_len=%d must be 16, 32, 64 or 128", c->block_len);
  if (c->capacity < 1 || c->capacity % c->block_len != 0)
    return fail(MSA_ERR_INVALID_ARG, "capacity=%d must be a positive multiple of block_len=%d",
                c->capacity, c->block_len);
  if (c->format != MSA_CACHE_INT8 && c->format != MSA_CACHE_E4M3)
    return fail(MSA_ERR_INVALID_ARG, "format must be MSA_CACHE_INT8 or MSA_CACHE_E4M3");
  if (static_cast<int64_t>(c->batch) * mem->H_kv > 65535)
    return fail(MSA_ERR_UNSUPPORTED, "batch * n_kv_heads = %lld exceeds 65535",
                (long long)c->batch * mem->H_kv);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->cache_len)
    return fail(MSA_ERR_INVALID_ARG, "null cache buffer");
  const msa_status on = current_device(mem->device, "memory");
  if (on != MSA_OK) return on;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
      !aligned16(c->weights))
    return fail(MSA_ERR_INVALID_ARG, "cache buffers must be 16-byte aligned");
  return MSA_OK;
}

int block_shift(const msa_cache8 *c) {
  return c->block_len == 16 ? 4 : c->block_len == 32 ? 5 : c->block_len == 64 ? 6 : 7;
}

template <typename T, int D, int FMT>
msa_status launch_append(const msa::AppendArgs &a, int B, bool set_len, cudaStream_t st) {
  const int tasks = a.bl * D / 16;
  const int blocks = static_cast<int>(
      std::min<int64_t>((static_cast<int64_t>(a.tokens) + a.bl - 2) / a.bl + 1, a.cap / a.bl + 1));
  if (blocks > 65535) return fail(MSA_ERR_UNSUPPORTED, "too many tokens for one append");
  const int units = std::max(1, 256 / tasks);  // (head, K or V) pairs a CTA
  const dim3 grid((2 * a.H_kv + units - 1) / units, blocks, B);
  auto kern = tasks == 64    ? msa::cache8_append_kernel<T, D, FMT, 1, 64>
              : tasks == 128 ? msa::cache8_append_kernel<T, D, FMT, 1, 128>
              : tasks == 256 ? msa::cache8_append_kernel<T, D, FMT, 1, 256>
              : tasks == 512 ? msa::cache8_append_kernel<T, D, FMT, 2, 256>
                             : msa::cache8_append_kernel<T, D, FMT, 4, 256>;
  MSA_CUDA(launch_pdl(kern, grid, dim3(256), 0, st, a, set_len ? 1 : 0));
  MSA_LAUNCHED("cache8_append_kernel");
  if (!set_len) {
    MSA_CUDA(launch_pdl(msa::cache8_advance_kernel, dim3((B + 255) / 256), dim3(256), 0, st,
                        a.cache_len, a.n_tokens, B, a.tokens, a.cap));
    MSA_LAUNCHED("cache8_advance_kernel");
  }
  return MSA_OK;
}

template <typename T, int D, int FMT>
msa_status launch_read(const msa_cache8 *c, const int32_t *begin, int rows, int H_kv, void *K,
                       void *V, cudaStream_t st) {
  const int64_t n = (static_cast<int64_t>(rows) * H_kv * (D / 16) + 255) / 256;
  if (n > 0x7FFFFF) return fail(MSA_ERR_UNSUPPORTED, "too many rows for one read");
  MSA_CUDA(launch_pdl(msa::cache8_read_kernel<T, D, FMT>, dim3(static_cast<unsigned>(n), 2, c->batch),
                      dim3(256), 0, st, static_cast<const uint8_t *>(c->k),
                      static_cast<const uint8_t *>(c->v), static_cast<const float *>(c->k_scale),
                      static_cast<const float *>(c->v_scale),
                      static_cast<const int32_t *>(c->cache_len), begin, rows, H_kv, c->capacity,
                      block_shift(c), static_cast<T *>(K), static_cast<T *>(V)));
  MSA_LAUNCHED("cache8_read_kernel");
  return MSA_OK;
}

// kernel template arguments (element type, head dim, format) from run-time values
template <typename F>
msa_status dispatch8(const msa_memory *mem, int format, F &&f) {
  auto fmt = [&](auto t, auto d) {
    return format == MSA_CACHE_INT8 ? f(t, d, std::integral_constant<int, MSA_CACHE_INT8>{})
                                    : f(t, d, std::integral_constant<int, MSA_CACHE_E4M3>{});
  };
  auto dim = [&](auto t) {
    return mem->D == 128 ? fmt(t, std::integral_constant<int, 128>{})
                         : fmt(t, std::integral_constant<int, 64>{});
  };
  return mem->dtype == MSA_BF16 ? dim(__nv_bfloat16{}) : dim(float{});
}

// Columns (token, head) of one kv head share an MMA's 8, 16 or 32 columns; more go to further CTAs.
// (fp32 at most 16: its heads and tails take twice the registers)
int attend8_nt(msa_dtype t, int64_t cols) { return cols <= 8 ? 1 : cols <= 16 || t == MSA_F32 ? 2 : 4; }

struct Attend8Plan {
  int n_split = 1, loc_split = 1, col_tiles = 1, table_cap = 0;
  bool tc = false;  // tcgen05: col_tiles is then the number of tile pairs
  size_t part_o = 0, part_ml = 0, ml = 0, scores = 0, q16 = 0, factor = 0, bytes = 0;
  int score_w = 0;
  bool weight_tc = false;
};

// Columns from which the weights' second pass runs on tcgen05, which takes tiles of 128 of them.
// tcgen05 against mma.sync: at 96 columns 14 against 21 us for one shape of 8,192 rows and 89 against
// 97 us for 16 of 4,096 (D = 64: 12 against 15 and 71 against 82); at 48 columns 14 against 16 us and
// 88 against 66 us.
constexpr int64_t kWeightTcCols = 96;

// Partial results of the splits, and the softmaxes' statistics where weights are tracked.
void plan_attend8_scratch(Attend8Plan &p, const msa_memory *mem, const msa_cache8 *c, size_t rows) {
  if (p.n_split > 1) {
    p.part_ml = round256(rows * p.n_split * mem->D * 4);
    p.bytes = p.part_ml + round256(rows * p.n_split * 2 * 4);
  }
  p.ml = p.bytes;
  if (c->weights) {
    p.bytes += round256(rows * 8);
    const size_t cols = rows / c->batch / mem->H_kv;
    if (cols <= 16) {
      p.score_w = cols <= 4 ? 4 : cols <= 8 ? 8 : 16;
      p.scores = p.bytes;
      p.bytes += round256(static_cast<size_t>(c->batch) * mem->H_kv * c->capacity * p.score_w * 4);
    }
    p.weight_tc = mem->dtype == MSA_BF16 && static_cast<int64_t>(cols) >= kWeightTcCols;
    if (p.weight_tc) {
      p.q16 = p.bytes;
      p.factor = p.q16 + round256(rows * mem->D * 2);
      p.bytes = p.factor + round256(rows * 4);
    }
  }
}

// Columns (tokens * heads of a group) from which the tcgen05 kernel takes over.  It widens every
// context row once for 256 columns, the other one once for 32: at 32 columns it takes 26 against
// 44 us for one query of 8,192 rows but 397 against 210 for 32 of them (bound by the widening); at
// 48 columns 27 against 42 and 397 against 385; at 128 columns 32 against 54 and 396 against 801.
constexpr int64_t kTcCols = 48;

Attend8Plan plan_attend8(const msa_memory *mem, const msa_cache8 *c, int T, int k, int H_q) {
  Attend8Plan p;
  const int64_t max_mem = static_cast<int64_t>(k) * mem->max_doc_chunks;
  p.table_cap = static_cast<int>(std::min<int64_t>(max_mem, msa::kMaxMemRows));
  const int64_t cols = static_cast<int64_t>(T) * (H_q / mem->H_kv);
  const int64_t bh = static_cast<int64_t>(c->batch) * mem->H_kv;
  const size_t rows = static_cast<size_t>(c->batch) * T * H_q;
  p.tc = mem->dtype == MSA_BF16 && mem->D == 128 && cols >= kTcCols &&
         msa::C8tSmem::bytes(p.table_cap) <= max_dyn_smem();
  if (p.tc) {
    // context splits that finish first, counting a CTA's set-up and its part of the merge as
    // eight blocks
    p.col_tiles = static_cast<int>((cols + 2 * msa::kC8tRows - 1) / (2 * msa::kC8tRows));
    const int64_t ctas = bh * p.col_tiles;
    const int64_t blocks = (c->capacity + max_mem + msa::kC8tBlk - 1) / msa::kC8tBlk;
    int64_t best = INT64_MAX;
    for (int s = 1; s <= 16 && (s == 1 || s * 4 <= blocks); ++s) {
      const int64_t waves = (ctas * s + num_sms() - 1) / num_sms();
      const int64_t cost = waves * ((blocks + s - 1) / s + 8);
      if (cost < best) {
        best = cost;
        p.n_split = p.loc_split = s;
      }
    }
    plan_attend8_scratch(p, mem, c, rows);
    return p;
  }
  const int per = 8 * attend8_nt(mem->dtype, cols);
  p.col_tiles = static_cast<int>((cols + per - 1) / per);
  const int64_t ctas = bh * p.col_tiles;
  // Splits of at most 2,048 local rows, so that ragged lengths spread over the SMs (64 queries of
  // up to 8,192 rows: 133 us at 4,096 rows a split, 124 at 2,048, 131 at 1,024).  Fewer CTAs than
  // fit the GPU at a time: as many splits as fill it once, down to 64 rows each.  Where the context
  // is split, the memory rows get splits of their own, so that the others need no chunk table; a
  // memory row counts as two local ones (bf16 against one byte).
  const bool bf16 = mem->dtype == MSA_BF16;
  const int64_t room = static_cast<int64_t>(num_sms()) * (per * (bf16 ? 1 : 2) == 8 ? 4 : per * (bf16 ? 1 : 2) == 16 ? 3 : 2);
  int64_t loc = (c->capacity + 2047) / 2048, own = 0;
  const bool fill = ctas * (loc + (max_mem > 0 ? 1 : 0)) < room;
  if (fill) loc = std::max<int64_t>(1, room / ctas);
  if (max_mem > 0 && (loc > 1 || !bf16)) {  // (fp32 memory rows are a kernel's of their own)
    own = std::max<int64_t>(1, loc * 2 * max_mem / (2 * max_mem + c->capacity));
    own = std::min<int64_t>(std::min<int64_t>(own, (max_mem + 63) / 64), msa::kC8MaxSplit - 64);
    if (fill) loc = std::max<int64_t>(1, loc - own);
  }
  loc = std::min<int64_t>(std::min<int64_t>(loc, (c->capacity + 63) / 64), 64);
  p.loc_split = static_cast<int>(loc);
  p.n_split = static_cast<int>(loc + own);
  plan_attend8_scratch(p, mem, c, rows);
  return p;
}

msa_status attend8_check(const msa_memory *mem, const msa_cache8 *c, int T, int k, int H_q) {
  const msa_status s = cache8_check(mem, c);
  if (s != MSA_OK) return s;
  if (T < 1) return fail(MSA_ERR_INVALID_ARG, "tokens must be >= 1");
  if (k < 0 || k > msa::kMaxTopK) return fail(MSA_ERR_INVALID_ARG, "k=%d out of range", k);
  if (H_q < mem->H_kv || H_q % mem->H_kv != 0)
    return fail(MSA_ERR_INVALID_ARG, "n_q_heads=%d must be a multiple of n_kv_heads=%d", H_q, mem->H_kv);
  if (H_q / mem->H_kv > 16)
    return fail(MSA_ERR_UNSUPPORTED, "GQA group %d exceeds 16", H_q / mem->H_kv);
  if (static_cast<int64_t>(k) * mem->max_doc_chunks > msa::kMaxMemRows)
    return fail(MSA_ERR_UNSUPPORTED, "k * max_doc_chunks = %lld exceeds %d retrieved rows",
                (long long)k * mem->max_doc_chunks, msa::kMaxMemRows);
  if (static_cast<int64_t>(c->batch) * T * H_q > 0x7FFFFFFF || static_cast<int64_t>(T) * (H_q / mem->H_kv) > 65535LL * 4)
    return fail(MSA_ERR_UNSUPPORTED, "batch * tokens * n_q_heads too large");
  return MSA_OK;
}

template <int FMT>
msa_status launch_prefill8(const msa::Attend8Args &a, const Attend8Plan &p, int B, cudaStream_t st) {
  auto kern = a.bl >= msa::kC8tBlk ? msa::cache8_prefill_tc_kernel<FMT, 1> : msa::cache8_prefill_tc_kernel<FMT, 4>;
  const int smem = msa::C8tSmem::bytes(p.table_cap);
  MSA_CUDA(allow_smem(kern, smem));
  const int64_t ctas = static_cast<int64_t>(B) * a.H_kv * p.col_tiles;
  if (ctas > 0x7FFFFFFF) return fail(MSA_ERR_UNSUPPORTED, "too many query tokens");
  MSA_CUDA(launch_pdl(kern, dim3(static_cast<unsigned>(ctas), p.n_split), dim3(msa::kC8tThreads), smem,
                      st, a, p.col_tiles));
  MSA_LAUNCHED("cache8_prefill_tc_kernel");
  return MSA_OK;
}

template <typename T, int D, int FMT, int NT>
msa_status launch_attend8(const msa::Attend8Args &a, const Attend8Plan &p, int B, uint8_t *ws,
                          cudaStream_t st) {
  constexpr bool kBf16 = sizeof(T) == 2;
  const dim3 block(32 * msa::kC8Warps);
  const int own = p.n_split - p.loc_split;
  if (kBf16 && D == 128 && p.tc) {
    const msa_status s = launch_prefill8<FMT>(a, p, B, st);
    if (s != MSA_OK) return s;
  } else {
    auto kern = msa::cache8_attend_kernel<T, D, NT, FMT>;
    const int smem = msa::Attend8Smem<D, NT>::bytes(kBf16 ? p.table_cap : 0);
    MSA_CUDA(allow_smem(kern, smem));
    MSA_CUDA(launch_pdl(kern, dim3(B * a.H_kv, kBf16 ? p.n_split : p.loc_split, p.col_tiles), block, smem,
                        st, a));
    MSA_LAUNCHED("cache8_attend_kernel");
    if (!kBf16 && own > 0) {
      auto mk = msa::cache8_memory_f32_kernel<D>;
      const int ms = msa::Memory8Smem<D>::bytes(p.table_cap);
      const int tiles = (a.T * a.G + msa::kC8Cols32 - 1) / msa::kC8Cols32;
      MSA_CUDA(allow_smem(mk, ms));
      MSA_CUDA(launch_pdl(mk, dim3(B * a.H_kv, own, tiles), block, ms, st, a));
      MSA_LAUNCHED("cache8_memory_f32_kernel");
    }
  }
  if (p.n_split > 1) {
    const int rows = B * a.T * a.H_kv * a.G;
    const bool many = p.n_split > 4;
    auto ck = many ? msa::cache8_combine_kernel<T, D, 4> : msa::cache8_combine_kernel<T, D, 1>;
    const unsigned grid = many ? rows : (static_cast<unsigned>(rows) + 3) / 4;
    MSA_CUDA(launch_pdl(ck, dim3(grid), dim3(128), 0, st, a, rows));
    MSA_LAUNCHED("cache8_combine_kernel");
  }
  if (a.scores) {
    auto sk = p.score_w == 4   ? msa::cache8_weight_scores_kernel<4>
              : p.score_w == 8 ? msa::cache8_weight_scores_kernel<8>
                               : msa::cache8_weight_scores_kernel<16>;
    MSA_CUDA(launch_pdl(sk, dim3((a.cap + 255) / 256, B * a.H_kv), dim3(256), 0, st, a));
    MSA_LAUNCHED("cache8_weight_scores_kernel");
  } else if (kBf16 && a.weights && p.weight_tc) {
    auto wk = msa::cache8_weight_tc_kernel<D, FMT>;
    auto *q16 = reinterpret_cast<__half *>(ws + p.q16);
    auto *factor = reinterpret_cast<float *>(ws + p.factor);
    const int64_t cols = static_cast<int64_t>(B) * a.T * a.H_kv * a.G;
    MSA_CUDA(launch_pdl(msa::cache8_q16_kernel<D>, dim3(static_cast<unsigned>((cols + 7) / 8)), dim3(256), 0,
                        st, a, B, q16, factor));
    MSA_LAUNCHED("cache8_q16_kernel");
    MSA_CUDA(allow_smem(wk, msa::CwSmem<D>::kBytes));
    MSA_CUDA(launch_pdl(wk, dim3((a.cap + msa::kCwRows - 1) / msa::kCwRows, B * a.H_kv),
                        dim3(msa::kCwThreads), msa::CwSmem<D>::kBytes, st, a,
                        static_cast<const __half *>(q16), static_cast<const float *>(factor)));
    MSA_LAUNCHED("cache8_weight_tc_kernel");
  } else if constexpr (NT == (kBf16 ? 4 : 2)) {  // (fewer columns left their scores behind)
    if (!a.weights) return MSA_OK;
    auto wk = msa::cache8_weight_kernel<T, D, NT, FMT>;
    const int smem = msa::Weight8Smem<D, NT>::kBytes;
    MSA_CUDA(allow_smem(wk, smem));
    // one round of columns: a CTA streams its share of the tiles, about eight CTAs an SM in all
    // (a CTA's set-up takes as long as a dozen tiles); more rounds: a CTA for every kC8wRows rows
    const int chunks = (a.cap + msa::kC8wRows - 1) / msa::kC8wRows;
    const bool stream = static_cast<int64_t>(a.T) * a.G <= 8 * NT;
    const int grid_x = stream ? std::min(chunks, (8 * num_sms() + B * a.H_kv - 1) / (B * a.H_kv)) : chunks;
    MSA_CUDA(launch_pdl(wk, dim3(grid_x, B * a.H_kv), block, smem, st, a, stream ? 1 : 0));
    MSA_LAUNCHED("cache8_weight_kernel");
  }
  return MSA_OK;
}

struct EvictPlan8 {
  size_t keys = 0, src = 0, lens = 0, bytes = 0;
};
EvictPlan8 plan_evict8(const msa_memory *mem, const msa_cache8 *c) {
  EvictPlan8 p;
  const size_t bh = static_cast<size_t>(c->batch) * mem->H_kv, nb = c->capacity / c->block_len;
  p.src = round256(bh * nb * 4);
  p.lens = p.src + round256(bh * (nb + 1) * 4);
  p.bytes = p.lens + round256(static_cast<size_t>(c->batch) * 2 * 4);
  return p;
}

}  // namespace

msa_status msa_host::cache8_attend(const msa_memory *mem, const void *content, const int32_t *ids,
                                   const int32_t *slots, int slot_chunks, int32_t k,
                                   const msa_cache8 *cache, int32_t tokens, int32_t n_q_heads,
                                   const void *Q, const int32_t *n_tokens, void *O, float *lse,
                                   float weight_decay, void *workspace, size_t workspace_bytes,
                                   cudaStream_t st) {
  const msa_status s = attend8_check(mem, cache, tokens, k, n_q_heads);
  if (s != MSA_OK) return s;
  if (!Q || !O || (k > 0 && (!content || !ids))) return fail(MSA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(Q) || !aligned16(O) || !aligned16(content) || !aligned16(workspace))
    return fail(MSA_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (std::isnan(weight_decay) || std::isinf(weight_decay))
    return fail(MSA_ERR_INVALID_ARG, "weight_decay must be finite");
  const bool track = weight_decay >= 0.0f;
  if (track && !cache->weights)
    return fail(MSA_ERR_INVALID_ARG, "weight_decay >= 0 needs a cache with weights");
  const Attend8Plan p = plan_attend8(mem, cache, tokens, k, n_q_heads);
  if (workspace_bytes < p.bytes || (p.bytes > 0 && !workspace))
    return fail(MSA_ERR_INVALID_ARG, "workspace too small: %zu < %zu", workspace_bytes, p.bytes);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  msa::Attend8Args a;
  a.content = content;
  a.ids = ids;
  a.doc_chunk_off = mem->d_doc_chunk_off;
  a.slots = slots;
  a.slot_chunks = slot_chunks;
  a.k = k;
  a.n_docs = mem->n_docs;
  a.table_cap = p.table_cap;
  a.k8 = static_cast<const uint8_t *>(cache->k);
  a.v8 = static_cast<const uint8_t *>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.cache_len = cache->cache_len;
  a.n_tokens = n_tokens;
  a.H_kv = mem->H_kv;
  a.G = n_q_heads / mem->H_kv;
  a.g_magic = a.G == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + a.G - 1) / a.G);
  a.T = tokens;
  a.cap = cache->capacity;
  a.bl = cache->block_len;
  a.bl_shift = block_shift(cache);
  a.Q = Q;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(mem->D)));
  a.n_split = p.n_split;
  a.loc_split = p.loc_split;
  a.O = O;
  a.lse = lse;
  a.scores = track && p.score_w ? reinterpret_cast<float *>(ws + p.scores) : nullptr;
  a.score_w = p.score_w;
  a.ml = track ? reinterpret_cast<float2 *>(ws + p.ml) : nullptr;
  a.part_o = reinterpret_cast<float *>(ws + p.part_o);
  a.part_ml = reinterpret_cast<float *>(ws + p.part_ml);
  a.weights = track ? cache->weights : nullptr;
  a.decay = weight_decay;
  const int nt = attend8_nt(mem->dtype, static_cast<int64_t>(tokens) * a.G);
  return dispatch8(mem, cache->format, [&](auto t, auto d, auto f) {
    using T = decltype(t);
    if (nt == 1) return launch_attend8<T, d.value, f.value, 1>(a, p, cache->batch, ws, st);
    if constexpr (sizeof(T) == 2)
      if (nt == 4) return launch_attend8<T, d.value, f.value, 4>(a, p, cache->batch, ws, st);
    return launch_attend8<T, d.value, f.value, 2>(a, p, cache->batch, ws, st);
  });
}

// ===================================================================== C ABI
extern "C" {

msa_status msa_rope_create(const msa_rope_config *cfg, msa_rope **out) {
  if (!cfg || !out) return fail(MSA_ERR_INVALID_ARG, "null config or output");
  *out = nullptr;
  if (cfg->head_dim < 2 || cfg->head_dim > msa::kRopeMaxDim || cfg->head_dim % 2 != 0)
    return fail(MSA_ERR_UNSUPPORTED, "head_dim=%d must be even and in [2, %d]", cfg->head_dim,
                msa::kRopeMaxDim);
  if (cfg->rotary_dim < 2 || cfg->rotary_dim > cfg->head_dim || cfg->rotary_dim % 2 != 0)
    return fail(MSA_ERR_INVALID_ARG, "rotary_dim=%d must be even and in [2, head_dim=%d]",
                cfg->rotary_dim, cfg->head_dim);
  if (!(cfg->theta > 1.0) || !std::isfinite(cfg->theta))
    return fail(MSA_ERR_INVALID_ARG, "theta must be finite and > 1");
  if (cfg->layout != MSA_ROPE_HALF && cfg->layout != MSA_ROPE_INTERLEAVED)
    return fail(MSA_ERR_INVALID_ARG, "layout=%d is not a msa_rope_layout", cfg->layout);
  if (cfg->scaling < MSA_ROPE_NONE || cfg->scaling > MSA_ROPE_YARN)
    return fail(MSA_ERR_INVALID_ARG, "scaling=%d is not a msa_rope_scaling", cfg->scaling);
  if (cfg->scaling != MSA_ROPE_NONE && (!(cfg->factor >= 1.0) || !std::isfinite(cfg->factor)))
    return fail(MSA_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (cfg->scaling == MSA_ROPE_NTK && cfg->rotary_dim == 2)
    return fail(MSA_ERR_INVALID_ARG, "NTK scaling needs rotary_dim > 2");
  if (cfg->scaling == MSA_ROPE_YARN && cfg->original_length < 1)
    return fail(MSA_ERR_INVALID_ARG, "YaRN scaling needs original_length >= 1");
  if (!std::isfinite(cfg->magnitude)) return fail(MSA_ERR_INVALID_ARG, "magnitude must be finite");
  msa_rope *r = new (std::nothrow) msa_rope();
  if (!r) return fail(MSA_ERR_OUT_OF_MEMORY, "could not allocate the rotary handle");
  try {
    std::vector<uint64_t> freq;
    rope_frequencies(cfg, freq, &r->magnitude);
    r->D = cfg->head_dim;
    r->r = cfg->rotary_dim;
    r->layout = cfg->layout;
    cudaError_t e = cudaGetDevice(&r->device);
    if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void **>(&r->d_freq), freq.size() * 8);
    if (e == cudaSuccess)
      e = cudaMemcpy(r->d_freq, freq.data(), freq.size() * 8, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) {
      cudaGetLastError();
      msa_rope_destroy(r);
      return e == cudaErrorMemoryAllocation
                 ? fail(MSA_ERR_OUT_OF_MEMORY, "could not allocate the rotary table")
                 : cuda_fail(e, "the rotary table");
    }
  } catch (const std::bad_alloc &) {
    msa_rope_destroy(r);
    return fail(MSA_ERR_OUT_OF_MEMORY, "could not allocate the rotary table");
  }
  *out = r;
  return MSA_OK;
}

msa_status msa_rope_destroy(msa_rope *rope) {
  if (!rope) return fail(MSA_ERR_INVALID_ARG, "null rope");
  cudaFree(rope->d_freq);
  delete rope;
  return MSA_OK;
}

msa_status msa_rope_apply(const msa_rope *rope, msa_dtype dtype, int64_t tokens,
                          const int64_t *positions, int32_t inverse, const void *q,
                          int32_t q_heads, int64_t q_stride, void *q_out, int64_t q_out_stride,
                          const void *k, int32_t k_heads, int64_t k_stride, void *k_out,
                          int64_t k_out_stride, msa_stream stream) {
  if (!rope) return fail(MSA_ERR_INVALID_ARG, "null rope");
  if (dtype != MSA_F32 && dtype != MSA_BF16)
    return fail(MSA_ERR_INVALID_ARG, "dtype must be MSA_F32 or MSA_BF16");
  if (tokens < 0 || q_heads < 0 || k_heads < 0 || q_heads > 4096 || k_heads > 4096 ||
      q_heads + k_heads < 1)
    return fail(MSA_ERR_INVALID_ARG, "tokens or head counts out of range");
  const msa::RopeSide qs{q, q_out, q_stride, q_out_stride, q_heads};
  const msa::RopeSide ks{k, k_out, k_stride, k_out_stride, k_heads};
  if (tokens == 0) return MSA_OK;
  if (!positions) return fail(MSA_ERR_INVALID_ARG, "null positions");
  const size_t es = elem_size(dtype);
  for (const msa::RopeSide *s : {&qs, &ks}) {
    if (s->heads == 0) continue;
    const int64_t row = static_cast<int64_t>(s->heads) * rope->D;
    if (!s->in || !s->out) return fail(MSA_ERR_INVALID_ARG, "null Q or K");
    if (s->in_stride < row || s->out_stride < row)
      return fail(MSA_ERR_INVALID_ARG, "a token stride is smaller than its heads");
    if (reinterpret_cast<uintptr_t>(s->in) % es || reinterpret_cast<uintptr_t>(s->out) % es)
      return fail(MSA_ERR_INVALID_ARG, "Q and K must be aligned to their elements");
    if (s->in == s->out && s->in_stride != s->out_stride)
      return fail(MSA_ERR_INVALID_ARG, "in place, the strides must be equal");
  }
  const msa_status on = current_device(rope->device, "rotary handle");
  if (on != MSA_OK) return on;
  const int inv = inverse ? 1 : 0;
  return dtype == MSA_BF16
             ? dispatch_rope<__nv_bfloat16>(rope, tokens, positions, inv, qs, ks, to_stream(stream))
             : dispatch_rope<float>(rope, tokens, positions, inv, qs, ks, to_stream(stream));
}

msa_status msa_cache8_append(const msa_memory *mem, const msa_cache8 *cache, const void *K,
                             const void *V, int32_t tokens, int64_t k_batch_stride,
                             int64_t k_token_stride, int64_t v_batch_stride, int64_t v_token_stride,
                             const int32_t *n_tokens, const int32_t *start, msa_stream stream) {
  const msa_status s = cache8_check(mem, cache);
  if (s != MSA_OK) return s;
  if (tokens < 1) return fail(MSA_ERR_INVALID_ARG, "tokens must be >= 1");
  if (!K || !V) return fail(MSA_ERR_INVALID_ARG, "null K or V");
  const int64_t unit = 16 / elem_size(mem->dtype);
  if (!aligned16(K) || !aligned16(V) || k_batch_stride % unit || k_token_stride % unit ||
      v_batch_stride % unit || v_token_stride % unit)
    return fail(MSA_ERR_INVALID_ARG, "K, V and their strides must be multiples of 16 bytes");
  if (k_batch_stride < 0 || k_token_stride < 0 || v_batch_stride < 0 || v_token_stride < 0)
    return fail(MSA_ERR_INVALID_ARG, "strides must not be negative");
  msa::AppendArgs a;
  a.K = K;
  a.V = V;
  a.kb = k_batch_stride;
  a.kt = k_token_stride;
  a.vb = v_batch_stride;
  a.vt = v_token_stride;
  a.tokens = tokens;
  a.H_kv = mem->H_kv;
  a.cap = cache->capacity;
  a.bl = cache->block_len;
  a.bl_shift = block_shift(cache);
  a.k8 = static_cast<uint8_t *>(cache->k);
  a.v8 = static_cast<uint8_t *>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.cache_len = cache->cache_len;
  a.n_tokens = n_tokens;
  a.start = start == cache->cache_len ? nullptr : start;
  a.weights = cache->weights;
  return dispatch8(mem, cache->format, [&](auto t, auto d, auto f) {
    return launch_append<decltype(t), d.value, f.value>(a, cache->batch, a.start != nullptr,
                                                        to_stream(stream));
  });
}

msa_status msa_cache8_read(const msa_memory *mem, const msa_cache8 *cache, const int32_t *begin,
                           int32_t rows, void *K_out, void *V_out, msa_stream stream) {
  const msa_status s = cache8_check(mem, cache);
  if (s != MSA_OK) return s;
  if (rows < 1) return fail(MSA_ERR_INVALID_ARG, "rows must be >= 1");
  if (!K_out || !V_out || !aligned16(K_out) || !aligned16(V_out))
    return fail(MSA_ERR_INVALID_ARG, "K_out and V_out must be given, 16-byte aligned");
  return dispatch8(mem, cache->format, [&](auto t, auto d, auto f) {
    return launch_read<decltype(t), d.value, f.value>(cache, begin, rows, mem->H_kv, K_out, V_out,
                                                      to_stream(stream));
  });
}

size_t msa_cache8_attend_workspace_size(const msa_memory *mem, const msa_cache8 *cache,
                                        int32_t tokens, int32_t k, int32_t n_q_heads) {
  if (attend8_check(mem, cache, tokens, k, n_q_heads) != MSA_OK) return 0;
  return plan_attend8(mem, cache, tokens, k, n_q_heads).bytes;
}

msa_status msa_cache8_attend(const msa_memory *mem, const void *content, const int32_t *ids,
                             int32_t k, const msa_cache8 *cache, int32_t tokens, int32_t n_q_heads,
                             const void *Q, const int32_t *n_tokens, void *O, float *lse,
                             float weight_decay, void *workspace, size_t workspace_bytes,
                             msa_stream stream) {
  return cache8_attend(mem, content, ids, nullptr, 0, k, cache, tokens, n_q_heads, Q, n_tokens, O,
                       lse, weight_decay, workspace, workspace_bytes, to_stream(stream));
}

size_t msa_cache8_evict_workspace_size(const msa_memory *mem, const msa_cache8 *cache) {
  if (cache8_check(mem, cache) != MSA_OK) return 0;
  return plan_evict8(mem, cache).bytes;
}

msa_status msa_cache8_evict(const msa_memory *mem, const msa_cache8 *cache, const msa_cache8 *out,
                            int32_t budget, int32_t recent, void *workspace,
                            size_t workspace_bytes, msa_stream stream) {
  msa_status s = cache8_check(mem, cache);
  if (s == MSA_OK) s = cache8_check(mem, out);
  if (s != MSA_OK) return s;
  if (!cache->weights || !out->weights)
    return fail(MSA_ERR_INVALID_ARG, "eviction needs caches with weights");
  if (out->batch != cache->batch || out->block_len != cache->block_len || out->format != cache->format)
    return fail(MSA_ERR_INVALID_ARG, "the caches differ in batch, block_len or format");
  if (budget < cache->block_len)
    return fail(MSA_ERR_INVALID_ARG, "budget=%d must be at least block_len=%d", budget, cache->block_len);
  if (recent < 0 || recent > budget)
    return fail(MSA_ERR_INVALID_ARG, "recent=%d must be in [0, budget=%d]", recent, budget);
  if (out->capacity < std::min(cache->capacity, budget))
    return fail(MSA_ERR_INVALID_ARG, "the receiving capacity %d is smaller than min(%d, budget=%d)",
                out->capacity, cache->capacity, budget);
  const bool in_place = out->k == cache->k;
  if (in_place != (out->v == cache->v) || in_place != (out->k_scale == cache->k_scale) ||
      in_place != (out->v_scale == cache->v_scale) || in_place != (out->weights == cache->weights) ||
      in_place != (out->cache_len == cache->cache_len) || (in_place && out->capacity != cache->capacity))
    return fail(MSA_ERR_INVALID_ARG, "out must be the same cache or share no buffer with it");
  // beyond the capacity they mean the capacity (2^31 - 1: keep everything)
  budget = std::min(budget, cache->capacity);
  recent = std::min(recent, budget);
  const EvictPlan8 p = plan_evict8(mem, cache);
  if (!workspace || !aligned16(workspace) || workspace_bytes < p.bytes)
    return fail(MSA_ERR_INVALID_ARG, "workspace missing, unaligned or too small: %zu < %zu",
                workspace_bytes, p.bytes);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  auto *keys = reinterpret_cast<uint32_t *>(ws + p.keys);
  auto *src = reinterpret_cast<int32_t *>(ws + p.src);
  auto *lens = reinterpret_cast<int32_t *>(ws + p.lens);
  const cudaStream_t st = to_stream(stream);
  const unsigned bh = static_cast<unsigned>(cache->batch * mem->H_kv);
  const int bl = cache->block_len;
  // the keys of up to 10,240 blocks fit in the 48 KB that need no opt-in beside the histogram
  const int nb = cache->capacity / bl, smem_keys = nb <= 10240 ? 1 : 0;
  MSA_CUDA(launch_pdl(msa::cache8_select_kernel, dim3(bh), dim3(msa::kSelThreads),
                      smem_keys ? static_cast<size_t>(nb) * 4 : 0, st,
                      static_cast<const float *>(cache->weights),
                      static_cast<const int32_t *>(cache->cache_len), mem->H_kv, cache->capacity, bl,
                      budget, recent, smem_keys, keys, src, lens));
  MSA_LAUNCHED("cache8_select_kernel");
  msa::EvictMove m;
  m.k8 = static_cast<const uint8_t *>(cache->k);
  m.v8 = static_cast<const uint8_t *>(cache->v);
  m.ks = cache->k_scale;
  m.vs = cache->v_scale;
  m.w = cache->weights;
  m.ok8 = static_cast<uint8_t *>(out->k);
  m.ov8 = static_cast<uint8_t *>(out->v);
  m.oks = out->k_scale;
  m.ovs = out->v_scale;
  m.ow = out->weights;
  m.out_len = out->cache_len;
  m.H_kv = mem->H_kv;
  m.cap = cache->capacity;
  m.out_cap = out->capacity;
  m.bl = bl;
  m.D = mem->D;
  const int streams = 2 * (bl * mem->D / 16) + bl / 4 + 2;
  const int live = (budget + bl - 1) / bl;
  const int parts = in_place ? 1 : std::max(1, std::min(live / msa::kMoveWave, 65535));
  MSA_CUDA(launch_pdl(msa::cache8_move_kernel, dim3((streams + 127) / 128, bh, parts), dim3(128), 0,
                      st, m, static_cast<const int32_t *>(src), static_cast<const int32_t *>(lens),
                      in_place ? 1 : 0));
  MSA_LAUNCHED("cache8_move_kernel");
  return MSA_OK;
}

}  // extern "C"
