// context.cuh -- the retrieved documents' chunk rows as an attention context:
// the chunk table that every attention kernel builds in shared memory.
#pragma once
#include "common.cuh"

namespace msa {

constexpr int kMaxMemRows = 4096;  // retrieved chunks per query (k * chunks per doc)
constexpr float kLog2e = 1.4426950408889634f;

// Chunk list of query b's retrieved documents in rank order -> table[0..n_mem).
// Warp 0 loads the k (<= 64) ranks' chunk counts in parallel (two ranks per
// lane) and prefix-sums them with shuffles; every thread then fills table
// entries from shared memory only (binary search over the prefix sums).
// Ids outside [0, n_docs) contribute no rows and raise MSA_DEVERR_BAD_DOC_ID.
// slots_b (nullable, [k]): chunk rows of rank r start at slots_b[r] *
// slot_chunks instead of doc_chunk_off[id] (device slot cache of a host tier).
// `pre` needs kMaxTopK + 1 ints and `base` kMaxTopK ints of shared memory.
__device__ __forceinline__ int build_chunk_table(const int32_t *__restrict__ ids_b, int k,
                                                 const int64_t *__restrict__ doc_chunk_off,
                                                 int n_docs, const int32_t *__restrict__ slots_b,
                                                 int slot_chunks, int *table, int *pre,
                                                 int *base, int table_cap) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int cnt[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane + 32 * h;
      if (r < k) {
        const int d = ids_b[r];
        if (d >= 0 && d < n_docs) {
          const int64_t c0 = doc_chunk_off[d];
          cnt[h] = static_cast<int>(doc_chunk_off[d + 1] - c0);
          base[r] = slots_b ? slots_b[r] * slot_chunks : static_cast<int>(c0);
        } else {
          raise_device_error(MSA_DEVERR_BAD_DOC_ID);
          base[r] = 0;
        }
      }
    }
    int run = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int v = cnt[h];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      const int r = lane + 32 * h;
      const int excl = run + v - cnt[h];
      // a rank that would overflow the table contributes nothing (host validation keeps
      // k * max_doc_chunks <= table_cap, so this does not happen)
      if (r < k) pre[r] = excl + cnt[h] > table_cap ? min(excl, table_cap) : excl;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) pre[k] = min(run, table_cap);
  }
  __syncthreads();
  const int n_mem = pre[k];
  for (int x = threadIdx.x; x < n_mem; x += blockDim.x) {
    int lo = 0, hi = k - 1;  // last rank r with pre[r] <= x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    table[x] = base[lo] + (x - pre[lo]);
  }
  __syncthreads();
  return n_mem;
}

// One warp's part of the chunk table of query b: pre[0..k] (context rows before each rank) and
// base[0..k) (each rank's first chunk row).  Returns n_mem in every lane.
__device__ __forceinline__ int chunk_prefix_warp(const int32_t *__restrict__ ids_b, int k,
                                                 const int64_t *__restrict__ doc_chunk_off,
                                                 int n_docs, const int32_t *__restrict__ slots_b,
                                                 int slot_chunks, int *pre, int *base,
                                                 int table_cap, int lane) {
  int cnt[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = lane + 32 * h;
    if (r < k) {
      const int d = ids_b[r];
      if (d >= 0 && d < n_docs) {
        const int64_t c0 = doc_chunk_off[d];
        cnt[h] = static_cast<int>(doc_chunk_off[d + 1] - c0);
        base[r] = slots_b ? slots_b[r] * slot_chunks : static_cast<int>(c0);
      } else {
        raise_device_error(MSA_DEVERR_BAD_DOC_ID);
        base[r] = 0;
      }
    }
  }
  int run = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = cnt[h];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const int r = lane + 32 * h;
    const int excl = run + v - cnt[h];
    // (a rank that would overflow the table contributes nothing; host validation keeps
    // k * max_doc_chunks <= table_cap)
    if (r < k) pre[r] = excl + cnt[h] > table_cap ? min(excl, table_cap) : excl;
    run += __shfl_sync(0xffffffffu, v, 31);
  }
  const int n_mem = min(run, table_cap);
  if (lane == 0) pre[k] = n_mem;
  __syncwarp();
  return n_mem;
}

// Chunk row of context row x < n_mem.
__device__ __forceinline__ int chunk_row(const int *pre, const int *base, int k, int x) {
  int lo = 0, hi = k - 1;  // last rank r with pre[r] <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return base[lo] + (x - pre[lo]);
}

// The chunk table of query b built by one warp (the loader): table[x] = chunk
// row of context row x < n_mem, ranks in order; the same rows as
// build_chunk_table.  Returns n_mem in every lane.
__device__ __forceinline__ int build_chunk_table_warp(const int32_t *__restrict__ ids_b, int k,
                                                      const int64_t *__restrict__ doc_chunk_off,
                                                      int n_docs, const int32_t *__restrict__ slots_b,
                                                      int slot_chunks, int *table, int *pre,
                                                      int *base, int table_cap, int lane) {
  const int n_mem = chunk_prefix_warp(ids_b, k, doc_chunk_off, n_docs, slots_b, slot_chunks, pre, base,
                                      table_cap, lane);
  for (int x = lane; x < n_mem; x += 32) table[x] = chunk_row(pre, base, k, x);
  __syncwarp();
  return n_mem;
}

}  // namespace msa
