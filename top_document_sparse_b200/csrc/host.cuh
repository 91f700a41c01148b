// host.cuh -- host-side helpers shared by the translation units of libmsa.so:
// statuses and the thread's last error, launch checking and counting,
// programmatic dependent launches, TMA maps.
#pragma once
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>
#include <utility>

#include "common.cuh"

namespace msa_host {

inline thread_local std::string g_last_error;

inline msa_status fail(msa_status s, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline msa_status cuda_fail(cudaError_t e, const char *what) {
  return fail(MSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define MSA_CUDA(call)                                 \
  do {                                                 \
    cudaError_t e_ = (call);                           \
    if (e_ != cudaSuccess) return cuda_fail(e_, #call); \
  } while (0)

// Every kernel launch is followed by MSA_LAUNCHED: it checks the launch and
// counts it (msa_launch_count).
inline std::atomic<uint64_t> g_launches{0};

#define MSA_LAUNCHED(what)                              \
  do {                                                  \
    cudaError_t e_ = cudaGetLastError();                \
    if (e_ != cudaSuccess) return cuda_fail(e_, what);  \
    g_launches.fetch_add(1, std::memory_order_relaxed); \
  } while (0)

// Launch with programmatic stream serialization: the kernel may start while
// the previous kernel on the stream drains (it calls griddep_wait() before
// its first global memory access), which hides the launch and the kernel's
// setup behind the previous kernel's tail.  Used for the per-token decode
// path, where a step is a chain of short dependent kernels.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Same, with thread-block clusters of cluster_x CTAs along x (1: none).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               cudaStream_t st, unsigned cluster_x, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster_x;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster_x > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline int round32(int x) { return (x + 31) / 32 * 32; }

inline int num_sms() {
  static int n = 0;
  if (n == 0) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 148;
  }
  return n;
}

inline int max_dyn_smem() {
  static int n = 0;
  if (n == 0) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (n <= 0) n = 232448;
  }
  return n;
}

// ---------------------------------------------------------------- TMA maps
inline PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D bf16 map over a row-major [rows][cols] array, box {64 cols, box_rows},
// 128-byte swizzle, out-of-range rows read as zero.
inline msa_status make_map_bf16(CUtensorMap *map, const void *base, int64_t rows, int64_t cols,
                         int box_rows) {
  auto fn = encode_tiled();
  if (!fn) return fail(MSA_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MSA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return MSA_OK;
}

// 3-D bf16 map over [d2][d1][d0] with the given byte strides of dimensions 1 and 2, box
// {64, box1, box2}, 128-byte swizzle, out-of-range elements read as zero.
inline msa_status make_map_bf16_3d(CUtensorMap *map, const void *base, int64_t d0, int64_t d1, int64_t d2,
                            int64_t stride1, int64_t stride2, int box1, int box2) {
  auto fn = encode_tiled();
  if (!fn) return fail(MSA_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1),
                        static_cast<cuuint64_t>(d2)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride1), static_cast<cuuint64_t>(stride2)};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MSA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return MSA_OK;
}

// ---------------------------------------------------------------- helpers
inline size_t elem_size(msa_dtype t) { return t == MSA_BF16 ? 2 : 4; }

// The device error word of the kernels in serve.cu (each translation unit has
// a word of its own): enqueue a read into *bits and a clear on `st`.
cudaError_t take_serve_error(unsigned int *bits, cudaStream_t st);

// The 8-bit cache's attention over memory rows in `content`, or in a slot cache (slots, [batch][k],
// of slot_chunks rows each); see msa_cache8_attend.
msa_status cache8_attend(const msa_memory *mem, const void *content, const int32_t *ids,
                         const int32_t *slots, int slot_chunks, int32_t k, const msa_cache8 *cache,
                         int32_t tokens, int32_t n_q_heads, const void *Q, const int32_t *n_tokens,
                         void *O, float *lse, float weight_decay, void *workspace,
                         size_t workspace_bytes, cudaStream_t st);

}  // namespace msa_host
