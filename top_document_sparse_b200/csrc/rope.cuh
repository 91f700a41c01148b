// rope.cuh -- rotary positions of Q and K heads in one launch: half or
// interleaved pairs, part of a head, any per-pair frequencies.
//   (a, b) -> magnitude * (a cos - b sin, b cos + a sin), angle = position * freq_i
// The frequency of a pair is a 64-bit fraction of a turn, so position * freq
// modulo 2^64 is the angle modulo one turn, exact at any position: the top 32
// bits go to sincospi, an error of 2^-25 turns at most.
// The work is bytes: every element is read and written once.  A CTA takes the
// heads of a few tokens; the angles of a token are computed once, into shared
// memory, and used by all of its heads.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace msa {

constexpr int kRopeThreads = 512;  // most threads of a block
constexpr int kRopeMaxDim = 512;

struct RopeSide {  // one of Q and K: heads of `D` elements, strides in elements
  const void *in;
  void *out;
  int64_t in_stride, out_stride;
  int heads;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
  T v[V];
};

// One task: V elements of a rotated half (with their V partners), V / 2
// interleaved pairs, or V elements of the rest of the head.
template <typename T, int V, bool INTER>
__device__ __forceinline__ void rope_task(const T *in, T *out, int task, int rot_tasks, int r,
                                          const float2 *cs) {
  using Vec = RopeVec<T, V>;
  if (task >= rot_tasks) {
    const int e = r + (task - rot_tasks) * V;
    *reinterpret_cast<Vec *>(out + e) = *reinterpret_cast<const Vec *>(in + e);
    return;
  }
  if constexpr (INTER) {
    // V = 1 stands for one pair moved by scalar loads (rows without alignment)
    constexpr int N = V == 1 ? 2 : V;
    const int e = task * N;
    T x[N], y[N];
    if constexpr (V == 1) {
      x[0] = in[e];
      x[1] = in[e + 1];
    } else {
      *reinterpret_cast<Vec *>(x) = *reinterpret_cast<const Vec *>(in + e);
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 c = cs[(e + i) >> 1];
      const float a = Elem<T>::to_f(x[i]), b = Elem<T>::to_f(x[i + 1]);
      y[i] = Elem<T>::from_f(a * c.x - b * c.y);
      y[i + 1] = Elem<T>::from_f(b * c.x + a * c.y);
    }
    if constexpr (V == 1) {
      out[e] = y[0];
      out[e + 1] = y[1];
    } else {
      *reinterpret_cast<Vec *>(out + e) = *reinterpret_cast<const Vec *>(y);
    }
  } else {
    const int e = task * V, half = r >> 1;
    const Vec xa = *reinterpret_cast<const Vec *>(in + e);
    const Vec xb = *reinterpret_cast<const Vec *>(in + e + half);
    Vec ya, yb;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 c = cs[e + i];
      const float a = Elem<T>::to_f(xa.v[i]), b = Elem<T>::to_f(xb.v[i]);
      ya.v[i] = Elem<T>::from_f(a * c.x - b * c.y);
      yb.v[i] = Elem<T>::from_f(b * c.x + a * c.y);
    }
    *reinterpret_cast<Vec *>(out + e) = ya;
    *reinterpret_cast<Vec *>(out + e + half) = yb;
  }
}

// grid ceil(tokens / tok_cta), block <= kRopeThreads, shared tok_cta * r / 2 float2.
// per_head = rot_tasks + the tasks of the copied rest (0 where the rest stays
// in place).
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const uint64_t *__restrict__ freq, int r, int D, float magnitude, int inverse,
            const int64_t *__restrict__ positions, int64_t tokens, int tok_cta, RopeSide q,
            RopeSide k, int rot_tasks, int per_head) {
  extern __shared__ float2 rope_cs[];
  griddep_wait();
  griddep_launch();
  const int half = r >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok_cta;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tok_cta), tokens - t0));
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int t = i / half, p = i - t * half;
    const uint64_t turn = static_cast<uint64_t>(positions[t0 + t]) * freq[p];
    float s, c;
    // the signed top half is the angle in units of 2^-32 turns, within half a turn
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
    rope_cs[i] = make_float2(c * magnitude, (inverse ? -s : s) * magnitude);
  }
  __syncthreads();
  const int per_token = (q.heads + k.heads) * per_head;
  for (int i = threadIdx.x; i < nt * per_token; i += blockDim.x) {
    const int t = i / per_token, j = i - t * per_token;
    const int h = j / per_head, task = j - h * per_head;
    const bool is_q = h < q.heads;
    const RopeSide &s = is_q ? q : k;
    const int hh = is_q ? h : h - q.heads;
    const T *in = static_cast<const T *>(s.in) + (t0 + t) * s.in_stride + hh * D;
    T *out = static_cast<T *>(s.out) + (t0 + t) * s.out_stride + hh * D;
    rope_task<T, V, INTER>(in, out, task, rot_tasks, r, rope_cs + t * half);
  }
}

}  // namespace msa
