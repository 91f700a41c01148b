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

// One task: V elements of a rotated half with their V partners, V interleaved elements (one pair
// for V = 1, moved by scalar loads: rows without alignment), or V elements of the rest of the head.
template <typename T, int V, bool INTER>
struct RopeTask {
  static constexpr int N = INTER && V == 1 ? 2 : V;
  using Vec = RopeVec<T, V>;
  T x[2 * N];  // interleaved: N elements
  T *out;
  const float2 *cs;
  int e;       // first element
  bool rot;

  __device__ __forceinline__ void load(const T *in, T *o, int task, int rot_tasks, int r,
                                       const float2 *token_cs) {
    rot = task < rot_tasks;
    e = rot ? task * N : r + (task - rot_tasks) * V;
    out = o + e;
    cs = token_cs;
    if constexpr (INTER && V == 1) {
      x[0] = in[e];
      if (rot) x[1] = in[e + 1];
    } else {
      *reinterpret_cast<Vec *>(x) = *reinterpret_cast<const Vec *>(in + e);
      if (!INTER && rot) *reinterpret_cast<Vec *>(x + N) = *reinterpret_cast<const Vec *>(in + e + (r >> 1));
    }
  }
  __device__ __forceinline__ void store(int r) {
    if constexpr (INTER) {
      if (rot) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float2 c = cs[(e + i) >> 1];
          const float a = Elem<T>::to_f(x[i]), b = Elem<T>::to_f(x[i + 1]);
          x[i] = Elem<T>::from_f(a * c.x - b * c.y);
          x[i + 1] = Elem<T>::from_f(b * c.x + a * c.y);
        }
      }
    } else if (rot) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 c = cs[e + i];
        const float a = Elem<T>::to_f(x[i]), b = Elem<T>::to_f(x[N + i]);
        x[i] = Elem<T>::from_f(a * c.x - b * c.y);
        x[N + i] = Elem<T>::from_f(b * c.x + a * c.y);
      }
    }
    if constexpr (INTER && V == 1) {
      out[0] = x[0];
      if (rot) out[1] = x[1];
    } else {
      *reinterpret_cast<Vec *>(out) = *reinterpret_cast<const Vec *>(x);
      if (!INTER && rot) *reinterpret_cast<Vec *>(out + (r >> 1)) = *reinterpret_cast<const Vec *>(x + N);
    }
  }
};

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
  const int per_token = (q.heads + k.heads) * per_head;
  const int total = nt * per_token;
  using Task = RopeTask<T, V, INTER>;
  auto load = [&](Task &task, int i) {
    const int t = i / per_token, j = i - t * per_token;
    const int h = j / per_head;
    const bool is_q = h < q.heads;
    const RopeSide &s = is_q ? q : k;
    const int hh = is_q ? h : h - q.heads;
    task.load(static_cast<const T *>(s.in) + (t0 + t) * s.in_stride + hh * D,
              static_cast<T *>(s.out) + (t0 + t) * s.out_stride + hh * D, j - h * per_head, rot_tasks, r,
              rope_cs + t * half);
  };
  // a thread's first elements are under way while the angles are computed
  Task task;
  int i = threadIdx.x;
  if (i < total) load(task, i);
  for (int a = threadIdx.x; a < nt * half; a += blockDim.x) {
    const int t = a / half, p = a - t * half;
    const uint64_t turn = static_cast<uint64_t>(positions[t0 + t]) * freq[p];
    float s, c;
    // the signed top half is the angle in units of 2^-32 turns, within half a turn
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
    rope_cs[a] = make_float2(c * magnitude, (inverse ? -s : s) * magnitude);
  }
  __syncthreads();
  while (i < total) {
    task.store(r);
    i += blockDim.x;
    if (i < total) load(task, i);
  }
}

}  // namespace msa
