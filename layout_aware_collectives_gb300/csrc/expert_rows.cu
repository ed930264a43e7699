// Tokens' rows to their experts and back: one pass over the rows, bound by
// HBM.  A thread takes 16 bytes of a token's row (V = 8; single elements where
// rows do not start on 16 bytes) and the same of each of its topk rows.
#include "compute_device.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;  // rows of a token on their way at a time

template <int V>
struct Piece {
  uint32_t w[V == 8 ? 4 : 1];
};

template <int V>
__device__ __forceinline__ Piece<V> load(const uint16_t* p) {
  Piece<V> r;
  if constexpr (V == 8) {
    const uint4 q = __ldcs((const uint4*)p);
    r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
  } else {
    r.w[0] = *p;
  }
  return r;
}
template <int V>
__device__ __forceinline__ void store(uint16_t* p, const Piece<V>& v) {
  if constexpr (V == 8)
    *(uint4*)p = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  else
    *p = (uint16_t)v.w[0];
}
template <int V>
__device__ __forceinline__ void values(const Piece<V>& v, float (&f)[V]) {
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(v.w[i]), f[2 * i + 1] = bf16_hi(v.w[i]);
  } else {
    f[0] = bf16_lo(v.w[0]);
  }
}
template <int V>
__device__ __forceinline__ Piece<V> rounded(const float (&f)[V]) {
  Piece<V> r;
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  } else {
    r.w[0] = to_bf16(f[0]);
  }
  return r;
}

// Threads of a token: a power of two of lanes, so that small rows share a
// warp and large ones take a whole CTA.
struct Shape {
  int lanes, tokens;  // threads of a token; tokens of a CTA
  int64_t pieces;     // of a row
};

// The address of a slot's row, or NULL outside the rows.
__device__ __forceinline__ int64_t row_of(const RowsArgs& a, int64_t pair) {
  const int s = a.slots[pair];
  return s >= 0 && s < a.num_rows ? s : -1;
}

template <int V>
__global__ void __launch_bounds__(kThreads) gather_kernel(RowsArgs a, Shape s) {
  after_previous();
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  if (t >= a.tokens) return;
  const int64_t p0 = t * a.topk;
  for (int64_t q = threadIdx.x % s.lanes; q < s.pieces; q += s.lanes) {
    const Piece<V> v = load<V>(a.in + t * a.ld_in + q * V);
    for (int j = 0; j < a.topk; ++j) {
      const int64_t r = row_of(a, p0 + j);
      if (r >= 0) store<V>(a.out + r * a.ld_out + q * V, v);
    }
  }
}

template <int V>
__global__ void __launch_bounds__(kThreads) combine_kernel(RowsArgs a, Shape s) {
  after_previous();
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  if (t >= a.tokens) return;
  const int64_t p0 = t * a.topk;
  for (int64_t q = threadIdx.x % s.lanes; q < s.pieces; q += s.lanes) {
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.topk; j0 += kAtOnce) {
      Piece<V> v[kAtOnce];
      float w[kAtOnce];
      bool in[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int64_t r = j0 + j < a.topk ? row_of(a, p0 + j0 + j) : -1;
        in[j] = r >= 0;
        w[j] = in[j] && a.weights ? a.weights[p0 + j0 + j] : 1.0f;
        if (in[j]) v[j] = load<V>(a.in + r * a.ld_in + q * V);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (!in[j]) continue;
        float f[V];
        values<V>(v[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
      }
    }
    store<V>(a.out + t * a.ld_out + q * V, rounded<V>(sum));
  }
}

// The weights' gradients are sums along a row: of each thread's pieces in
// order, then over the token's threads in a fixed order.
template <int V>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(RowsArgs a, Shape s) {
  after_previous();
  __shared__ float parts[kThreads / 32][kAtOnce];
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  const bool mine = t < a.tokens;
  const int64_t p0 = t * a.topk;
  const int me = threadIdx.x % s.lanes;
  for (int j0 = 0; j0 < a.topk; j0 += kAtOnce) {
    float dot[kAtOnce], w[kAtOnce];
    int64_t r[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      dot[j] = 0.0f;
      r[j] = mine && j0 + j < a.topk ? row_of(a, p0 + j0 + j) : -1;
      w[j] = r[j] >= 0 && a.weights ? a.weights[p0 + j0 + j] : 1.0f;
    }
    if (mine)
      for (int64_t q = me; q < s.pieces; q += s.lanes) {
        float d[V];
        values<V>(load<V>(a.in + t * a.ld_in + q * V), d);
        Piece<V> v[kAtOnce];
        if (a.dweights)
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
            if (r[j] >= 0) v[j] = load<V>(a.rows + r[j] * a.ld_rows + q * V);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          if (r[j] < 0) continue;
          float f[V];
          if (a.out) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = w[j] * d[i];
            store<V>(a.out + r[j] * a.ld_out + q * V, rounded<V>(f));
          }
          if (a.dweights) {
            values<V>(v[j], f);
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
          }
        }
      }
    if (!a.dweights) continue;
    const int within = min(s.lanes, 32);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      for (int d = within >> 1; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
    if (s.lanes > 32) {
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) parts[threadIdx.x >> 5][j] = dot[j];
      __syncthreads();
      const int w0 = (threadIdx.x - me) >> 5;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        dot[j] = 0.0f;
        for (int k = 0; k < s.lanes / 32; ++k) dot[j] += parts[w0 + k][j];
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (mine && me == j % s.lanes && j0 + j < a.topk) a.dweights[p0 + j0 + j] = dot[j];
  }
}

Shape shape_of(const RowsArgs& a, int v) {
  Shape s{1, 0, a.hidden / v};
  while (s.lanes < kThreads && s.lanes < s.pieces) s.lanes *= 2;
  s.tokens = kThreads / s.lanes;
  return s;
}

template <class K8, class K1>
cudaError_t run(K8 vec, K1 single, const RowsArgs& a, bool by8, cudaStream_t stream) {
  const Shape s = shape_of(a, by8 ? 8 : 1);
  return launch_early(by8 ? vec : single, dim3((unsigned)ceil_div(a.tokens, s.tokens)), kThreads, 0, 0, stream, a, s);
}

bool by8(const RowsArgs& a) {
  return a.hidden % 8 == 0 && a.ld_in % 8 == 0 && (!a.out || a.ld_out % 8 == 0) && (!a.dweights || a.ld_rows % 8 == 0);
}

}  // namespace

cudaError_t launch_expert_gather(const RowsArgs& a, cudaStream_t stream) {
  return run(gather_kernel<8>, gather_kernel<1>, a, by8(a), stream);
}

cudaError_t launch_expert_combine(const RowsArgs& a, cudaStream_t stream) {
  return run(combine_kernel<8>, combine_kernel<1>, a, by8(a), stream);
}

cudaError_t launch_expert_combine_backward(const RowsArgs& a, cudaStream_t stream) {
  return run(combine_backward_kernel<8>, combine_backward_kernel<1>, a, by8(a), stream);
}

}  // namespace tide
