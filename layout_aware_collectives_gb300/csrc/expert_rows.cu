// Tokens' rows to their experts and back: one pass over the rows, bound by
// HBM.  A thread takes 16 bytes of a token's row and the same of each of its
// topk rows.  8191 tokens of 2048 there, 8 choices each: 48 us (6.3 TB/s); 4096
// of them back 25 (6.0), backward 51 (5.6); with 10 choices, which take two turns
// of eight, 37, 38 and 73 (5.0 TB/s).  Rows that do not start on 16 bytes
// take windows of as many, or single elements: 2000 of 2049 there 22 us, back 27,
// backward 52.
#include "compute_device.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;

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
// warp and large ones take up to a whole CTA.
struct Shape {
  int lanes, tokens;  // threads of a token; tokens of a CTA
  int64_t pieces;     // of a row
};

// K of a token's slots (from pair `p` on, `left` of which there are), those
// outside the rows as -1, and the weights.
template <int K>
struct Slots {
  int64_t row[K];
  float w[K];

  __device__ __forceinline__ void load(const RowsArgs& a, int64_t p, int left) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int s = j < left ? a.slots[p + j] : -1;
      row[j] = s >= 0 && s < a.num_rows ? s : -1;
      w[j] = j < left && a.weights ? a.weights[p + j] : 1.0f;
    }
  }
};

template <int V, int K>
__global__ void __launch_bounds__(kThreads) gather_kernel(RowsArgs a, Shape s) {
  after_previous();
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  if (t >= a.tokens) return;
  const int64_t p0 = t * a.topk;
  for (int j0 = 0; j0 < a.topk; j0 += K) {
    Slots<K> at;
    at.load(a, p0 + j0, a.topk - j0);
    for (int64_t q = threadIdx.x % s.lanes; q < s.pieces; q += s.lanes) {
      const Piece<V> v = load<V>(a.in + t * a.ld_in + q * V);
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (at.row[j] >= 0) store<V>(a.out + at.row[j] * a.ld_out + q * V, v);
    }
  }
}

// U pieces of a row at a time, so that U K loads of a thread are on their way.
template <int K, int U>
__global__ void __launch_bounds__(kThreads) combine_kernel(RowsArgs a, Shape s) {
  constexpr int V = 8;
  after_previous();
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  if (t >= a.tokens) return;
  const int64_t p0 = t * a.topk;
  Slots<K> at;
  at.load(a, p0, a.topk);
  for (int64_t q = threadIdx.x % s.lanes; q < s.pieces; q += U * s.lanes) {
    float sum[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) sum[u][i] = 0.0f;
    for (int j0 = 0;;) {
      Piece<V> v[U][K];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (at.row[j] >= 0 && q + u * s.lanes < s.pieces) v[u][j] = load<V>(a.in + at.row[j] * a.ld_in + (q + u * s.lanes) * V);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < K; ++j) {
          if (at.row[j] < 0 || q + u * s.lanes >= s.pieces) continue;
          float f[V];
          values<V>(v[u][j], f);
#pragma unroll
          for (int i = 0; i < V; ++i) sum[u][i] = fmaf(at.w[j], f[i], sum[u][i]);
        }
      if (a.topk <= K) break;
      // more choices than are held at a time: round to the first ones again
      j0 = j0 + K < a.topk ? j0 + K : 0;
      at.load(a, p0 + j0, a.topk - j0);
      if (j0 == 0) break;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (q + u * s.lanes < s.pieces) store<V>(a.out + t * a.ld_out + (q + u * s.lanes) * V, rounded<V>(sum[u]));
  }
}

// The weights' gradients are sums along a row: of each thread's pieces in
// order, then over the token's threads in a fixed order.
template <int V, int K, int U>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(RowsArgs a, Shape s) {
  after_previous();
  __shared__ float parts[kThreads / 32][K];
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  const bool mine = t < a.tokens;
  const int64_t p0 = t * a.topk;
  const int me = threadIdx.x % s.lanes;
  for (int j0 = 0; j0 < a.topk; j0 += K) {
    float dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) dot[j] = 0.0f;
    if (mine) {
      Slots<K> at;
      at.load(a, p0 + j0, a.topk - j0);
      for (int64_t q = me; q < s.pieces; q += U * s.lanes) {
        Piece<V> dy[U], v[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t c = q + u * s.lanes;
          if (c >= s.pieces) continue;
          dy[u] = load<V>(a.in + t * a.ld_in + c * V);
          if (a.dweights)
#pragma unroll
            for (int j = 0; j < K; ++j)
              if (at.row[j] >= 0) v[u][j] = load<V>(a.rows + at.row[j] * a.ld_rows + c * V);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t c = q + u * s.lanes;
          if (c >= s.pieces) continue;
          float d[V];
          values<V>(dy[u], d);
#pragma unroll
          for (int j = 0; j < K; ++j) {
            if (at.row[j] < 0) continue;
            float f[V];
            if (a.out) {
#pragma unroll
              for (int i = 0; i < V; ++i) f[i] = at.w[j] * d[i];
              store<V>(a.out + at.row[j] * a.ld_out + c * V, rounded<V>(f));
            }
            if (a.dweights) {
              values<V>(v[u][j], f);
#pragma unroll
              for (int i = 0; i < V; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
            }
          }
        }
      }
    }
    if (!a.dweights) continue;
#pragma unroll
    for (int j = 0; j < K; ++j)
      for (int d = min(s.lanes, 32) >> 1; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
    if (s.lanes > 32) {
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int j = 0; j < K; ++j) parts[threadIdx.x >> 5][j] = dot[j];
      __syncthreads();
      const int w0 = (threadIdx.x - me) >> 5;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        dot[j] = 0.0f;
        for (int w = 0; w < s.lanes / 32; ++w) dot[j] += parts[w0 + w][j];
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (mine && me == j % s.lanes && j0 + j < a.topk) a.dweights[p0 + j0 + j] = dot[j];
  }
}

// ------------------------------------------- rows that do not start on 16 bytes

// Such rows are written by windows of 8 elements that start on 16 bytes; the
// same elements of another row lie in two blocks of 16 bytes, and are put together
// from them.  A row's first and last window have elements outside it, which are
// read where the matrix has them and count for nothing; a window whose blocks
// pass the matrix's ends is read by elements.  (4183 tokens of 4039, 5 choices:
// there 109 us by elements, 55 by windows; back 158 and 68.  Backward, whose
// windows take registers for two rows of each choice: 161 and 164 at best, and
// 53 and 71 for 2000 of 2049, so by elements.)

// Where a matrix's elements lie.
struct Extent {
  uintptr_t lo, hi;
  __device__ __forceinline__ Extent(const uint16_t* p, int64_t rows, int64_t ld, int64_t cols)
      : lo((uintptr_t)p), hi((uintptr_t)(p + (rows - 1) * ld + cols)) {}
  // Whether the blocks of the 8 elements from p on lie within.
  __device__ __forceinline__ bool holds(const uint16_t* p) const {
    const uintptr_t first = (uintptr_t)p & ~(uintptr_t)15;
    return first >= lo && first + ((uintptr_t)p & 15 ? 32 : 16) <= hi;
  }
};

__device__ __forceinline__ int phase_of(const uint16_t* p) { return (int)((uintptr_t)p >> 1 & 7); }

// The blocks of 8 elements, and those elements out of them.
struct Blocks {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4* q = (const uint4*)((uintptr_t)p & ~(uintptr_t)15);
    a = q[0];
    b = (uintptr_t)p & 15 ? q[1] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ Piece<8> at(uint32_t by) const {  // from so many bytes on
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = by & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = by & 4 ? w[i + 1] : w[i];
    Piece<8> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __funnelshift_r(w[i], w[i + 1], by & 2 ? 16 : 0);
    return r;
  }
};
// The 8 elements from e on of a row of `cols`, 0 for those outside it.
__device__ __noinline__ uint4 by_elements(const uint16_t* row, int64_t e, int64_t cols) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i >= 0 && e + i < cols) w[i / 2] |= (uint32_t)row[e + i] << (i % 2 * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ Piece<8> window(const uint16_t* row, int64_t e, int64_t cols, const Extent& x) {
  if (x.holds(row + e)) {
    Blocks b;
    b.load(row + e);
    return b.at((uintptr_t)(row + e) & 15);
  }
  const uint4 q = by_elements(row, e, cols);
  return Piece<8>{{q.x, q.y, q.z, q.w}};
}
// The 15 elements that windows of other rows, by their phases, have here: from
// 7 before the q-th 8 on.
__device__ __forceinline__ Blocks around(const uint16_t* row, int64_t q, int64_t cols, const Extent& x) {
  const Piece<8> a = window(row, q * 8 - 7, cols, x), b = window(row, q * 8 + 1, cols, x);
  return Blocks{make_uint4(a.w[0], a.w[1], a.w[2], a.w[3]), make_uint4(b.w[0], b.w[1], b.w[2], b.w[3])};
}
// To the 8 elements from e on of a row of `cols`, those outside it left out.
__device__ __forceinline__ void store_window(uint16_t* row, int64_t e, int64_t cols, const Piece<8>& v) {
  if (e >= 0 && e + 8 <= cols) {
    store<8>(row + e, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i >= 0 && e + i < cols) row[e + i] = (uint16_t)(v.w[i / 2] >> (i % 2 * 16));
}

template <int K>
__global__ void __launch_bounds__(kThreads) gather_windows_kernel(RowsArgs a, Shape s) {
  after_previous();
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  if (t >= a.tokens) return;
  const Extent x(a.in, a.tokens, a.ld_in, a.hidden);
  const uint16_t* from = a.in + t * a.ld_in;
  const int64_t p0 = t * a.topk;
  for (int j0 = 0; j0 < a.topk; j0 += K) {
    Slots<K> at;
    at.load(a, p0 + j0, a.topk - j0);
    for (int64_t q = threadIdx.x % s.lanes; q < s.pieces; q += s.lanes) {
      const Blocks v = around(from, q, a.hidden, x);
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (at.row[j] < 0) continue;
        uint16_t* to = a.out + at.row[j] * a.ld_out;
        const int phase = phase_of(to);
        if (q * 8 - phase < a.hidden) store_window(to, q * 8 - phase, a.hidden, v.at(2 * (7 - phase)));
      }
    }
  }
}

template <int K>
__global__ void __launch_bounds__(kThreads) combine_windows_kernel(RowsArgs a, Shape s) {
  after_previous();
  const int64_t t = (int64_t)blockIdx.x * s.tokens + threadIdx.x / s.lanes;
  if (t >= a.tokens) return;
  const Extent x(a.in, a.num_rows, a.ld_in, a.hidden);
  uint16_t* to = a.out + t * a.ld_out;
  const int64_t p0 = t * a.topk;
  Slots<K> at;
  at.load(a, p0, a.topk);
  for (int64_t q = threadIdx.x % s.lanes; q < s.pieces; q += s.lanes) {
    const int64_t e = q * 8 - phase_of(to);
    if (e >= a.hidden) break;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    const auto add = [&](const Piece<8>& v, float w) {
      float f[8];
      values<8>(v, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, f[i], sum[i]);
    };
    for (int j0 = 0;;) {
      bool within = true;
#pragma unroll
      for (int j = 0; j < K; ++j) within = within && (at.row[j] < 0 || x.holds(a.in + at.row[j] * a.ld_in + e));
      if (within) {
        Blocks b[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (at.row[j] >= 0) b[j].load(a.in + at.row[j] * a.ld_in + e);
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (at.row[j] >= 0) add(b[j].at((uintptr_t)(a.in + at.row[j] * a.ld_in + e) & 15), at.w[j]);
      } else {
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (at.row[j] >= 0) {
            const uint4 v = by_elements(a.in + at.row[j] * a.ld_in, e, a.hidden);
            add(Piece<8>{{v.x, v.y, v.z, v.w}}, at.w[j]);
          }
      }
      if (a.topk <= K) break;
      j0 = j0 + K < a.topk ? j0 + K : 0;
      at.load(a, p0 + j0, a.topk - j0);
      if (j0 == 0) break;
    }
    store_window(to, e, a.hidden, rounded<8>(sum));
  }
}

// As many lanes a token as it takes to give every SM `busy` threads, and no
// more than a row has pieces: fewer threads that stay longer wait less for
// slots, more have more loads on their way.  (4093 tokens x 2048 x 8, backward:
// 51 us with 256 to 768 threads, 57 with 1024, 79 with a CTA a token; results
// of 4096 x 4096 x 2 back: 19.6, 21 and 32; 8191 x 2048 x 8 there: 53 with up
// to 1024, 48.6 with 2048.)
Shape shape_of(const RowsArgs& a, int64_t pieces, int64_t busy, int sms) {
  Shape s{1, 0, pieces};
  while (s.lanes < kThreads && s.lanes < s.pieces && (s.lanes < 32 || s.lanes * a.tokens < sms * busy)) s.lanes *= 2;
  s.tokens = kThreads / s.lanes;
  return s;
}

cudaError_t run(void (*kernel)(RowsArgs, Shape), const RowsArgs& a, int64_t pieces, int64_t busy, int sms, cudaStream_t stream) {
  const Shape s = shape_of(a, pieces, busy, sms);
  return launch_early(kernel, dim3((unsigned)ceil_div(a.tokens, s.tokens)), kThreads, 0, 0, stream, a, s);
}

bool by8(const RowsArgs& a) {
  return a.hidden % 8 == 0 && a.ld_in % 8 == 0 && (!a.out || a.ld_out % 8 == 0) && (!a.dweights || a.ld_rows % 8 == 0);
}

// At most, of one row.
int64_t windows(const RowsArgs& a) { return (a.hidden + 14) / 8; }

}  // namespace

cudaError_t launch_expert_gather(const RowsArgs& a, int sms, cudaStream_t stream) {
  if (by8(a)) return run(a.topk <= 2 ? gather_kernel<8, 2> : gather_kernel<8, 8>, a, a.hidden / 8, 2048, sms, stream);
  // a short row's ends, which are written by elements, cost more than the rest
  // saves (4000 tokens of 333, 8 choices, their order too: 22 us, 19 by
  // elements; 8000 of 1023, 10 choices: 69 and 101)
  if (a.hidden < 512) return run(a.topk <= 2 ? gather_kernel<1, 2> : gather_kernel<1, 8>, a, a.hidden, 2048, sms, stream);
  return run(a.topk <= 2 ? gather_windows_kernel<2> : gather_windows_kernel<8>, a, windows(a), 2048, sms, stream);
}

cudaError_t launch_expert_combine(const RowsArgs& a, int sms, cudaStream_t stream) {
  if (by8(a)) {
    if (a.topk <= 4) return run(a.topk <= 2 ? combine_kernel<2, 4> : combine_kernel<4, 2>, a, a.hidden / 8, 512, sms, stream);
    return run(combine_kernel<8, 1>, a, a.hidden / 8, 2048, sms, stream);
  }
  return run(a.topk <= 2   ? combine_windows_kernel<2>
             : a.topk <= 4 ? combine_windows_kernel<4>
                           : combine_windows_kernel<8>,
             a, windows(a), 512, sms, stream);
}

cudaError_t launch_expert_combine_backward(const RowsArgs& a, int sms, cudaStream_t stream) {
  if (by8(a)) return run(a.topk <= 2 ? combine_backward_kernel<8, 2, 1> : combine_backward_kernel<8, 8, 1>, a, a.hidden / 8, 512, sms, stream);
  return run(a.topk <= 2 ? combine_backward_kernel<1, 2, 8> : combine_backward_kernel<1, 8, 4>, a, a.hidden, 256, sms, stream);
}

}  // namespace tide
