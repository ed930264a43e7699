// Plain tiled kernels of the feed-forward unit's products, for every size,
// stride and alignment.  Single elements are loaded, products and sums are
// fp32 on the CUDA cores: these are the right answers where rows do not
// start on 16 bytes, which the tensor-core kernels' copies need, not the
// fast ones (1000 x 500 x 8000, forward and backward in bf16: 3.4 ms, where
// 1000 x 512 x 8192 takes 0.06).
#include "compute_device.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;
constexpr int kTm = 32;   // rows of a tile
constexpr int kTn = 128;  // columns of a tile: one scale block
constexpr int kTk = 16;   // contraction step

// Each thread owns rows ty + 8 i (i < 4) and columns tx + 32 j (j < 4): a
// warp is one row of tx, so its column accesses are neighbours.
struct Tile4 {
  float v[4][4];
};

__device__ __forceinline__ void clear(Tile4& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) t.v[i][j] = 0.0f;
}

// c += A[rows of the tile, k0..] B[k0.., columns of the tile], both read by
// single elements through `av(row, k)` and `bv(k, col)`, which return 0 out
// of range.  AK / BK: consecutive k are neighbours in memory (else
// consecutive rows / columns are), which decides the order threads load in.
template <bool AK, bool BK, class Av, class Bv>
__device__ __forceinline__ void step(float (*as)[kTm + 1], float (*bs)[kTn + 1], Tile4& c, Av av, Bv bv) {
  const int t = threadIdx.x, tx = t & 31, ty = t >> 5;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTm * kTk / kThreads; ++i) {
    const int e = t + i * kThreads;
    const int k = AK ? e % kTk : e / kTm, r = AK ? e / kTk : e % kTm;
    as[k][r] = av(r, k);
  }
#pragma unroll
  for (int i = 0; i < kTn * kTk / kThreads; ++i) {
    const int e = t + i * kThreads;
    const int k = BK ? e % kTk : e / kTn, n = BK ? e / kTk : e % kTn;
    bs[k][n] = bv(k, n);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTk; ++k) {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = as[k][ty + 8 * i];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = bs[k][tx + 32 * j];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c.v[i][j] = fmaf(a[i], b[j], c.v[i][j]);
  }
}

// Both projections of a 32 x 128 tile, then either h (and the checkpoint) or
// dG, dU (and h).  The tile is one scale block wide, so a row's maximum is a
// warp's.
template <int ACT, bool GRAD>
__global__ void __launch_bounds__(kThreads) gated_simple_kernel(GatedArgs a) {
  __shared__ float as[kTk][kTm + 1];
  __shared__ float bs[kTk][kTn + 1];
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = (int64_t)blockIdx.y * kTn;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  Tile4 g, u;
  clear(g);
  clear(u);
  for (int64_t k0 = 0; k0 < a.hidden; k0 += kTk) {
    auto xv = [&](int r, int k) {
      return row0 + r < a.tokens && k0 + k < a.hidden ? bf16_value(a.x[(row0 + r) * a.ldx + k0 + k]) : 0.0f;
    };
    auto wv = [&](const uint16_t* w, int k, int n) {
      return col0 + n < a.ffn && k0 + k < a.hidden ? bf16_value(w[(col0 + n) * a.hidden + k0 + k]) : 0.0f;
    };
    step<true, true>(as, bs, g, xv, [&](int k, int n) { return wv(a.wg, k, n); });
    step<true, true>(as, bs, u, xv, [&](int k, int n) { return wv(a.wu, k, n); });
  }
  const int64_t nb = (a.ffn + kBlock - 1) / kBlock;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + ty + 8 * i;
    if (row >= a.tokens) continue;  // the whole warp
    float gmax = 0.0f, umax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t col = col0 + tx + 32 * j;
      gmax = fmaxf(gmax, fabsf(no_infinity(g.v[i][j])));  // columns past the end hold 0
      umax = fmaxf(umax, fabsf(no_infinity(u.v[i][j])));
      if (col >= a.ffn) continue;
      if (GRAD) {
        const float d = bf16_value(a.dh[row * a.lddh + col]);
        const float2 t = activation_grad<ACT>(g.v[i][j]);
        a.dg[row * a.ffn + col] = to_bf16(d * u.v[i][j] * t.y);
        a.du[row * a.ffn + col] = to_bf16(d * t.x);
        if (a.h) a.h[row * a.ldh + col] = to_bf16(t.x * u.v[i][j]);
      } else {
        a.h[row * a.ldh + col] = to_bf16(activation<ACT>(g.v[i][j]) * u.v[i][j]);
      }
    }
    if constexpr (!GRAD) {
      if (!a.g8) continue;
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        gmax = fmaxf(gmax, __shfl_xor_sync(0xffffffffu, gmax, d));
        umax = fmaxf(umax, __shfl_xor_sync(0xffffffffu, umax, d));
      }
      const uint32_t eg = scale_exponent(gmax), eu = scale_exponent(umax);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t col = col0 + tx + 32 * j;
        if (col >= a.ffn) continue;
        a.g8[row * a.ffn + col] = (uint8_t)pack_e4m3(no_infinity(g.v[i][j]) * exponent_inverse(eg), 0.0f);
        a.u8[row * a.ffn + col] = (uint8_t)pack_e4m3(no_infinity(u.v[i][j]) * exponent_inverse(eu), 0.0f);
      }
      if (tx == 0) {
        a.gs[row * nb + blockIdx.y] = exponent_value(eg);
        a.us[row * nb + blockIdx.y] = exponent_value(eu);
      }
    }
  }
}

__device__ __forceinline__ void write_tile(const Tile4& c, uint16_t* out, int64_t ld, int64_t row0, int64_t col0,
                                           int64_t rows, int64_t cols) {
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = row0 + ty + 8 * i, col = col0 + tx + 32 * j;
      if (row < rows && col < cols) out[row * ld + col] = to_bf16(c.v[i][j]);
    }
}

// dX = dG Wg + dU Wu.
__global__ void __launch_bounds__(kThreads) dx_simple_kernel(GatedArgs a) {
  __shared__ float as[kTk][kTm + 1];
  __shared__ float bs[kTk][kTn + 1];
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = (int64_t)blockIdx.y * kTn;
  Tile4 c;
  clear(c);
  for (int64_t k0 = 0; k0 < a.ffn; k0 += kTk) {
    auto dv = [&](const uint16_t* d, int r, int k) {
      return row0 + r < a.tokens && k0 + k < a.ffn ? bf16_value(d[(row0 + r) * a.ffn + k0 + k]) : 0.0f;
    };
    auto wv = [&](const uint16_t* w, int k, int n) {
      return col0 + n < a.hidden && k0 + k < a.ffn ? bf16_value(w[(k0 + k) * a.hidden + col0 + n]) : 0.0f;
    };
    step<true, false>(as, bs, c, [&](int r, int k) { return dv(a.dg, r, k); },
                      [&](int k, int n) { return wv(a.wg, k, n); });
    step<true, false>(as, bs, c, [&](int r, int k) { return dv(a.du, r, k); },
                      [&](int k, int n) { return wv(a.wu, k, n); });
  }
  write_tile(c, a.dx, a.lddx, row0, col0, a.tokens, a.hidden);
}

// dWg = dG^T X (z = 0), dWu = dU^T X (z = 1).
__global__ void __launch_bounds__(kThreads) dw_simple_kernel(GatedArgs a) {
  __shared__ float as[kTk][kTm + 1];
  __shared__ float bs[kTk][kTn + 1];
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = (int64_t)blockIdx.y * kTn;
  const uint16_t* d = blockIdx.z ? a.du : a.dg;
  Tile4 c;
  clear(c);
  for (int64_t k0 = 0; k0 < a.tokens; k0 += kTk)
    step<false, false>(
        as, bs, c,
        [&](int r, int k) {
          return row0 + r < a.ffn && k0 + k < a.tokens ? bf16_value(d[(k0 + k) * a.ffn + row0 + r]) : 0.0f;
        },
        [&](int k, int n) {
          return col0 + n < a.hidden && k0 + k < a.tokens ? bf16_value(a.x[(k0 + k) * a.ldx + col0 + n]) : 0.0f;
        });
  write_tile(c, blockIdx.z ? a.dwu : a.dwg, a.hidden, row0, col0, a.ffn, a.hidden);
}

// out = sum over 128-wide blocks of sa sb (codes' product).
__global__ void __launch_bounds__(kThreads) matmul_simple_kernel(MatmulArgs a) {
  __shared__ float as[kTk][kTm + 1];
  __shared__ float bs[kTk][kTn + 1];
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = (int64_t)blockIdx.y * kTn;
  const int64_t nb = (a.k + kBlock - 1) / kBlock;
  const int ty = threadIdx.x >> 5;
  Tile4 sum;
  clear(sum);
  for (int64_t kb = 0; kb < nb; ++kb) {
    Tile4 c;
    clear(c);
    for (int64_t k0 = kb * kBlock; k0 < a.k && k0 < (kb + 1) * kBlock; k0 += kTk)
      step<true, true>(
          as, bs, c,
          [&](int r, int k) {
            return row0 + r < a.m && k0 + k < a.k ? e4m3_values(a.a[(row0 + r) * a.k + k0 + k]).x : 0.0f;
          },
          [&](int k, int n) {
            return col0 + n < a.n && k0 + k < a.k ? e4m3_values(a.b[(col0 + n) * a.k + k0 + k]).x : 0.0f;
          });
    const auto scale = [&](float s) { return a.any_scales ? s : power_of_two(s); };
    const float sb = scale(a.sb[blockIdx.y * nb + kb]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = row0 + ty + 8 * i;
      const float s = row < a.m ? scale(a.sa[row * nb + kb]) * sb : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum.v[i][j] = fmaf(c.v[i][j], s, sum.v[i][j]);
    }
  }
  write_tile(sum, a.out, a.ldo, row0, col0, a.m, a.n);
}

dim3 grid_of(int64_t rows, int64_t cols, unsigned z = 1) {
  return dim3((unsigned)ceil_div(rows, kTm), (unsigned)ceil_div(cols, kTn), z);
}

template <int ACT>
cudaError_t gated(const GatedArgs& a, bool grad, cudaStream_t stream) {
  if (grad)
    gated_simple_kernel<ACT, true><<<grid_of(a.tokens, a.ffn), kThreads, 0, stream>>>(a);
  else
    gated_simple_kernel<ACT, false><<<grid_of(a.tokens, a.ffn), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_forward_simple(const GatedArgs& a, cudaStream_t stream) {
  return a.act == TIDE_ACT_SILU ? gated<TIDE_ACT_SILU>(a, false, stream) : gated<TIDE_ACT_GELU>(a, false, stream);
}

cudaError_t launch_gated_grad_simple(const GatedArgs& a, cudaStream_t stream) {
  return a.act == TIDE_ACT_SILU ? gated<TIDE_ACT_SILU>(a, true, stream) : gated<TIDE_ACT_GELU>(a, true, stream);
}

cudaError_t launch_gated_dx_simple(const GatedArgs& a, cudaStream_t stream) {
  dx_simple_kernel<<<grid_of(a.tokens, a.hidden), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_gated_dw_simple(const GatedArgs& a, cudaStream_t stream) {
  dw_simple_kernel<<<grid_of(a.ffn, a.hidden, 2), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_fp8_matmul_simple(const MatmulArgs& a, cudaStream_t stream) {
  matmul_simple_kernel<<<grid_of(a.m, a.n), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tide
