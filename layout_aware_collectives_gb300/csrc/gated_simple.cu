// The feed-forward unit's products for every size, stride and alignment, where
// rows do not start on 16 bytes as the tensor-map copies of the other kernels
// need.  Elements are loaded one by one, a tile ahead, and multiplied by warp
// instructions of the tensor cores; sums are fp32.
//
// Bound by the loads, 64 x 128 tiles of single elements: 1000 x 500 x 8001 in
// bf16 takes 167 us forward and 0.9 ms backward, where 1000 x 512 x 8192 takes
// 19 and 62.  (Loads of a step that wait for one another, as conditional ones
// do, made it 519 and 2.7 ms; fp32 products on the CUDA cores 758 and 3.4.)
#include "compute_device.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;  // 2 x 4 warps of 32 x 32
constexpr int kTm = 64;        // rows of a tile
constexpr int kTn = 128;       // columns of a tile: one scale block
constexpr int kTk = 32;        // contraction step: 16 words of two elements
constexpr int kPitch = 20;     // words of a row in shared memory: a fragment's rows fall into different banks

// One warp's 32 x 32 sums: [row / 16][column / 8], element i of a fragment at
// row lane / 4 + 8 (i / 2), column 2 (lane % 4) + i % 2.
struct Sums {
  float v[2][4][4];
};

__device__ __forceinline__ void clear(Sums& s) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) s.v[i][j][q] = 0.0f;
}

// Columns of tiles run along blockIdx.y and, WIDE, past kAcross of them, which
// a grid's y does not hold, along blockIdx.z in runs of kAcross.  (Taken that
// way or along x for every width, 1000 x 500 x 8001 forward takes 180 us and
// not 168: blockIdx.y's range spares 64-bit products of addresses.)
constexpr int64_t kAcross = 32768;
template <bool WIDE>
__device__ __forceinline__ int64_t first_col(unsigned run) {
  return WIDE ? (run * kAcross + blockIdx.y) * kTn : (int64_t)blockIdx.y * kTn;
}

struct At {
  int row, col;
};
// Where element q of fragment (i, j) lies in the tile.
__device__ __forceinline__ At element(int i, int j, int q) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  return At{(warp & 1) * 32 + i * 16 + (lane >> 2) + 8 * (q >> 1), (warp >> 1) * 32 + j * 8 + 2 * (lane & 3) + (q & 1)};
}

__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What an element out of range is read from: so every load is made, and all of
// a step's are on their way together.
__device__ uint32_t nothing = 0;

// Two elements of a step: where they lie.
template <class T>
struct Two {
  const T *lo, *hi;
};

// Elements k and k + 1 of `size`, at `at` and `stride` on; if `in`, in range.
template <class T>
__device__ __forceinline__ Two<T> two(const T* at, int64_t stride, int64_t k, int64_t size, bool in) {
  return Two<T>{in && k < size ? at : (const T*)&nothing, in && k + 1 < size ? at + stride : (const T*)&nothing};
}

__device__ __forceinline__ uint32_t word(uint16_t lo, uint16_t hi) { return (uint32_t)lo | (uint32_t)hi << 16; }
// Two codes as bf16, which holds every e4m3 value.
__device__ __forceinline__ uint32_t word(uint8_t lo, uint8_t hi) {
  const float2 v = e4m3_values((uint16_t)(lo | hi << 8));
  return pack_bf16(v.x, v.y);
}

// sums[p] += A B_p over `steps` steps of the contraction.  a(step, row, w) and
// b(step, p, column, w) say where word w (elements 2 w and 2 w + 1) of a row's
// or a column's step lies.  AK / BK: the contraction lies along memory (else
// rows / columns do), which decides who loads what.
template <class T, int PRODUCTS, bool AK, bool BK, class A, class B>
__device__ __forceinline__ void multiply(int64_t steps, Sums (&sums)[PRODUCTS], A a, B b) {
  constexpr int kWords = kTk / 2;
  constexpr int kA = kTm * kWords / kThreads, kB = kTn * kWords / kThreads;
  __shared__ uint32_t as[kTm * kPitch], bs[PRODUCTS][kTn * kPitch];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  T ra[kA][2], rb[PRODUCTS][kB][2];
  const auto a_row = [&](int i) { return AK ? (t + i * kThreads) / kWords : (t + i * kThreads) % kTm; };
  const auto a_word = [&](int i) { return AK ? (t + i * kThreads) % kWords : (t + i * kThreads) / kTm; };
  const auto b_col = [&](int i) { return BK ? (t + i * kThreads) / kWords : (t + i * kThreads) % kTn; };
  const auto b_word = [&](int i) { return BK ? (t + i * kThreads) % kWords : (t + i * kThreads) / kTn; };
  const auto load = [&](int64_t s) {
#pragma unroll
    for (int i = 0; i < kA; ++i) {
      const Two<T> at = a(s, a_row(i), a_word(i));
      ra[i][0] = *at.lo, ra[i][1] = *at.hi;
    }
#pragma unroll
    for (int p = 0; p < PRODUCTS; ++p)
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        const Two<T> at = b(s, p, b_col(i), b_word(i));
        rb[p][i][0] = *at.lo, rb[p][i][1] = *at.hi;
      }
  };
  if (steps > 0) load(0);
  for (int64_t s = 0; s < steps; ++s) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kA; ++i) as[a_row(i) * kPitch + a_word(i)] = word(ra[i][0], ra[i][1]);
#pragma unroll
    for (int p = 0; p < PRODUCTS; ++p)
#pragma unroll
      for (int i = 0; i < kB; ++i) bs[p][b_col(i) * kPitch + b_word(i)] = word(rb[p][i][0], rb[p][i][1]);
    __syncthreads();
    if (s + 1 < steps) load(s + 1);
#pragma unroll
    for (int k = 0; k < kWords; k += 8) {
      uint32_t fa[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t* at = as + ((warp & 1) * 32 + i * 16 + (lane >> 2)) * kPitch + k + (lane & 3);
        fa[i][0] = at[0], fa[i][1] = at[8 * kPitch], fa[i][2] = at[4], fa[i][3] = at[8 * kPitch + 4];
      }
#pragma unroll
      for (int p = 0; p < PRODUCTS; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t* at = bs[p] + ((warp >> 1) * 32 + j * 8 + (lane >> 2)) * kPitch + k + (lane & 3);
          const uint32_t b0 = at[0], b1 = at[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) mma16(sums[p].v[i][j], fa[i], b0, b1);
        }
    }
  }
}

// A block's magnitudes, row by row: the largest over the tile's four warps of
// columns.  `best` is this thread's largest for each of its four rows.
__device__ __forceinline__ void row_maxima(float (&best)[2][2]) {
  __shared__ float part[4][kTm];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float m = best[i][h];
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      if ((lane & 3) == 0) part[warp >> 1][element(i, 0, 2 * h).row] = m;
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = element(i, 0, 2 * h).row;
      best[i][h] = fmaxf(fmaxf(part[0][row], part[1][row]), fmaxf(part[2][row], part[3][row]));
    }
}

// Codes and scales of one pre-activation's tile, which is one scale block wide.
__device__ __forceinline__ void put_blocks(const Sums& s, uint8_t* codes, float* scales, int64_t row0, int64_t col0,
                                           const GatedArgs& a) {
  const int64_t nb = (a.ffn + kBlock - 1) / kBlock;
  float best[2][2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)  // columns past the end hold 0 (or NaN, which is passed over)
        best[i][q >> 1] = fmaxf(best[i][q >> 1], fabsf(no_infinity(s.v[i][j][q])));
  row_maxima(best);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = row0 + element(i, 0, 2 * h).row;
      if (row >= a.tokens) continue;
      const uint32_t e = scale_exponent(best[i][h]);
      if (element(0, 0, 0).col == 0) scales[row * nb + col0 / kBlock] = exponent_value(e);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t col = col0 + element(i, j, q).col;
          if (col < a.ffn)
            codes[row * a.ffn + col] = (uint8_t)pack_e4m3(no_infinity(s.v[i][j][2 * h + q]) * exponent_inverse(e), 0.0f);
        }
    }
}

// Both projections of a tile, then either h (and the checkpoint) or dG, dU
// (and h).
template <int ACT, bool GRAD, bool WIDE>
__global__ void __launch_bounds__(kThreads) gated_simple_kernel(GatedArgs a) {
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = first_col<WIDE>(blockIdx.z);
  if (WIDE && col0 >= a.ffn) return;
  Sums sums[2];
  clear(sums[0]);
  clear(sums[1]);
  multiply<uint16_t, 2, true, true>(
      (a.hidden + kTk - 1) / kTk, sums,
      [&](int64_t s, int r, int w) {
        const int64_t k = s * kTk + 2 * w;
        return two(a.x + (row0 + r) * a.ldx + k, 1, k, a.hidden, row0 + r < a.tokens);
      },
      [&](int64_t s, int p, int n, int w) {
        const int64_t k = s * kTk + 2 * w;
        return two((p ? a.wu : a.wg) + (col0 + n) * a.hidden + k, 1, k, a.hidden, col0 + n < a.ffn);
      });
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const At at = element(i, j, q);
        const int64_t row = row0 + at.row, col = col0 + at.col;
        if (row >= a.tokens || col >= a.ffn) continue;
        const float g = sums[0].v[i][j][q], u = sums[1].v[i][j][q];
        if (GRAD) {
          const float d = bf16_value(a.dh[row * a.lddh + col]);
          const float2 t = activation_grad<ACT>(g);
          a.dg[row * a.ffn + col] = to_bf16(d * u * t.y);
          a.du[row * a.ffn + col] = to_bf16(d * t.x);
          if (a.h) a.h[row * a.ldh + col] = to_bf16(t.x * u);
        } else {
          a.h[row * a.ldh + col] = to_bf16(activation<ACT>(g) * u);
        }
      }
  if constexpr (!GRAD) {
    if (!a.g8) return;
    put_blocks(sums[0], a.g8, a.gs, row0, col0, a);
    put_blocks(sums[1], a.u8, a.us, row0, col0, a);
  }
}

__device__ __forceinline__ void write_tile(const Sums& s, uint16_t* out, int64_t ld, int64_t row0, int64_t col0,
                                           int64_t rows, int64_t cols) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const At at = element(i, j, q);
        const int64_t row = row0 + at.row, col = col0 + at.col;
        if (row < rows && col < cols) out[row * ld + col] = to_bf16(s.v[i][j][q]);
      }
}

// dX = dG Wg + dU Wu.
template <bool WIDE>
__global__ void __launch_bounds__(kThreads) dx_simple_kernel(GatedArgs a) {
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = first_col<WIDE>(blockIdx.z);
  if (WIDE && col0 >= a.hidden) return;
  const int64_t half = (a.ffn + kTk - 1) / kTk;
  Sums sums[1];
  clear(sums[0]);
  multiply<uint16_t, 1, true, false>(
      2 * half, sums,
      [&](int64_t s, int r, int w) {
        const int64_t k = (s < half ? s : s - half) * kTk + 2 * w;
        const uint16_t* d = s < half ? a.dg : a.du;
        return two(d + (row0 + r) * a.ffn + k, 1, k, a.ffn, row0 + r < a.tokens);
      },
      [&](int64_t s, int, int n, int w) {
        const int64_t k = (s < half ? s : s - half) * kTk + 2 * w;
        const uint16_t* wt = s < half ? a.wg : a.wu;
        return two(wt + k * a.hidden + col0 + n, a.hidden, k, a.ffn, col0 + n < a.hidden);
      });
  write_tile(sums[0], a.dx, a.lddx, row0, col0, a.tokens, a.hidden);
}

// dWg = dG^T x (z = 0; WIDE: even), dWu = dU^T x (z = 1; odd).
template <bool WIDE>
__global__ void __launch_bounds__(kThreads) dw_simple_kernel(GatedArgs a) {
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = first_col<WIDE>(blockIdx.z >> 1);
  if (WIDE && col0 >= a.hidden) return;
  const uint16_t* d = (WIDE ? blockIdx.z & 1 : blockIdx.z) ? a.du : a.dg;
  Sums sums[1];
  clear(sums[0]);
  multiply<uint16_t, 1, false, false>(
      (a.tokens + kTk - 1) / kTk, sums,
      [&](int64_t s, int r, int w) {
        const int64_t k = s * kTk + 2 * w;
        return two(d + k * a.ffn + row0 + r, a.ffn, k, a.tokens, row0 + r < a.ffn);
      },
      [&](int64_t s, int, int n, int w) {
        const int64_t k = s * kTk + 2 * w;
        return two(a.x + k * a.ldx + col0 + n, a.ldx, k, a.tokens, col0 + n < a.hidden);
      });
  write_tile(sums[0], (WIDE ? blockIdx.z & 1 : blockIdx.z) ? a.dwu : a.dwg, a.hidden, row0, col0, a.ffn, a.hidden);
}

// out = sum over 128-wide blocks of sa sb (codes' product).
template <bool WIDE>
__global__ void __launch_bounds__(kThreads) matmul_simple_kernel(MatmulArgs a) {
  const int64_t row0 = (int64_t)blockIdx.x * kTm, col0 = first_col<WIDE>(blockIdx.z);
  if (WIDE && col0 >= a.n) return;
  const int64_t nb = (a.k + kBlock - 1) / kBlock;
  Sums total;
  clear(total);
  for (int64_t kb = 0; kb < nb; ++kb) {
    Sums sums[1];
    clear(sums[0]);
    const int64_t k0 = kb * kBlock, wide = a.k - k0 < kBlock ? a.k - k0 : kBlock;
    multiply<uint8_t, 1, true, true>(
        (wide + kTk - 1) / kTk, sums,
        [&](int64_t s, int r, int w) {
          const int64_t k = s * kTk + 2 * w;
          return two(a.a + (row0 + r) * a.k + k0 + k, 1, k, wide, row0 + r < a.m);
        },
        [&](int64_t s, int, int n, int w) {
          const int64_t k = s * kTk + 2 * w;
          return two(a.b + (col0 + n) * a.k + k0 + k, 1, k, wide, col0 + n < a.n);
        });
    const auto scale = [&](float s) { return a.any_scales ? s : power_of_two(s); };
    float sb = scale(a.sb[(WIDE ? col0 / kTn : blockIdx.y) * nb + kb]);
    const float power = leave_power(sb);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = row0 + element(i, 0, 2 * h).row;
        const float s = row < a.m ? take_power(scale(a.sa[row * nb + kb]), power) : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            total.v[i][j][2 * h + q] = fmaf(sums[0].v[i][j][2 * h + q] * sb, s, total.v[i][j][2 * h + q]);
      }
  }
  write_tile(total, a.out, a.ldo, row0, col0, a.m, a.n);
}

template <class Args>
using Kernel = void (*)(Args);

// The kernel for so many columns, on its grid.
template <class Args>
cudaError_t run(Kernel<Args> usual, Kernel<Args> wide, int64_t rows, int64_t cols, unsigned z, const Args& a,
                cudaStream_t stream) {
  const unsigned down = (unsigned)ceil_div(rows, kTm);
  const int64_t tiles = ceil_div(cols, kTn);
  if (tiles <= kAcross)
    usual<<<dim3(down, (unsigned)tiles, z), kThreads, 0, stream>>>(a);
  else
    wide<<<dim3(down, (unsigned)kAcross, z * (unsigned)ceil_div(tiles, kAcross)), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int ACT, bool GRAD>
cudaError_t gated(const GatedArgs& a, cudaStream_t stream) {
  return run<GatedArgs>(gated_simple_kernel<ACT, GRAD, false>, gated_simple_kernel<ACT, GRAD, true>, a.tokens, a.ffn, 1, a,
                        stream);
}

}  // namespace

cudaError_t launch_gated_forward_simple(const GatedArgs& a, cudaStream_t stream) {
  return a.act == TIDE_ACT_SILU ? gated<TIDE_ACT_SILU, false>(a, stream) : gated<TIDE_ACT_GELU, false>(a, stream);
}

cudaError_t launch_gated_grad_simple(const GatedArgs& a, cudaStream_t stream) {
  return a.act == TIDE_ACT_SILU ? gated<TIDE_ACT_SILU, true>(a, stream) : gated<TIDE_ACT_GELU, true>(a, stream);
}

cudaError_t launch_gated_dx_simple(const GatedArgs& a, cudaStream_t stream) {
  return run<GatedArgs>(dx_simple_kernel<false>, dx_simple_kernel<true>, a.tokens, a.hidden, 1, a, stream);
}

cudaError_t launch_gated_dw_simple(const GatedArgs& a, cudaStream_t stream) {
  return run<GatedArgs>(dw_simple_kernel<false>, dw_simple_kernel<true>, a.ffn, a.hidden, 2, a, stream);
}

cudaError_t launch_fp8_matmul_simple(const MatmulArgs& a, cudaStream_t stream) {
  return run<MatmulArgs>(matmul_simple_kernel<false>, matmul_simple_kernel<true>, a.m, a.n, 1, a, stream);
}

}  // namespace tide
