// The 8-bit block format of activations and weights: store, restore, and the
// gated block's gradients from stored pre-activations.
//
// Every kernel here is one pass over its data, bound by HBM: 28672 x 8192 to
// 128 x 128 blocks 100 us (7.0 TB/s), to 1 x 128 blocks 120 us (5.9; one
// scale written for each 128 codes), back 105 us (6.7); the gradients of 4096
// x 28672 stored pre-activations 140 us (6.7).  Rows that do not start on 16
// bytes are taken by single elements, 32 threads side by side: 8191 x 20001
// to blocks in 162-227 us (2.2-3.0 TB/s), back in 121 (4.1).  A restore into
// strided rows takes them so whatever the stride: 28672 x 8192 in 593 us (1.2).
#include "compute_device.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;
// Up to here indexes are 32-bit (no grid overshoots it by 2^30), whose
// divisions are a third of the 64-bit ones' instructions.
constexpr int64_t kSmall = (int64_t)3 << 30;

template <class... P, class... A>
cudaError_t run(void (*kernel)(P...), unsigned grid, cudaStream_t stream, const A&... args) {
  return launch_early(kernel, dim3(grid), kThreads, 0, 0, stream, args...);
}

// ------------------------------------------------------------------ store

// Magnitudes of packed bf16 are ordered as 16-bit whole numbers, infinity at
// 0x7f80 and NaN above: two elements a comparison.
constexpr uint32_t kInf16 = 0x7f80;

template <int N>
__device__ __forceinline__ uint32_t packed_max(const uint32_t (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = __vmaxu2(m, v[i] & 0x7fff7fffu);
  return m;
}
// The same without infinities and NaN.
template <int N>
__device__ __forceinline__ uint32_t packed_max_finite(const uint32_t (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t lo = v[i] & 0x7fffu, hi = (v[i] >> 16) & 0x7fffu;
    m = __vmaxu2(m, (lo < kInf16 ? lo : 0) | ((hi < kInf16 ? hi : 0) << 16));
  }
  return m;
}
__device__ __forceinline__ uint32_t fold(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// 8 packed bf16 to 8 codes.
template <bool CLEAN>
__device__ __forceinline__ uint2 codes8(const uint32_t (&w)[4], float inv) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(w[j]);
    f[2 * j + 1] = bf16_hi(w[j]);
  }
  if (!CLEAN)
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = no_infinity(f[j]);
  return make_uint2(pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// One scale for each 1 x 128: half a warp takes a block, 8 columns (16
// bytes) a lane, so the block's maximum is four shuffles and nothing is read
// twice.  U blocks are loaded before the first is reduced.
template <int U, class Index>
__global__ void __launch_bounds__(kThreads) store_rows_kernel(Fp8Args a, Index blocks_per_row, Index blocks) {
  after_previous();
  const int lane = threadIdx.x & 15;
  const Index group = (Index)blockIdx.x * (U * kThreads / 16) + (threadIdx.x >> 4);
  uint32_t v[U][4];
  int64_t row[U], col[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Index blk = group + (Index)(i * (kThreads / 16));
    const Index r = blk / blocks_per_row;
    row[i] = blk < blocks ? (int64_t)r : -1;
    col[i] = (int64_t)(blk - r * blocks_per_row) * kBlock + lane * 8;
    uint4 q = make_uint4(0, 0, 0, 0);
    if (row[i] >= 0 && col[i] < a.cols) q = __ldcs((const uint4*)(a.bf16 + row[i] * a.ld + col[i]));
    v[i][0] = q.x, v[i][1] = q.y, v[i][2] = q.z, v[i][3] = q.w;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    uint32_t m = packed_max(v[i]);
#pragma unroll
    for (int d = 8; d; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = fold(m);
    const bool clean = !__any_sync(0xffffffffu, m >= kInf16);
    if (!clean) {
      m = packed_max_finite(v[i]);
#pragma unroll
      for (int d = 8; d; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
      m = fold(m);
    }
    const uint32_t e = scale_exponent(bf16_lo(m));
    const float inv = exponent_inverse(e);
    if (row[i] < 0) continue;
    if (col[i] < a.cols)
      __stcs((uint2*)(a.codes + row[i] * a.cols + col[i]), clean ? codes8<true>(v[i], inv) : codes8<false>(v[i], inv));
    if (lane == 0) a.scales[row[i] * blocks_per_row + col[i] / kBlock] = exponent_value(e);
  }
}

// The same for rows whose stride or width is no multiple of 8: a warp takes
// a block, 4 single columns a lane, 32 apart.
template <int U, class Index>
__global__ void __launch_bounds__(kThreads) store_rows_any_kernel(Fp8Args a, Index blocks_per_row, Index blocks) {
  after_previous();
  const int lane = threadIdx.x & 31;
  const Index warp = (Index)blockIdx.x * (U * kThreads / 32) + (threadIdx.x >> 5);
  uint16_t v[U][4];
  int wide[U];  // columns of the block from this lane's first on
  int64_t at[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Index blk = warp + (Index)(i * (kThreads / 32));
    const Index r = blk / blocks_per_row, b = blk - r * blocks_per_row;
    const int64_t col = (int64_t)b * kBlock + lane;
    wide[i] = blk < blocks ? (int)min((int64_t)kBlock, a.cols - col) : 0;
    at[i] = (int64_t)r * a.cols + col;
    const uint16_t* src = a.bf16 + (int64_t)r * a.ld + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = 32 * j < wide[i] ? src[32 * j] : 0;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float f[4], amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = no_infinity(bf16_value(v[i][j]));
      amax = fmaxf(amax, fabsf(f[j]));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    const uint32_t e = scale_exponent(amax);
    const float inv = exponent_inverse(e);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (32 * j < wide[i]) a.codes[at[i] + 32 * j] = (uint8_t)pack_e4m3(f[j] * inv, 0.0f);
    const Index blk = warp + (Index)(i * (kThreads / 32));
    if (lane == 0 && blk < blocks) a.scales[blk] = exponent_value(e);
  }
}

// One scale for each 128 x 128: a CTA holds the whole block in registers
// (VEC: 8 16-byte vectors a thread; else 64 single columns), so it is read
// once.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) store_square_kernel(Fp8Args a, uint32_t blocks_per_row) {
  after_previous();
  constexpr int kPerLoad = VEC ? 8 : 1;
  constexpr int kLanes = kBlock / kPerLoad;        // threads across a row
  constexpr int kRows = kThreads / kLanes;         // rows a pass
  constexpr int kPasses = kBlock / kRows;
  constexpr int kWords = VEC ? 4 : 1;
  __shared__ uint32_t part[2][kThreads / 32];
  const uint32_t br = blockIdx.x / blocks_per_row, bc = blockIdx.x - br * blocks_per_row;
  const int64_t col = (int64_t)bc * kBlock + (threadIdx.x % kLanes) * kPerLoad;
  const int64_t row0 = (int64_t)br * kBlock + threadIdx.x / kLanes;
  const int high = col < a.cols ? (int)min((int64_t)kBlock, a.rows - row0) : 0;  // rows from this thread's first on
  const uint16_t* src = a.bf16 + row0 * a.ld + col;
  uint8_t* dst = a.codes + row0 * a.cols + col;
  uint32_t v[kPasses][kWords];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const bool in = p * kRows < high;
    if constexpr (VEC) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (in) q = __ldcs((const uint4*)src);
      v[p][0] = q.x, v[p][1] = q.y, v[p][2] = q.z, v[p][3] = q.w;
    } else {
      v[p][0] = in ? *src : 0;
    }
    src += kRows * a.ld;
  }
  // the block's maximum, of 32-bit words that each hold two magnitudes
  const auto all = [&](uint32_t m, int turn) {
#pragma unroll
    for (int d = 16; d; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = __vmaxu2(m, part[turn][w]);
    return fold(m);
  };
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) m = __vmaxu2(m, packed_max(v[p]));
  m = all(m, 0);
  const bool clean = m < kInf16;  // the same for the whole CTA
  if (!clean) {
    m = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) m = __vmaxu2(m, packed_max_finite(v[p]));
    m = all(m, 1);
  }
  const uint32_t e = scale_exponent(bf16_lo(m));
  const float inv = exponent_inverse(e);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    if (p * kRows < high) {
      if constexpr (VEC)
        __stcs((uint2*)dst, clean ? codes8<true>(v[p], inv) : codes8<false>(v[p], inv));
      else
        *dst = (uint8_t)pack_e4m3(no_infinity(bf16_lo(v[p][0])) * inv, 0.0f);
    }
    dst += kRows * a.cols;
  }
  if (threadIdx.x == 0) a.scales[blockIdx.x] = exponent_value(e);
}

// ---------------------------------------------------------------- restore

__device__ __forceinline__ float scale_at(const Fp8Args& a, int64_t blocks_per_row, int64_t row, int64_t col) {
  return a.scales[(a.block_rows == 1 ? row : row / kBlock) * blocks_per_row + col / kBlock];
}

// Contiguous on both sides: the matrix is one run of elements, taken 8 at a
// time (8 bytes of codes, 16 of bf16) whatever the width; a group of 8 that
// passes a block's or a row's end looks its scales up one by one.
template <int U, class Index>
__device__ __forceinline__ void restore_flat(const Fp8Args& a, int64_t blocks_per_row, Index numel, unsigned cta) {
  const Index cols = (Index)a.cols;
  uint2 c[U];
  Index at[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    at[i] = (((Index)cta * U + i) * kThreads + threadIdx.x) * 8;
    c[i] = make_uint2(0, 0);
    if (at[i] + 8 <= numel) c[i] = __ldcs((const uint2*)(a.codes + at[i]));
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (at[i] >= numel) continue;
    Index row = at[i] / cols, col = at[i] - row * cols;
    if (at[i] + 8 > numel) {
      for (Index e = at[i]; e < numel; ++e) {
        a.bf16[e] = to_bf16(e4m3_values(a.codes[e]).x * scale_at(a, blocks_per_row, row, col));
        if (++col == cols) ++row, col = 0;
      }
      continue;
    }
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = j < 2 ? c[i].x : c[i].y;
      const float2 t = e4m3_values((uint16_t)(w >> (16 * (j & 1))));
      f[2 * j] = t.x;
      f[2 * j + 1] = t.y;
    }
    if (col + 8 <= cols && (col & (kBlock - 1)) <= kBlock - 8) {
      const float s = scale_at(a, blocks_per_row, row, col);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] *= scale_at(a, blocks_per_row, row, col);
        if (++col == cols) ++row, col = 0;
      }
    }
    __stcs((uint4*)(a.bf16 + at[i]), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                               pack_bf16(f[6], f[7])));
  }
}

template <int U, class Index>
__global__ void __launch_bounds__(kThreads) restore_flat_kernel(Fp8Args a, int64_t blocks_per_row, Index numel) {
  after_previous();
  restore_flat<U>(a, blocks_per_row, numel, blockIdx.x);
}

// Strided destination rows: one element a thread and step.
__global__ void __launch_bounds__(kThreads) restore_any_kernel(Fp8Args a, int64_t blocks_per_row, int64_t numel) {
  after_previous();
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < numel; e += (int64_t)gridDim.x * kThreads) {
    const int64_t row = e / a.cols, col = e - row * a.cols;
    a.bf16[row * a.ld + col] = to_bf16(e4m3_values(a.codes[e]).x * scale_at(a, blocks_per_row, row, col));
  }
}

// ------------------------------------------------- gradients from the codes

// dU = dh act(g), dG = dh u act'(g) and, where asked, h = act(g) u, with g
// and u read from their codes: 4 bytes in and 4 (6) out an element, so the
// pre-activations are never spelled out in memory.  V = 8 columns a thread
// where rows allow 16-byte accesses, else 1.  CTAs past the gradients'
// restore the input `x`, if it is kept in 8 bits too: one launch for both.
constexpr int kRestoreUnroll = 4;

template <int ACT, int V, class Index>
__global__ void __launch_bounds__(kThreads)
    grad_stored_kernel(GatedArgs a, Index groups_per_row, Index groups, unsigned ctas, Fp8Args x) {
  after_previous();
  if (blockIdx.x >= ctas) {
    restore_flat<kRestoreUnroll, Index>(x, (x.cols + kBlock - 1) / kBlock, (Index)(x.rows * x.cols), blockIdx.x - ctas);
    return;
  }
  const int64_t nb = (a.ffn + kBlock - 1) / kBlock;
  const Index i = (Index)blockIdx.x * kThreads + threadIdx.x;
  if (i >= groups) return;
  const Index r = i / groups_per_row;
  const int64_t row = r, col = (int64_t)(i - r * groups_per_row) * V;
  const int64_t at = row * a.ffn + col, sat = row * nb + col / kBlock;
  const float sg = a.gs[sat], su = a.us[sat];
  float g[V], u[V], d[V], dg[V], du[V], h[V];
  if constexpr (V == 8) {
    const uint2 cg = __ldcs((const uint2*)(a.g8 + at)), cu = __ldcs((const uint2*)(a.u8 + at));
    const uint4 cd = __ldcs((const uint4*)(a.dh + row * a.lddh + col));
    const uint32_t w[4] = {cd.x, cd.y, cd.z, cd.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 tg = e4m3_values((uint16_t)((j < 2 ? cg.x : cg.y) >> (16 * (j & 1))));
      const float2 tu = e4m3_values((uint16_t)((j < 2 ? cu.x : cu.y) >> (16 * (j & 1))));
      g[2 * j] = tg.x, g[2 * j + 1] = tg.y;
      u[2 * j] = tu.x, u[2 * j + 1] = tu.y;
      d[2 * j] = bf16_lo(w[j]), d[2 * j + 1] = bf16_hi(w[j]);
    }
  } else {
    g[0] = e4m3_values(a.g8[at]).x;
    u[0] = e4m3_values(a.u8[at]).x;
    d[0] = bf16_value(a.dh[row * a.lddh + col]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float gv = g[j] * sg, uv = u[j] * su;
    const float2 t = activation_grad<ACT>(gv);
    du[j] = d[j] * t.x;
    dg[j] = d[j] * uv * t.y;
    h[j] = t.x * uv;
  }
  if constexpr (V == 8) {
    *(uint4*)(a.dg + at) = make_uint4(pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3]), pack_bf16(dg[4], dg[5]),
                                      pack_bf16(dg[6], dg[7]));
    *(uint4*)(a.du + at) = make_uint4(pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3]), pack_bf16(du[4], du[5]),
                                      pack_bf16(du[6], du[7]));
    if (a.h)
      *(uint4*)(a.h + row * a.ldh + col) = make_uint4(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]),
                                                      pack_bf16(h[4], h[5]), pack_bf16(h[6], h[7]));
  } else {
    a.dg[at] = to_bf16(dg[0]);
    a.du[at] = to_bf16(du[0]);
    if (a.h) a.h[row * a.ldh + col] = to_bf16(h[0]);
  }
}

template <int ACT>
cudaError_t grad_stored(const GatedArgs& a, const Fp8Args& x, cudaStream_t stream) {
  const bool vec = a.ffn % 8 == 0 && a.lddh % 8 == 0 && (!a.h || a.ldh % 8 == 0);
  const int64_t per_row = vec ? a.ffn / 8 : a.ffn, groups = per_row * a.tokens, more = x.rows * x.cols;
  const unsigned ctas = (unsigned)ceil_div(groups, kThreads);
  const unsigned grid = ctas + (unsigned)ceil_div(more, (int64_t)kThreads * 8 * kRestoreUnroll);
  const bool small = groups <= kSmall && more <= kSmall;
  if (vec && small) return run(grad_stored_kernel<ACT, 8, uint32_t>, grid, stream, a, (uint32_t)per_row, (uint32_t)groups, ctas, x);
  if (vec) return run(grad_stored_kernel<ACT, 8, int64_t>, grid, stream, a, per_row, groups, ctas, x);
  if (small) return run(grad_stored_kernel<ACT, 1, uint32_t>, grid, stream, a, (uint32_t)per_row, (uint32_t)groups, ctas, x);
  return run(grad_stored_kernel<ACT, 1, int64_t>, grid, stream, a, per_row, groups, ctas, x);
}

}  // namespace

cudaError_t launch_fp8_store(const Fp8Args& a, cudaStream_t stream) {
  const int64_t per_row = ceil_div(a.cols, kBlock);
  const bool vec = a.cols % 8 == 0 && a.ld % 8 == 0;
  if (a.block_rows != 1) {
    const unsigned grid = (unsigned)(per_row * ceil_div(a.rows, kBlock));
    return run(vec ? store_square_kernel<true> : store_square_kernel<false>, grid, stream, a, (uint32_t)per_row);
  }
  constexpr int kUnroll = 2;
  const int64_t blocks = per_row * a.rows;
  const unsigned grid = (unsigned)ceil_div(blocks, (int64_t)kUnroll * (vec ? kThreads / 16 : kThreads / 32));
  const bool small = blocks <= kSmall;
  if (vec && small) return run(store_rows_kernel<kUnroll, uint32_t>, grid, stream, a, (uint32_t)per_row, (uint32_t)blocks);
  if (vec) return run(store_rows_kernel<kUnroll, int64_t>, grid, stream, a, per_row, blocks);
  if (small) return run(store_rows_any_kernel<kUnroll, uint32_t>, grid, stream, a, (uint32_t)per_row, (uint32_t)blocks);
  return run(store_rows_any_kernel<kUnroll, int64_t>, grid, stream, a, per_row, blocks);
}

cudaError_t launch_fp8_restore(const Fp8Args& a, cudaStream_t stream) {
  const int64_t per_row = ceil_div(a.cols, kBlock), numel = a.rows * a.cols;
  if (a.ld != a.cols) {
    const int64_t grid = ceil_div(numel, kThreads);
    return run(restore_any_kernel, (unsigned)(grid < 65536 ? grid : 65536), stream, a, per_row, numel);
  }
  const unsigned grid = (unsigned)ceil_div(numel, (int64_t)kThreads * 8 * kRestoreUnroll);
  if (numel <= kSmall) return run(restore_flat_kernel<kRestoreUnroll, uint32_t>, grid, stream, a, per_row, (uint32_t)numel);
  return run(restore_flat_kernel<kRestoreUnroll, int64_t>, grid, stream, a, per_row, numel);
}

cudaError_t launch_gated_grad_stored(const GatedArgs& a, const Fp8Args& x, cudaStream_t stream) {
  return a.act == TIDE_ACT_SILU ? grad_stored<TIDE_ACT_SILU>(a, x, stream) : grad_stored<TIDE_ACT_GELU>(a, x, stream);
}

}  // namespace tide
