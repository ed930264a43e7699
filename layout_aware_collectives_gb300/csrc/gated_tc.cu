// The gated block's products on the tensor cores, one persistent kernel in
// four forms:
//   forward   [gate | up] = x [Wg | Wu]^T, then h (and the 8-bit checkpoint)
//   grad      the same products again, then dG, dU (and h) from dh
//   dx        dX = [dG dU] [Wg; Wu], one sum over both halves
//   dw        dWg = dG^T x and dWu = dU^T x
//
// A pair of CTAs (two SMs) works on one 256 x 256 tile of sums: each CTA
// loads 128 rows of A and half of B's 256 columns, one MMA instruction of the
// pair reads both halves, so every operand byte is loaded into one SM only.
// In the forward form CTA 0's half of B is 128 features of Wg and CTA 1's the
// same 128 features of Wu: each CTA's accumulator then holds its tokens' gate
// and up sums side by side, and the product needs no exchange.
//
// Roles: warp 0 loads (6 stages of 32 KiB), warp 1 of the pair's first CTA
// issues the MMAs, warps 4-7 read finished sums out of TMEM, which holds two
// accumulators so that they do so while the next tile is summed.  Bound by
// the tensor cores at every large size.
#include "compute_device.cuh"
#include "tc_device.cuh"
#include "tc_host.h"

namespace tide {
namespace {

using namespace tc;

enum Form { kForward = 0, kGrad = 1, kDx = 2, kDw = 3 };

constexpr int kStages = 6;
constexpr int kStep = 64;                     // contraction of one stage
constexpr int kHalf = 128;                    // rows of A, columns of B in one CTA
constexpr uint32_t kOperand = kHalf * kStep * 2;  // bytes of either in one stage
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kThreads = 256;
constexpr int kEpiWarps = 4;
constexpr int kBoxes = 4;                     // boxes in flight for each warp
constexpr size_t kSmem = 1024 + kStages * kStage + kEpiWarps * kBoxes * kBox;

struct Params {
  CUtensorMap a[2], b[2];  // the two halves (gate, up) of each operand, where a form has two
  CUtensorMap out[3];      // forward: h; grad: dG, dU, h; dx: dX; dw: dWg, dWu
  int rows, cols;          // of one output
  int tiles_m, tiles_n, tiles;
  int steps;               // stages of one tile's sum
  int half_steps;          // dx: stages of the first half
  // epilogue
  uint8_t *g8, *u8;
  float *gs, *us;
  const uint16_t* dh;
  int64_t lddh;
  bool with_h;
  int* err;
  uint64_t limit_ns, stall_ns;
};

// 32 codes of one row.  Rows are whole multiples of 8 codes.
__device__ __forceinline__ void put_codes(uint8_t* dst, const uint32_t (&v)[32], float inv, int valid, bool clean) {
  uint32_t c[8];
  if (clean) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = pack_e4m3x4(as_f(v[4 * i]) * inv, as_f(v[4 * i + 1]) * inv, as_f(v[4 * i + 2]) * inv, as_f(v[4 * i + 3]) * inv);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = pack_e4m3x4(no_infinity(as_f(v[4 * i])) * inv, no_infinity(as_f(v[4 * i + 1])) * inv,
                         no_infinity(as_f(v[4 * i + 2])) * inv, no_infinity(as_f(v[4 * i + 3])) * inv);
  }
  if (((uintptr_t)dst & 15) == 0 && valid >= 32) {
    ((uint4*)dst)[0] = make_uint4(c[0], c[1], c[2], c[3]);
    ((uint4*)dst)[1] = make_uint4(c[4], c[5], c[6], c[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (8 * i < valid) ((uint2*)dst)[i] = make_uint2(c[2 * i], c[2 * i + 1]);
  }
}

template <int FORM, int ACT>
__device__ __forceinline__ void epilogue(const Params& p, const TileAt& t, uint32_t tmem, int row0, Outbox<kBoxes>& out) {
  const int row = row0 + out.lane;
  const bool any = row0 < p.rows, mine = row < p.rows;
  if constexpr (FORM == kForward || FORM == kGrad) {
    const int col0 = t.n * kHalf;
    float ginv = 0.0f, uinv = 0.0f;
    bool clean = true;  // no infinities to be made NaN in the codes
    if constexpr (FORM == kForward) {
      if (p.g8) {  // the tile is one scale block wide: a thread holds a whole block of its token
        float gmax = 0.0f, umax = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t g[32], u[32];
          tmem_read32x2(tmem + c * 32, tmem + kHalf + c * 32, g, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            gmax = fmaxf(gmax, fabsf(as_f(g[i])));
            umax = fmaxf(umax, fabsf(as_f(u[i])));
          }
        }
        clean = !__any_sync(0xffffffffu, gmax == CUDART_INF_F || umax == CUDART_INF_F);
        if (!clean) {  // again without the infinities
          gmax = umax = 0.0f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t g[32], u[32];
            tmem_read32x2(tmem + c * 32, tmem + kHalf + c * 32, g, u);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              gmax = fmaxf(gmax, fabsf(no_infinity(as_f(g[i]))));
              umax = fmaxf(umax, fabsf(no_infinity(as_f(u[i]))));
            }
          }
        }
        const uint32_t eg = scale_exponent(gmax), eu = scale_exponent(umax);
        ginv = exponent_inverse(eg), uinv = exponent_inverse(eu);
        if (mine) {
          const int64_t nb = (p.cols + kBlock - 1) / kBlock;
          p.gs[row * nb + t.n] = exponent_value(eg);
          p.us[row * nb + t.n] = exponent_value(eu);
        }
      }
    }
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      const int col = col0 + c * 32;
      if (!any || col >= p.cols) break;
      uint32_t g[32], u[32], o[16];
      tmem_read32x2(tmem + c * 32, tmem + kHalf + c * 32, g, u);
      if constexpr (FORM == kForward) {
        if (p.g8 && mine) {
          put_codes(p.g8 + (int64_t)row * p.cols + col, g, ginv, p.cols - col, clean);
          put_codes(p.u8 + (int64_t)row * p.cols + col, u, uinv, p.cols - col, clean);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[i] = pack_bf16(activation<ACT>(as_f(g[2 * i])) * as_f(u[2 * i]),
                           activation<ACT>(as_f(g[2 * i + 1])) * as_f(u[2 * i + 1]));
        out.put(&p.out[0], o, col, row0);
      } else {
        uint32_t o1[16], o2[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 d = make_uint4(0, 0, 0, 0);
          if (mine && col + 8 * q < p.cols) d = __ldcs((const uint4*)(p.dh + row * p.lddh + col + 8 * q));
          const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 4 * q + j;
            const float d0 = bf16_lo(w[j]), d1 = bf16_hi(w[j]);
            const float2 t0 = activation_grad<ACT>(as_f(g[2 * i])), t1 = activation_grad<ACT>(as_f(g[2 * i + 1]));
            const float u0 = as_f(u[2 * i]), u1 = as_f(u[2 * i + 1]);
            o[i] = pack_bf16(d0 * u0 * t0.y, d1 * u1 * t1.y);
            o1[i] = pack_bf16(d0 * t0.x, d1 * t1.x);
            o2[i] = pack_bf16(t0.x * u0, t1.x * u1);
          }
        }
        out.put(&p.out[0], o, col, row0);
        out.put(&p.out[1], o1, col, row0);
        if (p.with_h) out.put(&p.out[2], o2, col, row0);
      }
    }
  } else {
    const CUtensorMap* map = &p.out[FORM == kDw ? t.z : 0];
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      const int col = t.n * 2 * kHalf + c * 32;
      if (!any || col >= p.cols) break;
      uint32_t v[32], o[16];
      tmem_read(tmem + c * 32, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = pack_bf16(as_f(v[2 * i]), as_f(v[2 * i + 1]));
      out.put(map, o, col, row0);
    }
  }
}

template <int FORM, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) gated_tc_kernel(const __grid_constant__ Params p) {
  constexpr bool kAMn = FORM == kDw, kBMn = FORM == kDx || FORM == kDw;
  constexpr uint32_t kInstr = instr_desc(1, kAMn, kBMn, 256, 256);
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_at;
  __shared__ int stop;

  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  const auto full = [&](int s) { return bar0 + 8u * s; };
  const auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  const auto sums_full = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  const auto sums_empty = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };
  const uint32_t spare = bar0 + 8u * (2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const Watch watch{&stop, p.err, p.limit_ns};

  if (threadIdx.x == 0) {
    stop = 0;
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(sums_full(b), 1), bar_init(sums_empty(b), 2 * kEpiWarps);
    bar_init(spare, 1);
    bar_init_fence();
    for (int i = 0; i < 2; ++i) prefetch_map(&p.a[i]), prefetch_map(&p.b[i]);
  }
  if (warp == 2) tmem_alloc<2>(smem_addr(&tmem_at), 512);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_at;

  if (p.stall_ns) {  // test: a wait on a barrier nothing arrives on runs out
    if (threadIdx.x == 0) bar_wait(spare, 0, Watch{&stop, p.err, p.stall_ns});
  } else if (warp == 0) {
    if (lane == 0) {
      int j = 0;  // stages filled so far
      bool go = true;
      for (int t = pair; t < p.tiles && go; t += pairs) {
        const TileAt at = tile_at(p.tiles_m, p.tiles_n, t);
        for (int k = 0; k < p.steps; ++k, ++j) {
          const int s = j % kStages;
          if (j >= kStages && !bar_wait(empty(s), (j / kStages + 1) & 1, watch)) {
            go = false;
            break;
          }
          if (rank == 0) bar_expect(full(s), 2 * kStage);
          const uint32_t bar = peer_addr(full(s), 0);
          const uint32_t a = smem + s * kStage, b = a + kOperand;
          const int second = FORM == kDx && k >= p.half_steps;
          const int k0 = (k - (second ? p.half_steps : 0)) * kStep;
          const int row = (at.m * 2 + rank) * kHalf, col = (at.n * 2 + rank) * kHalf;
          if constexpr (kAMn) {
            load_box<true>(a, &p.a[at.z], row, k0, bar);
            load_box<true>(a + kOperand / 2, &p.a[at.z], row + 64, k0, bar);
          } else {
            load_box<true>(a, &p.a[second], k0, row, bar);
          }
          if constexpr (kBMn) {
            load_box<true>(b, &p.b[second], col, k0, bar);
            load_box<true>(b + kOperand / 2, &p.b[second], col + 64, k0, bar);
          } else {
            load_box<true>(b, &p.b[rank], k0, at.n * kHalf, bar);
          }
        }
      }
      // the MMAs' last arrivals reach this CTA while it is still there
      for (int i = max(0, j - kStages); i < j && go; ++i) go = bar_wait(empty(i % kStages), (i / kStages) & 1, watch);
      // after a wait that ran out: both CTAs' copies in flight, with a limit
      // again; the peer's memory stays until the cluster's last barrier
      if (!go && rank == 0) {
        int never = 0;
        for (int i = max(0, j - kStages); i < j; ++i)
          bar_wait(full(i % kStages), (i / kStages) & 1, Watch{&never, p.err, p.limit_ns / 16});
      }
    }
  } else if (warp == 1 && rank == 0) {
    if (lane == 0) {
      int j = 0, i = 0;  // stages used, tiles done
      bool go = true;
      for (int t = pair; t < p.tiles && go; t += pairs, ++i) {
        const int b = i & 1;
        if (i >= 2 && !bar_wait(sums_empty(b), (i / 2 + 1) & 1, watch)) break;
        fence_after();
        for (int k = 0; k < p.steps; ++k, ++j) {
          const int s = j % kStages;
          if (!bar_wait(full(s), (j / kStages) & 1, watch)) {
            go = false;
            break;
          }
          fence_after();
          const uint32_t a = smem + s * kStage;
          // a 32-byte step of the contraction lies 32 bytes on (K-major) or
          // two groups of 8 rows on (MN-major)
          const uint64_t da = operand_desc(a, kAMn ? kOperand / 2 : 16), db = operand_desc(a + kOperand, kBMn ? kOperand / 2 : 16);
#pragma unroll
          for (int q = 0; q < kStep / 16; ++q)
            mma<2, false>(tmem + b * 256, da + q * ((kAMn ? 2048 : 32) >> 4), db + q * ((kBMn ? 2048 : 32) >> 4), kInstr,
                          k > 0 || q > 0);
          mma_commit<2>(empty(s));
        }
        if (go) mma_commit<2>(sums_full(b));
      }
      if (*watch.stop) {  // the MMAs in flight, with a limit
        int never = 0;
        mma_commit<2>(spare);
        bar_wait(spare, 0, Watch{&never, p.err, p.limit_ns / 16});
      }
    }
  } else if (warp >= 4) {
    Outbox<kBoxes> out{smem + kStages * kStage + (warp - 4) * kBoxes * kBox, 0, lane};
    int i = 0;
    for (int t = pair; t < p.tiles; t += pairs, ++i) {
      const int b = i & 1;
      if (!bar_wait_warp(sums_full(b), (i / 2) & 1, watch)) break;
      fence_after();
      const TileAt at = tile_at(p.tiles_m, p.tiles_n, t);
      const uint32_t lanes = (uint32_t)(warp - 4) * 32;
      epilogue<FORM, ACT>(p, at, tmem + (lanes << 16) + b * 256, (at.m * 2 + rank) * kHalf + lanes, out);
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_peer(peer_addr(sums_empty(b), 0));
    }
    if (lane == 0) stores_done();
  }
  __syncthreads();
  cluster_sync();
  if (warp == 2) tmem_free<2>(tmem, 512);
}

template <int FORM, int ACT>
cudaError_t launch(Params& p, const TcLaunch& l, cudaStream_t stream) {
  static const cudaError_t ready =
      cudaFuncSetAttribute(gated_tc_kernel<FORM, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (ready != cudaSuccess) return ready;
  p.err = l.err;
  p.limit_ns = TIDE_BULK_TIMEOUT_NS;
  p.stall_ns = l.stall_ns;
  const int pairs = p.tiles < l.pairs ? p.tiles : l.pairs;
  gated_tc_kernel<FORM, ACT><<<2 * pairs, kThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

bool rows16(int64_t width, int64_t ld) { return width % 8 == 0 && ld % 8 == 0; }

// Operand boxes: 64 of the contraction x 128 rows (K-major), or 64 columns x
// 64 of the contraction (MN-major); both are 128 bytes wide.
bool map_k(CUtensorMap* m, const uint16_t* p, int64_t cols, int64_t rows, int64_t ld) {
  return make_map(m, p, 2, cols, rows, ld, kStep, kHalf, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_mn(CUtensorMap* m, const uint16_t* p, int64_t cols, int64_t rows, int64_t ld) {
  return make_map(m, p, 2, cols, rows, ld, 64, kStep, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_out(CUtensorMap* m, const uint16_t* p, int64_t cols, int64_t rows, int64_t ld) {
  return make_map(m, p, 2, cols, rows, ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

bool fill_pre(Params* p, const GatedArgs& a) {
  p->rows = (int)a.tokens, p->cols = (int)a.ffn;
  p->tiles_m = (int)ceil_div(a.tokens, 2 * kHalf), p->tiles_n = (int)ceil_div(a.ffn, kHalf);
  p->tiles = p->tiles_m * p->tiles_n;
  p->steps = (int)ceil_div(a.hidden, kStep);
  if (!map_k(&p->a[0], a.x, a.hidden, a.tokens, a.ldx)) return false;
  p->a[1] = p->a[0];
  return map_k(&p->b[0], a.wg, a.hidden, a.ffn, a.hidden) && map_k(&p->b[1], a.wu, a.hidden, a.ffn, a.hidden);
}

}  // namespace

int gated_tc_pairs() {
  // The clusters the device holds at one time: a GPC with an odd number of
  // SMs leaves one without a partner.
  cudaFuncSetAttribute(gated_tc_kernel<kDx, 0>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(2);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmem;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gated_tc_kernel<kDx, 0>, &c) != cudaSuccess) return 0;
  return n;
}

bool gated_tc_takes(const GatedArgs& a) { return a.hidden >= 8 && rows16(a.hidden, a.hidden) && rows16(a.ffn, a.ffn); }

cudaError_t launch_gated_forward_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  if (!fill_pre(&p, a) || !map_out(&p.out[0], a.h, a.ffn, a.tokens, a.ldh)) return cudaErrorInvalidValue;
  p.g8 = a.g8, p.gs = a.gs, p.u8 = a.u8, p.us = a.us;
  return a.act == TIDE_ACT_SILU ? launch<kForward, TIDE_ACT_SILU>(p, l, stream)
                                : launch<kForward, TIDE_ACT_GELU>(p, l, stream);
}

cudaError_t launch_gated_grad_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  if (!fill_pre(&p, a) || !map_out(&p.out[0], a.dg, a.ffn, a.tokens, a.ffn) ||
      !map_out(&p.out[1], a.du, a.ffn, a.tokens, a.ffn) || (a.h && !map_out(&p.out[2], a.h, a.ffn, a.tokens, a.ldh)))
    return cudaErrorInvalidValue;
  p.with_h = a.h != nullptr;
  p.dh = a.dh, p.lddh = a.lddh;
  return a.act == TIDE_ACT_SILU ? launch<kGrad, TIDE_ACT_SILU>(p, l, stream) : launch<kGrad, TIDE_ACT_GELU>(p, l, stream);
}

cudaError_t launch_gated_dx_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  p.rows = (int)a.tokens, p.cols = (int)a.hidden;
  p.tiles_m = (int)ceil_div(a.tokens, 2 * kHalf), p.tiles_n = (int)ceil_div(a.hidden, 2 * kHalf);
  p.tiles = p.tiles_m * p.tiles_n;
  p.half_steps = (int)ceil_div(a.ffn, kStep), p.steps = 2 * p.half_steps;
  if (!map_k(&p.a[0], a.dg, a.ffn, a.tokens, a.ffn) || !map_k(&p.a[1], a.du, a.ffn, a.tokens, a.ffn) ||
      !map_mn(&p.b[0], a.wg, a.hidden, a.ffn, a.hidden) || !map_mn(&p.b[1], a.wu, a.hidden, a.ffn, a.hidden) ||
      !map_out(&p.out[0], a.dx, a.hidden, a.tokens, a.lddx))
    return cudaErrorInvalidValue;
  return launch<kDx, 0>(p, l, stream);
}

cudaError_t launch_gated_dw_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  p.rows = (int)a.ffn, p.cols = (int)a.hidden;
  p.tiles_m = (int)ceil_div(a.ffn, 2 * kHalf), p.tiles_n = (int)ceil_div(a.hidden, 2 * kHalf);
  if ((int64_t)p.tiles_m * p.tiles_n > INT32_MAX / 2) return cudaErrorInvalidValue;
  p.tiles = 2 * p.tiles_m * p.tiles_n;
  p.steps = (int)ceil_div(a.tokens, kStep);
  if (!map_mn(&p.a[0], a.dg, a.ffn, a.tokens, a.ffn) || !map_mn(&p.a[1], a.du, a.ffn, a.tokens, a.ffn) ||
      !map_mn(&p.b[0], a.x, a.hidden, a.tokens, a.ldx) || !map_out(&p.out[0], a.dwg, a.hidden, a.ffn, a.hidden) ||
      !map_out(&p.out[1], a.dwu, a.hidden, a.ffn, a.hidden))
    return cudaErrorInvalidValue;
  p.b[1] = p.b[0];
  return launch<kDw, 0>(p, l, stream);
}

}  // namespace tide
