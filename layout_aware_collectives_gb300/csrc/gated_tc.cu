// The gated block's products on the tensor cores, one persistent kernel in
// three forms:
//   forward   [gate | up] = x [Wg | Wu]^T, then h (and the 8-bit checkpoint)
//   grad      the same products again, then dG, dU (and h) from dh
//   back      dX = [dG dU] [Wg; Wu], one sum over both halves, and
//             dWg = dG^T x, dWu = dU^T x: independent tiles of one launch, so
//             that neither waits for the other's last ones
//
// A pair of CTAs (two SMs) works on one 256 x 256 tile of sums: each CTA
// loads 128 rows of A and half of B's 256 columns, one MMA instruction of the
// pair reads both halves, so every operand byte is loaded into one SM only.
// In the forward form CTA 0's half of B is 128 features of Wg and CTA 1's the
// same 128 features of Wu: each CTA's accumulator then holds its tokens' gate
// and up sums side by side, and the product needs no exchange.
//
// Roles: warps 0 and 3 load (6 stages of 32 KiB), warp 1 of the pair's first CTA
// issues the MMAs, warps from 4 on read finished sums out of TMEM, which holds two
// accumulators so that they do so while the next tile is summed.
//
// Bound by the tensor cores at every large size: 2048 x 4096 x 14336 forward
// 236-282 us (1.7-2.04 PFLOP/s; their pipe 94% busy), dX and dW of it 490-600
// us (94% busy), the longer times with the card at its power cap, where a
// plain library product of the forward's size takes 271.
#include "compute_device.cuh"
#include "gated_finish.cuh"
#include "tc_device.cuh"
#include "tc_host.h"

namespace tide {
namespace {

using namespace tc;

enum Form { kForward = 0, kGrad = 1, kBack = 2 };

constexpr int kStages = 6;
constexpr int kStep = 64;                     // contraction of one stage
constexpr int kHalf = 128;                    // rows of A, columns of B in one CTA
constexpr uint32_t kOperand = kHalf * kStep * 2;  // bytes of either in one stage
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kAllBoxes = 16;                 // boxes of results in flight
constexpr size_t kSmem = 1024 + kStages * kStage + kAllBoxes * kBox;
// Eight warps read finished sums, each 32 rows of one half of the columns:
// with a short contraction there is little of the next tile's sum to do it
// behind (64 tokens of the 8B-shaped block: dW 70 us with four, 52 with
// eight, 49 with two boxes of results behind one fence, 38 with the copies and
// MMAs from an elected thread).
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kBoxes = kAllBoxes / kEpiWarps;
constexpr int kJoinThreads = 256;

// Stages of part z of `split` of a sum of `steps`.
struct Share {
  int least, more;  // stages of each part; parts with one more

  Share() = default;
  Share(int steps, int split) : least(steps / split), more(steps % split) {}
  __device__ __forceinline__ int from(int z) const { return z * least + min(z, more); }
};

struct Params : GatedOut {  // of forward and grad
  // forward, grad: a = x, b = Wg, Wu; out = h, or dG, dU, h
  // back: dX: a = dG, dU, b = Wg, Wu, out[0]; dW: wa = dG, dU, wb = x, out[1..2]
  CUtensorMap a[2], b[2], wa[2], wb, outs[3];
  int rows, cols;  // of the outputs (back: of dX)
  TileGrid grid;
  int tiles;
  int steps;       // stages of one tile's sum
  int half_steps;  // back: stages of dX's first half
  // back: parts of dX's and of dW's sums, each in its own tile; forward,
  // grad: pairs of a cluster
  int split, w_split;
  Share share, w_share;
  float *parts, *w_parts;  // of [split, cols, rows], [w_split, half, cols, w_rows], where there are several
  TileGrid w_grid;
  int w_rows, w_tiles, w_steps;  // back: dW, both halves' tiles
  // back: who takes which tile (work_at).  dX's for each pair, and how many
  // pairs have one more; the others; dW's that go to those first, and how
  // many that is for each, and how many have one more
  int each, full, light, first, first_each, first_more;
  bool one_a, one_b;  // back: wa's, b's and wb's operands are one box each (map_mn)
  int* err;
  uint64_t limit_ns, stall_ns, late_ns;
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

// 128 columns x 64 of the contraction: a box of both halves, or one each.
__device__ __forceinline__ void load_mn(uint32_t dst, const CUtensorMap* m, int col, int k0, uint32_t bar, bool one) {
  if (one) {
    load_box3<true>(dst, m, 0, k0, col / 64, bar);
  } else {
    load_box<true>(dst, m, col, k0, bar);
    load_box<true>(dst + kOperand / 2, m, col + 64, k0, bar);
  }
}

// One tile of a pair's work.
struct Work {
  TileAt at;
  bool w;      // a tile of dW
  int half;    // of dW
  float* part;  // this part of the sums, [cols, rows], where there are several
  int k0, k1;  // stages of the whole sum
};

// The pair's i-th tile; false past the last.  Tiles go round the pairs in
// turn.  In the back form dX's tiles come first; where they do not come out
// even, the pairs that are one short take as many tiles of dW as one of dX is
// worth before the rest goes round, beginning with them again.
template <int FORM>
__device__ __forceinline__ bool work_at(const Params& p, int pair, int pairs, int part, int i, Work& r) {
  int t = pair + i * pairs;
  r.w = false;
  if (FORM != kBack) {
    if (t >= p.tiles) return false;
    r.at = tile_at(p.grid, t);
    r.k0 = p.share.from(part), r.k1 = p.share.from(part + 1);
    return true;
  }
  if (t < p.tiles) {
    r.at = tile_at(p.grid, t);
    r.k0 = p.share.from(r.at.z), r.k1 = p.share.from(r.at.z + 1);
    r.part = p.split > 1 ? p.parts + (int64_t)r.at.z * p.rows * p.cols : nullptr;
    return true;
  }
  const int l = pair - p.full;  // among those without one more, if not below 0
  i -= p.each + (l < 0);
  const int mine = l >= 0 ? p.first_each + (l < p.first_more) : 0;
  if (i < mine)
    t = l + i * p.light;
  else
    t = p.first + (l >= 0 ? l : p.light + pair) + (i - mine) * pairs;
  if (t >= p.w_tiles) return false;
  r.w = true;
  r.at = tile_at(p.w_grid, t);
  r.half = r.at.z & 1;
  const int z = r.at.z >> 1;
  r.k0 = p.w_share.from(z), r.k1 = p.w_share.from(z + 1);
  r.part = p.w_split > 1 ? p.w_parts + (int64_t)r.at.z * p.w_rows * p.cols : nullptr;
  return true;
}

// The two warps of 32 tokens, which meet in the epilogue of a checkpoint's
// tiles, enter it together or not at all: each has its own wait for the sums,
// and one's may run out where the other's does not.
__device__ __forceinline__ bool both_halves(int rows32, bool go) {
  uint32_t both;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %2, 0; bar.red.and.pred q, %1, 64, p; selp.b32 %0, 1, 0, q; }"
               : "=r"(both)
               : "r"(1 + rows32), "r"((uint32_t)go)
               : "memory");
  return both != 0;
}

template <int FORM, int ACT>
__device__ __forceinline__ void epilogue(const Params& p, const Work& work, uint32_t tmem, int row0, int half,
                                         uint32_t* maxima, const uint4 (&dh)[8], Outbox<kBoxes>& out) {
  const TileAt& t = work.at;
  const int row = row0 + out.lane, rows = work.w ? p.w_rows : p.rows;
  const bool any = row0 < rows, mine = row < rows;
  if constexpr (FORM == kForward || FORM == kGrad) {
    const int col0 = t.n * kHalf;
    float ginv = 0.0f, uinv = 0.0f;
    bool clean = true;  // no infinities to be made NaN in the codes
    if constexpr (FORM == kForward) {
      if (p.g8) {
        // The tile is one scale block wide: a thread holds half a block of
        // its token, and meets the thread that holds the other half.  The
        // block's exponent is the larger of the halves'.
        const auto meet = [&](float g, float u) {
          const auto code = [](float m) { return m == 0.0f ? 0u : m == CUDART_INF_F ? 255u : scale_exponent(m); };
          const uint32_t mine = code(g) | (code(u) << 16);
          uint32_t* at = maxima + (row & (kHalf - 1));
          at[half * kHalf] = mine;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + ((row0 >> 5) & 3)) : "memory");
          const uint32_t both = __vmaxu2(mine, at[(half ^ 1) * kHalf]);
          asm volatile("bar.sync %0, 64;" ::"r"(1 + ((row0 >> 5) & 3)) : "memory");
          return both;
        };
        float gmax = 0.0f, umax = 0.0f;
#pragma unroll
        for (int c = 2 * half; c < 2 * half + 2; ++c) {
          uint32_t g[32], u[32];
          tmem_read32x2(tmem + c * 32, tmem + kHalf + c * 32, g, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            gmax = fmaxf(gmax, fabsf(as_f(g[i])));
            umax = fmaxf(umax, fabsf(as_f(u[i])));
          }
        }
        uint32_t top = meet(gmax, umax);
        // the same for both warps: each sees both halves' maxima of 32 rows
        clean = !__any_sync(0xffffffffu, (top & 0xffffu) == 255u || (top >> 16) == 255u);
        if (!clean) {  // again without the infinities
          gmax = umax = 0.0f;
#pragma unroll 1
          for (int c = 2 * half; c < 2 * half + 2; ++c) {
            uint32_t g[32], u[32];
            tmem_read32x2(tmem + c * 32, tmem + kHalf + c * 32, g, u);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              gmax = fmaxf(gmax, fabsf(no_infinity(as_f(g[i]))));
              umax = fmaxf(umax, fabsf(no_infinity(as_f(u[i]))));
            }
          }
          top = meet(gmax, umax);
        }
        const uint32_t eg = (top & 0xffffu) ? top & 0xffffu : 127u, eu = (top >> 16) ? top >> 16 : 127u;
        ginv = exponent_inverse(eg), uinv = exponent_inverse(eu);
        if (mine && half == 0) {
          const int64_t nb = (p.cols + kBlock - 1) / kBlock;
          p.gs[row * nb + t.n] = exponent_value(eg);
          p.us[row * nb + t.n] = exponent_value(eu);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 2 * half + h, col = col0 + c * 32;
      if (!any || col >= p.cols) break;
      uint32_t o[16];
      if constexpr (FORM == kForward) {
        uint32_t g[32], u[32];
        tmem_read32x2(tmem + c * 32, tmem + kHalf + c * 32, g, u);
        if (p.g8 && mine) {
          put_codes(p.g8 + (int64_t)row * p.cols + col, g, ginv, p.cols - col, clean);
          put_codes(p.u8 + (int64_t)row * p.cols + col, u, uinv, p.cols - col, clean);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[i] = pack_bf16(activation<ACT>(as_f(g[2 * i])) * as_f(u[2 * i]),
                           activation<ACT>(as_f(g[2 * i + 1])) * as_f(u[2 * i + 1]));
        out.put(&p.outs[0], o, col, row0);
      } else {
        uint32_t o1[16], o2[16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // 16 columns at a time, for the registers
          uint32_t g[16], u[16];
          const uint4 d0 = dh[4 * h + 2 * q], d1 = dh[4 * h + 2 * q + 1];
          const uint32_t w[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
          tmem_read(tmem + c * 32 + 16 * q, g);
          tmem_read(tmem + kHalf + c * 32 + 16 * q, u);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int i = 8 * q + j;
            const float d0 = bf16_lo(w[j]), d1 = bf16_hi(w[j]);
            const float2 t0 = activation_grad<ACT>(as_f(g[2 * j])), t1 = activation_grad<ACT>(as_f(g[2 * j + 1]));
            const float u0 = as_f(u[2 * j]), u1 = as_f(u[2 * j + 1]);
            o[i] = pack_bf16(d0 * u0 * t0.y, d1 * u1 * t1.y);
            o1[i] = pack_bf16(d0 * t0.x, d1 * t1.x);
            o2[i] = pack_bf16(t0.x * u0, t1.x * u1);
          }
        }
        out.put2(&p.outs[0], o, col, &p.outs[1], o1, col, row0);
        if (p.out) out.put(&p.outs[2], o2, col, row0);
      }
    }
  } else {
    const CUtensorMap* map = &p.outs[work.w ? 1 + work.half : 0];
#pragma unroll 1
    for (int c = half * 4; c < half * 4 + 4; c += 2) {
      const int col = t.n * 2 * kHalf + c * 32;
      if (!any || col >= p.cols) break;
      uint32_t v[32], u[32];
      tmem_read32x2(tmem + c * 32, tmem + c * 32 + 32, v, u);
      if (work.part) {
        // a column of the warp's 32 rows lies together, so its threads do
        uint32_t* to = (uint32_t*)work.part + (int64_t)col * rows + row;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (mine && col + i < p.cols) to[(int64_t)i * rows] = v[i];
          if (mine && col + 32 + i < p.cols) to[(int64_t)(32 + i) * rows] = u[i];
        }
        continue;
      }
      uint32_t o0[16], o1[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        o0[i] = pack_bf16(as_f(v[2 * i]), as_f(v[2 * i + 1]));
        o1[i] = pack_bf16(as_f(u[2 * i]), as_f(u[2 * i + 1]));
      }
      out.put2(map, o0, col, map, o1, col + 32, row0, col + 32 < p.cols);
    }
  }
}

// SPLIT (forward, grad): where the tiles leave SMs without work, a cluster of
// two to four pairs works on one, each pair on a part of the contraction; the
// sums meet over distributed shared memory, in the order of the parts (512 x
// 7168 x 2048, 32 tiles: 34.8 us by single pairs, 24.5 in twos; 532 x 16480 x
// 656, 18 tiles: 72.7 and, in threes, 32).  A stage takes 0.27 us, the sums'
// meeting some 4.
template <int FORM, int ACT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) gated_tc_kernel(const __grid_constant__ Params p) {
  constexpr bool kBMn = FORM == kBack;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kStages + 6];
  __shared__ uint32_t maxima[FORM == kForward ? 2 * kHalf : 1];  // of the checkpoint's half blocks, as exponents
  __shared__ uint32_t tmem_at;
  __shared__ int stop;

  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  const auto full = [&](int s) { return bar0 + 8u * s; };
  const auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  const auto sums_full = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  const auto sums_empty = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };
  const uint32_t spare = bar0 + 8u * (2 * kStages + 4), silent = spare + 8;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t cta = cluster_rank(), rank = cta & 1, leader = SPLIT ? cta & ~1u : 0;
  const uint16_t both = (uint16_t)(3u << leader);  // the pair's CTAs
  const int split = SPLIT ? p.split : 1, part = SPLIT ? cta >> 1 : 0;
  const int pair = blockIdx.x / (2 * split), pairs = gridDim.x / (2 * split);
  const Watch watch{&stop, p.err, p.limit_ns};
  const bool late = p.late_ns && warp == 4;  // test: this warp waits for sums where nothing arrives
  const Watch sums_watch{&stop, p.err, late ? p.late_ns : p.limit_ns};

  if (threadIdx.x == 0) {
    stop = 0;
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(sums_full(b), 1), bar_init(sums_empty(b), 2 * kEpiWarps);
    bar_init(spare, 1), bar_init(silent, 1);
    bar_init_fence();
    prefetch_map(FORM == kBack && !p.tiles ? &p.wa[0] : &p.a[0]), prefetch_map(FORM == kBack && !p.tiles ? &p.wb : &p.b[0]);
  }
  if (warp == 2) tmem_alloc<2>(smem_addr(&tmem_at), 512);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_at;
  after_previous();

  if (p.stall_ns) {  // test: a wait on a barrier nothing arrives on runs out
    if (threadIdx.x == 0) bar_wait(silent, 0, Watch{&stop, p.err, p.stall_ns});
  } else if (warp == 0 || warp == 3) {
    // One thread loads A, another B: issuing a copy takes long enough that
    // one thread with all four of a stage fell behind the MMAs.
    if (elected()) {
      const bool load_a = warp == 0;
      int j = 0;  // stages filled so far
      bool go = true;
      Work work;
      for (int i = 0; go && work_at<FORM>(p, pair, pairs, part, i, work); ++i) {
        const TileAt& at = work.at;
        const int row = (at.m * 2 + rank) * kHalf, col = (at.n * 2 + rank) * kHalf;
        for (int k = work.k0; k < work.k1; ++k, ++j) {
          const int s = j % kStages;
          if (j >= kStages && !bar_wait(empty(s), (j / kStages + 1) & 1, watch)) {
            go = false;
            break;
          }
          if (load_a && rank == 0) bar_expect(full(s), 2 * kStage);
          const uint32_t bar = peer_addr(full(s), leader);
          const uint32_t a = smem + s * kStage, b = a + kOperand;
          if constexpr (FORM != kBack) {
            if (load_a)
              load_box<true>(a, &p.a[0], k * kStep, row, bar);
            else
              load_box<true>(b, &p.b[rank], k * kStep, at.n * kHalf, bar);
          } else {
            const int second = !work.w && k >= p.half_steps, k0 = (k - (second ? p.half_steps : 0)) * kStep;
            if (!load_a) {
              const CUtensorMap* mb = work.w ? &p.wb : &p.b[second];
              load_mn(b, mb, col, k0, bar, p.one_b);
            } else if (work.w) {
              load_mn(a, &p.wa[work.half], row, k0, bar, p.one_a);
            } else {
              load_box<true>(a, &p.a[second], k0, row, bar);
            }
          }
        }
      }
      // the MMAs' last arrivals reach this CTA while it is still there
      for (int i = max(0, j - kStages); i < j && go; ++i) go = bar_wait(empty(i % kStages), (i / kStages) & 1, watch);
      // after a wait that ran out: both CTAs' copies in flight, with a limit
      // again; the peer's memory stays until the cluster's last barrier
      if (!go && rank == 0)
        for (int i = max(0, j - kStages); i < j; ++i) await(full(i % kStages), (i / kStages) & 1, watch);
    }
  } else if (warp == 1 && rank == 0) {
    if (elected()) {
      int j = 0, i = 0;  // stages used, tiles done
      bool go = true;
      Work work;
      for (; go && work_at<FORM>(p, pair, pairs, part, i, work); ++i) {
        const int b = i & 1;
        const bool a_mn = FORM == kBack && work.w;
        const uint32_t instr = instr_desc(1, 0, kBMn, 256, 256) | (a_mn ? instr_desc_a_mn : 0);
        // a 32-byte step of the contraction lies 32 bytes on (K-major) or two
        // groups of 8 rows on (MN-major)
        const uint32_t a_lbo = a_mn ? kOperand / 2 : 16, a_next = (a_mn ? 2048 : 32) >> 4;
        if (i >= 2 && !bar_wait<kPeer>(sums_empty(b), (i / 2 + 1) & 1, watch)) break;
        fence_after();
        for (int k = work.k0; k < work.k1; ++k, ++j) {
          const int s = j % kStages;
          if (!bar_wait(full(s), (j / kStages) & 1, watch)) {
            go = false;
            break;
          }
          fence_after();
          const uint32_t a = smem + s * kStage;
          const uint64_t da = operand_desc(a, a_lbo), db = operand_desc(a + kOperand, kBMn ? kOperand / 2 : 16);
#pragma unroll
          for (int q = 0; q < kStep / 16; ++q)
            mma<2, false>(tmem + b * 256, da + q * a_next, db + q * ((kBMn ? 2048 : 32) >> 4), instr, k > work.k0 || q > 0);
          mma_commit<2>(empty(s), both);
        }
        if (go) mma_commit<2>(sums_full(b), both);
      }
      mma_commit<2>(spare, (uint16_t)(1u << leader));
    }
  } else if (warp >= 4) {
    Outbox<kBoxes> out{smem + kStages * kStage + (warp - 4) * kBoxes * kBox, 0, lane};
    Work work;
    for (int i = 0; work_at<FORM>(p, pair, pairs, part, i, work); ++i) {
      const int b = i & 1;
      uint4 dh[8];
      if constexpr (FORM == kGrad && !SPLIT) {  // 64 columns of dh on their way while the sums are not there yet
        const int row = (work.at.m * 2 + rank) * kHalf + (warp & 3) * 32 + lane;
        const int col = work.at.n * kHalf + ((warp - 4) >> 2) * 64;
        const uint4* from = (const uint4*)(p.dh + row * p.lddh + col);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          dh[j] = row < p.rows && col + 8 * j < p.cols ? __ldcs(from + j) : make_uint4(0, 0, 0, 0);
      }
      bool go = bar_wait_warp(late ? silent : sums_full(b), (i / 2) & 1, sums_watch);
      if constexpr (FORM == kForward && !SPLIT) {
        if (p.g8) go = both_halves(warp & 3, go);
      }
      if (!go) break;
      fence_after();
      const uint32_t lanes = (uint32_t)(warp & 3) * 32;
      if constexpr (SPLIT) {
        leave_sums(smem, tmem + (lanes << 16), lanes + lane, (warp - 4) >> 2 << 2);
        fence_before();
        break;
      }
      epilogue<FORM, ACT>(p, work, tmem + (lanes << 16) + b * 256, (work.at.m * 2 + rank) * kHalf + lanes, (warp - 4) >> 2, maxima, dh, out);
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_peer(peer_addr(sums_empty(b), leader));
    }
    if (lane == 0) stores_done();
  }
  __syncthreads();
  if (stop && warp == 1 && rank == 0 && !p.stall_ns) {
    await(spare, 0, watch);  // the MMAs in flight
    __syncwarp();
  }
  cluster_sync();
  if constexpr (SPLIT) {
    // Each CTA finishes its share of the pair's rows.
    const TileAt at = tile_at(p.grid, pair);
    const int row0 = (at.m * 2 + rank) * kHalf, r1 = min(kHalf * (part + 1) / split, p.rows - row0);
    if (!p.stall_ns) {
      for (int r = kHalf * part / split + warp; r < r1; r += kThreads / 32) {
        float4 sum[2];
        split_sums(smem, r, lane, rank, split, sum);
        if constexpr (FORM == kForward)
          finish_forward<ACT>(p, row0 + r, at.n, lane, sum[0], sum[1]);
        else
          finish_grad<ACT>(p, row0 + r, at.n, lane, sum[0], sum[1]);
      }
    }
    cluster_sync();  // the others have read this CTA's sums
  }
  if (warp == 2) tmem_free<2>(tmem, 512);
}

// Results from the parts of their sums, in the parts' order.  A part lies
// column by column, `out0`'s parts before `out1`'s: 32 rows x COLS columns a
// CTA, turned in shared memory, AT_ONCE parts of COLS / 8 columns a thread on
// their way at a time.  Few parts are many bytes each, many parts a latency
// for every turn: 64 columns and 4 parts, 32 and 8 or 16 and 16 (256 x 4096
// of 4 parts: 8 us less than in 16 columns; 849 x 144 of 19: 5 us less than in
// 64).
struct Join {
  const float* parts;
  int split;
  uint16_t* out[2];
  int64_t ld;
  int rows, cols;
};

template <int COLS, int AT_ONCE>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(Join a) {
  after_previous();
  constexpr int kCols = COLS / 8;
  __shared__ float tile[COLS][33];
  const int row0 = blockIdx.x * 32, col0 = blockIdx.y * COLS;
  const int r = threadIdx.x & 31, c0 = threadIdx.x >> 5;
  const int64_t numel = (int64_t)a.rows * a.cols, next = numel * gridDim.z;
  float sum[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
  if (row0 + r < a.rows) {
    const float* from = a.parts + blockIdx.z * numel + (int64_t)(col0 + c0) * a.rows + row0 + r;
    for (int s = 0; s < a.split; s += AT_ONCE) {
      float v[AT_ONCE][kCols];
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          v[q][i] = s + q < a.split && col0 + c0 + 8 * i < a.cols ? from[(s + q) * next + (int64_t)8 * i * a.rows] : 0.0f;
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i] += v[q][i];
    }
  }
#pragma unroll
  for (int i = 0; i < kCols; ++i) tile[c0 + 8 * i][r] = sum[i];
  __syncthreads();
  const int row = threadIdx.x / kCols, col = threadIdx.x % kCols * 8;
  if (row >= 32 || row0 + row >= a.rows || col0 + col >= a.cols) return;  // widths are multiples of 8
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16(tile[col + 2 * i][row], tile[col + 2 * i + 1][row]);
  uint16_t* out = blockIdx.z ? a.out[1] : a.out[0];
  *(uint4*)(out + (int64_t)(row0 + row) * a.ld + col0 + col) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <int COLS, int AT_ONCE>
cudaError_t join(const Join& a, int outputs, cudaStream_t stream) {
  return launch_early(join_kernel<COLS, AT_ONCE>,
                      dim3((unsigned)ceil_div(a.rows, 32), (unsigned)ceil_div(a.cols, COLS), outputs), kJoinThreads, 0, 0,
                      stream, a);
}
cudaError_t join(const Join& a, int outputs, cudaStream_t stream) {
  return a.split <= 4   ? join<64, 4>(a, outputs, stream)
         : a.split <= 8 ? join<32, 8>(a, outputs, stream)
                        : join<16, 16>(a, outputs, stream);
}

// Pairs that share a tile of the forward or grad form.  (300 x 1024 x 2048,
// 32 tiles of 16 stages: 9.0 us whole, 9.5 in twos; 1021 x 2048 x 768, 24 of
// 32: 12.9 and 11.9.)
int split_pre(int64_t tiles, int64_t steps, const TcDevice& dev) { return dev.gated.split(tiles, steps, 24); }

int pairs_of(const Params& p, const TcLaunch& l) {
  return p.tiles + p.w_tiles < l.dev->pairs ? p.tiles + p.w_tiles : l.dev->pairs;
}

template <int FORM, int ACT>
cudaError_t launch(Params& p, const TcLaunch& l, cudaStream_t stream) {
  p.err = l.err;
  p.limit_ns = TIDE_BULK_TIMEOUT_NS;
  p.stall_ns = l.stall_ns, p.late_ns = l.late_ns;
  if constexpr (FORM != kBack) {
    p.split = split_pre(p.tiles, p.steps, *l.dev);
    p.share = Share(p.steps, p.split);
    if (p.split > 1)
      return launch_early(gated_tc_kernel<FORM, ACT, true>, dim3(2 * p.split * p.tiles), kThreads, kSmem, 2 * p.split, stream, p);
  }
  return launch_early(gated_tc_kernel<FORM, ACT, false>, dim3(2 * pairs_of(p, l)), kThreads, kSmem, 2, stream, p);
}

bool rows16(int64_t width, int64_t ld) { return width % 8 == 0 && ld % 8 == 0; }

// Operand boxes: 64 of the contraction x 128 rows (K-major), or 64 columns x
// 64 of the contraction (MN-major); both are 128 bytes wide.  Where the width
// is a multiple of 64 the latter's matrix is taken as slabs of 64 columns, so
// that one box holds two of them: the fewer boxes a stage has, the less its
// loads lag (70B-shaped dX and dW: 5.25 ms with four boxes by one thread, 4.81
// by two threads, 4.74 with two boxes).
bool map_k(CUtensorMap* m, const uint16_t* p, int64_t cols, int64_t rows, int64_t ld) {
  return make_map(m, p, 2, cols, rows, ld, kStep, kHalf, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_mn(CUtensorMap* m, const uint16_t* p, int64_t cols, int64_t rows, int64_t ld) {
  return cols % 64 == 0 ? make_slab_map(m, p, cols, rows, ld, kStep)
                        : make_map(m, p, 2, cols, rows, ld, 64, kStep, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_out(CUtensorMap* m, const uint16_t* p, int64_t cols, int64_t rows, int64_t ld) {
  return make_map(m, p, 2, cols, rows, ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

bool fill_pre(Params* p, const GatedArgs& a) {
  p->rows = (int)a.tokens, p->cols = p->features = (int)a.ffn;
  p->grid = TileGrid((int)ceil_div(a.tokens, 2 * kHalf), (int)ceil_div(a.ffn, kHalf));
  p->tiles = p->grid.all.d;
  p->steps = (int)ceil_div(a.hidden, kStep);
  if (!map_k(&p->a[0], a.x, a.hidden, a.tokens, a.ldx)) return false;
  p->a[1] = p->a[0];
  return map_k(&p->b[0], a.wg, a.hidden, a.ffn, a.hidden) && map_k(&p->b[1], a.wu, a.hidden, a.ffn, a.hidden);
}

// Parts of the sums of dX or dW.  Where there are fewer than half as many
// tiles as pairs (dX of few tokens, dW of a small block), the contraction is
// split and the parts, in fp32, are joined by another kernel.  In stages (0.27
// us): a tile's share, 18 for the join, and one for each 650 KB of parts.
// (256 tokens of the 8B-shaped block: 16 tiles of 448 stages, 130 -> 52 us
// in 4 parts; 1021 x 2048 x 768, 32 tiles of 24: 11 us whole, 18 in two.)
int split_of(int64_t tiles, int64_t steps, int pairs, int64_t part_bytes, int64_t room) {
  int best = 1;
  double least = (double)steps;
  for (int s = 2; s <= pairs / tiles && 4 * s <= steps && s * part_bytes <= room; ++s) {
    const double cost = (double)steps / s + 18 + (double)s * part_bytes / 650e3;
    if (cost < least) least = cost, best = s;
  }
  return best;
}

// The parts of at most one tile for each of a GB300's 76 pairs.
int64_t parts_bytes(int64_t tiles, int64_t part_bytes) { return tiles ? 76 / tiles * part_bytes : 0; }

}  // namespace

cudaError_t gated_tc_prepare(TcDevice* dev) {
  void (*const kernels[])(Params) = {
      gated_tc_kernel<kForward, TIDE_ACT_SILU, false>, gated_tc_kernel<kForward, TIDE_ACT_GELU, false>,
      gated_tc_kernel<kForward, TIDE_ACT_SILU, true>,  gated_tc_kernel<kForward, TIDE_ACT_GELU, true>,
      gated_tc_kernel<kGrad, TIDE_ACT_SILU, false>,    gated_tc_kernel<kGrad, TIDE_ACT_GELU, false>,
      gated_tc_kernel<kGrad, TIDE_ACT_SILU, true>,     gated_tc_kernel<kGrad, TIDE_ACT_GELU, true>,
      gated_tc_kernel<kBack, 0, false>};
  for (auto k : kernels) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
  }
  // the split kernels take the same shape
  const cudaError_t held = dev->gated.prepare((const void*)gated_tc_kernel<kForward, TIDE_ACT_SILU, true>, kThreads, kSmem);
  if (held != cudaSuccess) return held;
  // The pairs the device holds at one time: a GPC with an odd number of
  // SMs leaves one without a partner.
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim = {2, 1, 1};
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(2);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmem;
  c.attrs = &cluster;
  c.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(&dev->pairs, gated_tc_kernel<kBack, 0, false>, &c);
}

int64_t gated_dx_parts_bytes(int64_t tokens, int64_t hidden) {
  return parts_bytes(ceil_div(tokens, 2 * kHalf) * ceil_div(hidden, 2 * kHalf), 4 * tokens * hidden);
}
int64_t gated_dw_parts_bytes(int64_t hidden, int64_t ffn) {
  return parts_bytes(2 * ceil_div(ffn, 2 * kHalf) * ceil_div(hidden, 2 * kHalf), 8 * ffn * hidden);
}

int gated_tc_split(const GatedArgs& a, const TcDevice& dev) {
  return split_pre(ceil_div(a.tokens, 2 * kHalf) * ceil_div(a.ffn, kHalf), ceil_div(a.hidden, kStep), dev);
}

bool gated_tc_takes(const GatedArgs& a) { return a.hidden >= 8 && rows16(a.hidden, a.hidden) && rows16(a.ffn, a.ffn); }

cudaError_t launch_gated_forward_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  if (!fill_pre(&p, a) || !map_out(&p.outs[0], a.h, a.ffn, a.tokens, a.ldh)) return cudaErrorInvalidValue;
  p.out = a.h, p.ldo = a.ldh, p.g8 = a.g8, p.gs = a.gs, p.u8 = a.u8, p.us = a.us;
  return a.act == TIDE_ACT_SILU ? launch<kForward, TIDE_ACT_SILU>(p, l, stream)
                                : launch<kForward, TIDE_ACT_GELU>(p, l, stream);
}

cudaError_t launch_gated_grad_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  if (!fill_pre(&p, a) || !map_out(&p.outs[0], a.dg, a.ffn, a.tokens, a.ffn) ||
      !map_out(&p.outs[1], a.du, a.ffn, a.tokens, a.ffn) || (a.h && !map_out(&p.outs[2], a.h, a.ffn, a.tokens, a.ldh)))
    return cudaErrorInvalidValue;
  p.out = a.h, p.ldo = a.ldh, p.dh = a.dh, p.lddh = a.lddh, p.dg = a.dg, p.du = a.du;
  return a.act == TIDE_ACT_SILU ? launch<kGrad, TIDE_ACT_SILU>(p, l, stream) : launch<kGrad, TIDE_ACT_GELU>(p, l, stream);
}

cudaError_t launch_gated_back_tc(const GatedArgs& a, bool dx, bool dw, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  p.cols = (int)a.hidden;
  p.one_a = a.ffn % 64 == 0, p.one_b = a.hidden % 64 == 0;
  if (dx) {
    p.rows = (int)a.tokens;
    p.grid = TileGrid((int)ceil_div(a.tokens, 2 * kHalf), (int)ceil_div(a.hidden, 2 * kHalf));
    p.half_steps = (int)ceil_div(a.ffn, kStep), p.steps = 2 * p.half_steps;
    p.split = split_of(p.grid.all.d, p.steps, l.dev->pairs, 4 * a.tokens * a.hidden, a.dx_parts_bytes);
    p.share = Share(p.steps, p.split);
    p.parts = a.dx_parts;
    p.tiles = p.grid.all.d * p.split;
    if (!map_k(&p.a[0], a.dg, a.ffn, a.tokens, a.ffn) || !map_k(&p.a[1], a.du, a.ffn, a.tokens, a.ffn) ||
        !map_mn(&p.b[0], a.wg, a.hidden, a.ffn, a.hidden) || !map_mn(&p.b[1], a.wu, a.hidden, a.ffn, a.hidden) ||
        !map_out(&p.outs[0], a.dx, a.hidden, a.tokens, a.lddx))
      return cudaErrorInvalidValue;
  }
  if (dw) {
    p.w_rows = (int)a.ffn;
    p.w_grid = TileGrid((int)ceil_div(a.ffn, 2 * kHalf), (int)ceil_div(a.hidden, 2 * kHalf));
    p.w_tiles = 2 * p.w_grid.all.d;
    p.w_steps = (int)ceil_div(a.tokens, kStep);
    p.w_split = split_of(p.w_tiles, p.w_steps, l.dev->pairs, 8 * a.ffn * a.hidden, a.dw_parts_bytes);
    p.w_share = Share(p.w_steps, p.w_split);
    p.w_parts = a.dw_parts;
    p.w_tiles *= p.w_split;
    if (!map_mn(&p.wa[0], a.dg, a.ffn, a.tokens, a.ffn) || !map_mn(&p.wa[1], a.du, a.ffn, a.tokens, a.ffn) ||
        !map_mn(&p.wb, a.x, a.hidden, a.tokens, a.ldx) || !map_out(&p.outs[1], a.dwg, a.hidden, a.ffn, a.hidden) ||
        !map_out(&p.outs[2], a.dwu, a.hidden, a.ffn, a.hidden))
      return cudaErrorInvalidValue;
  }
  // What a tile of either takes: its stages, at least the four that writing it
  // takes, and about one for its way in and out.
  const int x_part = dx ? p.share.least : 0, w_part = dw && p.w_share.least > 4 ? p.w_share.least : 4;
  const int pairs = pairs_of(p, l), extra = (x_part + 1 + (w_part + 1) / 2) / (w_part + 1);
  p.each = p.tiles / pairs, p.full = p.tiles % pairs, p.light = pairs - p.full;
  p.first = !p.full ? 0 : p.w_tiles < p.light * extra ? p.w_tiles : p.light * extra;
  p.first_each = p.first / p.light, p.first_more = p.first % p.light;
  cudaError_t e = launch<kBack, 0>(p, l, stream);
  if (e == cudaSuccess && p.split > 1)
    e = join(Join{p.parts, p.split, {a.dx, nullptr}, a.lddx, p.rows, p.cols}, 1, stream);
  if (e == cudaSuccess && p.w_split > 1)
    e = join(Join{p.w_parts, p.w_split, {a.dwg, a.dwu}, a.hidden, p.w_rows, p.cols}, 2, stream);
  return e;
}

}  // namespace tide
