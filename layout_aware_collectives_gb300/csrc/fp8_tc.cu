// Product of two matrices held in 8-bit blocks, on the tensor cores.
//
//   out[i, j] = sum_b sa[i, b] sb[j / 128, b] sum_{k in b} a[i, k] b[j, k]
//
// A block is 128 steps of the contraction: one pipeline stage.  A pair of
// CTAs works on a 256 x 256 tile, each with 128 rows of A and 128 of B as in
// the gated block's kernel.  Two kernels:
//
// scaled_kernel: scales that are powers of two.  The tensor cores take them
// as exponent bytes beside the codes, so the whole contraction is summed in
// TMEM at their 8-bit rate.  Four warps write each stage's scales to TMEM.
// 4096 x 8192 x 28672: 525-555 us in short bursts (3.5-3.7 PFLOP/s), 634 in a
// run of passes (3.0), by what the card's power management allows: with all-zero
// codes the same kernel takes 427 us, 4.5 PFLOP/s, which is the tensor cores'
// nominal rate.  Reading a quarter less
// from L2, by sharing rows between two pairs, changed nothing.
//
// summed_kernel: any scales.  A block's sums go from one of two TMEM
// accumulators, times sa sb, into fp32 sums in the registers of 8 warps (one
// fused multiply-add each, a row's scale being a thread's; times the one and
// then the other where fp32 does not hold their product) while the tensor
// cores sum the next block into the other.  A block is 512 cycles of the
// tensor cores, but handing an accumulator there and back takes some 1,500:
// the barriers' way between the two CTAs, TMEM reads and the multiply-adds
// between them; and TMEM holds no third accumulator (4096 x 8192 x 28672: 664 us
// in short bursts, 745 in a run of passes, 2.6-2.9 PFLOP/s; 630 with all-zero
// codes).
#include "compute_device.cuh"
#include "tc_device.cuh"
#include "tc_host.h"

namespace tide {
namespace {

using namespace tc;

constexpr int kStages = 6;
constexpr int kHalf = 128;
constexpr uint32_t kOperand = kHalf * kBlock;  // bytes of either operand in one stage
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kSumWarps = 8;
constexpr int kThreads = 128 + 32 * kSumWarps;
constexpr int kBoxes = 2;
constexpr size_t kSmem = 1024 + kStages * kStage + kSumWarps * kBoxes * kBox;

struct Params {
  CUtensorMap a, b, out;
  const float *sa, *sb;
  int rows, cols;
  TileGrid grid;
  int tiles;
  int blocks;  // of the contraction
  int split;   // pairs of a cluster, which share its blocks
  uint16_t* to;  // out and its rows' length
  int64_t ldo;
  int* err;
  uint64_t limit_ns, stall_ns, late_ns;
};

template <int C>
__device__ __forceinline__ void add32(uint64_t (&sum)[kHalf / 2], const uint32_t (&v)[32], uint64_t s) {
#pragma unroll
  for (int i = 0; i < 16; ++i) fma2(sum[C * 16 + i], v[2 * i], v[2 * i + 1], s);
}

__device__ __forceinline__ void times32(uint32_t (&v)[32], float w) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(as_f(v[i]) * w);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) summed_kernel(const __grid_constant__ Params p) {
  constexpr uint32_t kInstr = instr_desc(0, 0, 0, 256, 256);
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kStages + 6];
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
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const Watch watch{&stop, p.err, p.limit_ns};
  const bool late = p.late_ns && warp == 4;  // test: this warp waits for sums where nothing arrives
  const Watch sums_watch{&stop, p.err, late ? p.late_ns : p.limit_ns};

  if (threadIdx.x == 0) {
    stop = 0;
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(sums_full(b), 1), bar_init(sums_empty(b), 2 * kSumWarps);
    bar_init(spare, 1), bar_init(silent, 1);
    bar_init_fence();
    prefetch_map(&p.a), prefetch_map(&p.b), prefetch_map(&p.out);
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
  } else if (warp < 4) {
    // 384 threads start with 168 registers each (64,512); this warpgroup goes
    // down to 56 and the two that hold sums go up to 216: 62,464.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if ((warp == 0 || warp == 3) && elected()) {
      const bool load_a = warp == 0;  // one thread loads A, another B
      int j = 0;  // stages filled so far
      bool go = true;
      for (int t = pair; t < p.tiles && go; t += pairs) {
        const TileAt at = tile_at(p.grid, t);
        for (int k = 0; k < p.blocks; ++k, ++j) {
          const int s = j % kStages;
          if (j >= kStages && !bar_wait(empty(s), (j / kStages + 1) & 1, watch)) {
            go = false;
            break;
          }
          if (load_a && rank == 0) bar_expect(full(s), 2 * kStage);
          const uint32_t bar = peer_addr(full(s), 0);
          const uint32_t a = smem + s * kStage;
          if (load_a)
            load_box<true>(a, &p.a, k * kBlock, (at.m * 2 + rank) * kHalf, bar);
          else
            load_box<true>(a + kOperand, &p.b, k * kBlock, (at.n * 2 + rank) * kHalf, bar);
        }
      }
      // the MMAs' last arrivals reach this CTA while it is still there
      for (int i = max(0, j - kStages); i < j && go; ++i) go = bar_wait(empty(i % kStages), (i / kStages) & 1, watch);
      // after a wait that ran out: both CTAs' copies in flight, with a limit
      // again; the peer's memory stays until the cluster's last barrier
      if (!go && rank == 0)
        for (int i = max(0, j - kStages); i < j; ++i) await(full(i % kStages), (i / kStages) & 1, watch);
    } else if (warp == 1 && rank == 0 && elected()) {
      int j = 0;  // blocks so far
      bool go = true;
      for (int t = pair; t < p.tiles && go; t += pairs) {
        for (int k = 0; k < p.blocks; ++k, ++j) {
          const int s = j % kStages, b = j & 1;
          if ((j >= 2 && !bar_wait<kPeer>(sums_empty(b), (j / 2 + 1) & 1, watch)) || !bar_wait(full(s), (j / kStages) & 1, watch)) {
            go = false;
            break;
          }
          fence_after();
          const uint32_t a = smem + s * kStage;
          const uint64_t da = operand_desc(a, 16), db = operand_desc(a + kOperand, 16);
#pragma unroll
          for (int q = 0; q < kBlock / 32; ++q) mma<2, true>(tmem + b * 256, da + q * 2, db + q * 2, kInstr, q > 0);
          mma_commit<2>(empty(s));
          mma_commit<2>(sums_full(b));
        }
      }
      mma_commit<2>(spare, 1);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int w = warp - 4, half = w >> 2;
    const uint32_t lanes = (uint32_t)(w & 3) * 32;
    Outbox<kBoxes> out{smem + kStages * kStage + w * kBoxes * kBox, 0, lane};
    const uint32_t taddr = tmem + (lanes << 16) + half * kHalf;
    int j = 0;
    bool go = true;
    for (int t = pair; t < p.tiles && go; t += pairs) {
      const TileAt at = tile_at(p.grid, t);
      const int row0 = (at.m * 2 + rank) * kHalf + lanes, row = row0 + lane;
      const int col0 = (at.n * 2 + half) * kHalf;
      // rows and columns past the end take any scale that is there: their
      // codes are zeros, or they are not written
      const float* sa = p.sa + (int64_t)min(row, p.rows - 1) * p.blocks;
      const float* sb = p.sb + (int64_t)(min(col0, p.cols - 1) / kBlock) * p.blocks;
      uint64_t sum[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) sum[i] = 0;
      float next_a = __ldg(sa), next_b = __ldg(sb);
      for (int k = 0; k < p.blocks; ++k, ++j) {
        const int b = j & 1;
        float both = next_a * next_b, w = next_b;
        const bool apart = __any_sync(0xffffffffu, !normal(both));  // the sums times w, then times both
        if (apart) {
          const float power = leave_power(w);
          both = take_power(next_a, power);
        }
        const uint64_t s = twice(both);
        if (k + 1 < p.blocks) next_a = __ldg(sa + k + 1), next_b = __ldg(sb + k + 1);
        if (!bar_wait_warp(late ? silent : sums_full(b), (j / 2) & 1, sums_watch)) {
          go = false;
          break;
        }
        fence_after();
        // Each half of the sums is on its way while the other is added.
        uint32_t v[32], x[32];
        const uint32_t from = taddr + b * 256;
        tmem_issue32(from, v);
        tmem_issue32(from + 32, x);
        tmem_arrived(v, x);
        if (apart) times32(v, w), times32(x, w);
        add32<0>(sum, v, s);
        tmem_issue32(from + 64, v);
        add32<1>(sum, x, s);
        tmem_issue32(from + 96, x);
        tmem_arrived(v, x);
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive_peer(peer_addr(sums_empty(b), 0));
        if (apart) times32(v, w), times32(x, w);
        add32<2>(sum, v, s);
        add32<3>(sum, x, s);
      }
      if (!go) break;
#pragma unroll
      for (int c = 0; c < kHalf / 32; ++c) {
        const int col = col0 + c * 32;
        if (row0 < p.rows && col < p.cols) {
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = pack_bf16(as_f((uint32_t)sum[c * 16 + i]), as_f((uint32_t)(sum[c * 16 + i] >> 32)));
          out.put(&p.out, o, col, row0);
        }
      }
    }
    if (lane == 0) stores_done();
  }
  __syncthreads();
  if (stop && warp == 1 && rank == 0 && !p.stall_ns) {
    await(spare, 0, watch);  // the MMAs in flight
    __syncwarp();
  }
  cluster_sync();
  if (warp == 2) tmem_free<2>(tmem, 512);
}

// ------------------------------------------------------ powers of two only

// TMEM: a tile's 256 columns of sums start at 0 or at 160 in turn, the
// scales' ring takes 6 x 12 from 416 on.  Two tiles' sums share 96 columns;
// those are read first, and the next tile starts as soon as they are.
constexpr int kOdd = 160;
constexpr int kShared = 3;  // chunks of 32 columns
constexpr int kScales = 416;
constexpr int kScaledThreads = 384;  // loads, MMAs, -, -, 4 warps of results, 4 of scales
constexpr int kScaledBoxes = 3;
constexpr size_t kScaledSmem = 1024 + kStages * kStage + 4 * kScaledBoxes * kBox;
static_assert(kHalf * kSumRow <= kStages * kStage, "the sums lie where the stages were");

// SPLIT: where the tiles leave SMs without work, a cluster of two to four
// pairs works on one, each pair on a part of the contraction; the sums meet
// over distributed shared memory, in the order of the parts (1024 x 1024 x
// 8192, 16 tiles: 25.2 us by single pairs, 14.9 in threes and fours;
// 1021 x 768 x 2048, 12 tiles: 9.7, in twos 8.9).  A stage takes 0.33 us, the
// sums' meeting some 4.
template <bool SPLIT>
__global__ void __launch_bounds__(kScaledThreads, 1) scaled_kernel(const __grid_constant__ Params p) {
  constexpr uint32_t kInstr = instr_desc_scaled(256, 256);
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t words[2][4][kHalf];  // scales of two batches of four blocks
  __shared__ uint32_t tmem_at;
  __shared__ int stop;

  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  const auto full = [&](int s) { return bar0 + 8u * s; };
  const auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  const uint32_t sums_full = bar0 + 8u * (2 * kStages), sums_empty = sums_full + 8, spare = sums_full + 16, silent = sums_full + 24;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t cta = cluster_rank(), rank = cta & 1, leader = SPLIT ? cta & ~1u : 0;
  const uint16_t both = (uint16_t)(3u << leader);  // the pair's CTAs
  const int split = SPLIT ? p.split : 1, part = cta >> 1;
  const int pair = blockIdx.x / (2 * split), pairs = gridDim.x / (2 * split);
  const int k0 = SPLIT ? p.blocks * part / split : 0, k1 = SPLIT ? p.blocks * (part + 1) / split : p.blocks;
  const Watch watch{&stop, p.err, p.limit_ns};
  const bool late = p.late_ns && warp == 4;  // test: this warp waits for sums where nothing arrives
  const Watch sums_watch{&stop, p.err, late ? p.late_ns : p.limit_ns};

  if (threadIdx.x == 0) {
    stop = 0;
    // full: the copies, and four warps' scales in each CTA
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1 + 2 * 4), bar_init(empty(s), 1);
    bar_init(sums_full, 1), bar_init(sums_empty, 2 * 4), bar_init(spare, 1), bar_init(silent, 1);
    bar_init_fence();
    prefetch_map(&p.a), prefetch_map(&p.b), prefetch_map(&p.out);
  }
  if (warp == 2) tmem_alloc<2>(smem_addr(&tmem_at), 512);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_at;
  after_previous();

  // SPLIT: half of the columns' sums of this warp's 32 rows
  const auto leave_half = [&](int first) {
    if (!bar_wait_warp(late ? silent : sums_full, 0, sums_watch)) return;
    fence_after();
    const uint32_t lanes = (uint32_t)(warp & 3) * 32;
    leave_sums(smem, tmem + (lanes << 16), lanes + lane, first);
    fence_before();
  };

  if (p.stall_ns) {  // test: a wait on a barrier nothing arrives on runs out
    if (threadIdx.x == 0) bar_wait(silent, 0, Watch{&stop, p.err, p.stall_ns});
  } else if (warp == 0 || warp == 3) {
    if (elected()) {
      const bool load_a = warp == 0;  // one thread loads A, another B
      int j = 0;  // stages filled so far
      bool go = true;
      for (int t = pair; t < p.tiles && go; t += pairs) {
        const TileAt at = tile_at(p.grid, t);
        for (int k = k0; k < k1; ++k, ++j) {
          const int s = j % kStages;
          if (j >= kStages && !bar_wait(empty(s), (j / kStages + 1) & 1, watch)) {
            go = false;
            break;
          }
          if (load_a && rank == 0) bar_expect(full(s), 2 * kStage);
          const uint32_t bar = peer_addr(full(s), leader);
          const uint32_t a = smem + s * kStage;
          if (load_a)
            load_box<true>(a, &p.a, k * kBlock, (at.m * 2 + rank) * kHalf, bar);
          else
            load_box<true>(a + kOperand, &p.b, k * kBlock, (at.n * 2 + rank) * kHalf, bar);
        }
      }
      // the MMAs' last arrivals reach this CTA while it is still there
      for (int i = max(0, j - kStages); i < j && go; ++i) go = bar_wait(empty(i % kStages), (i / kStages) & 1, watch);
      // after a wait that ran out: both CTAs' copies in flight, with a limit
      // again; the peer's memory stays until the cluster's last barrier
      if (!go && rank == 0)
        for (int i = max(0, j - kStages); i < j; ++i) await(full(i % kStages), (i / kStages) & 1, watch);
    }
  } else if (warp == 1) {
    if (rank == 0 && elected()) {
      int j = 0, i = 0;  // blocks and tiles so far
      bool go = true;
      for (int t = pair; t < p.tiles && go; t += pairs, ++i) {
        if (i > 0 && !bar_wait<kPeer>(sums_empty, (i + 1) & 1, watch)) break;
        fence_after();
        const uint32_t sums = tmem + (i & 1) * kOdd;
        for (int k = k0; k < k1; ++k, ++j) {
          const int s = j % kStages;
          if (!bar_wait<kOwnAndPeer>(full(s), (j / kStages) & 1, watch)) {
            go = false;
            break;
          }
          fence_after();
          const uint32_t a = smem + s * kStage, scales = tmem + kScales + s * 12;
          const uint64_t da = operand_desc(a, 16), db = operand_desc(a + kOperand, 16);
#pragma unroll
          for (int q = 0; q < kBlock / 32; ++q)
            mma_scaled(sums, da + q * 2, db + q * 2, kInstr, scales, scales + 4, k > k0 || q > 0);
          mma_commit<2>(empty(s), both);
        }
        if (go) mma_commit<2>(sums_full, both);
      }
      mma_commit<2>(spare, (uint16_t)(1u << leader));
    }
  } else if (warp >= 8) {
    // Scales.  Every warp writes all 128 rows' (A, 4 columns) and both column
    // blocks' (B, 8 columns) to its own 32 lanes.  Four blocks at a time, a
    // batch ahead, each warp fetches 32 rows' and the four exchange them: a
    // load that touches 32 rows takes L1 32 cycles, and with every warp
    // fetching all rows these loads were 40% slower than the products.
    const int w = warp & 3;
    const uint32_t mine = tmem + ((uint32_t)w * 32 << 16) + kScales;
    int j = 0, batch = 0;
    bool go = true;
    for (int t = pair; t < p.tiles; t += pairs) {
      const TileAt at = tile_at(p.grid, t);
      // rows and columns past the end take any scale that is there
      const float* sa = p.sa + (int64_t)min((int)(at.m * 2 + rank) * kHalf + w * 32 + lane, p.rows - 1) * p.blocks;
      const float* sb = p.sb + (int64_t)min(at.n * 2 + (lane & 1), (p.cols - 1) / kBlock) * p.blocks;
      float next_a[4], next_b[4];
      const auto fetch = [&](int k) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          next_a[q] = __ldg(sa + min(k + q, k1 - 1));
          next_b[q] = __ldg(sb + min(k + q, k1 - 1));
        }
      };
      fetch(k0);
      for (int k = k0; k < k1; k += 4, ++batch) {
        uint32_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          words[batch & 1][q][w * 32 + lane] = exponent_bytes(next_a[q]);
          b[q] = exponent_bytes(next_b[q]);
        }
        if (k + 4 < k1) fetch(k + 4);
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (k + q >= k1) break;
          const int s = j % kStages;
          // a warp whose wait ran out goes on meeting the others at the barrier
          go = go && (j < kStages || bar_wait_warp(empty(s), (j / kStages + 1) & 1, watch));
          if (!go) continue;
          fence_after();
          const uint32_t to = mine + s * 12;
          const uint32_t b0 = __shfl_sync(0xffffffffu, b[q], 0), b1 = __shfl_sync(0xffffffffu, b[q], 1);
          const uint32_t* row = words[batch & 1][q] + lane;
          tmem_write4(to, row[0], row[32], row[64], row[96]);
          tmem_write4(to + 4, b0, b0, b0, b0);
          tmem_write4(to + 8, b1, b1, b1, b1);
          tmem_written();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive_peer(peer_addr(full(s), leader));
          ++j;
        }
      }
    }
    if constexpr (SPLIT) leave_half(4);
  } else if (warp >= 4) {
    if constexpr (SPLIT) leave_half(0);
    Outbox<kScaledBoxes> out{smem + kStages * kStage + (warp - 4) * kScaledBoxes * kBox, 0, lane};
    const uint32_t lanes = (uint32_t)(warp - 4) * 32;
    int i = 0;
    for (int t = pair; t < p.tiles && !SPLIT; t += pairs, ++i) {
      if (!bar_wait_warp(late ? silent : sums_full, i & 1, sums_watch)) break;
      fence_after();
      const TileAt at = tile_at(p.grid, t);
      const int row0 = (at.m * 2 + rank) * kHalf + lanes, col0 = at.n * 2 * kHalf;
      const uint32_t sums = tmem + (lanes << 16) + (i & 1) * kOdd;
      const int first = i & 1 ? 0 : 8 - kShared;  // the chunks the next tile shares
      uint32_t o[kShared][16];
#pragma unroll
      for (int c = 0; c < kShared; ++c) {
        uint32_t v[32];
        tmem_read(sums + (first + c) * 32, v);
#pragma unroll
        for (int q = 0; q < 16; ++q) o[c][q] = pack_bf16(as_f(v[2 * q]), as_f(v[2 * q + 1]));
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_peer(peer_addr(sums_empty, leader));
#pragma unroll
      for (int c = 0; c < kShared; ++c) {
        const int col = col0 + (first + c) * 32;
        if (row0 < p.rows && col < p.cols) out.put(&p.out, o[c], col, row0);
      }
#pragma unroll 1
      for (int c = 0; c < 8 - kShared; ++c) {
        const int chunk = i & 1 ? kShared + c : c, col = col0 + chunk * 32;
        uint32_t v[32];
        tmem_read(sums + chunk * 32, v);
        if (row0 >= p.rows || col >= p.cols) continue;
#pragma unroll
        for (int q = 0; q < 16; ++q) o[0][q] = pack_bf16(as_f(v[2 * q]), as_f(v[2 * q + 1]));
        out.put(&p.out, o[0], col, row0);
      }
      fence_before();
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
    const int row0 = (at.m * 2 + rank) * kHalf, col0 = at.n * 2 * kHalf + lane * 4;
    const int r1 = min(kHalf * (part + 1) / split, p.rows - row0);
    if (!p.stall_ns) {
      for (int r = kHalf * part / split + warp; r < r1; r += kScaledThreads / 32) {
        float4 sum[2];
        split_sums(smem, r, lane, rank, split, sum);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = col0 + c * kHalf;
          if (col < p.cols)
            *(uint2*)(p.to + (int64_t)(row0 + r) * p.ldo + col) =
                make_uint2(pack_bf16(sum[c].x, sum[c].y), pack_bf16(sum[c].z, sum[c].w));
        }
      }
    }
    cluster_sync();  // the others have read this CTA's sums
  }
  if (warp == 2) tmem_free<2>(tmem, 512);
}

}  // namespace

cudaError_t fp8_tc_prepare(TcDevice* dev) {
  cudaError_t e = cudaFuncSetAttribute(summed_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(scaled_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScaledSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(scaled_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScaledSmem);
  if (e == cudaSuccess) e = dev->fp8.prepare((const void*)scaled_kernel<true>, kScaledThreads, kScaledSmem);
  return e;
}

int fp8_tc_split(const MatmulArgs& a, const TcDevice& dev) {
  if (a.any_scales) return 1;
  return dev.fp8.split(ceil_div(a.m, 2 * kHalf) * ceil_div(a.n, 2 * kHalf), ceil_div(a.k, kBlock), 16);
}

cudaError_t launch_fp8_matmul_tc(const MatmulArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  p.sa = a.sa, p.sb = a.sb;
  p.rows = (int)a.m, p.cols = (int)a.n;
  p.grid = TileGrid((int)ceil_div(a.m, 2 * kHalf), (int)ceil_div(a.n, 2 * kHalf));
  p.tiles = p.grid.all.d;
  p.blocks = (int)ceil_div(a.k, kBlock);
  p.to = a.out, p.ldo = a.ldo;
  p.err = l.err;
  p.limit_ns = TIDE_BULK_TIMEOUT_NS;
  p.stall_ns = l.stall_ns, p.late_ns = l.late_ns;
  if (!make_map(&p.a, a.a, 1, a.k, a.m, a.k, kBlock, kHalf, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.b, a.b, 1, a.k, a.n, a.k, kBlock, kHalf, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.out, a.out, 2, a.n, a.m, a.ldo, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const int pairs = p.tiles < l.dev->pairs ? p.tiles : l.dev->pairs;
  p.split = fp8_tc_split(a, *l.dev);
  if (p.split > 1)
    return launch_early(scaled_kernel<true>, dim3(2 * p.split * p.tiles), kScaledThreads, kScaledSmem, 2 * p.split, stream, p);
  return a.any_scales ? launch_early(summed_kernel, dim3(2 * pairs), kThreads, kSmem, 0, stream, p)
                      : launch_early(scaled_kernel<false>, dim3(2 * pairs), kScaledThreads, kScaledSmem, 2, stream, p);
}

}  // namespace tide
