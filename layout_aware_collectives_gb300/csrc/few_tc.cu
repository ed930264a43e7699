// The gated block, forward and backward, and the 8-bit product for few tokens
// (one to a few hundred), where the weights' bytes are what counts.
//
// The tiles of gated_tc.cu and fp8_tc.cu put 256 tokens on the tensor cores'
// rows; with few tokens most of those are padding and few tiles are left to
// share out.  Here the weights take the rows: a CTA multiplies 128 of them
// (for the gated block 128 of Wg and the same 128 of Wu) by NT = 16 to 64
// tokens, and a cluster of up to 8 CTAs splits the contraction.  Each CTA
// leaves its sums in its shared memory, [token][feature] in fp32; then every
// CTA of the cluster finishes its share of the tokens, adding the others'
// sums over distributed shared memory in the order of their ranks, so the
// result does not depend on timing.
//
// Bound by HBM: the weights stream through a ring of 5-12 stages of 18-40 KiB
// (a ring of 3-6, with room for two CTAs to an SM, was slower for the gated
// block, 8192 x 28672 gate and up 152 us against 140, and faster for the 8-bit
// product, 43.8 against 45.5).  One token: 4096 x 14336 gate and up 36 us (6.5
// TB/s; once they flow the rest is the ramp), their dX 37 us, an 8192 x 28672
// 8-bit product 41 us (5.7 TB/s).  Small blocks take 4-7 us of waits one after
// the other: the first stage's 0.6 us, 0.15-0.3 us a stage, the clusters'
// meetings 0.7 us each.
#include "compute_device.cuh"
#include "gated_finish.cuh"
#include "tc_device.cuh"
#include "tc_host.h"

namespace tide {
namespace {

using namespace tc;

constexpr int kRows = 128;             // weights of a tile
constexpr uint32_t kRowBytes = 128;    // of either operand in one stage
constexpr uint32_t kWeights = kRows * kRowBytes;
constexpr int kThreads = 192;          // loads, MMAs, 4 warps for the sums

// What is computed: h, dG and dU (and h), the 8-bit product, or dX.  For dX
// the rows are the hidden features, columns of Wg and Wu, which lie along
// memory (MN-major), and the contraction runs over dG's features and then
// dU's.
enum Kind { kForward = 0, kGrad = 1, kFp8 = 2, kDx = 3 };

template <int KIND, int NT>
struct Shape {
  static constexpr bool FP8 = KIND == kFp8;
  static constexpr int kParts = KIND == kFp8 || KIND == kDx ? 1 : 2;  // weight tiles of a stage
  static constexpr uint32_t kStage = kParts * kWeights + NT * kRowBytes;
  static constexpr uint32_t kBudget = FP8 && NT <= 32 ? 108 * 1024 : 210 * 1024;
  static constexpr int kStages = kBudget / kStage < 12 ? kBudget / kStage : 12;
  static constexpr int kBufs = FP8 ? 4 : 1;  // accumulators of kParts * NT columns
  static constexpr int kColumns = kBufs * kParts * NT < 32 ? 32 : kBufs * kParts * NT;
  static constexpr uint32_t kSums = kParts * NT * kRows * 4;
  static constexpr size_t kSmem = 1024 + (kStages * kStage > kSums ? kStages * kStage : kSums);
};

struct Params : GatedOut {  // 8-bit product, dX: out, ldo and features of it
  CUtensorMap w[2], x[2];
  int tokens, steps, step_elems;
  int half_steps;  // dX: stages of dG's half
  bool one_box;    // dX: a stage's weights are one box of two slabs
  // 8-bit
  const float *sx, *sw;
  bool any_scales;
  int* err;
  uint64_t limit_ns, stall_ns, late_ns;
};

// Sums of the cluster's CTAs' sums at N addresses, in rank order.  Four ranks'
// reads are on their way before the first is added.
template <int N>
__device__ __forceinline__ void cluster_sums(const uint32_t (&addr)[N], int split, float4 (&v)[N]) {
  constexpr int kAtOnce = 4;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int r = 0; r < split; r += kAtOnce) {
    float4 a[kAtOnce][N];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
      for (int i = 0; i < N; ++i)
        a[q][i] = r + q < split ? peer_read(peer_addr(addr[i], r + q)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i].x += a[q][i].x, v[i].y += a[q][i].y, v[i].z += a[q][i].z, v[i].w += a[q][i].w;
  }
}
__device__ __forceinline__ float4 own_read(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ void sums_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int KIND, int NT, int ACT>
__global__ void __launch_bounds__(kThreads) few_tc_kernel(const __grid_constant__ Params p) {
  using S = Shape<KIND, NT>;
  constexpr bool FP8 = S::FP8;
  constexpr bool kMn = KIND == kDx;
  constexpr uint32_t kInstr = instr_desc(FP8 ? 0 : 1, kMn, 0, kRows, NT);
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * S::kStages + 2 * S::kBufs + 2];
  __shared__ __align__(16) float scales[4][FP8 ? NT : 4];
  __shared__ uint32_t tmem_at;
  __shared__ int stop;

  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  const auto full = [&](int s) { return bar0 + 8u * s; };
  const auto empty = [&](int s) { return bar0 + 8u * (S::kStages + s); };
  const auto sums_full = [&](int b) { return bar0 + 8u * (2 * S::kStages + b); };
  const auto sums_empty = [&](int b) { return bar0 + 8u * (2 * S::kStages + S::kBufs + b); };
  const uint32_t spare = bar0 + 8u * (2 * S::kStages + 2 * S::kBufs), silent = spare + 8;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x;  // the cluster is a row of the grid
  const int token0 = blockIdx.y * NT, feature0 = blockIdx.z * kRows;
  const int k0 = (int)((int64_t)p.steps * rank / split), k1 = (int)((int64_t)p.steps * (rank + 1) / split);
  const Watch watch{&stop, p.err, p.limit_ns};
  const bool late = p.late_ns && warp == 2;  // test: this warp waits for sums where nothing arrives
  const Watch sums_watch{&stop, p.err, late ? p.late_ns : p.limit_ns};

  if (threadIdx.x == 0) {
    stop = 0;
    for (int s = 0; s < S::kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < S::kBufs; ++b) bar_init(sums_full(b), 1), bar_init(sums_empty(b), 4);
    bar_init(spare, 1), bar_init(silent, 1);
    bar_init_fence();
    prefetch_map(&p.w[0]), prefetch_map(&p.x[0]);
  }
  if (warp == 1) tmem_alloc<1>(smem_addr(&tmem_at), S::kColumns);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_at;
  after_previous();
  bool done = false;  // this warp has its sums in shared memory
  int filled = 0;     // stages this thread has filled

  if (p.stall_ns) {  // test: a wait on a barrier nothing arrives on runs out
    if (threadIdx.x == 0) bar_wait(silent, 0, Watch{&stop, p.err, p.stall_ns});
  } else if (warp == 0) {
    if (elected()) {
      int j = 0;
      for (int k = k0; k < k1; ++k, ++j) {
        const int s = j % S::kStages;
        if (j >= S::kStages && !bar_wait(empty(s), (j / S::kStages + 1) & 1, watch)) break;
        const uint32_t at = smem + s * S::kStage;
        bar_expect(full(s), S::kStage);
        if constexpr (KIND == kDx) {
          const int second = k >= p.half_steps, f = (k - (second ? p.half_steps : 0)) * p.step_elems;
          if (p.one_box) {
            load_box3<false>(at, &p.w[second], 0, f, feature0 / 64, full(s));
          } else {
            load_box<false>(at, &p.w[second], feature0, f, full(s));
            load_box<false>(at + kWeights / 2, &p.w[second], feature0 + 64, f, full(s));
          }
          load_box<false>(at + kWeights, &p.x[second], f, token0, full(s));
        } else {
#pragma unroll
          for (int i = 0; i < S::kParts; ++i)
            load_box<false>(at + i * kWeights, &p.w[i], k * p.step_elems, feature0, full(s));
          load_box<false>(at + S::kParts * kWeights, &p.x[0], k * p.step_elems, token0, full(s));
        }
      }
      filled = j;
    }
  } else if (warp == 1) {
    if (elected()) {
      int j = 0;
      for (int k = k0; k < k1; ++k, ++j) {
        const int s = j % S::kStages, b = j % S::kBufs;
        if ((FP8 && j >= S::kBufs && !bar_wait(sums_empty(b), (j / S::kBufs + 1) & 1, watch)) ||
            !bar_wait(full(s), (j / S::kStages) & 1, watch))
          break;
        fence_after();
        const uint32_t at = smem + s * S::kStage;
        const uint64_t dx = operand_desc(at + S::kParts * kWeights, 16);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < S::kParts; ++i)
            mma<1, FP8>(tmem + (b * S::kParts + i) * NT,
                        operand_desc(at + i * kWeights, kMn ? kWeights / 2 : 16) + q * ((kMn ? 2048 : 32) >> 4), dx + q * 2,
                        kInstr, q > 0 || (!FP8 && j > 0));
        mma_commit<1>(empty(s));
        if (FP8 || k + 1 == k1) mma_commit<1>(sums_full(b));
      }
      mma_commit<1>(spare);
    }
  } else {
    const int lanes = (warp & 3) * 32, feature = lanes + lane;  // TMEM lanes follow the warp's index modulo 4
    const uint32_t mine = tmem + ((uint32_t)lanes << 16);
    constexpr int kChunk = NT < 32 ? NT : 32;
    const auto leave = [&](int row, float v) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(smem + (uint32_t)(row * kRows + feature) * 4), "f"(v) : "memory");
    };
    if constexpr (FP8) {
      const int e = threadIdx.x - 64;  // the token whose scales this thread fetches
      const float* sx = p.sx + (int64_t)min(token0 + e, p.tokens - 1) * p.steps;
      const float* sw = p.sw + (int64_t)blockIdx.z * p.steps;
      uint64_t sum[NT / 2];
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) sum[i] = 0;
      // Each step's scales: the tokens' in shared memory, the weights' as the
      // result.  A step ahead, behind the issue of the read of the sums.
      float next_x = 0.0f, next_w = 0.0f;
      const auto fetch = [&](int k) {
        if (k >= k1) return;
        next_w = __ldg(sw + k);
        if (e < NT) next_x = __ldg(sx + k);
      };
      const auto prepare = [&](int k, int j) {
        float w = p.any_scales ? next_w : power_of_two(next_w);
        const float power = leave_power(w);
        if (e < NT) scales[j & 3][e] = take_power(p.any_scales ? next_x : power_of_two(next_x), power);
        fetch(k + 1);
        return twice(w);
      };
      fetch(k0);
      uint64_t next = prepare(k0, 0);
      done = true;
      int j = 0;
      for (int k = k0; k < k1; ++k, ++j) {
        const int b = j % S::kBufs;
        sums_barrier();
        // a warp whose wait ran out goes on meeting the others at the barrier
        done = done && bar_wait_warp(late ? silent : sums_full(b), (j / S::kBufs) & 1, sums_watch);
        if (!done) continue;
        fence_after();
        const uint64_t w = next;
        uint32_t v[NT / kChunk][kChunk];
        if constexpr (NT == 16) {
          tmem_issue16(mine + b * NT, v[0]);
        } else {
#pragma unroll
          for (int c = 0; c < NT / kChunk; ++c) tmem_issue32(mine + b * NT + c * kChunk, v[c]);
        }
        next = prepare(k + 1, j + 1);
        if constexpr (NT == 64)
          tmem_arrived(v[0], v[1]);
        else
          tmem_arrived(v[0]);
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(sums_empty(b));
#pragma unroll
        for (int c = 0; c < NT / kChunk; ++c)
#pragma unroll
          for (int i = 0; i < kChunk; i += 4) {
            const ulonglong2 s = *(const ulonglong2*)&scales[j & 3][c * kChunk + i];
            uint64_t* to = sum + (c * kChunk + i) / 2;
            mul_fma2(to[0], v[c][i], v[c][i + 1], w, s.x);
            mul_fma2(to[1], v[c][i + 2], v[c][i + 3], w, s.y);
          }
      }
      if (done) {
        // every warp's last read of the stages is over: all MMAs completed
#pragma unroll
        for (int i = 0; i < NT; ++i) leave(i, as_f((uint32_t)(sum[i / 2] >> 32 * (i & 1))));
      }
    } else {
      done = k0 < k1 ? bar_wait_warp(late ? silent : sums_full(0), 0, sums_watch) : true;
      if (done) {
        fence_after();
#pragma unroll 1
        for (int c = 0; c < S::kParts * NT / kChunk; ++c) {
          uint32_t v[kChunk];
          if (k0 < k1)
            tmem_read(mine + c * kChunk, v);
          else
            for (int i = 0; i < kChunk; ++i) v[i] = 0;
#pragma unroll
          for (int i = 0; i < kChunk; ++i) leave(c * kChunk + i, as_f(v[i]));
        }
      }
    }
  }
  __syncthreads();
  if (stop && !p.stall_ns) {  // copies and MMAs in flight, with a limit again
    for (int i = max(0, filled - S::kStages); i < filled; ++i) await(full(i % S::kStages), (i / S::kStages) & 1, watch);
    if (warp == 1) await(spare, 0, watch);
    __syncwarp();
  }
  if (split > 1) cluster_sync();
  if (!p.stall_ns) {
    constexpr int kWarps = kThreads / 32;
    const int col = feature0 + lane * 4;
    const int live = min(NT, p.tokens - token0);
    // One token's results from its sums.
    const auto finish = [&](int t, const float4* v) {
      const int64_t token = token0 + t;
      if constexpr (KIND == kForward)
        finish_forward<ACT>(p, token, blockIdx.z, lane, v[0], v[1]);
      else if constexpr (KIND == kGrad)
        finish_grad<ACT>(p, token, blockIdx.z, lane, v[0], v[1]);
      else if (col < p.features)
        put_bf16(p.out + token * p.ldo + col, v[0]);
    };
    const auto sums_at = [&](int t, int q) { return smem + (uint32_t)((q * NT + t) * kRows + lane * 4) * 4; };
    constexpr int P = S::kParts;
    const int each = kWarps * split;
    for (int t = rank * kWarps + warp; t < live; t += 2 * each) {
      uint32_t addr[2 * P];
      float4 v[2 * P];
      const bool two = t + each < live;
#pragma unroll
      for (int q = 0; q < P; ++q) addr[q] = sums_at(t, q), addr[P + q] = sums_at(t + each, q);
      if (split == 1) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
          v[q] = own_read(addr[q]);
          if (two) v[P + q] = own_read(addr[P + q]);
        }
      } else if (two) {
        cluster_sums(addr, split, v);
      } else {
        const uint32_t (&first)[P] = *(const uint32_t(*)[P])addr;
        float4 (&w)[P] = *(float4(*)[P])v;
        cluster_sums(first, split, w);
      }
      finish(t, v);
      if (two) finish(t + each, v + P);
    }
  }
  if (split > 1) cluster_sync();  // the others have read this CTA's sums
  if (warp == 1) tmem_free<1>(tmem, S::kColumns);
}

constexpr int tile_index(int nt) { return nt == 16 ? 0 : nt == 32 ? 1 : 2; }

template <int KIND, int NT, int ACT>
cudaError_t prepare(TcDevice* dev) {
  using S = Shape<KIND, NT>;
  cudaError_t e = cudaFuncSetAttribute(few_tc_kernel<KIND, NT, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  for (int n = 2; n <= kMaxCluster && e == cudaSuccess; ++n) {
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {(unsigned)n, 1, 1};
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(n);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = S::kSmem;
    c.attrs = &cluster;
    c.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&dev->few[KIND][tile_index(NT)][ACT][n], few_tc_kernel<KIND, NT, ACT>, &c);
  }
  return e;
}

template <int KIND, int ACT = 0>
cudaError_t prepare_tiles(TcDevice* dev) {
  cudaError_t e = prepare<KIND, 16, ACT>(dev);
  if (e == cudaSuccess) e = prepare<KIND, 32, ACT>(dev);
  return e == cudaSuccess ? prepare<KIND, 64, ACT>(dev) : e;
}

// CTAs that share a tile's contraction: up to one for each SM, all at work at
// one time, each with at least four stages of it, or, where more than four
// exchange 64 tokens' gate and up sums, twelve (fewer save less than the
// exchange takes).  (16 tiles of 64 tokens, gated, 8192 x 2048: 18.1 us split
// in four, 17.6 in six, 28.1 in eight, where the last clusters wait for the
// first; 4096 x 2048: 12.4 in four, 12.9 in six; dX of 7 x 2048 x 8192: 15.6
// in four, 13.0 in six.)
template <int KIND, int NT, int ACT>
int split_of(int64_t tiles, int64_t steps, const TcDevice& dev) {
  const FewClusters& clusters = dev.few[KIND][tile_index(NT)][ACT];
  constexpr int kMany = NT == 64 && Shape<KIND, NT>::kParts == 2 ? 12 : 4;  // stages, of more than four
  int s = kMaxCluster;
  while (s > 1 && (s * tiles > dev.sms || clusters[s] < tiles || steps < (s > 4 ? kMany : 4) * s)) --s;
  return s;
}

template <int KIND, int NT, int ACT>
cudaError_t launch(Params& p, const TcLaunch& l, cudaStream_t stream) {
  using S = Shape<KIND, NT>;
  p.err = l.err;
  p.limit_ns = TIDE_BULK_TIMEOUT_NS;
  p.stall_ns = l.stall_ns, p.late_ns = l.late_ns;
  const int64_t tiles_t = ceil_div(p.tokens, NT), tiles_f = ceil_div(p.features, kRows);
  const int split = split_of<KIND, NT, ACT>(tiles_t * tiles_f, p.steps, *l.dev);
  return launch_early(few_tc_kernel<KIND, NT, ACT>, dim3(split, (unsigned)tiles_t, (unsigned)tiles_f), kThreads, S::kSmem,
                      (unsigned)split, stream, p);
}

int tile_of(int64_t tokens) { return tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64; }

// One tile of tokens, or so few tiles in all that the 256-token tiles of the
// other kernels would leave most SMs without work.
bool few(int64_t tokens, int64_t features, int64_t most) {
  const int64_t tiles = ceil_div(features, kRows);
  return tiles <= 65535 && (tokens <= 64 || tiles * ceil_div(tokens, 64) <= most);
}

template <int KIND, int ACT = 0>
cudaError_t launch_tile(Params& p, int nt, const TcLaunch& l, cudaStream_t stream) {
  return nt == 16   ? launch<KIND, 16, ACT>(p, l, stream)
         : nt == 32 ? launch<KIND, 32, ACT>(p, l, stream)
                    : launch<KIND, 64, ACT>(p, l, stream);
}

// Both kinds of the gated block: operands and sizes.
template <int KIND>
cudaError_t gated(Params& p, const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  constexpr int kElems = kRowBytes / 2;
  const int nt = tile_of(a.tokens);
  p.tokens = (int)a.tokens, p.features = (int)a.ffn;
  p.steps = (int)ceil_div(a.hidden, kElems), p.step_elems = kElems;
  p.out = a.h, p.ldo = a.ldh;
  if (!make_map(&p.w[0], a.wg, 2, a.hidden, a.ffn, a.hidden, kElems, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.w[1], a.wu, 2, a.hidden, a.ffn, a.hidden, kElems, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.x[0], a.x, 2, a.hidden, a.tokens, a.ldx, kElems, nt, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return a.act == TIDE_ACT_SILU ? launch_tile<KIND, TIDE_ACT_SILU>(p, nt, l, stream)
                                : launch_tile<KIND, TIDE_ACT_GELU>(p, nt, l, stream);
}

}  // namespace

cudaError_t few_tc_prepare(TcDevice* dev) {
  cudaError_t (*const all[])(TcDevice*) = {prepare_tiles<kForward, TIDE_ACT_SILU>, prepare_tiles<kForward, TIDE_ACT_GELU>,
                                  prepare_tiles<kGrad, TIDE_ACT_SILU>,    prepare_tiles<kGrad, TIDE_ACT_GELU>,
                                  prepare_tiles<kFp8>,                    prepare_tiles<kDx>};
  for (auto p : all) {
    const cudaError_t e = p(dev);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Past 64 tokens the 256-row tiles read fewer operand bytes; they are ahead
// for the gated block from about half as many of these tiles as SMs (1021 x
// 2048 x 768, 96 tiles: 19.6 us, 11.8 there), for the 8-bit product from two
// thirds (128 x 28672 x 8192, 128 tiles: 87 us, 76 there).  Below that it goes
// by the stages of a CTA, in microseconds:
//                    here                     256-row tiles
//   gated            0.24 each and 3          0.265 and 4.3
//     split          0.3 and 6.2              0.265 and 7.6
//     checkpoint     4 more, by the split     1.1 more
//   8-bit            0.35 and 3               0.33 and 4
//     split          0.35 and 4.5             0.33 and 7
// (Gated, 420 x 10864 x 208: 14.0 here, 19.1 there; 123 x 7712 x 960 15.4 and
// 17.0; 110 x 11584 x 3104 34.4 and 34.2; 1162 x 12880 x 544 62.9 and 35.7.
// 8-bit, 420 x 208 x 10864: 8.8 and 15.2; 123 x 960 x 7712 8.8 and 11.7; 110
// x 3104 x 11584 21.6 and 15.3; 1162 x 544 x 12880 40.0 and 18.0.)  Clusters are
// the forward kernel's for its gradients too, which take the same shared memory
// and threads.
bool gated_few_takes(const GatedArgs& a, const TcLaunch& l) {
  if (a.tokens <= 64 || !few(a.tokens, a.ffn, l.dev->sms / 2)) return few(a.tokens, a.ffn, 0);
  const int64_t steps = ceil_div(a.hidden, kRowBytes / 2);
  const int split = split_of<kForward, 64, TIDE_ACT_SILU>(ceil_div(a.tokens, 64) * ceil_div(a.ffn, kRows), steps, *l.dev);
  const int there = gated_tc_split(a, *l.dev);
  const double here = split > 1 ? 0.3 * steps / split + 6.2 : 0.24 * steps + 3;
  return here + (a.g8 ? 4.0 / split : 0) <= 0.265 * steps / there + (there > 1 ? 7.6 : 4.3) + (a.g8 ? 1.1 : 0);
}
// dX up to 64 tokens, where it saves more than its own launch takes beside
// dW's: from 12 M weights on (a whole backward pass in a graph, here and in
// 256-row tiles: 1 x 4096 x 14336 122 and 130 us, 8 x 8192 x 1792 35.6 and
// 41.4, 37 x 2048 x 4096 25.0 and 24.7, 64 x 512 x 2048 18.5 and 16.5).  In
// microseconds dX takes 0.21 a stage and 3 more here, in 256-row tiles 0.3 and
// 4, or 8 where their sums are split (4 x 4096 x 14336: 37 against 54; 2 x 336 x
// 25264, where a cluster's 8 CTAs are too few: 23 against 19).
bool gated_dx_few_takes(const GatedArgs& a, const TcLaunch& l) {
  if (a.tokens > 64 || a.hidden * a.ffn < (12 << 20) || !few(a.tokens, a.hidden, 0)) return false;
  const int64_t steps = 2 * ceil_div(a.ffn, kRowBytes / 2), tiles = ceil_div(a.hidden, kRows);
  const int64_t large = ceil_div(a.hidden, 256);
  const int split = split_of<kDx, 64, 0>(tiles, steps, *l.dev);
  const int64_t parts = l.dev->pairs / large > 1 ? l.dev->pairs / large : 1;
  return 0.21 * steps / split + 3 <= 0.3 * steps / parts + (parts > 1 ? 8 : 4);
}

bool fp8_few_takes(const MatmulArgs& a, const TcLaunch& l) {
  if (a.m <= 64 || !few(a.m, a.n, 2 * l.dev->sms / 3)) return few(a.m, a.n, 0);
  const int64_t steps = ceil_div(a.k, kRowBytes);
  const int split = split_of<kFp8, 64, 0>(ceil_div(a.m, 64) * ceil_div(a.n, kRows), steps, *l.dev), there = fp8_tc_split(a, *l.dev);
  return 0.35 * steps / split + (split > 1 ? 4.5 : 3) <= 0.33 * steps / there + (there > 1 ? 7 : 4);
}

cudaError_t launch_gated_forward_few(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  p.g8 = a.g8, p.gs = a.gs, p.u8 = a.u8, p.us = a.us;
  return gated<kForward>(p, a, l, stream);
}

cudaError_t launch_gated_grad_few(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  Params p{};
  p.dh = a.dh, p.lddh = a.lddh, p.dg = a.dg, p.du = a.du;
  return gated<kGrad>(p, a, l, stream);
}

cudaError_t launch_gated_dx_few(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream) {
  constexpr int kElems = kRowBytes / 2;
  const int nt = tile_of(a.tokens);
  const uint16_t *w[2] = {a.wg, a.wu}, *d[2] = {a.dg, a.du};
  Params p{};
  p.tokens = (int)a.tokens, p.features = (int)a.hidden;
  p.half_steps = (int)ceil_div(a.ffn, kElems), p.steps = 2 * p.half_steps, p.step_elems = kElems;
  p.one_box = a.hidden % 64 == 0;
  p.out = a.dx, p.ldo = a.lddx;
  for (int i = 0; i < 2; ++i)
    if (!(p.one_box ? make_slab_map(&p.w[i], w[i], a.hidden, a.ffn, a.hidden, kElems)
                    : make_map(&p.w[i], w[i], 2, a.hidden, a.ffn, a.hidden, 64, kElems, CU_TENSOR_MAP_SWIZZLE_128B)) ||
        !make_map(&p.x[i], d[i], 2, a.ffn, a.tokens, a.ffn, kElems, nt, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  return launch_tile<kDx>(p, nt, l, stream);
}

cudaError_t launch_fp8_matmul_few(const MatmulArgs& a, const TcLaunch& l, cudaStream_t stream) {
  const int nt = tile_of(a.m);
  Params p{};
  p.tokens = (int)a.m, p.features = (int)a.n;
  p.steps = (int)ceil_div(a.k, kRowBytes), p.step_elems = kRowBytes;
  p.out = a.out, p.ldo = a.ldo;
  p.sx = a.sa, p.sw = a.sb, p.any_scales = a.any_scales;
  if (!make_map(&p.w[0], a.b, 1, a.k, a.n, a.k, kRowBytes, kRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&p.x[0], a.a, 1, a.k, a.m, a.k, kRowBytes, nt, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return launch_tile<kFp8>(p, nt, l, stream);
}

}  // namespace tide
