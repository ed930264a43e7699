// The products of Newton-Schulz orthogonalisation on the tensor cores, one
// persistent kernel in four forms:
//   gram    A = X X^T, kept as O and its diagonal
//   square  B = b A + c A A from O O, kept as P and its diagonal
//   update  the next X = (a + E) X + P X
//   last    the same to the caller's matrices, in bf16
// A and B are symmetric: only tiles on and above the diagonal are summed, and
// written to both places.
//
// As in the gated block, a pair of CTAs works on one 256 x 256 tile: each
// loads 128 rows of the left operand and half of the right one's columns, one
// MMA instruction of the pair reads both halves.  Warps 0 and 3 load (6 stages
// of 32 KiB), warp 1 of the pair's first CTA issues the MMAs, warps from 4 on
// read finished sums out of TMEM, which holds two accumulators so that they do
// so while the next tile is summed.
#include "ortho.cuh"
#include "tc_device.cuh"
#include "tc_host.h"

namespace tide {
namespace {

using namespace tc;

constexpr int kStages = 6;
constexpr int kStep = 64;
constexpr int kHalf = 128;
constexpr uint32_t kOperand = kHalf * kStep * 2;
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kAllBoxes = 16;
constexpr size_t kSmem = 1024 + kStages * kStage + kAllBoxes * kBox;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kBoxes = kAllBoxes / kEpiWarps;

struct Params {
  CUtensorMap left, right;  // operands
  CUtensorMap out[2];       // gram: O, update: the next X, hi and lo; square: P
  int m, wide, steps;       // rows and columns of the result, stages of a tile's sum
  TileGrid grid;            // update, last
  Divisor each;             // gram, square: tiles of a matrix
  int tiles;
  int64_t first;            // matrix, of this launch
  const __half *hi, *lo;    // square: O, update: X
  int64_t ld;               // of those
  float *d, *e;             // diagonals of A and B
  float a, b, c;
  float sum_scale, in_scale, out_scale;  // factors of the sums, of hi and lo, of what is kept
  bool tall;
  int64_t ld_out;
  int* err;
  uint64_t limit_ns, stall_ns, late_ns;
};

template <int FORM>
__device__ __forceinline__ bool work_at(const Params& p, int pair, int pairs, int i, TileAt& r) {
  const int t = pair + i * pairs;
  if (t >= p.tiles) return false;
  if constexpr (FORM == kUpdate || FORM == kLast) {
    r = tile_at(p.grid, t);
  } else {
    // down the columns of the triangle m <= n
    r.z = p.each.of(t);
    const int q = t - r.z * p.each.d;
    int n = (int)((sqrtf(8.0f * (float)q + 1.0f) - 1.0f) * 0.5f);
    while (n * (n + 1) / 2 > q) --n;
    while ((n + 1) * (n + 2) / 2 <= q) ++n;
    r.n = n, r.m = q - n * (n + 1) / 2;
  }
  r.z += (int)p.first;
  return true;
}

// Two floats to packed fp16, to nearest even: `lo` in the low half.
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ float2 unpack_half(uint32_t v) { return __half22float2(*(const __half2*)&v); }

// Results on their way out: 32 x 32 boxes of one warp, as they are or turned.
struct Boxes : Outbox<kBoxes> {
  // 64-byte swizzle, as in fill(): row c of the box is column c of the sums
  __device__ __forceinline__ uint32_t fill_turned(const uint32_t (&p)[16]) {
    const uint32_t box = base + (uint32_t)(next % kBoxes) * kBox;
    ++next;
    const uint32_t piece = lane >> 3, at = box + (lane & 7) * 2;
#pragma unroll
    for (uint32_t c = 0; c < 32; ++c)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + c * 64 + ((piece ^ ((c >> 1) & 3)) << 4)),
                   "h"((uint16_t)(p[c / 2] >> (16 * (c & 1))))
                   : "memory");
    return box;
  }
  template <bool TURNED>
  __device__ __forceinline__ void put(const CUtensorMap* m0, const uint32_t (&p0)[16], const CUtensorMap* m1,
                                      const uint32_t (&p1)[16], int col, int row, int z) {
    if (lane == 0) stores_read<kBoxes - 2>();
    __syncwarp();
    const uint32_t b0 = TURNED ? fill_turned(p0) : fill(p0);
    uint32_t b1 = 0;
    if (m1) b1 = TURNED ? fill_turned(p1) : fill(p1);
    async_fence();
    __syncwarp();
    if (lane == 0) {
      store_box3(m0, TURNED ? row : col, TURNED ? col : row, z, b0);
      if (m1) store_box3(m1, TURNED ? row : col, TURNED ? col : row, z, b1);
    }
  }
};

// hi and lo of 32 neighbours.
__device__ __forceinline__ void load_terms(const Params& p, int64_t at, bool in, uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 h = in ? *(const uint4*)(p.hi + at + 8 * q) : zero, l = in ? *(const uint4*)(p.lo + at + 8 * q) : zero;
    hi[4 * q] = h.x, hi[4 * q + 1] = h.y, hi[4 * q + 2] = h.z, hi[4 * q + 3] = h.w;
    lo[4 * q] = l.x, lo[4 * q + 1] = l.y, lo[4 * q + 2] = l.z, lo[4 * q + 3] = l.w;
  }
}
__device__ __forceinline__ float2 both_terms(uint32_t hi, uint32_t lo, float scale) {
  const float2 h = unpack_half(hi), l = unpack_half(lo);
  return make_float2((h.x + l.x) * scale, (h.y + l.y) * scale);
}

// 32 columns of the last result's row: one lane a row.
__device__ __forceinline__ void put_last(const Params& p, uint16_t* dst, const float (&y)[32], int row0, int col, Boxes& out) {
  const int lane = out.lane, row = row0 + lane;
  if (p.tall) {  // a column's rows lie together, and so do the lanes
    if (row >= p.m) return;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col + i < p.wide) dst[(int64_t)(col + i) * p.ld_out + row] = to_bf16(y[i]);
    return;
  }
  uint32_t o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
  if (((uintptr_t)dst & 15) == 0 && p.ld_out % 8 == 0 && col + 32 <= p.wide) {
    if (row >= p.m) return;
    uint4* to = (uint4*)(dst + (int64_t)row * p.ld_out + col);
#pragma unroll
    for (int q = 0; q < 4; ++q) to[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    return;
  }
  // rows that do not start on 16 bytes: a row at a time, an element a lane
  __syncwarp();
  const uint32_t box = out.fill(o);
  __syncwarp();
  for (int r = 0; r < 32 && row0 + r < p.m; ++r) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];"
                 : "=h"(v)
                 : "r"(box + r * 64 + ((((uint32_t)lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2));
    if (col + lane < p.wide) dst[(int64_t)(row0 + r) * p.ld_out + col + lane] = v;
  }
}

// A warp's 32 rows and 128 columns of a tile.
template <int FORM>
__device__ __forceinline__ void epilogue(const Params& p, const OrthoTargets& targets, const TileAt& t, uint32_t tmem, int row0,
                                         int half, Boxes& out) {
  const int lane = out.lane, row = row0 + lane;
  const bool mine = row < p.m;
  if (row0 >= p.m) return;
  const int64_t at = (int64_t)t.z * p.m + row;
  float di = 0.0f;  // square: A's diagonal here, update: a + B's
  if (FORM == kSquare && mine) di = p.d[at];
  if (FORM >= kUpdate && mine) di = p.a + p.e[at];
#pragma unroll 1
  for (int c = half * 4; c < half * 4 + 4; ++c) {
    const int col = t.n * 2 * kHalf + c * 32;
    if (col >= p.wide) break;
    uint32_t hi[16], lo[16], v[32];
    if constexpr (FORM != kGram) load_terms(p, at * p.ld + col, mine, hi, lo);
    float dj = 0.0f;
    if (FORM == kSquare && col + lane < p.wide) dj = p.d[(int64_t)t.z * p.m + col + lane];
    tmem_read(tmem + c * 32, v);
    float y[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) y[i] = as_f(v[i]) * p.sum_scale;
    if constexpr (FORM == kSquare) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 o = both_terms(hi[i], lo[i], p.in_scale);
        const float d0 = __shfl_sync(0xffffffffu, dj, 2 * i), d1 = __shfl_sync(0xffffffffu, dj, 2 * i + 1);
        // A A = O O + D O + O D + D D
        y[2 * i] = fmaf(p.c, fmaf(di + d0, o.x, y[2 * i]), p.b * o.x);
        y[2 * i + 1] = fmaf(p.c, fmaf(di + d1, o.y, y[2 * i + 1]), p.b * o.y);
      }
    }
    if constexpr (FORM == kGram || FORM == kSquare) {
      if (t.m == t.n && (row0 >> 5) == (col >> 5)) {  // the diagonal's box
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i == lane) {
            if (mine) (FORM == kGram ? p.d : p.e)[at] = FORM == kGram ? y[i] : y[i] + di * fmaf(p.c, di, p.b);
            y[i] = 0.0f;
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 x = both_terms(hi[i], lo[i], p.in_scale);
        y[2 * i] = fmaf(di, x.x, y[2 * i]);
        y[2 * i + 1] = fmaf(di, x.y, y[2 * i + 1]);
      }
    }
    if constexpr (FORM == kLast) {
      put_last(p, targets.p[t.z - p.first], y, row0, col, out);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float y0 = y[2 * i] * p.out_scale, y1 = y[2 * i + 1] * p.out_scale;
        hi[i] = pack_half(y0, y1);
        const float2 h = unpack_half(hi[i]);
        lo[i] = pack_half(y0 - h.x, y1 - h.y);
      }
      const CUtensorMap* second = FORM == kSquare ? nullptr : &p.out[1];
      out.put<false>(&p.out[0], hi, second, lo, col, row0, t.z);
      if (FORM != kUpdate && t.m != t.n) out.put<true>(&p.out[0], hi, second, lo, col, row0, t.z);
    }
  }
}

template <int FORM>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ OrthoTargets targets) {
  constexpr bool kBMn = FORM == kUpdate || FORM == kLast;
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
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const Watch watch{&stop, p.err, p.limit_ns};
  const bool late = p.late_ns && warp == 4;  // test: this warp waits for sums where nothing arrives
  const Watch sums_watch{&stop, p.err, late ? p.late_ns : p.limit_ns};

  if (threadIdx.x == 0) {
    stop = 0;
    for (int s = 0; s < kStages; ++s) bar_init(full(s), 1), bar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(sums_full(b), 1), bar_init(sums_empty(b), 2 * kEpiWarps);
    bar_init(spare, 1), bar_init(silent, 1);
    bar_init_fence();
    prefetch_map(&p.left), prefetch_map(&p.right);
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
    // One thread loads the left operand, another the right one.
    if (elected()) {
      const bool left = warp == 0;
      int j = 0;  // stages filled so far
      bool go = true;
      TileAt at;
      for (int i = 0; go && work_at<FORM>(p, pair, pairs, i, at); ++i) {
        const int row = (at.m * 2 + rank) * kHalf, col = (at.n * 2 + rank) * kHalf;
        for (int k = 0; k < p.steps; ++k, ++j) {
          const int s = j % kStages;
          if (j >= kStages && !bar_wait(empty(s), (j / kStages + 1) & 1, watch)) {
            go = false;
            break;
          }
          if (left && rank == 0) bar_expect(full(s), 2 * kStage);
          const uint32_t bar = peer_addr(full(s), 0);
          const uint32_t a = smem + s * kStage, b = a + kOperand;
          if (left)
            load_box3<true>(a, &p.left, k * kStep, row, at.z, bar);
          else if (kBMn)
            load_box4(b, &p.right, 0, k * kStep, col / 64, at.z, bar);
          else
            load_box3<true>(b, &p.right, k * kStep, col, at.z, bar);
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
      constexpr uint32_t kInstr = instr_desc(0, 0, kBMn, 256, 256);  // fp16 operands
      int j = 0;  // stages used
      bool go = true;
      TileAt at;
      for (int i = 0; go && work_at<FORM>(p, pair, pairs, i, at); ++i) {
        const int b = i & 1;
        if (i >= 2 && !bar_wait<kPeer>(sums_empty(b), (i / 2 + 1) & 1, watch)) break;
        fence_after();
        for (int k = 0; k < p.steps; ++k, ++j) {
          const int s = j % kStages;
          if (!bar_wait(full(s), (j / kStages) & 1, watch)) {
            go = false;
            break;
          }
          fence_after();
          const uint32_t a = smem + s * kStage;
          const uint64_t da = operand_desc(a, 16), db = operand_desc(a + kOperand, kBMn ? kOperand / 2 : 16);
#pragma unroll
          for (int q = 0; q < kStep / 16; ++q)
            mma<2, false>(tmem + b * 256, da + q * (32 >> 4), db + q * ((kBMn ? 2048 : 32) >> 4), kInstr, k > 0 || q > 0);
          mma_commit<2>(empty(s));
        }
        if (go) mma_commit<2>(sums_full(b));
      }
      mma_commit<2>(spare, 1);
    }
  } else if (warp >= 4) {
    Boxes out;
    out.base = smem + kStages * kStage + (warp - 4) * kBoxes * kBox, out.next = 0, out.lane = lane;
    TileAt at;
    for (int i = 0; work_at<FORM>(p, pair, pairs, i, at); ++i) {
      const int b = i & 1;
      if (!bar_wait_warp(late ? silent : sums_full(b), (i / 2) & 1, sums_watch)) break;
      fence_after();
      const uint32_t lanes = (uint32_t)(warp & 3) * 32;
      epilogue<FORM>(p, targets, at, tmem + (lanes << 16) + b * 256, (at.m * 2 + rank) * kHalf + lanes, (warp - 4) >> 2, out);
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_peer(peer_addr(sums_empty(b), 0));
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

template <int FORM>
cudaError_t launch(Params& p, const OrthoTargets& targets, const TcLaunch& l, cudaStream_t stream) {
  p.err = l.err;
  p.limit_ns = TIDE_BULK_TIMEOUT_NS;
  p.stall_ns = l.stall_ns, p.late_ns = l.late_ns;
  const int pairs = p.tiles < l.dev->pairs ? p.tiles : l.dev->pairs;
  return launch_early(ortho_tc_kernel<FORM>, dim3(2 * pairs), kThreads, kSmem, 2, stream, p, targets);
}

bool map_k(CUtensorMap* map, const __half* plane, int64_t cols, const OrthoPlan& p, int64_t ld) {
  return make_stack_map(map, plane, cols, p.m, p.count, ld, kStep, kHalf, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_out(CUtensorMap* map, const __half* plane, int64_t cols, const OrthoPlan& p, int64_t ld) {
  return make_stack_map(map, plane, cols, p.m, p.count, ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace

cudaError_t ortho_prepare(TcDevice*) {
  void (*const kernels[])(Params, OrthoTargets) = {ortho_tc_kernel<kGram>, ortho_tc_kernel<kSquare>, ortho_tc_kernel<kUpdate>,
                                                   ortho_tc_kernel<kLast>};
  for (auto k : kernels) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_ortho_product(OrthoForm form, const OrthoPlan& p, const OrthoStep& s, int turn, const OrthoArgs& a,
                                 const TcLaunch& l, cudaStream_t stream) {
  Params k{};
  OrthoTargets targets{};
  const __half *const *x = p.x[turn], *const *next = p.x[turn ^ 1];
  const bool update = form >= kUpdate;
  const int64_t down = ceil_div(p.m, 2 * kHalf), across = ceil_div(p.n, 2 * kHalf);
  k.m = p.m, k.wide = update ? p.n : p.m;
  k.d = p.d, k.e = p.e;
  k.a = s.a, k.b = s.b, k.c = s.c;
  k.tall = p.tall, k.ld_out = a.ld_dst;
  bool ok = true;
  if (form == kGram) {
    k.steps = (int)ceil_div(p.n, kStep);
    k.sum_scale = 1.0f / (s.x_scale * s.x_scale), k.out_scale = s.a_scale;
    ok = map_k(&k.left, x[0], p.n, p, p.ld_x) && map_out(&k.out[0], p.o[0], p.m, p, p.ld_a) &&
         map_out(&k.out[1], p.o[1], p.m, p, p.ld_a);
    k.right = k.left;
  } else if (form == kSquare) {
    k.steps = (int)ceil_div(p.m, kStep);
    k.hi = p.o[0], k.lo = p.o[1], k.ld = p.ld_a;
    k.sum_scale = 1.0f / (s.a_scale * s.a_scale), k.in_scale = 1.0f / s.a_scale, k.out_scale = s.b_scale;
    ok = map_k(&k.left, p.o[0], p.m, p, p.ld_a) && map_out(&k.out[0], p.p, p.m, p, p.ld_a);
    k.right = k.left;
  } else {
    k.steps = (int)ceil_div(p.m, kStep);
    k.hi = x[0], k.lo = x[1], k.ld = p.ld_x;
    k.sum_scale = 1.0f / (s.b_scale * s.x_scale), k.in_scale = 1.0f / s.x_scale, k.out_scale = s.next_scale;
    ok = map_k(&k.left, p.p, p.m, p, p.ld_a) && make_slab_stack_map(&k.right, x[0], p.m, p.count, p.ld_x, kStep);
    if (form == kUpdate)
      ok = ok && map_out(&k.out[0], next[0], p.n, p, p.ld_x) && map_out(&k.out[1], next[1], p.n, p, p.ld_x);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int64_t each = update ? down * across : down * (down + 1) / 2;
  if (each > INT32_MAX) return cudaErrorInvalidValue;
  // as many matrices as a launch counts tiles, and the last form's table holds
  int64_t most = INT32_MAX / 2 / each;
  if (most < 1) most = 1;
  if (form == kLast && most > kOrthoTable) most = kOrthoTable;
  for (k.first = 0; k.first < p.count; k.first += most) {
    const int64_t some = p.count - k.first < most ? p.count - k.first : most;
    k.tiles = (int)(some * each);
    if (update)
      k.grid = TileGrid((int)down, (int)across);
    else
      k.each = Divisor((int)each);
    if (form == kLast)
      for (int64_t i = 0; i < some; ++i) targets.p[i] = a.dst[k.first + i];
    const cudaError_t e = form == kGram     ? launch<kGram>(k, targets, l, stream)
                          : form == kSquare ? launch<kSquare>(k, targets, l, stream)
                          : form == kUpdate ? launch<kUpdate>(k, targets, l, stream)
                                            : launch<kLast>(k, targets, l, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tide
