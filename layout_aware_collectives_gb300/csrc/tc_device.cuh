// Device helpers of the tensor-core kernels: mbarriers with bounded waits,
// tensor-map copies, and the 5th-generation tensor-core instructions with
// their shared-memory and instruction descriptors.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "tc_host.h"

namespace tide {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Address in CTA `rank`'s shared memory of what has this address here.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ float4 peer_read(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One thread of a converged warp, for the copies and the MMAs: what it issues
// behind `lane == 0` instead takes longer (dX of 7 tokens, 2048 x 8192: 24.1 us
// against 18.7).  The warp's index comes from a shuffle for the same reason.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.b32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}

// ---------------------------------------------------------------- mbarriers

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrives on a barrier of another CTA of the cluster (a peer_addr).  It tells
// of reads and writes of TMEM, which have completed (tcgen05.wait) and which
// fence_before and the waiting thread's fence_after put in order around the
// barrier: between those it has to order execution in the cluster, and no
// memory.  (A release at cluster scope waits for a memory barrier every time:
// 4096 x 8192 x 28672 8-bit product 1445 us instead of 530.)
__device__ __forceinline__ void bar_arrive_peer(uint32_t peer_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_bar) : "memory");
}
// What a wait orders: memory of this CTA; execution in the cluster, where a
// peer's bar_arrive_peer is waited for; or, for copies and those, both.
enum Order { kOwn, kPeer, kOwnAndPeer };
template <Order O = kOwn>
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
#define TIDE_TRY_WAIT(order)                                                                                          \
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity." order ".shared::cta.b64 p, [%1], %2; selp.b32 %0, 1, 0, p; }" \
               : "=r"(ok)                                                                                             \
               : "r"(bar), "r"(parity)                                                                                \
               : "memory")
  if constexpr (O == kOwn) TIDE_TRY_WAIT("acquire.cta");
  if constexpr (O == kPeer) TIDE_TRY_WAIT("relaxed.cluster");
  if constexpr (O == kOwnAndPeer) TIDE_TRY_WAIT("acquire.cluster");
#undef TIDE_TRY_WAIT
  return ok != 0;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// What a wait that runs out does: the handle's error word is set and every
// role of this CTA leaves its loop.
struct Watch {
  volatile int* stop;   // shared
  int* err;             // host-visible
  uint64_t limit_ns;
};

template <Order O>
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, const Watch& w) {
  const uint64_t t0 = now_ns();
  while (!bar_try<O>(bar, parity)) {
    if (*w.stop) return false;
    if (now_ns() - t0 > w.limit_ns) {
      *w.stop = 1;
      *(volatile int*)w.err = kDevErrTimeout;
      return false;
    }
  }
  return true;
}
template <Order O = kOwn>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Watch& w) {
  return bar_try<O>(bar, parity) || bar_wait_slow<O>(bar, parity, w);
}
// The same for a whole warp, which leaves together.
__device__ __forceinline__ bool bar_wait_warp(uint32_t bar, uint32_t parity, const Watch& w) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, w));
}

// What is in flight after a wait ran out: copies, or MMAs (whose issuing thread
// ends with a commit on a spare barrier).  Every role has left, so `stop` is
// set, and a CTA frees TMEM and ends only behind these.  Where no wait ran out
// the last sums were waited for, and with them all of it.
__device__ __forceinline__ void await(uint32_t bar, uint32_t parity, const Watch& w) {
  int never = 0;
  bar_wait(bar, parity, Watch{&never, w.err, w.limit_ns / 16});
}

// ------------------------------------------------------- tensor-map copies

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// A box of a 2-D tensor into this CTA's shared memory.  PAIR: `bar` may be
// the pair's leader's barrier (a peer_addr).
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// The same of a 3-D tensor.
template <bool PAIR>
__device__ __forceinline__ void load_box3(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// A box of shared memory to a 2-D tensor, clipped at its end.
__device__ __forceinline__ void store_box(const CUtensorMap* m, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m), "r"(x),
               "r"(y), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void stores_read() {  // all but the last N groups have been read from shared memory
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------ tensor cores

template <int GROUP>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t columns) {
  if constexpr (GROUP == 2)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns) : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns) : "memory");
}
template <int GROUP>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
  if constexpr (GROUP == 2) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns));
  } else {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns));
  }
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory descriptor of an operand tile with 128-byte swizzle (8 rows
// of 128 bytes repeat).  K-major: a row is 64 (bf16) or 128 (8-bit) steps of
// the contraction, SBO = 1024 steps 8 rows on.  MN-major: a row is 64 rows or
// columns of the operand, SBO steps 8 of the contraction on and LBO 64 rows
// or columns on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo) {
  constexpr uint32_t kSbo = 1024;
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(kSbo >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor: fp32 sums, A and B of type `ab` (bf16: 1 in
// kind::f16; e4m3: 0 in kind::f8f6f4), majors 1 = MN.
constexpr uint32_t instr_desc(uint32_t ab, uint32_t a_mn, uint32_t b_mn, uint32_t m, uint32_t n) {
  return (1u << 4) | (ab << 7) | (ab << 10) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

constexpr uint32_t instr_desc_a_mn = 1u << 15;  // A's major, where it is known at run time

// D (+)= A B for one step of the contraction (32 bytes of it).
template <int GROUP, bool FP8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  const uint32_t p = add ? 1u : 0u;
#define TIDE_MMA(group, kind)                                                                               \
  asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::" group ".kind::" kind       \
               " [%0], %1, %2, %3, p; }" ::"r"(d),                                                          \
               "l"(a), "l"(b), "r"(idesc), "r"(p)                                                           \
               : "memory")
  if constexpr (GROUP == 2 && FP8) TIDE_MMA("2", "f8f6f4");
  if constexpr (GROUP == 2 && !FP8) TIDE_MMA("2", "f16");
  if constexpr (GROUP == 1 && FP8) TIDE_MMA("1", "f8f6f4");
  if constexpr (GROUP == 1 && !FP8) TIDE_MMA("1", "f16");
#undef TIDE_MMA
}

// Instruction descriptor of the block-scaled 8-bit form: e4m3 operands, both
// K-major, scales that are powers of two (E8M0).
constexpr uint32_t instr_desc_scaled(uint32_t m, uint32_t n) { return ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24); }

// D (+)= (A * scales) (B * scales) for 32 steps of the contraction by a pair.
// A's scale of row r lies in column r / 32 of sa, lane r % 32 of each of the
// four groups of 32 lanes, and B's alike; a scale for 32 steps is one byte of
// that column's word.
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                           bool add) {
  const uint32_t p = add ? 1u : 0u;
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %6, 0;\n tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(p)
      : "memory");
}

// Four or eight columns of this warp's TMEM lanes, one lane a thread.
__device__ __forceinline__ void tmem_write4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_written() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrives on `bar` (at this address in both CTAs of a pair, `ctas` being
// their bits among the cluster's) once the MMAs issued so far have completed.
template <int GROUP>
__device__ __forceinline__ void mma_commit(uint32_t bar, uint16_t ctas = 3) {
  if constexpr (GROUP == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(ctas)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

#define TIDE_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                      "=r"(v[i + 6]), "=r"(v[i + 7])
#define TIDE_R32(v) TIDE_R8(v, 0), TIDE_R8(v, 8), TIDE_R8(v, 16), TIDE_R8(v, 24)

// 32 (or 16) columns of this warp's 32 TMEM lanes, one lane a thread; waits for them.
__device__ __forceinline__ void tmem_read(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : TIDE_R32(v)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_read(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : TIDE_R8(v, 0), TIDE_R8(v, 8)
      : "r"(addr)
      : "memory");
}
// The same without the wait: `v` may be used after tmem_arrived(v).
__device__ __forceinline__ void tmem_issue32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : TIDE_R32(v)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_issue16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : TIDE_R8(v, 0), TIDE_R8(v, 8)
      : "r"(addr)
      : "memory");
}
#define TIDE_RW8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), \
                       "+r"(v[i + 6]), "+r"(v[i + 7])
#define TIDE_RW32(v) TIDE_RW8(v, 0), TIDE_RW8(v, 8), TIDE_RW8(v, 16), TIDE_RW8(v, 24)
// Waits for every read issued so far; no use of v moves ahead of it.
__device__ __forceinline__ void tmem_arrived(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : TIDE_RW8(v, 0), TIDE_RW8(v, 8)::"memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : TIDE_RW32(v)::"memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&v)[32], uint32_t (&w)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : TIDE_RW32(v), TIDE_RW32(w)::"memory");
}

// The same for two runs of 32 columns.
__device__ __forceinline__ void tmem_read32x2(uint32_t a0, uint32_t a1, uint32_t (&v)[32], uint32_t (&w)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
      "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : TIDE_R32(v), TIDE_R32(w)
      : "r"(a0), "r"(a1)
      : "memory");
}

struct TileAt {
  int z, m, n;  // which of several products; tile indices
};

// No division: with few stages a tile they were a quarter of its time.
__device__ __forceinline__ TileAt tile_at(const TileGrid& g, int t) {
  TileAt r;
  r.z = g.all.of(t);
  t -= r.z * g.all.d;
  const int band = g.band.of(t), first = band * kBand;
  t -= band * g.band.d;
  if (first + kBand <= g.tiles_m) {
    r.n = t / kBand;
    r.m = first + t % kBand;
  } else {
    r.n = g.last.of(t);
    r.m = first + t - r.n * g.last.d;
  }
  return r;
}

__device__ __forceinline__ float as_f(uint32_t v) { return __uint_as_float(v); }

// Results on their way out: 32 x 32 boxes of one warp, a ring of BOXES.
constexpr uint32_t kBox = 32 * 32 * 2;  // 32 rows of 32 bf16

template <int BOXES>
struct Outbox {
  uint32_t base;
  int next;
  int lane;

  // 64-byte swizzle: 16-byte piece c of row r lies at piece c ^ (r / 2 % 4)
  __device__ __forceinline__ uint32_t fill(const uint32_t (&p)[16]) {
    const uint32_t box = base + (uint32_t)(next % BOXES) * kBox;
    ++next;
    const uint32_t row_at = box + lane * 64, turn = (lane >> 1) & 3;
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_at + ((c ^ turn) << 4)), "r"(p[4 * c]),
                   "r"(p[4 * c + 1]), "r"(p[4 * c + 2]), "r"(p[4 * c + 3])
                   : "memory");
    return box;
  }

  __device__ __forceinline__ void put(const CUtensorMap* map, const uint32_t (&p)[16], int col, int row) {
    if (lane == 0) stores_read<BOXES - 1>();
    __syncwarp();
    const uint32_t box = fill(p);
    async_fence();
    __syncwarp();
    if (lane == 0) store_box(map, col, row, box);
  }
  // Two at once, behind one fence, the second only if `two`.
  __device__ __forceinline__ void put2(const CUtensorMap* map0, const uint32_t (&p0)[16], int col0, const CUtensorMap* map1,
                                       const uint32_t (&p1)[16], int col1, int row, bool two = true) {
    if (lane == 0) stores_read<BOXES - 2>();
    __syncwarp();
    const uint32_t box0 = fill(p0);
    uint32_t box1 = 0;
    if (two) box1 = fill(p1);
    async_fence();
    __syncwarp();
    if (lane == 0) {
      store_box(map0, col0, row, box0);
      if (two) store_box(map1, col1, row, box1);
    }
  }
};

// A pair's sums of its part of a contraction, on their way to the cluster's
// other pairs: 128 rows of 256 fp32 a CTA, where its stages were (their
// products have completed).  16-byte piece c of row r lies at c ^ (r % 8).
constexpr uint32_t kSumRow = 256 * 4;

// Four of the eight chunks of 32 columns, from this warp's 32 TMEM lanes.
__device__ __forceinline__ void leave_sums(uint32_t smem, uint32_t tmem, int row, int first) {
  const uint32_t to = smem + row * kSumRow, turn = row & 7;
#pragma unroll 1
  for (uint32_t c = first; c < first + 4; ++c) {
    uint32_t v[32];
    tmem_read(tmem + c * 32, v);
#pragma unroll
    for (uint32_t q = 0; q < 8; ++q)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((c * 8 + q) ^ turn) << 4)), "r"(v[4 * q]),
                   "r"(v[4 * q + 1]), "r"(v[4 * q + 2]), "r"(v[4 * q + 3])
                   : "memory");
  }
}

// The whole contraction's sums of row `row` and columns lane * 4 on, and 128
// columns further, in the parts' order.  rank: in the pair.
__device__ __forceinline__ void split_sums(uint32_t smem, int row, int lane, uint32_t rank, int split, float4 (&sum)[2]) {
  const uint32_t from = smem + row * kSumRow + ((lane ^ (row & 7)) << 4);
  float4 v[kMaxSplit][2];
#pragma unroll
  for (int q = 0; q < kMaxSplit; ++q)
    if (q < split) {
      const uint32_t a = peer_addr(from, 2 * q + rank);
      v[q][0] = peer_read(a), v[q][1] = peer_read(a + kSumRow / 2);
    }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    sum[c] = v[0][c];
#pragma unroll
    for (int q = 1; q < kMaxSplit; ++q)
      if (q < split) sum[c].x += v[q][c].x, sum[c].y += v[q][c].y, sum[c].z += v[q][c].z, sum[c].w += v[q][c].w;
  }
}

}  // namespace tc
}  // namespace tide
