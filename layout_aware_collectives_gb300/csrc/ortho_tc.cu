// The products of Newton-Schulz orthogonalisation on the tensor cores, one
// persistent kernel in four forms:
//   gram    A = X X^T
//   sym     s2 L R + s1 L + s0 of two symmetric matrices that commute
//   update  the next X = L X
//   last    the same to the caller's matrices, in bf16
// What gram and sym make is symmetric: only tiles on and above the diagonal
// are summed, and written to both places.
//
// Update's and last's tiles are of X turned, X^T L (L is symmetric): the long
// side lies along a tile's 256 rows, and the short one along its columns, of
// which a tile may have 64.  With X as it is, a matrix of 33 rows left seven of
// eight warps without results (25 of 3582 x 33, in pairs of steps: 204 us, 153 turned;
// level where both sides are long).
//
// As in the gated block, a pair of CTAs works on one tile of 256 rows and 256
// columns (or 128 or 64, where there are few tiles): each loads 128 rows of the
// left operand and half of the right one's columns, one MMA instruction of the
// pair reads both halves.  Warps 0 and 3 load (5 stages of 32 KiB), warp 1 of the
// pair's first CTA issues the MMAs, warps from 4 on read finished sums out of
// TMEM, which holds two accumulators so that they do so while the next tile is
// summed.
//
// What those warps add to the sums (32 x 32 elements of two planes at a time)
// is copied to shared memory while the elements before are at work, and what
// they make of it goes out by way of the same place.  TMA does neither: each of
// its copies here would stand behind the operands' large ones.  The sums come
// out of TMEM as fragments, so that a piece is stored turned, for the tile's
// other place, by the same instructions.
//
// Bound by the tensor cores where sums are long: one 14336 x 4096, gram 148 us
// (1.72 PFLOP/s of the half that is summed), sym 50 (1.46: 136 tiles on 76
// pairs), update 288 (1.67).  By the way out where they are short, 3.3 us a tile
// of gram, 5.3 of sym, 8 of update: 128 of 768 x 2048, gram 139 us, sym 84,
// update 290, which is also 80% of what their bytes take.
#include <cmath>

#include "ortho.cuh"
#include "tc_device.cuh"
#include "tc_host.h"

namespace tide {
namespace {

using namespace tc;

constexpr int kStages = 5;
constexpr int kStep = 64;
constexpr int kHalf = 128;
constexpr uint32_t kOperand = kHalf * kStep * 2;
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kSlot = 2 * kBox;  // boxes of two planes
constexpr int kSlots = 2;             // of a warp
constexpr size_t kSmem = 1024 + kStages * kStage + kEpiWarps * kSlots * kSlot;

// One product, as the kernels take it.
struct Phase {
  int form;
  int left, right;          // maps of the operands
  int left_lo;              // and of X's lo, where a sum has two terms
  int term;                 // stages of a term
  const __half* in[2];      // planes that are added: sym: left, right; update, last: X, hi and lo
  __half* out[2];           // gram, sym: the one; update: the next X, hi and lo
  int64_t ld;               // of those
  int m, wide, steps;       // rows and columns of the result (update, last: of X turned), stages of a tile's sum
  int planes;               // of `in`
  int width;                // columns of a tile
  TileGrid grid;            // update, last
  Divisor each;             // gram, sym: tiles of a matrix
  Divisor segments;         // gram: sums of a matrix, a result each; in a chain 1
  int tiles;
  const float *left_d, *right_d;  // diagonals
  float* out_d;
  float s2, s1, s0;
  float rest;               // update, last: the factor of X's lo in rows whose diagonal is near it; 0: as of its hi
  float sum_scale, left_scale, right_scale, out_scale;  // factors of the sums, of `in`, of what is kept
  bool tall;
  int64_t ld_out;
};

// The operands that products have: left ones of gram, sym and update, right
// ones of the same; those of X's lo last.
enum Map { kLeftX = 0, kLeftT = 2, kWideX = 5, kRightX = 7, kRightT = 9, kUpdateT = 12, kWideLo = 14,
           kMaps = 16 };

struct Limits {
  int* err;
  uint64_t limit_ns, stall_ns, late_ns;
};

struct Params {  // of one product of all matrices
  CUtensorMap left, right, left_lo;
  Phase phase;
  int64_t first;  // matrix, of this launch
  Limits limits;
};

constexpr int kMaxPhases = 24;
struct ChainParams {  // of all products of each matrix
  CUtensorMap maps[kMaps];
  int used;  // of those
  Phase phase[kMaxPhases];
  int phases;
  int64_t first;
  Limits limits;
};

// The pairs that share a phase's tiles, which of them this is, and the first
// of their matrices.
struct Team {
  int pair, pairs;
  int z0;
  uint32_t rank;  // of this CTA in its pair
};

// A kernel of one form knows it; one of all forms looks it up (kAny) but for
// results' way out (one code for all of them there: 704 x 256 94 us instead of 87).
constexpr int kAny = -1;
template <int FORM>
__device__ __forceinline__ int form_of(const Phase& p) {
  return FORM == kAny ? p.form : FORM;
}

template <int FORM>
__device__ __forceinline__ bool work_at(const Phase& p, const Team& team, int i, TileAt& r) {
  const int t = team.pair + i * team.pairs;
  if (t >= p.tiles) return false;
  if (form_of<FORM>(p) >= kUpdate) {
    r = tile_at(p.grid, t);
  } else {
    // Down the columns: the tiles of rows up to the diagonal's.  One, two or
    // four columns of tiles end at the same row.
    const int turns = p.width == 256 ? 0 : p.width == 128 ? 1 : 2;  // 2^turns of them
    r.z = p.each.of(t);
    const int q = t - r.z * p.each.d;
    int n = (int)((__fsqrt_rn(8.0f * (float)(q >> turns) + 1.0f) - 1.0f) * 0.5f);
    while (((n * (n + 1) / 2) << turns) > q) --n;
    while ((((n + 1) * (n + 2) / 2) << turns) <= q) ++n;
    const int rest = q - ((n * (n + 1) / 2) << turns), high = n + 1;
    const int column = (rest >= high) + (rest >= 2 * high) + (rest >= 3 * high);  // of up to four
    r.n = (n << turns) + column, r.m = rest - column * high;
  }
  r.z += team.z0;
  return true;
}

// A warp's 32 x 32 elements of one plane in shared memory, 64-byte swizzle: 16-byte
// piece c of row r lies at piece c ^ (r / 2 % 4).
__device__ __forceinline__ uint32_t piece_at(uint32_t row, uint32_t piece) { return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }

// Where a lane's part of a box begins; the rest of it is constants further.
struct Places {
  uint32_t line;    // eight rows of four pieces at a time: row lane / 4, piece lane % 4
  uint32_t rows;    // 16 rows as fragments
  uint32_t turned;  // and turned
  __device__ __forceinline__ explicit Places(uint32_t lane)
      : line(piece_at(lane >> 2, lane & 3)),
        rows(piece_at(lane & 15, lane >> 4)),
        turned(piece_at((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1)) {}
};
// 16 rows of a box, the first or the second, as the tensor cores' fragments
// have them: register 2 g + h of a lane holds columns 8 g + 2 (lane % 4) and the
// next one of row 8 h + lane / 4.
__device__ __forceinline__ void get_rows(uint32_t box, const Places& at, int q, uint32_t (&v)[8]) {
#pragma unroll
  for (uint32_t g = 0; g < 4; g += 2)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[2 * g]), "=r"(v[2 * g + 1]), "=r"(v[2 * g + 2]), "=r"(v[2 * g + 3])
                 : "r"(box + (at.rows ^ (g << 4)) + q * 1024)
                 : "memory");
}
// Turned: column c of them is row c of the box.
__device__ __forceinline__ void get_turned(uint32_t box, const Places& at, int q, uint32_t (&v)[8]) {
#pragma unroll
  for (uint32_t g = 0; g < 4; g += 2)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[2 * g]), "=r"(v[2 * g + 1]), "=r"(v[2 * g + 2]), "=r"(v[2 * g + 3])
                 : "r"(box + (at.turned ^ (q << 5)) + g * 512)
                 : "memory");
}
template <bool TURNED>
__device__ __forceinline__ void get_box(uint32_t box, const Places& at, uint32_t (&v)[2][8]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if constexpr (TURNED)
      get_turned(box, at, q, v[q]);
    else
      get_rows(box, at, q, v[q]);
  }
}
__device__ __forceinline__ void put_rows(uint32_t box, const Places& at, int q, const uint32_t (&v)[8]) {
#pragma unroll
  for (uint32_t g = 0; g < 4; g += 2)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(box + (at.rows ^ (g << 4)) + q * 1024),
                 "r"(v[2 * g]), "r"(v[2 * g + 1]), "r"(v[2 * g + 2]), "r"(v[2 * g + 3])
                 : "memory");
}
__device__ __forceinline__ void put_turned(uint32_t box, const Places& at, int q, const uint32_t (&v)[8]) {
#pragma unroll
  for (uint32_t g = 0; g < 4; g += 2)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(box + (at.turned ^ (q << 5)) + g * 512),
                 "r"(v[2 * g]), "r"(v[2 * g + 1]), "r"(v[2 * g + 2]), "r"(v[2 * g + 3])
                 : "memory");
}
// 32 columns of 16 TMEM lanes, likewise: sums 4 g + 2 h and the next one.  They
// may be used after tmem_arrived.
__device__ __forceinline__ void tmem_rows(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : TIDE_R8(v, 0), TIDE_R8(v, 8)
      : "r"(addr)
      : "memory");
}

// A box of a plane, `from` and `to` being this lane's first piece.  Planes' rows
// are whole 64s wide, so a box has all its columns; `rows` of its rows are there.
__device__ __forceinline__ void ask_box(uint32_t box, const Places& at, const __half* from, int64_t ld8, int rows) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(box + at.line + q * 512),
                 "l"(q * 8 < rows ? from + q * ld8 : from), "r"(q * 8 < rows ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void asked() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void arrived() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}
template <class T>
__device__ __forceinline__ void send_box(uint32_t box, const Places& at, T* to, int64_t ld8, int rows) {
  uint4 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[q].x), "=r"(v[q].y), "=r"(v[q].z), "=r"(v[q].w)
                 : "r"(box + at.line + q * 512)
                 : "memory");
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q * 8 < rows) *(uint4*)(to + q * ld8) = v[q];
}

// A warp's way through its 32 x 32 pieces of the pair's tiles.
template <int FORM>
struct Cursor {
  int i;      // tile
  TileAt at;
  int row0, col, left;  // of the piece; pieces left in this tile, it among them
  int64_t mine;         // of a plane: this lane's first piece of the box
  bool more;

  // Rows of the box that are there, from this lane's first one on.
  __device__ __forceinline__ int rows(const Phase& p, int lane) const {
    return (form_of<FORM>(p) >= kUpdate ? p.wide - col : p.m - row0) - (lane >> 2);
  }

  // The i-th tile, or the next that has a piece for this warp.
  __device__ __forceinline__ void open(const Phase& p, const Team& team, int first, int half, int lanes, int lane) {
    const bool turned = form_of<FORM>(p) >= kUpdate;
    for (i = first;; ++i) {
      more = work_at<FORM>(p, team, i, at);
      if (!more) return;
      row0 = (at.m * 2 + (int)team.rank) * kHalf + lanes;
      col = at.n * p.width + half * (p.width / 2);
      left = row0 >= p.m || col >= p.wide ? 0 : min(p.width / 64, (p.wide - col + 31) / 32);
      // (update: X's rows are the result's columns)
      mine = ((int64_t)at.z * p.wide + (turned ? col : row0) + (lane >> 2)) * p.ld + (turned ? row0 : col) + (lane & 3) * 8;
      if (left) return;
    }
  }
  __device__ __forceinline__ void step(const Phase& p, const Team& team, int half, int lanes, int lane) {
    col += 32, mine += form_of<FORM>(p) >= kUpdate ? 32 * p.ld : 32;
    if (--left == 0) open(p, team, i + 1, half, lanes, lane);
  }
};

// 32 x 32 results to the caller: `rows` and `cols` of which there are.
__device__ __forceinline__ void send_last(uint32_t box, const Places& at, uint16_t* to, int64_t ld, int rows, int cols, int lane) {
  if (((uintptr_t)to & 15) == 0 && ld % 8 == 0 && cols >= 32) {
    send_box(box, at, to + (lane >> 2) * ld + (lane & 3) * 8, 8 * ld, rows - (lane >> 2));
    return;
  }
  to += lane;
  for (int r = 0; r < 32 && r < rows; r += 8, to += 8 * ld) {
    uint16_t v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v[q]) : "r"(box + piece_at(r + q, lane >> 3) + (lane & 7) * 2) : "memory");
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (r + q < rows && lane < cols) to[q * ld] = v[q];
  }
}

// Two 32-bit operations as one instruction.
__device__ __forceinline__ uint64_t two(uint32_t a, uint32_t b) { return (uint64_t)b << 32 | a; }
__device__ __forceinline__ uint64_t two(float a, float b) { return two(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ uint64_t two_halves(uint32_t v) {
  const float2 f = unpack_half(v);
  return two(f.x, f.y);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t muladd2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Diagonals' elements of a piece: left's of row row0 + lane, right's of column
// col + lane.
struct Diagonals {
  float di, dj;
};

// What becomes of 32 x 32 sums.
template <int FORM>
__device__ __forceinline__ void finish(const Phase& p, uint16_t* dst, const Cursor<FORM>& now, const Places& at, int lane,
                                       uint32_t tmem, uint32_t slot, Diagonals d) {
  const int form = form_of<FORM>(p);
  const TileAt& t = now.at;
  const int row0 = now.row0, col = now.col;
  uint32_t sums[2][16], a[2][8], b[2][8];
  tmem_rows(tmem, sums[0]);
  tmem_rows(tmem + (16u << 16), sums[1]);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[0][i] = a[1][i] = 0;
  constexpr bool kTurned = FORM >= kUpdate;
  if (form != kGram) get_box<kTurned>(slot, at, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) b[0][i] = a[0][i], b[1][i] = a[1][i];
  if (p.planes == 2) get_box<kTurned>(slot + kBox, at, b);
  // What is kept is scale * (s2 (sum + di right + left dj) + s1 left), or
  // scale * (sum + dj hi + dj or rest lo): each factor with its scales taken together.
  const float k0 = p.sum_scale * p.out_scale * p.s2;
  const uint64_t k2 = two(k0, k0);
  const float by_row = d.di * p.s2 * p.right_scale * p.out_scale;
  uint64_t by_col[4], by_lo[4];  // of the fragments' columns
  if (form != kGram) {
    const float own = fmaf(d.dj, p.s2, p.s1) * p.left_scale * p.out_scale;
#pragma unroll
    for (int g = 0; g < 4; ++g)
      by_col[g] = two(__shfl_sync(0xffffffffu, own, g * 8 + (lane & 3) * 2), __shfl_sync(0xffffffffu, own, g * 8 + (lane & 3) * 2 + 1));
    // (a row whose diagonal is far from L(0) lies in directions that do not grow)
    const float rest = p.rest * p.left_scale * p.out_scale, least = 0.75f * rest * rest;
    const auto lo_by = [&](uint32_t v) { return __uint_as_float(v) * rest > least ? rest : __uint_as_float(v); };
#pragma unroll
    for (int g = 0; g < 4; ++g) by_lo[g] = two(lo_by((uint32_t)by_col[g]), lo_by((uint32_t)(by_col[g] >> 32)));
  }
  const bool upper = form < kUpdate && t.n * p.width / (2 * kHalf) != t.m;  // above the diagonal's tiles
  tmem_arrived(sums[0]);
  tmem_arrived(sums[1]);
  __syncwarp();  // every lane has its part of the slot
  uint32_t hi[2][8], lo[2][8];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint64_t by[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float v = __shfl_sync(0xffffffffu, by_row, q * 16 + h * 8 + (lane >> 2));
      by[h] = two(v, v);
    }
    uint64_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = mul2(two(sums[q][2 * i], sums[q][2 * i + 1]), k2);
      if (FORM == kGram) continue;
      y[i] = muladd2(two_halves(a[q][i]), by_col[i >> 1], y[i]);
      y[i] = muladd2(two_halves(b[q][i]), form == kSym ? by[i & 1] : by_lo[i >> 1], y[i]);
    }
    if (form == kLast) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[q][i] = pack_bf16(__uint_as_float((uint32_t)y[i]), __uint_as_float((uint32_t)(y[i] >> 32)));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[q][i] = pack_half(__uint_as_float((uint32_t)y[i]), __uint_as_float((uint32_t)(y[i] >> 32)));
    }
    if (form == kUpdate) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t rest = muladd2(two_halves(hi[q][i]), two(-1.0f, -1.0f), y[i]);
        lo[q][i] = pack_half(__uint_as_float((uint32_t)rest), __uint_as_float((uint32_t)(rest >> 32)));
      }
    }
  }
  if (form < kUpdate && !upper && row0 == col) {
    // The diagonal's elements go to their own place, and 0 to the plane's: row
    // r and column c of a fragment meet where 8 g + 2 (lane % 4) + {0, 1} = r.
    const int off = (lane >> 2) - 2 * (lane & 3);
    float* diagonal = p.out_d + ((int64_t)t.z * p.wide + row0 + (lane >> 2));
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 2 * (2 * q + h) + h, r = q * 16 + h * 8 + (lane >> 2);
        float v = as_f(off ? sums[q][2 * i + 1] : sums[q][2 * i]) * p.sum_scale;
        const float dl = __shfl_sync(0xffffffffu, d.di, r), dr = __shfl_sync(0xffffffffu, d.dj, r);
        v = fmaf(p.s2, fmaf(dl, dr, v), fmaf(p.s1, dl, p.s0));
        if ((off == 0 || off == 1) && row0 + r < p.m) diagonal[q * 16 + h * 8] = v;
        hi[q][i] &= off == 0 ? 0xffff0000u : off == 1 ? 0xffffu : 0xffffffffu;
      }
  }
  if (form == kUpdate || (form == kLast && !p.tall)) {
    put_turned(slot, at, 0, hi[0]);
    put_turned(slot, at, 1, hi[1]);
  } else {
    put_rows(slot, at, 0, hi[0]);
    put_rows(slot, at, 1, hi[1]);
  }
  if (form == kUpdate) {
    put_turned(slot + kBox, at, 0, lo[0]);
    put_turned(slot + kBox, at, 1, lo[1]);
  }
  if (upper) {
    put_turned(slot + kBox, at, 0, hi[0]);
    put_turned(slot + kBox, at, 1, hi[1]);
  }
  __syncwarp();
  if (form == kLast) {
    if (p.tall)
      send_last(slot, at, dst + (int64_t)row0 * p.ld_out + col, p.ld_out, p.m - row0, p.wide - col, lane);
    else
      send_last(slot, at, dst + (int64_t)col * p.ld_out + row0, p.ld_out, p.wide - col, p.m - row0, lane);
  } else {
    const int64_t ld8 = 8 * p.ld;
    const int rows = now.rows(p, lane);
    send_box(slot, at, p.out[0] + now.mine, ld8, rows);
    if (form == kUpdate || upper) {
      const int64_t turned = ((int64_t)t.z * p.wide + col + (lane >> 2)) * p.ld + row0 + (lane & 3) * 8;
      send_box(slot + kBox, at, upper ? p.out[0] + turned : p.out[1] + now.mine, ld8, upper ? p.wide - col - (lane >> 2) : rows);
    }
  }
  __syncwarp();
}

// Barriers of a CTA.
struct Bars {
  uint32_t at;
  __device__ __forceinline__ uint32_t full(int s) const { return at + 8u * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return at + 8u * (kStages + s); }
  __device__ __forceinline__ uint32_t sums_full(int b) const { return at + 8u * (2 * kStages + b); }
  __device__ __forceinline__ uint32_t sums_empty(int b) const { return at + 8u * (2 * kStages + 2 + b); }
  __device__ __forceinline__ uint32_t spare() const { return at + 8u * (2 * kStages + 4); }
  __device__ __forceinline__ uint32_t silent() const { return at + 8u * (2 * kStages + 5); }
};
constexpr int kBars = 2 * kStages + 6;

// What every form's kernel begins with; returns TMEM's address.
__device__ __forceinline__ uint32_t set_up(const Bars& bars, int* stop, uint32_t* tmem_at, int warp) {
  if (threadIdx.x == 0) {
    *stop = 0;
    for (int s = 0; s < kStages; ++s) bar_init(bars.full(s), 1), bar_init(bars.empty(s), 1);
    for (int b = 0; b < 2; ++b) bar_init(bars.sums_full(b), 1), bar_init(bars.sums_empty(b), 2 * kEpiWarps);
    bar_init(bars.spare(), 1), bar_init(bars.silent(), 1);
    bar_init_fence();
  }
  if (warp == 2) tmem_alloc<2>(smem_addr(tmem_at), 512);
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  return *tmem_at;
}

// A phase's first tile, found ahead of it.
struct First {
  TileAt at;
  bool more;
};
__device__ __forceinline__ First first_of(const Phase& p, const Team& team) {
  First f;
  f.more = work_at<kAny>(p, team, 0, f.at);
  return f;
}

// One thread loads the left operand, another the right one.  j: stages
// filled so far.  `leader`: the pair's first CTA's rank in the cluster.
template <int FORM>
__device__ __forceinline__ bool load_phase(const Phase& p, const CUtensorMap* map, const CUtensorMap* map_lo, const Team& team,
                                           const First& first, bool left, uint32_t smem, const Bars& bars, uint32_t leader,
                                           const Watch& watch, int& j) {
  const bool a_mn = form_of<FORM>(p) >= kUpdate;  // the left operand's major
  const uint32_t leaders = peer_addr(bars.full(0), leader);
  const uint32_t bytes = 2 * kOperand + p.width * (kStep * 2);
  const bool expects = left && team.rank == 0;
  const int steps = p.steps;
  int s = j % kStages, parity = (j / kStages + 1) & 1;
  TileAt at = first.at;
  bool more = first.more;
  for (int next = 1; more; more = work_at<FORM>(p, team, next++, at)) {
    const int row = (at.m * 2 + team.rank) * kHalf, col = at.n * p.width + (int)team.rank * (p.width / 2);
    int z = at.z, from = 0;
    if (FORM == kGram) {
      z = p.segments.of(at.z);
      from = (at.z - z * p.segments.d) * p.term * kStep;
    }
    // X's lo before its hi: a sum loses of its own size with every product that is added
    const CUtensorMap* now = steps > p.term ? map_lo : map;
    for (int i = 0, k = 0; i < steps; ++i, ++j) {
      if (j >= kStages && !bar_wait(bars.empty(s), parity, watch)) return false;
      if (expects) bar_expect(bars.full(s), bytes);
      const uint32_t bar = leaders + 8u * s;
      const uint32_t a = smem + s * kStage, b = a + kOperand;
      if (!left)
        load_box3<true>(b, now, from + k * kStep, col, z, bar);
      else if (a_mn)
        load_box4(a, now, 0, k * kStep, row / 64, z, bar);
      else
        load_box3<true>(a, now, from + k * kStep, row, z, bar);
      if (++s == kStages) s = 0, parity ^= 1;
      if (++k == p.term) k = 0, now = map;
    }
  }
  return true;
}
// The MMAs' last arrivals reach this CTA while it is still there.  After a wait
// that ran out: both CTAs' copies in flight, with a limit again; the peer's
// memory stays until the cluster's last barrier.
__device__ __forceinline__ void load_end(bool go, const Team& team, const Bars& bars, const Watch& watch, int j) {
  for (int i = max(0, j - kStages); i < j && go; ++i) go = bar_wait(bars.empty(i % kStages), (i / kStages) & 1, watch);
  if (!go && team.rank == 0)
    for (int i = max(0, j - kStages); i < j; ++i) await(bars.full(i % kStages), (i / kStages) & 1, watch);
}

// j: stages used so far, done: tiles.  `ctas`: the pair's bits among the cluster's.
template <int FORM>
__device__ __forceinline__ bool mma_phase(const Phase& p, const Team& team, uint32_t smem, uint32_t tmem, const Bars& bars,
                                          uint16_t ctas, const Watch& watch, int& j, int& done) {
  const bool a_mn = form_of<FORM>(p) >= kUpdate;
  const uint32_t instr = instr_desc(0, a_mn, 0, 256, 0) | (uint32_t)(p.width >> 3) << 17;  // fp16 operands
  const uint32_t a_lbo = a_mn ? kOperand / 2 : 16, a_next = (a_mn ? 2048 : 32) >> 4;
  const int steps = p.steps;
  int s = j % kStages, parity = (j / kStages) & 1;
  TileAt at;
  for (int i = 0; work_at<FORM>(p, team, i, at); ++i, ++done) {
    const int b = done & 1;
    if (done >= 2 && !bar_wait<kPeer>(bars.sums_empty(b), (done / 2 + 1) & 1, watch)) return false;
    fence_after();
    for (int k = 0; k < steps; ++k, ++j) {
      if (!bar_wait(bars.full(s), parity, watch)) return false;
      fence_after();
      const uint32_t a = smem + s * kStage;
      const uint64_t da = operand_desc(a, a_lbo), db = operand_desc(a + kOperand, 16);
#pragma unroll
      for (int q = 0; q < kStep / 16; ++q)
        mma<2, false>(tmem + b * 256, da + q * a_next, db + q * (32 >> 4), instr, k > 0 || q > 0);
      mma_commit<2>(bars.empty(s), ctas);
      if (++s == kStages) s = 0, parity ^= 1;
    }
    mma_commit<2>(bars.sums_full(b), ctas);
  }
  return true;
}

template <int FORM>
__device__ __forceinline__ bool finish_phase(const Phase& p, const OrthoTargets& targets, const Team& team, int64_t first,
                                             uint32_t slots, uint32_t tmem, const Bars& bars, uint32_t leader, bool late,
                                             const Watch& watch, int warp, int lane, int& done) {
  const int half = warp >> 2, lanes = (warp & 3) * 32;
  // Pieces in turn, slot by slot; `next` is the one whose copies go out.
  const int form = form_of<FORM>(p);
  const bool in = form != kGram;
  const Places places(lane);
  Cursor<FORM> now, next;
  now.open(p, team, 0, half, lanes, lane);
  next = now;
  int slot = 0;  // of the piece at hand, and of the next to be asked for
  // of the piece at hand and the next: moved on, not chosen by slot, so that
  // nothing waits for the last one's
  static_assert(kSlots == 2, "two pieces on their way");
  Diagonals here{0.0f, 0.0f}, then{0.0f, 0.0f};
  const auto ask = [&](int to) {
    here = then;
    if (in && next.more) {
      const int64_t z = (int64_t)next.at.z * p.wide;
      if (form == kSym) then.di = next.row0 + lane < p.m ? __ldcg(p.left_d + z + next.row0 + lane) : 0.0f;
      then.dj = next.col + lane < p.wide ? __ldcg(p.right_d + z + next.col + lane) : 0.0f;
      const int rows = next.rows(p, lane);
      // (a lane without a row of its own names the piece's first)
      const int64_t from = rows > 0 ? next.mine : next.mine - (int64_t)(lane >> 2) * p.ld;
      ask_box(slots + to * kSlot, places, p.in[0] + from, 8 * p.ld, rows);
      if (p.planes == 2) ask_box(slots + to * kSlot + kBox, places, p.in[1] + from, 8 * p.ld, rows);
      next.step(p, team, half, lanes, lane);
    }
    if (in) asked();  // an empty group past the last, so that their number says which have arrived
  };
  for (int s = 0; s < kSlots; ++s) ask(s);
  TileAt at;
  bool go = true;
  // every tile's sums are waited for and handed back, a piece of it here or not
  for (int i = 0; work_at<FORM>(p, team, i, at); ++i, ++done) {
    const int b = done & 1;
    go = bar_wait_warp(late ? bars.silent() : bars.sums_full(b), (done / 2) & 1, watch);
    if (!go) break;
    fence_after();
    while (now.more && now.i == i) {
      if (in) arrived<kSlots - 1>();
      finish<FORM>(p, form == kLast ? targets.p[at.z - first] : nullptr, now, places, lane,
                   tmem + ((uint32_t)lanes << 16) + b * 256 + (now.col - at.n * p.width), slots + slot * kSlot, here);
      ask(slot);
      slot ^= 1;
      now.step(p, team, half, lanes, lane);
    }
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive_peer(peer_addr(bars.sums_empty(b), leader));
  }
  if (in) arrived<0>();
  return go;
}

// One product of all matrices, its tiles over all pairs.
template <int FORM>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ OrthoTargets targets) {
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bar_words[kBars];
  __shared__ uint32_t tmem_at;
  __shared__ int stop;
  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const Bars bars{smem_addr(bar_words)};
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Team team{(int)blockIdx.x / 2, (int)gridDim.x / 2, (int)p.first, cluster_rank()};
  const Watch watch{&stop, p.limits.err, p.limits.limit_ns};
  const bool late = p.limits.late_ns && warp == 4;  // test: this warp waits for sums where nothing arrives
  if (threadIdx.x == 0) prefetch_map(&p.left), prefetch_map(&p.right);
  if (threadIdx.x == 0 && p.phase.term < p.phase.steps) prefetch_map(&p.left_lo);
  const uint32_t tmem = set_up(bars, &stop, &tmem_at, warp);
  after_previous();

  int j = 0, done = 0;
  if (p.limits.stall_ns) {  // test: a wait on a barrier nothing arrives on runs out
    if (threadIdx.x == 0) bar_wait(bars.silent(), 0, Watch{&stop, p.limits.err, p.limits.stall_ns});
  } else if (warp == 0 || warp == 3) {
    if (elected()) {
      const bool left = warp == 0;
      const bool go = load_phase<FORM>(p.phase, left ? &p.left : &p.right, left ? &p.left_lo : &p.right, team,
                                       first_of(p.phase, team), left, smem, bars, 0, watch, j);
      load_end(go, team, bars, watch, j);
    }
  } else if (warp == 1 && team.rank == 0) {
    if (elected()) {
      mma_phase<FORM>(p.phase, team, smem, tmem, bars, 3, watch, j, done);
      mma_commit<2>(bars.spare(), 1);
    }
  } else if (warp >= 4) {
    finish_phase<FORM>(p.phase, targets, team, p.first, smem + kStages * kStage + (warp - 4) * kSlots * kSlot, tmem, bars, 0, late,
                       Watch{&stop, p.limits.err, late ? p.limits.late_ns : p.limits.limit_ns}, warp - 4, lane, done);
  }
  __syncthreads();
  if (stop && warp == 1 && team.rank == 0 && !p.limits.stall_ns) {
    await(bars.spare(), 0, watch);  // the MMAs in flight
    __syncwarp();
  }
  cluster_sync();
  if (warp == 2) tmem_free<2>(tmem, 512);
}

// All products of one matrix by a cluster of one to eight pairs, which meet
// between two products: what a launch, its set-up and its last tiles cost is
// paid once, and a matrix's planes stay in L2 from one product to the next.
__global__ void __launch_bounds__(kThreads, 1)
    ortho_chain_kernel(const __grid_constant__ ChainParams p, const __grid_constant__ OrthoTargets targets) {
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bar_words[kBars];
  __shared__ uint32_t tmem_at;
  __shared__ int stop, ended_at;  // the phase that a wait ran out in
  __shared__ Phase at_hand[2];    // and the next one, which has time to come
  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const Bars bars{smem_addr(bar_words)};
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t cta = cluster_rank(), leader = cta & ~1u;
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint16_t both = (uint16_t)(3u << leader);
  const Team team{(int)cta / 2, (int)ctas / 2, (int)(p.first + blockIdx.x / ctas), cta & 1};
  const Watch watch{&stop, p.limits.err, p.limits.limit_ns};
  const bool late = p.limits.late_ns && warp == 4;
  const Watch sums_watch{&stop, p.limits.err, late ? p.limits.late_ns : p.limits.limit_ns};
  const uint32_t slots = smem + kStages * kStage + (warp - 4) * kSlots * kSlot;
  const auto fetch = [&](int n, int from, int by) {
    static_assert(sizeof(Phase) % 4 == 0, "copied by words");
    for (int i = from; i < (int)(sizeof(Phase) / 4); i += by) ((uint32_t*)&at_hand[n & 1])[i] = ((const uint32_t*)&p.phase[n])[i];
  };
  if (threadIdx.x == 0) ended_at = INT32_MAX;
  fetch(0, threadIdx.x, kThreads);
  if (threadIdx.x < p.used) prefetch_map(&p.maps[threadIdx.x]);
  const uint32_t tmem = set_up(bars, &stop, &tmem_at, warp);
  after_previous();

  int j = 0, done = 0;
  bool go = true, ended = false;
  First first{};
  if (warp == 0 || warp == 3) first = first_of(p.phase[0], team);
  if (p.limits.stall_ns && threadIdx.x == 0) bar_wait(bars.silent(), 0, Watch{&stop, p.limits.err, p.limits.stall_ns});
  const int phases = p.limits.stall_ns ? 0 : p.phases;
  for (int n = 0; n < phases; ++n) {
    const Phase& f = at_hand[n & 1];
    if (warp == 2 && n + 1 < phases) fetch(n + 1, lane, 32);
    if (warp == 0 || warp == 3) {
      if (elected()) {
        const bool left = warp == 0;
        go = load_phase<kAny>(f, &p.maps[left ? f.left : f.right], &p.maps[left ? f.left_lo : f.right], team, first, left, smem,
                              bars, leader, watch, j);
        if (!go || n == phases - 1)
          load_end(go, team, bars, watch, j);
        else
          first = first_of(p.phase[n + 1], team);
      }
    } else if (warp == 1 && team.rank == 0) {
      if (elected()) go = mma_phase<kAny>(f, team, smem, tmem, bars, both, watch, j, done);
    } else if (warp >= 4) {
      if (f.form == kGram)
        finish_phase<kGram>(f, targets, team, p.first, slots, tmem, bars, leader, late, sums_watch, warp - 4, lane, done);
      else if (f.form == kSym)
        finish_phase<kSym>(f, targets, team, p.first, slots, tmem, bars, leader, late, sums_watch, warp - 4, lane, done);
      else if (f.form == kUpdate)
        finish_phase<kUpdate>(f, targets, team, p.first, slots, tmem, bars, leader, late, sums_watch, warp - 4, lane, done);
      else
        finish_phase<kLast>(f, targets, team, p.first, slots, tmem, bars, leader, late, sums_watch, warp - 4, lane, done);
      publish();  // these results, to others' reads and copies of them
    }
    __syncthreads();
    // A wait that ran out ends all of the cluster at this phase: who tells the
    // others does so before they meet, and one that is a phase ahead names its own.
    if (stop && threadIdx.x < ctas) peer_write(peer_addr(smem_addr(&ended_at), threadIdx.x), n);
    if (stop) publish();
    cluster_meet();
    ended = *(volatile int*)&ended_at <= n;
    if (ended) break;
  }
  if (ended) {  // copies and MMAs in flight
    if (warp == 0 || warp == 3) {
      if (elected() && go) load_end(false, team, bars, watch, j);
    } else if (warp == 1 && team.rank == 0) {
      if (elected()) mma_commit<2>(bars.spare(), (uint16_t)(1u << leader));
      __syncwarp();
      await(bars.spare(), 0, watch);
    }
  }
  __syncwarp();
  cluster_sync();
  if (warp == 2) tmem_free<2>(tmem, 512);
}

// Columns of the tiles of each form.
struct Widths {
  int gram, sym, update;
  int of(int form) const { return form == kGram ? gram : form == kSym ? sym : update; }
};

bool map_of(CUtensorMap* map, int which, const OrthoPlan& p, const Widths& w) {
  const auto k = [&](const __half* plane, int64_t cols, int64_t ld, int rows) {
    return make_stack_map(map, plane, cols, p.m, p.count, ld, kStep, rows, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (which < kLeftT) return k(p.x[which - kLeftX][0], p.n, p.ld_x, kHalf);
  if (which < kWideX) return k(p.t[which - kLeftT], p.m, p.ld_a, kHalf);
  if (which < kRightX) return make_slab_stack_map(map, p.x[which - kWideX][0], p.m, p.count, p.ld_x, kStep, kHalf / 64);
  if (which < kRightT) return k(p.x[which - kRightX][0], p.n, p.ld_x, w.gram / 2);
  if (which < kUpdateT) return k(p.t[which - kRightT], p.m, p.ld_a, w.sym / 2);
  if (which < kWideLo) return k(p.t[which - kUpdateT], p.m, p.ld_a, w.update / 2);
  return make_slab_stack_map(map, p.x[which - kWideLo][1], p.m, p.count, p.ld_x, kStep, kHalf / 64);
}

Limits limits_of(const TcLaunch& l) { return Limits{l.err, TIDE_BULK_TIMEOUT_NS, l.stall_ns, l.late_ns}; }

// Tiles on and above the diagonal of [m, m].
int64_t triangle(int64_t m, int64_t width) {
  const int64_t across = 2 * kHalf / width, columns = ceil_div(m, width), whole = columns / across, rest = columns % across;
  return across * (whole * (whole + 1) / 2) + rest * (whole + 1);
}

// A product, but for how many tiles there are.
Phase phase_of(const OrthoPlan& p, const OrthoProduct& q, const Widths& w, int64_t ld_dst) {
  Phase k{};
  const bool update = q.form >= kUpdate;
  k.width = w.of(q.form);
  k.form = q.form;
  k.left = q.form == kGram ? kLeftX + q.turn : q.form == kSym ? kLeftT + q.left : kWideX + q.turn;
  k.right = q.form == kGram ? kRightX + q.turn : (update ? kUpdateT : kRightT) + q.right;
  k.m = update ? p.n : p.m, k.wide = p.m;
  const bool parted = q.form == kGram && p.segments > 1;
  k.steps = (int)ceil_div(parted ? kOrthoSegment : q.form == kGram ? p.n : p.m, kStep);
  k.segments = Divisor(parted ? p.segments : 1);
  k.term = k.steps;
  if (update) k.steps *= p.x_terms;
  k.left_lo = update && p.x_terms > 1 ? kWideLo + q.turn : k.left;
  k.rest = q.rest;
  k.planes = q.form == kGram ? 0 : q.form == kSym && q.left == q.right ? 1 : 2;
  k.in[0] = update ? p.x[q.turn][0] : p.t[q.left], k.in[1] = update ? p.x[q.turn][1] : p.t[q.right];
  k.out[0] = update ? p.x[q.turn ^ 1][0] : parted ? p.part_t : p.t[q.out], k.out[1] = p.x[q.turn ^ 1][1];
  k.ld = update ? p.ld_x : p.ld_a;
  k.left_d = p.d[q.left], k.right_d = p.d[q.right], k.out_d = parted ? p.part_d : p.d[q.out];
  k.s2 = q.s2, k.s1 = q.s1, k.s0 = q.s0;
  k.sum_scale = 1.0f / (q.left_scale * q.right_scale);
  k.left_scale = 1.0f / q.left_scale, k.right_scale = 1.0f / q.right_scale;
  k.out_scale = q.form == kLast ? 1.0f : q.out_scale;
  k.tall = p.tall, k.ld_out = ld_dst;
  if (update)
    k.grid = TileGrid((int)ceil_div(p.n, 2 * kHalf), (int)ceil_div(p.m, k.width));
  else
    k.each = Divisor((int)triangle(p.m, k.width));
  return k;
}
int64_t tiles_of(const Phase& k) { return k.form >= kUpdate ? k.grid.all.d : k.each.d; }

cudaError_t launch_product(const OrthoPlan& p, const OrthoProduct& q, const Widths& w, const OrthoArgs& a, const TcLaunch& l,
                           cudaStream_t stream) {
  Params k{};
  OrthoTargets targets{};
  k.phase = phase_of(p, q, w, a.ld_dst);
  k.limits = limits_of(l);
  if (!map_of(&k.left, k.phase.left, p, w) || !map_of(&k.right, k.phase.right, p, w)) return cudaErrorInvalidValue;
  if (k.phase.term < k.phase.steps && !map_of(&k.left_lo, k.phase.left_lo, p, w)) return cudaErrorInvalidValue;
  // as many matrices (or segments) as a launch counts tiles, and the last form's table holds
  const int64_t each = tiles_of(k.phase);
  int64_t most = INT32_MAX / 2 / each;
  if (most < 1) return cudaErrorInvalidValue;
  if (q.form == kLast && most > kOrthoTable) most = kOrthoTable;
  const int64_t count = p.count * k.phase.segments.d;
  for (k.first = 0; k.first < count; k.first += most) {
    const int64_t some = count - k.first < most ? count - k.first : most;
    k.phase.tiles = (int)(some * each);
    if (q.form == kLast)
      for (int64_t i = 0; i < some; ++i) targets.p[i] = a.dst[k.first + i];
    const int pairs = k.phase.tiles < l.dev->pairs ? k.phase.tiles : l.dev->pairs;
    const auto kernel = q.form == kGram     ? ortho_tc_kernel<kGram>
                        : q.form == kSym    ? ortho_tc_kernel<kSym>
                        : q.form == kUpdate ? ortho_tc_kernel<kUpdate>
                                            : ortho_tc_kernel<kLast>;
    const cudaError_t e = launch_early(kernel, dim3(2 * pairs), kThreads, kSmem, 2, stream, k, targets);
    if (e != cudaSuccess) return e;
  }
  return k.phase.segments.d > 1 ? launch_ortho_join(p, q.out, stream) : cudaSuccess;
}

cudaError_t launch_chain(const OrthoPlan& p, const OrthoProduct* q, int products, const Widths& w, int pairs, const OrthoArgs& a,
                         const TcLaunch& l, cudaStream_t stream) {
  ChainParams k{};
  OrthoTargets targets{};
  k.phases = products;
  k.limits = limits_of(l);
  for (int i = 0; i < products; ++i) {
    k.phase[i] = phase_of(p, q[i], w, a.ld_dst);
    k.phase[i].tiles = (int)tiles_of(k.phase[i]);
  }
  k.used = p.x_terms > 1 ? kMaps : kWideLo;
  for (int i = 0; i < k.used; ++i)
    if (!map_of(&k.maps[i], i, p, w)) return cudaErrorInvalidValue;
  for (k.first = 0; k.first < p.count; k.first += kOrthoTable) {
    const int64_t some = p.count - k.first < kOrthoTable ? p.count - k.first : kOrthoTable;
    for (int64_t i = 0; i < some; ++i) targets.p[i] = a.dst[k.first + i];
    const cudaError_t e = launch_early(ortho_chain_kernel, dim3((unsigned)(2 * pairs * some)), kThreads, kSmem, 2 * pairs, stream, k, targets);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// How a call's products are shared out.
struct Way {
  int pairs;  // of a cluster for each matrix; 0: every product by all pairs
  Widths widths;
};

// By the time it takes, in stages of 256 columns (0.27 us): a tile's sum or its
// results' way out, whichever is longer, as one hides behind the other but for the
// last; and what a product costs besides, in a chain or alone, where half of the
// device's SMs is free for the next one's CTAs to set up or is not.  Measured, in
// us (all pairs; one, two, three, four, six, eight pairs a matrix): 704 x 256 83;
// 174, 116, 97, 92, 77, 76.  128 x 2048 97; 218, 144, 128, 111, 110, 94.  64 of 256 x
// 704 229; 205, 255, 306, 456, 595, 726.  16 of 300 x 300 127; 224, 137, 111, 187,
// 150, 218.  100 of 128 x 512 165; 190, 208, 329, 406, 732, 840.  512 x 768 109; 377,
// 251, 180, 175, 122, 122.
constexpr double kMeet = 12, kLaunch = 16, kLaunchFull = 18;
double way_out(int width) { return 4.4 + width / 22.0; }
double product_time(int64_t tiles, int64_t pairs, int steps, int width) {
  const double sum = steps * (width == 256 ? 1.0 : width == 128 ? 0.65 : 0.55), out = way_out(width);
  return (double)ceil_div(tiles, pairs) * std::fmax(sum, out) + std::fmin((double)steps, out);
}

Way way_of(const OrthoPlan& p, const OrthoProduct* q, int products, const TcDevice& dev) {
  int number[3] = {};  // of products: gram, sym, update and last
  for (int i = 0; i < products; ++i) ++number[q[i].form == kGram ? 0 : q[i].form == kSym ? 1 : 2];
  const int64_t down = ceil_div(p.n, 2 * kHalf);
  const int long_steps = (int)ceil_div(p.n < kOrthoSegment ? p.n : kOrthoSegment, kStep), short_steps = (int)ceil_div(p.m, kStep);
  // the widths that take the least time with so many pairs for so many matrices
  const auto best_of = [&](int64_t matrices, int64_t pairs, bool chain, Widths* w) {
    double least[3] = {};
    for (int width = 64; width <= 256; width *= 2) {
      int* const at[3] = {&w->gram, &w->sym, &w->update};
      for (int f = 0; f < 3; ++f) {
        const int64_t tiles = matrices * (f < 2 ? triangle(p.m, width) : down * ceil_div(p.m, width)) * (f == 0 ? p.segments : 1);
        const double t = product_time(tiles, pairs, f == 0 ? long_steps : f == 1 ? short_steps : short_steps * p.x_terms, width) +
                         (chain ? kMeet : 2 * tiles > pairs ? kLaunchFull : kLaunch);
        if (width == 64 || t <= least[f]) least[f] = t, *at[f] = width;
      }
    }
    return number[0] * least[0] + number[1] * least[1] + number[2] * least[2];
  };
  Way best{};
  double least = best_of(p.count, dev.pairs, false, &best.widths);
  for (int pairs = 1; pairs <= kMaxTeam && products <= kMaxPhases && p.segments == 1; ++pairs) {
    const int held = pairs == 1 ? dev.pairs : dev.ortho[pairs];
    if (held < 1) continue;
    Way way{pairs, {}};
    const double all = (double)ceil_div(p.count, held) * best_of(1, pairs, true, &way.widths) + kLaunch;
    if (all < least) least = all, best = way;
  }
  return best;
}

}  // namespace

cudaError_t ortho_prepare(TcDevice* dev) {
  void (*const kernels[])(Params, OrthoTargets) = {ortho_tc_kernel<kGram>, ortho_tc_kernel<kSym>, ortho_tc_kernel<kUpdate>,
                                                   ortho_tc_kernel<kLast>};
  for (auto k : kernels) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = cudaFuncSetAttribute(ortho_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(ortho_chain_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e != cudaSuccess ? e : held_clusters((const void*)ortho_chain_kernel, kThreads, kSmem, kMaxTeam, dev->ortho);
}

cudaError_t launch_ortho_products(const OrthoPlan& p, const OrthoProduct* q, int products, const OrthoArgs& a, const TcLaunch& l,
                                  cudaStream_t stream) {
  const Way way = way_of(p, q, products, *l.dev);
  if (way.pairs) return launch_chain(p, q, products, way.widths, way.pairs, a, l, stream);
  for (int i = 0; i < products; ++i) {
    const cudaError_t e = launch_product(p, q[i], way.widths, a, l, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tide
