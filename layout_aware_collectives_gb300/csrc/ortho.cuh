// Newton-Schulz orthogonalisation: what its kernels share.
//
// One step takes X [m, n], m <= n (the matrix, or its transpose where it has
// more rows), to C X, C = a + b A + c A A, A = X X^T.  Where m is large two steps
// may share one pass over X: the second's A is C A C, and X becomes C' C X.
//
// X is kept as two fp16 terms (hi + lo: 22 bits) of a power-of-two scale, the
// symmetric matrices as one, all but their diagonals, which are kept in fp32
// beside them.  The products take hi alone.  What its rounding leaves would be
// 0.002-0.003 of the result, as much as the result's own rounding to bf16 or
// twice that, were it not for the diagonals: near the end A is close to the
// identity, and the diagonals carry most of a product.  With L = D + P, P's
// diagonal 0,
//   L L' = P P' + D P' + P D' + D D',   L X = P X + D X,
// and the tensor cores see the first terms only.
//
// Next to a low rank that is not enough: small singular values grow by a in every
// step, by 485 in five, and with them whatever a step leaves in their directions.
// There L is L(0), its value at A = 0 (a, or a a' of two steps), while D is less
// by some 1 / m of what L takes from the large ones: P lo, which the products pass
// over, has the difference, and so left 0.02 of the result of 8 rows, 0.01 of 33,
// 0.005 of 128, for a floor of noise below rank one.  So while later steps may still
// stretch things by more than 8, lo is multiplied by L(0): what that leaves, (L -
// L(0)) lo, lies in directions with large singular values, which do not grow.  In
// the last steps all are near 1, and lo is multiplied by D, which is nearer to L
// on average, as it is in rows whose diagonal is below 3/4 of L(0): such a row lies
// in directions that do not grow.  Short sides of up to 64 have lo in the product
// itself, a second term of its sums, which are a stage long.
//
// What all this leaves, in 2^-9 of the result's norm (rounding it to bf16 leaves
// 0.85 of that), the largest of noise, noise of 1e-1 to 1e-5 over rank one, spectra
// of e^-4 to e^-14 and columns of very different sizes:
//   17 x 40  33 x 2500  64 x 200  128 x 1000  256 x 704  512 x 1024, steps apart
//   0.6      0.4        0.4       0.4         0.4        0.35
//   (7.9     5.0        2.6       2.1         1.2        1.0, in pairs, lo by D)
//   384 x 1024  768 x 2048, in pairs
//   1.1         0.95
// Pairs leave more, as A's rounding passes through C on both sides, a a of it; the
// more rows, the less.  Of 200,000 matrices made to be hard, two or three levels of
// singular values left up to 2.1 (in pairs 3.4).  Where a few elements make up a
// matrix, roundings average out over nothing: permutations with up to 5.4, a dozen
// elements with up to 7.8, A's diagonal itself being off by 2^-11.
#pragma once

#include <cuda_fp16.h>

#include "compute_device.cuh"

namespace tide {

enum OrthoForm { kGram = 0, kSym = 1, kUpdate = 2, kLast = 3 };

// Columns of X that one of gram's sums takes.  The tensor cores' fp32 sums lose
// some 2^-24 of themselves with every 16 products that are added, always downwards:
// 3.7e-4 of A after 65536 columns, 1.5e-3 after four times as many, 8.5e-2 after
// 2^24.  Longer rows are summed in segments of as many, each to a plane of its
// own, which are added up afterwards.
constexpr int64_t kOrthoSegment = 65536;

// Short sides of up to so many rows take no tensor cores, but 32-bit arithmetic
// throughout (ortho.cu).
constexpr int kShortSide = 16;

constexpr int kOrthoTable = 128;  // matrices of a launch that goes by the caller's pointers

// The workspace's parts.
struct OrthoPlan {
  int m, n;
  int64_t count, ld_x, ld_a;  // row strides: whole 128-byte lines
  bool tall;
  __half* x[2][2];  // of two turns: hi, lo [count, m, ld_x]
  __half* t[3];     // symmetric matrices without their diagonals [count, m, ld_a]
  float* d[3];      // the diagonals [count, m]
  int x_terms;      // of update's and last's sums: 1, or 2 with X's lo
  int segments;     // of gram's sums; where there is more than one:
  __half* part_t;   // [count, segments, m, ld_a]
  float* part_d;    // [count, segments, m]
  // short sides: X [count, m, ld_x], and A's parts of two turns [count, spans,
  // m (m + 1) / 2]
  float* short_x;
  double* short_a[2];
  int spans, span;  // of X's columns, 64 at a time: so many a span
  double* norms;    // parts of the sums of squares [count, parts]
  int parts;
};

// One product of every matrix.  A plane holds values times its scale.
struct OrthoProduct {
  OrthoForm form;
  int turn;            // which X is read
  int left, right;     // kSym: t's; kUpdate, kLast: X turned, times the right t
  int out;             // kGram, kSym: a t
  float s2, s1, s0;    // kSym: s2 (left right) + s1 left + s0
  float left_scale, right_scale, out_scale;
  float rest;  // kUpdate, kLast: the factor of X's lo; 0: the right t's diagonal
};

// The caller's matrices of one launch.
struct OrthoTargets {
  uint16_t* p[kOrthoTable];
};

// A from its segments (ortho.cu).
cudaError_t launch_ortho_join(const OrthoPlan& p, int out, cudaStream_t stream);

// The products in order (ortho_tc.cu); the last form's results go to the
// caller's matrices.
cudaError_t launch_ortho_products(const OrthoPlan& p, const OrthoProduct* q, int products, const OrthoArgs& a,
                                  const TcLaunch& l, cudaStream_t stream);

__device__ __forceinline__ float2 unpack_half(uint32_t v) { return __half22float2(*(const __half2*)&v); }

// Two floats as packed fp16, to nearest even: `a` in the low half.
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *(const uint32_t*)&h;
}

// Two floats as two fp16 terms each, to nearest even: `a` in the low halves.
__device__ __forceinline__ void split_half2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *(const uint32_t*)&h, lo = *(const uint32_t*)&l;
}

}  // namespace tide
