// Newton-Schulz orthogonalisation: what its kernels share.
//
// One step takes X [m, n], m <= n (the matrix, or its transpose where it has
// more rows), to a X + B X, B = b A + c A A, A = X X^T.  X and A are kept as
// two fp16 terms (hi + lo: 22 bits) of power-of-two scales; the products take
// hi alone.  What its rounding leaves would be 0.002-0.003 of the result, as
// much as the result's own rounding to bf16 or twice that, were it not for
// the diagonals: near the end A is close to the identity and its diagonal,
// and B's, carry most of a product.  So they are kept apart in fp32:
//   A A = O O + D O + O D + D D   with A = O + D, O's diagonal 0,
//   B X = P X + E X               with B = P + E, likewise,
// and the products see O and P only.  That leaves 0.0002-0.0007.
#pragma once

#include <cuda_fp16.h>

#include "compute_device.cuh"

namespace tide {

enum OrthoForm { kGram = 0, kSquare = 1, kUpdate = 2, kLast = 3 };

constexpr int kOrthoTable = 128;  // matrices of a launch that goes by the caller's pointers

// The workspace's parts, and a step's scales: a plane holds values times its
// scale.
struct OrthoPlan {
  int m, n;
  int64_t count, ld_x, ld_a;  // row strides: whole 128-byte lines
  bool tall;
  __half *x[2][2];  // of two turns: hi, lo [count, m, ld_x]
  __half *o[2];     // A without its diagonal: hi, lo [count, m, ld_a]
  __half *p;        // B without its diagonal: hi [count, m, ld_a]
  float *d, *e;     // their diagonals [count, m]
  double *norms;    // parts of the sums of squares [count, parts]
  int parts;
};

struct OrthoStep {
  float a, b, c;
  float x_scale, a_scale, b_scale, next_scale;  // of X, A, B and the next X
};

// The caller's matrices of one launch.
struct OrthoTargets {
  uint16_t* p[kOrthoTable];
};

// One product of every matrix (ortho_tc.cu): X by turn, the last step's result
// to the caller's matrices.
cudaError_t launch_ortho_product(OrthoForm form, const OrthoPlan& p, const OrthoStep& s, int turn, const OrthoArgs& a,
                                 const TcLaunch& l, cudaStream_t stream);

// v as two fp16 terms.
__device__ __forceinline__ void split_half(float v, __half& hi, __half& lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}

}  // namespace tide
