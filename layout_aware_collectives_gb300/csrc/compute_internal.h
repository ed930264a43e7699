// Internal interface between the feed-forward unit's C ABI (compute_api.cpp)
// and its kernels (gated_tc.cu, few_tc.cu, fp8_tc.cu, fp8_blocks.cu,
// gated_simple.cu).
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

#include <mutex>

#include "tide.h"
#include "tide_internal.h"

namespace tide {

constexpr int kBlock = 128;  // columns (and, for weights, rows) that share one scale

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A bf16 matrix [rows, cols] beside its 8-bit blocks.  ld is the bf16
// matrix's row stride in elements; codes are contiguous.
struct Fp8Args {
  int64_t rows, cols, ld;
  uint16_t* bf16;  // read by the store, written by the restore
  uint8_t* codes;
  float* scales;  // [ceil(rows / block_rows), ceil(cols / 128)]
  int block_rows;  // 1 or 128
};

// One call of the gated block, forward or backward.  Null pointers leave an
// output out.
struct GatedArgs {
  int64_t tokens, hidden, ffn;
  int act;
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* wg;
  const uint16_t* wu;
  uint16_t* h;
  int64_t ldh;
  uint8_t* g8;  // checkpoint of the two pre-activations
  float* gs;
  uint8_t* u8;
  float* us;
  // backward
  const uint16_t* dh;
  int64_t lddh;
  uint16_t* dx;
  int64_t lddx;
  uint16_t* dwg;
  uint16_t* dwu;
  uint16_t* dg;  // [tokens, ffn] each, workspace; bf16, the operands of dX's and dW's products
  uint16_t* du;
  float *dx_parts, *dw_parts;  // of dX's and dW's sums, workspace
  int64_t dx_parts_bytes, dw_parts_bytes;
};

struct MatmulArgs {
  int64_t m, n, k;
  const uint8_t* a;
  const float* sa;
  const uint8_t* b;
  const float* sb;
  uint16_t* out;
  int64_t ldo;
  bool any_scales;  // else powers of two
};

// Bytes <-> blocks (fp8_blocks.cu).
cudaError_t launch_fp8_store(const Fp8Args& a, cudaStream_t stream);
cudaError_t launch_fp8_restore(const Fp8Args& a, cudaStream_t stream);

// dG, dU (and h) from the checkpoint's codes, and the input from its own
// where `x` has any (fp8_blocks.cu).
cudaError_t launch_gated_grad_stored(const GatedArgs& a, const Fp8Args& x, cudaStream_t stream);

// Plain tiled kernels for every size and stride (gated_simple.cu).
cudaError_t launch_gated_forward_simple(const GatedArgs& a, cudaStream_t stream);
cudaError_t launch_gated_grad_simple(const GatedArgs& a, cudaStream_t stream);
cudaError_t launch_gated_dx_simple(const GatedArgs& a, cudaStream_t stream);
cudaError_t launch_gated_dw_simple(const GatedArgs& a, cudaStream_t stream);
cudaError_t launch_fp8_matmul_simple(const MatmulArgs& a, cudaStream_t stream);

// Launches a kernel that may begin before the work ahead of it on the stream
// has ended (programmatic dependent launch): it calls after_previous() before
// it touches memory, so only its set-up overlaps.  cluster: CTAs of a
// cluster, 0 where the kernel fixes it.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, unsigned cluster,
                         cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {cluster, 1, 1};
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = at;
  c.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Clusters of 2 to 4 pairs of CTAs that work on one tile, each pair on a part
// of its contraction.  A cluster lies within one GPC, so the device holds
// fewer than it has SMs by their size.
constexpr int kMaxSplit = 4;
struct PairClusters {
  int held[kMaxSplit + 1];  // at one time, of so many pairs

  cudaError_t prepare(const void* kernel, int threads, size_t smem);
  // Pairs for a tile: as many as all tiles find at one time, each with at
  // least eight stages, or 1, as with fewer stages than `least` in all.
  int split(int64_t tiles, int64_t stages, int least) const {
    int s = stages < least ? 1 : kMaxSplit;
    while (s > 1 && (held[s] < tiles || stages < 8 * s)) --s;
    return s;
  }
};

// Clusters of 2 to 8 CTAs of the few-token kernels, likewise: of so many CTAs
// that the device holds at one time.
constexpr int kMaxCluster = 8;
using FewClusters = int[kMaxCluster + 1];

// What a device holds at one time, which the splits go by.  A handle keeps its
// own device's.
struct TcDevice {
  int sms;
  int pairs;               // of CTAs
  PairClusters gated, fp8;  // of the split kernels
  FewClusters few[4][3][2];  // by kind, tile of tokens and activation
};

// What a tensor-core launch takes from its handle.
struct TcLaunch {
  const TcDevice* dev;
  int* err;   // the handle's error word
  uint64_t stall_ns;  // test: a wait that must run out
  uint64_t late_ns;   // test: the same of one warp, beside others whose do not
};

// Tensor-core kernels of the gated block (gated_tc.cu).  They take matrices
// whose rows start on 16 bytes.
// prepare: sets a file's kernels up on the current device (shared-memory
// limits, what the device holds at one time); once for each handle.
cudaError_t gated_tc_prepare(TcDevice* dev);
cudaError_t fp8_tc_prepare(TcDevice* dev);
cudaError_t few_tc_prepare(TcDevice* dev);
bool gated_tc_takes(const GatedArgs& a);
// Pairs of CTAs that share a tile's contraction in forward and grad.
int gated_tc_split(const GatedArgs& a, const TcDevice& dev);
// Workspace for the parts of dX's and dW's sums.
int64_t gated_dx_parts_bytes(int64_t tokens, int64_t hidden);
int64_t gated_dw_parts_bytes(int64_t hidden, int64_t ffn);
cudaError_t launch_gated_forward_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream);
cudaError_t launch_gated_grad_tc(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream);
// dX, dWg and dWu, or either.
cudaError_t launch_gated_back_tc(const GatedArgs& a, bool dx, bool dw, const TcLaunch& l, cudaStream_t stream);

// Tensor-core product of 8-bit blocks (fp8_tc.cu): k a multiple of 16, n and
// the output's stride of 8.
// Pairs of CTAs that share a tile's contraction there.
int fp8_tc_split(const MatmulArgs& a, const TcDevice& dev);
cudaError_t launch_fp8_matmul_tc(const MatmulArgs& a, const TcLaunch& l, cudaStream_t stream);

// The same two products for few tokens (few_tc.cu).
bool gated_few_takes(const GatedArgs& a, const TcLaunch& l);
bool fp8_few_takes(const MatmulArgs& a, const TcLaunch& l);
cudaError_t launch_gated_grad_few(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream);
bool gated_dx_few_takes(const GatedArgs& a, const TcLaunch& l);
cudaError_t launch_gated_dx_few(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream);
cudaError_t launch_gated_forward_few(const GatedArgs& a, const TcLaunch& l, cudaStream_t stream);
cudaError_t launch_fp8_matmul_few(const MatmulArgs& a, const TcLaunch& l, cudaStream_t stream);

}  // namespace tide

struct tide_compute_s {
  int device = -1;  // bound by the first call
  tide::TcDevice dev{};  // written once, before `device`
  // Error word: pinned host memory that a kernel writes when a bounded wait
  // runs out, so that nothing has to be zeroed on a stream.
  int* err = nullptr;
  int* d_err = nullptr;
  int64_t test_stall_ns = 0, test_late_ns = 0;
  std::mutex mu;
};
