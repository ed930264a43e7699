// C ABI of the feed-forward unit: argument checks, the handle's device
// binding, and the choice between the kernels.
#include <cstring>
#include <new>
#include <string>

#include "compute_checks.h"

using namespace tide;

namespace {

tide_status_t check_gated(const GatedArgs& a, const char* what) {
  TIDE_TRY(check_dims(a.tokens, a.hidden, what));
  TIDE_TRY(check_dims(a.tokens, a.ffn, what));
  TIDE_TRY(check_dims(a.ffn, a.hidden, what));
  if (a.act != TIDE_ACT_SILU && a.act != TIDE_ACT_GELU) return invalid(std::string(what) + ": unknown activation");
  TIDE_TRY(check_buffer(a.wg, a.ffn * a.hidden, "w_gate"));
  return check_buffer(a.wu, a.ffn * a.hidden, "w_up");
}

tide_status_t check_checkpoint(const tide_gated_checkpoint_t* c, int64_t tokens, int64_t hidden, int64_t ffn) {
  TIDE_TRY(check_blocks(c->gate_codes, c->gate_scales, tokens, ffn, "checkpoint gate"));
  TIDE_TRY(check_blocks(c->up_codes, c->up_scales, tokens, ffn, "checkpoint up"));
  if (c->x_codes || c->x_scales) TIDE_TRY(check_blocks(c->x_codes, c->x_scales, tokens, hidden, "checkpoint x"));
  return TIDE_OK;
}

// Offsets of the workspace's parts.
struct Workspace {
  int64_t dg, du, x, dx_parts, dw_parts, bytes;
};
Workspace workspace_of(int64_t tokens, int64_t hidden, int64_t ffn) {
  Workspace w{};
  if (tokens == 0) return w;
  w.du = round256(2 * tokens * ffn);
  w.x = w.du + round256(2 * tokens * ffn);
  w.dx_parts = w.x + round256(2 * tokens * hidden);
  w.dw_parts = w.dx_parts + round256(gated_dx_parts_bytes(tokens, hidden));
  w.bytes = w.dw_parts + round256(gated_dw_parts_bytes(hidden, ffn));
  return w;
}

}  // namespace

// Binds the handle to the current device on first use.
tide_status_t tide::bind(tide_compute_s* c, cudaStream_t stream) {
  std::lock_guard<std::mutex> g(c->mu);
  int dev = 0;
  TIDE_TRY(current_device(c, &dev));
  if (c->device >= 0) return TIDE_OK;
  if (capturing(stream))
    return set_error(TIDE_ERR_UNSUPPORTED,
                     "the handle's first call sets it up on the device and cannot be captured; make one call before");
  cudaError_t e = cudaDeviceGetAttribute(&c->dev.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(MultiProcessorCount)");
  e = gated_tc_prepare(&c->dev);
  if (e == cudaSuccess) e = fp8_tc_prepare(&c->dev);
  if (e == cudaSuccess) e = few_tc_prepare(&c->dev);
  if (e == cudaSuccess) e = ortho_prepare(&c->dev);
  if (e != cudaSuccess) return cuda_fail(e, "set-up of the tensor-core kernels");
  if (c->dev.pairs < 1) return set_error(TIDE_ERR_CUDA, "the device holds no pair of tensor-core CTAs");
  if (!c->err) {
    e = cudaHostAlloc((void**)&c->err, sizeof(int), cudaHostAllocMapped);
    if (e != cudaSuccess) return cuda_fail(e, "cudaHostAlloc(error word)");
    *c->err = 0;
    e = cudaHostGetDevicePointer((void**)&c->d_err, c->err, 0);
    if (e != cudaSuccess) return cuda_fail(e, "cudaHostGetDevicePointer(error word)");
  }
  c->device = dev;
  return TIDE_OK;
}

extern "C" {

tide_status_t tide_compute_create(tide_compute_t* out) try {
  if (!out) return invalid("out is NULL");
  *out = new (std::nothrow) tide_compute_s();
  return *out ? TIDE_OK : set_error(TIDE_ERR_OUT_OF_MEMORY, "host allocation failed");
}
TIDE_CATCH

void tide_compute_destroy(tide_compute_t c) {
  if (!c) return;
  if (c->err && cudaFreeHost(c->err) != cudaSuccess) cudaGetLastError();
  delete c;
}

tide_status_t tide_compute_check_device(tide_compute_t c) try {
  if (!c) return invalid("compute is NULL");
  std::lock_guard<std::mutex> g(c->mu);
  if (c->device < 0) return TIDE_OK;  // nothing launched yet
  int dev = 0;
  TIDE_TRY(current_device(c, &dev));  // another device's end says nothing of this handle's kernels
  const cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  volatile int* err = c->err;
  if (*err == 0) return TIDE_OK;
  *err = 0;
  return set_error(TIDE_ERR_TIMEOUT, "a bounded wait in a tensor-core kernel ran out; its outputs are incomplete");
}
TIDE_CATCH

tide_status_t tide_compute_set_test_stall(tide_compute_t c, int64_t ns) try {
  if (!c || ns < 0) return invalid("NULL handle or negative time");
  std::lock_guard<std::mutex> g(c->mu);
  c->test_stall_ns = ns;
  return TIDE_OK;
}
TIDE_CATCH

tide_status_t tide_compute_set_test_late_warp(tide_compute_t c, int64_t ns) try {
  if (!c || ns < 0) return invalid("NULL handle or negative time");
  std::lock_guard<std::mutex> g(c->mu);
  c->test_late_ns = ns;
  return TIDE_OK;
}
TIDE_CATCH

tide_status_t tide_fp8_store(tide_compute_t c, int64_t rows, int64_t cols, const uint16_t* src, int64_t ld_src,
                             uint8_t* codes, float* scales, int32_t block_rows, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  if (block_rows != 1 && block_rows != kBlock) return invalid("block_rows must be 1 or 128");
  TIDE_TRY(check_dims(rows, cols, "tide_fp8_store"));
  TIDE_TRY(check_matrix(src, rows, cols, ld_src, "src"));
  TIDE_TRY(check_blocks(codes, scales, rows, cols, "destination"));
  if (rows * cols == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  const Fp8Args a{rows, cols, ld_src, const_cast<uint16_t*>(src), codes, scales, block_rows};
  return launched(launch_fp8_store(a, stream), "tide_fp8_store");
}
TIDE_CATCH

tide_status_t tide_fp8_restore(tide_compute_t c, int64_t rows, int64_t cols, const uint8_t* codes,
                               const float* scales, int32_t block_rows, uint16_t* dst, int64_t ld_dst,
                               cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  if (block_rows != 1 && block_rows != kBlock) return invalid("block_rows must be 1 or 128");
  TIDE_TRY(check_dims(rows, cols, "tide_fp8_restore"));
  TIDE_TRY(check_blocks(codes, scales, rows, cols, "source"));
  TIDE_TRY(check_matrix(dst, rows, cols, ld_dst, "dst"));
  if (rows * cols == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  const Fp8Args a{rows,       cols, ld_dst, dst, const_cast<uint8_t*>(codes), const_cast<float*>(scales),
                  block_rows};
  return launched(launch_fp8_restore(a, stream), "tide_fp8_restore");
}
TIDE_CATCH

tide_status_t tide_fp8_matmul(tide_compute_t c, int64_t m, int64_t n, int64_t k, const uint8_t* a,
                              const float* a_scales, const uint8_t* b, const float* b_scales, int32_t any_scales,
                              uint16_t* out, int64_t ld_out, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  TIDE_TRY(check_dims(m, k, "tide_fp8_matmul"));
  TIDE_TRY(check_dims(n, k, "tide_fp8_matmul"));
  TIDE_TRY(check_dims(m, n, "tide_fp8_matmul"));
  TIDE_TRY(check_blocks(a, a_scales, m, k, "a"));
  TIDE_TRY(check_blocks(b, b_scales, n, k, "b"));
  TIDE_TRY(check_matrix(out, m, n, ld_out, "out"));
  if (m * n == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  if (k == 0)  // an empty sum
    return launched(cudaMemset2DAsync(out, ld_out * 2, 0, n * 2, m, stream), "tide_fp8_matmul");
  const MatmulArgs args{m, n, k, a, a_scales, b, b_scales, out, ld_out, any_scales != 0};
  if (k % 16 == 0 && n % 8 == 0 && ld_out % 8 == 0) {
    const TcLaunch l = launch_of(c);
    return launched(fp8_few_takes(args, l) ? launch_fp8_matmul_few(args, l, stream)
                                                 : launch_fp8_matmul_tc(args, l, stream),
                    "tide_fp8_matmul");
  }
  return launched(launch_fp8_matmul_simple(args, stream), "tide_fp8_matmul");
}
TIDE_CATCH

tide_status_t tide_gated_forward(tide_compute_t c, int64_t tokens, int64_t hidden, int64_t ffn, tide_activation_t act,
                                 const uint16_t* x, int64_t ld_x, const uint16_t* w_gate, const uint16_t* w_up,
                                 uint16_t* h, int64_t ld_h, const tide_gated_checkpoint_t* ck, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  GatedArgs a{};
  a.tokens = tokens, a.hidden = hidden, a.ffn = ffn, a.act = act;
  a.x = x, a.ldx = ld_x, a.wg = w_gate, a.wu = w_up, a.h = h, a.ldh = ld_h;
  TIDE_TRY(check_gated(a, "tide_gated_forward"));
  TIDE_TRY(check_matrix(x, tokens, hidden, ld_x, "x"));
  TIDE_TRY(check_matrix(h, tokens, ffn, ld_h, "h"));
  if (ck) {
    TIDE_TRY(check_checkpoint(ck, tokens, hidden, ffn));
    a.g8 = ck->gate_codes, a.gs = ck->gate_scales, a.u8 = ck->up_codes, a.us = ck->up_scales;
  }
  if (tokens == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  if (ck && ck->x_codes && hidden) {
    const Fp8Args s{tokens, hidden, ld_x, const_cast<uint16_t*>(x), ck->x_codes, ck->x_scales, 1};
    TIDE_TRY(launched(launch_fp8_store(s, stream), "tide_gated_forward"));
  }
  if (ffn == 0) return TIDE_OK;
  if (gated_tc_takes(a) && ld_x % 8 == 0 && ld_h % 8 == 0) {
    const TcLaunch l = launch_of(c);
    return launched(gated_few_takes(a, l) ? launch_gated_forward_few(a, l, stream)
                                                : launch_gated_forward_tc(a, l, stream),
                    "tide_gated_forward");
  }
  return launched(launch_gated_forward_simple(a, stream), "tide_gated_forward");
}
TIDE_CATCH

tide_status_t tide_gated_workspace(int64_t tokens, int64_t hidden, int64_t ffn, int64_t* bytes) try {
  if (!bytes) return invalid("bytes is NULL");
  *bytes = 0;
  TIDE_TRY(check_dims(tokens, hidden, "tide_gated_workspace"));
  TIDE_TRY(check_dims(tokens, ffn, "tide_gated_workspace"));
  TIDE_TRY(check_dims(ffn, hidden, "tide_gated_workspace"));
  *bytes = workspace_of(tokens, hidden, ffn).bytes;
  return TIDE_OK;
}
TIDE_CATCH

tide_status_t tide_gated_backward(tide_compute_t c, int64_t tokens, int64_t hidden, int64_t ffn,
                                  tide_activation_t act, const uint16_t* dh, int64_t ld_dh, const uint16_t* x,
                                  int64_t ld_x, const uint16_t* w_gate, const uint16_t* w_up,
                                  const tide_gated_checkpoint_t* ck, uint16_t* dx, int64_t ld_dx, uint16_t* dw_gate,
                                  uint16_t* dw_up, uint16_t* h, int64_t ld_h, void* workspace,
                                  int64_t workspace_bytes, cudaStream_t stream) try {
  const char* what = "tide_gated_backward";
  if (!c) return invalid("compute is NULL");
  GatedArgs a{};
  a.tokens = tokens, a.hidden = hidden, a.ffn = ffn, a.act = act;
  a.x = x, a.ldx = ld_x, a.wg = w_gate, a.wu = w_up, a.h = h, a.ldh = ld_h;
  a.dh = dh, a.lddh = ld_dh, a.dx = dx, a.lddx = ld_dx, a.dwg = dw_gate, a.dwu = dw_up;
  TIDE_TRY(check_gated(a, what));
  TIDE_TRY(check_matrix(dh, tokens, ffn, ld_dh, "dh"));
  const bool x8 = ck && ck->x_codes;
  if (ck) {
    TIDE_TRY(check_checkpoint(ck, tokens, hidden, ffn));
    a.g8 = ck->gate_codes, a.gs = ck->gate_scales, a.u8 = ck->up_codes, a.us = ck->up_scales;
  }
  const int64_t weights = ffn * hidden;
  if (!dw_gate != !dw_up && weights) return invalid("dw_gate and dw_up: both or neither");
  if (!x8 && (!ck || dw_gate)) TIDE_TRY(check_matrix(x, tokens, hidden, ld_x, "x"));
  if (dx) TIDE_TRY(check_matrix(dx, tokens, hidden, ld_dx, "dx"));
  if (dw_gate) TIDE_TRY(check_buffer(dw_gate, weights, "dw_gate"));
  if (dw_up) TIDE_TRY(check_buffer(dw_up, weights, "dw_up"));
  if (h) TIDE_TRY(check_matrix(h, tokens, ffn, ld_h, "h"));
  const Workspace w = workspace_of(tokens, hidden, ffn);
  TIDE_TRY(check_buffer(workspace, w.bytes, "workspace"));
  if (workspace_bytes < w.bytes)
    return invalid("workspace: " + std::to_string(w.bytes) + " bytes are needed, " + std::to_string(workspace_bytes) +
                   " given");
  if (hidden == 0 && !h) return TIDE_OK;
  if (tokens == 0 && (!dw_gate || !weights)) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  if (tokens == 0) {  // gradients of no tokens
    TIDE_TRY(launched(cudaMemsetAsync(dw_gate, 0, weights * 2, stream), what));
    return launched(cudaMemsetAsync(dw_up, 0, weights * 2, stream), what);
  }
  if (ffn == 0) {
    if (!dx || !hidden) return TIDE_OK;
    return launched(cudaMemset2DAsync(dx, ld_dx * 2, 0, hidden * 2, tokens, stream), what);
  }
  a.dg = (uint16_t*)((char*)workspace + w.dg);
  a.du = (uint16_t*)((char*)workspace + w.du);
  a.dx_parts = (float*)((char*)workspace + w.dx_parts), a.dx_parts_bytes = w.dw_parts - w.dx_parts;
  a.dw_parts = (float*)((char*)workspace + w.dw_parts), a.dw_parts_bytes = w.bytes - w.dw_parts;
  const TcLaunch l = launch_of(c);
  const bool tc = gated_tc_takes(a);
  Fp8Args xr{};
  if (x8 && dw_gate && hidden) {  // the restored input takes x's place
    xr = Fp8Args{tokens, hidden, hidden, (uint16_t*)((char*)workspace + w.x), ck->x_codes, ck->x_scales, 1};
    a.x = xr.bf16, a.ldx = hidden;
  }
  if (ck)
    TIDE_TRY(launched(launch_gated_grad_stored(a, xr, stream), what));
  else if (tc && ld_x % 8 == 0 && ld_dh % 8 == 0 && (!h || ld_h % 8 == 0))
    TIDE_TRY(launched(gated_few_takes(a, l) ? launch_gated_grad_few(a, l, stream) : launch_gated_grad_tc(a, l, stream), what));
  else
    TIDE_TRY(launched(launch_gated_grad_simple(a, stream), what));
  if (hidden == 0) return TIDE_OK;
  const bool dx_tc = dx && tc && ld_dx % 8 == 0, dw_tc = dw_gate && tc && a.ldx % 8 == 0;
  const bool dx_few = dx_tc && gated_dx_few_takes(a, l);
  if (dx_few) TIDE_TRY(launched(launch_gated_dx_few(a, l, stream), what));
  if ((dx_tc && !dx_few) || dw_tc) TIDE_TRY(launched(launch_gated_back_tc(a, dx_tc && !dx_few, dw_tc, l, stream), what));
  if (dx && !dx_tc) TIDE_TRY(launched(launch_gated_dx_simple(a, stream), what));
  if (dw_gate && !dw_tc) TIDE_TRY(launched(launch_gated_dw_simple(a, stream), what));
  return TIDE_OK;
}
TIDE_CATCH

}  // extern "C"
