// C ABI of the expert layer: routing, experts' rows, orthogonalised updates.
#include <cmath>
#include <cstring>

#include "compute_checks.h"

using namespace tide;

namespace {

constexpr int64_t kMaxSide = (int64_t)1 << 30;  // of a matrix to orthogonalise: tiles pass its end
constexpr int64_t kMaxShort = (int64_t)1 << 17;  // of its short side: sums along it are not parted
const float kCoefficients[3] = {3.4445f, -4.7750f, 2.0315f};

// An array of `bytes`-sized elements, aligned to them.
tide_status_t check_array(const void* p, int64_t numel, int bytes, const char* what) {
  if (numel == 0) return TIDE_OK;
  if (!p) return invalid(std::string(what) + " is NULL");
  if ((uintptr_t)p & (uintptr_t)(bytes - 1))
    return set_error(TIDE_ERR_MISALIGNED, std::string(what) + " is not aligned to its elements");
  return TIDE_OK;
}

tide_status_t check_type(tide_dtype_t type) {
  return type == TIDE_BF16 || type == TIDE_FP32 ? TIDE_OK : invalid("unknown element type");
}

tide_status_t check_router(const tide_router_t* r, int64_t tokens) {
  if (!r) return invalid("router is NULL");
  if (r->experts < 1 || r->experts > TIDE_MAX_EXPERTS) return invalid("router: experts out of range");
  if (r->topk < 1 || r->topk > TIDE_MAX_TOPK || r->topk > r->experts) return invalid("router: topk out of range");
  if (r->score != TIDE_SCORE_SOFTMAX && r->score != TIDE_SCORE_SIGMOID) return invalid("router: unknown score");
  if (r->groups < 1 || r->groups > 32 || r->experts % r->groups) return invalid("router: groups of one size, 1 to 32, are wanted");
  if (r->top_groups < 1 || r->top_groups > r->groups) return invalid("router: top_groups out of range");
  if (r->group_best != 1 && r->group_best != 2) return invalid("router: group_best must be 1 or 2");
  if (r->topk > r->top_groups * (r->experts / r->groups)) return invalid("router: the best groups hold fewer than topk experts");
  return check_dims(tokens, r->experts, "router");
}

// A matrix of `rows` rows of `cols` elements, `ld` apart, aligned to them.
tide_status_t check_typed(const void* p, int64_t rows, int64_t cols, int64_t ld, tide_dtype_t type, const char* what) {
  TIDE_TRY(check_array(p, rows * cols, type == TIDE_BF16 ? 2 : 4, what));
  if (ld < cols || (rows && ld > kMaxNumel / rows)) return invalid(std::string(what) + ": row stride out of range");
  return TIDE_OK;
}

RouterArgs router_args(const tide_router_t* r, int64_t tokens, tide_dtype_t type, const void* logits, int64_t ld) {
  RouterArgs a{};
  a.tokens = tokens;
  a.experts = r->experts, a.topk = r->topk, a.score = r->score;
  a.groups = r->groups, a.top_groups = r->top_groups, a.group_best = r->group_best;
  a.renormalize = r->renormalize != 0, a.scale = r->scale;
  a.bf16 = type == TIDE_BF16, a.logits = logits, a.ld = ld;
  return a;
}

tide_status_t check_pairs(int64_t tokens, int64_t topk, const char* what) {
  if (tokens < 0 || topk < 1 || topk > 1024 || tokens > kMaxDim / topk) return invalid(std::string(what) + ": sizes out of range");
  return TIDE_OK;
}

tide_status_t check_rows(int64_t tokens, int64_t hidden, int64_t topk, int64_t num_rows, const int32_t* slots,
                         const char* what) {
  TIDE_TRY(check_pairs(tokens, topk, what));
  TIDE_TRY(check_dims(tokens, hidden, what));
  TIDE_TRY(check_dims(num_rows, hidden, what));
  return check_array(slots, tokens * topk, 4, "slots");
}

}  // namespace

extern "C" {

tide_status_t tide_route(tide_compute_t c, int64_t tokens, const tide_router_t* router, tide_dtype_t type,
                         const void* logits, int64_t ld_logits, const float* bias, int32_t* ids, float* weights,
                         cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  TIDE_TRY(check_router(router, tokens));
  TIDE_TRY(check_type(type));
  TIDE_TRY(check_typed(logits, tokens, router->experts, ld_logits, type, "logits"));
  if (bias) TIDE_TRY(check_array(bias, router->experts, 4, "bias"));
  TIDE_TRY(check_array(ids, tokens * router->topk, 4, "ids"));
  TIDE_TRY(check_array(weights, tokens * router->topk, 4, "weights"));
  if (tokens == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  RouterArgs a = router_args(router, tokens, type, logits, ld_logits);
  a.bias = bias, a.ids = ids, a.weights = weights;
  return launched(launch_route(a, stream), "tide_route");
}
TIDE_CATCH

tide_status_t tide_route_backward(tide_compute_t c, int64_t tokens, const tide_router_t* router, tide_dtype_t type,
                                  const void* logits, int64_t ld_logits, const int32_t* ids, const float* dweights,
                                  void* dlogits, int64_t ld_dlogits, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  TIDE_TRY(check_router(router, tokens));
  TIDE_TRY(check_type(type));
  TIDE_TRY(check_typed(logits, tokens, router->experts, ld_logits, type, "logits"));
  TIDE_TRY(check_array(ids, tokens * router->topk, 4, "ids"));
  TIDE_TRY(check_array(dweights, tokens * router->topk, 4, "dweights"));
  TIDE_TRY(check_typed(dlogits, tokens, router->experts, ld_dlogits, type, "dlogits"));
  if (tokens == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  RouterArgs a = router_args(router, tokens, type, logits, ld_logits);
  a.ids = const_cast<int32_t*>(ids), a.dweights = dweights, a.dlogits = dlogits, a.ldd = ld_dlogits;
  return launched(launch_route_backward(a, stream), "tide_route_backward");
}
TIDE_CATCH

tide_status_t tide_expert_slots_workspace(int64_t tokens, int64_t topk, int64_t experts, int64_t* bytes) try {
  if (!bytes) return invalid("bytes is NULL");
  *bytes = 0;
  TIDE_TRY(check_pairs(tokens, topk, "tide_expert_slots_workspace"));
  if (experts < 1 || experts > TIDE_MAX_EXPERTS) return invalid("tide_expert_slots_workspace: experts out of range");
  *bytes = slots_workspace_bytes(tokens * topk, experts);
  return TIDE_OK;
}
TIDE_CATCH

tide_status_t tide_expert_slots(tide_compute_t c, int64_t tokens, int64_t topk, int64_t experts, const int32_t* ids,
                                int32_t* slots, int32_t* offsets, void* workspace, int64_t workspace_bytes,
                                cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  TIDE_TRY(check_pairs(tokens, topk, "tide_expert_slots"));
  if (experts < 1 || experts > TIDE_MAX_EXPERTS) return invalid("tide_expert_slots: experts out of range");
  const int64_t pairs = tokens * topk, need = slots_workspace_bytes(pairs, experts);
  TIDE_TRY(check_array(ids, pairs, 4, "ids"));
  TIDE_TRY(check_array(slots, pairs, 4, "slots"));
  TIDE_TRY(check_array(offsets, experts + 1, 4, "offsets"));
  TIDE_TRY(check_buffer(workspace, need, "workspace"));
  if (workspace_bytes < need)
    return invalid("workspace: " + std::to_string(need) + " bytes are needed, " + std::to_string(workspace_bytes) + " given");
  TIDE_TRY(bind(c, stream));
  if (pairs == 0) return launched(cudaMemsetAsync(offsets, 0, (experts + 1) * 4, stream), "tide_expert_slots");
  const SlotsArgs a{pairs, (int)experts, ids, slots, offsets, (int32_t*)workspace};
  return launched(launch_expert_slots(a, stream), "tide_expert_slots");
}
TIDE_CATCH

tide_status_t tide_expert_gather(tide_compute_t c, int64_t tokens, int64_t hidden, int64_t topk, const uint16_t* x,
                                 int64_t ld_x, const int32_t* slots, uint16_t* rows, int64_t num_rows,
                                 int64_t ld_rows, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  TIDE_TRY(check_rows(tokens, hidden, topk, num_rows, slots, "tide_expert_gather"));
  TIDE_TRY(check_matrix(x, tokens, hidden, ld_x, "x"));
  TIDE_TRY(check_matrix(rows, num_rows, hidden, ld_rows, "rows"));
  if (tokens == 0 || hidden == 0 || num_rows == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  RowsArgs a{};
  a.tokens = tokens, a.hidden = hidden, a.num_rows = num_rows, a.topk = (int)topk, a.slots = slots;
  a.in = x, a.ld_in = ld_x, a.out = rows, a.ld_out = ld_rows;
  return launched(launch_expert_gather(a, launch_of(c).dev->sms, stream), "tide_expert_gather");
}
TIDE_CATCH

tide_status_t tide_expert_combine(tide_compute_t c, int64_t tokens, int64_t hidden, int64_t topk,
                                  const uint16_t* rows, int64_t num_rows, int64_t ld_rows, const int32_t* slots,
                                  const float* weights, uint16_t* y, int64_t ld_y, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  TIDE_TRY(check_rows(tokens, hidden, topk, num_rows, slots, "tide_expert_combine"));
  TIDE_TRY(check_matrix(rows, num_rows, hidden, ld_rows, "rows"));
  if (weights) TIDE_TRY(check_array(weights, tokens * topk, 4, "weights"));
  TIDE_TRY(check_matrix(y, tokens, hidden, ld_y, "y"));
  if (tokens == 0 || hidden == 0) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  RowsArgs a{};
  a.tokens = tokens, a.hidden = hidden, a.num_rows = num_rows, a.topk = (int)topk, a.slots = slots;
  a.weights = weights, a.in = rows, a.ld_in = ld_rows, a.out = y, a.ld_out = ld_y;
  return launched(launch_expert_combine(a, launch_of(c).dev->sms, stream), "tide_expert_combine");
}
TIDE_CATCH

tide_status_t tide_expert_combine_backward(tide_compute_t c, int64_t tokens, int64_t hidden, int64_t topk,
                                           const uint16_t* dy, int64_t ld_dy, const uint16_t* rows, int64_t num_rows,
                                           int64_t ld_rows, const int32_t* slots, const float* weights,
                                           uint16_t* drows, int64_t ld_drows, float* dweights, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  TIDE_TRY(check_rows(tokens, hidden, topk, num_rows, slots, "tide_expert_combine_backward"));
  TIDE_TRY(check_matrix(dy, tokens, hidden, ld_dy, "dy"));
  if (dweights) {
    TIDE_TRY(check_matrix(rows, num_rows, hidden, ld_rows, "rows"));
    TIDE_TRY(check_array(dweights, tokens * topk, 4, "dweights"));
  }
  if (weights) TIDE_TRY(check_array(weights, tokens * topk, 4, "weights"));
  if (drows) TIDE_TRY(check_matrix(drows, num_rows, hidden, ld_drows, "drows"));
  if (tokens == 0 || (!drows && !dweights) || (hidden == 0 && !dweights)) return TIDE_OK;
  TIDE_TRY(bind(c, stream));
  if (hidden == 0) return launched(cudaMemsetAsync(dweights, 0, tokens * topk * 4, stream), "tide_expert_combine_backward");
  RowsArgs a{};
  a.tokens = tokens, a.hidden = hidden, a.num_rows = num_rows, a.topk = (int)topk, a.slots = slots;
  a.weights = weights, a.in = dy, a.ld_in = ld_dy, a.rows = rows, a.ld_rows = ld_rows;
  a.out = drows, a.ld_out = ld_drows, a.dweights = dweights;
  return launched(launch_expert_combine_backward(a, launch_of(c).dev->sms, stream), "tide_expert_combine_backward");
}
TIDE_CATCH

tide_status_t tide_orthogonalize_workspace(int64_t count, int64_t rows, int64_t cols, int64_t* bytes) try {
  if (!bytes) return invalid("bytes is NULL");
  *bytes = 0;
  TIDE_TRY(check_dims(rows, cols, "tide_orthogonalize"));
  if (rows > kMaxSide || cols > kMaxSide || (rows > kMaxShort && cols > kMaxShort))
    return invalid("tide_orthogonalize: sizes out of range");
  const int64_t numel = rows * cols;
  if (count < 0 || count > kMaxDim || (numel != 0 && count > kMaxNumel / numel))
    return invalid("tide_orthogonalize: count out of range");
  if (numel != 0 && count != 0) *bytes = ortho_workspace_bytes(count, rows, cols);
  return TIDE_OK;
}
TIDE_CATCH

tide_status_t tide_orthogonalize(tide_compute_t c, int64_t count, int64_t rows, int64_t cols, tide_dtype_t type,
                                 const void* const* src, int64_t ld_src, uint16_t* const* dst, int64_t ld_dst,
                                 int32_t steps, const float* coefficients, float eps, void* workspace,
                                 int64_t workspace_bytes, cudaStream_t stream) try {
  if (!c) return invalid("compute is NULL");
  int64_t need = 0;
  TIDE_TRY(tide_orthogonalize_workspace(count, rows, cols, &need));
  TIDE_TRY(check_type(type));
  if (steps < 0 || steps > TIDE_MAX_ORTHOGONALIZE_STEPS) return invalid("steps out of range");
  if (!(eps >= 0.0f) || std::isinf(eps)) return invalid("eps must be finite and not negative");
  float own[3 * TIDE_MAX_ORTHOGONALIZE_STEPS];
  for (int s = 0; s < steps; ++s)
    memcpy(own + 3 * s, coefficients ? coefficients + 3 * s : kCoefficients, sizeof(kCoefficients));
  if (!ortho_bounded(steps, own)) return invalid("coefficients: not finite, or singular values would pass 2^16");
  if (count == 0 || rows * cols == 0) return TIDE_OK;
  if (!src || !dst) return invalid("a table of matrices is NULL");
  for (int64_t i = 0; i < count; ++i) {
    TIDE_TRY(check_typed(src[i], rows, cols, ld_src, type, "src"));
    TIDE_TRY(check_typed(dst[i], rows, cols, ld_dst, TIDE_BF16, "dst"));
  }
  TIDE_TRY(check_buffer(workspace, need, "workspace"));
  if (workspace_bytes < need)
    return invalid("workspace: " + std::to_string(need) + " bytes are needed, " + std::to_string(workspace_bytes) + " given");
  TIDE_TRY(bind(c, stream));
  const OrthoArgs a{count, rows, cols, type == TIDE_BF16, src, ld_src, dst, ld_dst, steps, own, eps, (char*)workspace};
  return launched(launch_orthogonalize(a, launch_of(c), stream), "tide_orthogonalize");
}
TIDE_CATCH

}  // extern "C"
