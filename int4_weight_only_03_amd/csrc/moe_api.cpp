// C-ABI layer of the mixture-of-experts entry points: argument validation and
// workspace layout.

#include "../../include/w4a16.h"
#include "w4a16_internal.h"

#include <algorithm>
#include <cstdint>

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && a0 < b0 + nb && b0 < a0 + na;
}

struct Range {
  const void *p;
  size_t n;
};

// whether any of the `no` written ranges overlaps another or one of the `ni` read ones
bool any_overlap(const Range *out, int no, const Range *in, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = i + 1; j < no; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    for (int j = 0; j < ni; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
  }
  return false;
}

bool dtype_ok(int32_t dtype) {
  return dtype == W4A16_DTYPE_F32 || dtype == W4A16_DTYPE_F16 || dtype == W4A16_DTYPE_BF16;
}

size_t dtype_size(int32_t dtype) { return dtype == W4A16_DTYPE_F32 ? 4 : 2; }

constexpr int64_t kMaxSlots = 0x7fffffff;

int route_extents(int64_t T, int64_t E, int64_t topk) {
  if (T < 0 || E <= 0 || topk <= 0 || topk > E) return W4A16_ERR_ARG;
  if (E > W4A16_ROUTE_MAX_EXPERTS || topk > W4A16_ROUTE_MAX_TOPK ||
      T > W4A16_ROUTE_MAX_TOKENS || T > kMaxSlots / topk)
    return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// extents of the experts' products: rows of activations, slots, experts,
// outputs and features
int experts_extents(int64_t rows, int64_t R, int64_t E, int64_t N, int64_t K, int32_t group,
                    int32_t dtype) {
  if (group != W4A16_GROUP || !dtype_ok(dtype)) return W4A16_ERR_ARG;
  if (rows < 0 || R < 0 || E <= 0 || N < 0 || K <= 0) return W4A16_ERR_ARG;
  if (K % W4A16_GROUP != 0) return W4A16_ERR_SHAPE;
  if (rows > W4A16_MAX_M || R > W4A16_MAX_M || E > 65535 || N > W4A16_MAX_N / 2 - 4 ||
      K > W4A16_MAX_K)
    return W4A16_ERR_SHAPE;
  // tiles are counted in 32 bits
  const int64_t active = std::min(R, E);
  if (((R + 15 * active) / 16 + 1) * ((N + 15) / 16 + 1) > kMaxSlots / 2) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

size_t combine_rows_bytes(int64_t R, int64_t N) {
  return (size_t(R) * size_t((N + 3) / 4 * 4) * 4 + 255) / 256 * 256;
}

// The launchers refuse a grid that the hardware cannot take as an invalid
// configuration.
int status(hipError_t e) {
  if (e == hipErrorInvalidConfiguration) return W4A16_ERR_SHAPE;
  return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP;
}

}  // namespace

extern "C" {

size_t w4a16_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t topk) {
  if (route_extents(T, E, topk) != W4A16_OK) return 0;
  return w4a16::route_workspace_bytes(long(T), int(E));
}

int w4a16_moe_route(const void *logits, const float *bias, const int32_t *num_tokens,
                    int32_t *ids, float *weights, int32_t *slots, int32_t *token_index,
                    int32_t *expert_offsets, int64_t T, int64_t E, int64_t topk, int32_t score,
                    int64_t groups, int64_t group_limit, int32_t group_top, int32_t renormalize,
                    float scale, int32_t dtype, void *workspace, size_t workspace_bytes,
                    void *stream) {
  const int st = route_extents(T, E, topk);
  if (st != W4A16_OK) return st;
  if (!dtype_ok(dtype) || (score != W4A16_SCORE_SOFTMAX && score != W4A16_SCORE_SIGMOID))
    return W4A16_ERR_ARG;
  if (groups <= 0 || groups > E || E % groups != 0 || group_limit <= 0 || group_limit > groups ||
      (group_top != 1 && group_top != 2))
    return W4A16_ERR_ARG;
  if (groups > W4A16_ROUTE_MAX_GROUPS) return W4A16_ERR_SHAPE;
  if (!(scale - scale == 0.0f)) return W4A16_ERR_ARG;  // NaN or infinite
  if (!expert_offsets) return W4A16_ERR_ARG;
  if (T > 0 && (!logits || !ids || !weights || !slots || !token_index)) return W4A16_ERR_ARG;
  if (!aligned(logits, dtype_size(dtype)) || !aligned(bias, 4) || !aligned(num_tokens, 4) ||
      !aligned(ids, 4) || !aligned(weights, 4) || !aligned(slots, 4) || !aligned(token_index, 4) ||
      !aligned(expert_offsets, 4))
    return W4A16_ERR_ALIGN;
  const size_t need = w4a16::route_workspace_bytes(long(T), int(E));
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return W4A16_ERR_ARG;
  const size_t list = size_t(T) * size_t(topk) * 4;
  const Range out[] = {{ids, list}, {weights, list}, {slots, list}, {token_index, list},
                       {expert_offsets, size_t(E + 1) * 4}, {need ? workspace : nullptr, need}};
  const Range in[] = {{logits, size_t(T) * size_t(E) * dtype_size(dtype)},
                      {bias, size_t(E) * 4}, {num_tokens, 4}};
  if (any_overlap(out, 6, in, 3)) return W4A16_ERR_ARG;
  (void)hipGetLastError();

  w4a16::MoeRoute r;
  r.logits = logits;
  r.bias = bias;
  r.num_tokens = num_tokens;
  r.ids = ids;
  r.weights = weights;
  r.slots = slots;
  r.token_index = token_index;
  r.expert_offsets = expert_offsets;
  r.T = int(T);
  r.E = int(E);
  r.topk = int(topk);
  r.groups = int(groups);
  r.group_limit = int(group_limit);
  r.group_top = group_top;
  r.sigmoid = score == W4A16_SCORE_SIGMOID;
  r.renormalize = renormalize != 0;
  r.dtype = dtype;
  r.scale = scale;
  return status(w4a16::launch_route(r, workspace, reinterpret_cast<hipStream_t>(stream)));
}

int w4a16_experts_kernel(int64_t R, int64_t E, int32_t dtype) {
  if (R <= 0 || E <= 0 || R > W4A16_MAX_M || E > 65535 || !dtype_ok(dtype)) return 0;
  return w4a16::experts_kernel(long(R), long(E), dtype);
}

size_t w4a16_grouped_swiglu_workspace_bytes(int64_t T, int64_t R, int64_t E, int64_t F, int64_t K,
                                            int32_t dtype) {
  if (experts_extents(T, R, E, F, K, W4A16_GROUP, dtype) != W4A16_OK || R == 0 || F == 0) return 0;
  return w4a16::experts_workspace_bytes(long(T), long(R), long(E), int(K), dtype);
}

int w4a16_gemm_grouped_swiglu(const void *X, const int32_t *token_index,
                              const int32_t *expert_offsets, const int32_t *qweight,
                              const float *scales, void *H, int64_t T, int64_t R, int64_t E,
                              int64_t F, int64_t K, int32_t group, int32_t dtype, void *workspace,
                              size_t workspace_bytes, void *stream) {
  const int st = experts_extents(T, R, E, F, K, group, dtype);
  if (st != W4A16_OK || R == 0 || F == 0) return st;
  if (T == 0) return W4A16_ERR_ARG;  // slots but no tokens to read
  if (!X || !token_index || !expert_offsets || !qweight || !scales || !H) return W4A16_ERR_ARG;
  const size_t size = dtype_size(dtype);
  if (!aligned(X, 16) || !aligned(qweight, 16) || !aligned(scales, 4) || !aligned(H, size) ||
      !aligned(token_index, 4) || !aligned(expert_offsets, 4))
    return W4A16_ERR_ALIGN;
  const size_t need = w4a16::experts_workspace_bytes(long(T), long(R), long(E), int(K), dtype);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return W4A16_ERR_ARG;
  const size_t rows = size_t(E) * 2 * size_t(F);
  const Range out[] = {{H, size_t(R) * size_t(F) * size}, {need ? workspace : nullptr, need}};
  const Range in[] = {{X, size_t(T) * size_t(K) * size},
                      {token_index, size_t(R) * 4},
                      {expert_offsets, size_t(E + 1) * 4},
                      {qweight, rows * size_t(K) / 2},
                      {scales, rows * size_t(K / W4A16_GROUP) * 4}};
  if (any_overlap(out, 2, in, 5)) return W4A16_ERR_ARG;
  (void)hipGetLastError();

  w4a16::MoeExperts p;
  p.X = X;
  p.token_index = token_index;
  p.expert_offsets = expert_offsets;
  p.qweight = qweight;
  p.scales = scales;
  p.Y = H;
  p.workspace = workspace;
  p.rows_x = int(T);
  p.R = int(R);
  p.E = int(E);
  p.N = int(F);
  p.K = int(K);
  p.ldy = int(F);
  p.dtype = dtype;
  p.swiglu = true;
  return status(w4a16::launch_experts(p, reinterpret_cast<hipStream_t>(stream)));
}

size_t w4a16_grouped_combine_workspace_bytes(int64_t T, int64_t topk, int64_t E, int64_t N,
                                             int64_t K, int32_t dtype) {
  if (T <= 0 || topk <= 0 || N <= 0 || T > kMaxSlots / topk) return 0;
  const int64_t R = T * topk;
  if (experts_extents(R, R, E, N, K, W4A16_GROUP, dtype) != W4A16_OK) return 0;
  return combine_rows_bytes(R, N) +
         w4a16::experts_workspace_bytes(long(R), long(R), long(E), int(K), dtype);
}

int w4a16_gemm_grouped_combine(const void *H, const int32_t *expert_offsets,
                               const int32_t *qweight, const float *scales, const int32_t *slots,
                               const float *weights, void *Y, int64_t T, int64_t topk, int64_t E,
                               int64_t N, int64_t K, int32_t group, int32_t dtype,
                               void *workspace, size_t workspace_bytes, void *stream) {
  if (T < 0 || topk <= 0) return W4A16_ERR_ARG;
  if (T > kMaxSlots / topk) return W4A16_ERR_SHAPE;
  const int64_t R = T * topk;
  const int st = experts_extents(R, R, E, N, K, group, dtype);
  if (st != W4A16_OK || R == 0 || N == 0) return st;
  if (!H || !expert_offsets || !qweight || !scales || !slots || !weights || !Y)
    return W4A16_ERR_ARG;
  const size_t size = dtype_size(dtype);
  if (!aligned(H, 16) || !aligned(qweight, 16) || !aligned(scales, 4) || !aligned(Y, size) ||
      !aligned(expert_offsets, 4) || !aligned(slots, 4) || !aligned(weights, 4))
    return W4A16_ERR_ALIGN;
  const size_t rows_bytes = combine_rows_bytes(R, N);
  const size_t need =
      rows_bytes + w4a16::experts_workspace_bytes(long(R), long(R), long(E), int(K), dtype);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return W4A16_ERR_ARG;
  const size_t rows = size_t(E) * size_t(N);
  const Range out[] = {{Y, size_t(T) * size_t(N) * size}, {workspace, need}};
  const Range in[] = {{H, size_t(R) * size_t(K) * size},
                      {expert_offsets, size_t(E + 1) * 4},
                      {qweight, rows * size_t(K) / 2},
                      {scales, rows * size_t(K / W4A16_GROUP) * 4},
                      {slots, size_t(R) * 4},
                      {weights, size_t(R) * 4}};
  if (any_overlap(out, 2, in, 6)) return W4A16_ERR_ARG;
  (void)hipGetLastError();

  w4a16::MoeExperts p;
  p.X = H;
  p.token_index = nullptr;
  p.expert_offsets = expert_offsets;
  p.qweight = qweight;
  p.scales = scales;
  p.Y = workspace;
  p.workspace = static_cast<unsigned char *>(workspace) + rows_bytes;
  p.rows_x = int(R);
  p.R = int(R);
  p.E = int(E);
  p.N = int(N);
  p.K = int(K);
  p.ldy = int((N + 3) / 4 * 4);
  p.dtype = dtype;
  p.swiglu = false;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (w4a16::experts_token(long(T), long(topk), int(N), int(K), dtype)) {
    p.Y = Y;
    return status(w4a16::launch_experts_token(p, slots, weights, int(topk), s));
  }
  const hipError_t e = w4a16::launch_experts(p, s);
  if (e != hipSuccess) return status(e);
  return status(w4a16::launch_combine(static_cast<const float *>(workspace), slots, weights, Y,
                                      int(T), int(topk), int(R), int(N), p.ldy, dtype, s));
}

}  // extern "C"
