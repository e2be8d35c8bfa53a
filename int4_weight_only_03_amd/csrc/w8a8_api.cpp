// C-ABI layer of the 8-bit floating-point operators: argument validation and the host
// quantizer of weights.  Compiled without FMA contraction or fast-math, so that the
// quantizer is bit-exact with any IEEE implementation of its stated fp32 steps.

#include "../../include/w8a8.h"
#include "w8a8_internal.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && a0 < b0 + nb && b0 < a0 + na;
}

bool dtype_ok(int32_t dtype) {
  return dtype == W4A16_DTYPE_F32 || dtype == W4A16_DTYPE_F16 || dtype == W4A16_DTYPE_BF16;
}

size_t dtype_size(int32_t dtype) { return dtype == W4A16_DTYPE_F32 ? 4 : 2; }

size_t blocks(int64_t n) { return size_t((n + W8A8_BLOCK - 1) / W8A8_BLOCK); }

int rows_extents(int64_t M, int64_t K, int32_t dtype, int64_t most_k) {
  if (M < 0 || K <= 0 || !dtype_ok(dtype)) return W4A16_ERR_ARG;
  if (K % 16 != 0 || M > W8A8_MAX_M || K > most_k) return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

// R: rows of Y; T: rows of X
int gemm_extents(int64_t T, int64_t R, int64_t E, int64_t N, int64_t K, int32_t block,
                 int32_t dtype) {
  if (block != W8A8_BLOCK || !dtype_ok(dtype)) return W4A16_ERR_ARG;
  if (T < 0 || R < 0 || E <= 0 || N < 0 || K <= 0) return W4A16_ERR_ARG;
  if (K % 16 != 0 || T > W8A8_MAX_M || R > W8A8_MAX_M || E > 65535 || N > W8A8_MAX_N ||
      K > W8A8_MAX_K)
    return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

int status(hipError_t e) {
  if (e == hipErrorInvalidConfiguration) return W4A16_ERR_SHAPE;
  return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP;
}

// the common part of both products; pointers and lists that are not used are NULL
int gemm(const uint8_t *X, const float *xs, const int32_t *token_index,
         const int32_t *expert_offsets, const uint8_t *W, const float *ws, void *Y, int64_t T,
         int64_t R, int64_t E, int64_t N, int64_t K, int32_t dtype, void *stream) {
  if (!X || !xs || !W || !ws || !Y) return W4A16_ERR_ARG;
  const size_t size = dtype_size(dtype);
  if (!aligned(X, 16) || !aligned(xs, 4) || !aligned(token_index, 4) ||
      !aligned(expert_offsets, 4) || !aligned(W, 16) || !aligned(ws, 4) || !aligned(Y, size))
    return W4A16_ERR_ALIGN;
  const size_t y = size_t(R) * size_t(N) * size, KB = blocks(K);
  if (overlaps(Y, y, X, size_t(T) * size_t(K)) || overlaps(Y, y, xs, size_t(T) * KB * 4) ||
      overlaps(Y, y, token_index, size_t(R) * 4) ||
      overlaps(Y, y, expert_offsets, size_t(E + 1) * 4) ||
      overlaps(Y, y, W, size_t(E) * size_t(N) * size_t(K)) ||
      overlaps(Y, y, ws, size_t(E) * blocks(N) * KB * 4))
    return W4A16_ERR_ARG;
  (void)hipGetLastError();

  w4a16::Gemm8 p;
  p.X = X;
  p.xs = xs;
  p.token_index = token_index;
  p.expert_offsets = expert_offsets;
  p.W = W;
  p.ws = ws;
  p.Y = Y;
  p.rows_x = int(T);
  p.R = int(R);
  p.E = int(E);
  p.N = int(N);
  p.K = int(K);
  p.dtype = dtype;
  return status(w4a16::launch_gemm8(p, reinterpret_cast<hipStream_t>(stream)));
}

// w to the nearest e4m3 value, ties to even, magnitudes past 448 to 448; w is finite
uint8_t to_e4m3(float w) {
  uint32_t bits;
  std::memcpy(&bits, &w, 4);
  const uint8_t sign = uint8_t(bits >> 24 & 0x80);
  const float m = std::fabs(w);
  if (m >= 448.0f) return sign | 0x7E;
  if (m < 0x1p-6f)  // subnormal: steps of 2^-9, the 8th of which is the least normal's code
    return sign | uint8_t(std::nearbyint(m * 0x1p9f));
  // 20 mantissa bits go: half of them and the last that stays, for ties to even
  bits &= 0x7fffffffu;
  bits += 0x7ffffu + (bits >> 20 & 1u);
  return sign | uint8_t((bits >> 20) - ((127 - 7) << 3));
}

}  // namespace

extern "C" {

int w8a8_quantize_weights(const float *W, uint8_t *codes, float *scales, int64_t N, int64_t K,
                          int32_t block) {
  if (block != W8A8_BLOCK || N < 0 || K <= 0) return W4A16_ERR_ARG;
  if (K % 16 != 0 || N > W8A8_MAX_N || K > W8A8_MAX_K) return W4A16_ERR_SHAPE;
  if (N == 0) return W4A16_OK;
  if (!W || !codes || !scales) return W4A16_ERR_ARG;
  const size_t total = size_t(N) * size_t(K);
  for (size_t i = 0; i < total; ++i)
    if (!std::isfinite(W[i])) return W4A16_ERR_NONFINITE;
  const int64_t KB = int64_t(blocks(K));
  for (int64_t n0 = 0; n0 < N; n0 += W8A8_BLOCK) {
    const int64_t n1 = std::min(n0 + W8A8_BLOCK, N);
    for (int64_t b = 0; b < KB; ++b) {
      const int64_t k0 = b * W8A8_BLOCK, k1 = std::min(k0 + W8A8_BLOCK, K);
      float most = 0.0f;
      for (int64_t n = n0; n < n1; ++n)
        for (int64_t k = k0; k < k1; ++k) most = std::fmax(most, std::fabs(W[n * K + k]));
      const float scale = most == 0.0f ? 0.0f : std::fmax(most / 448.0f, 0x1p-126f);
      scales[n0 / W8A8_BLOCK * KB + b] = scale;
      for (int64_t n = n0; n < n1; ++n)
        for (int64_t k = k0; k < k1; ++k)
          codes[n * K + k] = scale == 0.0f ? 0 : to_e4m3(W[n * K + k] / scale);
    }
  }
  return W4A16_OK;
}

int w8a8_quantize(const void *X, const int32_t *num_rows, uint8_t *codes, float *scales,
                  int64_t M, int64_t K, int32_t swiglu, int32_t dtype, void *stream) {
  const int st = rows_extents(M, K, dtype, W8A8_MAX_K);
  if (st != W4A16_OK || M == 0) return st;
  if (!X || !codes || !scales) return W4A16_ERR_ARG;
  if (!aligned(X, 16) || !aligned(num_rows, 4) || !aligned(codes, 16) || !aligned(scales, 4))
    return W4A16_ERR_ALIGN;
  const size_t x = size_t(M) * size_t(K) * (swiglu ? 2 : 1) * dtype_size(dtype),
               c = size_t(M) * size_t(K), s = size_t(M) * blocks(K) * 4;
  if (overlaps(codes, c, scales, s) || overlaps(codes, c, X, x) || overlaps(scales, s, X, x) ||
      overlaps(codes, c, num_rows, 4) || overlaps(scales, s, num_rows, 4))
    return W4A16_ERR_ARG;
  (void)hipGetLastError();
  w4a16::Rows8 p;
  p.X = X;
  p.num_rows = num_rows;
  p.codes = codes;
  p.scales = scales;
  p.M = int(M);
  p.K = int(K);
  p.dtype = dtype;
  p.swiglu = swiglu != 0;
  return status(w4a16::launch_rows8(p, reinterpret_cast<hipStream_t>(stream)));
}

int w8a8_rms_norm(const void *X, const void *residual, const void *weight, void *H, void *Y,
                  uint8_t *codes, float *scales, int64_t M, int64_t K, float eps, int32_t dtype,
                  int32_t weight_dtype, void *stream) {
  const int st = rows_extents(M, K, dtype, W8A8_NORM_MAX_K);
  if (st != W4A16_OK) return st;
  if (!(eps > 0.0f) || std::isinf(eps) ||
      (weight_dtype != dtype && weight_dtype != W4A16_DTYPE_F32))
    return W4A16_ERR_ARG;
  if (M == 0) return W4A16_OK;
  if (!X || !weight || !codes != !scales || (!H && !Y && !codes)) return W4A16_ERR_ARG;
  if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(H, 16) ||
      !aligned(Y, 16) || !aligned(codes, 16) || !aligned(scales, 4))
    return W4A16_ERR_ALIGN;
  struct Range {
    const void *p;
    size_t n;
  };
  const size_t x = size_t(M) * size_t(K) * dtype_size(dtype);
  const Range out[] = {{H, x}, {Y, x}, {codes, size_t(M) * size_t(K)},
                       {scales, size_t(M) * blocks(K) * 4}};
  const Range in[] = {{weight, size_t(K) * dtype_size(weight_dtype)}, {X, x}, {residual, x}};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return W4A16_ERR_ARG;
    for (int j = 0; j < 3; ++j) {
      if (i == 0 && j > 0 && H == in[j].p) continue;  // in place
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return W4A16_ERR_ARG;
    }
  }
  (void)hipGetLastError();
  w4a16::Norm8 p;
  p.X = X;
  p.residual = residual;
  p.weight = weight;
  p.H = H;
  p.Y = Y;
  p.codes = codes;
  p.scales = scales;
  p.M = int(M);
  p.K = int(K);
  p.dtype = dtype;
  p.weight_f32 = weight_dtype == W4A16_DTYPE_F32;
  p.eps = eps;
  return status(w4a16::launch_norm8(p, reinterpret_cast<hipStream_t>(stream)));
}

int w8a8_gemm(const uint8_t *X, const float *xs, const uint8_t *W, const float *ws, void *Y,
              int64_t M, int64_t N, int64_t K, int32_t block, int32_t dtype, void *stream) {
  const int st = gemm_extents(M, M, 1, N, K, block, dtype);
  if (st != W4A16_OK || M == 0 || N == 0) return st;
  return gemm(X, xs, nullptr, nullptr, W, ws, Y, M, M, 1, N, K, dtype, stream);
}

int w8a8_gemm_grouped(const uint8_t *X, const float *xs, const int32_t *token_index,
                      const int32_t *expert_offsets, const uint8_t *W, const float *ws, void *Y,
                      int64_t T, int64_t R, int64_t E, int64_t N, int64_t K, int32_t block,
                      int32_t dtype, void *stream) {
  const int st = gemm_extents(T, R, E, N, K, block, dtype);
  if (st != W4A16_OK || R == 0 || N == 0) return st;
  if (!expert_offsets || T == 0 || (!token_index && T < R)) return W4A16_ERR_ARG;
  return gemm(X, xs, token_index, expert_offsets, W, ws, Y, T, R, E, N, K, dtype, stream);
}

int w8a8_kernel(int64_t R, int64_t E) {
  if (R <= 0 || E < 0 || R > W8A8_MAX_M || E > 65535) return 0;
  return w4a16::gemm8_kernel(long(R), long(E), E > 0);
}

}  // extern "C"
