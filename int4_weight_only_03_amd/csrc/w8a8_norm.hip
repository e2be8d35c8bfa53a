// Residual addition, RMS norm and rows to e4m3 in one pass:
//     h = x + r,  y = h * w / sqrt(mean(h^2) + eps),  y to e4m3 by groups of 128.
//
// Bound by HBM (x, r read, H, Y, codes written, each once): a row stays in registers,
// 8 neighbouring values to a lane and vector, so that the 128 values of a scale are in
// 16 neighbouring lanes; its sum of squares meets in LDS once.  4096 x 7168 in bf16 with all
// outputs: 265 MB in 56.5 us, 4.7 TB/s of the 4.96 that a copy reaches; a single row 3.3 us.

#include "w8a8_common.h"
#include "gemv_common.h"

#include <algorithm>

namespace w4a16 {
namespace {

struct NormArgs {
  const void *X, *residual, *weight;
  void *H, *Y;
  uint8_t *codes;
  float *scales;
  int M, K, KB;
  bool weight_f32;
  float eps;
};

// sum / largest over the TPR threads of a row, in all of them; `lds`: one word a wave.
// TPR = 64: a wave of its own, no LDS.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *lds) {
  v = segment_sum<64>(v);
  v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += lds[i];
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_most(uint32_t v, float *lds) {
  v = row_max(v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, uint32_t(__builtin_amdgcn_readlane(int(v), 16 * i)));
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = __uint_as_float(m);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) m = max(m, __float_as_uint(lds[i]));
  }
  return m;
}

// TPR threads a row, V vectors of 8 values each.  A workgroup of 64 threads a row takes
// 4 rows.
template <typename XT, int TPR, int V>
__global__ void __launch_bounds__(TPR == 64 ? 256 : TPR)
rms_norm_rows(NormArgs a) {
  constexpr int kWaves = TPR / 64;
  __shared__ float lds[3 * kWaves];
  const int t = threadIdx.x % TPR;
  const long row = TPR == 64 ? long(blockIdx.x) * 4 + (threadIdx.x >> 6) : long(blockIdx.x);
  if (row >= a.M) return;  // TPR = 64: whole waves, which meet no barrier
  const int K = a.K;
  const XT *x = static_cast<const XT *>(a.X) + row * K;
  const XT *r = static_cast<const XT *>(a.residual) + row * K;
  float h[V][8];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int k = 8 * (t + j * TPR);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = 0.0f;
    if (k < K) load8(x + k, h[j]);
  }
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int k = 8 * (t + j * TPR);
      if (k < K) {
        float v[8];
        load8(r + k, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] += v[i];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(h[j][i], h[j][i], sum);
  if (a.H) {
    XT *o = static_cast<XT *>(a.H) + row * K;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int k = 8 * (t + j * TPR);
      if (k < K) store8(o + k, h[j]);
    }
  }
  sum = row_sum<TPR>(sum, lds);
  // 2^e scales the row where its squares or their sum with eps leave fp32's range, or come so
  // near its least (their sum, or eps) that bits of it are lost
  float factor;
  if (!(sum < 0x1p127f) || a.eps >= 0x1p126f ||
      (sum < 0x1p-60f && a.eps < 0x1p-60f)) {  // the same in all lanes
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(h[j][i]) & 0x7fffffffu);
    m = row_most<TPR>(m, lds + kWaves);
    if (m >= 0x7f800000u) {
      factor = m > 0x7f800000u ? __uint_as_float(m) : 0.0f;  // NaN, or 1 / infinity
    } else {
      // |h| < 2^e, and eps 2^-2e no larger than 4
      const int most = m == 0 ? -149 : ilogbf(__uint_as_float(m)) + 1;
      const int e = max(most, ilogbf(a.eps) / 2);
      sum = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[j][i] = ldexpf(h[j][i], -e);
          sum = fmaf(h[j][i], h[j][i], sum);
        }
      sum = row_sum<TPR>(sum, lds + 2 * kWaves);
      factor = 1.0f / sqrtf(sum / float(K) + ldexpf(a.eps, -2 * e));
    }
  } else {
    factor = 1.0f / sqrtf(sum / float(K) + a.eps);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int k = 8 * (t + j * TPR);
    if (k - 8 * (t % kLanes8) >= K) continue;  // the whole group is behind the row
    float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (k < K) {
      if (a.weight_f32)
        load8(static_cast<const float *>(a.weight) + k, y);
      else
        load8(static_cast<const XT *>(a.weight) + k, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[j][i] * factor * y[i];
      if (a.Y) store8(static_cast<XT *>(a.Y) + row * K + k, y);
    }
    if (a.codes) {
      float s;
      const uint2 c = quantize8(y, s);
      if (k < K) *reinterpret_cast<uint2 *>(a.codes + row * K + k) = c;
      if (t % kLanes8 == 0) a.scales[row * a.KB + k / kBlock8] = s;
    }
  }
}

template <typename XT, int TPR, int V>
hipError_t run_norm_with(const NormArgs &a, hipStream_t stream) {
  const long blocks = TPR == 64 ? (long(a.M) + 3) / 4 : long(a.M);
  constexpr int threads = TPR == 64 ? 256 : TPR;
  if (blocks > kMaxBlocks * 256 / threads) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((rms_norm_rows<XT, TPR, V>), dim3(unsigned(blocks)), dim3(threads), 0, stream,
                     a);
  return hipGetLastError();
}

template <typename XT>
hipError_t run_norm(const NormArgs &a, hipStream_t stream) {
  // few rows: one vector a thread (us with 256 threads of 4 vectors, with 1024 of one; bf16, K =
  // 7168: 1 row 4.9, 3.2; 256 6.5, 4.5; 512 8.7, 7.5; 1024 11.4, 11.5; K = 2080, where three
  // quarters of the 1024 have nothing: 1 row 3.5, 2.9; 256 4.0, 3.5; 512 4.35, 4.25)
  if (a.M <= 512 && a.K > 256 && a.K <= 8192)
    return a.K <= 2048 ? run_norm_with<XT, 256, 1>(a, stream)
                       : run_norm_with<XT, 1024, 1>(a, stream);
  if (a.K <= 2048) return run_norm_with<XT, 64, 4>(a, stream);
  if (a.K <= 8192) return run_norm_with<XT, 256, 4>(a, stream);
  return run_norm_with<XT, 1024, 4>(a, stream);
}

}  // namespace

hipError_t launch_norm8(const Norm8 &p, hipStream_t stream) {
  NormArgs a;
  a.X = p.X;
  a.residual = p.residual;
  a.weight = p.weight;
  a.H = p.H;
  a.Y = p.Y;
  a.codes = p.codes;
  a.scales = p.scales;
  a.M = p.M;
  a.K = p.K;
  a.KB = blocks8(p.K);
  a.weight_f32 = p.weight_f32;
  a.eps = p.eps;
  switch (p.dtype) {
    case W4A16_DTYPE_F32: return run_norm<float>(a, stream);
    case W4A16_DTYPE_F16: return run_norm<_Float16>(a, stream);
    default: return run_norm<Bf16>(a, stream);
  }
}

}  // namespace w4a16
