// Rows to e4m3 with one fp32 scale per 128 values, plain or silu(gate) * up of rows
// [gate | up].
//
// Bound by HBM: 2 or 4 bytes a value read (twice that with swiglu), 1 + 1/32 written.
// 16 lanes take the 128 values of a scale, 8 each (one 16-byte load of 16-bit values):
// its largest magnitude is four DPP steps away, no LDS, no barrier.  32768 x 2 x 2048 in bf16:
// 338 MB in 61 us, 5.5 TB/s (a copy reaches 4.96, a stream of reads 6.3).

#include "w8a8_common.h"

#include <algorithm>

namespace w4a16 {
namespace {

// silu(g) * u = g / (1 + exp(-g)) * u.  exp(x) = 2^(x log2 e): the exponent's rounding (up to
// 2^-17 absolute) is taken out again to first order.  The sum is taken a quarter as large, so
// that its reciprocal is a normal number as long as exp(-g) is one (g > -88.72; below it the
// sum is infinite and the result 0).  v_exp_f32 and v_rcp_f32 are within a unit of 2^-23; the
// correction, the sum and two products add half a unit each: 4 units, 2.0 at most measured.  The
// compiler's expf and division made the kernel bound by VALU (32768 x 2 x 2048 in bf16: 80 us),
// the quotient mended by its remainder takes 67 us for 63.
__device__ __forceinline__ float silu_fast(float g, float u) {
  constexpr float kHigh = 0x1.715476p+0f, kLow = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;
  const float a = __builtin_amdgcn_fmed3f(g, -200.0f, 200.0f);  // e and its product stay finite
  const float p = a * -kHigh;
  const float e = fmaf(a, -kLow, fmaf(a, -kHigh, -p));
  const float x = __builtin_amdgcn_exp2f(p);
  const float d = fmaf(x, fmaf(e, 0.25f * kLn2, 0.25f), 0.25f);  // (1 + exp(-g)) / 4
  return 0.25f * g * __builtin_amdgcn_rcpf(d) * u;
}

constexpr int kRowsThreads = 256;
constexpr int kRowsGroups = kRowsThreads / kLanes8;

template <typename XT, bool kSw>
__global__ void __launch_bounds__(kRowsThreads)
quantize_rows(const XT *__restrict__ X, const int32_t *__restrict__ num_rows,
              uint8_t *__restrict__ codes, float *__restrict__ scales, int M, int K, int KB) {
  const int rows = num_rows ? min(max(*num_rows, 0), M) : M;
  const long total = long(rows) * KB;
  const int at = threadIdx.x / kLanes8;
  const int lane = threadIdx.x % kLanes8;
  for (long first = long(blockIdx.x) * kRowsGroups; first < total;
       first += long(gridDim.x) * kRowsGroups) {
    const long g = first + at;
    if (g >= total) return;  // all 16 lanes of a group
    const long row = (total >> 31) == 0 ? long(uint32_t(g) / uint32_t(KB)) : g / KB;
    const int k = int(g - row * KB) * kBlock8 + 8 * lane;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (k < K) {
      if constexpr (kSw) {
        float u[8];
        load8(X + row * (2 * long(K)) + k, v);
        load8(X + row * (2 * long(K)) + K + k, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = silu_fast(v[i], u[i]);
      } else {
        load8(X + row * K + k, v);
      }
    }
    float s;
    const uint2 c = quantize8(v, s);
    if (k < K) *reinterpret_cast<uint2 *>(codes + row * K + k) = c;
    if (lane == 0) scales[g] = s;
  }
}

template <typename XT>
hipError_t run_rows(const Rows8 &p, hipStream_t stream) {
  const int KB = blocks8(p.K);
  const long blocks = std::min((long(p.M) * KB + kRowsGroups - 1) / kRowsGroups, kMaxBlocks);
  const XT *X = static_cast<const XT *>(p.X);
  if (p.swiglu)
    hipLaunchKernelGGL((quantize_rows<XT, true>), dim3(unsigned(blocks)), dim3(kRowsThreads), 0,
                       stream, X, p.num_rows, p.codes, p.scales, p.M, p.K, KB);
  else
    hipLaunchKernelGGL((quantize_rows<XT, false>), dim3(unsigned(blocks)), dim3(kRowsThreads), 0,
                       stream, X, p.num_rows, p.codes, p.scales, p.M, p.K, KB);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows8(const Rows8 &p, hipStream_t stream) {
  switch (p.dtype) {
    case W4A16_DTYPE_F32: return run_rows<float>(p, stream);
    case W4A16_DTYPE_F16: return run_rows<_Float16>(p, stream);
    default: return run_rows<Bf16>(p, stream);
  }
}

}  // namespace w4a16
