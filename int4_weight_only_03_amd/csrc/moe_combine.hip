// Combination of an MoE layer's routed slots into its tokens:
// Y[t][n] = sum_j weights[t][j] * D[slots[t][j]][n], D the experts' down
// projections in fp32 (not rounded before the sum), the terms added in order
// of j in fp32 and rounded once.  Slots below 0 (places no expert took) add
// nothing; a token without experts becomes 0.
//
// Bound by reading D (16384 slots of 7168 columns into 4096 tokens: 104 us, 5.1
// TB/s with what is written, a plain copy's rate).

#include "moe_common.h"

#include <algorithm>

namespace w4a16 {
namespace {

constexpr int kCbThreads = 256;

// A workgroup takes 4 * kCbThreads columns of one token, a thread 4 of them.
// ldd is a multiple of 4; kVec: so is N, and Y's rows are aligned to 4 values.
template <typename YT, bool kVec>
__global__ void __launch_bounds__(kCbThreads)
combine_slots(const float *__restrict__ D, const int32_t *__restrict__ slots,
              const float *__restrict__ weights, YT *__restrict__ Y, int topk, int R, int N,
              int ldd, int blocks_n) {
  const long t = blockIdx.x / unsigned(blocks_n);
  const int n = int(blockIdx.x % unsigned(blocks_n)) * 4 * kCbThreads + 4 * int(threadIdx.x);
  if (n >= N) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < topk; ++j) {
    const int slot = slots[t * topk + j];
    if (slot < 0) continue;
    const float w = weights[t * topk + j];
    const float4 d = *reinterpret_cast<const float4 *>(D + long(std::min(slot, R - 1)) * ldd + n);
    v[0] = fmaf(w, d.x, v[0]);
    v[1] = fmaf(w, d.y, v[1]);
    v[2] = fmaf(w, d.z, v[2]);
    v[3] = fmaf(w, d.w, v[3]);
  }
  YT *y = Y + t * N + n;
  if constexpr (kVec) {
    struct alignas(4 * sizeof(YT)) Four {
      YT v[4];
    };
    *reinterpret_cast<Four *>(y) =
        Four{{from_f32<YT>(v[0]), from_f32<YT>(v[1]), from_f32<YT>(v[2]), from_f32<YT>(v[3])}};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) y[i] = from_f32<YT>(v[i]);
  }
}

template <typename YT>
hipError_t run_combine(const float *D, const int32_t *slots, const float *weights, void *Y, int T,
                       int topk, int R, int N, int ldd, hipStream_t stream) {
  const int blocks_n = (N + 4 * kCbThreads - 1) / (4 * kCbThreads);
  const long blocks = long(T) * blocks_n;
  if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
  YT *y = static_cast<YT *>(Y);
  if (N % 4 == 0 && reinterpret_cast<uintptr_t>(Y) % (4 * sizeof(YT)) == 0)
    hipLaunchKernelGGL((combine_slots<YT, true>), dim3(unsigned(blocks)), dim3(kCbThreads), 0,
                       stream, D, slots, weights, y, topk, R, N, ldd, blocks_n);
  else
    hipLaunchKernelGGL((combine_slots<YT, false>), dim3(unsigned(blocks)), dim3(kCbThreads), 0,
                       stream, D, slots, weights, y, topk, R, N, ldd, blocks_n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine(const float *D, const int32_t *slots, const float *weights, void *Y,
                          int T, int topk, int R, int N, int ldd, int dtype, hipStream_t stream) {
  switch (dtype) {
    case W4A16_DTYPE_F32:
      return run_combine<float>(D, slots, weights, Y, T, topk, R, N, ldd, stream);
    case W4A16_DTYPE_F16:
      return run_combine<_Float16>(D, slots, weights, Y, T, topk, R, N, ldd, stream);
    default:
      return run_combine<Bf16>(D, slots, weights, Y, T, topk, R, N, ldd, stream);
  }
}

}  // namespace w4a16
