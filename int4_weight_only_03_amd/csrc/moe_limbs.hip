// fp16 limbs of the activations of the experts' products, made once in the
// workspace for all the workgroups that read them.
//
// A row is scaled by a power of two (its largest magnitude into [2^14, 2^15);
// fp16 rows stay as they are) and kept as one limb (fp16, bf16: exact for every
// value within 2^-28 of its row's largest) or two (fp32: hi = f16(x'), lo =
// f16((x' - hi) 2^11), 22 significant bits down to 2^-28 of the row's largest,
// below that an absolute error under 2^-50 of it: without the 2^11 the low limb
// would reach fp16's subnormals, 2^-39 of it, and rows that span 2^26 the end of
// the tolerance).  Each 8 values are stored in the order of the nibble conversion,
// x0 x4 x1 x5 x2 x6 x3 x7.
//
// Layout: limb plane l of row t at (l * rows + t) * KP fp16 values, KP = K
// rounded up to 64 (zeros behind K), then one fp32 factor 2^-e per row.
//
// Bound by reading the rows once (their second pass is served by the caches)
// and, for a few rows, by launch latency.

#include "moe_common.h"
#include "limbs.h"

#include <algorithm>

namespace w4a16 {
namespace {

__device__ __forceinline__ void read8(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void read8(const _Float16 *p, float (&v)[8]) {
  const half8_t a = *reinterpret_cast<const half8_t *>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = float(a[i]);
}
__device__ __forceinline__ void read8(const Bf16 *p, float (&v)[8]) {
  const u32x4m a = *reinterpret_cast<const u32x4m *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}

// A workgroup of NTHR threads takes every gridDim.x-th row.  A thread's first 8
// values stay in registers between the two passes, the others are read again.
template <typename XT, int NTHR>
__global__ void __launch_bounds__(NTHR)
experts_limbs(const XT *__restrict__ X, _Float16 *__restrict__ limbs, float *__restrict__ factor,
              int rows, int K, int KP) {
  __shared__ float part[NTHR / 64];
  const int tid = threadIdx.x;
  for (long t = blockIdx.x; t < rows; t += gridDim.x) {
    const XT *x = X + t * K;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (8 * tid < K) read8(x + 8 * tid, v);
    int e = 0;
    if constexpr (!__is_same(XT, _Float16)) {
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[i]));
      for (int k = 8 * (tid + NTHR); k < K; k += 8 * NTHR) {
        float u[8];
        read8(x + k, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(u[i]));
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
      if ((tid & 63) == 0) part[tid >> 6] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NTHR / 64; ++i) mx = fmaxf(mx, part[i]);
      e = std::min(row_exponent(mx), 149);  // 2^-149 is the least fp32 number
      __syncthreads();  // before the next row's parts
    }
    if (tid == 0) factor[t] = ldexpf(1.0f, -e);
    _Float16 *hi = limbs + t * KP, *lo = hi + long(rows) * KP;
    for (int k = 8 * tid; k < KP; k += 8 * NTHR) {
      if (k >= 8 * NTHR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (k < K) read8(x + k, v);
      }
      half8_t h, l;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = (i >> 1) + 4 * (i & 1);  // x0 x4 x1 x5 x2 x6 x3 x7
        const float s = ldexpf(v[j], e);
        h[i] = _Float16(s);
        l[i] = _Float16((s - float(h[i])) * kLowScale);
      }
      *reinterpret_cast<half8_t *>(hi + k) = h;
      if constexpr (sizeof(XT) == 4) *reinterpret_cast<half8_t *>(lo + k) = l;
    }
  }
}

template <typename XT, int NTHR>
hipError_t run_limbs(const MoeExperts &p, hipStream_t stream) {
  const LimbLayout at = limb_layout(p.workspace, p.rows_x, p.K, p.dtype);
  const long grid = std::min(long(p.rows_x), (1L << 32) / NTHR - 8);
  hipLaunchKernelGGL((experts_limbs<XT, NTHR>), dim3(unsigned(grid)), dim3(NTHR), 0, stream,
                     static_cast<const XT *>(p.X), at.limbs, at.factor, p.rows_x, p.K, at.KP);
  return hipGetLastError();
}

template <typename XT>
hipError_t run_limbs_row(const MoeExperts &p, hipStream_t stream) {
  // Threads by the row's length (fp32, us with 256 and 1024; 16 rows of 7168: 4.6,
  // 3.7; 4096 rows of 7168: 48.6, 37.2, of 4096: 25.4, 26.4, of 2048: 11.6, 17.2).
  return p.K > 4096 ? run_limbs<XT, 1024>(p, stream) : run_limbs<XT, 256>(p, stream);
}

}  // namespace

LimbLayout limb_layout(void *workspace, long rows, int K, int dtype) {
  LimbLayout at;
  at.KP = (K + 63) / 64 * 64;
  at.limbs = static_cast<_Float16 *>(workspace);
  at.factor = reinterpret_cast<float *>(at.limbs + size_t(dtype == W4A16_DTYPE_F32 ? 2 : 1) *
                                                       size_t(rows) * size_t(at.KP));
  return at;
}

size_t limb_bytes(long rows, int K, int dtype) {
  const size_t KP = size_t(K + 63) / 64 * 64;
  return (size_t(rows) * KP * (dtype == W4A16_DTYPE_F32 ? 4 : 2) + size_t(rows) * 4 + 255) / 256 *
         256;
}

hipError_t launch_limbs(const MoeExperts &p, hipStream_t stream) {
  switch (p.dtype) {
    case W4A16_DTYPE_F32: return run_limbs_row<float>(p, stream);
    case W4A16_DTYPE_F16: return run_limbs_row<_Float16>(p, stream);
    default: return run_limbs_row<Bf16>(p, stream);
  }
}

}  // namespace w4a16
