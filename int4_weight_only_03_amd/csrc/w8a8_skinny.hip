// 8-bit products for few rows: Y[r] = x_r . W_e^T, weights and activations from memory
// to registers.
//
// Arithmetic: e4m3 codes become fp16, exactly; 16x16x32 fp16 matrix instructions with
// fp32 accumulation add up a block of 128 features, and one fp32 FMA per output and
// block applies its scales.  (The fp8 instructions add 8 products at a time in a window
// that ends 13 bits below the largest, and there is nothing to gain from their rate here.)
//
// Mapping: A is 16 rows of W, B 16 slots, so that a lane's 4 sums are neighbouring
// outputs of one slot.  Lane (c, R) (c = lane % 16, R = lane / 16) loads 16 bytes at 16 R
// and at 64 + 16 R of a block of row c of each; any order of k that both operands share
// gives the same sum.  A wave takes 16 MT slots of one expert by 16 NT rows of W, KW
// waves of a workgroup its blocks in turn; their sums are added in wave order in LDS.

#include "w8a8_common.h"

#include <algorithm>

namespace w4a16 {
namespace {

struct SkinnyArgs {
  const uint8_t *X;
  const float *xs;
  const int32_t *token_index, *offsets;
  const uint8_t *W;
  const float *ws;
  void *Y;
  int rows_x, R, E, N, K, KB, NB, tiles_n;
  bool vec;  // rows of Y begin and end at 4 outputs
};

// 8 codes to fp16, exactly
__device__ __forceinline__ half8v widen(uint32_t lo, uint32_t hi) {
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false),
               b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true),
               c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false),
               d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return half8v{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <int MT, int NT, int KW, int P, typename OT>
__global__ void __launch_bounds__(64 * KW) gemm8_skinny(SkinnyArgs a) {
  __shared__ f32x4 part[KW > 1 ? KW : 1][MT * NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, R = lane >> 4;
  const int item = blockIdx.x / unsigned(a.tiles_n), tile = blockIdx.x % unsigned(a.tiles_n);
  int e = 0, row0 = item * 16 * MT, rows = std::min(16 * MT, a.R - row0);
  if (a.offsets) {
    const ExpertItem it = find_item(a.offsets, a.E, a.R, 16 * MT, item);
    if (it.e < 0) return;  // uniform over the workgroup
    e = it.e;
    row0 = it.row0;
    rows = it.rows;
  }
  const int n0 = tile * 16 * NT;
  const long K = a.K;

  const uint8_t *wrow[NT], *xrow[MT];
  const float *xscale[MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    wrow[n] = a.W + (long(e) * a.N + std::min(n0 + 16 * n + c, a.N - 1)) * K;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int slot = row0 + std::min(16 * m + c, rows - 1);
    long row = slot;
    if (a.token_index) row = std::min(std::max(a.token_index[slot], 0), a.rows_x - 1);
    xrow[m] = a.X + row * K;
    xscale[m] = a.xs + row * a.KB;
  }
  const float *wscale = a.ws + (long(e) * a.NB + n0 / kBlock8) * a.KB;

  struct Step {
    u32x4m w[NT][2], x[MT][2];
    float s[MT], t;
  };
  auto load = [&](Step &s, int b) {
    const int k0 = kBlock8 * b + 16 * R, k1 = k0 + 64;
    // behind the row's end its last 16 bytes are read, and zeros taken
    const int at0 = std::min(k0, a.K - 16), at1 = std::min(k1, a.K - 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s.w[n][0] = *reinterpret_cast<const u32x4m *>(wrow[n] + at0);
      s.w[n][1] = *reinterpret_cast<const u32x4m *>(wrow[n] + at1);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      s.x[m][0] = *reinterpret_cast<const u32x4m *>(xrow[m] + at0);
      s.x[m][1] = *reinterpret_cast<const u32x4m *>(xrow[m] + at1);
      s.s[m] = xscale[m][b];
    }
    s.t = wscale[b];
  };
  f32x4 acc[MT][NT];
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = zero;
  auto multiply = [&](Step &s, int b) {
    if (kBlock8 * (b + 1) > a.K) {
      const u32x4m none = {0, 0, 0, 0};
      const int k0 = kBlock8 * b + 16 * R, k1 = k0 + 64;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s.w[n][0] = k0 < a.K ? s.w[n][0] : none;
        s.w[n][1] = k1 < a.K ? s.w[n][1] : none;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        s.x[m][0] = k0 < a.K ? s.x[m][0] : none;
        s.x[m][1] = k1 < a.K ? s.x[m][1] : none;
      }
    }
    half8v w[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) w[n][j] = widen(s.w[n][j / 2][2 * (j & 1)], s.w[n][j / 2][2 * (j & 1) + 1]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      half8v x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = widen(s.x[m][j / 2][2 * (j & 1)], s.x[m][j / 2][2 * (j & 1) + 1]);
      const float f = s.s[m] * s.t;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 d = zero;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[n][j], x[j], d, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = fmaf(f, d[i], acc[m][n][i]);
      }
    }
  };

  Step step[P];
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (wave + p * KW < a.KB) load(step[p], wave + p * KW);
  for (int b = wave; b < a.KB; b += P * KW) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = b + p * KW;
      if (at < a.KB) multiply(step[p], at);
      if (at + P * KW < a.KB) load(step[p], at + P * KW);
    }
  }

  auto store = [&](int m, int n, f32x4 v) {
    const int i = 16 * m + c, at = n0 + 16 * n + 4 * R;
    if (i >= rows) return;
    OT *y = static_cast<OT *>(a.Y) + long(row0 + i) * a.N + at;
    if (a.vec) {
      struct alignas(4 * sizeof(OT)) Four {
        OT v[4];
      };
      if (at < a.N)
        *reinterpret_cast<Four *>(y) =
            Four{{from_f32<OT>(v[0]), from_f32<OT>(v[1]), from_f32<OT>(v[2]), from_f32<OT>(v[3])}};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (at + q < a.N) y[q] = from_f32<OT>(v[q]);
    }
  };
  if constexpr (KW == 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) store(m, n, acc[m][n]);
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) part[wave][m * NT + n][lane] = acc[m][n];
    __syncthreads();
    for (int i = wave; i < MT * NT; i += KW) {
      f32x4 v = part[0][i][lane];
#pragma unroll
      for (int w = 1; w < KW; ++w) v += part[w][i][lane];
      store(i / NT, i % NT, v);
    }
  }
}

template <int MT, int NT, int KW, int P, typename OT>
hipError_t run_skinny(const Gemm8 &p, hipStream_t stream) {
  SkinnyArgs a;
  a.X = p.X;
  a.xs = p.xs;
  a.token_index = p.token_index;
  a.offsets = p.expert_offsets;
  a.W = p.W;
  a.ws = p.ws;
  a.Y = p.Y;
  a.rows_x = p.rows_x;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.K = p.K;
  a.KB = blocks8(p.K);
  a.NB = blocks8(p.N);
  a.tiles_n = (p.N + 16 * NT - 1) / (16 * NT);
  a.vec = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.Y) % (4 * sizeof(OT)) == 0;
  const long items = p.expert_offsets ? max_items(p.R, p.E, 16 * MT) : (long(p.R) + 16 * MT - 1) / (16 * MT);
  const long blocks = items * a.tiles_n;
  if (blocks > kMaxBlocks * 4 / KW) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm8_skinny<MT, NT, KW, P, OT>), dim3(unsigned(blocks)), dim3(64 * KW), 0,
                     stream, a);
  return hipGetLastError();
}

template <typename OT>
hipError_t run_skinny_type(const Gemm8 &p, hipStream_t stream) {
  // Waves of a tile and rows of W by whether the workgroups are many (us with 8 waves and 16
  // rows, 4 and 32: 1 row of 4096 x 7168 7.1, 10.8; 244 slots of 60 experts of 2080 x 1408
  // 56.8, 36.0; 64 of 32 experts of 4096 x 7168 159, 156).
  return p.expert_offsets ? run_skinny<1, 2, 4, 2, OT>(p, stream)
                          : run_skinny<1, 1, 8, 2, OT>(p, stream);
}

}  // namespace

hipError_t launch_gemm8_skinny(const Gemm8 &p, hipStream_t stream) {
  switch (p.dtype) {
    case W4A16_DTYPE_F32: return run_skinny_type<float>(p, stream);
    case W4A16_DTYPE_F16: return run_skinny_type<_Float16>(p, stream);
    default: return run_skinny_type<Bf16>(p, stream);
  }
}

}  // namespace w4a16
