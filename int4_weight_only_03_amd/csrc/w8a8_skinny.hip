// 8-bit products for few rows: Y[r] = x_r . W_e^T, weights and activations from memory
// to registers.  Bound by HBM where there are many experts (64 slots of 32 experts of 4096 x
// 7168: 940 MB in 155 us, 6.1 TB/s, a stream of reads alone reaches 6.3), by latency for one
// (4096 x 7168: 29 MB in 7.1 us, 2 of them the launch).
//
// Arithmetic: e4m3 codes become fp16, exactly; 16x16x32 fp16 matrix instructions with
// fp32 accumulation add up a block of 128 features, and one fp32 FMA per output and
// block applies its scales.  (The fp8 instructions add 8 products at a time in a window
// that ends 13 bits below the largest, and there is nothing to gain from their rate here.)
//
// Mapping: A is 16 rows of W, B 16 slots, so that a lane's 4 sums are neighbouring
// outputs of one slot.  Lane (c, R) (c = lane % 16, R = lane / 16) loads 16 bytes at 16 R
// and at 64 + 16 R of a block of row c of each; any order of k that both operands share
// gives the same sum.  A wave takes 16 slots of one expert by 16 NT rows of W, KW
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
  int turn;  // blocks that a tile of W begins behind the one before it
  bool vec;  // rows of Y begin and end at 4 outputs
};

constexpr int kSkinnySlots = 16;
constexpr int kSkinnyAhead = 2;  // blocks of a wave in flight (4: 7.6 us for 7.1, one row)

template <int NT, int KW, typename OT>
__global__ void __launch_bounds__(64 * KW) gemm8_skinny(SkinnyArgs a) {
  constexpr int P = kSkinnyAhead;
  __shared__ f32x4 part[KW][NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, R = lane >> 4;
  const int item = blockIdx.x / unsigned(a.tiles_n), tile = blockIdx.x % unsigned(a.tiles_n);
  int e = 0, row0 = item * kSkinnySlots, rows = std::min(kSkinnySlots, a.R - row0);
  if (a.offsets) {
    const ExpertItem it = find_item(a.offsets, a.E, a.R, kSkinnySlots, item);
    if (it.e < 0) return;  // uniform over the workgroup
    e = it.e;
    row0 = it.row0;
    rows = it.rows;
  }
  const int n0 = tile * 16 * NT;
  const long K = a.K;

  const uint8_t *wrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    wrow[n] = a.W + (long(e) * a.N + std::min(n0 + 16 * n + c, a.N - 1)) * K;
  long row = row0 + std::min(c, rows - 1);
  if (a.token_index) row = std::min(std::max(a.token_index[row], 0), a.rows_x - 1);
  const uint8_t *xrow = a.X + row * K;
  const float *xscale = a.xs + row * a.KB;
  const float *wscale = a.ws + (long(e) * a.NB + n0 / kBlock8) * a.KB;

  struct Step {
    u32x4m w[NT][2], x[2];
    float s, t;
  };
  // Rows of 4096 bytes, or a multiple, have their blocks in the same few channels of memory:
  // there tiles begin 2 KB behind each other and go round (64 slots of 32 experts of 4096 x
  // 8192: 229 us, 180 so; of 4096 x 4096 98, 92; 1 row 6.1, 5.7); other lengths need none of it
  // and lose up to 3% (32 experts of 4096 x 2048 46.2, 46.6; of 4096 x 6144 133.8, 134.6; 1 row of
  // the latter 6.6, 6.8).  By the tile of W alone: a slot's sums have the same order whatever
  // other slots there are.
  const int turn = a.turn ? int(unsigned(tile) * unsigned(a.turn) % unsigned(a.KB)) : 0;
  auto block_of = [&](int i) { return i + turn < a.KB ? i + turn : i + turn - a.KB; };
  auto load = [&](Step &s, int i) {
    const int b = block_of(i);
    // behind the row's end its last 16 bytes are read, and zeros taken
    const int at0 = std::min(kBlock8 * b + 16 * R, a.K - 16),
              at1 = std::min(kBlock8 * b + 16 * R + 64, a.K - 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s.w[n][0] = *reinterpret_cast<const u32x4m *>(wrow[n] + at0);
      s.w[n][1] = *reinterpret_cast<const u32x4m *>(wrow[n] + at1);
    }
    s.x[0] = *reinterpret_cast<const u32x4m *>(xrow + at0);
    s.x[1] = *reinterpret_cast<const u32x4m *>(xrow + at1);
    s.s = xscale[b];
    s.t = wscale[b];
  };
  f32x4 acc[NT];
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = zero;
  auto multiply = [&](Step &s, int i) {
    const int b = block_of(i);
    if (kBlock8 * (b + 1) > a.K) {
      const u32x4m none = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (kBlock8 * b + 16 * R + 64 * h < a.K) continue;
        s.x[h] = none;
#pragma unroll
        for (int n = 0; n < NT; ++n) s.w[n][h] = none;
      }
    }
    half8v x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[j] = widen8(s.x[j / 2][2 * (j & 1)], s.x[j / 2][2 * (j & 1) + 1]);
    const float f = s.s * s.t;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 d = zero;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            widen8(s.w[n][j / 2][2 * (j & 1)], s.w[n][j / 2][2 * (j & 1) + 1]), x[j], d, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(f, d[i], acc[n][i]);
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

#pragma unroll
  for (int n = 0; n < NT; ++n) part[wave][n][lane] = acc[n];
  __syncthreads();
  if (wave >= NT || c >= rows) return;
  f32x4 v = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < KW; ++w) v += part[w][wave][lane];
  const int at = n0 + 16 * wave + 4 * R;
  OT *y = static_cast<OT *>(a.Y) + long(row0 + c) * a.N + at;
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
}

template <int NT, int KW, typename OT>
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
  a.turn = p.K % 4096 == 0 ? 2048 / kBlock8 : 0;
  a.vec = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.Y) % (4 * sizeof(OT)) == 0;
  const long items = p.expert_offsets
                         ? max_items(p.R, p.E, kSkinnySlots)
                         : (long(p.R) + kSkinnySlots - 1) / kSkinnySlots;
  const long blocks = items * a.tiles_n;
  if (blocks > kMaxBlocks * 4 / KW) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm8_skinny<NT, KW, OT>), dim3(unsigned(blocks)), dim3(64 * KW), 0,
                     stream, a);
  return hipGetLastError();
}

template <typename OT>
hipError_t run_skinny_type(const Gemm8 &p, hipStream_t stream) {
  // Waves of a tile and rows of W by whether the workgroups are many (us with 8 waves and 16
  // rows, 4 and 32: 1 row of 4096 x 7168 7.1, 10.8; 244 slots of 60 experts of 2080 x 1408
  // 56.8, 36.0; 64 of 32 experts of 4096 x 7168 159, 156).
  return p.expert_offsets ? run_skinny<2, 4, OT>(p, stream)
                          : run_skinny<1, 8, OT>(p, stream);
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
