// Experts' W4A16 products for many slots per expert (prompts): the products of
// moe_skinny.hip in 128 x 128 tiles on the fp16 matrix instructions.
//
// The activations come as fp16 limbs that moe_limbs.hip makes in the workspace,
// once for all the tiles that read them: one limb for fp16 and bf16, two for
// fp32.
//
// The tile kernel: v_mfma_f32_16x16x32_f16 on limbs and the exact codes q - 8
// (K: one group of 32; every product exact in fp32), one fp32 FMA per output
// and group for the scale, the row's power of two undone at the store.  A
// workgroup takes 128 slots of one expert by 128 rows of W (gate/up form: 64
// gate rows and the up rows of the same outputs, so that both sums of an
// output lie in one lane); wave (wm, wn) of its 4 waves 64 x 64 of them.
//
// Per stage of two groups: the limbs come to LDS by direct copies (gathered
// rows, 128 bytes each), the weight words through registers, converted once
// per workgroup into an LDS image of codes; both images are double buffered
// and a stage has one barrier.  While a stage's products run, the next stage's
// copies fly and its codes are converted.
//
// Tiles are dealt so that each XCD works a contiguous run of them (the
// hardware deals workgroups round-robin over the 8 XCDs), row blocks of an
// expert fastest: the tiles an XCD holds at once share weight rows and slots.
//
// Bound: VALU issue.  Per stage and wave 32 L matrix instructions (16 cycles
// each; L limbs) against 128 FMAs for the scales, 36 for the conversion and
// about 30 others of 4 cycles.

#include "moe_common.h"
#include "gemv_common.h"
#include "limbs.h"

#include <algorithm>

namespace w4a16 {
namespace {

typedef __attribute__((address_space(3))) void et_lds_void;

constexpr int kEtThreads = 256;

__device__ __forceinline__ void et_wait_vm0() {
  __builtin_amdgcn_s_waitcnt(0x70 | (15 << 8));  // vmcnt(0)
}
__device__ __forceinline__ void et_wait_lgkm0() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | 0x70);  // lgkmcnt(0)
}
// Direct copy of 16 bytes per lane, lane i to lds + 16 i; as asm so that the
// compiler does not wait for it at every LDS read (the kernel's own waits and
// barriers order the copies).  The LDS address is wave-uniform (m0).
__device__ __forceinline__ void et_copy16(const void *src, const void *lds) {
  const uint32_t at = uint32_t(reinterpret_cast<uintptr_t>((const et_lds_void *)lds));
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 1\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(src), "s"(at) : "memory", "m0");
}
__device__ __forceinline__ void et_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

struct TileArgs {
  const _Float16 *limbs;
  const float *factor;
  const int32_t *token_index, *offsets;
  const unsigned char *qw;
  const float *sc;
  void *Y;
  int rows_x, R, E, N, G, KP, ldy, tiles_n;
};

// L limbs, OT the output type (kSw: the activations' type, else fp32)
template <int L, typename OT, bool kSw>
__global__ void __launch_bounds__(kEtThreads, L == 1 ? 2 : 1) experts_tile(TileArgs a) {
  // Images of a stage (64 k): row r at 128 r, logical chunk x (16 bytes: 8
  // values of one group's block x % 4, group x / 4) at chunk x ^ ((r / 2) % 8),
  // so that the 16 rows an operand read touches fall in distinct banks.
  __shared__ __align__(16) unsigned char et_a0[L * 16384];
  __shared__ __align__(16) unsigned char et_a1[L * 16384];
  __shared__ __align__(16) unsigned char et_c0[16384];
  __shared__ __align__(16) unsigned char et_c1[16384];
  __shared__ __align__(16) float et_s0[256];  // scales: row n, group q at 2 n + q
  __shared__ __align__(16) float et_s1[256];
  constexpr int NO = kSw ? 64 : 128;  // outputs per tile
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int c = lane & 15, R = lane >> 4;
  const int G = a.G, N = a.N;

  // tile of this workgroup: XCD b % 8 takes a contiguous run of the tiles
  // there are; within an expert its row blocks are fastest
  ExpertItem it = find_item(a.offsets, a.E, a.R, 128, 0);
  const long tiles = long(it.total) * a.tiles_n;
  const long run = (tiles + 7) / 8;
  const long index = long(blockIdx.x >> 3);
  const long tile = long(blockIdx.x & 7) * run + index;
  if (index >= run || tile >= tiles) return;  // uniform over the workgroup
  it = find_item(a.offsets, a.E, a.R, 128, int(tile / a.tiles_n));
  // tiles of this expert: it.blocks x tiles_n, from item (its first block) on
  const long first = (tile / a.tiles_n - it.block) * a.tiles_n;
  const int within = int(tile - first);
  const int bm = within % it.blocks, bn = within / it.blocks;
  int e0, e1;
  expert_slots(a.offsets, it.e, a.R, e0, e1);
  const int row0 = e0 + bm * 128, rows = std::min(128, e1 - row0);
  const int n0 = bn * NO;

  // Limb copies: copy j (wave w issues j = 4w .. 4w+3 of each limb): lane i
  // writes 16 B at 1024 j + 16 i: row 8 j + i / 8, chunk i % 8, which holds
  // logical chunk (i % 8) ^ ((row / 2) % 8).  Rows past the item repeat its last.
  const unsigned char *asrc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 8 * (4 * wave + j) + lane / 8;
    const int slot = row0 + std::min(r, rows - 1);
    long row = slot;
    if (a.token_index) row = std::min(std::max(a.token_index[slot], 0), a.rows_x - 1);
    asrc[j] = reinterpret_cast<const unsigned char *>(a.limbs + row * a.KP) +
              16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  const long plane = long(a.rows_x) * a.KP * 2;
  auto copy_stage = [&](unsigned char *img, int p) {
#pragma unroll
    for (int l = 0; l < L; ++l)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        et_copy16(asrc[j] + l * plane + long(p) * 128, img + 16384 * l + 1024 * (4 * wave + j));
  };
  // Weights: thread t takes image row t / 2, group t % 2 of each stage.  Gate/up
  // form: image rows 64 wn + 0..31 are gate rows of outputs 32 wn .. +31, rows
  // 64 wn + 32..63 the up rows of the same.  Rows past N read row N - 1.
  const int cr = tid >> 1, ch = tid & 1;
  long wrow;
  if constexpr (kSw)
    wrow = std::min(n0 + 32 * (cr >> 6) + (cr & 31), N - 1) + ((cr & 32) ? long(N) : 0);
  else
    wrow = std::min(n0 + cr, N - 1);
  wrow += long(it.e) * (kSw ? 2 * long(N) : long(N));
  const unsigned char *wsrc = a.qw + wrow * G * 16;
  const float *ssrc = a.sc + wrow * G;
  const int P = (G + 1) / 2;
  struct W {
    u32x4m w;
    float s;
  };
  auto load_w = [&](int p) -> W {
    const int g = 2 * p + ch, gc = std::min(g, G - 1);
    W v;
    v.w = *reinterpret_cast<const u32x4m *>(wsrc + long(gc) * 16);
    v.s = g < G ? ssrc[gc] : 0.0f;  // behind the last group the limbs are 0 too
    return v;
  };
  uint32_t cwrite[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cwrite[i] = uint32_t(cr * 128 + 16 * ((4 * ch + i) ^ ((cr >> 1) & 7)));
  auto convert = [&](const W &v, unsigned char *cimg, float *simg) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<half8_t *>(cimg + cwrite[i]) = nibbles_to_f16(v.w[i]);
    simg[tid] = v.s;
  };

  // operand reads: limbs of row 64 wm + 16 u + c at aread[q] + 2048 u, codes of
  // image row 64 wn + 16 t + c at cread[q] + 2048 t
  uint32_t aread[2], cread[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int ra = 64 * wm + c, rc = 64 * wn + c;
    aread[q] = uint32_t(ra * 128 + 16 * ((4 * q + R) ^ ((ra >> 1) & 7)));
    cread[q] = uint32_t(rc * 128 + 16 * ((4 * q + R) ^ ((rc >> 1) & 7)));
  }
  float acc[4][4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[u][t][r] = 0.0f;
  const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  auto products = [&](const unsigned char *img, const unsigned char *cimg, const float *simg) {
    float2 s[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      s[t] = *reinterpret_cast<const float2 *>(simg + 2 * (64 * wn + 16 * t + c));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      half8_t x[L][4], b[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) b[t] = *reinterpret_cast<const half8_t *>(cimg + cread[q] + 2048 * t);
#pragma unroll
      for (int l = 0; l < L; ++l)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          x[l][u] = *reinterpret_cast<const half8_t *>(img + 16384 * l + aread[q] + 2048 * u);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          floatx4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[0][u], b[t], zero, 0, 0, 0);
          if constexpr (L == 2)
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[L - 1][u], b[t], d, 0, 0, 0);
          const float sq = q == 0 ? s[t].x : s[t].y;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[u][t][r] = fmaf(sq, d[r], acc[u][t][r]);
        }
    }
  };

  copy_stage(et_a0, 0);
  {
    const W w0 = load_w(0);
    convert(w0, et_c0, et_s0);
  }
  W next = load_w(std::min(1, P - 1));
  // Two stages per iteration (images by p % 2).  At a stage's start its copies
  // have landed in this wave and its codes are written; past the barrier that
  // holds for every wave, and every wave is past the stage before, whose images
  // are then filled again.
  for (int pb = 0; pb < P; pb += 2) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int p = pb + v;
      if (p < P) {
        et_wait_vm0();
        et_wait_lgkm0();
        et_barrier();
        if (p + 1 < P) copy_stage(v ? et_a0 : et_a1, p + 1);
        const W w = next;
        next = load_w(std::min(p + 2, P - 1));
        if (p + 1 < P) convert(w, v ? et_c0 : et_c1, v ? et_s0 : et_s1);
        products(v ? et_a1 : et_a0, v ? et_c1 : et_c0, v ? et_s1 : et_s0);
      }
    }
  }

  OT *y = static_cast<OT *>(a.Y);
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 64 * wm + 16 * u + 4 * R + r;
      if (m >= rows) continue;
      const int slot = row0 + m;
      long row = slot;
      if (a.token_index) row = std::min(std::max(a.token_index[slot], 0), a.rows_x - 1);
      const float f = a.factor[row];
      const long at = long(slot) * a.ldy;
      if constexpr (kSw) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int n = n0 + 32 * wn + 16 * t + c;
          if (n < N) y[at + n] = from_f32<OT>(silu_mul(acc[u][t][r] * f, acc[u][t + 2][r] * f));
        }
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int n = n0 + 64 * wn + 16 * t + c;
          if (n < N) y[at + n] = from_f32<OT>(acc[u][t][r] * f);
        }
      }
    }
}

template <typename XT, bool kSw>
hipError_t run_tile(const MoeExperts &p, hipStream_t stream) {
  using OT = typename std::conditional<kSw, XT, float>::type;
  constexpr int L = sizeof(XT) == 4 ? 2 : 1;
  const LimbLayout at = limb_layout(p.workspace, p.rows_x, p.K, p.dtype);
  TileArgs a;
  a.KP = at.KP;
  a.limbs = at.limbs;
  a.factor = at.factor;
  a.token_index = p.token_index;
  a.offsets = p.expert_offsets;
  a.qw = reinterpret_cast<const unsigned char *>(p.qweight);
  a.sc = p.scales;
  a.Y = p.Y;
  a.rows_x = p.rows_x;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.G = p.K / kGroup;
  a.ldy = p.ldy;
  a.tiles_n = (p.N + (kSw ? 64 : 128) - 1) / (kSw ? 64 : 128);
  const long tiles = long(a.tiles_n) * max_items(p.R, p.E, 128);
  if (tiles < 1 || tiles > 0x7ffffff0L) return hipErrorInvalidValue;
  const hipError_t e = launch_limbs(p, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((experts_tile<L, OT, kSw>), dim3(unsigned((tiles + 7) / 8 * 8)),
                     dim3(kEtThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename XT>
hipError_t run_tile_type(const MoeExperts &p, hipStream_t stream) {
  return p.swiglu ? run_tile<XT, true>(p, stream) : run_tile<XT, false>(p, stream);
}

}  // namespace

int experts_kernel(long R, long E) {
  const long active = std::max(1L, std::min(R, E));
  return R >= 64 * active ? W4A16_EXPERTS_TILE : W4A16_EXPERTS_SKINNY;
}

size_t experts_workspace_bytes(long rows_x, long R, long E, int K, int dtype) {
  // the skinny kernel takes 16-bit activations as they are
  if (experts_kernel(R, E) != W4A16_EXPERTS_TILE && dtype != W4A16_DTYPE_F32) return 0;
  return limb_bytes(rows_x, K, dtype);
}

hipError_t launch_experts_tile(const MoeExperts &p, hipStream_t stream) {
  switch (p.dtype) {
    case W4A16_DTYPE_F32: return run_tile_type<float>(p, stream);
    case W4A16_DTYPE_F16: return run_tile_type<_Float16>(p, stream);
    default: return run_tile_type<Bf16>(p, stream);
  }
}

hipError_t launch_experts(const MoeExperts &p, hipStream_t stream) {
  return experts_kernel(p.R, p.E) == W4A16_EXPERTS_TILE ? launch_experts_tile(p, stream)
                                                       : launch_experts_skinny(p, stream);
}

}  // namespace w4a16
