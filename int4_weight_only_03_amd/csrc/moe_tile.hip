// Experts' W4A16 products for many slots per expert (prompts): the products of
// moe_skinny.hip in tiles of up to 128 slots by 256 rows on the fp16 matrix instructions.
//
// The activations come as fp16 limbs that moe_limbs.hip makes in the workspace,
// once for all the tiles that read them: one limb for fp16 and bf16, two for
// fp32.
//
// The tile kernel: v_mfma_f32_16x16x32_f16 (K: one group of 32), fp32
// accumulation, the row's power of two undone at the store.  A workgroup takes
// 16 U slots (U = 8, 4 or 2, by the mean number of an expert) of one expert by
// 256 rows of W (gate/up form: 128 gate rows and the up rows of the same
// outputs, so that both sums of an output lie in one lane); each of its 4 waves
// all of the slots by 64 of the rows, so that no weight is converted twice.
// The weights:
//   fp32, fp16  the exact codes q - 8 (for fp32's low limbs times their 2^-11),
//         every product exact in fp32, one fp32 FMA per output and group for the
//         scale;
//   bf16  the same with tiles of 32 slots.  Larger ones take (q - 8) * scale * 2^10 in
//         fp16, the scale rounded to it and the product, so that the products of
//         all groups add up inside the matrix instructions.  That saves the FMAs,
//         256 VALU instructions of a wave's 400 per stage (us without and with it,
//         32 experts of 2 x 1024 x 4096: mean 32 84, 84; 128 166, 121; 256 272, 220;
//         512 418, 338; of 2 x 2048 x 7168, mean 512: 1257 to 1287, 1000).  The two
//         roundings change a product by at most 2^-10 of it.  The scale's is common
//         to a group, so a sum is off by up to 2^-10 sum |x w|; where scales are
//         spread over their binades its root mean square is under 2^-12
//         sqrt(sum of the groups' sums squared + sum (x w)^2) (0.78 measured at 32 to
//         7168 features), beside the 2^-8 of the result that storing it rounds by.
//         fp16's 2^-11 leaves no such room.  A scale outside [2^-20, 4) would leave
//         fp16's range: its group counts as 0 there, and a stage with such a
//         group adds its exact codes' products, scaled in fp32, by themselves.
//
// Stages of two groups.  Limbs (gathered rows, 128 bytes a stage) come to LDS by
// direct copies one stage ahead, weight words and scales for two stages at once
// (64 and 16 bytes a row), two stages ahead; both have two images, and a stage
// one barrier.  A wave copies the weights and scales of its own rows.  Copied
// stage by stage, 32 and 8 bytes a row, their requests held up all others (32
// experts of 2 x 2048 x 7168, 16384 slots in bf16: 1127 us; so 1034).  With the
// steps since then 990 us, 0.97 PFLOP/s (limbs included; 1068 under the profiler's
// trace), the matrix units busy half of the time: bound by their issue together
// with the conversion's.
//
// Tiles are dealt so that each XCD works a contiguous run of them (the
// hardware deals workgroups round-robin over the 8 XCDs), row blocks of an
// expert fastest: the tiles an XCD holds at once share weight rows and slots.

#include "moe_common.h"
#include "gemv_common.h"
#include "limbs.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

typedef __attribute__((address_space(3))) void et_lds_void;

constexpr int kEtThreads = 256;

template <int VM>
__device__ __forceinline__ void et_wait_vm() {  // at most VM copies still in flight
  static_assert(VM >= 0 && VM < 64, "wait count");
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | 0x70 | (15 << 8));
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
__device__ __forceinline__ void et_copy4(const void *src, const void *lds) {
  const uint32_t at = uint32_t(reinterpret_cast<uintptr_t>((const et_lds_void *)lds));
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 1\n\tglobal_load_lds_dword %0, off"
               :: "v"(src), "s"(at) : "memory", "m0");
}
__device__ __forceinline__ void et_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr float kFold = 1024.0f;  // power of two of folded weights

// whether a scale times kFold is folded in (0 is: its products are 0 either way)
__device__ __forceinline__ bool foldable(float s) {
  const float m = fabsf(s);
  return bool(int(m == 0.0f) | (int(m >= 0x1p-10f) & int(m < 4096.0f)));
}

struct TileArgs {
  const _Float16 *limbs;
  const float *factor;
  const int32_t *token_index, *offsets;
  const unsigned char *qw;
  const float *sc;
  void *Y;
  int rows_x, R, E, N, G, KP, ldy, tiles_n;
  bool pairs;  // rows of Y begin and end at pairs of outputs (gate/up form)
};

// U: row tiles of 16 slots, L limbs, OT the output type (kSw: the activations'
// type, else fp32), kFolded: weights with their scales.
template <int U, int L, typename OT, bool kSw, bool kFolded>
__global__ void __launch_bounds__(kEtThreads, 2) experts_tile(TileArgs a) {
  static_assert(!kFolded || L == 1, "folded weights have fp16's precision");
  // Limbs of a stage (64 k): row r at 128 r, logical chunk x (16 bytes: 8 values
  // of one group's block x % 4, group x / 4) at chunk x ^ ((r / 2) % 8), so that
  // the 16 rows an operand read touches fall in distinct banks.
  // Weights of two stages: W row n at 64 n, its 16 bytes of group q (0..3) at
  // chunk q ^ ((n / 4) % 4), for the same reason.  Their scales: group q of row n
  // at 16 n + 4 q.
  constexpr int kRows = 16 * U, kLimb = kRows * 128;
  constexpr int kA = L * kLimb, kW = 16384, kS = 4096;
  __shared__ __align__(16) unsigned char et_mem[2 * (kA + kW + kS)];
  __shared__ __align__(16) float et_factor[kRows];
  unsigned char *const a_mem = et_mem, *const w_mem = et_mem + 2 * kA,
                      *const s_mem = w_mem + 2 * kW;
  constexpr int kPairCopies = 8;            // weights and scales, of a wave
  constexpr int NO = kSw ? 128 : 256;       // outputs per tile
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, R = lane >> 4;
  const int G = a.G, N = a.N;

  // tile of this workgroup: XCD b % 8 takes a contiguous run of the tiles
  // there are; within an expert its row blocks are fastest
  ExpertItem it = find_item(a.offsets, a.E, a.R, kRows, 0);
  const long tiles = long(it.total) * a.tiles_n;
  const long run = (tiles + 7) / 8;
  const long index = long(blockIdx.x >> 3);
  const long tile = long(blockIdx.x & 7) * run + index;
  if (index >= run || tile >= tiles) return;  // uniform over the workgroup
  it = find_item(a.offsets, a.E, a.R, kRows, int(tile / a.tiles_n));
  // tiles of this expert: it.blocks x tiles_n, from item (its first block) on
  const long first = (tile / a.tiles_n - it.block) * a.tiles_n;
  const int within = int(tile - first);
  const int bm = within % it.blocks, bn = within / it.blocks;
  int e0, e1;
  expert_slots(a.offsets, it.e, a.R, e0, e1);
  const int row0 = e0 + bm * kRows, rows = std::min(kRows, e1 - row0);
  const int n0 = bn * NO;

  // Limb copies: copy j (wave w issues j = w U/2 .. of each limb): lane i writes
  // 16 B at 1024 j + 16 i: row 8 j + i / 8, chunk i % 8, which holds logical
  // chunk (i % 8) ^ ((row / 2) % 8).  Rows past the item repeat its last.
  const unsigned char *asrc[U / 2];
#pragma unroll
  for (int j = 0; j < U / 2; ++j) {
    const int r = 8 * (wave * (U / 2) + j) + lane / 8;
    const int slot = row0 + std::min(r, rows - 1);
    long row = slot;
    if (a.token_index) row = std::min(std::max(a.token_index[slot], 0), a.rows_x - 1);
    asrc[j] = reinterpret_cast<const unsigned char *>(a.limbs + row * a.KP) +
              16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  const long plane = long(a.rows_x) * a.KP * 2;
  // Row of W of row i of this wave's 64, dealt so that a lane's sums of a slot
  // are neighbouring outputs: row 16 t + c is that of output 64 w + 4 c + t; in
  // the gate/up form t = 0, 1 are the gate rows of outputs 32 w + 2 c + t, t = 2, 3
  // the up rows of the same.  Rows past N read row N - 1.
  auto w_row = [&](int i) -> long {
    const int t = i >> 4, at = i & 15;
    long n;
    if constexpr (kSw)
      n = std::min(n0 + 32 * wave + 2 * at + (t & 1), N - 1) + (t >= 2 ? long(N) : 0);
    else
      n = std::min(n0 + 64 * wave + 4 * at + t, N - 1);
    return n + long(it.e) * (kSw ? 2 * long(N) : long(N));
  };
  // Weight copies j = 0..3: lane i writes 16 B: row 16 j + i / 4, chunk i % 4.
  // Scale copies: lane i writes 4 B: row 16 j + i / 4, group i % 4.
  const unsigned char *wsrc[4];
  const float *ssrc[4];
  int wq[4];  // the lane's group of the two stages
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 16 * j + lane / 4;
    wq[j] = (lane & 3) ^ ((i >> 2) & 3);
    wsrc[j] = a.qw + (w_row(i) * G + wq[j]) * 16;
    ssrc[j] = a.sc + w_row(i) * G + (lane & 3);
  }
  const int P = (G + 1) / 2;
  // limbs of a stage; called for the stages in order
  auto copy_limbs = [&](unsigned char *img) {
#pragma unroll
    for (int l = 0; l < L; ++l)
#pragma unroll
      for (int j = 0; j < U / 2; ++j)
        et_copy16(asrc[j] + l * plane, img + l * kLimb + 1024 * (wave * (U / 2) + j));
#pragma unroll
    for (int j = 0; j < U / 2; ++j) asrc[j] += 128;
  };
  // weights and scales of stages 2 k and 2 k + 1; called in order
  auto copy_pair = [&](unsigned char *wimg, unsigned char *simg, int k) {
    if (4 * k + 4 > G) {
      // groups past G read group G - 1 again (their limbs are 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wsrc[j] -= 16 * std::max(4 * k + wq[j] - (G - 1), 0);
        ssrc[j] -= std::max(4 * k + (lane & 3) - (G - 1), 0);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      et_copy16(wsrc[j], wimg + 4096 * wave + 1024 * j);
      et_copy4(ssrc[j], simg + 1024 * wave + 256 * j);
      wsrc[j] += 64;
      ssrc[j] += 4;
    }
  };

  // operand reads: limbs of row 16 u + c at aread[q] + 2048 u; words of row
  // 16 t + c, group q, at cread[q] + 1024 t (^ 32 for the images' second stage);
  // its scales at sread + 256 t (+ 8)
  uint32_t aread[2], cread[2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    aread[q] = uint32_t(c * 128 + 16 * ((4 * q + R) ^ ((c >> 1) & 7)));
#pragma unroll
  for (int q = 0; q < 2; ++q)
    cread[q] = uint32_t(4096 * wave + 64 * c + 16 * (q ^ (c >> 2)) + 4 * R);
  const uint32_t sread = uint32_t(1024 * wave + 16 * c);

  floatx4 acc[U][4];
  const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[u][t] = zero;

  // The scales times kFold.  Groups whose scale cannot be folded in are done
  // here (none in an ordinary stage: one look at the largest and the least of
  // the wave's) and left with 0.
  auto fold_scales = [&](const unsigned char *img, const unsigned char *wimg, int p,
                         float2 (&s)[4]) {
    const uint32_t h = p & 1;
    float most = 0.0f, least = 1.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s[t].x *= kFold;
      s[t].y *= kFold;
      most = fmaxf(fmaxf(most, fabsf(s[t].x)), fabsf(s[t].y));
      least = fminf(fminf(least, fabsf(s[t].x)), fabsf(s[t].y));
    }
    if (__ballot(!(most < 4096.0f) | (least < 0x1p-10f)) == 0) return;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float &m = q == 0 ? s[t].x : s[t].y;
        if (__ballot(!foldable(m)) == 0) continue;
        const float sq = foldable(m) || 2 * p + q >= G ? 0.0f : m;
        m = foldable(m) ? m : 0.0f;
        const half8_t b =
            nibbles_to_f16(*reinterpret_cast<const uint32_t *>(wimg + (cread[q] ^ 32 * h) + 1024 * t));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const half8_t x = *reinterpret_cast<const half8_t *>(img + aread[q] + 2048 * u);
          const floatx4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, b, zero, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[u][t][r] = sq != 0.0f ? fmaf(sq, d[r], acc[u][t][r]) : acc[u][t][r];
        }
      }
    }
  };
  auto products = [&](const unsigned char *img, const unsigned char *wimg,
                      const unsigned char *simg, int p) {
    const uint32_t h = p & 1;
    float2 s[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      s[t] = *reinterpret_cast<const float2 *>(simg + sread + 256 * t + 8 * h);
    if constexpr (kFolded) fold_scales(img, wimg, p, s);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        w[t] = *reinterpret_cast<const uint32_t *>(wimg + (cread[q] ^ 32 * h) + 1024 * t);
      half8_t b[4], low[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        b[t] = nibbles_to_f16(w[t]);
        if constexpr (kFolded) {
          const _Float16 f = _Float16(q == 0 ? s[t].x : s[t].y);
          b[t] = b[t] * half8_t{f, f, f, f, f, f, f, f};
        }
        if constexpr (L == 2) {  // the low limbs' codes, exact
          const _Float16 f = _Float16(1.0f / kLowScale);
          low[t] = b[t] * half8_t{f, f, f, f, f, f, f, f};
        }
      }
      if constexpr (kFolded) __builtin_amdgcn_s_setprio(2);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        half8_t x[L];
#pragma unroll
        for (int l = 0; l < L; ++l)
          x[l] = *reinterpret_cast<const half8_t *>(img + l * kLimb + aread[q] + 2048 * u);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if constexpr (kFolded) {
            acc[u][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[0], b[t], acc[u][t], 0, 0, 0);
          } else {
            floatx4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[0], b[t], zero, 0, 0, 0);
            if constexpr (L == 2)
              d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[L - 1], low[t], d, 0, 0, 0);
            const float sq = q == 0 ? s[t].x : s[t].y;
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[u][t][r] = fmaf(sq, d[r], acc[u][t][r]);
          }
        }
      }
    }
  };

  // Folded weights: the wave that has come to its products goes first until the
  // stage's end, while the other wave of its SIMD converts or copies (us without
  // and with it, bf16, 32 experts: 2 x 2048 x 7168, mean 512: 1002, 967; 2 x 1024
  // x 4096, mean 150: 134, 124; 688: 400, 373; but 325: 216, 229, a launch whose
  // last tiles leave half the card empty.  fp16 and fp32 lose, 2 to 10 %).
  //
  // At a stage's start its copies have landed in this wave; past the barrier
  // they have in every wave, and every wave is past the stage before, whose
  // limbs' image is then filled again, and past the two stages before an even
  // stage, whose weights' image is.
  copy_limbs(a_mem);
  copy_pair(w_mem, s_mem, 0);
  // the rows' factors for the store, on their way with the first copies (read
  // there row by row, they cost a tenth of a tile's time)
  if (tid < kRows) {
    long row = row0 + std::min(tid, rows - 1);
    if (a.token_index) row = std::min(std::max(a.token_index[row], 0), a.rows_x - 1);
    et_factor[tid] = a.factor[row];
  }
  for (int p = 0; p < P; ++p) {
    const int k = p >> 1;
    const bool odd = p & 1, more = p + 1 < P;
    // the limbs of an odd stage were asked for before the next weights
    if (odd && more)
      et_wait_vm<kPairCopies>();
    else
      et_wait_vm<0>();
    et_wait_lgkm0();
    et_barrier();
    if (more) copy_limbs(a_mem + (~p & 1) * kA);
    if (!odd && p + 2 < P) copy_pair(w_mem + (~k & 1) * kW, s_mem + (~k & 1) * kS, k + 1);
    products(a_mem + (p & 1) * kA, w_mem + (k & 1) * kW, s_mem + (k & 1) * kS, p);
    if constexpr (kFolded) __builtin_amdgcn_s_setprio(0);
  }

  OT *y = static_cast<OT *>(a.Y);
  constexpr float f0 = kFolded ? 1.0f / kFold : 1.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const floatx4 f = *reinterpret_cast<const floatx4 *>(et_factor + 16 * u + 4 * R);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 16 * u + 4 * R + r;
      if (m >= rows) continue;
      const long at = long(row0 + m) * a.ldy;
      if constexpr (kSw) {
        const int n = n0 + 32 * wave + 2 * c;
        OT h[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
          h[t] = from_f32<OT>(silu_mul(acc[u][t][r] * f0 * f[r], acc[u][t + 2][r] * f0 * f[r]));
        if (a.pairs) {
          struct alignas(2 * sizeof(OT)) Two {
            OT v[2];
          };
          if (n < N) *reinterpret_cast<Two *>(y + at + n) = Two{{h[0], h[1]}};
        } else {
          if (n < N) y[at + n] = h[0];
          if (n + 1 < N) y[at + n + 1] = h[1];
        }
      } else {
        // rows of Y have room for a multiple of 4 outputs
        const int n = n0 + 64 * wave + 4 * c;
        const floatx4 d = {acc[u][0][r], acc[u][1][r], acc[u][2][r], acc[u][3][r]};
        if (n < N) *reinterpret_cast<floatx4 *>(y + at + n) = d * f0 * f[r];
      }
    }
  }
}

template <typename XT, bool kSw, int U>
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
  a.pairs = p.N % 2 == 0 && reinterpret_cast<uintptr_t>(p.Y) % (2 * sizeof(OT)) == 0;
  a.tiles_n = (p.N + (kSw ? 128 : 256) - 1) / (kSw ? 128 : 256);
  const long tiles = long(a.tiles_n) * max_items(p.R, p.E, 16 * U);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  const hipError_t e = launch_limbs(p, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((experts_tile<U, L, OT, kSw, __is_same(XT, Bf16) && (U > 2)>),
                     dim3(unsigned((tiles + 7) / 8 * 8)), dim3(kEtThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename XT, bool kSw>
hipError_t run_tile_rows(const MoeExperts &p, hipStream_t stream) {
  // Slots per tile by the mean of an expert (32 experts of 2 x 1024 x 4096, us
  // with 32, 64 and 128 slots; bf16: mean 48 88, 98, 112; 56 109, 98, 123; 96
  // 140, 118, 136; 128 164, 150, 137.  fp16, whose FMAs grow with every slot: 48
  // 89, 110, 150; 256 279, 263, 292; 512 512, 455, 446.  fp32, with 32 and 64:
  // 48 106, 138; 64 145, 139; 128 slots leave room for one workgroup only on a
  // compute unit).
  const double mean = double(p.R) / double(std::max(1, std::min(p.R, p.E)));
  if (mean <= 52) return run_tile<XT, kSw, 2>(p, stream);
  if constexpr (sizeof(XT) == 4) return run_tile<XT, kSw, 4>(p, stream);
  else if (mean <= (__is_same(XT, Bf16) ? 110 : 320)) return run_tile<XT, kSw, 4>(p, stream);
  else return run_tile<XT, kSw, 8>(p, stream);
}

template <typename XT>
hipError_t run_tile_type(const MoeExperts &p, hipStream_t stream) {
  return p.swiglu ? run_tile_rows<XT, true>(p, stream) : run_tile_rows<XT, false>(p, stream);
}

}  // namespace

// Mean slots per expert up to which the skinny kernel is the faster one (32
// experts of 2 x 1024 x 4096, us skinny against the best tile: bf16 24 73, 82;
// 32 87, 85; 48 119, 88; fp32 8 69, 72; 12 83, 80; 24 111, 95).
int experts_kernel(long R, long E, int dtype) {
  const long active = std::max(1L, std::min(R, E));
  return R > (dtype == W4A16_DTYPE_F32 ? 10 : 28) * active ? W4A16_EXPERTS_TILE
                                                          : W4A16_EXPERTS_SKINNY;
}

size_t experts_workspace_bytes(long rows_x, long R, long E, int K, int dtype) {
  // the skinny kernel takes 16-bit activations as they are
  if (experts_kernel(R, E, dtype) != W4A16_EXPERTS_TILE && dtype != W4A16_DTYPE_F32) return 0;
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
  return experts_kernel(p.R, p.E, p.dtype) == W4A16_EXPERTS_TILE ? launch_experts_tile(p, stream)
                                                       : launch_experts_skinny(p, stream);
}

}  // namespace w4a16
