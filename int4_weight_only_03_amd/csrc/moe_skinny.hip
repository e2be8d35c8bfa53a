// Experts' W4A16 products for few slots per expert, in fp32, fp16 and bf16:
// D[r] = x_r . W_e^T for every slot r of expert e (stored as fp32, for the
// combination of slots), or the fused gate/up form H[r] = silu(x_r . gate_e^T)
// * (x_r . up_e^T) in the activations' type.  The pages run their MoE experts
// and the SwiGLU MLP through the INT4 path ("The Quiet Commit: How a Single
// Documentation Edit Marks the Completion of a Major Engineering Milestone",
// section "The INT4 Milestone").
//
// Bound by reading the active experts' weights (5/8 byte a weight; 147 MB for one
// token of 8 experts of 2 x 2048 x 7168 in 33 us, 4.4 TB/s, where the loads alone
// take 28): the weights and the activations go from memory straight to registers,
// P steps of 4 groups ahead, and nothing waits at a barrier before the end.  They
// are read once for every 16 slots of an expert, so twice from 17 to the 28 slots
// where the tile kernel takes over (the second time mostly from the caches).
//
// Arithmetic, on 16x16x32 matrix instructions (A: 16 slots, B: 16 rows of W,
// K: one group of 32), fp32 accumulation, one fp32 FMA per output and group
// for the group's scale:
//   fp32  two fp16 limbs of each activation, from moe_limbs.hip, and the exact
//         codes q - 8 (every product exact in fp32); the low limb's sum takes its
//         2^-11 with one FMA, the row's power of two is undone at the store;
//   fp16  the activations as they are and the exact codes q - 8;
//   bf16  the activations as they are and (q + 16) 2^-12, which two VALU
//         instructions per pair of codes make: an instruction on a B of -24 2^-12
//         throughout gives the accumulator that takes the offset out again, and
//         the store undoes 2^-12.  The terms are up to 31 + 24 units of the scale
//         instead of 8 and cancel, so the fp32 sums lose up to 3 bits more (2^-21
//         beside an output rounded to 2^-8); nothing is spent per activation.
//         With the power of two no group's sum leaves fp32's range: 32 (31 + 24)
//         2^-12 of bf16's largest number is less than half of it, and 2^-12 of its
//         least, 2^-133, is a multiple of fp32's least.  (Without it activations
//         from 3e35 on overflowed.)
//
// Mapping: lane (c, R) (c = lane % 16, R = lane / 16) loads the 16 bytes of
// group 4 s + R of W row c (64 contiguous bytes of each of 16 rows per
// instruction); two lane swaps across the four lane rows give it word R of
// each of the step's 4 groups, its B operand.  Its A operand is k = 8R .. 8R+7
// of the slot in tile row c, D holds tile rows 4R .. 4R+3 of W row c.  Slot i
// of 16 stands in tile row 4 (i % 4) + i / 4, so that up to 4 MR slots fill only
// the first MR of D's registers and the others cost no scale FMA.
//
// A wave takes 4 MR slots of one expert by NT x 16 rows of W (gate tiles, then
// the up tiles of the same outputs); KW waves of a workgroup share a tile and
// its steps in turn, and their sums are added in wave order in LDS.  So the
// waves read a row's next 64 bytes each at about the same time, and a cache line
// that two steps share is fetched once (taking blocks of 4 steps in turn: 342 MB
// fetched for 215 at 2080 features, whose rows end inside a line, and 61.7 us;
// so 290 MB and 59.1 us with 2 waves, 212 MB and 56.0 us with 4).  The next
// steps' weights fly while one is worked on.  The scales of a wave's 4 steps come
// in one load per 16 rows of W (16 bytes a step and row) and pass through the
// wave's own LDS words: loaded step by step they cost more than the weights
// (measured on 147 MB in this pattern, loads alone: 22.4 us without scales, 34.8
// with them step by step, 27.9 by blocks).

#include "moe_common.h"
#include "gemv_common.h"
#include "limbs.h"

#include <algorithm>

namespace w4a16 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kEsWaves = 4;
constexpr int kEsThreads = 64 * kEsWaves;
constexpr int kEsBlock = 16;  // groups of a block: 4 steps of 4
constexpr int kTokenWaves = 16;  // most waves of a workgroup of the one-token form
constexpr int P = 2;          // steps in flight of a wave

// 8 activations x0..x7 in the order x0 x4 x1 x5 x2 x6 x3 x7 (that of the
// nibble conversions)
__device__ __forceinline__ u32x4m interleave8(u32x4m a) {
  return u32x4m{__builtin_amdgcn_perm(a.z, a.x, 0x05040100u),
                __builtin_amdgcn_perm(a.z, a.x, 0x07060302u),
                __builtin_amdgcn_perm(a.w, a.y, 0x05040100u),
                __builtin_amdgcn_perm(a.w, a.y, 0x07060302u)};
}

constexpr float kBf16Scale = 4096.0f;  // what the bf16 form's codes are divided by

// bf16 (q + 16) 2^-12 of the 8 nibbles of w: dword p holds nibbles p and p + 4.  A
// bf16 has 7 bits behind the leading one, so a nibble stands at bits 3..6 of those of
// 16 2^-12 = 0x3B80.
__device__ __forceinline__ bf16x8 nibbles_to_bf16_16(uint32_t w) {
  const uint32_t p0 = __builtin_amdgcn_bitop3_b32(w << 3, 0x00780078u, 0x3B803B80u, 0xEA);
  const uint32_t p1 = __builtin_amdgcn_bitop3_b32(w >> 1, 0x00780078u, 0x3B803B80u, 0xEA);
  const uint32_t p2 = __builtin_amdgcn_bitop3_b32(w >> 5, 0x00780078u, 0x3B803B80u, 0xEA);
  const uint32_t p3 = __builtin_amdgcn_bitop3_b32(w >> 9, 0x00780078u, 0x3B803B80u, 0xEA);
  return __builtin_bit_cast(bf16x8, u32x4m{p0, p1, p2, p3});
}

// k = 8R .. 8R+7 of one group of one slot: fp32 its two limbs (in the nibble
// conversion's order), else the activations
template <typename XT>
struct XChunk {
  u32x4m v[sizeof(XT) == 4 ? 2 : 1];
};

struct ExpertArgs {
  const void *X;               // rows of ldx values: limbs (fp32) or activations
  const float *factor;         // 2^-e of a row (fp32)
  const int32_t *token_index;  // slot -> row of X, or null: the slot itself
  const int32_t *offsets;      // [E + 1]
  const uint4 *qw;             // [E][N or 2N][G] groups of 16 bytes
  const float *sc;             // [E][N or 2N][G]
  void *Y;                     // [R][ldy]
  int rows_x, ldx, R, E, N, G, ldy, tiles_n;
  // one-token form: Y[n] = sum_j weights[j] * D[slots[j]][n], in XT
  const int32_t *slots;
  const float *weights;
  int topk;
};

__device__ __forceinline__ long row_of(const ExpertArgs &a, int slot) {
  return a.token_index ? std::min(std::max(a.token_index[slot], 0), a.rows_x - 1) : slot;
}

// The item of one slot, of whichever expert owns it (none: e = -1, as for a slot
// below 0).  Every lane gets the same answer.
__device__ __forceinline__ ExpertItem slot_item(const int32_t *__restrict__ offsets, int E, int R,
                                                int slot) {
  ExpertItem it = {-1, min(max(slot, 0), R - 1), 1, 0, 1, 1};
  if (slot < 0) return it;
  int owner = 0;  // experts that end before it
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + int(threadIdx.x & 63);
    owner += __popcll(__ballot(e < E && offsets[min(e, E - 1) + 1] <= it.row0));
  }
  int r0 = 0, r1 = 0;
  if (owner < E) expert_slots(offsets, owner, R, r0, r1);
  if (it.row0 >= r0 && it.row0 < r1) it.e = owner;
  return it;
}

// kSw: W has 2N rows, Y is XT; else Y is fp32.
// kToken: the combination for a single token in the same launch.  KW waves a slot
// and all of its slots make a workgroup, which adds them up in the order of the
// choices and stores Y in XT.
template <typename XT, int MR, int KW, bool kSw, bool kToken>
__global__ void __launch_bounds__(kToken ? 64 * kTokenWaves : kEsThreads, kToken ? 4 : 2)
experts_skinny(ExpertArgs a) {
  static_assert(!kToken || (MR == 1 && !kSw), "one slot of a down projection");
  constexpr int NT = kToken ? 2 : 4;  // tiles of 16 rows of W of a wave
  constexpr int NO = kSw ? NT / 2 : NT;
  constexpr int B = 4 * MR;  // slots of an item
  constexpr bool kLimbs = sizeof(XT) == 4;
  constexpr float kOnce = __is_same(XT, Bf16) ? kBf16Scale : 1.0f;  // factor of the sums
  // per wave: a block's scales, row n of the tile at 64 n; at the end the sums
  constexpr int kTile = MR * NT * 64;
  constexpr int kWaveLds = KW > 1 && kTile > NT * 256 ? kTile : NT * 256;
  __shared__ __align__(16) float es_lds[(kToken ? kTokenWaves : kEsWaves) * kWaveLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int c = lane & 15, R = lane >> 4;
  float *mem = es_lds + wave * kWaveLds;
  const int kw = KW > 1 ? wave % KW : 0;
  int n0;
  ExpertItem it;
  if constexpr (kToken) {
    n0 = int(blockIdx.x) * 16 * NO;
    it = slot_item(a.offsets, a.E, a.R, a.slots[wave / KW]);
  } else {
    const long tile = long(blockIdx.x) * (kEsWaves / KW) + wave / KW;
    const int item = int(tile / a.tiles_n);
    n0 = int(tile - long(item) * a.tiles_n) * 16 * NO;
    it = find_item(a.offsets, a.E, a.R, B, item);
  }
  const int G = a.G, N = a.N;

  float acc[NT][MR];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < MR; ++r) acc[t][r] = 0.0f;

  // The wave's j-th step of 4 groups; its steps come in blocks of 4.
  auto step_of = [&](int j) { return j * KW + kw; };
  const int steps = (G + 3) / 4, own = (steps - kw + KW - 1) / KW;
  const int mine = it.e >= 0 ? (own + 3) / 4 : 0;
  if (mine > 0) {
    // The tile's first row of W and its scales (gate; the up rows are N
    // further), and this lane's row offsets from them (below 2^23 bytes).
    // Rows past N read row N - 1.
    const long row = long(it.e) * (kSw ? 2 * long(N) : long(N)) + n0;
    const char *wbase = reinterpret_cast<const char *>(a.qw) + row * G * 16;
    const char *sbase = reinterpret_cast<const char *>(a.sc) + row * G * 4;
    const long up_w = kSw ? long(N) * G * 16 : 0, up_s = kSw ? long(N) * G * 4 : 0;
    uint32_t woff[NO], soff[NO];
#pragma unroll
    for (int t = 0; t < NO; ++t) {
      woff[t] = uint32_t(std::min(n0 + 16 * t + c, N - 1) - n0) * uint32_t(G) * 16u;
      soff[t] = uint32_t(std::min(n0 + 16 * t + lane / 4, N - 1) - n0) * uint32_t(G) * 4u;
    }
    // the activations (slots past the item repeat its last)
    const int slot = (c >> 2) + 4 * std::min(c & 3, MR - 1);
    const char *const xrow = static_cast<const char *>(a.X) +
                             2 * (row_of(a, it.row0 + std::min(slot, it.rows - 1)) * a.ldx + 8 * R);
    const long plane = 2 * long(a.rows_x) * a.ldx;

    // step j of block b; groups past G read group G - 1 and are left out later.
    // Weights and activations are loaded together and equally far ahead: loads
    // complete in order, so a wait for activations loaded late would be a wait
    // for every weight asked for before them.
    struct Ops {
      u32x4m w[NT];
      XChunk<XT> x[4];
    };
    auto load = [&](Ops &o, int b, int j) {
      const int g0 = 4 * step_of(4 * b + j);
      const uint32_t gw = 16u * uint32_t(std::min(g0 + R, G - 1));
#pragma unroll
      for (int t = 0; t < NT; ++t)
        o.w[t] = *reinterpret_cast<const u32x4m *>(wbase + (t < NO ? 0 : up_w) + (woff[t % NO] + gw));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const long g = 64 * long(std::min(g0 + q, G - 1));
        o.x[q].v[0] = *reinterpret_cast<const u32x4m *>(xrow + g);
        if constexpr (kLimbs) o.x[q].v[1] = *reinterpret_cast<const u32x4m *>(xrow + plane + g);
      }
    };
    // Scales of block b: lane l takes those of step l % 4 for row l / 4 of each
    // tile, shares that would pass G moved back to end there.
    auto load_s = [&](f32x4u (&s)[NT], int b) {
      const uint32_t at = 4u * uint32_t(std::min(4 * step_of(4 * b + (lane & 3)), G - 4));
#pragma unroll
      for (int t = 0; t < NT; ++t)
        s[t] = *reinterpret_cast<const f32x4u *>(sbase + (t < NO ? 0 : up_s) + (soff[t % NO] + at));
    };
    // the same for rows of fewer than 4 groups
    auto load_few = [&](f32x4u (&s)[NT]) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[t][i] = *reinterpret_cast<const float *>(
              sbase + (t < NO ? 0 : up_s) + (soff[t % NO] + 4u * uint32_t(std::min(i, G - 1))));
    };
    // Into the wave's words, group q of row n of the block at 16 n + q: a whole
    // block, or the last one, whose moved shares write their groups' own places.
    float *keep = mem + 16 * (lane / 4);
    auto keep_s = [&](const f32x4u (&s)[NT]) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        *reinterpret_cast<float4 *>(keep + 256 * t + 4 * (lane & 3)) =
            make_float4(s[t][0], s[t][1], s[t][2], s[t][3]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    auto keep_last = [&](const f32x4u (&s)[NT], int b) {
      const int g = 4 * (lane & 3);
      const int moved = G >= 4 ? std::max(4 * step_of(4 * b + (lane & 3)) - (G - 4), 0) : 0;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i >= moved) keep[256 * t + g + i - moved] = s[t][i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };

    const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    auto group = [&](const Ops &o, const float4 (&sc)[NT], int q) {
      const u32x4m xa = kLimbs ? o.x[q].v[0] : interleave8(o.x[q].v[0]);
      floatx4 d0 = zero;
      if constexpr (__is_same(XT, Bf16)) {
        const bf16x8 off = __builtin_bit_cast(
            bf16x8, u32x4m{0xBBC0BBC0u, 0xBBC0BBC0u, 0xBBC0BBC0u, 0xBBC0BBC0u});  // -24 2^-12
        d0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa), off, zero, 0, 0,
                                                     0);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        floatx4 d;
        if constexpr (__is_same(XT, Bf16)) {
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa),
                                                      nibbles_to_bf16_16(o.w[t][q]), d0, 0, 0, 0);
        } else {
          const half8_t b = nibbles_to_f16(o.w[t][q]);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, xa), b, zero, 0, 0, 0);
          if constexpr (kLimbs) {
            const floatx4 low = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                __builtin_bit_cast(half8_t, o.x[q].v[sizeof(XT) / 4]), b, zero, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < MR; ++r) d[r] = fmaf(low[r], 1.0f / kLowScale, d[r]);
          }
        }
        const float s = q == 0 ? sc[t].x : q == 1 ? sc[t].y : q == 2 ? sc[t].z : sc[t].w;
#pragma unroll
        for (int r = 0; r < MR; ++r) acc[t][r] = fmaf(s, d[r], acc[t][r]);
      }
    };
    // left: groups of the step that there are
    auto process = [&](Ops &o, int j, int left) {
      float4 sc[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sc[t] = *reinterpret_cast<const float4 *>(mem + 16 * (16 * t + c) + 4 * j);
        transpose_words(o.w[t]);
      }
      // one group at a time: letting the scheduler mix them costs registers
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q < left) group(o, sc, q);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // A ring of P steps: a step's registers are refilled after their last use,
    // which keeps them over the loop's back edge.
    Ops ring[P];
    f32x4u s[NT];
    if (G >= 4)
      load_s(s, 0);
    else
      load_few(s);
#pragma unroll
    for (int j = 0; j < P; ++j) load(ring[j], 0, j);
    int b = 0;
    for (; b + 1 < mine; ++b) {  // every block but a wave's last is whole
      keep_s(s);
      load_s(s, b + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        process(ring[j % P], j, 4);
        load(ring[j % P], j + P < 4 ? b : b + 1, (j + P) % 4);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    keep_last(s, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int left = G - 4 * step_of(4 * b + j);
      if (left <= 0) break;
      process(ring[j % P], j, left);
      if (j + P < 4) load(ring[j % P], b, j + P);
    }
  }

  if constexpr (kToken) {
    // the slot stands in tile row 0: lanes 0..15 hold its outputs
    __shared__ int es_there[kTokenWaves];
    float f = kOnce;
    if constexpr (kLimbs) f = a.factor[it.row0];
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (R == 0) mem[16 * t + c] = acc[t][0] * f;
    if (lane == 0) es_there[wave] = it.e >= 0;
    __syncthreads();
    const int n = n0 + int(threadIdx.x);
    if (threadIdx.x >= 16 * NT || n >= N) return;
    float y = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
      if (!es_there[j * KW]) continue;
      const float *d = es_lds + j * KW * kWaveLds + threadIdx.x;
      float sum = d[0];
#pragma unroll
      for (int k = 1; k < KW; ++k) sum += d[k * kWaveLds];
      y = fmaf(a.weights[j], sum, y);
    }
    static_cast<XT *>(a.Y)[n] = from_f32<XT>(y);
    return;
  }
  if constexpr (KW > 1) {
    // sums of the tile's waves, in their order, on the first of them (each wave
    // is past its own words)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < MR; ++r) mem[(t * MR + r) * 64 + lane] = acc[t][r];
    __syncthreads();
    if (kw != 0) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < MR; ++r)
#pragma unroll
        for (int k = 1; k < KW; ++k) acc[t][r] += mem[k * kWaveLds + (t * MR + r) * 64 + lane];
  }
  if (it.e < 0) return;
#pragma unroll
  for (int r = 0; r < MR; ++r) {
    const int m = R + 4 * r;
    if (m >= it.rows) continue;
    float f = kOnce;
    if constexpr (kLimbs) f = a.factor[row_of(a, it.row0 + m)];
    const long y = long(it.row0 + m) * a.ldy;
#pragma unroll
    for (int t = 0; t < NO; ++t) {
      const int n = n0 + 16 * t + c;
      if (n >= N) continue;
      const float g = acc[t][r] * f;
      if constexpr (kSw)
        static_cast<XT *>(a.Y)[y + n] = from_f32<XT>(silu_mul(g, acc[t + NO][r] * f));
      else
        static_cast<float *>(a.Y)[y + n] = g;
    }
  }
}

template <typename XT, int MR, int KW, bool kSw>
hipError_t run_skinny(ExpertArgs a, hipStream_t stream) {
  constexpr int NO = kSw ? 2 : 4;
  a.tiles_n = (a.N + 16 * NO - 1) / (16 * NO);
  const long tiles = long(a.tiles_n) * max_items(a.R, a.E, 4 * MR);
  const long blocks = (tiles * KW + kEsWaves - 1) / kEsWaves;
  if (blocks > kMaxBlocks) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((experts_skinny<XT, MR, KW, kSw, false>), dim3(unsigned(blocks)),
                     dim3(kEsThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename XT, bool kSw, int KW>
hipError_t run_skinny_rows(const ExpertArgs &a, hipStream_t stream) {
  // slots per item: enough for one item of most experts (32 experts of 2 x 1024
  // x 4096, mean 4: 47 us with 8, 41 with 16; with row tiles of 32 and 64
  // slots means of 12 to 24 took 72 to 91 us, with several items of 16 58 to 75)
  const double mean = double(a.R) / double(std::max(1, std::min(a.R, a.E)));
  if (mean <= 1.25) return run_skinny<XT, 1, KW, kSw>(a, stream);
  if (mean <= 3.0) return run_skinny<XT, 2, KW, kSw>(a, stream);
  return run_skinny<XT, 4, KW, kSw>(a, stream);
}

template <typename XT, bool kSw>
hipError_t run_skinny_type(const ExpertArgs &a, hipStream_t stream) {
  // Waves per tile: as many as there are blocks for up to 2; up to 4 where few
  // tiles leave the card to fill (K = 7168, one token, 32 tiles: 15.8 against
  // 24.5 us with 2; 512 tiles: 37.2 against 35.2) and where rows of W are no whole
  // 64 bytes, so that more waves share their lines (32 experts of 2 x 1024, us
  // with 2 and 4: 16 tokens, top 4, K = 7200: bf16 72.5, 70.7, fp32 83.8, 81.2; 64
  // tokens: 108, 93 and 130, 117; but K = 2080 in fp32 37.0, 38.3, and whole rows
  // of 7168 60.7, 63.7 and 91.8, 85.4).
  const int blocks = (a.G + kEsBlock - 1) / kEsBlock;
  const long tiles = (long(a.N) + 31) / 32 * std::min(a.R, a.E);
  const bool ragged = a.G % 4 != 0 && blocks >= (sizeof(XT) == 4 ? 8 : 4);
  if (ragged || (blocks >= 4 && tiles < 512)) return run_skinny_rows<XT, kSw, 4>(a, stream);
  if (blocks >= 2) return run_skinny_rows<XT, kSw, 2>(a, stream);
  return run_skinny_rows<XT, kSw, 1>(a, stream);
}

template <typename XT>
hipError_t run_token(const ExpertArgs &a, hipStream_t stream) {
  // waves of a slot: what the workgroup has room for, while each has a block
  const int blocks = (a.G + kEsBlock - 1) / kEsBlock;
  const int kw = std::min(kTokenWaves / a.topk, blocks);
  const dim3 grid(unsigned((a.N + 31) / 32));
  if (kw >= 4)
    hipLaunchKernelGGL((experts_skinny<XT, 1, 4, false, true>), grid, dim3(64 * 4 * a.topk), 0,
                       stream, a);
  else if (kw >= 2)
    hipLaunchKernelGGL((experts_skinny<XT, 1, 2, false, true>), grid, dim3(64 * 2 * a.topk), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((experts_skinny<XT, 1, 1, false, true>), grid, dim3(64 * a.topk), 0, stream,
                       a);
  return hipGetLastError();
}

// The arguments of a call; fp32 activations' limbs are made on the way.
hipError_t prepare(const MoeExperts &p, ExpertArgs &a, hipStream_t stream) {
  a.X = p.X;
  a.ldx = p.K;
  a.factor = nullptr;
  if (p.dtype == W4A16_DTYPE_F32) {
    const LimbLayout at = limb_layout(p.workspace, p.rows_x, p.K, p.dtype);
    const hipError_t e = launch_limbs(p, stream);
    if (e != hipSuccess) return e;
    a.X = at.limbs;
    a.factor = at.factor;
    a.ldx = at.KP;
  }
  a.token_index = p.token_index;
  a.offsets = p.expert_offsets;
  a.qw = reinterpret_cast<const uint4 *>(p.qweight);
  a.sc = p.scales;
  a.Y = p.Y;
  a.rows_x = p.rows_x;
  a.R = p.R;
  a.E = p.E;
  a.N = p.N;
  a.G = p.K / kGroup;
  a.ldy = p.ldy;
  a.tiles_n = 0;
  a.slots = nullptr;
  a.weights = nullptr;
  a.topk = 0;
  return hipSuccess;
}

}  // namespace

// Where the one-token form is the faster: a launch less (4.5 us), but a workgroup
// has all of a column's slots to read, at 28 bytes a ns (20 with two limbs) where
// the tiles of the general form share them out over the card, 4200 a ns (bf16, us
// general against one-token: 8 slots of 7168 x 2048 22.2, 18.0; 4 of 7168 x 512
// 9.8, 5.1; 8 of 2080 x 1408 13.1, 12.1, fp32 16.6, 18.2; 2 of 1024 x 4096 12.0,
// 8.7, 4 of them 12.9, 15.1).
bool experts_token(long T, long topk, int N, int K, int dtype) {
  const long groups = (long(N) + 31) / 32;
  if (T != 1 || topk > kTokenWaves || groups > kMaxBlocks / 4) return false;
  const double bytes = 20.0 * K * topk;  // of a workgroup: 32 rows, 5/8 byte a weight
  return bytes / (dtype == W4A16_DTYPE_F32 ? 20e3 : 28e3) <= 4.5 + groups * bytes / 4.2e6;
}

hipError_t launch_experts_token(const MoeExperts &p, const int32_t *slots, const float *weights,
                                int topk, hipStream_t stream) {
  ExpertArgs a;
  const hipError_t e = prepare(p, a, stream);
  if (e != hipSuccess) return e;
  a.slots = slots;
  a.weights = weights;
  a.topk = topk;
  switch (p.dtype) {
    case W4A16_DTYPE_F32: return run_token<float>(a, stream);
    case W4A16_DTYPE_F16: return run_token<_Float16>(a, stream);
    default: return run_token<Bf16>(a, stream);
  }
}

hipError_t launch_experts_skinny(const MoeExperts &p, hipStream_t stream) {
  ExpertArgs a;
  const hipError_t e = prepare(p, a, stream);
  if (e != hipSuccess) return e;
  switch (p.dtype) {
    case W4A16_DTYPE_F32:
      return p.swiglu ? run_skinny_type<float, true>(a, stream)
                      : run_skinny_type<float, false>(a, stream);
    case W4A16_DTYPE_F16:
      return p.swiglu ? run_skinny_type<_Float16, true>(a, stream)
                      : run_skinny_type<_Float16, false>(a, stream);
    default:
      return p.swiglu ? run_skinny_type<Bf16, true>(a, stream)
                      : run_skinny_type<Bf16, false>(a, stream);
  }
}

}  // namespace w4a16
