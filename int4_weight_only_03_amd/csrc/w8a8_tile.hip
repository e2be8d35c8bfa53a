// 8-bit products for many rows: Y[r] = x_r . W_e^T in tiles on the matrix instructions.
//
// Arithmetic: the sum over a block of 128 features is one 16x16x128 fp8 instruction (A: 16
// rows of W, B: 16 slots, C: 0), and one fp32 FMA per output adds it up with its scales'
// product.  The fp8 instructions add products 8 at a time, each cut off 13 bits below the
// largest one's power of two (measured; the sums of 8 then add up in fp32), which moves a
// result by at most 7 * 2^-13 of sum |x w| and, on normally distributed values, by 2^-16.1 in
// the root mean square (2^-14.9 where a hundredth of the activations is 20 times the others,
// 2^-14.05 where the weights are so too).  Stored bf16 results are further off by 0.0% to 0.1%
// for it, fp16 ones by 0.2%, 1.2% and 4% (6.5% with a twentieth of both 50 times the others), and
// anything that is exact takes twice the time (4096 x 4096 x 7168: 101 us, 218).  fp32 outputs
// take the codes as fp16, exactly, on the 16x16x32 fp16 instructions instead.
//
// A tile is 16 WU GU slots by 16 WT GT rows of W: GU x GT waves take 16 WU slots by 16 WT rows
// each, in turn, so that a half-full tile's work is spread over them.  G such groups of
// waves share a tile and take its blocks of features in turn; their sums are added in LDS at
// the end, in the order of the groups.  A stage is one block for each group.  Rows of 128
// bytes, and the slots' scales, come to LDS by direct copies into a ring of S stages, S - 1 of
// them in flight, and one barrier a stage; the rows of W go on to registers while the
// products before them are still under way, so that their image is free a stage earlier and a
// stage begins with the fetch of 16 slots.
//
// Few tiles are bound by latency: a stage takes 0.4 us whatever is in it (64 x 64, one group,
// 256 x 4096 x 7168: 19.6 us), so groups and small tiles, which put more of K and more of the
// card to work, win until the tiles are more than the card (64 x 64 with two groups 16.9; 64
// rows with 32 x 32 and four 10.5).  The largest are bound by power: 256 x 256 runs 8192 x 8192
// x 8192 in 455 us, 2.4 PFLOP/s, the matrix units busy for 56% of the cycles at 1.9 GHz (2.4
// without load); left out, the copies between L2 and LDS would save 18%, the FMAs 5%, operand
// reads from LDS nothing.  Instructions and FMAs alone, in registers, reach 3.7 PFLOP/s.
// Tried without gain there: operands 1 to 3 steps ahead, copies at once or spread over the
// stage, half of the waves half a stage behind the others, scales 4 blocks at a time, 32x32x64
// instructions (3.3 PFLOP/s in registers).  By expert (16384 slots of 32 experts of 4096 x 7168,
// shares from half to one and a half times the mean): part-filled tiles behind all the others
// 578 us for 537, as they read their weights once more, all at one time; XCDs' runs cut by
// cost, a half-full tile as half of one, 611 for 550; to every XCD an eighth of every expert's
// tiles 563 for 555.  What stands idle leaves power to the others, so what counts is the
// products that padding adds, not how evenly they are dealt.
//
// Tiles are dealt so that each XCD works a contiguous run of them (the hardware deals
// workgroups round-robin over the 8 XCDs); see in_band for their order.

#include "w8a8_choice.h"
#include "w8a8_common.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void t8_lds_void;

struct TileArgs {
  const uint8_t *X;
  const float *xs;
  const int32_t *token_index, *offsets;
  const uint8_t *W;
  const float *ws;
  void *Y;
  int rows_x, R, E, N, K, KB, NB, tiles_n;
  bool vec;  // rows of Y begin and end at 16 bytes
};

template <int VM>
__device__ __forceinline__ void t8_wait_copies() {  // at most VM still in flight
  static_assert(VM >= 0 && VM < 64, "wait count");
  __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | 0x70 | (15 << 8));
}
__device__ __forceinline__ void t8_wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | 0x70);  // lgkmcnt(0)
}
__device__ __forceinline__ void t8_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// Direct copy of 16 bytes per lane (from base + offset, or from `from`), lane i to
// lds + 16 i; as asm so that the compiler does not wait for it at every LDS read (the
// kernel's own waits and barriers order the copies).  The LDS address is wave-uniform (m0).
__device__ __forceinline__ void t8_copy16(const uint8_t *base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 1\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(offset), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void t8_copy16(const uint8_t *from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 1\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(from), "s"(lds) : "memory", "m0");
}

__device__ __forceinline__ void t8_copy4(const float *from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 1\n\tglobal_load_lds_dword %0, off"
               :: "v"(from), "s"(lds) : "memory", "m0");
}

// One block of features of 16 rows: 32 codes to a lane, as they are or in fp16.
template <bool kExact>
struct Operand;
template <>
struct Operand<false> {
  i32x8 v;
  __device__ __forceinline__ void set(u32x4m a, u32x4m b) {
    v = i32x8{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
  }
};
template <>
struct Operand<true> {
  half8v v[4];
  __device__ __forceinline__ void set(u32x4m a, u32x4m b) {
    v[0] = widen8(a.x, a.y);
    v[1] = widen8(a.z, a.w);
    v[2] = widen8(b.x, b.y);
    v[3] = widen8(b.z, b.w);
  }
};
__device__ __forceinline__ f32x4 block_sum(const Operand<false> &w, const Operand<false> &x) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, zero, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_sum(const Operand<true> &w, const Operand<true> &x) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[j], x.v[j], d, 0, 0, 0);
  return d;
}

// Tile `i` of `tiles_m` x `tiles_n`: bands of kBand blocks of slots, in a band the blocks of
// slots fastest, so that the 32 tiles that an XCD holds at once are about 4 x 8 and share
// their operands in its L2 (8192 x 8192 x 8192: 556 us with all of an expert's blocks of slots
// fastest, 494 so; 4 and 8 of them alike).
constexpr int kBand = 4;
__device__ __forceinline__ void in_band(long i, int tiles_m, int tiles_n, int &bm, int &bn) {
  const long band = i / (long(kBand) * tiles_n);
  const int within = int(i - band * kBand * tiles_n);
  const int high = std::min(kBand, tiles_m - int(band) * kBand);
  bm = int(band) * kBand + within % high;
  bn = within / high;
}

template <int WU, int WT, int GU, int GT, int G, int S, typename OT, bool kExact>
__global__ void __launch_bounds__(64 * GU * GT * G, G * GU * GT > 8 ? G * GU * GT / 4 : 2)
gemm8_tile(TileArgs a) {
  constexpr int kWaves = GU * GT;  // of a group
  constexpr int TM = 16 * WU * GU, TN = 16 * WT * GT;  // slots and rows of W of a tile
  constexpr int kX = TM * 128, kImage = kX + TN * 128;
  static_assert(128 % (16 * WT) == 0, "a wave's rows of W share their scales");
  constexpr int kS = TM;  // slots' scales in LDS
  static_assert(TM % kWaves == 0 && TM / kWaves <= 64, "a wave copies its share of the scales");
  // Row r at 128 r, logical chunk x (16 bytes) at chunk x ^ ((r / 2) % 8), so that the 16
  // rows an operand read touches fall in distinct banks.
  __shared__ __align__(16) unsigned char mem[S * G * kImage];
  constexpr int kWB = (TN + 127) / 128;  // blocks of W rows
  static_assert((TN % 128 == 0 || 128 % TN == 0) && kWB <= kWaves, "blocks of W rows");
  __shared__ __align__(16) float scale[S * G * kS];  // of the slots, by blocks
  __shared__ __align__(16) float wscale[2 * kWB * 64];  // of W's blocks, by runs of 64
  const int tid = threadIdx.x, lane = tid & 63;
  const int kg = G == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6) / kWaves;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) - kg * kWaves;
  const int c = lane & 15, R = lane >> 4;
  const int wu = wave % GU, wt = wave / GU;

  // tile of this workgroup: XCD b % 8 takes a contiguous run of the tiles there are
  int e = 0, bm, bn, e0 = 0, e1 = a.R;
  {
    const long index = long(blockIdx.x >> 3);
    if (a.offsets) {
      ExpertItem it = find_item(a.offsets, a.E, a.R, TM, 0);
      const long tiles = long(it.total) * a.tiles_n, run = (tiles + 7) / 8;
      const long tile = long(blockIdx.x & 7) * run + index;
      if (index >= run || tile >= tiles) return;  // uniform over the workgroup
      it = find_item(a.offsets, a.E, a.R, TM, int(tile / a.tiles_n));
      in_band(tile - (tile / a.tiles_n - it.block) * a.tiles_n, it.blocks, a.tiles_n, bm, bn);
      e = it.e;
      expert_slots(a.offsets, e, a.R, e0, e1);
    } else {
      const int tiles_m = (a.R + TM - 1) / TM;
      const long tiles = long(tiles_m) * a.tiles_n, run = (tiles + 7) / 8;
      const long tile = long(blockIdx.x & 7) * run + index;
      if (index >= run || tile >= tiles) return;
      in_band(tile, tiles_m, a.tiles_n, bm, bn);
    }
  }
  const int row0 = e0 + bm * TM, rows = std::min(TM, e1 - row0);
  const int n0 = bn * TN;
  const long K = a.K;

  // Copies: wave w issues those of 8 rows each from w on, kWaves apart, of both operands.
  // Lane i copies 16 bytes of row 8 j + i / 8.  Slots past the item repeat its last, rows of W
  // past N repeat row N - 1.  LDS row 16 t + i of a wave's strip of W holds its row
  // 4 WT (i / 4) + 4 t + i % 4, so that a lane's sums are neighbouring outputs.
  constexpr int kXC = TM / 8 / kWaves, kWC = TN / 8 / kWaves, kAll = kXC + kWC + 1;  // 1: scales
  static_assert(TM % (8 * kWaves) == 0 && TN % (8 * kWaves) == 0 && kWaves % 2 == 0,
                "copies deal out evenly");
  const uint8_t *wbase = a.W + (long(e) * a.N + n0) * K;
  const uint8_t *xat[kXC];
  uint32_t wat[kWC];
#pragma unroll
  for (int j = 0; j < kXC; ++j) {
    long row = row0 + std::min(8 * (wave + j * kWaves) + lane / 8, rows - 1);
    if (a.token_index) row = std::min(std::max(a.token_index[row], 0), a.rows_x - 1);
    xat[j] = a.X + row * K;
  }
#pragma unroll
  for (int j = 0; j < kWC; ++j) {
    const int r = 8 * (wave + j * kWaves) + lane / 8;
    const int strip = r / (16 * WT), t = r % (16 * WT) / 16, i = r % 16;
    const int n = std::min(16 * WT * strip + 4 * WT * (i / 4) + 4 * t + i % 4, a.N - 1 - n0);
    wat[j] = uint32_t(n) * uint32_t(a.K);
  }
  // the chunk that a lane copies, the same in all of a wave's copies: their blocks of 8 rows
  // are all even or all odd
  const uint32_t chunk = 16 * ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>((const t8_lds_void *)mem));
  // the ring of S stages of G blocks
  auto image_of = [&](int p) { return uint32_t(p & (S * G - 1)); };
  // where a lane reads in its rows for block p; behind their end (the last block of K may be
  // shorter than 128) their last 16 bytes once more
  auto offset_of = [&](int p) {
    return std::min(uint32_t(p) * kBlock8 + chunk, uint32_t(a.K) - 16);
  };
  // copy j of block p's slots and of its rows of W
  auto copy_x = [&](int j, int p, uint32_t at) {
    t8_copy16(xat[j] + at, lds0 + image_of(p) * kImage + 1024 * (wave + j * kWaves));
  };
  auto copy_w = [&](int j, int p, uint32_t at) {
    t8_copy16(wbase, wat[j] + at, lds0 + image_of(p) * kImage + kX + 1024 * (wave + j * kWaves));
  };
  // zeros in place of W's codes that were copied from behind the rows' end, and of X's
  auto clear_behind = [&](int p, uint32_t to, int copies) {
    if (uint32_t(p) * kBlock8 + chunk < uint32_t(a.K)) return;
#pragma unroll
    for (int j = 0; j < copies; ++j)
      *reinterpret_cast<u32x4m *>(mem + image_of(p) * kImage + to + 1024 * (wave + j * kWaves) +
                                  16 * lane) = u32x4m{0, 0, 0, 0};
  };

  // scales: every wave copies those of as many slots, so that every wave has as many copies
  // in flight (a lane's lies in a cache line of its own: where all waves copied 64 slots' each,
  // most of them twice, 256 x 256 took 10% longer)
  constexpr int kSC = kS / kWaves;
  const uint32_t scale0 = uint32_t(reinterpret_cast<uintptr_t>((const t8_lds_void *)scale));
  const float *sx = a.xs;
  {
    long row = row0 + std::min(kSC * wave + lane, rows - 1);
    if (a.token_index) row = std::min(std::max(a.token_index[row], 0), a.rows_x - 1);
    sx += row * a.KB;
  }
  auto copy_scales = [&](int p) {
    if (lane < kSC)
      t8_copy4(sx + std::min(p, a.KB - 1), scale0 + (image_of(p) * kS + kSC * wave) * 4);
  };
  // scales of W: wave i copies those of block i of the tile's rows, of 64 blocks of K at once
  const uint32_t wscale0 = uint32_t(reinterpret_cast<uintptr_t>((const t8_lds_void *)wscale));
  auto copy_wscales = [&](int p) {
    if (kg > 0 || wave >= kWB) return;
    const long block = long(e) * a.NB + std::min(n0 / kBlock8 + wave, a.NB - 1);
    t8_copy4(a.ws + block * a.KB + std::min(p + lane, a.KB - 1),
             wscale0 + ((p >> 6 & 1) * kWB + wave) * 256);
  };

  // operand reads: the wave's slots 16 (GU u + wu) + c, chunks R and 4 + R
  uint32_t read[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) read[q] = uint32_t(c * 128 + 16 * ((4 * q + R) ^ ((c >> 1) & 7)));
  const uint32_t xread = uint32_t(16 * wu) * 128, wread = kX + uint32_t(16 * WT * wt) * 128;
  const int sread = 16 * wu + c;

  constexpr int kDelay = 2;
  f32x4 acc[WU][WT];
#pragma unroll
  for (int u = 0; u < WU; ++u)
#pragma unroll
    for (int t = 0; t < WT; ++t) acc[u][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // The products of block p with the wave's first A tiles of 16 slots, and, between them, the
  // copies for S - 1 stages on and the fetch of the next block's rows of W.  The FMAs of a sum
  // stand kDelay products behind it (right behind it they would wait 12 cycles each: 125 us of
  // 4096 x 4096 x 7168 then, 114 so); slots are fetched kAhead steps of WT products ahead.
  u32x4m wraw[WT][2];
  auto fetch_w = [&](int t, int p) {
    const unsigned char *img = mem + image_of(p) * kImage + wread + 2048 * t;
    wraw[t][0] = *reinterpret_cast<const u32x4m *>(img + read[0]);
    wraw[t][1] = *reinterpret_cast<const u32x4m *>(img + read[1]);
  };
  auto multiply = [&](auto active, int p) {
    constexpr int A = decltype(active)::value;
    constexpr int kAhead = A > 1 && A < 6 ? 2 : 1, kN = A * WT, kIssue = kN / 2;
    const unsigned char *img = mem + image_of(p) * kImage;
    // behind the last block it is copied once more, into images that nobody reads again:
    // without a condition every wave has as many copies in flight
    const uint32_t xoff = offset_of(p + (S - 1) * G), woff = offset_of(p + S * G);
    const float *s = scale + int(image_of(p)) * kS + sread;
    const float fw = wscale[((p >> 6 & 1) * kWB + 16 * WT * wt / kBlock8) * 64 + (p & 63)];
    Operand<kExact> w[WT], x[kAhead + 1];
#pragma unroll
    for (int t = 0; t < WT; ++t) w[t].set(wraw[t][0], wraw[t][1]);
    f32x4 d[kDelay];
    float f[kAhead + 1], g = 0.0f;
    auto fetch = [&](int u) {
      const unsigned char *at = img + xread + 2048 * GU * u;
      x[u % (kAhead + 1)].set(*reinterpret_cast<const u32x4m *>(at + read[0]),
                              *reinterpret_cast<const u32x4m *>(at + read[1]));
      f[u % (kAhead + 1)] = s[16 * GU * u];
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(u);
    __builtin_amdgcn_sched_barrier(0);
    copy_scales(p + (S - 1) * G);
#pragma unroll
    for (int i = 0; i < kN + kDelay; ++i) {
      const int u = i / WT, t = i % WT;
      f32x4 now;
      if (i < kN) now = block_sum(w[t], x[u % (kAhead + 1)]);
      __builtin_amdgcn_sched_barrier(0);
      if (i >= kDelay) {
        const int v = (i - kDelay) / WT, o = (i - kDelay) % WT;
        if (o == 0) g = f[v % (kAhead + 1)] * fw;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[v][o][r] = fmaf(g, d[i % kDelay][r], acc[v][o][r]);
        // here, not sunk to where the sums are used next: their products would stay in
        // registers till then
        asm volatile("" : "+v"(acc[v][o]));
      }
      if (i < kN) d[i % kDelay] = now;
      if (i < kN && t == kDelay - 1 && u + kAhead < A) fetch(u + kAhead);
#pragma unroll
      for (int j = 0; j < kXC + kWC; ++j) {
        if (j * kIssue / (kXC + kWC) != i) continue;
        if (j < kXC)
          copy_x(j, p + (S - 1) * G, xoff);
        else
          copy_w(j - kXC, p + S * G, woff);
      }
      if (i >= kN - WT && i < kN) fetch_w(t, p + G);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // At a stage's start its copies have landed in this wave; past the barrier they have in
  // every wave, and every wave is past the stage before, whose image is then filled again.
  copy_wscales(0);
#pragma unroll
  for (int j = 0; j < kWC; ++j) copy_w(j, kg, offset_of(kg));
  for (int q = 0; q < S - 1; ++q) {
    const int p = q * G + kg;
    copy_scales(p);
#pragma unroll
    for (int j = 0; j < kXC; ++j) copy_x(j, p, offset_of(p));
#pragma unroll
    for (int j = 0; j < kWC; ++j) copy_w(j, p + G, offset_of(p + G));
  }
  // waits until the copies of all but the last n stages are here
  auto landed = [&](auto n) {
    constexpr int kStages = decltype(n)::value;
    t8_wait_copies<kStages * kAll>();
  };
  landed(std::integral_constant<int, S - 1>());
  if (kBlock8 * (kg + 1) > a.K) clear_behind(kg, kX, kWC);
  t8_wait_lds();
  t8_barrier();
#pragma unroll
  for (int t = 0; t < WT; ++t) fetch_w(t, kg);
  // the first stage in which a block may be short
  const int last = a.K % kBlock8 ? a.KB - 2 * G : a.KB;
  auto stages = [&](auto active) {
    for (int q = 0; q < a.KB; q += G) {
      const int p = q + kg;  // the group's block
      landed(std::integral_constant<int, S - 2>());
      if (q >= last) {
        clear_behind(p, 0, kXC);
        clear_behind(p + G, kX, kWC);
      }
      t8_wait_lds();
      t8_barrier();
      if ((q & 63) == 0 && q + 64 < a.KB) copy_wscales(q + 64);
      if (p < a.KB) multiply(active, p);
    }
  };
  // A tile that is half full, or less, does half the products (4096 tokens, 4 of 32 experts of
  // 4096 x 7168: 628 us without, 595 so), a large one that is three quarters full those (16384
  // slots of such experts with shares from half to one and a half times the mean: 555, 550).
  if (WU >= 4 && rows <= TM / 4)
    stages(std::integral_constant<int, WU >= 4 ? WU / 4 : WU>());
  else if (WU >= 4 && rows <= TM / 2)
    stages(std::integral_constant<int, WU >= 4 ? WU / 2 : WU>());
  else if (WU >= 8 && rows <= 3 * TM / 4)
    stages(std::integral_constant<int, WU >= 8 ? 3 * WU / 4 : WU>());
  else
    stages(std::integral_constant<int, WU>());
  t8_wait_copies<0>();  // the LDS is the next workgroup's, or the sums'

  if constexpr (G > 1) {
    // the groups' sums, added in their order; group i takes the slots u = i, i + G, ...
    static_assert(sizeof(mem) >= G * kWaves * WU * WT * 1024, "room for all sums");
    static_assert(WU % G == 0 || G % WU == 0, "slots deal out evenly");
    t8_barrier();
    f32x4 *const sums = reinterpret_cast<f32x4 *>(mem);
#pragma unroll
    for (int u = 0; u < WU; ++u)
#pragma unroll
      for (int t = 0; t < WT; ++t)
        sums[((kg * kWaves + wave) * WU * WT + u * WT + t) * 64 + lane] = acc[u][t];
    t8_wait_lds();
    t8_barrier();
#pragma unroll
    for (int u = 0; u < WU; ++u) {
      if (u % G != kg) continue;
#pragma unroll
      for (int t = 0; t < WT; ++t) {
        f32x4 v = sums[(wave * WU * WT + u * WT + t) * 64 + lane];
#pragma unroll
        for (int i = 1; i < G; ++i)
          v += sums[((i * kWaves + wave) * WU * WT + u * WT + t) * 64 + lane];
        acc[u][t] = v;
      }
    }
  }

  OT *y = static_cast<OT *>(a.Y) + long(row0) * a.N + n0;
  const int n = 16 * WT * wt + 4 * WT * R, cols = std::min(TN, a.N - n0);  // of the tile
  // Whole vectors straight from the sums, where they are a good part of a cache line: of fp32
  // in tiles of 128 rows a lane's 16 outputs take four stores, each to 64 places, and the way
  // through LDS below is the faster (4096 x 4096 x 1024: 51.6 us, 44.3 so; 64 x 64 tiles and
  // 16-bit outputs lose by it: 500 x 1408 x 2064 11.9, 12.3; 4096 x 4096 x 1024 in bf16 22.5,
  // 26.2).
  if (a.vec && (sizeof(OT) == 2 || WT < 4)) {
    constexpr int kV = std::min(int(16 / sizeof(OT)), 4 * WT);
    struct alignas(kV * sizeof(OT)) Some {
      OT v[kV];
    };
#pragma unroll
    for (int u = 0; u < WU; ++u) {
      const int m = 16 * (GU * u + wu) + c;
      if (m >= rows || u % G != kg) continue;
#pragma unroll
      for (int v = 0; v < 4 * WT / kV; ++v) {
        Some o;
#pragma unroll
        for (int i = 0; i < kV; ++i)
          o.v[i] = from_f32<OT>(acc[u][(kV * v + i) / 4][(kV * v + i) % 4]);
        if (n + kV * v < cols) *reinterpret_cast<Some *>(y + long(m) * a.N + n + kV * v) = o;
      }
    }
    return;
  }
  // Rows that begin anywhere: to LDS first, each row as far behind a multiple of 16 bytes as
  // in memory, so that whole 16 bytes of it are read and stored (4096 x 4095 x 7168, bf16: 107
  // us, 144 with single outputs stored from the sums).
  constexpr int kV = 16 / sizeof(OT), kPitch = TN + kV, kChunks = TN / kV + 1;
  constexpr int kPart = WU * 16 * GU * kPitch * sizeof(OT) <= sizeof(mem) ? WU : WU / 2;
  static_assert(kPart * 16 * GU * kPitch * sizeof(OT) <= sizeof(mem), "room for the outputs");
  OT *const out = reinterpret_cast<OT *>(mem);
  auto behind = [&](int m) {
    return int((reinterpret_cast<uintptr_t>(y + long(m) * a.N) & 15) / sizeof(OT));
  };
#pragma unroll
  for (int u0 = 0; u0 < WU; u0 += kPart) {
    t8_wait_lds();
    t8_barrier();  // nobody reads what is there any more
    const int m0 = 16 * GU * u0, m1 = std::min(rows, m0 + 16 * GU * kPart);
#pragma unroll
    for (int u = u0; u < u0 + kPart; ++u) {
      const int m = 16 * (GU * u + wu) + c;
      if (m >= rows || u % G != kg) continue;
      OT *to = out + (m - m0) * kPitch + behind(m) + n;
#pragma unroll
      for (int i = 0; i < 4 * WT; ++i) to[i] = from_f32<OT>(acc[u][i / 4][i % 4]);
    }
    t8_wait_lds();
    t8_barrier();
    for (int i = tid; i < (m1 - m0) * kChunks; i += 64 * kWaves * G) {
      const int m = m0 + i / kChunks, at = kV * (i % kChunks);
      struct alignas(16) Chunk {
        OT v[kV];
      };
      const Chunk o = *reinterpret_cast<const Chunk *>(out + (m - m0) * kPitch + at);
      const int first = at - behind(m);  // column
      OT *to = y + long(m) * a.N + first;
      if (first >= 0 && first + kV <= cols) {
        *reinterpret_cast<Chunk *>(to) = o;
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (first + j >= 0 && first + j < cols) to[j] = o.v[j];
      }
    }
  }
}

TileCall call_of(const Gemm8 &p) { return {p.R, p.E, p.N, p.K, p.expert_offsets != nullptr}; }

template <int WU, int WT, int GU, int GT, int G, int S, typename OT, bool kExact>
hipError_t run_tile8(const Gemm8 &p, hipStream_t stream) {
  constexpr int TM = 16 * WU * GU, TN = 16 * WT * GT;
  TileArgs a;
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
  a.tiles_n = int((long(p.N) + TN - 1) / TN);
  constexpr int kV = 16 / sizeof(OT);
  a.vec = p.N % kV == 0 && reinterpret_cast<uintptr_t>(p.Y) % 16 == 0;
  const long tiles = tiles_of(TM, TN, call_of(p), p.R);
  if (tiles > most_tiles(GU * GT * G)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm8_tile<WU, WT, GU, GT, G, S, OT, kExact>),
                     dim3(unsigned((tiles + 7) / 8 * 8)), dim3(64 * GU * GT * G), 0, stream, a);
  return hipGetLastError();
}

template <typename OT>
hipError_t run_type8(const Gemm8 &p, hipStream_t stream) {
  switch (least(kChoices, call_of(p), p.R).choice) {
    case -1: return hipErrorInvalidConfiguration;
    case 0: return run_tile8<1, 1, 1, 2, 4, 4, OT, false>(p, stream);
    case 1: return run_tile8<1, 1, 2, 2, 4, 4, OT, false>(p, stream);
    case 2: return run_tile8<1, 2, 2, 2, 2, 4, OT, false>(p, stream);
    case 3: return run_tile8<2, 2, 2, 2, 2, 4, OT, false>(p, stream);
    case 4: return run_tile8<2, 2, 2, 2, 1, 4, OT, false>(p, stream);
    case 5: return run_tile8<2, 4, 2, 2, 1, 4, OT, false>(p, stream);
    case 6: return run_tile8<4, 4, 2, 2, 1, 4, OT, false>(p, stream);
    case 7: return run_tile8<4, 4, 2, 2, 1, 2, OT, false>(p, stream);
    default: return run_tile8<8, 4, 2, 4, 1, 2, OT, false>(p, stream);
  }
}

hipError_t run_exact8(const Gemm8 &p, hipStream_t stream) {
  switch (least(kExactChoices, call_of(p), p.R).choice) {
    case -1: return hipErrorInvalidConfiguration;
    case 0: return run_tile8<1, 1, 1, 2, 4, 4, float, true>(p, stream);
    case 1: return run_tile8<1, 1, 2, 2, 4, 4, float, true>(p, stream);
    case 2: return run_tile8<1, 2, 2, 2, 2, 4, float, true>(p, stream);
    case 3: return run_tile8<2, 2, 2, 2, 2, 4, float, true>(p, stream);
    case 4: return run_tile8<2, 2, 2, 2, 1, 4, float, true>(p, stream);
    default: return run_tile8<4, 4, 2, 2, 1, 2, float, true>(p, stream);
  }
}

}  // namespace

// Few rows: the skinny kernel.  Of one expert (4096 rows of W x 7168, us skinny against the
// tiles): 1 row 7.1, 7.7 (fp32 outputs 7.2, 9.3), 4 rows 7.8, 7.8, 16 rows 10.4, 8.1; of many by
// their mean (32 of the same): 2 155, 159; 8 167, 160 (fp32 168, 170); 10 175, 160 (176, 171); 16
// 246, 162 (247, 177); 60 of 2080 x 1408 with 4 36.1, 36.9 (36.5, 41.3), with 10 39.4, 37.4
// (39.8, 44.3).  Up to 10 they are within a tenth of each other, either way, and the skinny
// kernel's sums are exact.
int gemm8_kernel(long R, long E, bool grouped) {
  if (!grouped) return R <= 4 ? W8A8_KERNEL_SKINNY : W8A8_KERNEL_TILE;
  return R <= 10 * std::max(1L, std::min(R, E)) ? W8A8_KERNEL_SKINNY : W8A8_KERNEL_TILE;
}

hipError_t launch_gemm8(const Gemm8 &p, hipStream_t stream) {
  return gemm8_kernel(p.R, p.E, p.expert_offsets != nullptr) == W8A8_KERNEL_TILE
             ? launch_gemm8_tile(p, stream)
             : launch_gemm8_skinny(p, stream);
}

hipError_t launch_gemm8_tile(const Gemm8 &p, hipStream_t stream) {
  auto run = [&](const Gemm8 &part) {
    switch (p.dtype) {
      case W4A16_DTYPE_F32: return run_exact8(part, stream);
      case W4A16_DTYPE_F16: return run_type8<_Float16>(part, stream);
      default: return run_type8<Bf16>(part, stream);
    }
  };
  const bool exact = p.dtype == W4A16_DTYPE_F32;
  const long rows = exact ? rows_before_rest(kExactChoices, call_of(p))
                          : rows_before_rest(kChoices, call_of(p));
  Gemm8 part = p;
  part.R = part.rows_x = int(rows);
  if (p.expert_offsets) part.rows_x = p.rows_x;
  const hipError_t e = run(part);
  if (e != hipSuccess || rows >= p.R) return e;
  part.R = part.rows_x = int(p.R - rows);
  part.X += rows * p.K;
  part.xs += rows * blocks8(p.K);
  part.Y = static_cast<unsigned char *>(p.Y) + rows * p.N * (exact ? 4 : 2);
  return run(part);
}

}  // namespace w4a16
