// Shared by the mixture-of-experts kernels (moe_route.hip, moe_skinny.hip,
// moe_tile.hip, moe_combine.hip): stores of the three activation types and the
// assignment of workgroups to (expert, block of slots) items.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "w4a16_internal.h"

namespace w4a16 {
namespace {

struct Bf16 {
  uint16_t v;
};
typedef unsigned int u32x4m __attribute__((ext_vector_type(4)));

// power of two that the low limb of an fp32 activation is carried with
constexpr float kLowScale = 2048.0f;

// fp32 to the activation type, to nearest even (one rounding per output)
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ _Float16 from_f32<_Float16>(float x) {
  return _Float16(x);
}
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float x) {
  return Bf16{__builtin_bit_cast(uint16_t, __bf16(x))};
}

// Slots [r0, r1) of expert e, clamped into [0, R] (malformed offsets give
// wrong values, never an access out of bounds).
__device__ __forceinline__ void expert_slots(const int32_t *__restrict__ offsets, int e, int R,
                                             int &r0, int &r1) {
  r0 = min(max(offsets[e], 0), R);
  r1 = min(max(offsets[e + 1], r0), R);
}

// A launch of 256 threads a workgroup has at most this many (2^32 threads).
constexpr long kMaxBlocks = (1L << 24) - 8;

struct ExpertItem {
  int e;      // expert, -1 behind the last item
  int row0;   // first slot of the item
  int rows;   // slots of the item, at most B
  int block;  // which block of B slots of the expert
  int blocks; // the expert's number of blocks
  int total;  // items of the launch
};

// More items than any launch has workgroups for.  A lane's count stops there, so that
// the counts of lists that overlap (malformed offsets, up to E / 2 times R slots) do
// not pass 32 bits: an item would be looked for where there is none, and its first
// slot lie out of range.
constexpr int kMostItems = 1 << 24;

// Item `item` of the list (expert, block of up to B of its slots), experts
// ascending.  Every lane of a wave calls it with the same arguments and gets
// the same answer.  Lane l counts the blocks of experts l*per .. l*per+per-1
// (one round of loads for up to 64 experts, independent loads after that), a
// scan over the wave finds the owner, and the owner walks its experts.
__device__ __forceinline__ ExpertItem find_item(const int32_t *__restrict__ offsets, int E, int R,
                                                int B, int item) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < E) {
      int r0, r1;
      expert_slots(offsets, e, R, r0, r1);
      mine = min(mine + (r1 - r0 + B - 1) / B, kMostItems);
    }
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(incl, d, 64);
    if (lane >= d) incl += up;
  }
  ExpertItem it;
  it.total = __builtin_amdgcn_readlane(incl, 63);
  it.e = -1;
  it.row0 = it.rows = it.block = it.blocks = 0;
  if (item >= it.total) return it;
  const unsigned long long over = __ballot(incl > item);
  const int owner = __builtin_ctzll(over);
  int rest = item - (incl - mine);  // the owner's: item within its experts
  int e = 0, row0 = 0, rows = 0, block = 0, blocks = 0;
  if (lane == owner) {
    for (int i = 0; i < per; ++i) {
      e = lane * per + i;
      if (e >= E) break;  // not reached: the owner has more than `rest` blocks
      int r0, r1;
      expert_slots(offsets, e, R, r0, r1);
      const int n = (r1 - r0 + B - 1) / B;
      if (rest < n) {
        block = rest;
        blocks = n;
        row0 = r0 + rest * B;
        rows = min(B, r1 - row0);
        break;
      }
      rest -= n;
    }
  }
  it.e = __builtin_amdgcn_readlane(e, owner);
  it.row0 = __builtin_amdgcn_readlane(row0, owner);
  it.rows = __builtin_amdgcn_readlane(rows, owner);
  it.block = __builtin_amdgcn_readlane(block, owner);
  it.blocks = __builtin_amdgcn_readlane(blocks, owner);
  return it;
}

// The most items there can be: every expert with a slot adds at most one
// partly filled block.
inline long max_items(long R, long E, long B) {
  const long active = R < E ? R : E;
  return (R + (B - 1) * active) / B;
}

// Lane row R (16 lanes) holds words 0..3 of group R in v0..v3; afterwards word
// R of groups 0..3 (permlane32_swap exchanges the upper half of its first
// operand with the lower half of its second, permlane16_swap the odd 16-lane
// rows of the first with the even rows of the second).
__device__ __forceinline__ void transpose_words(u32x4m &v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v = u32x4m{c[0], c[1], d[0], d[1]};
}

}  // namespace
}  // namespace w4a16
