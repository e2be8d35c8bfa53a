// Experts' W4A16 products for few slots per expert, in fp32, fp16 and bf16:
// D[r] = x_r . W_e^T for every slot r of expert e (stored as fp32, for the
// combination of slots), or the fused gate/up form H[r] = silu(x_r . gate_e^T)
// * (x_r . up_e^T) in the activations' type.  The pages run their MoE experts
// and the SwiGLU MLP through the INT4 path ("The Quiet Commit: How a Single
// Documentation Edit Marks the Completion of a Major Engineering Milestone",
// section "The INT4 Milestone").
//
// Bound by reading the active experts' weights once (5/8 byte a weight): the
// weights and the activations go from memory straight to registers, P steps of
// 4 groups ahead, and nothing waits at a barrier before the end.
//
// Arithmetic, on 16x16x32 matrix instructions (A: 16 slots, B: 16 rows of W,
// K: one group of 32), fp32 accumulation, one fp32 FMA per output and group
// for the group's scale:
//   fp32  two fp16 limbs of each activation, scaled by a power of two per slot
//         and pair of groups, the low limb x2^11 and met by the codes x2^-11
//         (22 significant bits; every product exact in fp32);
//   fp16  the activations as they are and the exact codes q - 8;
//   bf16  the activations as they are and q + 16, which two VALU instructions
//         per pair of codes make: an instruction on a B of -24 throughout gives
//         the accumulator that takes the offset out again.  The terms are up
//         to 31 + 24 units of the scale instead of 8 and cancel, so the fp32
//         sums lose up to 3 bits more (2^-21 beside an output rounded to
//         2^-8); nothing is spent per activation.
//
// Mapping: lane (c, R) (c = lane % 16, R = lane / 16) loads the 16 bytes of
// group 4 s + R of W row c (64 contiguous bytes of each of 16 rows per
// instruction); two lane swaps across the four lane rows give it word R of
// each of the step's 4 groups, its B operand.  Its A operand is k = 8R .. 8R+7
// of slot c, D holds slots 4R .. 4R+3 of W row c.  A workgroup takes MT x 16
// slots of one expert by NT x 16 rows of W (gate tiles, then the up tiles of
// the same outputs); its 8 waves take steps in turn (neighbouring waves read
// neighbouring bytes) and their sums are added in wave order in LDS.

#include "moe_common.h"
#include "gemv_common.h"
#include "limbs.h"

#include <algorithm>

namespace w4a16 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kEsWaves = 8;
constexpr int kEsThreads = 64 * kEsWaves;

// 8 activations x0..x7 in the order x0 x4 x1 x5 x2 x6 x3 x7 (that of the
// nibble conversions)
__device__ __forceinline__ u32x4m interleave8(u32x4m a) {
  return u32x4m{__builtin_amdgcn_perm(a.z, a.x, 0x05040100u),
                __builtin_amdgcn_perm(a.z, a.x, 0x07060302u),
                __builtin_amdgcn_perm(a.w, a.y, 0x05040100u),
                __builtin_amdgcn_perm(a.w, a.y, 0x07060302u)};
}

// bf16 q + 16 of the 8 nibbles of w: dword p holds nibbles p and p + 4.  In
// [16, 32) a bf16 has 3 bits behind the point, so a nibble stands at bits 3..6.
__device__ __forceinline__ bf16x8 nibbles_to_bf16_16(uint32_t w) {
  const uint32_t p0 = __builtin_amdgcn_bitop3_b32(w << 3, 0x00780078u, 0x41804180u, 0xEA);
  const uint32_t p1 = __builtin_amdgcn_bitop3_b32(w >> 1, 0x00780078u, 0x41804180u, 0xEA);
  const uint32_t p2 = __builtin_amdgcn_bitop3_b32(w >> 5, 0x00780078u, 0x41804180u, 0xEA);
  const uint32_t p3 = __builtin_amdgcn_bitop3_b32(w >> 9, 0x00780078u, 0x41804180u, 0xEA);
  return __builtin_bit_cast(bf16x8, u32x4m{p0, p1, p2, p3});
}

template <typename XT>
struct XChunk;  // k = 8R .. 8R+7 of one group of one slot
template <>
struct XChunk<float> {
  float4 lo, hi;
};
template <>
struct XChunk<_Float16> {
  u32x4m v;
};
template <>
struct XChunk<Bf16> {
  u32x4m v;
};

struct ExpertArgs {
  const void *X;               // [rows][K] activations
  const int32_t *token_index;  // slot -> row of X, or null: the slot itself
  const int32_t *offsets;      // [E + 1]
  const uint4 *qw;             // [E][N or 2N][G] groups of 16 bytes
  const float *sc;             // [E][N or 2N][G]
  void *Y;                     // [R][ldy]
  int rows_x, R, E, N, G, ldy, tiles_n;
};

// kSw: W has 2N rows, Y is XT; else Y is fp32.
template <typename XT, int MT, int NT, int P, bool kSw>
__global__ void __launch_bounds__(kEsThreads) experts_skinny(ExpertArgs a) {
  constexpr int NO = kSw ? NT / 2 : NT;
  constexpr bool kLimbs = sizeof(XT) == 4;
  constexpr int kTile = MT * NT * 256;
  __shared__ __align__(16) float red[kEsWaves * kTile];
  __shared__ __align__(16) float es_inv[kLimbs ? kEsWaves * 16 * MT : 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int c = lane & 15, R = lane >> 4;
  const int item = int(blockIdx.x / unsigned(a.tiles_n));
  const int n0 = int(blockIdx.x - unsigned(item) * unsigned(a.tiles_n)) * 16 * NO;
  const ExpertItem it = find_item(a.offsets, a.E, a.R, 16 * MT, item);
  if (it.e < 0) return;  // uniform over the workgroup
  const int G = a.G, N = a.N;
  const long K = long(G) * kGroup;

  // this lane's rows of W (clamped: rows past N are computed and not stored)
  const uint4 *wrow[NT];
  const float *srow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const long n = std::min(n0 + 16 * (t % NO) + c, N - 1) + (kSw && t >= NO ? long(N) : 0);
    const long row = long(it.e) * (kSw ? 2 * long(N) : long(N)) + n;
    wrow[t] = a.qw + row * G;
    srow[t] = a.sc + row * G;
  }
  // and of the activations (slots past the item repeat its last)
  const XT *xrow[MT];
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const int slot = it.row0 + std::min(16 * u + c, it.rows - 1);
    long row = slot;
    if (a.token_index) row = std::min(std::max(a.token_index[slot], 0), a.rows_x - 1);
    xrow[u] = static_cast<const XT *>(a.X) + row * K + 8 * R;
  }

  struct Ops {
    u32x4m w[NT];
    float4 s[NT];
    XChunk<XT> x[MT][4];
  };
  const int S = G / 4;  // whole steps
  auto load_x = [&](XChunk<XT> &d, int u, long g) {
    if constexpr (kLimbs) {
      const float4 *p = reinterpret_cast<const float4 *>(xrow[u] + g * kGroup);
      d.lo = p[0];
      d.hi = p[1];
    } else {
      d.v = *reinterpret_cast<const u32x4m *>(xrow[u] + g * kGroup);
    }
  };
  auto load = [&](Ops &o, int s) {
    const long g = 4 * long(s);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      o.w[t] = __builtin_nontemporal_load(reinterpret_cast<const u32x4m *>(wrow[t] + g + R));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f32x4u v = *reinterpret_cast<const f32x4u *>(srow[t] + g);
      o.s[t] = make_float4(v.x, v.y, v.z, v.w);
    }
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) load_x(o.x[u][q], u, g + q);
  };
  // the step past the whole ones: groups past G read group G - 1 and are
  // left out of the products
  auto load_tail = [&](Ops &o) {
    const long g = 4 * long(S);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      o.w[t] = *reinterpret_cast<const u32x4m *>(wrow[t] + std::min(g + R, long(G) - 1));
      o.s[t].x = srow[t][std::min(g + 0, long(G) - 1)];
      o.s[t].y = srow[t][std::min(g + 1, long(G) - 1)];
      o.s[t].z = srow[t][std::min(g + 2, long(G) - 1)];
      o.s[t].w = srow[t][std::min(g + 3, long(G) - 1)];
    }
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) load_x(o.x[u][q], u, std::min(g + q, long(G) - 1));
  };

  float acc[MT][NT][4];
#pragma unroll
  for (int u = 0; u < MT; ++u)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[u][t][r] = 0.0f;
  const floatx4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  // one group's products of 16-bit activations
  auto group16 = [&](const Ops &o, const u32x4m (&w)[NT], int q) {
#pragma unroll
    for (int u = 0; u < MT; ++u) {
      if constexpr (!kLimbs) {
        const u32x4m xa = interleave8(o.x[u][q].v);
        floatx4 d0 = zero;
        if constexpr (sizeof(XT) == 2 && !__is_same(XT, _Float16)) {
          const bf16x8 off = __builtin_bit_cast(
              bf16x8, u32x4m{0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u});  // -24
          d0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa), off, zero, 0,
                                                       0, 0);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          floatx4 d;
          if constexpr (__is_same(XT, _Float16))
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, xa),
                                                       nibbles_to_f16(w[t][q]), zero, 0, 0, 0);
          else
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa),
                                                        nibbles_to_bf16_16(w[t][q]), d0, 0, 0, 0);
          const float s4[4] = {o.s[t].x, o.s[t].y, o.s[t].z, o.s[t].w};
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[u][t][r] = fmaf(s4[q], d[r], acc[u][t][r]);
        }
      }
    }
  };
  // a pair of groups' products of fp32 activations (two: the pair is whole)
  float *inv = es_inv + wave * 16 * MT;
  auto pair32 = [&](const Ops &o, const u32x4m (&w)[NT], int q0, bool two) {
    if constexpr (kLimbs) {
      float up[MT];
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        // the slot's largest magnitude in the pair: this lane's 16 values,
        // then the slot's 4 lanes
        const float4 a0 = o.x[u][q0].lo, a1 = o.x[u][q0].hi;
        const float4 a2 = o.x[u][q0 + 1].lo, a3 = o.x[u][q0 + 1].hi;
        const float t0 = limb_absmax3(a0.x, a0.y, a0.z), t1 = limb_absmax3(a0.w, a1.x, a1.y);
        const float t2 = limb_absmax3(a1.z, a1.w, a2.x), t3 = limb_absmax3(a2.y, a2.z, a2.w);
        const float t4 = limb_absmax3(a3.x, a3.y, a3.z), t5 = limb_absmax3(t0, t1, a3.w);
        float mx = limb_absmax3(t2, t3, t4);
        mx = limb_absmax3(mx, t5, 0.0f);
        const auto h32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx),
                                                          false, false);
        mx = limb_absmax3(__uint_as_float(h32[0]), __uint_as_float(h32[1]), 0.0f);
        const auto h16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(mx), __float_as_uint(mx),
                                                          false, false);
        mx = limb_absmax3(__uint_as_float(h16[0]), __uint_as_float(h16[1]), 0.0f);
        // e in [-113, 116]: 2^-e and 2^(e+11) are normal, x 2^(e+11) finite
        const int e = std::min(row_exponent(mx), 116);
        if (R == 0) inv[16 * u + c] = __int_as_float((127 - e) << 23);
        up[u] = __int_as_float((127 + e + 11) << 23);
      }
      // this wave's own words (its LDS operations complete in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      float4 fac[MT];
#pragma unroll
      for (int u = 0; u < MT; ++u)
        fac[u] = *reinterpret_cast<const float4 *>(inv + 16 * u + 4 * R);
      float ss[MT][NT][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q == 1 && !two) break;
        half8_t hi[MT], lo[MT];
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          const float4 x0 = o.x[u][q0 + q].lo, x1 = o.x[u][q0 + q].hi;
          const float va[4] = {x0.x, x0.y, x0.z, x0.w}, vb[4] = {x1.x, x1.y, x1.z, x1.w};
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            limb_split2(va[i] * up[u], vb[i] * up[u], 0x1p-11f, -2048.0f, hw[i], lw[i]);
          hi[u] = __builtin_bit_cast(half8_t, make_uint4(hw[0], hw[1], hw[2], hw[3]));
          lo[u] = __builtin_bit_cast(half8_t, make_uint4(lw[0], lw[1], lw[2], lw[3]));
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const half8_t b = nibbles_to_f16(w[t][q0 + q]);
          const _Float16 k2 = (_Float16)0x1p-11f;
          const half8_t b2 = b * half8_t{k2, k2, k2, k2, k2, k2, k2, k2};  // exact in fp16
          const float s4[4] = {o.s[t].x, o.s[t].y, o.s[t].z, o.s[t].w};
          const float sq = s4[q0 + q];
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            floatx4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi[u], b, zero, 0, 0, 0);
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo[u], b2, d, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              ss[u][t][r] = q == 0 ? sq * d[r] : fmaf(sq, d[r], ss[u][t][r]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const float f[4] = {fac[u].x, fac[u].y, fac[u].z, fac[u].w};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[u][t][r] = fmaf(ss[u][t][r], f[r], acc[u][t][r]);
      }
    }
  };
  // left: groups of the step (4, or fewer in the last one)
  auto process = [&](const Ops &o, int left) {
    u32x4m w[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w[t] = o.w[t];
      transpose_words(w[t]);
    }
    if constexpr (kLimbs) {
      pair32(o, w, 0, left > 1);
      if (left > 2) pair32(o, w, 2, left > 3);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < left) group16(o, w, q);
    }
  };

  // wave w takes steps w, w + 8, ...; a ring of P steps in registers
  Ops ring[P];
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (wave + p * kEsWaves < S) load(ring[p], wave + p * kEsWaves);
  for (int s = wave; s < S; s += P * kEsWaves) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = s + p * kEsWaves;
      if (at >= S) break;
      process(ring[p], 4);
      // refilled after its last use: the ring keeps its registers over the
      // loop's back edge, and a step waits for its own loads only
      __builtin_amdgcn_sched_barrier(0);
      if (at + P * kEsWaves < S) load(ring[p], at + P * kEsWaves);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // the last G % 4 groups, on the wave whose turn it would be
  if (G % 4 != 0 && wave == S % kEsWaves) {
    Ops o;
    load_tail(o);
    process(o, G % 4);
  }

#pragma unroll
  for (int u = 0; u < MT; ++u)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[wave * kTile + ((u * NT + t) * 4 + r) * 64 + lane] = acc[u][t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NO * 256; i += kEsThreads) {
    const int l = i & 63, r = (i >> 6) & 3, ut = i >> 8;
    const int u = ut / NO, t = ut - u * NO;
    const int at = ((u * NT + t) * 4 + r) * 64 + l;
    const int m = 16 * u + 4 * (l >> 4) + r, n = n0 + 16 * t + (l & 15);
    if (m >= it.rows || n >= N) continue;
    float g = 0.0f, v = 0.0f;
#pragma unroll
    for (int w = 0; w < kEsWaves; ++w) {
      g += red[w * kTile + at];
      if constexpr (kSw) v += red[w * kTile + at + NO * 256];
    }
    const long y = long(it.row0 + m) * a.ldy + n;
    if constexpr (kSw)
      static_cast<XT *>(a.Y)[y] = from_f32<XT>(silu_mul(g, v));
    else
      static_cast<float *>(a.Y)[y] = g;
  }
}

template <typename XT, int MT, int NT, int P, bool kSw>
hipError_t run_skinny(ExpertArgs a, hipStream_t stream) {
  constexpr int NO = kSw ? NT / 2 : NT;
  a.tiles_n = (a.N + 16 * NO - 1) / (16 * NO);
  const long blocks = long(a.tiles_n) * max_items(a.R, a.E, 16 * MT);
  if (blocks < 1 || blocks > 0x7fffffffL) return hipErrorInvalidValue;
  hipLaunchKernelGGL((experts_skinny<XT, MT, NT, P, kSw>), dim3(unsigned(blocks)),
                     dim3(kEsThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename XT, bool kSw>
hipError_t run_skinny_type(const ExpertArgs &a, hipStream_t stream) {
  switch (experts_skinny_rows(a.R, a.E)) {
    case 16: return run_skinny<XT, 1, 4, 2, kSw>(a, stream);
    case 32: return run_skinny<XT, 2, 4, 2, kSw>(a, stream);
    default: return run_skinny<XT, 4, 2, sizeof(XT) == 4 ? 1 : 2, kSw>(a, stream);
  }
}

}  // namespace

// slots per workgroup: enough for one block of most experts
int experts_skinny_rows(long R, long E) {
  const double mean = double(R) / double(std::max(1L, std::min(R, E)));
  return mean <= 10.0 ? 16 : mean <= 24.0 ? 32 : 64;
}

hipError_t launch_experts_skinny(const MoeExperts &p, hipStream_t stream) {
  ExpertArgs a;
  a.X = p.X;
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
