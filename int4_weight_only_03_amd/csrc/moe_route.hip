// Routing of tokens to experts, and the slot lists of the grouped products.
//
// The pages' engine routes every token of an MoE layer before its INT4 experts
// run ("The Quiet Commit: How a Single Documentation Edit Marks the Completion
// of a Major Engineering Milestone", section "The Context: A Native DDTree
// Engine Takes Shape").
//
// Mathematics, per token: score s_e = 1 / (1 + exp(-l_e)) or softmax(l)_e, key
// c_e = s_e + b_e; with groups, a group is worth the sum of its one or two
// largest keys and only experts of the best groups stay; the topk largest keys
// are taken, ties to the lowest index; weights are the chosen scores
// (optionally divided by their sum) times a factor.  An expert whose logit or
// key is NaN or -inf is masked: never taken, and a token with too few experts
// left gets empty places (-1).
//
// The choice is that of 64-bit keys.  Without a bias the scores are in the
// logits' order, so the logits themselves are compared.  Otherwise a token's
// keys are computed in fp32 first; if any two values whose order decides
// something lie closer than their errors, the token is done again with 64-bit
// keys (about 1 token in 1000 at 256 experts).
//
// Slots are sorted by expert, then token.  A block of tokens counts its
// choices per expert; a second kernel sums the blocks before its own and ranks
// each choice inside its block (past 2^14 tokens or so a small kernel between adds
// the counts up, so that reading them does not grow with the square of the tokens).
// A token takes an expert at most once, so 64
// tokens' choices of an expert are one 64-bit mask, ORed together in LDS (any
// order gives the same mask), and a choice's rank is a population count: no
// result depends on the order of atomics.  One block of up to 64 tokens does
// both in one launch, and one wave does a single token.
//
// A token is worked on by LP lanes, expert e in register e / LP of lane e % LP:
// by a whole wave where tokens are few (a pick's chain of dependent reductions
// is what takes the time), by 16 lanes, four tokens a wave, where they are many
// (the same instructions serve four tokens).
//
// Bound: at few tokens by launch and the picks' latency (one token of 256 experts
// 6.3 us, 64 of 160 12.0); at many by VALU issue of the selection (16384 of 256
// experts: 26 us to choose, 7 of them the few tokens' 64-bit keys at the end, and
// 8 for the lists, where reading the logits takes 4).

#include "moe_common.h"

#include <algorithm>
#include <cmath>

namespace w4a16 {
namespace {

constexpr int kRtWaves = 16;
constexpr int kRtThreads = 64 * kRtWaves;
constexpr int kRtMaxBlocks = 256; // blocks of the second kernel

struct RouteArgs {
  const void *logits;
  const float *bias;           // [E] or null
  const int32_t *num_tokens;   // [1] or null
  int32_t *ids;                // [T][topk]
  float *weights;              // [T][topk]
  int32_t *slots;              // [T][topk]
  int32_t *token_index;        // [T * topk]
  int32_t *offsets;            // [E + 1]
  int32_t *counts;             // [blocks][padded(E)]
  int T, E, topk, groups, group_limit, group_top, sigmoid, renormalize, dtype;
  float scale;
  int at_once, blocks;         // the first kernel's tokens per block, blocks
  int chunk;                   // the second's tokens per block (a multiple of 64)
  int step;                    // blocks of the first that a row of counts it reads stands for
};

// row of the counts: a multiple of 4 experts
__host__ __device__ constexpr int padded(int E) { return (E + 3) & ~3; }

constexpr float kNegInf = -__builtin_huge_valf();

// fp32: exp2 of the rounded product; the product's rounding is an error of
// |x| 2^-24 of the result, at most 0.37 * 2^-24 absolute for x <= 0, and so is
// the instruction's, 2^-23 relative
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }  // 1 ulp
__device__ __forceinline__ double inverse(double x) { return 1.0 / x; }

__device__ __forceinline__ float read_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}

// A lane of the other half of this lane's aligned run of 2 D lanes (the xor
// partner, or for D = 4 and 8 the mirrored lane: the same where each half holds
// one value throughout, as it does in a butterfly).
template <int D>
__device__ __forceinline__ int other_half(int v) {
  if constexpr (D == 1) {
    return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xf, 0xf, false);
  } else if constexpr (D == 2) {
    return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xf, 0xf, false);
  } else if constexpr (D == 4) {
    return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xf, 0xf, false);
  } else if constexpr (D == 8) {
    return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xf, 0xf, false);
  } else if constexpr (D == 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(uint32_t(v), uint32_t(v), false, false);
    return int((threadIdx.x & 16) ? p[0] : p[1]);
  } else {
    const auto p = __builtin_amdgcn_permlane32_swap(uint32_t(v), uint32_t(v), false, false);
    return int((threadIdx.x & 32) ? p[0] : p[1]);
  }
}
template <int D>
__device__ __forceinline__ float other_half(float v) {
  return __int_as_float(other_half<D>(__float_as_int(v)));
}
template <int D>
__device__ __forceinline__ double other_half(double v) {
  return __hiloint2double(other_half<D>(__double2hiint(v)), other_half<D>(__double2loint(v)));
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

// over a token's LP lanes; every lane gets the result
template <int LP, typename V>
__device__ __forceinline__ V token_max(V v) {
  v = larger(v, other_half<1>(v));
  v = larger(v, other_half<2>(v));
  v = larger(v, other_half<4>(v));
  v = larger(v, other_half<8>(v));
  if constexpr (LP == 64) {
    v = larger(v, other_half<16>(v));
    v = larger(v, other_half<32>(v));
  }
  return v;
}
template <int LP>
__device__ __forceinline__ int token_min(int v) {
  v = min(v, other_half<1>(v));
  v = min(v, other_half<2>(v));
  v = min(v, other_half<4>(v));
  v = min(v, other_half<8>(v));
  if constexpr (LP == 64) {
    v = min(v, other_half<16>(v));
    v = min(v, other_half<32>(v));
  }
  return v;
}
template <int LP>
__device__ __forceinline__ double token_sum(double v) {
  v += other_half<1>(v);
  v += other_half<2>(v);
  v += other_half<4>(v);
  v += other_half<8>(v);
  if constexpr (LP == 64) {
    v += other_half<16>(v);
    v += other_half<32>(v);
  }
  return v;
}

// the value of lane I of this lane's row of 16
template <int I>
__device__ __forceinline__ int row_lane(int v) {
  return __builtin_amdgcn_update_dpp(v, v, 0x150 + I, 0xf, 0xf, false);
}
template <int I>
__device__ __forceinline__ float row_lane(float v) {
  return __int_as_float(row_lane<I>(__float_as_int(v)));
}
template <int I>
__device__ __forceinline__ double row_lane(double v) {
  return __hiloint2double(row_lane<I>(__double2hiint(v)), row_lane<I>(__double2loint(v)));
}

// the two largest values of both halves
template <int D, typename KT>
__device__ __forceinline__ void merge_two(KT &m1, KT &m2) {
  const KT o1 = other_half<D>(m1), o2 = other_half<D>(m2);
  m2 = o1 > m1 ? (m1 > o2 ? m1 : o2) : (o1 > m2 ? o1 : m2);
  m1 = o1 > m1 ? o1 : m1;
}

// What an fp32 score is off by: at most 5 * 2^-24.  Sigmoid: s (1 - s) |x| 2^-24 < 0.3
// (the exponent's rounding), 0.5 (exp2, 1 ulp of e s^2), 1 (the sum) and 2 (the
// reciprocal, 1 ulp) of 2^-24 times s.  Softmax: terms 0.4 + 2, the products and the
// reciprocal of their sum 5 in proportion to s, which two scores share 1 of.  A bias
// added rounds once more, by 2^-24 of the key.
constexpr float kUnit = 0x1p-24f;

// whether two fp32 keys lie closer than their errors (and the difference's rounding)
template <typename KT>
__device__ __forceinline__ bool too_close(KT hi, KT lo) {
  if constexpr (sizeof(KT) == 8) return false;  // 64-bit keys decide as they are
  const float d = float(hi) - float(lo);
  return !(d > 12 * kUnit + 4 * kUnit * fmaxf(fabsf(float(hi)), fabsf(float(lo))));
}

// What the sum of n keys of magnitudes `size` together is off by: 5 units and its
// rounding for each, and the roundings of their sum and of adding this error to it.
// The keys may cancel, so their sum says nothing of it (one expert favoured by 10^4
// beside one disfavoured by as much: worth about 1, off by up to 10^-3).
__device__ __forceinline__ float worth_error(int n, float size) {
  return kUnit * (6.0f * float(n) + 3.0f * size);
}

// Rank of a group of value `value` among a token's: h runs over the groups, g is
// its own index.  Group g is held by lanes g L .. g L + L - 1 of the token's.
template <typename KT>
__device__ __forceinline__ int above(KT v, int h, KT value, int g) {
  return (v > value || (v == value && h < g)) ? 1 : 0;
}
template <int I, typename KT>
__device__ __forceinline__ void rank_row(KT value, int g, int L, int groups, int &rank) {
  if ((I & (L - 1)) == 0 && I < groups * L)  // uniform
    rank += above(row_lane<I>(value), I / L, value, g);
  if constexpr (I < 15) rank_row<I + 1>(value, g, L, groups, rank);
}

// The logits of up to 64 tokens that threads work on together: row t - first of
// them starts at base + (t - first) * E elements.  Reads past the last row give
// 0 (and are masked), so a lane needs no clamp and its reads differ in constants.
struct Rows {
  const char *base;  // uniform
  uint32_t bytes;    // of all the rows
  uint32_t at;       // this lane's token's row, elements
  int E, dtype;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, int(bytes), 0x00027000);
}

// logits of experts r LP + l, masked ones (NaN, -inf, none there, token not
// live) -inf
template <int LP, int NV>
__device__ __forceinline__ void load_logits(const Rows &w, bool live, float (&x)[NV]) {
  const int l = threadIdx.x & (LP - 1);
  const __amdgpu_buffer_rsrc_t rs = resource(w.base, w.bytes);
  const uint32_t at = w.at + uint32_t(l);
  if (w.dtype == W4A16_DTYPE_F32) {
#pragma unroll
    for (int r = 0; r < NV; ++r)
      x[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, int(at * 4) + r * LP * 4, 0, 0));
  } else {
    uint16_t h[NV];
#pragma unroll
    for (int r = 0; r < NV; ++r)
      h[r] = __builtin_amdgcn_raw_buffer_load_b16(rs, int(at * 2) + r * LP * 2, 0, 0);
#pragma unroll
    for (int r = 0; r < NV; ++r)
      x[r] = w.dtype == W4A16_DTYPE_F16 ? float(__builtin_bit_cast(_Float16, h[r]))
                                        : __uint_as_float(uint32_t(h[r]) << 16);
  }
#pragma unroll
  for (int r = 0; r < NV; ++r)
    x[r] = (live && r * LP + l < w.E && x[r] > kNegInf) ? x[r] : kNegInf;
}

__device__ __forceinline__ float load_logit(const Rows &w, int e) {
  const __amdgpu_buffer_rsrc_t rs = resource(w.base, w.bytes);
  const uint32_t at = w.at + uint32_t(e);
  if (w.dtype == W4A16_DTYPE_F32)
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, int(at * 4), 0, 0));
  const uint16_t h = __builtin_amdgcn_raw_buffer_load_b16(rs, int(at * 2), 0, 0);
  return w.dtype == W4A16_DTYPE_F16 ? float(__builtin_bit_cast(_Float16, h))
                                    : __uint_as_float(uint32_t(h) << 16);
}

// What a token's selection needs of the call.
struct Select {
  const float *bias;
  int topk, groups, group_limit, group_top;
};

// Order a token's experts by keys of type KT; false on a lane of a token that
// fp32 cannot tell.  kBias: keys are s + b, else the logits.  keys: the token's
// LDS room of LP * NV values (used with groups only).  top: largest logit, sum:
// sum of exp(l - top) (softmax).  Lane j of the token leaves with its j-th
// choice, -1 where none.
template <typename KT, int LP, int NV, bool kBias, bool kSigmoid>
__device__ __forceinline__ bool select_experts(const Select &a, int E, const float (&x)[NV],
                                               float top, double sum, KT *keys, int &chosen) {
  const int l = threadIdx.x & (LP - 1);
  const bool grouped = a.group_limit < a.groups;
  // groups are valued by the keys, or by the scores where two are added
  const bool scores = kBias || (grouped && a.group_top == 2);
  const KT low = KT(kNegInf);
  KT key[NV];
#pragma unroll
  for (int r = 0; r < NV; ++r) key[r] = KT(x[r]);
  if (scores) {
    KT value[NV];
    const KT over = kSigmoid ? KT(1) : inverse(KT(sum));
#pragma unroll
    for (int r = 0; r < NV; ++r) {
      const KT p = exp_of(kSigmoid ? -KT(x[r]) : KT(x[r]) - KT(top));
      value[r] = kSigmoid ? inverse(KT(1) + p) : (x[r] == top ? KT(1) : p) * over;
    }
    if constexpr (kBias) {
      const __amdgpu_buffer_rsrc_t rs = resource(a.bias, uint32_t(E) * 4u);
      float b[NV];
#pragma unroll
      for (int r = 0; r < NV; ++r)
        b[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, 4 * l + r * LP * 4, 0, 0));
#pragma unroll
      for (int r = 0; r < NV; ++r) {
        value[r] += KT(b[r]);
        value[r] = value[r] > low ? value[r] : low;  // a NaN or -inf bias masks
      }
    }
#pragma unroll
    for (int r = 0; r < NV; ++r) {
      value[r] = x[r] > kNegInf ? value[r] : low;
      if (kBias) key[r] = value[r];
    }
    if (grouped) {
#pragma unroll
      for (int r = 0; r < NV; ++r) keys[r * LP + l] = value[r];
    }
  } else if (grouped) {
#pragma unroll
    for (int r = 0; r < NV; ++r) keys[r * LP + l] = key[r];
  }
  bool sure = true;
  if (grouped) {
    // groups side by side, L lanes (a power of two) each, a lane taking every
    // L-th of the group's experts; the two largest are merged across them
    const int L = 1 << (31 - __clz(LP / a.groups));
    const int gs = E / a.groups;
    const int g = l / L;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    KT m1 = low, m2 = low;
    if (g < a.groups)
      for (int i = l - g * L; i < gs; i += L) {
        const KT v = keys[g * gs + i];
        m2 = v > m1 ? m1 : (v > m2 ? v : m2);
        m1 = v > m1 ? v : m1;
      }
    if (L > 1) merge_two<1>(m1, m2);
    if (L > 2) merge_two<2>(m1, m2);
    if (L > 4) merge_two<4>(m1, m2);
    if (L > 8) merge_two<8>(m1, m2);
    if (LP == 64 && L > 16) merge_two<16>(m1, m2);
    if (LP == 64 && L > 32) merge_two<32>(m1, m2);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // before the room is written again
    __builtin_amdgcn_wave_barrier();
    const bool two = a.group_top == 2 && m2 > low;
    const KT value = two ? m1 + m2 : m1;
    int rank = 0;
    if constexpr (LP == 64) {
      for (int h = 0; h < a.groups; ++h) rank += above(read_lane(value, h * L), h, value, g);
    } else {
      rank_row<0>(value, g, L, a.groups, rank);
    }
    const bool open = g < a.groups && m1 > low, keep = open && rank < a.group_limit;
    const unsigned long long kept = __ballot(keep) >> ((threadIdx.x & 63) & ~(LP - 1));
    if constexpr (sizeof(KT) == 4) {
      // The least that a kept group can be worth against the most that another can.
      // A worth past fp32's range has an infinite error: a group kept above, or left
      // below, everything is passed over (NaN), any other leaves the token unsure.
      if (scores) {
        const float error = worth_error(two ? 2 : 1, fabsf(m1) + (two ? fabsf(m2) : 0.0f));
        const float least = -token_max<LP>(keep ? error - value : low);
        const float most = token_max<LP>(open && !keep ? value + error : low);
        sure = least > most;
      }
    }
    // e / gs = (e * ceil(2^20 / gs)) >> 20 for e < 1024 (gs < 1024: two groups
    // at least)
    const uint32_t over_gs = ((1u << 20) + uint32_t(gs) - 1) / uint32_t(gs);
#pragma unroll
    for (int r = 0; r < NV; ++r) {
      const uint32_t of = (uint32_t(r * LP + l) * over_gs) >> 20;
      key[r] = ((kept >> ((of * L) & 63)) & 1) ? key[r] : low;
    }
  }
  // topk + 1 picks: the last shows how near the first one left out comes
  chosen = -1;
  KT last = low;
  for (int j = 0; j <= a.topk; ++j) {
    KT m = key[0];
#pragma unroll
    for (int r = 1; r < NV; ++r) m = larger(m, key[r]);
    m = token_max<LP>(m);
    if (kBias && j > 0 && m > low && too_close(last, m)) sure = false;
    last = m;
    if (j == a.topk) break;
    int at = 0x7fffffff;  // the lowest expert that has it
#pragma unroll
    for (int r = NV - 1; r >= 0; --r) at = key[r] == m ? r * LP + l : at;
    at = token_min<LP>(at);
#pragma unroll
    for (int r = 0; r < NV; ++r) key[r] = at - l == r * LP ? low : key[r];
    if (l == j && m > low) chosen = at;
  }
  return sure;
}

// The selection in 64 bits: out of line, taken by few waves.
template <int LP, int NV, bool kBias, bool kSigmoid>
__device__ __noinline__ int select_64(Rows w, Select a, bool live, float top, double *keys) {
  // what is uniform comes in vector registers
  w.base = reinterpret_cast<const char *>(
      uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(uint64_t(w.base))))) |
      uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(uint64_t(w.base) >> 32)))) << 32);
  a.bias = reinterpret_cast<const float *>(
      uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(uint64_t(a.bias))))) |
      uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(uint64_t(a.bias) >> 32)))) << 32);
  w.bytes = uint32_t(__builtin_amdgcn_readfirstlane(int(w.bytes)));
  w.E = __builtin_amdgcn_readfirstlane(w.E);
  w.dtype = __builtin_amdgcn_readfirstlane(w.dtype);
  a.topk = __builtin_amdgcn_readfirstlane(a.topk);
  a.groups = __builtin_amdgcn_readfirstlane(a.groups);
  a.group_limit = __builtin_amdgcn_readfirstlane(a.group_limit);
  a.group_top = __builtin_amdgcn_readfirstlane(a.group_top);
  float x[NV];
  load_logits<LP, NV>(w, live, x);
  double sum = 0.0;
  if constexpr (!kSigmoid) {
#pragma unroll
    for (int r = 0; r < NV; ++r) {
      const double p = exp(double(x[r]) - double(top));
      sum += x[r] == top ? 1.0 : p;
    }
    sum = token_sum<LP>(sum);
  }
  int id;
  select_experts<double, LP, NV, kBias, kSigmoid>(a, w.E, x, top, sum, keys, id);
  return id;
}

// A token by LP lanes: lane j < topk leaves with its j-th choice and weight.
// Every token of the wave takes part, those that are not there (live false)
// with every expert masked.
template <int LP, int NV, bool kBias, bool kSigmoid>
__device__ __forceinline__ void route_token(const RouteArgs &a, const Rows &w, bool live,
                                            double *keys, int &id, float &weight) {
  const Select sel = {a.bias, a.topk, a.groups, a.group_limit, a.group_top};
  float x[NV];
  load_logits<LP, NV>(w, live, x);
  const bool grouped = a.group_limit < a.groups;
  const bool scores = kBias || (grouped && a.group_top == 2);
  float top = 0.0f;
  double sum = 1.0;
  if constexpr (!kSigmoid) {
    float m = x[0];
#pragma unroll
    for (int r = 1; r < NV; ++r) m = fmaxf(m, x[r]);
    top = token_max<LP>(m);
    if (scores || !a.renormalize) {
      // fp32 terms summed in 64 bits: the error of the sum is the terms' own
      double s = 0.0;
#pragma unroll
      for (int r = 0; r < NV; ++r) {
        const float p = expf(x[r] - top);
        s += double(x[r] == top ? 1.0f : p);
      }
      sum = token_sum<LP>(s);
    }
  }
  const bool sure = select_experts<float, LP, NV, kBias, kSigmoid>(
      sel, w.E, x, top, sum, reinterpret_cast<float *>(keys), id);
  if (__ballot(!sure) != 0) id = select_64<LP, NV, kBias, kSigmoid>(w, sel, live, top, keys);
  // the chosen scores, one per lane, in 64 bits (a score of 1e-40 still has a
  // share of the chosen ones' sum)
  const float c = load_logit(w, max(id, 0));
  const double p = exp(kSigmoid ? -double(c) : double(c) - double(top));
  double s = kSigmoid ? 1.0 / (1.0 + p) : (c == top ? 1.0 : p) / sum;
  s = id >= 0 ? s : 0.0;
  if (a.renormalize) {
    const double all = token_sum<LP>(s);
    s = all > 0.0 ? s / all : 0.0;
  }
  weight = float(s * double(a.scale));
}

__device__ __forceinline__ int live_tokens(const RouteArgs &a) {
  return a.num_tokens ? min(max(*a.num_tokens, 0), a.T) : a.T;
}

// Choices of tokens [t0, t0 + n), n <= kRtThreads / LP, into memory and, if
// kept, into LDS.
template <int LP, int NV, bool kBias, bool kSigmoid>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, int t0, int n, double *keys,
                                             int32_t *kept, int *hist) {
  const int l = threadIdx.x & (LP - 1), mine = threadIdx.x / LP, t = t0 + mine;
  double *room = keys + (a.group_limit < a.groups ? mine * LP * NV : 0);
  const int size = a.dtype == W4A16_DTYPE_F32 ? 4 : 2;
  Rows w;
  w.base = static_cast<const char *>(a.logits) + long(t0) * a.E * size;
  w.bytes = uint32_t(n) * uint32_t(a.E) * uint32_t(size);
  w.at = uint32_t(mine) * uint32_t(a.E);
  w.E = a.E;
  w.dtype = a.dtype;
  int id = -1;
  float weight = 0.0f;
  route_token<LP, NV, kBias, kSigmoid>(a, w, mine < n && t < live_tokens(a), room, id, weight);
  if (mine < n && l < a.topk) {
    a.ids[long(t) * a.topk + l] = id;
    a.weights[long(t) * a.topk + l] = weight;
    if (kept) kept[mine * a.topk + l] = id;
    if (hist && id >= 0) atomicAdd(&hist[id], 1);
  }
}

// In place: v[e] (e < E <= kRtThreads) becomes the sum of v[0..e-1], v[E] the
// total.  part: kRtWaves words.  Ends with a barrier.
__device__ __forceinline__ void scan_experts(int *v, int E, int *part) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int own = tid < E ? v[tid] : 0;
  int incl = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(incl, d, 64);
    if (lane >= d) incl += up;
  }
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += part[w];
  if (tid < E) v[tid] = before + incl - own;
  if (tid == E - 1) v[E] = before + incl;
  __syncthreads();
}

// Ranks of the choices of up to 64 tokens from t0 on: base[e] is the slot of
// the first of them that chose e, advanced past them.  ids: their choices.
__device__ __forceinline__ void place_choices(const RouteArgs &a, int t0, int n,
                                              const int32_t *ids, unsigned long long *mask,
                                              int *base) {
  const int tid = threadIdx.x;
  if (tid < a.E) mask[tid] = 0;
  __syncthreads();
  for (int i = tid; i < n * a.topk; i += kRtThreads) {
    const int id = ids[i];
    if (id >= 0) atomicOr(&mask[id], 1ull << (i / a.topk));
  }
  __syncthreads();
  for (int i = tid; i < n * a.topk; i += kRtThreads) {
    const int id = ids[i], t = i / a.topk;
    int slot = -1;
    if (id >= 0) {
      slot = base[id] + __popcll(mask[id] & ((1ull << t) - 1));
      a.token_index[slot] = t0 + t;
    }
    a.slots[long(t0) * a.topk + i] = slot;
  }
  __syncthreads();
  if (tid < a.E) base[tid] += __popcll(mask[tid]);
}

// LDS: masks [E], then `keys` of the tokens, then base [E + 1], part, the kept
// choices (one-launch form).
__host__ __device__ constexpr size_t route_lds(int E, int keys, int kept) {
  return size_t(E) * 8 + size_t(keys) * 8 + (size_t(E) + 1 + kRtWaves + kept) * 4;
}

// One token: its choices in the order of the experts are the slots, so a choice's
// slot is the number of chosen experts before its own; one wave, no barrier.
template <int NV, bool kBias, bool kSigmoid>
__global__ void __launch_bounds__(64) route_one(RouteArgs a) {
  extern __shared__ __align__(16) unsigned char rt_lds[];
  const int lane = threadIdx.x;
  const int size = a.dtype == W4A16_DTYPE_F32 ? 4 : 2;
  const Rows row = {static_cast<const char *>(a.logits), uint32_t(a.E) * uint32_t(size), 0, a.E,
                    a.dtype};
  int id = -1;
  float w = 0.0f;
  route_token<64, NV, kBias, kSigmoid>(a, row, live_tokens(a) > 0,
                                       reinterpret_cast<double *>(rt_lds), id, w);
  int slot = 0, n = 0;
  int start[NV + 1];  // chosen experts before 64 r + lane (the last: before 64 NV, lane 0)
#pragma unroll
  for (int r = 0; r <= NV; ++r) start[r] = 0;
  for (int j = 0; j < a.topk; ++j) {
    const int other = __builtin_amdgcn_readlane(id, j);
    if (other < 0) break;  // nor is there any behind it
    ++n;
    slot += other < id ? 1 : 0;
#pragma unroll
    for (int r = 0; r <= NV; ++r) start[r] += other < 64 * r + lane ? 1 : 0;
  }
  if (lane < a.topk) {
    a.ids[lane] = id;
    a.weights[lane] = w;
    a.slots[lane] = id < 0 ? -1 : slot;
    if (id >= 0) a.token_index[slot] = 0;
    if (lane >= n) a.token_index[lane] = -1;
  }
#pragma unroll
  for (int r = 0; r <= NV; ++r)
    if (64 * r + lane <= a.E) a.offsets[64 * r + lane] = start[r];
}

// Block b routes tokens [b kAtOnce, (b + 1) kAtOnce) and writes its counts.
// kSingle: there is one block, which builds the lists too.
template <int LP, int NV, bool kBias, bool kSigmoid, bool kSingle>
__global__ void __launch_bounds__(kRtThreads) route_choose(RouteArgs a) {
  extern __shared__ __align__(16) unsigned char rt_lds[];
  constexpr int kAtOnce = kRtThreads / LP;
  const bool grouped = a.group_limit < a.groups;
  auto *mask = reinterpret_cast<unsigned long long *>(rt_lds);
  auto *keys = reinterpret_cast<double *>(mask + a.E);
  auto *base = reinterpret_cast<int *>(keys + (grouped ? kRtThreads * NV : 0));
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * kAtOnce, n = min(kAtOnce, a.T - t0);
  if (tid < a.E) base[tid] = 0;
  __syncthreads();
  if constexpr (!kSingle) {
    route_tokens<LP, NV, kBias, kSigmoid>(a, t0, n, keys, nullptr, base);
    __syncthreads();
    const int row = padded(a.E);
    if (tid < row) a.counts[long(blockIdx.x) * row + tid] = tid < a.E ? base[tid] : 0;
  } else {
    int *part = base + a.E + 1;
    int32_t *kept = part + kRtWaves;
    route_tokens<LP, NV, kBias, kSigmoid>(a, t0, n, keys, kept, base);
    __syncthreads();
    scan_experts(base, a.E, part);
    for (int e = tid; e <= a.E; e += kRtThreads) a.offsets[e] = base[e];
    for (int r = base[a.E] + tid; r < a.T * a.topk; r += kRtThreads) a.token_index[r] = -1;
    __syncthreads();
    place_choices(a, 0, a.T, kept, mask, base);
  }
}

// Block b: the counts of the first kernel's blocks that make the second's block b,
// added up in place of the first of them.
__global__ void __launch_bounds__(kRtThreads) route_sums(RouteArgs a) {
  extern __shared__ __align__(16) unsigned char rt_lds[];
  auto *total = reinterpret_cast<int *>(rt_lds);  // [row]
  const int row = padded(a.E), tid = threadIdx.x;
  const int first = int(blockIdx.x) * a.step, end = min(first + a.step, a.blocks);
  if (tid < row) total[tid] = 0;
  __syncthreads();
  int width = 16;
  while (4 * width < row) width <<= 1;
  const int e = 4 * (tid & (width - 1));
  if (e < row) {
    int4 all = make_int4(0, 0, 0, 0);
#pragma unroll 8
    for (int k = first + tid / width; k < end; k += kRtThreads / width) {
      const int4 c = *reinterpret_cast<const int4 *>(a.counts + long(k) * row + e);
      all.x += c.x;
      all.y += c.y;
      all.z += c.z;
      all.w += c.w;
    }
    atomicAdd(&total[e], all.x);
    atomicAdd(&total[e + 1], all.y);
    atomicAdd(&total[e + 2], all.z);
    atomicAdd(&total[e + 3], all.w);
  }
  __syncthreads();
  if (tid < row) a.counts[long(first) * row + tid] = total[tid];
}

// Block b: slots of tokens [b chunk, (b + 1) chunk) from the counts of the first
// kernel's `blocks` blocks of at_once tokens, a row of them in every `step`.
__global__ void __launch_bounds__(kRtThreads) route_lists(RouteArgs a) {
  extern __shared__ __align__(16) unsigned char rt_lds[];
  const int row = padded(a.E);
  auto *mask = reinterpret_cast<unsigned long long *>(rt_lds);  // [E]
  auto *total = reinterpret_cast<int *>(mask + a.E);            // [row + 1]
  int *before = total + row + 1;                                // [row]
  int *part = before + row;                                     // [kRtWaves]
  const int tid = threadIdx.x;
  // rows of counts, and the row of its first token
  const int rows = (a.blocks + a.step - 1) / a.step;
  const int first = int(blockIdx.x) * (a.chunk / a.at_once / a.step);
  if (tid < row) total[tid] = before[tid] = 0;
  __syncthreads();
  // four experts a thread side by side, the blocks dealt to the thread groups
  // that are left, all of a group's loads in flight
  int width = 16;
  while (4 * width < row) width <<= 1;
  const int e = 4 * (tid & (width - 1));
  if (e < row) {
    int4 all = make_int4(0, 0, 0, 0), mine = all;
    const int step = kRtThreads / width;
#pragma unroll 8
    for (int k = tid / width; k < rows; k += step) {
      const int4 c = *reinterpret_cast<const int4 *>(a.counts + long(k) * a.step * row + e);
      const int own = k < first ? -1 : 0;
      all.x += c.x;
      all.y += c.y;
      all.z += c.z;
      all.w += c.w;
      mine.x += c.x & own;
      mine.y += c.y & own;
      mine.z += c.z & own;
      mine.w += c.w & own;
    }
    atomicAdd(&total[e], all.x);
    atomicAdd(&total[e + 1], all.y);
    atomicAdd(&total[e + 2], all.z);
    atomicAdd(&total[e + 3], all.w);
    atomicAdd(&before[e], mine.x);
    atomicAdd(&before[e + 1], mine.y);
    atomicAdd(&before[e + 2], mine.z);
    atomicAdd(&before[e + 3], mine.w);
  }
  __syncthreads();
  scan_experts(total, a.E, part);
  if (blockIdx.x == 0)
    for (int i = tid; i <= a.E; i += kRtThreads) a.offsets[i] = total[i];
  const long R = long(a.T) * a.topk;
  for (long r = total[a.E] + long(blockIdx.x) * kRtThreads + tid; r < R;
       r += long(gridDim.x) * kRtThreads)
    a.token_index[r] = -1;
  if (tid < a.E) before[tid] += total[tid];
  const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  for (int t = t0; t < t1; t += 64)  // place_choices begins and ends past barriers
    place_choices(a, t, min(64, t1 - t), a.ids + long(t) * a.topk, mask, before);
}

// Lanes per token: 16 (four tokens a wave) past 16 tokens, while their experts,
// choices and groups fit 16 lanes, but a whole wave for many experts and few
// tokens, whose blocks of 16 tokens fit the card at once.  us with 64 and 16 lanes
// (8 of E by sigmoid, bias and groups): E = 128, 64 tokens 13.8, 11.7, 4096 19.6,
// 19.3, 8192 27.0, 20.3; E = 160, 64 tokens 13.9, 13.5, 1024 17.1, 17.7, 8192
// 30.2, 23.7; E = 256, 64 tokens 14.0, 17.1, 4096 21.5, 25.7, 6000 29.3, 27.6,
// 16384 50.8, 33.7.
int lanes_per_token(long T, int E, int topk, int groups) {
  const bool fits = E <= 256 && topk <= 16 && groups <= 16;
  const bool rather = E <= 128 || T > 256 * kRtWaves || (T <= 64 && E <= 192);
  return T > 16 && fits && rather ? 16 : 64;
}

// blocks of the first kernel; one builds the lists as well
long choose_blocks(long T, int lanes) {
  const long at_once = kRtThreads / lanes;
  return std::max((T + at_once - 1) / at_once, 1L);
}

// Whether the counts are added up by the second kernel's blocks first (per_list: the
// first kernel's blocks in each; 1: they are not).  Each of up to 256 blocks reads all
// the counts there are, which grow with the tokens and the experts; added up they are
// 256 rows (bf16, us without and with the launch more: 32768 tokens of 64 experts, 2
// blocks each, 18.0, 19.6; 65536, 4, 27.4, 27.1; of 256 59.2, 52.8; 32768 of 1000, 8
// blocks each, 151, 67; 2^21 of 1000 11585, 3071).
int counts_step(int per_list) { return per_list >= 4 ? per_list : 1; }

template <int LP, int NV, bool kBias, bool kSigmoid>
hipError_t run_route(const RouteArgs &a, hipStream_t stream) {
  const bool grouped = a.group_limit < a.groups;
  if constexpr (LP == 64) {
    if (a.T == 1) {
      hipLaunchKernelGGL((route_one<NV, kBias, kSigmoid>), dim3(1), dim3(64),
                         grouped ? LP * NV * 8 : 0, stream, a);
      return hipGetLastError();
    }
  }
  const int keys = grouped ? kRtThreads * NV : 0;
  // (past 192 experts 16 lanes have more than one block)
  if constexpr (LP == 64 || NV < 16) {
    if (a.blocks == 1) {
      hipLaunchKernelGGL((route_choose<LP, NV, kBias, kSigmoid, true>), dim3(1), dim3(kRtThreads),
                         route_lds(a.E, keys, a.T * a.topk), stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((route_choose<LP, NV, kBias, kSigmoid, false>), dim3(a.blocks),
                     dim3(kRtThreads), route_lds(a.E, keys, 0), stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned lists = unsigned((a.T + a.chunk - 1) / a.chunk);
  if (a.step > 1) {
    hipLaunchKernelGGL(route_sums, dim3(lists), dim3(kRtThreads), size_t(padded(a.E)) * 4, stream,
                       a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t lds = size_t(a.E) * 8 + (2 * size_t(padded(a.E)) + 1 + kRtWaves) * 4;
  hipLaunchKernelGGL(route_lists, dim3(lists), dim3(kRtThreads), lds, stream, a);
  return hipGetLastError();
}

template <int LP, int NV>
hipError_t run_route_keys(const RouteArgs &a, hipStream_t stream) {
  if (a.bias)
    return a.sigmoid ? run_route<LP, NV, true, true>(a, stream)
                     : run_route<LP, NV, true, false>(a, stream);
  return a.sigmoid ? run_route<LP, NV, false, true>(a, stream)
                   : run_route<LP, NV, false, false>(a, stream);
}

hipError_t run_route_size(const RouteArgs &a, hipStream_t stream) {
  if (lanes_per_token(a.T, a.E, a.topk, a.groups) == 16) {
    if (a.E <= 64) return run_route_keys<16, 4>(a, stream);
    if (a.E <= 128) return run_route_keys<16, 8>(a, stream);
    if (a.E <= 192) return run_route_keys<16, 12>(a, stream);
    return run_route_keys<16, 16>(a, stream);
  }
  if (a.E <= 64) return run_route_keys<64, 1>(a, stream);
  if (a.E <= 256) return run_route_keys<64, 4>(a, stream);
  if (a.E <= 512) return run_route_keys<64, 8>(a, stream);
  return run_route_keys<64, 16>(a, stream);
}

}  // namespace

// the groups are not known here: room for the form with more blocks
size_t route_workspace_bytes(long T, int E) {
  const long blocks = choose_blocks(T, 64);
  return blocks > 1 ? size_t(blocks) * padded(E) * 4 : 0;
}

hipError_t launch_route(const MoeRoute &r, void *workspace, hipStream_t stream) {
  RouteArgs a;
  a.logits = r.logits;
  a.bias = r.bias;
  a.num_tokens = r.num_tokens;
  a.ids = r.ids;
  a.weights = r.weights;
  a.slots = r.slots;
  a.token_index = r.token_index;
  a.offsets = r.expert_offsets;
  a.counts = static_cast<int32_t *>(workspace);
  a.T = r.T;
  a.E = r.E;
  a.topk = r.topk;
  a.groups = r.groups;
  a.group_limit = r.group_limit;
  a.group_top = r.group_top;
  a.sigmoid = r.sigmoid;
  a.renormalize = r.renormalize;
  a.scale = r.scale;
  const int lanes = lanes_per_token(r.T, r.E, r.topk, r.groups);
  a.at_once = kRtThreads / lanes;
  a.blocks = int(choose_blocks(r.T, lanes));
  a.chunk = int(64 * ((long(r.T) + 64L * kRtMaxBlocks - 1) / (64L * kRtMaxBlocks)));
  a.step = counts_step(a.chunk / a.at_once);
  a.dtype = r.dtype;
  return run_route_size(a, stream);
}

}  // namespace w4a16
