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
// keys are computed in fp32 first, with an error below kTol(key); if any two
// values whose order decides something lie closer than twice that, the token
// is done again with 64-bit keys (about 1 token in 500 at 256 experts).
//
// Slots are sorted by expert, then token.  A block of tokens counts its
// choices per expert; a second kernel sums the blocks before its own and ranks
// each choice inside its block.  A token takes an expert at most once, so 64
// tokens' choices of an expert are one 64-bit mask, ORed together in LDS (any
// order gives the same mask), and a choice's rank is a population count: no
// result depends on the order of atomics.  One block of up to 64 tokens does
// both in one launch.
//
// Bound: at few tokens by launch and load latency; at many by VALU issue of
// the selection (about 700 instructions a token at 256 experts, top 8 of 4 out
// of 8 groups).

#include "moe_common.h"

#include <algorithm>
#include <cmath>

namespace w4a16 {
namespace {

constexpr int kRtWaves = 16;
constexpr int kRtThreads = 64 * kRtWaves;
constexpr int kRtSingle = 64;     // tokens of the one-launch form
constexpr int kRtMaxBlocks = 256; // blocks of the first kernel

struct RouteArgs {
  const void *logits;
  const float *bias;           // [E] or null
  const int32_t *num_tokens;   // [1] or null
  int32_t *ids;                // [T][topk]
  float *weights;              // [T][topk]
  int32_t *slots;              // [T][topk]
  int32_t *token_index;        // [T * topk]
  int32_t *offsets;            // [E + 1]
  int32_t *counts;             // [blocks][E]
  int T, E, topk, groups, group_limit, group_top, sigmoid, renormalize;
  float scale;
  int chunk, blocks;           // tokens per block, blocks
};

constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float wave_max(float v) {
  // row shifts 1, 2, 4, 8, then rows 0 and 2 into 1 and 3, then row 1 into 2
  // and 3: lane 63 holds the maximum (lanes without a source keep their own)
#define W4A16_RT_STEP(CTRL, ROWS)                                                            \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(                                   \
                   __float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xf, false)))
  W4A16_RT_STEP(0x111, 0xf);
  W4A16_RT_STEP(0x112, 0xf);
  W4A16_RT_STEP(0x114, 0xf);
  W4A16_RT_STEP(0x118, 0xf);
  W4A16_RT_STEP(0x142, 0xa);
  W4A16_RT_STEP(0x143, 0xc);
#undef W4A16_RT_STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmax(v, __shfl_xor(v, d, 64));
  return v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// Bound of twice the error of a fp32 key or of a sum of two: scores are at
// most 1 with a relative error below 12 * 2^-24 (exp 1 ulp, the softmax sum of
// up to 1024 terms in 64 bits, one division), each addition rounds once.
template <typename KT>
__device__ __forceinline__ bool too_close(KT hi, KT lo) {
  if constexpr (sizeof(KT) == 8) return false;  // 64-bit keys decide as they are
  const float d = float(hi) - float(lo);
  return !(d > 4e-6f + 1e-6f * fmaxf(fabsf(float(hi)), fabsf(float(lo))));
}

template <int NV>
struct Token {
  float x[NV];      // logits of experts 64 r + lane; masked ones -inf
  float chosen_x;   // lane j: logit of the j-th choice
  int chosen;       // lane j: its expert, -1 where none
};

// Order the token's experts by keys of type KT; returns false if fp32 cannot
// tell.  kBias: keys are s + b, else the logits.  keys: this wave's LDS room
// for E values (used with groups only).  top: largest logit, sum: sum of
// exp(l - top) (softmax).
template <typename KT, int NV, bool kBias>
__device__ __forceinline__ bool select_experts(const RouteArgs &a, Token<NV> &tk,
                                               const float (&b)[NV], const int (&grp)[NV],
                                               float top, double sum, KT *keys) {
  const int lane = threadIdx.x & 63;
  const bool grouped = a.group_limit < a.groups;
  const KT low = KT(kNegInf);
  KT key[NV];
  KT gkey[NV];  // what groups are valued by
#pragma unroll
  for (int r = 0; r < NV; ++r) {
    const float x = tk.x[r];
    key[r] = KT(x);
    gkey[r] = key[r];
    if (kBias || grouped) {
      KT s;
      if (a.sigmoid)
        s = KT(1) / (KT(1) + exp_of(-KT(x)));
      else
        s = (x == top ? KT(1) : exp_of(KT(x) - KT(top))) / KT(sum);
      if (kBias) {
        s += KT(b[r]);
        if (!(s > low)) s = low;  // a NaN or -inf bias masks
        key[r] = x > kNegInf ? s : low;
      }
      gkey[r] = x > kNegInf ? s : low;
    }
  }
  bool sure = true;
  if (grouped) {
    // groups side by side: 64 / groups lanes (a power of two) per group, each
    // taking every L-th of its experts, the two largest merged across them
    const int L = 1 << (31 - __clz(64 / a.groups));
    const int gs = a.E / a.groups;
    const int g = lane / L;
#pragma unroll
    for (int r = 0; r < NV; ++r)
      if (64 * r + lane < a.E) keys[64 * r + lane] = gkey[r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    KT m1 = low, m2 = low;
    if (g < a.groups)
      for (int i = lane - g * L; i < gs; i += L) {
        const KT v = keys[g * gs + i];
        m2 = v > m1 ? m1 : (v > m2 ? v : m2);
        m1 = v > m1 ? v : m1;
      }
    for (int d = 1; d < L; d <<= 1) {
      const KT o1 = __shfl_xor(m1, d, 64), o2 = __shfl_xor(m2, d, 64);
      m2 = o1 > m1 ? (m1 > o2 ? m1 : o2) : (o1 > m2 ? o1 : m2);
      m1 = o1 > m1 ? o1 : m1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // before the room is written again
    __builtin_amdgcn_wave_barrier();
    KT value = m1;
    if (a.group_top == 2 && m2 > low) value += m2;
    int rank = 0;
    bool near = false;
    for (int h = 0; h < a.groups; ++h) {
      const KT v = __shfl(value, h * L, 64);
      rank += (v > value || (v == value && h < g)) ? 1 : 0;
      near |= h != g && m1 > low && v > low && too_close(v > value ? v : value, v > value ? value : v);
    }
    const unsigned long long kept =
        __ballot(g < a.groups && m1 > low && rank < a.group_limit);
    sure = __ballot(near && g < a.groups) == 0;
#pragma unroll
    for (int r = 0; r < NV; ++r)
      if (!((kept >> (grp[r] * L)) & 1)) key[r] = low;
  }
  // topk + 1 picks: the last shows how near the first one left out comes
  tk.chosen = -1;
  tk.chosen_x = 0.0f;
  KT last = low;
  for (int j = 0; j <= a.topk; ++j) {
    KT m = key[0];
#pragma unroll
    for (int r = 1; r < NV; ++r) m = key[r] > m ? key[r] : m;
    m = wave_max(m);
    if (!(m > low)) break;
    if (kBias && j > 0 && too_close(last, m)) sure = false;
    last = m;
    if (j == a.topk) break;
    bool done = false;
#pragma unroll
    for (int r = 0; r < NV; ++r) {
      const unsigned long long at = __ballot(key[r] == m);
      if (!done && at != 0) {
        const int l = __builtin_ctzll(at);
        const float x =
            __int_as_float(__builtin_amdgcn_readlane(__float_as_int(tk.x[r]), l));
        if (lane == j) {
          tk.chosen = 64 * r + l;
          tk.chosen_x = x;
        }
        if (lane == l) key[r] = low;
        done = true;
      }
    }
  }
  return sure;
}

// One token by one wave: lane j < topk leaves with its j-th choice and weight.
template <typename LT, int NV, bool kBias>
__device__ __forceinline__ void route_token(const RouteArgs &a, int t, const float (&b)[NV],
                                            const int (&grp)[NV], double *keys, int &id,
                                            float &weight) {
  const int lane = threadIdx.x & 63;
  const LT *row = static_cast<const LT *>(a.logits) + long(t) * a.E;
  Token<NV> tk;
#pragma unroll
  for (int r = 0; r < NV; ++r) {
    const int e = 64 * r + lane;
    const float x = to_f32(row[min(e, a.E - 1)]);
    tk.x[r] = (e < a.E && x > kNegInf) ? x : kNegInf;  // a NaN is masked too
  }
  const bool grouped = a.group_limit < a.groups;
  float top = 0.0f;
  double sum = 1.0;
  if (!a.sigmoid) {
    float m = tk.x[0];
#pragma unroll
    for (int r = 1; r < NV; ++r) m = fmaxf(m, tk.x[r]);
    top = wave_max(m);
    if (kBias || grouped || !a.renormalize) {
      // fp32 terms summed in 64 bits: the error of the sum is the terms' own
      double s = 0.0;
#pragma unroll
      for (int r = 0; r < NV; ++r)
        s += tk.x[r] > kNegInf ? (tk.x[r] == top ? 1.0 : double(expf(tk.x[r] - top))) : 0.0;
      sum = wave_sum(s);
    }
  }
  bool sure;
  if constexpr (!kBias) {
    sure = select_experts<float, NV, false>(a, tk, b, grp, top, sum,
                                            reinterpret_cast<float *>(keys));
  } else {
    sure = select_experts<float, NV, true>(a, tk, b, grp, top, sum,
                                           reinterpret_cast<float *>(keys));
  }
  if (!sure) {  // uniform over the wave
    if (!a.sigmoid) {
      double s = 0.0;
#pragma unroll
      for (int r = 0; r < NV; ++r)
        s += tk.x[r] > kNegInf ? (tk.x[r] == top ? 1.0 : exp(double(tk.x[r]) - double(top))) : 0.0;
      sum = wave_sum(s);
    }
    select_experts<double, NV, kBias>(a, tk, b, grp, top, sum, keys);
  }
  // the chosen scores, one per lane, in 64 bits (a score of 1e-40 still has a
  // share of the chosen ones' sum)
  double s = 0.0;
  if (tk.chosen >= 0) {
    const double x = tk.chosen_x;
    if (a.sigmoid)
      s = 1.0 / (1.0 + exp(-x));
    else
      s = (tk.chosen_x == top ? 1.0 : exp(x - double(top))) / sum;
  }
  if (a.renormalize) {
    const double all = wave_sum(s);
    s = all > 0.0 ? s / all : 0.0;
  }
  id = tk.chosen;
  weight = float(s * double(a.scale));
}

__device__ __forceinline__ int live_tokens(const RouteArgs &a) {
  return a.num_tokens ? min(max(*a.num_tokens, 0), a.T) : a.T;
}

// Choices of this block's tokens [t0, t1), into memory and, if kept, into LDS.
template <typename LT, int NV, bool kBias>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, int t0, int t1, double *keys,
                                             int32_t *kept, int *hist) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int live = live_tokens(a);
  float b[NV];
  int grp[NV];
#pragma unroll
  for (int r = 0; r < NV; ++r) {
    const int e = min(64 * r + lane, a.E - 1);
    b[r] = kBias ? a.bias[e] : 0.0f;
    grp[r] = e / (a.E / a.groups);
  }
  double *mine = keys + long(wave) * (a.group_limit < a.groups ? a.E : 0);
  for (int t = t0 + wave; t < t1; t += kRtWaves) {
    int id = -1;
    float w = 0.0f;
    if (t < live) route_token<LT, NV, kBias>(a, t, b, grp, mine, id, w);
    if (lane < a.topk) {
      a.ids[long(t) * a.topk + lane] = id;
      a.weights[long(t) * a.topk + lane] = w;
      if (kept) kept[(t - t0) * a.topk + lane] = id;
      if (hist && id >= 0) atomicAdd(&hist[id], 1);
    }
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

// LDS: masks [E], then the per-wave keys, then base [E + 1], part, the kept
// choices (one-launch form).
__host__ __device__ constexpr size_t route_lds(int E, bool grouped, int kept) {
  return size_t(E) * 8 + (grouped ? size_t(kRtWaves) * E * 8 : 0) +
         (size_t(E) + 1 + kRtWaves + kept) * 4;
}

// kSingle: T <= 64, choices and lists.  Otherwise block b routes tokens
// [b chunk, (b + 1) chunk) and writes its counts.
template <typename LT, int NV, bool kBias, bool kSingle>
__global__ void __launch_bounds__(kRtThreads) route_choose(RouteArgs a) {
  extern __shared__ __align__(16) unsigned char rt_lds[];
  const bool grouped = a.group_limit < a.groups;
  auto *mask = reinterpret_cast<unsigned long long *>(rt_lds);
  auto *keys = reinterpret_cast<double *>(mask + a.E);
  auto *base = reinterpret_cast<int *>(keys + (grouped ? kRtWaves * a.E : 0));
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  if (tid < a.E) base[tid] = 0;
  __syncthreads();
  if constexpr (!kSingle) {
    route_tokens<LT, NV, kBias>(a, t0, t1, keys, nullptr, base);
    __syncthreads();
    if (tid < a.E) a.counts[long(blockIdx.x) * a.E + tid] = base[tid];
  } else {
    int *part = base + a.E + 1;
    int32_t *kept = part + kRtWaves;
    route_tokens<LT, NV, kBias>(a, t0, t1, keys, kept, base);
    __syncthreads();
    scan_experts(base, a.E, part);
    for (int e = tid; e <= a.E; e += kRtThreads) a.offsets[e] = base[e];
    for (int r = base[a.E] + tid; r < a.T * a.topk; r += kRtThreads) a.token_index[r] = -1;
    __syncthreads();
    place_choices(a, 0, a.T, kept, mask, base);
  }
}

// Block b: slots of tokens [b chunk, (b + 1) chunk) from the counts.
__global__ void __launch_bounds__(kRtThreads) route_lists(RouteArgs a) {
  extern __shared__ __align__(16) unsigned char rt_lds[];
  auto *mask = reinterpret_cast<unsigned long long *>(rt_lds);
  auto *total = reinterpret_cast<int *>(mask + a.E);  // [E + 1]
  int *before = total + a.E + 1;                      // [E]
  int *part = before + a.E;                           // [kRtWaves]
  const int tid = threadIdx.x;
  if (tid < a.E) total[tid] = before[tid] = 0;
  __syncthreads();
  // experts side by side, the blocks dealt to the thread groups that are left
  int width = 64;
  while (width < a.E) width <<= 1;
  const int e = tid & (width - 1);
  if (e < a.E) {
    int all = 0, mine = 0;
    const int step = kRtThreads / width;
#pragma unroll 4
    for (int k = tid / width; k < a.blocks; k += step) {
      const int c = a.counts[long(k) * a.E + e];
      all += c;
      if (k < int(blockIdx.x)) mine += c;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&before[e], mine);
  }
  __syncthreads();
  scan_experts(total, a.E, part);
  if (blockIdx.x == 0)
    for (int i = tid; i <= a.E; i += kRtThreads) a.offsets[i] = total[i];
  const long R = long(a.T) * a.topk;
  for (long r = total[a.E] + long(blockIdx.x) * kRtThreads + tid; r < R;
       r += long(a.blocks) * kRtThreads)
    a.token_index[r] = -1;
  if (tid < a.E) before[tid] += total[tid];
  const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
  for (int t = t0; t < t1; t += 64)  // place_choices begins and ends past barriers
    place_choices(a, t, min(64, t1 - t), a.ids + long(t) * a.topk, mask, before);
}

struct RoutePlan {
  int chunk, blocks;
};

// One launch up to 64 tokens; above, blocks of a multiple of 16 tokens (one
// per wave at a time), at most 256 blocks.
RoutePlan plan_route(long T) {
  RoutePlan p;
  if (T <= kRtSingle) {
    p.chunk = kRtSingle;
    p.blocks = 1;
    return p;
  }
  const long per = (T + long(kRtWaves) * kRtMaxBlocks - 1) / (long(kRtWaves) * kRtMaxBlocks);
  p.chunk = int(per * kRtWaves);
  p.blocks = int((T + p.chunk - 1) / p.chunk);
  return p;
}

template <typename LT, int NV, bool kBias>
hipError_t run_route(const RouteArgs &a, hipStream_t stream) {
  const bool grouped = a.group_limit < a.groups;
  if (a.T <= kRtSingle) {
    const size_t lds = route_lds(a.E, grouped, a.T * a.topk);
    hipLaunchKernelGGL((route_choose<LT, NV, kBias, true>), dim3(1), dim3(kRtThreads), lds,
                       stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((route_choose<LT, NV, kBias, false>), dim3(a.blocks), dim3(kRtThreads),
                     route_lds(a.E, grouped, 0), stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = size_t(a.E) * 8 + (2 * size_t(a.E) + 1 + kRtWaves) * 4;
  hipLaunchKernelGGL(route_lists, dim3(a.blocks), dim3(kRtThreads), lds, stream, a);
  return hipGetLastError();
}

template <typename LT, int NV>
hipError_t run_route_bias(const RouteArgs &a, hipStream_t stream) {
  return a.bias ? run_route<LT, NV, true>(a, stream) : run_route<LT, NV, false>(a, stream);
}

template <typename LT>
hipError_t run_route_type(const RouteArgs &a, hipStream_t stream) {
  if (a.E <= 64) return run_route_bias<LT, 1>(a, stream);
  if (a.E <= 128) return run_route_bias<LT, 2>(a, stream);
  if (a.E <= 256) return run_route_bias<LT, 4>(a, stream);
  if (a.E <= 512) return run_route_bias<LT, 8>(a, stream);
  return run_route_bias<LT, 16>(a, stream);
}

}  // namespace

size_t route_workspace_bytes(long T, int E) {
  const RoutePlan p = plan_route(T);
  return p.blocks > 1 ? size_t(p.blocks) * E * 4 : 0;
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
  const RoutePlan p = plan_route(r.T);
  a.chunk = p.chunk;
  a.blocks = p.blocks;
  switch (r.dtype) {
    case W4A16_DTYPE_F32: return run_route_type<float>(a, stream);
    case W4A16_DTYPE_F16: return run_route_type<_Float16>(a, stream);
    default: return run_route_type<Bf16>(a, stream);
  }
}

}  // namespace w4a16
