// Routing by a rule: scores, a bias for balance, groups of experts, and weights.
//
//   s_e = 1 / (1 + e^-l_e)   or   e^(l_e - max l) / sum_i e^(l_i - max l)
//   c_e = s_e + bias_e
//   a group of E / G neighbouring experts is worth max c, or the sum of its two largest c;
//   the top_groups worthiest stay (equal ones: the lower group first); of their experts the
//   k with the largest c are taken (equal ones: the lower id first), in that order
//   w_j = scale * s_j, or scale * s_j / sum_i s_i over the k taken
//
// all in binary64: a score's last bit decides between near experts. One wavefront takes one
// token: lane l holds experts l, l + 64, ... in registers. Bound by the vector units: binary64
// for every expert costs some 35 instructions of double length each.
//
// Sigmoid scores are therefore taken in fp32 first (rule_fast): the groups are kept by fp32
// worths where these are further apart than their errors, every expert that could be among the k
// best becomes a candidate, and the candidates, at most one a lane, get their binary64 scores,
// by which they are ranked. Where groups are too near or candidates too many, and for scores
// that are not finite, the whole rule runs in binary64 (wave_rule, which softmax always does:
// its sum needs every exponential). The fused kernel holds both, and the grouping: it spills
// scalar registers into lanes of vector registers (76 at 512 experts, 131 at 1024; k_rule_topk 47
// at 1024). 4 tokens, us: 256 experts 6.1, 512 experts 7.0 (softmax 8.6), 1024 experts 9.6.
//
// Groups go through LDS: 64 / G lanes (a power of two) scan one group each. The k best are found
// as in the plain router, by a threshold on order-preserving images: every expert of the top k
// has an image of at least the k-th largest of the lanes' largest ones, and the few that do are
// ranked by counting.
#include "qmoe_route_dev.h"

namespace qmoe {
namespace {

// Order-preserving unsigned image of a double (-0 as +0). NaN and -inf are 1, the lowest of a
// valid expert (0 marks none), so that they are taken last and in the order of their ids.
__device__ __forceinline__ uint64_t order_image(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  const uint64_t o = u >> 63 ? ~u : u | 0x8000000000000000ull;
  return v > -__builtin_inf() ? o : 1ull;
}

__device__ __forceinline__ double shfl_xor_f64(double v, int mask) { return __shfl_xor(v, mask); }

struct RuleArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int n, E, k, dtype;
  int softmax, groups, top_groups, top2, renormalize;
  int lanes;  // lanes a group, a power of two
  double scale;
};

template <int KPL>
struct RuleScratch {
  uint32_t hi[kWave], lo[kWave];  // images of the candidates; fast: their logits and biases
  int id[kWave];
  int slot_id[MOE_MAX_TOP_K];
  double score[KPL * kWave];
};

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The two largest of the union of (a, b) and (c, d), each with its larger first.
__device__ __forceinline__ void top2_merge(double& a, double& b, double c, double d) {
  const double low = fmin(a, c);
  a = fmax(a, c);
  b = fmax(low, fmax(b, d));
}

template <int KPL>
struct RuleRow {
  float l[KPL], b[KPL];  // logits and biases of experts lane, lane + 64, ...
};

// Every load is issued before the first is used.
template <int KPL>
__device__ __forceinline__ void load_row(const RuleArgs& a, int t, RuleRow<KPL>& v) {
  const int lane = threadIdx.x & (kWave - 1), E = a.E;
  const size_t row = (size_t)t * E;
  if (a.dtype == MOE_F32) {
    const float* p = static_cast<const float*>(a.logits) + row;
#pragma unroll
    for (int i = 0; i < KPL; ++i) v.l[i] = p[min(lane + kWave * i, E - 1)];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + row;
    uint32_t h[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) h[i] = p[min(lane + kWave * i, E - 1)];
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      v.l[i] = a.dtype == MOE_BF16 ? __uint_as_float(h[i] << 16) : half_bits_to_float(h[i]);
  }
#pragma unroll
  for (int i = 0; i < KPL; ++i) v.b[i] = 0.0f;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < KPL; ++i) v.b[i] = a.bias[min(lane + kWave * i, E - 1)];
  }
}

// Ranks the candidates by (image, lower id): lane q holds candidate q < total. Slots get the lanes.
__device__ __forceinline__ int rank_of(uint64_t mine, int id, int total) {
  int rank = 0;
  for (int q = 0; q < total; ++q) {
    const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), q) << 32 |
                       (uint32_t)__builtin_amdgcn_readlane((int)mine, q);
    const int oi = __builtin_amdgcn_readlane(id, q);
    rank += o > mine || (o == mine && oi < id);
  }
  return rank;
}

// Weights of the slots: lane j < k holds slot j's expert and binary64 score.
__device__ __forceinline__ void store_slots(const RuleArgs& a, int t, int id, double score) {
  const int lane = threadIdx.x & (kWave - 1), k = a.k;
  double sum = 1.0;
  if (a.renormalize) {
    sum = 0.0;
    for (int j = 0; j < k; ++j) sum += readlane_f64(score, j);  // slot order
  }
  if (lane < k) {
    a.ids[(size_t)t * k + lane] = id;
    a.w[(size_t)t * k + lane] = (float)(sum > 0.0 ? score / sum * a.scale : 0.0);
  }
}

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// Sigmoid scores by fp32 first; false where that cannot decide. An fp32 score is off by less than
// 2^-21 (the exponential's argument by |l| 2^-24 of itself, which times the slope s (1 - s) stays
// under 2^-24; the exponential, the sum and the reciprocal by an ulp each) and c by 2^-24 of
// itself more: within 2^-20 (1 + |c|).
template <int KPL>
__device__ __forceinline__ bool rule_fast(const RuleArgs& a, int t, const RuleRow<KPL>& v,
                                          RuleScratch<KPL>* sc, int& my_id) {
  const int lane = threadIdx.x & (kWave - 1);
  const int E = a.E, k = a.k;
  constexpr float kErr = 0x1p-20f;
  float c[KPL];
  bool odd = false;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    c[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-v.l[i])) + v.b[i];
    odd |= !(fabsf(c[i]) < __builtin_inff());
  }
  if (__ballot(odd)) return false;

  uint64_t kept = ~0ull;
  const int size = E / a.groups;
  if (a.top_groups < a.groups) {
    float* score = reinterpret_cast<float*>(sc->score);
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lane + kWave * i < E) score[lane + kWave * i] = c[i];
    wave_sync();
    const int g = lane / a.lanes, sub = lane & (a.lanes - 1);
    float m1 = -__builtin_inff(), m2 = m1;
    if (g < a.groups)
      for (int j = sub; j < size; j += a.lanes) {
        const float x = score[g * size + j];
        m2 = fmaxf(m2, fminf(m1, x));
        m1 = fmaxf(m1, x);
      }
    for (int m = 1; m < a.lanes; m <<= 1) {
      const float o1 = __shfl_xor(m1, m), o2 = __shfl_xor(m2, m);
      m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
      m1 = fmaxf(m1, o1);
    }
    const bool two = a.top2 && size > 1;
    const float worth = two ? m1 + m2 : m1;
    const float err = 2.0f * kErr * (2.0f + fabsf(m1) + (two ? fabsf(m2) : 0.0f));
    int rank = 0;
    for (int q = 0; q < a.groups; ++q) {
      const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(worth), q * a.lanes));
      rank += o > worth || (o == worth && q < g);
    }
    const bool in = g < a.groups, stays = in && rank < a.top_groups;
    // the least of the kept and the largest of the others, each at the wrong end of its error
    const float least = -wave_max_f32(stays ? err - worth : -__builtin_inff());
    const float most = wave_max_f32(in && !stays ? worth + err : -__builtin_inff());
    if (!(least > most)) return false;
    const uint64_t stay = __ballot(stays && sub == 0);
    kept = 0;
    for (int q = 0; q < a.groups; ++q) kept |= (stay >> (q * a.lanes) & 1ull) << q;
  }

  bool in[KPL];
  uint32_t lmax = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + kWave * i;
    in[i] = e < E && (a.top_groups >= a.groups || (kept >> (min(e, E - 1) / size) & 1));
    lmax = max(lmax, in[i] ? order_bits(c[i]) : 0u);
  }
  // a threshold that at least k lanes reach, to 20 bits; 0 where fewer lanes than k hold an expert
  uint32_t T = 0;
  for (int b = 31; b >= 12; --b) {
    const uint32_t u = T | (1u << b);
    if (__popcll(__ballot(lmax >= u)) >= k) T = u;
  }
  const float Tf = order_bits_to_float(T);
  const float from = T ? Tf - 4.0f * kErr * (1.0f + fabsf(Tf)) : -__builtin_inff();
  const uint64_t below = (1ull << lane) - 1ull;
  int total = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const bool cand = in[i] && c[i] >= from;
    const uint64_t b = __ballot(cand);
    const int pos = total + __popcll(b & below);
    if (cand && pos < kWave) {
      sc->hi[pos] = __float_as_uint(v.l[i]);
      sc->lo[pos] = __float_as_uint(v.b[i]);
      sc->id[pos] = lane + kWave * i;
    }
    total += __popcll(b);
  }
  if (total > kWave) return false;
  wave_sync();
  const int at = min(lane, total - 1);
  const double s = 1.0 / (1.0 + exp(-(double)__uint_as_float(sc->hi[at])));
  const int id = sc->id[at];
  const uint64_t mine = lane < total ? order_image(s + (double)__uint_as_float(sc->lo[at])) : 0ull;
  const int rank = rank_of(mine, id, total);
  if (lane < total && rank < k) sc->slot_id[rank] = lane;
  wave_sync();
  const int from_lane = sc->slot_id[min(lane, k - 1)];
  my_id = __shfl(id, from_lane);
  store_slots(a, t, my_id, __shfl(s, from_lane));
  return true;
}

// One token by one wavefront; every lane returns the expert of slot `lane` (lane < k).
template <int KPL>
__device__ __forceinline__ int wave_rule(const RuleArgs& a, int t, RuleScratch<KPL>* sc) {
  const int lane = threadIdx.x & (kWave - 1);
  const int E = a.E, k = a.k;
  const double none = -__builtin_inf();
  RuleRow<KPL> row;
  load_row(a, t, row);
  int fast_id = 0;
  if (!a.softmax && rule_fast(a, t, row, sc, fast_id)) return fast_id;
  wave_sync();
  const float(&lv)[KPL] = row.l, (&bv)[KPL] = row.b;

  double s[KPL];
  if (a.softmax) {
    float top = -__builtin_inff();  // fmaxf passes over NaN
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lane + kWave * i < E) top = fmaxf(top, lv[i]);
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      // the largest stands for 1 even where it is infinite; -inf and NaN for 0
      const double x = lv[i] == top ? 0.0 : (double)lv[i] - (double)top;
      s[i] = lane + kWave * i < E && lv[i] > -__builtin_inff() ? exp(x) : 0.0;
      sum += s[i];
    }
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) sum += shfl_xor_f64(sum, m);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) s[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      s[i] = lv[i] > -__builtin_inff() ? 1.0 / (1.0 + exp(-(double)lv[i])) : 0.0;
  }

  double c[KPL];
#pragma unroll
  for (int i = 0; i < KPL; ++i) c[i] = lv[i] == lv[i] ? s[i] + (double)bv[i] : none;
#pragma unroll
  for (int i = 0; i < KPL; ++i)
    if (!(c[i] > none)) c[i] = none, s[i] = 0.0;  // never with a weight

  uint64_t kept = ~0ull;  // groups that stay
  const int size = E / a.groups;
  if (a.top_groups < a.groups) {
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lane + kWave * i < E) sc->score[lane + kWave * i] = c[i];
    wave_sync();
    const int g = lane / a.lanes, sub = lane & (a.lanes - 1);
    double m1 = none, m2 = none;
    if (g < a.groups)
      for (int j = sub; j < size; j += a.lanes) top2_merge(m1, m2, sc->score[g * size + j], none);
    for (int m = 1; m < a.lanes; m <<= 1) {
      const double o1 = shfl_xor_f64(m1, m), o2 = shfl_xor_f64(m2, m);
      top2_merge(m1, m2, o1, o2);
    }
    // one expert a group: its own score is the sum
    const uint64_t worth = g < a.groups ? order_image(a.top2 && size > 1 ? m1 + m2 : m1) : 0ull;
    int rank = 0;
    for (int q = 0; q < a.groups; ++q) {
      const int from = q * a.lanes;
      const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(worth >> 32), from) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)worth, from);
      rank += o > worth || (o == worth && q < g);
    }
    const uint64_t stay = __ballot(g < a.groups && rank < a.top_groups && sub == 0);
    kept = 0;
    for (int q = 0; q < a.groups; ++q) kept |= (stay >> (q * a.lanes) & 1ull) << q;
    wave_sync();
  }

  uint64_t key[KPL];
  uint32_t lmax = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const int e = lane + kWave * i;
    const bool in = e < E && (a.top_groups >= a.groups || (kept >> (min(e, E - 1) / size) & 1));
    key[i] = in ? order_image(c[i]) : 0ull;
    // the image of an expert that comes last has an empty upper half
    lmax = max(lmax, in ? max((uint32_t)(key[i] >> 32), 1u) : 0u);
  }
  // the largest threshold that at least k lanes reach; fewer lanes than k may hold an expert
  // when groups are small: then it stays at 0 and the rounds below select
  uint32_t T = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t v = T | (1u << b);
    if (__popcll(__ballot(lmax >= v)) >= k) T = v;
  }
  const uint64_t below = (1ull << lane) - 1ull;
  int total = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) {
    const bool in = key[i] != 0ull && max((uint32_t)(key[i] >> 32), 1u) >= T;
    const uint64_t b = __ballot(in);
    const int pos = total + __popcll(b & below);
    if (in && pos < kWave) {
      sc->hi[pos] = (uint32_t)(key[i] >> 32);
      sc->lo[pos] = (uint32_t)key[i];
      sc->id[pos] = lane + kWave * i;
    }
    total += __popcll(b);
  }
  wave_sync();
  int my_id = 0;
  if (total <= kWave) {
    const uint64_t mine = lane < total ? (uint64_t)sc->hi[lane] << 32 | sc->lo[lane] : 0ull;
    const int mi = lane < total ? sc->id[lane] : 0x7fffffff;
    const int rank = rank_of(mine, mi, total);
    if (lane < total && rank < k) sc->slot_id[rank] = mi;
    wave_sync();
    if (lane < k) my_id = sc->slot_id[lane];
  } else {
    for (int j = 0; j < k; ++j) {
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) best = max(best, key[i]);
      const uint32_t hi = wave_max_u32((uint32_t)(best >> 32));
      const uint32_t lo = wave_max_u32((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
      best = (uint64_t)hi << 32 | lo;
      int slot = 0;
      uint64_t hit = 0;
#pragma unroll
      for (int i = KPL - 1; i >= 0; --i) {
        const uint64_t b = __ballot(key[i] == best);
        if (b) slot = i, hit = b;
      }
      const int owner = __builtin_ctzll(hit);
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (i == slot && lane == owner) key[i] = 0ull;
      if (lane == j) my_id = owner + kWave * slot;
    }
  }
  // the scores of the experts taken, through LDS (without groups their c never went there)
#pragma unroll
  for (int i = 0; i < KPL; ++i)
    if (lane + kWave * i < E) sc->score[lane + kWave * i] = s[i];
  wave_sync();
  store_slots(a, t, my_id, lane < k ? sc->score[my_id] : 0.0);
  return my_id;
}

constexpr int kRuleWaves = 4;

template <int KPL>
__global__ __launch_bounds__(kRuleWaves * kWave) void k_rule_topk(RuleArgs a) {
  __shared__ RuleScratch<KPL> s_rule[kRuleWaves];
  const int wave = threadIdx.x / kWave;
  const int t = blockIdx.x * kRuleWaves + wave;
  if (t < a.n) wave_rule<KPL>(a, t, &s_rule[wave]);
}

// Up to kFusedRouteTokens tokens: selection and grouping in one workgroup and one launch.
constexpr int kFusedWaves = 8;

template <int KPL>
__global__ __launch_bounds__(kFusedWaves * kWave) void k_rule_fused(RuleArgs a, int32_t* offsets,
                                                                    int32_t* pair_index) {
  __shared__ union {
    RuleScratch<KPL> rule[kFusedWaves];
    struct {
      int hist[kFusedWaves * MOE_MAX_EXPERTS];
      int off[MOE_MAX_EXPERTS + 1];
      int wsum[kFusedWaves];
    } group;
  } s;
  __shared__ __attribute__((aligned(16))) int s_ids[kSmallPairs + 4];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int P = a.n * a.k;
  for (int t = wave; t < a.n; t += kFusedWaves) {
    const int id = wave_rule<KPL>(a, t, &s.rule[wave]);
    if (P <= kSmallPairs && lane < a.k) s_ids[t * a.k + lane] = id;
    wave_sync();
  }
  if (P <= kSmallPairs && threadIdx.x < 4 && P + (int)threadIdx.x < ((P + 3) & ~3))
    s_ids[P + threadIdx.x] = 0x7fffffff;
  __threadfence_block();
  __syncthreads();
  if (P <= kWave)
    group_tiny(s_ids, P, a.E, offsets, pair_index);
  else if (P <= kSmallPairs)
    group_small(s_ids, P, a.E, offsets, pair_index);
  else
    group_block<kFusedWaves>(a.ids, P, a.E, s.group.hist, s.group.off, s.group.wsum, offsets,
                             pair_index);
}

template <int KPL>
hipError_t launch(const RuleArgs& a, const moe_routing* out, void* ws, hipStream_t stream) {
  if (a.n <= kFusedRouteTokens) {
    hipLaunchKernelGGL(k_rule_fused<KPL>, dim3(1), dim3(kFusedWaves * kWave), 0, stream, a,
                       out->expert_offsets, out->pair_index);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_rule_topk<KPL>, dim3((a.n + kRuleWaves - 1) / kRuleWaves),
                     dim3(kRuleWaves * kWave), 0, stream, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  return launch_route_group(out->topk_ids, a.n * a.k, a.E, out, ws, stream);
}

}  // namespace

hipError_t launch_route_scored(const void* logits, int dtype, int n, int E, int k,
                               const moe_route_rule& rule, const moe_routing* out, void* ws,
                               hipStream_t stream) {
  RuleArgs a{};
  a.logits = logits;
  a.bias = rule.bias;
  a.ids = out->topk_ids;
  a.w = out->topk_w;
  a.n = n;
  a.E = E;
  a.k = k;
  a.dtype = dtype;
  a.softmax = rule.score == MOE_SCORE_SOFTMAX;
  a.groups = rule.groups;
  a.top_groups = rule.top_groups;
  a.top2 = rule.group_score == MOE_GROUP_TOP2;
  a.renormalize = rule.renormalize != 0;
  a.lanes = 1;
  while (2 * a.lanes * a.groups <= kWave) a.lanes *= 2;
  a.scale = (double)rule.scale;
  const int kpl = (E + kWave - 1) / kWave;
  if (kpl <= 1) return launch<1>(a, out, ws, stream);
  if (kpl <= 2) return launch<2>(a, out, ws, stream);
  if (kpl <= 4) return launch<4>(a, out, ws, stream);
  if (kpl <= 8) return launch<8>(a, out, ws, stream);
  return launch<16>(a, out, ws, stream);
}

}  // namespace qmoe
