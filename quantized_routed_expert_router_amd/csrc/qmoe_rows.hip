// Norm and rotation of query and key heads, and the append to a paged key-value cache.
#include "qmoe_attn_internal.h"

namespace qmoe {
namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsWaves = kRowsThreads / kWave;
[[maybe_unused]] constexpr int kMaxAngles = 128;  // rot_dim / 2

struct RowsParams {
  HeadView q, k, v, q_out, k_out;
  const int32_t* positions;
  const int32_t* slots;
  const float* q_norm;
  const float* k_norm;
  const float* inv_freq;
  const float* k_scale;
  const float* v_scale;
  char* ck;
  char* cv;
  float eps, weight_offset;
  int n, rot, interleaved;
  int parts, iters_per_part;  // waves of a token's query and key rows, row groups of each
  int vparts;                 // waves of a token's value heads (append)
  int num_slots, page_shift, kv_heads;
};

enum CacheKind { kNoCache = 0, kCache16 = 1, kCacheE4m3 = 2 };

#if defined(__HIP_DEVICE_COMPILE__)

template <typename A>
__device__ __forceinline__ float widen1(uint32_t half) {
  const uint16_t b = (uint16_t)half;
  return (float)bits_as<typename A::T>(b);
}

// sin and cos of r in [-pi/4, pi/4] by their Taylor sums to r^9 and r^10: the terms left out
// are below 2^-28.
__device__ __forceinline__ void sin_cos_octant(float r, float& s, float& c) {
  const float z = r * r;
  float ps = __builtin_fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  ps = __builtin_fmaf(z, ps, 1.0f / 120.0f);
  ps = __builtin_fmaf(z, ps, -1.0f / 6.0f);
  s = __builtin_fmaf(r * z, ps, r);
  float pc = __builtin_fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  pc = __builtin_fmaf(z, pc, -1.0f / 720.0f);
  pc = __builtin_fmaf(z, pc, 1.0f / 24.0f);
  pc = __builtin_fmaf(z, pc, -0.5f);
  c = __builtin_fmaf(z, pc, 1.0f);
}

// cos and sin of the token's angles into the wave's part of LDS: angle i in entry i. The
// product and the reduction to a quarter turn are in binary64 (positions far into a context
// leave no fraction bits in fp32), the functions of the reduced angle in fp32.
__device__ __forceinline__ void token_angles(const RowsParams& p, int position, int lane,
                                             float* cs, float* sn) {
  const double pos = (double)position;
  for (int i = lane; i < p.rot / 2; i += kWave) {
    const double a = pos * (double)p.inv_freq[i];
    const double quarters = __builtin_rint(a * 0.63661977236758134308);
    double r = __builtin_fma(-quarters, 1.57079632679489655800, a);
    r = __builtin_fma(-quarters, 6.12323399573676603587e-17, r);
    float s, c;
    sin_cos_octant((float)r, s, c);
    // quarters modulo 4, exact up to 2^53
    const int n = (int)(quarters - 4.0 * __builtin_floor(quarters * 0.25));
    const float x = n & 1 ? s : c, y = n & 1 ? c : s;
    cs[i] = n == 1 || n == 2 ? -x : x;
    sn[i] = n >= 2 ? -y : y;
  }
  // the wave's own writes, read back by the same wave
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Sum over the LPR (8, 16 or 32) neighbouring lanes of a row, in every one of them.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + bits_as<float>(
                 __builtin_amdgcn_update_dpp(0, bits_as<int>(x), CTRL, 0xf, 0xf, true));
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  x = add_dpp<0xb1>(x);                          // quad_perm 1 0 3 2
  x = add_dpp<0x4e>(x);                          // quad_perm 2 3 0 1
  x = add_dpp<0x141>(x);                         // row_half_mirror
  if constexpr (LPR >= 16) x = add_dpp<0x140>(x);  // row_mirror
  if constexpr (LPR >= 32) x += __shfl_xor(x, 16);
  return x;
}

// 1 / sqrt(x): the hardware's (1 ulp), with small arguments scaled into its range.
__device__ __forceinline__ float inv_sqrt(float x) {
  const bool small = x < 0x1p-96f;
  const float r = __builtin_amdgcn_rsqf(small ? x * 0x1p64f : x);
  return small ? r * 0x1p32f : r;
}

struct Weights {
  f32x4 lo, hi;
};
__device__ __forceinline__ f32x4 load4(const float* p) {  // 4-byte aligned
  f32x4 v;
  __builtin_memcpy(&v, p, sizeof v);
  return v;
}

// One wave's share of a token's query and key rows: LPR = D/8 lanes hold one row, 8
// elements a lane, 64/LPR rows at a time, first the query heads, then the key heads. A
// lane's 8 elements are 4 rotation pairs: 4 elements of the first half and their partners
// in the second (interleaved, or beyond the rotation: 8 consecutive ones), so that the
// rotation needs no other lane.
template <typename A, int D, int CACHE>
__device__ __forceinline__ void rows_wave(const RowsParams& p, int token, int part, int lane,
                                          float* cs, float* sn) {
  typedef typename A::V4 V4;
  constexpr int LPR = D / 8, RPI = kWave / LPR;
  const int sub = lane / LPR, j = lane % LPR;
  const int qgroups = (p.q.heads + RPI - 1) / RPI;
  const int it0 = part * p.iters_per_part;
  const int it1 = min(it0 + p.iters_per_part, qgroups + (p.k.heads + RPI - 1) / RPI);
  if (it0 >= it1) return;
  const bool turned = 8 * j < p.rot;
  const bool halves = turned && !p.interleaved;
  const int e0 = halves ? 4 * j : 8 * j, e1 = halves ? p.rot / 2 + 4 * j : 8 * j + 4;

  struct Raw {
    u32x2 lo, hi;
  };
  auto load = [&](int it) -> Raw {
    const bool is_q = it < qgroups;
    const HeadView& v = is_q ? p.q : p.k;
    const uint32_t row = (uint32_t)min((is_q ? it : it - qgroups) * RPI + sub, v.heads - 1);
    const char* at = v.data + 2 * ((uint64_t)(uint32_t)token * (uint32_t)v.token_stride +
                                   (uint64_t)row * (uint32_t)v.head_stride);
    return {*reinterpret_cast<const u32x2*>(at + 2 * e0),
            *reinterpret_cast<const u32x2*>(at + 2 * e1)};
  };
  // everything that the first rows need is on its way before the angles are computed
  Raw next = load(it0);
  Raw after = load(min(it0 + 1, it1 - 1));
  Weights wq{1.0f, 1.0f}, wk{1.0f, 1.0f};
  if (p.q_norm) wq = {load4(p.q_norm + e0), load4(p.q_norm + e1)};
  if (p.k_norm) wk = {load4(p.k_norm + e0), load4(p.k_norm + e1)};
  int slot = 0;
  if constexpr (CACHE != kNoCache) slot = p.slots[token];
  f32x4 c4 = 1.0f, s4 = 0.0f;
  if (p.rot > 0) {
    token_angles(p, p.positions[token], lane, cs, sn);
    if (turned) {
      c4 = *reinterpret_cast<const f32x4*>(cs + 4 * j);
      s4 = *reinterpret_cast<const f32x4*>(sn + 4 * j);
    }
  }
  if (p.q_norm) wq = {wq.lo + p.weight_offset, wq.hi + p.weight_offset};
  if (p.k_norm) wk = {wk.lo + p.weight_offset, wk.hi + p.weight_offset};
  const bool stored = slot >= 0 && slot < p.num_slots;

  for (int it = it0; it < it1; ++it) {
    const Raw raw = next;
    next = after;
    after = load(min(it + 2, it1 - 1));
    const bool is_q = it < qgroups;
    const HeadView& in = is_q ? p.q : p.k;
    const int row = (is_q ? it : it - qgroups) * RPI + sub;
    f32x4 lo = __builtin_convertvector(bits_as<V4>(raw.lo), f32x4);
    f32x4 hi = __builtin_convertvector(bits_as<V4>(raw.hi), f32x4);
    if (is_q ? p.q_norm != nullptr : p.k_norm != nullptr) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ss = __builtin_fmaf(lo[e], lo[e], ss);
        ss = __builtin_fmaf(hi[e], hi[e], ss);
      }
      const float inv = inv_sqrt(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
      lo *= inv;
      hi *= inv;
      if (is_q) {
        lo *= wq.lo;
        hi *= wq.hi;
      } else {
        lo *= wk.lo;
        hi *= wk.hi;
      }
    }
    if (p.rot > 0) {
      f32x4 x = lo, y = hi;
      if (p.interleaved) {
        x = f32x4{lo[0], lo[2], hi[0], hi[2]};
        y = f32x4{lo[1], lo[3], hi[1], hi[3]};
      }
      f32x4 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = __builtin_fmaf(x[e], c4[e], -(y[e] * s4[e]));
        b[e] = __builtin_fmaf(y[e], c4[e], x[e] * s4[e]);
      }
      if (turned) {
        lo = p.interleaved ? f32x4{a[0], b[0], a[1], b[1]} : a;
        hi = p.interleaved ? f32x4{a[2], b[2], a[3], b[3]} : b;
      }
    }
    if (row >= in.heads) continue;
    if (is_q || CACHE == kNoCache) {
      const HeadView& o = is_q ? p.q_out : p.k_out;
      char* at = o.data + 2 * ((uint64_t)(uint32_t)token * (uint32_t)o.token_stride +
                               (uint64_t)(uint32_t)row * (uint32_t)o.head_stride);
      *reinterpret_cast<u32x2*>(at + 2 * e0) = bits_as<u32x2>(__builtin_convertvector(lo, V4));
      *reinterpret_cast<u32x2*>(at + 2 * e1) = bits_as<u32x2>(__builtin_convertvector(hi, V4));
    } else if (stored) {
      const long long page = slot >> p.page_shift;
      const long long at = (((page * p.kv_heads + row) << p.page_shift) +
                            (slot & ((1 << p.page_shift) - 1))) * D;
      if constexpr (CACHE == kCacheE4m3) {
        const float scale = p.k_scale ? p.k_scale[row] : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = lo[e] / scale;
          hi[e] = hi[e] / scale;
        }
        *reinterpret_cast<uint32_t*>(p.ck + at + e0) =
            pack_e4m3(lo[0], lo[1]) | pack_e4m3(lo[2], lo[3]) << 16;
        *reinterpret_cast<uint32_t*>(p.ck + at + e1) =
            pack_e4m3(hi[0], hi[1]) | pack_e4m3(hi[2], hi[3]) << 16;
      } else {
        *reinterpret_cast<u32x2*>(p.ck + 2 * (at + e0)) =
            bits_as<u32x2>(__builtin_convertvector(lo, V4));
        *reinterpret_cast<u32x2*>(p.ck + 2 * (at + e1)) =
            bits_as<u32x2>(__builtin_convertvector(hi, V4));
      }
    }
  }
}

// One wave's share of the value heads of one run: the tokens from `token` on that go to
// consecutive slots of one group of 8 rows. Only the first token of such a run does the
// work, so a column's 8 rows leave as one 16-byte (8-byte) word when the run is whole.
template <typename A, int D, int CACHE>
__device__ __forceinline__ void values_wave(const RowsParams& p, int token, int part, int lane) {
  const int slot = p.slots[token];
  if (slot < 0 || slot >= p.num_slots) return;
  const int r0 = slot & 7;
  if (r0 != 0 && token > 0 && p.slots[token - 1] == slot - 1) return;
  int m = 1;
  while (m < 8 - r0 && token + m < p.n && p.slots[token + m] == slot + m) ++m;

  constexpr int PAIRS = D / 2;  // two adjacent columns a lane
  const int total = p.kv_heads * PAIRS;
  const long long page = slot >> p.page_shift;
  const int group = (slot & ((1 << p.page_shift) - 1)) >> 3;
  for (int idx = part * kWave + lane; idx < total; idx += p.vparts * kWave) {
    const int h = idx / PAIRS, d = 2 * (idx % PAIRS);
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = i < m ? *reinterpret_cast<const uint32_t*>(
                         p.v.data + 2 * ((long long)(token + i) * p.v.token_stride +
                                         (long long)h * p.v.head_stride + d))
                   : 0u;
    const long long at =
        ((((page * p.kv_heads + h) << p.page_shift) >> 3) + group) * (8 * D) + 8 * d;
    if constexpr (CACHE == kCacheE4m3) {
      const float scale = p.v_scale ? p.v_scale[h] : 1.0f;
      uint32_t code[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        code[i] = pack_e4m3(widen1<A>(x[i] & 0xffffu) / scale, widen1<A>(x[i] >> 16) / scale);
      if (m == 8) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] = (code[4 * i] & 0xffu) | (code[4 * i + 1] & 0xffu) << 8 |
                 (code[4 * i + 2] & 0xffu) << 16 | (code[4 * i + 3] & 0xffu) << 24;
          w[2 + i] = code[4 * i] >> 8 | (code[4 * i + 1] >> 8) << 8 |
                     (code[4 * i + 2] >> 8) << 16 | (code[4 * i + 3] >> 8) << 24;
        }
        *reinterpret_cast<u32x4*>(p.cv + at) = w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < m) {
            p.cv[at + r0 + i] = (char)(code[i] & 0xffu);
            p.cv[at + 8 + r0 + i] = (char)(code[i] >> 8);
          }
      }
    } else {
      char* to = p.cv + 2 * at;
      if (m == 8) {
        u32x4 even, odd;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          even[i] = (x[2 * i] & 0xffffu) | x[2 * i + 1] << 16;
          odd[i] = x[2 * i] >> 16 | (x[2 * i + 1] & 0xffff0000u);
        }
        reinterpret_cast<u32x4*>(to)[0] = even;
        reinterpret_cast<u32x4*>(to)[1] = odd;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < m) {
            reinterpret_cast<uint16_t*>(to)[r0 + i] = (uint16_t)(x[i] & 0xffffu);
            reinterpret_cast<uint16_t*>(to)[8 + r0 + i] = (uint16_t)(x[i] >> 16);
          }
      }
    }
  }
}

#endif  // __HIP_DEVICE_COMPILE__

// Norm, rotation and append: every row is read once and written once, so memory bounds it
// (and the launch, at a few tokens). A wave takes `iters_per_part` groups of one token's
// rows: the angles cost about as much as ten rows and are computed once for all of them.
// 8192 tokens, 32 + 8 heads of 128, bf16: 30 us, 5.5 TB/s moved (a copy of 2 GB reaches
// 4.9; a part of this chunk stays in the last cache). 4 tokens: 3.7 us.
template <typename A, int D, int CACHE>
__global__ __launch_bounds__(kRowsThreads) void k_rows(RowsParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __align__(16) float angles[kRowsWaves][2][kMaxAngles];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  const int token = blockIdx.x * kRowsWaves + wave, part = blockIdx.y;
  if (token >= p.n) return;
  if (part < p.parts)
    rows_wave<A, D, CACHE>(p, token, part, lane, angles[wave][0], angles[wave][1]);
  else if constexpr (CACHE != kNoCache)
    values_wave<A, D, CACHE>(p, token, part - p.parts, lane);
#endif
}

template <typename A, int D, int CACHE>
hipError_t launch_one(const RowsParams& p, hipStream_t stream) {
  const unsigned blocks = (unsigned)((p.n + kRowsWaves - 1) / kRowsWaves);
  const unsigned parts = (unsigned)(p.parts + (CACHE != kNoCache ? p.vparts : 0));
  k_rows<A, D, CACHE><<<dim3(blocks, parts), dim3(kRowsThreads), 0, stream>>>(p);
  return hipGetLastError();
}

template <typename A, int CACHE>
hipError_t launch_dim(const RowsParams& p, int D, hipStream_t stream) {
  if (D == 64) return launch_one<A, 64, CACHE>(p, stream);
  if (D == 128) return launch_one<A, 128, CACHE>(p, stream);
  return launch_one<A, 256, CACHE>(p, stream);
}

template <typename A>
hipError_t launch_type(const RowsParams& p, int D, int kind, hipStream_t stream) {
  if (kind == kNoCache) return launch_dim<A, kNoCache>(p, D, stream);
  if (kind == kCache16) return launch_dim<A, kCache16>(p, D, stream);
  return launch_dim<A, kCacheE4m3>(p, D, stream);
}

}  // namespace

hipError_t launch_rows(const RowsArgs& a) {
  RowsParams p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_out = a.q_out;
  p.k_out = a.k_out;
  p.positions = a.positions;
  p.slots = a.slots;
  p.q_norm = a.p.q_norm;
  p.k_norm = a.p.k_norm;
  p.inv_freq = a.p.inv_freq;
  p.eps = a.p.eps;
  p.weight_offset = a.p.weight_offset;
  p.n = a.n;
  p.rot = a.p.rot_dim;
  p.interleaved = a.p.interleaved != 0;
  const int per_iter = kWave / (a.D / 8);
  const int iters = (a.q.heads + per_iter - 1) / per_iter + (a.k.heads + per_iter - 1) / per_iter;
  // enough waves for 8 on every CU; beyond that a token's rows stay with one wave
  const int want = 8 * a.num_cus;
  p.parts = std::max(1, std::min(iters, (want + a.n - 1) / a.n));
  p.iters_per_part = (iters + p.parts - 1) / p.parts;
  p.parts = (iters + p.iters_per_part - 1) / p.iters_per_part;
  int kind = kNoCache;
  if (a.cache) {
    kind = a.cache->dtype == MOE_E4M3 ? kCacheE4m3 : kCache16;
    p.k_scale = a.cache->k_scale;
    p.v_scale = a.cache->v_scale;
    p.ck = (char*)a.cache->k;
    p.cv = (char*)a.cache->v;
    p.kv_heads = a.cache->kv_heads;
    p.num_slots = a.cache->num_pages * a.cache->page_size;
    while ((1 << p.page_shift) < a.cache->page_size) ++p.page_shift;
    const int viters = (p.kv_heads * (a.D / 2) + kWave - 1) / kWave;
    p.vparts = std::max(1, std::min(viters, (want + a.n - 1) / a.n));
  }
  return a.dtype == MOE_BF16 ? launch_type<Bf16>(p, a.D, kind, a.stream)
                             : launch_type<F16>(p, a.D, kind, a.stream);
}

}  // namespace qmoe
