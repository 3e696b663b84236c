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
__device__ __forceinline__ f32x8 widen(const u32x4& w) {
  return __builtin_convertvector(bits_as<typename A::V8>(w), f32x8);
}

template <typename A>
__device__ __forceinline__ float widen1(uint32_t half) {
  const uint16_t b = (uint16_t)half;
  return (float)bits_as<typename A::T>(b);
}

// cos and sin of the token's angles into the wave's part of LDS: angle i in entry i. The
// product and the reduction to (-pi, pi) are in binary64 (positions far into a context
// leave no fraction bits in fp32), the functions of the reduced angle in fp32.
__device__ __forceinline__ void token_angles(const RowsParams& p, int token, int lane, float* cs,
                                             float* sn) {
  const double pos = (double)p.positions[token];
  for (int i = lane; i < p.rot / 2; i += kWave) {
    const double a = pos * (double)p.inv_freq[i];
    const double turns = __builtin_rint(a * 0.15915494309189533577);
    double r = __builtin_fma(-turns, 6.28318530717958623200, a);
    r = __builtin_fma(-turns, 2.44929359829470641435e-16, r);
    float s, c;
    sincosf((float)r, &s, &c);
    cs[i] = c;
    sn[i] = s;
  }
  // the wave's own writes, read back by the same wave
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One wave's share of a token's query and key rows: LPR = D/8 lanes hold one row, 8
// elements a lane, 64/LPR rows at a time.
template <typename A, int D, int CACHE>
__device__ __forceinline__ void rows_wave(const RowsParams& p, int token, int part, int lane,
                                          float* cs, float* sn) {
  constexpr int LPR = D / 8, RPI = kWave / LPR;
  const int sub = lane / LPR, j = lane % LPR;
  const int hq = p.q.heads, rows = hq + p.k.heads;
  const int half = p.rot / 2;

  if (p.rot > 0) token_angles(p, token, lane, cs, sn);
  // this lane's 8 elements: which angles turn them, and which lane holds their partners
  const bool turned = 8 * j < p.rot;
  const bool second = !p.interleaved && 8 * j >= half;
  const int first_angle = !turned ? 0 : p.interleaved ? 4 * j : 8 * j - (second ? half : 0);
  const int hop = turned && !p.interleaved ? (second ? -half / 8 : half / 8) : 0;
  f32x8 c8, s8;  // interleaved: entries 0..3
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool live = turned && (!p.interleaved || e < 4);
    c8[e] = live ? cs[first_angle + e] : 1.0f;
    s8[e] = live ? sn[first_angle + e] : 0.0f;
  }
  f32x8 wq, wk;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wq[e] = p.q_norm ? p.q_norm[8 * j + e] + p.weight_offset : 1.0f;
    wk[e] = p.k_norm ? p.k_norm[8 * j + e] + p.weight_offset : 1.0f;
  }
  int slot = 0;
  bool stored = true;
  if constexpr (CACHE != kNoCache) {
    slot = p.slots[token];
    stored = slot >= 0 && slot < p.num_slots;
  }

  const int it0 = part * p.iters_per_part;
  const int it1 = min(it0 + p.iters_per_part, (rows + RPI - 1) / RPI);
  auto source = [&](int it) -> const u32x4* {
    const int r = min(it * RPI + sub, rows - 1);
    const HeadView& v = r < hq ? p.q : p.k;
    const long long h = r < hq ? r : r - hq;
    return reinterpret_cast<const u32x4*>(
        v.data + 2 * ((long long)token * v.token_stride + h * v.head_stride + 8 * j));
  };
  if (it0 >= it1) return;
  u32x4 next = *source(it0);
  for (int it = it0; it < it1; ++it) {
    const u32x4 raw = next;
    if (it + 1 < it1) next = *source(it + 1);
    const int r = it * RPI + sub;
    const bool is_q = r < hq;
    f32x8 y = widen<A>(raw);
    const bool normed = is_q ? p.q_norm != nullptr : p.k_norm != nullptr;
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(y[e], y[e], ss);
#pragma unroll
    for (int m = 1; m < LPR; m *= 2) ss += __shfl_xor(ss, m);
    const float inv = normed ? 1.0f / sqrtf(ss * (1.0f / D) + p.eps) : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * (is_q ? wq[e] : wk[e]);
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = y[2 * e], b = y[2 * e + 1];
        if (turned) {
          y[2 * e] = a * c8[e] - b * s8[e];
          y[2 * e + 1] = b * c8[e] + a * s8[e];
        }
      }
    } else if (p.rot > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl(y[e], lane + hop);
        const float cross = second ? other * s8[e] : -(other * s8[e]);
        if (turned) y[e] = y[e] * c8[e] + cross;
      }
    }
    if (r >= rows) continue;
    if (is_q || CACHE == kNoCache) {
      const HeadView& o = is_q ? p.q_out : p.k_out;
      const long long h = is_q ? r : r - hq;
      const u32x4 w = bits_as<u32x4>(__builtin_convertvector(y, typename A::V8));
      *reinterpret_cast<u32x4*>(
          o.data + 2 * ((long long)token * o.token_stride + h * o.head_stride + 8 * j)) = w;
    } else if (stored) {
      const int h = r - hq;
      const long long page = slot >> p.page_shift;
      const long long at = (((page * p.kv_heads + h) << p.page_shift) +
                            (slot & ((1 << p.page_shift) - 1))) * D + 8 * j;
      if constexpr (CACHE == kCacheE4m3) {
        const float scale = p.k_scale ? p.k_scale[h] : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] / scale;
        const u32x2 w = {pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16,
                         pack_e4m3(y[4], y[5]) | pack_e4m3(y[6], y[7]) << 16};
        *reinterpret_cast<u32x2*>(p.ck + at) = w;
      } else {
        *reinterpret_cast<u32x4*>(p.ck + 2 * at) =
            bits_as<u32x4>(__builtin_convertvector(y, typename A::V8));
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
template <typename A, int D, int CACHE>
__global__ __launch_bounds__(kRowsThreads) void k_rows(RowsParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float angles[kRowsWaves][2][kMaxAngles];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  const int id = blockIdx.x * kRowsWaves + wave;
  const int nrows = p.n * p.parts;
  if (id < nrows) {
    rows_wave<A, D, CACHE>(p, id / p.parts, id % p.parts, lane, angles[wave][0], angles[wave][1]);
  } else if constexpr (CACHE != kNoCache) {
    const int v = id - nrows;
    if (v < p.n * p.vparts) values_wave<A, D, CACHE>(p, v / p.vparts, v % p.vparts, lane);
  }
#endif
}

template <typename A, int D, int CACHE>
hipError_t launch_one(const RowsParams& p, hipStream_t stream) {
  const long long waves =
      (long long)p.n * p.parts + (CACHE != kNoCache ? (long long)p.n * p.vparts : 0);
  const unsigned blocks = (unsigned)((waves + kRowsWaves - 1) / kRowsWaves);
  k_rows<A, D, CACHE><<<dim3(blocks), dim3(kRowsThreads), 0, stream>>>(p);
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
  const int iters = (a.q.heads + a.k.heads + per_iter - 1) / per_iter;
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
