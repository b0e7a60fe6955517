// moe_route.hip -- the top-k router and its gradient.
//
// A wave takes a token: its E logits sit in the wave's registers (logit
// 64 i + lane in register i), the k largest are taken one after the other by
// a maximum over the wave, and the softmax sum is one more reduction.  The
// slots then have to be put in expert order, stably: a slot's row is
//   (slots of smaller experts) + (slots of its expert in earlier blocks)
//   + (those earlier in its block),
// the last from a match of expert numbers inside a wave and a scan over the
// block's waves, without atomics.  Up to kRouteSmall slots one workgroup does
// all of it; past that three launches do (choose, scan, place).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "a2av.h"
#include "moe.h"

namespace a2av {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxE = 1024;

__device__ inline float load_value(const void* p, int64_t i, int dtype) {
  if (dtype == A2AV_FP32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  if (dtype == A2AV_BF16) return __uint_as_float(uint32_t(h) << 16);
  return float(__builtin_bit_cast(_Float16, h));
}

__device__ inline void store_value(void* p, int64_t i, int dtype, float v) {
  if (dtype == A2AV_FP32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == A2AV_BF16)
    static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, __bf16(v));
  else
    static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, _Float16(v));
}

// Rising unsigned keys in the order of the logits: 0 for -inf (not to be
// chosen), NaN on top, both zeros alike.
__device__ inline uint32_t key_of(float v) {
  v += 0.0f;
  const uint32_t b = __float_as_uint(v);
  if (v != v) return 0xffffffffu;
  if (b == 0xff800000u) return 0;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ inline uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint32_t u = __shfl_xor(v, d);
    v = u > v ? u : v;
  }
  return v;
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ inline int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// One token by one wave: writes experts and weights, and the experts to LDS.
template <int PER>
__device__ inline void choose(const RouteParams& p, int t, int32_t* ids) {
  const int lane = threadIdx.x & 63;
  float v[PER];
  uint32_t key[PER];
  const int64_t at = int64_t(t) * p.stride;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 64 + lane;
    v[i] = e < p.E ? load_value(p.logits, at + e, p.dtype) : -__builtin_inff();
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = key_of(v[i]);

  float most = 0.0f, picked = 0.0f;  // picked: lane j holds slot j
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = key[i] > m ? key[i] : m;
    m = wave_max(m);
    if (m == 0) break;
    int e = -1;
    float val = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t at_i = __ballot(key[i] == m);
      if (e < 0 && at_i) {
        const int l = __ffsll((unsigned long long)at_i) - 1;
        e = i * 64 + l;
        val = __shfl(v[i], l);
        if (lane == l) key[i] = 0;
      }
    }
    if (j == 0) most = val;
    if (lane == j) {
      mine = e;
      picked = expf(val - most);
    }
  }
  float total;
  if (p.renorm) {
    total = picked;
  } else {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) total += v[i] == -__builtin_inff() ? 0.0f : expf(v[i] - most);
  }
  total = wave_sum(total);
  if (lane < p.k) {
    const int64_t s = int64_t(t) * p.k + lane;
    p.experts[s] = mine;
    p.weights[s] = mine >= 0 ? picked / total : 0.0f;
    ids[lane] = mine;
  }
}

// Ranks of the slots [first, first + kThreads) of a block among the block's
// slots of the same expert; run[e] counts those of earlier slots and is moved
// on.  ids in LDS, -1 = empty.  All threads of the workgroup call it.
__device__ inline int rank_slots(const int32_t* ids, int first, int n, int E,
                                 uint16_t (*hist)[kMaxE], int32_t* run) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kWaves * E; i += kThreads) hist[i / E][i % E] = 0;
  __syncthreads();
  const int s = first + tid;
  const int e = s < n ? ids[s] : -1;
  uint64_t same = __ballot(e >= 0);
  for (int b = 1; b < E; b <<= 1) {
    const bool bit = (e & b) != 0;
    const uint64_t m = __ballot(bit);
    same &= bit ? m : ~m;
  }
  const int below = __popcll(same & ((1ull << lane) - 1));
  if (e >= 0 && below == 0) hist[wave][e] = uint16_t(__popcll(same));
  __syncthreads();
  for (int i = tid; i < E; i += kThreads) {
    int at = run[i];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int c = hist[w][i];
      hist[w][i] = uint16_t(at);  // at most kRouteSmall or 64 k slots in a block
      at += c;
    }
    run[i] = at;
  }
  __syncthreads();
  const int r = e >= 0 ? hist[wave][e] + below : -1;
  __syncthreads();
  return r;
}

// The first rows of the experts, from their counts in LDS (in place).
__device__ inline int first_rows(int32_t* counts, int E) {
  __shared__ int32_t all;
  __syncthreads();
  if (threadIdx.x < 64) {
    int at = 0;
    for (int b = 0; b < E; b += 64) {
      const int e = b + int(threadIdx.x);
      const int c = e < E ? counts[e] : 0;
      const int in = wave_scan(c);
      if (e < E) counts[e] = at + in - c;
      at += __shfl(in, 63);
    }
    if (threadIdx.x == 0) all = at;
  }
  __syncthreads();
  return all;
}

template <int PER>
__global__ __launch_bounds__(kThreads) void route_small(const RouteParams p) {
  __shared__ int32_t ids[kRouteSmall];
  __shared__ uint16_t hist[kWaves][kMaxE];
  __shared__ int32_t run[kMaxE];
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int t = wave; t < p.tokens; t += kWaves) choose<PER>(p, t, ids + t * p.k);
  for (int i = tid; i < p.E; i += kThreads) run[i] = 0;
  __syncthreads();
  const int n = p.tokens * p.k;
  int rank[kRouteSmall / kThreads];
#pragma unroll
  for (int q = 0; q < kRouteSmall / kThreads; ++q) {
    rank[q] = -1;
    if (q * kThreads < n) rank[q] = rank_slots(ids, q * kThreads, n, p.E, hist, run);
  }
  for (int i = tid; i < p.E; i += kThreads) p.counts[i] = run[i];
  const int all = first_rows(run, p.E);
#pragma unroll
  for (int q = 0; q < kRouteSmall / kThreads; ++q) {
    const int s = q * kThreads + tid;
    if (s >= n) continue;
    const int r = rank[q] >= 0 ? run[ids[s]] + rank[q] : -1;
    p.place[s] = r;
    if (r >= 0) p.order[r] = s / p.k;
    if (s >= all) p.order[s] = -1;
  }
}

// Choose: kRouteTokens tokens; the slots' ranks in the block go to place, the
// block's counts to hist[e][block].
template <int PER>
__global__ __launch_bounds__(kThreads) void route_choose(const RouteParams p, int blocks) {
  __shared__ int32_t ids[kRouteTokens * 16];
  __shared__ uint16_t hist[kWaves][kMaxE];
  __shared__ int32_t run[kMaxE];
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int t0 = b * kRouteTokens;
    const int nt = p.tokens - t0 < kRouteTokens ? p.tokens - t0 : kRouteTokens;
    for (int t = wave; t < nt; t += kWaves) choose<PER>(p, t0 + t, ids + t * p.k);
    for (int i = tid; i < p.E; i += kThreads) run[i] = 0;
    __syncthreads();
    const int n = nt * p.k;
    for (int f = 0; f < n; f += kThreads) {
      const int r = rank_slots(ids, f, n, p.E, hist, run);
      if (f + tid < n) p.place[int64_t(t0) * p.k + f + tid] = r;
    }
    for (int i = tid; i < p.E; i += kThreads) p.hist[int64_t(i) * blocks + b] = run[i];
    __syncthreads();
  }
}

// Scan: a wave per expert turns its blocks' counts into the slots of that
// expert in earlier blocks.
__global__ __launch_bounds__(64) void route_scan(const RouteParams p, int blocks) {
  const int e = blockIdx.x, lane = threadIdx.x;
  int32_t* h = p.hist + int64_t(e) * blocks;
  int at = 0;
  for (int b = 0; b < blocks; b += 64) {
    const int c = b + lane < blocks ? h[b + lane] : 0;
    const int in = wave_scan(c);
    if (b + lane < blocks) h[b + lane] = at + in - c;
    at += __shfl(in, 63);
  }
  if (lane == 0) p.counts[e] = at;
}

__global__ __launch_bounds__(kThreads) void route_place(const RouteParams p, int blocks) {
  __shared__ int32_t first[kMaxE];
  const int tid = threadIdx.x;
  for (int i = tid; i < p.E; i += kThreads) first[i] = p.counts[i];
  const int all = first_rows(first, p.E);
  for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int t0 = b * kRouteTokens;
    const int nt = p.tokens - t0 < kRouteTokens ? p.tokens - t0 : kRouteTokens;
    const int n = nt * p.k;
    for (int f = tid; f < n; f += kThreads) {
      const int64_t s = int64_t(t0) * p.k + f;
      const int e = p.experts[s];
      int r = -1;
      if (e >= 0) {
        r = first[e] + p.hist[int64_t(e) * blocks + b] + p.place[s];
        p.order[r] = t0 + f / p.k;
      }
      p.place[s] = r;
      if (s >= all) p.order[s] = -1;
    }
  }
}

template <int PER>
__global__ __launch_bounds__(256) void route_back(const RouteBackParams p) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); t < p.tokens;
       t += int64_t(gridDim.x) * 4) {
    int e = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < p.k) {
      const int64_t s = t * p.k + lane;
      e = p.experts[s];
      if (e >= p.E) e = -1;
      if (e >= 0) {
        w = p.weights[s];
        dw = p.dweights[s];
      }
    }
    const float mean = wave_sum(e >= 0 ? w * dw : 0.0f);
    float q[PER], gr[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) q[i] = gr[i] = 0.0f;
    if (!p.renorm) {
      float most = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int x = i * 64 + lane;
        q[i] = x < p.E ? load_value(p.logits, t * p.stride + x, p.dtype) : -__builtin_inff();
        most = q[i] > most || q[i] != q[i] ? q[i] : most;
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) {
        const float u = __shfl_xor(most, d);
        most = u > most || u != u ? u : most;
      }
      if (most == -__builtin_inff()) most = 0.0f;
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        q[i] = q[i] == -__builtin_inff() ? 0.0f : expf(q[i] - most);
        total += q[i];
      }
      total = wave_sum(total);
#pragma unroll
      for (int i = 0; i < PER; ++i) q[i] = total == 0.0f ? 0.0f : q[i] / total;
    }
    for (int j = 0; j < p.k; ++j) {
      const int ej = __shfl(e, j);
      const float wj = __shfl(w, j), dj = __shfl(dw, j);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (ej == i * 64 + lane) {
          gr[i] = dj;
          if (p.renorm) q[i] = wj;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = i * 64 + lane;
      if (x < p.E) store_value(p.dlogits, t * p.E + x, p.dtype, q[i] == 0.0f ? 0.0f : q[i] * (gr[i] - mean));
    }
  }
}

// f(std::integral_constant) with the registers per lane that E logits need.
template <class F>
void with_per(int E, F f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_route(const RouteParams& p, hipStream_t stream) {
  (void)hipGetLastError();
  if (int64_t(p.tokens) * p.k <= kRouteSmall) {
    with_per(p.E, [&](auto per) {
      route_small<decltype(per)::value><<<dim3(1), dim3(kThreads), 0, stream>>>(p);
    });
    return hipGetLastError();
  }
  const int blocks = (p.tokens + kRouteTokens - 1) / kRouteTokens;
  const int grid = blocks < 65536 ? blocks : 65536;
  with_per(p.E, [&](auto per) {
    route_choose<decltype(per)::value><<<dim3(grid), dim3(kThreads), 0, stream>>>(p, blocks);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_scan<<<dim3(p.E), dim3(64), 0, stream>>>(p, blocks);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_place<<<dim3(grid), dim3(kThreads), 0, stream>>>(p, blocks);
  return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackParams& p, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  (void)hipGetLastError();
  const int64_t want = (int64_t(p.tokens) + 3) / 4;
  const int grid = int(want < 65536 ? want : 65536);
  with_per(p.E, [&](auto per) {
    route_back<decltype(per)::value><<<dim3(grid), dim3(256), 0, stream>>>(p);
  });
  return hipGetLastError();
}

}  // namespace a2av
