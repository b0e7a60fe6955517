// moe_route.hip -- the top-k router and its gradient.
//
// A wave takes a token: its E logits sit in the wave's registers (logit
// PER * lane + i in register i), the k largest are taken one after the other by
// a maximum over the wave, and the softmax sum is one more reduction.  The
// slots then have to be put in expert order, stably: a slot's row is
//   (slots of smaller experts) + (slots of its expert in earlier blocks)
//   + (those earlier in its block),
// the last from a match of expert numbers inside a wave and a scan over the
// block's waves, without atomics.  For few tokens one workgroup does all of it;
// past that three launches do (choose, scan, place).
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

// Rising unsigned keys in the order of the logits: NaN on top, both zeros alike,
// -inf (not to be chosen) at kNoKey.
constexpr uint32_t kNoKey = 0x007fffffu;
__device__ inline uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t key = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  return v != v ? 0xffffffffu : key;
}
// The logit of a key (any NaN for that of NaN).
__device__ inline float of_key(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Reductions over the wave by lane moves inside rows of 16 lanes and from row to
// row: the result stands in lane 63.  Six moves of the vector unit; through LDS
// (shuffles) the same took 2.5 times as long.
template <class F>
__device__ inline int wave_reduce(int v, int none, F f) {
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x111, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x112, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x114, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x118, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x142, 0xa, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x143, 0xc, 0xf, false));
  return v;
}

__device__ inline uint32_t wave_max(uint32_t v) {
  const auto f = [](int a, int b) { return int(uint32_t(a) > uint32_t(b) ? a : b); };
  return uint32_t(__builtin_amdgcn_readlane(wave_reduce(int(v), 0, f), 63));
}

__device__ inline float wave_fmax(float v) {
  const auto f = [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  };
  const int none = __float_as_int(-__builtin_inff());
  return __int_as_float(
      __builtin_amdgcn_readlane(wave_reduce(__float_as_int(v), none, f), 63));
}

__device__ inline float wave_sum(float v) {
  const auto f = [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  };
  return __int_as_float(__builtin_amdgcn_readlane(wave_reduce(__float_as_int(v), 0, f), 63));
}

__device__ inline int wave_scan(int v) {
  return wave_reduce(v, 0, [](int a, int b) { return a + b; });
}

// exp(x), x <= 0 or NaN, within 2 steps: 2^t for t = x log2(e) rounded, times
// 1 + ln(2) (x log2(e) - t).  Results below the normal numbers are 0.
__device__ inline float exp_of(float x) {
  const float t = x * 1.44269504f;
  const float r = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269504f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return x < -150.0f ? 0.0f : fmaf(e, r * 0.693147181f, e);
}

// A row of E logits: PER of them in a row to a lane, -inf past the end.  VEC:
// every lane's are one aligned piece of the row or all past its end.
template <int PER>
struct Row {
  float v[PER];

  __device__ void load(const void* p, int64_t at, int E, int dtype, bool vec) {
    const int e0 = (threadIdx.x & 63) * PER;
    if (PER > 1 && vec) {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = -__builtin_inff();
      if (e0 >= E) return;
      if (dtype == A2AV_FP32) {
        constexpr int kN = PER < 4 ? PER : 4;
        typedef float Piece __attribute__((ext_vector_type(kN < 2 ? 2 : kN)));
#pragma unroll
        for (int i = 0; i < PER; i += kN) {
          const Piece w = *reinterpret_cast<const Piece*>(static_cast<const float*>(p) + at + e0 + i);
#pragma unroll
          for (int j = 0; j < kN; ++j) v[i + j] = w[j];
        }
      } else {
        constexpr int kN = PER < 8 ? PER : 8;
        typedef uint16_t Piece __attribute__((ext_vector_type(kN < 2 ? 2 : kN)));
#pragma unroll
        for (int i = 0; i < PER; i += kN) {
          const Piece w =
              *reinterpret_cast<const Piece*>(static_cast<const uint16_t*>(p) + at + e0 + i);
#pragma unroll
          for (int j = 0; j < kN; ++j)
            v[i + j] = dtype == A2AV_BF16 ? __uint_as_float(uint32_t(w[j]) << 16)
                                          : float(__builtin_bit_cast(_Float16, uint16_t(w[j])));
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[i] = e0 + i < E ? load_value(p, at + e0 + i, dtype) : -__builtin_inff();
  }

  // dtype's rounding of x, contiguous from p[at] on.
  __device__ static void store(void* p, int64_t at, int E, int dtype, bool vec,
                               const float (&x)[PER]) {
    const int e0 = (threadIdx.x & 63) * PER;
    if (PER > 1 && vec) {
      if (e0 >= E) return;
      if (dtype == A2AV_FP32) {
        constexpr int kN = PER < 4 ? PER : 4;
        typedef float Piece __attribute__((ext_vector_type(kN < 2 ? 2 : kN)));
#pragma unroll
        for (int i = 0; i < PER; i += kN) {
          Piece w;
#pragma unroll
          for (int j = 0; j < kN; ++j) w[j] = x[i + j];
          *reinterpret_cast<Piece*>(static_cast<float*>(p) + at + e0 + i) = w;
        }
      } else {
        constexpr int kN = PER < 8 ? PER : 8;
        typedef uint16_t Piece __attribute__((ext_vector_type(kN < 2 ? 2 : kN)));
#pragma unroll
        for (int i = 0; i < PER; i += kN) {
          Piece w;
#pragma unroll
          for (int j = 0; j < kN; ++j)
            w[j] = dtype == A2AV_BF16 ? __builtin_bit_cast(uint16_t, __bf16(x[i + j]))
                                      : __builtin_bit_cast(uint16_t, _Float16(x[i + j]));
          *reinterpret_cast<Piece*>(static_cast<uint16_t*>(p) + at + e0 + i) = w;
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < E) store_value(p, at + e0 + i, dtype, x[i]);
  }
};

// Whether rows of E logits from p on, `stride` apart, are whole pieces.
template <int PER>
__device__ inline bool row_pieces(const void* p, int64_t stride, int E, int dtype) {
  const int size = dtype == A2AV_FP32 ? 4 : 2;
  const int piece = PER * size < 16 ? PER * size : 16;
  return E % PER == 0 && (stride * size) % piece == 0 &&
         reinterpret_cast<uintptr_t>(p) % uintptr_t(piece) == 0;
}

// One token by one wave: writes experts and weights, and the experts to LDS.
template <int PER>
__device__ inline void choose(const RouteParams& p, int t, const float (&v)[PER], int32_t* ids) {
  const int lane = threadIdx.x & 63;
  // Each lane's keys in falling order, equal ones in their own (neighbours
  // change places only when out of order), and which logits they were, 4 bits
  // each: the choice below looks at first keys alone.
  uint32_t key[PER];
  int id[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    key[i] = key_of(v[i]);
    id[i] = i;
  }
#pragma unroll
  for (int n = 1; n < PER; ++n)
#pragma unroll
    for (int i = n; i > 0; --i) {
      const bool swap = key[i] > key[i - 1];
      const uint32_t hi = swap ? key[i] : key[i - 1], lo = swap ? key[i - 1] : key[i];
      const int hi_id = swap ? id[i] : id[i - 1], lo_id = swap ? id[i - 1] : id[i];
      key[i - 1] = hi, key[i] = lo;
      id[i - 1] = hi_id, id[i] = lo_id;
    }
  uint64_t ids_left = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) ids_left |= uint64_t(id[i]) << (4 * i);
  if (PER <= 8) ids_left = uint32_t(ids_left);

  // Lane j keeps slot j: the largest first key, of the first lane that has it.
  int mine = -1;
  uint32_t mine_key = 0;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t m = wave_max(key[0]);
    if (m <= kNoKey) break;
    const int l = __ffsll((unsigned long long)__ballot(key[0] == m)) - 1;
    const int e = l * PER + (PER > 1 ? __builtin_amdgcn_readlane(int(ids_left), l) & 15 : 0);
    if (lane == j) {
      mine = e;
      mine_key = m;
    }
    if (lane == l) {
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) key[i] = key[i + 1];
      key[PER - 1] = 0;
      if (PER <= 8) ids_left = uint32_t(ids_left) >> 4;
      else ids_left >>= 4;
    }
  }
  const float most = of_key(uint32_t(__builtin_amdgcn_readlane(int(mine_key), 0)));
  const float picked = mine >= 0 ? exp_of(of_key(mine_key) - most) : 0.0f;
  float total = picked;
  if (!p.renorm) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) total += v[i] == -__builtin_inff() ? 0.0f : exp_of(v[i] - most);
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
      at += __builtin_amdgcn_readlane(in, 63);
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
  const bool vec = row_pieces<PER>(p.logits, p.stride, p.E, p.dtype);
  for (int t = wave; t < p.tokens; t += kWaves) {
    Row<PER> row;
    row.load(p.logits, t * p.stride, p.E, p.dtype, vec);
    choose<PER>(p, t, row.v, ids + t * p.k);
  }
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

// Choose: p.per_block tokens; the slots' ranks in the block go to place, the
// block's counts to hist[e][block].
template <int PER>
__global__ __launch_bounds__(kThreads) void route_choose(const RouteParams p, int blocks) {
  __shared__ int32_t ids[kRouteMost * 16];
  __shared__ uint16_t hist[kWaves][kMaxE];
  __shared__ int32_t run[kMaxE];
  const int tid = threadIdx.x, wave = tid >> 6;
  const bool vec = row_pieces<PER>(p.logits, p.stride, p.E, p.dtype);
  for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int t0 = b * p.per_block;
    const int nt = p.tokens - t0 < p.per_block ? p.tokens - t0 : p.per_block;
    // The next token's logits are on their way while one is chosen from.
    Row<PER> row, next;
    if (wave < nt) next.load(p.logits, (t0 + wave) * p.stride, p.E, p.dtype, vec);
    for (int t = wave; t < nt; t += kWaves) {
      row = next;
      if (t + kWaves < nt) next.load(p.logits, (t0 + t + kWaves) * p.stride, p.E, p.dtype, vec);
      choose<PER>(p, t0 + t, row.v, ids + t * p.k);
    }
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
    at += __builtin_amdgcn_readlane(in, 63);
  }
  if (lane == 0) p.counts[e] = at;
}

__global__ __launch_bounds__(kThreads) void route_place(const RouteParams p, int blocks) {
  __shared__ int32_t first[kMaxE];
  const int tid = threadIdx.x;
  for (int i = tid; i < p.E; i += kThreads) first[i] = p.counts[i];
  const int all = first_rows(first, p.E);
  for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int t0 = b * p.per_block;
    const int nt = p.tokens - t0 < p.per_block ? p.tokens - t0 : p.per_block;
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
  const bool vec = row_pieces<PER>(p.logits, p.stride, p.E, p.dtype);
  const bool vec_out = row_pieces<PER>(p.dlogits, p.E, p.E, p.dtype);
  const int64_t step = int64_t(gridDim.x) * 4;
  // A value per expert and wave, zeros but where a slot's lane has put its own:
  // each lane takes the values of its logits from there at once (32768 x 256,
  // top 8, FP32: 21.6 us with a lane read and branches per slot, 15.3 so).
  __shared__ __attribute__((aligned(16))) float of_expert[4][64 * PER];
  float* const mine = of_expert[threadIdx.x >> 6];
#pragma unroll
  for (int i = 0; i < PER; ++i) mine[lane * PER + i] = 0.0f;
  auto in_order = [] {  // a wave's LDS accesses are done in order: keep theirs
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  struct Slots {
    int e;
    float w, dw;
  };
  auto slots = [&](int64_t t) {
    Slots s{-1, 0.0f, 0.0f};
    if (lane < p.k) s = Slots{p.experts[t * p.k + lane], p.weights[t * p.k + lane],
                              p.dweights[t * p.k + lane]};
    return s;
  };
  int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  Row<PER> next;
  Slots next_slots{-1, 0.0f, 0.0f};
  if (t < p.tokens) {
    next_slots = slots(t);
    if (!p.renorm) next.load(p.logits, t * p.stride, p.E, p.dtype, vec);
  }
  for (; t < p.tokens; t += step) {
    const Row<PER> row = next;
    Slots s = next_slots;
    if (t + step < p.tokens) {  // on their way while this token is done
      next_slots = slots(t + step);
      if (!p.renorm) next.load(p.logits, (t + step) * p.stride, p.E, p.dtype, vec);
    }
    if (s.e >= p.E) s.e = -1;
    const float mean = wave_sum(s.e >= 0 ? s.w * s.dw : 0.0f);
    // The slot's dweight, or with renorm its whole gradient.
    in_order();
    if (s.e >= 0) mine[s.e] = !p.renorm ? s.dw : s.w == 0.0f ? 0.0f : s.w * (s.dw - mean);
    in_order();
    float gr[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) gr[i] = mine[lane * PER + i];
    in_order();
    if (s.e >= 0) mine[s.e] = 0.0f;
    if (!p.renorm) {
      float most = row.v[0];  // of the numbers: a NaN makes the sum NaN by itself
#pragma unroll
      for (int i = 1; i < PER; ++i) most = fmaxf(most, row.v[i]);
      most = wave_fmax(most);
      float q[PER], total = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        q[i] = row.v[i] == -__builtin_inff() ? 0.0f : exp_of(row.v[i] - most);
        total += q[i];
      }
      total = wave_sum(total);
      // Times the inverse: one rounding more than a quotient per logit (half a step,
      // 2^-24 of the gradient), for one division per token.
      const float inverse = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        q[i] *= inverse;
        // -inf is asked for by itself: beside a NaN its q, 0 times NaN, is not 0.
        const bool none = row.v[i] == -__builtin_inff() || q[i] == 0.0f;
        gr[i] = none ? 0.0f : q[i] * (gr[i] - mean);
      }
    }
    Row<PER>::store(p.dlogits, t * p.E, p.E, p.dtype, vec_out, gr);
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

hipError_t launch_route(RouteParams p, hipStream_t stream) {
  (void)hipGetLastError();
  p.per_block = route_per_block(p.tokens);
  if (route_is_small(p.tokens, p.E, p.k)) {
    with_per(p.E, [&](auto per) {
      route_small<decltype(per)::value><<<dim3(1), dim3(kThreads), 0, stream>>>(p);
    });
    return hipGetLastError();
  }
  const int blocks = route_blocks(p.tokens);
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
  const int grid = int(want < 2048 ? want : 2048);  // 8 waves per SIMD
  with_per(p.E, [&](auto per) {
    route_back<decltype(per)::value><<<dim3(grid), dim3(256), 0, stream>>>(p);
  });
  return hipGetLastError();
}

}  // namespace a2av
