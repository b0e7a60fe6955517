// moe_route.hip -- the top-k router, the router by groups, and their gradients.
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
//
// The router by groups compares sums that FP32 rounds.  It chooses in FP32 wherever the
// bounds of every sum's own error tell experts and groups apart, and does the other tokens
// again in 64 bits, so that the choice is that of 64 bits; up to 256 experts 16 lanes take
// a token and a wave four of them.
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
    load_from((threadIdx.x & 63) * PER, p, at, E, dtype, vec);
  }
  __device__ void load_from(int e0, const void* p, int64_t at, int E, int dtype, bool vec) {
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

// The k largest of a wave's values, in falling order, equal ones by their number:
// lane j gets the j-th, its number in `mine` and its key, -1 where there is none left
// but -inf.  Returns the key of the largest that is left.
template <int PER>
__device__ inline uint32_t take_largest(const float (&v)[PER], int k, int& mine,
                                        uint32_t& mine_key) {
  const int lane = threadIdx.x & 63;
  // Each lane's keys in falling order, equal ones in their own (neighbours
  // change places only when out of order), and which values they were, 4 bits
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
  mine = -1;
  mine_key = 0;
  for (int j = 0; j < k; ++j) {
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
  return key[0];
}

// One token by one wave: writes experts and weights, and the experts to LDS.
template <int PER>
__device__ inline void choose(const RouteParams& p, int t, const float (&v)[PER], int32_t* ids) {
  const int lane = threadIdx.x & 63;
  int mine;
  uint32_t mine_key;
  take_largest<PER>(v, p.k, mine, mine_key);
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

// ------------------------------------------------------------------ the router by groups

// Rising unsigned keys in the order of the numbers, NaN on top, as key_of's.
__device__ inline uint64_t key64_of(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));
  const uint64_t key = b ^ (uint64_t(int64_t(b) >> 63) | 1ull << 63);
  return v != v ? ~0ull : key;
}
__device__ inline double of_key64(uint64_t key) {
  return __longlong_as_double(int64_t(key >> 63 ? key & ~(1ull << 63) : ~key));
}

__device__ inline uint64_t lane64(uint64_t v, int lane) {
  return uint64_t(uint32_t(__builtin_amdgcn_readlane(int(uint32_t(v)), lane))) |
         uint64_t(uint32_t(__builtin_amdgcn_readlane(int(uint32_t(v >> 32)), lane))) << 32;
}
__device__ inline double wave_sum64(double v) {
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// One token by one wave, as the definition says it: scores in 64 bits.  A lane has NE
// neighbouring experts, so that the first of equal ones is the first lane's first.
template <int NE>
__device__ inline void choose_grouped(const RouteParams& p, int t, const float* bias, int32_t* ids,
                                      float* scratch) {
  const int lane = threadIdx.x & 63, size = p.E / p.groups, e0 = lane * NE;
  const float none = -__builtin_inff();
  auto in_order = [] {  // a wave's LDS accesses are done in order: keep theirs
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  Row<NE> l;
  l.load(p.logits, int64_t(t) * p.stride, p.E, p.dtype,
         row_pieces<NE>(p.logits, p.stride, p.E, p.dtype));
  double most = 0.0, sum_of_exp = 1.0;
  if (!p.sigmoid) {
    float top = none;
#pragma unroll
    for (int i = 0; i < NE; ++i) top = fmaxf(top, l.v[i]);
    most = double(wave_fmax(top));
  }
  double x[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const double v = double(l.v[i]);
    x[i] = l.v[i] == none ? 0.0 : exp(p.sigmoid ? -v : v - most);
  }
  if (!p.sigmoid) {
    sum_of_exp = x[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) sum_of_exp += x[i];
    sum_of_exp = wave_sum64(sum_of_exp);
  }
  auto score = [&](double y) { return p.sigmoid ? 1.0 / (1.0 + y) : y / sum_of_exp; };
  uint64_t key[NE];  // 0: not to be chosen
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const double c = p.bias ? score(x[i]) + double(bias[e0 + i]) : score(x[i]);
    key[i] = l.v[i] == none || c == -__builtin_inf() ? 0 : key64_of(c);
  }
  uint64_t allowed = ~0ull;
  if (p.groups > 1) {
    uint64_t* const keys = reinterpret_cast<uint64_t*>(scratch);
    in_order();
#pragma unroll
    for (int i = 0; i < NE; ++i) keys[e0 + i] = key[i];
    in_order();
    int span = 64;  // lanes of a group
    while (span * p.groups > 64) span >>= 1;
    const int g = lane / span;
    uint64_t one = 0, two = 0;
    if (g < p.groups)
      for (int i = lane & (span - 1); i < size; i += span) {
        const uint64_t k = keys[g * size + i];
        two = k > one ? one : k > two ? k : two;
        one = k > one ? k : one;
      }
    for (int d = 1; d < span; d <<= 1) {
      const uint64_t a = __shfl_xor((unsigned long long)one, d);
      const uint64_t b = __shfl_xor((unsigned long long)two, d);
      const uint64_t low = a < one ? a : one, high = b > two ? b : two;
      one = a > one ? a : one;
      two = low > high ? low : high;
    }
    uint64_t group_key = 0;
    if (one) {
      double sum = one == ~0ull ? __builtin_nan("") : of_key64(one);
      if (p.group_best == 2 && two) sum += two == ~0ull ? __builtin_nan("") : of_key64(two);
      group_key = key64_of(sum);
    }
    int rank = 0;
    for (int i = 0; i < p.groups; ++i) {
      const uint64_t k = lane64(group_key, i * span);
      rank += k > group_key || (k == group_key && i < g);
    }
    const uint64_t lanes = __ballot(group_key != 0 && rank < p.top_groups);
    allowed = 0;
    for (int i = 0; i < p.groups; ++i) allowed |= (lanes >> (i * span) & 1) << i;
  }
  // In whose order experts are taken, 0 for those of other groups.  No other key has
  // zeros for its upper half.
  int group = p.groups > 1 ? e0 / size : 0, in_group = e0 - group * size;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if (!(allowed >> (group & 63) & 1)) key[i] = 0;
    else if (key[i] && !p.bias) key[i] = uint64_t(key_of(l.v[i])) << 32;
    if (++in_group == size) in_group = 0, ++group;
  }
  double* const powers = reinterpret_cast<double*>(scratch);
  in_order();
#pragma unroll
  for (int i = 0; i < NE; ++i) powers[e0 + i] = x[i];
  in_order();
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    uint64_t top = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NE; ++i)
      if (key[i] > top) top = key[i], at = i;
    const uint32_t hi = wave_max(uint32_t(top >> 32));
    if (!hi) break;
    bool is = uint32_t(top >> 32) == hi;
    uint64_t who = __ballot(is);
    if (who & (who - 1)) {
      const uint32_t lo = wave_max(is ? uint32_t(top) : 0u);
      is = is && uint32_t(top) == lo;
      who = __ballot(is);
    }
    const int from = __ffsll((unsigned long long)who) - 1;
    const int e = from * NE + __builtin_amdgcn_readlane(at, from);
    if (lane == j) mine = e;
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (i == at) key[i] = 0;
    }
  }
  const double s = mine >= 0 ? score(powers[mine]) : 0.0;
  double total = 1.0;
  if (p.renorm) {  // over the lanes that have slots
    total = s;
    for (int d = 1; d < 16; d <<= 1) total += __shfl_xor(total, d);
  }
  if (lane < p.k) {
    const int64_t slot = int64_t(t) * p.k + lane;
    p.experts[slot] = mine;
    p.weights[slot] = mine < 0 || total == 0.0 ? 0.0f : float(double(p.scale) * (s / total));
    ids[lane] = mine;
  }
}

// A lane's value from the lane that its own number with the bits of D (1 to 8) changed
// names, where the lanes of each smaller block hold one value already: moves inside
// rows of 16, mirrored halves and rows doing for 4 and 8.
template <int D>
__device__ inline float other_lanes(float v) {
  constexpr int kCtrl = D == 1 ? 0xb1 : D == 2 ? 0x4e : D == 4 ? 0x141 : 0x140;
  if constexpr (D <= 8)
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
  else
    return __shfl_xor(v, D);
}

// The largest two of the values of blocks of `span` lanes (a power of two).
template <int D>
__device__ inline void join_best(float& one, float& two, int span) {
  if (D < span) {
    const float a = other_lanes<D>(one), b = other_lanes<D>(two);
    two = fmaxf(fminf(one, a), fmaxf(two, b));
    one = fmaxf(one, a);
    if constexpr (D < 32) join_best<D * 2>(one, two, span);
  }
}

// f(0) .. f(15), each number as a type.
template <int N = 0, class F>
__device__ inline void each16(F f) {
  f(std::integral_constant<int, N>{});
  if constexpr (N < 15) each16<N + 1>(f);
}

// What a lane keeps over its tokens, of which each has LANES: how the groups lie among
// its experts.
template <int PER, int LANES>
struct Groups {
  uint64_t number = 0;   // the PER experts' groups after the first's, 4 bits each
  int first;             // group of the lane's first expert
  int span;              // lanes of a group, when they hold nothing else; else 0
  int size;

  __device__ void init(const RouteParams& p) {
    const int e0 = (threadIdx.x & (LANES - 1)) * PER;
    size = p.E / p.groups;
    first = e0 / size;
    int in_group = e0 - first * size, after = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      number |= uint64_t(after) << (4 * i);
      if (++in_group == size) in_group = 0, ++after;
    }
    const int lanes = size / PER;
    span = size % PER == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  }
};

// How far apart sums of score and bias have to be, in FP32, to stand in their true
// order, as a part of `reach`, the token's largest score (sigmoid: 1), and of the sum
// itself.  One step is 2^-23 of a value; exp is within 2 steps, the inverse within one.
// Sigmoid: past 1/2 a quarter of exp's error, half a step of 1 + x and one of the
// inverse, 2^-22; below 1/2 half of exp's and a product's half step more, of less than
// 1/2, which is less.  Two are off by 2^-21, and by 2^-23 of the sums for adding the bias.
// Softmax: exp's 2 steps, its argument's rounding (y e^y < 0.37) and the product with the
// inverse, 2^-21.6 each.  What all have in common, the sum's error, moves two by its part
// of their distance: 2 steps of exp, 5 half steps of arguments (the mean of |y| over 1024
// terms), 22 of 16 and 6 additions, 5 of the inverse, 2^-18.8.  Together 2^-18.4.
__device__ inline float apart(const RouteParams& p) { return p.sigmoid ? 0x1p-20f : 0x1p-18f; }

// A group's score from its best sums `one` and `two` (-inf where it has none).  A sum past
// the range stays a number, so that the group counts as one with experts; its group_off is
// infinite.
__device__ inline float group_score(const RouteParams& p, float one, float two) {
  if (p.group_best == 1 || two == -__builtin_inff()) return one;
  return fmaxf(one + two, -0x1.fffffep127f);
}

// How far that may be off: `one` and `two` have their own errors, which their sum, if they
// are of opposite signs, may be smaller than.  The bound rises with a sum's magnitude less
// than the sum, so it holds for whichever are the best in 64 bits.
__device__ inline float group_off(const RouteParams& p, float reach, float one, float two) {
  float size = fabsf(one);
  if (p.group_best == 2 && two != -__builtin_inff()) size += fabsf(two);
  return apart(p) * (reach + size);
}

// Without a bias a group of one best score stands by its best logit, exactly.  Whether
// scores of 64 bits tell other logits from `l`: the next one lies 2^-24 |l| away or more, and
// so, 2^-40 at least, does its exponential as a part of itself; a sigmoid's part of that is
// e^-l, 2^-43 at least.  Past these limits scores of 64 bits meet, as 1 or as 0.
__device__ inline bool logit_tells(const RouteParams& p, float l, float most) {
  return p.sigmoid ? l >= -600.0f && l <= 16.0f : l - most >= -600.0f;
}
// Nearer to 0 than 2^-16 logits other than `l` have to be at least twice that.
__device__ inline bool beside_zero(float l, float other) {
  return fabsf(l) < 0x1p-16f && other != l && fabsf(other) < 0x1p-15f;
}

// Whether a slot's score s, of exp(y), may lose places to FP32's smallest numbers, which the
// sum over the slots or the scale can bring back; past -800 it is 0 in 64 bits too.
__device__ inline bool too_small(float y, float s) { return !(s > 0x1p-100f) && y >= -800.0f; }

// choose_grouped in FP32, as far as that can tell the experts and groups apart; false,
// and nothing written, when it cannot (256 tokens of 256 experts: 13 us, 16 with
// every one by 64 bits; 4096 tokens 22 and 41).
template <int PER>
__device__ inline bool choose_near(const RouteParams& p, int t, const float (&v)[PER],
                                   const Groups<PER, 64>& groups, const float* bias,
                                   int32_t* ids, float* scratch) {
  const int lane = threadIdx.x & 63;
  const float none = -__builtin_inff();
  auto in_order = [] {  // a wave's LDS accesses are done in order: keep theirs
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  float c[PER], most = 0.0f, total = 1.0f, reach = 1.0f;
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float x = exp_of(-fabsf(v[i]));
      c[i] = (v[i] > 0.0f ? 1.0f : x) * __builtin_amdgcn_rcpf(1.0f + x);
    }
  } else {
    most = v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) most = fmaxf(most, v[i]);
    most = wave_fmax(most);
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = v[i] == none ? 0.0f : exp_of(v[i] - most);
      total += c[i];
    }
    total = wave_sum(total);
    reach = 1.0f / total;
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] *= reach;
  }
  bool odd = false;  // NaN or infinities to compare
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] += bias[lane * PER + i];
    if (v[i] == none) c[i] = none;
    odd = odd || !(c[i] <= 0x1p126f);
  }
  if (__ballot(odd)) return false;

  uint64_t allowed = ~0ull;
  if (p.groups > 1) {
    // Without a bias the best scores are those of the best logits.
    const bool by_logit = !p.bias && p.group_best == 1;
    // Every lane of a block of `span` lanes gets its group's score.
    int span = groups.span, group = groups.first;
    float one = none, two = none;
    auto add = [&](float x) {  // the middle one of three is the second of all
      two = __builtin_amdgcn_fmed3f(one, two, x);
      one = fmaxf(one, x);
    };
    if (span) {
#pragma unroll
      for (int i = 0; i < PER; ++i) add(by_logit ? v[i] : c[i]);
    } else {  // by way of LDS: the lanes share out among as many groups as there can be
      span = 64;
      while (span * p.groups > 64) span >>= 1;
      group = lane / span;
      in_order();
#pragma unroll
      for (int i = 0; i < PER; ++i) scratch[lane * PER + i] = by_logit ? v[i] : c[i];
      in_order();
      if (group < p.groups)
        for (int i = lane & (span - 1); i < groups.size; i += span)
          add(scratch[group * groups.size + i]);
    }
    join_best<1>(one, two, span);
    const bool mine = group < p.groups;
    float score = group_score(p, one, two);
    if (!mine) score = none;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const float s =
          __int_as_float(__builtin_amdgcn_readlane(__float_as_int(score), g * span));
      rank += s > score || (s == score && g < group);
    }
    const bool is = mine && score != none;
    if (by_logit) {
      const uint64_t last = __ballot(is && rank == p.top_groups - 1);
      if (last && __ballot(is && rank == p.top_groups)) {
        const float l = __int_as_float(__builtin_amdgcn_readlane(
            __float_as_int(score), __ffsll((unsigned long long)last) - 1));
        if (!logit_tells(p, l, most) || __ballot(is && beside_zero(l, score))) return false;
      }
    } else {  // the least that one taken can be, and the most that another can
      const float off = group_off(p, reach, one, two);
      const float least = -wave_fmax(is && rank < p.top_groups ? off - score : none);
      const float other = wave_fmax(is && rank >= p.top_groups ? score + off : none);
      if (!(least > other)) return false;
    }
    const uint64_t lanes = __ballot(is && rank < p.top_groups);
    if (groups.span) {
      allowed = lanes >> lane & 1 ? ~0ull : 0;  // a lane is in one group
    } else {
      allowed = 0;
      for (int g = 0; g < p.groups; ++g) allowed |= (lanes >> (g * span) & 1) << g;
    }
  }
  float by[PER];
  uint64_t number = groups.number;
  asm volatile("" : "+v"(number));  // not PER numbers kept over the tokens
  allowed >>= groups.span || p.groups == 1 ? 0 : groups.first & 63;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool ok = allowed >> (number >> (4 * i) & 15) & 1;
    by[i] = ok && c[i] != none ? (p.bias ? c[i] : v[i]) : none;
  }
  if (p.bias) {  // the slots' logits are looked up there: of their keys only the sums are known
    in_order();
#pragma unroll
    for (int i = 0; i < PER; ++i) scratch[lane * PER + i] = v[i];
    in_order();
  }
  int mine;
  uint32_t mine_key;
  uint32_t rest = take_largest<PER>(by, p.k, mine, mine_key);
  const int n = __popcll(__ballot(mine >= 0));
  float l = of_key(mine_key);  // the slot's logit
  if (p.bias) {
    const float sum = l;
    if (mine >= 0) l = scratch[mine];
    // Each slot's sum against the next one's, the last one's against what is left.
    rest = wave_max(rest);
    uint32_t below = uint32_t(__builtin_amdgcn_update_dpp(0, int(mine_key), 0x101, 0xf, 0xf, true));
    if (lane == n - 1) below = rest;
    const bool near = lane < n && below > kNoKey &&
                      !(sum - of_key(below) > apart(p) * (reach + fabsf(sum)));
    if (__ballot(near)) {
      // Of the same logit and bias: a tie in any number of bits.
      const int e = __builtin_amdgcn_update_dpp(-1, mine, 0x101, 0xf, 0xf, false);
      bool same = false;
      if (near && lane < n - 1 && e >= 0)
        same = scratch[e] == l && p.bias[e] == p.bias[mine];
      if (__ballot(near && !same)) return false;
    }
  }
  float s = 0.0f;
  bool small = false;
  if (mine >= 0) {
    const float y = p.sigmoid ? -fabsf(l) : l - most, x = exp_of(y);
    s = !p.sigmoid ? x : (l > 0.0f ? 1.0f : x) / (1.0f + x);
    small = too_small(y, s);
  }
  if (p.renorm) {
    total = wave_sum(s);
    small = small || (n && !(total > 0.0f));
  }
  if (__ballot(small)) return false;
  if (lane < p.k) {
    const int64_t slot = int64_t(t) * p.k + lane;
    p.experts[slot] = mine;
    p.weights[slot] = mine >= 0 ? p.scale * (s / total) : 0.0f;
    ids[lane] = mine;
  }
  return true;
}

// ---- four tokens by a wave, 16 lanes (a row of lane moves) to each

// f over each row of 16, in all of its lanes.
template <class F>
__device__ inline float row_all(float v, F f) {
  v = f(v, other_lanes<1>(v));
  v = f(v, other_lanes<2>(v));
  v = f(v, other_lanes<4>(v));
  return f(v, other_lanes<8>(v));
}
__device__ inline float row_fmax(float v) {
  return row_all(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float row_sum(float v) {
  return row_all(v, [](float a, float b) { return a + b; });
}
__device__ inline uint32_t row_max(uint32_t v) {
  const auto f = [](float a, float b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    return __uint_as_float(x > y ? x : y);
  };
  return __float_as_uint(row_all(__uint_as_float(v), f));
}
// The bits of a row's lanes.
__device__ inline uint32_t row_ballot(bool v) {
  const uint64_t all = __ballot(v);
  const uint32_t half = threadIdx.x & 32 ? uint32_t(all >> 32) : uint32_t(all);
  return half >> (threadIdx.x & 16) & 0xffff;
}

// f(a, b) for the pairs of a sorting network of N places (a power of two), by merging
// sorted halves of even and odd places.
template <int N, class F>
__device__ inline void sorting_network(F f) {
#pragma unroll
  for (int len = 1; len < N; len *= 2)
#pragma unroll
    for (int d = len; d > 0; d /= 2)
#pragma unroll
      for (int j = d % len; j + d < N; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d && i + j + d < N; ++i)
          if ((i + j) / (2 * len) == (i + j + d) / (2 * len)) f(i + j, i + j + d);
}

// choose_near for a token in each row: 400 vector instructions per token of 256 experts
// for the wave's 700 (32768 of them: 66 -> 39 us), the reductions being four moves for
// four tokens.  `ids` and `scratch` are the row's.  False in the lanes of a row whose
// token has to go by 64 bits.
template <int PER>
__device__ inline bool choose_rows(const RouteParams& p, int64_t t, bool there,
                                   const float (&v)[PER], const Groups<PER, 16>& groups,
                                   const float* bias, int32_t* ids, float* scratch) {
  const int q = threadIdx.x & 15;
  const float none = -__builtin_inff();
  auto in_order = [] {  // a wave's LDS accesses are done in order: keep theirs
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  float c[PER], most = 0.0f, total = 1.0f, reach = 1.0f;
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float x = exp_of(-fabsf(v[i]));
      c[i] = (v[i] > 0.0f ? 1.0f : x) * __builtin_amdgcn_rcpf(1.0f + x);
    }
  } else {
    most = v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) most = fmaxf(most, v[i]);
    most = row_fmax(most);
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = v[i] == none ? 0.0f : exp_of(v[i] - most);
      total += c[i];
    }
    total = row_sum(total);
    reach = 1.0f / total;
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] *= reach;
  }
  bool slow = false;  // NaN or infinities to compare, or values too near each other
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] += bias[q * PER + i];
    if (v[i] == none) c[i] = none;
    slow = slow || !(c[i] <= 0x1p126f);
  }

  uint32_t allowed = 0xffff;  // by lanes: a group's are its `span` from group * span on
  int span = groups.span;
  if (p.groups > 1) {
    const bool by_logit = !p.bias && p.group_best == 1;
    int group = groups.first;
    float one = none, two = none;
    auto add = [&](float x) {  // the middle one of three is the second of all
      two = __builtin_amdgcn_fmed3f(one, two, x);
      one = fmaxf(one, x);
    };
    if (span) {
#pragma unroll
      for (int i = 0; i < PER; ++i) add(by_logit ? v[i] : c[i]);
    } else {
      span = 16;
      while (span * p.groups > 16) span >>= 1;
      group = q / span;
      in_order();
#pragma unroll
      for (int i = 0; i < PER; ++i) scratch[q * PER + i] = by_logit ? v[i] : c[i];
      in_order();
      if (group < p.groups)
        for (int i = q & (span - 1); i < groups.size; i += span)
          add(scratch[group * groups.size + i]);
    }
    join_best<1>(one, two, span);
    float score = group_score(p, one, two);
    if (group >= p.groups) score = none;
    int above = 0;  // lanes of groups before this one
    each16([&](auto n) {
      const float s = __int_as_float(__builtin_amdgcn_update_dpp(
          0, __float_as_int(score), 0x150 + decltype(n)::value, 0xf, 0xf, true));
      above += s > score || (s == score && decltype(n)::value < group * span);
    });
    const bool is = score != none, in = above < p.top_groups * span;
    if (by_logit) {
      const float l = row_fmax(is && above == (p.top_groups - 1) * span ? score : none);
      const bool more = row_ballot(is && !in) != 0;
      slow = slow || (more && (!logit_tells(p, l, most) || (is && beside_zero(l, score))));
    } else {  // the least that one taken can be, and the most that another can
      const float off = group_off(p, reach, one, two);
      const float least = -row_fmax(is && in ? off - score : none);
      const float other = row_fmax(is && !in ? score + off : none);
      slow = slow || !(least > other);
    }
    allowed = row_ballot(is && in);
  }
  // A bit for each of the lane's experts whose group is taken.
  uint32_t taken = allowed >> (groups.first * span & 15) & 1 ? 0xffff : 0;
  if (p.groups > 1 && !groups.span) {
    uint64_t number = groups.number;
    asm volatile("" : "+v"(number));  // not PER numbers kept over the tokens
    taken = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = groups.first + int(number >> (4 * i) & 15);
      taken |= (allowed >> (g * span & 15) & 1) << i;
    }
  }
  // The values' keys and, below them, places, the first of equal ones on top: as the
  // bits of positive doubles, which have a maximum and a minimum of one instruction.
  double key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float by = (taken >> i & 1) && c[i] != none ? (p.bias ? c[i] : v[i]) : none;
    key[i] = __longlong_as_double(int64_t(key_of(by)) << 30 | (PER - 1 - i));
  }
  const auto key_bits = [](double k) { return uint64_t(__double_as_longlong(k)); };
  if (p.bias) {  // the slots' logits are looked up there: of their keys only the sums are known
    in_order();
#pragma unroll
    for (int i = 0; i < PER; ++i) scratch[q * PER + i] = v[i];
    in_order();
  }
  sorting_network<PER>([&](int a, int b) {
    double hi, lo;  // in asm: the compiler would first make quiet what it takes for a NaN
    asm("v_max_f64 %0, %2, %3\n\tv_min_f64 %1, %2, %3"
        : "=&v"(hi), "=&v"(lo)
        : "v"(key[a]), "v"(key[b]));
    key[a] = hi, key[b] = lo;
  });
  // Lane j keeps slot j's key, its expert goes to ids.
  uint32_t mine_key = 0;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t top = uint32_t(key_bits(key[0]) >> 30), m = row_max(top);
    const bool some = m > kNoKey;
    if (!__ballot(some)) break;
    if (q == j && some) mine_key = m;
    const uint32_t has = row_ballot(top == m);
    if (some && (has & ((2u << q) - 1)) == 1u << q) {  // the first lane of them
      if (there) ids[j] = q * PER + PER - 1 - int(uint32_t(key_bits(key[0])) & 15);
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) key[i] = key[i + 1];
      key[PER - 1] = 0.0;
    }
  }
  const int n = __popc(row_ballot(mine_key > kNoKey));
  in_order();
  const int mine = there && q < n ? ids[q] : -1;
  float l = of_key(mine_key);  // the slot's logit
  if (p.bias) {
    const float sum = l;
    if (mine >= 0) l = scratch[mine];
    // Each slot's sum against the next one's, the last one's against what is left.
    const uint32_t rest = row_max(uint32_t(key_bits(key[0]) >> 30));
    uint32_t below = uint32_t(__builtin_amdgcn_update_dpp(0, int(mine_key), 0x101, 0xf, 0xf, true));
    if (q == n - 1) below = rest;
    const bool near = q < n && below > kNoKey &&
                      !(sum - of_key(below) > apart(p) * (reach + fabsf(sum)));
    if (__ballot(near)) {
      // Of the same logit and bias: a tie in any number of bits.
      const int e = __builtin_amdgcn_update_dpp(-1, mine, 0x101, 0xf, 0xf, false);
      bool same = false;
      if (near && q < n - 1 && e >= 0 && mine >= 0)
        same = scratch[e] == l && p.bias[e] == p.bias[mine];
      slow = slow || (near && !same);
    }
  }
  float s = 0.0f;
  if (q < n) {
    const float y = p.sigmoid ? -fabsf(l) : l - most, x = exp_of(y);
    s = !p.sigmoid ? x : (l > 0.0f ? 1.0f : x) / (1.0f + x);
    slow = slow || too_small(y, s);
  }
  if (p.renorm) {
    total = row_sum(s);
    slow = slow || (n && !(total > 0.0f));
  }
  const bool done = row_ballot(slow) == 0;
  if (there && done && q < p.k) {
    p.experts[t * p.k + q] = mine;
    p.weights[t * p.k + q] = mine >= 0 ? p.scale * (s / total) : 0.0f;
    ids[q] = mine;
  }
  return done;
}

// The bias to LDS, zeros past its end and where there is none.
__device__ inline void put_bias(const RouteParams& p, float* bias, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) bias[i] = p.bias && i < p.E ? p.bias[i] : 0.0f;
  __syncthreads();
}

// How a workgroup's waves share out its tokens t0 .. t0 + n.  ROWS: four to a wave.
template <int PER, bool GROUPED, bool ROWS>
__device__ inline void choose_all(const RouteParams& p, int t0, int n, const float* bias,
                                  int32_t* ids, float* scratch) {
  const int wave = threadIdx.x >> 6;
  const bool vec = row_pieces<PER>(p.logits, p.stride, p.E, p.dtype);
  if constexpr (ROWS) {
    const int row = threadIdx.x >> 4 & 3, e0 = (threadIdx.x & 15) * PER;
    Groups<PER, 16> groups;
    groups.init(p);
    // Registers are for more waves, not for the next tokens' logits.
    for (int first = wave * 4; first < n; first += kWaves * 4) {
      const int t = first + row;
      Row<PER> logits;  // -inf for a row without a token
      logits.load_from(e0, p.logits, int64_t(t0 + t) * p.stride, t < n ? p.E : 0, p.dtype, vec);
      const bool done = choose_rows<PER>(p, t0 + t, t < n, logits.v, groups, bias,
                                         ids + t * p.k, scratch + row * 16 * PER);
      const uint64_t left = __ballot(!done);
      for (int r = 0; r < 4; ++r)
        if (first + r < n && left >> (r * 16) & 1)
          choose_grouped<PER / 4>(p, t0 + first + r, bias, ids + (first + r) * p.k, scratch);
    }
  } else {
    Groups<GROUPED ? PER : 1, 64> groups;
    if constexpr (GROUPED) groups.init(p);
    // The next token's logits are on their way while one is chosen from.
    Row<PER> row, next;
    if (wave < n) next.load(p.logits, int64_t(t0 + wave) * p.stride, p.E, p.dtype, vec);
    for (int t = wave; t < n; t += kWaves) {
      row = next;
      if (t + kWaves < n)
        next.load(p.logits, int64_t(t0 + t + kWaves) * p.stride, p.E, p.dtype, vec);
      if constexpr (GROUPED) {
        if (!choose_near<PER>(p, t0 + t, row.v, groups, bias, ids + t * p.k, scratch))
          choose_grouped<PER>(p, t0 + t, bias, ids + t * p.k, scratch);
      } else {
        choose<PER>(p, t0 + t, row.v, ids + t * p.k);
      }
    }
  }
}

// ------------------------------------------------------------------ the slots' order

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

template <int PER, bool GROUPED, bool ROWS>
__global__ __launch_bounds__(kThreads) void route_small(const RouteParams p) {
  __shared__ int32_t ids[kRouteSmall];
  __shared__ uint16_t hist[kWaves][kMaxE];
  __shared__ int32_t run[kMaxE];
  constexpr int kScratch = GROUPED ? (ROWS ? 64 : 128) * PER : 1;
  __shared__ __attribute__((aligned(16))) float scratch[GROUPED ? kWaves : 1][kScratch];
  __shared__ __attribute__((aligned(16))) float bias[GROUPED ? (ROWS ? 16 : 64) * PER : 1];
  const int tid = threadIdx.x, wave = tid >> 6;
  if constexpr (GROUPED) put_bias(p, bias, (ROWS ? 16 : 64) * PER);
  choose_all<PER, GROUPED, ROWS>(p, 0, p.tokens, bias, ids, scratch[GROUPED ? wave : 0]);
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
template <int PER, bool GROUPED, bool ROWS>
__global__ __launch_bounds__(kThreads, ROWS ? 4 : 1) void route_choose(const RouteParams p,
                                                                       int blocks) {
  __shared__ int32_t ids[kRouteMost * 16];
  __shared__ uint16_t hist[kWaves][kMaxE];
  __shared__ int32_t run[kMaxE];
  constexpr int kScratch = GROUPED ? (ROWS ? 64 : 128) * PER : 1;
  __shared__ __attribute__((aligned(16))) float scratch[GROUPED ? kWaves : 1][kScratch];
  __shared__ __attribute__((aligned(16))) float bias[GROUPED ? (ROWS ? 16 : 64) * PER : 1];
  const int tid = threadIdx.x, wave = tid >> 6;
  if constexpr (GROUPED) put_bias(p, bias, (ROWS ? 16 : 64) * PER);
  for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int t0 = b * p.per_block;
    const int nt = p.tokens - t0 < p.per_block ? p.tokens - t0 : p.per_block;
    choose_all<PER, GROUPED, ROWS>(p, t0, nt, bias, ids, scratch[GROUPED ? wave : 0]);
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

// The gradient of the router by groups.  With u = w / scale and g the slots'
// dweights, a chosen expert's score has the gradient scale / sum of scores *
// sum_i u_i (g_j - g_i) when renormalised (equal terms cancel exactly: one expert
// alone gets 0), else scale * g_j; sigmoid's slope is s (1 - s), so that only the
// chosen logits are read.  Softmax without renormalisation reaches every logit.
// 32768 x 256, top 8, sigmoid: 13 us, 36 MB; a wave per token waits for its slots and
// then for their logits.  Those of the next tokens loaded ahead: 15 to 16.
template <int PER>
__global__ __launch_bounds__(256) void route_grouped_back(const RouteBackParams p) {
  const int lane = threadIdx.x & 63;
  const bool all = !p.sigmoid && !p.renorm;
  const bool vec = row_pieces<PER>(p.logits, p.stride, p.E, p.dtype);
  const bool vec_out = row_pieces<PER>(p.dlogits, p.E, p.E, p.dtype);
  const int64_t step = int64_t(gridDim.x) * 4;
  __shared__ __attribute__((aligned(16))) float of_expert[4][64 * PER];
  float* const mine = of_expert[threadIdx.x >> 6];
#pragma unroll
  for (int i = 0; i < PER; ++i) mine[lane * PER + i] = 0.0f;
  auto in_order = [] {  // a wave's LDS accesses are done in order: keep theirs
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  const float inverse_scale = 1.0f / p.scale;
  for (int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); t < p.tokens; t += step) {
    int e = -1;
    float w = 0.0f, g = 0.0f, l = 0.0f;
    if (lane < p.k) {
      e = p.experts[t * p.k + lane];
      if (e >= p.E) e = -1;
      if (e >= 0) {
        w = p.weights[t * p.k + lane];
        g = p.dweights[t * p.k + lane];
        if (p.sigmoid) l = load_value(p.logits, t * p.stride + e, p.dtype);
      }
    }
    Row<PER> row;
    if (all) row.load(p.logits, t * p.stride, p.E, p.dtype, vec);
    float d = p.scale * g;
    if (!all) {
      d = g;
      if (p.renorm) {
        d = 0.0f;
        for (int i = 0; i < p.k; ++i) {
          const float wi = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), i));
          const float gi = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), i));
          if (wi != 0.0f) d = fmaf(wi * inverse_scale, g - gi, d);
        }
      }
      if (p.sigmoid) {  // 1 - s, without a difference of near numbers
        const float x = exp_of(-fabsf(l));
        d *= (l > 0.0f ? x : 1.0f) / (1.0f + x);
      }
      d = w == 0.0f ? 0.0f : w * d;
    }
    in_order();
    if (e >= 0) mine[e] = d;
    in_order();
    float gr[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) gr[i] = mine[lane * PER + i];
    in_order();
    if (e >= 0) mine[e] = 0.0f;
    if (all) {
      const float mean = wave_sum(e >= 0 ? w * g : 0.0f);
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
      const float inverse = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        q[i] *= inverse;
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

template <int PER, bool GROUPED, bool ROWS>
static hipError_t launch_route_of(const RouteParams& p, hipStream_t stream) {
  if (route_is_small(p.tokens, p.E, p.k)) {
    route_small<PER, GROUPED, ROWS><<<dim3(1), dim3(kThreads), 0, stream>>>(p);
    return hipGetLastError();
  }
  const int blocks = (p.tokens + p.per_block - 1) / p.per_block;
  const int grid = blocks < 65536 ? blocks : 65536;
  route_choose<PER, GROUPED, ROWS><<<dim3(grid), dim3(kThreads), 0, stream>>>(p, blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_scan<<<dim3(p.E), dim3(64), 0, stream>>>(p, blocks);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_place<<<dim3(grid), dim3(kThreads), 0, stream>>>(p, blocks);
  return hipGetLastError();
}

// The router by groups with a wave to each token is the shorter way as long as no wave
// has two of them (to 2303 tokens where they are too many for one workgroup).  us of
// four tokens to a wave and of one, 256 experts in 8 groups: 1 token 9.3 and 7.1, 8
// tokens 9.6 and 7.9, 12 tokens 9.6 and 10.0, 48 tokens 14.5 and 24.0; in three launches
// 64 tokens 16.2 and 12.5, 1024 tokens 17.1 and 13.3, 2048 tokens 19.8 and 18.3, 4096
// tokens 22.6 and 22.4, 8192 tokens 23.8 and 29.1; 64 experts in one group, 8 tokens 6.1
// and 5.3, 2048 tokens 11.7 and 11.3, 4096 tokens 13.6 and 14.5.  (How many one workgroup
// takes is the plain router's rule, with its figures; by the ones above three launches
// would be the shorter way for 48 tokens already.)
static bool a_token_each(const RouteParams& p) {
  return p.tokens <= kWaves ||
         (!route_is_small(p.tokens, p.E, p.k) && route_per_block(p.tokens) <= kWaves);
}

hipError_t launch_route(RouteParams p, hipStream_t stream) {
  (void)hipGetLastError();
  p.per_block = route_per_block(p.tokens);
  hipError_t e = hipSuccess;
  if (!p.groups) {
    with_per(p.E, [&](auto per) {
      e = launch_route_of<decltype(per)::value, false, false>(p, stream);
    });
  } else if (p.E <= 256 && p.groups <= 16 && !a_token_each(p)) {
    // Four tokens to a wave: every wave of a block has some.
    if (p.per_block < kWaves * 4) p.per_block = kWaves * 4;
    if (p.E <= 64) e = launch_route_of<4, true, true>(p, stream);
    else if (p.E <= 128) e = launch_route_of<8, true, true>(p, stream);
    else e = launch_route_of<16, true, true>(p, stream);
  } else {
    with_per(p.E, [&](auto per) {
      e = launch_route_of<decltype(per)::value, true, false>(p, stream);
    });
  }
  return e;
}

hipError_t launch_route_back(const RouteBackParams& p, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  (void)hipGetLastError();
  const int64_t want = (int64_t(p.tokens) + 3) / 4;
  const int grid = int(want < 2048 ? want : 2048);  // 8 waves per SIMD
  with_per(p.E, [&](auto per) {
    if (p.grouped)
      route_grouped_back<decltype(per)::value><<<dim3(grid), dim3(256), 0, stream>>>(p);
    else
      route_back<decltype(per)::value><<<dim3(grid), dim3(256), 0, stream>>>(p);
  });
  return hipGetLastError();
}

}  // namespace a2av
