// moe_rows.hip -- the weighted return of rows to their tokens, its gradients,
// and the 4-bit format of rows.  All of it is bound by memory: each kernel
// reads and writes every row once, 16 bytes per lane where the rows' alignment
// allows it.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "a2av.h"
#include "moe.h"

namespace a2av {
namespace {

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <int DT>
struct Elem {
  using type = uint16_t;
  __device__ static float up(uint16_t h) {
    if constexpr (DT == A2AV_BF16) return __uint_as_float(uint32_t(h) << 16);
    return float(__builtin_bit_cast(_Float16, h));
  }
  __device__ static uint16_t down(float v) {
    if constexpr (DT == A2AV_BF16) return __builtin_bit_cast(uint16_t, __bf16(v));
    return __builtin_bit_cast(uint16_t, _Float16(v));
  }
};
template <>
struct Elem<A2AV_FP32> {
  using type = float;
  __device__ static float up(float v) { return v; }
  __device__ static float down(float v) { return v; }
};

// N elements as they lie in memory, 16 bytes of them where a row has as many.
// ALIGNED: at a multiple of their size; else at any element (the loads and
// stores are the same instructions, which take every address).  Kept apart from
// their values as floats, so that several are in flight before the first is
// looked at.
template <int DT, int N, bool ALIGNED>
struct __attribute__((packed, aligned(ALIGNED ? sizeof(typename Elem<DT>::type) * N
                                              : sizeof(typename Elem<DT>::type)))) Pack {
  typename Elem<DT>::type e[N];
  __device__ float operator[](int i) const { return Elem<DT>::up(e[i]); }
};

// STREAM, here and below: past the caches.  Stores: 235 MB of dequantised rows
// took 67 us and take 48.  Loads: to combine 65536 rows of 14 KiB took 255 us and
// takes 208 (5.1 TB/s).  Both, in the gradient of that: 415 and 395.
template <int DT, int N, bool ALIGNED, bool STREAM = false>
__device__ inline Pack<DT, N, ALIGNED> load_n(const typename Elem<DT>::type* p) {
  using P = Pack<DT, N, ALIGNED>;
  if constexpr (STREAM && ALIGNED && sizeof(P) == 16)
    return __builtin_bit_cast(P, __builtin_nontemporal_load(reinterpret_cast<const uint4v*>(p)));
  else
    return *reinterpret_cast<const P*>(p);
}

template <int DT, int N, bool ALIGNED, bool STREAM = false>
__device__ inline void store_n(typename Elem<DT>::type* p, const float (&v)[N]) {
  Pack<DT, N, ALIGNED> k;
#pragma unroll
  for (int i = 0; i < N; ++i) k.e[i] = Elem<DT>::down(v[i]);
  if constexpr (STREAM && ALIGNED && sizeof(k) == 16)
    __builtin_nontemporal_store(__builtin_bit_cast(uint4v, k), reinterpret_cast<uint4v*>(p));
  else
    *reinterpret_cast<Pack<DT, N, ALIGNED>*>(p) = k;
}

// Where piece i of a row begins: the last one is moved back to end with the row
// (its first elements are the one before's last).
template <int N>
__device__ inline int piece_at(int i, int width) {
  return i * N + N <= width ? i * N : width - N;
}

constexpr int kSlots = 8;  // slots whose rows are in flight together

// A token's row in pieces of N elements, one piece per lane; `across` lanes
// (a power of two, 256 at most) per token and workgroup column.  WAVE: across
// is 64 at least, so that a wave has one token and its places and weights are
// scalars.  The rows of eight slots are loaded before the first is used; an
// empty slot loads nothing then, else row 0, whose value it drops.
template <int DT, int N, bool ALIGNED, bool WAVE>
__global__ __launch_bounds__(256) void combine_kernel(const CombineParams p, int across) {
  using T = typename Elem<DT>::type;
  const int pieces = (p.width + N - 1) / N;
  const int per_wg = 256 / across;
  const int piece0 = blockIdx.y * across + (threadIdx.x & (across - 1));
  for (int64_t t0 = int64_t(blockIdx.x) * per_wg; t0 < p.tokens; t0 += int64_t(gridDim.x) * per_wg) {
    int64_t t = t0 + threadIdx.x / across;
    if (WAVE) t = t0 + __builtin_amdgcn_readfirstlane(threadIdx.x / across);
    if (t >= p.tokens) continue;
    const int32_t* place = p.place + t * p.k;
    const float* w = p.weights ? p.weights + t * p.k : nullptr;
    for (int piece = piece0; piece < pieces; piece += gridDim.y * across) {
      const int at = piece_at<N>(piece, p.width);
      float sum[N];
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] = 0.0f;
      for (int j0 = 0; j0 < p.k; j0 += kSlots) {
        Pack<DT, N, ALIGNED> v[kSlots];
        float wj[kSlots];
        bool here[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          const bool slot = j0 + j < p.k;
          const int32_t r = slot ? place[j0 + j] : -1;
          here[j] = r >= 0 && r < p.y_rows;
          if (!here[j] && r != -1 && p.status) *p.status = A2AV_ERR_INVALID_ARGS;
          wj[j] = here[j] ? (w ? w[j0 + j] : 1.0f) : 0.0f;
          if (WAVE ? here[j] : slot && p.y_rows > 0)
            v[j] = load_n<DT, N, ALIGNED, true>(static_cast<const T*>(p.y) +
                                                int64_t(here[j] ? r : 0) * p.y_stride + at);
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (here[j]) {
#pragma unroll
            for (int i = 0; i < N; ++i) sum[i] = fmaf(wj[j], v[j][i], sum[i]);
          }
      }
      store_n<DT, N, ALIGNED, true>(static_cast<T*>(p.out) + t * p.o_stride + at, sum);
    }
  }
}

// One workgroup per token: dout's row is read once for eight slots, each slot's
// row of y once, and its row of dy is written in the same pass.
template <int DT, int N, bool ALIGNED, int THREADS>
__global__ __launch_bounds__(THREADS) void combine_back_kernel(const CombineParams p) {
  using T = typename Elem<DT>::type;
  __shared__ float part[THREADS / 64][kSlots];
  const int pieces = (p.width + N - 1) / N;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
      int32_t row[kSlots];
      float w[kSlots], dot[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        row[j] = -1;
        w[j] = 1.0f;
        dot[j] = 0.0f;
        if (j0 + j < p.k) {
          const int32_t r = p.place[t * p.k + j0 + j];
          if (r >= 0 && r < p.y_rows)
            row[j] = r;
          else if (r != -1 && p.status && tid == 0)
            *p.status = A2AV_ERR_INVALID_ARGS;
          if (p.weights) w[j] = p.weights[t * p.k + j0 + j];
        }
      }
      const bool want_dots = p.dweights != nullptr;
      for (int piece = tid; piece < pieces; piece += THREADS) {
        const int at = piece_at<N>(piece, p.width);
        const auto d = load_n<DT, N, ALIGNED>(static_cast<const T*>(p.dout) + t * p.o_stride + at);
        Pack<DT, N, ALIGNED> v[kSlots];
        if (want_dots) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (row[j] >= 0)
              v[j] = load_n<DT, N, ALIGNED, true>(static_cast<const T*>(p.y) +
                                                  int64_t(row[j]) * p.y_stride + at);
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (row[j] >= 0) {
            float g[N];
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = w[j] * d[i];
            store_n<DT, N, ALIGNED, true>(static_cast<T*>(p.dy) + int64_t(row[j]) * p.dy_stride + at, g);
          }
        if (want_dots) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (row[j] >= 0) {
#pragma unroll
              for (int i = 0; i < N; ++i)
                if (ALIGNED || at + i >= piece * N) dot[j] = fmaf(d[i], v[j][i], dot[j]);
            }
        }
      }
      if (want_dots) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
#pragma unroll
          for (int s = 32; s; s >>= 1) dot[j] += __shfl_xor(dot[j], s);
          if (lane == 0) part[wave][j] = dot[j];
        }
        __syncthreads();
        if (tid < kSlots && j0 + tid < p.k) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < THREADS / 64; ++i) sum += part[i][tid];
          p.dweights[t * p.k + j0 + tid] = sum;
        }
        __syncthreads();
      }
    }
  }
}

// ------------------------------------------------------------------ 4-bit rows

// Four lanes per block of 32, 8 values each.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void quantize_kernel(const Mx4Params p) {
  using T = typename Elem<DT>::type;
  const int64_t all = int64_t(p.rows) * p.blocks * 4;
  for (int64_t q = int64_t(blockIdx.x) * 256 + threadIdx.x; q < all;
       q += int64_t(gridDim.x) * 256) {
    const int64_t block = q >> 2;
    const int64_t row = block / p.blocks;
    const int b = int(block - row * p.blocks);
    const int col = b * 32 + int(q & 3) * 8;
    const T* x = static_cast<const T*>(p.x) + row * p.stride + col;
    float v[8];
    if constexpr (WHOLE) {
      if constexpr (DT == A2AV_FP32) {
        const auto lo = load_n<DT, 4, true>(x), hi = load_n<DT, 4, true>(x + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lo[i], v[i + 4] = hi[i];
      } else {
        const auto w = load_n<DT, 8, true>(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[i];
      }
    } else if (col + 8 <= p.cols) {
      const auto w = load_n<DT, 8, false>(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = col + i < p.cols ? Elem<DT>::up(x[i]) : 0.0f;
    }
    uint32_t top = 0;  // magnitudes order like their bits
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = __float_as_uint(v[i]) & 0x7fffffffu;
      top = m > top ? m : top;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      const uint32_t u = __shfl_xor(top, d);
      top = u > top ? u : top;
    }
    // floor(log2) - 2 + 127 is the exponent field less 2; the rest follows
    // from exact products with 2^(127 - s).
    const int field = int(top >> 23);
    const int s = field == 255 ? 255 : field > 2 ? field - 2 : 0;
    uint32_t codes = 0;
    if (s != 255) {
      const float up = __uint_as_float(uint32_t(254 - s) << 23);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[0] * up, v[1] * up, 1.0f, 0);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2] * up, v[3] * up, 1.0f, 1);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[4] * up, v[5] * up, 1.0f, 2);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[6] * up, v[7] * up, 1.0f, 3);
    }
    reinterpret_cast<uint32_t*>(p.codes)[q] = codes;
    if ((q & 3) == 0) p.scales[block] = uint8_t(s);
  }
}

template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void dequantize_kernel(const Mx4Params p) {
  using T = typename Elem<DT>::type;
  const int64_t all = int64_t(p.rows) * p.blocks * 4;
  for (int64_t q = int64_t(blockIdx.x) * 256 + threadIdx.x; q < all;
       q += int64_t(gridDim.x) * 256) {
    const int64_t block = q >> 2;
    const int64_t row = block / p.blocks;
    const int b = int(block - row * p.blocks);
    const int col = b * 32 + int(q & 3) * 8;
    const uint32_t codes = reinterpret_cast<const uint32_t*>(p.codes_in)[q];
    const uint32_t s = p.scales_in[block];
    // 2^(s - 127); below the normal numbers for s = 0, NaN for s = 255.
    const float step = __uint_as_float(s == 255 ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = codes >> (4 * i) & 15;
      // Twice the magnitude as a whole number: 0 1 2 3 4 6 8 12.
      const uint32_t m = 0xc8643210u >> (4 * (c & 7)) & 15;
      v[i] = 0.5f * float(int(m)) * step;
      v[i] = c & 8 ? -v[i] : v[i];
    }
    T* x = static_cast<T*>(p.out) + row * p.stride + col;
    if constexpr (WHOLE) {
      if constexpr (DT == A2AV_FP32) {
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        store_n<DT, 4, true, true>(x, lo);
        store_n<DT, 4, true, true>(x + 4, hi);
      } else {
        store_n<DT, 8, true, true>(x, v);
      }
    } else if (col + 8 <= p.cols) {
      store_n<DT, 8, false>(x, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < p.cols) x[i] = Elem<DT>::down(v[i]);
    }
  }
}

template <class F>
hipError_t with_dtype(int dtype, F f) {
  (void)hipGetLastError();
  if (dtype == A2AV_FP32) f(std::integral_constant<int, A2AV_FP32>{});
  else if (dtype == A2AV_BF16) f(std::integral_constant<int, A2AV_BF16>{});
  else f(std::integral_constant<int, A2AV_FP16>{});
  return hipGetLastError();
}

int size_of(int dtype) { return dtype == A2AV_FP32 ? 4 : 2; }

// Whether rows of `width` elements at these addresses and strides (elements)
// are whole 16-byte pieces.
bool aligned(int dtype, int64_t width, const void* a, int64_t sa, const void* b, int64_t sb,
             const void* c, int64_t sc) {
  const int n = 16 / size_of(dtype);
  const uintptr_t at = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                       reinterpret_cast<uintptr_t>(c);
  return at % 16 == 0 && width % n == 0 && sa % n == 0 && sb % n == 0 && sc % n == 0;
}

}  // namespace

// f(pieces' length, whether they are aligned) for rows of `width` elements.
template <int DT, class F>
static void with_pieces(bool fast, int width, F f) {
  constexpr int N = DT == A2AV_FP32 ? 4 : 8;
  using One = std::integral_constant<int, 1>;
  using Many = std::integral_constant<int, N>;
  if (fast) f(Many{}, std::true_type{});
  else if (width >= N) f(Many{}, std::false_type{});
  else f(One{}, std::false_type{});
}

hipError_t launch_combine(const CombineParams& p, hipStream_t stream) {
  const bool fast = aligned(p.dtype, p.width, p.y, p.y_stride, p.out, p.o_stride, nullptr, 0);
  return with_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    with_pieces<DT>(fast, p.width, [&](auto n, auto is_aligned) {
      constexpr int N = decltype(n)::value;
      constexpr bool kAligned = decltype(is_aligned)::value;
      const int pieces = (p.width + N - 1) / N;
      // The power of two that leaves the fewest lanes without a piece.
      int across = 1;
      while (across < pieces && across < 256) across *= 2;
      const auto lanes = [&](int a) { return (pieces + a - 1) / a * a; };
      while (across > 64 && lanes(across / 2) < lanes(across)) across /= 2;
      const int64_t wgs = (int64_t(p.tokens) * across + 255) / 256;
      const int cols = (pieces + across - 1) / across;
      const dim3 grid(uint32_t(wgs < (1 << 20) ? wgs : (1 << 20)), uint32_t(cols < 64 ? cols : 64));
      if constexpr (N > 1)  // single elements: rows of fewer than 8
        if (across >= 64)
          return combine_kernel<DT, N, kAligned, true><<<grid, dim3(256), 0, stream>>>(p, across);
      combine_kernel<DT, N, kAligned, false><<<grid, dim3(256), 0, stream>>>(p, across);
    });
  });
}

hipError_t launch_combine_back(const CombineParams& p, hipStream_t stream) {
  const bool fast = aligned(p.dtype, p.width, p.y, p.y_stride, p.dout, p.o_stride, p.dy,
                            p.dy_stride);
  const dim3 grid(uint32_t(p.tokens < (1 << 20) ? p.tokens : (1 << 20)));
  return with_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    with_pieces<DT>(fast, p.width, [&](auto n, auto is_aligned) {
      constexpr int N = decltype(n)::value;
      constexpr bool kAligned = decltype(is_aligned)::value;
      if constexpr (N > 1)
        if ((p.width + N - 1) / N > 64)
          return combine_back_kernel<DT, N, kAligned, 256><<<grid, dim3(256), 0, stream>>>(p);
      combine_back_kernel<DT, N, kAligned, 64><<<grid, dim3(64), 0, stream>>>(p);
    });
  });
}

hipError_t launch_mx4_quantize(const Mx4Params& p, hipStream_t stream) {
  const int n = 16 / size_of(p.dtype);
  const bool whole = p.cols % 32 == 0 && p.stride % n == 0 &&
                     reinterpret_cast<uintptr_t>(p.x) % 16 == 0;
  const int64_t want = (int64_t(p.rows) * p.blocks * 4 + 255) / 256;
  const dim3 grid(uint32_t(want < (1 << 20) ? want : (1 << 20)));
  return with_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (whole)
      quantize_kernel<DT, true><<<grid, dim3(256), 0, stream>>>(p);
    else
      quantize_kernel<DT, false><<<grid, dim3(256), 0, stream>>>(p);
  });
}

hipError_t launch_mx4_dequantize(const Mx4Params& p, hipStream_t stream) {
  const int n = 16 / size_of(p.dtype);
  const bool whole = p.cols % 32 == 0 && p.stride % n == 0 &&
                     reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  const int64_t want = (int64_t(p.rows) * p.blocks * 4 + 255) / 256;
  const dim3 grid(uint32_t(want < (1 << 20) ? want : (1 << 20)));
  return with_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (whole)
      dequantize_kernel<DT, true><<<grid, dim3(256), 0, stream>>>(p);
    else
      dequantize_kernel<DT, false><<<grid, dim3(256), 0, stream>>>(p);
  });
}

}  // namespace a2av
