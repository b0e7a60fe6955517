// moe_rows.hip -- the weighted return of rows to their tokens, its gradients,
// and the 4-bit and 8-bit formats of rows and weights.  All of it is bound by memory: each kernel
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

// ------------------------------------------------------------------ 8-bit rows and weights

// The scale byte of a block from the bits of its largest magnitude: the least s
// with 448 * 2^(s - 127) at or above it.  448 is 1.75 * 2^8: a mantissa past
// 1.75, 0x600000, carries into the exponent.
__device__ inline int fp8_scale(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  const int s = int((top + 0x1fffffu) >> 23) - 8;
  return s > 0 ? s : 0;
}

// 4 codes; the products with 2^(127 - s) are exact, so that each value is
// rounded once.
__device__ inline uint32_t fp8_codes(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// 8 values of a row of `cols` from column `col` on, zeros past its end; kept as they
// lie in memory until they are looked at, so that several are in flight.
template <int DT, bool WHOLE>
struct Eight {
  using T = typename Elem<DT>::type;
  static constexpr int kN = DT == A2AV_FP32 && WHOLE ? 4 : 8;
  Pack<DT, kN, WHOLE> part[8 / kN];
  __device__ void load(const T* x, int col, int cols) {
    if (WHOLE || col + 8 <= cols) {
#pragma unroll
      for (int i = 0; i < 8 / kN; ++i) part[i] = load_n<DT, kN, WHOLE, true>(x + i * kN);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) part[i / kN].e[i % kN] = col + i < cols ? x[i] : T(0);
    }
  }
  __device__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[i / kN][i % kN];
  }
};

// The pieces of 8 values are numbered through, 16 to a block; a workgroup takes
// kPieces * 256 of them in a row, each thread every 256th.
constexpr int kPieces = 2;
struct Piece8 {
  int64_t row;
  int b, col;
  // Piece `first` + `i`, where `first` begins block b0 of row0.
  __device__ static Piece8 at(int64_t row0, int b0, int i, int blocks) {
    const uint32_t lb = uint32_t(b0) + uint32_t(i >> 4), rows = lb / uint32_t(blocks);
    const int b = int(lb - rows * uint32_t(blocks));
    return Piece8{row0 + rows, b, b * 128 + (i & 15) * 8};
  }
};

__device__ inline uint32_t top_of(const float (&v)[8]) {
  uint32_t top = 0;  // magnitudes order like their bits
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __float_as_uint(v[i]) & 0x7fffffffu;
    top = m > top ? m : top;
  }
  return top;
}

__device__ inline uint2 eight_codes(const float (&v)[8], int s) {
  if (s == 255) return uint2{0, 0};
  const float up = __uint_as_float(uint32_t(254 - s) << 23);
  return uint2{fp8_codes(v[0] * up, v[1] * up, v[2] * up, v[3] * up),
               fp8_codes(v[4] * up, v[5] * up, v[6] * up, v[7] * up)};
}

// The largest over each row of 16 lanes, in all of them, by moves inside the row.
__device__ inline uint32_t row_max(uint32_t v) {
  const auto with = [](uint32_t a, int b) { return a > uint32_t(b) ? a : uint32_t(b); };
  v = with(v, __builtin_amdgcn_update_dpp(0, int(v), 0xb1, 0xf, 0xf, true));   // its neighbour
  v = with(v, __builtin_amdgcn_update_dpp(0, int(v), 0x4e, 0xf, 0xf, true));   // the next two
  v = with(v, __builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xf, 0xf, true));  // half, mirrored
  return with(v, __builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xf, 0xf, true));
}

// Sixteen lanes per block of 128, 8 values each, two pieces of each thread on their way
// before the first is looked at (four: 2 us more).  16384 x 7168, bf16, to codes and
// back: 110 us, 6.4 TB/s.  Codes stored past the caches are 8 us faster by themselves and
// then 12 slower to read, and something always reads them next.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void fp8_rows_kernel(const Fp8Params p) {
  using T = typename Elem<DT>::type;
  const int64_t all = p.rows * p.blocks * 16;
  const int pitch = (p.blocks + 3) / 4 * 4, tid = threadIdx.x;
  constexpr int kEach = kPieces * 256;
  const int64_t step = int64_t(gridDim.x) * kEach;
  for (int64_t first = int64_t(blockIdx.x) * kEach; first < all; first += step) {
    const int64_t row0 = (first >> 4) / p.blocks;
    const int b0 = int((first >> 4) - row0 * p.blocks);
    const int left = int(all - first < kEach ? all - first : kEach);
    Eight<DT, WHOLE> x[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const Piece8 c = Piece8::at(row0, b0, u * 256 + tid, p.blocks);
      if (u * 256 + tid < left)
        x[u].load(static_cast<const T*>(p.x) + c.row * p.stride + c.col, c.col, p.cols);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = u * 256 + tid;
      if (i >= left) break;  // 16 lanes have the same block
      const Piece8 c = Piece8::at(row0, b0, i, p.blocks);
      float v[8];
      x[u].values(v);
      const int s = fp8_scale(row_max(top_of(v)));
      reinterpret_cast<uint2*>(p.codes)[first + i] = eight_codes(v, s);
      if ((i & 15) == 0) {
        uint8_t* to = p.scales + c.row * pitch;
        to[c.b] = uint8_t(s);
        if (c.b == p.blocks - 1)
          for (int k = p.blocks; k < pitch; ++k) to[k] = 0;
      }
    }
  }
}

// A workgroup per 128 x 128 block of a weight, 16 rows at a time, all of it read once
// and held in registers between its maximum and its codes.  16 x 2048 x 7168, bf16: 122
// us, 5.8 TB/s.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void fp8_weights_kernel(const Fp8Params p) {
  using T = typename Elem<DT>::type;
  __shared__ uint32_t tops[16];
  const int tid = threadIdx.x, pitch = (p.blocks + 3) / 4 * 4;
  const int tall = (p.n + 127) / 128;
  const int64_t all = p.rows / p.n * tall * p.blocks;
  for (int64_t block = blockIdx.x; block < all; block += gridDim.x) {
    const int64_t strip = block / p.blocks, e = strip / tall;
    const int b = int(block - strip * p.blocks);
    const int n0 = int(strip - e * tall) * 128;
    const int col = b * 128 + (tid & 15) * 8;
    Eight<DT, WHOLE> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = n0 + i * 16 + (tid >> 4);
      if (n < p.n)
        x[i].load(static_cast<const T*>(p.x) + (e * p.n + n) * p.stride + col, col, p.cols);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (n0 + i * 16 + (tid >> 4) >= p.n) continue;
      float v[8];
      x[i].values(v);
      const uint32_t u = top_of(v);
      top = u > top ? u : top;
    }
    top = row_max(top);
    if ((tid & 15) == 0) tops[tid >> 4] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) top = tops[i] > top ? tops[i] : top;
    __syncthreads();
    const int s = fp8_scale(top);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = n0 + i * 16 + (tid >> 4);
      if (n >= p.n) continue;
      float v[8];
      x[i].values(v);
      reinterpret_cast<uint2*>(p.codes)[(e * p.n + n) * (p.blocks * 16) + b * 16 + (tid & 15)] =
          eight_codes(v, s);
    }
    if (tid == 0) {
      uint8_t* to = p.scales + strip * pitch;
      to[b] = uint8_t(s);
      if (b == p.blocks - 1)
        for (int i = p.blocks; i < pitch; ++i) to[i] = 0;
    }
  }
}

// Rows and, with n, weights.  16384 x 7168 to bf16: 50 us, 7.1 TB/s (codes from the
// caches); 16 x 2048 x 7168: 96 us, 7.3 TB/s.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void fp8_values_kernel(const Fp8Params p) {
  using T = typename Elem<DT>::type;
  const int64_t all = p.rows * p.blocks * 16;
  const int pitch = (p.blocks + 3) / 4 * 4, tid = threadIdx.x;
  constexpr int kEach = kPieces * 256;
  const int64_t step = int64_t(gridDim.x) * kEach;
  for (int64_t first = int64_t(blockIdx.x) * kEach; first < all; first += step) {
    const int64_t row0 = (first >> 4) / p.blocks;
    const int b0 = int((first >> 4) - row0 * p.blocks);
    const int left = int(all - first < kEach ? all - first : kEach);
    uint2 codes[kPieces];
    uint32_t scales[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = u * 256 + tid;
      if (i >= left) continue;
      const Piece8 c = Piece8::at(row0, b0, i, p.blocks);
      int64_t strip = c.row;
      if (p.n) {
        const int64_t e = c.row / p.n;
        strip = e * ((p.n + 127) / 128) + (c.row - e * p.n) / 128;
      }
      codes[u] = reinterpret_cast<const uint2*>(p.codes_in)[first + i];
      scales[u] = p.scales_in[strip * pitch + c.b];
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = u * 256 + tid;
      if (i >= left) break;
      const Piece8 c = Piece8::at(row0, b0, i, p.blocks);
      const uint32_t s = scales[u];
      // 2^(s - 127); below the normal numbers for s = 0, NaN for s = 255.
      const float step = __uint_as_float(s == 255 ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const int w = int(j ? codes[u].y : codes[u].x);
        v[j] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * step;
        v[j + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * step;
        v[j + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * step;
        v[j + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * step;
      }
      T* x = static_cast<T*>(p.out) + c.row * p.stride + c.col;
      if constexpr (WHOLE && DT == A2AV_FP32) {
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        store_n<DT, 4, true, true>(x, lo);
        store_n<DT, 4, true, true>(x + 4, hi);
      } else if (WHOLE || c.col + 8 <= p.cols) {
        store_n<DT, 8, WHOLE, true>(x, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c.col + j < p.cols) x[j] = Elem<DT>::down(v[j]);
      }
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

// Whether rows of x or out are whole blocks of aligned pieces.
static bool whole_rows(const Fp8Params& p, const void* rows) {
  return p.cols % 128 == 0 && p.stride % (16 / size_of(p.dtype)) == 0 &&
         reinterpret_cast<uintptr_t>(rows) % 16 == 0;
}

hipError_t launch_fp8_quantize(const Fp8Params& p, hipStream_t stream) {
  const bool whole = whole_rows(p, p.x);
  const int64_t want = p.n ? p.rows / p.n * ((p.n + 127) / 128) * p.blocks
                           : (p.rows * p.blocks * 16 + kPieces * 256 - 1) / (kPieces * 256);
  const dim3 grid(uint32_t(want < (1 << 20) ? want : (1 << 20)));
  return with_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (p.n && whole)
      fp8_weights_kernel<DT, true><<<grid, dim3(256), 0, stream>>>(p);
    else if (p.n)
      fp8_weights_kernel<DT, false><<<grid, dim3(256), 0, stream>>>(p);
    else if (whole)
      fp8_rows_kernel<DT, true><<<grid, dim3(256), 0, stream>>>(p);
    else
      fp8_rows_kernel<DT, false><<<grid, dim3(256), 0, stream>>>(p);
  });
}

hipError_t launch_fp8_dequantize(const Fp8Params& p, hipStream_t stream) {
  const bool whole = whole_rows(p, p.out);
  const int64_t want = (p.rows * p.blocks * 16 + kPieces * 256 - 1) / (kPieces * 256);
  const dim3 grid(uint32_t(want < (1 << 20) ? want : (1 << 20)));
  return with_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (whole)
      fp8_values_kernel<DT, true><<<grid, dim3(256), 0, stream>>>(p);
    else
      fp8_values_kernel<DT, false><<<grid, dim3(256), 0, stream>>>(p);
  });
}

}  // namespace a2av
