// moe_tiles.h -- what the kernels of the products grouped by expert share
// (moe_gemm.hip, moe_fp8.hip): how a workgroup finds its tile from the counts,
// the loads that go straight to LDS, the stores of a tile's sums, the launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>
#include <utility>

#include "a2av.h"
#include "moe.h"

namespace a2av {
namespace {

typedef short short4v __attribute__((ext_vector_type(4)));
typedef short short8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) uint16_t lds_u16;

// What a load reads in place of bytes past an operand's end.
__device__ const uint32_t g_zeros[4] = {0, 0, 0, 0};

// 16 bytes per lane from `src` to LDS at base + 16 * lane, without registers in
// between.  In asm because the compiler, which cannot tell the two LDS buffers
// apart, would wait for it before the next LDS read; the kernel waits itself.
__device__ inline void load_to_lds(const uint8_t* src, uint32_t base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(base), "v"(src)
               : "memory");
}

__device__ inline void wait_loads_and_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Inclusive sum over the wave, by lane moves inside rows of 16 and from row to
// row.
__device__ inline int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31
  return v;
}

__device__ inline int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Row tiles of c rows; c may be 2^31 - 1.
__device__ inline int tiles_of(int c, int BM) { return c > 0 ? (c - 1) / BM + 1 : 0; }

// Where a tile of grouped rows lies: expert e, rows [row0, row0 + m).
struct Span {
  int e;
  int m;
  int64_t row0;
};

// The counts of 64 experts from `b` on, one per lane, with the sums before
// them; every wave does this for itself.
struct Counts {
  int c;          // this lane's count
  int rows, tiles;  // inclusive sums over the 64
  int64_t rows_before = 0, tiles_before = 0;

  // Takes the next 64; false when one is negative or the sum passes nrows.
  __device__ bool take(const int32_t* counts, int E, int b, int BM, int64_t nrows) {
    const int lane = threadIdx.x & 63;
    c = b + lane < E ? counts[b + lane] : 0;
    if (__ballot(c < 0)) return false;
    // Two halves of 16 bits each keep the sums inside 32 bits.
    const int lo = wave_scan(c & 0xffff), hi = wave_scan(c >> 16);
    const int64_t sum = int64_t(lane_value(lo, 63)) + (int64_t(lane_value(hi, 63)) << 16);
    if (rows_before + sum > nrows) return false;
    rows = lo + (hi << 16);
    tiles = wave_scan(tiles_of(c, BM));
    return true;
  }
  __device__ void pass() {
    rows_before += lane_value(rows, 63);
    tiles_before += lane_value(tiles, 63);
  }
  __device__ Span at(int b, int lane) const {
    const int cl = lane_value(c, lane);
    return Span{b + lane, cl, rows_before + lane_value(rows, lane) - cl};
  }
};

// The block of the output that a workgroup computes: rows out_row0 .. + rm of
// the output (dw: of the expert's matrix), columns c0 .. + cn.
struct Tile {
  Span span;
  int64_t out_row0, c0;
  int rm, cn;
};

// Checks the counts and finds this workgroup's tile; false when it has none.
// Tiles stand in groups of kGroup row tiles that walk the columns together, and
// 32 in a row go to one XCD (workgroups go round the 8 XCDs in turn, each with
// 32 CUs and an L2 of its own), the next 32 to the next: an expert with many
// rows is spread over all of them.
// SPLIT, for tiles that fill a CU: what is left after whole rounds of 256 tiles,
// when it is at most half a round, is cut into quarters, so that the last round
// is not a whole tile long for a few CUs while the others have none (16384 rows
// of 16 experts, 2048 x 7168, bf16: 2.25 rounds; 550 us in whole tiles).
// *part is the quarter, -1 for a whole tile.
template <int MODE, int BM, int BN, bool SPLIT>
__device__ inline bool find_work(const GmmParams& p, Tile* t, int* part) {
  Counts k;
  bool ok = true;
  for (int b = 0; b < p.E && ok; b += 64) {
    if (b) k.pass();
    ok = k.take(p.counts, p.E, b, BM, p.nrows);
  }
  if (!ok) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && p.status)
      *p.status = A2AV_ERR_INVALID_ARGS;
    return false;
  }
  // The host refuses products of 2^31 tiles and more.
  const uint32_t row_tiles = uint32_t(k.tiles_before + lane_value(k.tiles, 63));
  const uint32_t out_cols = MODE == kGmmFwd ? p.N : p.K;
  const uint32_t col_tiles = (out_cols + BN - 1) / BN;
  const uint32_t per_e = (uint32_t(p.N) + BM - 1) / BM;  // dw: row tiles of an expert
  const uint32_t tm_all = MODE == kGmmDw ? uint32_t(p.E) * per_e : row_tiles;
  const uint32_t total = tm_all * col_tiles;
  const uint32_t wg = blockIdx.y * gridDim.x + blockIdx.x;
  const uint32_t whole = total / 256 * 256, rest = total - whole;
  const bool cut = SPLIT && rest <= 128;
  uint32_t tile;
  *part = -1;
  if (wg < whole) {
    tile = ((wg >> 8) * 8 + (wg & 7)) * 32 + (wg >> 3 & 31);
  } else {
    const uint32_t n = cut ? rest * 4 : rest, per = (n + 7) / 8;
    const uint32_t i = (wg - whole) >> 3, u = ((wg - whole) & 7) * per + i;
    if (i >= per || u >= n) return false;
    tile = whole + (cut ? u >> 2 : u);
    if (cut) *part = int(u & 3);
  }
  constexpr uint32_t kGroup = 4;
  const uint32_t grp = tile / (kGroup * col_tiles);
  const uint32_t in_grp = tile - grp * kGroup * col_tiles;
  const uint32_t grp_rows = tm_all - grp * kGroup < kGroup ? tm_all - grp * kGroup : kGroup;
  const uint32_t tn = in_grp / grp_rows;
  const uint32_t tm = grp * kGroup + (in_grp - tn * grp_rows);
  const int want = MODE == kGmmDw ? int(tm / per_e) : 0;  // dw: the tile's expert
  int b = 0;
  if (p.E > 64) {  // the counts again, as far as the tile's expert
    k = Counts{};
    k.take(p.counts, p.E, 0, BM, p.nrows);
    while (MODE == kGmmDw ? b + 64 <= want : k.tiles_before + lane_value(k.tiles, 63) <= tm) {
      k.pass();
      b += 64;
      k.take(p.counts, p.E, b, BM, p.nrows);
    }
  }
  if constexpr (MODE == kGmmDw) {
    t->span = k.at(b, want - b);
    t->out_row0 = int64_t(tm - want * per_e) * BM;
    t->rm = int(p.N - t->out_row0 < BM ? p.N - t->out_row0 : BM);
  } else {
    const uint64_t past = __ballot(k.tiles_before + k.tiles > tm);
    const int lane = __ffsll((unsigned long long)past) - 1;
    t->span = k.at(b, lane);
    const int first = lane ? lane_value(k.tiles, lane - 1) : 0;
    const int off = int(tm - k.tiles_before - first) * BM;
    t->span.row0 += off;
    t->span.m -= off;
    if (t->span.m > BM) t->span.m = BM;
    t->out_row0 = t->span.row0;
    t->rm = t->span.m;
  }
  t->c0 = int64_t(tn) * BN;
  t->cn = int(out_cols - tn * BN < BN ? out_cols - tn * BN : BN);
  if (*part >= 0) {
    const int r = (*part & 1) * (BM / 2), c = (*part >> 1) * (BN / 2);
    if (r >= t->rm || c >= t->cn) return false;
    t->out_row0 += r;
    if (MODE != kGmmDw) t->span.row0 += r;
    t->rm = t->rm - r < BM / 2 ? t->rm - r : BM / 2;
    t->c0 += c;
    t->cn = t->cn - c < BN / 2 ? t->cn - c : BN / 2;
  }
  return true;
}

__device__ inline uint16_t round16(float v, int type) {
  if (type == A2AV_BF16) return __builtin_bit_cast(uint16_t, __bf16(v));
  return __builtin_bit_cast(uint16_t, _Float16(v));
}

// A lane holds 4 columns (4g .. 4g + 3 of a fragment) of output row l16, stored
// at once at any alignment of an element.
// ready(a) is called before the sums of fragment row a are looked at.
struct Ready {
  __device__ void operator()(int) const {}
};
template <int MODE, int TM, int TN, int FM, int FN, class At = Ready>
__device__ inline void store_tile(const GmmParams& p, const Tile& t, const float4v (&acc)[FM][FN],
                                  int wm, int wn, At ready = {}) {
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int64_t first = MODE == kGmmDw ? int64_t(t.span.e) * p.N + t.out_row0 : t.out_row0;
  struct __attribute__((packed, aligned(4))) Loose32 {
    float4v v;
  };
  struct __attribute__((packed, aligned(2))) Loose16 {
    uint64_t v;
  };
#pragma unroll
  for (int a = 0; a < FM; ++a) {
    ready(a);
    const int r = wm * TM + a * 16 + l16;
    if (r >= t.rm) continue;
#pragma unroll
    for (int d = 0; d < FN; ++d) {
      const int col = wn * TN + d * 16 + g * 4;
      if (col >= t.cn) continue;
      const int64_t at = (first + r) * p.out_stride + t.c0 + col;
      const float4v v = acc[a][d];
      const bool whole = col + 4 <= t.cn;
      if (p.out_type == A2AV_FP32) {
        float* o = reinterpret_cast<float*>(p.out) + at;
        if (whole)
          reinterpret_cast<Loose32*>(o)->v = v;
        else
          for (int i = 0; i < 4 && col + i < t.cn; ++i) o[i] = v[i];
      } else {
        uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at;
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = round16(v[i], p.out_type);
        if (whole)
          reinterpret_cast<Loose16*>(o)->v = __builtin_bit_cast(uint64_t, h);
        else
          for (int i = 0; i < 4 && col + i < t.cn; ++i) o[i] = h[i];
      }
    }
  }
}

// The same through LDS (free by now, a part of it per wave): the fragments'
// pieces of 8 or 16 bytes become rows, which leave in whole lines.  Straight
// from the fragments every line of the output was written in four parts, and a
// 256 x 256 tile took 14 us to store.
// Half the sums at a time if all of them do not fit into kBytes.
template <int MODE, int TM, int TN, int FM, int FN, int ES, int kBytes>
__device__ inline void store_rows(const GmmParams& p, const Tile& t, const float4v (&acc)[FM][FN],
                                  int wm, int wn, uint8_t* lds) {
  constexpr int kRow = TN * ES, kChunks = kRow / 16;
  constexpr int kSwizzle = (kChunks < 16 ? kChunks : 16) - 1;
  constexpr int kBatch = kRow * TM <= kBytes ? FM : FM / 2;  // fragment rows at once
  static_assert(kBatch * 16 * kRow <= kBytes, "the batch fits");
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int64_t first = MODE == kGmmDw ? int64_t(t.span.e) * p.N + t.out_row0 : t.out_row0;
  const int64_t col0 = t.c0 + wn * TN;
  const int cols = t.cn - wn * TN;
  const bool wide = ((p.out_stride * ES) & 15) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
#pragma unroll
  for (int a0 = 0; a0 < FM; a0 += kBatch) {
#pragma unroll
    for (int a = 0; a < kBatch; ++a) {
      uint8_t* row = lds + (a * 16 + l16) * kRow;
#pragma unroll
      for (int d = 0; d < FN; ++d) {
        const float4v v = acc[a0 + a][d];
        if constexpr (ES == 4) {
          *reinterpret_cast<float4v*>(row + ((d * 4 + g) ^ (l16 & kSwizzle)) * 16) = v;
        } else {
          uint16_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = round16(v[i], p.out_type);
          *reinterpret_cast<uint64_t*>(row + ((d * 2 + (g >> 1)) ^ (l16 & kSwizzle)) * 16 +
                                       (g & 1) * 8) = __builtin_bit_cast(uint64_t, h);
        }
      }
    }
    constexpr int kAtOnce = 64 / kChunks;  // rows per store of the wave
    const int ch = lane % kChunks, col = ch * (16 / ES);
#pragma unroll 4
    for (int r = lane / kChunks; r < kBatch * 16; r += kAtOnce) {
      const int out_row = wm * TM + a0 * 16 + r;
      const int4v v = *reinterpret_cast<const int4v*>(lds + r * kRow + (ch ^ (r & kSwizzle)) * 16);
      if (out_row >= t.rm || col >= cols) continue;
      uint8_t* o = p.out + ((first + out_row) * p.out_stride + col0 + col) * ES;
      if (wide && col + 16 / ES <= cols) {
        *reinterpret_cast<int4v*>(o) = v;
      } else if constexpr (ES == 4) {
        for (int i = 0; i < 4 && col + i < cols; ++i) reinterpret_cast<int*>(o)[i] = v[i];
      } else {
        for (int i = 0; i < 8 && col + i < cols; ++i)
          reinterpret_cast<uint16_t*>(o)[i] = uint16_t(uint32_t(v[i / 2]) >> (16 * (i & 1)));
      }
    }
  }
}

// f(0), f(1), .., each number as a type.
template <int... I, class F>
__device__ inline void each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}

// A sum may be looked at 7 wait states after its last product at the earliest.
// The compiler keeps that distance along a straight run of code, but not across
// the branch at a loop's end (nor for products written in asm): every run of
// products ends with it.  Without it a 64 x 64 tile of one step lost the last
// register of its last sums.
__device__ inline void end_of_products() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7");
  __builtin_amdgcn_sched_barrier(0);
}

template <int N>
__device__ inline void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// load_to_lds with a uniform base and a 32-bit offset per lane.
__device__ inline void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(to), "v"(offset), "s"(base)
               : "memory");
}

// 4 bytes per lane from `src` to LDS at base + 4 * lane.
__device__ inline void load_word_to_lds(const void* src, uint32_t base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(base), "v"(src)
               : "memory");
}

template <class T>
__device__ inline const T* uniform(const T* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const T*>(uint64_t(hi) << 32 | lo);
}

// Launches `kernel` over the tiles that the counts can need: they stay on the
// device, so as many row tiles as there can be.
template <int MODE, int BM, int BN, class Kernel>
hipError_t launch_tiles(Kernel kernel, int threads, const GmmParams& p, hipStream_t stream) {
  const int64_t cols = MODE == kGmmFwd ? p.N : p.K;
  const int64_t col_tiles = (cols + BN - 1) / BN;
  const int64_t used = p.E < p.nrows ? p.E : p.nrows;
  const int64_t row_tiles = MODE == kGmmDw ? int64_t(p.E) * ((p.N + BM - 1) / BM)
                                           : (p.nrows + used * (BM - 1)) / BM;
  if (row_tiles * col_tiles <= 0) return hipSuccess;
  if (row_tiles > 0x7fff0000 / col_tiles) return hipErrorInvalidConfiguration;
  // Quarters of up to 128 tiles come on top.
  const int64_t grid = (row_tiles * col_tiles + (BM == 256 ? 3 * 128 : 0) + 7) / 8 * 8;
  // A launch's threads have to stay below 2^32 in x: long ones go on in y.
  const int64_t gx = grid < (1 << 20) ? grid : (1 << 20);
  const int64_t gy = (grid + gx - 1) / gx;
  (void)hipGetLastError();
  kernel<<<dim3(uint32_t(gx), uint32_t(gy)), dim3(uint32_t(threads)), 0, stream>>>(p);
  return hipGetLastError();
}

// Row tiles of nrows rows, about: the counts stay on the device, and most experts
// are taken to have up to a third more rows than the mean.
inline int64_t expected_row_tiles(const GmmParams& p, int BM) {
  const int64_t used = p.E < p.nrows ? p.E : p.nrows;
  const int64_t mean = (p.nrows + used - 1) / used;
  const int64_t most = p.E == 1 ? mean : mean + mean / 3;
  return used * ((most + BM - 1) / BM);
}

}  // namespace
}  // namespace a2av
