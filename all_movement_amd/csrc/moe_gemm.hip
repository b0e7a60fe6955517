// moe_gemm.hip -- the products grouped by expert with ragged sizes.
//
// Rows stand in expert order, counts[e] of them for expert e; with r a row of
// expert e
//   forward  y [r][n] = sum_k x[index[r]][k] W[e][n][k]
//   dx       dx[r][k] = sum_n dy[r][n] W[e][n][k]
//   dw       dW[e][n][k] = sum_r dy[r][n] x[index[r]][k]
// One tile kernel computes all three: a BM x BN tile of the output in FP32
// accumulators, 128 bytes of the reduction (64 elements of 16 bits, 256 of 4)
// per step through two LDS buffers.  An operand is "along" when the reduction
// runs along its rows (x, dy, and W in the forward product) and "across" when
// it runs over its rows (W in dx, both in dw); an across tile is read from LDS
// with the transposing read, so no operand is ever transposed in memory.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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

__device__ inline int wave_scan(int v) {  // inclusive, 64 lanes
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// Where a tile of grouped rows lies: expert e, rows [row0, row0 + m).
struct Span {
  int e;
  int m;
  int64_t row0;
};

// Row tiles of c rows; c may be 2^31 - 1.
__device__ inline int tiles_of(int c, int BM) { return c > 0 ? (c - 1) / BM + 1 : 0; }

// Checks the counts; false when one is negative or they sum to more than
// nrows.  total_tiles: row tiles of BM over all experts.  Every wave does it
// for itself, 64 counts at a time.
__device__ inline bool check_counts(const int32_t* counts, int E, int64_t nrows, int BM,
                                    int64_t* total_tiles) {
  const int lane = threadIdx.x & 63;
  int64_t rows = 0, tiles = 0;
  bool ok = true;
  for (int b = 0; b < E; b += 64) {
    const int c = b + lane < E ? counts[b + lane] : 0;
    ok = ok && __ballot(c < 0) == 0;
    // Two halves of 16 bits each keep the wave's sums inside 32 bits.
    const int lo = __shfl(wave_scan(c & 0xffff), 63), hi = __shfl(wave_scan(c >> 16), 63);
    rows += int64_t(lo) + (int64_t(hi) << 16);
    ok = ok && rows <= nrows;
    if (!ok) return false;
    tiles += __shfl(wave_scan(tiles_of(c, BM)), 63);
  }
  *total_tiles = tiles;
  return true;
}

// The row tile `t` (counts checked).
__device__ inline Span find_tile(const int32_t* counts, int E, int BM, int64_t t) {
  const int lane = threadIdx.x & 63;
  int64_t rows = 0, tiles = 0;
  for (int b = 0; b < E; b += 64) {
    const int c = b + lane < E ? counts[b + lane] : 0;
    const int n = tiles_of(c, BM);
    const int in = wave_scan(n), cs = wave_scan(c);
    const uint64_t past = __ballot(tiles + in > t);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = __shfl(in - n, l), r0 = __shfl(cs - c, l), cl = __shfl(c, l);
      const int off = int(t - tiles - first) * BM;
      Span s;
      s.e = b + l;
      s.row0 = rows + r0 + off;
      s.m = cl - off < BM ? cl - off : BM;
      return s;
    }
    tiles += __shfl(in, 63);
    rows += __shfl(cs, 63);
  }
  return Span{0, 0, 0};
}

// The rows of expert e (counts checked).
__device__ inline Span find_expert(const int32_t* counts, int E, int e) {
  const int lane = threadIdx.x & 63;
  int64_t rows = 0;
  for (int b = 0; b < e; b += 64) {
    const int c = b + lane < e ? counts[b + lane] : 0;
    rows += __shfl(wave_scan(c), 63);
  }
  (void)E;
  return Span{e, counts[e], rows};
}

// 8 elements of 16 bits at any 2-byte address, the first n of them (0..8).
__device__ inline int4v load_part(const uint8_t* p, int n) {
  struct __attribute__((packed, aligned(2))) Loose {
    int4v v;
  };
  if (n >= 8) return reinterpret_cast<const Loose*>(p)->v;
  int4v r = {0, 0, 0, 0};
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = 0;
    if (2 * i < n) w = h[2 * i];
    if (2 * i + 1 < n) w |= uint32_t(h[2 * i + 1]) << 16;
    r[i] = int(w);
  }
  return r;
}

// One operand's tile of SPAN outputs x 128 bytes of reduction, loaded by NW
// waves as 16-byte chunks.
//   along:  LDS [SPAN][8 chunks], chunk c of row r at c ^ (r & 7)
//   across: LDS [64][SPAN / 8 chunks], chunk c of row r at c ^ f(r),
//           f(r) = 2 (r & 3) + 8 (r >> 3 & 1)
// so that the reads of one fragment spread over all LDS banks.
template <bool ALONG, int SPAN, int NW, bool DIRECT>
struct Loader {
  static constexpr int kChunks = SPAN * 8;
  static constexpr int kPer = kChunks / (NW * 64);  // chunks per lane
  static_assert(kChunks % (NW * 64) == 0, "a tile is a whole number of wave loads");
  const uint8_t* ptr[kPer];
  int32_t left[kPer];   // along: elements of the row from this chunk on; across: columns from it
  int4v staged[DIRECT ? 1 : kPer];
  int wave, lane;

  __device__ static int across_swizzle(int r) { return 2 * (r & 3) | (8 & r); }
  __device__ int chunk(int i) const { return (wave * kPer + i) * 64 + lane; }
  // Where chunk i lies: row of the LDS tile and chunk in that row.
  __device__ int lds_row(int i) const { return ALONG ? chunk(i) / 8 : chunk(i) / (SPAN / 8); }
  __device__ int col(int i) const {
    const int r = lds_row(i);
    return ALONG ? (chunk(i) % 8) ^ (r & 7) : (chunk(i) % (SPAN / 8)) ^ across_swizzle(r);
  }
};

template <int TY>
__device__ inline float4v mma(int4v a, int4v b, float4v c) {
  if constexpr (TY == kGmmBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

__device__ inline float4v mma_mx4(int4v a, int4v b, float4v c, int sa, int sb, int byte) {
  const int8v x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const int8v y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  if (byte == 0)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 1, sa, 1, sb);
}

__device__ inline uint16_t round16(float v, int type) {
  if (type == A2AV_BF16) return __builtin_bit_cast(uint16_t, __bf16(v));
  return __builtin_bit_cast(uint16_t, _Float16(v));
}

// BM rows x BN columns of the output by WM x WN waves.
template <int TY, int MODE, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM* WN * 64) void gmm_kernel(const GmmParams p) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr bool kColsAlong = MODE == kGmmFwd;  // the operand of the output's columns
  constexpr bool kRowsAlong = MODE != kGmmDw;   // the operand of the output's rows
  constexpr int kStep = TY == kGmmMX4 ? 256 : 64;  // reduction elements per step
  constexpr int kPerChunk = kStep / 8;
  constexpr int kBuf = (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBuf];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, l16 = lane & 15;

  int64_t row_tiles = 0;
  if (!check_counts(p.counts, p.E, p.nrows, BM, &row_tiles)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && p.status) *p.status = A2AV_ERR_INVALID_ARGS;
    return;
  }

  // The tile of this workgroup.  Workgroups go round the 8 XCDs in turn, each
  // with an L2 of its own: every XCD takes one contiguous eighth of the tiles.
  const int64_t out_cols = MODE == kGmmFwd ? p.N : p.K;
  const int64_t col_tiles = (out_cols + BN - 1) / BN;
  const int64_t tm_all = MODE == kGmmDw ? int64_t(p.E) * ((p.N + BM - 1) / BM) : row_tiles;
  const int64_t total = tm_all * col_tiles;
  const int64_t per = (total + 7) / 8;
  const int64_t wg = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t in_xcd = wg / 8;
  const int64_t tile = (wg % 8) * per + in_xcd;
  if (in_xcd >= per || tile >= total) return;
  constexpr int kGroup = 4;  // row tiles that walk the columns together
  const int64_t grp = tile / (kGroup * col_tiles);
  const int64_t in_grp = tile - grp * kGroup * col_tiles;
  const int64_t grp_rows = tm_all - grp * kGroup < kGroup ? tm_all - grp * kGroup : kGroup;
  const int64_t tm = grp * kGroup + in_grp % grp_rows;
  const int64_t tn = in_grp / grp_rows;

  // The output block [r0, r0 + rm) x [c0, ..) and the reduction's length.
  Span s;
  int64_t out_row0;
  int rm;
  int64_t red;
  if constexpr (MODE == kGmmDw) {
    const int64_t per_e = (p.N + BM - 1) / BM;
    const int e = int(tm / per_e);
    s = find_expert(p.counts, p.E, e);
    out_row0 = (tm - e * per_e) * BM;
    rm = int(p.N - out_row0 < BM ? p.N - out_row0 : BM);
    red = s.m;
  } else {
    s = find_tile(p.counts, p.E, BM, tm);
    out_row0 = s.row0;
    rm = s.m;
    red = MODE == kGmmFwd ? p.K : p.N;
  }
  const int64_t c0 = tn * BN;
  const int cn = int(out_cols - c0 < BN ? out_cols - c0 : BN);
  const int steps = int((red + kStep - 1) / kStep);

  // ---- the loaders: where each chunk of a lane begins, without the step.
  Loader<kRowsAlong, BM, NW, DIRECT> q;
  Loader<kColsAlong, BN, NW, DIRECT> c;
  q.wave = c.wave = wave;
  q.lane = c.lane = lane;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(g_zeros);
  const int64_t e_rows = int64_t(s.e) * p.N;  // first row of the expert's weight
  bool bad_row = false;

#pragma unroll
  for (int i = 0; i < q.kPer; ++i) {
    const int r = q.lds_row(i), ch = q.col(i);
    if constexpr (kRowsAlong) {
      int64_t row = s.row0 + (r < rm ? r : rm - 1);
      bool ok = true;
      if (MODE == kGmmFwd && p.index) {
        row = p.index[row];
        ok = row >= 0 && row < p.x_rows;
        bad_row = bad_row || !ok;
      }
      q.ptr[i] = ok ? p.rows + row * p.row_stride + ch * 16 : nullptr;
      q.left[i] = int(red - ch * kPerChunk);
    } else {
      q.ptr[i] = p.rows + (s.row0 + r) * p.row_stride + (out_row0 + ch * 8) * 2;
      q.left[i] = rm - ch * 8;
    }
  }
#pragma unroll
  for (int i = 0; i < c.kPer; ++i) {
    const int r = c.lds_row(i), ch = c.col(i);
    if constexpr (kColsAlong) {
      const int64_t row = e_rows + c0 + (r < cn ? r : cn - 1);
      c.ptr[i] = p.other + row * p.other_stride + ch * 16;
      c.left[i] = int(red - ch * kPerChunk);
    } else if constexpr (MODE == kGmmDx) {
      c.ptr[i] = p.other + (e_rows + r) * p.other_stride + (c0 + ch * 8) * 2;
      c.left[i] = cn - ch * 8;
    } else {
      c.ptr[i] = p.other + (c0 + ch * 8) * 2;  // the row comes with each step
      c.left[i] = cn - ch * 8;
    }
  }

  const uint32_t lds0 = uint32_t(uintptr_t((lds_u8*)lds));

  // Loads step k into buffer k & 1 (or, not DIRECT, into registers).
  auto load_one = [&](auto& ld, auto along, int i, int k, uint32_t base, const uint8_t* ptr) {
    constexpr bool kAlong = decltype(along)::value;
    int n;  // elements of the chunk that exist
    if (kAlong) {
      n = ld.left[i] - k * kStep;
    } else {
      n = ld.lds_row(i) + k * 64 < red ? ld.left[i] : 0;
    }
    if (!ptr) n = 0;
    if constexpr (DIRECT) {
      load_to_lds(n > 0 ? ptr : zeros,
                  __builtin_amdgcn_readfirstlane(base + (wave * ld.kPer + i) * 1024));
    } else {
      ld.staged[i] = n > 0 ? load_part(ptr, n) : int4v{0, 0, 0, 0};
    }
  };
  auto issue = [&](int k) {
    const uint32_t base = lds0 + (k & 1) * kBuf;
    constexpr auto row_kind = std::integral_constant<bool, kRowsAlong>{};
    constexpr auto col_kind = std::integral_constant<bool, kColsAlong>{};
#pragma unroll
    for (int i = 0; i < q.kPer; ++i) {
      const uint8_t* ptr = q.ptr[i];
      if (ptr) ptr += kRowsAlong ? int64_t(k) * 128 : int64_t(k) * 64 * p.row_stride;
      load_one(q, row_kind, i, k, base, ptr);
    }
#pragma unroll
    for (int i = 0; i < c.kPer; ++i) {
      const uint8_t* ptr = c.ptr[i];
      if constexpr (kColsAlong) {
        ptr += int64_t(k) * 128;
      } else if constexpr (MODE == kGmmDx) {
        ptr += int64_t(k) * 64 * p.other_stride;
      } else {
        const int64_t r = int64_t(k) * 64 + c.lds_row(i);
        int64_t row = s.row0 + r;
        if (p.index && r < red) {
          row = p.index[row];
          if (row < 0 || row >= p.x_rows) {
            bad_row = true;
            row = -1;
          }
        }
        ptr = row < 0 ? nullptr : ptr + row * p.other_stride;
      }
      load_one(c, col_kind, i, k, base + BM * 128, ptr);
    }
  };
  auto put_staged = [&](int k) {
    if constexpr (!DIRECT) {
      uint8_t* b = lds + (k & 1) * kBuf;
#pragma unroll
      for (int i = 0; i < q.kPer; ++i)
        *reinterpret_cast<int4v*>(b + q.chunk(i) * 16) = q.staged[i];
#pragma unroll
      for (int i = 0; i < c.kPer; ++i)
        *reinterpret_cast<int4v*>(b + BM * 128 + c.chunk(i) * 16) = c.staged[i];
    }
  };

  float4v acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = float4v{0, 0, 0, 0};

  // Scale bytes of this lane's rows, MX4: row l16 of each fragment.
  const uint8_t* qs[TY == kGmmMX4 ? FM : 1];
  const uint8_t* cs[TY == kGmmMX4 ? FN : 1];
  if constexpr (TY == kGmmMX4) {
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      const int r = wm * TM + f * 16 + l16;
      int64_t row = s.row0 + (r < rm ? r : rm - 1);
      if (p.index) row = p.index[row];
      qs[f] = row >= 0 && row < p.x_rows ? p.row_scales + row * p.blocks : nullptr;
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      const int r = wn * TN + f * 16 + l16;
      cs[f] = p.other_scales + (e_rows + c0 + (r < cn ? r : cn - 1)) * p.blocks;
    }
  }

  // Reads fragment f (16 outputs from `first` on) of reduction part kk: along,
  // the lane's 16 bytes are one chunk; across, two transposed 4 x 16 blocks.
  auto fragment = [&](auto along, auto span, const uint8_t* tile_lds, int first, int kk) -> int4v {
    constexpr bool kAlong = decltype(along)::value;
    constexpr int kSpan = decltype(span)::value;
    if constexpr (kAlong) {
      const int r = first + l16;
      const int ch = (TY == kGmmMX4 ? g * 2 + kk : kk * 4 + g) ^ (l16 & 7);
      return *reinterpret_cast<const int4v*>(tile_lds + r * 128 + ch * 16);
    } else {
      const int r = kk * 32 + g * 8 + (l16 >> 2);
      const int ch = (first / 8 + ((l16 & 3) >> 1)) ^ (2 * (l16 >> 2) | (8 * (g & 1)));
      const uint8_t* a = tile_lds + r * (kSpan * 2) + ch * 16 + (l16 & 1) * 8;
      const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) short4v*)(a));
      const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) short4v*)(a + 4 * kSpan * 2));
      const short8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(int4v, v);
    }
  };
  auto compute = [&](int k) {
    const uint8_t* b = lds + (k & 1) * kBuf;
    constexpr auto row_kind = std::integral_constant<bool, kRowsAlong>{};
    constexpr auto col_kind = std::integral_constant<bool, kColsAlong>{};
    int sq[TY == kGmmMX4 ? FM : 1], sc[TY == kGmmMX4 ? FN : 1];
    if constexpr (TY == kGmmMX4) {
      // Blocks 2g and 2g + 1 of the step; past the row's end the codes are
      // zero and the scale has to be a number.
      const int b0 = k * 8 + g * 2;
      auto two = [&](const uint8_t* at) {
        int v = 0x7f7f;
        if (at && b0 + 1 < p.blocks) {
          v = at[b0] | at[b0 + 1] << 8;
        } else if (at && b0 < p.blocks) {
          v = at[b0] | 0x7f00;
        }
        return v;
      };
#pragma unroll
      for (int f = 0; f < FM; ++f) sq[f] = two(qs[f]);
#pragma unroll
      for (int f = 0; f < FN; ++f) sc[f] = two(cs[f]);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      int4v fc[FN], fq[FM];
#pragma unroll
      for (int f = 0; f < FN; ++f)
        fc[f] = fragment(col_kind, std::integral_constant<int, BN>{}, b + BM * 128,
                         wn * TN + f * 16, kk);
#pragma unroll
      for (int f = 0; f < FM; ++f)
        fq[f] = fragment(row_kind, std::integral_constant<int, BM>{}, b, wm * TM + f * 16, kk);
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int d = 0; d < FN; ++d) {
          if constexpr (TY == kGmmMX4)
            acc[a][d] = mma_mx4(fc[d], fq[a], acc[a][d], sc[d], sq[a], kk);
          else
            acc[a][d] = mma<TY>(fc[d], fq[a], acc[a][d]);
        }
    }
  };

  if (steps > 0) {
    issue(0);
    put_staged(0);
  }
  for (int k = 0; k < steps; ++k) {
    wait_loads_and_barrier();
    if (k + 1 < steps) issue(k + 1);
    compute(k);
    if (k + 1 < steps) put_staged(k + 1);
  }
  if (bad_row && p.status) *p.status = A2AV_ERR_INVALID_ARGS;

  // A lane holds 4 columns (4g .. 4g + 3 of a fragment) of output row l16.
  const int64_t out_first = MODE == kGmmDw ? e_rows + out_row0 : out_row0;
  const bool wide = (p.out_stride & 3) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
#pragma unroll
  for (int a = 0; a < FM; ++a) {
    const int r = wm * TM + a * 16 + l16;
    if (r >= rm) continue;
#pragma unroll
    for (int d = 0; d < FN; ++d) {
      const int col = wn * TN + d * 16 + g * 4;
      if (col >= cn) continue;
      const int64_t at = (out_first + r) * p.out_stride + c0 + col;
      const float4v v = acc[a][d];
      const bool whole = wide && col + 4 <= cn;
      if (p.out_type == A2AV_FP32) {
        float* o = reinterpret_cast<float*>(p.out) + at;
        if (whole)
          *reinterpret_cast<float4v*>(o) = v;
        else
          for (int i = 0; i < 4 && col + i < cn; ++i) o[i] = v[i];
      } else {
        uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at;
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = round16(v[i], p.out_type);
        if (whole)
          *reinterpret_cast<uint64_t*>(o) = __builtin_bit_cast(uint64_t, h);
        else
          for (int i = 0; i < 4 && col + i < cn; ++i) o[i] = h[i];
      }
    }
  }
}

template <int TY, int MODE, int BM, int BN, int WM, int WN, bool DIRECT>
hipError_t launch_tiles(const GmmParams& p, hipStream_t stream) {
  const int64_t cols = MODE == kGmmFwd ? p.N : p.K;
  const int64_t col_tiles = (cols + BN - 1) / BN;
  // The counts stay on the device: as many row tiles as they can need.
  const int64_t used = p.E < p.nrows ? p.E : p.nrows;
  const int64_t row_tiles = MODE == kGmmDw ? int64_t(p.E) * ((p.N + BM - 1) / BM)
                                           : (p.nrows + used * (BM - 1)) / BM;
  const int64_t grid = (row_tiles * col_tiles + 7) / 8 * 8;
  if (grid <= 0) return hipSuccess;
  // A launch's threads have to stay below 2^32 in x: long ones go on in y.
  const int64_t gx = grid < (1 << 20) ? grid : (1 << 20);
  const int64_t gy = (grid + gx - 1) / gx;
  if (gy > 65535) return hipErrorInvalidConfiguration;
  (void)hipGetLastError();
  gmm_kernel<TY, MODE, BM, BN, WM, WN, DIRECT>
      <<<dim3(uint32_t(gx), uint32_t(gy)), dim3(WM * WN * 64), 0, stream>>>(p);
  return hipGetLastError();
}

template <int TY, int MODE>
hipError_t launch_mode(const GmmParams& p, bool direct, hipStream_t stream) {
  if constexpr (TY == kGmmMX4) {
    (void)direct;
    return launch_tiles<TY, MODE, 128, 128, 2, 2, true>(p, stream);
  } else {
    if (direct) return launch_tiles<TY, MODE, 128, 128, 2, 2, true>(p, stream);
    return launch_tiles<TY, MODE, 128, 128, 2, 2, false>(p, stream);
  }
}

}  // namespace

hipError_t launch_gmm(const GmmParams& p, GmmType type, GmmMode mode, hipStream_t stream) {
  // The loads to LDS move aligned chunks of 16 bytes: every row has to begin
  // and end on one.
  const uintptr_t bases = reinterpret_cast<uintptr_t>(p.rows) | reinterpret_cast<uintptr_t>(p.other);
  const bool direct = ((bases | uint64_t(p.row_stride) | uint64_t(p.other_stride)) & 15) == 0 &&
                      ((p.N | p.K) & 7) == 0;
  if (type == kGmmMX4) return launch_mode<kGmmMX4, kGmmFwd>(p, true, stream);
  if (type == kGmmBF16) {
    if (mode == kGmmFwd) return launch_mode<kGmmBF16, kGmmFwd>(p, direct, stream);
    if (mode == kGmmDx) return launch_mode<kGmmBF16, kGmmDx>(p, direct, stream);
    return launch_mode<kGmmBF16, kGmmDw>(p, direct, stream);
  }
  if (mode == kGmmFwd) return launch_mode<kGmmFP16, kGmmFwd>(p, direct, stream);
  if (mode == kGmmDx) return launch_mode<kGmmFP16, kGmmDx>(p, direct, stream);
  return launch_mode<kGmmFP16, kGmmDw>(p, direct, stream);
}

}  // namespace a2av
