// moe_gemm.hip -- the products grouped by expert with ragged sizes.
//
// Rows stand in expert order, counts[e] of them for expert e; with r a row of
// expert e
//   forward  y [r][n] = sum_k x[index[r]][k] W[e][n][k]
//   dx       dx[r][k] = sum_n dy[r][n] W[e][n][k]
//   dw       dW[e][n][k] = sum_r dy[r][n] x[index[r]][k]
// Each kernel sums in FP32:
//   gmm_large, gmm_small  256 x 256 and 128 x 128 tiles of the output, 128 bytes of
//       the reduction (64 elements of 16 bits, 256 of 4) per stage, brought straight
//       to LDS: rows whose pieces of 16 bytes are aligned
//   gmm_kernel  64 x 64 and 128 x 128 tiles with loads by way of registers: every
//       alignment and stride; in 4 bits straight to LDS, for any number of blocks
//   gmm_few  few rows per expert, forward: W streams into registers
// An operand is "along" when the reduction runs along its rows (x, dy, and W in
// the forward product) and "across" when it runs over its rows (W in dx, both in
// dw); a tile kernel reads an across tile from LDS with the transposing read, so
// no operand is ever transposed in memory.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>
#include <utility>

#include "a2av.h"
#include "moe.h"
#include "moe_tiles.h"

namespace a2av {
namespace {

// 8 elements of 16 bits at any 2-byte address, the first n of them (0..8).
__device__ inline int4v load_part(const uint8_t* p, int n) {
  struct __attribute__((packed, aligned(2))) Loose {
    int4v v;
  };
  // As global memory: where the compiler cannot see that, it counts the load
  // as one of LDS too, and any wait is then for all of them.
  if (n >= 8)
    return reinterpret_cast<const __attribute__((address_space(1))) Loose*>(uintptr_t(p))->v;
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

// The last n (1..7) elements of 8, moved to the front, with zeros after them.
__device__ inline int4v last_part(int4v v, int n) {
  const uint64_t lo = uint32_t(v[0]) | uint64_t(uint32_t(v[1])) << 32;
  const uint64_t hi = uint32_t(v[2]) | uint64_t(uint32_t(v[3])) << 32;
  const int drop = 16 * (8 - n);  // bits, 16..112
  const uint64_t a = drop < 64 ? lo >> drop | hi << (64 - drop) : hi >> (drop - 64);
  const uint64_t b = drop < 64 ? hi >> drop : 0;
  return int4v{int(uint32_t(a)), int(a >> 32), int(uint32_t(b)), int(b >> 32)};
}

// Chunk c of row r of an across tile lies at c ^ across_swizzle(r), so that the
// transposing read, 4 rows x 32 bytes by 16 lanes, meets every bank once.
template <int SPAN>
__device__ inline int across_swizzle(int r) {
  return (2 * (r & 3) | (8 & r)) & (SPAN / 8 - 1);
}

// One operand's tile of SPAN outputs x 128 bytes of reduction, loaded by NW
// waves as 16-byte chunks.
//   along:  LDS [SPAN][8 chunks], chunk c of row r at c ^ (r & 7)
//   across: LDS [64][SPAN / 8 chunks], chunk c of row r at c ^ f(r),
//           f(r) = 2 (r & 3) + 8 (r >> 3 & 1)
// so that the reads of one fragment spread over all LDS banks.
// AHEAD: the steps on their way in registers; 0: loads go straight to LDS.
template <bool ALONG, int SPAN, int NW, int AHEAD>
struct Loader {
  static constexpr int kChunks = SPAN * 8;
  static constexpr int kPer = kChunks / (NW * 64);  // chunks per lane
  static_assert(kChunks % (NW * 64) == 0, "a tile is a whole number of wave loads");
  const uint8_t* ptr[kPer];
  int32_t left[kPer];   // along: elements of the row from this chunk on; across: columns from it
  int4v staged[AHEAD ? AHEAD : 1][AHEAD ? kPer : 1];  // by the step's number % AHEAD
  int wave, lane;

  __device__ int chunk(int i) const { return (wave * kPer + i) * 64 + lane; }
  // Where chunk i lies: row of the LDS tile and chunk in that row.
  __device__ int lds_row(int i) const { return ALONG ? chunk(i) / 8 : chunk(i) / (SPAN / 8); }
  __device__ int col(int i) const {
    const int r = lds_row(i);
    return ALONG ? (chunk(i) % 8) ^ (r & 7) : (chunk(i) % (SPAN / 8)) ^ across_swizzle<SPAN>(r);
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

// BM rows x BN columns of the output by WM x WN waves.
template <int TY, int MODE, int BM, int BN, int WM, int WN, bool DIRECT, bool SHORT = false>
__global__ __launch_bounds__(WM* WN * 64) void gmm_kernel(const GmmParams p) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr bool kColsAlong = MODE == kGmmFwd;  // the operand of the output's columns
  constexpr bool kRowsAlong = MODE != kGmmDw;   // the operand of the output's rows
  constexpr int kStep = TY == kGmmMX4 ? 256 : 64;  // reduction elements per step
  constexpr int kPerChunk = kStep / 8;
  // Loads run kAhead steps ahead: straight to LDS into the other buffer, or by
  // way of registers, which the step before puts into LDS.  Four steps ahead were
  // no faster (dx 14.3 us for 13.8 at the sizes below) and cost waves.
  constexpr int kAhead = DIRECT ? 1 : 2;
  constexpr bool kSkip = MODE == kGmmDw && BM == 64;  // no loads of rows that are not there
  constexpr int kBuf = (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBuf];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, l16 = lane & 15;

  Tile t;
  int part;
  if (!find_work<MODE, BM, BN, false>(p, &t, &part)) return;
  const Span s = t.span;
  const int64_t out_row0 = t.out_row0, c0 = t.c0;
  const int rm = t.rm, cn = t.cn;
  const int64_t red = MODE == kGmmDw ? s.m : MODE == kGmmFwd ? p.K : p.N;
  const int steps = int((red + kStep - 1) / kStep);

  // ---- the loaders: where each chunk of a lane begins, without the step.
  Loader<kRowsAlong, BM, NW, DIRECT ? 0 : kAhead> q;
  Loader<kColsAlong, BN, NW, DIRECT ? 0 : kAhead> c;
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

  // Not DIRECT: the chunk that a row ends in is loaded as the row's last 8
  // elements and moved into place on its way to LDS, so that no step waits for
  // it where it is loaded (1539 rows of 7 experts, 1001 x 523: dx 28 us when its
  // elements were joined there, 19 so).  Rows shorter than 8 (SHORT) are
  // loaded by element.
  if constexpr (!DIRECT && !SHORT) {
    // Across, it is the same chunk in every step.
#pragma unroll
    for (int i = 0; i < q.kPer; ++i)
      if (!kRowsAlong && q.left[i] > 0 && q.left[i] < 8)
        q.ptr[i] -= 2 * (8 - q.left[i]);
#pragma unroll
    for (int i = 0; i < c.kPer; ++i)
      if (!kColsAlong && c.left[i] > 0 && c.left[i] < 8)
        c.ptr[i] -= 2 * (8 - c.left[i]);
  }
  // Loads step k into buffer k & 1 (or, not DIRECT, into registers).
  auto load_one = [&](auto& ld, auto along, int i, int k, auto set, uint32_t base,
                      const uint8_t* ptr) {
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
      // Without a branch: across one, the compiler waits for all loads at once
      // (1539 rows of 7 experts, 1001 x 523: dx 18.1 -> 13.6 us, with the loop
      // below).  dw's small tiles have reductions of few steps, and rows that
      // are not there are better skipped (15.8 -> 12.7; large ones 44.5 -> 48).
      int4v v = {0, 0, 0, 0};
      if constexpr (SHORT) {
        if (n > 0) v = load_part(ptr, n);
      } else if constexpr (kSkip) {
        if (n > 0) v = load_part(ptr, 8);
      } else {
        if (kAlong && n < 8) ptr -= 2 * (8 - n);
        v = load_part(n > 0 ? ptr : zeros, 8);
      }
      ld.staged[decltype(set)::value][i] = v;
    }
  };
  // dw: the rows of x of the next step to issue, read a step ahead so that
  // their latency passes under a step's products; -1 reads zeros.
  int next_row[MODE == kGmmDw ? c.kPer : 1];
  auto read_rows = [&](int k) {
    if constexpr (MODE == kGmmDw) {
#pragma unroll
      for (int i = 0; i < c.kPer; ++i) {
        const int r = k * 64 + c.lds_row(i);
        int row = -1;
        if (r < red) {
          row = int(s.row0 + r);
          if (p.index) row = p.index[row];
        }
        next_row[i] = row;
      }
    }
  };
  auto check_rows = [&](int k) {
    if constexpr (MODE == kGmmDw) {
#pragma unroll
      for (int i = 0; i < c.kPer; ++i) {
        const int row = next_row[i];
        if (row < 0 || row >= p.x_rows) {
          bad_row = bad_row || k * 64 + c.lds_row(i) < red;
          next_row[i] = -1;
        }
      }
    }
  };
  auto issue = [&](int k, auto set) {
    check_rows(k);
    const uint32_t base = lds0 + (k & 1) * kBuf;
    constexpr auto row_kind = std::integral_constant<bool, kRowsAlong>{};
    constexpr auto col_kind = std::integral_constant<bool, kColsAlong>{};
#pragma unroll
    for (int i = 0; i < q.kPer; ++i) {
      const uint8_t* ptr = q.ptr[i];
      if (ptr) ptr += kRowsAlong ? int64_t(k) * 128 : int64_t(k) * 64 * p.row_stride;
      load_one(q, row_kind, i, k, set, base, ptr);
    }
#pragma unroll
    for (int i = 0; i < c.kPer; ++i) {
      const uint8_t* ptr = c.ptr[i];
      if constexpr (kColsAlong) {
        ptr += int64_t(k) * 128;
      } else if constexpr (MODE == kGmmDx) {
        ptr += int64_t(k) * 64 * p.other_stride;
      } else {
        const int row = next_row[i];
        ptr = row < 0 ? nullptr : ptr + int64_t(row) * p.other_stride;
      }
      load_one(c, col_kind, i, k, set, base + BM * 128, ptr);
    }
  };
  auto put_staged = [&](int k, auto set) {
    if constexpr (!DIRECT) {
      constexpr int kSet = decltype(set)::value;
      uint8_t* b = lds + (kSet & 1) * kBuf;
      auto placed = [&](const auto& ld, auto along, int i) {
        int4v v = ld.staged[kSet][i];
        const int n = ld.left[i] - (decltype(along)::value ? k * kStep : 0);
        if (!SHORT && n > 0 && n < 8) v = last_part(v, n);
        return v;
      };
#pragma unroll
      for (int i = 0; i < q.kPer; ++i)
        *reinterpret_cast<int4v*>(b + q.chunk(i) * 16) =
            placed(q, std::integral_constant<bool, kRowsAlong>{}, i);
#pragma unroll
      for (int i = 0; i < c.kPer; ++i)
        *reinterpret_cast<int4v*>(b + BM * 128 + c.chunk(i) * 16) =
            placed(c, std::integral_constant<bool, kColsAlong>{}, i);
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
      const int ch = (first / 8 + ((l16 & 3) >> 1)) ^ across_swizzle<kSpan>(r);
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
    end_of_products();
  };

  using Sets = std::make_integer_sequence<int, kAhead>;
  if (steps > 0) {
    read_rows(0);
    each(Sets{}, [&](auto set) {
      constexpr int k = decltype(set)::value;
      if (k < steps) {
        issue(k, set);
        read_rows(k + 1);
      }
    });
    put_staged(0, std::integral_constant<int, 0>{});
  }
  // k % kAhead is `set`; `inner`: kAhead more steps follow.
  auto step = [&](int k, auto set, auto inner) {
    if constexpr (DIRECT) {
      wait_loads_and_barrier();
    } else {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    if (decltype(inner)::value || k + kAhead < steps) {
      issue(k + kAhead, set);
      read_rows(k + kAhead + 1);
    }
    compute(k);
    if (decltype(inner)::value || k + 1 < steps)
      put_staged(k + 1, std::integral_constant<int, (decltype(set)::value + 1) % kAhead>{});
  };
  // Without conditions a wait for a step's loads leaves those of later ones on
  // their way.
  int k = 0;
  for (; !kSkip && k + 2 * kAhead <= steps; k += kAhead)
    each(Sets{}, [&](auto set) { step(k + decltype(set)::value, set, std::true_type{}); });
  for (; k < steps; k += kAhead)
    each(Sets{}, [&](auto set) {
      if (k + decltype(set)::value < steps)
        step(k + decltype(set)::value, set, std::false_type{});
    });
  if (bad_row && p.status) *p.status = A2AV_ERR_INVALID_ARGS;

  store_tile<MODE, TM, TN, FM, FN>(p, t, acc, wm, wn);
}

// ------------------------------------------------------------------ the pipelined tile kernel

// One operand's 128 bytes x SPAN outputs of a stage in LDS, brought by wave
// loads of 64 chunks of 16 bytes.
//   along:  [SPAN][8 chunks], chunk c of row r at c ^ (r & 7): the 8 lanes that
//           read 128 bytes together, one chunk of 8 rows, meet every bank once.
//   across: 64 rows of SPAN / 8 chunks in units of one wave load (2 rows of 256
//           outputs or 4 of 128) whose rows alternate every 32 bytes: the
//           transposing read takes 32 bytes of 4 rows by 16 lanes, which are
//           128 bytes in a row for SPAN 128, and for 256 two runs of 64 that
//           the units' pitch of 1024 + 64 bytes puts into other banks.
template <bool ALONG, int SPAN>
struct Layout {
  static constexpr int kRows = ALONG ? 8 : 512 / SPAN;  // LDS rows of a wave load
  static constexpr int kPitch = !ALONG && SPAN == 256 ? 1024 + 64 : 1024;
  static constexpr int kLoads = SPAN / 8;
  static constexpr int kBytes = kLoads * kPitch;
  static_assert(ALONG || SPAN == 256 || SPAN == 128, "rows of a unit");
  // Row (of the wave load) and chunk that lane l brings.
  __device__ static int row(int l) { return ALONG ? l >> 3 : l >> 1 & (kRows - 1); }
  __device__ static int chunk(int l) {
    if (ALONG) return (l ^ l >> 3) & 7;
    return l / (2 * kRows) * 2 + (l & 1);
  }
  // Where a lane reads its part of the fragment of outputs 0 .. 15 in half kk
  // of the stage; those of fragment f lie f * kFragment further.
  static constexpr int kFragment = ALONG ? 2048 : kRows * 32;
  // PAIRS: a lane takes chunks 2g and 2g + 1 in the two halves (any share of
  // the chunks is right that both operands follow), so that the two scale
  // bytes that go with them lie side by side.
  template <bool PAIRS>
  __device__ static uint32_t read_at(int lane, int kk) {
    const int g = lane >> 4, l = lane & 15;
    if (ALONG) return uint32_t(l * 128 + ((PAIRS ? 2 * g + kk : kk * 4 + g) ^ (l & 7)) * 16);
    const int r = kk * 32 + g * 8 + (l >> 2);
    return uint32_t(r / kRows * kPitch + (r % kRows) * 32 + (l & 3) * 8);
  }
  __device__ static int4v read(uint32_t at) {
    if constexpr (ALONG) {
      return *(const __attribute__((address_space(3))) int4v*)(uintptr_t(at));
    } else {
      typedef __attribute__((address_space(3))) short4v lds_short4;
      const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)(uintptr_t(at)));
      const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_short4*)(uintptr_t(at)) + 4 / kRows * kPitch / 8);
      return __builtin_bit_cast(
          int4v, short8v(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)));
    }
  }
};

// acc += a b with the sums in the accumulation registers, or with VECTOR in the
// vector registers.
#define A2AV_MMA(op, tail, ...)                                                        \
  if constexpr (VECTOR)                                                                \
    asm("v_mfma_" op " %0, %1, %2, %0" tail : "+v"(acc) : "v"(a), "v"(b) __VA_ARGS__); \
  else                                                                                 \
    asm("v_mfma_" op " %0, %1, %2, %0" tail : "+a"(acc) : "v"(a), "v"(b) __VA_ARGS__)
template <int TY, int BYTE, bool VECTOR>
__device__ inline void mma_acc(float4v& acc, int4v a, int4v b, int sa, int sb) {
  if constexpr (TY == kGmmBF16) {
    A2AV_MMA("f32_16x16x32_bf16", "");
  } else if constexpr (TY == kGmmFP16) {
    A2AV_MMA("f32_16x16x32_f16", "");
  } else if constexpr (BYTE == 0) {
    A2AV_MMA("scale_f32_16x16x128_f8f6f4", ", %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4", , "v"(sa),
             "v"(sb));
  } else {
    A2AV_MMA("scale_f32_16x16x128_f8f6f4",
             ", %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4", , "v"(sa), "v"(sb));
  }
}
#undef A2AV_MMA

// BM x BN of the output by WM x WN waves, one per SIMD, 128 bytes of the
// reduction (64 elements of 16 bits, 256 of 4) per stage, through NB LDS
// buffers.  A stage has two halves of 64 bytes.  While a wave multiplies the
// fragments of one half it reads those of the next into other registers.  Once
// the second half's are read stands the stage's one barrier: past it nobody
// reads the stage's buffer again, and the loads of stage s + NB go there; before
// it everybody waits for his loads of stage s + 1.
// Loads past the last stage read zeros.  Every row of every operand begins and
// ends on a 16-byte chunk, and the rows that a tile reads lie within 4 GiB of
// its first.
template <int TY, int MODE, int BM, int BN, int NB>
struct PipeShape {
  static constexpr int WM = 2, WN = 2, NW = WM * WN;
  using Q = Layout<MODE != kGmmDw, BM>;   // the operand of the output's rows
  using C = Layout<MODE == kGmmFwd, BN>;  // the operand of the output's columns
  static constexpr int kBuf = Q::kBytes + C::kBytes;
  // Scales: 16 bytes (2 stages) of every row of the tile, as many sets
  // as the buffers' stages span; dw: 64
  // indexes per wave, four sets.
  static constexpr int kScaleSet = (BM + BN) * 16, kScaleSets = NB / 2 + 1;
  static constexpr int kLds =
      NB * kBuf + (TY == kGmmMX4 ? kScaleSets * kScaleSet : MODE == kGmmDw ? NW * 1024 : 0);
};

template <int TY, int MODE, int BM, int BN, int NB>
__device__ inline void gmm_tile(const GmmParams& p, const Tile& t, uint8_t* lds) {
  using Shape = PipeShape<TY, MODE, BM, BN, NB>;
  constexpr int WM = Shape::WM, WN = Shape::WN, NW = Shape::NW;
  constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr bool kColsAlong = MODE == kGmmFwd;
  constexpr bool kRowsAlong = MODE != kGmmDw;
  using Q = typename Shape::Q;
  using C = typename Shape::C;
  constexpr int kStage = TY == kGmmMX4 ? 256 : 64;
  constexpr int kPerChunk = kStage / 8;
  constexpr int kBuf = Shape::kBuf;
  constexpr int kQ = Q::kLoads / NW, kC = C::kLoads / NW;  // loads per wave and stage
  static_assert(Q::kLoads % NW == 0 && C::kLoads % NW == 0, "whole wave loads");
  constexpr bool kGather = MODE == kGmmDw;
  constexpr bool kScales = TY == kGmmMX4;
  constexpr int kScaleSet = Shape::kScaleSet;
  constexpr int kIndexes = kGather ? kC * C::kRows : 64;  // dw: rows of x per wave and stage

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, l16 = lane & 15;

  const int rm = __builtin_amdgcn_readfirstlane(t.rm);
  const int cn = __builtin_amdgcn_readfirstlane(t.cn);
  const int red = __builtin_amdgcn_readfirstlane(MODE == kGmmDw ? t.span.m
                                                 : MODE == kGmmFwd ? p.K : p.N);
  const int stages = (red + kStage - 1) / kStage;
  const int64_t e_rows = int64_t(t.span.e) * p.N;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(g_zeros);
  bool bad_row = false;

  // ---- Where each chunk of this lane begins: base + offset, moved on by a
  // uniform step per stage.  Outputs past the tile's edge read a row or chunk
  // inside it: they are not stored.
  const uint8_t* qbase;
  const uint8_t* cbase;
  uint32_t qo[kQ], co[kC];
  const int64_t qstep = kRowsAlong ? 128 : 64 * p.row_stride;
  const int64_t cstep = kColsAlong ? 128 : kGather ? 0 : 64 * p.other_stride;
  if constexpr (kRowsAlong) {
    qbase = p.rows + (MODE == kGmmFwd && p.index ? 0 : t.span.row0 * p.row_stride);
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      int r = (wave * kQ + i) * Q::kRows + Q::row(lane);
      r = r < rm ? r : rm - 1;
      uint32_t row = uint32_t(r);
      if (MODE == kGmmFwd && p.index) {
        const int64_t x = p.index[t.span.row0 + r];
        const bool ok = x >= 0 && x < p.x_rows;
        bad_row = bad_row || !ok;
        row = ok ? uint32_t(x) : 0xffffffffu;
      }
      qo[i] = row == 0xffffffffu ? row : row * uint32_t(p.row_stride) + Q::chunk(lane) * 16;
    }
  } else {
    qbase = p.rows + t.span.row0 * p.row_stride + t.out_row0 * 2;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int ch = Q::chunk(lane);
      qo[i] = uint32_t((wave * kQ + i) * Q::kRows + Q::row(lane)) * uint32_t(p.row_stride) +
              (ch * 8 < rm ? ch * 16 : 0);
    }
  }
  if constexpr (kColsAlong) {
    cbase = p.other + (e_rows + t.c0) * p.other_stride;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int r = (wave * kC + i) * C::kRows + C::row(lane);
      co[i] = uint32_t(r < cn ? r : cn - 1) * uint32_t(p.other_stride) + C::chunk(lane) * 16;
    }
  } else {
    cbase = p.other + (MODE == kGmmDx ? e_rows * p.other_stride : 0) + t.c0 * 2;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int ch = C::chunk(lane);
      co[i] = ch * 8 < cn ? ch * 16 : 0;
      if (MODE == kGmmDx)
        co[i] += uint32_t((wave * kC + i) * C::kRows + C::row(lane)) * uint32_t(p.other_stride);
    }
  }
  qbase = uniform(qbase);
  cbase = uniform(cbase);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(uint32_t(uintptr_t((lds_u8*)lds)));
  const uint32_t extra0 = lds0 + NB * kBuf;

  // ---- dw: the rows of x.  Each wave keeps the indexes of its own chunks'
  // rows for kSet stages in LDS, four sets: entry (stage, load, row of the load).
  // A set is loaded at least NB - 1 stages before its first index is read, when
  // the waits of that many stages have covered it.
  constexpr int kSet = 64 / kIndexes;
  static_assert(!kGather || (2 * kSet - NB - 1 >= NB - 1 && NB <= 4), "indexes in time");
  int next_row[kGather ? kC : 1];
  auto index_row = [&](int s, int at) { return s * 64 + wave * kIndexes + at; };
  typedef __attribute__((address_space(3))) int lds_int;
  auto load_index = [&](int s) {  // the kSet stages from s (a multiple) on
    if constexpr (kGather) {
      const uint32_t to = extra0 + wave * 1024 + (s / kSet & 3) * 256;
      const int r = index_row(s + lane / kIndexes, lane % kIndexes);
      if (p.index)
        load_word_to_lds(r < red ? static_cast<const void*>(p.index + t.span.row0 + r)
                                 : static_cast<const void*>(zeros),
                         to);
      else
        *(lds_int*)(uintptr_t(to + lane * 4)) = int(t.span.row0) + r;
    }
  };
  auto read_rows = [&](int s) {  // for the loads of stage s
    if constexpr (kGather) {
      const uint32_t at =
          extra0 + wave * 1024 + ((s & (4 * kSet - 1)) * kIndexes + C::row(lane)) * 4;
#pragma unroll
      for (int i = 0; i < kC; ++i)
        next_row[i] = ((const lds_int*)(uintptr_t(at)))[i * C::kRows];
    }
  };
  // ---- scales: a thread brings 16 bytes of a row of the tile (rows operand
  // first) for two stages.
  constexpr int kS = kScales ? (BM + BN) / (NW * 64) : 1;
  const uint8_t* sp[kS];
  if constexpr (kScales) {
    static_assert((BM + BN) % (NW * 64) == 0, "whole wave loads of scales");
#pragma unroll
    for (int i = 0; i < kS; ++i) {
      const int r = i * NW * 64 + tid;
      if (r < BM) {
        int64_t row = t.span.row0 + (r < rm ? r : rm - 1);
        if (p.index) row = p.index[row];
        sp[i] = row >= 0 && row < p.x_rows ? p.row_scales + row * p.blocks : nullptr;
      } else {
        sp[i] = p.other_scales + (e_rows + t.c0 + (r - BM < cn ? r - BM : cn - 1)) * p.blocks;
      }
    }
  }
  auto load_scales = [&](int s) {  // of the stages s and s + 1, s even
    if constexpr (kScales) {
#pragma unroll
      for (int i = 0; i < kS; ++i)
        load_to_lds(s < stages && sp[i] ? sp[i] + s * 8 : zeros,
                    extra0 + (s >> 1) % Shape::kScaleSets * kScaleSet + (i * NW + wave) * 1024);
    }
  };

  // ---- load i of stage s, into buffer s % NB.  FAST: all of it exists.
  auto load_one = [&](int s, int i, auto fast) {
    const bool is_q = i < kQ;
    const uint32_t to = lds0 + s % NB * kBuf +
                        (is_q ? (wave * kQ + i) * Q::kPitch
                              : Q::kBytes + (wave * kC + i - kQ) * C::kPitch);
    if (is_q) {
      const uint8_t* from = qbase + s * qstep;
      if constexpr (decltype(fast)::value) {
        load_to_lds(from, qo[i], to);
      } else {
        const int at = kRowsAlong ? s * kStage + Q::chunk(lane) * kPerChunk
                                  : s * 64 + (wave * kQ + i) * Q::kRows + Q::row(lane);
        load_to_lds(at < red && qo[i] != 0xffffffffu ? from + qo[i] : zeros, to);
      }
    } else {
      const int j = i - kQ;
      const uint8_t* from = cbase + s * cstep;
      if constexpr (kGather)
        from += uint64_t(uint32_t(next_row[j])) * uint32_t(p.other_stride) + co[j];
      else if constexpr (!decltype(fast)::value)
        from += co[j];
      if constexpr (decltype(fast)::value) {
        if constexpr (kGather) load_to_lds(from, to);
        else load_to_lds(from, co[j], to);
      } else {
        const int at = kColsAlong ? s * kStage + C::chunk(lane) * kPerChunk
                                  : s * 64 + (wave * kC + j) * C::kRows + C::row(lane);
        const bool have =
            at < red && (!kGather || (next_row[j] >= 0 && next_row[j] < p.x_rows));
        load_to_lds(have ? from : zeros, to);
      }
    }
  };
  constexpr auto kFast = std::true_type{};
  constexpr auto kCareful = std::false_type{};

  float4v acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = float4v{0, 0, 0, 0};

  // Fragments of 16 outputs x 64 bytes, one set per half, and their scales (the
  // bytes of both halves).
  int4v fq[2][FM], fc[2][FN];
  int sq[2][kScales ? FM : 1] = {}, sc[2][kScales ? FN : 1] = {};
  uint32_t q_lane[2], c_lane[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    q_lane[kk] = lds0 + Q::template read_at<kScales>(lane, kk) + wm * FM * Q::kFragment;
    c_lane[kk] = lds0 + Q::kBytes + C::template read_at<kScales>(lane, kk) + wn * FN * C::kFragment;
  }
  const uint32_t s_lane = extra0 + l16 * 16 + g * 2;
  // Reads fragment f (columns' first) of half kk, and its scale.
  auto read_one = [&](int kk, int f, uint32_t qa, uint32_t ca, uint32_t sa) {
    if (f < FN) {
      fc[kk][f] = C::read(ca + f * C::kFragment);
      if constexpr (kScales)
        sc[kk][f] = *((const lds_u16*)(uintptr_t(sa)) + (BM + wn * TN + f * 16) * 8);
    } else {
      fq[kk][f - FN] = Q::read(qa + (f - FN) * Q::kFragment);
      if constexpr (kScales)
        sq[kk][f - FN] = *((const lds_u16*)(uintptr_t(sa)) + (wm * TM + (f - FN) * 16) * 8);
    }
  };

  if (kGather) {
    load_index(0);
    load_index(kSet);
    wait_loads<0>();
  }
#pragma unroll
  for (int s = 0; s < NB; s += 2) load_scales(s);
#pragma unroll
  for (int s = 0; s < NB; ++s) {
    read_rows(s);
#pragma unroll
    for (int i = 0; i < kQ + kC; ++i) load_one(s, i, kCareful);
  }
  read_rows(NB);
  if constexpr (kGather) {
    if (p.index)  // a look at all of them, under the first loads, so that the rest need none
      for (int s = 0; s < stages; s += kSet) {
        const int r = index_row(s + lane / kIndexes, lane % kIndexes);
        const int x = r < red ? p.index[t.span.row0 + r] : 0;
        bad_row = bad_row || (r < red && (x < 0 || x >= p.x_rows));
      }
  }
  // A wave that names a row outside x takes the careful loads throughout.
  const bool careful = __ballot(bad_row) != 0;
  wait_loads<(NB - 1) * (kQ + kC)>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int f = 0; f < FN + FM; ++f) read_one(0, f, q_lane[0], c_lane[0], s_lane);

  // Products of the two halves, numbered through; the reads of the second
  // half's fragments, the barrier, the loads and the reads of the next stage's
  // first half are spread between them.  One wave load occupies the path to
  // LDS for 16 cycles, as long as a product: 4 waves keep below its rate with
  // one load per 5 products.
  // Sums from kVector on stay in vector registers: with all 256 accumulation
  // registers of a lane taken the compiler moves sums about between products.
  constexpr int kVector = FM * FN < 64 ? FM * FN : kScales ? 60 : 56;
  constexpr int kHalf = FM * FN, kReads = FM + FN, kAll = kQ + kC;
  constexpr int kBarrier = kHalf / 2;
  auto products = [&](int s, auto which, auto fast) {
    constexpr int kk = decltype(which)::value;
    const uint32_t buf = (s + kk) % NB * kBuf;  // of the fragments to read, half kk ^ 1
    uint32_t qa = q_lane[kk ^ 1] + buf, ca = c_lane[kk ^ 1] + buf;
    uint32_t sa =
        kScales ? s_lane + ((s + kk) >> 1) % Shape::kScaleSets * kScaleSet + ((s + kk) & 1) * 8 : 0;
    // One address register per operand; the fragments are offsets in the
    // instructions.
    asm("" : "+v"(qa), "+v"(ca), "+v"(sa));
    // Whatever the compiler does to the fragments' registers is done before
    // the first product, with the distance that products need.
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      asm volatile("" : "+v"(fc[kk][f]));
      if constexpr (kScales) asm volatile("" : "+v"(sc[kk][f]));
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      asm volatile("" : "+v"(fq[kk][f]));
      if constexpr (kScales) asm volatile("" : "+v"(sq[kk][f]));
    }
    asm volatile("s_nop 1");
    __builtin_amdgcn_sched_barrier(0);
    // The compiler would gather the products and put each read right before
    // its use: it keeps this order.
#pragma unroll
    for (int a = 0; a < FM; ++a) {
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        const int n = a * FN + b, m = kk * kHalf + n;
        if (a * FN + b >= kVector)
          mma_acc<TY, kk, true>(acc[a][b], fc[kk][b], fq[kk][a], sc[kk][kScales ? b : 0],
                                sq[kk][kScales ? a : 0]);
        else
          mma_acc<TY, kk, false>(acc[a][b], fc[kk][b], fq[kk][a], sc[kk][kScales ? b : 0],
                                 sq[kk][kScales ? a : 0]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < kReads; ++r)
          if (n == (kk == 0 ? r * (kBarrier * 3 / 4) / kReads : r * (kHalf * 3 / 4) / kReads)) {
            read_one(kk ^ 1, r, qa, ca, sa);
            __builtin_amdgcn_sched_barrier(0);
          }
        if (m == kBarrier - 1) {
          // The loads of stage s + 1 and all before them have arrived.
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NB - 2) * kAll) : "memory");
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          if constexpr (kScales) {
            if ((s & 1) == 0) load_scales(s + NB);
          }
          if constexpr (kGather) {
            if ((s & (kSet - 1)) == 0) load_index(s + 2 * kSet);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < kAll; ++i)
          if (m == kBarrier + i * (kHalf * 5 / 4) / kAll) {
            load_one(s + NB, i, fast);
            __builtin_amdgcn_sched_barrier(0);
          }
      }
    }
  };
  auto stage = [&](int s, auto fast) {
    products(s, std::integral_constant<int, 0>{}, fast);
    products(s, std::integral_constant<int, 1>{}, fast);
    end_of_products();
    read_rows(s + NB + 1);
  };
  int s = 0;
  if (!careful)
    for (; (s + NB + 1) * kStage <= red; ++s) stage(s, kFast);
  for (; s < stages; ++s) stage(s, kCareful);
  // The loads still in flight write to this workgroup's LDS; the last products
  // have to end before their sums are read.
  asm volatile("s_waitcnt vmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      if (a * FN + b >= kVector)
        asm volatile("" : "+v"(acc[a][b]));
      else
        asm volatile("" : "+a"(acc[a][b]));
    }
  if (bad_row && p.status) *p.status = A2AV_ERR_INVALID_ARGS;
  __syncthreads();  // everybody's reads and loads are done
  constexpr int kPart = NB * kBuf / NW / 1024 * 1024;
  constexpr bool kFp32 = MODE == kGmmDw || TY == kGmmMX4;  // the others' types are 16 bits
  if (kFp32 && p.out_type == A2AV_FP32)
    store_rows<MODE, TM, TN, FM, FN, 4, kPart>(p, t, acc, wm, wn, lds + wave * kPart);
  else
    store_rows<MODE, TM, TN, FM, FN, 2, kPart>(p, t, acc, wm, wn, lds + wave * kPart);
}

// 256 x 256 tiles, one workgroup per CU.
template <int TY, int MODE>
__global__ __launch_bounds__(256, 1) void gmm_large(const GmmParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[PipeShape<TY, MODE, 256, 256, 2>::kLds];
  static_assert(PipeShape<TY, MODE, 128, 128, 4>::kLds <= sizeof(lds), "quarters fit");
  Tile t;
  int part;
  if (!find_work<MODE, 256, 256, true>(p, &t, &part)) return;
  if (part < 0)
    gmm_tile<TY, MODE, 256, 256, 2>(p, t, lds);
  else
    gmm_tile<TY, MODE, 128, 128, 4>(p, t, lds);
}

// 128 x 128 tiles, two workgroups per CU.
template <int TY, int MODE, int NB>
__global__ __launch_bounds__(256, NB == 2 ? 2 : 1) void gmm_small(const GmmParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[PipeShape<TY, MODE, 128, 128, NB>::kLds];
  Tile t;
  int part;
  if (!find_work<MODE, 128, 128, false>(p, &t, &part)) return;
  gmm_tile<TY, MODE, 128, 128, NB>(p, t, lds);
}

// ------------------------------------------------------------------ few rows per expert

// MT x 16 rows and FN x 16 columns by NW waves that share out the reduction.
// With few rows an expert's weight is read for little work, and its bytes are
// the time: every wave streams its part of W straight into registers (nothing
// of it is used twice, so LDS would only be a detour), 4 steps of 64 bytes per
// row at a time, and the waves' sums meet in LDS, in the order of the waves.  32
// rows of 8 experts, 2048 x 7168: bf16 45 us, 5.2 TB/s of W; 4 bits 14 us, 4.5.
template <int TY, int MT, int FN, int NW>
__global__ __launch_bounds__(NW * 64, 4) void gmm_few(const GmmParams p) {
  constexpr int BM = MT * 16, BN = FN * 16, U = 4;
  constexpr int kStep = TY == kGmmMX4 ? 128 : 32;  // reduction elements per product
  __shared__ float part[NW][MT * FN][64 * 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, l16 = lane & 15;
  Tile t;
  int cut;
  if (!find_work<kGmmFwd, BM, BN, false>(p, &t, &cut)) return;
  const int64_t w0 = int64_t(t.span.e) * p.N + t.c0;
  const int K = p.K;
  constexpr int kPerChunk = kStep / 4;

  const uint8_t* x[MT];
  const uint8_t* w[FN];
  const uint8_t* xs[TY == kGmmMX4 ? MT : 1];
  const uint8_t* ws[TY == kGmmMX4 ? FN : 1];
  // A row outside x reads row 0 and is made zeros before the products, as in the
  // tile kernels, so that W's NaN and infinities show in it with every kernel.
  int mask[MT];
  bool bad_row = false;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = i * 16 + l16;
    int64_t row = t.span.row0 + (r < t.rm ? r : t.rm - 1);
    mask[i] = -1;
    if (p.index) {
      row = p.index[row];
      if (row < 0 || row >= p.x_rows) {
        row = 0;
        mask[i] = 0;
        bad_row = true;
      }
    }
    x[i] = p.rows + row * p.row_stride + g * 16;
    if constexpr (TY == kGmmMX4) xs[i] = p.row_scales + row * p.blocks;
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    const int c = f * 16 + l16;
    const int64_t row = w0 + (c < t.cn ? c : t.cn - 1);
    w[f] = p.other + row * p.other_stride + g * 16;
    if constexpr (TY == kGmmMX4) ws[f] = p.other_scales + row * p.blocks;
  }
  // The scale of this lane's chunk in a step.  Whole groups of steps take a row's
  // 16 bytes with one load (a byte each cost 7 of 24 us of 62 MB of weights).
  auto scale = [&](const uint8_t* at, int step) -> int { return at[step * 4 + g]; };
  auto scales = [&](const uint8_t* at, int step) -> int4v {
    struct __attribute__((packed, aligned(1))) Loose {
      int4v v;
    };
    return reinterpret_cast<const Loose*>(at + step * 4)->v;
  };

  float4v acc[MT][FN];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[i][f] = float4v{0, 0, 0, 0};

  // 16 bytes of a row, at any address, of which n elements exist.
  auto load = [&](const uint8_t* from, int n) -> int4v {
    if constexpr (TY == kGmmMX4)
      return n > 0 ? *reinterpret_cast<const int4v*>(from) : int4v{0, 0, 0, 0};
    else
      return load_part(from, n);
  };
  // Steps first .. first + n of 64 bytes; TAIL: some may lie past the end.
  auto run = [&](int first, auto n, auto tail) {
    constexpr int kN = decltype(n)::value;
    int4v wv[kN][FN], xv[kN][MT];
    int wsv[kN][FN], xsv[kN][MT];
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const int left =
          decltype(tail)::value ? K - (first + u) * kStep - g * kPerChunk : kPerChunk;
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        wv[u][f] = load(w[f] + int64_t(first + u) * 64, left);
        if constexpr (TY == kGmmMX4 && decltype(tail)::value)
          wsv[u][f] = left > 0 ? scale(ws[f], first + u) : 0x7f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xv[u][i] = load(x[i] + int64_t(first + u) * 64, left);
        if constexpr (TY == kGmmMX4 && decltype(tail)::value)
          xsv[u][i] = left > 0 ? scale(xs[i], first + u) : 0x7f;
      }
    }
    if constexpr (TY == kGmmMX4 && !decltype(tail)::value) {
      static_assert(kN == 4, "16 scales");
      int4v wg[FN], xg[MT];
#pragma unroll
      for (int f = 0; f < FN; ++f) wg[f] = scales(ws[f], first);
#pragma unroll
      for (int i = 0; i < MT; ++i) xg[i] = scales(xs[i], first);
#pragma unroll
      for (int u = 0; u < kN; ++u) {
#pragma unroll
        for (int f = 0; f < FN; ++f) wsv[u][f] = int(uint32_t(wg[f][u]) >> (8 * g));
#pragma unroll
        for (int i = 0; i < MT; ++i) xsv[u][i] = int(uint32_t(xg[i][u]) >> (8 * g));
      }
    }
#pragma unroll
    for (int u = 0; u < kN; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int4v row = xv[u][i] & mask[i];
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          if constexpr (TY == kGmmMX4)  // row 0's scale may be NaN
            acc[i][f] = mma_mx4(wv[u][f], row, acc[i][f], wsv[u][f], xsv[u][i] & mask[i], 0);
          else
            acc[i][f] = mma<TY>(wv[u][f], row, acc[i][f]);
        }
      }
    end_of_products();
  };
  // Waves take groups of U steps in turn.
  const int steps = (K + kStep - 1) / kStep;
  const int whole = K / kStep / U * U;
  for (int s = wave * U; s < whole; s += NW * U)
    run(s, std::integral_constant<int, U>{}, std::false_type{});
  for (int s = whole + wave; s < steps; s += NW)
    run(s, std::integral_constant<int, 1>{}, std::true_type{});
  if (bad_row && p.status) *p.status = A2AV_ERR_INVALID_ARGS;

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f)
      *reinterpret_cast<float4v*>(&part[wave][i * FN + f][lane * 4]) = acc[i][f];
  __syncthreads();
  // Element (r, c): column c % 16 = 4g + j of fragment (r / 16, c / 16), lane 16 g + r % 16.
  for (int q = tid; q < BM * BN; q += NW * 64) {
    const int r = q / BN, c = q % BN;
    if (r >= t.rm || c >= t.cn) continue;
    const int at = ((c & 15) >> 2) * 64 + (r & 15) * 4 + (c & 3);
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += part[i][(r >> 4) * FN + (c >> 4)][at];
    const int64_t o = (t.out_row0 + r) * p.out_stride + t.c0 + c;
    if (p.out_type == A2AV_FP32)
      reinterpret_cast<float*>(p.out)[o] = v;
    else
      reinterpret_cast<uint16_t*>(p.out)[o] = round16(v, p.out_type);
  }
}

template <int TY, int MODE>
hipError_t launch_mode(const GmmParams& p, bool direct, hipStream_t stream) {
  if constexpr (MODE == kGmmFwd) {
    // The streaming kernel reads W once per row tile: it pays while the rows of an
    // expert mostly fit into one tile, and otherwise while about one workgroup is on
    // every CU (4 bits: two), more of them for short rows, whose products take less
    // than a tile's start (as much as 1 KiB of a row; 512 bytes count at least).  Over
    // some 700 sizes that it was not made with (1 to 64 experts of 3 to 60 rows, some
    // with a hot one, N to 4096, K to 7168) the kernel chosen takes 1.01 to 1.03 times
    // the fastest one's time in each of the four kinds below, and by 12 and 40 rows per
    // expert alone 1.10 to 1.21.
    // us of it and of the tile kernel in its place (in brackets its workgroups):
    //   bf16, 64 experts of 2048 x 2048: 8 rows each 104 and 136, 12 rows 113 and 136,
    //   16 rows 141 and 136, 24 rows 179 and 137; half of 640 rows on one expert 120
    //   and 136.  8 of 2048 x 7168: 12 rows 52 and 59, 16 rows (512) 63 and 59; 4 of
    //   them: 24 rows (256) 41 and 54; one: 40 rows (192) 24 and 46.  One of 256 x
    //   4096: 512 rows (256) 15 and 30, 2048 rows (1024) 46 and 30.
    //   Unaligned, 2001 x 7001, 8 rows: 8 experts (504) 94 and 72, one (63) 48 and 57;
    //   257 x 4001, 512 rows in tiles of 32 (144) 42 and 35.
    //   4 bits, 64 of 2048 x 2048: 12 rows 35 and 36, 24 rows 44 and 38; 8 of 2048 x
    //   7168: 24 rows (512) 18 and 24, 40 rows (1024) 30 and 25.
    //   4 bits of other scale groups, whose tile kernel is slower, 8 of 2048 x 7200: 40
    //   rows (1024) 34 and 49, 64 rows (1536) 42 and 51; 64 of 2048 x 1408: 32 rows
    //   (8192) 44 and 37.
    constexpr int kWaves = TY == kGmmMX4 ? 4 : 8;  // a row of 4 bits is a quarter as long
    const int64_t bytes = TY == kGmmMX4 ? p.K / 2 : p.K * int64_t(2);
    const int64_t row = bytes < 512 ? 512 : bytes;
    const auto at_once = [&](int BM, int limit) {
      const int64_t wgs = expected_row_tiles(p, BM) * ((int64_t(p.N) + 31) / 32);
      return wgs <= limit + (direct ? limit * 1024 / row : 0);
    };
    if (p.x_rows > 0) {  // it reads row 0 for rows outside x
      const bool one_tile = p.nrows <= int64_t(p.E) * 12 && (direct || TY == kGmmMX4);
      if (one_tile || at_once(16, 256))
        return launch_tiles<MODE, 16, 32>(gmm_few<TY, 1, 2, kWaves>, kWaves * 64, p, stream);
      if (at_once(32, TY == kGmmMX4 ? (direct ? 512 : 1536) : direct ? 256 : 0))
        return launch_tiles<MODE, 32, 32>(gmm_few<TY, 2, 2, kWaves>, kWaves * 64, p, stream);
    }
  }
  if (direct) {
    // Rows of an expert (dw: of the reduction, which no tile cuts).  us of the large
    // tiles and the small ones, bf16, 64 experts of 2048 x 2048: 96 rows each 155 and
    // 141, dx 139 and 119; 128 rows 157 and 158, 142 and 145; 160 rows 161 and 178,
    // 144 and 176.  8 experts of 2048 x 7168: 96 rows 79 and 79, dx 66 and 56; 160 rows
    // 83 and 83, 68 and 84.
    if (MODE == kGmmDw || p.nrows / p.E >= 160)
      return launch_tiles<MODE, 256, 256>(gmm_large<TY, MODE>, 256, p, stream);
    if constexpr (MODE != kGmmDw) {
      const int64_t cols = MODE == kGmmFwd ? p.N : p.K;
      // More tiles than CUs: two workgroups on each hide each other's ends.  Else one,
      // with four stages of loads in flight.  us of two stages and four, bf16, 64 rows
      // of each expert, 2048 x 2048: 16 experts (256 tiles) 43 and 40, dx 40 and 35; 32
      // (512) 73 and 75, 60 and 63.  12 rows, 8 of 7168 x 2048 (448): 54 and 59, 4 bits
      // (16 rows) 16 and 22; 32 of 4096 x 1024 (1024): 54 and 62.  8 of 2048 x 7168
      // (128): 103 and 71.  24 of 4096 x 2048 (768), an exception: 113 and 107.
      if (expected_row_tiles(p, 128) * ((cols + 127) / 128) > 256)
        return launch_tiles<MODE, 128, 128>(gmm_small<TY, MODE, 2>, 256, p, stream);
      return launch_tiles<MODE, 128, 128>(gmm_small<TY, MODE, 4>, 256, p, stream);
    }
  }
  if constexpr (TY != kGmmMX4) {
    if (p.K < 8 || (MODE != kGmmFwd && p.N < 8))  // rows of an operand
      return launch_tiles<MODE, 64, 64>(gmm_kernel<TY, MODE, 64, 64, 2, 2, false, true>, 256, p,
                                        stream);
    const int64_t used = p.E < p.nrows ? p.E : p.nrows;
    const int64_t cols = ((MODE == kGmmFwd ? p.N : p.K) + 127) / 128;
    const int64_t rows = MODE == kGmmDw ? int64_t(p.E) * ((p.N + 127) / 128)
                                        : p.nrows / 128 + used / 2;
    // Too few tiles for two on every CU: quarters of them.  us of 64 x 64 tiles and
    // of 128 x 128, bf16: 8 experts of 256 rows, 2001 x 1003 (320 tiles), 35 and 43, dx
    // 34 and 45; 512 rows (576) 55 and 63, 54 and 65; 16 of 300 rows, 2001 x 2003 (720)
    // 156 and 118, 158 and 121.  dw, 8 of 256 rows: 1001 x 1003 (512) 24 and 26, 2001 x
    // 2003 (2048) 76 and 88; of 4096 rows 789 and 782; one of 8192, 4001 x 4003: 775, 719.
    if (rows * cols < 512)
      return launch_tiles<MODE, 64, 64>(gmm_kernel<TY, MODE, 64, 64, 2, 2, false>, 256, p, stream);
  }
  return launch_tiles<MODE, 128, 128>(gmm_kernel<TY, MODE, 128, 128, 2, 2, TY == kGmmMX4>, 256, p,
                                      stream);
}

}  // namespace

hipError_t launch_gmm(const GmmParams& p, GmmType type, GmmMode mode, hipStream_t stream) {
  // The loads to LDS move aligned chunks of 16 bytes: every row has to begin
  // and end on one.
  const uintptr_t bases = reinterpret_cast<uintptr_t>(p.rows) | reinterpret_cast<uintptr_t>(p.other);
  // They go by 32-bit offsets from a tile's first row (x that the forward product
  // gathers: from its first; the weight gradient's x by 64 bits).  Anything else
  // takes the kernel with plain loads.
  const int64_t far = (int64_t(1) << 32) - 256;
  const bool all_x = mode == kGmmFwd && p.index;
  const int chunked = mode == kGmmFwd ? p.K : p.N | p.K;  // widths that loads run along
  const bool direct = ((bases | uint64_t(p.row_stride) | uint64_t(p.other_stride)) & 15) == 0 &&
                      (chunked & 7) == 0 && p.row_stride <= far / 256 &&
                      p.other_stride <= far / 256 &&
                      (!all_x || p.row_stride <= far / (p.x_rows + 1));
  if (type == kGmmMX4) {
    const uintptr_t scales = reinterpret_cast<uintptr_t>(p.row_scales) |
                             reinterpret_cast<uintptr_t>(p.other_scales) | uintptr_t(p.blocks);
    return launch_mode<kGmmMX4, kGmmFwd>(p, direct && scales % 16 == 0, stream);
  }
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
