// moe_fp8.hip -- the products grouped by expert on 8-bit rows and weights.
//
// With r a row of expert e, b a block of 128 of the reduction and 2^s the scales
//   forward  y [r][n] = sum_b 2^(sx[index[r]][b] + sw[e][n / 128][b]) sum_k x[index[r]][k] W[e][n][k]
//   dx       dx[r][k] = sum_b 2^(sdy[r][b] + sw[e][b][k / 128]) sum_n dy[r][n] W[e][n][k]
// A block is 128 bytes of a row and one matrix instruction, 16 x 16 x 128, which
// takes both scales as powers of two at no cost.  (FP32 scales would cost four
// multiply-adds per instruction and keep the sums out of the accumulation
// registers.)  It adds eight neighbouring products after cutting them at 2^-13 of
// the largest's binade, the eights and the blocks in FP32.  The format fills every
// row up to whole blocks, so there are no other alignments.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>
#include <utility>

#include "a2av.h"
#include "moe.h"
#include "moe_tiles.h"

namespace a2av {
namespace {

typedef int int2v __attribute__((ext_vector_type(2)));

__device__ inline float4v mma_fp8(int8v a, int8v b, float4v c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

// Bytes of scales of a row of `blocks` blocks.
__host__ __device__ inline int64_t scale_bytes(int64_t blocks) { return (blocks + 3) / 4 * 4; }

// One operand's 128 bytes x SPAN outputs of a stage in LDS, as chunks of 16 bytes.
//   along:  [SPAN][8 chunks], chunk c of row r at c ^ (r & 7): the 8 lanes that
//           read 128 bytes together, one chunk of 8 rows, meet every bank once.
//   across: [16 groups of 8 rows][SPAN / 16 chunks][8 rows]: the transposing read
//           takes a chunk's 8 rows, 128 bytes on end, by 16 lanes.
// A lane of group g takes the chunks (along) or rows (across) of 16 g and 64 + 16 g;
// any share of the block is right that both operands follow.
template <bool ALONG, int SPAN>
struct Block {
  static constexpr int kBytes = SPAN * 128;
  __device__ static int row(int q) {
    return ALONG ? q / 8 : q / (SPAN / 2) * 8 + (q & 7);
  }
  __device__ static int chunk(int q) {
    return ALONG ? (q ^ q >> 3) & 7 : q / 8 % (SPAN / 16);
  }
  // The fragment of the outputs f * 16 .. + 15.
  __device__ static int8v read(const uint8_t* at, int f) {
    const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
    if constexpr (ALONG) {
      const uint8_t* r = at + (f * 16 + l) * 128;
      const int4v lo = *reinterpret_cast<const int4v*>(r + (g ^ (l & 7)) * 16);
      const int4v hi = *reinterpret_cast<const int4v*>(r + ((4 + g) ^ (l & 7)) * 16);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      typedef __attribute__((address_space(3))) int2v lds_int2;
      int8v v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int eight = (i >> 1) * 8 + g * 2 + (i & 1);
        const int2v w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (lds_int2*)(at + eight * (SPAN * 8) + f * 128 + l * 8));
        v[2 * i] = w[0];
        v[2 * i + 1] = w[1];
      }
      return v;
    }
  }
};

// BM x BN of the output by 2 x 2 waves, a block per step, the next one's loads on
// their way to the other LDS buffer.
template <int MODE, int BM, int BN>
__global__ __launch_bounds__(256) void fp8_kernel(const GmmParams p) {
  constexpr int TM = BM / 2, TN = BN / 2, FM = TM / 16, FN = TN / 16;
  using Q = Block<true, BM>;               // the operand of the output's rows
  using C = Block<MODE == kGmmFwd, BN>;    // the operand of the output's columns
  constexpr int kBuf = Q::kBytes + C::kBytes;
  constexpr int kQ = BM * 8 / 256, kC = BN * 8 / 256;  // chunks per lane
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBuf];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  Tile t;
  int part;
  if (!find_work<MODE, BM, BN, false>(p, &t, &part)) return;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(g_zeros);
  const int w_blocks = (p.N + 127) / 128;  // of an expert's rows
  const int steps = MODE == kGmmFwd ? p.blocks : w_blocks;
  const int64_t e_rows = int64_t(t.span.e) * p.N;
  bool bad_row = false;

  const uint8_t* q[kQ];
  const uint8_t* c[kC];
  int c_row[kC];
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int at = (wave * kQ + i) * 64 + lane, r = Q::row(at);
    int64_t row = t.span.row0 + (r < t.rm ? r : t.rm - 1);
    bool ok = true;
    if (MODE == kGmmFwd && p.index) {
      row = p.index[row];
      ok = row >= 0 && row < p.x_rows;
      bad_row = bad_row || !ok;
    }
    q[i] = ok ? p.rows + row * p.row_stride + Q::chunk(at) * 16 : nullptr;
  }
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int at = (wave * kC + i) * 64 + lane, r = C::row(at), ch = C::chunk(at);
    c_row[i] = r;
    if constexpr (MODE == kGmmFwd)
      c[i] = p.other + (e_rows + t.c0 + (r < t.cn ? r : t.cn - 1)) * p.other_stride + ch * 16;
    else
      c[i] = p.other + (e_rows + r) * p.other_stride + t.c0 + (ch * 16 < t.cn ? ch * 16 : 0);
  }
  // This lane's scales: rows l16 of the fragments, and the weight's block.
  const uint8_t* qs[FM];
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int r = wm * TM + f * 16 + l16;
    int64_t row = t.span.row0 + (r < t.rm ? r : t.rm - 1);
    if (MODE == kGmmFwd && p.index) row = p.index[row];
    qs[f] = MODE == kGmmDx || (row >= 0 && row < p.x_rows) ? p.row_scales + row * scale_bytes(steps)
                                                           : nullptr;
  }
  const int64_t s_stride = scale_bytes(p.blocks);
  auto w_scale = [&](int b, int f) -> int {
    const int64_t col = t.c0 + wn * TN + f * 16;
    int64_t nb = MODE == kGmmFwd ? col / 128 : b, kb = MODE == kGmmFwd ? b : col / 128;
    if (nb >= w_blocks) nb = w_blocks - 1;
    if (kb >= p.blocks) kb = p.blocks - 1;
    return p.other_scales[(int64_t(t.span.e) * w_blocks + nb) * s_stride + kb];
  };

  const uint32_t lds0 = uint32_t(uintptr_t((lds_u8*)lds));
  auto issue = [&](int b) {
    const uint32_t base = lds0 + (b & 1) * kBuf;
#pragma unroll
    for (int i = 0; i < kQ; ++i)
      load_to_lds(q[i] ? q[i] + int64_t(b) * 128 : zeros,
                  __builtin_amdgcn_readfirstlane(base + (wave * kQ + i) * 1024));
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const uint8_t* from = c[i] + (MODE == kGmmFwd ? int64_t(b) * 128 : b * 128 * p.other_stride);
      // Rows of the next expert, or of none, are zeros: their codes may be NaN.
      if (MODE == kGmmDx && b * 128 + c_row[i] >= p.N) from = zeros;
      load_to_lds(from, __builtin_amdgcn_readfirstlane(base + Q::kBytes + (wave * kC + i) * 1024));
    }
  };

  float4v acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int d = 0; d < FN; ++d) acc[a][d] = float4v{0, 0, 0, 0};
  issue(0);
  for (int b = 0; b < steps; ++b) {
    wait_loads_and_barrier();
    if (b + 1 < steps) issue(b + 1);
    const uint8_t* buf = lds + (b & 1) * kBuf;
    int sc[FN], sq[FM];
    int8v fc[FN];
#pragma unroll
    for (int d = 0; d < FN; ++d) {
      sc[d] = w_scale(b, d);
      fc[d] = C::read(buf + Q::kBytes, wn * FN + d);
    }
#pragma unroll
    for (int a = 0; a < FM; ++a) sq[a] = qs[a] ? qs[a][b] : 127;
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      const int8v fq = Q::read(buf, wm * FM + a);
#pragma unroll
      for (int d = 0; d < FN; ++d) acc[a][d] = mma_fp8(fc[d], fq, acc[a][d], sc[d], sq[a]);
    }
    end_of_products();
  }
  if (bad_row && p.status) *p.status = A2AV_ERR_INVALID_ARGS;
  store_tile<MODE, TM, TN, FM, FN>(p, t, acc, wm, wn);
}

}  // namespace

hipError_t launch_gmm_fp8(const GmmParams& p, GmmMode mode, hipStream_t stream) {
  if (mode == kGmmFwd)
    return launch_tiles<kGmmFwd, 128, 128>(fp8_kernel<kGmmFwd, 128, 128>, 256, p, stream);
  return launch_tiles<kGmmDx, 128, 128>(fp8_kernel<kGmmDx, 128, 128>, 256, p, stream);
}

}  // namespace a2av
