// moe.h -- what the host checks (moe_host.hip) hand to the kernels of the
// operators around the exchange (moe_gemm.hip, moe_route.hip, moe_rows.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace a2av {

// Element kinds of the grouped products.
enum GmmType { kGmmBF16 = 0, kGmmFP16 = 1, kGmmMX4 = 2 };
// Which operands the reduction runs along: forward (both rows), input
// gradient (the weight's columns), weight gradient (both columns).
enum GmmMode { kGmmFwd = 0, kGmmDx = 1, kGmmDw = 2 };

struct GmmParams {
  const uint8_t* rows;     // x or dy: the operand whose rows are the grouped rows
  const uint8_t* other;    // w (fwd, dx) or x (dw)
  const uint8_t* row_scales;    // MX4: [x_rows, B] and [E, N, B]
  const uint8_t* other_scales;
  uint8_t* out;
  const int32_t* counts;
  const int32_t* index;    // may be null
  int32_t* status;         // may be null
  int64_t row_stride;      // bytes
  int64_t other_stride;    // bytes from one row of `other` to the next
  int64_t out_stride;      // elements
  int64_t x_rows;          // rows that index may name
  int64_t nrows;           // grouped rows
  int32_t E;
  int32_t N, K;            // of the weights
  int32_t blocks;          // scale blocks of a row (MX4), of a weight's row (8 bits)
  int32_t out_type;        // a2av_dtype of out
};

struct RouteParams {
  const void* logits;
  int64_t stride;
  int32_t tokens, E, k, renorm, dtype;
  int32_t* experts;
  float* weights;
  int32_t* counts;
  int32_t* order;
  int32_t* place;
  int32_t* hist;           // workspace [E][blocks]
  int32_t per_block;       // tokens of a block (set by launch_route)
  // The router by groups: groups > 0.
  int32_t groups, top_groups, group_best, sigmoid;
  const float* bias;       // may be null
  float scale;
};

struct RouteBackParams {
  const void* logits;
  int64_t stride;
  int32_t tokens, E, k, renorm, dtype;
  const int32_t* experts;
  const float* weights;
  const float* dweights;
  void* dlogits;
  int32_t grouped, sigmoid;
  float scale;
};

struct CombineParams {
  const void* y;
  const void* dout;
  const int32_t* place;
  const float* weights;    // may be null: every weight 1
  void* out;               // forward
  void* dy;                // backward
  float* dweights;         // backward; may be null
  int32_t* status;
  int64_t y_stride, o_stride, dy_stride;  // elements; o_stride of out or dout
  int64_t y_rows;
  int32_t tokens, k, width, dtype;
};

struct Mx4Params {
  const void* x;
  void* out;
  const uint8_t* codes_in;
  const uint8_t* scales_in;
  uint8_t* codes;
  uint8_t* scales;
  int64_t stride;
  int32_t rows, cols, blocks, dtype;
};

// 8-bit rows (n = 0), or weights [rows / n, n, cols].
struct Fp8Params {
  const void* x;
  void* out;
  const uint8_t* codes_in;
  const uint8_t* scales_in;
  uint8_t* codes;
  uint8_t* scales;
  int64_t stride;          // elements, of x or out
  int64_t rows;
  int32_t n, cols, blocks, dtype;
};

hipError_t launch_gmm(const GmmParams& p, GmmType type, GmmMode mode, hipStream_t stream);
hipError_t launch_gmm_fp8(const GmmParams& p, GmmMode mode, hipStream_t stream);
hipError_t launch_route(RouteParams p, hipStream_t stream);
hipError_t launch_route_back(const RouteBackParams& p, hipStream_t stream);
hipError_t launch_combine(const CombineParams& p, hipStream_t stream);
hipError_t launch_combine_back(const CombineParams& p, hipStream_t stream);
hipError_t launch_mx4_quantize(const Mx4Params& p, hipStream_t stream);
hipError_t launch_mx4_dequantize(const Mx4Params& p, hipStream_t stream);
hipError_t launch_fp8_quantize(const Fp8Params& p, hipStream_t stream);
hipError_t launch_fp8_dequantize(const Fp8Params& p, hipStream_t stream);

// The router's blocks: tokens of one workgroup of its first kernel, 8 to 64, so
// that there are 256 blocks (one per CU) as soon as there are tokens for it.
constexpr int kRouteMost = 64;
inline int32_t route_per_block(int64_t tokens) {
  const int64_t n = (tokens / 256 + 7) / 8 * 8;
  return int32_t(n < 8 ? 8 : n > kRouteMost ? kRouteMost : n);
}
inline int32_t route_blocks(int64_t tokens) {
  const int32_t n = route_per_block(tokens);
  return int32_t((tokens + n - 1) / n);
}
// Few tokens: one workgroup does everything and needs no workspace.  Against the
// three launches (k = 2): 64 experts, 32 tokens 5.3 us and 7.5, 128 tokens 13.8
// and 8.3; 256 experts 7.4 and 8.5, 19.4 and 9.3; 512 experts, 16 tokens 11.0
// and 12.1, 32 tokens 17.6 and 12.4.
constexpr int kRouteSmall = 1024;  // slots
inline bool route_is_small(int64_t tokens, int32_t E, int32_t k) {
  return tokens * k <= kRouteSmall && tokens <= (E <= 64 ? 64 : E <= 256 ? 48 : 16);
}

}  // namespace a2av
