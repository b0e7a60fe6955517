// moe_host.hip -- the entry points of include/a2av_moe.h: host checks, then
// the launches of moe_gemm.hip, moe_fp8.hip, moe_route.hip and moe_rows.hip.  No device
// code, no state: what an operator needs comes with the call.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "a2av_moe.h"
#include "moe.h"

namespace {

using namespace a2av;

constexpr int64_t kMax31 = 0x7fffffff;

int64_t size_of(int32_t dtype) { return dtype == A2AV_FP32 ? 4 : 2; }

bool is_float(int32_t dtype) {
  return dtype == A2AV_FP32 || dtype == A2AV_FP16 || dtype == A2AV_BF16;
}

bool is_16bit(int32_t dtype) { return dtype == A2AV_FP16 || dtype == A2AV_BF16; }

struct Operand {
  const void* p;
  int64_t bytes;
  bool out;
  int64_t align;  // bytes the address has to be a multiple of
  bool optional = false;
  int64_t stride = 0, width = 0;  // bytes of strided rows; 0: all of it is one run
};

// Bytes from a matrix's first row to the end of its last.
// Each is below 2^31; what no address space holds is cut to 2^60.
int64_t extent(int64_t rows, int64_t stride, int64_t width, int64_t size) {
  if (rows <= 0 || width <= 0) return 0;
  const int64_t n = (rows - 1) * stride + width;
  return n < (int64_t(1) << 58) ? n * size : int64_t(1) << 60;
}

// A matrix's rows; of bad sizes, something that must not be NULL.
Operand matrix(const void* p, bool bad, int64_t rows, int64_t stride, int64_t width, int64_t size,
               bool out, bool optional = false) {
  if (bad) return Operand{p, 1, out, size, optional};
  return Operand{p, extent(rows, stride, width, size), out, size, optional, stride * size,
                 width * size};
}

// NULLPTR, then nothing else; the addresses' other checks come last.
bool any_null(std::initializer_list<Operand> all) {
  for (const Operand& o : all)
    if (!o.p && !o.optional && o.bytes > 0) return true;
  return false;
}

// sum over i < n of floor((a i + b) / m), modulo 2^64, by the steps of Euclid's
// algorithm on a and m.
uint64_t sum_of_floors(uint64_t n, uint64_t m, uint64_t a, uint64_t b) {
  uint64_t sum = 0;
  for (;;) {
    sum += (n & 1 ? n * ((n - 1) / 2) : n / 2 * (n - 1)) * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const uint64_t top = a * n + b;
    if (top < m) return sum;
    n = top / m;
    b = top % m;
    const uint64_t t = m;
    m = a;
    a = t;
  }
}

// Whether two operands share a byte: rows of one may lie between the other's
// (columns of one buffer).
bool share_bytes(const Operand& one, const Operand& two) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(one.p), y = reinterpret_cast<uintptr_t>(two.p);
  if (!(x < y + uintptr_t(two.bytes) && y < x + uintptr_t(one.bytes))) return false;
  const bool swap = two.stride == two.width;
  const Operand& a = swap ? two : one;
  const Operand& b = swap ? one : two;
  // Larger than any address space (cut by extent): the rows are not told apart.
  if (b.stride == b.width || a.bytes >= int64_t(1) << 60 || b.bytes >= int64_t(1) << 60)
    return true;
  // at + i step, `len` bytes: the rows of a, from the start of b on.
  int64_t at = reinterpret_cast<intptr_t>(a.p) - reinterpret_cast<intptr_t>(b.p);
  const bool rows = a.stride > a.width;
  const int64_t len = rows ? a.width : a.bytes, step = rows ? a.stride : 1;
  int64_t n = rows ? (a.bytes - len) / step + 1 : 1;
  if (at + len <= 0) {  // rows before b
    const int64_t before = -(at + len) / step + 1;
    if (before >= n) return false;
    n -= before;
    at += before * step;
  }
  if (at >= b.bytes) return false;
  if (at <= 0) return true;
  const int64_t inside = (b.bytes - at + step - 1) / step;
  if (inside < n) n = inside;
  // Each of these begins before b's end, so it shares a byte with a row of b
  // exactly if its place in b's stride is less than b.width, or less than `len`
  // before the next row: if (at + len - 1) mod b.stride < b.width + len - 1.
  const int64_t hit = b.width + len - 1;
  if (hit >= b.stride) return true;
  const uint64_t m = uint64_t(b.stride), from = uint64_t(at + len - 1) % m, a1 = uint64_t(step) % m;
  return sum_of_floors(uint64_t(n), m, a1, from + m) !=
         sum_of_floors(uint64_t(n), m, a1, from + m - uint64_t(hit));
}

// Misaligned, or an output that shares a byte with another operand.
bool bad_addresses(std::initializer_list<Operand> all) {
  for (const Operand& o : all)
    if (o.p && o.bytes > 0 && reinterpret_cast<uintptr_t>(o.p) % uintptr_t(o.align)) return true;
  for (const Operand* a = all.begin(); a != all.end(); ++a)
    for (const Operand* b = a + 1; b != all.end(); ++b) {
      if (!(a->out || b->out) || !a->p || !b->p || a->bytes <= 0 || b->bytes <= 0) continue;
      if (share_bytes(*a, *b)) return true;
    }
  return false;
}

int launched(hipError_t e) { return e == hipSuccess ? A2AV_OK : A2AV_ERR_HIP; }

// Sizes stay a factor of two inside 32 bits: the kernels add a tile to them.
constexpr int64_t kMostSize = int64_t(1) << 30;
bool bad_size(int64_t v, int64_t least) { return v < least || v > kMostSize; }

// The sizes that all grouped products check alike.
bool bad_gmm_sizes(int64_t x_rows, int64_t rows, int32_t E, int64_t N, int64_t K,
                   const int32_t* index) {
  return bad_size(x_rows, 0) || bad_size(rows, 0) || E < 1 || E > 4096 || bad_size(N, 1) ||
         bad_size(K, 1) || N * K > (int64_t(1) << 58) / E || (!index && x_rows < rows);
}

int check_route_sizes(int64_t tokens, int32_t E, int32_t k) {
  if (tokens < 0 || E < 1 || E > 1024 || k < 1 || k > 16 || k > E) return A2AV_ERR_INVALID_ARGS;
  return tokens > kMostSize / k ? A2AV_ERR_INVALID_ARGS : A2AV_OK;
}

bool bad_groups(int32_t E, int32_t k, int32_t groups, int32_t top_groups, int32_t group_best) {
  return groups < 1 || groups > 64 || E % groups || top_groups < 1 || top_groups > groups ||
         k > top_groups * (E / groups) || group_best < 1 || group_best > 2;
}

// The scale is a positive number that has an inverse.
bool bad_scores(int32_t scores, float scale) {
  return (scores != A2AV_MOE_SOFTMAX && scores != A2AV_MOE_SIGMOID) ||
         !(scale >= 0x1p-100f && scale <= 0x1p100f);
}

// Blocks of 128 of a row of 8-bit values, and the scale bytes of such a row.
int64_t blocks128(int64_t n) { return (n + 127) / 128; }
int64_t fp8_pitch(int64_t n) { return (blocks128(n) + 3) / 4 * 4; }

int fp8_rows(const void* x, int64_t x_stride, int64_t rows, int64_t cols, int32_t dtype,
             const uint8_t* codes, const uint8_t* scales, bool quantize, hipStream_t stream) {
  const bool sizes_bad = bad_size(rows, 0) || bad_size(cols, 1) || x_stride < cols ||
                         x_stride > kMax31;
  const std::initializer_list<Operand> all = {
      matrix(x, sizes_bad, rows, x_stride, cols, size_of(dtype), !quantize),
      {codes, sizes_bad ? 1 : rows * blocks128(cols) * 128, quantize, 16},
      {scales, sizes_bad ? 1 : rows * fp8_pitch(cols), quantize, 4}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (rows == 0) return A2AV_OK;
  Fp8Params p{};
  p.x = x;
  p.out = const_cast<void*>(x);
  p.codes = const_cast<uint8_t*>(codes);
  p.scales = const_cast<uint8_t*>(scales);
  p.codes_in = codes;
  p.scales_in = scales;
  p.stride = x_stride;
  p.rows = rows;
  p.cols = int32_t(cols);
  p.blocks = int32_t(blocks128(cols));
  p.dtype = dtype;
  return launched(quantize ? launch_fp8_quantize(p, stream) : launch_fp8_dequantize(p, stream));
}

int fp8_weights(const void* w, int32_t E, int64_t N, int64_t K, int32_t dtype, const uint8_t* codes,
                const uint8_t* scales, bool quantize, hipStream_t stream) {
  const bool sizes_bad = E < 1 || E > 4096 || bad_size(N, 1) || bad_size(K, 1) ||
                         N * K > (int64_t(1) << 58) / E;
  const int64_t z = size_of(dtype);
  const std::initializer_list<Operand> all = {
      {w, sizes_bad ? 1 : E * N * K * z, !quantize, z},
      {codes, sizes_bad ? 1 : E * N * blocks128(K) * 128, quantize, 16},
      {scales, sizes_bad ? 1 : E * blocks128(N) * fp8_pitch(K), quantize, 4}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  Fp8Params p{};
  p.x = w;
  p.out = const_cast<void*>(w);
  p.codes = const_cast<uint8_t*>(codes);
  p.scales = const_cast<uint8_t*>(scales);
  p.codes_in = codes;
  p.scales_in = scales;
  p.stride = K;
  p.rows = E * N;
  p.n = int32_t(N);
  p.cols = int32_t(K);
  p.blocks = int32_t(blocks128(K));
  p.dtype = dtype;
  return launched(quantize ? launch_fp8_quantize(p, stream) : launch_fp8_dequantize(p, stream));
}

// The 8-bit products: rows of x (forward) or dy, of `red` values each, give rows
// of `out` values.
int gmm_fp8(GmmMode mode, const uint8_t* x_codes, const uint8_t* x_scales, int64_t x_rows,
            const uint8_t* w_codes, const uint8_t* w_scales, const int32_t* counts,
            const int32_t* index, void* y, int64_t y_stride, int64_t rows, int32_t E, int64_t N,
            int64_t K, int32_t y_dtype, int32_t* status, hipStream_t stream) {
  const int64_t out = mode == kGmmFwd ? N : K, red = mode == kGmmFwd ? K : N;
  const bool sizes_bad = bad_gmm_sizes(x_rows, rows, E, N, K, index) || y_stride < out ||
                         y_stride > kMax31;
  const bool some = sizes_bad || rows > 0;
  const std::initializer_list<Operand> all = {
      {x_codes, sizes_bad ? 1 : x_rows * blocks128(red) * 128, false, 16},
      {x_scales, sizes_bad ? 1 : x_rows * fp8_pitch(red), false, 4},
      {w_codes, sizes_bad ? 1 : E * N * blocks128(K) * 128, false, 16},
      {w_scales, sizes_bad ? 1 : E * blocks128(N) * fp8_pitch(K), false, 4},
      {counts, sizes_bad ? 1 : int64_t(E) * 4, false, 4},
      {index, sizes_bad ? 1 : rows * 4, false, 4, true},
      matrix(y, sizes_bad, rows, y_stride, out, size_of(y_dtype), true),
      {status, 4, true, 4, true}};
  if (some && any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(y_dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (rows == 0) return A2AV_OK;
  GmmParams p{};
  p.rows = x_codes;
  p.other = w_codes;
  p.row_scales = x_scales;
  p.other_scales = w_scales;
  p.out = static_cast<uint8_t*>(y);
  p.counts = counts;
  p.index = index;
  p.status = status;
  p.row_stride = blocks128(red) * 128;
  p.other_stride = blocks128(K) * 128;
  p.out_stride = y_stride;
  p.x_rows = x_rows;
  p.nrows = rows;
  p.E = E;
  p.N = int32_t(N);
  p.K = int32_t(K);
  p.blocks = int32_t(blocks128(K));
  p.out_type = y_dtype;
  return launched(launch_gmm_fp8(p, mode, stream));
}

}  // namespace

extern "C" {

int a2av_moe_route_workspace(int64_t tokens, int32_t E, int32_t k, int64_t* bytes) {
  if (!bytes) return A2AV_ERR_NULLPTR;
  const int st = check_route_sizes(tokens, E, k);
  if (st != A2AV_OK) return st;
  *bytes = route_is_small(tokens, E, k) ? 0 : int64_t(route_blocks(tokens)) * E * 4;
  return A2AV_OK;
}

int a2av_moe_route(const void* logits, int64_t logits_stride, int64_t tokens, int32_t E, int32_t k,
                   int32_t renormalize, int32_t dtype, int32_t* experts, float* weights,
                   int32_t* counts, int32_t* order, int32_t* place, void* workspace,
                   int64_t workspace_bytes, void* stream) {
  const int64_t slots = tokens > 0 && k > 0 && tokens <= kMax31 && k <= kMax31 ? tokens * k : 0;
  int64_t need = 0;
  const int sizes = a2av_moe_route_workspace(tokens, E, k, &need);
  const bool bad = sizes != A2AV_OK || logits_stride < E || logits_stride > kMax31;
  const int64_t z = size_of(dtype);
  const std::initializer_list<Operand> all = {
      matrix(logits, bad && slots > 0, bad ? 0 : tokens, logits_stride, E, z, false),
      {experts, slots * 4, true, 4},   {weights, slots * 4, true, 4},
      {counts, int64_t(E > 0 ? E : 0) * 4, true, 4},
      {order, slots * 4, true, 4},     {place, slots * 4, true, 4},
      {workspace, need, true, 16}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (bad || workspace_bytes < need || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  RouteParams p{};
  p.logits = logits;
  p.stride = logits_stride;
  p.tokens = int32_t(tokens);
  p.E = E;
  p.k = k;
  p.renorm = renormalize != 0;
  p.dtype = dtype;
  p.experts = experts;
  p.weights = weights;
  p.counts = counts;
  p.order = order;
  p.place = place;
  p.hist = static_cast<int32_t*>(workspace);
  return launched(launch_route(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_route_backward(const void* logits, int64_t logits_stride, int64_t tokens, int32_t E,
                            int32_t k, int32_t renormalize, int32_t dtype, const int32_t* experts,
                            const float* weights, const float* dweights, void* dlogits,
                            void* stream) {
  const int sizes = check_route_sizes(tokens, E, k);
  const int64_t slots = sizes ? (tokens > 0) : tokens * k;
  const bool bad = sizes != A2AV_OK || logits_stride < E || logits_stride > kMax31;
  const int64_t z = size_of(dtype);
  const std::initializer_list<Operand> all = {
      matrix(logits, bad && slots > 0, bad ? 0 : tokens, logits_stride, E, z, false),
      {experts, slots * 4, false, 4},
      {weights, slots * 4, false, 4},
      {dweights, slots * 4, false, 4},
      {dlogits, sizes ? slots : tokens * E * z, true, z}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  RouteBackParams p{};
  p.logits = logits;
  p.stride = logits_stride;
  p.tokens = int32_t(tokens);
  p.E = E;
  p.k = k;
  p.renorm = renormalize != 0;
  p.dtype = dtype;
  p.experts = experts;
  p.weights = weights;
  p.dweights = dweights;
  p.dlogits = dlogits;
  return launched(launch_route_back(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_route_grouped(const void* logits, int64_t logits_stride, const float* bias,
                           int64_t tokens, int32_t E, int32_t k, int32_t groups, int32_t top_groups,
                           int32_t group_best, int32_t scores, int32_t renormalize, float scale,
                           int32_t dtype, int32_t* experts, float* weights, int32_t* counts,
                           int32_t* order, int32_t* place, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  const int64_t slots = tokens > 0 && k > 0 && tokens <= kMax31 && k <= kMax31 ? tokens * k : 0;
  int64_t need = 0;
  const int sizes = a2av_moe_route_workspace(tokens, E, k, &need);
  const bool bad = sizes != A2AV_OK || logits_stride < E || logits_stride > kMax31 ||
                   bad_groups(E, k, groups, top_groups, group_best) || bad_scores(scores, scale);
  const int64_t z = size_of(dtype);
  const std::initializer_list<Operand> all = {
      matrix(logits, bad && slots > 0, bad ? 0 : tokens, logits_stride, E, z, false),
      {bias, int64_t(E > 0 ? E : 0) * 4, false, 4, true},
      {experts, slots * 4, true, 4},   {weights, slots * 4, true, 4},
      {counts, int64_t(E > 0 ? E : 0) * 4, true, 4},
      {order, slots * 4, true, 4},     {place, slots * 4, true, 4},
      {workspace, need, true, 16}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (bad || workspace_bytes < need || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  RouteParams p{};
  p.logits = logits;
  p.stride = logits_stride;
  p.tokens = int32_t(tokens);
  p.E = E;
  p.k = k;
  p.renorm = renormalize != 0;
  p.dtype = dtype;
  p.experts = experts;
  p.weights = weights;
  p.counts = counts;
  p.order = order;
  p.place = place;
  p.hist = static_cast<int32_t*>(workspace);
  p.groups = groups;
  p.top_groups = top_groups;
  p.group_best = group_best;
  p.sigmoid = scores == A2AV_MOE_SIGMOID;
  p.bias = bias;
  p.scale = scale;
  return launched(launch_route(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_route_grouped_backward(const void* logits, int64_t logits_stride, int64_t tokens,
                                    int32_t E, int32_t k, int32_t scores, int32_t renormalize,
                                    float scale, int32_t dtype, const int32_t* experts,
                                    const float* weights, const float* dweights, void* dlogits,
                                    void* stream) {
  const int sizes = check_route_sizes(tokens, E, k);
  const int64_t slots = sizes ? (tokens > 0) : tokens * k;
  const bool bad = sizes != A2AV_OK || logits_stride < E || logits_stride > kMax31 ||
                   bad_scores(scores, scale);
  const int64_t z = size_of(dtype);
  const std::initializer_list<Operand> all = {
      matrix(logits, bad && slots > 0, bad ? 0 : tokens, logits_stride, E, z, false),
      {experts, slots * 4, false, 4},
      {weights, slots * 4, false, 4},
      {dweights, slots * 4, false, 4},
      {dlogits, sizes ? slots : tokens * E * z, true, z}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  RouteBackParams p{};
  p.logits = logits;
  p.stride = logits_stride;
  p.tokens = int32_t(tokens);
  p.E = E;
  p.k = k;
  p.renorm = renormalize != 0;
  p.dtype = dtype;
  p.experts = experts;
  p.weights = weights;
  p.dweights = dweights;
  p.dlogits = dlogits;
  p.grouped = 1;
  p.sigmoid = scores == A2AV_MOE_SIGMOID;
  p.scale = scale;
  return launched(launch_route_back(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_gmm(const void* x, int64_t x_stride, int64_t x_rows, const void* w,
                 const int32_t* counts, const int32_t* index, void* y, int64_t y_stride,
                 int64_t rows, int32_t E, int64_t N, int64_t K, int32_t dtype, int32_t* status,
                 void* stream) {
  const bool sizes_bad = bad_gmm_sizes(x_rows, rows, E, N, K, index) || x_stride < K ||
                         x_stride > kMax31 || y_stride < N || y_stride > kMax31;
  const bool some = sizes_bad || rows > 0;
  const std::initializer_list<Operand> all = {
      matrix(x, sizes_bad, x_rows, x_stride, K, 2, false),
      {w, sizes_bad ? 1 : E * N * K * 2, false, 2},
      {counts, sizes_bad ? 1 : int64_t(E) * 4, false, 4},
      {index, sizes_bad ? 1 : rows * 4, false, 4, true},
      matrix(y, sizes_bad, rows, y_stride, N, 2, true),
      {status, 4, true, 4, true}};
  if (some && any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_16bit(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (rows == 0) return A2AV_OK;
  GmmParams p{};
  p.rows = static_cast<const uint8_t*>(x);
  p.other = static_cast<const uint8_t*>(w);
  p.out = static_cast<uint8_t*>(y);
  p.counts = counts;
  p.index = index;
  p.status = status;
  p.row_stride = x_stride * 2;
  p.other_stride = K * 2;
  p.out_stride = y_stride;
  p.x_rows = x_rows;
  p.nrows = rows;
  p.E = E;
  p.N = int32_t(N);
  p.K = int32_t(K);
  p.out_type = dtype;
  return launched(launch_gmm(p, dtype == A2AV_BF16 ? kGmmBF16 : kGmmFP16, kGmmFwd,
                             static_cast<hipStream_t>(stream)));
}

int a2av_moe_gmm_dx(const void* dy, int64_t dy_stride, const void* w, const int32_t* counts,
                    void* dx, int64_t dx_stride, int64_t rows, int32_t E, int64_t N, int64_t K,
                    int32_t dtype, int32_t* status, void* stream) {
  const bool sizes_bad = bad_gmm_sizes(rows, rows, E, N, K, nullptr) || dy_stride < N ||
                         dy_stride > kMax31 || dx_stride < K || dx_stride > kMax31;
  const bool some = sizes_bad || rows > 0;
  const std::initializer_list<Operand> all = {
      matrix(dy, sizes_bad, rows, dy_stride, N, 2, false),
      {w, sizes_bad ? 1 : E * N * K * 2, false, 2},
      {counts, sizes_bad ? 1 : int64_t(E) * 4, false, 4},
      matrix(dx, sizes_bad, rows, dx_stride, K, 2, true),
      {status, 4, true, 4, true}};
  if (some && any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_16bit(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (rows == 0) return A2AV_OK;
  GmmParams p{};
  p.rows = static_cast<const uint8_t*>(dy);
  p.other = static_cast<const uint8_t*>(w);
  p.out = static_cast<uint8_t*>(dx);
  p.counts = counts;
  p.status = status;
  p.row_stride = dy_stride * 2;
  p.other_stride = K * 2;
  p.out_stride = dx_stride;
  p.x_rows = rows;
  p.nrows = rows;
  p.E = E;
  p.N = int32_t(N);
  p.K = int32_t(K);
  p.out_type = dtype;
  return launched(launch_gmm(p, dtype == A2AV_BF16 ? kGmmBF16 : kGmmFP16, kGmmDx,
                             static_cast<hipStream_t>(stream)));
}

int a2av_moe_gmm_dw(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                    int64_t x_rows, const int32_t* counts, const int32_t* index, void* dw,
                    int64_t rows, int32_t E, int64_t N, int64_t K, int32_t dtype, int32_t dw_dtype,
                    int32_t* status, void* stream) {
  const bool sizes_bad = bad_gmm_sizes(x_rows, rows, E, N, K, index) || dy_stride < N ||
                         dy_stride > kMax31 || x_stride < K || x_stride > kMax31;
  const int64_t dz = size_of(dw_dtype);
  const std::initializer_list<Operand> all = {
      matrix(dy, sizes_bad, rows, dy_stride, N, 2, false),
      matrix(x, sizes_bad, rows ? x_rows : 0, x_stride, K, 2, false),
      {counts, sizes_bad ? 1 : int64_t(E) * 4, false, 4},
      {index, sizes_bad ? 1 : rows * 4, false, 4, true},
      {dw, sizes_bad ? 1 : E * N * K * dz, true, dz},
      {status, 4, true, 4, true}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_16bit(dtype) || (dw_dtype != dtype && dw_dtype != A2AV_FP32))
    return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  GmmParams p{};
  p.rows = static_cast<const uint8_t*>(dy);
  p.other = static_cast<const uint8_t*>(x);
  p.out = static_cast<uint8_t*>(dw);
  p.counts = counts;
  p.index = index;
  p.status = status;
  p.row_stride = dy_stride * 2;
  p.other_stride = x_stride * 2;
  p.out_stride = K;
  p.x_rows = x_rows;
  p.nrows = rows;
  p.E = E;
  p.N = int32_t(N);
  p.K = int32_t(K);
  p.out_type = dw_dtype;
  return launched(launch_gmm(p, dtype == A2AV_BF16 ? kGmmBF16 : kGmmFP16, kGmmDw,
                             static_cast<hipStream_t>(stream)));
}

int a2av_moe_combine(const void* y, int64_t y_stride, int64_t y_rows, const int32_t* place,
                     const float* weights, void* out, int64_t out_stride, int64_t tokens,
                     int32_t k, int64_t width, int32_t dtype, int32_t* status, void* stream) {
  const bool sizes_bad = bad_size(y_rows, 0) || bad_size(tokens, 0) || bad_size(width, 1) ||
                         k < 1 || k > 64 || y_stride < width || y_stride > kMax31 ||
                         out_stride < width || out_stride > kMax31;
  const int64_t z = size_of(dtype);
  const std::initializer_list<Operand> all = {
      matrix(y, sizes_bad, tokens ? y_rows : 0, y_stride, width, z, false),
      {place, sizes_bad ? 1 : tokens * k * 4, false, 4},
      {weights, sizes_bad ? 1 : tokens * k * 4, false, 4, true},
      matrix(out, sizes_bad, tokens, out_stride, width, z, true),
      {status, 4, true, 4, true}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (tokens == 0) return A2AV_OK;
  CombineParams p{};
  p.y = y;
  p.place = place;
  p.weights = weights;
  p.out = out;
  p.status = status;
  p.y_stride = y_stride;
  p.o_stride = out_stride;
  p.y_rows = y_rows;
  p.tokens = int32_t(tokens);
  p.k = k;
  p.width = int32_t(width);
  p.dtype = dtype;
  return launched(launch_combine(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_combine_backward(const void* dout, int64_t dout_stride, const void* y,
                              int64_t y_stride, int64_t y_rows, const int32_t* place,
                              const float* weights, void* dy, int64_t dy_stride, float* dweights,
                              int64_t tokens, int32_t k, int64_t width, int32_t dtype,
                              int32_t* status, void* stream) {
  const bool sizes_bad = bad_size(y_rows, 0) || bad_size(tokens, 0) || bad_size(width, 1) ||
                         k < 1 || k > 64 || y_stride < width || y_stride > kMax31 ||
                         dout_stride < width || dout_stride > kMax31 || dy_stride < width ||
                         dy_stride > kMax31;
  const int64_t z = size_of(dtype);
  const std::initializer_list<Operand> all = {
      matrix(dout, sizes_bad, tokens, dout_stride, width, z, false),
      // y is only read for dweights
      matrix(y, sizes_bad, tokens ? y_rows : 0, y_stride, width, z, false, dweights == nullptr),
      {place, sizes_bad ? 1 : tokens * k * 4, false, 4},
      {weights, sizes_bad ? 1 : tokens * k * 4, false, 4, true},
      matrix(dy, sizes_bad, tokens ? y_rows : 0, dy_stride, width, z, true),
      {dweights, sizes_bad ? 1 : tokens * k * 4, true, 4, weights == nullptr},
      {status, 4, true, 4, true}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (tokens == 0) return A2AV_OK;
  CombineParams p{};
  p.y = y;
  p.dout = dout;
  p.place = place;
  p.weights = weights;
  p.dy = dy;
  p.dweights = dweights;
  p.status = status;
  p.y_stride = y_stride;
  p.o_stride = dout_stride;
  p.dy_stride = dy_stride;
  p.y_rows = y_rows;
  p.tokens = int32_t(tokens);
  p.k = k;
  p.width = int32_t(width);
  p.dtype = dtype;
  return launched(launch_combine_back(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_mx4_quantize(const void* x, int64_t x_stride, int64_t rows, int64_t cols,
                          int32_t dtype, uint8_t* codes, uint8_t* scales, void* stream) {
  const bool sizes_bad = bad_size(rows, 0) || bad_size(cols, 1) || x_stride < cols ||
                         x_stride > kMax31;
  const int64_t z = size_of(dtype), blocks = (cols + 31) / 32;
  const std::initializer_list<Operand> all = {
      matrix(x, sizes_bad, rows, x_stride, cols, z, false),
      {codes, sizes_bad ? 1 : rows * blocks * 16, true, 16},
      {scales, sizes_bad ? 1 : rows * blocks, true, 1}};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (rows == 0) return A2AV_OK;
  Mx4Params p{};
  p.x = x;
  p.codes = codes;
  p.scales = scales;
  p.stride = x_stride;
  p.rows = int32_t(rows);
  p.cols = int32_t(cols);
  p.blocks = int32_t(blocks);
  p.dtype = dtype;
  return launched(launch_mx4_quantize(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                            int32_t dtype, void* x, int64_t x_stride, void* stream) {
  const bool sizes_bad = bad_size(rows, 0) || bad_size(cols, 1) || x_stride < cols ||
                         x_stride > kMax31;
  const int64_t z = size_of(dtype), blocks = (cols + 31) / 32;
  const std::initializer_list<Operand> all = {
      {codes, sizes_bad ? 1 : rows * blocks * 16, false, 16},
      {scales, sizes_bad ? 1 : rows * blocks, false, 1},
      matrix(x, sizes_bad, rows, x_stride, cols, z, true)};
  if (any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (rows == 0) return A2AV_OK;
  Mx4Params p{};
  p.out = x;
  p.codes_in = codes;
  p.scales_in = scales;
  p.stride = x_stride;
  p.rows = int32_t(rows);
  p.cols = int32_t(cols);
  p.blocks = int32_t(blocks);
  p.dtype = dtype;
  return launched(launch_mx4_dequantize(p, static_cast<hipStream_t>(stream)));
}

int a2av_moe_gmm_mx4(const uint8_t* x_codes, const uint8_t* x_scales, int64_t x_rows,
                     const uint8_t* w_codes, const uint8_t* w_scales, const int32_t* counts,
                     const int32_t* index, void* y, int64_t y_stride, int64_t rows, int32_t E,
                     int64_t N, int64_t K, int32_t y_dtype, int32_t* status, void* stream) {
  const bool sizes_bad = bad_gmm_sizes(x_rows, rows, E, N, K, index) || y_stride < N ||
                         y_stride > kMax31;
  const bool some = sizes_bad || rows > 0;
  const int64_t z = size_of(y_dtype), blocks = (K + 31) / 32;
  const std::initializer_list<Operand> all = {
      {x_codes, sizes_bad ? 1 : x_rows * blocks * 16, false, 16},
      {x_scales, sizes_bad ? 1 : x_rows * blocks, false, 1},
      {w_codes, sizes_bad ? 1 : E * N * blocks * 16, false, 16},
      {w_scales, sizes_bad ? 1 : E * N * blocks, false, 1},
      {counts, sizes_bad ? 1 : int64_t(E) * 4, false, 4},
      {index, sizes_bad ? 1 : rows * 4, false, 4, true},
      matrix(y, sizes_bad, rows, y_stride, N, z, true),
      {status, 4, true, 4, true}};
  if (some && any_null(all)) return A2AV_ERR_NULLPTR;
  if (!is_float(y_dtype)) return A2AV_ERR_UNSUPPORTED_DTYPE;
  if (sizes_bad || bad_addresses(all)) return A2AV_ERR_INVALID_ARGS;
  if (rows == 0) return A2AV_OK;
  GmmParams p{};
  p.rows = x_codes;
  p.other = w_codes;
  p.row_scales = x_scales;
  p.other_scales = w_scales;
  p.out = static_cast<uint8_t*>(y);
  p.counts = counts;
  p.index = index;
  p.status = status;
  p.row_stride = blocks * 16;
  p.other_stride = blocks * 16;
  p.out_stride = y_stride;
  p.x_rows = x_rows;
  p.nrows = rows;
  p.E = E;
  p.N = int32_t(N);
  p.K = int32_t(blocks * 32);
  p.blocks = int32_t(blocks);
  p.out_type = y_dtype;
  return launched(launch_gmm(p, kGmmMX4, kGmmFwd, static_cast<hipStream_t>(stream)));
}

int a2av_moe_fp8_quantize(const void* x, int64_t x_stride, int64_t rows, int64_t cols,
                          int32_t dtype, uint8_t* codes, uint8_t* scales, void* stream) {
  return fp8_rows(x, x_stride, rows, cols, dtype, codes, scales, true,
                  static_cast<hipStream_t>(stream));
}

int a2av_moe_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                            int32_t dtype, void* x, int64_t x_stride, void* stream) {
  return fp8_rows(x, x_stride, rows, cols, dtype, codes, scales, false,
                  static_cast<hipStream_t>(stream));
}

int a2av_moe_fp8_quantize_weights(const void* w, int32_t E, int64_t N, int64_t K, int32_t dtype,
                                  uint8_t* codes, uint8_t* scales, void* stream) {
  return fp8_weights(w, E, N, K, dtype, codes, scales, true, static_cast<hipStream_t>(stream));
}

int a2av_moe_fp8_dequantize_weights(const uint8_t* codes, const uint8_t* scales, int32_t E,
                                    int64_t N, int64_t K, int32_t dtype, void* w, void* stream) {
  return fp8_weights(w, E, N, K, dtype, codes, scales, false, static_cast<hipStream_t>(stream));
}

int a2av_moe_gmm_fp8(const uint8_t* x_codes, const uint8_t* x_scales, int64_t x_rows,
                     const uint8_t* w_codes, const uint8_t* w_scales, const int32_t* counts,
                     const int32_t* index, void* y, int64_t y_stride, int64_t rows, int32_t E,
                     int64_t N, int64_t K, int32_t y_dtype, int32_t* status, void* stream) {
  return gmm_fp8(kGmmFwd, x_codes, x_scales, x_rows, w_codes, w_scales, counts, index, y, y_stride,
                 rows, E, N, K, y_dtype, status, static_cast<hipStream_t>(stream));
}

int a2av_moe_gmm_fp8_dx(const uint8_t* dy_codes, const uint8_t* dy_scales, const uint8_t* w_codes,
                        const uint8_t* w_scales, const int32_t* counts, void* dx, int64_t dx_stride,
                        int64_t rows, int32_t E, int64_t N, int64_t K, int32_t dx_dtype,
                        int32_t* status, void* stream) {
  return gmm_fp8(kGmmDx, dy_codes, dy_scales, rows, w_codes, w_scales, counts, nullptr, dx,
                 dx_stride, rows, E, N, K, dx_dtype, status, static_cast<hipStream_t>(stream));
}

}  // extern "C"
