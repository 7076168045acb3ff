// C entry points of the 4-bit (MXFP4) product, of expert routing with its balance
// loss and of the low-rank adapters (include/imc.h): argument checks, scratch, launches.  As everywhere in the
// library, every check runs before anything is enqueued.
#include <cmath>

#include "adapters.cuh"
#include "mx_internal.cuh"

using namespace imc;
using namespace imc::mx;

namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;
constexpr int kMaxExperts = 1024, kMaxChosen = 32, kMaxGroups = 32;
// codes and scales of one operand stay below 2^40 bytes, so no size below overflows
constexpr double kMaxBytes = 1099511627776.0;

bool float_type(int dtype) { return dtype == IMC_F32 || dtype == IMC_F16 || dtype == IMC_BF16; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool dims_ok(int64_t a, int64_t b, int64_t c) {
  return a >= 0 && b >= 0 && c >= 0 && a <= kMaxDim && b <= kMaxDim && c <= kMaxDim;
}
bool store_ok(int64_t batch, int64_t rows, int64_t cols) {
  return (double)batch * ((double)rows + 128.0) * ((double)cols + 128.0) < kMaxBytes;
}
// Bytes from the first to the last element of a strided [batch][rows][cols].
uint64_t span(int dtype, int64_t batch, int64_t rows, int64_t cols, int64_t batch_stride,
              int64_t row_stride) {
  if (batch == 0 || rows == 0 || cols == 0) return 0;
  return (uint64_t)((batch - 1) * batch_stride + (rows - 1) * row_stride + cols) *
         dtype_bytes(dtype);
}
// Rows a matrix needs that holds `slots` rows sorted by expert, each expert's
// run starting at a multiple of 128.
int64_t sorted_rows(int64_t slots, int64_t E) {
  return ceil_div(slots + 127 * (slots < E ? slots : E), ATOM_ROWS) * ATOM_ROWS;
}

// Room for M tokens quantised for a product, whichever layout it takes.
size_t tokens_bytes(int64_t M, int64_t K) {
  const int64_t a = store_of(1, M, K).bytes;
  const int64_t b = M > ATOM_ROWS ? store_of(1, M, K, TILES_224).bytes : a;
  return (size_t)(a > b ? a : b);
}

QuantArgs quant_args(const void* x, int64_t batch, int64_t rows, int64_t cols,
                     int64_t batch_stride, int64_t row_stride, bool transpose, void* q) {
  QuantArgs a = {};
  a.x = x;
  a.batch = batch;
  a.rows = rows;
  a.cols = cols;
  a.batch_stride = batch_stride;
  a.row_stride = row_stride;
  a.q = static_cast<uint8_t*>(q);
  a.st = transpose ? store_of(batch, cols, rows) : store_of(batch, rows, cols);
  a.share = 1;
  return a;
}

// A call's scratch: the caller's buffer, or (workspace null) one from the
// library's pool, released on the stream at the end of the call.
struct Scratch {
  void* p = nullptr;
  bool pool = false;
  cudaStream_t s;
  explicit Scratch(cudaStream_t st) : s(st) {}
  int take(void* workspace, size_t need) {
    p = workspace;
    if (workspace || need == 0) return IMC_OK;
    if (scratch_alloc(&p, need, s) != cudaSuccess) return IMC_ERR_CUDA;
    pool = true;
    return IMC_OK;
  }
  cudaError_t give(cudaError_t e) {
    if (!pool) return e;
    const cudaError_t f = cudaFreeAsync(p, s);
    return e != cudaSuccess ? e : f;
  }
};
int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace) return IMC_OK;
  return bytes < need || !aligned(workspace, 16) ? IMC_ERR_ARG : IMC_OK;
}

}  // namespace

extern "C" {

size_t mxfp4_bytes(int64_t batch, int64_t rows, int64_t cols) {
  if (!dims_ok(batch, rows, cols) || !store_ok(batch, rows, cols)) return 0;
  return (size_t)store_of(batch, rows, cols).bytes;
}

int mxfp4_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols,
                   int64_t batch_stride, int64_t row_stride, int transpose, void* q,
                   void* stream) {
  if (!float_type(dtype) || (transpose != 0 && transpose != 1)) return IMC_ERR_ARG;
  if (!dims_ok(batch, rows, cols) || !store_ok(batch, rows, cols) ||
      !store_ok(batch, cols, rows) || row_stride < (rows > 1 ? cols : 0) || batch_stride < 0)
    return IMC_ERR_SHAPE;
  if (batch == 0 || rows == 0 || cols == 0) return finish_empty();
  if (!x || !q) return IMC_ERR_NULL;
  if (!aligned(q, 16) || !aligned(x, (uintptr_t)dtype_bytes(dtype))) return IMC_ERR_ARG;
  const QuantArgs a =
      quant_args(x, batch, rows, cols, batch_stride, row_stride, transpose != 0, q);
  if (ranges_overlap(q, (uint64_t)a.st.bytes, x,
                     span(dtype, batch, rows, cols, batch_stride, row_stride)))
    return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  return finish_call(launch_quantize(a, dtype, transpose != 0, (cudaStream_t)stream),
                     IMC_KERNEL_MXFP4);
}

int mxfp4_dequantize(const void* q, int64_t batch, int64_t rows, int64_t cols, int dtype,
                     void* out, void* stream) {
  if (!float_type(dtype)) return IMC_ERR_ARG;
  if (!dims_ok(batch, rows, cols) || !store_ok(batch, rows, cols)) return IMC_ERR_SHAPE;
  if (batch == 0 || rows == 0 || cols == 0) return finish_empty();
  if (!q || !out) return IMC_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, (uintptr_t)dtype_bytes(dtype))) return IMC_ERR_ARG;
  const Store st = store_of(batch, rows, cols);
  if (ranges_overlap(out, (uint64_t)(batch * rows * cols) * dtype_bytes(dtype), q,
                     (uint64_t)st.bytes))
    return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  return finish_call(launch_dequantize(static_cast<const uint8_t*>(q), st, dtype, out,
                                       (cudaStream_t)stream),
                     IMC_KERNEL_MXFP4);
}

size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t K, int x_dtype) {
  if (x_dtype == IMC_MXFP4 || product_fused(M) || mxfp4_bytes(1, M, K) == 0) return 0;
  return tokens_bytes(M, K);
}

int mxfp4_linear(const void* x, int x_dtype, int64_t row_stride, const void* w, const float* bias,
                 void* out, int out_dtype, int64_t M, int64_t N, int64_t K, int flags,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if ((!float_type(x_dtype) && x_dtype != IMC_MXFP4) || !float_type(out_dtype) ||
      (flags & ~IMC_ACT_RELU))
    return IMC_ERR_ARG;
  const bool raw = x_dtype != IMC_MXFP4;
  if (!dims_ok(M, N, K) || K == 0 || !store_ok(1, M, K) || !store_ok(1, N, K) ||
      (raw && row_stride < (M > 1 ? K : 0)))
    return IMC_ERR_SHAPE;
  if (M == 0 || N == 0) return finish_empty();
  if (!x || !w || !out) return IMC_ERR_NULL;
  if (!aligned(w, 16) || !aligned(out, (uintptr_t)dtype_bytes(out_dtype)) ||
      !aligned(x, raw ? (uintptr_t)dtype_bytes(x_dtype) : 16) || !aligned(bias, 4))
    return IMC_ERR_ARG;
  const uint64_t out_bytes = (uint64_t)M * N * dtype_bytes(out_dtype);
  const uint64_t x_bytes = raw ? span(x_dtype, 1, M, K, 0, row_stride) : mxfp4_bytes(1, M, K);
  const uint64_t w_bytes = mxfp4_bytes(1, N, K);
  if (ranges_overlap(out, out_bytes, x, x_bytes) || ranges_overlap(out, out_bytes, w, w_bytes) ||
      ranges_overlap(out, out_bytes, bias, (uint64_t)N * 4))
    return IMC_ERR_ALIAS;
  const size_t need = mxfp4_linear_workspace_bytes(M, K, x_dtype);
  if (need) {
    const int ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != IMC_OK) return ws;
    if (ranges_overlap(workspace, need, out, out_bytes) ||
        ranges_overlap(workspace, need, x, x_bytes) ||
        ranges_overlap(workspace, need, w, w_bytes) ||
        ranges_overlap(workspace, need, bias, (uint64_t)N * 4))
      return IMC_ERR_ALIAS;
  }
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  if (!product_supported()) return IMC_ERR_DEVICE;
  cudaStream_t s = (cudaStream_t)stream;
  ProductArgs p = {};
  p.x = static_cast<const uint8_t*>(x);
  p.w = static_cast<const uint8_t*>(w);
  p.bias = bias;
  p.out = out;
  p.out_dtype = out_dtype;
  p.relu = flags & IMC_ACT_RELU ? 1 : 0;
  p.M = p.x_rows = M;
  p.N = N;
  p.K = K;
  p.x_shift = 7;
  Scratch sc(s);
  cudaError_t e = cudaSuccess;
  if (raw && need == 0) {
    p.raw = x;
    p.raw_dtype = x_dtype;
    p.raw_stride = row_stride;
    p.share = 1;
  } else if (raw) {
    if (sc.take(workspace, need) != IMC_OK) return IMC_ERR_CUDA;
    QuantArgs a = quant_args(x, 1, M, K, 0, row_stride, false, sc.p);
    p.x_shift = product_atom_shift(M, N, K);
    a.st = store_of(1, M, K, p.x_shift);
    e = launch_quantize(a, x_dtype, false, s);
    p.x = static_cast<const uint8_t*>(sc.p);
    p.inputs_ready = true;
  }
  if (e == cudaSuccess) e = launch_product(p, s);
  return finish_call(sc.give(e), IMC_KERNEL_MXFP4);
}

size_t mxfp4_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!dims_ok(M, N, K) || !store_ok(1, M, N) || !store_ok(1, K, N) || !store_ok(1, K, M)) return 0;
  const int64_t sizes[4] = {(int64_t)tokens_bytes(M, N), store_of(1, K, N).bytes,
                            (int64_t)tokens_bytes(N, M), store_of(1, K, M).bytes};
  int64_t sum = 0;
  for (int64_t v : sizes) sum += ceil_div(v, 512) * 512;
  return (size_t)sum;
}

int mxfp4_linear_backward(const void* grad, const void* x, const void* w, int dtype,
                          int64_t M, int64_t N, int64_t K, void* grad_x, void* grad_w,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!float_type(dtype)) return IMC_ERR_ARG;
  if (!dims_ok(M, N, K) || !store_ok(1, M, N) || !store_ok(1, K, N) || !store_ok(1, K, M) ||
      M == 0 || N == 0 || K == 0)
    return IMC_ERR_SHAPE;
  if (!grad_x && !grad_w) return finish_empty();
  if (!grad || (grad_x && !w) || (grad_w && !x)) return IMC_ERR_NULL;
  const uint64_t b = (uint64_t)dtype_bytes(dtype);
  if (!aligned(grad, b) || !aligned(x, b) || !aligned(w, b) || !aligned(grad_x, b) ||
      !aligned(grad_w, b))
    return IMC_ERR_ARG;
  const void* in[3] = {grad, grad_w ? x : nullptr, grad_x ? w : nullptr};
  const uint64_t in_bytes[3] = {(uint64_t)M * N * b, (uint64_t)M * K * b, (uint64_t)N * K * b};
  const uint64_t gx = (uint64_t)M * K * b, gw = (uint64_t)N * K * b;
  const size_t need = mxfp4_linear_backward_workspace_bytes(M, N, K);
  const int ws = check_workspace(workspace, workspace_bytes, need);
  if (ws != IMC_OK) return ws;
  for (int i = 0; i < 3; ++i)
    if (ranges_overlap(grad_x, gx, in[i], in_bytes[i]) ||
        ranges_overlap(grad_w, gw, in[i], in_bytes[i]) ||
        ranges_overlap(workspace, need, in[i], in_bytes[i]))
      return IMC_ERR_ALIAS;
  if (ranges_overlap(grad_x, gx, grad_w, gw) || ranges_overlap(workspace, need, grad_x, gx) ||
      ranges_overlap(workspace, need, grad_w, gw))
    return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  if (!product_supported()) return IMC_ERR_DEVICE;
  cudaStream_t s = (cudaStream_t)stream;
  Scratch sc(s);
  if (sc.take(workspace, need) != IMC_OK) return IMC_ERR_CUDA;
  // grad along its rows and, transposed, along its columns: read once for both
  uint8_t* at = static_cast<uint8_t*>(sc.p);
  auto room = [&](int64_t bytes) {
    uint8_t* q = at;
    at += ceil_div(bytes, 512) * 512;
    return q;
  };
  uint8_t *g_rows = room((int64_t)tokens_bytes(M, N)), *g_cols = room((int64_t)tokens_bytes(N, M)),
          *w_cols = room(store_of(1, K, N).bytes), *x_cols = room(store_of(1, K, M).bytes);
  // grad's rows are the tokens of the first product, its columns of the second
  const int shift_x = product_atom_shift(M, K, N), shift_w = product_atom_shift(N, K, M);
  cudaError_t e;
  if (grad_w) {
    QuantArgs a = quant_args(grad, 1, M, N, 0, N, true, g_cols);
    a.st = store_of(1, N, M, shift_w);
    a.q_rows = grad_x ? g_rows : nullptr;
    a.st_rows = store_of(1, M, N, shift_x);
    e = launch_quantize(a, dtype, true, s);
  } else {
    QuantArgs a = quant_args(grad, 1, M, N, 0, N, false, g_rows);
    a.st = store_of(1, M, N, shift_x);
    e = launch_quantize(a, dtype, false, s);
  }
  // out[rows, cols]: the contraction of two operands quantised along `depth`
  auto product = [&](const uint8_t* a, int shift, int64_t rows, const uint8_t* c, int64_t cols,
                     int64_t depth, void* out) {
    ProductArgs p = {};
    p.x = a;
    p.x_shift = shift;
    p.w = c;
    p.out = out;
    p.out_dtype = dtype;
    p.M = p.x_rows = rows;
    p.N = cols;
    p.K = depth;
    if (e == cudaSuccess) e = launch_product(p, s);
  };
  const QuantArgs w_args = quant_args(w, 1, N, K, 0, K, true, w_cols),
                  x_args = quant_args(x, 1, M, K, 0, K, true, x_cols);
  if (e == cudaSuccess)
    e = grad_x && grad_w ? launch_quantize_two(w_args, x_args, dtype, s)
                         : launch_quantize(grad_x ? w_args : x_args, dtype, true, s);
  if (grad_x) product(g_rows, shift_x, M, w_cols, K, N, grad_x);  // grad [M,N] . w [N,K]
  if (grad_w) product(g_cols, shift_w, N, x_cols, K, M, grad_w);  // grad^T [N,M] . x [M,K]
  return finish_call(sc.give(e), IMC_KERNEL_MXFP4);
}

}  // extern "C"

namespace {
bool route_dims_ok(int64_t T, int64_t E, int64_t k) {
  return T >= 0 && E >= 1 && E <= kMaxExperts && k >= 1 && k <= kMaxChosen && k <= E &&
         T * k <= kMaxDim - 1;
}
}  // namespace

extern "C" {

int moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t row_stride,
              const float* bias, int64_t k, int score, int64_t groups, int64_t top_groups,
              int renormalize, double scale, float* weights, int32_t* experts, void* stream) {
  if (!float_type(dtype) || (score != IMC_SCORE_SOFTMAX && score != IMC_SCORE_SIGMOID) ||
      (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
    return IMC_ERR_ARG;
  if (T < 0 || T > kMaxDim || !route_dims_ok(T, E, k) || row_stride < (T > 1 ? E : 0) ||
      groups < 1 || groups > kMaxGroups || E % groups != 0 || top_groups < 1 ||
      top_groups > groups || k > E / groups * top_groups)
    return IMC_ERR_SHAPE;
  if (T == 0) return finish_empty();
  if (!logits || !weights || !experts) return IMC_ERR_NULL;
  if (!aligned(logits, (uintptr_t)dtype_bytes(dtype)) || !aligned(weights, 4) ||
      !aligned(experts, 4) || !aligned(bias, 4))
    return IMC_ERR_ARG;
  const uint64_t in = span(dtype, 1, T, E, 0, row_stride), slots = (uint64_t)(T * k) * 4;
  if (ranges_overlap(weights, slots, logits, in) || ranges_overlap(experts, slots, logits, in) ||
      ranges_overlap(weights, slots, bias, (uint64_t)E * 4) ||
      ranges_overlap(experts, slots, bias, (uint64_t)E * 4) ||
      ranges_overlap(weights, slots, experts, slots))
    return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  RouteArgs a = {};
  a.logits = logits;
  a.T = T;
  a.ld = row_stride;
  a.E = (int)E;
  a.k = (int)k;
  a.groups = (int)groups;
  a.top_groups = (int)top_groups;
  a.size = (int)(E / groups);
  a.inv_size = (uint32_t)(((1 << 20) + a.size - 1) / a.size);
  a.sigmoid = score == IMC_SCORE_SIGMOID ? 1 : 0;
  a.renorm = renormalize;
  a.scale = (float)scale;
  a.bias = bias;
  a.weights = weights;
  a.experts = experts;
  return finish_call(launch_route(a, dtype, (cudaStream_t)stream), IMC_KERNEL_EXPERTS);
}

int moe_route_backward(const float* grad_weights, const void* logits, int dtype, int64_t T,
                       int64_t E, int64_t row_stride, const int32_t* experts, int64_t k, int score,
                       int renormalize, double scale, void* grad_logits, void* stream) {
  if (!float_type(dtype) || (score != IMC_SCORE_SOFTMAX && score != IMC_SCORE_SIGMOID) ||
      (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
    return IMC_ERR_ARG;
  if (T < 0 || T > kMaxDim || !route_dims_ok(T, E, k) || row_stride < (T > 1 ? E : 0))
    return IMC_ERR_SHAPE;
  if (T == 0) return finish_empty();
  if (!grad_weights || !logits || !experts || !grad_logits) return IMC_ERR_NULL;
  const uint64_t b = (uint64_t)dtype_bytes(dtype);
  if (!aligned(logits, b) || !aligned(grad_logits, b) || !aligned(grad_weights, 4) ||
      !aligned(experts, 4))
    return IMC_ERR_ARG;
  const uint64_t out = (uint64_t)(T * E) * b, slots = (uint64_t)(T * k) * 4;
  if (ranges_overlap(grad_logits, out, logits, span(dtype, 1, T, E, 0, row_stride)) ||
      ranges_overlap(grad_logits, out, grad_weights, slots) ||
      ranges_overlap(grad_logits, out, experts, slots))
    return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  RouteArgs a = {};
  a.logits = logits;
  a.T = T;
  a.ld = row_stride;
  a.E = (int)E;
  a.k = (int)k;
  a.sigmoid = score == IMC_SCORE_SIGMOID ? 1 : 0;
  a.renorm = renormalize;
  a.scale = (float)scale;
  a.experts = const_cast<int32_t*>(experts);
  return finish_call(launch_route_backward(a, dtype, grad_weights, grad_logits,
                                           (cudaStream_t)stream),
                     IMC_KERNEL_EXPERTS);
}

int64_t moe_layout_size(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || T > kMaxDim || E < 1 || E > kMaxExperts || k < 1 || k > kMaxChosen ||
      T * k > kMaxDim - 1)
    return 0;
  const int64_t n = T * k, ctas = layout_ctas(n);
  if (sorted_at(sorted_rows(n, E), TILES_224) > kMaxDim) return 0;  // places are 32-bit
  return 2 * E + 3 + 3 * n + (ctas > 1 ? ctas * (E + 1) : 0);
}

int moe_layout(const int32_t* experts, int64_t T, int64_t k, int64_t E, int32_t* layout,
               void* stream) {
  const int64_t size = moe_layout_size(T, k, E);
  if (size == 0) return IMC_ERR_SHAPE;
  const int64_t n = T * k;
  if (!layout || (n > 0 && !experts)) return IMC_ERR_NULL;
  if (!aligned(layout, 4) || !aligned(experts, 4)) return IMC_ERR_ARG;
  if (ranges_overlap(layout, (uint64_t)size * 4, experts, (uint64_t)n * 4)) return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  int32_t *offsets = layout, *starts = offsets + E + 2, *order = starts + E + 1, *dest = order + n;
  return finish_call(launch_layout(experts, (int)n, (int)E, offsets, starts, order, dest,
                                   dest + n, dest + 2 * n, (cudaStream_t)stream),
                     IMC_KERNEL_EXPERTS);
}

size_t mxfp4_experts_linear_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t K) {
  if (moe_layout_size(T, k, E) == 0 || T == 0) return 0;
  if (experts_fused(T * k, E)) return 0;
  const int64_t rows = sorted_rows(T * k, E);
  if (rows > kMaxDim / 2 || !dims_ok(0, 0, K) || !store_ok(4, rows, K)) return 0;
  const int shift = experts_atom_shift(T * k, E);
  return (size_t)store_of(1, sorted_at(rows, shift), K, shift).bytes;
}

int mxfp4_experts_linear(const void* x, int x_dtype, int64_t x_rows, int64_t row_stride,
                         const void* w, const float* bias, const int32_t* layout, void* out,
                         int out_dtype, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K,
                         int flags, void* workspace, size_t workspace_bytes, void* stream) {
  if (!float_type(x_dtype) || !float_type(out_dtype) || (flags & ~IMC_ACT_RELU)) return IMC_ERR_ARG;
  const int64_t size = moe_layout_size(T, k, E), n = T * k;
  if (size == 0 || !dims_ok(x_rows, N, K) || K == 0 || (x_rows != T && x_rows != n) ||
      row_stride < (x_rows > 1 ? K : 0) || sorted_rows(n, E) > kMaxDim / 2 ||
      !store_ok(4, sorted_rows(n, E), K) || !store_ok(E, N, K))
    return IMC_ERR_SHAPE;
  if (T == 0 || N == 0) return finish_empty();
  if (!x || !w || !layout || !out) return IMC_ERR_NULL;
  if (!aligned(w, 16) || !aligned(out, (uintptr_t)dtype_bytes(out_dtype)) ||
      !aligned(x, (uintptr_t)dtype_bytes(x_dtype)) || !aligned(bias, 4) || !aligned(layout, 4))
    return IMC_ERR_ARG;
  const uint64_t out_bytes = (uint64_t)n * N * dtype_bytes(out_dtype);
  const size_t need = mxfp4_experts_linear_workspace_bytes(T, k, E, K);
  const int ws = check_workspace(workspace, workspace_bytes, need);
  if (ws != IMC_OK) return ws;
  const void* in[4] = {x, w, bias, layout};
  const uint64_t in_bytes[4] = {span(x_dtype, 1, x_rows, K, 0, row_stride), mxfp4_bytes(E, N, K),
                                (uint64_t)E * N * 4, (uint64_t)size * 4};
  for (int i = 0; i < 4; ++i)
    if (ranges_overlap(out, out_bytes, in[i], in_bytes[i]) ||
        ranges_overlap(workspace, need, in[i], in_bytes[i]))
      return IMC_ERR_ALIAS;
  if (ranges_overlap(workspace, need, out, out_bytes)) return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  if (!product_supported()) return IMC_ERR_DEVICE;
  cudaStream_t s = (cudaStream_t)stream;
  ProductArgs p = {};
  p.w = static_cast<const uint8_t*>(w);
  p.bias = bias;
  p.out = out;
  p.out_dtype = out_dtype;
  p.relu = flags & IMC_ACT_RELU ? 1 : 0;
  p.N = N;
  p.K = K;
  p.E = (int)E;
  p.slots = (int)n;
  p.offsets = layout;
  p.starts = layout + E + 2;
  p.order = p.starts + E + 1;
  const int shift = experts_atom_shift(n, E);
  p.x_rows = sorted_at(sorted_rows(n, E), shift);
  if (need == 0) {
    p.raw = x;
    p.raw_dtype = x_dtype;
    p.raw_stride = row_stride;
    p.share = x_rows == n ? 1 : (int)k;
    return finish_call(launch_product(p, s), IMC_KERNEL_MXFP4);
  }
  Scratch sc(s);
  if (sc.take(workspace, need) != IMC_OK) return IMC_ERR_CUDA;
  p.x = static_cast<const uint8_t*>(sc.p);
  QuantArgs qa = quant_args(x, 1, x_rows, K, 0, row_stride, false, sc.p);
  qa.st = store_of(1, p.x_rows, K, shift);
  qa.dest = p.order + (shift == TILES_224 ? 2 * n : n);
  qa.share = x_rows == n ? 1 : (int)k;
  cudaError_t e = launch_quantize(qa, x_dtype, false, s);
  p.inputs_ready = true;
  if (e == cudaSuccess) e = launch_product(p, s);
  return finish_call(sc.give(e), IMC_KERNEL_MXFP4);
}

size_t mxfp4_experts_weight_grad_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N,
                                                 int64_t K) {
  if (moe_layout_size(T, k, E) == 0 || T == 0 || !dims_ok(0, N, K)) return 0;
  const int64_t rows = sorted_rows(T * k, E);
  if (rows > kMaxDim || !store_ok(1, N, rows) || !store_ok(1, K, rows)) return 0;
  return (size_t)(ceil_div(store_of(1, N, rows).bytes, 512) * 512 + store_of(1, K, rows).bytes);
}

int mxfp4_experts_weight_grad(const void* grad, const void* x, int dtype, int64_t x_rows,
                              const int32_t* layout, void* grad_w, int64_t T, int64_t k, int64_t E,
                              int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (!float_type(dtype)) return IMC_ERR_ARG;
  const int64_t size = moe_layout_size(T, k, E), n = T * k;
  if (size == 0 || T == 0 || !dims_ok(x_rows, N, K) || N == 0 || K == 0 ||
      (x_rows != T && x_rows != n) || sorted_rows(n, E) > kMaxDim ||
      !store_ok(1, N, sorted_rows(n, E)) || !store_ok(1, K, sorted_rows(n, E)) ||
      (double)E * N * K > kMaxBytes)
    return IMC_ERR_SHAPE;
  if (!grad || !x || !layout || !grad_w) return IMC_ERR_NULL;
  const uint64_t b = (uint64_t)dtype_bytes(dtype);
  if (!aligned(grad, b) || !aligned(x, b) || !aligned(grad_w, b) || !aligned(layout, 4))
    return IMC_ERR_ARG;
  const size_t need = mxfp4_experts_weight_grad_workspace_bytes(T, k, E, N, K);
  const int ws = check_workspace(workspace, workspace_bytes, need);
  if (ws != IMC_OK) return ws;
  const uint64_t out_bytes = (uint64_t)E * N * K * b;
  const void* in[3] = {grad, x, layout};
  const uint64_t in_bytes[3] = {(uint64_t)n * N * b, (uint64_t)x_rows * K * b, (uint64_t)size * 4};
  for (int i = 0; i < 3; ++i)
    if (ranges_overlap(grad_w, out_bytes, in[i], in_bytes[i]) ||
        ranges_overlap(workspace, need, in[i], in_bytes[i]))
      return IMC_ERR_ALIAS;
  if (ranges_overlap(workspace, need, grad_w, out_bytes)) return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  if (!product_supported()) return IMC_ERR_DEVICE;
  cudaStream_t s = (cudaStream_t)stream;
  Scratch sc(s);
  if (sc.take(workspace, need) != IMC_OK) return IMC_ERR_CUDA;
  const int64_t rows = sorted_rows(n, E);
  uint8_t* g_cols = static_cast<uint8_t*>(sc.p);
  uint8_t* x_cols = g_cols + ceil_div(store_of(1, N, rows).bytes, 512) * 512;
  auto quantize = [&](const void* src, int64_t cols, int share, uint8_t* q) {
    QuantArgs a = quant_args(src, 1, rows, cols, 0, cols, true, q);
    a.offsets = layout;
    a.starts = layout + E + 2;
    a.order = a.starts + E + 1;
    a.E = (int)E;
    a.share = share;
    return launch_quantize(a, dtype, true, s);
  };
  cudaError_t e = quantize(grad, N, 1, g_cols);
  if (e == cudaSuccess) e = quantize(x, K, x_rows == n ? 1 : (int)k, x_cols);
  ProductArgs p = {};
  p.x = g_cols;
  p.w = x_cols;
  p.out = grad_w;
  p.out_dtype = dtype;
  p.x_shift = 7;
  p.M = p.x_rows = N;
  p.N = K;
  p.K = rows;
  p.E = (int)E;
  p.starts = layout + E + 2;
  p.groups = true;
  if (e == cudaSuccess) e = launch_product(p, s);
  return finish_call(sc.give(e), IMC_KERNEL_MXFP4);
}

}  // extern "C"

namespace {
int combine_call(const void* y, int dtype, const float* weights, int64_t T, int64_t k, int64_t N,
                 void* out, int out_dtype, void* stream) {
  if (!float_type(dtype) || !float_type(out_dtype)) return IMC_ERR_ARG;
  if (!dims_ok(T, k, N) || k < 1 || k > kMaxChosen || (double)T * k * N > kMaxBytes)
    return IMC_ERR_SHAPE;
  if (T == 0 || N == 0) return finish_empty();
  if (!y || !out) return IMC_ERR_NULL;
  const uint64_t b = (uint64_t)dtype_bytes(dtype), ob = (uint64_t)dtype_bytes(out_dtype);
  const uint64_t out_bytes = (uint64_t)T * N * ob;
  if (!aligned(y, b) || !aligned(out, ob) || !aligned(weights, 4)) return IMC_ERR_ARG;
  if (ranges_overlap(out, out_bytes, y, (uint64_t)T * k * N * b) ||
      ranges_overlap(out, out_bytes, weights, (uint64_t)T * k * 4))
    return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  return finish_call(launch_combine(y, weights, dtype, T, (int)k, N, out, out_dtype,
                                    (cudaStream_t)stream),
                     IMC_KERNEL_EXPERTS);
}
}  // namespace

extern "C" {

int moe_combine(const void* y, int dtype, const float* weights, int64_t T, int64_t k, int64_t N,
                void* out, void* stream) {
  return combine_call(y, dtype, weights, T, k, N, out, dtype, stream);
}

int moe_combine_f32(const float* y, const float* weights, int64_t T, int64_t k, int64_t N, void* out,
                    int out_dtype, void* stream) {
  return combine_call(y, IMC_F32, weights, T, k, N, out, out_dtype, stream);
}

int moe_combine_backward(const void* grad, const void* y, int dtype, const float* weights,
                         int64_t T, int64_t k, int64_t N, void* grad_y, float* grad_weights,
                         void* stream) {
  if (!float_type(dtype)) return IMC_ERR_ARG;
  if (!dims_ok(T, k, N) || k < 1 || k > kMaxChosen || (double)T * k * N > kMaxBytes)
    return IMC_ERR_SHAPE;
  if (T == 0) return finish_empty();
  if (!weights || !grad_weights || (N > 0 && (!grad || !y || !grad_y))) return IMC_ERR_NULL;
  const uint64_t b = (uint64_t)dtype_bytes(dtype);
  if (!aligned(grad, b) || !aligned(y, b) || !aligned(grad_y, b) || !aligned(weights, 4) ||
      !aligned(grad_weights, 4))
    return IMC_ERR_ARG;
  const uint64_t y_bytes = (uint64_t)T * k * N * b, w_bytes = (uint64_t)T * k * 4;
  const void* in[3] = {grad, y, weights};
  const uint64_t in_bytes[3] = {(uint64_t)T * N * b, y_bytes, w_bytes};
  for (int i = 0; i < 3; ++i)
    if (ranges_overlap(grad_y, y_bytes, in[i], in_bytes[i]) ||
        ranges_overlap(grad_weights, w_bytes, in[i], in_bytes[i]))
      return IMC_ERR_ALIAS;
  if (ranges_overlap(grad_y, y_bytes, grad_weights, w_bytes)) return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  return finish_call(launch_combine_backward(grad, y, weights, dtype, T, (int)k, N, grad_y,
                                             grad_weights, (cudaStream_t)stream),
                     IMC_KERNEL_EXPERTS);
}

}  // extern "C"

namespace {
constexpr int64_t kMaxRows = 1 << 27, kMaxWidth = 1 << 20;  // grids stay below 2^31 blocks

bool adapter_dims_ok(int64_t T, int64_t L, int64_t r, int64_t K, int64_t N) {
  return T >= 0 && T <= kMaxRows && L >= 1 && L <= kMaxExperts && r >= 1 && r <= kMaxRank &&
         K >= 1 && K <= kMaxWidth && N >= 0 && N <= kMaxWidth && (double)T * K < kMaxBytes && (double)T * N < kMaxBytes &&
         (double)L * r * K < kMaxBytes && (double)L * r * N < kMaxBytes;
}
struct Range {
  const void* p;
  uint64_t bytes;
};
bool overlaps_any(const Range& out, const Range* in, int n) {
  for (int i = 0; i < n; ++i)
    if (ranges_overlap(out.p, out.bytes, in[i].p, in[i].bytes)) return true;
  return false;
}
}  // namespace

extern "C" {

size_t lowrank_linear_workspace_bytes(int64_t T, int64_t L, int64_t r) {
  if (T < 1 || T > kMaxRows || L < 1 || L > kMaxExperts || r < 1 || r > kMaxRank) return 0;
  return adapters_bytes(T, L, r);
}

int lowrank_linear(const void* x, int dtype, int64_t row_stride, const void* a, const void* b,
                    const float* scale, const int32_t* layout, const void* base, void* out,
                    int64_t T, int64_t L, int64_t r, int64_t K, int64_t N, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!float_type(dtype)) return IMC_ERR_ARG;
  if (!adapter_dims_ok(T, L, r, K, N) || row_stride < (T > 1 ? K : 0)) return IMC_ERR_SHAPE;
  if (T == 0 || N == 0) return finish_empty();
  if (!x || !a || !b || !layout || !out) return IMC_ERR_NULL;
  const uint64_t e = (uint64_t)dtype_bytes(dtype);
  if (!aligned(x, e) || !aligned(a, e) || !aligned(b, e) || !aligned(scale, 4) ||
      !aligned(layout, 4) || !aligned(base, e) || !aligned(out, e))
    return IMC_ERR_ARG;
  const uint64_t out_bytes = (uint64_t)T * N * e;
  const Range in[6] = {{x, span(dtype, 1, T, K, 0, row_stride)},
                       {a, (uint64_t)L * r * K * e},
                       {b, (uint64_t)L * N * r * e},
                       {scale, (uint64_t)L * 4},
                       {layout, (uint64_t)moe_layout_size(T, 1, L) * 4},
                       {base == out ? nullptr : base, out_bytes}};
  if (overlaps_any({out, out_bytes}, in, 6)) return IMC_ERR_ALIAS;
  const size_t need = lowrank_linear_workspace_bytes(T, L, r);
  if (need) {
    const int ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != IMC_OK) return ws;
    const Range room = {workspace, need}, res[2] = {{base, out_bytes}, {out, out_bytes}};
    if (workspace && (overlaps_any(room, in, 5) || overlaps_any(room, res, 2))) return IMC_ERR_ALIAS;
  }
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  cudaStream_t s = (cudaStream_t)stream;
  Scratch sc(s);
  if (sc.take(workspace, need) != IMC_OK) return IMC_ERR_CUDA;
  AdapterArgs p = {};
  p.workspace = sc.p;
  p.x = x;
  p.ld = row_stride;
  p.a = a;
  p.b = b;
  p.scale = scale;
  p.offsets = layout;
  p.order = layout + 2 * L + 3;
  p.base = base;
  p.out = out;
  p.T = T;
  p.K = K;
  p.N = N;
  p.L = (int)L;
  p.r = (int)r;
  return finish_call(sc.give(launch_adapters(p, dtype, s)), IMC_KERNEL_ADAPTERS);
}

size_t lowrank_linear_backward_workspace_bytes(int64_t T, int64_t r) {
  if (T < 1 || T > kMaxRows || r < 1 || r > kMaxRank) return 0;
  return adapters_backward_bytes(T, r);
}

int lowrank_linear_backward(const void* grad, const void* x, const void* a, const void* b,
                             int dtype, const float* scale, const int32_t* layout,
                             const void* base, void* grad_x, void* grad_a, void* grad_b, int64_t T,
                             int64_t L, int64_t r, int64_t K, int64_t N, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (!float_type(dtype)) return IMC_ERR_ARG;
  if (!adapter_dims_ok(T, L, r, K, N) || T == 0 || N == 0) return IMC_ERR_SHAPE;
  if (!grad_x && !grad_a && !grad_b) return finish_empty();
  if (!grad || !x || !a || !b || !layout) return IMC_ERR_NULL;
  const uint64_t e = (uint64_t)dtype_bytes(dtype);
  if (!aligned(grad, e) || !aligned(x, e) || !aligned(a, e) || !aligned(b, e) ||
      !aligned(scale, 4) || !aligned(layout, 4) || !aligned(base, e) || !aligned(grad_x, e) ||
      !aligned(grad_a, e) || !aligned(grad_b, e))
    return IMC_ERR_ARG;
  const size_t need = lowrank_linear_backward_workspace_bytes(T, r);
  const int ws = check_workspace(workspace, workspace_bytes, need);
  if (ws != IMC_OK) return ws;
  const uint64_t row_bytes = (uint64_t)T * K * e;
  const Range in[7] = {{grad, (uint64_t)T * N * e},
                       {x, row_bytes},
                       {a, (uint64_t)L * r * K * e},
                       {b, (uint64_t)L * N * r * e},
                       {scale, (uint64_t)L * 4},
                       {layout, (uint64_t)moe_layout_size(T, 1, L) * 4},
                       {base, grad_x ? row_bytes : 0}};
  const Range out[4] = {{grad_x, row_bytes},
                        {grad_a, (uint64_t)L * r * K * e},
                        {grad_b, (uint64_t)L * N * r * e},
                        {workspace, need}};
  for (int i = 0; i < 4; ++i) {
    const bool in_place = i == 0 && base == grad_x;
    if (out[i].p && (overlaps_any(out[i], in, in_place ? 6 : 7) || overlaps_any(out[i], out, i)))
      return IMC_ERR_ALIAS;
  }
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  cudaStream_t s = (cudaStream_t)stream;
  Scratch sc(s);
  if (sc.take(workspace, need) != IMC_OK) return IMC_ERR_CUDA;
  AdapterGradArgs p = {};
  p.grad = grad;
  p.x = x;
  p.a = a;
  p.b = b;
  p.scale = scale;
  p.offsets = layout;
  p.order = layout + 2 * L + 3;
  p.base = base;
  p.grad_x = grad_x;
  p.grad_a = grad_a;
  p.grad_b = grad_b;
  p.T = T;
  p.K = K;
  p.N = N;
  p.L = (int)L;
  p.r = (int)r;
  p.workspace = sc.p;
  return finish_call(sc.give(launch_adapters_backward(p, dtype, s)), IMC_KERNEL_ADAPTERS);
}

}  // extern "C"

namespace {
// What moe_balance and its gradient have in common; IMC_OK or the status.
int balance_args(BalanceArgs& p, const void* logits, int dtype, int64_t T, int64_t E,
                 int64_t row_stride, const int32_t* experts, int64_t k, int score,
                 const int32_t* offsets, int64_t S) {
  if (!float_type(dtype) || (score != IMC_SCORE_SOFTMAX && score != IMC_SCORE_SIGMOID))
    return IMC_ERR_ARG;
  if (T < 0 || T > kMaxRows || !route_dims_ok(T, E, k) || row_stride < (T > 1 ? E : 0) || S < 0 ||
      S > kMaxRows || S * E > kMaxDim || (!offsets && S != 1))
    return IMC_ERR_SHAPE;
  if (!aligned(logits, (uintptr_t)dtype_bytes(dtype)) || !aligned(experts, 4) ||
      !aligned(offsets, 4))
    return IMC_ERR_ARG;
  p = {};
  p.logits = logits;
  p.T = T;
  p.ld = row_stride;
  p.E = (int)E;
  p.k = (int)k;
  p.S = (int)S;
  p.sigmoid = score == IMC_SCORE_SIGMOID ? 1 : 0;
  p.experts = experts;
  p.offsets = offsets;
  return IMC_OK;
}
}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(int64_t T, int64_t S, int64_t E) {
  if (T < 0 || T > kMaxRows || S < 1 || S > kMaxRows || E < 1 || E > kMaxExperts || S * E > kMaxDim)
    return 0;
  return balance_bytes(T, S, E);
}

int moe_balance(const void* logits, int dtype, int64_t T, int64_t E, int64_t row_stride,
                const int32_t* experts, int64_t k, int score, const int32_t* offsets, int64_t S,
                float* loss, int32_t* counts, void* workspace, size_t workspace_bytes,
                void* stream) {
  BalanceArgs p;
  const int rc = balance_args(p, logits, dtype, T, E, row_stride, experts, k, score, offsets, S);
  if (rc != IMC_OK) return rc;
  if (S == 0) return finish_empty();
  if ((T > 0 && (!logits || !experts)) || !loss || !counts) return IMC_ERR_NULL;
  if (!aligned(loss, 4) || !aligned(counts, 4)) return IMC_ERR_ARG;
  const Range in[3] = {{logits, span(dtype, 1, T, E, 0, row_stride)},
                       {experts, (uint64_t)(T * k) * 4},
                       {offsets, (uint64_t)(S + 1) * 4}};
  const Range out[2] = {{loss, (uint64_t)S * 4}, {counts, (uint64_t)(S * E) * 4}};
  if (overlaps_any(out[0], in, 3) || overlaps_any(out[1], in, 3) || overlaps_any(out[1], out, 1))
    return IMC_ERR_ALIAS;
  const size_t need = moe_balance_workspace_bytes(T, S, E);
  if (need) {
    const int ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != IMC_OK) return ws;
    const Range room = {workspace, need};
    if (workspace && (overlaps_any(room, in, 3) || overlaps_any(room, out, 2))) return IMC_ERR_ALIAS;
  }
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  cudaStream_t s = (cudaStream_t)stream;
  Scratch sc(s);
  if (sc.take(workspace, need) != IMC_OK) return IMC_ERR_CUDA;
  p.workspace = sc.p;
  p.loss = loss;
  p.counts = counts;
  return finish_call(sc.give(launch_balance(p, dtype, s)), IMC_KERNEL_EXPERTS);
}

int moe_balance_backward(const float* grad_loss, const void* logits, int dtype, int64_t T,
                         int64_t E, int64_t row_stride, const int32_t* experts, int64_t k,
                         int score, const int32_t* counts, const int32_t* offsets, int64_t S,
                         const float* grad_weights, int renormalize, double scale,
                         void* grad_logits, void* stream) {
  BalanceArgs p;
  const int rc = balance_args(p, logits, dtype, T, E, row_stride, experts, k, score, offsets, S);
  if (rc != IMC_OK) return rc;
  if ((renormalize != 0 && renormalize != 1) || !std::isfinite(scale)) return IMC_ERR_ARG;
  if (T == 0) return finish_empty();
  if (!logits || !grad_logits || (S > 0 && (!grad_loss || !counts)) || (grad_weights && !experts))
    return IMC_ERR_NULL;
  const uint64_t b = (uint64_t)dtype_bytes(dtype);
  if (!aligned(grad_loss, 4) || !aligned(counts, 4) || !aligned(grad_weights, 4) ||
      !aligned(grad_logits, b))
    return IMC_ERR_ARG;
  const Range in[6] = {{logits, span(dtype, 1, T, E, 0, row_stride)},
                       {experts, (uint64_t)(T * k) * 4},
                       {offsets, (uint64_t)(S + 1) * 4},
                       {grad_loss, (uint64_t)S * 4},
                       {counts, (uint64_t)(S * E) * 4},
                       {grad_weights, (uint64_t)(T * k) * 4}};
  if (overlaps_any({grad_logits, (uint64_t)(T * E) * b}, in, 6)) return IMC_ERR_ALIAS;
  const int dev = require_device();
  if (dev != IMC_OK) return dev;
  p.grad_loss = grad_loss;
  p.counts = const_cast<int32_t*>(counts);
  p.grad_weights = grad_weights;
  p.renorm = renormalize;
  p.scale = (float)scale;
  p.grad = grad_logits;
  return finish_call(launch_balance_backward(p, dtype, (cudaStream_t)stream), IMC_KERNEL_EXPERTS);
}

}  // extern "C"
