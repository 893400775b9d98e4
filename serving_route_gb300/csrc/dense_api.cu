// dense_api.cu -- the calls of the dense products (include/megamoe.h): argument checks,
// workspaces, and the launches of dense.cu.
#include <cstring>
#include <new>

#include "dense.h"
#include "internal.h"

using namespace mm;

struct moe_fp8_linear_handle {
  int rows, cols, device, sms;
  int64_t max_tokens;
  bool withhold;
  const uint8_t* codes;
  uint32_t* status;
  uint8_t* sb;   // E8M0 scales of the weight blocks
  uint8_t* xq;   // rows of x quantised within the call
  uint8_t* xs;
};

struct moe_mlp_handle {
  int hidden, inter, device, sms;
  DenseType type;
  DenseAct act;
  int64_t max_tokens;
  bool withhold, withhold_last;
  const void *w1, *w2;
  uint32_t* status;
  void* h;       // [max_tokens, inter]
  void* dgu;     // [max_tokens, 2 inter]
};

namespace {

constexpr size_t kAlign = 1024;
constexpr int64_t kMaxTokens = 1 << 24;

size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }
uint8_t* aligned(void* p) { return reinterpret_cast<uint8_t*>(((uintptr_t)p + kAlign - 1) / kAlign * kAlign); }
bool off(const void* p, size_t a) { return !p || (uintptr_t)p % a != 0; }

moe_status this_device(int* device, int* sms) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;  // built for sm_103a only
  *device = dev;
  return dense_set_attributes() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Launches go to the current device: it has to be the handle's.
bool elsewhere(int device) {
  int dev = -1;
  return cudaGetDevice(&dev) != cudaSuccess || dev != device;
}

// The bytes from the first of `rows` rows to the last one's end.
struct Span {
  uintptr_t a, b;
  Span(const void* p, int64_t rows, int64_t ld, int64_t cols, size_t size)
      : a((uintptr_t)p), b(p && rows ? a + ((rows - 1) * ld + cols) * size : a) {}
  bool meets(const Span& o) const { return a < b && o.a < o.b && a < o.b && o.a < b; }  // (an empty one nothing)
};

moe_status read_word(const uint32_t* d_status, uint32_t* h_status, cudaStream_t stream) {
  if (cudaMemcpyAsync(h_status, d_status, 4, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

// The status word since it was last read; a handle whose kernel gave up a wait starts afresh.
moe_status read_status(uint32_t* d_status, uint32_t* h_status, cudaStream_t stream) {
  const moe_status st = read_word(d_status, h_status, stream);
  if (st != MOE_OK || !*h_status) return st;
  if (cudaMemsetAsync(d_status, 0, kAlign, stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_ERR_DEVICE_TIMEOUT;
}

struct LinearLayout {
  size_t sb, xq, xs, bytes;
  LinearLayout(int rows, int cols, int64_t T) {
    sb = kAlign;
    xq = sb + up((size_t)((rows + 127) / 128) * scale_pitch(cols));
    xs = xq + up((size_t)T * cols);
    bytes = xs + up((size_t)T * scale_pitch(cols)) + kAlign;
  }
};

struct MlpLayout {
  size_t h, dgu, bytes;
  MlpLayout(int inter, int64_t T) {
    h = kAlign;
    dgu = h + up((size_t)T * inter * 2);
    bytes = dgu + up((size_t)T * inter * 4) + kAlign;
  }
};

DenseGemm linear_product(const moe_fp8_linear_handle* h, int64_t T, void* y, bool f32) {
  DenseGemm g = {};
  g.b = {h->codes, h->cols, h->rows, false};
  g.M = (int)T;
  g.N = h->rows;
  g.K = h->cols;
  g.type = kE4M3;
  g.epi = kEpiStore;
  g.sb = h->sb;
  g.out = y;
  g.ld_out = h->rows;
  g.out_f32 = f32;
  g.status = h->status;
  g.withhold = h->withhold;
  return g;
}

// The rows of x in BF16: rounded by the product itself, or before it.
void linear_rows(DenseGemm& g, const moe_fp8_linear_handle* h, const uint16_t* x, int64_t stride) {
  if (g.M <= kFusedTokens) {
    g.x = x;
    g.ldx = stride;
  } else {
    g.a = {h->xq, h->cols, g.M, false};
    g.sa = h->xs;
    g.sa_pitch = scale_pitch(h->cols);
    g.early = true;
  }
}

// The block's products, but for what the caller gives.
DenseGemm mlp_product(const moe_mlp_handle* h, DenseEpi epi, DenseOperand a, DenseOperand b, int M, int N, int K) {
  DenseGemm g = {};
  g.a = a;
  g.b = b;
  g.M = M;
  g.N = N;
  g.K = K;
  g.type = h->type;
  g.epi = epi;
  g.act = h->act;
  g.ld_out = N;
  g.status = h->status;
  g.withhold = h->withhold || (h->withhold_last && epi == kEpiStore);  // (a call ends with these)
  return g;
}

DenseGemm gate_product(const moe_mlp_handle* h, int T, const void* x, int64_t stride) {  // h, from x W1^T
  DenseGemm g = mlp_product(h, kEpiGate, {x, stride, T, false}, {h->w1, h->hidden, 2 * h->inter, false}, T, h->inter, h->hidden);
  g.out = h->h;
  return g;
}

DenseGemm down_product(const moe_mlp_handle* h, int T) {  // h W2^T
  DenseGemm g = mlp_product(h, kEpiStore, {h->h, h->inter, T, false}, {h->w2, h->inter, h->hidden, false}, T, h->hidden,
                            h->inter);
  g.early = true;
  return g;
}

DenseGemm grad_product(const moe_mlp_handle* h, int T, const void* dy, int64_t stride) {  // dg, du (and h), from dy W2
  DenseGemm g = mlp_product(h, kEpiGrad, {dy, stride, T, false}, {h->w2, h->inter, h->inter, true}, T, h->inter, h->hidden);
  g.dgu = h->dgu;
  return g;
}

DenseGemm dx_product(const moe_mlp_handle* h, int T) {  // (dg, du) W1
  return mlp_product(h, kEpiStore, {h->dgu, 2 * h->inter, T, false}, {h->w1, h->hidden, h->hidden, true}, T, h->hidden,
                     2 * h->inter);
}

DenseGemm dw1_product(const moe_mlp_handle* h, int T, const void* x, int64_t stride) {  // (dg, du)^T x
  return mlp_product(h, kEpiStore, {h->dgu, 2 * h->inter, 2 * h->inter, true}, {x, stride, h->hidden, true}, 2 * h->inter,
                     h->hidden, T);
}

DenseGemm dw2_product(const moe_mlp_handle* h, int T, const void* dy, int64_t stride) {  // dy^T h
  return mlp_product(h, kEpiStore, {dy, stride, h->hidden, true}, {h->h, h->inter, h->inter, true}, h->hidden, h->inter, T);
}

bool mlp_dims_ok(int32_t hidden, int32_t inter) {
  return hidden % 8 == 0 && inter % 8 == 0 && hidden <= 65536 && inter <= 65536;
}

}  // namespace

extern "C" {

moe_status moe_fp8_linear_workspace_query(int32_t rows, int32_t cols, int64_t max_tokens, size_t* workspace_bytes) {
  if (!workspace_bytes || rows < 1 || cols < 1 || max_tokens < 1) return MOE_ERR_INVALID_ARG;
  if (cols % 128 || cols > 32768 || rows > (1 << 24) || max_tokens > kMaxTokens) return MOE_ERR_UNSUPPORTED;
  *workspace_bytes = LinearLayout(rows, cols, max_tokens).bytes;
  return MOE_OK;
}

moe_status moe_fp8_linear_create(int32_t rows, int32_t cols, uint32_t flags, int64_t max_tokens, const uint8_t* d_codes,
                                 const float* d_scales, void* d_workspace, size_t workspace_bytes,
                                 struct CUstream_st* stream, moe_fp8_linear_handle** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  size_t need = 0;
  moe_status st = moe_fp8_linear_workspace_query(rows, cols, max_tokens, &need);
  if (st != MOE_OK) return st;
  if (flags & ~MOE_FLAG_WATCHDOG_TEST) return MOE_ERR_UNSUPPORTED;
  if (off(d_codes, 16) || off(d_scales, 4) || off(d_workspace, 16)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((st = this_device(&dev, &sms)) != MOE_OK) return st;
  const LinearLayout l(rows, cols, max_tokens);
  uint8_t* b = aligned(d_workspace);
  uint32_t* status = reinterpret_cast<uint32_t*>(b);
  uint32_t bits = 0;
  if (cudaMemsetAsync(b, 0, kAlign, stream) != cudaSuccess ||
      dense_scales_to_e8m0(d_scales, (rows + 127) / 128, cols / 128, scale_pitch(cols), b + l.sb, status, stream) !=
          cudaSuccess ||
      read_word(status, &bits, stream) != MOE_OK)
    return MOE_ERR_CUDA;
  if (bits & MOE_DEV_BAD_SCALE) return MOE_ERR_BAD_SCALE;
  moe_fp8_linear_handle* h = new (std::nothrow) moe_fp8_linear_handle;
  if (!h) return MOE_ERR_INVALID_ARG;
  memset(h, 0, sizeof(*h));
  h->rows = rows;
  h->cols = cols;
  h->device = dev;
  h->sms = sms;
  h->max_tokens = max_tokens;
  h->withhold = (flags & MOE_FLAG_WATCHDOG_TEST) != 0;
  h->codes = d_codes;
  h->status = status;
  h->sb = b + l.sb;
  h->xq = b + l.xq;
  h->xs = b + l.xs;
  *out = h;
  return MOE_OK;
}

moe_status moe_fp8_linear(moe_fp8_linear_handle* h, const uint16_t* d_x, int64_t x_stride, int64_t num_tokens,
                          void* d_y, int32_t y_float32, struct CUstream_st* stream) {
  if (!h || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  if (off(d_x, 16) || off(d_y, y_float32 ? 4 : 2) || x_stride < h->cols || x_stride % 8 || elsewhere(h->device))
    return MOE_ERR_INVALID_ARG;
  const Span y(d_y, num_tokens, h->rows, h->rows, y_float32 ? 4 : 2);
  if (y.meets(Span(d_x, num_tokens, x_stride, h->cols, 2)) || y.meets(Span(h->codes, h->rows, h->cols, h->cols, 1)))
    return MOE_ERR_INVALID_ARG;
  DenseGemm g = linear_product(h, num_tokens, d_y, y_float32 != 0);
  linear_rows(g, h, d_x, x_stride);
  if (!g.x && dense_quantize_rows(d_x, x_stride, num_tokens, h->cols, h->xq, h->xs, h->sms, stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  return dense_gemm(g, h->sms, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_fp8_linear_quantized(moe_fp8_linear_handle* h, const uint8_t* d_xq, const uint8_t* d_xq_scale,
                                    int64_t num_tokens, void* d_y, int32_t y_float32, struct CUstream_st* stream) {
  if (!h || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  if (off(d_xq, 16) || !d_xq_scale || off(d_y, y_float32 ? 4 : 2) || elsewhere(h->device)) return MOE_ERR_INVALID_ARG;
  const Span y(d_y, num_tokens, h->rows, h->rows, y_float32 ? 4 : 2);
  if (y.meets(Span(d_xq, num_tokens, h->cols, h->cols, 1)) ||
      y.meets(Span(d_xq_scale, num_tokens, h->cols / 128, h->cols / 128, 1)) ||
      y.meets(Span(h->codes, h->rows, h->cols, h->cols, 1)))
    return MOE_ERR_INVALID_ARG;
  DenseGemm g = linear_product(h, num_tokens, d_y, y_float32 != 0);
  g.a = {d_xq, h->cols, (int)num_tokens, false};
  g.sa = d_xq_scale;
  g.sa_pitch = h->cols / 128;
  return dense_gemm(g, h->sms, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_fp8_linear_plan(moe_fp8_linear_handle* h, int64_t num_tokens, int32_t quantized, moe_dense_launch* out) {
  if (!h || !out || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  *out = moe_dense_launch{};
  if (num_tokens == 0) return MOE_OK;
  DenseGemm g = linear_product(h, num_tokens, nullptr, false);
  const uint16_t row = 0;  // (some address: the choice reads none)
  if (!quantized) linear_rows(g, h, &row, h->cols);
  *out = dense_choice(&g, 1, h->sms);
  return MOE_OK;
}

moe_status moe_fp8_linear_read_status(moe_fp8_linear_handle* h, uint32_t* h_status, struct CUstream_st* stream) {
  if (!h || !h_status || elsewhere(h->device)) return MOE_ERR_INVALID_ARG;
  return read_status(h->status, h_status, stream);
}

void moe_fp8_linear_destroy(moe_fp8_linear_handle* h) { delete h; }

moe_status moe_mlp_workspace_query(int32_t hidden, int32_t inter, int64_t max_tokens, size_t* workspace_bytes) {
  if (!workspace_bytes || hidden < 1 || inter < 1 || max_tokens < 1) return MOE_ERR_INVALID_ARG;
  if (!mlp_dims_ok(hidden, inter) || max_tokens > kMaxTokens) return MOE_ERR_UNSUPPORTED;
  *workspace_bytes = MlpLayout(inter, max_tokens).bytes;
  return MOE_OK;
}

moe_status moe_mlp_create(int32_t hidden, int32_t inter, int32_t fp16, int32_t activation, uint32_t flags,
                          int64_t max_tokens, const uint16_t* d_w1, const uint16_t* d_w2, void* d_workspace, size_t workspace_bytes,
                          struct CUstream_st* stream, moe_mlp_handle** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  size_t need = 0;
  moe_status st = moe_mlp_workspace_query(hidden, inter, max_tokens, &need);
  if (st != MOE_OK) return st;
  if ((activation != MOE_ACT_SILU && activation != MOE_ACT_GELU_TANH) ||
      (flags & ~(MOE_FLAG_WATCHDOG_TEST | MOE_FLAG_WATCHDOG_LAST_TEST)))
    return MOE_ERR_UNSUPPORTED;
  if (off(d_w1, 16) || off(d_w2, 16) || off(d_workspace, 16)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((st = this_device(&dev, &sms)) != MOE_OK) return st;
  const MlpLayout l(inter, max_tokens);
  uint8_t* b = aligned(d_workspace);
  // (finished before the handle exists: its calls may be on other streams)
  if (cudaMemsetAsync(b, 0, kAlign, stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  moe_mlp_handle* h = new (std::nothrow) moe_mlp_handle;
  if (!h) return MOE_ERR_INVALID_ARG;
  memset(h, 0, sizeof(*h));
  h->hidden = hidden;
  h->inter = inter;
  h->device = dev;
  h->sms = sms;
  h->type = fp16 ? kFP16 : kBF16;
  h->act = activation == MOE_ACT_SILU ? kSilu : kGeluTanh;
  h->max_tokens = max_tokens;
  h->withhold = (flags & MOE_FLAG_WATCHDOG_TEST) != 0;
  h->withhold_last = (flags & MOE_FLAG_WATCHDOG_LAST_TEST) != 0;
  h->w1 = d_w1;
  h->w2 = d_w2;
  h->status = reinterpret_cast<uint32_t*>(b);
  h->h = b + l.h;
  h->dgu = b + l.dgu;
  *out = h;
  return MOE_OK;
}

moe_status moe_mlp_forward(moe_mlp_handle* h, const uint16_t* d_x, int64_t x_stride, int64_t num_tokens,
                           uint16_t* d_y, void* d_saved, int32_t saved_float32, struct CUstream_st* stream) {
  if (!h || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  const int H = h->hidden, I = h->inter;
  if (off(d_x, 16) || off(d_y, 16) || (d_saved && off(d_saved, 16)) || x_stride < H || x_stride % 8 ||
      elsewhere(h->device))
    return MOE_ERR_INVALID_ARG;
  const Span x(d_x, num_tokens, x_stride, H, 2), y(d_y, num_tokens, H, H, 2),
      saved(d_saved, num_tokens, 2 * I, 2 * I, saved_float32 ? 4 : 2), w1(h->w1, 2 * I, H, H, 2), w2(h->w2, H, I, I, 2);
  // y is stored after all of x has been read: it may be x itself
  if (saved.meets(x) || saved.meets(y) || (x.meets(y) && !(d_x == d_y && x_stride == H)) || y.meets(w1) || y.meets(w2) ||
      saved.meets(w1) || saved.meets(w2))
    return MOE_ERR_INVALID_ARG;
  DenseGemm g = gate_product(h, (int)num_tokens, d_x, x_stride);
  g.saved = d_saved;
  g.saved_f32 = saved_float32 != 0;
  if (dense_gemm(g, h->sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
  DenseGemm d = down_product(h, (int)num_tokens);
  d.out = d_y;
  return dense_gemm(d, h->sms, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_mlp_backward(moe_mlp_handle* h, const uint16_t* d_dy, int64_t dy_stride, const uint16_t* d_x,
                            int64_t x_stride, const void* d_saved, int32_t saved_float32, int64_t num_tokens,
                            uint16_t* d_dx, void* d_dw1, void* d_dw2, int32_t dw_float32, int32_t accumulate,
                            struct CUstream_st* stream) {
  if (!h || num_tokens < 0 || (accumulate && !dw_float32)) return MOE_ERR_INVALID_ARG;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  const int H = h->hidden, I = h->inter, T = (int)num_tokens;
  const size_t ds = dw_float32 ? 4 : 2;
  if ((d_dw1 && off(d_dw1, 16)) || (d_dw2 && off(d_dw2, 16)) || elsewhere(h->device)) return MOE_ERR_INVALID_ARG;
  if (T && (off(d_dy, 16) || off(d_x, 16) || off(d_saved, 16) || (d_dx && off(d_dx, 16)) || dy_stride < H ||
            dy_stride % 8 || x_stride < H || x_stride % 8))
    return MOE_ERR_INVALID_ARG;
  const Span in[5] = {Span(d_dy, T, dy_stride, H, 2), Span(d_x, T, x_stride, H, 2),
                      Span(d_saved, T, 2 * I, 2 * I, saved_float32 ? 4 : 2), Span(h->w1, 2 * I, H, H, 2),
                      Span(h->w2, H, I, I, 2)};
  const Span out[3] = {Span(d_dx, T, H, H, 2), Span(d_dw1, 2 * I, H, H, ds), Span(d_dw2, H, I, I, ds)};
  for (int i = 0; i < 3; ++i) {
    for (const Span& s : in)
      if (out[i].meets(s)) return MOE_ERR_INVALID_ARG;
    if (out[i].meets(out[(i + 1) % 3])) return MOE_ERR_INVALID_ARG;
  }
  if (T == 0) {  // the weights' gradients are sums over no rows
    if (accumulate) return MOE_OK;
    if (d_dw1 && cudaMemsetAsync(d_dw1, 0, 2 * ds * H * I, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (d_dw2 && cudaMemsetAsync(d_dw2, 0, ds * H * I, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  DenseGemm g = grad_product(h, T, d_dy, dy_stride);
  g.out = d_dw2 ? h->h : nullptr;
  g.saved = const_cast<void*>(d_saved);
  g.saved_f32 = saved_float32 != 0;
  if (dense_gemm(g, h->sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
  // what these read the product above has written, or the caller
  DenseGemm d[3] = {};
  int count = 0;
  auto add = [&](const DenseGemm& p, void* to, bool weights) {
    d[count] = p;
    d[count].out = to;
    d[count].out_f32 = weights && dw_float32;
    d[count++].accumulate = weights && accumulate;
  };
  if (d_dx) add(dx_product(h, T), d_dx, false);
  if (d_dw1) add(dw1_product(h, T, d_x, x_stride), d_dw1, true);
  if (d_dw2) add(dw2_product(h, T, d_dy, dy_stride), d_dw2, true);
  return !count || dense_gemms(d, count, h->sms, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_mlp_plan(moe_mlp_handle* h, int64_t num_tokens, moe_dense_launch out[4]) {
  if (!h || !out || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  memset(out, 0, 4 * sizeof(*out));
  const int T = (int)num_tokens;
  if (T == 0) return MOE_OK;
  DenseGemm g[3] = {gate_product(h, T, nullptr, h->hidden), down_product(h, T), grad_product(h, T, nullptr, h->hidden)};
  for (int i = 0; i < 3; ++i) out[i] = dense_choice(&g[i], 1, h->sms);
  DenseGemm d[3] = {dx_product(h, T), dw1_product(h, T, nullptr, h->hidden), dw2_product(h, T, nullptr, h->hidden)};
  out[3] = dense_choice(d, 3, h->sms);
  return MOE_OK;
}

moe_status moe_mlp_read_status(moe_mlp_handle* h, uint32_t* h_status, struct CUstream_st* stream) {
  if (!h || !h_status || elsewhere(h->device)) return MOE_ERR_INVALID_ARG;
  return read_status(h->status, h_status, stream);
}

void moe_mlp_destroy(moe_mlp_handle* h) { delete h; }

}  // extern "C"
