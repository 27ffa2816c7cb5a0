// C ABI of the block norms (blocknorm.h): argument checks and launches.
#include "api_check.h"
#include "blocknorm.h"
#include "blocknorm_launch.h"

namespace blocknorm {
namespace {

using api::fail;
using api::Span;

constexpr unsigned long long kMaxBytes = 1ull << 46;

int check_dims(long long rows, int H, int D) {
  if (rows < 0 || H < 0) return fail(WKV7_ERR_INVALID, "rows and heads must be >= 0 (got %lld, %d)", rows, H);
  if (D < 1 || D > kMaxD) return fail(WKV7_ERR_INVALID, "D must be 1 to %d (got %d)", kMaxD, D);
  if (rows >= 1ll << 30 || (H && rows * H >= 1ll << 31) || (unsigned long long)rows * H * D * 4 >= kMaxBytes)
    return fail(WKV7_ERR_INVALID, "too many rows");
  return WKV7_OK;
}
// Bytes an input of `rows` rows of `row` values, `stride` apart, spans.
int span_bytes(unsigned long long* out, long long* stride, long long rows, long long row, int es, const char* name) {
  if (rows <= 1) *stride = row;
  if (*stride < row || *stride >= 1ll << 40) return fail(WKV7_ERR_INVALID, "%s: rows of %lld values %lld apart", name, row, *stride);
  *out = rows ? ((unsigned long long)(rows - 1) * *stride + row) * es : 0;
  return *out < kMaxBytes ? WKV7_OK : fail(WKV7_ERR_INVALID, "%s too large", name);
}
int check_types(int bf16, int residual_bf16) {
  return !bf16 && residual_bf16 ? fail(WKV7_ERR_INVALID, "an fp32 x needs an fp32 residual") : WKV7_OK;
}
int launched(cudaError_t e) {
  return e == cudaSuccess ? WKV7_OK : fail(WKV7_ERR_CUDA, "block norm launch: %s", cudaGetErrorString(e));
}
// No rows: the sums over them are 0.
int zero_sums(float* a, float* b, int D, cudaStream_t s) {
  for (float* p : {a, b})
    if (p) {
      const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)D * 4, s);
      if (e != cudaSuccess) return launched(e);
    }
  return WKV7_OK;
}

}  // namespace
}  // namespace blocknorm

using namespace blocknorm;

extern "C" {

size_t blocknorm_part_bytes(long long rows, int D, int sums) {
  if (rows < 0 || D < 1 || D > kMaxD || sums < 1 || sums > 2) return 0;
  return (size_t)part_rows(rows, D) * sums * D * 4;
}

int blocknorm_add_forward(const void* x, const void* residual, const float* weight, const float* scale, void* h, void* n,
                          float* rstd, long long x_stride, long long residual_stride, long long rows, int D, float eps,
                          int bf16, int residual_bf16, void* stream) {
  int rc = check_dims(rows, 1, D);
  if (rc || (rc = check_types(bf16, residual_bf16))) return rc;
  if (!rows) return WKV7_OK;  // whose buffers may all be NULL
  const int es = bf16 ? 2 : 4, rs = residual_bf16 ? 2 : 4;
  const unsigned long long m = (unsigned long long)rows * D, vec = (unsigned long long)D * 4;
  unsigned long long xb = 0, rb = 0;
  if (!x) x_stride = D;
  if (x && (rc = span_bytes(&xb, &x_stride, rows, D, es, "x"))) return rc;
  if ((rc = span_bytes(&rb, &residual_stride, rows, D, rs, "residual"))) return rc;
  if (!x && (scale || h)) return fail(WKV7_ERR_INVALID, "scale and h belong to x");
  // h may be written over residual: a row is read before it is written
  const bool over = h && h == residual && residual_stride == D;
  const Span ins[4] = {{x, xb, "x", false}, {residual, over ? 0 : rb, "residual", true}, {weight, vec, "weight", true}, {scale, vec, "scale", false}};
  const Span outs[3] = {{n, m * es, "n", true}, {h, m * rs, "h", x != nullptr}, {rstd, (unsigned long long)rows * 4, "rstd", false}};
  if (over && !residual) return fail(WKV7_ERR_INVALID, "residual must not be NULL");
  if ((rc = api::check_spans(ins, outs))) return rc;
  Args p{};
  p.a = x, p.b = residual, p.w = weight, p.scale = scale, p.out = n, p.h = h, p.rstd = rstd;
  p.rows = rows, p.a_t = x_stride, p.b_t = residual_stride, p.H = 1, p.D = D, p.eps = eps;
  return launched(launch_add(p, bf16, residual_bf16, false, static_cast<cudaStream_t>(stream)));
}

int blocknorm_add_backward(const void* x, const void* residual, const float* weight, const float* scale,
                           const float* rstd, const void* dn, const void* dh, void* dresidual, void* dx, float* dweight,
                           float* dscale, void* part, long long x_stride, long long residual_stride, long long rows,
                           int D, int bf16, int residual_bf16, void* stream) {
  int rc = check_dims(rows, 1, D);
  if (rc || (rc = check_types(bf16, residual_bf16))) return rc;
  const unsigned long long vec = (unsigned long long)D * 4;
  if (!rows) {  // no terms: the sums are 0, and every other buffer may be NULL
    const Span none[1] = {{nullptr, 0, "", false}};
    const Span sums[2] = {{dweight, vec, "dweight", true}, {dscale, vec, "dscale", false}};
    return (rc = api::check_spans(none, sums)) ? rc : zero_sums(dweight, dscale, D, static_cast<cudaStream_t>(stream));
  }
  const int es = bf16 ? 2 : 4, rs = residual_bf16 ? 2 : 4;
  const unsigned long long m = (unsigned long long)rows * D;
  unsigned long long xb = 0, rb = 0;
  if (!x) x_stride = D;
  if (x && (rc = span_bytes(&xb, &x_stride, rows, D, es, "x"))) return rc;
  if ((rc = span_bytes(&rb, &residual_stride, rows, D, rs, "residual"))) return rc;
  if (!x && (scale || dx)) return fail(WKV7_ERR_INVALID, "scale and dx belong to x");
  if (!scale != !dscale) return fail(WKV7_ERR_INVALID, "dscale belongs to scale");
  const Span ins[7] = {{x, xb, "x", false}, {residual, rb, "residual", true}, {weight, vec, "weight", true}, {scale, vec, "scale", false},
                       {rstd, (unsigned long long)rows * 4, "rstd", true}, {dn, m * es, "dn", true}, {dh, m * rs, "dh", false}};
  const Span outs[5] = {{dresidual, m * rs, "dresidual", true}, {dx, m * es, "dx", scale != nullptr}, {dweight, vec, "dweight", true},
                        {dscale, vec, "dscale", false}, {part, rows ? blocknorm_part_bytes(rows, D, 2) : 0, "part", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  Args p{};
  p.a = x, p.b = residual, p.w = weight, p.scale = scale, p.rstd = const_cast<float*>(rstd), p.dout = dn, p.dh = dh;
  p.da = dx, p.db = dresidual, p.dw = dweight, p.dscale = dscale, p.part = static_cast<float*>(part);
  p.rows = rows, p.a_t = x_stride, p.b_t = residual_stride, p.H = 1, p.D = D;
  return launched(launch_add(p, bf16, residual_bf16, true, static_cast<cudaStream_t>(stream)));
}

int blocknorm_gated_forward(const void* o, const void* z, const float* weight, void* y, float* rstd, long long o_stride,
                            long long z_stride, long long tokens, int H, int D, float eps, int bf16, void* stream) {
  int rc = check_dims(tokens, H, D);
  if (rc) return rc;
  const int es = bf16 ? 2 : 4;
  const unsigned long long m = (unsigned long long)tokens * H * D;
  unsigned long long ob = 0, zb = 0;
  if ((rc = span_bytes(&ob, &o_stride, tokens, (long long)H * D, es, "o"))) return rc;
  if ((rc = span_bytes(&zb, &z_stride, tokens, (long long)H * D, es, "z"))) return rc;
  const Span ins[3] = {{o, ob, "o", true}, {z, zb, "z", true}, {weight, (unsigned long long)D * 4, "weight", true}};
  const Span outs[2] = {{y, m * es, "y", true}, {rstd, m / D * 4, "rstd", false}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!m) return WKV7_OK;
  Args p{};
  p.a = o, p.b = z, p.w = weight, p.out = y, p.rstd = rstd;
  p.rows = tokens * H, p.a_t = o_stride, p.b_t = z_stride, p.H = H, p.D = D, p.eps = eps;
  return launched(launch_gated(p, bf16, false, static_cast<cudaStream_t>(stream)));
}

int blocknorm_gated_backward(const void* o, const void* z, const float* weight, const float* rstd, const void* dy,
                             void* d_o, void* dz, float* dweight, void* part, long long o_stride, long long z_stride,
                             long long tokens, int H, int D, int bf16, void* stream) {
  int rc = check_dims(tokens, H, D);
  if (rc) return rc;
  const int es = bf16 ? 2 : 4;
  const unsigned long long m = (unsigned long long)tokens * H * D, vec = (unsigned long long)D * 4;
  unsigned long long ob = 0, zb = 0;
  if ((rc = span_bytes(&ob, &o_stride, tokens, (long long)H * D, es, "o"))) return rc;
  if ((rc = span_bytes(&zb, &z_stride, tokens, (long long)H * D, es, "z"))) return rc;
  const Span ins[5] = {{o, ob, "o", true}, {z, zb, "z", true}, {weight, vec, "weight", true}, {rstd, m / D * 4, "rstd", true}, {dy, m * es, "dy", true}};
  const Span outs[4] = {{d_o, m * es, "d_o", true}, {dz, m * es, "dz", true}, {dweight, vec, "dweight", true},
                        {part, m ? blocknorm_part_bytes(tokens * H, D, 1) : 0, "part", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!m) return zero_sums(dweight, nullptr, D, static_cast<cudaStream_t>(stream));
  Args p{};
  p.a = o, p.b = z, p.w = weight, p.rstd = const_cast<float*>(rstd), p.dout = dy;
  p.da = d_o, p.db = dz, p.dw = dweight, p.part = static_cast<float*>(part);
  p.rows = tokens * H, p.a_t = o_stride, p.b_t = z_stride, p.H = H, p.D = D;
  return launched(launch_gated(p, bf16, true, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
