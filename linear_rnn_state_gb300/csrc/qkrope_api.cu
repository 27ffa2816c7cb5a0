// C ABI of the norms of queries and keys with the position rotation (qkrope.h):
// argument checks and launches.
#include "api_check.h"
#include "qkrope.h"
#include "qkrope_launch.h"

namespace qkrope {
namespace {

using api::fail;
using api::Span;

constexpr unsigned long long kMaxBytes = 1ull << 46;

struct Sizes {
  unsigned long long q, k, qd, kd;  // bytes that the inputs span, and dense
};
int check(Sizes* z, Args& p, long long tokens, long long T, int es) {
  if (tokens < 0 || p.Hq < 0 || p.Hk < 0) return fail(WKV7_ERR_INVALID, "tokens and heads must be >= 0 (got %lld, %d, %d)", tokens, p.Hq, p.Hk);
  if (p.D < 8 || p.D > kMaxD || p.D % 8) return fail(WKV7_ERR_INVALID, "D must be a multiple of 8 from 8 to %d (got %d)", kMaxD, p.D);
  if (p.half < 0 || p.half > p.D / 2) return fail(WKV7_ERR_INVALID, "half must be 0 to D / 2 (got %d of %d)", p.half, p.D);
  if (!p.positions && tokens && (T < 1 || T > 1ll << 31)) return fail(WKV7_ERR_INVALID, "T must be 1 to 2^31 without positions (got %lld)", T);
  const unsigned long long H = (unsigned long long)p.Hq + p.Hk;
  if (tokens >= 1ll << 31 || H >= 1ull << 20 || (unsigned long long)tokens * H >= 1ull << 31 || (unsigned long long)tokens * H * p.D * 4 >= kMaxBytes)
    return fail(WKV7_ERR_INVALID, "too many tokens or heads");
  long long* const strides[2] = {&p.q_t, &p.k_t};
  const int heads[2] = {p.Hq, p.Hk};
  unsigned long long* const spans[2] = {&z->q, &z->k};
  for (int i = 0; i < 2; ++i) {
    const long long row = (long long)heads[i] * p.D;
    if (tokens <= 1 || !row) *strides[i] = row;
    if (*strides[i] < row || *strides[i] % 8 || *strides[i] >= 1ll << 40)
      return fail(WKV7_ERR_INVALID, "%s: tokens of %lld values %lld apart (a multiple of 8, at least the heads)", i ? "k" : "q", row, *strides[i]);
    *spans[i] = tokens && row ? api::span_bytes(tokens - 1, *strides[i], 0, 0, row, es) : 0;
    if (*spans[i] >= kMaxBytes) return fail(WKV7_ERR_INVALID, "%s too large", i ? "k" : "q");
  }
  z->qd = (unsigned long long)tokens * p.Hq * p.D * es, z->kd = (unsigned long long)tokens * p.Hk * p.D * es;
  p.rows = tokens * (long long)H, p.T = T;
  return WKV7_OK;
}
int launched(cudaError_t e) { return e == cudaSuccess ? WKV7_OK : fail(WKV7_ERR_CUDA, "query and key norm launch: %s", cudaGetErrorString(e)); }

}  // namespace
}  // namespace qkrope

using namespace qkrope;

extern "C" {

size_t qkrope_part_bytes(long long tokens, int Hq, int Hk, int D) {
  if (tokens < 0 || tokens >= 1ll << 31 || Hq < 0 || Hk < 0 || D < 8 || D > kMaxD || D % 8) return 0;
  return (size_t)part_rows(tokens * ((long long)Hq + Hk)) * 2 * D * 4;
}

int qkrope_forward(const void* q, const void* k, const float* q_weight, const float* k_weight, const double* freq,
                   const int* positions, void* q_out, void* k_out, long long q_stride, long long k_stride,
                   long long tokens, long long T, int Hq, int Hk, int D, int half, int interleaved, float eps, int bf16,
                   void* stream) {
  Args p{};
  p.q = q, p.k = k, p.wq = q_weight, p.wk = k_weight, p.freq = freq, p.positions = positions, p.qo = q_out, p.ko = k_out;
  p.q_t = q_stride, p.k_t = k_stride, p.Hq = Hq, p.Hk = Hk, p.D = D, p.half = half, p.interleaved = interleaved, p.eps = eps;
  Sizes z;
  int rc = check(&z, p, tokens, T, bf16 ? 2 : 4);
  if (rc || !p.rows) return rc;
  const unsigned long long vec = (unsigned long long)D * 4;
  const Span ins[6] = {{q, z.q, "q", true}, {k, z.k, "k", true}, {q_weight, Hq ? vec : 0, "q_weight", true}, {k_weight, Hk ? vec : 0, "k_weight", true},
                       {freq, (unsigned long long)half * 8, "freq", true}, {positions, (unsigned long long)tokens * 4, "positions", false, 4}};
  const Span outs[2] = {{q_out, z.qd, "q_out", true}, {k_out, z.kd, "k_out", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  return launched(launch(p, bf16, false, static_cast<cudaStream_t>(stream)));
}

int qkrope_backward(const void* q, const void* k, const float* q_weight, const float* k_weight, const double* freq,
                    const int* positions, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                    float* dk_weight, void* part, long long q_stride, long long k_stride, long long tokens, long long T,
                    int Hq, int Hk, int D, int half, int interleaved, float eps, int bf16, void* stream) {
  Args p{};
  p.q = q, p.k = k, p.wq = q_weight, p.wk = k_weight, p.freq = freq, p.positions = positions, p.dqo = dq_out, p.dko = dk_out;
  p.qo = dq, p.ko = dk, p.dwq = dq_weight, p.dwk = dk_weight, p.part = static_cast<float*>(part);
  p.q_t = q_stride, p.k_t = k_stride, p.Hq = Hq, p.Hk = Hk, p.D = D, p.half = half, p.interleaved = interleaved, p.eps = eps;
  Sizes z;
  int rc = check(&z, p, tokens, T, bf16 ? 2 : 4);
  if (rc) return rc;
  const unsigned long long vec = (unsigned long long)D * 4, some = p.rows ? ~0ull : 0ull;
  const Span ins[8] = {{q, z.q, "q", true}, {k, z.k, "k", true}, {q_weight, some & (Hq ? vec : 0), "q_weight", true},
                       {k_weight, some & (Hk ? vec : 0), "k_weight", true}, {freq, some & ((unsigned long long)half * 8), "freq", true},
                       {positions, (unsigned long long)tokens * 4, "positions", false, 4}, {dq_out, z.qd, "dq_out", true}, {dk_out, z.kd, "dk_out", true}};
  const Span outs[5] = {{dq, z.qd, "dq", true}, {dk, z.kd, "dk", true}, {dq_weight, vec, "dq_weight", true}, {dk_weight, vec, "dk_weight", true},
                        {part, some & (unsigned long long)qkrope_part_bytes(tokens, Hq, Hk, D), "part", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!p.rows) {  // no terms
    cudaError_t e = cudaMemsetAsync(dq_weight, 0, vec, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, vec, s);
    return launched(e);
  }
  return launched(launch(p, bf16, true, s));
}

}  // extern "C"
