// C ABI of the gated delta rule (gdr.h): argument checks, the regions of the
// caller's buffers, and the launches.
#include <algorithm>
#include <initializer_list>

#ifdef WKV7_DEBUG
#include <atomic>
#include "gdr_debug.h"
#endif

#include "api_check.h"
#include "gdr.h"
#include "gdr_launch.h"

namespace gdr {
namespace {

using api::fail;
using api::Span;

constexpr unsigned long long kMaxBytes = 1ull << 46, kMaxBlocks = 1ull << 31;

#ifdef WKV7_DEBUG
std::atomic<int> g_debug_skip_tile{0}, g_debug_skip_t{0};  // gdr_debug.h
#endif

int check_dims(int B, int T, int Hk, int Hv, int K, int V, const char* rows) {
  if (B < 0 || T < 0 || Hk < 0 || Hv < 0) return fail(WKV7_ERR_INVALID, "%s, T, Hk and Hv must be >= 0 (got %d, %d, %d, %d)", rows, B, T, Hk, Hv);
  if (Hk > Hv || (Hk ? Hv % Hk : Hv)) return fail(WKV7_ERR_INVALID, "Hv must be a multiple of Hk (got %d, %d)", Hv, Hk);
  if (K < 8 || K > kMaxDim || K % 8 || V < 8 || V > kMaxDim || V % 8)
    return fail(WKV7_ERR_INVALID, "K and V must be multiples of 8 from 8 to %d (got %d, %d)", kMaxDim, K, V);
  if ((unsigned long long)B * T >= 1ull << 40 || (unsigned long long)B * T * Hv >= kMaxBytes / (4 * kMaxDim))
    return fail(WKV7_ERR_INVALID, "%s * T * Hv too large", rows);
  return WKV7_OK;
}

// Strides of q, k, v: the given ones, checked, or the dense ones. bytes: what
// each tensor spans.
int set_strides(long long (&out)[6], unsigned long long (&bytes)[3], const long long* given, int B, int T, int Hk, int Hv,
                int K, int V, int es) {
  const long long row[3] = {(long long)Hk * K, (long long)Hk * K, (long long)Hv * V};
  const char* const names[3] = {"q", "k", "v"};
  for (int i = 0; i < 3; ++i) {
    long long b = row[i] * T, t = row[i];
    if (given) b = given[2 * i], t = given[2 * i + 1];
    if (given && ((T > 1 && (t < row[i] || t % 8 || t > 1ll << 40)) || (B > 1 && (b < 0 || b % 8 || b > 1ll << 45))))
      return fail(WKV7_ERR_INVALID, "%s: strides must be multiples of 8, a token's at least its heads (got %lld, %lld)", names[i], b, t);
    if (B <= 1) b = 0;
    if (T <= 1) t = 0;
    out[2 * i] = b, out[2 * i + 1] = t;
    bytes[i] = B && T && Hv ? ((unsigned long long)(B - 1) * b + (unsigned long long)(T - 1) * t + row[i]) * es : 0;
    if (bytes[i] >= kMaxBytes) return fail(WKV7_ERR_INVALID, "%s too large", names[i]);
  }
  return WKV7_OK;
}

// Fills a shape; nseq < 0 for dense batches.
int set_shape(Shape& s, int B, int T, int Hk, int Hv, int K, int V, int nseq) {
  int rc = check_dims(B, T, Hk, Hv, K, V, "B");
  if (rc) return rc;
  if (nseq >= 0 && B != 1) return fail(WKV7_ERR_INVALID, "packed sequences lie in one batch row (got B = %d)", B);
  s = Shape{};
  s.B = B, s.T = T, s.Hk = Hk, s.Hv = Hv, s.K = K, s.V = V;
  s.nseq = nseq >= 0 ? nseq : B;
  s.packed = nseq >= 0;
  const unsigned long long slots = slot_count(B, T, s.nseq, nseq >= 0);
  if (slots * (Hv ? Hv : 1) * v_tiles(V) >= kMaxBlocks || (unsigned long long)s.nseq * Hv * v_tiles(V) >= kMaxBlocks)
    return fail(WKV7_ERR_INVALID, "too many chunks");
  s.slots = (int)slots;
  return WKV7_OK;
}

size_t align128(size_t x) { return (x + 127) & ~(size_t)127; }

// Packed, but no sequence at all: outputs of tokens are 0.
int zero_tokens(std::initializer_list<Span> outs, cudaStream_t stream) {
  for (const Span& x : outs) {
    const cudaError_t e = x.bytes ? cudaMemsetAsync(const_cast<void*>(x.p), 0, x.bytes, stream) : cudaSuccess;
    if (e != cudaSuccess) return fail(WKV7_ERR_CUDA, "%s: %s", x.name, cudaGetErrorString(e));
  }
  return WKV7_OK;
}

// The regions of `saved` from p on; returns the bytes.
size_t place_saved(Buffers& b, const Shape& s, bool bf16, bool for_backward, char* p) {
  const Layout l = layout(s, bf16);
  char* at = p;
  auto take = [&](size_t bytes) {
    char* r = at;
    at += align128(bytes);
    return r;
  };
  b.k_img = take(l.n_k * l.kq_img);
  b.q_img = take(l.n_k * l.kq_img);
  b.rows = reinterpret_cast<Rows*>(take(l.n_k * sizeof(Rows)));
  b.t_img = take(l.n_v * Layout::tp_img);
  b.p_img = take(l.n_v * Layout::tp_img);
  b.scal = reinterpret_cast<Scal*>(take(l.n_v * sizeof(Scal)));
  if (for_backward) b.f_rec = take(l.n_t * l.f_rec);
  b.carry = segments_of(s) > 1 ? reinterpret_cast<float*>(take((size_t)s.nseq * s.Hv * s.V * s.K * 4)) : nullptr;
  return at - p;
}
size_t place_workspace(Buffers& b, const Shape& s, bool bf16, char* p) {
  const Layout l = layout(s, bf16);
  char* at = p;
  auto take = [&](size_t bytes) {
    char* r = at;
    at += align128(bytes);
    return r;
  };
  b.b_rec = take(l.n_t * l.b_rec);
  b.carry_back = segments_of(s) > 1 ? reinterpret_cast<float*>(take((size_t)s.nseq * s.Hv * s.V * s.K * 4)) : nullptr;
  b.dq_part = b.dk_part = nullptr;
  if (needs_terms(s, l.parts)) {
    const size_t bytes = (size_t)s.B * s.T * s.Hv * s.K * 4;
    b.dq_part = reinterpret_cast<float*>(take(bytes));
    b.dk_part = reinterpret_cast<float*>(take(bytes));
  }
  return at - p;
}

int copy_state(float* dst, const float* src, size_t bytes, cudaStream_t stream) {
  if (!dst || !bytes) return WKV7_OK;
  const cudaError_t e = src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(dst, 0, bytes, stream);
  return e == cudaSuccess ? WKV7_OK : fail(WKV7_ERR_CUDA, "state copy: %s", cudaGetErrorString(e));
}

int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? WKV7_OK : fail(WKV7_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

int forward_impl(bool bf16, const void* q, const void* k, const void* v, const float* g, const float* beta,
                 const float* s_init, const int* starts, void* o, float* s_final, void* saved, const long long* strides,
                 float scale, int l2norm, int for_backward, int B, int T, int Hk, int Hv, int K, int V, int nseq,
                 cudaStream_t stream) {
  if (!starts) nseq = -1;
  if (starts && nseq < 0) return fail(WKV7_ERR_INVALID, "nseq must be >= 0 with seq_starts (got %d)", nseq);
  Args a{};
  int rc = set_shape(a.s, B, T, Hk, Hv, K, V, nseq);
  if (rc) return rc;
  const int es = bf16 ? 2 : 4;
  long long st[6];
  unsigned long long in_bytes[3];
  if ((rc = set_strides(st, in_bytes, strides, B, T, Hk, Hv, K, V, es))) return rc;
  const unsigned long long rows = (unsigned long long)B * T * Hv, state = (unsigned long long)a.s.nseq * Hv * V * K * 4;
  const size_t need = place_saved(a.b, a.s, bf16, for_backward, static_cast<char*>(saved));
  const Span ins[7] = {{q, in_bytes[0], "q", true}, {k, in_bytes[1], "k", true}, {v, in_bytes[2], "v", true},
                       {g, rows * 4, "g", true, 4}, {beta, rows * 4, "beta", true, 4}, {s_init, state, "s_init", false},
                       {starts, starts ? ((unsigned long long)nseq + 1) * 4 : 0, "seq_starts", false, 4}};
  const Span outs[3] = {{o, rows * V * es, "o", true}, {s_final, state, "s_final", false}, {saved, rows ? need : 0, "saved", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!Hv) return WKV7_OK;
  if (!a.s.nseq) return zero_tokens({outs[0]}, stream);
  if (!rows) return copy_state(s_final, s_init, state, stream);
  a.s.starts = starts;
  a.s.l2norm = l2norm, a.s.scale = scale;
  a.small = is_small(a.s);
  a.s.q_b = st[0], a.s.q_t = st[1], a.s.k_b = st[2], a.s.k_t = st[3], a.s.v_b = st[4], a.s.v_t = st[5];
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.s_init = s_init, a.o = o, a.s_final = s_final;
#ifdef WKV7_DEBUG
  a.skip_t = g_debug_skip_t.load();
#endif
  if ((rc = wkv7::api_status_word(&a.status))) return rc;
  const int parts = segments_of(a.s), chunks = (T + kC - 1) / kC, each = (chunks + parts - 1) / parts;
  if (parts > 1) a.small = 0;
  for (int at = 0; at < chunks || at == 0; at += each) {
    if (parts > 1) {
      a.seg0 = at, a.segn = std::min(each, chunks - at);
      if (at) a.s_init = a.s_final;
      if (!s_final) a.s_final = a.b.carry;
    }
    if ((rc = launched(launch_prep(a, bf16, stream), "chunk preparation"))) return rc;
    if ((rc = launched(launch_fwd(a, bf16, for_backward, stream), "forward"))) return rc;
    if (parts == 1) break;
  }
  if (a.s.packed) {
    const Gaps gaps{{static_cast<uint32_t*>(o)}, {(long long)Hv * V * es / 4}};
    return launched(launch_gaps(a, gaps, stream), "gaps");
  }
  return WKV7_OK;
}

int backward_impl(bool bf16, const void* q, const void* k, const void* v, const float* g, const float* beta,
                  const void* d_o, const float* dS_final, const int* starts, const void* saved, void* workspace, void* dq,
                  void* dk, void* dv, float* dg, float* dbeta, float* dS_init, const long long* strides, float scale,
                  int l2norm, int B, int T, int Hk, int Hv, int K, int V, int nseq, cudaStream_t stream) {
  if (!starts) nseq = -1;
  if (starts && nseq < 0) return fail(WKV7_ERR_INVALID, "nseq must be >= 0 with seq_starts (got %d)", nseq);
  Args a{};
  int rc = set_shape(a.s, B, T, Hk, Hv, K, V, nseq);
  if (rc) return rc;
  const int es = bf16 ? 2 : 4;
  long long st[6];
  unsigned long long in_bytes[3];
  if ((rc = set_strides(st, in_bytes, strides, B, T, Hk, Hv, K, V, es))) return rc;
  const unsigned long long rows = (unsigned long long)B * T * Hv, keys = (unsigned long long)B * T * Hk * K * es,
                           state = (unsigned long long)a.s.nseq * Hv * V * K * 4;
  const size_t have = place_saved(a.b, a.s, bf16, true, const_cast<char*>(static_cast<const char*>(saved)));
  const size_t need = place_workspace(a.b, a.s, bf16, static_cast<char*>(workspace));
  const Span ins[9] = {{q, in_bytes[0], "q", true}, {k, in_bytes[1], "k", true}, {v, in_bytes[2], "v", true},
                       {g, rows * 4, "g", true, 4}, {beta, rows * 4, "beta", true, 4}, {d_o, rows * V * es, "d_o", true},
                       {dS_final, state, "dS_final", false},
                       {starts, starts ? ((unsigned long long)nseq + 1) * 4 : 0, "seq_starts", false, 4},
                       {saved, rows ? have : 0, "saved", true}};
  const Span outs[7] = {{dq, keys, "dq", true}, {dk, keys, "dk", true}, {dv, rows * V * es, "dv", true},
                        {dg, rows * 4, "dg", true, 4}, {dbeta, rows * 4, "dbeta", true, 4}, {dS_init, state, "dS_init", false},
                        {workspace, rows ? need : 0, "workspace", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!Hv) return WKV7_OK;
  if (!a.s.nseq) return zero_tokens({outs[0], outs[1], outs[2], outs[3], outs[4]}, stream);
  if (!rows) return copy_state(dS_init, dS_final, state, stream);
  a.s.starts = starts;
  a.s.l2norm = l2norm, a.s.scale = scale;
  a.small = is_small(a.s);
  a.s.q_b = st[0], a.s.q_t = st[1], a.s.k_b = st[2], a.s.k_t = st[3], a.s.v_b = st[4], a.s.v_t = st[5];
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.d_o = d_o, a.dS_final = dS_final;
  a.dq = dq, a.dk = dk, a.dv = dv, a.dg = dg, a.dbeta = dbeta, a.dS_init = dS_init;
#ifdef WKV7_DEBUG
  a.skip_tile = g_debug_skip_tile.load(), a.skip_t = g_debug_skip_t.load();
#endif
  if ((rc = wkv7::api_status_word(&a.status))) return rc;
  const int parts = segments_of(a.s), chunks = (T + kC - 1) / kC, each = (chunks + parts - 1) / parts;
  if (parts > 1) a.small = 0;
  if (parts == 1) {
    if ((rc = launched(launch_bwd(a, bf16, stream), "backward"))) return rc;
    if ((rc = launched(launch_grad(a, bf16, stream), "gradients")) || !a.s.packed) return rc;
    auto words = [](void* p) { return static_cast<uint32_t*>(p); };
    const long long wk = (long long)Hk * K * es / 4, wv = (long long)Hv * V * es / 4;
    const Gaps gaps{{words(dq), words(dk), words(dv), words(dg), words(dbeta)}, {wk, wk, wv, Hv, Hv}};
    return launched(launch_gaps(a, gaps, stream), "gaps");
  }
  // from the last segment to the first: the chain of one, then the gradients of the one after it beside that chain
  if (!dS_init) a.dS_init = a.b.carry_back;
  const int last = (chunks - 1) / each * each;
  Args after{};
  for (int at = last; at >= 0; at -= each) {
    a.seg0 = at, a.segn = std::min(each, chunks - at);
    if ((rc = launched(launch_bwd(a, bf16, stream), "backward"))) return rc;
    if (at < last && (rc = launched(launch_grad(after, bf16, stream), "gradients"))) return rc;
    after = a;
    a.dS_final = a.dS_init;
  }
  return launched(launch_grad(after, bf16, stream), "gradients");
}

int step_impl(bool bf16, const void* q, const void* k, const void* v, const float* g, const float* beta, float* state,
              const int* slots, void* o, const long long* strides, float scale, int l2norm, int R, int T, int Hk, int Hv,
              int K, int V, int n_slots, cudaStream_t stream) {
  int rc = check_dims(R, T, Hk, Hv, K, V, "R");
  if (rc) return rc;
  if (n_slots < 0 || (!slots && R > n_slots)) return fail(WKV7_ERR_INVALID, "%d states for %d requests", n_slots, R);
  const int es = bf16 ? 2 : 4;
  long long st[6];
  unsigned long long in_bytes[3];
  if ((rc = set_strides(st, in_bytes, strides, R, T, Hk, Hv, K, V, es))) return rc;
  const unsigned long long rows = (unsigned long long)R * T * Hv, pool = (unsigned long long)n_slots * Hv * V * K * 4;
  if (pool >= kMaxBytes || (unsigned long long)R * Hv * 16 >= kMaxBlocks) return fail(WKV7_ERR_INVALID, "too many states");
  const Span ins[6] = {{q, in_bytes[0], "q", true}, {k, in_bytes[1], "k", true}, {v, in_bytes[2], "v", true},
                       {g, rows * 4, "g", true, 4}, {beta, rows * 4, "beta", true, 4}, {slots, (unsigned long long)R * 4, "slots", false, 4}};
  const Span outs[2] = {{state, pool, "state", rows != 0}, {o, rows * V * es, "o", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!rows) return WKV7_OK;
  StepArgs a{};
  a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.state = state, a.slots = slots, a.o = o;
  a.R = R, a.T = T, a.Hk = Hk, a.Hv = Hv, a.K = K, a.V = V, a.n_slots = n_slots, a.l2norm = l2norm, a.scale = scale;
  a.q_b = st[0], a.q_t = st[1], a.k_b = st[2], a.k_t = st[3], a.v_b = st[4], a.v_t = st[5];
  return launched(launch_step(a, bf16, stream), "step");
}

}  // namespace
}  // namespace gdr

extern "C" {

#ifdef WKV7_DEBUG
int gdr_debug_skip_tile(int tile) {
  gdr::g_debug_skip_tile.store(tile > 0 ? tile : 0);
  return WKV7_OK;
}
int gdr_debug_skip_t(int step) {
  gdr::g_debug_skip_t.store(step > 0 ? step : 0);
  return WKV7_OK;
}
#endif

size_t gdr_saved_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16, int for_backward) {
  gdr::Shape s;
  if (gdr::set_shape(s, B, T, Hk, Hv, K, V, nseq)) return 0;
  gdr::Buffers b;
  return gdr::place_saved(b, s, bf16, for_backward, nullptr);
}
size_t gdr_backward_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16) {
  gdr::Shape s;
  if (gdr::set_shape(s, B, T, Hk, Hv, K, V, nseq)) return 0;
  gdr::Buffers b;
  return gdr::place_workspace(b, s, bf16, nullptr);
}

int gdr_forward(const float* q, const float* k, const float* v, const float* g, const float* beta, const float* s_init,
                const int* seq_starts, float* o, float* s_final, void* saved, const long long* strides, float scale,
                int l2norm, int for_backward, int B, int T, int Hk, int Hv, int K, int V, int nseq, void* stream) {
  return gdr::forward_impl(false, q, k, v, g, beta, s_init, seq_starts, o, s_final, saved, strides, scale, l2norm,
                           for_backward, B, T, Hk, Hv, K, V, nseq, static_cast<cudaStream_t>(stream));
}
int gdr_forward_bf16(const wkv7_bf16* q, const wkv7_bf16* k, const wkv7_bf16* v, const float* g, const float* beta,
                     const float* s_init, const int* seq_starts, wkv7_bf16* o, float* s_final, void* saved,
                     const long long* strides, float scale, int l2norm, int for_backward, int B, int T, int Hk, int Hv,
                     int K, int V, int nseq, void* stream) {
  return gdr::forward_impl(true, q, k, v, g, beta, s_init, seq_starts, o, s_final, saved, strides, scale, l2norm,
                           for_backward, B, T, Hk, Hv, K, V, nseq, static_cast<cudaStream_t>(stream));
}
int gdr_backward(const float* q, const float* k, const float* v, const float* g, const float* beta, const float* d_o,
                 const float* dS_final, const int* seq_starts, const void* saved, void* workspace, float* dq, float* dk,
                 float* dv, float* dg, float* dbeta, float* dS_init, const long long* strides, float scale, int l2norm,
                 int B, int T, int Hk, int Hv, int K, int V, int nseq, void* stream) {
  return gdr::backward_impl(false, q, k, v, g, beta, d_o, dS_final, seq_starts, saved, workspace, dq, dk, dv, dg, dbeta,
                            dS_init, strides, scale, l2norm, B, T, Hk, Hv, K, V, nseq, static_cast<cudaStream_t>(stream));
}
int gdr_backward_bf16(const wkv7_bf16* q, const wkv7_bf16* k, const wkv7_bf16* v, const float* g, const float* beta,
                      const wkv7_bf16* d_o, const float* dS_final, const int* seq_starts, const void* saved,
                      void* workspace, wkv7_bf16* dq, wkv7_bf16* dk, wkv7_bf16* dv, float* dg, float* dbeta,
                      float* dS_init, const long long* strides, float scale, int l2norm, int B, int T, int Hk, int Hv,
                      int K, int V, int nseq, void* stream) {
  return gdr::backward_impl(true, q, k, v, g, beta, d_o, dS_final, seq_starts, saved, workspace, dq, dk, dv, dg, dbeta,
                            dS_init, strides, scale, l2norm, B, T, Hk, Hv, K, V, nseq, static_cast<cudaStream_t>(stream));
}
int gdr_step(const float* q, const float* k, const float* v, const float* g, const float* beta, float* state,
             const int* slots, float* o, const long long* strides, float scale, int l2norm, int R, int T, int Hk, int Hv,
             int K, int V, int n_slots, void* stream) {
  return gdr::step_impl(false, q, k, v, g, beta, state, slots, o, strides, scale, l2norm, R, T, Hk, Hv, K, V, n_slots,
                        static_cast<cudaStream_t>(stream));
}
int gdr_step_bf16(const wkv7_bf16* q, const wkv7_bf16* k, const wkv7_bf16* v, const float* g, const float* beta,
                  float* state, const int* slots, wkv7_bf16* o, const long long* strides, float scale, int l2norm, int R,
                  int T, int Hk, int Hv, int K, int V, int n_slots, void* stream) {
  return gdr::step_impl(true, q, k, v, g, beta, state, slots, o, strides, scale, l2norm, R, T, Hk, Hv, K, V, n_slots,
                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"
