// C ABI of linear attention with a decay (linattn.h): argument checks, the
// regions of the caller's buffers, and the launches.
#include <algorithm>
#include <initializer_list>

#ifdef WKV7_DEBUG
#include <atomic>
#endif

#include "api_check.h"
#include "linattn.h"
#include "linattn_launch.h"
#include "linattn_maps.h"

namespace linattn {
namespace {

using api::fail;
using api::Span;

constexpr unsigned long long kMaxBytes = 1ull << 46, kMaxBlocks = 1ull << 31;

#ifdef WKV7_DEBUG
std::atomic<int> g_debug_what{0}, g_debug_n{0};  // linattn_debug.h
#endif

int check_dims(int B, int T, int Hk, int Hv, int K, int V, const char* rows) {
  if (B < 0 || T < 0 || Hk < 0 || Hv < 0) return fail(WKV7_ERR_INVALID, "%s, T, Hk and Hv must be >= 0 (got %d, %d, %d, %d)", rows, B, T, Hk, Hv);
  if (Hk > Hv || (Hk ? Hv % Hk : Hv)) return fail(WKV7_ERR_INVALID, "Hv must be a multiple of Hk (got %d, %d)", Hv, Hk);
  if (K < 8 || K > kMaxDim || K % 8 || V < 8 || V > kMaxDim || V % 8)
    return fail(WKV7_ERR_INVALID, "K and V must be multiples of 8 from 8 to %d (got %d, %d)", kMaxDim, K, V);
  if (T > 1 << 30 || (unsigned long long)B * T >= 1ull << 40 || (unsigned long long)B * T * Hv >= kMaxBytes / (4 * kMaxDim))
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
    bytes[i] = B && T && Hv ? api::span_bytes(B - 1, b, T - 1, t, row[i], es) : 0;
    if (bytes[i] >= kMaxBytes) return fail(WKV7_ERR_INVALID, "%s too large", names[i]);
  }
  return WKV7_OK;
}

// Fills a shape; nseq < 0 for dense batches.
int set_shape(Shape& s, int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16) {
  int rc = check_dims(B, T, Hk, Hv, K, V, "B");
  if (rc) return rc;
  if (nseq >= 0 && B != 1) return fail(WKV7_ERR_INVALID, "packed sequences lie in one batch row (got B = %d)", B);
  s = Shape{};
  s.B = B, s.T = T, s.Hk = Hk, s.Hv = Hv, s.K = K, s.V = V;
  s.nseq = nseq >= 0 ? nseq : B;
  s.packed = nseq >= 0;
  s.C = on_tcgen05(K, V, bf16) ? kCBf16 : kCF32;
  const unsigned long long slots = slot_count(B, T, s.nseq, s.packed, s.C), heads = Hv ? Hv : 1;
  if (slots * heads * 2 >= kMaxBlocks || (unsigned long long)s.nseq * heads * 16 >= kMaxBlocks)
    return fail(WKV7_ERR_INVALID, "too many chunks");
  s.slots = (int)slots;
  return WKV7_OK;
}

struct Place {
  char* at;
  char* const start;
  template <typename T>
  void take(T*& p, size_t count) {
    p = reinterpret_cast<T*>(at);
    at += (count * sizeof(T) + 127) & ~(size_t)127;
  }
  void* bytes(size_t n) {
    char* p;
    take(p, n);
    return p;
  }
};
// On tcgen05: how many chunks a segment of a chain has; 0: chains go whole. Chains (sequences, heads and slices of
// 64 values) run one an SM at a time. Segments fill the GPU, at the price of a pass for their sums, which measures as
// much as the chain itself in bfloat16 and half of it in fp32, of launches and the join (4 steps' worth, and 6), and of two steps'
// worth for each block's beginning; they are taken where that saves a tenth of the steps that follow one another. 8192
// tokens, us whole and in segments: bfloat16 32 heads of 64 150 and 91, 64 heads 150 and 160; fp32 32 heads 347 and 160, 64 heads
// 351 and 300, 80 heads 359 and 519. Of packed sequences the lengths are not known here, and may be alike or one long and
// some short ones: the longest is taken for three times the mean, or for all there is. 8190 tokens, 32 heads of 64, bfloat16: three
// alike 67 whole and 121 in segments, one of 7900 and two short ones 154 and 102; six 71 and 126, 153 and 105 (16 heads: 42 and
// 76, 150 and 66); fp32, three: 134 and 226, 344 and 169. Whole loses more where it loses.
int segment_chunks(const Shape& s, bool bf16) {
  const long long heads = (long long)s.Hv * ((s.V + 63) / 64), lines = heads * s.nseq;
  const int chunks = (s.T + s.C - 1) / s.C;
  if (chunks < 8 || !lines) return 0;
  auto steps = [&](long long blocks, int each) { return (blocks + kSms - 1) / kSms * (each + 2); };
  const bool several = s.packed && s.nseq > 1;  // (one packed sequence is a dense one)
  const long long total = several ? (s.T / s.C + s.nseq) * heads : chunks * lines;
  const long long longest = several ? std::min<long long>(chunks, (chunks * 3ll + s.nseq - 1) / s.nseq) : chunks;
  const long long whole = several ? std::max(longest, total / kSms) + 2 : steps(lines, chunks);
  int best = 0;
  long long least = whole * 9;
  for (int n = 2; n <= 64 && n <= chunks / 2; ++n) {
    const int each = (chunks + n - 1) / n;
    const long long cost = steps(several ? (total + each - 1) / each : lines * n, each) * (bf16 ? 20 : 15) + (bf16 ? 40 : 60);
    if (cost < least) least = cost, best = each;
  }
  return best;
}
// How many chunks or segments have their states in fp32.
long long stretches(const Shape& s, bool bf16) {
  if (!on_tcgen05(s.K, s.V, bf16)) return s.slots;
  const int each = segment_chunks(s, bf16);
  return each ? slot_count(s.B, s.T, s.nseq, s.packed, each * s.C) : 0;
}
// The regions of `saved`, and of the backward's workspace, from p on; returns the bytes.
size_t place_saved(Args& a, bool bf16, bool for_backward, char* p) {
  const Shape& s = a.s;
  const size_t n = (size_t)s.slots * s.Hv;
  Place x{p, p};
  const bool tc = on_tcgen05(s.K, s.V, bf16);
  if (tc && for_backward) a.images = x.bytes(n * image_bytes(s.K, s.V));
  const size_t m = (size_t)stretches(s, bf16) * s.Hv;
  x.take(a.states, m * s.V * s.K);
  x.take(a.decay, m);
  return x.at - x.start;
}
size_t place_workspace(Args& a, bool bf16, char* p) {
  const Shape& s = a.s;
  const size_t n = (size_t)s.slots * s.Hv;
  Place x{p, p};
  const bool tc = on_tcgen05(s.K, s.V, bf16);
  if (tc) a.dimages = x.bytes(n * image_bytes(s.K, s.V));
  const size_t m = (size_t)stretches(s, bf16) * s.Hv;
  x.take(a.dstates, m * s.V * s.K);
  x.take(a.decay, m);
  if (s.fixed) {
    x.take(a.dg, (size_t)s.B * s.T * s.Hv);
    x.take(a.part, (size_t)kParts * s.Hv);
  }
  return x.at - x.start;
}

int zero_all(std::initializer_list<Span> outs, cudaStream_t stream) {
  for (const Span& x : outs) {
    const cudaError_t e = x.p && x.bytes ? cudaMemsetAsync(const_cast<void*>(x.p), 0, x.bytes, stream) : cudaSuccess;
    if (e != cudaSuccess) return fail(WKV7_ERR_CUDA, "%s: %s", x.name, cudaGetErrorString(e));
  }
  return WKV7_OK;
}
int copy_state(float* dst, const float* src, size_t bytes, cudaStream_t stream) {
  if (!dst || !bytes) return WKV7_OK;
  const cudaError_t e = src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(dst, 0, bytes, stream);
  return e == cudaSuccess ? WKV7_OK : fail(WKV7_ERR_CUDA, "state copy: %s", cudaGetErrorString(e));
}
int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? WKV7_OK : fail(WKV7_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}
// On tcgen05: o, or dv.
int chains(const Maps& maps, Args& a, bool bf16, bool backward, bool keep, cudaStream_t stream) {
#ifdef WKV7_DEBUG
  a.skip_what = g_debug_what.load(), a.skip_n = g_debug_n.load();
#endif
  const int each = segment_chunks(a.s, bf16);
  auto run = [&](Way way, bool images) {
    return launched(bf16 ? launch_chain(maps, a, backward, each, way, images, stream) : launch_chain32(a, backward, each, way, images, stream), "chain");
  };
  if (!each) return run(kWhole, keep);
  int rc = run(kSums, false);
  if (!rc) rc = launched(launch_join(a, backward, each * a.s.C, stream), "join");
  return rc ? rc : run(kResume, keep);
}
uint32_t* words(void* p) { return static_cast<uint32_t*>(p); }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  return fn;
}
// [B][T][H][D] with token and batch strides. A batch row that is every batch row's (stride 0) is one.
bool make_map(CUtensorMap& map, const void* p, int B, int T, int H, int D, long long t, long long b) {
  const cuuint64_t row = (cuuint64_t)H * D * 2, ts = t ? (cuuint64_t)t * 2 : row, bs = b ? (cuuint64_t)b * 2 : ts * T;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)(b ? B : 1)}, strides[3] = {(cuuint64_t)D * 2, ts, bs};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)kCBf16, 1}, one[4] = {1, 1, 1, 1};
  return encoder()(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool make_maps(Maps& m, const Args& a) {
  const Shape& s = a.s;
  if (!encoder()) return false;
  return make_map(m.q, a.q, s.B, s.T, s.Hk, s.K, s.q_t, s.q_b) && make_map(m.k, a.k, s.B, s.T, s.Hk, s.K, s.k_t, s.k_b) &&
         make_map(m.v, a.v, s.B, s.T, s.Hv, s.V, s.v_t, s.v_b) &&
         (!a.d_o || make_map(m.d, a.d_o, s.B, s.T, s.Hv, s.V, 0, s.B > 1 ? (long long)s.T * s.Hv * s.V : 0));
}

}  // namespace linattn

using namespace linattn;

extern "C" {

#ifdef WKV7_DEBUG
int linattn_debug_skip(int what, int n) {
  linattn::g_debug_what.store(n > 0 ? what : 0), linattn::g_debug_n.store(n);
  return WKV7_OK;
}
#endif

size_t linattn_saved_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16, int for_backward) {
  Args a{};
  if (set_shape(a.s, B, T, Hk, Hv, K, V, nseq, bf16)) return 0;
  return place_saved(a, bf16, for_backward, nullptr);
}
size_t linattn_backward_bytes(int B, int T, int Hk, int Hv, int K, int V, int nseq, int g_fixed, int bf16) {
  Args a{};
  if (set_shape(a.s, B, T, Hk, Hv, K, V, nseq, bf16)) return 0;
  a.s.fixed = g_fixed;
  return place_workspace(a, bf16, nullptr);
}

int linattn_forward(const void* q, const void* k, const void* v, const float* g, const float* s_init,
                    const int* seq_starts, void* o, float* s_final, void* saved, const long long* strides, float scale,
                    int g_fixed, int for_backward, int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16, void* stream_) {
  const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (!seq_starts) nseq = -1;
  if (seq_starts && nseq < 0) return fail(WKV7_ERR_INVALID, "nseq must be >= 0 with seq_starts (got %d)", nseq);
  Args a{};
  int rc = set_shape(a.s, B, T, Hk, Hv, K, V, nseq, bf16);
  if (rc) return rc;
  const int es = bf16 ? 2 : 4;
  long long st[6];
  unsigned long long in_bytes[3];
  if ((rc = set_strides(st, in_bytes, strides, B, T, Hk, Hv, K, V, es))) return rc;
  const unsigned long long rows = (unsigned long long)B * T * Hv, state = (unsigned long long)a.s.nseq * Hv * V * K * 4;
  const size_t need = place_saved(a, bf16, for_backward, static_cast<char*>(saved));
  const Span ins[6] = {{q, in_bytes[0], "q", true}, {k, in_bytes[1], "k", true}, {v, in_bytes[2], "v", true},
                       {g, rows ? (g_fixed ? Hv : rows) * 4 : 0, "g", true, 4}, {s_init, state, "s_init", false},
                       {seq_starts, seq_starts ? ((unsigned long long)nseq + 1) * 4 : 0, "seq_starts", false, 4}};
  const Span outs[3] = {{o, rows * V * es, "o", true}, {s_final, state, "s_final", false}, {saved, rows ? need : 0, "saved", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!Hv) return WKV7_OK;
  if (!a.s.nseq) return zero_all({outs[0]}, stream);
  if (!rows) return copy_state(s_final, s_init, state, stream);
  a.s.starts = seq_starts, a.s.scale = scale, a.s.fixed = g_fixed;
  a.s.q_b = st[0], a.s.q_t = st[1], a.s.k_b = st[2], a.s.k_t = st[3], a.s.v_b = st[4], a.s.v_t = st[5];
  a.q = q, a.k = k, a.v = v, a.g = g, a.s_init = s_init, a.o = o, a.s_final = s_final;
  if (on_tcgen05(K, V, bf16)) {
    Maps maps;
    if (bf16 && !make_maps(maps, a)) return fail(WKV7_ERR_CUDA, "no tensor maps of q, k and v");
    if ((rc = wkv7::api_status_word(&a.status)) || (rc = chains(maps, a, bf16, false, for_backward, stream))) return rc;
  } else {
    if ((rc = launched(launch_states(a, false, stream), "states"))) return rc;
    if ((rc = launched(launch_rows_o(a, stream), "forward"))) return rc;
  }
  if (!a.s.packed) return WKV7_OK;
  return launched(launch_gaps(a, Gaps{{words(o)}, {(long long)Hv * V * es / 4}}, stream), "gaps");
}

int linattn_backward(const void* q, const void* k, const void* v, const float* g, const void* d_o,
                     const float* dS_final, const int* seq_starts, const void* saved, void* workspace, void* dq,
                     void* dk, void* dv, float* dg, float* dS_init, const long long* strides, float scale, int g_fixed,
                     int B, int T, int Hk, int Hv, int K, int V, int nseq, int bf16, void* stream_) {
  const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (!seq_starts) nseq = -1;
  if (seq_starts && nseq < 0) return fail(WKV7_ERR_INVALID, "nseq must be >= 0 with seq_starts (got %d)", nseq);
  Args a{};
  int rc = set_shape(a.s, B, T, Hk, Hv, K, V, nseq, bf16);
  if (rc) return rc;
  a.s.fixed = g_fixed;
  const int es = bf16 ? 2 : 4;
  long long st[6];
  unsigned long long in_bytes[3];
  if ((rc = set_strides(st, in_bytes, strides, B, T, Hk, Hv, K, V, es))) return rc;
  const unsigned long long rows = (unsigned long long)B * T * Hv, keys = (unsigned long long)B * T * Hk * K * es,
                           state = (unsigned long long)a.s.nseq * Hv * V * K * 4,
                           gs = (g_fixed ? Hv : rows) * 4;
  const size_t have = place_saved(a, bf16, true, const_cast<char*>(static_cast<const char*>(saved)));
  const size_t need = place_workspace(a, bf16, static_cast<char*>(workspace));
  const Span ins[8] = {{q, in_bytes[0], "q", true}, {k, in_bytes[1], "k", true}, {v, in_bytes[2], "v", true},
                       {g, rows ? gs : 0, "g", true, 4}, {d_o, rows * V * es, "d_o", true}, {dS_final, state, "dS_final", false},
                       {seq_starts, seq_starts ? ((unsigned long long)nseq + 1) * 4 : 0, "seq_starts", false, 4},
                       {saved, rows ? have : 0, "saved", true}};
  const Span outs[6] = {{dq, keys, "dq", true}, {dk, keys, "dk", true}, {dv, rows * V * es, "dv", true},
                        {dg, gs, "dg", false, 4}, {dS_init, state, "dS_init", false}, {workspace, rows ? need : 0, "workspace", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!Hv) return WKV7_OK;
  if (!a.s.nseq) return zero_all({outs[0], outs[1], outs[2], outs[3]}, stream);
  if (!rows) {
    if (g_fixed && (rc = zero_all({outs[3]}, stream))) return rc;
    return copy_state(dS_init, dS_final, state, stream);
  }
  a.s.starts = seq_starts, a.s.scale = scale;
  a.s.q_b = st[0], a.s.q_t = st[1], a.s.k_b = st[2], a.s.k_t = st[3], a.s.v_b = st[4], a.s.v_t = st[5];
  a.q = q, a.k = k, a.v = v, a.g = g, a.d_o = d_o, a.dS_final = dS_final;
  a.dq = dq, a.dk = dk, a.dv = dv, a.dS_init = dS_init;
  if (g_fixed)
    a.dg_fixed = dg;
  else
    a.dg = dg;
  if (!dg) a.dg = nullptr;
  if (on_tcgen05(K, V, bf16)) {
    Maps maps;
    if (bf16 && !make_maps(maps, a)) return fail(WKV7_ERR_CUDA, "no tensor maps of q, k, v and d_o");
    if ((rc = wkv7::api_status_word(&a.status)) || (rc = chains(maps, a, bf16, true, true, stream))) return rc;
    if ((rc = launched(launch_grad(maps, a, bf16, stream), "gradients"))) return rc;
  } else {
    if ((rc = launched(launch_states(a, true, stream), "states"))) return rc;
    if ((rc = launched(launch_rows_grad(a, stream), "gradients"))) return rc;
  }
  if (a.s.packed) {
    const long long wk = (long long)Hk * K * es / 4, wv = (long long)Hv * V * es / 4;
    const Gaps gaps{{words(dq), words(dk), words(dv), words(a.dg)}, {wk, wk, wv, Hv}};
    if ((rc = launched(launch_gaps(a, gaps, stream), "gaps"))) return rc;
  }
  return a.dg_fixed ? launched(launch_dg_sums(a, stream), "sums of dg") : WKV7_OK;
}

int linattn_step(const void* q, const void* k, const void* v, const float* g, float* state, const int* slots, void* o,
                 const long long* strides, float scale, int g_fixed, int R, int T, int Hk, int Hv, int K, int V,
                 int n_slots, int bf16, void* stream) {
  int rc = check_dims(R, T, Hk, Hv, K, V, "R");
  if (rc) return rc;
  if (n_slots < 0 || (!slots && R > n_slots)) return fail(WKV7_ERR_INVALID, "%d states for %d requests", n_slots, R);
  const int es = bf16 ? 2 : 4;
  long long st[6];
  unsigned long long in_bytes[3];
  if ((rc = set_strides(st, in_bytes, strides, R, T, Hk, Hv, K, V, es))) return rc;
  const unsigned long long rows = (unsigned long long)R * T * Hv, pool = (unsigned long long)n_slots * Hv * V * K * 4;
  if (pool >= kMaxBytes || (unsigned long long)R * Hv * 16 >= kMaxBlocks) return fail(WKV7_ERR_INVALID, "too many states");
  const Span ins[5] = {{q, in_bytes[0], "q", true}, {k, in_bytes[1], "k", true}, {v, in_bytes[2], "v", true},
                       {g, rows ? (g_fixed ? Hv : rows) * 4 : 0, "g", true, 4}, {slots, (unsigned long long)R * 4, "slots", false, 4}};
  const Span outs[2] = {{state, pool, "state", rows != 0}, {o, rows * V * es, "o", true}};
  if ((rc = api::check_spans(ins, outs))) return rc;
  if (!rows) return WKV7_OK;
  StepArgs a{};
  a.q = q, a.k = k, a.v = v, a.g = g, a.state = state, a.slots = slots, a.o = o;
  a.R = R, a.T = T, a.Hk = Hk, a.Hv = Hv, a.K = K, a.V = V, a.n_slots = n_slots, a.fixed = g_fixed, a.scale = scale;
  a.q_b = st[0], a.q_t = st[1], a.k_b = st[2], a.k_t = st[3], a.v_b = st[4], a.v_t = st[5];
  return launched(launch_step(a, bf16, static_cast<cudaStream_t>(stream)), "step");
}

}  // extern "C"
